// Checks and size rules of the C ABI shared by its translation units.
#pragma once
#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>

#include "moe_api.h"

#define MOE_TRY(x)                   \
  do {                               \
    const moe_status _st = (x);      \
    if (_st != MOE_OK) return _st;   \
  } while (0)

namespace moe {
namespace api {

moe_status check_config(const moe_config* c);
moe_status check_tokens(const moe_config* c, int32_t T);
int32_t capacity(const moe_config* c, int32_t T);
int slots(const moe_config* c);                              // route slots per token
int64_t max_rows(const moe_config* c, int32_t T);            // padded rows
int64_t max_blocks(const moe_config* c, int32_t T);
int64_t max_tiles(const moe_config* c, int32_t T, int tile_rows);
int sm_count();
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode();
moe_status last_error();
moe_status need(const void* p);                              // present and 16-byte aligned
moe_status optional(const void* p);                          // absent or 16-byte aligned

}  // namespace api
}  // namespace moe
