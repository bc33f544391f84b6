"""A GEMM whose bounded waits ran out leaves nothing behind: the call enqueued right after it gives the usual bits.

The limits run from one at which the first wait gives up to ones that some
roles see through and others do not, so that CTAs end at different points with
loads in flight; nothing is synchronised between the two calls."""
import pytest

pytestmark = pytest.mark.gpu

LIMITS_NS = (1, 400, 1500, 4000, 10000, 30000)


def _rand(g, *shape, low=0, high=256):
    import torch
    return torch.randint(low, high, shape, generator=g, device="cuda", dtype=torch.uint8)


def _dispatch(moe, cfg, idx, T, k, N):
    import torch
    e = dict(device="cuda", dtype=torch.int32)
    ids, blocks, npad = (torch.full((n,), -9, **e) for n in (moe.moe_max_padded_rows(cfg, T), moe.moe_max_blocks(cfg, T), 1))
    moe.moe_dispatch_align(cfg, idx, torch.empty(T * k, dtype=torch.uint8, device="cuda"), torch.empty(T * k, **e), ids,
                           blocks, npad, torch.empty(N, **e), torch.empty(1, **e), moe.workspace(cfg, T))
    return ids, blocks, npad


def _check(moe, cfg, call, ws):
    """call(cfg) runs the operator and returns its outputs, fresh ones."""
    import torch
    moe.moe_clear_device_status(ws)
    want = call(cfg)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status(ws) == 0
    gave_up = 0
    for ns in LIMITS_NS:
        short = moe.moe_config.from_buffer_copy(cfg)
        short.debug_wait_ns = ns
        for _ in range(6):
            call(short)
            got = call(cfg)
            status = moe.moe_get_device_status(ws)
            gave_up += status != 0
            assert status in (0, moe.MOE_DEV_ERR_TIMEOUT)
            for a, b in zip(got, want):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16)), ns
            moe.moe_clear_device_status(ws)
    assert gave_up >= 6      # those of 1 ns


@pytest.mark.parametrize("T,N,k,Is", [
    (9, 8, 2, 1024),       # operands swapped, and the shared expert
    (70, 2, 1, 0),         # 64-column items
    (300, 8, 2, 0),        # wider ones
    (900, 8, 2, 14336)])    # CTA pairs
def test_mx_ffn(T, N, k, Is):
    import torch
    import invariant_expert_routing_gb300 as moe
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    H, I = 4096, 14336   # an epilogue's wait for a 14336-deep tile outlasts the hardware's own suspension
    cfg = moe.make_config(H, N, k, I, 16, shared_intermediate=Is)
    scale = dict(low=118, high=122)
    w = [_rand(g, N, 2 * I, H // 2), _rand(g, N, 2 * I, H // 32, **scale),
         _rand(g, N, H, I // 2), _rand(g, N, H, I // 32, **scale)]
    w += [_rand(g, 1, 2 * Is, H // 2), _rand(g, 1, 2 * Is, H // 32, **scale),
          _rand(g, 1, H, Is // 2), _rand(g, 1, H, Is // 32, **scale)] if Is else [None] * 4
    codes, scales = _rand(g, T, H // 2), _rand(g, T, H // 32, low=124, high=128)
    idx = torch.rand(T, N, generator=g, device="cuda").topk(k, 1).indices.sort(1).values.int()
    ids, blocks, npad = _dispatch(moe, cfg, idx, T, k, N)
    ws = moe.workspace_mx(cfg, T)

    def call(c):
        y = torch.zeros(ids.numel(), H, dtype=torch.bfloat16, device="cuda")
        ysh = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") if Is else None
        moe.moe_expert_ffn_mx(c, codes, scales, *w, ids, blocks, npad, y, ysh, ws)
        return [y] if ysh is None else [y, ysh]
    _check(moe, cfg, call, ws)


@pytest.mark.parametrize("H,I,T,N,k,flags", [
    (4096, 14336, 20, 4, 2, 0),        # CTA pairs, decode instances
    (14336, 4096, 600, 4, 2, 0),       # CTA pairs
    (4096, 14336, 600, 4, 2, 0),       # wide W2 items
    (14336, 4096, 600, 4, 2, 0x2000),  # W13 on single CTAs
    (640, 14336, 600, 4, 2, 0)])       # W2 on single CTAs
def test_bf16_ffn(H, I, T, N, k, flags):
    import torch
    import invariant_expert_routing_gb300 as moe
    g = torch.Generator(device="cuda")
    g.manual_seed(T + I)
    cfg = moe.make_config(H, N, k, I, 16, debug_flags=flags)
    rand = lambda *s: 0.05 * torch.randn(*s, generator=g, device="cuda")
    h, w13, w2 = rand(T, H).bfloat16(), rand(N, H, 2 * I).bfloat16(), rand(N, I, H).bfloat16()
    idx = torch.rand(T, N, generator=g, device="cuda").topk(k, 1).indices.sort(1).values.int()
    ids, blocks, npad = _dispatch(moe, cfg, idx, T, k, N)
    ws = moe.workspace(cfg, T)

    def call(c):
        y = torch.zeros(ids.numel(), H, dtype=torch.bfloat16, device="cuda")
        moe.moe_expert_ffn(c, h, w13, w2, None, None, ids, blocks, npad, y, None, ws)
        return [y]
    _check(moe, cfg, call, ws)
