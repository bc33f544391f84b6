"""Bounded waits that run out in the forms of the grouped products that test_gpu_train_waits does not reach: items of two
groups of features (four stages, one accumulator), and weight gradients added to earlier ones (four stages, copies of what is
added in flight), with segments of several parts.  Which kernel a call launches is read from a captured graph."""
import ctypes
import re

import pytest

from tests.test_gpu_mx import moe, torch_  # noqa: F401
from tests.test_gpu_train import _gen, _randn

pytestmark = pytest.mark.gpu

T, N, K_CHOICES, B, K, F = 4000, 4, 2, 8, 136, 2048      # some 2000 rows an expert

# the forms, and the kernel's mode (csrc/grouped.cu: enum Mode)
FORMS = {"in place": 1, "gather": 1, "transposed": 3, "transposed gather": 3, "wgrad add": 5, "wgrad add gather": 5,
         "wgrad add in place": 5}


class _Params(ctypes.Structure):   # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p), ("sizes", ctypes.c_uint * 7), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _kernels(call):
    """The names of the kernels that a call launches."""
    torch = torch_()
    try:
        graph = torch.cuda.CUDAGraph(keep_graph=True)
    except TypeError:
        pytest.skip("this PyTorch cannot keep the captured cudaGraph_t")
    with torch.cuda.graph(graph):
        call()
    cu, handle = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(graph.raw_cuda_graph())
    n = ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(handle, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(handle, nodes, ctypes.byref(n)) == 0
    names = []
    for node in nodes:
        t, p, name = ctypes.c_int(-1), _Params(), ctypes.c_char_p()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(t)) == 0
        if t.value == 0:   # CU_GRAPH_NODE_TYPE_KERNEL
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            get, f = (cu.cuFuncGetName, p.func) if p.func else (cu.cuKernelGetName, p.kern)
            assert get(ctypes.byref(name), ctypes.c_void_p(f)) == 0
            names.append(name.value.decode())
    return names


@pytest.mark.parametrize("form", FORMS)
def test_wait_runs_out_and_reports(moe, form):
    torch = torch_()
    from tests import train_ref as R
    G = R.Groups(T, N, K_CHOICES, B, seed=5)
    assert min(G.counts) > 768
    gather, out = form.endswith("gather"), {}
    for limit in (0, 1, 20000, 1, 0):   # none, 1 ns, 20 us
        cfg = moe.make_config(128, N, K_CHOICES, 128, B, debug_wait_ns=limit)
        ws, g = moe.workspace_grouped(cfg, T), _gen(1)
        x = _randn(g, T, K) if gather else G.grouped(K, g)
        if form.startswith("wgrad"):
            dy, add = G.grouped(F, g), torch.randn(N, K, F, generator=g, device="cuda")
            y = add if form.endswith("in place") else torch.zeros_like(add)

            def call():
                moe.moe_grouped_wgrad(cfg, T, x, dy, G.ids, G.dcounts, y, ws, dw_add=add, gather_x=gather)
        else:
            tr = form.startswith("transposed")
            w, y = _randn(g, *((N, F, K) if tr else (N, K, F))), torch.zeros(G.rows, F, dtype=torch.bfloat16, device="cuda")

            def call():
                moe.moe_grouped_gemm(cfg, T, x, w, G.ids, G.dcounts, y, ws, gather=gather, transposed=tr)
        call()
        torch.cuda.synchronize()
        status = moe.moe_get_device_status(ws)
        if limit == 1:
            assert status == moe.MOE_DEV_ERR_TIMEOUT
        elif limit == 0:
            assert status == 0
            assert torch.equal(out.setdefault("y", y), y)
        else:
            assert status in (0, moe.MOE_DEV_ERR_TIMEOUT)
    name, = _kernels(call)
    assert re.search(r"grouped_kernelILNS[^E]*4ModeE(\d+)E", name).group(1) == str(FORMS[form]), name
