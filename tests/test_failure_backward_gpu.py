"""Failure detection in the tensor-core backward, without faulting the GPU: a test-only
build never issues the loads of one step and lowers every wait's bound to 5 ms.  Both
kernels must time out, leave by their abort paths and return, and the next call must be
right."""
import ctypes

import pytest
import torch

import score_ref as R
from gpu_util import build_test_library
from test_scored_gpu import inputs

pytestmark = pytest.mark.gpu
TIMEOUT = -5


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from sliding_window_attention_fwd_b200 import binding as b

    path = build_test_library(str(tmp_path_factory.mktemp("withheld")),
                              ["SWA_TEST_WITHHOLD_TILE=1", "SWA_WAIT_LIMIT_NS=5000000ull"])
    lib = ctypes.CDLL(path)
    for n in ("swa_backward_scored", "swa_device_error"):
        getattr(lib, n).argtypes = getattr(b._lib, n).argtypes
    return lib


@pytest.mark.parametrize("cap,docs", [(20.0, True), (0.0, True), (0.0, False)])  # (last: the band)
@pytest.mark.parametrize("H,Hkv", [(2, 2), (16, 2), (32, 32)])
@pytest.mark.parametrize("D", [64, 128])
def test_backward_gives_up(lib, D, H, Hkv, cap, docs):
    import sliding_window_attention_fwd_b200 as swa
    from sliding_window_attention_fwd_b200 import binding as b

    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    # long walks, of which one step's loads are missing; then walks of one step each (one
    # tile, one head per kv head)
    for N, heads, kv, code in ((700, H, Hkv, TIMEOUT), (128, Hkv, Hkv, 0)):
        q, k, v, do = inputs(1, N, heads, kv, D, 51)
        cu = [[0, 40, N]] if docs else None
        t = torch.tensor(cu, dtype=torch.int32, device="cuda") if docs else None
        lse = torch.empty(1, heads, N, device="cuda")
        kw = {"win_left": -1, "win_right": 0, "softcap": cap, "cu_docs": t}
        out = swa.swa_forward_scored(q, k, v, lse=lse, **kw)
        g = [torch.empty_like(x) for x in (q, k, v)]
        delta = torch.empty(heads * N, device="cuda")
        sc = b.SwaScore(cap, None, t.data_ptr() if docs else None, None, 2 if docs else 0)
        args = [x.data_ptr() for x in (q, k, v, out, do, lse, *g, delta)]
        assert lib.swa_backward_scored(*args, 1, heads, kv, N, D, -1, 0, ctypes.addressof(sc), 0.0,
                                       stream) == 0
        assert lib.swa_device_error(stream) == code
    ref = R.forward(q, k, v, -1, 0, cap, None, cu, dout=do)
    R.check(dict(zip(("dq", "dk", "dv"), g)), ref, ("dq", "dk", "dv"))
    assert lib.swa_device_error(stream) == 0
