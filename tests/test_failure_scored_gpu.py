"""Failure detection in the kernels of the shaped scores and of the shared-prefix decode,
without faulting the GPU: a test-only build never loads one key tile and lowers every
wait's bound to 5 ms.  The kernels must time out, leave by their abort paths and return,
and the next call must be right."""
import ctypes

import pytest
import torch

import score_ref as R
from gpu_util import build_test_library
from test_decode_shared_gpu import build, reference
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
    for n in ("swa_forward_scored", "swa_decode_shared", "swa_device_error"):
        getattr(lib, n).argtypes = getattr(b._lib, n).argtypes
    return lib


def stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("H,N", [(2, 600), (64, 700)])  # one and two heads per CTA
@pytest.mark.parametrize("D", [64, 128])
def test_forward_gives_up(lib, H, N, D):
    from sliding_window_attention_fwd_b200 import binding as b

    for n, code in ((N, TIMEOUT), (128, 0)):  # one key tile: nothing is withheld
        q, k, v, _ = inputs(1, n, H, H // 2, D)
        cu = torch.tensor([[0, 40, n]], dtype=torch.int32, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(1, H, n, device="cuda")
        sc = b.SwaScore(20.0, None, cu.data_ptr(), None, 2)
        assert lib.swa_forward_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                      lse.data_ptr(), 1, H, H // 2, n, D, -1, 0,
                                      ctypes.addressof(sc), 0.0, stream()) == 0
        assert lib.swa_device_error(stream()) == code
    R.check({"out": out, "lse": lse}, R.forward(q, k, v, -1, 0, 20.0, None, cu.cpu()),
            ("out", "lse"))
    assert lib.swa_device_error(stream()) == 0


@pytest.mark.parametrize("P,B,tail", [(8192, 64, 40),   # the prefix's walks give up
                                      (0, 2, 600)])     # the own keys' do
@pytest.mark.parametrize("D", [64, 128])
def test_decode_gives_up(lib, P, B, tail, D):
    H, Hkv, page, W = 32, 8, 64, 4096
    for p, n, code in ((P, tail, TIMEOUT), (min(P, 100), 20, 0)):
        q, kp, vp, ptab, table, pos = build(p, [p + n] * (B if code else 2), H, Hkv, D, page)
        out, lse = torch.empty_like(q), torch.empty(q.shape[0], H, device="cuda")
        ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
        dptab, dtable, dpos = ptab.cuda(), table.cuda(), pos.cuda()
        assert lib.swa_decode_shared(q.data_ptr(), kp.data_ptr(), vp.data_ptr(), out.data_ptr(),
                                     lse.data_ptr(), dptab.data_ptr(), p, dtable.data_ptr(),
                                     dpos.data_ptr(), q.shape[0], H, Hkv, D, page,
                                     kp.shape[0] // page, table.shape[1], W, 1, n + 1, 20.0, None,
                                     0.0, ws.data_ptr(), ws.numel(), stream()) == 0
        assert lib.swa_device_error(stream()) == code
    R.check({"out": out, "lse": lse},
            reference(q, kp, vp, ptab, table, pos, p, page, W, True, 20.0, None), ("out", "lse"))
