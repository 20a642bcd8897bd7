"""The kernels' waits hold however late a warp comes: many calls whose last key tile has
rows to clear, with slow and quick softmax steps, none of which may give up."""
import pytest
import torch

from test_decode_shared_gpu import build
from test_scored_gpu import inputs, slopes_of

pytestmark = pytest.mark.gpu
FORMS = [(0.0, False), (50.0, False), (0.0, True), (20.0, True)]


@pytest.fixture(scope="module")
def swa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import sliding_window_attention_fwd_b200 as m
    return m


def repeat(swa, call, times=300):
    """Every call gives the same bits, and none times out."""
    first = call()
    assert swa.swa_device_error() == 0
    for _ in range(times):
        got = call()
        assert swa.swa_device_error() == 0
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.parametrize("cap,bias", FORMS)
@pytest.mark.parametrize("H,Hkv,N,D", [(32, 8, 700, 128), (32, 8, 700, 64), (32, 8, 1300, 128)])
@pytest.mark.parametrize("std", [2.0, 60.0])  # most scores near zero; at the cap
def test_forward(swa, cap, bias, H, Hkv, N, D, std):
    q, k, v, _ = inputs(1, N, H, Hkv, D, 41, std=std)
    q, k = q.abs(), k.abs()
    kw = {"win_left": 150, "win_right": 0, "softcap": cap, "slopes": slopes_of(H) if bias else None}

    def call():
        out = torch.full_like(q, float("nan"))
        lse = torch.full((1, H, N), float("nan"), device="cuda")
        swa.swa_forward_scored(q, k, v, out=out, lse=lse, **kw)
        return out, lse
    repeat(swa, call)


@pytest.mark.parametrize("cap,bias", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [20, 140])
def test_decode(swa, cap, bias, D, B):
    P = 1000  # (its last key tile ends inside)
    q, kp, vp, ptab, table, pos = build(P, [P + b % 90 for b in range(B)], 32, 8, D, 64, seed=42,
                                        std=60.0)
    args = (ptab.cuda(), P, table.cuda(), pos.cuda(), 64, 200)
    kw = {"softcap": cap, "slopes": slopes_of(32) if bias else None}

    def call():
        out = torch.full_like(q, float("nan"))
        swa.swa_decode_shared(q, kp, vp, *args, out=out, **kw)
        return (out,)
    repeat(swa, call)
