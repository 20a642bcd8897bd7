"""The score cap over its whole range, 0 < softcap <= 1e30, against the 64-bit form: a cap
far above the scores leaves them as they are, one far below makes them equal."""
import pytest
import torch

import score_ref as R
from test_decode_shared_gpu import build, reference
from test_scored_gpu import inputs, slopes_of

pytestmark = pytest.mark.gpu
NAMES = ("out", "lse", "dq", "dk", "dv")
LARGE = [1e3, 8e3, 2e4, 1e6, 1e9, 1e30]


@pytest.fixture(scope="module")
def swa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import sliding_window_attention_fwd_b200 as m
    return m


def score_error(u_abs, cap, slope, dist):
    """score_ref's bound with a cap term that goes by the score.  For |u| <= 1/2, u = scale
    q . k / cap, the capped score is a polynomial that fits tanh u to 5.5e-7 of itself,
    after at most eight fp32 roundings (8 * 2^-24 = 4.8e-7): 1.1e-6 of the score.  Past it
    tanh u = 1 - 2 / (e^2u + 1): the exponential is off by 2^-22 + 2^-23 of itself, which
    moves the quotient by at most 0.4 times that, its sum and reciprocal add 1.5 (2^-24 +
    2^-23), the difference 2^-24: 4.7e-7, 1.1e-6 of a tanh of at least 0.46.  With two
    roundings of the product that is below 1.3e-6 of the score, which is at most u_abs
    and at most the cap."""
    e = 134 * R.HALF_F32 * u_abs + 7.6e-5
    if cap > 0:
        e = e + 1.3e-6 * u_abs.clamp(max=cap)
    if slope is not None:
        e = e + 4 * R.HALF_F32 * abs(slope) * dist
    return e


@pytest.fixture(autouse=True)
def tight(monkeypatch):
    monkeypatch.setattr(R, "score_error", score_error)


def both(swa, q, k, v, do, L, cap, slopes=None, cu=None):
    kw = {"win_left": L, "win_right": 0, "softcap": cap, "slopes": slopes,
          "cu_docs": None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")}
    lse = torch.empty(q.shape[0], q.shape[2], q.shape[1], device="cuda")
    out = swa.swa_forward_scored(q, k, v, lse=lse, **kw)
    g = swa.swa_backward_scored(q, k, v, out, do, lse, **kw)
    torch.cuda.synchronize()
    assert swa.swa_device_error() == 0
    return {"out": out, "lse": lse, **dict(zip(("dq", "dk", "dv"), g))}


@pytest.mark.parametrize("cap", LARGE)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("H,Hkv,N,D", [(2, 1, 300, 128), (3, 3, 300, 64), (32, 8, 700, 128)])
def test_large_caps(swa, cap, bias, H, Hkv, N, D):
    q, k, v, do = inputs(1, N, H, Hkv, D, 11)
    sl = slopes_of(H) if bias else None
    cu = [[0, N // 3, N - 9]]
    got = both(swa, q, k, v, do, 100, cap, sl, cu)
    real = slice(0, N - 9)
    for t in (q, k, v, do):
        t[:, N - 9:] = 0
    ref = R.forward(q, k, v, 100, 0, cap, sl, cu, dout=do)
    R.check(got, ref, NAMES, f"cap {cap}")
    if cap >= 1e9:  # (u^2 / 3 is far below a rounding of the score: the plain scores' results)
        R.check(got, R.forward(q, k, v, 100, 0, 0.0, sl, cu, dout=do), NAMES, "without the cap")
    assert got["out"][:, real].abs().max() > 0


@pytest.mark.parametrize("cap", [2e3, 2e4])
@pytest.mark.parametrize("D", [64, 128])
def test_large_scores_beside_usual_ones(swa, cap, D):
    """Some rows' scores reach the cap, their neighbours' stay near zero."""
    q, k, v, do = inputs(1, 300, 2, 1, D, 12)
    q[:, ::37] *= cap / 4
    got = both(swa, q, k, v, do, 100, cap)
    R.check(got, R.forward(q, k, v, 100, 0, cap, dout=do), NAMES)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("cap", [1e-10, 1e-40])  # (1e-40 is subnormal in fp32)
def test_tiny_caps(swa, cap, D, bias):
    """All scores equal up to the bias, rows whose products are zero among them."""
    q, k, v, do = inputs(1, 300, 4, 2, D, 13)
    q[:, 7::50] = 0
    sl = slopes_of(4) if bias else None
    got = both(swa, q, k, v, do, 100, cap, sl)
    R.check(got, R.forward(q, k, v, 100, 0, cap, sl, dout=do), NAMES)


@pytest.mark.parametrize("scale", [1e-12, 40.0])
@pytest.mark.parametrize("cap", [1e-6, 1e30])
def test_caps_far_from_the_scale(swa, scale, cap):
    q, k, v, _ = inputs(1, 200, 2, 1, 128, 14, std=2.0 if scale < 1 else 2.0 ** -9)
    lse = torch.empty(1, 2, 200, device="cuda")
    out = swa.swa_forward_scored(q, k, v, lse=lse, win_left=64, win_right=0, softcap=cap,
                                 scale=scale)
    ref = R.forward(q, k, v, 64, 0, cap, scale=scale)
    R.check({"out": out, "lse": lse}, ref, ("out", "lse"))


@pytest.mark.parametrize("cap", LARGE + [1e-40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P,B,bias", [(0, 3, False), (300, 5, True), (1030, 70, False)])
def test_decode(swa, cap, D, P, B, bias):
    pos = [P + (41 * b) % 150 for b in range(B)]
    q, kp, vp, ptab, table, ps = build(P, pos, 8, 2, D, 64, seed=15)
    q[0, 1] = 0
    sl = slopes_of(8) if bias else None
    lse = torch.empty(B, 8, device="cuda")
    out = swa.swa_decode_shared(q, kp, vp, ptab.cuda(), P, table.cuda(), ps.cuda(), 64, 100,
                                lse=lse, softcap=cap, slopes=sl)
    ref = reference(q, kp, vp, ptab, table, ps, P, 64, 100, True, cap, sl)
    R.check({"out": out, "lse": lse}, ref, ("out", "lse"), f"cap {cap}")


@pytest.mark.parametrize("size", [1e-14, 1e13])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("cap", [0.0, 50.0, 51.0])
@pytest.mark.parametrize("D", [64, 128])
def test_sizes_of_v(swa, size, sign, cap, D):
    """Small and large values under scores at the cap (far from 0 without one)."""
    q, k, v, _ = inputs(1, 200, 2, 1, D, 16, std=60.0 if cap else 4.0)
    q, k, v = q.abs(), k.abs() * sign, (v.double() * size).to(v.dtype)
    lse = torch.empty(1, 2, 200, device="cuda")
    # (one document, so that the uncapped call takes the shaped form too)
    cu = torch.tensor([[0, 200]], dtype=torch.int32, device="cuda")
    out = swa.swa_forward_scored(q, k, v, lse=lse, win_left=150, win_right=0, softcap=cap,
                                 cu_docs=cu)
    ref = R.forward(q, k, v, 150, 0, cap)
    ref["e_out"] = ref["e_out"] - 1e-30  # (which would be most of a small value's bound)
    R.check({"out": out, "lse": lse}, ref, ("out", "lse"))
