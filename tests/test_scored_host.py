"""Host checks of the operators with shaped scores, of the shared-prefix decode and of
the rotated paged append: what the C entries and the binding refuse (no GPU call is
reached), the order of the arguments they hand on, and the 64-bit reference itself."""
import ctypes
import math

import pytest
import torch

import score_ref as R
import sliding_window_attention_fwd_b200 as swa
from sliding_window_attention_fwd_b200 import binding as b

OK, ARG, ALIGN, UNSUP = 0, -1, -2, -3
A = 0x10000  # a fake 16-byte aligned address: validation never reads it
L = b._lib
BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
nan = float("nan")


def score(softcap=0.0, slopes=None, cu=None, prefix=None, n=0):
    return b.SwaScore(softcap, slopes, cu, prefix, n)


def fwd(q=A, k=A, v=A, out=A, lse=None, B=1, H=4, Hkv=2, N=64, D=128, sc=None):
    p = None if sc is None else ctypes.c_void_p(ctypes.addressof(sc))
    return L.swa_forward_scored(q, k, v, out, lse, B, H, Hkv, N, D, 8, 0, p, 0.0, None)


def bwd(q=A, out=A, dout=A, lse=A, dq=A, dk=A, dv=A, delta=A, B=1, H=4, Hkv=2, N=64, D=128, sc=None):
    p = None if sc is None else ctypes.c_void_p(ctypes.addressof(sc))
    return L.swa_backward_scored(q, A, A, out, dout, lse, dq, dk, dv, delta, B, H, Hkv, N, D, 8, 0,
                                 p, 0.0, None)


SCORES = [
    (dict(softcap=-1.0), ARG), (dict(softcap=nan), ARG), (dict(softcap=math.inf), ARG),
    (dict(softcap=2e30), ARG), (dict(n=-1), ARG), (dict(n=3), ARG), (dict(cu=A), ARG),
    (dict(prefix=A), ARG), (dict(slopes=A + 2), ALIGN), (dict(cu=A + 1, n=2), ALIGN),
    (dict(cu=A, prefix=A + 2, n=2), ALIGN),
]


@pytest.mark.parametrize("kw,code", SCORES)
def test_score_blocks_refused(kw, code):
    assert fwd(sc=score(**kw)) == code
    assert bwd(sc=score(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(out=None), ARG), (dict(H=4, Hkv=3), ARG), (dict(N=-1), ARG),
    (dict(q=A + 8), ALIGN), (dict(lse=A + 2), ALIGN), (dict(D=96), UNSUP), (dict(D=32), UNSUP),
    (dict(N=0), OK), (dict(B=0), OK), (dict(N=0, sc=score(20.0, A, A, A, 3)), OK),
])
def test_forward_refusals(kw, code):
    assert fwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dout=None), ARG), (dict(lse=None), ARG), (dict(dq=None), ARG), (dict(delta=None), ARG),
    (dict(dk=A + 8), ALIGN), (dict(delta=A + 2), ALIGN), (dict(D=256), UNSUP), (dict(N=0), OK),
])
def test_backward_refusals(kw, code):
    assert bwd(**kw) == code


def rope(q=A, k=A, v=A, qs=512, ks=256, vs=256, inv=A, rot=128, cu=A, pos0=A, table=A, qo=A,
         qos=512, kp=A, vp=A, T=4, B=2, H=4, Hkv=2, D=128, page=64, n=9, cols=5):
    return L.swa_rope_append_paged(q, k, v, qs, ks, vs, inv, rot, 0, cu, pos0, table, qo, qos, kp,
                                   vp, T, B, H, Hkv, D, page, n, cols, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(inv=None), ARG), (dict(cu=None), ARG), (dict(qo=None), ARG),
    (dict(vp=None), ARG), (dict(T=-1), ARG), (dict(B=-1), ARG), (dict(H=0), ARG),
    (dict(page=0), ARG), (dict(n=0), ARG), (dict(cols=0), ARG), (dict(rot=144), ARG),
    (dict(rot=-16), ARG), (dict(qs=504), ARG), (dict(ks=248), ARG), (dict(qos=8), ARG),
    (dict(q=A + 8), ALIGN), (dict(kp=A + 2), ALIGN), (dict(qs=516), ALIGN), (dict(vs=260), ALIGN),
    (dict(pos0=A + 4), ALIGN), (dict(cu=A + 2), ALIGN), (dict(rot=0), UNSUP), (dict(rot=24), UNSUP),
    (dict(D=96, rot=96), UNSUP), (dict(H=5000, qs=5000 * 128, qos=5000 * 128), UNSUP),
    (dict(T=0), OK), (dict(B=0), OK),
])
def test_rope_refusals(kw, code):
    assert rope(**kw) == code


def shared(q=A, kp=A, vp=A, out=A, lse=None, ptab=A, P=100, table=A, pos=A, B=2, H=8, Hkv=2, D=128,
           page=64, n=9, cols=5, W=64, keep=1, tail=10, cap=0.0, slopes=None, ws=A, nbytes=1 << 40):
    return L.swa_decode_shared(q, kp, vp, out, lse, ptab, P, table, pos, B, H, Hkv, D, page, n,
                               cols, W, keep, tail, cap, slopes, 0.0, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(table=None), ARG), (dict(ptab=None), ARG), (dict(ws=None), ARG),
    (dict(pos=None), ARG), (dict(P=-1), ARG), (dict(W=0), ARG), (dict(tail=-1), ARG),
    (dict(cap=-2.0), ARG), (dict(cap=nan), ARG), (dict(H=9), ARG), (dict(nbytes=64), ARG),
    (dict(cols=0), ARG), (dict(q=A + 8), ALIGN), (dict(ws=A + 8), ALIGN), (dict(pos=A + 4), ALIGN),
    (dict(slopes=A + 1), ALIGN), (dict(D=96), UNSUP), (dict(H=18), UNSUP), (dict(page=96), UNSUP),
    (dict(page=1 << 20, n=1 << 12), UNSUP), (dict(P=2 ** 31 - 1), UNSUP), (dict(B=0), OK),
])
def test_shared_refusals(kw, code):
    assert shared(**kw) == code


def test_shared_workspace_grows_with_the_call():
    f = swa.swa_decode_shared_workspace_bytes
    assert f(0, 8, 2, 128, 100, 64, 5) == 0 and f(2, 9, 2, 128, 100, 64, 5) == 0
    assert f(2, 8, 2, 96, 100, 64, 5) == 0 and f(2, 18, 2, 128, 100, 64, 5) == 0
    one = f(1, 8, 2, 128, 100, 64, 5)
    # without a prefix no part of it, however many rows there are
    assert f(9999, 64, 8, 64, 0, 64, 5) == 9999 * 64 * 65 * 4
    assert one >= 2 * 8 * 129 * 4  # a prefix part and an own part
    assert f(1, 8, 2, 128, 0, 64, 5) >= 8 * 129 * 4
    for tail in (0, 1, 10 ** 4, 2 ** 31 - 1):
        assert 0 < f(64, 32, 8, 128, 8192, 2 ** 31 - 1 if tail < 10 ** 6 else 4096, tail) < 2 ** 31


# ------------------------------------------------------------------ the binding
# CPU tensors of the right shapes get as far as the placement check, which shows that
# the shape checks took them; a wrong argument is named before that.
CUDA_ONLY = "must be a (contiguous )?CUDA tensor"


def t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def score_args():
    return dict(q=t(2, 50, 8, 64), k=t(2, 50, 2, 64), v=t(2, 50, 2, 64), out=t(2, 50, 8, 64),
                lse=t(2, 8, 50, dtype=F32), win_left=7, win_right=0, softcap=20.0,
                slopes=t(8, dtype=F32), cu_docs=t(2, 4, dtype=I32), prefix=t(2, 3, dtype=I32))


SCORE_BAD = [
    dict(q=t(2, 50, 8, 32)), dict(q=t(50, 8, 64)), dict(q=t(2, 50, 8, 64, dtype=F32)),
    dict(k=t(2, 49, 2, 64)), dict(k=t(2, 50, 64)), dict(v=t(2, 50, 4, 64)), dict(out=t(2, 50, 2, 64)),
    dict(lse=t(2, 50, 8, dtype=F32)), dict(lse=t(2, 8, 50)), dict(slopes=t(7, dtype=F32)),
    dict(slopes=t(8)), dict(cu_docs=t(2, 1, dtype=I32), prefix=None), dict(cu_docs=t(1, 4, dtype=I32)),
    dict(cu_docs=t(2, 4, dtype=I64)), dict(cu_docs=None), dict(prefix=t(2, 4, dtype=I32)),
]


@pytest.mark.parametrize("bad", SCORE_BAD)
def test_scored_tensors_checked(bad):
    with pytest.raises(ValueError, match="expected|needs cu_docs"):
        b.swa_forward_scored(**(score_args() | bad))
    with pytest.raises(ValueError, match="expected|needs cu_docs"):
        b.swa_backward_scored(dout=t(2, 50, 8, 64), **(score_args() | bad))


def test_scored_placement_checked():
    with pytest.raises(ValueError, match=CUDA_ONLY):
        b.swa_forward_scored(**score_args())
    args = score_args() | dict(dout=t(2, 50, 8, 64))
    with pytest.raises(ValueError, match=CUDA_ONLY):
        b.swa_backward_scored(**args)
    with pytest.raises(ValueError, match="required"):
        b.swa_backward_scored(**(args | dict(out=None)))
    with pytest.raises(ValueError, match="required"):
        b.swa_backward_scored(**(args | dict(lse=None)))
    with pytest.raises(ValueError, match="expected a torch tensor"):
        b.swa_forward_scored(**(score_args() | dict(q=[1.0])))
    e = torch.empty(2, 0, 4, 64, dtype=BF)  # also where there is nothing to do
    with pytest.raises(ValueError, match=CUDA_ONLY):
        b.swa_forward_scored(e, e, e)


def rope_args():
    return dict(q=t(9, 4, 64), k=t(9, 2, 64), v=t(9, 2, 64), inv_freq=t(16, dtype=F32),
                cu=t(4, dtype=I32), pos0=t(3, dtype=I64), block_table=t(3, 5, dtype=I32),
                k_pages=t(96, 2, 64), v_pages=t(96, 2, 64), page_size=48, q_out=t(9, 4, 64))


@pytest.mark.parametrize("bad", [
    dict(k=t(8, 2, 64)), dict(v=t(9, 1, 64)), dict(cu=t(3, dtype=I32)), dict(cu=t(4, dtype=I64)),
    dict(page_size=50), dict(page_size=0), dict(page_size=-48), dict(v_pages=t(96, 2, 32)),
    dict(k_pages=t(96, 4, 64), v_pages=t(96, 4, 64)), dict(inv_freq=t(16)),
    dict(inv_freq=t(2, 8, dtype=F32)), dict(pos0=t(3, dtype=I32)),
    dict(block_table=t(2, 5, dtype=I32)), dict(block_table=t(15, dtype=I32)),
    dict(q_out=t(9, 2, 64)), dict(q=t(9, 256)),
])
def test_rope_tensors_checked(bad):
    with pytest.raises(ValueError, match="expected"):
        b.swa_rope_append_paged(**(rope_args() | bad))


def test_rope_placement_checked():
    with pytest.raises(ValueError, match=CUDA_ONLY):
        b.swa_rope_append_paged(**rope_args())


def shared_args():
    return dict(q=t(3, 8, 128), k_pages=t(320, 2, 128), v_pages=t(320, 2, 128),
                prefix_table=t(2, dtype=I32), n_prefix=100, block_table=t(3, 4, dtype=I32),
                pos=t(3, dtype=I64), page_size=64, W=33, out=t(3, 8, 128),
                lse=t(3, 8, dtype=F32), slopes=t(8, dtype=F32))


@pytest.mark.parametrize("bad", [
    dict(n_prefix=129), dict(n_prefix=-1), dict(page_size=96), dict(page_size=0),
    dict(block_table=t(2, 4, dtype=I32)), dict(block_table=t(3, 4, dtype=I64)),
    dict(v_pages=t(320, 4, 128)), dict(k_pages=t(320, 2, 64), v_pages=t(320, 2, 64)),
    dict(pos=t(2, dtype=I64)), dict(pos=t(3, dtype=I32)), dict(out=t(3, 8, 64)),
    dict(lse=t(8, 3, dtype=F32)), dict(slopes=t(2, dtype=F32)), dict(prefix_table=t(2, dtype=I64)),
    dict(q=t(3, 8, 128, dtype=F32)),
])
def test_shared_tensors_checked(bad):
    with pytest.raises(ValueError, match="expected"):
        b.swa_decode_shared(**(shared_args() | bad))


def test_shared_placement_checked():
    with pytest.raises(ValueError, match=CUDA_ONLY):
        b.swa_decode_shared(**shared_args())


@pytest.mark.parametrize("call,args,bad", [
    (b.swa_rope_append_paged, rope_args, dict(page_size="48")),
    (b.swa_decode_shared, shared_args, dict(W=1.5)),
    (b.swa_decode_shared, shared_args, dict(n_prefix=None)),
])
def test_numbers_of_the_wrong_kind(call, args, bad):
    with pytest.raises(TypeError):
        call(**(args() | bad))


@pytest.mark.parametrize("bad", [dict(W=2 ** 31), dict(page_size=2 ** 40), dict(n_prefix=-2 ** 31 - 1)])
def test_numbers_out_of_range(bad):
    with pytest.raises(ValueError):
        b.swa_decode_shared(**(shared_args() | bad))


# ------------------------------------------------------------------ the reference
@pytest.mark.parametrize("cap,bias,cu,pre,L_,R_", [
    (0.0, False, None, None, -1, 0), (3.0, True, [[0, 5, 17]], [[3, 20]], 6, 0),
    (5.0, False, [[2, 2, 9, 15]], None, -1, -1), (0.0, True, [[0, 18]], [[7]], 4, 2),
])
def test_reference_gradients(cap, bias, cu, pre, L_, R_):
    """The reference's gradients are those that differentiation of its forward gives, and
    its key sets those of the definition, element by element."""
    g = torch.Generator().manual_seed(1)
    B, N, H, Hkv, D = 1, 18, 4, 2, 8
    q, k, v, do = (torch.randn(B, N, h, D, generator=g, dtype=torch.float64)
                   for h in (H, Hkv, Hkv, H))
    sl = torch.tensor([0.5, 0.25, 0.125, 0.0625]) if bias else None
    c = None if cu is None else cu[0]
    seen = R.seen_keys(N, L_, R_, c, None if pre is None else pre[0])
    for i in range(N):
        m = None if c is None else [x for x in range(len(c) - 1) if c[x] <= i < c[x + 1]]
        for j in range(N):
            if c is None:
                lo, hi = 0, N - 1
                pe = 0
            elif m:
                lo, hi = c[m[0]], c[m[0] + 1] - 1
                pe = lo + (min(pre[0][m[0]], hi + 1 - lo) if pre else 0)
            else:
                lo, hi, pe = 1, 0, 0
            if lo <= hi:
                last = hi if R_ < 0 else min(hi, max(i + R_, pe - 1))
                first = lo if L_ < 0 else max(lo, i - L_)
            else:
                first, last = 1, 0
            assert bool(seen[i, j]) == (first <= j <= last), (i, j)
    ref = R.forward(q, k, v, L_, R_, cap, sl, cu, pre, dout=do)
    x = [a.clone().requires_grad_() for a in (q, k, v)]
    dist = (torch.arange(N)[:, None] - torch.arange(N)).abs().double()
    out = []
    for h in range(H):
        s = x[0][0, :, h] @ x[1][0, :, h // 2].T / math.sqrt(D)
        s = cap * torch.tanh(s / cap) if cap > 0 else s
        s = s - (float(sl[h]) * dist if bias else 0)
        p = torch.softmax(s.masked_fill(~seen, -1e300), -1) * seen
        out.append(p @ x[2][0, :, h // 2])
    out = torch.stack(out, 1)[None] * seen.any(1)[None, :, None, None]
    torch.testing.assert_close(out.detach(), ref["out"], rtol=1e-11, atol=1e-12)
    for got, n in zip(torch.autograd.grad(out, x, do), ("dq", "dk", "dv")):
        torch.testing.assert_close(got, ref[n], rtol=1e-10, atol=1e-11)
