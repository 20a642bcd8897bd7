"""A row that sees a NaN score is NaN, however few keys it sees, and no other row is."""
import pytest
import torch

from test_decode_shared_gpu import build
from test_scored_gpu import inputs, slopes_of

pytestmark = pytest.mark.gpu
FORMS = [(0.0, False), (20.0, False), (0.0, True), (20.0, True), (60.0, False)]


@pytest.fixture(scope="module")
def swa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import sliding_window_attention_fwd_b200 as m
    return m


def expect(got, want, bad):
    """got NaN where bad (rows), elsewhere want's bits."""
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("cap,bias", FORMS)
@pytest.mark.parametrize("H,Hkv,N,D", [(2, 1, 300, 128), (2, 1, 300, 64), (3, 3, 300, 128),
                                       (32, 8, 1300, 128), (32, 8, 1300, 64)])
def test_forward(swa, cap, bias, H, Hkv, N, D):
    L, cu = 20, [0, 1, 70, 200, N - 5]
    q, k, v, _ = inputs(1, N, H, Hkv, D, 21)
    kw = {"win_left": L, "win_right": 0, "softcap": cap, "slopes": slopes_of(H) if bias else None,
          "cu_docs": torch.tensor([cu], dtype=torch.int32, device="cuda")}

    def run(q, k):
        lse = torch.empty(1, H, N, device="cuda")
        out = swa.swa_forward_scored(q, k, v, lse=lse, **kw)
        return out, lse.transpose(1, 2)
    want, want_lse = run(q, k)
    # queries with one key, a few, and a window's worth across a tile border
    rows = [0, 1, 3, 70, 75, 130, N - 6]
    bad = torch.zeros(1, N, H, dtype=torch.bool, device="cuda")
    bad[:, rows, 1] = True
    q2 = q.clone()
    q2[:, rows, 1, 5] = float("nan")
    got, lse = run(q2, k)
    expect(got, want, bad)
    expect(lse, want_lse, bad)
    # keys at a document's first position: its first rows see little else
    k2 = k.clone()
    bad[:] = False
    grp = H // Hkv
    for j, e in ((0, 1), (1, 70), (200, N - 5)):
        k2[:, j, 0, 7] = float("nan")
        bad[:, j:min(j + L + 1, e), :grp] = True
    got, lse = run(q, k2)
    expect(got, want, bad)
    expect(lse, want_lse, bad)


@pytest.mark.parametrize("cap,bias", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [4, 140])  # one and two query tiles per CTA
def test_shared_prefix(swa, cap, bias, D, B):
    P, page, H, Hkv = 300, 64, 8, 2
    pos = [[3, 0, 299, 310][b % 4] for b in range(B)]
    q, kp, vp, ptab, table, ps = build(P, pos, H, Hkv, D, page, seed=22)
    args = (ptab.cuda(), P, table.cuda(), ps.cuda(), page, 30)
    kw = {"softcap": cap, "slopes": slopes_of(H) if bias else None}

    def run(q, kp, keep):
        lse = torch.empty(B, H, device="cuda")
        return swa.swa_decode_shared(q, kp, vp, *args, lse=lse, keep_prefix=keep, **kw), lse
    for keep in (True, False):
        want, want_lse = run(q, kp, keep)
        bad = torch.zeros(B, H, dtype=torch.bool, device="cuda")
        bad[0, 2] = bad[1, 0] = bad[2, 7] = bad[3, 4] = True
        q2 = q.clone()
        q2[bad] = float("nan")
        got, lse = run(q2, kp, keep)
        expect(got, want, bad)
        expect(lse, want_lse, bad)
        k2 = kp.clone()
        k2[int(ptab[0]) * page, 1, 3] = float("nan")  # position 0
        bad[:] = False
        seen = [keep or p < 30 for p in pos]
        bad[torch.tensor(seen, device="cuda"), 4:] = True
        got, lse = run(q, k2, keep)
        expect(got, want, bad)
        expect(lse, want_lse, bad)


@pytest.mark.parametrize("cap,bias", FORMS)
@pytest.mark.parametrize("H,Hkv,N,D", [(2, 1, 300, 128), (3, 3, 300, 64), (32, 8, 1300, 128)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_infinities_stay_with_the_rows_that_see_them(swa, cap, bias, H, Hkv, N, D, value):
    L, cu = 40, [0, 90, 200, N - 5]
    q, k, v, _ = inputs(1, N, H, Hkv, D, 23)
    kw = {"win_left": L, "win_right": 0, "softcap": cap, "slopes": slopes_of(H) if bias else None,
          "cu_docs": torch.tensor([cu], dtype=torch.int32, device="cuda")}
    want = swa.swa_forward_scored(q, k, v, **kw)
    hit = torch.zeros(1, N, H, dtype=torch.bool, device="cuda")
    for j, e in ((10, 90), (100, 200), (230, N - 5)):
        k[:, j, 0, 3] = value
        hit[:, j:min(j + L + 1, e), :H // Hkv] = True
    for i in (60, 150, 285):
        q[:, i, H - 1, 9] = value
        hit[:, i, H - 1] = True
    got = swa.swa_forward_scored(q, k, v, **kw)
    assert torch.equal(got[~hit], want[~hit])
