"""A row's result goes by what the row sees: neither padding nor another document or
sequence changes a bit of it, whatever (finite) values they hold."""
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


@pytest.mark.parametrize("cap,bias", FORMS)
@pytest.mark.parametrize("H,Hkv,N,D", [(2, 1, 300, 128), (3, 3, 300, 64), (32, 8, 1300, 128),
                                       (32, 8, 1300, 64)])
@pytest.mark.parametrize("what", ["padding", "document"])
def test_forward_and_gradients(swa, cap, bias, H, Hkv, N, D, what):
    cu = [5, 100, 200, N - 10]
    mine = torch.zeros(N, dtype=torch.bool, device="cuda")
    mine[5:N - 10] = True
    if what == "document":
        mine[100:200] = False
    kw = {"win_left": 150, "win_right": 0, "softcap": cap,
          "slopes": slopes_of(H) if bias else None,
          "cu_docs": torch.tensor([cu], dtype=torch.int32, device="cuda")}
    results = []
    for factor in (1.0, 300.0):
        q, k, v, do = inputs(1, N, H, Hkv, D, 31)
        for t in (q, k, v, do):
            t[:, ~mine] *= factor
        lse = torch.empty(1, H, N, device="cuda")
        out = swa.swa_forward_scored(q, k, v, lse=lse, **kw)
        g = swa.swa_backward_scored(q, k, v, out, do, lse, **kw)
        results.append([out[:, mine], lse[:, :, mine], *(x[:, mine] for x in g)])
    for a, b in zip(*results):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("cap,bias", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [4, 140])
def test_decode(swa, cap, bias, D, B):
    P, page, H, Hkv = 700, 64, 8, 2
    pos = [P + (b * 29) % 100 for b in range(B)]
    q, kp, vp, ptab, table, ps = build(P, pos, H, Hkv, D, page, seed=32)
    args = (ptab.cuda(), P, table.cuda(), ps.cuda(), page, 200)
    kw = {"softcap": cap, "slopes": slopes_of(H) if bias else None}
    want = swa.swa_decode_shared(q, kp, vp, *args, **kw)
    q[2] *= 300.0
    got = swa.swa_decode_shared(q, kp, vp, *args, **kw)
    rest = [b for b in range(B) if b != 2]
    assert torch.equal(got[rest], want[rest])
