"""Rotated append into a paged cache (C ABI) against the 64-bit rotation: every element
of the rotated queries, the pages row by row, and what must stay untouched."""
import pytest
import torch

import score_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def swa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import sliding_window_attention_fwd_b200 as m
    return m


def freqs(rot, base=10000.0):
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    return (base ** (-i / rot)).float().cuda()


def make(lens, pos0, H, Hkv, D, page, packed, extra=0, seed=0):
    """Inputs of a call; `extra` rows of no sequence behind the last one."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens) + extra
    if packed:
        qkv = torch.randn(T, (H + 2 * Hkv) * D, generator=g, device="cuda").to(BF)
        q, k, v = qkv.split((H * D, Hkv * D, Hkv * D), 1)
        q, k, v = q.unflatten(1, (H, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))
    else:
        q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").to(BF) for h in (H, Hkv, Hkv))
    need = [0 if n == 0 or p < 0 else (p + n - 1) // page - p // page + 1
            for n, p in zip(lens, pos0)]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed))
    cols = max([(p + n - 1) // page + 1 for n, p in zip(lens, pos0) if n and p >= 0] + [1])
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    at = 0
    for b, (n, p) in enumerate(zip(need, pos0)):
        if n:
            table[b, p // page:p // page + n] = order[at:at + n].to(torch.int32)
            at += n
    kp = torch.randn(n_pages * page, Hkv, D, generator=g, device="cuda").to(BF)
    vp = torch.randn(n_pages * page, Hkv, D, generator=g, device="cuda").to(BF)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    return q, k, v, cu.cuda(), torch.tensor(pos0, dtype=torch.int64).cuda(), table.cuda(), kp, vp


def expected(q, k, v, inv, cu, pos0, table, kp, vp, page, inter, q_out):
    """(values, bounds) of q_out, k_pages, v_pages in 64 bits."""
    eq, ek, ev = q_out.double(), kp.double(), vp.double()
    bq, bk = torch.zeros_like(eq), torch.zeros_like(ek)
    for b in range(pos0.shape[0]):
        a, e = int(cu[b]), int(cu[b + 1])
        p0 = int(pos0[b])
        if p0 < 0 or a == e:
            continue
        pos = torch.arange(p0, p0 + e - a, device="cuda")
        eq[a:e] = R.rotate(q[a:e], pos, inv, inter)
        bq[a:e] = R.rotate_error(q[a:e], eq[a:e], inv, inter)
        lp = pos // page
        there = lp < table.shape[1]
        pg = torch.where(there, table[b, lp.clamp(max=table.shape[1] - 1)].long(), -1)
        there &= (pg >= 0) & (pg < kp.shape[0] // page)
        row = (pg * page + pos % page)[there]
        y = R.rotate(k[a:e], pos, inv, inter)
        ek[row], bk[row] = y[there], R.rotate_error(k[a:e], y, inv, inter)[there]
        ev[row] = v[a:e].double()[there]
    return (eq, ek, ev), (bq, bk)


def run(swa, lens, pos0, H, Hkv, D, page, rot, inter, packed, extra=0, table_edit=None,
        in_place=False, seed=0):
    q, k, v, cu, p0, table, kp, vp = make(lens, pos0, H, Hkv, D, page, packed, extra, seed)
    if table_edit:
        table_edit(table, kp.shape[0] // page)
    inv = freqs(rot)
    q0 = q.clone()
    q_out = q if in_place else torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    want, bound = expected(q0, k, v, inv, cu, p0, table, kp, vp, page, inter, q_out)
    got = swa.swa_rope_append_paged(q, k, v, inv, cu, p0, table, kp, vp, page, q_out=q_out,
                                    interleaved=inter)
    torch.cuda.synchronize()
    assert got is q_out and swa.swa_device_error() == 0
    assert ((q_out.double() - want[0]).abs() <= bound[0]).all()
    assert ((kp.double() - want[1]).abs() <= bound[1]).all()
    assert torch.equal(vp.double(), want[2])


@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 16), (64, 64), (64, 32), (64, 16)])
@pytest.mark.parametrize("inter", [False, True])
def test_rotations(swa, D, rot, inter):
    run(swa, [1, 5, 0, 70, 3], [0, 62, 9, 131, 100000], 6, 2, D, 64, rot, inter, packed=False)


@pytest.mark.parametrize("lens,pos0,H,Hkv,page", [
    ([1], [0], 1, 1, 64),                                    # one token, one head
    ([1] * 64, [1000 * i + 7 for i in range(64)], 32, 8, 256),  # a decoding step
    ([0, 0, 0], [1, 2, 3], 4, 4, 64),                        # nothing
    ([0, 9, 0, 0, 2, 0], [5, 63, 5, 5, 64, 5], 4, 1, 64),    # empty sequences between
    ([300, 1, 1200], [0, 500, 77], 8, 2, 128),               # four tokens a block
    ([1025], [3], 2, 2, 1),                                  # pages of one row
    ([40, 41], [10, 30], 12, 12, 48),                        # pages of any size
])
@pytest.mark.parametrize("packed", [False, True])
def test_shapes(swa, lens, pos0, H, Hkv, page, packed):
    run(swa, lens, pos0, H, Hkv, 128, page, 128, False, packed, seed=len(lens))


def test_many_sequences(swa):
    """The search of a token's sequence over more boundaries than a warp's lanes squared."""
    lens = [(7 * i) % 3 for i in range(1500)]
    run(swa, lens, [i % 90 for i in range(1500)], 2, 1, 64, 64, 64, False, True)


def test_far_positions(swa):
    """Positions past 2^24 (the angle is reduced in 64 bits)."""
    T, p = 3, (1 << 31) + 12345
    q, k, v, cu, _, _, kp, vp = make([T], [0], 2, 1, 128, 64, False)
    inv = freqs(128)
    pos0 = torch.tensor([p], dtype=torch.int64, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")  # the page is missing
    before = kp.clone()
    got = swa.swa_rope_append_paged(q, k, v, inv, cu, pos0, table, kp, vp, 64)
    want = R.rotate(q, torch.arange(p, p + T, device="cuda"), inv, False)
    # the 64-bit angle itself is off by 2^-53 of some 2^31 rad
    assert ((got.double() - want).abs() <= R.rotate_error(q, want, inv, False) + 1e-5).all()
    assert torch.equal(kp, before)


def test_inactive_sequences_and_rows_of_none(swa):
    run(swa, [4, 6, 5], [3, -1, 70], 4, 2, 128, 64, 128, False, True, extra=5)
    run(swa, [700, 600], [-5, 70], 4, 2, 64, 64, 64, True, False, extra=9)


def test_missing_pages(swa):
    def edit(table, n):
        table[0, 0], table[1, 1] = -1, n
    run(swa, [100, 130], [10, 20], 4, 2, 128, 64, 128, False, False, table_edit=edit)


def test_in_place_queries(swa):
    run(swa, [33, 1], [10, 2000], 4, 2, 128, 64, 64, False, True, in_place=True)
    run(swa, [33, 1], [10, 2000], 4, 2, 64, 64, 64, True, False, in_place=True)


def test_large_offsets(swa):
    """A cache whose element offsets pass 2^32."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    Hkv, D, page = 8, 128, 64
    rows = ((1 << 32) // (Hkv * D) + 4 * page) // page * page
    kp, vp = (torch.zeros(rows, Hkv, D, dtype=BF, device="cuda") for _ in range(2))
    q, k, v, cu, pos0, _, _, _ = make([3], [5], 8, Hkv, D, page, False)
    table = torch.tensor([[rows // page - 1]], dtype=torch.int32, device="cuda")
    inv = freqs(D)
    swa.swa_rope_append_paged(q, k, v, inv, cu, pos0, table, kp, vp, page)
    want = R.rotate(k, torch.arange(5, 8, device="cuda"), inv, False)
    at = rows - page + 5
    assert ((kp[at:at + 3].double() - want).abs() <= R.rotate_error(k, want, inv, False)).all()
    assert torch.equal(vp[at:at + 3], v)
    assert not kp[:at].any() and not vp[:at].any()


def test_captured_and_on_a_stream(swa):
    q, k, v, cu, pos0, table, kp, vp = make([5, 6], [60, 3], 4, 2, 128, 64, True)
    inv = freqs(128)
    k2, v2 = kp.clone(), vp.clone()
    want = swa.swa_rope_append_paged(q, k, v, inv, cu, pos0, table, kp, vp, 64)
    out = torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        swa.swa_rope_append_paged(q, k, v, inv, cu, pos0, table, k2, v2, 64, q_out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(k2, kp) and torch.equal(v2, vp)


def test_token_strides_refused(swa):
    q, k, v, cu, pos0, table, kp, vp = make([5, 6], [60, 3], 4, 2, 64, 64, True)
    inv = freqs(64)

    def call(**kw):
        a = dict(q=q, k=k, v=v, inv_freq=inv, cu=cu, pos0=pos0, block_table=table, k_pages=kp,
                 v_pages=vp, page_size=64) | kw
        return swa.swa_rope_append_paged(**a)
    wide = torch.zeros(11, 4, 128, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        call(q=wide[:, :, :64])
    with pytest.raises(ValueError, match="contiguous"):
        call(q=wide[:, :, ::2])
    with pytest.raises(ValueError, match="overlap"):
        call(q=q[:1].expand(11, 4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        call(q_out=torch.zeros(11, 4, 64, dtype=BF))
    with pytest.raises(ValueError, match="CUDA"):
        call(cu=cu.cpu())
    with pytest.raises(swa.SwaError):  # tokens not on 16-byte boundaries
        odd = torch.zeros(11, 4 * 64 + 4, dtype=BF, device="cuda")
        call(q=odd[:, :256].unflatten(1, (4, 64)))
    with pytest.raises(swa.SwaError):
        call(inv_freq=inv[:12].contiguous())
    one = q[:1].as_strided((1, 4, 64), (3, 64, 1))  # one token: its stride does not matter
    call(q=one, k=k[:1], v=v[:1], cu=torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda"))
    none = q[:0]  # nothing to do
    assert call(q=none, k=k[:0], v=v[:0]).shape == (0, 4, 64)
    torch.cuda.synchronize()
    assert swa.swa_device_error() == 0
