"""Decode behind a shared prefix against the 64-bit form, and the serving loop it
belongs to: rotated append, then decode."""
import math

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


def build(P, pos, H, Hkv, D, page, seed=0, std=2.0):
    """A pool whose unused rows hold NaN, tables, and per sequence the keys by position."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(pos)
    shared = -(-P // page)
    own = [0 if p < P else p // page - P // page + 1 for p in pos]
    n = shared + sum(own) + 2
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    cols = max([p // page + 1 for p in pos] + [1])
    ptab = torch.full((max(shared, 1),), -1, dtype=torch.int32)
    ptab[:shared] = order[:shared]
    table = torch.full((B, cols), -1, dtype=torch.int32)
    kp = torch.full((n * page, Hkv, D), float("nan"), dtype=BF, device="cuda")
    vp = torch.full_like(kp, float("nan"))

    def fill(page_of, a, e):
        j = torch.arange(a, max(a, e))
        if len(j):
            row = (page_of[j // page].long() * page + j % page).cuda()
            for t in (kp, vp):
                t[row] = torch.randn(len(j), Hkv, D, generator=g, device="cuda").to(BF)
    fill(ptab, 0, P)
    at = shared
    for b, p in enumerate(pos):
        table[b, P // page:P // page + own[b]] = order[at:at + own[b]]
        at += own[b]
        fill(table[b], P, p + 1)
    q = (torch.randn(B, H, D, generator=g, device="cuda") * std).to(BF)
    return q, kp, vp, ptab, table, torch.tensor(pos, dtype=torch.int64)


def reference(q, kp, vp, ptab, table, pos, P, page, W, keep, cap, slopes, scale=0.0):
    B, H, D = q.shape
    Hkv = kp.shape[1]
    scale = scale if scale > 0 else 1.0 / math.sqrt(D)

    def z(*s):
        return torch.zeros(*s, dtype=torch.float64, device="cuda")
    ref = {"out": z(B, H, D), "e_out": z(B, H, D), "lse": z(B, H), "e_lse": z(B, H)}
    for b, p in enumerate(pos.tolist()):
        j = torch.tensor([x for x in range(p + 1) if x > p - W or (keep and x < P)],
                         dtype=torch.int64)
        if not len(j):
            ref["lse"][b] = -math.inf
            continue
        pg = torch.where(j < P, ptab[(j // page).clamp(max=len(ptab) - 1)],
                         table[b, (j // page).clamp(max=table.shape[1] - 1)])
        gone = (pg < 0).cuda()
        row = (pg.clamp(min=0).long() * page + j % page).cuda()
        dist = (p - j).double().cuda()[None]
        for h in range(H):
            g = h // (H // Hkv)
            k, v = (torch.where(gone[:, None], 0.0, t[row, g].double()) for t in (kp, vp))
            r = R.attention(q[b, h][None], k, v, torch.ones(1, len(j), dtype=torch.bool,
                                                            device="cuda"),
                            scale, cap, None if slopes is None else float(slopes[h]), dist)
            for n in ref:
                ref[n][b, h] = r[n][0]
    # parts are joined by e^(lse_i - lse): two fp32 exponentials and logarithms of lse
    big = torch.where(torch.isinf(ref["lse"]), 0.0, ref["lse"]).abs() + 1.0
    ref["e_lse"] += 16 * R.HALF_F32 * big
    ref["e_out"] += (32 * R.HALF_F32 * big)[..., None] * ref["e_out"] / R.HALF_BF16
    return ref


def run(swa, P, pos, H, Hkv, D, page, W, keep=True, cap=0.0, bias=False, max_tail=None, scale=0.0,
        edit=None, std=2.0):
    q, kp, vp, ptab, table, ps = build(P, pos, H, Hkv, D, page, seed=P + len(pos), std=std)
    if edit:
        edit(ptab, table)
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)],
                          device="cuda") if bias else None
    nan = float("nan")
    out, lse = torch.full_like(q, nan), torch.full((len(pos), H), nan, device="cuda")
    swa.swa_decode_shared(q, kp, vp, ptab.cuda(), P, table.cuda(), ps.cuda(), page, W, out=out,
                          lse=lse, keep_prefix=keep, max_tail=max_tail, softcap=cap,
                          slopes=slopes, scale=scale)
    torch.cuda.synchronize()
    assert swa.swa_device_error() == 0
    R.check({"out": out, "lse": lse},
            reference(q, kp, vp, ptab, table, ps, P, page, W, keep, cap, slopes, scale),
            ("out", "lse"))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [0, 1, 63, 64, 65, 128, 300, 1024])
def test_prefix_lengths(swa, P, D):
    pos = [P, P + 1, P + 70, P + 200, P + 127]
    run(swa, P, pos, 8, 2, D, 64, 100)
    run(swa, P, pos, 8, 2, D, 128, 100, keep=False, cap=20.0)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 1), (12, 12), (6, 2), (10, 2), (16, 16)])
@pytest.mark.parametrize("D", [64, 128])
def test_head_layouts(swa, H, Hkv, D):
    run(swa, 200, [200, 333, 260], H, Hkv, D, 64, 90, cap=30.0, bias=True)


@pytest.mark.parametrize("B", [1, 2, 31, 33, 64, 100])
@pytest.mark.parametrize("D", [64, 128])
def test_batches(swa, B, D):
    """Query rows of one, two and more tiles, with partly filled last ones."""
    run(swa, 260, [260 + (37 * b) % 150 for b in range(B)], 8, 2, D, 64, 64, keep=B % 2 == 0,
        bias=B > 32)


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("W", [1, 64, 129, 5000])
def test_windows(swa, W, keep):
    """Windows that end behind the prefix, inside it and before it."""
    run(swa, 500, [500, 530, 700, 900], 4, 2, 128, 64, W, keep=keep, cap=50.0)


def test_positions_inside_the_prefix_and_inactive_sequences(swa):
    run(swa, 400, [0, 5, 399, 400, 450], 4, 2, 128, 64, 200)
    run(swa, 400, [-1, 5, -7, 480, -2 ** 40], 4, 2, 64, 64, 200, keep=False)
    run(swa, 400, [-1, -1], 4, 2, 128, 64, 200)


@pytest.mark.parametrize("max_tail", [0, 1, 300, 3000, 2 ** 31 - 1])
def test_max_tail_only_splits(swa, max_tail):
    run(swa, 130, [2300, 130, 1500], 4, 2, 128, 64, 2100, max_tail=max_tail)
    run(swa, 130, [2300, 130, 1500], 4, 2, 64, 64, 2100, max_tail=max_tail, bias=True)


def test_missing_pages_read_as_zero_keys(swa):
    def edit(ptab, table):
        ptab[1] = -1
        table[0, 5] = -1
    run(swa, 256, [400, 300], 4, 2, 128, 64, 500, edit=edit)
    run(swa, 256, [400, 300], 4, 2, 64, 64, 500, edit=edit, cap=20.0)


def test_scale_and_scores_past_the_cap(swa):
    run(swa, 300, [350, 420], 4, 1, 128, 64, 64, cap=2.0, std=6.0)
    run(swa, 300, [350, 420], 4, 1, 64, 64, 64, scale=0.4)


def test_without_a_prefix_it_is_the_paged_decode(swa):
    q, kp, vp, ptab, table, pos = build(0, [1000, 20, 513], 8, 2, 128, 64)
    kp, vp = kp.nan_to_num(), vp.nan_to_num()  # swa_decode_paged wants finite pages
    a = swa.swa_decode_paged(q, kp, vp, table.cuda(), pos.cuda(), 64, 300)
    b = swa.swa_decode_shared(q, kp, vp, ptab.cuda(), 0, table.cuda(), pos.cuda(), 64, 300)
    assert (a.float() - b.float()).abs().max() <= 4 * R.HALF_BF16 * a.float().abs().max()


def test_large_offsets(swa):
    """A page pool whose element offsets pass 2^32, its last pages in use."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    H, Hkv, D, page, P, W = 8, 8, 128, 64, 150, 100
    q, k0, v0, ptab, table, pos = build(P, [200, 333], H, Hkv, D, page)
    rows = ((1 << 32) // (Hkv * D) + k0.shape[0]) // page * page
    kp, vp = (torch.zeros(rows, Hkv, D, dtype=BF, device="cuda") for _ in range(2))
    kp[-k0.shape[0]:], vp[-v0.shape[0]:] = k0, v0
    want = swa.swa_decode_shared(q, k0, v0, ptab.cuda(), P, table.cuda(), pos.cuda(), page, W)
    up = (rows - k0.shape[0]) // page
    ptab, table = torch.where(ptab < 0, ptab, ptab + up), torch.where(table < 0, table, table + up)
    got = swa.swa_decode_shared(q, kp, vp, ptab.cuda(), P, table.cuda(), pos.cuda(), page, W)
    assert torch.equal(got, want)


def test_nan_of_a_seen_key_stays_visible_and_where_it_is(swa):
    """A NaN score makes its row NaN, whichever part holds it, and no other row."""
    P, page, H, Hkv = 300, 64, 8, 2
    q, kp, vp, ptab, table, pos = build(P, [P + 400, P + 9, P + 130], H, Hkv, 128, page, seed=5)
    args = (ptab.cuda(), P, table.cuda(), pos.cuda(), page, 1000)
    want = swa.swa_decode_shared(q, kp, vp, *args)
    j = P + 200  # a key of sequence 0 alone
    own = kp.clone()
    own[int(table[0, j // page]) * page + j % page, 1, 3] = float("nan")
    got = swa.swa_decode_shared(q, own, vp, *args)
    assert torch.isnan(got[0, 4:]).all()
    assert torch.equal(got[0, :4], want[0, :4]) and torch.equal(got[1:], want[1:])
    first = kp.clone()
    first[int(ptab[1]) * page + 7, 0, 3] = float("nan")
    got = swa.swa_decode_shared(q, first, vp, *args)
    assert torch.isnan(got[:, :4]).all() and torch.equal(got[:, 4:], want[:, 4:])
    bad = q.clone()
    bad[1, 2, 0] = float("nan")
    lse = torch.empty(3, H, device="cuda")
    got = swa.swa_decode_shared(bad, kp, vp, *args, lse=lse)
    assert torch.isnan(got[1, 2]).all() and torch.isnan(lse[1, 2])
    keep = torch.ones(3, H, dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("D", [64, 128])
def test_prefix_rows_that_no_query_sees_may_hold_nan(swa, D):
    """In front of every window, and behind every position inside the prefix."""
    P, page, W, pos = 500, 64, 90, [333, 350, 401]
    q, kp, vp, ptab, table, ps = build(P, pos, 8, 2, D, page, seed=6)
    args = (ptab.cuda(), P, table.cuda(), ps.cuda(), page, W)
    want = swa.swa_decode_shared(q, kp, vp, *args, keep_prefix=False)
    for j in [*range(0, 333 - W + 1), *range(402, P)]:
        row = int(ptab[j // page]) * page + j % page
        kp[row] = vp[row] = float("nan")
    assert torch.equal(swa.swa_decode_shared(q, kp, vp, *args, keep_prefix=False), want)


def test_many_rows_without_a_prefix(swa):
    """More rows than the SMs take at once, no prefix and no prefix pages."""
    B, H, Hkv, page = 1200, 64, 8, 64
    q, kp, vp, ptab, table, pos = build(0, [b % 5 for b in range(B)], H, Hkv, 64, page, seed=7)
    got = swa.swa_decode_shared(q, kp, vp, ptab.cuda(), 0, table.cuda(), pos.cuda(), page, 8)
    some = list(range(0, B, 173))
    ref = reference(q[some], kp, vp, ptab, table[some], pos[some], 0, page, 8, True, 0.0, None)
    R.check({"out": got[some]}, ref, ("out",))
    for b in range(20, B, 5):  # (every fifth sequence has one key: its value)
        row = int(table[b, 0]) * page
        if int(pos[b]) == 0:
            assert torch.equal(got[b], vp[row].repeat_interleave(H // Hkv, 0))


def test_captured_and_at_once(swa):
    """Two captured decodes of different sizes replayed in turn; two calls at once."""
    sides, st = [], [torch.cuda.Stream() for _ in range(2)]
    for i, (P, pos) in enumerate(((300, [310, 420, 300]), (2000, [2500 + b for b in range(40)]))):
        q, kp, vp, ptab, table, ps = build(P, pos, 8, 2, 128, 64, seed=i)
        args = (q, kp, vp, ptab.cuda(), P, table.cuda(), ps.cuda(), 64, 256)
        want = swa.swa_decode_shared(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = swa.swa_decode_shared(*args)
        sides.append((args, want, graph, got))
    for _ in range(3):
        for args, want, graph, got in sides:
            got.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
    outs = [[], []]
    for _ in range(5):
        for i in range(2):
            outs[i].append(swa.swa_decode_shared(*sides[i][0], stream=st[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, sides[i][1])


def test_serving_loop(swa):
    """A shared prompt is appended once, then three sequences grow token by token:
    append with rotation, decode behind the prefix, as one program uses them."""
    H, Hkv, D, page, P, W, steps = 4, 2, 128, 64, 150, 64, 70
    g = torch.Generator(device="cuda").manual_seed(3)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda").to(BF)
    inv = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    B, shared = 3, -(-P // page)
    per = (P + steps - 1) // page - P // page + 1
    n = shared + B * per
    kp, vp = rnd(n * page, Hkv, D), rnd(n * page, Hkv, D)
    ptab = torch.arange(shared, dtype=torch.int32, device="cuda")
    table = torch.full((B, P // page + per), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        table[b, P // page:] = torch.arange(shared + b * per, shared + (b + 1) * per,
                                            dtype=torch.int32)
    z = torch.zeros(1, dtype=torch.int64, device="cuda")
    prompt = [rnd(P, h, D) for h in (H, Hkv, Hkv)]
    swa.swa_rope_append_paged(*prompt, inv, torch.tensor([0, P], dtype=torch.int32, device="cuda"),
                              z, ptab[None], kp, vp, page)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    for t in range(steps):
        pos = torch.full((B,), P + t, dtype=torch.int64, device="cuda")
        q = swa.swa_rope_append_paged(rnd(B, H, D), rnd(B, Hkv, D), rnd(B, Hkv, D), inv, cu, pos,
                                      table, kp, vp, page)
        out, lse = torch.empty_like(q), torch.empty(B, H, device="cuda")
        swa.swa_decode_shared(q, kp, vp, ptab, P, table, pos, page, W, out=out, lse=lse,
                              softcap=30.0)
        if t % 23 == 0 or t == steps - 1:
            ref = reference(q, kp, vp, ptab.cpu(), table.cpu(), pos.cpu(), P, page, W, True, 30.0,
                            None)
            R.check({"out": out, "lse": lse}, ref, ("out", "lse"), f"step {t}")
    assert swa.swa_device_error() == 0
