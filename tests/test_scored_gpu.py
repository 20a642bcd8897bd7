"""Attention with shaped scores, forward and backward, against the 64-bit form with
bounds derived from the roundings (score_ref)."""
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


def inputs(B, N, H, Hkv, D, seed=0, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(h, s=1.0):
        return (torch.randn(B, N, h, D, generator=g, device="cuda") * s).to(BF)
    return n(H, std), n(Hkv), n(Hkv), n(H)


def slopes_of(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")


def poison(t, cu):
    """NaN and infinities in the padding rows of t."""
    for b, c in enumerate(cu):
        t[b, :c[0]] = float("nan")
        t[b, c[-1]:] = float("inf")
        t[b, c[-1]::2] = float("nan")


def run(swa, B, N, H, Hkv, D, L, Rr, cap=0.0, bias=False, cu=None, pre=None, scale=0.0, std=2.0,
        seed=0):
    q, k, v, do = inputs(B, N, H, Hkv, D, seed, std)
    if cu is not None:
        for t in (q, k, v, do):
            poison(t, cu)
    kw = {"win_left": L, "win_right": Rr, "softcap": cap, "scale": scale,
          "slopes": slopes_of(H) if bias else None,
          "cu_docs": None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"),
          "prefix": None if pre is None else torch.tensor(pre, dtype=torch.int32, device="cuda")}
    nan = float("nan")
    out, lse = torch.full_like(q, nan), torch.full((B, H, N), nan, device="cuda")
    swa.swa_forward_scored(q, k, v, out=out, lse=lse, **kw)
    g = {n: torch.full_like(t, nan) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    swa.swa_backward_scored(q, k, v, out, do, lse, **g, **kw)
    torch.cuda.synchronize()
    assert swa.swa_device_error() == 0
    ref = R.forward(q, k, v, L, Rr, cap, kw["slopes"], cu, pre, scale, do)
    R.check({"out": out, "lse": lse, **g}, ref, ("out", "lse", "dq", "dk", "dv"))


@pytest.mark.parametrize("cap,bias", [(0.0, False), (50.0, False), (0.0, True), (20.0, True)])
@pytest.mark.parametrize("H,Hkv,D", [(4, 2, 128), (3, 3, 128), (4, 2, 64), (3, 3, 64)])
def test_scores(swa, cap, bias, H, Hkv, D):
    run(swa, 2, 300, H, Hkv, D, 100, 0, cap, bias)


@pytest.mark.parametrize("cap", [0.5, 3.0])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_past_the_cap(swa, cap, D):
    """Most scores lie past the cap."""
    run(swa, 1, 200, 2, 1, D, -1, 0, cap, False, std=6.0)


@pytest.mark.parametrize("cap", [50.0, 51.0])  # with and without a running maximum
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [-1.0, 1.0, 0.0])
def test_saturated_scores(swa, cap, D, sign):
    """Every score at the cap: below zero, above it, or some of each."""
    for H, Hkv, N in ((2, 1, 200), (32, 8, 700)):
        q, k, v, do = inputs(1, N, H, Hkv, D, std=60.0)
        if sign:
            q, k = q.abs(), k.abs() * sign
        kw = {"win_left": 150, "win_right": 0, "softcap": cap}
        lse = torch.empty(1, H, N, device="cuda")
        out = swa.swa_forward_scored(q, k, v, lse=lse, **kw)
        g = swa.swa_backward_scored(q, k, v, out, do, lse, **kw)
        torch.cuda.synchronize()
        ref = R.forward(q, k, v, 150, 0, cap, None, None, None, 0.0, do)
        R.check({"out": out, "lse": lse, **dict(zip(("dq", "dk", "dv"), g))}, ref,
                ("out", "lse", "dq", "dk", "dv"))


@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 127, 128, 129, 257, 700])
def test_lengths(swa, N):
    run(swa, 1, N, 2, 1, 128, -1, 0, 30.0, True)
    run(swa, 2, N, 2, 2, 64, 70, 5, 30.0, True)


@pytest.mark.parametrize("L,Rr", [(-1, -1), (0, 0), (0, -1), (5, 3), (128, 128), (-1, 200),
                                  (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows(swa, L, Rr):
    run(swa, 1, 400, 4, 2, 128, L, Rr, 20.0, True)
    run(swa, 1, 400, 4, 2, 64, L, Rr, 20.0, False, cu=[[0, 100, 391]], pre=[[60, 150]])


@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 1), (12, 1), (6, 2), (10, 2), (16, 16)])
def test_head_layouts(swa, H, Hkv):
    run(swa, 1, 150, H, Hkv, 128, 90, 0, 20.0, True, cu=[[0, 50, 140]])
    run(swa, 1, 150, H, Hkv, 64, 90, 0, 20.0, True, cu=[[0, 50, 140]])


DOCS = {
    "one": [[0, 520]],
    "tiles": [[0, 128, 256, 520]],
    "ragged": [[0, 1, 2, 130, 131, 400, 517]],
    "empty documents": [[0, 0, 0, 77, 77, 300, 300, 300]],
    "padding on both sides": [[200, 290, 310, 385]],
    "padding of whole tiles": [[257, 258, 300]],
    "nothing": [[0, 0, 0]],
    "nothing, at the end": [[520, 520]],
    "single tokens": [list(range(0, 520, 1))],
}


@pytest.mark.parametrize("name", DOCS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [False, True])
def test_documents(swa, name, D, prefix):
    cu = DOCS[name]
    pre = [[(3 * (e - a)) // (2 + m % 4) for m, (a, e) in enumerate(zip(c, c[1:]))] for c in cu]
    run(swa, 1, 520, 4, 2, D, 150, 0, 20.0, False, cu=cu, pre=pre if prefix else None)
    run(swa, 1, 520, 2, 2, D, -1, 0, 0.0, True, cu=cu, pre=pre if prefix else None)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (20.0, True)])
def test_two_heads_per_cta(swa, D, cap, bias):
    """Enough work to fill the SMs with two heads per CTA."""
    cu = [[0, 100, 101, 600, 700], [30, 260, 260, 500, 650]]
    pre = [[40, 5, 300, 0], [10, 0, 100, 1000]]
    run(swa, 2, 705, 32, 8, D, 300, 0, cap, bias, cu=cu, pre=pre)
    run(swa, 1, 705, 64, 16, D, 130, 90, cap, bias)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 20.0, 80.0])
def test_more_items_than_a_wave(swa, D, cap):
    """Several items per SM, of many lengths and some empty: tiles of padding, single
    tokens, more documents than lanes."""
    cu = [[0] + list(range(300, 340)) + [900, 990], [400] * 30 + list(range(401, 413)) + [450],
          [0] * 20 + list(range(0, 1000, 45))]
    assert len({len(c) for c in cu}) == 1
    run(swa, 3, 1000, 32, 8, D, 200, 0, cap, False, cu=cu)
    run(swa, 2, 1030, 32, 8, D, -1, -1, cap, False, cu=[[0, 513, 1030], [129, 140, 640]])


@pytest.mark.parametrize("D", [64, 128])
def test_many_key_tiles(swa, D):
    """Packed documents over more key tiles than SMs (their longest walks go first)."""
    cu = [[0, 700, 701, 900, 1390], [130, 131, 131, 500, 1400]]
    pre = [[40, 5, 100, 0], [1, 0, 100, 1000]]
    run(swa, 2, 1400, 16, 8, D, -1, 0, 20.0, False, cu=cu, pre=pre)
    run(swa, 2, 1400, 16, 8, D, 600, 40, 0.0, True, cu=cu)


def test_batch_of_different_documents(swa):
    cu = [[0, 100, 300], [10, 10, 290], [0, 0, 0]]
    pre = [[0, 40], [7, 1000], [-3, 5]]
    run(swa, 3, 300, 4, 2, 128, 120, 0, 50.0, False, cu=cu, pre=pre)
    run(swa, 3, 300, 4, 4, 64, -1, -1, 50.0, True, cu=cu)


def test_scale(swa):
    run(swa, 1, 200, 2, 1, 128, 64, 0, 20.0, False, scale=0.3)


def test_steep_bias_and_large_scores(swa):
    """Scores far apart: rows whose maximum moves by much between key tiles."""
    q, k, v, do = inputs(1, 700, 2, 1, 128, 3, std=8.0)
    for sl in ([1.5, 0.75], [-0.5, -0.25]):
        s = torch.tensor(sl, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(1, 2, 700, device="cuda")
        swa.swa_forward_scored(q, k, v, out=out, lse=lse, win_left=-1, win_right=0, slopes=s)
        dq, dk, dv = swa.swa_backward_scored(q, k, v, out, do, lse, win_left=-1, win_right=0,
                                             slopes=s)
        ref = R.forward(q, k, v, -1, 0, 0.0, s, dout=do)
        R.check({"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, ref,
                ("out", "lse", "dq", "dk", "dv"))


def test_plain_scores_equal_the_plain_forward(swa):
    q, k, v, do = inputs(2, 333, 4, 2, 128)
    lse, lse2 = (torch.empty(2, 4, 333, device="cuda") for _ in range(2))
    a = swa.swa_forward(q, k, v, lse=lse, win_left=99, win_right=0)
    b = swa.swa_forward_scored(q, k, v, lse=lse2, win_left=99, win_right=0)
    assert torch.equal(a, b) and torch.equal(lse, lse2)
    ga = swa.swa_backward(q, k, v, a, do, lse, win_left=99, win_right=0)
    gb = swa.swa_backward_scored(q, k, v, a, do, lse, win_left=99, win_right=0)
    for x, y in zip(ga, gb):
        assert torch.equal(x, y)


def test_gradients_against_differences(swa):
    """<dq, x> + <dk, y> + <dv, z> against a central difference of the 64-bit loss."""
    B, N, H, Hkv, D = 1, 140, 2, 1, 64
    q, k, v, do = inputs(B, N, H, Hkv, D, 5)
    cu, pre = [[0, 60, 133]], [[20, 30]]
    sl = slopes_of(H)
    kw = {"win_left": 50, "win_right": 0, "softcap": 10.0, "slopes": sl,
          "cu_docs": torch.tensor(cu, dtype=torch.int32, device="cuda"),
          "prefix": torch.tensor(pre, dtype=torch.int32, device="cuda")}
    lse = torch.empty(B, H, N, device="cuda")
    out = swa.swa_forward_scored(q, k, v, lse=lse, **kw)
    grads = swa.swa_backward_scored(q, k, v, out, do, lse, **kw)
    ref = R.forward(q, k, v, 50, 0, 10.0, sl, cu, pre, dout=do)
    gen = torch.Generator(device="cuda").manual_seed(9)
    dirs = [torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64)
            for t in (q, k, v)]

    def loss(h):
        x = [t.double() + h * d for t, d in zip((q, k, v), dirs)]
        return float((R.forward(*x, 50, 0, 10.0, sl, cu, pre)["out"] * do.double()).sum())
    h = 1e-5
    fd = (loss(h) - loss(-h)) / (2 * h)
    got = sum(float((g.double() * d).sum()) for g, d in zip(grads, dirs))
    exact = sum(float((ref[n] * d).sum()) for n, d in zip(("dq", "dk", "dv"), dirs))
    # the formula's own derivative: the difference's third-order term and cancellation
    assert abs(fd - exact) <= 1e-5 * max(1.0, abs(exact))
    bound = sum(float((ref["e_" + n] * d.abs()).sum()) for n, d in zip(("dq", "dk", "dv"), dirs))
    assert abs(got - fd) <= bound


def test_same_bits_every_time(swa):
    q, k, v, do = inputs(2, 500, 8, 2, 128, 7)
    kw = {"win_left": 200, "win_right": 0, "softcap": 30.0}
    lse = torch.empty(2, 8, 500, device="cuda")
    out = swa.swa_forward_scored(q, k, v, lse=lse, **kw)
    first = swa.swa_backward_scored(q, k, v, out, do, lse, **kw)
    for _ in range(3):
        for a, b in zip(first, swa.swa_backward_scored(q, k, v, out, do, lse, **kw)):
            assert torch.equal(a, b)


def test_captured_steps(swa):
    """Two captured training steps of different sizes, replayed in turn and against
    eager calls; calls on another stream."""
    cases = []
    s = torch.cuda.Stream()
    for N, cap in ((200, 20.0), (900, 0.0)):
        q, k, v, do = inputs(1, N, 4, 2, 64, N)
        kw = {"win_left": 100, "win_right": 0, "softcap": cap, "slopes": slopes_of(4)}
        lse = torch.empty(1, 4, N, device="cuda")

        def step(q=q, k=k, v=v, do=do, lse=lse, kw=kw, **st):
            out = swa.swa_forward_scored(q, k, v, lse=lse, **kw, **st)
            return (out, *swa.swa_backward_scored(q, k, v, out, do, lse, **kw, **st))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for st in (s, s.cuda_stream):
            got = step(stream=st)
            s.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        cases.append((graph, got, want, step))  # (step keeps the captured inputs alive)
    for _ in range(3):
        for graph, got, want, _ in cases:
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_two_calls_at_once(swa):
    """The calls share nothing: two backward passes on two streams."""
    st = [torch.cuda.Stream() for _ in range(2)]
    data, want = [], []
    for i in range(2):
        q, k, v, do = inputs(1, 1200, 8, 2, 128, i)
        lse = torch.empty(1, 8, 1200, device="cuda")
        out = swa.swa_forward_scored(q, k, v, lse=lse, win_left=400, win_right=0, softcap=20.0)
        data.append((q, k, v, out, do, lse))
        want.append(swa.swa_backward_scored(*data[i], win_left=400, win_right=0, softcap=20.0))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            got[i].append(swa.swa_backward_scored(*data[i], win_left=400, win_right=0,
                                                  softcap=20.0, stream=st[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for a, b in zip(g, want[i]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, True)])
def test_nan_of_a_seen_key_stays_visible_and_where_it_is(swa, cap, bias):
    """A NaN key makes the rows that see it NaN, and no others."""
    q, k, v, _ = inputs(1, 300, 4, 2, 128)
    cu = torch.tensor([[0, 120, 290]], dtype=torch.int32, device="cuda")
    kw = {"win_left": 50, "win_right": 0, "softcap": cap, "slopes": slopes_of(4) if bias else None,
          "cu_docs": cu}
    want = swa.swa_forward_scored(q, k, v, **kw)
    k[0, 100, 1, 5] = float("nan")
    lse = torch.empty(1, 4, 300, device="cuda")
    got = swa.swa_forward_scored(q, k, v, lse=lse, **kw)
    sees = torch.zeros(300, dtype=torch.bool)
    sees[100:120] = True  # (the next document begins at 120)
    assert torch.isnan(got[0, sees, 2:]).all() and torch.isnan(lse[0, 2:, sees]).all()
    assert torch.equal(got[0, ~sees], want[0, ~sees])
    assert torch.equal(got[:, :, :2], want[:, :, :2])


def test_unbounded_windows_of_plain_scores(swa):
    q, k, v, do = inputs(1, 300, 4, 2, 128)
    lse = [torch.empty(1, 4, 300, device="cuda") for _ in range(2)]
    res = []
    for i, (a, b) in enumerate(((-1, -1), (2 ** 31 - 1, 2 ** 31 - 1))):
        out = swa.swa_forward_scored(q, k, v, lse=lse[i], win_left=a, win_right=b)
        res.append((out, *swa.swa_backward_scored(q, k, v, out, do, lse[i], win_left=a,
                                                  win_right=b)))
    ref = R.forward(q, k, v, -1, -1, 0.0, None, None, None, 0.0, do)
    for i, r in enumerate(res):
        R.check({"lse": lse[i], **dict(zip(("out", "dq", "dk", "dv"), r))}, ref,
                ("out", "lse", "dq", "dk", "dv"))


def test_results_belong_to_the_stream_of_the_call(swa):
    """Memory that another stream's work may still use is not taken for results."""
    q, k, v, do = inputs(1, 2048, 8, 2, 128)
    lse = torch.empty(1, 8, 2048, device="cuda")
    want = swa.swa_forward_scored(q, k, v, win_left=64, win_right=0, softcap=20.0, lse=lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = torch.empty_like(q)
    at = held.data_ptr()
    del held
    out = swa.swa_forward_scored(q, k, v, win_left=64, win_right=0, softcap=20.0, stream=side)
    grads = swa.swa_backward_scored(q, k, v, want, do, lse, win_left=64, win_right=0, softcap=20.0,
                                    stream=side)
    assert at not in [t.data_ptr() for t in (out, *grads)]
    assert torch.empty_like(q).data_ptr() == at  # (it was free)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("D", [64, 128])
def test_forwards_of_several_waves_at_once_and_captured(swa, D):
    """Forwards whose CTAs take several items: in two streams at once, each beside the
    other's, and replayed from graphs in turn."""
    st, calls = [torch.cuda.Stream() for _ in range(2)], []
    for i, (N, cu) in enumerate(((2000, [0, 700, 701, 1900]), (1500, [40, 600, 1500]))):
        q, k, v, _ = inputs(1, N, 32, 8, D, seed=i)
        kw = {"win_left": 900, "win_right": 0, "softcap": 30.0 * i,
              "cu_docs": torch.tensor([cu], dtype=torch.int32, device="cuda")}
        calls.append((q, k, v, kw))
    want = [swa.swa_forward_scored(q, k, v, **kw) for q, k, v, kw in calls]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (q, k, v, kw) in enumerate(calls):
            outs[i].append(swa.swa_forward_scored(q, k, v, stream=st[i], **kw))
    graphs = []
    torch.cuda.synchronize()
    for i, (q, k, v, kw) in enumerate(calls):
        assert all(torch.equal(o, want[i]) for o in outs[i])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = swa.swa_forward_scored(q, k, v, **kw)
        graphs.append((graph, got))
    for _ in range(3):
        for i, (graph, got) in enumerate(graphs):
            got.zero_()
        torch.cuda.synchronize()
        for i, (graph, got) in enumerate(graphs):
            with torch.cuda.stream(st[i]):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got, want[i]) for i, (_, got) in enumerate(graphs))
    assert swa.swa_device_error() == 0
