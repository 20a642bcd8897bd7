"""Plain 64-bit forms of the operators with shaped scores, of the shared-prefix
decode and of the rotated paged append, with bounds on what bf16 operands and
fp32 sums may cost (half a step of bf16 is 2^-8 relative, of fp32 2^-24)."""
import math

import torch

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
HALF_F32 = torch.finfo(torch.float32).eps / 2


def seen_keys(N, L, R, cu=None, pre=None):
    """[N, N] bool: which keys each row sees (cu: boundaries, pre: prefix lengths)."""
    i = torch.arange(N)
    band = torch.ones(N, N, dtype=torch.bool)
    back = i[:, None] - i[None, :]
    if L >= 0:
        band &= back <= L
    ahead = back >= -R if R >= 0 else torch.ones_like(band)
    if cu is None:
        return band & ahead
    seen = torch.zeros(N, N, dtype=torch.bool)
    for m, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        ok = ahead.clone()
        if pre is not None:
            p = a + min(pre[m], e - a)
            ok[a:p, a:p] = True
        seen[a:e, a:e] = (band & ok)[a:e, a:e]
    return seen


def shaped(u, cap, slope, dist):
    """Scores of the raw products u, and the derivative of the cap."""
    if cap > 0:
        t = torch.tanh(u / cap)
        s, f = cap * t, 1.0 - t * t
    else:
        s, f = u, torch.ones_like(u)
    return (s if slope is None else s - slope * dist), f


def score_error(u_abs, cap, slope, dist):
    """Bound on a score's error: the fp32 sum of u (the tensor core adds its D products
    in fp32, u_abs = scale sum |q||k| large enough for any order), the cap (its tanh is
    within 1e-6 of itself), the bias (one rounding of slope, distance and product each)
    and the change to units of log2 (two roundings); the polynomial exp2 adds 7.6e-5
    relative to P."""
    e = 130 * HALF_F32 * u_abs
    if cap > 0:
        e = e + cap * 1e-6
    if slope is not None:
        e = e + 4 * HALF_F32 * abs(slope) * dist
    return e + 4 * HALF_F32 * u_abs + 7.6e-5


def attention(q, k, v, seen, scale, cap, slope, dist, dout=None):
    """One head in 64 bits: q [n, D], k and v [m, D], seen [n, m].  Returns a dict of
    out, lse (and dq, dk, dv) with bounds e_out, ... on the library's errors."""
    q, k, v = q.double(), k.double(), v.double()
    u = q @ k.T * scale
    ua = q.abs() @ k.abs().T * scale
    s, f = shaped(u, cap, slope, dist)
    ds_err = torch.where(seen, score_error(ua, cap, slope, dist), 0.0)
    some = seen.any(1)
    x = s.masked_fill(~seen, -math.inf)
    x = torch.where(some[:, None], x, 0.0)
    lse = torch.where(some, torch.logsumexp(x, 1), -math.inf)
    p = torch.where(seen, torch.exp(x - torch.where(some, lse, 0.0)[:, None]), 0.0)
    out = p @ v
    # lse moves by at most the largest score error of the row; P relative to
    # that twice (score and sum)
    e_lse = ds_err.amax(1) + 2.0 ** -20 + 4 * HALF_F32 * torch.where(some, lse, 0.0).abs()
    rel = ds_err + e_lse[:, None]
    r = {"out": out, "lse": lse, "e_lse": e_lse}
    r["e_out"] = ((rel + HALF_BF16) * p) @ v.abs() * 1.01 + HALF_BF16 * out.abs() + 1e-30
    if dout is not None:
        do = dout.double()
        dp = do @ v.T
        delta = (do * out).sum(1, keepdim=True)
        e_delta = (do.abs() * r["e_out"]).sum(1, keepdim=True) + 130 * HALF_F32 * (
            do.abs() * out.abs()).sum(1, keepdim=True)
        e_dp = 130 * HALF_F32 * (do.abs() @ v.abs().T)
        ds = p * (dp - delta) * f
        e_f = 4e-6 if cap > 0 else 0.0
        e_ds = (rel + HALF_BF16 + 4 * HALF_F32) * ds.abs() + p * f * (e_delta + e_dp) \
            + p * (dp - delta).abs() * e_f
        r["dq"], r["dk"], r["dv"] = ds @ k * scale, ds.T @ q * scale, p.T @ do
        many = 2048 * HALF_F32
        r["e_dq"] = (e_ds @ k.abs() + many * (ds.abs() @ k.abs())) * scale * 1.02
        r["e_dk"] = (e_ds.T @ q.abs() + many * (ds.abs().T @ q.abs())) * scale * 1.02
        r["e_dv"] = (((rel + HALF_BF16) * p).T @ do.abs() + many * (p.T @ do.abs())) * 1.02
        # (rounding of the result: of dk / dv once per kv head, added by the caller)
    return r


def forward(q, k, v, L, R, cap=0.0, slopes=None, cu=None, pre=None, scale=0.0, dout=None):
    """The whole forward (and backward) [B, N, H, D] in 64 bits with bounds."""
    B, N, H, D = q.shape
    Hkv = k.shape[2]
    scale = scale if scale > 0 else 1.0 / math.sqrt(D)
    dev = q.device
    i = torch.arange(N, device=dev)
    dist = (i[:, None] - i).abs().double()

    def z(*sh):
        return torch.zeros(*sh, dtype=torch.float64, device=dev)

    got = {"out": z(B, N, H, D), "e_out": z(B, N, H, D), "lse": z(B, H, N), "e_lse": z(B, H, N)}
    if dout is not None:
        for n, heads in (("dq", H), ("dk", Hkv), ("dv", Hkv)):
            got[n], got["e_" + n] = z(B, N, heads, D), z(B, N, heads, D)
    for b in range(B):
        c = None if cu is None else [int(x) for x in cu[b]]
        pr = None if pre is None else [int(x) for x in pre[b]]
        seen = seen_keys(N, L, R, c, pr).to(dev)
        real = seen.any(1)
        for h in range(H):
            g = h // (H // Hkv)
            # padding holds nothing that counts
            t = [torch.where(real[:, None], x[b, :, hh].double(), 0.0)
                 for x, hh in ((q, h), (k, g), (v, g))]
            do = None if dout is None else torch.where(real[:, None], dout[b, :, h].double(), 0.0)
            r = attention(*t, seen, scale, cap, None if slopes is None else float(slopes[h]), dist,
                          do)
            for n in ("out", "e_out"):
                got[n][b, :, h] = r[n]
            for n in ("lse", "e_lse"):
                got[n][b, h] = r[n]
            if dout is not None:
                got["dq"][b, :, h], got["e_dq"][b, :, h] = r["dq"], r["e_dq"]
                for n in ("dk", "e_dk", "dv", "e_dv"):
                    got[n][b, :, g] += r[n]
    if dout is not None:
        for n in ("dq", "dk", "dv"):
            got["e_" + n] += HALF_BF16 * (got[n].abs() + got["e_" + n]) + 1e-30
    return got


def check(got, ref, names, what=""):
    """Every element of got[name] within ref's bound; the infinities of lse alike."""
    for n in names:
        g, r, e = got[n].double(), ref[n], ref["e_" + n]
        inf = torch.isinf(r)
        assert torch.equal(g[inf], r[inf]), f"{what} {n}: infinities differ"
        d = (g - r)[~inf].abs()
        assert torch.isfinite(d).all(), f"{what} {n}: non-finite values"
        over = d - e[~inf]
        worst = float(over.max()) if over.numel() else 0.0
        assert worst <= 0, f"{what} {n}: past its bound by {worst:.3e} (error {float(d.max()):.3e})"


def rotate(x, pos, inv_freq, interleaved):
    """x [n, heads, D] at positions [n], rotated in 64 bits."""
    x = x.double()
    rot = 2 * inv_freq.shape[0]
    a = pos.double()[:, None] * inv_freq.double()
    c, s = a.cos()[:, None], a.sin()[:, None]
    y = x.clone()
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def rotate_error(x, y, inv_freq, interleaved):
    """Bound on a rotated element: its rounding to bf16, and sin / cos and the products
    in fp32 (the reduced angle is off by half a step of at most one turn, 2^-24 * pi)."""
    x = x.double().abs()
    rot = 2 * inv_freq.shape[0]
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    e = torch.zeros_like(x)
    e[..., first] = e[..., second] = (x[..., first] + x[..., second]) * (2.0 ** -21)
    return (HALF_BF16 * (y.abs() + e) + e) * torch.cat(
        (torch.ones(rot), torch.zeros(x.shape[-1] - rot))).to(x)
