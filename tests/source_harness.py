"""64-bit values and error bounds for the source-side operators' tests.
Everything here is computed from the definitions, in float64, without the
library."""
from __future__ import annotations

import torch

E4M3_HALF = 2.0 ** -4    # half a step of E4M3, relative ...
E4M3_TINY = 2.0 ** -10   # ... and below its smallest normal number, absolute
FP32_HALF = 2.0 ** -24
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
SMALLEST_SCALE = 2.0 ** -100


# ------------------------------------------------------------------- E4M3
def check_e4m3(q, scale, want, err):
    """E4M3 vectors (last dimension) with FP32 scales against float64 values
    that are known to +- err: the scale is the largest magnitude / 448 (its own
    rounding: one division), every value within half a step of want / scale."""
    big = want.abs().amax(-1)
    slack = err.amax(-1) / 448
    s = scale.double()
    s_want = (big / 448).clamp_min(SMALLEST_SCALE)
    off = (s - s_want).abs()
    assert (off <= slack + 2 * FP32_HALF * s_want).all(), f"scales off by {(off / s_want).max().item():.3g}"
    # The reciprocal and the product with it: 2^-23 of the quotient. At the top,
    # values up to the slack above 448 scales round to 448.
    v = q.double() * s[..., None]
    tol = E4M3_HALF * (want.abs() + err) + E4M3_TINY * s[..., None] + err + 4 * FP32_HALF * want.abs()
    bad = ~((v - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values off, first at {bad.nonzero()[0].tolist()}"


# -------------------------------------------------------------------- norm
def norm(x, residual, weight, eps, terms):
    """(r, y, error of y before rounding) in float64. `terms`: values that one
    thread sums one after another; five shuffles twice and a division follow, the
    root takes half of the sum's error, the reciprocal root is good to 2^-22 and
    r and the two products round three times."""
    r = x.double() if residual is None else x.double() + residual.double()
    y = r * (r.square().mean(-1, keepdim=True) + eps).rsqrt() * weight.double()
    err = (((terms + 16) / 2 + 4) + 4 + 3) * FP32_HALF * y.abs()
    return r, y, err


# ------------------------------------------------------------------ rotary
def rotate(x, positions, inv_freq, interleaved, factor):
    """(value, error before rounding) of [T, heads, D] in float64. The angle's
    remainder (at most pi) rounds to FP32 with 2^-23, sine and cosine err by two
    steps (2^-23), the factor and the rotation round three times."""
    x = x.double()
    R = 0 if inv_freq is None else inv_freq.numel()
    if not R:
        return x, torch.zeros_like(x)
    angle = positions.double()[:, None, None] * inv_freq.double()
    cos, sin = angle.cos() * factor, angle.sin() * factor
    at = torch.arange(R, device=x.device)
    i, j = (2 * at, 2 * at + 1) if interleaved else (at, at + R)
    a, b = x[..., i], x[..., j]
    y, err = x.clone(), torch.zeros_like(x)
    y[..., i], y[..., j] = a * cos - b * sin, b * cos + a * sin
    err[..., i] = err[..., j] = (a.abs() + b.abs()) * abs(factor) * (2.0 ** -22 + 4 * FP32_HALF)
    return y, err


# --------------------------------------------------------------- attention
def attention(q, k_cache, v_cache, table, lengths, scale, window=0, k_scale=None, v_scale=None):
    """(out, lse, error of out before rounding, error of lse), float64,
    sequence by sequence and head by head.

    Scores: FP32 sums of D products (each addition truncated at worst) and four
    roundings. Their error e moves a probability by e (relative), twice with the
    sum; exponentials err by 2^-21 with their arguments' rounding (2^-23 of the
    score's distance from the maximum, at most a few hundred where the result
    counts). Probabilities: two BF16 parts (2^-16), or FP16 (2^-11, and 2^-25 of
    the largest contribution). Sums over n tokens: n truncated additions."""
    B, Hq, D = q.shape
    pages, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    fp8 = k_scale is not None
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    err = torch.zeros_like(out)
    lse = torch.full((B, Hq), float("-inf"), dtype=torch.float64, device=q.device)
    lse_err = torch.zeros_like(lse)
    for b, n in enumerate(lengths.tolist()):
        n = min(max(n, 0), table.shape[1] * page)
        at = torch.arange(max(n - window, 0) if window else 0, n, device=q.device)
        where = table[b].long()[at // page]
        ok = (where >= 0) & (where < pages)
        at, where = at[ok], where[ok]
        if not len(at):
            continue
        for h in range(Hkv):
            k, v = k_cache[where, h, at % page].double(), v_cache[where, h, at % page].double()
            if fp8:
                ks, vs = k_scale[where, h, at % page].double(), v_scale[where, h, at % page].double()
                k, v = k * ks[:, None], v * vs[:, None]
            mine = slice(h * G, (h + 1) * G)
            qd = q[b, mine].double()
            s = scale * (qd @ k.t())
            e = (D + 8) * 2 * FP32_HALF * abs(scale) * (qd.abs() @ k.abs().t())
            if fp8:  # queries in FP16, 2^-25 of the row's largest
                e = e + 2.0 ** -25 * abs(scale) * qd.abs().amax(-1, keepdim=True) * k.abs().sum(-1)
            top = s.amax(-1, keepdim=True)
            e = (e + 2.0 ** -23 * ((s - top).abs().clamp_max(200) + s.abs()) + 2.0 ** -21).amax(-1, keepdim=True)
            p = torch.softmax(s, -1)
            mag = p @ v.abs()
            m = len(at)
            rel = 2 * e + (m + 64) * 2 * FP32_HALF + (2.0 ** -11 if fp8 else 2.0 ** -16)
            out[b, mine] = p @ v
            err[b, mine] = rel * mag
            if fp8:
                most = (p * vs).amax(-1, keepdim=True)
                err[b, mine] += 2.0 ** -24 * most * (v.abs() / vs.clamp_min(1e-300)[:, None]).sum(0)
            lse[b, mine] = torch.logsumexp(s, -1)
            lse_err[b, mine] = (e + (m + 64) * 2 * FP32_HALF).squeeze(-1) + 2.0 ** -22 * lse[b, mine].abs()
    return out, lse, err, lse_err


def check_lse(got, want, err):
    none = want == float("-inf")
    assert torch.equal(got == float("-inf"), none)
    off = (got.double() - want).abs()[~none]
    assert (off <= err[~none] + FP32_HALF * want[~none].abs() + 1e-30).all(), off.max().item()


def paged(lengths, page, Hkv, D, fp8, generator, width=None, spare=2, spoil=True):
    """A cache whose sequences lie on shuffled pages: (k, v, k_scale, v_scale,
    table, lengths). What no sequence owns is NaN, table entries behind a
    sequence's pages are numbers of no page."""
    dev = generator.device
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    width = max(need + [0]) + 1 if width is None else width
    ids = torch.randperm(pages, generator=generator, device=dev).int()
    table = torch.full((len(lengths), width), 0x7fffffff, dtype=torch.int32, device=dev)
    table[:, ::2] = -1
    at = 0
    owned = torch.zeros(pages, page, dtype=torch.bool, device=dev)
    for b, n in enumerate(lengths):
        table[b, :need[b]] = ids[at:at + need[b]]
        for i in range(need[b]):
            owned[ids[at + i].long(), :min(page, n - i * page)] = True
        at += need[b]
    got = []
    for _ in range(2):
        x = torch.randn(pages, Hkv, page, D, generator=generator, device=dev)
        dead = ~owned[:, None, :].expand(pages, Hkv, page)
        if fp8:
            scale = torch.rand(pages, Hkv, page, generator=generator, device=dev) * 0.02 + 0.002
            x = (x * 100).clamp(-448, 448).to(FP8)
            if spoil:
                x.view(torch.uint8)[dead] = 0x7F
                scale[dead] = float("nan")
        else:
            x, scale = x.to(BF16), None
            if spoil:
                x[dead] = float("nan")
        got.append((x, scale))
    (k, ks), (v, vs) = got
    return k, v, ks, vs, table, torch.tensor(lengths, dtype=torch.int32, device=dev)
