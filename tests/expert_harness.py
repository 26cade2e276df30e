"""Ragged layouts, 64-bit values and error bounds for the expert operators'
tests. Everything here is computed from the definitions, in float64, without
the library."""
from __future__ import annotations

import torch

HALF_BF16 = 2.0 ** -8   # half a step of BF16, relative
FP32_STEP = 2.0 ** -23  # one truncated FP32 operation, relative


def ragged(counts, alpha, tail=0):
    """(ends, num_rows, [(start, end)]) of groups with these counts."""
    at, ends, spans = 0, [], []
    for c in counts:
        at = -(-at // alpha) * alpha
        spans.append((at, at + c))
        at += c
        ends.append(at)
    return ends, at + tail, spans


def product(x, w, spans, x_scale=None, w_scale=None):
    """(sum, sum of magnitudes) of every row against its group's weight,
    float64 on x's device; rows outside the spans are NaN."""
    R, K = x.shape
    y = torch.full((R, w.shape[1]), float("nan"), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    for g, (a, b) in enumerate(spans):
        if b <= a:
            continue
        xd, wd = x[a:b].double(), w[g].double()
        if x_scale is not None:
            xd = xd * x_scale[a:b].double().repeat_interleave(128, 1)
            wd = wd * w_scale[g].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        y[a:b] = xd @ wd.t()
        mag[a:b] = xd.abs() @ wd.abs().t()
    return y, mag


def product_error(mag, K):
    """Bound on an FP32 sum of K products (each add truncated at worst, every
    partial sum at most `mag`), plus four scalings."""
    return (K + 4) * FP32_STEP * mag


def silu(g):
    return g * torch.sigmoid(g)


def gated(y, mag, K):
    """(value, error bound before rounding) of silu(gate) * up for sums with
    product_error: |silu'| <= 1.1, and 2^-18 relative for exp, the division
    and the products."""
    g, u = y.chunk(2, 1)
    eg, eu = product_error(mag, K).chunk(2, 1)
    v = silu(g) * u
    err = 1.1 * eg * (u.abs() + eu) + silu(g).abs() * eu + 2.0 ** -18 * v.abs()
    return v, err


def check_bf16(got, want, err, rows):
    """got (BF16) within the error bound and half a step of want, on rows."""
    g, w, e = got.double()[rows], want[rows], err[rows]
    off = (g - w).abs()
    tol = e + HALF_BF16 * (w.abs() + e) + 1e-36
    bad = ~(off <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} values off; worst "
                           f"{(off / tol)[bad].max().item():.3g} of the bound at {bad.nonzero()[0].tolist()}")


def live_rows(R, spans, device="cpu"):
    m = torch.zeros(R, dtype=torch.bool, device=device)
    for a, b in spans:
        m[a:b] = True
    return m


def quantise_rows(v):
    """E4M3 values and FP32 scales of blocks of 128 columns."""
    b = v.view(v.shape[0], -1, 128)
    s = b.abs().amax(-1).clamp_min(1e-30) / 448.0
    return (b / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(v.shape), s


def quantise_weight(v):
    G, N, K = v.shape
    b = v.view(G, N // 128, 128, K // 128, 128)
    s = b.abs().amax(dim=(2, 4)).clamp_min(1e-30) / 448.0
    return (b / s[:, :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(G, N, K), s


def route_reference(logits, top_k, scoring="softmax", bias=None, renormalize=True, scale=1.0):
    """(ids, weights float64) from the definition, token by token."""
    ids, ws = [], []
    for row in logits.double().tolist():
        n = len(row)
        b = bias.double().tolist() if bias is not None else [0.0] * n
        ok = [e for e in range(n) if row[e] == row[e] and row[e] != float("-inf")
              and b[e] == b[e] and b[e] != float("-inf")]
        big = float(torch.finfo(torch.float32).max)
        l = torch.tensor([min(row[e], big) for e in ok], dtype=torch.float64)
        log_s = torch.log_softmax(l, 0) if scoring == "softmax" else torch.nn.functional.logsigmoid(l)
        s = log_s.exp().tolist()
        key = [s[i] + b[e] if bias is not None else min(row[e], big) for i, e in enumerate(ok)]
        order = sorted(range(len(ok)), key=lambda i: (-key[i], ok[i]))[:top_k]
        # s / sum of the selected s, whatever both underflow to
        w = torch.softmax(log_s[order], 0).tolist() if renormalize else [s[i] for i in order]
        pad = top_k - len(order)
        ids.append([ok[i] for i in order] + [-1] * pad)
        ws.append([scale * v for v in w] + [0.0] * pad)
    T = logits.shape[0]
    return (torch.tensor(ids, dtype=torch.int64).view(T, top_k),
            torch.tensor(ws, dtype=torch.float64).view(T, top_k))
