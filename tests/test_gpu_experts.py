"""The expert operators (afd_route_topk, afd_grouped_linear, afd_gated_rows,
afd_adapter_add) against float64 values from their definitions, at the sizes
and masks where they can go wrong, and their refusals that need a GPU."""
import math
import os
import subprocess
import sys

import pytest
import torch

import combine_attention_ffn_gb300 as lib
import expert_harness as eh
from combine_attention_ffn_gb300 import afd

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_attention_ffn_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------ grouped product
COUNTS = {
    "one-row": [0, 1, 0],
    "empty": [0, 0, 0, 0],
    "small": [3, 0, 8, 9, 16, 17, 1, 0],
    "tile-edges": [255, 256, 257, 0, 127, 128, 129, 1],
    "one-large": [0, 700, 2],
    "many": [(7 * i * i) % 23 for i in range(130)],
}


def _grouped_case(counts, alpha, K, N, gated, fp8, seed, tail=5):
    g = _gen(seed)
    ends, R, spans = eh.ragged(counts, alpha, tail)
    W = 2 * N if gated else N
    x = torch.randn(max(R, 1), K, generator=g, device="cuda")
    w = torch.randn(len(counts), W, K, generator=g, device="cuda") * K ** -0.5
    xs = ws = None
    if fp8:
        x, xs = eh.quantise_rows(x)
        w, ws = eh.quantise_weight(w)
    else:
        x, w = x.to(BF16), w.to(BF16)
    # what lies outside every expert's range must neither be used nor written
    dead = ~eh.live_rows(x.shape[0], spans, "cuda")
    if fp8:
        x.view(torch.uint8)[dead] = 0x7F
        xs[dead] = float("nan")
    else:
        x[dead] = float("nan")
    return x, xs, w, ws, torch.tensor(ends, dtype=torch.int32, device="cuda"), spans, dead


def _grouped_check(x, xs, w, ws, ends, spans, dead, alpha, gated, **kw):
    R, K = x.shape
    N = w.shape[1] // 2 if gated else w.shape[1]
    out = torch.full((R, N), 7.0, dtype=BF16, device="cuda")
    error = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.grouped_linear(x, w, ends, expert_alignment=alpha, gated=gated, x_scale=xs, weight_scale=ws,
                             out=out, error=error, **kw)
    assert got is out
    y, mag = eh.product(x, w, spans, xs, ws)
    want, err = eh.gated(y, mag, K) if gated else (y, eh.product_error(mag, K))
    eh.check_bf16(out, want, err, ~dead)
    assert (out[dead] == 7.0).all()
    assert error.item() == 0
    return out


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", sorted(COUNTS))
def test_grouped_bf16_counts(name, gated):
    case = _grouped_case(COUNTS[name], 128 if name != "many" else 1, 192, 320, gated, False, 11)
    _grouped_check(*case, 128 if name != "many" else 1, gated)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K,N", [(8, 8), (8, 1), (64, 7), (72, 129), (2048, 256), (200, 1000), (1000, 65)])
def test_grouped_bf16_sizes(K, N, gated):
    case = _grouped_case([5, 0, 131, 16], 1, K, N, gated, False, K * 7 + N)
    _grouped_check(*case, 1, gated)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", sorted(COUNTS))
def test_grouped_fp8_counts(name, gated):
    case = _grouped_case(COUNTS[name], 16, 256, 384, gated, True, 12)
    _grouped_check(*case, 16, gated)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K,N", [(128, 128), (128, 256), (1152, 128), (2048, 640)])
def test_grouped_fp8_sizes(K, N, gated):
    case = _grouped_case([5, 0, 131, 16], 1, K, N, gated, True, K + N)
    _grouped_check(*case, 1, gated)


def test_grouped_most_experts():
    counts = [(i * 5) % 4 for i in range(1024)]
    _grouped_check(*_grouped_case(counts, 1, 64, 64, False, False, 3), 1, False)


@pytest.mark.parametrize("gated", [False, True])
def test_grouped_more_tiles_than_are_listed(gated):
    """Over 100 tiles for every pair of CTAs, of several widths."""
    counts = [(i * 7) % 5 + (90 if i % 50 == 0 else 0) for i in range(1024)]
    _grouped_check(*_grouped_case(counts, 1, 64, 2048 // (1 + gated), gated, False, 4), 1, gated)


@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_strided_rows(fp8):
    """x and out are columns of wider buffers."""
    x, xs, w, ws, ends, spans, dead = _grouped_case([3, 200, 0, 40], 64, 256, 128, True, fp8, 5)
    wide = torch.zeros(x.shape[0], 3 * 256, dtype=BF16, device="cuda")
    wide = wide.to(x.dtype) if not fp8 else torch.zeros(x.shape[0], 768, dtype=torch.uint8, device="cuda").view(FP8)
    wide[:, 256:512] = x
    outs = torch.full((x.shape[0], 131), 3.0, dtype=BF16, device="cuda")
    lib.grouped_linear(wide[:, 256:512], w, ends, expert_alignment=64, gated=True, x_scale=xs, weight_scale=ws,
                       out=outs[:, 2:130])
    plain = lib.grouped_linear(x, w, ends, expert_alignment=64, gated=True, x_scale=xs, weight_scale=ws)
    assert torch.equal(outs[:, 2:130][~dead], plain[~dead])
    assert (outs[:, :2] == 3.0).all() and (outs[:, 130:] == 3.0).all()


def test_grouped_offsets_past_32_bits():
    """Rows and weights whose byte offsets pass 32 bits (x of 4.3 GB, weights of 4.5 GB)."""
    alpha, K, N, G, far = 1 << 20, 2048, 2048, 540, 531
    counts = [0] * G
    counts[0], counts[far] = 3, 21
    ends, R, spans = eh.ragged(counts[:far + 1], alpha)
    ends += [R] * (G - far - 1)  # the last groups are empty
    x = torch.zeros(R, K, dtype=BF16, device="cuda")
    x[R - 21:] = torch.randn(21, K, generator=_gen(1), device="cuda").to(BF16)
    x[:3] = x[R - 3:]
    w = torch.zeros(G, N, K, dtype=BF16, device="cuda")
    for g in (0, far):
        w[g] = (torch.randn(N, K, generator=_gen(2 + g), device="cuda") * K ** -0.5).to(BF16)
    out = torch.zeros(R, N, dtype=BF16, device="cuda")
    lib.grouped_linear(x, w, torch.tensor(ends, dtype=torch.int32, device="cuda"), expert_alignment=alpha, out=out)
    for g, (a, b) in ((0, spans[0]), (far, spans[far])):
        y, mag = eh.product(x[a:b], w[g:g + 1], [(0, b - a)])
        eh.check_bf16(out[a:b], y, eh.product_error(mag, K), torch.ones(b - a, dtype=torch.bool, device="cuda"))
    assert (out[3:R - 21] == 0).all()


def test_grouped_bad_ends_stay_inside_the_buffers():
    """Ends beyond num_rows count as num_rows; negative ones as empty groups."""
    x, xs, w, ws, ends, spans, dead = _grouped_case([4, 4, 4], 1, 64, 32, False, False, 8, tail=0)
    ends = torch.tensor([-5, 6, 1 << 30], dtype=torch.int32, device="cuda")
    out = torch.full((12, 32), 7.0, dtype=BF16, device="cuda")
    lib.grouped_linear(x, w, ends, out=out)
    y, mag = eh.product(x, w, [(0, 0), (0, 6), (6, 12)])
    eh.check_bf16(out, y, eh.product_error(mag, 64), torch.ones(12, dtype=torch.bool, device="cuda"))


def test_grouped_infinities_stay_in_their_row():
    case = _grouped_case([9, 20], 1, 64, 64, False, False, 9)
    x, _, w, _, ends, spans, dead = case
    clean = lib.grouped_linear(x, w, ends)
    x[4, 3], x[12, 5], x[13, 0] = float("inf"), float("nan"), float("-inf")
    out = lib.grouped_linear(x, w, ends)
    hit = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    hit[[4, 12, 13]] = True
    assert torch.equal(out[~hit & ~dead], clean[~hit & ~dead])
    assert not torch.isfinite(out[hit]).any()


@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_repeats_bit_for_bit_on_other_streams_and_in_graphs(fp8):
    """The same call twice, on two streams at once, and replayed from two
    graphs at once with new inputs gives the same bits."""
    case = _grouped_case([40, 300, 0, 7, 513], 16, 512, 384, True, fp8, 21, tail=90)
    x, xs, w, ws, ends, spans, dead = case
    call = lambda out: lib.grouped_linear(x, w, ends, expert_alignment=16, gated=True, x_scale=xs,
                                          weight_scale=ws, out=out)
    first = _grouped_check(*case, 16, True)
    outs = [torch.zeros_like(first) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):
        with torch.cuda.stream(s):
            call(o)
    graphs = []
    torch.cuda.synchronize()
    for o in outs[2:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(o)
        graphs.append(g)
    for o in outs[2:]:
        o.zero_()
    torch.cuda.synchronize()
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[~dead], first[~dead])
    # new routing and rows under the captured call
    counts = [1, 0, 400, 500, 20]
    x2, xs2, _, _, ends2, spans2, _ = _grouped_case(counts, 16, 512, 384, True, fp8, 22)
    n = min(x.shape[0], x2.shape[0])
    assert ends2.max() <= x.shape[0]
    x.view(torch.uint8).zero_()
    x[:n] = x2[:n]
    if fp8:
        xs.fill_(1.0)
        xs[:n] = xs2[:n]
    ends.copy_(ends2)
    graphs[0].replay()
    torch.cuda.synchronize()
    y, mag = eh.product(x, w, spans2, xs, ws)
    want, err = eh.gated(y, mag, 512)
    eh.check_bf16(outs[2], want, err, eh.live_rows(x.shape[0], spans2, "cuda"))


# ------------------------------------------------------------- gated rows
@pytest.mark.parametrize("N", [1, 8, 100, 257, 1024])
@pytest.mark.parametrize("name", ["empty", "small", "many"])
def test_gated_rows(name, N):
    ends, R, spans = eh.ragged(COUNTS[name], 16, 3)
    h = (torch.randn(R, 2 * N, generator=_gen(N), device="cuda") * 3).to(BF16)
    ends = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out = torch.full((R, N), 7.0, dtype=BF16, device="cuda")
    lib.gated_rows(h, ends, expert_alignment=16, out=out)
    live = eh.live_rows(R, spans, "cuda")
    g, u = h.double().chunk(2, 1)
    v = eh.silu(g) * u
    eh.check_bf16(out, v, 2.0 ** -18 * v.abs(), live)
    assert (out[~live] == 7.0).all()
    # in place, into the first half
    lib.gated_rows(h, ends, expert_alignment=16, out=h[:, :N])
    assert torch.equal(h[:, :N][live], out[live])
    assert torch.equal(h[:, :N].double()[~live], g[~live])


def test_gated_rows_extremes():
    h = torch.tensor([[-1e4, 200.0, float("inf"), 0.0, 2.0, 2.0, 2.0, float("inf")],
                      [float("nan"), 1.0, -90.0, 3e38, 1.0, float("-inf"), 3e38, 3e38]], device="cuda").to(BF16)
    ends = torch.tensor([2], dtype=torch.int32, device="cuda")
    out = lib.gated_rows(h, ends)
    g, u = h.float().chunk(2, 1)
    want = (g * torch.sigmoid(g) * u).to(BF16)
    want[1, 2] = out[1, 2]  # silu(-90) is around the smallest normal number: checked below
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    ok = ~torch.isnan(want)
    inf = torch.isinf(want)
    assert torch.equal(out[inf], want[inf])
    assert torch.allclose(out[ok & ~inf].float(), want[ok & ~inf].float(), rtol=2 ** -7, atol=1e-30)
    assert abs(out[1, 2].item()) <= 3e38 * 90 * math.exp(-90) * (1 + 2 ** -7)


# --------------------------------------------------------------- adapters
def _adapter_case(R, K, N, rank, S, seed, tokens):
    g = _gen(seed)
    x = torch.randn(R, K, generator=g, device="cuda").to(BF16)
    base = torch.randn(R, N, generator=g, device="cuda").to(BF16)
    down = (torch.randn(S, rank, K, generator=g, device="cuda") * K ** -0.5).to(BF16)
    up = (torch.randn(S, N, rank, generator=g, device="cuda") * rank ** -0.5).to(BF16)
    scales = torch.rand(S, generator=g, device="cuda") + 0.5
    slots = torch.randint(-1, S + 1, (tokens,), generator=g, device="cuda").int()
    return x, base, down, up, scales, slots


def _adapter_want(base, x, down, up, scales, slot):
    """(value, error bound): slot [R] int64 per row, outside [0, S) none. The
    down sums err as FP32 sums of K products; they enter the up product with
    at least 16 bits (2^-16 relative)."""
    S, rank, K = down.shape
    want, err = base.double(), torch.zeros(base.shape, dtype=torch.float64, device=base.device)
    for a in range(S):
        rows = (slot == a).nonzero()[:, 0]
        if not len(rows):
            continue
        d, u, sc = down[a].double(), up[a].double(), scales[a].double()
        t = x[rows].double() @ d.t()
        et = K * eh.FP32_STEP * (x[rows].double().abs() @ d.abs().t()) + 2.0 ** -16 * t.abs()
        want[rows] += sc * (t @ u.t())
        err[rows] = sc * (et @ u.abs().t()) + (2 * rank + 4) * eh.FP32_STEP * (
            sc * (t.abs() @ u.abs().t()) + base[rows].double().abs())
    return want, err


@pytest.mark.parametrize("rank", [8, 16, 32, 64])
@pytest.mark.parametrize("R,K,N", [(1, 16, 8), (2, 256, 24), (17, 2048, 264), (33, 48, 1000), (300, 1040, 512),
                                   (513, 16, 8), (600, 2048, 264), (700, 1040, 1000)])  # (from 513 on not a row at a time)
def test_adapters_of_own_tokens(R, K, N, rank):
    x, base, down, up, scales, slots = _adapter_case(R, K, N, rank, 5, R + rank, R)
    want, err = _adapter_want(base, x, down, up, scales, slots.long())
    out = lib.adapter_add(base, x, down, up, slots, scales, out=torch.empty_like(base))
    every = torch.ones(R, dtype=torch.bool, device="cuda")
    eh.check_bf16(out, want, err, every)
    none = (slots < 0) | (slots >= 5)
    assert torch.equal(out[none], base[none])
    again = base.clone()
    assert lib.adapter_add(again, x, down, up, slots, scales) is again
    assert torch.equal(again, out)


@pytest.mark.parametrize("rank", [8, 16, 32, 64])
@pytest.mark.parametrize("R,K,N", [(1, 128, 8), (17, 2048, 264), (300, 1152, 512), (513, 128, 8), (700, 2048, 264)])
def test_adapters_of_fp8_rows(R, K, N, rank):
    _, base, down, up, scales, slots = _adapter_case(R, K, N, rank, 5, R + rank, R)
    q, qs = eh.quantise_rows(torch.randn(R, K, generator=_gen(R), device="cuda"))
    x = q.double() * qs.double().repeat_interleave(128, 1)
    dead = slots < 0
    q.view(torch.uint8)[dead], qs[dead] = 0x7F, float("nan")  # rows without an adapter are not read
    x[dead] = 0
    want, err = _adapter_want(base, x, down, up, scales, slots.long())
    wide = torch.zeros(R, 2 * K, dtype=torch.uint8, device="cuda").view(FP8)
    wide[:, K:] = q
    for rows in (q, wide[:, K:]):
        out = lib.adapter_add(base, rows, down, up, slots, scales, x_scale=qs, out=torch.empty_like(base))
        eh.check_bf16(out, want, err, torch.ones(R, dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("run", [1, 40])
@pytest.mark.parametrize("alpha", [1, 16])
@pytest.mark.parametrize("counts", [(30, 0, 1, 70, 5, 16), (300, 0, 1, 270, 5, 16)])
def test_adapters_of_received_rows(counts, alpha, run):
    """Rows in an exchange's order: padding (row_src -1), a row_src that names
    no token, and rows behind the last end stay as they were."""
    K, N, rank, S, top_k, tokens = 128, 136, 16, 6, 3, sum(counts) // 2 + 9
    ends, R, spans = eh.ragged(list(counts), alpha, 9)
    x, base, down, up, scales, _ = _adapter_case(R, K, N, rank, S, 4, tokens)
    slots = (torch.arange(tokens, device="cuda") // run * 7 % (S + 2) - 1).int()
    live = eh.live_rows(R, spans, "cuda")
    src = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    src[live] = (torch.randperm(tokens * top_k, generator=_gen(9), device="cuda")[: int(live.sum())]).int().sort().values
    src[ends[-1]:] = 5                       # stale
    src[3] = tokens * top_k                  # names no token
    live[3] = False
    x[~live] = float("nan")
    out = torch.full_like(base, 7.0)
    lib.adapter_add(base, x, down, up, slots, scales, row_src=src, top_k=top_k, out=out,
                    ends=torch.tensor(ends, dtype=torch.int32, device="cuda"))
    slot = slots[(src.long().clamp_min(0) // top_k).clamp_max(tokens - 1)].long()
    slot[~live] = -1
    want, err = _adapter_want(base, x, down, up, scales, slot)
    eh.check_bf16(out, want, err, live)
    assert (out[~live] == 7.0).all()


@pytest.mark.parametrize("rank", [8, 64])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("tokens", [1, 4, 8, 60])
def test_adapters_few_rows_of_a_long_layout(tokens, in_place, rank):
    """A decode step in a padded layout: few live rows, far apart."""
    K, N, S, top_k, groups, alpha = 144, 264, 3, 8, 300, 128
    g = _gen(tokens + rank)
    routes = torch.randint(0, groups, (tokens * top_k,), generator=g, device="cuda").sort().values
    counts = torch.bincount(routes, minlength=groups).tolist()
    ends, R, spans = eh.ragged(counts, alpha, 9)
    x, base, down, up, scales, slots = _adapter_case(R, K, N, rank, S, 4, tokens)
    live = eh.live_rows(R, spans, "cuda")
    src = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    src[live] = torch.randperm(tokens * top_k, generator=g, device="cuda").int()
    x[~live] = float("nan")
    slot = slots[src.long().clamp_min(0) // top_k].long()
    slot[~live] = -1
    want, err = _adapter_want(base, x, down, up, scales, slot)
    before = base.clone()
    out = base if in_place else torch.full_like(base, 7.0)
    lib.adapter_add(base, x, down, up, slots, scales, row_src=src, top_k=top_k, out=out,
                    ends=torch.tensor(ends, dtype=torch.int32, device="cuda"))
    eh.check_bf16(out, want, err, live)
    assert torch.equal(out[~live], before[~live]) if in_place else (out[~live] == 7.0).all()


@pytest.mark.parametrize("R", [90, 690])
def test_adapters_strided_and_captured(R):
    K, N, rank, S = 256, 128, 32, 3
    x, base, down, up, scales, slots = _adapter_case(R, K, N, rank, S, 6, R)
    want = lib.adapter_add(base, x, down, up, slots, scales, out=torch.empty_like(base))
    xw = torch.full((R, 3 * K), float("nan"), dtype=BF16, device="cuda")
    xw[:, K:2 * K] = x
    bw = torch.full((R, N + 16), 5.0, dtype=BF16, device="cuda")
    bw[:, 8:8 + N] = base
    lib.adapter_add(bw[:, 8:8 + N], xw[:, K:2 * K], down, up, slots, scales)
    assert torch.equal(bw[:, 8:8 + N], want) and (bw[:, :8] == 5).all() and (bw[:, 8 + N:] == 5).all()
    out = torch.zeros_like(base)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.adapter_add(base, x, down, up, slots, scales, out=out)
    out.zero_()
    slots.copy_((slots + 2) % 4 - 1)
    g.replay()
    torch.cuda.synchronize()
    want, err = _adapter_want(base, x, down, up, scales, slots.long())
    eh.check_bf16(out, want, err, torch.ones(R, dtype=torch.bool, device="cuda"))


def test_adapters_many_rows():
    """More rows than the grouping keeps in registers, and uneven groups."""
    R, K, N, rank, S = 40_000, 32, 24, 8, 300
    x, base, down, up, scales, slots = _adapter_case(R, K, N, rank, S, 7, R)
    slots[: R // 2] = 3
    out = lib.adapter_add(base, x, down, up, slots, scales, out=torch.empty_like(base))
    s = slots.long()
    ok = (s >= 0) & (s < S)
    d, u = down.double()[s.clamp(0, S - 1)], up.double()[s.clamp(0, S - 1)]
    t = torch.einsum("rk,rjk->rj", x.double(), d)
    sc = torch.where(ok, scales.double()[s.clamp(0, S - 1)], 0.0)[:, None]
    want = base.double() + sc * torch.einsum("rj,rnj->rn", t, u)
    et = K * eh.FP32_STEP * torch.einsum("rk,rjk->rj", x.double().abs(), d.abs()) + 2.0 ** -16 * t.abs()
    err = sc * torch.einsum("rj,rnj->rn", et, u.abs()) + (2 * rank + 4) * eh.FP32_STEP * (want.abs() + base.double().abs() + sc * (
        t.abs()[:, None, :] * u.abs()).sum(-1))
    eh.check_bf16(out, want, err, torch.ones(R, dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("R", [70, 670])
def test_adapters_keep_requests_apart(R):
    """An adapter full of infinities and NaN reaches its own rows only; so do rows of NaN."""
    K, N, rank, S = 64, 40, 16, 4
    x, base, down, up, scales, _ = _adapter_case(R, K, N, rank, S, 8, R)
    slots = (torch.arange(R, device="cuda") % 4).int()
    clean = lib.adapter_add(base, x, down, up, slots, scales, out=torch.empty_like(base))
    down[2], up[1] = float("inf"), float("nan")
    x[3] = float("nan")
    out = lib.adapter_add(base, x, down, up, slots, scales, out=torch.empty_like(base))
    own = (slots == 1) | (slots == 2)
    own[3] = True
    assert torch.equal(out[~own], clean[~own])
    assert not torch.isfinite(out[own]).any()


@pytest.mark.parametrize("R", [500, 1500])
def test_adapters_two_streams_at_once(R):
    K, N, rank, S = 512, 256, 32, 6
    a, b = (_adapter_case(R, K, N, rank, S, seed, R) for seed in (1, 2))
    call = lambda c, **kw: lib.adapter_add(c[1], c[0], c[2], c[3], c[5], c[4], out=torch.empty_like(c[1]), **kw)
    want = [call(a), call(b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[call(c, stream=s) for _ in range(20)] for c, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


# ------------------------------------------------------------------ router
def _route_check(logits, top_k, **kw):
    ids, w = lib.route_topk(logits, top_k, **kw)
    want_ids, want_w = eh.route_reference(logits.cpu(), top_k, **{
        k: (v.cpu() if isinstance(v, torch.Tensor) else v) for k, v in kw.items()})
    assert torch.equal(ids.cpu(), want_ids)
    # exp (2 units), a sum over the experts, a quotient and two products: 2^-17 relative;
    # scores below the normal range are flushed or lose digits
    assert ((w.double().cpu() - want_w).abs() <= 2.0 ** -17 * want_w.abs() + 1e-36).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 8, 8), (5, 33, 4), (64, 128, 8), (9, 200, 10), (7, 1024, 32), (130, 96, 8)])
def test_router(T, E, K, with_bias, scoring):
    for dtype in (torch.float32, BF16):
        logits = (torch.randn(T, E, generator=_gen(T * E + K), device="cuda") * 2).to(dtype)
        bias = torch.randn(E, generator=_gen(5), device="cuda") * 0.1 if with_bias else None
        _route_check(logits, K, scoring=scoring, bias=bias)
        _route_check(logits, K, scoring=scoring, bias=bias, renormalize=False, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_router_ties_and_masks(scoring):
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(torch.float32).min
    rows = [[0.0] * 40,
            [1.0, -0.0, 0.0, 1.0] * 10,
            [-inf] * 40,
            [nan] * 39 + [1.0],
            [-inf] * 37 + [3.0, nan, 2.0],
            [low] * 40,
            [low] * 20 + [1.0] * 2 + [low] * 18,
            [inf, 1.0, inf] + [0.0] * 37,
            [-200.0] * 40]
    logits = torch.tensor(rows, device="cuda")
    _route_check(logits, 6, scoring=scoring)
    _route_check(logits, 6, scoring=scoring, renormalize=False)
    bias = torch.zeros(40, device="cuda")
    _route_check(logits, 6, scoring=scoring, bias=bias)
    bias[3], bias[5], bias[7], bias[39] = nan, -inf, 4.0, 4.0
    _route_check(logits, 6, scoring=scoring, bias=bias)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_router_keys_closer_than_fp32(scoring):
    """Biased keys that differ by less than FP32 resolves are ordered as in 64 bits."""
    T, E = 200, 64
    base = torch.randn(T, E, generator=_gen(3), device="cuda") * 0.5
    l = base.double()
    s = torch.softmax(l, -1) if scoring == "softmax" else torch.sigmoid(l)
    bias = (0.75 - s[0]).float()  # token 0: every key is 0.75 up to FP32's rounding
    logits = base[:1].repeat(T, 1) + torch.randn(T, E, generator=_gen(4), device="cuda") * 1e-6
    _route_check(logits, 8, scoring=scoring, bias=bias)


def test_router_live_tokens_strides_and_dispatch():
    """A bucket's padding gets -1; logits may be strided; the outputs feed a dispatch."""
    T, live, E, K, H = 48, 31, 16, 4, 256
    wide = torch.randn(T, 3 * E, generator=_gen(8), device="cuda")
    wide[live:] = float("nan")
    n = torch.tensor([live], dtype=torch.int32, device="cuda")
    ids, w = lib.route_topk(wide[:, E:2 * E], K, live_tokens=n)
    want_ids, want_w = eh.route_reference(wide[:live, E:2 * E].cpu(), K)
    assert torch.equal(ids[:live].cpu(), want_ids)
    assert (ids[live:] == -1).all() and (w[live:] == 0).all()
    assert w[:live].double().cpu().sub(want_w).abs().max() <= 2.0 ** -17
    x = torch.randn(T, H, generator=_gen(9), device="cuda").to(BF16)
    with afd.Buffer(1, 1, E, K, H, T) as buf:
        buf.source_dispatch(0, x, ids, w, bucket=T)
        r = buf.worker_receive(0, bucket=T)
        assert r.ends[-1].item() == live * K
        buf.worker_reply(0, r.rows, r.receipt)
        out = buf.source_collect(0, num_tokens=T)
        torch.cuda.synchronize()
        assert buf.get_error()[0] == 0
    sum_w = w.double().sum(1, keepdim=True)
    assert ((out.double() - x.double() * sum_w).abs() <= (eh.HALF_BF16 + 2 ** -20) * (x.double() * sum_w).abs()).all()


def test_router_captured_with_new_logits():
    T, E, K = 20, 128, 8
    logits = torch.randn(T, E, generator=_gen(1), device="cuda")
    lib.route_topk(logits, K)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ids, w = lib.route_topk(logits, K)
    logits.copy_(torch.randn(T, E, generator=_gen(2), device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    want_ids, want_w = eh.route_reference(logits.cpu(), K)
    assert torch.equal(ids.cpu(), want_ids)
    assert w.double().cpu().sub(want_w).abs().max() <= 2.0 ** -17


# ------------------------------------------------------- the operators together
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("fp8", [False, True])
def test_whole_expert_path(fp8, T):
    """Router -> dispatch -> product -> adapters -> activation -> product ->
    reply -> collect, for two sources and two workers, eagerly and replayed
    from one graph with new tokens, against float64 values token by token."""
    A, F, E, K, H, I, rank, S, alpha = 2, 2, 8, 3, 256, 128, 8, 2, 16
    Ef, bucket = E // F, 64
    g = _gen(31)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    gate_w = rnd(E, H) * H ** -0.5
    w13, w2 = rnd(E, 2 * I, H) * H ** -0.5, rnd(E, H, I) * I ** -0.5
    s13 = s2 = None
    if fp8:
        w13, s13 = eh.quantise_weight(w13)
    else:
        w13 = w13.to(BF16)
    w2 = w2.to(BF16)
    down, up = (rnd(S, rank, H) * H ** -0.5).to(BF16), rnd(S, 2 * I, rank).to(BF16)
    scales = torch.tensor([0.5, 1.5], device="cuda")
    slots = torch.randint(-1, S, (A * bucket,), generator=g, device="cuda").int()
    x = [rnd(T, H) for _ in range(A)]
    xb = [v.to(BF16) for v in x]
    if fp8:
        q = [eh.quantise_rows(v) for v in x]
        rows, row_scales = [a for a, _ in q], [b for _, b in q]
        xv = [a.double() * b.double().repeat_interleave(128, 1) for a, b in q]
    else:
        rows, row_scales, xv = xb, [None] * A, [v.double() for v in xb]
    logits = [v.float() @ gate_w.t() for v in xb]
    outs = [torch.zeros(T, H, dtype=BF16, device="cuda") for _ in range(A)]
    buf = afd.Buffer(A, F, E, K, H, bucket, alpha, "fp8" if fp8 else "bf16")

    def step():
        routes = [lib.route_topk(l, K) for l in logits]
        for s in range(A):
            buf.source_dispatch(s, rows[s], *routes[s], row_scales[s], bucket=bucket)
        replies = []  # kept until they are collected
        for f in range(F):
            r = buf.worker_receive(f, bucket=bucket)
            mine = slice(f * Ef, (f + 1) * Ef)
            kw = dict(expert_alignment=alpha)
            h = lib.grouped_linear(r.rows, w13[mine], r.ends, x_scale=r.row_scales,
                                   weight_scale=None if s13 is None else s13[mine], **kw)
            lib.adapter_add(h, r.rows, down, up, slots, scales, row_src=r.row_src, ends=r.ends, top_k=K,
                            x_scale=r.row_scales)
            a = lib.gated_rows(h, r.ends, **kw)
            replies.append(lib.grouped_linear(a, w2[mine], r.ends, **kw))
            buf.worker_reply(f, replies[f], r.receipt)
        buf.source_collect_all(outs=outs)
        return routes

    def check(routes):
        w13v = w13.double()
        if fp8:
            w13v = w13v * s13.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
        for s in range(A):
            ids, w = routes[s]
            for t in range(T):
                want = torch.zeros(H, dtype=torch.float64, device="cuda")
                mag = torch.zeros_like(want)
                a = int(slots[s * bucket + t])
                for k in range(K):
                    e = int(ids[t, k])
                    h = w13v[e] @ xv[s][t]
                    if a >= 0:
                        h = h + scales[a].double() * (up[a].double() @ (down[a].double() @ xv[s][t]))
                    gt, u = h.chunk(2)
                    act = eh.silu(gt) * u
                    want += w[t, k].double() * (w2[e].double() @ act)
                    # roundings to BF16: h twice (1.1 |gate| u + silu u each), the activation, the reply
                    off = 2 * eh.HALF_BF16 * (1.1 * gt.abs() * u.abs() + act.abs()) + eh.HALF_BF16 * act.abs()
                    mag += w[t, k].double() * (w2[e].double().abs() @ off + eh.HALF_BF16 * (w2[e].double() @ act).abs())
                tol = 1.05 * mag + eh.HALF_BF16 * want.abs() + 1e-6
                assert ((outs[s][t].double() - want).abs() <= tol).all()

    try:
        routes = step()
        torch.cuda.synchronize()
        assert buf.get_error()[0] == 0
        check(routes)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step()
        for s in range(A):
            logits[s].copy_(rnd(T, E))
        graph.replay()
        torch.cuda.synchronize()
        check(captured)
    finally:
        torch.cuda.synchronize()
        buf.close()


def test_calls_on_a_given_stream():
    """stream=: the operators run there, and so do the tensors they make."""
    side = torch.cuda.Stream()
    ends = torch.tensor([3, 9], dtype=torch.int32, device="cuda")
    x = torch.randn(9, 128, generator=_gen(1), device="cuda").to(BF16)
    w = torch.randn(2, 256, 128, generator=_gen(2), device="cuda").to(BF16)
    logits = torch.randn(9, 16, generator=_gen(3), device="cuda")
    want = (*lib.route_topk(logits, 2), lib.grouped_linear(x, w, ends, gated=True), lib.gated_rows(x, ends))
    torch.cuda.synchronize()
    got = (*lib.route_topk(logits, 2, stream=side), lib.grouped_linear(x, w, ends, gated=True, stream=side),
           lib.gated_rows(x, ends, stream=side))
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_first_calls_inside_a_capture():
    """A process whose first call of every operator is captured (nothing has to be set up eagerly)."""
    code = """
import torch, combine_attention_ffn_gb300 as lib
d = "cuda"
ends = torch.tensor([3, 9], dtype=torch.int32, device=d)
x = torch.randn(9, 128, device=d).bfloat16(); w = torch.randn(2, 256, 128, device=d).bfloat16()
q = x.to(torch.float8_e4m3fn); qw = w.to(torch.float8_e4m3fn)
xs, ws = torch.ones(9, 1, device=d), torch.ones(2, 2, 1, device=d)
logits = torch.randn(9, 16, device=d)
down, up = torch.randn(2, 16, 128, device=d).bfloat16(), torch.randn(2, 256, 16, device=d).bfloat16()
slots, scales = torch.tensor([0, 1, -1] * 3, dtype=torch.int32, device=d), torch.ones(2, device=d)
def step():
    h = lib.grouped_linear(x, w, ends)
    return [*lib.route_topk(logits, 2), lib.adapter_add(h, x, down, up, slots, scales), lib.gated_rows(h, ends),
            lib.grouped_linear(x, w, ends, gated=True), lib.grouped_linear(q, qw, ends, x_scale=xs, weight_scale=ws)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay(); torch.cuda.synchronize()
for a, b in zip(got, step()):
    assert torch.equal(a, b)
print("captured first: ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=120)
    assert r.returncode == 0 and "captured first: ok" in r.stdout, r.stderr[-2000:]


# ---------------------------------------------------------------- refusals
def test_refusals_of_unreachable_and_unaligned_buffers():
    """Host memory, misaligned bases and bad shapes raise before anything runs."""
    ends = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    w = torch.zeros(2, 32, 64, dtype=BF16, device="cuda")
    out = torch.full((4, 32), 7.0, dtype=BF16, device="cuda")

    def refused(status, fn, *a, **kw):
        with pytest.raises(afd.AfdError) as e:
            fn(*a, **kw)
        assert e.value.status == status

    refused(afd.ERR_ARG, lib.grouped_linear, x, w.cpu(), ends, out=out)
    refused(afd.ERR_ARG, lib.grouped_linear, x, w.cpu().pin_memory(), ends, out=out)
    refused(afd.ERR_ARG, lib.grouped_linear, x, w, ends.cpu(), out=out)
    shifted = torch.zeros(4 * 64 + 1, dtype=BF16, device="cuda")[1:].view(4, 64)
    refused(afd.ERR_UNSUPPORTED, lib.grouped_linear, shifted, w, ends, out=out)
    wide = torch.zeros(4, 68, dtype=BF16, device="cuda")[:, :64]
    refused(afd.ERR_UNSUPPORTED, lib.grouped_linear, wide, w, ends, out=out)
    refused(afd.ERR_ARG, lib.grouped_linear, x, w, ends, out=out, gated=True)
    refused(afd.ERR_ARG, lib.grouped_linear, x, w, ends, out=out, expert_alignment=0)
    refused(afd.ERR_ARG, lib.grouped_linear, x, w, ends[:1], out=out)
    refused(afd.ERR_ARG, lib.grouped_linear, x.half(), w.half(), ends, out=out)
    refused(afd.ERR_ARG, lib.gated_rows, x.cpu(), ends)
    refused(afd.ERR_ARG, lib.route_topk, torch.zeros(3, 8), 2, ids=torch.zeros(3, 2, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    assert (out == 7.0).all()


def test_row_operators_take_pinned_host_buffers():
    """Router, activation and adapters read and write page-locked host memory in place."""
    pin = lambda t: t.cpu().pin_memory()
    logits = torch.randn(5, 16, generator=_gen(1), device="cuda")
    ids, w = lib.route_topk(logits, 3)
    pids, pw = (torch.zeros(5, 3, dtype=d).pin_memory() for d in (torch.int64, torch.float32))
    lib.route_topk(pin(logits), 3, ids=pids, weights=pw)
    ends = torch.tensor([4, 5], dtype=torch.int32, device="cuda")
    h = torch.randn(5, 64, generator=_gen(2), device="cuda").to(BF16)
    act, pact = lib.gated_rows(h, ends), torch.zeros(5, 32, dtype=BF16).pin_memory()
    lib.gated_rows(pin(h), pin(ends), out=pact)
    for R in (20, 520):
        case = _adapter_case(R, 64, 40, 16, 3, 3, R)
        x, base, down, up, scales, slots = case
        want = lib.adapter_add(base, x, down, up, slots, scales, out=torch.empty_like(base))
        px, pbase, pdown, pup, pscales, pslots = (pin(t) for t in case)
        lib.adapter_add(pbase, px, pdown, pup, pslots, pscales)
        torch.cuda.synchronize()
        assert torch.equal(pbase, want.cpu())
    assert torch.equal(pids, ids.cpu()) and torch.equal(pw, w.cpu())
    assert torch.equal(pact, act.cpu())
