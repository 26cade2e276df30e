"""Decode attention over E4M3 caches whose value scales are infinite, very large
or very unlike each other: the scores' log-sum is of the scores alone, whatever
the values weigh, in a warp, across a block's warps and across blocks; weak tokens
beside strong ones keep their part of the result."""
import math

import pytest
import torch

import combine_attention_ffn_gb300 as lib
import expert_harness as eh
import source_harness as sh

pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
INF = float("inf")

# Tokens of the sequences under test: one tile, what a block takes whole, what
# blocks share; and a batch whose warps have whole sequences.
LENGTHS = {"tile": [16], "block": [700], "blocks": [9000], "batch": [(i * 37) % 150 + 1 for i in range(400)]}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_attention_ffn_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _place(case, b, token):
    """(page, place) of a token."""
    page = case[0].shape[2]
    return case[4][b, token // page].long(), token % page


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [3, 16])
@pytest.mark.parametrize("name", sorted(LENGTHS))
def test_lse_beside_an_infinite_value_scale(name, G, D):
    """What the cache write stores for a vector with an infinity: its head's
    result is NaN, the scores' log-sum as without it."""
    lengths = LENGTHS[name]
    case = sh.paged(lengths, 16, 2, D, True, _gen(1))
    k, v, ks, vs, table, n = case
    q = torch.randn(len(lengths), 2 * G, D, generator=_gen(2), device="cuda").to(BF16)
    clean, clean_lse = lib.decode_attention(q, k, v, table, n, k_scale=ks, v_scale=vs, return_lse=True)
    hit = torch.zeros(len(lengths), 2 * G, dtype=torch.bool, device="cuda")
    for b in range(0, len(lengths), 3):
        for token in {0, lengths[b] // 2, lengths[b] - 1} if b % 2 == 0 else {lengths[b] // 3}:
            page, at = _place(case, b, token)
            vs[page, 1, at] = INF
            v.view(torch.uint8)[page, 1, at] = 0
            v.view(torch.uint8)[page, 1, at, token % D] = 0x7F
        hit[b, G:] = True
    out, lse = lib.decode_attention(q, k, v, table, n, k_scale=ks, v_scale=vs, return_lse=True)
    _, want, _, err = sh.attention(q, k, v, table, n, D ** -0.5, 0, ks, vs)
    sh.check_lse(lse, want, err)
    assert torch.isnan(out[hit]).all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


def _scored(scores, vs, v, D, G):
    """One sequence of one KV head whose tokens have these scores (scale 1), and
    G equal queries that ask for them: column 0 of a key is its score's sign,
    its scale the score's size."""
    n, page = len(scores), 16
    pages = -(-n // page)
    k = torch.zeros(pages * page, D, device="cuda")
    k[:n, 0] = torch.where(scores < 0, -1.0, 1.0)
    rows = lambda t: torch.cat([t, t.new_zeros(pages * page - n, *t.shape[1:])])
    cache = lambda t: t.view(pages, 1, page, *t.shape[1:])
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    q = torch.zeros(1, G, D, dtype=BF16, device="cuda")
    q[..., 0] = 1
    return q, (cache(k.to(FP8)), cache(rows(v).to(FP8)), cache(rows(scores.abs())), cache(rows(vs)), table,
               torch.tensor([n], dtype=torch.int32, device="cuda"))


def _call(q, case):
    k, v, ks, vs, table, n = case
    out, lse = lib.decode_attention(q, k, v, table, n, scale=1.0, k_scale=ks, v_scale=vs, return_lse=True)
    want, want_lse, err, lse_err = sh.attention(q, k, v, table, n, 1.0, 0, ks, vs)
    return out[0], lse[0], want[0], want_lse[0], err[0], lse_err[0]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 16])
@pytest.mark.parametrize("n", [60, 2000, 20000])
@pytest.mark.parametrize("e", [60, 80, 100, 119])
def test_one_very_large_value_scale(e, n, G, D):
    """A token whose values are 2^e beside many that score 2^-8 of it (119: the
    largest that BF16 values lead to). Up to 2^80 the result is right, above it
    right or not finite; the log-sum is right either way."""
    scores = torch.full((n,), -8 * math.log(2), device="cuda")
    vs = torch.full((n,), 0.01, device="cuda")
    scores[n // 3], vs[n // 3] = 0.0, 2.0 ** e
    v = (torch.randn(n, D, generator=_gen(3), device="cuda") * 100).clamp(-448, 448)
    out, lse, want, want_lse, err, lse_err = _call(*_scored(scores, vs, v, D, G))
    sh.check_lse(lse, want_lse, lse_err)
    ok = torch.ones(G, dtype=torch.bool, device="cuda")
    if e > 80:
        ok = torch.isfinite(out).all(-1)
    eh.check_bf16(out, want, err, ok)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 16])
@pytest.mark.parametrize("n", [60, 700, 9000])
@pytest.mark.parametrize("e", [0, 30, 60, 80])
@pytest.mark.parametrize("first", [True, False])
def test_values_of_zero_beside_large_ones(first, e, n, G, D):
    """The first half of a sequence, or the last tenth, has values of scale 2^e, the
    rest none (scale 0, or the smallest one): equal scores count alike in the
    log-sum, whatever the parts that are joined hold."""
    scores = torch.zeros(n, device="cuda")
    vs = torch.full((n,), 2.0 ** e, device="cuda")
    none = torch.arange(n, device="cuda") >= n // 2 if first else torch.arange(n, device="cuda") < n - n // 10
    vs[none] = torch.where(torch.arange(int(none.sum()), device="cuda") % 40 < 20, 0.0, 2.0 ** -100)
    v = (torch.randn(n, D, generator=_gen(4), device="cuda") * 100).clamp(-448, 448)
    v[none] = 0
    out, lse, want, want_lse, err, lse_err = _call(*_scored(scores, vs, v, D, G))
    sh.check_lse(lse, want_lse, lse_err)
    eh.check_bf16(out, want, err, torch.ones(G, dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 16])
@pytest.mark.parametrize("n", [64, 700, 9000])
@pytest.mark.parametrize("weak", [24.3, 25.5, 28.0])
def test_a_weak_tail_beside_strong_tokens(weak, n, G, D):
    """One token in 32 weighs 2^weak of every other one; in the odd columns only
    the weak ones have values. Weights are FP16 with 2^7 for a warp's largest: half of
    FP16's smallest step is 2^-32 of that. The rest of the bound: 2^-11 for a weight's own
    rounding; scores up to 28 (base 2) with three roundings and the exponential's 2^-22, less
    than 2^-18; sums as in the harness."""
    strong = torch.arange(n, device="cuda") % 32 == 5
    scores = torch.where(strong, 0.0, -weak * math.log(2))
    vs = torch.full((n,), 0.01, device="cuda")
    v = torch.rand(n, D, generator=_gen(5), device="cuda") * 400 + 40
    v[:, 1::2] *= ~strong[:, None]
    q, case = _scored(scores, vs, v, D, G)
    out = lib.decode_attention(q, case[0], case[1], case[4], case[5], scale=1.0, k_scale=case[2], v_scale=case[3])[0]
    p = torch.softmax(scores.double(), 0)
    codes = case[1].view(-1, D)[:n].double()
    want = p * vs.double() @ codes
    rel = 2.0 ** -11 + 2.0 ** -17 + (n + 64) * 2 * sh.FP32_HALF
    err = rel * want + 2.0 ** -32 * (p * vs.double()).max() * codes.sum(0)
    assert (err[1::2] < 0.1 * want[1::2]).all()
    eh.check_bf16(out, want.expand(G, D), err.expand(G, D), torch.ones(G, dtype=torch.bool, device="cuda"))
