"""How decode attention cuts its work into shares, checked without an error
bound that could hide a tile: equal scores (scale 0), so that every token
weighs the same, and values that say which tile they belong to. A result is
then a tile's number of tokens over the sequence's, exact up to its rounding,
and a tile that is lost or counted twice shows.

The lengths meet the kernel's own limits: the longest sequence that a block
takes whole (6 tiles a warp where tables allow no more, 4 by the lengths), and
lines of work that fill all warps' shares exactly, or miss that by a place."""
import pytest
import torch

import combine_attention_ffn_gb300 as lib
import expert_harness as eh
import source_harness as sh

BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
WARPS = 8  # of a block
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def built():
    from combine_attention_ffn_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _shape(D, fp8):
    """Tokens of a tile, and what a segment counts beside its tiles."""
    return 4096 // (D * (1 if fp8 else 2)), 2 if fp8 and D == 128 else 1


def _warps():
    return min(torch.cuda.get_device_properties(0).multi_processor_count, 160) * WARPS


def _marks(n, first, tile, D, device):
    """Column of every token: its tile's number, counted from `first`."""
    return (first + torch.arange(n, device=device) // tile) % D


def _want(marks, D):
    """(out, lse) of one sequence."""
    n = len(marks)
    if not n:
        return torch.zeros(D, dtype=torch.float64, device=marks.device), float("-inf")
    count = torch.bincount(marks, minlength=D).double()
    return count / n, torch.tensor(float(n), dtype=torch.float64).log().item()


def _check(out, lse, want, want_lse, tiles):
    """out [rows, D] and lse [rows]. Sums are exact (whole numbers below 2^24,
    times a power of two); the division and the product round once each, the
    base-2 logarithm is good to 2^-22 of its value, the rest of lse to three
    roundings of values a little larger than it. `tiles`: a row's tokens over
    those of a tile; the bounds are far below what one tile changes."""
    eh.check_bf16(out, want, 4 * sh.FP32_HALF * want, torch.ones(out.shape[0], dtype=torch.bool, device=out.device))
    empty = want_lse == float("-inf")
    assert torch.equal(lse == float("-inf"), empty)
    tol = (2.0 ** -20 * want_lse + 2.0 ** -20)[~empty]
    assert (tol * 8 < 1 / tiles[~empty]).all()
    off = (lse.double() - want_lse).abs()[~empty]
    assert (off <= tol).all(), f"lse off by {(off / tol).max().item():.3g} of the bound"


def _run(lengths, D, fp8, Hkv=1, G=1, window=0, page=64, width=None, seed=1):
    tile, _ = _shape(D, fp8)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v, ks, vs, table, n = sh.paged(lengths, page, Hkv, D, fp8, g, width=width)
    want = torch.zeros(len(lengths), Hkv, D, dtype=torch.float64, device="cuda")
    want_lse = torch.zeros(len(lengths), Hkv, dtype=torch.float64, device="cuda")
    tiles = torch.zeros_like(want_lse)
    first = 0
    for b, m in enumerate(lengths):
        at = torch.arange(m, device="cuda")
        where = table[b].long()[at // page]
        for h in range(Hkv):
            marks = _marks(m, first + 7 * h, tile, D, "cuda")
            v[where, h, at % page] = torch.nn.functional.one_hot(marks, D).to(v.dtype)
            if fp8:
                vs[where, h, at % page] = 1.0
            seen = marks[max(0, m - window):] if window else marks
            want[b, h], want_lse[b, h] = _want(seen, D)
            tiles[b, h] = len(seen) / tile
        first += -(-m // tile)
    q = torch.randn(len(lengths), Hkv * G, D, generator=g, device="cuda").to(BF16)
    out, lse = lib.decode_attention(q, k, v, table, n, scale=0.0, window=window, k_scale=ks, v_scale=vs, return_lse=True)
    rows = lambda t: t.repeat_interleave(G, 1).flatten(0, 1)
    _check(out.flatten(0, 1), lse.flatten(), rows(want), rows(want_lse), rows(tiles))


FORMS = pytest.mark.parametrize("D,fp8", [(64, False), (64, True), (128, False), (128, True)])


@gpu
@FORMS
@pytest.mark.parametrize("G", [1, 16])
def test_a_block_or_shares(built, D, fp8, G):
    """Around the longest sequence that a block takes whole, by its table's width and by its length."""
    tile, _ = _shape(D, fp8)
    for tiles in (1, WARPS - 1, WARPS, WARPS + 1, 4 * WARPS - 1, 4 * WARPS, 4 * WARPS + 1, 6 * WARPS - 1, 6 * WARPS, 6 * WARPS + 1):
        for n in (tiles * tile, tiles * tile - tile + 1):
            for page, width in ((16, -(-n // 16)), (16, 5000)):
                _run([n], D, fp8, G=G, page=page, width=width)
                _run([n], D, fp8, G=G, page=page, width=width, window=max(1, n - tile // 2))


@gpu
@FORMS
def test_full_shares_of_one_sequence(built, D, fp8):
    """Lines of k places a warp, of one less and of one more, for the smallest
    share (a beginning and a tile) and what comes next."""
    tile, begin = _shape(D, fp8)
    for k in (1, 1 + begin, 2 + begin, 3 + begin):
        for off in (-1, 0, 1):
            tiles = k * _warps() - begin + off
            for short in (0, tile - 1):
                _run([tiles * tile - short], D, fp8)


def _split(total, parts, begin, rng):
    """`parts` sequences whose tiles and beginnings make `total` places."""
    cuts = sorted(rng.sample(range(1, total - parts * (1 + begin)), parts - 1))
    free = [b - a for a, b in zip([0] + cuts, cuts + [total - parts * (1 + begin)])]
    return [1 + f for f in free]


@gpu
@FORMS
@pytest.mark.parametrize("B", [5, 33, 300])
def test_full_shares_of_many_sequences(built, B, D, fp8):
    """The same with sequences of any length, empty ones among them: up to 32
    every warp finds its share by itself, with more the block does, and above 256
    a thread has several."""
    import random

    rng = random.Random(B + D)
    tile, begin = _shape(D, fp8)
    live = B - B // 5
    for k in (1 + begin, 2 + begin):
        for off in (-1, 0, 1):
            lengths = [t * tile - rng.choice([0, 0, 1, tile - 1]) for t in _split(k * _warps() + off, live, begin, rng)]
            lengths += [0] * (B - live)
            rng.shuffle(lengths)
            _run(lengths, D, fp8)


@gpu
@FORMS
@pytest.mark.parametrize("seed", range(3))
def test_drawn_shares(built, seed, D, fp8):
    """Several KV heads, chunks of heads, windows and pages."""
    import random

    rng = random.Random(100 * seed + D + fp8)
    for _ in range(4):
        B, most = rng.choice([1, 3, 20, 40, 500]), rng.choice([100, 3000, 20000])
        lengths = [rng.randint(0, max(1, min(most, 200000 // B))) for _ in range(B)]
        _run(lengths, D, fp8, Hkv=rng.choice([1, 2, 3]), G=rng.choice([1, 4, 9, 20]), window=rng.choice([0, 0, rng.randint(1, most)]),
             page=rng.choice([1, 16, 24, 64]), seed=seed)


def test_the_check_notices_a_tile():
    """A tile lost, one counted twice, and a share's edge off by a tile (one lost, its neighbour twice), in a long sequence."""
    D, tile, tiles = 64, 64, 3600
    marks = _marks(tiles * tile - 5, 3, tile, D, "cpu")
    want, lse = _want(marks, D)
    one = lambda m: tuple(t if torch.is_tensor(t) else torch.tensor([t], dtype=torch.float64) for t in _want(m, D))

    def check(m):
        got, got_lse = one(m)
        _check(got[None].to(BF16), got_lse.float(), want[None], torch.tensor([lse], dtype=torch.float64),
               torch.tensor([len(marks) / tile]))

    check(marks)
    at = 1700 * tile
    for wrong in (torch.cat([marks[:at], marks[at + tile:]]), torch.cat([marks[:at], marks[at - tile:]]),
                  torch.cat([marks[:at], marks[at - tile:at], marks[at + tile:]]), marks[:-tile], marks[tile:]):
        with pytest.raises(AssertionError):
            check(wrong)
