"""norm_rows: E4M3 values are the FP32 quotient by the block's scale, rounded to
nearest even: bit for bit, at values that FP32 holds exactly."""
import math
import random

import pytest
import torch

import combine_attention_ffn_gb300 as lib

pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_attention_ffn_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _check(y, got):
    """The scale is a product with FP32's 1 / 448, 2^-100 at least."""
    y = y.float().view(*got.scales.shape, 128)
    scale = (y.abs().amax(-1) * torch.tensor(1 / 448, device="cuda")).clamp_min(2.0 ** -100)
    assert torch.equal(got.scales, scale)
    want = (y / scale[..., None]).to(FP8)
    values = got.fp8_rows.view(*scale.shape, 128)
    off = (values.view(torch.uint8) != want.view(torch.uint8)).sum().item()
    assert off == 0, f"{off} of {want.numel()} values are not the rounded quotient"


@pytest.mark.parametrize("H", [128, 2048, 4096, 16384, 32768])
def test_ties(H):
    """Rows of +-1 (mean square 1, eps 0): y is the weight exactly, here whole
    numbers whose quotients often lie between two E4M3 values."""
    g = torch.Generator(device="cuda").manual_seed(H)
    x = (torch.randint(0, 2, (8, H), generator=g, device="cuda") * 2 - 1).to(BF16)
    for most in (3, 14, 200):
        w = torch.randint(-most, most + 1, (H,), generator=g, device="cuda").float().to(BF16)
        got = lib.norm_rows(x, w, eps=0.0, fp8=True)
        assert torch.equal(got.rows, x * w)
        _check(x * w, got)


def _squares(n, total, rng):
    """n whole numbers whose squares sum to `total`."""
    while True:
        got = [rng.randint(1, 25) for _ in range(n - 3)]
        rest = total - sum(t * t for t in got)
        if rest < 0:
            continue
        a = math.isqrt(rest)
        for b in range(math.isqrt(rest - a * a), -1, -1):
            c = math.isqrt(rest - a * a - b * b)
            if a * a + b * b + c * c == rest and a < 256:
                return got + [a, b, c]


@pytest.mark.parametrize("seed", range(8))
def test_products_of_two_bf16_numbers(seed):
    """Rows of sixteenths whose mean square is 1: y is a product of two BF16
    numbers, whose quotients come within a step of a border (a product with the scale's
    reciprocal puts one in 40,000 on the wrong side)."""
    rng, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
    groups = torch.tensor([_squares(16, 16 * 256, rng) for _ in range(200)], device="cuda").float() / 16
    T, H = 256, 4096
    x = groups[torch.randint(0, 200, (T, H // 16), generator=g, device="cuda")].view(T, H)
    x = x * (torch.randint(0, 2, (T, H), generator=g, device="cuda") * 2 - 1)
    assert (x.square().mean(1) == 1).all() and torch.equal(x, x.to(BF16).float())
    w = (1 + (0.3 if seed % 2 else 1.0) * torch.randn(H, generator=g, device="cuda")).to(BF16)
    got = lib.norm_rows(x.to(BF16), w, eps=0.0, fp8=True)
    assert torch.equal(got.rows, (x * w.float()).to(BF16))
    _check(x * w.float(), got)


@pytest.mark.parametrize("e", [-126, -115, -105, -100, -98, -95, -92, -90, -88, -85, -60, 0, 60, 110])
def test_scales_from_the_smallest_to_the_largest(e):
    """The same with weights around 2^e: the scale at its floor, just above it
    (where a quotient's remainder is no normal number) and near the top."""
    g = torch.Generator(device="cuda").manual_seed(e + 200)
    x = (torch.randint(0, 2, (4, 4096), generator=g, device="cuda") * 2 - 1).to(BF16)
    w = (torch.randint(-200, 201, (4096,), generator=g, device="cuda").double() * 2.0 ** e).to(BF16)
    got = lib.norm_rows(x, w, eps=0.0, fp8=True)
    assert torch.equal(got.rows, x * w)
    _check(x * w, got)


def test_infinities_still_spoil_their_block_alone():
    x = torch.ones(2, 256, device="cuda").to(BF16)
    w = torch.ones(256, device="cuda").to(BF16)
    w[5] = float("inf")
    w[200] = float("nan")
    got = lib.norm_rows(x, w, eps=0.0, fp8=True)
    decoded = got.fp8_rows.float().view(2, 2, 128) * got.scales[..., None]
    assert torch.isnan(decoded).all()
    w[200] = 1.0
    got = lib.norm_rows(x, w, eps=0.0, fp8=True)
    decoded = got.fp8_rows.float().view(2, 2, 128) * got.scales[..., None]
    assert torch.isnan(decoded[:, 0]).all() and (decoded[:, 1] == 1.0).all()
