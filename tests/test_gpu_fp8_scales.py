"""grouped_linear with E4M3 scales over their whole range: the product of a
row's and a weight's anywhere in FP32's normal range, each of them by itself
anywhere, and zero."""
import pytest
import torch

import combine_attention_ffn_gb300 as lib
import expert_harness as eh

pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_attention_ffn_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _check(got, want, err):
    """Within the sums' error and half a BF16 step (2^-134 below its normal
    range) of the value."""
    tol = err + eh.HALF_BF16 * (want.abs() + err) + 2.0 ** -134
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist())


def _run(counts, K, N, gated, value_exp, x_exp, w_exp, seed):
    """Values around 2^value_exp; scales around 2^x_exp [R, K/128] and 2^w_exp
    [G, W/128, K/128] (exponents as tensors or numbers)."""
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda") + 1.0
    ends, R, spans = eh.ragged(counts, 16, 5)
    W = 2 * N if gated else N
    x = (torch.randn(R, K, generator=g, device="cuda") * 2.0 ** value_exp).to(FP8)
    w = (torch.randn(len(counts), W, K, generator=g, device="cuda") * 2.0 ** value_exp).to(FP8)
    power = lambda e, like: torch.ldexp(like, torch.as_tensor(e, device="cuda"))
    xs, ws = power(x_exp, rand(R, K // 128)), power(w_exp, rand(len(counts), W // 128, K // 128))
    live = eh.live_rows(R, spans, "cuda")
    out = torch.full((R, N), 7.0, dtype=BF16, device="cuda")
    lib.grouped_linear(x, w, torch.tensor(ends, dtype=torch.int32, device="cuda"), expert_alignment=16, gated=gated,
                       x_scale=xs, weight_scale=ws, out=out)
    y, mag = eh.product(x, w, spans, xs, ws)
    want, err = eh.gated(y, mag, K) if gated else (y, eh.product_error(mag, K))
    assert want[live].abs().max() < 3e38 and want[live].abs().median() > 2.0 ** -126  # ordinary numbers
    _check(out[live], want[live], err[live])
    assert (out[~live] == 7.0).all()


@pytest.mark.parametrize("counts", [[3, 0, 40], [300, 17]])
@pytest.mark.parametrize("value,xe,we", [(6, -100, -26), (6, -26, -100), (6, -126, 0), (6, 0, -126), (6, -63, -63),
                                         (-8, 100, 25), (-8, 25, 100), (-8, 126, -1), (-8, -1, 126), (-8, 62, 63)])
def test_products_of_scales_at_the_ends_of_fp32(counts, value, xe, we):
    _run(counts, 384, 256, False, value, xe, we, 3)


@pytest.mark.parametrize("counts", [[3, 0, 40], [300, 17]])
def test_mixed_rows_and_blocks(counts):
    """Rows and K blocks of far apart scales, and scales of zero."""
    ends, R, _ = eh.ragged(counts, 16, 5)
    r = torch.arange(R, device="cuda")[:, None]
    for only in ((r % 7 == 3), (r % 64 < 32), (r % 2 == 0)):
        xe = torch.where(only & (torch.arange(3, device="cuda") != 1), -100, 0).int()
        _run(counts, 384, 256, False, 6, xe, -20, 4)
    xe = torch.full((R, 3), -3, dtype=torch.int32, device="cuda")
    xe[::3, 1] = -400  # a scale of zero
    _run(counts, 384, 256, False, 6, xe, -3, 5)


@pytest.mark.parametrize("counts", [[3, 0, 40], [300, 17]])
@pytest.mark.parametrize("gate_e,up_e", [(-100, 25), (-110, 24)])
def test_gated(counts, gate_e, up_e):
    """x_scale 2^100: the gate's product is small, the up projection's near the top."""
    we = torch.tensor([gate_e, gate_e, up_e, up_e], device="cuda").view(1, 4, 1).expand(len(counts), 4, 3)
    _run(counts, 384, 256, True, -8, 100, we, 6)


def test_zero_blocks_under_scales_of_nothing():
    """Values of zero give zero under scales whose product FP32 does not hold."""
    x, w = torch.zeros(40, 256, device="cuda").to(FP8), torch.ones(1, 128, 256, device="cuda").to(FP8)
    for a, b in ((1e-30, 1e-30), (0.0, 1.0), (1.0, 0.0), (2.0 ** -149, 2.0 ** -149)):
        out = lib.grouped_linear(x, w, torch.tensor([40], dtype=torch.int32, device="cuda"),
                                 x_scale=torch.full((40, 2), a, device="cuda"), weight_scale=torch.full((1, 1, 2), b, device="cuda"))
        assert (out == 0).all()
