"""adapter_add at the ends of FP32's range: the low-rank product of many rows,
kept as two BF16, stays the number that FP32 holds."""
import pytest
import torch

import combine_attention_ffn_gb300 as lib
import expert_harness as eh

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_attention_ffn_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("rank", [8, 32])
@pytest.mark.parametrize("R", [90, 690])  # few rows, many rows
def test_products_beyond_the_largest_bf16(R, rank):
    """scale * down x between the largest BF16 (3.39e38) and the largest FP32
    number (3.40e38), brought down again by up; infinities stay infinite."""
    K, N = 16, 24
    x = torch.zeros(R, K, dtype=BF16, device="cuda")
    x[:, 0] = torch.where(torch.arange(R, device="cuda") % 2 == 0, 1.0, -1.0).to(BF16)
    down = torch.zeros(3, rank, K, dtype=BF16, device="cuda")
    down[:, :, 0] = 1.0
    up = torch.randn(3, N, rank, generator=torch.Generator("cuda").manual_seed(1), device="cuda").mul_(2.0 ** -126).to(BF16)
    scales = torch.tensor([3.4e38, 3.4028234663852886e38, float("inf")], device="cuda")
    slots = (torch.arange(R, device="cuda") // 2 % 3).int()
    base = torch.zeros(R, N, dtype=BF16, device="cuda")
    out = lib.adapter_add(base, x, down, up, slots, scales, out=torch.empty_like(base))
    t = x[:, 0].double() * scales[slots.long()].double()
    want = t[:, None] * up.double()[slots.long()].sum(-1)
    # the low-rank product to 16 bits, rank sums of FP32
    err = t.abs()[:, None] * up.double().abs()[slots.long()].sum(-1) * (2.0 ** -16 + (2 * rank + 4) * eh.FP32_STEP)
    finite = slots < 2
    eh.check_bf16(out, want, err, finite)
    assert not torch.isfinite(out[~finite]).any()
