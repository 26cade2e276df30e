"""gated_rows with rows wider than a warp's one pass (1,024 columns) and at the
edges of its 16-byte path, out of place and over its own input."""
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


@pytest.mark.parametrize("N", [1016, 1025, 1032, 2048, 2056, 5000, 7168])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_wide_rows_and_in_place(N, pad):
    """`pad` more columns behind every row: other strides, with 3 no 16-byte path."""
    g = torch.Generator("cuda").manual_seed(N + pad)
    ends, R, spans = eh.ragged([3, 0, 1, 40, 17, 260], 16, 3)
    live = eh.live_rows(R, spans, "cuda")
    wide = (torch.randn(R, 2 * N + pad, generator=g, device="cuda") * 3).to(BF16)
    h = wide[:, :2 * N]
    before = wide.clone()
    ends = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out = torch.full((R, N + pad), 7.0, dtype=BF16, device="cuda")
    lib.gated_rows(h, ends, expert_alignment=16, out=out[:, :N])
    gate, up = h.double().chunk(2, 1)
    v = eh.silu(gate) * up
    eh.check_bf16(out[:, :N], v, 2.0 ** -18 * v.abs(), live)
    assert (out[~live] == 7.0).all() and (out[:, N:] == 7.0).all() and torch.equal(wide, before)
    lib.gated_rows(h, ends, expert_alignment=16, out=h[:, :N])
    assert torch.equal(wide[live][:, :N], out[live][:, :N])
    assert torch.equal(wide[:, N:], before[:, N:]) and torch.equal(wide[~live], before[~live])
