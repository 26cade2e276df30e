"""The products and the adapters at widths of the wide exchanges (hidden 4,096
and 7,168), where K and N pass what the other tests use."""
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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("K,N,gated", [(4096, 1536, True), (7168, 2048, True), (2048, 7168, False), (4096, 4096, False)])
def test_products(K, N, gated, fp8):
    g = torch.Generator("cuda").manual_seed(K + N)
    ends, R, spans = eh.ragged([1, 0, 37, 290], 128, 7)
    W = 2 * N if gated else N
    x, w = torch.randn(R, K, generator=g, device="cuda"), torch.randn(4, W, K, generator=g, device="cuda") * K ** -0.5
    xs = ws = None
    if fp8:
        (x, xs), (w, ws) = eh.quantise_rows(x), eh.quantise_weight(w)
    else:
        x, w = x.to(BF16), w.to(BF16)
    out = torch.full((R, N), 7.0, dtype=BF16, device="cuda")
    lib.grouped_linear(x, w, torch.tensor(ends, dtype=torch.int32, device="cuda"), expert_alignment=128, gated=gated,
                       x_scale=xs, weight_scale=ws, out=out)
    y, mag = eh.product(x, w, spans, xs, ws)
    want, err = eh.gated(y, mag, K) if gated else (y, eh.product_error(mag, K))
    live = eh.live_rows(R, spans, "cuda")
    eh.check_bf16(out, want, err, live)
    assert (out[~live] == 7.0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rank", [8, 64])
@pytest.mark.parametrize("R", [33, 600])  # a row at a time, and grouped
@pytest.mark.parametrize("K,N", [(4096, 7168), (7168, 4104)])
def test_adapters(K, N, R, rank, fp8):
    g = torch.Generator("cuda").manual_seed(K + N + R)
    S = 5
    x = torch.randn(R, K, generator=g, device="cuda")
    base = torch.randn(R, N, generator=g, device="cuda").to(BF16)
    down = (torch.randn(S, rank, K, generator=g, device="cuda") * K ** -0.5).to(BF16)
    up = (torch.randn(S, N, rank, generator=g, device="cuda") * rank ** -0.5).to(BF16)
    scales = torch.rand(S, generator=g, device="cuda") + 0.5
    slots = torch.randint(-1, S + 1, (R,), generator=g, device="cuda").int()
    xs = None
    if fp8:
        x, xs = eh.quantise_rows(x)
        value = x.double() * xs.double().repeat_interleave(128, 1)
    else:
        x = x.to(BF16)
        value = x.double()
    out = lib.adapter_add(base, x, down, up, slots, scales, x_scale=xs, out=torch.empty_like(base))
    want, err = base.double(), torch.zeros(R, N, dtype=torch.float64, device="cuda")
    for a in range(S):
        rows = (slots == a).nonzero()[:, 0]
        d, u, sc = down[a].double(), up[a].double(), scales[a].double()
        t = value[rows] @ d.t()
        # the down sums of K products, the low-rank product to 16 bits, the up sums
        et = (K + 4) * eh.FP32_STEP * (value[rows].abs() @ d.abs().t()) + 2.0 ** -16 * t.abs()
        want[rows] += sc * (t @ u.t())
        err[rows] = sc * (et @ u.abs().t()) + (2 * rank + 4) * eh.FP32_STEP * (
            sc * (t.abs() @ u.abs().t()) + base[rows].double().abs())
    eh.check_bf16(out, want, err, torch.ones(R, dtype=torch.bool, device="cuda"))
