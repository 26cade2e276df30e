"""grouped_linear's give-up path: with a limit of 0 every role of the kernel
gives up before its first wait, the call's `error` word says so, and the
context and later calls are as before. Nothing on the GPU stalls for this."""
import pytest
import torch

import combine_attention_ffn_gb300 as lib
import expert_harness as eh
from combine_attention_ffn_gb300 import afd

BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _limit():
    from combine_attention_ffn_gb300 import build

    build.build()
    yield
    lib.set_product_wait_limit()


def test_limits_that_are_none():
    for bad in (-1, 1 << 63):
        with pytest.raises(afd.AfdError) as e:
            lib.set_product_wait_limit(bad)
        assert e.value.status == afd.ERR_ARG
    assert afd.load_library().afd_set_product_wait_limit(-1) == afd.ERR_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_gives_up_and_says_so(fp8, gated):
    g = torch.Generator("cuda").manual_seed(1)
    ends, R, spans = eh.ragged([5, 0, 300, 40], 16, 3)
    K, N = 512, 256
    W = 2 * N if gated else N
    x, w = torch.randn(R, K, generator=g, device="cuda"), torch.randn(4, W, K, generator=g, device="cuda") * K ** -0.5
    xs = ws = None
    if fp8:
        (x, xs), (w, ws) = eh.quantise_rows(x), eh.quantise_weight(w)
    else:
        x, w = x.to(BF16), w.to(BF16)
    ends = torch.tensor(ends, dtype=torch.int32, device="cuda")
    live = eh.live_rows(R, spans, "cuda")
    y, mag = eh.product(x, w, spans, xs, ws)
    want, err = eh.gated(y, mag, K) if gated else (y, eh.product_error(mag, K))
    error, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((R, N), 7.0, dtype=BF16, device="cuda")

    def call():
        lib.grouped_linear(x, w, ends, expert_alignment=16, gated=gated, x_scale=xs, weight_scale=ws, out=out, error=error)

    graph = torch.cuda.CUDAGraph()
    for limit, status in ((0, afd.ERR_TIMEOUT), (afd.PRODUCT_WAIT_CYCLES, 0), (0, afd.ERR_TIMEOUT), (1 << 62, 0)):
        lib.set_product_wait_limit(limit)
        error.zero_()
        out.fill_(7.0)
        for _ in range(3):  # (TMEM and shared memory are free again each time)
            call()
        assert error.item() == status
        assert (out[~live] == 7.0).all()
        if status == 0:
            eh.check_bf16(out, want, err, live)
        else:
            lib.grouped_linear(x, w, ends, expert_alignment=16, gated=gated, x_scale=xs, weight_scale=ws, out=out)
            torch.cuda.synchronize()
    # a captured call keeps the limit it was captured with
    with torch.cuda.graph(graph):
        call()
    lib.set_product_wait_limit(0)
    error.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert error.item() == 0
    eh.check_bf16(out, want, err, live)
