"""Decode attention where scores are infinite: +infinity spoils its head's
result and log-sum, -infinity leaves its token out, and a head whose scores are all
-infinity is one that sees nothing."""
import pytest
import torch

import combine_attention_ffn_gb300 as lib
import expert_harness as eh
import source_harness as sh

pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_attention_ffn_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 20, 700, 9000])
def test_infinite_scores(n, fp8):
    """Keys of column 0 alone; head 0 asks for +1, head 1 for -1."""
    page, D = 16, 64
    k, v, ks, vs, table, lengths = sh.paged([n], page, 1, D, fp8, torch.Generator(device="cuda").manual_seed(n))
    at = torch.arange(n, device="cuda")
    where = table[0].long()[at // page], 0, at % page
    k[where] = torch.zeros(n, D, device="cuda").to(k.dtype)
    keys = torch.rand(n, device="cuda") + 0.5

    def put(infinite):
        x = torch.where(infinite, float("inf"), keys)
        if fp8:
            k[where[0], 0, where[2], 0] = torch.ones(n, device="cuda").to(FP8)
            ks[where] = x
        else:
            k[where[0], 0, where[2], 0] = x.to(BF16)

    q = torch.zeros(1, 2, D, dtype=BF16, device="cuda")
    q[0, 0, 0], q[0, 1, 0] = 1, -1
    call = lambda: lib.decode_attention(q, k, v, table, lengths, k_scale=ks, v_scale=vs, return_lse=True)
    put(at == n // 2)
    out, lse = call()
    assert torch.isnan(out[0, 0]).all() and torch.isnan(lse[0, 0])
    if n > 1:  # head 1: as if the token were not there
        x = torch.where(at == n // 2, 0.0, keys if fp8 else keys.to(BF16).float()).double()
        p = torch.exp(-x / 8) * (at != n // 2)
        values = v[where].double() * (vs[where].double()[:, None] if fp8 else 1)
        want, total = p @ values / p.sum(), p.sum()
        err = (2.0 ** -11 + 2.0 ** -16 + (n + 64) * 2 * sh.FP32_HALF) * (p @ values.abs() / total)
        eh.check_bf16(out[0, 1:], want[None], err[None], torch.ones(1, dtype=torch.bool, device="cuda"))
        assert abs(lse[0, 1].item() - total.log().item()) <= 2.0 ** -14  # (a lane adds 150 terms at most)
    put(at >= 0)
    out, lse = call()
    assert torch.isnan(out[0, 0]).all() and torch.isnan(lse[0, 0])
    assert (out[0, 1].view(torch.int16) == 0).all() and lse[0, 1] == float("-inf")
