"""Sizes that 32 bits do not hold: the binding refuses them (ctypes would cut
them to their low bits). Meta tensors stand in for the memory; no GPU."""
import pytest
import torch

import combine_attention_ffn_gb300 as lib
from combine_attention_ffn_gb300 import afd

BIG = 1 << 32


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def ints(*shape):
    return meta(*shape, dtype=torch.int32)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_attention_ffn_gb300 import build

    afd.load_library(build.build())


@pytest.mark.parametrize("call", [
    lambda: lib.route_topk(meta(BIG + 4, 1), 1),
    lambda: lib.route_topk(meta(4, BIG + 8), 1),
    lambda: lib.route_topk(meta(0, 8), BIG + 1),
    lambda: lib.grouped_linear(meta(4, BIG + 64), meta(1, 8, BIG + 64), ints(1)),
    lambda: lib.grouped_linear(meta(4, 64), meta(1, BIG + 8, 64), ints(1)),
    lambda: lib.grouped_linear(meta(4, 64), meta(BIG + 1, 8, 64), ints(BIG + 1)),
    lambda: lib.grouped_linear(meta(4, 64), meta(1, 8, 64), ints(1), expert_alignment=BIG + 16),
    lambda: lib.grouped_linear(meta(4, 64), meta(1, 8, 64), ints(1), expert_alignment=16 - BIG),
    lambda: lib.gated_rows(meta(4, 2 * BIG + 16), ints(1)),
    lambda: lib.gated_rows(meta(4, 16), ints(BIG + 1)),
    lambda: lib.gated_rows(meta(4, 16), ints(1), expert_alignment=BIG + 16),
    lambda: lib.adapter_add(meta(4, 64), meta(4, 32), meta(2, 16, 32), meta(2, 64, 16), ints(BIG + 4),
                            meta(2, dtype=torch.float32)),
    lambda: lib.adapter_add(meta(4, BIG + 64), meta(4, 32), meta(2, 16, 32), meta(2, BIG + 64, 16), ints(4),
                            meta(2, dtype=torch.float32)),
    lambda: lib.adapter_add(meta(4, 64), meta(4, BIG + 32), meta(2, 16, BIG + 32), meta(2, 64, 16), ints(4),
                            meta(2, dtype=torch.float32)),
    lambda: lib.adapter_add(meta(4, 64), meta(4, 32), meta(BIG + 2, 16, 32), meta(BIG + 2, 64, 16), ints(4),
                            meta(BIG + 2, dtype=torch.float32)),
    lambda: lib.adapter_add(meta(4, 64), meta(4, 32), meta(2, 16, 32), meta(2, 64, 16), ints(4),
                            meta(2, dtype=torch.float32), row_src=ints(4), ends=ints(1), top_k=BIG + 1),
    lambda: lib.adapter_add(meta(4, 64), meta(4, 32), meta(2, 16, 32), meta(2, 64, 16), ints(4),
                            meta(2, dtype=torch.float32), row_src=ints(4), ends=ints(BIG + 1)),
])
def test_refused(call):
    with pytest.raises(afd.AfdError) as e:
        call()
    assert e.value.status == afd.ERR_UNSUPPORTED
