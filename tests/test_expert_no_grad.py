"""The expert operators have no backward pass: a call whose result autograd
would take for a constant is refused, and taken under no_grad."""
import pytest
import torch

import combine_attention_ffn_gb300 as lib
from combine_attention_ffn_gb300 import afd

BF16, FP8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_attention_ffn_gb300 import build

    afd.load_library(build.build())


def _calls(device):
    """(name, arguments that may carry gradients, call)"""
    def z(*s, dtype=BF16):
        return torch.zeros(*s, dtype=dtype, device=device)

    ends = torch.tensor([2, 4], dtype=torch.int32, device=device)
    slots = z(4, dtype=torch.int32)
    return [
        ("route", dict(logits=z(4, 8, dtype=F32), bias=z(8, dtype=F32), weights=z(4, 2, dtype=F32)),
         lambda logits, **kw: lib.route_topk(logits, 2, **kw)),
        ("product", dict(x=z(4, 64), weight=z(2, 32, 64), out=z(4, 32)),
         lambda x, weight, out: lib.grouped_linear(x, weight, ends, out=out)),
        ("fp8 product", dict(x_scale=z(4, 1, dtype=F32), weight_scale=z(2, 1, 1, dtype=F32)),
         lambda **kw: lib.grouped_linear(z(4, 128, dtype=FP8), z(2, 128, 128, dtype=FP8), ends, **kw)),
        ("gated", dict(h=z(4, 16), out=z(4, 8)), lambda h, out: lib.gated_rows(h, ends, out=out)),
        ("adapters", dict(base=z(4, 64), x=z(4, 32), down=z(2, 16, 32), up=z(2, 64, 16), scales=z(2, dtype=F32), out=z(4, 64)),
         lambda base, x, down, up, scales, out: lib.adapter_add(base, x, down, up, slots, scales, out=out)),
    ]


CASES = [(i, name) for i, (_, args, _) in enumerate(_calls("cpu")) for name in args]


@pytest.mark.parametrize("i,name", CASES)
def test_refused_with_gradients(i, name):
    _, args, call = _calls("cpu")[i]
    args[name].requires_grad_()
    with pytest.raises(afd.AfdError) as e:
        call(**args)
    assert e.value.status == afd.ERR_UNSUPPORTED and "backward" in str(e.value)


@pytest.mark.gpu
@pytest.mark.parametrize("i,name", CASES)
def test_taken_without(i, name):
    _, args, call = _calls("cuda")[i]
    want = call(**{k: v.clone() for k, v in args.items()})
    args[name].requires_grad_()
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            got = call(**args)
        for a, b in zip(got if isinstance(got, tuple) else [got], want if isinstance(want, tuple) else [want]):
            assert torch.equal(a, b)
    with pytest.raises(afd.AfdError):
        call(**args)
