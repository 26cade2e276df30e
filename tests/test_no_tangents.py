"""The context-free operators have no forward-mode derivative: a dual tensor,
whose tangent the result would lack, is refused, and its primal taken."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import test_expert_no_grad as experts
import test_source_refusals as sources
from combine_attention_ffn_gb300 import afd

CALLS = ([(experts._calls, i, name) for i, (_, args, _) in enumerate(experts._calls("cpu")) for name in args]
         + [(sources._grad_calls, i, name) for i, (args, _) in enumerate(sources._grad_calls("cpu")) for name in args])


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_attention_ffn_gb300 import build

    afd.load_library(build.build())


def _case(calls, i, device):
    *_, args, call = calls(device)[i]
    return args, call


@pytest.mark.parametrize("calls,i,name", CALLS)
def test_dual_tensors_are_refused(calls, i, name):
    args, call = _case(calls, i, "cpu")
    for mode in (torch.enable_grad, torch.no_grad):
        with mode(), fw.dual_level():
            with pytest.raises(afd.AfdError) as e:
                call(**{**args, name: fw.make_dual(args[name], torch.ones_like(args[name]))})
        assert e.value.status == afd.ERR_UNSUPPORTED and "forward-mode" in str(e.value)


@pytest.mark.gpu
@pytest.mark.parametrize("calls,i,name", CALLS)
def test_plain_tensors_are_taken_inside_a_dual_level(calls, i, name):
    args, call = _case(calls, i, "cuda")
    with fw.dual_level():
        dual = fw.make_dual(args[name], torch.ones_like(args[name]))
        call(**args)
        call(**{**args, name: fw.unpack_dual(dual).primal})
    call(**args)
