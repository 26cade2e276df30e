"""route_topk with a bias where FP32 cannot order the keys: the selection is
that of 64-bit keys, ties to the lowest index, also where equal experts stand
between the last slot and a better one, and where an expert with a large score
hides behind one with a small score."""
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


def _check(logits, bias, K, scoring, **kw):
    ids, w = lib.route_topk(logits.cuda(), K, scoring=scoring, bias=bias.cuda(), **kw)
    want_ids, want_w = eh.route_reference(logits, K, scoring=scoring, bias=bias, **kw)
    assert torch.equal(ids.cpu(), want_ids)
    # as in test_gpu_experts.py: exp, a sum, a quotient and two products
    assert ((w.double().cpu() - want_w).abs() <= 2.0 ** -17 * want_w.abs() + 1e-36).all()


def _scores(logits, scoring):
    l = logits.double()
    return torch.softmax(l, -1) if scoring == "softmax" else torch.sigmoid(l)


def test_a_tie_before_a_better_expert():
    """Three keys that round to one FP32 number; the third is the largest."""
    l = torch.tensor([[0.12573022, 0.12573022, 0.64042264]])
    b = torch.tensor([-0.013210487, -0.013210487, -0.13666826])
    assert eh.route_reference(l, 1, scoring="sigmoid", bias=b)[0].item() == 2
    _check(l, b, 1, "sigmoid")


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,distinct", [(3, 1, 2), (8, 1, 3), (12, 4, 3), (64, 8, 5), (64, 8, 40), (200, 10, 4), (1024, 32, 7)])
def test_equal_experts_at_the_last_slot(E, K, distinct, scoring, dtype):
    """Every key is 0.75 up to a few units of FP32; experts come in copies."""
    for seed in range(12):
        g = torch.Generator().manual_seed(1000 * seed + E + K)
        of = torch.randint(0, distinct, (E,), generator=g)
        values = (torch.randn(distinct, generator=g) * 0.7).to(dtype)
        l = values[of].view(1, E)
        s = _scores(l, scoring)
        nudge = torch.randint(-1, 2, (distinct,), generator=g)[of].double() * 2.0 ** -25
        b = (0.75 + nudge - s[0]).float()
        assert all(len(set(b[of == i].tolist())) <= 1 for i in range(distinct))
        _check(l.expand(3, E).contiguous(), b, K, scoring)
        _check(l, b, K, scoring, renormalize=False, scale=1.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(6, 1), (64, 4), (256, 8)])
def test_large_scores_behind_small_ones(E, K, scoring):
    """Keys around 0.01 of scores between 1e-6 and 0.9: what FP32 makes of a
    large score is off by more than the gap of two small ones'."""
    for seed in range(25):
        g = torch.Generator().manual_seed(seed)
        l = torch.randn(1, E, generator=g) * 3 - (4 if scoring == "sigmoid" else 0)
        s = _scores(l, scoring)
        b = (0.01 + torch.randn(E, generator=g).double() * 2e-8 - s[0]).float()
        _check(l.expand(3, E).contiguous(), b, K, scoring)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(128, 8), (1024, 32), (40, 32)])
def test_all_experts_equal(E, K, scoring):
    """A fresh router: no logit and no bias stands out; also groups of equal ones."""
    _check(torch.zeros(3, E), torch.zeros(E), K, scoring)
    _check(torch.full((3, E), -2.5), torch.full((E,), 0.125), K, scoring)
    _check((torch.arange(E) % 3).float().view(1, E), torch.zeros(E), K, scoring)
    l = torch.zeros(2, E)
    l[:, E // 2] = 1e-7  # one that FP32 barely tells apart
    _check(l, torch.zeros(E), K, scoring)
