"""Refusals of the expert operators that the library makes on the host before
any CUDA call, through the C ABI and the binding (these run without a GPU)."""
import ctypes

import pytest
import torch

import combine_attention_ffn_gb300 as pkg
from combine_attention_ffn_gb300 import afd

P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    from combine_attention_ffn_gb300 import build

    return afd.load_library(build.build())


def _route(lib, **over):
    a = dict(logits=P, dtype=afd.FP32, stride=64, bias=None, live=None, T=4, E=64, K=8, scoring=0, renorm=1,
             scale=1.0, ids=P, weights=P)
    a.update(over)
    return lib.afd_route_topk(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), afd.ERR_ARG), (dict(K=0), afd.ERR_ARG), (dict(K=65), afd.ERR_ARG), (dict(K=33), afd.ERR_ARG),
    (dict(E=0, K=1), afd.ERR_ARG), (dict(stride=63), afd.ERR_ARG), (dict(logits=None), afd.ERR_ARG),
    (dict(ids=None), afd.ERR_ARG), (dict(weights=None), afd.ERR_ARG), (dict(dtype=afd.FP8_E4M3), afd.ERR_ARG),
    (dict(scoring=2), afd.ERR_ARG), (dict(renorm=2), afd.ERR_ARG), (dict(E=1025, stride=1025), afd.ERR_UNSUPPORTED),
    (dict(T=(1 << 31) - (1 << 20)), afd.ERR_UNSUPPORTED),
    (dict(T=0, logits=None, ids=None, weights=None), afd.OK)])
def test_router(lib, over, status):
    assert _route(lib, **over) == status


def _grouped(lib, **over):
    a = dict(x=P, x_stride=256, x_scale=None, w=P, w_scale=None, ends=P, G=4, alpha=1, R=16, K=256, N=128,
             dtype=afd.BF16, gated=0, out=P, out_stride=128, error=None)
    a.update(over)
    return lib.afd_grouped_linear(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=afd.FP32), afd.ERR_ARG), (dict(G=0), afd.ERR_ARG), (dict(alpha=0), afd.ERR_ARG),
    (dict(R=-1), afd.ERR_ARG), (dict(K=0, x_stride=0), afd.ERR_ARG), (dict(N=0), afd.ERR_ARG), (dict(gated=2), afd.ERR_ARG),
    (dict(x_stride=255), afd.ERR_ARG), (dict(out_stride=127), afd.ERR_ARG), (dict(x=None), afd.ERR_ARG),
    (dict(w=None), afd.ERR_ARG), (dict(ends=None), afd.ERR_ARG), (dict(out=None), afd.ERR_ARG),
    (dict(x_scale=P), afd.ERR_ARG), (dict(w_scale=P), afd.ERR_ARG), (dict(dtype=afd.FP8_E4M3), afd.ERR_ARG),
    (dict(G=1025), afd.ERR_UNSUPPORTED), (dict(R=(1 << 31) - (1 << 20) - 1), afd.ERR_UNSUPPORTED),
    (dict(alpha=(1 << 31) - 1), afd.ERR_UNSUPPORTED), (dict(K=252), afd.ERR_UNSUPPORTED),
    (dict(x_stride=260), afd.ERR_UNSUPPORTED),
    (dict(dtype=afd.FP8_E4M3, x_scale=P, w_scale=P, K=192), afd.ERR_UNSUPPORTED),
    (dict(dtype=afd.FP8_E4M3, x_scale=P, w_scale=P, N=64), afd.ERR_UNSUPPORTED),
    (dict(N=1 << 24, out_stride=1 << 24, R=1 << 30), afd.ERR_UNSUPPORTED), (dict(N=(1 << 24) + 1, out_stride=1 << 25), afd.ERR_UNSUPPORTED),
    (dict(x=ctypes.c_void_p(4104)), afd.ERR_UNSUPPORTED), (dict(w=ctypes.c_void_p(4104)), afd.ERR_UNSUPPORTED),
    (dict(ends=ctypes.c_void_p(4098)), afd.ERR_ARG), (dict(out=ctypes.c_void_p(4097)), afd.ERR_ARG),
    (dict(R=0, x=None, out=None), afd.OK)])
def test_grouped(lib, over, status):
    assert _grouped(lib, **over) == status


def _gated(lib, **over):
    a = dict(h=P, h_stride=64, ends=P, G=4, alpha=1, R=16, N=32, out=P, out_stride=32)
    a.update(over)
    return lib.afd_gated_rows(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(G=0), afd.ERR_ARG), (dict(alpha=0), afd.ERR_ARG), (dict(R=-1), afd.ERR_ARG), (dict(N=0), afd.ERR_ARG),
    (dict(ends=None), afd.ERR_ARG), (dict(h=None), afd.ERR_ARG), (dict(out=None), afd.ERR_ARG),
    (dict(h_stride=63), afd.ERR_ARG), (dict(out_stride=31), afd.ERR_ARG), (dict(G=1025), afd.ERR_UNSUPPORTED),
    (dict(R=(1 << 31) - (1 << 20) - 1), afd.ERR_UNSUPPORTED), (dict(alpha=(1 << 31) - 1), afd.ERR_UNSUPPORTED),
    (dict(N=(1 << 24) + 1, h_stride=1 << 26, out_stride=1 << 25), afd.ERR_UNSUPPORTED),
    (dict(R=0, h=None, out=None), afd.OK)])
def test_gated_rows(lib, over, status):
    assert _gated(lib, **over) == status


def _adapter(lib, **over):
    a = dict(base=P, base_stride=64, x=P, x_stride=128, x_scale=None, down=P, up=P, slots=P, scales=P, row_src=None, ends=None, G=0,
             top_k=1, R=8, tokens=8, S=2, rank=16, K=128, N=64, out=P, out_stride=64, ws=None, ws_bytes=0)
    a.update(over)
    return lib.afd_adapter_add(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(R=-1), afd.ERR_ARG), (dict(S=0), afd.ERR_ARG), (dict(rank=0), afd.ERR_ARG), (dict(K=0), afd.ERR_ARG),
    (dict(N=0), afd.ERR_ARG), (dict(base_stride=56), afd.ERR_ARG), (dict(x_stride=120), afd.ERR_ARG),
    (dict(out_stride=56), afd.ERR_ARG), (dict(tokens=7), afd.ERR_ARG), (dict(row_src=P), afd.ERR_ARG),
    (dict(row_src=P, ends=P, G=1, top_k=0), afd.ERR_ARG), (dict(base=None), afd.ERR_ARG), (dict(x=None), afd.ERR_ARG),
    (dict(down=None), afd.ERR_ARG), (dict(up=None), afd.ERR_ARG), (dict(slots=None), afd.ERR_ARG),
    (dict(scales=None), afd.ERR_ARG), (dict(out=None), afd.ERR_ARG), (dict(rank=24), afd.ERR_UNSUPPORTED),
    (dict(rank=128), afd.ERR_UNSUPPORTED), (dict(K=120), afd.ERR_UNSUPPORTED), (dict(x_scale=P, K=64), afd.ERR_UNSUPPORTED),
    (dict(x_scale=P, x_stride=136), afd.ERR_UNSUPPORTED),
    (dict(N=60, base_stride=60, out_stride=60), afd.ERR_UNSUPPORTED), (dict(base_stride=68), afd.ERR_UNSUPPORTED),
    (dict(R=(1 << 31) - (1 << 20), tokens=(1 << 31) - 1), afd.ERR_UNSUPPORTED),
    (dict(N=(1 << 24) + 8, base_stride=1 << 25, out_stride=1 << 25), afd.ERR_UNSUPPORTED),
    (dict(K=(1 << 24) + 16, x_stride=1 << 25), afd.ERR_UNSUPPORTED),
    (dict(S=1024, ws_bytes=1 << 20), afd.ERR_UNSUPPORTED), (dict(R=1 << 20, tokens=1 << 20, ws=None, ws_bytes=1 << 40), afd.ERR_ARG),
    (dict(R=1 << 20, tokens=1 << 20, ws=P, ws_bytes=1 << 26), afd.ERR_ARG),
    (dict(R=0, base=None, x=None, out=None, ws=None, ws_bytes=0), afd.OK)])
def test_adapters(lib, over, status):
    assert _adapter(lib, **over) == status


def test_adapter_workspace(lib):
    size = lib.afd_adapter_workspace_bytes
    for R, S, rank in ((100_000, 1023, 64), (1 << 28, 5, 64), (65_536, 3, 32)):
        assert size(R, R, 0, S, rank, 2048, 2048) == (R + S + 2 + 3) // 4 * 16 + 4 * R * rank
        assert size(R, 65, 8, S, rank, 2048, 2048) == size(R, R, 0, S, rank, 2048, 2048)
        assert size(R, 16, 8, S, rank, 2048, 2048) == 0  # few rows can be live
    for rows, rank, K, N, few in ((512, 8, 16, 8, True), (513, 8, 16, 8, False), (512, 16, 2048, 2048, True),
                                  (512, 16, 2048, 2560, False), (160, 64, 2048, 2048, True),
                                  (161, 64, 2048, 2048, False), (64, 64, 7168, 2048, True),
                                  (128, 64, 7168, 2048, False), (1, 64, 16, 2 ** 31 - 8, False)):
        assert (size(rows, rows, 0, 4, rank, K, N) == 0) == few
    assert size(0, 0, 0, 1, 8, 16, 8) == 0
    for bad in ((-1, 0, 0, 1, 8, 16, 8), (1, -1, 0, 1, 8, 16, 8), (1, 1, -1, 1, 8, 16, 8), (1, 1, 0, 0, 8, 16, 8),
                (1, 1, 0, 1, 0, 16, 8), (1, 1, 0, 1, 8, 0, 8), (1, 1, 0, 1, 8, 16, 0)):
        assert size(*bad) == -1


def test_binding_refuses_wrong_types_and_shapes(lib):
    bf = torch.bfloat16
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype)
    ends = z(2, dtype=torch.int32)
    calls = [
        lambda: pkg.route_topk(z(4, 8, dtype=torch.float16), 2),
        lambda: pkg.route_topk(z(4, 8), 2, scoring="tanh"),
        lambda: pkg.route_topk(z(4, 8), 2, bias=z(8)),
        lambda: pkg.route_topk(z(4, 8), 2, ids=z(4, 2, dtype=torch.int32)),
        lambda: pkg.route_topk(z(8, 4).t(), 2),
        lambda: pkg.route_topk(z(4, 8), 2, live_tokens=z(1, dtype=torch.int64)),
        lambda: pkg.grouped_linear(z(4, 64), z(2, 32, 128), ends),
        lambda: pkg.grouped_linear(z(4, 64), z(2, 31, 64), ends, gated=True),
        lambda: pkg.grouped_linear(z(4, 64), z(2, 32, 64), ends.long()),
        lambda: pkg.grouped_linear(z(4, 64), z(2, 32, 64, dtype=torch.float32), ends),
        lambda: pkg.grouped_linear(z(4, 64), z(2, 32, 64), ends, x_scale=z(4, 1, dtype=torch.float32)),
        lambda: pkg.grouped_linear(z(4, 128).to(torch.float8_e4m3fn), z(2, 128, 128).to(torch.float8_e4m3fn), ends),
        lambda: pkg.grouped_linear(z(4, 64), z(2, 32, 64), ends, out=z(4, 31)),
        lambda: pkg.grouped_linear(z(4, 64), z(2, 64, 64).transpose(1, 2), ends),
        lambda: pkg.gated_rows(z(4, 7), ends),
        lambda: pkg.gated_rows(z(4, 8), ends, out=z(4, 8)),
        lambda: pkg.adapter_add(z(4, 64), z(4, 128).to(torch.float8_e4m3fn), z(2, 16, 128), z(2, 64, 16), z(4, dtype=torch.int32),
                                z(2, dtype=torch.float32)),
        lambda: pkg.adapter_add(z(4, 64), z(4, 128), z(2, 16, 128), z(2, 64, 16), z(4, dtype=torch.int32),
                                z(2, dtype=torch.float32), x_scale=z(4, 1, dtype=torch.float32)),
        lambda: pkg.adapter_add(z(4, 64), z(4, 32), z(2, 16, 32), z(2, 64, 8), z(4, dtype=torch.int32), z(2, dtype=torch.float32)),
        lambda: pkg.adapter_add(z(4, 64), z(4, 32), z(2, 16, 32), z(2, 64, 16), z(3, dtype=torch.int32), z(2, dtype=torch.float32)),
        lambda: pkg.adapter_add(z(4, 64), z(4, 32), z(2, 16, 32), z(2, 64, 16), z(4, dtype=torch.int32), z(2, dtype=torch.float32),
                                row_src=z(4, dtype=torch.int32)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(afd.AfdError) as e:
            call()
        assert e.value.status == afd.ERR_ARG, i
