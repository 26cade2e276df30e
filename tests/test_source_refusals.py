"""Refusals of the source-side operators that the library makes on the host
before any CUDA call, through the C ABI and the binding, and what the binding
refuses by itself (these run without a GPU)."""
import ctypes

import pytest
import torch

import combine_attention_ffn_gb300 as pkg
from combine_attention_ffn_gb300 import afd

P, ODD, OFF8 = ctypes.c_void_p(4096), ctypes.c_void_p(4097), ctypes.c_void_p(4104)
BF16, F32, FP8, I32, I64 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32, torch.int64


@pytest.fixture(scope="module")
def lib():
    from combine_attention_ffn_gb300 import build

    return afd.load_library(build.build())


def _norm(lib, **over):
    a = dict(x=P, x_stride=256, res=P, res_stride=256, weight=P, eps=1e-6, T=4, H=256, res_out=P, res_out_stride=256,
             out=P, out_stride=256, fp8=P, scale=P)
    a.update(over)
    return lib.afd_norm_rows(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), afd.ERR_ARG), (dict(H=0), afd.ERR_ARG), (dict(x_stride=255), afd.ERR_ARG), (dict(res_stride=255), afd.ERR_ARG),
    (dict(res_out_stride=255), afd.ERR_ARG), (dict(out_stride=255), afd.ERR_ARG), (dict(eps=-1.0), afd.ERR_ARG),
    (dict(eps=float("nan")), afd.ERR_ARG), (dict(scale=None), afd.ERR_ARG), (dict(fp8=None), afd.ERR_ARG),
    (dict(res=None), afd.ERR_ARG), (dict(x=None), afd.ERR_ARG), (dict(weight=None), afd.ERR_ARG),
    (dict(res_out=None, out=None, fp8=None, scale=None), afd.ERR_ARG), (dict(x=ODD), afd.ERR_ARG), (dict(out=ODD), afd.ERR_ARG),
    (dict(scale=ctypes.c_void_p(4098)), afd.ERR_ARG), (dict(H=192), afd.ERR_UNSUPPORTED),
    (dict(x=OFF8), afd.ERR_UNSUPPORTED), (dict(weight=OFF8), afd.ERR_UNSUPPORTED), (dict(x_stride=260), afd.ERR_UNSUPPORTED),
    (dict(fp8=ctypes.c_void_p(4100)), afd.ERR_UNSUPPORTED), (dict(T=(1 << 31) - (1 << 20)), afd.ERR_UNSUPPORTED),
    (dict(H=32896, x_stride=32896, res_stride=32896, res_out_stride=32896, out_stride=32896), afd.ERR_UNSUPPORTED),
    (dict(H=(1 << 24) + 1, x_stride=1 << 25, res=None, res_out=None, out_stride=1 << 25, fp8=None, scale=None), afd.ERR_UNSUPPORTED),
    (dict(T=0, x=None, weight=None), afd.OK)])
def test_norm(lib, over, status):
    assert _norm(lib, **over) == status


def _descriptor(**over):
    a = dict(k=P, v=P, k_scale=None, v_scale=None, k_page_stride=4096, v_page_stride=4096, num_pages=4, page_size=16,
             num_kv_heads=2, head_dim=128, dtype=afd.BF16)
    a.update(over)
    return afd.Cache(*a.values())


CACHES = [
    (dict(num_pages=-1), afd.ERR_ARG), (dict(page_size=0), afd.ERR_ARG), (dict(num_kv_heads=0), afd.ERR_ARG),
    (dict(head_dim=0), afd.ERR_ARG), (dict(dtype=afd.FP32), afd.ERR_ARG), (dict(k_scale=P), afd.ERR_ARG),
    (dict(dtype=afd.FP8_E4M3), afd.ERR_ARG), (dict(dtype=afd.FP8_E4M3, k_scale=P), afd.ERR_ARG),
    (dict(dtype=afd.FP8_E4M3, k_scale=P, v_scale=ODD), afd.ERR_ARG), (dict(k=None), afd.ERR_ARG), (dict(v=None), afd.ERR_ARG),
    (dict(k_page_stride=4095), afd.ERR_ARG), (dict(v_page_stride=4088), afd.ERR_ARG), (dict(head_dim=96), afd.ERR_UNSUPPORTED),
    (dict(head_dim=256, k_page_stride=8192, v_page_stride=8192), afd.ERR_UNSUPPORTED), (dict(k_page_stride=4100), afd.ERR_UNSUPPORTED),
    (dict(k=OFF8), afd.ERR_UNSUPPORTED), (dict(v=OFF8), afd.ERR_UNSUPPORTED),
    (dict(num_kv_heads=1025, k_page_stride=1 << 22, v_page_stride=1 << 22), afd.ERR_UNSUPPORTED),
    (dict(num_pages=1 << 27), afd.ERR_UNSUPPORTED)]


def _write(lib, cache=None, **over):
    a = dict(q=P, q_stride=1024, k=P, k_stride=256, v=P, v_stride=256, positions=P, slots=P, inv_freq=P, pairs=64,
             interleaved=0, factor=1.0, T=4, Hq=8)
    b = dict(q_out=P, q_out_stride=1024)
    a.update({k: v for k, v in over.items() if k in a})
    b.update({k: v for k, v in over.items() if k in b})
    return lib.afd_cache_write(*a.values(), cache if cache is not None else _descriptor(), *b.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), afd.ERR_ARG), (dict(Hq=-1), afd.ERR_ARG), (dict(pairs=-1), afd.ERR_ARG), (dict(pairs=65), afd.ERR_ARG),
    (dict(interleaved=2), afd.ERR_ARG), (dict(q_stride=1023), afd.ERR_ARG), (dict(q_out_stride=1016), afd.ERR_ARG),
    (dict(k_stride=255), afd.ERR_ARG), (dict(v_stride=248), afd.ERR_ARG), (dict(q=None), afd.ERR_ARG), (dict(q_out=None), afd.ERR_ARG),
    (dict(k=None), afd.ERR_ARG), (dict(v=None), afd.ERR_ARG), (dict(slots=None), afd.ERR_ARG), (dict(positions=None), afd.ERR_ARG),
    (dict(inv_freq=None), afd.ERR_ARG), (dict(slots=ctypes.c_void_p(4100)), afd.ERR_ARG), (dict(inv_freq=ODD), afd.ERR_ARG),
    (dict(q_stride=1028), afd.ERR_UNSUPPORTED), (dict(k_stride=260), afd.ERR_UNSUPPORTED), (dict(q=OFF8), afd.ERR_UNSUPPORTED),
    (dict(v=OFF8), afd.ERR_UNSUPPORTED), (dict(q_out=OFF8), afd.ERR_UNSUPPORTED), (dict(T=(1 << 31) - (1 << 20)), afd.ERR_UNSUPPORTED),
    (dict(Hq=1025, q_stride=1 << 18, q_out_stride=1 << 18), afd.ERR_UNSUPPORTED),
    (dict(T=0, q=None, k=None, v=None, slots=None, positions=None, inv_freq=None, q_out=None), afd.OK)])
def test_write(lib, over, status):
    assert _write(lib, **over) == status


@pytest.mark.parametrize("over,status", CACHES)
def test_caches(lib, over, status):
    assert _write(lib, _descriptor(**over)) == status
    assert _attend(lib, _descriptor(**over)) == status


def _attend(lib, cache=None, **over):
    a = dict(q=P, q_stride=1024)
    b = dict(table=P, table_stride=100, max_pages=100, lengths=P, B=4, Hq=8, scale=0.1, window=0, out=P, out_stride=1024,
             lse=P, ws=P, ws_bytes=1 << 40)
    a.update({k: v for k, v in over.items() if k in a})
    b.update({k: v for k, v in over.items() if k in b})
    return lib.afd_decode_attention(*a.values(), cache if cache is not None else _descriptor(), *b.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), afd.ERR_ARG), (dict(Hq=0), afd.ERR_ARG), (dict(Hq=7), afd.ERR_ARG), (dict(max_pages=-1), afd.ERR_ARG),
    (dict(window=-1), afd.ERR_ARG), (dict(q_stride=1016), afd.ERR_ARG), (dict(out_stride=1016), afd.ERR_ARG),
    (dict(table_stride=99), afd.ERR_ARG), (dict(q=None), afd.ERR_ARG), (dict(out=None), afd.ERR_ARG), (dict(lengths=None), afd.ERR_ARG),
    (dict(table=None), afd.ERR_ARG), (dict(ws=None), afd.ERR_ARG), (dict(ws_bytes=1000), afd.ERR_ARG), (dict(ws=OFF8), afd.ERR_ARG),
    (dict(lse=ODD), afd.ERR_ARG), (dict(lengths=ODD), afd.ERR_ARG), (dict(table=ODD), afd.ERR_ARG),
    (dict(Hq=1026, q_stride=1 << 18, out_stride=1 << 18), afd.ERR_UNSUPPORTED), (dict(q=OFF8), afd.ERR_UNSUPPORTED),
    (dict(out=OFF8), afd.ERR_UNSUPPORTED), (dict(q_stride=1028), afd.ERR_UNSUPPORTED),
    (dict(max_pages=1 << 27, table_stride=1 << 27), afd.ERR_UNSUPPORTED), (dict(B=1 << 30), afd.ERR_UNSUPPORTED),
    (dict(B=0, q=None, out=None, lengths=None, table=None, ws=None, ws_bytes=0), afd.OK)])
def test_attention(lib, over, status):
    assert _attend(lib, **over) == status


def test_attention_workspace(lib):
    """A size that does not depend on the lengths; none where a block does for
    each sequence and KV head, however long it is."""
    size = lib.afd_decode_workspace_bytes
    for B, Hq, Hkv, D, pages, page in ((1, 8, 8, 128, 8, 16), (64, 64, 4, 64, 1000, 64), (1, 40, 1, 128, 1 << 26, 1)):
        assert size(B, Hq, Hkv, D, 8 * pages, page) == size(B, Hq, Hkv, D, 16 * pages, page) > 0
    assert size(1, 1, 1, 128, 1, 16) == size(1, 64, 4, 128, 48, 16) == size(148, 8, 1, 64, 6, 256) == 0
    assert size(1, 64, 4, 128, 49, 16) > 0 and size(149, 8, 1, 64, 6, 256) > 0 and size(1, 256, 8, 64, 7, 256) > 0
    assert size(0, 8, 8, 128, 8, 16) == 0 and size(4, 8, 8, 128, 0, 16) == 0
    for bad in ((-1, 8, 8, 128, 8, 16), (1, 8, 3, 128, 8, 16), (1, 0, 1, 128, 8, 16), (1, 8, 0, 128, 8, 16), (1, 8, 8, 96, 8, 16),
                (1, 8, 8, 128, -1, 16), (1, 8, 8, 128, 8, 0)):
        assert size(*bad) == -1


def z(*s, dtype=BF16):
    return torch.zeros(*s, dtype=dtype)


def _binding_calls():
    k, v = z(4, 2, 16, 64), z(4, 2, 16, 64)
    k8, ks = k.to(FP8), z(4, 2, 16, dtype=F32)
    t, n = z(3, 5, dtype=I32), z(3, dtype=I32)
    q, pos, slots, freq = z(3, 4, 64), z(3, dtype=I64), z(3, dtype=I64), z(32, dtype=F32)
    kv = z(3, 2, 64)
    attend, write = pkg.decode_attention, pkg.cache_write
    return [
        lambda: pkg.norm_rows(z(4, 8, dtype=F32), z(8)), lambda: pkg.norm_rows(z(4, 8), z(8, dtype=F32)),
        lambda: pkg.norm_rows(z(4, 8), z(7)), lambda: pkg.norm_rows(z(8), z(8)), lambda: pkg.norm_rows(z(4, 8), z(8), residual=z(4, 9)),
        lambda: pkg.norm_rows(z(4, 8), z(8), residual_out=z(4, 8)), lambda: pkg.norm_rows(z(4, 8), z(8), fp8=True),
        lambda: pkg.norm_rows(z(8, 4).t(), z(8)), lambda: pkg.norm_rows(z(4, 128), z(128), fp8_out=z(4, 128)),
        lambda: pkg.norm_rows(z(4, 128), z(128), scale_out=z(4, 2, dtype=F32)), lambda: pkg.norm_rows(z(4, 8), z(8), out=z(3, 8)),
        lambda: attend(q, k, z(4, 2, 16, 128), t, n), lambda: attend(q, k.float(), v.float(), t, n),
        lambda: attend(q, k8, v.to(FP8), t, n), lambda: attend(q, k8, v.to(FP8), t, n, k_scale=ks, v_scale=z(4, 2, 15, dtype=F32)),
        lambda: attend(q, k, v, t, n, k_scale=ks, v_scale=ks), lambda: attend(q, k.transpose(1, 2), v.transpose(1, 2), t, n),
        lambda: attend(z(3, 4, 128), k, v, t, n), lambda: attend(z(3, 256), k, v, t, n), lambda: attend(q, k, v, t.long(), n),
        lambda: attend(q, k, v, t, n.long()), lambda: attend(q, k, v, t, z(2, dtype=I32)), lambda: attend(q, k, v, z(2, 5, dtype=I32), n),
        lambda: attend(q, k, v, t, n, out=z(3, 5, 64)), lambda: attend(q, k, v, t, n, lse=z(3, 4)),
        lambda: attend(z(4, 3, 64).transpose(0, 1), k, v, t, n),
        lambda: write(q, kv, kv, pos.int(), slots, k, v, inv_freq=freq), lambda: write(q, kv, kv, pos, slots.int(), k, v, inv_freq=freq),
        lambda: write(q, kv, kv, pos, slots, k, v, inv_freq=freq.double()), lambda: write(q, kv, kv, None, slots, k, v, inv_freq=freq),
        lambda: write(q, z(3, 3, 64), kv, pos, slots, k, v), lambda: write(q, kv, z(2, 2, 64), pos, slots, k, v),
        lambda: write(q, kv, kv, pos, slots, k, v, q_out=z(3, 5, 64)), lambda: write(None, kv, kv, pos, slots, k, v, q_out=q),
        lambda: write(z(2, 4, 64), kv, kv, pos, slots, k, v), lambda: write(q, kv, kv, pos, slots, k8, v.to(FP8)),
        lambda: write(q, kv, kv, pos, z(2, dtype=I64), k, v),
    ]


@pytest.mark.parametrize("i", range(len(_binding_calls())))
def test_binding_refuses_wrong_types_and_shapes(lib, i):
    with pytest.raises(afd.AfdError) as e:
        _binding_calls()[i]()
    assert e.value.status == afd.ERR_ARG


def test_binding_refuses_sizes_beyond_32_bits(lib):
    """Views without memory behind them: sizes that ctypes would cut off."""
    big = 1 << 32
    wide = z(1).expand(1, big)
    k = z(1, 1, 1, 1).expand(1, 1, big, 64)
    q, t, n = z(1, 4, 64), z(1, 5, dtype=I32), z(1, dtype=I32)
    small = z(1, 1, 16, 64)
    for call in (lambda: pkg.norm_rows(wide, z(1).expand(big)), lambda: pkg.decode_attention(q, k, k, t, n),
                 lambda: pkg.decode_attention(q, small, small, t, n, window=big),
                 lambda: pkg.decode_attention(q, small, small, z(1, dtype=I32).expand(1, big), n),
                 lambda: pkg.cache_write(None, z(1, big, 1).expand(1, big, 64), small[0], None, z(1, dtype=I64), k, k)):
        with pytest.raises(afd.AfdError) as e:
            call()
        assert e.value.status == afd.ERR_UNSUPPORTED


def _grad_calls(device):
    """(arguments that may carry gradients, call)"""
    def zd(*s, dtype=BF16):
        return torch.zeros(*s, dtype=dtype, device=device)

    t, n, slots = zd(3, 5, dtype=I32), zd(3, dtype=I32), torch.arange(3, device=device)
    k, v = zd(4, 2, 16, 64), zd(4, 2, 16, 64)
    return [
        (dict(x=zd(3, 64), weight=zd(64), residual=zd(3, 64), out=zd(3, 64), residual_out=zd(3, 64)),
         lambda x, weight, **kw: pkg.norm_rows(x, weight, **kw)),
        (dict(x=zd(3, 128), weight=zd(128), scale_out=zd(3, 1, dtype=F32)),
         lambda x, weight, **kw: pkg.norm_rows(x, weight, fp8=True, **kw)),
        (dict(q=zd(3, 4, 64), k=zd(3, 2, 64), v=zd(3, 2, 64), inv_freq=zd(32, dtype=F32), k_cache=k, v_cache=v, q_out=zd(3, 4, 64)),
         lambda q, k, v, inv_freq, k_cache, v_cache, q_out: pkg.cache_write(q, k, v, slots, slots, k_cache, v_cache, inv_freq=inv_freq,
                                                                            q_out=q_out)),
        (dict(q=zd(3, 4, 64), k_cache=k, v_cache=v, out=zd(3, 4, 64), lse=zd(3, 4, dtype=F32)),
         lambda q, k_cache, v_cache, out, lse: pkg.decode_attention(q, k_cache, v_cache, t, n, out=out, lse=lse)),
        (dict(k_scale=zd(4, 2, 16, dtype=F32), v_scale=zd(4, 2, 16, dtype=F32)),
         lambda k_scale, v_scale: pkg.decode_attention(zd(3, 4, 64), k.to(FP8), v.to(FP8), t, n, k_scale=k_scale, v_scale=v_scale)),
    ]


GRADS = [(i, name) for i, (args, _) in enumerate(_grad_calls("cpu")) for name in args]


@pytest.mark.parametrize("i,name", GRADS)
def test_refused_with_gradients(lib, i, name):
    args, call = _grad_calls("cpu")[i]
    args[name].requires_grad_()
    with pytest.raises(afd.AfdError) as e:
        call(**args)
    assert e.value.status == afd.ERR_UNSUPPORTED and "backward" in str(e.value)


@pytest.mark.gpu
@pytest.mark.parametrize("i,name", GRADS)
def test_taken_without(lib, i, name):
    args, call = _grad_calls("cuda")[i]
    args[name].requires_grad_()
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            call(**args)
    with pytest.raises(afd.AfdError):
        call(**args)
