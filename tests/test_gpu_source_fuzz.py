"""Drawn cases of the source-side operators against float64 values: sizes, head
layouts, pages, windows, strides and padding in combinations that no hand-written
test makes."""
import random

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


def _every(n):
    return torch.ones(n, dtype=torch.bool, device="cuda")


def _attention_case(rng, g):
    D, fp8 = rng.choice([64, 128]), rng.random() < 0.5
    Hkv, G = rng.choice([1, 1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 5, 8, 9, 12, 16, 20])
    B = int(2 ** rng.uniform(0, 9.5))
    most = int(2 ** rng.uniform(0, min(14, 20 - B.bit_length())))
    shape = rng.choice(["even", "any", "few long"])
    lengths = [most if shape == "even" else rng.randint(0, most) if shape == "any" or rng.random() < 0.1 else rng.randint(0, 20)
               for _ in range(B)]
    page = rng.choice([1, 2, 7, 8, 16, 16, 24, 32, 48, 64, 128, 256])
    window = rng.choice([0, 0, rng.randint(1, most + 5)])
    return sh.paged(lengths, page, Hkv, D, fp8, g), Hkv * G, D, window


@pytest.mark.parametrize("seed", range(30))
def test_attention(seed):
    rng, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
    (k, v, ks, vs, table, lengths), Hq, D, window = _attention_case(rng, g)
    B = len(lengths)
    q = (torch.randn(B, Hq + rng.choice([0, 2]), D, generator=g, device="cuda") * rng.choice([0.5, 2, 8])).to(BF16)[:, :Hq]
    out, lse = lib.decode_attention(q, k, v, table, lengths, window=window, k_scale=ks, v_scale=vs, return_lse=True)
    want, want_lse, err, lse_err = sh.attention(q, k, v, table, lengths, D ** -0.5, window, ks, vs)
    eh.check_bf16(out.view(B * Hq, D), want.view(B * Hq, D), err.view(B * Hq, D), _every(B * Hq))
    sh.check_lse(lse, want_lse, lse_err)
    again = lib.decode_attention(q, k, v, table, lengths, window=window, k_scale=ks, v_scale=vs)
    assert torch.equal(again, out)


@pytest.mark.parametrize("seed", range(30))
def test_write(seed):
    rng, g = random.Random(1000 + seed), torch.Generator(device="cuda").manual_seed(seed)
    D, fp8, interleaved = rng.choice([64, 128]), rng.random() < 0.5, rng.random() < 0.5
    Hkv, Hq, page = rng.choice([1, 2, 3, 8]), rng.randint(0, 70), rng.choice([1, 5, 16, 64])
    T, R, factor = int(2 ** rng.uniform(0, 11)), rng.choice([0, rng.randint(1, D // 2), D // 4, D // 2]), rng.choice([1.0, 0.5, 1.25])
    pages = -(-T // page) + 2
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D + 8, generator=g, device="cuda").to(BF16)
    q, k, v, _ = qkv.split([Hq * D, Hkv * D, Hkv * D, 8], 1)
    q, k, v = q.unflatten(1, (Hq, D)) if Hq else None, k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))
    positions = torch.randint(0, rng.choice([10, 5000, 1 << 22]), (T,), generator=g, device="cuda")
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    slots[torch.rand(T, generator=g, device="cuda") < 0.2] = rng.choice([-1, pages * page, 1 << 40])
    inv_freq = (10000.0 ** (-torch.arange(R, device="cuda").double() / R)).float() if R else None
    caches = [torch.randn(pages, Hkv, page, D, generator=g, device="cuda").to(FP8 if fp8 else BF16) for _ in range(2)]
    scales = [torch.rand(pages, Hkv, page, generator=g, device="cuda") if fp8 else None for _ in range(2)]
    before = [c.clone() for c in caches]
    got = lib.cache_write(q, k, v, positions, slots, *caches, inv_freq=inv_freq, interleaved=interleaved, factor=factor,
                          k_scale=scales[0], v_scale=scales[1])
    if Hq:
        want, err = sh.rotate(q, positions, inv_freq, interleaved, factor)
        eh.check_bf16(got, want, err, _every(T))
    live = (slots >= 0) & (slots < pages * page)
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[slots[live]] = False
    for t, cache, scale, old, f in ((k, caches[0], scales[0], before[0], inv_freq), (v, caches[1], scales[1], before[1], None)):
        want, err = sh.rotate(t, positions, f, interleaved, factor if f is not None else 1.0)
        flat, old = (c.transpose(1, 2).flatten(0, 1) for c in (cache, old))
        if fp8:
            sh.check_e4m3(flat[slots[live]], scale.transpose(1, 2).flatten(0, 1)[slots[live]], want[live], err[live])
        else:
            eh.check_bf16(flat[slots[live]], want[live], err[live], _every(int(live.sum())))
        assert torch.equal(flat[rest].view(torch.uint8), old[rest].view(torch.uint8))


@pytest.mark.parametrize("seed", range(30))
def test_norm(seed):
    rng, g = random.Random(2000 + seed), torch.Generator(device="cuda").manual_seed(seed)
    fp8 = rng.random() < 0.5
    T, H = int(2 ** rng.uniform(0, 10)), 128 * rng.randint(1, 64) if fp8 else int(2 ** rng.uniform(0, 14))
    pad = rng.choice([0, 0, 8, 3 if not fp8 else 8])
    x = torch.randn(T, H + pad, generator=g, device="cuda").to(BF16)[:, :H]
    res = (torch.randn(T, H + pad, generator=g, device="cuda") * 4).to(BF16)[:, :H] if rng.random() < 0.7 else None
    w = torch.randn(H, generator=g, device="cuda").to(BF16)
    got = lib.norm_rows(x, w, residual=res, fp8=fp8, eps=1e-5)
    r, y, err = sh.norm(x, res, w, 1e-5, 64 if H % 8 == 0 and pad % 8 == 0 else H // 256 + 1)
    eh.check_bf16(got.rows, y, err, _every(T))
    if res is not None:
        eh.check_bf16(got.residual, r, sh.FP32_HALF * r.abs(), _every(T))
    if fp8:
        sh.check_e4m3(got.fp8_rows.view(T, -1, 128), got.scales, y.view(T, -1, 128), err.view(T, -1, 128))


def test_most_heads_and_no_sequences():
    """1,024 query heads, 3,000 sequences, none."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for lengths, Hkv, Hq in (([40, 3], 64, 1024), ([(i * 13) % 50 for i in range(3000)], 1, 2), ([], 2, 4)):
        k, v, ks, vs, table, n = sh.paged(lengths, 16, Hkv, 64, True, g)
        q = torch.randn(len(lengths), Hq, 64, generator=g, device="cuda").to(BF16)
        out, lse = lib.decode_attention(q, k, v, table, n, k_scale=ks, v_scale=vs, return_lse=True)
        assert out.shape == q.shape and lse.shape == q.shape[:2]
        if lengths:
            want, want_lse, err, lse_err = sh.attention(q, k, v, table, n, 0.125, 0, ks, vs)
            eh.check_bf16(out.flatten(0, 1), want.flatten(0, 1), err.flatten(0, 1), _every(out.shape[0] * Hq))
            sh.check_lse(lse, want_lse, lse_err)


def test_calls_of_unlike_shapes_side_by_side():
    """Calls on several streams at once, each with its own workspace, give what they give alone."""
    g = torch.Generator(device="cuda").manual_seed(2)
    rng = random.Random(3)
    calls = []
    for _ in range(6):
        (k, v, ks, vs, table, lengths), Hq, D, window = _attention_case(rng, g)
        q = torch.randn(len(lengths), Hq, D, generator=g, device="cuda").to(BF16)
        calls.append(lambda q=q, k=k, v=v, ks=ks, vs=vs, t=table, n=lengths, w=window, **kw:
                     lib.decode_attention(q, k, v, t, n, window=w, k_scale=ks, v_scale=vs, **kw))
    want = [call() for call in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[call(stream=s) for call, s in zip(calls, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for row in got:
        for a, b in zip(row, want):
            assert torch.equal(a, b)
