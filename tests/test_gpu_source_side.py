"""The source-side operators (afd_norm_rows, afd_cache_write,
afd_decode_attention) against float64 values from their definitions, at the
sizes, layouts and masks where they can go wrong."""
import pytest
import torch

import combine_attention_ffn_gb300 as lib
import expert_harness as eh
import source_harness as sh
from combine_attention_ffn_gb300 import afd

pytestmark = pytest.mark.gpu
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_attention_ffn_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _every(t):
    return torch.ones(t.shape[0], dtype=torch.bool, device=t.device)


# -------------------------------------------------------------------- norm
def _norm_case(T, H, seed, residual=True):
    g = _gen(seed)
    x = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    res = (torch.randn(T, H, generator=g, device="cuda") * 5).to(BF16) if residual else None
    return x, res, (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(BF16)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (1, 8), (5, 136), (2, 2048), (4, 2056), (700, 1000), (33, 4096), (7, 7168),
                                 (2, 8200), (2, 16392), (1, 32768), (1, 32776), (2, 4097)])
def test_norm_bf16(T, H, residual):
    x, res, w = _norm_case(T, H, T + H, residual)
    got = lib.norm_rows(x, w, eps=1e-5, residual=res)
    r, y, err = sh.norm(x, res, w, 1e-5, 64 if H <= 32768 and H % 8 == 0 else H // 256 + 1)
    eh.check_bf16(got.rows, y, err, _every(x))
    assert got.fp8_rows is None and got.scales is None
    if residual:
        eh.check_bf16(got.residual, r, sh.FP32_HALF * r.abs(), _every(x))
    else:
        assert got.residual is None


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("T,H", [(1, 128), (3, 384), (2, 2048), (65, 2176), (33, 4096), (7, 7168), (2, 16384), (1, 32768)])
def test_norm_fp8(T, H, rows):
    x, res, w = _norm_case(T, H, T + H)
    got = lib.norm_rows(x, w, residual=res, rows=rows, fp8=True)
    r, y, err = sh.norm(x, res, w, 1e-6, 64)
    sh.check_e4m3(got.fp8_rows.view(T, -1, 128), got.scales, y.view(T, -1, 128), err.view(T, -1, 128))
    assert got.scales.shape == (T, H // 128)
    if rows:
        eh.check_bf16(got.rows, y, err, _every(x))
        plain = lib.norm_rows(x, w, residual=res)
        assert torch.equal(plain.rows, got.rows) and torch.equal(plain.residual, got.residual)
    else:
        assert got.rows is None


def test_norm_strided_and_unaligned_rows():
    """Columns of wider arrays; an offset of one element takes the path for any alignment."""
    x, res, w = _norm_case(9, 512, 3)
    want = lib.norm_rows(x, w, residual=res)
    for shift in (8, 1):
        wide = [torch.full((9, 600), 3.0, dtype=BF16, device="cuda") for _ in range(4)]
        views = [t[:, shift:shift + 512] for t in wide]
        views[0].copy_(x)
        views[1].copy_(res)
        got = lib.norm_rows(views[0], w, residual=views[1], out=views[2], residual_out=views[3])
        assert got.rows is views[2] and got.residual is views[3]
        _, y, err = sh.norm(x, res, w, 1e-6, 64)
        eh.check_bf16(views[2], y, err, _every(x))
        assert torch.equal(views[3], want.residual)
        for t in wide[2:]:
            assert (t[:, :shift] == 3.0).all() and (t[:, shift + 512:] == 3.0).all()


@pytest.mark.parametrize("H", [1000, 1001, 4096])
def test_norm_in_place(H):
    x, res, w = _norm_case(17, H, 4)
    want = lib.norm_rows(x, w, residual=res)
    x2, res2 = x.clone(), res.clone()
    got = lib.norm_rows(x2, w, residual=res2, residual_out=res2, out=x2)
    assert got.residual is res2 and got.rows is x2
    assert torch.equal(res2, want.residual) and torch.equal(x2, want.rows)
    x2, res2 = x.clone(), res.clone()
    lib.norm_rows(x2, w, residual=res2, residual_out=x2)
    assert torch.equal(x2, want.residual) and torch.equal(res2, res)


def test_norm_extremes():
    """Rows of zeros, of tiny and of large numbers, and infinities and NaN that
    stay in their row."""
    H = 512
    x, _, w = _norm_case(8, H, 5, False)
    x[1] = 0
    x[2] *= 2.0 ** -40
    x[3] *= 2.0 ** 60  # (the sum of squares is about 2^129: not finite in FP32)
    x[4] *= 2.0 ** 50
    x[5, 3] = float("nan")
    x[6, 9] = float("inf")
    x[7, :128] = 0
    got = lib.norm_rows(x, w, fp8=True)
    fine = torch.tensor([0, 1, 2, 4, 7], device="cuda")
    _, y, err = sh.norm(x[fine], None, w, 1e-6, 64)
    eh.check_bf16(got.rows[fine], y, err, _every(fine))
    sh.check_e4m3(got.fp8_rows[fine].view(5, -1, 128), got.scales[fine], y.view(5, -1, 128), err.view(5, -1, 128))
    assert (got.scales[1] == 2.0 ** -100).all() and (got.fp8_rows[1].float() == 0).all()
    assert got.scales[7, 0] == 2.0 ** -100 and got.scales[7, 1] > 1e-4
    decoded = got.fp8_rows.float().view(8, -1, 128) * got.scales[..., None]
    assert torch.isnan(got.rows[5]).all() and torch.isnan(decoded[5]).all()
    assert torch.isnan(got.rows[6, 9]) and (got.rows[6, :9] == 0).all()
    assert torch.isnan(decoded[6, 0]).all() and (decoded[6, 1:] == 0).all()


def test_norm_repeats_on_other_streams_and_in_graphs():
    x, res, w = _norm_case(300, 2048, 6)
    first = lib.norm_rows(x, w, residual=res, fp8=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    others = []
    for s in streams:
        others.append(lib.norm_rows(x, w, residual=res, fp8=True, stream=s))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        captured = lib.norm_rows(x, w, residual=res, fp8=True)
    for t in captured:
        t.view(torch.uint8).zero_()
    g.replay()
    torch.cuda.synchronize()
    for got in others + [captured]:
        for a, b in zip(got, first):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    x.copy_(torch.randn(300, 2048, generator=_gen(7), device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, lib.norm_rows(x, w, residual=res, fp8=True)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------- cache
def _write_case(T, Hq, Hkv, D, page, R, fp8, seed, far=5000, spare=3):
    g = _gen(seed)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(BF16)
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
    pages = -(-max(T, 1) // page) + spare
    s = dict(q=q.unflatten(1, (Hq, D)) if Hq else None, k=k.unflatten(1, (Hkv, D)), v=v.unflatten(1, (Hkv, D)),
             positions=torch.randint(0, far, (T,), generator=g, device="cuda"),
             slots=torch.randperm(pages * page, generator=g, device="cuda")[:T],
             inv_freq=(10000.0 ** (-torch.arange(R, device="cuda").double() / R)).float() if R else None)
    if T > 2:
        s["slots"][1], s["slots"][T // 2 + 1] = -1, pages * page
    for name in ("k", "v"):
        c = torch.randn(pages, Hkv, page, D, generator=g, device="cuda")
        s[name + "_cache"] = c.to(FP8 if fp8 else BF16)
        s[name + "_scale"] = torch.rand(pages, Hkv, page, generator=g, device="cuda") if fp8 else None
    return s


def _write(s, **kw):
    return lib.cache_write(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                           inv_freq=s["inv_freq"], k_scale=s["k_scale"], v_scale=s["v_scale"], **kw)


def _flat(cache):
    """[slots, heads, ...] of [pages, heads, page, ...]"""
    return cache.transpose(1, 2).flatten(0, 1)


def _write_check(s, interleaved=False, factor=1.0, call=None):
    fp8 = s["k_scale"] is not None
    q, k, v = (None if s[n] is None else s[n].clone() for n in "qkv")
    before = {n: s[n].clone() for n in ("k_cache", "v_cache", "k_scale", "v_scale") if s[n] is not None}
    got = (call or (lambda: _write(s, interleaved=interleaved, factor=factor)))()
    if q is not None:
        want, err = sh.rotate(q, s["positions"], s["inv_freq"], interleaved, factor)
        eh.check_bf16(got, want, err, _every(q))
    slots = s["slots"]
    live = (slots >= 0) & (slots < _flat(s["k_cache"]).shape[0])
    for name, t in (("k", k), ("v", v)):
        want, err = (sh.rotate(t, s["positions"], s["inv_freq"], interleaved, factor) if name == "k"
                     else (t.double(), torch.zeros(t.shape, dtype=torch.float64, device="cuda")))
        flat = _flat(s[name + "_cache"])
        if fp8:
            scales = _flat(s[name + "_scale"])
            sh.check_e4m3(flat[slots[live]], scales[slots[live]], want[live], err[live])
        elif name == "v":
            assert torch.equal(flat[slots[live]], t[live])
        else:
            eh.check_bf16(flat[slots[live]], want[live], err[live], _every(slots[live]))
        rest = torch.ones(flat.shape[0], dtype=torch.bool, device="cuda")
        rest[slots[live]] = False
        assert torch.equal(flat[rest].view(torch.uint8), _flat(before[name + "_cache"])[rest].view(torch.uint8))
        if fp8:
            assert torch.equal(scales[rest], _flat(before[name + "_scale"])[rest])
    return got


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 0), (64, 5), (64, 16), (64, 32), (128, 1), (128, 20), (128, 32), (128, 63), (128, 64)])
def test_write_rotary_forms(D, R, interleaved, fp8):
    _write_check(_write_case(9, 4, 2, D, 16, R, fp8, D + R), interleaved, 0.75)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,page", [(1, 32, 4, 128, 16), (1, 1, 1, 64, 1), (2, 0, 3, 64, 24), (5, 7, 1, 128, 7),
                                             (130, 40, 8, 64, 32), (700, 6, 2, 128, 64), (3, 128, 8, 128, 1), (33, 3, 3, 64, 128)])
def test_write_sizes(T, Hq, Hkv, D, page, fp8):
    _write_check(_write_case(T, Hq, Hkv, D, page, D // 2, fp8, T + Hq))


def test_write_far_positions():
    """Angles of positions up to 2^31: 64 bits, where FP32 keeps nothing of them."""
    s = _write_case(64, 2, 1, 128, 16, 64, False, 1)
    s["positions"] = torch.randint(0, 1 << 31, (64,), generator=_gen(2), device="cuda")
    s["positions"][0], s["positions"][1] = 0, (1 << 31) - 1
    _write_check(s)


def test_write_pages_of_one_allocation_and_queries_in_place():
    for fp8 in (False, True):
        s = _write_case(21, 5, 2, 64, 8, 32, fp8, 11)
        pages = s["k_cache"].shape[0]
        both = torch.zeros(pages, 2, 2, 8, 64, dtype=BF16, device="cuda").to(FP8 if fp8 else BF16)
        both[:, 0], both[:, 1] = s["k_cache"], s["v_cache"]
        s["k_cache"], s["v_cache"] = both[:, 0], both[:, 1]
        q = s["q"]
        out = _write_check(s, call=lambda: _write(s, q_out=q))
        assert out is q


def test_write_infinities_and_zeros():
    s = _write_case(6, 1, 2, 64, 16, 0, True, 12)
    s["slots"][:] = torch.arange(6, device="cuda")
    s["k"][0, 0, 3], s["k"][2, 1, 5] = float("inf"), float("nan")
    s["v"][3, 0] = 0
    _write(s)
    k = _flat(s["k_cache"]).float() * _flat(s["k_scale"])[..., None]
    v = _flat(s["v_cache"]).float() * _flat(s["v_scale"])[..., None]
    assert torch.isnan(k[0, 0]).all() and torch.isnan(k[2, 1]).all()
    assert torch.isfinite(k[0, 1]).all() and torch.isfinite(k[2, 0]).all() and torch.isfinite(k[[1, 3, 4, 5]]).all()
    assert (v[3, 0] == 0).all() and _flat(s["v_scale"])[3, 0] == 2.0 ** -100


def test_write_nothing():
    s = _write_case(0, 4, 2, 64, 16, 32, False, 13)
    assert _write(s).shape == (0, 4, 64)
    s = _write_case(4, 4, 2, 64, 16, 32, False, 13)
    for n in ("k_cache", "v_cache"):
        s[n] = s[n][:0]
    want, err = sh.rotate(s["q"], s["positions"], s["inv_freq"], False, 1.0)
    eh.check_bf16(_write(s), want, err, _every(s["q"]))


def test_write_in_a_graph():
    s = _write_case(40, 8, 2, 128, 16, 64, True, 14)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = _write(s)
    s["k"].copy_(torch.randn(40, 2, 128, generator=_gen(3), device="cuda"))
    s["positions"] += 17
    _write_check(s, call=lambda: (g.replay(), out)[1])


# --------------------------------------------------------------- attention
def _attend(case, q, **kw):
    k, v, ks, vs, table, lengths = case
    return lib.decode_attention(q, k, v, table, lengths, k_scale=ks, v_scale=vs, return_lse=True, **kw)


def _attend_check(case, q, window=0, scale=None, **kw):
    k, v, ks, vs, table, lengths = case
    B, Hq, D = q.shape
    if scale is not None:
        kw["scale"] = scale
    out, lse = _attend(case, q, window=window, **kw)
    want, want_lse, err, lse_err = sh.attention(q, k, v, table, lengths, D ** -0.5 if scale is None else scale, window, ks, vs)
    eh.check_bf16(out.reshape(B * Hq, D), want.view(B * Hq, D), err.view(B * Hq, D),
                  torch.ones(B * Hq, dtype=torch.bool, device="cuda"))
    sh.check_lse(lse, want_lse, lse_err)
    empty = want_lse == float("-inf")
    assert (out[empty].view(torch.int16) == 0).all()
    return out, lse


def _queries(B, Hq, D, seed, spread=2.0):
    return (torch.randn(B, Hq, D, generator=_gen(seed), device="cuda") * spread).to(BF16)


LENGTHS = {
    "one": [1],
    "none": [0],
    "padding": [5, 0, 40, 0, 0],
    "tile-edges": [15, 16, 17, 31, 32, 33, 63, 64, 65, 1, 2],
    "long": [5000],
    "long-and-short": [1, 4097, 3, 0, 700, 2],
    "many": [(i * 37) % 150 for i in range(400)],
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", sorted(LENGTHS))
def test_attention_lengths(name, D, fp8):
    lengths = LENGTHS[name]
    case = sh.paged(lengths, 16, 2, D, fp8, _gen(len(name)))
    _attend_check(case, _queries(len(lengths), 10, D, 1))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (3, 1), (2, 7), (1, 8), (2, 9), (4, 16), (1, 17), (1, 40), (8, 3)])
def test_attention_heads(Hkv, G, D, fp8):
    case = sh.paged([70, 1, 300], 24, Hkv, D, fp8, _gen(Hkv + G))
    _attend_check(case, _queries(3, Hkv * G, D, 2))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 5, 16, 24, 64, 128, 1000])
def test_attention_pages(page, fp8):
    case = sh.paged([1, 130, 63, 257], page, 2, 128, fp8, _gen(page))
    _attend_check(case, _queries(4, 16, 128, 3))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 33, 100, 10000])
def test_attention_window(window, fp8):
    case = sh.paged([1, 16, 17, 0, 100, 640, 33], 16, 2, 64, fp8, _gen(window))
    _attend_check(case, _queries(7, 6, 64, 4), window=window)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_does_not_read_before_the_window(fp8):
    case = sh.paged([100], 10, 1, 64, fp8, _gen(5))
    q = _queries(1, 4, 64, 5)
    out, lse = _attend(case, q, window=25)
    k, v, ks, vs, table, _ = case
    for t in (k, v):
        if fp8:
            t.view(torch.uint8)[table[0, :7].long()] = 0x7F
        else:
            t[table[0, :7].long()] = float("nan")
    again, lse2 = _attend(case, q, window=25)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_bad_pages_and_lengths_stay_inside(fp8):
    """Numbers of no page hide their tokens, a length beyond the table ends
    there, a negative one is none."""
    k, v, ks, vs, table, lengths = sh.paged([50, 80, 20, 16], 16, 2, 64, fp8, _gen(6), width=5)
    table[0, 1], table[1, 0], table[3, 0] = -1, 1 << 30, k.shape[0]
    lengths = torch.tensor([50, 1 << 30, -7, 16], dtype=torch.int32, device="cuda")
    case = (k, v, ks, vs, table, lengths)
    out, lse = _attend_check(case, _queries(4, 4, 64, 6))
    assert (lse[2:] == float("-inf")).all()
    for n in (0, 1):  # a cache without pages, a table without any
        got, lse = lib.decode_attention(_queries(4, 4, 64, 6), k[:0] if n == 0 else k, v[:0] if n == 0 else v,
                                        table if n == 0 else table[:, :0], lengths, return_lse=True,
                                        k_scale=None if ks is None else ks[:0] if n == 0 else ks,
                                        v_scale=None if vs is None else vs[:0] if n == 0 else vs)
        assert (got == 0).all() and (lse == float("-inf")).all()


def test_attention_shared_pages():
    """Sequences with a common prefix on the same pages."""
    k, v, ks, vs, table, lengths = sh.paged([160, 170, 161], 16, 2, 128, False, _gen(7))
    table[1, :10] = table[0, :10]
    table[2, :10] = table[0, :10]
    _attend_check((k, v, ks, vs, table, lengths), _queries(3, 16, 128, 7))


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_strided(fp8):
    """Queries and outputs as parts of wider rows, keys and values in one allocation, a table with wider rows."""
    k, v, ks, vs, table, lengths = sh.paged([33, 500, 7], 16, 2, 64, fp8, _gen(8))
    both = torch.stack([k.view(torch.uint8), v.view(torch.uint8)], 1).view(k.dtype)
    wide = torch.full((3, 20), -5, dtype=torch.int32, device="cuda")
    wide = torch.cat([table, wide], 1)[:, :table.shape[1]]
    q = _queries(3, 6, 64, 8)
    qkv = torch.zeros(3, 10, 64, dtype=BF16, device="cuda")
    qkv[:, :6] = q
    outs = torch.full((3, 9, 64), 3.0, dtype=BF16, device="cuda")
    want, _ = _attend_check((k, v, ks, vs, table, lengths), q)
    got = lib.decode_attention(qkv[:, :6], both[:, 0], both[:, 1], wide, lengths, k_scale=ks, v_scale=vs, out=outs[:, 1:7])
    assert torch.equal(got, want) and (outs[:, 0] == 3.0).all() and (outs[:, 7:] == 3.0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("spread,scale", [(40.0, None), (0.0, None), (2.0, -0.5), (1.0, 0.0), (1e-30, 3.0)])
def test_attention_peaked_and_flat(spread, scale, fp8):
    case = sh.paged([600, 40], 16, 2, 128, fp8, _gen(9))
    _attend_check(case, _queries(2, 10, 128, 9, spread), scale=scale)


def test_attention_unlike_value_scales():
    """E4M3 values of very unlike scales, zeros among them: small ones count
    beside large ones of small probability."""
    k, v, ks, vs, table, lengths = sh.paged([200, 64, 33], 16, 2, 128, True, _gen(10))
    vs *= 2.0 ** torch.randint(-60, 10, vs.shape, generator=_gen(11), device="cuda").float()
    vs[table[1, 1].long()] = 0.0
    vs[table[2, 0].long()] = 2.0 ** -100
    vs[table[2, 1].long()] = 2.0 ** -100
    vs[table[2, 2].long()] = 2.0 ** -100
    _attend_check((k, v, ks, vs, table, lengths), _queries(3, 10, 128, 10))
    for t in range(4):  # a head of zero values: zero, with the scores' sum
        vs[table[1, t].long()] = 0.0
    out, lse = _attend_check((k, v, ks, vs, table, lengths), _queries(3, 10, 128, 10))
    assert (out[1] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_nan_and_infinity_stay_in_their_sequence(fp8):
    k, v, ks, vs, table, lengths = sh.paged([40, 41, 300, 301], 16, 2, 64, fp8, _gen(12))
    case, q = (k, v, ks, vs, table, lengths), _queries(4, 6, 64, 12)
    clean, _ = _attend(case, q)
    if fp8:
        ks[table[1, 0].long(), 0, 3] = float("nan")
        vs[table[3, 2].long(), 1, 5] = float("inf")
    else:
        k[table[1, 0].long(), 0, 3, 7] = float("nan")
        v[table[3, 2].long(), 1, 5] = float("inf")
    out, _ = _attend(case, q)
    hit = torch.zeros(4, 6, dtype=torch.bool, device="cuda")
    hit[1, :3], hit[3, 3:] = True, True
    assert torch.equal(out[~hit], clean[~hit])
    assert not torch.isfinite(out[hit]).any()


def test_attention_offsets_past_32_bits():
    """Pages whose byte offsets pass 32 bits, in a cache of 5 GB each."""
    page, D = 64, 128
    pages = 5 * (1 << 30) // (page * D * 2)
    k = torch.zeros(pages, 1, page, D, dtype=BF16, device="cuda")
    v = torch.zeros(pages, 1, page, D, dtype=BF16, device="cuda")
    ids = torch.tensor([pages - 1, 0, pages // 2 + 7, pages - 2], device="cuda")
    for t, seed in ((k, 1), (v, 2)):
        t[ids] = torch.randn(4, 1, page, D, generator=_gen(seed), device="cuda").to(BF16)
    table = ids.int()[None].contiguous()
    case = (k, v, None, None, table, torch.tensor([250], dtype=torch.int32, device="cuda"))
    _attend_check(case, _queries(1, 8, D, 13))
    s = dict(q=None, k=torch.randn(1, 1, D, generator=_gen(3), device="cuda").to(BF16),
             v=torch.randn(1, 1, D, generator=_gen(4), device="cuda").to(BF16), positions=None,
             slots=torch.tensor([(pages - 1) * page + 5], device="cuda"), inv_freq=None, k_cache=k, v_cache=v,
             k_scale=None, v_scale=None)
    assert _write(s) is None
    assert torch.equal(k[-1, 0, 5], s["k"][0, 0]) and torch.equal(v[-1, 0, 5], s["v"][0, 0])
    _attend_check(case, _queries(1, 8, D, 13))


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_repeats_on_other_streams_and_in_graphs(fp8):
    """The same call twice, on two streams at once and replayed from two graphs
    at once gives the same bits; a replay takes new lengths and queries."""
    lengths = [900, 0, 3, 2500, 64]
    case = sh.paged(lengths, 16, 2, 128, fp8, _gen(14), width=200, spoil=False)
    table = case[4]
    table[:, :] = torch.randint(0, case[0].shape[0], table.shape, generator=_gen(15), device="cuda").int()
    q = _queries(5, 16, 128, 14)
    first, first_lse = _attend_check(case, q)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [_attend(case, q, stream=s) for s in streams for _ in range(2)]
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = _attend(case, q)
        graphs.append((g, r))
        got.append(r)
    for g, r in graphs:
        r[0].zero_(), r[1].zero_()
    torch.cuda.synchronize()
    for s, (g, _) in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, first) and torch.equal(lse, first_lse)
    q.copy_(_queries(5, 16, 128, 16))
    case[5].copy_(torch.tensor([0, 3000, 17, 1, 1200], dtype=torch.int32))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    want, want_lse = _attend_check(case, q)
    assert torch.equal(graphs[0][1][0], want) and torch.equal(graphs[0][1][1], want_lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_of_more_warps_than_tiles_and_the_reverse(fp8):
    """Every number of tiles around the numbers of warps and blocks."""
    k, v, ks, vs, table, _ = sh.paged([4096], 64, 1, 64, fp8, _gen(17), spoil=False)
    q = _queries(1, 4, 64, 17)
    for n in [*range(1, 32 * 14, 31), 32 * 911, 32 * 912, 32 * 913, 32 * 2000 + 1]:
        wide = table[:, :64].repeat(1, -(-n // 4096))
        _attend_check((k, v, ks, vs, wide, torch.tensor([n], dtype=torch.int32, device="cuda")), q)


def test_page_locked_host_buffers():
    """Every buffer in page-locked host memory, read and written in place."""
    pin = lambda t: None if t is None else t.cpu().pin_memory()
    x, res, w = _norm_case(3, 256, 18)
    got, want = lib.norm_rows(pin(x), pin(w), residual=pin(res), fp8=True, out=pin(x), residual_out=pin(x),
                              fp8_out=pin(x.to(FP8)), scale_out=torch.zeros(3, 2).pin_memory()), lib.norm_rows(x, w, residual=res, fp8=True)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.cpu().view(torch.uint8))
    s = _write_case(5, 4, 2, 64, 16, 32, True, 19)
    host = {n: pin(t) for n, t in s.items()}
    out, mine = _write(s), _write(host, q_out=torch.zeros(5, 4, 64, dtype=BF16).pin_memory())
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), mine)
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        assert torch.equal(host[n].view(torch.uint8), s[n].cpu().view(torch.uint8))
    case = sh.paged([40, 3], 16, 2, 64, True, _gen(20), spoil=False)
    q = _queries(2, 4, 64, 20)
    want, want_lse = _attend(case, q)
    got, lse = _attend([pin(t) for t in case], pin(q), out=torch.zeros(2, 4, 64, dtype=BF16).pin_memory(),
                       lse=torch.zeros(2, 4).pin_memory())
    torch.cuda.synchronize()
    assert torch.equal(got, want.cpu()) and torch.equal(lse, want_lse.cpu())


def test_refusals_on_the_gpu():
    """Pageable buffers, and those that the host cannot check without a device."""
    x, res, w = _norm_case(3, 256, 21)
    case = sh.paged([40, 3], 16, 2, 64, False, _gen(22))
    q = _queries(2, 4, 64, 22)
    s = _write_case(5, 4, 2, 64, 16, 32, False, 23)
    calls = [lambda: lib.norm_rows(x, w.cpu(), residual=res), lambda: lib.norm_rows(x, w, out=torch.zeros(3, 256, dtype=BF16)),
             lambda: lib.decode_attention(q, case[0], case[1].cpu(), *case[4:]),
             lambda: lib.decode_attention(q, case[0], case[1], case[4].cpu(), case[5]),
             lambda: lib.cache_write(s["q"], s["k"], s["v"], s["positions"], s["slots"].cpu(), s["k_cache"], s["v_cache"]),
             lambda: lib.cache_write(s["q"], s["k"], s["v"].cpu(), s["positions"], s["slots"], s["k_cache"], s["v_cache"])]
    for i, call in enumerate(calls):
        with pytest.raises(afd.AfdError) as e:
            call()
        assert e.value.status == afd.ERR_ARG, i


def test_write_ties_go_where_the_division_puts_them():
    """BF16 values whose quotients by the scale lie on ties of E4M3: bit for bit what
    the division by the scale gives in FP32 (the scale: a product with FP32's 1 / 448)."""
    s = _write_case(300, 1, 4, 128, 16, 0, True, 24)
    s["slots"][:] = torch.arange(300, device="cuda")
    s["v"].copy_(torch.randint(-14, 15, s["v"].shape, generator=_gen(25), device="cuda").float())
    _write(s)
    for name in ("k", "v"):
        t = s[name].float()
        scale = t.abs().amax(-1) * torch.tensor(1 / 448, device="cuda")
        assert torch.equal(_flat(s[name + "_scale"])[:300], scale)
        want = (t / scale[..., None]).to(FP8)
        assert torch.equal(_flat(s[name + "_cache"])[:300].view(torch.uint8), want.view(torch.uint8))
