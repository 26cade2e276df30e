"""The Attention source's operators as they are measured: the norm that makes
the rows a dispatch takes, the rotary positions and cache write of new tokens,
and the attention of one new token a sequence over its paged cache.

Hidden sizes and token counts follow the exchange's own workloads (2,048 tokens
a source; hidden 2,048, 4,096 and 7,168); head counts, head sizes and pages are
generic.
"""
import math

import torch

own = False

BF16, F32, F64, FP8 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
EPS = 1e-6
SMALLEST_SCALE = 2.0 ** -100


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One decode token before an FP8 dispatch: rows for the router and rows with scales for the exchange.
        dict(name="norm-decode1", op="norm", T=1, H=2048, residual=True, fp8=True),
        # A decode batch of wide rows, BF16 exchange.
        dict(name="norm-decode128-wide", op="norm", T=128, H=7168, residual=True, fp8=False),
        # Two sources' full prefill buckets, FP8 exchange.
        dict(name="norm-prefill-fp8", op="norm", T=4096, H=4096, residual=True, fp8=True),
        # One decode token's rotation and cache write.
        dict(name="write-decode1", op="write", T=1, Hq=32, Hkv=4, D=128, page=16, fp8=False, R=64, interleaved=False, far=4096),
        # A decode batch at far positions into an E4M3 cache, a quarter of the batch padding.
        dict(name="write-decode128-fp8", op="write", T=128, Hq=64, Hkv=8, D=128, page=64, fp8=True, R=64, interleaved=False, far=1000000),
        # A prefill chunk, interleaved layout on half of the head, E4M3 cache.
        dict(name="write-prefill-fp8", op="write", T=8192, Hq=64, Hkv=8, D=128, page=64, fp8=True, R=32, interleaved=True, far=131072),
        # One short sequence: a chain of latencies.
        dict(name="attention-one-short", op="attention", B=1, most=200, ragged=False, Hq=32, Hkv=4, D=128, page=16, fp8=False, window=0),
        # One long sequence: split over its length.
        dict(name="attention-one-long", op="attention", B=1, most=131072, ragged=False, Hq=64, Hkv=8, D=128, page=64, fp8=False, window=0),
        # A decode batch of unlike lengths over an E4M3 cache, sixteen query heads a KV head.
        dict(name="attention-batch64-fp8", op="attention", B=64, most=16384, ragged=True, Hq=64, Hkv=4, D=128, page=64, fp8=True, window=0),
        # Many short sequences, small heads, an odd number of them, small pages.
        dict(name="attention-batch250-small", op="attention", B=250, most=1000, ragged=True, Hq=40, Hkv=8, D=64, page=16, fp8=False, window=0),
        # Sliding-window layers of long sequences.
        dict(name="attention-window-fp8", op="attention", B=96, most=20000, ragged=True, Hq=64, Hkv=8, D=64, page=32, fp8=True, window=1024),
        # The largest: a full decode batch over a BF16 cache.
        dict(name="attention-batch128", op="attention", B=128, most=8192, ragged=True, Hq=64, Hkv=8, D=128, page=64, fp8=False, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "write", "attention", "attention"])
    fp8 = rng.random() < 0.5
    if op == "norm":
        H = 128 * _log(rng, 2, 56) if fp8 else 8 * _log(rng, 16, 896)
        return dict(op=op, T=_log(rng, 1, 4096), H=H, residual=rng.random() < 0.7, fp8=fp8)
    Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16]), rng.choice([64, 128])
    case = dict(op=op, Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([1, 16, 24, 32, 64, 128]), fp8=fp8)
    if op == "write":
        return dict(case, T=_log(rng, 1, 4096), R=rng.choice([0, D // 8, D // 4, D // 2, D // 2]), interleaved=rng.random() < 0.5,
                    far=_log(rng, 100, 4000000))
    B = _log(rng, 1, 256)
    return dict(case, B=B, most=_log(rng, 1, min(131072, (1 << 30) // (B * Hkv * D))), ragged=rng.random() < 0.7,
                window=rng.choice([0, 0, 0, 128, 1000]))


# ------------------------------------------------------------------- inputs
def _lengths(case):
    """The sequences' lengths in order: the squares of even steps up to the
    largest, and one sequence in sixteen is the bucket's padding."""
    B, most = case["B"], case["most"]
    if not case["ragged"]:
        return [most] * B
    pad = B // 16
    return [max(1, round(most * ((i + 1) / (B - pad)) ** 2)) for i in range(B - pad)] + [0] * pad


def _live(case):
    """Tokens that the attention reads, for every sequence."""
    return [min(n, case["window"]) if case["window"] else n for n in _lengths(case)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def bf16(*shape):
        return torch.empty(*shape, dtype=BF16, device=dev).normal_(generator=g)

    s = dict(case=case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s.update(x=bf16(T, H), residual=bf16(T, H).mul_(4) if case["residual"] else None, weight=(1 + 0.2 * randn(H)).to(BF16))
        return s
    Hq, Hkv, D, page, fp8 = (case[k] for k in ("Hq", "Hkv", "D", "page", "fp8"))
    if case["op"] == "write":
        T, R = case["T"], case["R"]
        qkv = bf16(T, (Hq + 2 * Hkv) * D)
        q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
        s.update(q=q.unflatten(1, (Hq, D)), k=k.unflatten(1, (Hkv, D)), v=v.unflatten(1, (Hkv, D)))
        s["inv_freq"] = (500000.0 ** (-torch.arange(R, device=dev, dtype=F64) / max(R, 1))).to(F32) if R else None
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=dev)
        pages = -(-T // page) + 3
        slots = torch.randperm(pages * page, generator=g, device=dev)[:T]
        slots[torch.rand(T, generator=g, device=dev) < (0.25 if T > 1 else 0)] = -1
        s["slots"] = slots
        for name in ("k", "v"):
            s[name + "_cache"] = bf16(pages, Hkv, page, D).to(FP8 if fp8 else BF16)
            s[name + "_scale"] = torch.rand(pages, Hkv, page, generator=g, device=dev) if fp8 else None
        return s
    B = case["B"]
    order = torch.randperm(B, generator=torch.Generator().manual_seed(int(seed))).tolist()
    if case["ragged"]:  # (the padding of a bucket stays behind its sequences)
        live = B - B // 16
        order = [i for i in order if i < live] + list(range(live, B))
    lengths = [_lengths(case)[i] for i in order]
    need = [-(-n // page) for n in lengths]
    width, pages = max(need) + 1, sum(need) + 2
    ids = torch.randperm(pages, generator=g, device=dev).int()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = torch.zeros(B + 1, dtype=torch.int64)
    at[1:] = torch.tensor(need).cumsum(0)
    cols = torch.arange(width)
    mine = cols[None, :] < torch.tensor(need)[:, None]
    table, index = table.to(dev), (at[:-1, None] + cols).to(dev)
    mine = mine.to(dev)
    table[mine] = ids[index[mine]]
    s.update(q=(bf16(B, Hq, D).float() * 2).to(BF16), table=table, lengths=torch.tensor(lengths, dtype=torch.int32, device=dev))
    for name in ("k", "v"):
        if fp8:
            s[name + "_cache"] = torch.empty(pages, Hkv, page, D, dtype=FP8, device=dev)
            for p in range(0, pages, 4096):  # (the conversion's temporaries stay small)
                part = s[name + "_cache"][p:p + 4096]
                part.copy_((bf16(*part.shape) * 120).clamp_(-448, 448))
            s[name + "_scale"] = (torch.rand(pages, Hkv, page, generator=g, device=dev) + 0.5) / 120
        else:
            s[name + "_cache"], s[name + "_scale"] = bf16(pages, Hkv, page, D), None
    return s


# --------------------------------------------------------------- plain forms
def _quantise(y):
    """E4M3 values and FP32 scales of the last dimension's vectors."""
    scale = (y.abs().amax(-1) / 448).clamp_min(SMALLEST_SCALE)
    return (y / scale[..., None]).clamp(-448, 448).to(FP8), scale


def _norm(s):
    r = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    got = dict(rows=y.to(BF16))
    if s["residual"] is not None:
        got["residual"] = r.to(BF16)
    if s["case"]["fp8"]:
        q, got["scales"] = _quantise(y.unflatten(-1, (-1, 128)))
        got["fp8_rows"] = q.flatten(-2)
    return got


def _rotate(x, cos, sin, interleaved):
    """FP32 [T, heads, D] with the first pairs of columns rotated."""
    x, R = x.float(), cos.shape[-1]
    a, b = (x[..., 0:2 * R:2], x[..., 1:2 * R:2]) if interleaved else (x[..., :R], x[..., R:2 * R])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * R:]], -1)


def _write(s):
    case = s["case"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if case["R"]:  # far positions: the angles in 64 bits
        angle = (s["positions"].double()[:, None] * s["inv_freq"].double())[:, None]
        cos, sin = angle.cos().float(), angle.sin().float()
        q, k = (_rotate(t, cos, sin, case["interleaved"]) for t in (q, k))
    tokens = torch.nonzero(s["slots"] >= 0)[:, 0]
    pages, at = s["slots"][tokens] // case["page"], s["slots"][tokens] % case["page"]
    for name, t in (("k", k), ("v", v)):
        if case["fp8"]:
            values, scale = _quantise(t[tokens])
            s[name + "_scale"][pages, :, at] = scale
            s[name + "_cache"].view(torch.uint8)[pages, :, at] = values.view(torch.uint8)
        else:
            s[name + "_cache"][pages, :, at] = t[tokens].to(BF16)
    return dict(q=q.to(BF16), k=s["k_cache"], v=s["v_cache"], ks=s["k_scale"], vs=s["v_scale"])


def _attention(s):
    case = s["case"]
    B, Hq, Hkv, D, page = (case[k] for k in ("B", "Hq", "Hkv", "D", "page"))
    table = s["table"].long().clamp_min(0)
    at = torch.arange(table.shape[1] * page, device=table.device)
    seen = at < s["lengths"][:, None]
    if case["window"]:
        seen &= at >= s["lengths"][:, None] - case["window"]

    def heads(name):  # [B, Hkv, L, D]
        x = s[name + "_cache"][table].float()
        if case["fp8"]:
            x = x * s[name + "_scale"][table][..., None]
        return x.transpose(1, 2).flatten(2, 3)

    scores = s["q"].float().view(B, Hkv, Hq // Hkv, D) @ heads("k").transpose(2, 3) * D ** -0.5
    scores = scores.masked_fill(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp_min(torch.finfo(F32).min)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = p @ heads("v").masked_fill(~seen[:, None, :, None], 0)
    out = out / total.clamp_min(1e-30)
    lse = torch.where(total > 0, top + torch.log(total), float("-inf"))
    return dict(out=out.view(B, Hq, D).to(BF16), lse=lse.view(B, Hq))


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import combine_attention_ffn_gb300 as afd

        if op == "norm":
            got = afd.norm_rows(state["x"], state["weight"], eps=EPS, residual=state["residual"], fp8=case["fp8"])
            return {k: v for k, v in got._asdict().items() if v is not None}
        caches = (state["k_cache"], state["v_cache"])
        scales = dict(k_scale=state["k_scale"], v_scale=state["v_scale"])
        if op == "write":
            q = afd.cache_write(state["q"], state["k"], state["v"], state["positions"], state["slots"], *caches,
                                inv_freq=state["inv_freq"], interleaved=case["interleaved"], **scales)
            return dict(q=q, k=state["k_cache"], v=state["v_cache"], ks=state["k_scale"], vs=state["v_scale"])
        out, lse = afd.decode_attention(state["q"], *caches, state["table"], state["lengths"], window=case["window"],
                                        return_lse=True, **scales)
        return dict(out=out, lse=lse)
    return dict(norm=_norm, write=_write, attention=_attention)[op](state)


# ------------------------------------------------------------ least work
def work(case):
    op, fp8 = case["op"], case["fp8"]
    if op == "norm":
        T, H = case["T"], case["H"]
        n = T * H * (4 + (4 if case["residual"] else 0)) + 2 * H
        return dict(bytes=n + (T * H + T * (H // 128) * 4 if fp8 else 0), flops=6 * T * H)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    b = 1 if fp8 else 2
    if op == "write":
        T = case["T"]
        kept = T if T == 1 else T * 3 // 4
        n = T * ((Hq + Hkv) * D * 2 + Hq * D * 2 + 16) + kept * (Hkv * D * 2 + 2 * Hkv * (D * b + (4 if fp8 else 0)))
        return dict(bytes=n, flops=T * (Hq + Hkv) * (6 * case["R"] + (2 * D if fp8 else 0)))
    live = sum(_live(case))
    rows = case["B"] * Hq
    n = live * 2 * Hkv * (D * b + (4 if fp8 else 0)) + rows * (4 * D + 4) + 4 * sum(-(-n // case["page"]) for n in _live(case))
    return dict(bytes=n, flops=live * 4 * Hq * D)


# ------------------------------------------------------------------- exact
def _e4m3(y):
    scale = (y.abs().amax(-1) / 448).clamp_min(SMALLEST_SCALE)
    return (y / scale[..., None]).clamp(-448, 448).to(FP8).double(), scale


def exact(case, seed):
    """Row by row, token by token, sequence by sequence in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        got = dict(rows=torch.empty(s["x"].shape, dtype=F64, device=s["x"].device))
        got["residual"], got["fp8_rows"] = torch.empty_like(got["rows"]), torch.empty_like(got["rows"])
        got["scales"] = torch.empty(case["T"], case["H"] // 128, dtype=F64, device=s["x"].device)
        for a in range(0, case["T"], 512):
            rows = slice(a, a + 512)
            r = s["x"][rows].double() + (s["residual"][rows].double() if case["residual"] else 0)
            y = r * r.square().mean(-1, keepdim=True).add(EPS).rsqrt() * s["weight"].double()
            got["rows"][rows], got["residual"][rows] = y, r
            if case["fp8"]:
                q, got["scales"][rows] = _e4m3(y.view(y.shape[0], -1, 128))
                got["fp8_rows"][rows] = q.view(y.shape)
        keep = ["rows"] + ["residual"] * case["residual"] + ["fp8_rows", "scales"] * case["fp8"]
        return {k: got[k] for k in keep}
    page = case["page"]
    if case["op"] == "write":
        T, Hkv, D, R = case["T"], case["Hkv"], case["D"], case["R"]
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        if R:
            unit = torch.polar(torch.ones(T, 1, R, dtype=F64, device=q.device),
                               s["positions"].double()[:, None, None] * s["inv_freq"].double())
            at = torch.arange(R, device=q.device)
            first, second = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + R)
            for t in (q, k):
                z = torch.complex(t[..., first], t[..., second]) * unit
                t[..., first], t[..., second] = z.real, z.imag
        got = dict(q=q, ks=None, vs=None)
        live = s["slots"] >= 0
        for name, t in (("k", k), ("v", v)):
            flat = s[name + "_cache"].double().transpose(1, 2).reshape(-1, Hkv, D)
            if case["fp8"]:
                scale = s[name + "_scale"].double().transpose(1, 2).reshape(-1, Hkv)
                flat[s["slots"][live]], scale[s["slots"][live]] = _e4m3(t[live])
                got[name + "s"] = scale.view(-1, page, Hkv).transpose(1, 2)
            else:
                flat[s["slots"][live]] = t[live]
            got[name] = flat.view(-1, page, Hkv, D).transpose(1, 2)
        return got
    B, Hq, Hkv, D = (case[k] for k in ("B", "Hq", "Hkv", "D"))
    out = torch.zeros(B, Hq, D, dtype=F64, device=s["q"].device)
    lse = torch.full((B, Hq), float("-inf"), dtype=F64, device=s["q"].device)
    for b, n in enumerate(s["lengths"].tolist()):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        at = torch.arange(first, n, device=out.device)
        pages, where = s["table"][b].long()[at // page], at % page
        for h in range(Hkv):
            k, v = s["k_cache"][pages, h, where].double(), s["v_cache"][pages, h, where].double()
            if case["fp8"]:
                k, v = k * s["k_scale"][pages, h, where, None].double(), v * s["v_scale"][pages, h, where, None].double()
            mine = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            a = s["q"][b, mine].double() @ k.t() / math.sqrt(D)
            lse[b, mine] = a.logsumexp(-1)
            out[b, mine] = a.softmax(-1) @ v
    return dict(out=out, lse=lse)
