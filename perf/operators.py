"""The expert-worker operators as they are measured: the router that makes a
dispatch's IDs and weights, the experts' ragged matrix products, the gated
activation over received rows, and the low-rank adapters of many requests.

Shapes follow the exchange's own workloads (top-k 8 of 128 or 96 experts,
hidden 2,048, expert_alignment 128, uniform or Zipf-like routing); the experts'
inner sizes and the adapters' ranks are generic.
"""
import math

import torch

own = False

BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of two sources with one token each: 8 rows on 64 local experts.
        dict(name="experts-gated-decode1", op="experts", A=2, T=1, E=128, F=2, K=8, H=2048, N=1024, gated=True, fp8=False,
             alpha=128, zipf=False),
        # A decode step of 128 requests on the one-source, three-worker layout: skewed, unaligned, an odd inner size.
        dict(name="experts-gated-odd128", op="experts", A=1, T=128, E=96, F=3, K=8, H=2048, N=1000, gated=True, fp8=False,
             alpha=1, zipf=True),
        # A full prefill bucket: 2,048 tokens from each of two sources, about 256 rows per expert.
        dict(name="experts-gated-prefill", op="experts", A=2, T=2048, E=128, F=2, K=8, H=2048, N=1024, gated=True, fp8=False,
             alpha=128, zipf=False),
        # The down projection of the skewed three-source, one-worker layout: the largest ragged product.
        dict(name="experts-down-skewed", op="experts", A=3, T=2048, E=128, F=1, K=8, H=1024, N=2048, gated=False, fp8=False,
             alpha=128, zipf=True),
        # The FP8 exchange's rows (E4M3 with block scales) at prefill.
        dict(name="experts-gated-fp8-prefill", op="experts", A=2, T=2048, E=128, F=2, K=8, H=2048, N=1024, gated=True, fp8=True,
             alpha=128, zipf=False),
        # The FP8 down projection of an ordinary decode step.
        dict(name="experts-down-fp8-decode32", op="experts", A=2, T=32, E=128, F=2, K=8, H=1024, N=2048, gated=False, fp8=True,
             alpha=128, zipf=False),
        # The router of one decode token.
        dict(name="router-decode1", op="router", T=1, E=128, K=8, scoring="softmax", bias=False, bf16=False),
        # The router of a prefill bucket, with sigmoid scores and a balancing bias on the selection.
        dict(name="router-prefill", op="router", T=2048, E=128, K=8, scoring="sigmoid", bias=True, bf16=True),
        # The activation of a decode step (rows with adapters between product and activation).
        dict(name="gated-decode32", op="gated", A=2, T=32, E=128, F=2, K=8, N=1024, alpha=128),
        # ... and of a prefill bucket.
        dict(name="gated-prefill", op="gated", A=2, T=2048, E=128, F=2, K=8, N=1024, alpha=128),
        # Decode: every token another request, 16 adapters, rows in the order that the exchange gives them.
        dict(name="adapters-decode32", op="adapters", A=2, T=32, E=128, F=2, K=8, H=2048, N=2048, rank=16, S=16, run=1, alpha=128),
        # Prefill: requests of 256 tokens each, two in three with an adapter.
        dict(name="adapters-prefill", op="adapters", A=2, T=2048, E=128, F=2, K=8, H=2048, N=2048, rank=32, S=8, run=256, alpha=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["experts", "experts", "experts", "router", "gated", "adapters"])
    if op == "router":
        E = rng.choice([8, 32, 96, 128, 200, 256, 384])
        return dict(op=op, T=_log(rng, 1, 2048), E=E, K=rng.randint(1, min(E, 10)),
                    scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, bf16=rng.random() < 0.5)
    A, F, El = rng.choice([(1, 1, 32), (2, 2, 64), (1, 3, 32), (2, 1, 48), (2, 4, 16), (2, 2, 4)])
    case = dict(op=op, A=A, F=F, E=F * El, K=min(8, El, rng.choice([1, 2, 6, 8])), T=_log(rng, 1, 2048),
                alpha=rng.choice([1, 16, 64, 128]))
    if op == "experts":
        fp8 = rng.random() < 0.4
        wide = 128 if fp8 else rng.choice([8, 8, 64, 128])
        return dict(case, H=256 * rng.randint(1, 8) if fp8 or rng.random() < 0.5 else 8 * rng.randint(16, 256),
                    N=wide * max(1, _log(rng, 128, 1024) // wide), gated=rng.random() < 0.5, fp8=fp8, zipf=rng.random() < 0.5)
    if op == "gated":
        return dict(case, N=8 * _log(rng, 16, 128))
    return dict(case, H=256 * rng.randint(1, 8), N=8 * _log(rng, 16, 256), rank=rng.choice([8, 16, 32, 64]),
                S=_log(rng, 1, 32), run=rng.choice([1, 7, 64, 256]))


# ------------------------------------------------------------------- inputs
def _gen(seed, device):
    return torch.Generator(device=device).manual_seed(int(seed))


def _receive(case, seed, device):
    """Worker 0's received layout: ends [E/F], row_src [R] and the largest
    count, rows expert-major with aligned starts, tokens ascending inside."""
    g = _gen(seed, device)
    A, T, E, F, K, alpha = (case[k] for k in ("A", "T", "E", "F", "K", "alpha"))
    El, tokens = E // F, A * T
    if case.get("zipf"):
        p = torch.arange(1, E + 1, device=device, dtype=F32).pow(-1.2).log()
        keys = p - torch.rand(tokens, E, generator=g, device=device).clamp_min(1e-12).log().neg().clamp_min(1e-12).log()
        ids = keys.argsort(dim=1, descending=True)[:, :K]
        ids = torch.where(torch.rand(tokens, K, generator=g, device=device) < 0.1, E, ids)
    else:
        ids = torch.rand(tokens, E, generator=g, device=device).argsort(dim=1)[:, :K]
    flat = ids.reshape(-1)
    local = torch.where(flat < El, flat, El)
    order = local.argsort(stable=True)
    counts = torch.bincount(local, minlength=El + 1)[:El]
    aligned = (counts + alpha - 1) // alpha * alpha
    starts = aligned.cumsum(0) - aligned
    n = int(counts.sum())
    R = (tokens * min(K, El) + El * (alpha - 1) + alpha - 1) // alpha * alpha
    sorted_local, routes = local[order[:n]], order[:n]
    first = counts.cumsum(0) - counts
    rows = starts[sorted_local] + torch.arange(n, device=device) - first[sorted_local]
    row_src = torch.full((R,), -1, dtype=torch.int32, device=device)
    row_src[rows] = routes.int()
    return dict(ends=(starts + counts).int(), row_src=row_src, R=R, rows=n, used=int((counts > 0).sum()),
                most=int(counts.max()), starts=starts, counts=counts)


def _blocks(v):
    """E4M3 rows and their FP32 scales, one for every 128 columns (absmax / 448)."""
    b = v.view(*v.shape[:-1], -1, 128)
    s = b.abs().amax(-1) / 448.0
    return (b / s[..., None]).clamp(-448, 448).to(FP8).view(v.shape), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed + 1_000_003, dev)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    op, s = case["op"], dict(case=case)
    if op == "router":
        s["logits"] = (randn(case["T"], case["E"]) * 1.5).to(BF16 if case["bf16"] else F32)
        s["bias"] = randn(case["E"]) * 0.05 if case["bias"] else None
        return s
    lay = _receive(case, seed, dev)
    R, El = lay["R"], case["E"] // case["F"]
    s.update(ends=lay["ends"], row_src=lay["row_src"], most=lay["most"])
    if op == "experts":
        K, N = case["H"], case["N"] * (2 if case["gated"] else 1)
        x = randn(R, K)
        if case["fp8"]:
            s["x"], s["x_scale"] = _blocks(x)
            w = randn(El, N, K).mul_(K ** -0.5).view(El, N // 128, 128, K // 128, 128)
            ws = w.abs().amax(dim=(2, 4)) / 448.0
            s["w"] = (w / ws[:, :, None, :, None]).clamp(-448, 448).to(FP8).view(El, N, K)
            s["w_scale"] = ws
        else:
            s["x"], s["x_scale"], s["w_scale"] = x.to(BF16), None, None
            s["w"] = randn(El, N, K).mul_(K ** -0.5).to(BF16)
        s["out"] = torch.zeros(R, case["N"], dtype=BF16, device=dev)
    elif op == "gated":
        s["h"] = randn(R, 2 * case["N"]).to(BF16)
        s["out"] = torch.zeros(R, case["N"], dtype=BF16, device=dev)
    else:
        H, N, r, S, tokens = case["H"], case["N"], case["rank"], case["S"], case["A"] * case["T"]
        s["x"], s["base"] = randn(R, H).to(BF16), randn(R, N).to(BF16)
        s["down"] = randn(S, r, H).mul_(H ** -0.5).to(BF16)
        s["up"] = randn(S, N, r).mul_(r ** -0.5).to(BF16)
        s["scales"] = torch.rand(S, generator=g, device=dev) + 0.5
        requests = -(-tokens // case["run"])
        slot = torch.randint(0, S, (requests,), generator=g, device=dev)
        slot = torch.where(torch.rand(requests, generator=g, device=dev) < 1 / 3, -1, slot)
        s["token_slots"] = slot.repeat_interleave(case["run"])[:tokens].int()
        s["out"] = torch.zeros(R, N, dtype=BF16, device=dev)
    return s


# --------------------------------------------------------------- plain forms
def _row_index(s):
    """[El, most] row numbers of every expert and which of them are rows."""
    case, ends = s["case"], s["ends"].long()
    a = case["alpha"]
    starts = torch.cat([ends.new_zeros(1), (ends[:-1] + a - 1) // a * a])
    at = starts[:, None] + torch.arange(max(s["most"], 1), device=ends.device)
    return at, at < ends[:, None]


def _experts(s):
    case, (at, live) = s["case"], _row_index(s)
    x, w = s["x"][at.clamp_max(s["x"].shape[0] - 1)].float(), s["w"].float()
    if case["fp8"]:
        x = x * s["x_scale"][at.clamp_max(s["x"].shape[0] - 1)].repeat_interleave(128, -1)
        w = w * s["w_scale"].repeat_interleave(128, 1).repeat_interleave(128, 2)
    y = torch.bmm(x, w.transpose(1, 2))
    if case["gated"]:
        gate, up = y.chunk(2, -1)
        y = gate / (1 + torch.exp(-gate)) * up
    s["out"][at[live]] = y[live].to(BF16)
    return s["out"]


def _gated(s):
    at, live = _row_index(s)
    rows = at[live]
    gate, up = s["h"][rows].float().chunk(2, -1)
    s["out"][rows] = (gate / (1 + torch.exp(-gate)) * up).to(BF16)
    return s["out"]


def _adapters(s):
    K, S, r = s["case"]["K"], s["case"]["S"], s["case"]["rank"]
    rows = torch.nonzero(s["row_src"] >= 0)[:, 0]
    slot = s["token_slots"][(s["row_src"][rows] // K).long()].long()
    # every row against every adapter, and the products of the others left out
    t = s["x"][rows].float() @ s["down"].float().view(S * r, -1).t()
    mine = slot[:, None] == torch.arange(S, device=slot.device)
    t = t.view(-1, S, r) * (mine * s["scales"])[:, :, None]
    delta = t.view(-1, S * r) @ s["up"].float().transpose(1, 2).reshape(S * r, -1)
    s["out"][rows] = (s["base"][rows].float() + delta).to(BF16)
    return s["out"]


def _router(s):
    case, K = s["case"], s["case"]["K"]
    l = s["logits"].double()  # the choice lies next to a border: in 64 bits
    score = torch.softmax(l, -1) if case["scoring"] == "softmax" else 1 / (1 + torch.exp(-l))
    key = score + s["bias"].double() if case["bias"] else l
    ids = key.sort(dim=-1, descending=True, stable=True).indices[:, :K].contiguous()
    w = score.gather(1, ids)
    return ids, (w / w.sum(-1, keepdim=True)).float()


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import combine_attention_ffn_gb300 as afd

        if op == "router":
            return afd.route_topk(state["logits"], case["K"], scoring=case["scoring"], bias=state["bias"])
        if op == "experts":
            return afd.grouped_linear(state["x"], state["w"], state["ends"], expert_alignment=case["alpha"], gated=case["gated"],
                                      x_scale=state["x_scale"], weight_scale=state["w_scale"], out=state["out"])
        if op == "gated":
            return afd.gated_rows(state["h"], state["ends"], expert_alignment=case["alpha"], out=state["out"])
        return afd.adapter_add(state["base"], state["x"], state["down"], state["up"], state["token_slots"], state["scales"],
                               ends=state["ends"], row_src=state["row_src"], top_k=case["K"], out=state["out"])
    return dict(router=_router, experts=_experts, gated=_gated, adapters=_adapters)[op](state)


# ------------------------------------------------------------ least work
def work(case):
    op = case["op"]
    if op == "router":
        T, E, K = case["T"], case["E"], case["K"]
        return dict(bytes=T * E * (2 if case["bf16"] else 4) + T * K * 12 + (4 * E if case["bias"] else 0), flops=6 * T * E)
    lay = _receive(case, 0, torch.device("cpu"))
    rows, N, El = lay["rows"], case["N"], case["E"] // case["F"]
    if op == "gated":
        return dict(bytes=rows * N * 6 + 4 * El, flops=5 * rows * N)
    H = case["H"]
    if op == "experts":
        wide = N * (2 if case["gated"] else 1)
        b = 1 if case["fp8"] else 2
        scales = (rows * (H // 128) + lay["used"] * (wide // 128) * (H // 128)) * 4 if case["fp8"] else 0
        return dict(bytes=rows * H * b + lay["used"] * wide * H * b + rows * N * 2 + scales + 4 * El, flops=2 * rows * wide * H)
    # two rows in three have an adapter; the others are copied
    r, with_a = case["rank"], rows * 2 // 3
    used = min(case["S"], -(-case["A"] * case["T"] // case["run"]))
    return dict(bytes=with_a * H * 2 + rows * N * 4 + rows * 4 + used * r * (H + N) * 2, flops=2 * with_a * r * (H + N))


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """Expert by expert and row by row in 64 bits, from the definitions."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "router":
        l = s["logits"].double().cpu()
        if case["scoring"] == "softmax":
            e = (l - l.max(1, keepdim=True).values).exp()
            p = e / e.sum(1, keepdim=True)
        else:
            p = l.sigmoid()
        key = p + s["bias"].double().cpu() if case["bias"] else l
        ids = torch.tensor([sorted(range(case["E"]), key=lambda j: (-row[j], j))[: case["K"]] for row in key.tolist()])
        w = p.gather(1, ids)
        return ids, w / w.sum(1, keepdim=True)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    if op == "adapters":
        src = s["row_src"].long()
        slots = torch.where(src < 0, -2, s["token_slots"].long()[src.clamp_min(0) // case["K"]])
        out[slots > -2] = s["base"][slots > -2].double()
        for a in range(case["S"]):
            rows = torch.nonzero(slots == a)[:, 0]
            low = s["x"][rows].double() @ s["down"][a].double().t()
            out[rows] += s["scales"][a].double() * (low @ s["up"][a].double().t())
        return out
    at = 0
    for e, end in enumerate(s["ends"].tolist()):
        at = -(-at // case["alpha"]) * case["alpha"]
        if end > at:
            if op == "gated":
                y = s["h"][at:end].double()
            else:
                x, w = s["x"][at:end].double(), s["w"][e].double()
                if case["fp8"]:
                    x = (x.view(end - at, -1, 128) * s["x_scale"][at:end, :, None].double()).view(end - at, -1)
                    q = w.view(w.shape[0] // 128, 128, -1, 128) * s["w_scale"][e][:, None, :, None].double()
                    w = q.reshape(w.shape)
                y = x @ w.t()
            if op == "gated" or case["gated"]:
                gate, up = y[:, : case["N"]], y[:, case["N"]:]
                y = gate * gate.sigmoid() * up
            out[at:end] = y
            at = end
    return out
