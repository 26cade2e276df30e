"""A decode step of both roles on the library's operators: norm, projections,
rotary positions and cache write, attention over the cache, norm to FP8 rows,
router, FP8 dispatch, experts, reply, collect. Every stage against float64
values from the inputs it got, and several steps replayed from one graph against
the same steps called one by one."""
import os
import subprocess
import sys

import pytest
import torch

import combine_attention_ffn_gb300 as lib
import expert_harness as eh
import source_harness as sh
from combine_attention_ffn_gb300 import afd

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
A, F, E, K, H, I = 2, 2, 8, 2, 256, 128
HQ, HKV, D, PAGE, BUCKET, ALPHA = 6, 2, 64, 16, 64, 16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_attention_ffn_gb300 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Sources:
    """Weights, caches and the sequences of two sources; the last sequence of
    each is the bucket's padding."""

    def __init__(self, T, fp8_cache, seed=5):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.T, self.fp8 = T, fp8_cache
        self.w1, self.w2 = ((1 + 0.2 * rnd(H)).to(BF16) for _ in range(2))
        self.wqkv = (rnd(1, (HQ + 2 * HKV) * D, H) * H ** -0.5).to(BF16)
        self.wo = (rnd(1, H, HQ * D) * (HQ * D) ** -0.5).to(BF16)
        self.gate = (rnd(1, E, H) * 3 * H ** -0.5).to(BF16)
        self.w13, self.s13 = eh.quantise_weight(rnd(E, 2 * I, H) * H ** -0.5)
        self.down = (rnd(E, H, I) * I ** -0.5).to(BF16)
        self.inv_freq = (10000.0 ** (-torch.arange(D // 2, device="cuda").double() / (D // 2))).float()
        self.ends = torch.tensor([T], dtype=torch.int32, device="cuda")
        self.x = [rnd(T, H).to(BF16) for _ in range(A)]
        self.residual = [(3 * rnd(T, H)).to(BF16) for _ in range(A)]
        before = [(37 * i) % 150 for i in range(T)]  # tokens that a sequence has so far
        self.caches, self.tables, self.lengths = [], [], []
        for s in range(A):
            room = [n + 8 for n in before]
            k, v, ks, vs, table, _ = sh.paged(room, PAGE, HKV, D, fp8_cache, g, spoil=False)
            self.caches.append((k, v, ks, vs))
            self.tables.append(table)
            self.lengths.append(torch.tensor(before, dtype=torch.int32, device="cuda"))
        self.positions = [torch.zeros(T, dtype=torch.int64, device="cuda") for _ in range(A)]
        self.slots = [torch.zeros(T, dtype=torch.int64, device="cuda") for _ in range(A)]

    def advance(self):
        """The next token of every sequence: its position, slot and length."""
        for s in range(A):
            at = self.lengths[s].long()
            self.positions[s].copy_(at)
            self.slots[s].copy_(self.tables[s].gather(1, (at // PAGE)[:, None])[:, 0].long() * PAGE + at % PAGE)
            self.lengths[s] += 1
            if self.T > 1:  # the padding
                self.slots[s][-1], self.lengths[s][-1] = -1, 0

    def step(self, buf):
        """One layer; returns every stage's results."""
        T, got = self.T, []
        for s in range(A):
            k, v, ks, vs = self.caches[s]
            n = lib.norm_rows(self.x[s], self.w1, residual=self.residual[s])
            qkv = lib.grouped_linear(n.rows, self.wqkv, self.ends)
            q, kn, vn = (t.unflatten(1, (-1, D)) for t in qkv.split([HQ * D, HKV * D, HKV * D], 1))
            q = lib.cache_write(q, kn, vn, self.positions[s], self.slots[s], k, v, inv_freq=self.inv_freq, k_scale=ks, v_scale=vs)
            a, lse = lib.decode_attention(q, k, v, self.tables[s], self.lengths[s], k_scale=ks, v_scale=vs, return_lse=True)
            o = lib.grouped_linear(a.view(T, HQ * D), self.wo, self.ends)
            m = lib.norm_rows(o, self.w2, residual=n.residual, fp8=True)
            logits = lib.grouped_linear(m.rows, self.gate, self.ends)
            ids, w = lib.route_topk(logits, K)
            buf.source_dispatch(s, m.fp8_rows, ids, w, m.scales, bucket=BUCKET)
            got.append(dict(n=n, qkv=qkv, q=q, a=a, lse=lse, o=o, m=m, logits=logits, ids=ids, w=w))
        replies = []
        for f in range(F):
            r = buf.worker_receive(f, bucket=BUCKET)
            mine = slice(f * E // F, (f + 1) * E // F)
            act = lib.grouped_linear(r.rows, self.w13[mine], r.ends, expert_alignment=ALPHA, gated=True, x_scale=r.row_scales,
                                     weight_scale=self.s13[mine])
            replies.append(lib.grouped_linear(act, self.down[mine], r.ends, expert_alignment=ALPHA))
            buf.worker_reply(f, replies[f], r.receipt)
        outs = buf.source_collect_all(num_tokens=[T] * A)
        for s in range(A):
            got[s]["out"] = outs[s]
            # the next layer's inputs
            self.residual[s].copy_(got[s]["m"].residual)
            self.x[s].copy_(outs[s])
        return got, replies

    def check(self, got, x, residual):
        T, every = self.T, torch.ones(self.T, dtype=torch.bool, device="cuda")
        product = lambda t, w: eh.product(t, w, [(0, T)])
        for s in range(A):
            r = got[s]
            res, y, err = sh.norm(x[s], residual[s], self.w1, 1e-6, 64)
            eh.check_bf16(r["n"].rows, y, err, every)
            eh.check_bf16(r["n"].residual, res, sh.FP32_HALF * res.abs(), every)
            y, mag = product(r["n"].rows, self.wqkv)
            eh.check_bf16(r["qkv"], y, eh.product_error(mag, H), every)
            q, k, v = (t.unflatten(1, (-1, D)) for t in r["qkv"].split([HQ * D, HKV * D, HKV * D], 1))
            y, err = sh.rotate(q, self.positions[s], self.inv_freq, False, 1.0)
            eh.check_bf16(r["q"], y, err, every)
            live = self.slots[s] >= 0
            kc, vc, ks, vs = self.caches[s]
            for cache, scale, t, turned in ((kc, ks, k, True), (vc, vs, v, False)):
                y, err = sh.rotate(t, self.positions[s], self.inv_freq if turned else None, False, 1.0)
                flat = cache.transpose(1, 2).flatten(0, 1)[self.slots[s][live]]
                if self.fp8:
                    sh.check_e4m3(flat, scale.transpose(1, 2).flatten(0, 1)[self.slots[s][live]], y[live], err[live])
                else:
                    eh.check_bf16(flat, y[live], err[live], every[live])
            y, lse, err, lse_err = sh.attention(r["q"], kc, vc, self.tables[s], self.lengths[s], D ** -0.5, 0, ks, vs)
            eh.check_bf16(r["a"], y, err, every)
            sh.check_lse(r["lse"], lse, lse_err)
            y, mag = product(r["a"].view(T, -1), self.wo)
            eh.check_bf16(r["o"], y, eh.product_error(mag, HQ * D), every)
            res, y, err = sh.norm(r["o"], r["n"].residual, self.w2, 1e-6, 64)
            eh.check_bf16(r["m"].rows, y, err, every)
            sh.check_e4m3(r["m"].fp8_rows.view(T, -1, 128), r["m"].scales, y.view(T, -1, 128), err.view(T, -1, 128))
            ids, w = eh.route_reference(r["logits"].cpu(), K)
            assert torch.equal(r["ids"].cpu(), ids) and (r["w"].double().cpu() - w).abs().max() <= 2.0 ** -17
            rows = r["m"].fp8_rows.double() * r["m"].scales.double().repeat_interleave(128, 1)
            w13 = self.w13.double() * self.s13.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
            for t in range(T):
                want, off = torch.zeros(2, H, dtype=torch.float64, device="cuda")
                for k in range(K):
                    e, weight = int(ids[t, k]), float(r["w"][t, k])
                    g, u = (w13[e] @ rows[t]).chunk(2)
                    act = eh.silu(g) * u
                    y = self.down[e].double() @ act
                    want += weight * y
                    # the activation's rounding through the product, and the reply's
                    off += weight * eh.HALF_BF16 * (self.down[e].double().abs() @ act.abs() + y.abs())
                assert ((r["out"][t].double() - want).abs() <= 1.05 * off + eh.HALF_BF16 * want.abs() + 1e-6).all()


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_steps(fp8, T):
    eager, graphed = Sources(T, fp8), Sources(T, fp8)
    bufs = [afd.Buffer(A, F, E, K, H, BUCKET, ALPHA, "fp8") for _ in range(2)]
    try:
        # (the capture records a step and runs none of it)
        graphed.advance()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured, _ = graphed.step(bufs[1])
        for i in range(3):
            if i:
                graphed.advance()
            graph.replay()
            eager.advance()
            x, residual = [t.clone() for t in eager.x], [t.clone() for t in eager.residual]
            got, _ = eager.step(bufs[0])
            torch.cuda.synchronize()
            eager.check(got, x, residual)
            for s in range(A):
                for name in ("out", "q", "a", "lse", "logits", "ids", "w"):
                    assert torch.equal(captured[s][name], got[s][name]), (i, s, name)
                for a, b in zip(graphed.caches[s], eager.caches[s]):
                    if a is not None:
                        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert all(b.get_error()[0] == 0 for b in bufs)
    finally:
        torch.cuda.synchronize()
        for b in bufs:
            b.close()


def test_first_calls_inside_a_capture():
    """A process whose first call of every operator is captured (nothing has to be set up eagerly)."""
    code = """
import torch, combine_attention_ffn_gb300 as lib
d, bf = "cuda", torch.bfloat16
x, w = torch.randn(9, 256, device=d).to(bf), torch.ones(256, device=d).to(bf)
kc, vc = torch.zeros(40, 2, 16, 64, device=d).to(bf), torch.zeros(40, 2, 16, 64, device=d).to(bf)
k8, v8, s8 = kc.to(torch.float8_e4m3fn), vc.to(torch.float8_e4m3fn), torch.ones(2, 40, 2, 16, device=d)
q, k = torch.randn(9, 6, 64, device=d).to(bf), torch.randn(9, 2, 64, device=d).to(bf)
pos, slots = torch.arange(9, device=d), torch.arange(9, device=d) * 16
f = torch.rand(32, device=d)
table = torch.arange(40, dtype=torch.int32, device=d).repeat(9, 20)
lengths = torch.full((9,), 700, dtype=torch.int32, device=d)
def step():
    n = lib.norm_rows(x, w, residual=x, fp8=True)
    r = lib.cache_write(q, k, k, pos, slots, kc, vc, inv_freq=f)
    r8 = lib.cache_write(q, k, k, pos, slots, k8, v8, inv_freq=f, k_scale=s8[0], v_scale=s8[1])
    return [*n, r, r8, lib.decode_attention(r, kc, vc, table, lengths), lib.decode_attention(r, k8, v8, table, lengths, k_scale=s8[0], v_scale=s8[1])]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay(); torch.cuda.synchronize()
for a, b in zip(got, step()):
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
print("captured first: ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=120)
    assert r.returncode == 0 and "captured first: ok" in r.stdout, r.stderr[-2000:]


def test_calls_on_a_given_stream():
    """stream=: the operators run there, and so do the tensors they make."""
    src = Sources(4, True)
    src.advance()
    side = torch.cuda.Stream()
    k, v, ks, vs = src.caches[0]
    q = torch.randn(4, HQ, D, device="cuda").to(BF16)
    kn = torch.randn(4, HKV, D, device="cuda").to(BF16)

    def calls(**kw):
        return (*lib.norm_rows(src.x[0], src.w1, residual=src.residual[0], fp8=True, **kw),
                lib.cache_write(q, kn, kn, src.positions[0], src.slots[0], k, v, inv_freq=src.inv_freq, k_scale=ks, v_scale=vs, **kw),
                *lib.decode_attention(q, k, v, src.tables[0], src.lengths[0], k_scale=ks, v_scale=vs, return_lse=True, **kw))

    want = calls()
    torch.cuda.synchronize()
    got = calls(stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
