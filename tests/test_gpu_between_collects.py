"""An operator, or another context's exchange, between two collects of one
exchange. A combine that follows another one of its exchange directly starts
beside it; with other work of the library between them it must wait, because
that work lets its dependents start while it still reads, and what it reads
may be the memory of the second collect's `out` (handed over by the caller, or
by an allocator that got it back)."""
import numpy as np
import pytest
import torch

import combine_attention_ffn_gb300 as lib
import gpu_harness as GH
from combine_attention_ffn_gb300 import afd, build
from combine_attention_ffn_gb300 import workloads as W

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
H = 2048


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class _Gated:
    """16 K rows of 2 x 2048; source 1's `out` lies in the rows read last."""

    def __init__(self, T):
        R = 16384
        self.buf = torch.randn(R, 2 * H, generator=_gen(1), device="cuda").to(BF16)
        self.out1 = self.buf.view(-1)[-T * H:].view(T, H)
        self.ends = torch.tensor([R], dtype=torch.int32, device="cuda")
        self.res = torch.zeros(R, H, dtype=BF16, device="cuda")

    def run(self):
        lib.gated_rows(self.buf, self.ends, out=self.res)
        return self.res


class _Router:
    def __init__(self, T):
        E = 256
        self.buf = torch.randn(65536, E, generator=_gen(2), device="cuda").to(BF16)
        self.out1 = self.buf.view(-1)[-T * H:].view(T, H)
        self.bias = torch.randn(E, generator=_gen(3), device="cuda") * 0.1
        self.res = torch.zeros(65536, 8, dtype=torch.int64, device="cuda")
        self.w = torch.zeros(65536, 8, device="cuda")

    def run(self):
        lib.route_topk(self.buf, 8, bias=self.bias, ids=self.res, weights=self.w)
        return self.res


class _Product:
    def __init__(self, T):
        R, G = 16384, 32
        self.buf = torch.randn(R, H, generator=_gen(4), device="cuda").to(BF16)
        self.out1 = self.buf.view(-1)[-T * H:].view(T, H)
        self.w = (torch.randn(G, 1024, H, generator=_gen(5), device="cuda") * H ** -0.5).to(BF16)
        self.ends = torch.arange(1, G + 1, dtype=torch.int32, device="cuda") * (R // G)
        self.res = torch.zeros(R, 512, dtype=BF16, device="cuda")

    def run(self):
        lib.grouped_linear(self.buf, self.w, self.ends, gated=True, out=self.res)
        return self.res


class _Adapters:
    """Many rows (three launches and a workspace) or few (one launch); source
    1's `out` lies in the base rows, which the last launch reads."""

    def __init__(self, T, R=16384):
        self.buf = torch.randn(max(R, T), H, generator=_gen(6), device="cuda").to(BF16)
        self.out1 = self.buf.view(-1)[-T * H:].view(T, H)
        self.base = self.buf[-R:]
        self.x = torch.randn(R, 1024, generator=_gen(7), device="cuda").to(BF16)
        self.down = (torch.randn(4, 32, 1024, generator=_gen(8), device="cuda") / 32).to(BF16)
        self.up = torch.randn(4, H, 32, generator=_gen(9), device="cuda").to(BF16)
        self.slots = (torch.arange(R, device="cuda") % 5 - 1).int()
        self.scales = torch.ones(4, device="cuda")
        self.res = torch.zeros(R, H, dtype=BF16, device="cuda")

    def run(self):
        lib.adapter_add(self.base, self.x, self.down, self.up, self.slots, self.scales, out=self.res)
        return self.res


class _FewAdapters(_Adapters):
    def __init__(self, T):
        super().__init__(T, 100)


class _OtherContext:
    """Another context's combine, whose replies lie in source 1's `out`."""

    def __init__(self, T):
        self.other = afd.Buffer(1, 1, 16, 8, H, 512)
        n = self.other.recv_rows_for_bucket(512)
        self.buf = torch.randn(max(n, T), H, generator=_gen(10), device="cuda").to(BF16)
        self.out1 = self.buf.view(-1)[:T * H].view(T, H)
        self.rows = n
        self.x = torch.randn(512, H, generator=_gen(11), device="cuda").to(BF16)
        self.ids = torch.rand(512, 16, generator=_gen(12), device="cuda").argsort(1)[:, :8].contiguous()
        self.w = torch.rand(512, 8, generator=_gen(13), device="cuda")
        self.res = torch.zeros(512, H, dtype=BF16, device="cuda")

    def run(self):
        self.other.source_dispatch(0, self.x, self.ids, self.w, bucket=512)
        r = self.other.worker_receive(0, bucket=512)
        self.other.worker_reply(0, self.buf[:r.num_rows], r.receipt)
        self.other.source_collect(0, out=self.res)
        return self.res


WORK = dict(gated=_Gated, router=_Router, product=_Product, adapters=_Adapters, few=_FewAdapters, other=_OtherContext)


def _exchange(buf, wl, dev, between, outs):
    for s in range(wl.A):
        buf.source_dispatch(s, dev.x[s], dev.ids[s], dev.w[s], bucket=wl.bucket)
    for f in range(wl.F):
        r = buf.worker_receive(f, bucket=wl.bucket)
        buf.worker_reply(f, r.rows, r.receipt)
    buf.source_collect(0, out=outs[0])
    between()
    buf.source_collect(1, out=outs[1])


@pytest.mark.parametrize("T", [64, 2048])
@pytest.mark.parametrize("name", sorted(WORK))
def test_work_between_two_collects_keeps_its_inputs(name, T):
    wl = W.named("2A2F", T=T)
    inp = W.make_inputs(wl)
    exp = GH.expected(inp, GH.IDENTITY)
    buf = GH.make_buffer(wl)
    try:
        dev = GH.to_device(inp)
        work = WORK[name](T)
        before = work.buf.clone()
        want = work.run().clone()
        outs = [torch.empty(T, H, dtype=BF16, device="cuda"), work.out1]

        def check():
            torch.cuda.synchronize()
            assert torch.equal(work.res, want)
            GH.check_outputs(wl, outs, exp)

        for _ in range(4):
            work.buf.copy_(before)
            work.res.zero_()
            _exchange(buf, wl, dev, work.run, outs)
            check()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _exchange(buf, wl, dev, work.run, outs)
        for _ in range(4):
            work.buf.copy_(before)
            work.res.zero_()
            g.replay()
            check()
        del g
    finally:
        torch.cuda.synchronize()
        buf.close()


@pytest.mark.parametrize("name", ["gated", "adapters", "product"])
def test_a_replayed_graph_between_two_collects(name):
    """The operator's call is not seen then, but the combine starts only when
    the replayed graph has ended: results as above, and (phase-timer build) it
    has nothing left to wait for once its own sums are stored."""
    T = 64
    wl = W.named("2A2F", T=T)
    exp = GH.expected(W.make_inputs(wl), GH.IDENTITY)
    build.build()
    prev = afd.load_library()
    afd.use_library(build.build_timers())
    try:
        dev = GH.to_device(W.make_inputs(wl))
        work = WORK[name](T)
        before = work.buf.clone()
        want = work.run().clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            work.run()
        buf = GH.make_buffer(wl)
        outs = [torch.empty(T, H, dtype=BF16, device="cuda"), work.out1]
        try:
            for _ in range(4):
                work.buf.copy_(before)
                work.res.zero_()
                torch.cuda.synchronize()
                buf.phase_stamps(clear=True)
                _exchange(buf, wl, dev, g.replay, outs)
                torch.cuda.synchronize()
                assert torch.equal(work.res, want)
                GH.check_outputs(wl, outs, exp)
                st = buf.phase_stamps()[3].astype(np.int64)
                st = st[(st[:, :4] > 0).all(1)]
                assert len(st) and (st[:, 3] - st[:, 2]).max() < 3000  # ns; the operators take 17 us and more
            del g
        finally:
            torch.cuda.synchronize()
            buf.close()
    finally:
        afd._lib = prev


@pytest.mark.parametrize("T", [64, 2048])
def test_memory_freed_before_the_second_collect(T):
    """adapter_add's inputs and its workspace go back to the allocator when
    the call returns; the second collect's new tensor may get that block."""
    wl = W.named("2A2F", T=T)
    inp = W.make_inputs(wl)
    exp = GH.expected(inp, GH.IDENTITY)
    buf = GH.make_buffer(wl)
    try:
        dev = GH.to_device(inp)
        work = _Adapters(T)
        want = work.run().clone()
        for _ in range(6):
            outs = []

            def between():
                base = work.base.clone()
                lib.adapter_add(base, work.x.clone(), work.down, work.up, work.slots, work.scales, out=work.res)

            work.res.zero_()
            for s in range(wl.A):
                buf.source_dispatch(s, dev.x[s], dev.ids[s], dev.w[s], bucket=wl.bucket)
            for f in range(wl.F):
                r = buf.worker_receive(f, bucket=wl.bucket)
                buf.worker_reply(f, r.rows, r.receipt)
            outs.append(buf.source_collect(0, num_tokens=T))
            between()
            outs.append(buf.source_collect(1, num_tokens=T))
            torch.cuda.synchronize()
            assert torch.equal(work.res, want)
            GH.check_outputs(wl, outs, exp)
    finally:
        torch.cuda.synchronize()
        buf.close()


@pytest.mark.parametrize("name", [None, "gated", "router", "product", "adapters", "few", "other"])
def test_early_start_only_next_to_each_other(name):
    """The phase-timer build's stamps: the second combine is an early one with
    nothing of the library between the two collects, and never otherwise."""
    build.build()
    prev = afd.load_library()
    afd.use_library(build.build_timers())
    try:
        T = 64
        wl = W.named("2A2F", T=T)
        dev = GH.to_device(W.make_inputs(wl))
        outs = GH.alloc_outs(wl)  # apart from what the operator reads
        work = WORK[name](T) if name else None
        buf = GH.make_buffer(wl)
        try:
            torch.cuda.synchronize()
            buf.phase_stamps(clear=True)
            _exchange(buf, wl, dev, work.run if work else lambda: None, outs)
            torch.cuda.synchronize()
            early = buf.phase_stamps()[3].astype(np.int64)
            assert (early > 0).any() == (name is None)
        finally:
            buf.close()
    finally:
        afd._lib = prev


@pytest.mark.parametrize("T,shift", [(64, 0), (2048, 0), (2048, 1000), ((100, 2048), -64)])
def test_second_result_over_the_first(T, shift):
    """Collects into memory that the results share (the caller's own buffer,
    or a dropped result's block): the later one's rows are the ones that stay,
    and the combines do not run side by side."""
    wl = W.named("2A2F", T=T) if isinstance(T, int) else W.named("2A2F").with_tokens(T)
    exp = GH.expected(W.make_inputs(wl), GH.IDENTITY)
    build.build()
    prev = afd.load_library()
    afd.use_library(build.build_timers())
    try:
        dev = GH.to_device(W.make_inputs(wl))
        buf = GH.make_buffer(wl)
        mem = torch.zeros(2 * wl.bucket, H, dtype=BF16, device="cuda")
        at = 64
        outs = [mem[at:at + wl.T[0]], mem[at + shift:at + shift + wl.T[1]]]

        def check():
            torch.cuda.synchronize()
            got = outs[1].view(torch.int16).cpu().numpy().view(np.uint16)
            assert np.array_equal(got, exp["out"][1, :wl.T[1]])

        try:
            torch.cuda.synchronize()
            buf.phase_stamps(clear=True)
            for _ in range(4):
                _exchange(buf, wl, dev, lambda: None, outs)
                check()
            assert not (buf.phase_stamps()[3].astype(np.int64) > 0).any()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                _exchange(buf, wl, dev, lambda: None, outs)
            for _ in range(4):
                mem.zero_()
                g.replay()
                check()
            del g
        finally:
            torch.cuda.synchronize()
            buf.close()
    finally:
        afd._lib = prev
