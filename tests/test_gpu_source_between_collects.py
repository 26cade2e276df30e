"""The source-side operators between two collects of one exchange: the second
combine waits for them, though its `out` is memory that they read."""
import numpy as np
import pytest
import torch

import combine_attention_ffn_gb300 as lib
import gpu_harness as GH
import test_gpu_between_collects as between
from combine_attention_ffn_gb300 import afd, build
from combine_attention_ffn_gb300 import workloads as W

pytestmark = pytest.mark.gpu
BF16, H = torch.bfloat16, between.H


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class _Norm:
    """16 K rows; source 1's `out` lies in the last ones."""

    def __init__(self, T):
        self.buf = torch.randn(16384, H, generator=between._gen(1), device="cuda").to(BF16)
        self.out1 = self.buf[-T:]
        self.weight = torch.ones(H, dtype=BF16, device="cuda")
        self.res = torch.zeros_like(self.buf)

    def run(self):
        lib.norm_rows(self.buf, self.weight, out=self.res)
        return self.res


class _Write:
    """The keys of 8 K tokens; source 1's `out` lies in the last ones."""

    def __init__(self, T):
        tokens, heads, D = 8192, 16, 128
        self.buf = torch.randn(tokens, heads, D, generator=between._gen(2), device="cuda").to(BF16)
        self.out1 = self.buf.view(-1)[-T * H:].view(T, H)
        self.v = torch.zeros_like(self.buf)
        self.positions = torch.arange(tokens, device="cuda")
        self.freq = torch.rand(64, generator=between._gen(3), device="cuda")
        self.res, self.vc = (torch.zeros(tokens // 64, heads, 64, D, dtype=BF16, device="cuda") for _ in range(2))

    def run(self):
        lib.cache_write(None, self.buf, self.v, self.positions, self.positions, self.res, self.vc, inv_freq=self.freq)
        return self.res


class _Attention:
    """One sequence over 512 pages; source 1's `out` lies in the keys read last."""

    def __init__(self, T):
        pages, heads, D = 512, 2, 128
        self.buf = torch.randn(pages, heads, 64, D, generator=between._gen(4), device="cuda").to(BF16)
        self.out1 = self.buf.view(-1)[-T * H:].view(T, H)
        self.v = torch.randn(pages, heads, 64, D, generator=between._gen(5), device="cuda").to(BF16)
        self.table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
        self.lengths = torch.tensor([pages * 64], dtype=torch.int32, device="cuda")
        self.q = torch.randn(1, 16, D, generator=between._gen(6), device="cuda").to(BF16)
        self.res = torch.zeros(1, 16, D, dtype=BF16, device="cuda")

    def run(self):
        lib.decode_attention(self.q, self.buf, self.v, self.table, self.lengths, out=self.res)
        return self.res


WORK = dict(norm=_Norm, write=_Write, attention=_Attention)


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
        g = torch.cuda.CUDAGraph()
        for i in range(8):
            work.buf.copy_(before)
            work.res.zero_()
            if i == 4:
                with torch.cuda.graph(g):
                    between._exchange(buf, wl, dev, work.run, outs)
            if i < 4:
                between._exchange(buf, wl, dev, work.run, outs)
            else:
                g.replay()
            torch.cuda.synchronize()
            assert torch.equal(work.res, want)
            GH.check_outputs(wl, outs, exp)
        del g
    finally:
        torch.cuda.synchronize()
        buf.close()


@pytest.mark.parametrize("name", sorted(WORK))
def test_no_early_start_behind_them(name):
    """The phase-timer build's stamps: with an operator between the two collects the
    second combine is not one that starts early."""
    prev = afd.load_library()
    afd.use_library(build.build_timers())
    try:
        wl = W.named("2A2F", T=64)
        dev = GH.to_device(W.make_inputs(wl))
        work, buf = WORK[name](64), GH.make_buffer(wl)
        try:
            torch.cuda.synchronize()
            buf.phase_stamps(clear=True)
            between._exchange(buf, wl, dev, work.run, GH.alloc_outs(wl))
            torch.cuda.synchronize()
            assert not (buf.phase_stamps()[3].astype(np.int64) > 0).any()
        finally:
            buf.close()
    finally:
        afd._lib = prev
