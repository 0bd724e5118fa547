"""Decoder operators in use at the same time: threads on streams of their own,
and captured graphs replayed in turn with eager calls between them.  Results
are the lone calls' own, bit by bit."""
import os
import threading

import pytest
import torch

import implicit_gemm_nhwc_amd as igc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def setup_module(_):
    if not (os.path.exists(igc.LIB_PATH) and os.path.exists(igc.POISON_LIB_PATH)):
        import __graft_entry__
        __graft_entry__.build()


class _Step:
    """One step of a decoder's operators over inputs of its own; lengths above
    the split's least and below it, rows above one workgroup's."""

    def __init__(self, seed, tokens, heads, d, capacity):
        gen = torch.Generator().manual_seed(seed)

        def rnd(*shape):
            return torch.randn(*shape, generator=gen)

        b, c, page = 3, heads * d, 32
        self.entries = capacity // page
        self.x, self.dy = (rnd(b, tokens, c).bfloat16().to(DEV) for _ in range(2))
        self.w, self.bias = (1 + 0.3 * rnd(c)).to(DEV), (0.3 * rnd(c)).to(DEV)
        self.wq, self.ws = igc.quantize_rows(rnd(3 * c, c).bfloat16().to(DEV))
        self.cache = igc.KVCache.empty(b * self.entries, page, heads, d, device=DEV)
        for t in (self.cache.k, self.cache.v):
            t.copy_(torch.randint(-128, 128, t.shape, generator=gen, dtype=torch.int8))
        for t in (self.cache.k_scale, self.cache.v_scale):
            t.copy_(0.01 + 0.02 * torch.rand(t.shape, generator=gen))
        self.table = torch.randperm(b * self.entries, generator=gen).view(b, -1).int().to(DEV)
        self.lens = torch.tensor([capacity, capacity // 2, tokens], dtype=torch.int32, device=DEV)
        self.start = self.lens - tokens
        self.heads, self.d = heads, d

    def run(self):
        n = igc.layer_norm(self.x, self.w, self.bias)
        q, s = igc.quantize_rows(n)
        y = igc.linear_i8(q, s, self.wq, self.ws).view(*n.shape[:2], 3, self.heads, self.d)
        igc.kv_cache_write(self.cache, y[:, :, 1], y[:, :, 2], self.table, self.start)
        out, lse = igc.cache_attention(y[:, :, 0], self.cache, self.table, self.lens,
                                       return_lse=True)
        back = igc.kv_cache_read(self.cache, self.table, self.start, n.shape[1])
        return (out, lse, *back, *igc.layer_norm_bwd(self.dy, self.x, self.w))


STEPS = [(1, 1, 4, 128, 4096), (2, 5, 8, 80, 1024), (3, 40, 2, 64, 2048), (4, 1, 2, 32, 96)]


def _same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def test_threads_on_streams_of_their_own():
    steps = [_Step(*a) for a in STEPS]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = steps[i].run()
                stream.synchronize()
                if not _same(got, want[i]):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(steps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_graphs_replayed_in_turn():
    steps = [_Step(*a) for a in STEPS]
    want = [s.run() for s in steps]
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = s.run()
        graphs.append((g, got))
    for _ in range(4):
        for (g, got), s, w in zip(graphs, steps, want):
            for t in got:
                t.zero_()
            g.replay()
            assert _same(s.run(), w)   # eager, behind the replay
            torch.cuda.synchronize()
            assert _same(got, w)


# steps whose attention divides the card by the sequences' lengths
DIVIDED = [(5, 1, 32, 24, 4096), (6, 3, 40, 16, 2048), (7, 1, 4, 128, 65536)]


@pytest.mark.parametrize("run", [test_threads_on_streams_of_their_own, test_graphs_replayed_in_turn])
def test_with_divisions_by_lengths(run, monkeypatch):
    for seed, tokens, heads, d, capacity in DIVIDED:
        cache = igc.KVCache.empty(1, 32, heads, d, device=DEV)
        need = igc.cache_attn_fwd_workspace_bytes((3, tokens, heads, d), cache, capacity // 32,
                                                  torch.bfloat16)
        room = need // (heads * tokens * (d + 2) * 4)
        assert 3 < room < 3 * (capacity // 256)   # parts, of 256 keys at least
    monkeypatch.setitem(globals(), "STEPS", DIVIDED)
    run()
