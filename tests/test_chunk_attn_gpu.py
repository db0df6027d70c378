"""paged_chunk_attn against softmax attention in 64 bits.

An output is off by its own rounding and by that of each probability (half a step
of bf16 each, of values at most the largest |v|), and by fp32 arithmetic over the
slots, far below both (paged_plain.attention_tolerance); over e4m3 pages the
probabilities' fp16 rounding and the queries' are smaller still."""
import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu


def attend(q, K, V, first, scale, window, sinks):
    """q [n, Hq, D] at positions first.., K and V [N, Hkv, D], float64: [n, Hq, D]."""
    n, Hq, _ = q.shape
    G = Hq // K.shape[1]
    p, j = torch.arange(first, first + n)[:, None], torch.arange(K.shape[0])
    seen = (j <= p) & ((j > p - window) | (j < sinks)) if window else (j <= p)
    x = torch.einsum("nhd,khd->hnk", q.double(), K.repeat_interleave(G, 1)) * scale
    x = x.masked_fill(~seen[None], float("-inf"))
    w = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
    return torch.einsum("hnk,khd->nhd", w, V.repeat_interleave(G, 1))


class Call:
    """Sequences of (new rows, slots) over pages placed at random, and the call on them."""

    def __init__(self, sv, seqs, Hq, Hkv, D, page, layout="NHD", e4m3=False, window=0, sinks=0, seed=0, extra=0,
                 dirty=True, gain=1.0):
        self.sv, self.seqs, self.D, self.window, self.sinks = sv, seqs, D, window, sinks
        g = torch.Generator().manual_seed(seed)
        self.T = sum(n for n, _ in seqs)
        width = max([1] + [-(-L // page) for _, L in seqs])
        used = [-(-L // page) for _, L in seqs]
        pages = sum(used) + 3
        typ = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        shape = (pages, page, Hkv, D) if layout == "NHD" else (pages, Hkv, page, D)
        self.k, self.v = ((torch.randn(shape, generator=g) * gain).to(typ) for _ in range(2))
        self.ks, self.vs = ((torch.rand(Hkv, generator=g) + 0.5) if e4m3 else None for _ in range(2))
        order = torch.randperm(pages, generator=g).int()
        self.table = torch.full((len(seqs), width), -1, dtype=torch.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        self.lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
        self.cu = torch.tensor([0] + list(torch.tensor([n for n, _ in seqs]).cumsum(0)), dtype=torch.int32)
        # queries are slices of wider rows
        self.q = torch.randn(self.T + extra, Hq + 2 * Hkv, D, generator=g).bfloat16()
        self.scale, self.Hq, self.Hkv, self.page, self.layout = D ** -0.5, Hq, Hkv, page, layout
        self.want = []
        for b, (n, L) in enumerate(seqs):
            K = plain.gather(self.k.float(), self.table[b], L, page, layout, self.ks) if L else torch.zeros(0, Hkv, D, dtype=torch.float64)
            V = plain.gather(self.v.float(), self.table[b], L, page, layout, self.vs) if L else torch.zeros(0, Hkv, D, dtype=torch.float64)
            rows = self.q[int(self.cu[b]):int(self.cu[b + 1]), :Hq]
            o = attend(rows, K, V, L - n, self.scale, window, sinks) if L else torch.zeros(n, Hq, D, dtype=torch.float64)
            self.want.append(o)
        self.most = float(self.v.float().abs().max()) * (float(self.vs.max()) if e4m3 else 1.0)
        if dirty:  # NaN wherever no row of the sequence looks, the unused pages among it
            view = [x.float() for x in (self.k, self.v)]
            kept = torch.zeros(pages, page, dtype=torch.bool)
            for b, (n, L) in enumerate(seqs):
                low = max(0, L - n - window + 1) if window and n else (0 if n else L)
                for j in range(L):
                    if n and (j >= low or j < sinks):
                        kept[int(self.table[b, j // page]), j % page] = True
                for x in range(used[b]):  # entries of pages that no row looks at
                    if not kept[int(self.table[b, x])].any():
                        self.table[b, x] = 0x7fffffff
            for x in view:
                (x if layout == "NHD" else x.transpose(1, 2))[~kept] = float("nan")
            self.k, self.v = (x.to(typ) for x in view)

    def tensors(self):
        c = "cuda"
        cache = self.sv.PagedKV(self.k.to(c), self.v.to(c), layout=self.layout,
                                k_scale=None if self.ks is None else self.ks.to(c),
                                v_scale=None if self.vs is None else self.vs.to(c))
        q = self.q.to(c)
        o = torch.full((q.shape[0], self.Hq, self.D), 99.0, device=c, dtype=torch.bfloat16)
        ws = self.sv.workspace(self.sv.paged_chunk_attn_workspace_bytes(len(self.seqs), q.shape[0], self.Hq, self.Hkv, self.D))
        return q[:, :self.Hq], cache, self.table.to(c), self.lens.to(c), o, self.cu.to(c), ws

    def run(self, t=None):
        q, cache, table, lens, o, cu, ws = t or self.tensors()
        self.sv.paged_chunk_attn(q, cache, table, lens, o, cu, self.scale, window=self.window, sinks=self.sinks, workspace=ws)
        return o

    def check(self):
        o = self.run()
        assert self.sv.sv_last_device_error() == self.sv.SV_OK
        got = o[:self.T].double().cpu()
        assert torch.isfinite(got).all()
        want = torch.cat(self.want)
        off = (got - want).abs().max() if self.T else 0.0
        assert float(off) <= plain.attention_tolerance(self.most), float(off)
        for b, (n, L) in enumerate(self.seqs):  # rows before position 0 see nothing
            blind = min(n, max(0, n - L))
            assert bool((got[int(self.cu[b]):int(self.cu[b]) + blind] == 0).all())
        assert bool((o[self.T:] == 99.0).all())


RAGGED = [(1, 1), (3, 40), (77, 77), (1, 300), (130, 515), (64, 64)]


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 128), (8, 2, 128), (3, 3, 128), (6, 1, 256), (12, 2, 256), (2, 2, 256), (40, 1, 128)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_heads(cuda_lib, Hq, Hkv, D, e4m3):
    Call(cuda_lib, RAGGED, Hq, Hkv, D, 16, e4m3=e4m3, seed=Hq + D, extra=5).check()


@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("D,e4m3", [(128, False), (256, False), (128, True), (256, True)])
def test_pages(cuda_lib, page, layout, D, e4m3):
    Call(cuda_lib, [(100, 301), (33, 513), (2, 130)], 4, 2, D, page, layout=layout, e4m3=e4m3, seed=page).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (100, 0), (128, 4), (130, 33), (64, 200), (1000, 3), (17, 128)])
@pytest.mark.parametrize("D,e4m3,page", [(128, False, 16), (256, False, 64), (128, True, 32), (256, True, 48)])
def test_windows(cuda_lib, window, sinks, D, e4m3, page):
    Call(cuda_lib, [(1, 900), (150, 777), (300, 300), (20, 2000), (5, 3)], 4, 2, D, page, e4m3=e4m3, window=window,
         sinks=sinks, seed=window + sinks).check()


@pytest.mark.parametrize("seqs", [
    [(0, 0)], [(0, 50), (1, 1)], [(5, 0), (5, 3), (5, 5)], [(200, 60)], [(1, 0), (0, 7), (2, 9)],
], ids=["nothing", "no_rows", "short", "longer_than_the_cache", "mixed"])
@pytest.mark.parametrize("D,e4m3", [(128, False), (256, True)])
def test_rows_that_see_nothing(cuda_lib, seqs, D, e4m3):
    Call(cuda_lib, seqs, 4, 2, D, 16, e4m3=e4m3, seed=3, extra=2).check()


@pytest.mark.parametrize("seqs", [[(1, 20000)], [(3, 9001), (1, 12345)], [(61, 6000)], [(200, 8000), (1, 1), (7, 3333)]],
                         ids=["token", "two", "few", "three"])
@pytest.mark.parametrize("Hq,Hkv,D,e4m3", [(4, 1, 128, False), (6, 1, 256, False), (4, 1, 128, True), (6, 1, 256, True)])
def test_long_caches_are_cut_and_joined(cuda_lib, seqs, Hq, Hkv, D, e4m3):
    Call(cuda_lib, seqs, Hq, Hkv, D, 64, e4m3=e4m3, seed=5, dirty=False).check()


def test_a_window_behind_a_long_cache(cuda_lib):
    Call(cuda_lib, [(40, 15000), (600, 9000)], 4, 1, 128, 32, window=4000, sinks=70, seed=6).check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_sequences(cuda_lib, e4m3):
    """More than the prefix sums' place in the header holds."""
    Call(cuda_lib, [(i % 3, 1 + 7 * i % 90) for i in range(400)], 2, 1, 128, 16, e4m3=e4m3, seed=7).check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_scores_far_apart(cuda_lib, e4m3):
    """Logits of hundreds: the running maximum is raised over and over, in both pieces of cut items."""
    Call(cuda_lib, [(30, 3000), (129, 1000)], 4, 2, 128, 16, e4m3=e4m3, seed=8, gain=16.0, dirty=False).check()


def test_queries_of_any_size(cuda_lib):
    """Beside e4m3 pages queries are two e4m3 parts behind a power of two a row."""
    c = Call(cuda_lib, [(60, 200)], 4, 2, 128, 16, e4m3=True, seed=9, dirty=False)
    for size in (1e-30, 1e-3, 1e4, 1e30):
        c.q = (torch.randn(60, 8, 128, generator=torch.Generator().manual_seed(1)) * size).bfloat16()
        c.scale = 128 ** -0.5 / size
        K = plain.gather(c.k.float(), c.table[0], 200, 16, "NHD", c.ks)
        V = plain.gather(c.v.float(), c.table[0], 200, 16, "NHD", c.vs)
        c.want = [attend(c.q[:, :4], K, V, 140, c.scale, 0, 0)]
        if 1e-35 < c.scale < 1e35:
            c.check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_queries_that_are_not_finite(cuda_lib, e4m3):
    """They reach their own rows only, and none that sees nothing."""
    sv = cuda_lib
    c = Call(sv, [(5, 2), (9, 40)], 4, 2, 128, 16, e4m3=e4m3, seed=13, dirty=False)
    t = c.tensors()
    good = c.run(t).clone()
    t[0][0] = float("nan")             # rows 0..2 stand before position 0
    t[0][1, :, 3] = float("inf")
    t[0][8, 1, 100] = float("nan")
    t[0][9, 2, 5] = float("inf")
    o = c.run(t)
    assert sv.sv_last_device_error() == sv.SV_OK
    assert bool((o[:3] == 0).all())
    assert bool(o[8, 1].isnan().all())
    good[8, 1] = good[9, 2] = 0
    o[8, 1] = o[9, 2] = 0
    assert torch.equal(o, good)


def test_pages_lengths_and_offsets_out_of_range(cuda_lib):
    """Needed pages outside the cache count as zeros, lengths as the nearest in range; sequences
    whose offsets are out of order or range are left out; all are reported."""
    sv = cuda_lib
    for e4m3 in (False, True):
        c = Call(sv, [(4, 40), (5, 50)], 2, 1, 128, 16, e4m3=e4m3, seed=10, dirty=False)
        t = list(c.tensors())
        good = c.run(t).clone()
        assert sv.sv_last_device_error() == sv.SV_OK
        bad = t[2].clone()
        bad[0, 1], bad[1, 0] = 1 << 30, -5
        o = c.run([t[0], t[1], bad] + t[3:]).clone()
        assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
        for b, hole in ((0, 16), (1, 0)):
            n, L = c.seqs[b]
            K, V = (plain.gather(x.float(), c.table[b], L, 16, "NHD", s) for x, s in ((c.k, c.ks), (c.v, c.vs)))
            K[hole:hole + 16] = 0
            V[hole:hole + 16] = 0
            rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
            want = attend(c.q[rows, :2], K, V, L - n, c.scale, 0, 0)
            assert float((o[rows].double().cpu() - want).abs().max()) <= plain.attention_tolerance(c.most)
        lens = torch.tensor([-3, 1 << 20], dtype=torch.int32, device="cuda")
        c.run(t[:3] + [lens] + t[4:])
        assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
        for cu, left in (([0, 4, 10], 0), ([0, 4, 2], 0), ([-1, 4, 9], 1)):
            t[4].fill_(7.0)
            o = c.run(t[:5] + [torch.tensor(cu, dtype=torch.int32, device="cuda")] + t[6:])
            assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
            mine = slice(int(c.cu[left]), int(c.cu[left + 1]))
            assert torch.equal(o[mine], good[mine])
            other = slice(int(c.cu[1 - left]), int(c.cu[2 - left]))
            assert bool((o[other] == 7.0).all())
    assert sv.sv_last_device_error() == sv.SV_OK


@pytest.mark.parametrize("e4m3", [False, True])
def test_bits_repeat_and_a_captured_call_follows_its_inputs(cuda_lib, e4m3):
    sv = cuda_lib
    c = Call(sv, [(50, 3000), (3, 4000), (200, 300)], 4, 1, 128, 32, e4m3=e4m3, seed=11, dirty=False)
    t = c.tensors()
    first = c.run(t).clone()
    for _ in range(3):
        assert torch.equal(c.run(t), first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(t)
    graph.replay()
    assert torch.equal(t[4], first)
    t[3].copy_(torch.tensor([1000, 77, 300])), t[5].copy_(torch.tensor([0, 100, 101, 253]))
    graph.replay()
    got = t[4].clone()
    t[4].fill_(0)
    assert torch.equal(c.run(t), got) and not torch.equal(got, first)
    assert sv.sv_last_device_error() == sv.SV_OK


def test_single_tokens_as_paged_attn(cuda_lib):
    """One row each: what paged_attn gives, to rounding."""
    sv = cuda_lib
    c = Call(sv, [(1, L) for L in (1, 17, 400, 3000)], 8, 2, 128, 16, seed=12, dirty=False)
    t = c.tensors()
    a = c.run(t).clone()
    o = torch.empty_like(a)
    ws = sv.workspace(sv.paged_attn_workspace_bytes(4, 1, 8, 2, 128))
    sv.paged_attn(t[0], t[1], t[2], t[3], o, 1, c.scale, workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_OK
    assert float((a.float() - o.float()).abs().max()) <= 2 * plain.attention_tolerance(c.most)
