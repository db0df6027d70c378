"""A full-attention and a recurrent layer through the serving of three sequences.

Prompts come in chunks beside the tokens of sequences that already generate, then
all of them run verify steps:

  chunks   paged_kv_append -> paged_chunk_attn over the pages, and gdn_chunk over the
           pool of states: ragged rows of all sequences in one call each
  steps    paged_kv_append -> paged_attn, and gdn_step, which first applies what the last
           round accepted: captured once in a CUDA graph and replayed with new lengths,
           slots, counts and rows
  between  a sequence whose next rows go through gdn_chunk has its accepted rows
           committed first (gdn_step with M = 0)

The "projections" are random rows, as there is no model here; every output is
compared with a plain computation in 64 bits over the same rows.

    python examples/hybrid_serving.py [--e4m3] [--window 96 --sinks 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verify_08_gb300 as sv  # noqa: E402

HQ, HKV, D, PAGE, WIDTH = 16, 2, 128, 32, 16   # attention heads, pages, entries of a table's row
HK, HV, DK, DV = 4, 8, 128, 128                # recurrent heads
M, SCALE = 4, 128 ** -0.5
# rows of each sequence in the calls before the verify steps: prompts in pieces, single tokens between them
CHUNKS = [[100, 0, 33], [61, 90, 1], [1, 130, 1]]


class Sequence:
    """What a sequence has seen, for the plain forms (CPU, float64)."""

    def __init__(self):
        self.k, self.v = torch.zeros(0, HKV, D, dtype=torch.float64), torch.zeros(0, HKV, D, dtype=torch.float64)
        self.state = torch.zeros(HV, DV, DK, dtype=torch.float64)

    def attend(self, q, k, v, a):
        """Rows q behind what is kept and the rows before them: outputs; nothing is kept."""
        K, V = torch.cat((self.k, k)), torch.cat((self.v, v))
        j, p = torch.arange(len(K)), torch.arange(len(self.k), len(K))[:, None]
        seen = (j <= p) & ((j > p - a.window) | (j < a.sinks)) if a.window else j <= p
        x = torch.einsum("ihgd,nhd->hgin", q.double().view(-1, HKV, HQ // HKV, D), K) * SCALE
        w = torch.softmax(x.masked_fill(~seen, float("-inf")), -1)
        return torch.einsum("hgin,nhd->ihgd", w, V).reshape(-1, HQ, D)

    def recur(self, q, k, v, g, beta):
        """States after each row, and the outputs."""
        S, states, out = self.state, [self.state], []
        for t in range(len(q)):
            kt, qt = (x[t].double().repeat_interleave(HV // HK, 0) for x in (k, q))
            S = S * torch.exp(g[t].double())[:, None, None]
            u = beta[t].double()[:, None] * (v[t].double() - torch.einsum("hvk,hk->hv", S, kt))
            S = S + u[:, :, None] * kt[:, None, :]
            states.append(S)
            out.append(torch.einsum("hvk,hk->hv", S, qt))
        return states, torch.stack(out)

    def keep(self, k, v, state):
        self.k, self.v, self.state = torch.cat((self.k, k)), torch.cat((self.v, v)), state


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--e4m3", action="store_true", help="8-bit pages")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args(argv)
    sv.load()
    dev, gen = "cuda", torch.Generator().manual_seed(0)
    B = len(CHUNKS[0])
    seen = dict(window=a.window, sinks=a.sinks)
    typ = torch.float8_e4m3fn if a.e4m3 else torch.bfloat16

    # pages and states shared by the sequences, handed out in no order
    cache = sv.PagedKV(*(torch.zeros(B * WIDTH, PAGE, HKV, D, device=dev).to(typ) for _ in range(2)))
    table = torch.randperm(B * WIDTH, generator=gen).int().view(B, WIDTH)
    states = torch.zeros(B + 2, HV, DV, DK, device=dev)
    places = torch.tensor([4, 0, 3], dtype=torch.int32)
    on_gpu = dict(table=table.to(dev), places=places.to(dev))

    def slots_of(b, first, n):
        at = torch.arange(first, first + n)
        return table[b, at // PAGE].long() * PAGE + at % PAGE

    def projected(n):
        """Rows of both layers: attention q, k, v; recurrent q, k, v, log decay, strength."""
        r = lambda *s: torch.randn(*s, generator=gen)
        unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).bfloat16()
        return [r(n, HQ, D).bfloat16(), r(n, HKV, D).bfloat16(), r(n, HKV, D).bfloat16(), unit(r(n, HK, DK)),
                unit(r(n, HK, DK)), r(n, HV, DV).bfloat16(), -torch.rand(n, HV, generator=gen), torch.rand(n, HV, generator=gen)]

    def held(x):  # what a page keeps of a row
        return x.to(typ).double()

    seqs, worst = [Sequence() for _ in range(B)], dict(attention=0.0, outputs=0.0, states=0.0)

    def note(what, got, want):
        worst[what] = max(worst[what], float((got.double().cpu() - want).abs().max()) if want.numel() else 0.0)

    # ---- chunks ----
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    for sizes in CHUNKS:
        T, lens = sum(sizes), [len(s.k) + n for s, n in zip(seqs, sizes)]
        cu = torch.tensor([0] + sizes).cumsum(0).tolist()
        rows = projected(T)
        q, k, v, rq, rk, rv, rg, rb = (x.to(dev) for x in rows)
        slots = torch.cat([slots_of(b, len(seqs[b].k), n) for b, n in enumerate(sizes)])
        o, ro = torch.empty_like(q), torch.empty_like(rv)
        sv.paged_kv_append(k, v, cache, slots.to(dev))
        sv.paged_chunk_attn(q, cache, on_gpu["table"], ints(lens), o, ints(cu), SCALE,
                            workspace=sv.workspace(sv.paged_chunk_attn_workspace_bytes(B, T, HQ, HKV, D)), **seen)
        sv.gdn_chunk(states, on_gpu["places"], rq, rk, rv, rg, rb, ro, ints(cu),
                     workspace=sv.workspace(sv.gdn_chunk_workspace_bytes(B, T, HK, HV, DK, DV)))
        for b, s in enumerate(seqs):
            r = slice(cu[b], cu[b + 1])
            if not sizes[b]:
                continue
            q, k, v, *rec = (x[r] for x in rows)
            note("attention", o[r], s.attend(q, held(k), held(v), a))
            after, out = s.recur(*rec)
            note("outputs", ro[r], out)
            s.keep(held(k), held(v), after[-1])
    for b, s in enumerate(seqs):
        note("states", states[places[b]], s.state)
    assert sv.sv_last_device_error() == sv.SV_OK
    print(f"chunks of {CHUNKS} rows: largest differences {worst}")

    # ---- verify steps of M rows a sequence, in one graph ----
    new = [x.to(dev) for x in projected(B * M)]
    q, k, v, *rec = new
    tape = [torch.zeros_like(x) for x in rec[1:]]          # keys, values, decays, strengths of the last round
    counts = torch.zeros(B, dtype=torch.int32, device=dev)
    lens = ints([len(s.k) for s in seqs])
    slots = torch.full((B * M,), -1, dtype=torch.int64, device=dev)
    o, ro = torch.empty_like(q), torch.empty_like(rec[2])
    ws = sv.workspace(sv.paged_attn_workspace_bytes(B, M, HQ, HKV, D))

    def step():
        sv.paged_kv_append(k, v, cache, slots)
        sv.paged_attn(q, cache, on_gpu["table"], lens, o, M, SCALE, workspace=ws, **seen)
        sv.gdn_step(states, on_gpu["places"], *rec, ro, M, tape=tape, n_replay=counts)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # once outside the capture: slots of -1 and counts of 0 change nothing
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(a.steps):
        for t, x in zip(tape, rec[1:]):
            t.copy_(x)                                     # the last round's rows; `counts` says how many stay
        rows = projected(B * M)
        for x, r in zip(new, rows):
            x.copy_(r)
        slots.copy_(torch.cat([slots_of(b, len(s.k), M) for b, s in enumerate(seqs)]))
        lens.copy_(ints([len(s.k) + M for s in seqs]))
        graph.replay()
        taken = [1 + (n + b) % M for b in range(B)]        # the first row and some drafts
        for b, s in enumerate(seqs):
            r = slice(b * M, (b + 1) * M)
            qb, kb, vb, *recb = (x[r] for x in rows)
            note("attention", o[r], s.attend(qb, held(kb), held(vb), a))
            after, out = s.recur(*recb)
            note("outputs", ro[r], out)
            note("states", states[places[b]], s.state)     # as it stood before this round's rows
            s.keep(held(kb[:taken[b]]), held(vb[:taken[b]]), after[taken[b]])
        counts.copy_(ints(taken))

    # ---- the last round's accepted rows committed: chunks may follow ----
    sv.gdn_step(states, on_gpu["places"], *[None] * 6, 0, tape=rec[1:], n_replay=counts)
    for b, s in enumerate(seqs):
        note("states", states[places[b]], s.state)
    assert sv.sv_last_device_error() == sv.SV_OK
    assert not states[[1, 2]].any()                        # places of no sequence
    print(f"{a.steps} verify steps of {M} rows: largest differences {worst}, lengths {[len(s.k) for s in seqs]}")
    return worst


if __name__ == "__main__":
    main()
