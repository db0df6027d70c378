"""A layer's way through the paged cache: two prompts, then verify steps.

The four calls as a server uses them:

  prompts   qk_norm_rope -> paged_kv_append -> window_attn over the packed rows
  steps     paged_kv_append (queries, keys and values in one call) -> paged_attn,
            captured once in a CUDA graph and replayed with new lengths, slots
            and rows

The "projections" are random rows, as there is no model here; every output is
compared with a plain computation in 64 bits over the same rows.

    python examples/paged_serving.py [--e4m3] [--window 96 --sinks 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verify_08_gb300 as sv  # noqa: E402

HQ, HKV, D, PAGE, WIDTH, M, EPS = 24, 4, 256, 64, 16, 4, 1e-6
ROT = 64
INV_FREQ = 10000.0 ** (-torch.arange(0, ROT, 2, dtype=torch.float64) / ROT)
SCALE = D ** -0.5


def plain_rows(x, weight, positions):
    """Norm (zero-centred weights) and rotation of rows [T, heads, D], float64."""
    x = x.double()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (weight.double() + 1)
    a = positions.double()[:, None] * INV_FREQ.to(x.device)
    c, s = a.cos()[:, None], a.sin()[:, None]
    u, v = x[..., :ROT // 2], x[..., ROT // 2:ROT]
    return torch.cat((u * c - v * s, u * s + v * c, x[..., ROT:]), -1)


def plain_attention(q, k, v, first, window, sinks):
    """Rows q [n, HQ, D] at positions first.. over k and v [N, HKV, D], float64."""
    j = torch.arange(k.shape[0], device=q.device)
    p = (torch.arange(q.shape[0], device=q.device) + first)[:, None]
    seen = (j <= p) & ((j > p - window) | (j < sinks)) if window else j <= p
    x = torch.einsum("ihgd,nhd->hgin", q.double().view(-1, HKV, HQ // HKV, D), k.double()) * SCALE
    w = torch.softmax(x.masked_fill(~seen, float("-inf")), -1)
    return torch.einsum("hgin,nhd->ihgd", w, v.double()).reshape(-1, HQ, D)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--e4m3", action="store_true", help="8-bit pages")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    ap.add_argument("--steps", type=int, default=6)
    a = ap.parse_args(argv)
    sv.load()
    dev, g = "cuda", torch.Generator(device="cuda").manual_seed(0)
    prompts = [150, 37]
    B = len(prompts)
    seen = dict(window=a.window, sinks=a.sinks)
    phases = sv.rope_phases(INV_FREQ)
    qw, kw = ((torch.randn(D, generator=g, device=dev) * 0.1).bfloat16() for _ in range(2))
    norm = dict(q_weight=qw, k_weight=kw, eps=EPS, weight_offset=1.0)

    # a pool of pages shared by the sequences, handed out in no order
    typ = torch.float8_e4m3fn if a.e4m3 else torch.bfloat16
    pool = [torch.zeros(B * WIDTH, HKV, PAGE, D, device=dev).to(typ) for _ in range(2)]
    scales = [torch.full((HKV,), s, device=dev) for s in (0.02, 0.01)] if a.e4m3 else [None, None]
    cache = sv.PagedKV(*pool, layout="HND", k_scale=scales[0], v_scale=scales[1])
    table = torch.randperm(B * WIDTH, generator=g, device=dev).int().view(B, WIDTH)

    def slots_of(b, positions):
        return table[b, positions // PAGE].long() * PAGE + positions % PAGE

    def projected(n):  # queries, keys and values of n tokens, heads side by side
        return torch.randn(n, HQ + 2 * HKV, D, generator=g, device=dev).bfloat16()

    # ---- the prompts, packed ----
    x = projected(sum(prompts))
    q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
    pos = torch.cat([torch.arange(n, device=dev) for n in prompts])
    slots = torch.cat([slots_of(b, torch.arange(n, device=dev)) for b, n in enumerate(prompts)])
    cu = torch.tensor([0, prompts[0], sum(prompts)], dtype=torch.int32, device=dev)
    qr, kr = (torch.empty(len(x), h, D, dtype=torch.bfloat16, device=dev) for h in (HQ, HKV))
    o = torch.empty_like(qr)
    sv.qk_norm_rope(q, k, qr, kr, pos.int(), phases, **norm)
    sv.paged_kv_append(kr, v, cache, slots)
    sv.window_attn(qr, kr, v, o, cu, cu, SCALE,
                   workspace=sv.workspace(sv.window_attn_workspace_bytes(B, HQ, HKV, D)), **seen)
    worst, K, V = 0.0, [], []
    for b in range(B):
        r = slice(int(cu[b]), int(cu[b + 1]))
        K.append(plain_rows(k[r], kw, pos[r]))
        V.append(v[r].double())
        want = plain_attention(plain_rows(q[r], qw, pos[r]), K[b], V[b], 0, a.window, a.sinks)
        worst = max(worst, float((o[r] - want).abs().max()))
    print(f"prompts of {prompts} rows: largest difference {worst:.2e}")

    # ---- verify steps of M rows a sequence, in one graph ----
    x = projected(B * M)
    lens = torch.tensor(prompts, dtype=torch.int32, device=dev)
    pos = torch.zeros(B * M, dtype=torch.int32, device=dev)
    slots = torch.full((B * M,), -1, dtype=torch.int64, device=dev)
    qr, o = (torch.empty(B * M, HQ, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    ws = sv.workspace(sv.paged_attn_workspace_bytes(B, M, HQ, HKV, D))

    def step():
        sv.paged_kv_append(x[:, HQ:HQ + HKV], x[:, HQ + HKV:], cache, slots, q=x[:, :HQ], q_out=qr, positions=pos,
                           phases=phases, **norm)
        sv.paged_attn(qr, cache, table, lens, o, M, SCALE, workspace=ws, **seen)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # once outside the capture: slots of -1 write nothing
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    accepted = list(prompts)  # tokens of each sequence that stay
    for n in range(a.steps):
        x.copy_(projected(B * M))
        at = torch.tensor([[accepted[b] + i for i in range(M)] for b in range(B)], device=dev)
        pos.copy_(at.flatten())
        slots.copy_(torch.cat([slots_of(b, at[b]) for b in range(B)]))
        lens.copy_(at[:, -1] + 1)
        graph.replay()
        for b in range(B):
            r = slice(b * M, (b + 1) * M)
            K[b] = torch.cat((K[b][:accepted[b]], plain_rows(x[r, HQ:HQ + HKV], kw, pos[r])))
            V[b] = torch.cat((V[b][:accepted[b]], x[r, HQ + HKV:].double()))
            want = plain_attention(plain_rows(x[r, :HQ], qw, pos[r]), K[b], V[b], accepted[b], a.window, a.sinks)
            worst = max(worst, float((o[r] - want).abs().max()))
            accepted[b] += 1 + (n + b) % M  # the first row and some drafts; the rest is overwritten
    assert sv.sv_last_device_error() == sv.SV_OK
    print(f"{a.steps} verify steps of {M} rows: largest difference {worst:.2e}, lengths {accepted}")
    return worst


if __name__ == "__main__":
    main()
