"""What the paged-cache operators are measured on: their cases, inputs and plain forms.

Four operators that together take the rows of a layer's q/k/v projection to its attention output:

    qk_norm_rope     RMS norm of every query and key head and the position rotation, in one pass
    paged_kv_append  keys (normed and rotated on the way) and values written to the pages of a
                     cache shared by many sequences; the queries' rows in the same call
    paged_attn       the newest M rows of each sequence (M = 1: one new token) over that cache,
                     with a sliding window and a few first tokens that stay visible
    window_attn      the same attention for whole prompts, packed one after the other

``run`` computes them in elementary torch operations in 32 bits (angles in 64), or, where ``own`` is
true, through the package's entry points.  ``exact`` computes them in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
DEV = "cuda"


def _sv():
    import speculative_decoding_verify_08_gb300 as sv
    return sv


# ------------------------------------------------------------------ cases ----
# 24 query heads over 4 KV heads of 256 are this repository's own attention layer (a 27B-class
# hybrid target; norms with zero-centred weights, a quarter of the head rotated); 32 over 8 of 128 and 16 over 16 of 128 are
# the usual grouped and ungrouped layouts.
def listed():
    return [
        # the M = 4 rows of one sequence's verify step
        dict(name="norm_rope_verify_4", op="qk_norm_rope", tokens=4, hq=24, hkv=4, d=256, rot=64,
             offset=1.0, interleaved=False, far=40000),
        # the rows of a long prompt (or of several), odd in number
        dict(name="norm_rope_prompt_16381", op="qk_norm_rope", tokens=16381, hq=32, hkv=8, d=128, rot=128,
             offset=0.0, interleaved=False, far=131072),
        # one token for each of 61 sequences: queries, keys and values in one call
        dict(name="append_decode_61", op="paged_kv_append", tokens=61, hq=32, hkv=8, d=128, rot=128,
             offset=0.0, interleaved=True, far=131072, page=16, layout="NHD", e4m3=False, queries=True),
        # a prompt's keys and values into 8-bit pages, without the queries
        dict(name="append_prompt_30011_e4m3", op="paged_kv_append", tokens=30011, hq=24, hkv=4, d=256, rot=64,
             offset=1.0, interleaved=False, far=40000, page=64, layout="HND", e4m3=True, queries=False),
        # one new token of one short conversation: latency
        dict(name="decode_1x777", op="paged_attn", batch=1, rows=1, lo=777, hi=777, hq=24, hkv=4, d=256,
             page=16, layout="NHD", e4m3=False, window=0, sinks=0),
        # the verify step of one sequence at 32K
        dict(name="verify_1x32768", op="paged_attn", batch=1, rows=4, lo=32768, hi=32768, hq=24, hkv=4, d=256,
             page=64, layout="HND", e4m3=False, window=0, sinks=0),
        # one new token for 48 ragged conversations
        dict(name="decode_48_ragged", op="paged_attn", batch=48, rows=1, lo=40, hi=16000, hq=32, hkv=8, d=128,
             page=16, layout="NHD", e4m3=False, window=0, sinks=0),
        # the verify step of 24 ragged sequences over 8-bit pages
        dict(name="verify_24_ragged_e4m3", op="paged_attn", batch=24, rows=4, lo=500, hi=32000, hq=24, hkv=4, d=256,
             page=64, layout="HND", e4m3=True, window=0, sinks=0),
        # long conversations under a window with sinks, every head with keys of its own
        dict(name="decode_64_window", op="paged_attn", batch=64, rows=1, lo=2000, hi=120000, hq=16, hkv=16, d=128,
             page=32, layout="NHD", e4m3=False, window=4096, sinks=4),
        # short ragged prompts that arrive together, one of a single token
        dict(name="prompt_7_ragged", op="window_attn", batch=7, lo=1, hi=901, past=0, hq=32, hkv=8, d=128,
             window=0, sinks=0),
        # one long prompt under a window with sinks
        dict(name="prompt_8192_window", op="window_attn", batch=1, lo=8192, hi=8192, past=0, hq=32, hkv=8, d=128,
             window=1024, sinks=4),
        # one long prompt, fully causal, at the verify step's own heads
        dict(name="prompt_8000_causal", op="window_attn", batch=1, lo=8000, hi=8000, past=0, hq=24, hkv=4, d=256,
             window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "paged_kv_append", "paged_attn", "paged_attn", "window_attn", "window_attn"])
    hq, hkv, d = rng.choice([(24, 4, 256), (32, 8, 128), (16, 16, 128), (8, 1, 128), (12, 2, 256), (40, 8, 128)])
    if op in ("qk_norm_rope", "paged_kv_append"):
        if rng.random() < 0.2:
            d = 64
        c = dict(op=op, tokens=_log(rng, 1, 16000 if op == "qk_norm_rope" else 30000), hq=hq, hkv=hkv, d=d,
                 rot=rng.choice([d, d // 2, d // 4]), offset=rng.choice([0.0, 1.0]),
                 interleaved=rng.random() < 0.5, far=rng.choice([4096, 131072, 1000000]))
        if op == "qk_norm_rope":
            return c
        e4m3 = d != 64 and rng.random() < 0.5
        return dict(c, page=rng.choice([16, 32, 64, 128]), layout=rng.choice(["NHD", "HND"]), e4m3=e4m3,
                    queries=c["tokens"] < 12000 and rng.random() < 0.5)
    if op == "paged_attn":
        window = rng.choice([0, 0, 512, 4096])
        batch = _log(rng, 1, 64)
        hi = _log(rng, 16, min(32000, 700000 // batch))
        return dict(op=op, batch=batch, rows=rng.choice([1, 1, 2, 3, 4, 5, 8]), lo=max(8, hi // rng.choice([1, 3, 50])),
                    hi=hi, hq=hq, hkv=min(hkv, 8), d=d, page=rng.choice([16, 32, 64, 128]),
                    layout=rng.choice(["NHD", "HND"]), e4m3=rng.random() < 0.4, window=window,
                    sinks=rng.choice([0, 1, 4]) if window else 0)
    window = rng.choice([0, 0, 128, 1000])
    batch = _log(rng, 1, 16)
    hi = _log(rng, 5, 4096 if batch <= 2 else 1500)
    return dict(op=op, batch=batch, lo=max(1, hi // rng.choice([1, 3, 50])), hi=hi,
                past=rng.choice([0, 0, 333]), hq=hq, hkv=hkv, d=d, window=window,
                sinks=rng.choice([0, 1, 4]) if window else 0)


def _lens(case):
    """Lengths of the case's sequences: the longest, then spread over the logarithm of the range."""
    r = random.Random("%d %d %d" % (case["batch"], case["lo"], case["hi"]))
    return [case["hi"]] + [_log(r, case["lo"], case["hi"]) for _ in range(case["batch"] - 1)]


def _visible(n, m, window, sinks):
    """(slots that some of the newest m of n rows see, pairs of a row and a slot that it sees)."""
    i = np.arange(max(0, n - m), n, dtype=np.int64)
    if not len(i):
        return 0, 0
    if not window:
        return n, int((i + 1).sum())
    first = np.maximum(0, i - window + 1)
    pairs = i + 1 - first + np.minimum(sinks, first)
    slots = n - first[0] + min(sinks, int(first[0]))
    return int(slots), int(pairs.sum())


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "qk_norm_rope":
        t = case["tokens"]
        return dict(bytes=t * (4 * (hq + hkv) * d + 4), flops=t * (hq + hkv) * d * 8)
    if case["op"] == "paged_kv_append":
        t, c = case["tokens"], 1 if case["e4m3"] else 2
        heads = hq if case["queries"] else 0
        return dict(bytes=t * (2 * hkv * d * (2 + c) + 4 * heads * d + 12), flops=t * (heads + hkv) * d * 8)
    lens, w, s = _lens(case), case["window"], case["sinks"]
    if case["op"] == "paged_attn":
        seen = [_visible(n, case["rows"], w, s) for n in lens]
        c, rows = 1 if case["e4m3"] else 2, case["batch"] * case["rows"]
        slots, pairs = sum(x[0] for x in seen), sum(x[1] for x in seen)
        return dict(bytes=2 * c * hkv * d * slots + 4 * rows * hq * d + 4 * (-(-slots // case["page"])) + 4 * len(lens),
                    flops=4 * hq * d * pairs)
    rows = sum(lens)
    seen = [_visible(n + case["past"], n, w, s) for n in lens]
    return dict(bytes=4 * rows * hq * d + 4 * hkv * d * sum(x[0] for x in seen), flops=4 * hq * d * sum(x[1] for x in seen))


# ----------------------------------------------------------------- inputs ----
def _inv_freq(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _rotation(case, s, g):
    t, d = case["tokens"], case["d"]
    s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV, dtype=torch.int32)
    s["inv_freq"] = _inv_freq(case["rot"]).to(DEV)
    s["q_weight"] = (torch.randn(d, generator=g, device=DEV) * 0.1 + 1 - case["offset"]).bfloat16()
    s["k_weight"] = (torch.randn(d, generator=g, device=DEV) * 0.1 + 1 - case["offset"]).bfloat16()
    if own:
        s["phases"] = _sv().rope_phases(_inv_freq(case["rot"]))


def _heads(t, heads, d, g, gain=1.0):
    return (torch.randn((t, heads, d), generator=g, device=DEV) * gain).bfloat16()


def _cache(s, pages, case, g, filled):
    """Pages of keys and values: [pages, slots, heads, d] ("NHD") or [pages, heads, slots, d] ("HND")."""
    hkv, page, d = case["hkv"], case["page"], case["d"]
    shape = (pages, page, hkv, d) if case["layout"] == "NHD" else (pages, hkv, page, d)
    typ = torch.float8_e4m3fn if case["e4m3"] else torch.bfloat16
    for n in ("k_cache", "v_cache"):
        if filled:
            s[n] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16).to(typ)
        else:
            s[n] = torch.zeros(shape, device=DEV, dtype=typ)
    s["k_scale"] = s["v_scale"] = None
    if case["e4m3"]:
        s["k_scale"] = torch.rand(hkv, generator=g, device=DEV) * 0.1 + 0.02 if not filled else torch.rand(hkv, generator=g, device=DEV) + 0.5
        s["v_scale"] = torch.rand(hkv, generator=g, device=DEV) * 0.1 + 0.02 if not filled else torch.rand(hkv, generator=g, device=DEV) + 0.5
    if own:
        s["cache"] = _sv().PagedKV(s["k_cache"], s["v_cache"], layout=case["layout"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"])


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = dict(case=case, scale=d ** -0.5)
    if case["op"] in ("qk_norm_rope", "paged_kv_append"):
        t = case["tokens"]
        _rotation(case, s, g)
        # one projection's output rows: the queries', keys' and values' heads side by side
        rows = _heads(t, hq + 2 * hkv, d, g, gain=2.0)
        s["q"], s["k"], s["v"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        s["q_out"] = torch.empty((t, hq, d), device=DEV, dtype=torch.bfloat16)
        s["k_out"] = torch.empty((t, hkv, d), device=DEV, dtype=torch.bfloat16)
        if case["op"] == "paged_kv_append":
            page = case["page"]
            pages = -(-t // page) + 7
            _cache(s, pages, case, g, filled=False)
            if t <= 256:  # one token for each sequence: slots anywhere
                s["slots"] = torch.randperm(pages * page, generator=g, device=DEV)[:t]
            else:         # whole pages of a prompt, anywhere
                order = torch.randperm(pages, generator=g, device=DEV)
                at = torch.arange(t, device=DEV)
                s["slots"] = order[at // page] * page + at % page
        return s
    lens = _lens(case)
    random.Random(seed).shuffle(lens)
    if case["op"] == "paged_attn":
        b, m, page, w = case["batch"], case["rows"], case["page"], case["window"]
        s["q"] = _heads(b * m, hq, d, g)
        s["o"] = torch.empty_like(s["q"])
        s["max_len"] = max(lens)
        width = -(-max(lens) // page)
        # under a window only the pages that a row can still see are held; the others' entries are -1
        table, used = np.full((b, width), -1, dtype=np.int32), 0
        for i, n in enumerate(lens):
            held = np.arange(-(-n // page))
            if w:
                held = held[(held * page < case["sinks"]) | ((held + 1) * page > n - m - w + 1)]
            table[i, held] = np.arange(used, used + len(held))
            used += len(held)
        order = torch.randperm(used, generator=g, device=DEV).int()
        table = torch.from_numpy(table).to(DEV)
        s["block_table"] = torch.where(table < 0, table, order[table.clamp(min=0).long()])
        s["kv_lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
        _cache(s, used, case, g, filled=True)
        if own:
            sv = _sv()
            s["workspace"] = sv.workspace(sv.paged_attn_workspace_bytes(b, m, hq, hkv, d))
        return s
    nk = [n + case["past"] for n in lens]
    rows = _heads(sum(lens), hq, d, g)
    kv = _heads(sum(nk), 2 * hkv, d, g)
    s["q"], s["k"], s["v"] = rows, kv[:, :hkv], kv[:, hkv:]
    s["o"] = torch.empty_like(rows)
    s["max_q"], s["max_k"] = max(lens), max(nk)
    s["cu_q"] = torch.tensor([0] + np.cumsum(lens).tolist(), device=DEV, dtype=torch.int32)
    s["cu_k"] = torch.tensor([0] + np.cumsum(nk).tolist(), device=DEV, dtype=torch.int32)
    if own:
        sv = _sv()
        s["workspace"] = sv.workspace(sv.window_attn_workspace_bytes(case["batch"], hq, hkv, d))
    return s


# ------------------------------------------------------------- plain forms ----
def _norm_rope(x, weight, s):
    """Rows [T, heads, d] in 32 bits: x * rsqrt(mean(x^2) + eps) * (w + offset), then the rotation."""
    c = s["case"]
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (weight.float() + c["offset"])
    a = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    rot = c["rot"]
    if c["interleaved"]:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((u * cos - v * sin, u * sin + v * cos), -1).flatten(-2)
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((u * cos - v * sin, u * sin + v * cos), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _write(cache, x, slots, scale, c):
    if scale is not None:
        x = (x / scale[:, None]).clamp(-448.0, 448.0)
    page, at = slots // c["page"], slots % c["page"]
    view = cache if c["layout"] == "NHD" else cache.transpose(1, 2)
    if scale is None:
        view[page, at] = x.to(cache.dtype)
    else:
        view.view(torch.uint8)[page, at] = x.to(cache.dtype).view(torch.uint8)


def _gather(cache, page, at, scale, c):
    view = cache if c["layout"] == "NHD" else cache.transpose(1, 2)
    if scale is None:
        return view[page, at].float()
    return view.view(torch.uint8)[page, at].view(cache.dtype).float() * scale[:, None]


def _attend(q, k, v, seen, scale):
    """q [B, M, Hq, d], k and v [B, N, Hkv, d], seen [B, M, N]: softmax over the slots that a row sees,
    zeros for a row that sees none; 32 bits."""
    b, m, hq, d = q.shape
    hkv = k.shape[2]
    q = q.reshape(b, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(scale).reshape(b, hkv, -1, m, k.shape[1])
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == float("-inf"), torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(b, hkv, -1, k.shape[1]), v.permute(0, 2, 1, 3)).reshape(b, hkv, -1, m, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.permute(0, 3, 1, 2, 4).reshape(b, m, hq, d)


def _plain_paged(s):
    c, lens = s["case"], s["kv_lens"].long()
    b, m, w, sinks = c["batch"], c["rows"], c["window"], c["sinks"]
    if w:  # the sinks and the window's slots only
        at = torch.arange(sinks + w + m - 1, device=DEV)
        slot = torch.where(at < sinks, at, lens[:, None] - m - w + 1 + at - sinks)
        good = (slot >= 0) & (slot < lens[:, None]) & ((at < sinks) | (slot >= sinks))
    else:
        slot = torch.arange(s["max_len"], device=DEV).expand(b, -1)
        good = slot < lens[:, None]
    held = slot.clamp(0, s["max_len"] - 1)
    page = torch.gather(s["block_table"].long(), 1, held // c["page"])
    good = good & (page >= 0)
    page = page.clamp(min=0)
    k = _gather(s["k_cache"], page, held % c["page"], s["k_scale"], c)
    v = _gather(s["v_cache"], page, held % c["page"], s["v_scale"], c)
    p = lens[:, None] - m + torch.arange(m, device=DEV)
    seen = good[:, None] & (slot[:, None] <= p[..., None])
    if w:
        seen &= (slot[:, None] > p[..., None] - w) | (slot[:, None] < sinks)
    v = torch.where(good[..., None, None], v, torch.zeros_like(v))
    q = s["q"].float().view(b, m, c["hq"], c["d"])
    return _attend(q, k, v, seen, s["scale"]).to(s["q"].dtype).reshape(s["q"].shape)


def _plain_window(s):
    c, w, sinks = s["case"], s["case"]["window"], s["case"]["sinks"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    at_q = (cu_q[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    p = (nk - nq)[:, None] + i
    seen = (j < nk[:, None])[:, None] & (j <= p[..., None])
    if w:
        seen &= (j > p[..., None] - w) | (j < sinks)
    o = _attend(s["q"][at_q].float(), s["k"][at_k].float(), s["v"][at_k].float(), seen, s["scale"])
    row = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(cu_q, row, right=True) - 1
    return o[seq, row - cu_q[seq]].to(s["q"].dtype)


# -------------------------------------------------------------------- run ----
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        sv = _sv()
        if op == "qk_norm_rope":
            sv.qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["phases"],
                            q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                            weight_offset=c["offset"], interleaved=c["interleaved"])
            return s["q_out"], s["k_out"]
        if op == "paged_kv_append":
            with_q = dict(q=s["q"], q_out=s["q_out"], q_weight=s["q_weight"]) if c["queries"] else {}
            sv.paged_kv_append(s["k"], s["v"], s["cache"], s["slots"], positions=s["positions"], phases=s["phases"],
                               k_weight=s["k_weight"], eps=EPS, weight_offset=c["offset"],
                               interleaved=c["interleaved"], **with_q)
            return (s["k_cache"], s["v_cache"]) + ((s["q_out"],) if c["queries"] else ())
        if op == "paged_attn":
            sv.paged_attn(s["q"], s["cache"], s["block_table"], s["kv_lens"], s["o"], c["rows"], s["scale"],
                          window=c["window"], sinks=c["sinks"], workspace=s["workspace"])
            return s["o"]
        sv.window_attn(s["q"], s["k"], s["v"], s["o"], s["cu_q"], s["cu_k"], s["scale"],
                       window=c["window"], sinks=c["sinks"], workspace=s["workspace"])
        return s["o"]
    if op == "qk_norm_rope":
        return tuple(_norm_rope(s[n], s[n + "_weight"], s).bfloat16() for n in ("q", "k"))
    if op == "paged_kv_append":
        _write(s["k_cache"], _norm_rope(s["k"], s["k_weight"], s), s["slots"], s["k_scale"], c)
        _write(s["v_cache"], s["v"].float(), s["slots"], s["v_scale"], c)
        q = (_norm_rope(s["q"], s["q_weight"], s).bfloat16(),) if c["queries"] else ()
        return (s["k_cache"], s["v_cache"]) + q
    return _plain_paged(s) if op == "paged_attn" else _plain_window(s)


# ------------------------------------------------------------------ exact ----
def _exact_rows(x, w, s):
    """Norm and rotation by complex multiplication, 64 bits."""
    c = s["case"]
    rot = c["rot"]
    x = x.double()
    x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * (w.double() + c["offset"])
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.outer(s["positions"].double(), s["inv_freq"]))[:, None]
    out = x.clone()
    if c["interleaved"]:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turn
        out[..., 0:rot:2], out[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        out[..., :rot // 2], out[..., rot // 2:rot] = z.real, z.imag
    return out


def _exact_head(q, k, v, seen, scale):
    x = torch.einsum("mgd,nd->mgn", q, k) * scale
    x = x.masked_fill(~seen[:, None], float("-inf"))
    return torch.einsum("mgn,nd->mgd", torch.nan_to_num(torch.softmax(x, -1), nan=0.0), v)


def exact(case, seed):
    s = prepare(case, seed)
    c, hq, hkv, d = case, case["hq"], case["hkv"], case["d"]
    if c["op"] == "qk_norm_rope":
        return _exact_rows(s["q"], s["q_weight"], s), _exact_rows(s["k"], s["k_weight"], s)
    if c["op"] == "paged_kv_append":
        got = []
        for n, x in (("k", _exact_rows(s["k"], s["k_weight"], s)), ("v", s["v"].double())):
            cache = s[n + "_cache"].double()
            if s[n + "_scale"] is not None:
                x = (x / s[n + "_scale"].double()[None, :, None]).clamp(-448.0, 448.0)
            flat = cache if c["layout"] == "NHD" else cache.permute(0, 2, 1, 3).contiguous()
            flat.view(-1, hkv, d)[s["slots"]] = x
            got.append(flat if c["layout"] == "NHD" else flat.permute(0, 2, 1, 3).contiguous())
        return tuple(got) + ((_exact_rows(s["q"], s["q_weight"], s),) if c["queries"] else ())
    w, sinks, group = c["window"], c["sinks"], hq // hkv
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    if c["op"] == "paged_attn":
        m = c["rows"]
        for b, n in enumerate(s["kv_lens"].tolist()):
            j = torch.arange(n, device=DEV)
            if w:
                j = j[(j < sinks) | (j > n - m - w)]
            p = torch.arange(n - m, n, device=DEV)[:, None]
            seen = (j <= p) & ((j > p - w) | (j < sinks)) if w else j <= p
            page = s["block_table"][b].long()[j // c["page"]]
            for h in range(hkv):
                at = (page, j % c["page"], h) if c["layout"] == "NHD" else (page, h, j % c["page"])
                k, v = (s[x].view(torch.uint8)[at].view(s[x].dtype).double() if c["e4m3"] else s[x][at].double()
                        for x in ("k_cache", "v_cache"))
                if c["e4m3"]:
                    k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
                mine = slice(h * group, (h + 1) * group)
                out[b * m:(b + 1) * m, mine] = _exact_head(s["q"][b * m:(b + 1) * m, mine].double(), k, v, seen, s["scale"])
        return out
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(c["batch"]):
        q, k, v = s["q"][cu_q[b]:cu_q[b + 1]], s["k"][cu_k[b]:cu_k[b + 1]], s["v"][cu_k[b]:cu_k[b + 1]]
        j = torch.arange(len(k), device=DEV)
        p = (torch.arange(len(q), device=DEV) + len(k) - len(q))[:, None]
        seen = (j <= p) & ((j > p - w) | (j < sinks)) if w else j <= p
        for h in range(hq):
            o = _exact_head(q[:, h:h + 1].double(), k[:, h // group].double(), v[:, h // group].double(), seen, s["scale"])
            out[cu_q[b]:cu_q[b + 1], h:h + 1] = o
    return out
