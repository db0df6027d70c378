"""What the chunked-prefill operators are measured on: their cases, inputs and plain forms.

Three operators that take a chunk of new tokens of many sequences through a hybrid target's two
kinds of layer, and the steps that follow it:

    paged_chunk_attn  a chunk of new rows of each sequence over a paged cache that already holds
                      them: ragged, bf16 or e4m3 pages, with a sliding window and a few first
                      tokens that stay visible
    gdn_chunk         the gated delta rule over packed chunks, from the states of a pool and back
                      into it
    gdn_step          the newest rows of each sequence (one token, or the rows of a verify step)
                      over the same pool, after the accepted rows of the previous round

``run`` computes them in elementary torch operations in 32 bits (sums of decays in 64), or, where
``own`` is true, through the package's entry points.  ``exact`` computes them in 64 bits.
"""
import math
import random

import numpy as np
import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
CHUNK = 64  # tokens of a chunk in the plain form of gdn_chunk


def _sv():
    import speculative_decoding_verify_08_gb300 as sv
    return sv


# ------------------------------------------------------------------ cases ----
# 24 query heads over 4 KV heads of 256, and 48 value heads over 16 key heads of 128 x 128, are this
# repository's own attention and recurrent layers (a 27B-class hybrid target); 32 over 8 of 128 is the
# usual grouped layout.
def listed():
    return [
        # a chunk of a long conversation's prompt behind what the cache holds already
        dict(name="chunk_2048_past_30000", op="paged_chunk_attn", batch=1, lo=2048, hi=2048, past=30000, hq=24, hkv=4,
             d=256, page=64, layout="HND", e4m3=False, window=0, sinks=0),
        # prompts and rests of prompts that a scheduler packs into one call, some of a single token
        dict(name="chunk_13_ragged", op="paged_chunk_attn", batch=13, lo=1, hi=777, past=5000, hq=32, hkv=8, d=128,
             page=16, layout="NHD", e4m3=False, window=0, sinks=0),
        # a short follow-up question to a long document, 8-bit pages
        dict(name="chunk_61_past_16000_e4m3", op="paged_chunk_attn", batch=1, lo=61, hi=61, past=16000, hq=24, hkv=4,
             d=256, page=64, layout="HND", e4m3=True, window=0, sinks=0),
        # chunks of two long prompts under a window with sinks, 8-bit pages
        dict(name="chunk_2x4001_window_e4m3", op="paged_chunk_attn", batch=2, lo=4001, hi=4001, past=9000, hq=32, hkv=8,
             d=128, page=32, layout="NHD", e4m3=True, window=1024, sinks=4),
        # one long prompt through a recurrent layer
        dict(name="gdn_prompt_8192", op="gdn_chunk", batch=1, lo=8192, hi=8192, hk=16, hv=48, dk=128, dv=128),
        # ragged prompts that arrive together, some of a single token
        dict(name="gdn_prompt_11_ragged", op="gdn_chunk", batch=11, lo=1, hi=3001, hk=16, hv=48, dk=128, dv=128),
        # the rest of a prompt: latency
        dict(name="gdn_prompt_77", op="gdn_chunk", batch=1, lo=77, hi=77, hk=16, hv=48, dk=128, dv=128),
        # one new token of one conversation: latency
        dict(name="gdn_token_1", op="gdn_step", batch=1, rows=1, replay=0, commit=True, hk=16, hv=48, dk=128, dv=128),
        # one new token for each of 61 conversations
        dict(name="gdn_token_61", op="gdn_step", batch=61, rows=1, replay=0, commit=True, hk=16, hv=48, dk=128, dv=128),
        # the verify step of 24 sequences, after what each accepted of its last one
        dict(name="gdn_verify_24x4", op="gdn_step", batch=24, rows=4, replay=4, commit=False, hk=16, hv=48, dk=128, dv=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paged_chunk_attn", "paged_chunk_attn", "gdn_chunk", "gdn_chunk", "gdn_step"])
    if op == "paged_chunk_attn":
        hq, hkv, d = rng.choice([(24, 4, 256), (32, 8, 128), (8, 8, 128), (8, 1, 128), (12, 2, 256), (40, 8, 128)])
        window = rng.choice([0, 0, 0, 600, 4096])
        batch = _log(rng, 1, 24)
        hi = _log(rng, 1, 2048 if batch <= 3 else 800)
        past = rng.choice([0, _log(rng, 1, 30000 if batch <= 2 else 6000)])
        return dict(op=op, batch=batch, lo=max(1, hi // rng.choice([1, 3, 50])), hi=hi, past=past, hq=hq, hkv=hkv, d=d,
                    page=rng.choice([16, 32, 48, 64, 128]), layout=rng.choice(["NHD", "HND"]), e4m3=rng.random() < 0.4,
                    window=window, sinks=rng.choice([0, 1, 4, 50]) if window else 0)
    hk, hv, dk, dv = rng.choice([(16, 48, 128, 128), (16, 32, 128, 128), (4, 8, 128, 64), (8, 8, 64, 128), (2, 6, 128, 256),
                                 (4, 4, 64, 72)])
    if op == "gdn_chunk":
        batch = _log(rng, 1, 24)
        hi = _log(rng, 1, max(2, 8000 // batch) * (1 if batch < 3 else 3))
        return dict(op=op, batch=batch, lo=max(1, hi // rng.choice([1, 4, 60])), hi=hi, hk=hk, hv=hv, dk=dk, dv=dv)
    rows = rng.choice([1, 1, 2, 3, 4, 5, 8])
    return dict(op=op, batch=_log(rng, 1, 61), rows=rows, replay=rng.choice([0, rows]), commit=rng.random() < 0.5,
                hk=hk, hv=hv, dk=dk, dv=dv)


def _spread(case, lo, hi, what):
    """Lengths of the case's sequences: the longest, then spread over the logarithm of the range."""
    r = random.Random("%s %d %d %d" % (what, case["batch"], lo, hi))
    return [hi] + [_log(r, lo, hi) for _ in range(case["batch"] - 1)]


def _lens(case):
    """(new rows, rows of the cache) of each sequence: what came before is from 0 to `past` rows."""
    new = _spread(case, case["lo"], case["hi"], "new")
    past = [n - 1 for n in _spread(case, 1, case["past"] + 1, "past")]
    return new, [n + p for n, p in zip(new, past)]


def _visible(nq, n, window, sinks):
    """(slots that some of the newest nq of n rows see, pairs of a row and a slot that it sees)."""
    i = np.arange(n - nq, n, dtype=np.int64)
    if not window:
        return n, int((i + 1).sum())
    first = np.maximum(0, i - window + 1)
    pairs = i + 1 - first + np.minimum(sinks, first)
    return int(n - first[0] + min(sinks, int(first[0]))), int(pairs.sum())


def work(case):
    if case["op"] == "paged_chunk_attn":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        new, lens = _lens(case)
        seen = [_visible(m, n, case["window"], case["sinks"]) for m, n in zip(new, lens)]
        c, slots, pairs = 1 if case["e4m3"] else 2, sum(x[0] for x in seen), sum(x[1] for x in seen)
        return dict(bytes=2 * c * hkv * d * slots + 4 * sum(new) * hq * d + 4 * (-(-slots // case["page"])) + 8 * len(lens),
                    flops=4 * hq * d * pairs)
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    state = 8 * case["batch"] * hv * dv * dk
    row = 2 * (2 * hk * dk + 2 * hv * dv) + 8 * hv  # q, k, v, o and the two gates
    if case["op"] == "gdn_chunk":
        t = sum(_lens(dict(case, past=0))[0])
        return dict(bytes=state + t * row, flops=6 * t * hv * dk * dv)
    t, r = case["batch"] * case["rows"], sum(_replay(case))
    return dict(bytes=state + t * row + r * (2 * (hk * dk + hv * dv) + 8 * hv), flops=6 * t * hv * dk * dv + 4 * r * hv * dk * dv)


def _replay(case):
    """Rows of the last round that each sequence accepted."""
    r = random.Random("replay %d %d" % (case["batch"], case["replay"]))
    return [r.randint(0, case["replay"]) for _ in range(case["batch"])]


# ----------------------------------------------------------------- inputs ----
def _offsets(lens):
    return torch.tensor([0] + np.cumsum(lens).tolist(), device=DEV, dtype=torch.int32)


def _prepare_attn(case, s, seed, g):
    hq, hkv, d, page, w = case["hq"], case["hkv"], case["d"], case["page"], case["window"]
    new, lens = _lens(case)
    both = list(zip(new, lens))
    random.Random(seed).shuffle(both)
    new, lens = [x[0] for x in both], [x[1] for x in both]
    s["q"] = torch.randn((sum(new), hq, d), generator=g, device=DEV).bfloat16()
    s["o"] = torch.empty_like(s["q"])
    s["cu_q"], s["kv_lens"] = _offsets(new), torch.tensor(lens, device=DEV, dtype=torch.int32)
    s["max_new"], s["max_len"], s["scale"] = max(new), max(lens), d ** -0.5
    # under a window only the pages that a row can still see are held; the others' entries are -1
    table, used = np.full((len(lens), -(-max(lens) // page)), -1, dtype=np.int32), 0
    for i, (m, n) in enumerate(both):
        held = np.arange(-(-n // page))
        if w:
            held = held[(held * page < case["sinks"]) | ((held + 1) * page > n - m - w + 1)]
        table[i, held] = np.arange(used, used + len(held))
        used += len(held)
    order = torch.randperm(used, generator=g, device=DEV).int()
    table = torch.from_numpy(table).to(DEV)
    s["block_table"] = torch.where(table < 0, table, order[table.clamp(min=0).long()])
    shape = (used, page, hkv, d) if case["layout"] == "NHD" else (used, hkv, page, d)
    typ = torch.float8_e4m3fn if case["e4m3"] else torch.bfloat16
    for n in ("k_cache", "v_cache"):
        s[n] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16).to(typ)
    s["k_scale"] = s["v_scale"] = None
    if case["e4m3"]:
        s["k_scale"] = torch.rand(hkv, generator=g, device=DEV) + 0.5
        s["v_scale"] = torch.rand(hkv, generator=g, device=DEV) + 0.5
    if own:
        sv = _sv()
        s["cache"] = sv.PagedKV(s["k_cache"], s["v_cache"], layout=case["layout"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        s["workspace"] = sv.workspace(sv.paged_chunk_attn_workspace_bytes(len(lens), sum(new), hq, hkv, d))


def _recurrent_rows(case, t, g):
    """Rows of a recurrent layer: queries and keys of unit norm that point partly the same way, values, log decays
    and update strengths of the usual initialisation."""
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    rows = torch.empty((t, 2 * hk * dk + hv * dv), device=DEV, dtype=torch.bfloat16)
    lean = torch.randn((2 * hk, dk), generator=g, device=DEV) * 0.4
    qk = F.silu(torch.randn((t, 2 * hk, dk), generator=g, device=DEV) + lean)
    qk = qk / (qk.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    qk[:, :hk] *= dk ** -0.5
    rows[:, :2 * hk * dk] = qk.reshape(t, -1)
    rows[:, 2 * hk * dk:] = F.silu(torch.randn((t, hv * dv), generator=g, device=DEV) * 1.5)
    a = torch.rand(hv, generator=g, device=DEV) * 15 + 1
    step = torch.exp(torch.rand(hv, generator=g, device=DEV) * math.log(100.0) + math.log(0.001))
    bias = torch.log(torch.expm1(step))
    gate = -a * F.softplus(torch.randn((t, hv), generator=g, device=DEV) + bias)
    beta = torch.sigmoid(torch.randn((t, hv), generator=g, device=DEV))
    q, k, v = rows.split([hk * dk, hk * dk, hv * dv], 1)
    return q.unflatten(1, (hk, dk)), k.unflatten(1, (hk, dk)), v.unflatten(1, (hv, dv)), gate, beta


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case=case)
    if case["op"] == "paged_chunk_attn":
        _prepare_attn(case, s, seed, g)
        return s
    b, hv, dk, dv = case["batch"], case["hv"], case["dk"], case["dv"]
    s["states"] = torch.randn((b + 2, hv, dv, dk), generator=g, device=DEV) * 0.1
    s["slots"] = torch.randperm(b + 2, generator=g, device=DEV)[:b].int()
    if case["op"] == "gdn_chunk":
        lens = _lens(dict(case, past=0))[0]
        random.Random(seed).shuffle(lens)
        s["cu"], s["max_new"], t = _offsets(lens), max(lens), sum(lens)
    else:
        t = b * case["rows"]
        s["tape"] = s["n_replay"] = None
        if case["replay"]:
            s["tape"] = _recurrent_rows(case, b * case["replay"], g)[1:]
            n = _replay(case)
            random.Random(seed).shuffle(n)
            s["n_replay"] = torch.tensor(n, device=DEV, dtype=torch.int32)
    s["q"], s["k"], s["v"], s["g"], s["beta"] = _recurrent_rows(case, t, g)
    s["o"] = torch.empty((t, hv, dv), device=DEV, dtype=torch.bfloat16)
    if own and case["op"] == "gdn_chunk":
        sv = _sv()
        s["workspace"] = sv.workspace(sv.gdn_chunk_workspace_bytes(b, t, case["hk"], hv, dk, dv))
    return s


# ------------------------------------------------------------- plain forms ----
def _gather(cache, page, at, scale, c):
    view = cache if c["layout"] == "NHD" else cache.transpose(1, 2)
    if scale is None:
        return view[page, at].float()
    return view.view(torch.uint8)[page, at].view(cache.dtype).float() * scale[:, None]


def _plain_attn(s):
    """Every sequence's rows and slots padded to the longest; zeros for a row that sees none; 32 bits."""
    c, w, sinks = s["case"], s["case"]["window"], s["case"]["sinks"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    cu, lens = s["cu_q"].long(), s["kv_lens"].long()
    nq = cu[1:] - cu[:-1]
    b, i, j = len(lens), torch.arange(s["max_new"], device=DEV), torch.arange(s["max_len"], device=DEV)
    row = (cu[:-1, None] + i).clamp(max=len(s["q"]) - 1)
    page = s["block_table"].long()[:, j // c["page"]]
    good = (j < lens[:, None]) & (page >= 0)
    k, v = (_gather(s[n + "_cache"], page.clamp(min=0), (j % c["page"]).expand(b, -1), s[n + "_scale"], c) for n in ("k", "v"))
    v = torch.where(good[..., None, None], v, torch.zeros_like(v))
    p = (lens - nq)[:, None, None] + i[:, None]
    seen = good[:, None] & (j <= p)
    if w:
        seen &= (j > p - w) | (j < sinks)
    q = s["q"][row].float().reshape(b, -1, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["scale"]).reshape(b, hkv, -1, s["max_new"], s["max_len"])
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == float("-inf"), torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(b, hkv, -1, s["max_len"]), v.permute(0, 2, 1, 3)).reshape(b, hkv, -1, s["max_new"], d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(b, s["max_new"], hq, d)
    at = torch.arange(len(s["q"]), device=DEV)
    seq = torch.searchsorted(cu, at, right=True) - 1
    return o[seq, at - cu[seq]].to(s["q"].dtype)


def _key_heads(x, c):
    """Rows [..., hk, dk] as each value head's, in 32 bits: [..., hv, dk]."""
    return x.float().repeat_interleave(c["hv"] // c["hk"], -2)


def _plain_chunk(s):
    """Chunks of 64 tokens, all sequences padded to the longest: within a chunk the tokens' updates solve a
    triangular system, which the state at its start enters linearly; 32 bits."""
    c, cu = s["case"], s["cu"].long()
    lens, b = cu[1:] - cu[:-1], c["batch"]
    chunks = -(-s["max_new"] // CHUNK)
    i = torch.arange(chunks * CHUNK, device=DEV)
    inside = (i < lens[:, None])
    row = (cu[:-1, None] + i).clamp(max=len(s["q"]) - 1)

    def rows(x):  # [b, chunks, hv, CHUNK, ...], zeros past a sequence's end
        x = x[row]
        x = torch.where(inside.view(b, -1, *(1,) * (x.dim() - 2)), x, torch.zeros_like(x))
        return x.reshape(b, chunks, CHUNK, *x.shape[2:]).transpose(2, 3)

    q, k, v = rows(_key_heads(s["q"], c)), rows(_key_heads(s["k"], c)), rows(s["v"].float())
    beta, total = rows(s["beta"])[..., None], rows(s["g"]).double().cumsum(-1)
    low = torch.ones((CHUNK, CHUNK), device=DEV, dtype=torch.bool).tril()
    decay = torch.where(low, total[..., :, None] - total[..., None, :], torch.zeros((), device=DEV, dtype=torch.float64))
    decay = torch.where(low, decay.exp().float(), torch.zeros((), device=DEV))
    start, end = total.exp().float()[..., None], (total[..., -1:] - total).exp().float()[..., None]
    a = (beta * decay * torch.matmul(k, k.transpose(-1, -2))).tril(-1)
    t = torch.eye(CHUNK, device=DEV).expand_as(a).clone()
    for n in range(1, CHUNK):  # inverse of 1 + a, row by row
        t[..., n, :n] = -torch.matmul(a[..., n:n + 1, :n], t[..., :n, :n]).squeeze(-2)
    p = decay * torch.matmul(q, k.transpose(-1, -2))
    state = s["states"][s["slots"].long()].transpose(-1, -2).contiguous()
    o = torch.empty_like(v)
    for n in range(chunks):
        u = torch.matmul(t[:, n], beta[:, n] * (v[:, n] - start[:, n] * torch.matmul(k[:, n], state)))
        o[:, n] = start[:, n] * torch.matmul(q[:, n], state) + torch.matmul(p[:, n], u)
        state = start[:, n, :, -1:] * state + torch.matmul((end[:, n] * k[:, n]).transpose(-1, -2), u)
    s["states"][s["slots"].long()] = state.transpose(-1, -2)
    at = torch.arange(len(s["q"]), device=DEV)
    seq = torch.searchsorted(cu, at, right=True) - 1
    return o.transpose(2, 3).reshape(b, chunks * CHUNK, c["hv"], c["dv"])[seq, at - cu[seq]].bfloat16(), s["states"]


def _token(state, k, v, g, beta, c):
    k, g = _key_heads(k, c), g.exp()[..., None]
    u = beta[..., None] * (v.float() - g * torch.matmul(state, k[..., None]).squeeze(-1))
    return g[..., None] * state + u[..., None] * k[..., None, :]


def _plain_step(s):
    c, b, m, slots = s["case"], s["case"]["batch"], s["case"]["rows"], s["slots"].long()
    state = s["states"][slots]
    if s["tape"] is not None:
        tape = [x.unflatten(0, (b, c["replay"])) for x in s["tape"]]
        for i in range(c["replay"]):
            on = (s["n_replay"] > i)[:, None, None, None]
            state = torch.where(on, _token(state, *(x[:, i] for x in tape), c), state)
    kept, o = state, torch.empty((b, m, c["hv"], c["dv"]), device=DEV)
    q, *rows = (s[n].unflatten(0, (b, m)) for n in ("q", "k", "v", "g", "beta"))
    for i in range(m):
        state = _token(state, *(x[:, i] for x in rows), c)
        o[:, i] = torch.matmul(state, _key_heads(q[:, i], c)[..., None]).squeeze(-1)
    s["states"][slots] = state if c["commit"] else kept
    return o.reshape(b * m, c["hv"], c["dv"]).bfloat16(), s["states"]


# -------------------------------------------------------------------- run ----
def run(state):
    s, c = state, state["case"]
    if own:
        sv = _sv()
        if c["op"] == "paged_chunk_attn":
            sv.paged_chunk_attn(s["q"], s["cache"], s["block_table"], s["kv_lens"], s["o"], s["cu_q"], s["scale"],
                                window=c["window"], sinks=c["sinks"], workspace=s["workspace"])
            return s["o"]
        if c["op"] == "gdn_chunk":
            sv.gdn_chunk(s["states"], s["slots"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], s["cu"],
                         workspace=s["workspace"])
        else:
            sv.gdn_step(s["states"], s["slots"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], c["rows"],
                        tape=s["tape"], n_replay=s["n_replay"], commit=c["commit"])
        return s["o"], s["states"]
    if c["op"] == "paged_chunk_attn":
        return _plain_attn(s)
    return _plain_chunk(s) if c["op"] == "gdn_chunk" else _plain_step(s)


# ------------------------------------------------------------------ exact ----
def _exact_attn(s, c):
    hq, hkv, d, w, sinks = c["hq"], c["hkv"], c["d"], c["window"], c["sinks"]
    group, cu = hq // hkv, s["cu_q"].tolist()
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    for b, n in enumerate(s["kv_lens"].tolist()):
        mine, nq = slice(cu[b], cu[b + 1]), cu[b + 1] - cu[b]
        j = torch.arange(n, device=DEV)
        p = torch.arange(n - nq, n, device=DEV)[:, None]
        if w:
            j = j[(j < sinks) | (j > n - nq - w)]
        seen = (j <= p) & ((j > p - w) | (j < sinks)) if w else j <= p
        page, at = s["block_table"][b].long()[j // c["page"]], j % c["page"]
        for h in range(hkv):
            where = (page, at, h) if c["layout"] == "NHD" else (page, h, at)
            if c["e4m3"]:
                k, v = (s[x + "_cache"].view(torch.uint8)[where].view(torch.float8_e4m3fn).double() * s[x + "_scale"][h].double()
                        for x in ("k", "v"))
            else:
                k, v = s["k_cache"][where].double(), s["v_cache"][where].double()
            for e in range(h * group, (h + 1) * group):
                x = (s["q"][mine, e].double() @ k.T * s["scale"]).masked_fill(~seen, float("-inf"))
                out[mine, e] = torch.nan_to_num(torch.softmax(x, -1), nan=0.0) @ v
    return out


def _exact_tokens(state, rows, live, group):
    """The rule token by token: state [b, hv, dv, dk], rows a list of (q, k, v, g, beta) of all sequences,
    live a list of which of them the token belongs to."""
    out = []
    for (q, k, v, g, beta), on in zip(rows, live):
        k, a = k.double().repeat_interleave(group, 1), torch.exp(g.double())[..., None]
        old = (state * k[:, :, None, :]).sum(-1) * a
        new = state * a[..., None] + ((v.double() - old) * beta.double()[..., None])[..., None] * k[:, :, None, :]
        state = torch.where(on[:, None, None, None], new, state)
        out.append(None if q is None else (state * q.double().repeat_interleave(group, 1)[:, :, None, :]).sum(-1))
    return state, out


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "paged_chunk_attn":
        return _exact_attn(s, c)
    group, slots = c["hv"] // c["hk"], s["slots"].long()
    pool = s["states"].double()
    state, five = pool[slots], [s[n] for n in ("q", "k", "v", "g", "beta")]
    out = torch.zeros(s["o"].shape, device=DEV, dtype=torch.float64)
    if c["op"] == "gdn_chunk":
        first, last = s["cu"][:-1].long(), s["cu"][1:].long()
        for t in range(s["max_new"]):
            at, on = (first + t).clamp(max=len(out) - 1), first + t < last
            state, got = _exact_tokens(state, [[x[at] for x in five]], [on], group)
            out[at[on]] = got[0][on]
        pool[slots] = state
        return out, pool
    b, m, everyone = c["batch"], c["rows"], torch.ones(c["batch"], device=DEV, dtype=torch.bool)
    if s["tape"] is not None:
        tape = [[None] + [x[i::c["replay"]] for x in s["tape"]] for i in range(c["replay"])]
        state, _ = _exact_tokens(state, tape, [s["n_replay"] > i for i in range(c["replay"])], group)
    after, got = _exact_tokens(state, [[x[i::m] for x in five] for i in range(m)], [everyone] * m, group)
    for i in range(m):
        out[i::m] = got[i]
    pool[slots] = after if c["commit"] else state
    return out, pool
