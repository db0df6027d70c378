"""What the chunked calls are given beside their sequences, and beside one another
(GPU): rows of no sequence that hold anything, places out of range, odd value sizes,
several streams at once."""
import pytest
import torch

import gdn_plain as plain
from test_chunk_attn_gpu import Call

pytestmark = pytest.mark.gpu
STATE = 2.0 ** -14  # of a row's largest value, as in the calls' own tests


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def chunk(sv, states, slots, rows, o, cu):
    (T, Hk, dk), (_, Hv, dv) = rows[0].shape, rows[2].shape
    ws = sv.workspace(sv.gdn_chunk_workspace_bytes(len(slots), T, Hk, Hv, dk, dv))
    sv.gdn_chunk(states, slots, *rows, o, cu, workspace=ws)


# token by token, blocks, blocks prepared beside the chains
@pytest.mark.parametrize("n", [(5, 9), (40, 70), (1500, 900)])
def test_rows_of_no_sequence_hold_anything(cuda_lib, n):
    """NaN before, between and behind the sequences, and in a third one, stays there."""
    sv, (a, b) = cuda_lib, n
    T, Hk, Hv, dk, dv = 3 + a + b + 30, 1, 2, 64, 72
    r = plain.rows(T, Hk, Hv, dk, dv, 31)
    cu = ints(3, 3 + a, 3 + a + b, T - 20)     # the third sequence: NaN
    pool = torch.randn(3, Hv, dv, dk, generator=torch.Generator().manual_seed(1)).cuda()
    good, go = pool.clone(), torch.zeros(T, Hv, dv, device="cuda", dtype=torch.bfloat16)
    chunk(sv, good, ints(0, 2, 1), plain.on(r), go, cu)
    rows = plain.on(r)
    for x in rows:
        x[:3] = float("nan")
        x[3 + a + b:] = float("nan")
    states, o = pool.clone(), torch.full_like(go, 7.0)
    chunk(sv, states, ints(0, 2, 1), rows, o, cu)
    assert sv.sv_last_device_error() == sv.SV_OK
    mine = slice(3, 3 + a + b)
    assert torch.equal(o[mine], go[mine]) and torch.equal(states[[0, 2]], good[[0, 2]])
    assert bool((o[:3] == 7.0).all()) and bool((o[T - 20:] == 7.0).all())
    assert bool(o[3 + a + b:T - 20].isnan().all()) and bool(states[1].isnan().any())


@pytest.mark.parametrize("n", [(5, 9), (40, 70), (1500, 900)])
def test_places_out_of_range(cuda_lib, n):
    """A place past the pool counts as none (from zeros, not kept) and is reported."""
    sv, (a, b) = cuda_lib, n
    T, Hk, Hv, dk, dv = a + b, 2, 2, 64, 64
    rows = plain.on(plain.rows(T, Hk, Hv, dk, dv, 32))
    pool = torch.randn(3, Hv, dv, dk, generator=torch.Generator().manual_seed(2)).cuda()
    outs = []
    for slots in (ints(-1, 1), ints(3, 1), ints(0x7fffffff, 1)):
        states, o = pool.clone(), torch.zeros(T, Hv, dv, device="cuda", dtype=torch.bfloat16)
        chunk(sv, states, slots, rows, o, ints(0, a, T))
        assert sv.sv_last_device_error() == (sv.SV_OK if int(slots[0]) < 0 else sv.SV_ERR_INVALID_ARG)
        assert torch.equal(states[[0, 2]], pool[[0, 2]])
        outs.append((o, states))
    assert all(torch.equal(o, outs[0][0]) and torch.equal(s, outs[0][1]) for o, s in outs)


def output_reach(r, T):
    """What outputs of blocks of 64 tokens may be off by: o = e^G S q + sum_j P_j u_j takes S, P and u as
    one fp16 part each, off by at most 2^-11 of themselves, so o by 2^-11 of the first sum's absolute
    values and 2^-10 of the second's, however much of them cancels (a row of one value has no larger ones
    beside it to be measured by)."""
    Hv, dv, dk = r["v"].shape[1], r["v"].shape[2], r["k"].shape[2]
    group = Hv // r["k"].shape[1]
    S = S0 = torch.zeros(Hv, dv, dk, dtype=torch.float64)
    out, seen = [], []
    for t in range(T):
        if t % 64 == 0:
            S0, seen, G = S, [], torch.zeros(Hv, dtype=torch.float64)
        k, q = (r[n][t].double().repeat_interleave(group, 0) for n in ("k", "q"))
        g = r["g"][t].double()
        G = G + g
        S = S * torch.exp(g)[:, None, None]
        u = r["beta"][t].double()[:, None] * (r["v"][t].double() - torch.einsum("hvk,hk->hv", S, k))
        S = S + u[:, :, None] * k[:, None, :]
        seen.append((G, k, u))
        first = torch.exp(G)[:, None] * torch.einsum("hvk,hk->hv", S0.abs(), q.abs())
        second = sum((torch.exp(G - Gj) * (q * kj).sum(-1).abs())[:, None] * uj.abs() for Gj, kj, uj in seen)
        out.append(2.0 ** -11 * first + 2.0 ** -10 * second)
    return torch.stack(out)


@pytest.mark.parametrize("dv", [1, 5, 67])
def test_odd_value_sizes(cuda_lib, dv):
    """Values and outputs in padded rows; nothing of the padding is written."""
    sv, Hk, Hv, dk, T = cuda_lib, 1, 2, 64, 150
    r = plain.rows(T, Hk, Hv, dk, dv, 33)
    pad = (dv + 7) // 8 * 8
    q, k, v, g, beta = plain.on(r)
    wide = torch.full((T, Hv, pad), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide[..., :dv] = v
    out = torch.full((T, Hv, pad), 7.0, device="cuda", dtype=torch.bfloat16)
    v, o = wide[..., :dv], out[..., :dv]
    states = torch.zeros(2, Hv, dv, dk, device="cuda")
    chunk(sv, states, ints(1), [x[:140] for x in (q, k, v, g, beta)], o[:140], ints(0, 140))
    sv.gdn_step(states, ints(1), *(x[140:] for x in (q, k, v, g, beta)), o[140:], 10, commit=True)
    assert sv.sv_last_device_error() == sv.SV_OK
    S, want = plain.run(torch.zeros(Hv, dv, dk), r, 0, T)
    # and their rounding, half a step of bf16 (2^-8), once more 2^-16 of all for fp32's
    off = (o.double().cpu() - want).abs() - 2.0 ** -8 * want.abs() - 2.0 ** -16 * want.abs().max()
    assert bool((off <= output_reach(r, T)).all())
    plain.close(states[1], S, STATE, 0.0, "state")
    assert bool((out[..., dv:] == 7.0).all()) and not states[0].any()


@pytest.mark.parametrize("tape_M,M", [(0, 2), (8, 8), (16, 0), (7, 2), (0, 16), (1, 1)])
def test_many_states_of_128_columns(cuda_lib, tape_M, M):
    """Streamed tiles of two rows a thread, up to the most tokens that are streamed; a height that the
    tiles do not divide."""
    sv, B, Hk, Hv, dk, dv = cuda_lib, 40, 1, 4, 128, 264
    gen = torch.Generator().manual_seed(34)
    pool = torch.randn(B + 1, Hv, dv, dk, generator=gen) * 0.3
    slots = torch.randperm(B + 1, generator=gen)[:B].int()
    count = torch.randint(0, tape_M + 1, (B,), generator=gen).int()
    tape, own = (plain.rows(max(1, B * n), Hk, Hv, dk, dv, 35 + i) for i, n in enumerate((tape_M, M)))
    states, o = pool.cuda(), torch.zeros(B * M, Hv, dv, device="cuda")
    t = plain.on(tape)[1:] if tape_M else None
    sv.gdn_step(states, slots.cuda(), *(plain.on(own) if M else [None] * 5), o if M else None, M, tape=t,
                n_replay=count.cuda() if tape_M else None)
    assert sv.sv_last_device_error() == sv.SV_OK
    for b in range(B):
        S, _ = plain.run(pool[int(slots[b])], tape, b * tape_M, b * tape_M + int(count[b]), False)
        plain.close(states[int(slots[b])], S, 2.0 ** -18, 0.0, "state")
        if M:
            _, want = plain.run(S, own, b * M, (b + 1) * M)
            plain.close(o[b * M:(b + 1) * M], want, 2.0 ** -18, 0.0, "o")


def test_streams_at_once(cuda_lib):
    """Each call on a stream of its own, with a workspace of its own, over and over: the bits of one
    after the other."""
    sv = cuda_lib
    Hk, Hv, dk, dv, T = 2, 8, 128, 128, 2500
    works = []
    for seed in (41, 42):
        rows = plain.on(plain.rows(T, Hk, Hv, dk, dv, seed))
        ws = sv.workspace(sv.gdn_chunk_workspace_bytes(1, T, Hk, Hv, dk, dv))
        st, o = torch.zeros(1, Hv, dv, dk, device="cuda"), torch.zeros(T, Hv, dv, device="cuda", dtype=torch.bfloat16)

        def recur(rows=rows, ws=ws, st=st, o=o):
            st.zero_()
            sv.gdn_chunk(st, ints_0, *rows, o, cu, workspace=ws)
            return st, o
        works.append(recur)
    ints_0, cu = ints(0), ints(0, T)
    for seed, e4m3 in ((43, False), (44, True)):
        c = Call(sv, [(300, 2000), (40, 900)], 8, 2, 128, 16, e4m3=e4m3, seed=seed, dirty=False)
        t = c.tensors()
        works.append(lambda c=c, t=t: (c.run(t),))
    want = [[x.clone() for x in w()] for w in works]
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, w in zip(streams, works):
            with torch.cuda.stream(s):
                got.append(w())
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, h in zip(got, want) for x, y in zip(g, h))
    assert sv.sv_last_device_error() == sv.SV_OK
