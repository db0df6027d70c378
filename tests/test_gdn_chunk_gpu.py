"""gdn_chunk against the rule in 64 bits, token by token.

What a chunk's arithmetic may be off by: its operands are fp32 values held as two
fp16 parts (2^-22 of the value, or 2^-27 of the row's largest in the chunk), and
a state enters and leaves a chunk through three products of at most 128 terms
with fp32 sums, each term's share at most 2^-22 + 2^-23 of a sum of absolute
values that passes the row's largest by sqrt(128) < 2^4: 3 * 2^4 * 2^-21, once
more for what earlier chunks left: 2^-14 of a row's largest value.  Outputs add
operands of one fp16 part (2^-11 each way, of sums as above) and their own
rounding, half a step of bf16: 2^-8 of the row's largest in all beside it."""
import pytest
import torch

import gdn_plain as plain

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8
STATE, OUT = 2.0 ** -14, 2.0 ** -8


def chunk(sv, states, slots, r, o, cu):
    """The call with a workspace of its own."""
    (T, Hk, dk), (_, Hv, dv) = r[0].shape, r[2].shape
    ws = sv.workspace(sv.gdn_chunk_workspace_bytes(len(slots), T, Hk, Hv, dk, dv))
    sv.gdn_chunk(states, slots, *r, o, cu, workspace=ws)


def case(sv, lens, Hk, Hv, dk, dv, seed, slots=None, extra=0, **how):
    B, T = len(lens), sum(lens)
    gen = torch.Generator().manual_seed(seed)
    pool = torch.randn(B + 2, Hv, dv, dk, generator=gen) * 0.3
    slots = torch.randperm(B + 2, generator=gen)[:B].int() if slots is None else torch.tensor(slots, dtype=torch.int32)
    r = plain.rows(T + extra, Hk, Hv, dk, dv, seed + 1, **how)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    q, k, v, g, beta = plain.on(r)
    fused = torch.cat([x.flatten(1) for x in (q, k, v)], 1)  # slices of one projection's rows
    q, k, v = fused.split([Hk * dk, Hk * dk, Hv * dv], 1)
    q, k, v = q.unflatten(1, (Hk, dk)), k.unflatten(1, (Hk, dk)), v.unflatten(1, (Hv, dv))
    states, o = pool.cuda(), torch.full((T + extra, Hv, dv), 99.0, device="cuda", dtype=torch.bfloat16)
    chunk(sv, states, slots.cuda(), (q, k, v, g, beta), o, cu.cuda())
    assert sv.sv_last_device_error() == sv.SV_OK
    want, out = pool.double().clone(), []
    for b in range(B):
        at = int(slots[b])
        S = pool[at].double() if at >= 0 else torch.zeros(Hv, dv, dk, dtype=torch.float64)
        S, got = plain.run(S, r, int(cu[b]), int(cu[b + 1]))
        out.append(got)
        if at >= 0:
            want[at] = S
    plain.close(o[:T], torch.cat(out), OUT, BF16, "o")
    plain.close(states, want, STATE, 0.0, "states")
    assert bool((o[T:] == 99.0).all())  # rows behind the last sequence
    touched = {int(s) for s, n in zip(slots, lens) if s >= 0 and n}
    for s in set(range(B + 2)) - touched:
        assert torch.equal(states[s].cpu(), pool[s])


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 321])
def test_lengths(cuda_lib, n):
    case(cuda_lib, [n], 1, 2, 128, 128, seed=n)


@pytest.mark.parametrize("dk,dv", [(128, 8), (128, 72), (128, 128), (128, 136), (128, 256), (64, 64), (64, 128), (64, 200)])
def test_shapes(cuda_lib, dk, dv):
    case(cuda_lib, [70, 5, 130], 2, 4, dk, dv, seed=dk + dv)


@pytest.mark.parametrize("lens,Hk,Hv,dk,dv", [
    ([1100], 1, 2, 128, 128), ([3000, 1, 200], 2, 2, 128, 64), ([0, 2100], 1, 3, 64, 200), ([513, 512, 1200, 1900], 1, 1, 64, 8)])
def test_long_sequences_of_few_heads(cuda_lib, lens, Hk, Hv, dk, dv):
    """Later blocks are prepared beside the chains that take them."""
    case(cuda_lib, lens, Hk, Hv, dk, dv, seed=len(lens) + dk, extra=3)


def test_many_value_heads_of_a_key_head(cuda_lib):
    case(cuda_lib, [1030, 20], 1, 12, 64, 16, seed=21)


def test_ragged_with_empty_sequences_and_rows_behind(cuda_lib):
    case(cuda_lib, [0, 3, 0, 190, 64, 1, 0, 77], 2, 6, 128, 64, seed=4, extra=9)


def test_many_sequences(cuda_lib):
    case(cuda_lib, [1 + 7 * i % 83 for i in range(300)], 1, 1, 64, 16, seed=5)


def test_negative_slots(cuda_lib):
    case(cuda_lib, [66, 70, 3], 1, 2, 128, 64, seed=6, slots=[-1, 4, -3])


@pytest.mark.parametrize("how", [
    dict(decay=(1e-6, 1e-5)),                    # a state that hardly decays
    dict(decay=(5.0, 60.0)),                     # one that is forgotten at once
    dict(lean=5.0, beta=(0.9, 1.0)),             # keys nearly the same: the inverse is far from 1
    dict(lean=0.0, beta=(1.0, 2.0)),             # reflections
    dict(beta=(0.0, 1e-4)),
], ids=["keeps", "forgets", "leaning", "reflecting", "weak"])
def test_gates(cuda_lib, how):
    case(cuda_lib, [333], 1, 2, 128, 64, seed=7, **how)


def test_chunks_continue_one_another(cuda_lib):
    """A prompt in pieces ends where the whole one does, and steps go on from there."""
    sv = cuda_lib
    Hk, Hv, dk, dv = 2, 4, 128, 128
    r = plain.rows(300, Hk, Hv, dk, dv, 11)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = torch.zeros(1, Hv, dv, dk, device="cuda")
    outs = []
    for lo, hi in ((0, 100), (100, 101), (101, 230), (230, 296)):
        o = torch.empty(hi - lo, Hv, dv, device="cuda", dtype=torch.bfloat16)
        chunk(sv, a, one, [x[lo:hi] for x in plain.on(r)], o, torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"))
        outs.append(o)
    o = torch.empty(4, Hv, dv, device="cuda", dtype=torch.bfloat16)
    sv.gdn_step(a, one, *(x[296:] for x in plain.on(r)), o, 4, commit=True)
    assert sv.sv_last_device_error() == sv.SV_OK
    S, want = plain.run(torch.zeros(Hv, dv, dk), r, 0, 300)
    plain.close(torch.cat(outs + [o]), want, OUT, BF16, "o")
    plain.close(a[0], S, STATE, 0.0, "state")


def test_sizes_of_keys_values_and_states(cuda_lib):
    """Keys of other norms (with strengths to match), large and small values, queries of any size."""
    sv = cuda_lib
    T, Hk, Hv, dk, dv = 150, 2, 2, 128, 64
    for ks, vs, qs in ((1e-3, 1.0, 1.0), (300.0, 1e4, 1e-3), (1.0, 1e-5, 1e5), (1.0, 1e20, 1.0)):
        r = plain.rows(T, Hk, Hv, dk, dv, 12)
        r["k"], r["v"], r["q"] = ((r[n].float() * s).bfloat16() for n, s in (("k", ks), ("v", vs), ("q", qs)))
        r["beta"] = r["beta"] / ks ** 2
        pool = torch.randn(1, Hv, dv, dk, generator=torch.Generator().manual_seed(1)) * (vs / ks)
        states, o = pool.cuda(), torch.empty(T, Hv, dv, device="cuda", dtype=torch.bfloat16)
        chunk(sv, states, torch.zeros(1, dtype=torch.int32, device="cuda"), plain.on(r), o,
              torch.tensor([0, T], dtype=torch.int32, device="cuda"))
        assert sv.sv_last_device_error() == sv.SV_OK
        S, want = plain.run(pool[0], r, 0, T)
        plain.close(o, want, OUT, BF16, f"o {ks} {vs} {qs}")
        plain.close(states[0], S, STATE, 0.0, f"state {ks} {vs} {qs}")


def test_offsets_out_of_order(cuda_lib):
    """A sequence whose offsets are out of order or range is left out and reported."""
    sv = cuda_lib
    T, Hk, Hv, dk, dv = 100, 1, 2, 64, 64
    r = plain.rows(T, Hk, Hv, dk, dv, 13)
    pool = torch.randn(3, Hv, dv, dk, generator=torch.Generator().manual_seed(1))
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    for cu, bad in (([0, 40, 30, 100], 1), ([0, 40, 90, 101], 2), ([-1, 40, 90, 100], 0)):
        states, o = pool.cuda(), torch.full((T, Hv, dv), 99.0, device="cuda", dtype=torch.bfloat16)
        chunk(sv, states, slots, plain.on(r), o, torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
        for b in range(3):
            if b == bad:
                assert torch.equal(states[b].cpu(), pool[b])
            else:
                S, want = plain.run(pool[b], r, cu[b], cu[b + 1])
                plain.close(states[b], S, STATE, 0.0, "state")
    assert sv.sv_last_device_error() == sv.SV_OK


def test_offsets_that_fall_far(cuda_lib):
    """Sequences that share rows: nothing waits for what never comes, and the next call is right."""
    sv = cuda_lib
    T, Hk, Hv, dk, dv = 3200, 1, 2, 64, 64
    r = plain.on(plain.rows(T, Hk, Hv, dk, dv, 15))
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    states, o = torch.zeros(3, Hv, dv, dk, device="cuda"), torch.zeros(T, Hv, dv, device="cuda", dtype=torch.bfloat16)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good = [states.clone(), o.clone()]
    chunk(sv, good[0], slots, r, good[1], ints(0, 3000, 3100, 3200))
    assert sv.sv_last_device_error() == sv.SV_OK
    for cu in ((0, 3000, 100, 3200), (100, 3200, 0, 3100), (0, 3201, 0, 3200)):
        chunk(sv, states, slots, r, o, ints(*cu))
        assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
    states.zero_()
    chunk(sv, states, slots, r, o, ints(0, 3000, 3100, 3200))
    assert sv.sv_last_device_error() == sv.SV_OK
    assert torch.equal(states, good[0]) and torch.equal(o, good[1])


@pytest.mark.parametrize("lens", [[130, 7, 260], [1500, 7, 1700]])
def test_bits_repeat_and_a_captured_call_follows_its_inputs(cuda_lib, lens):
    sv = cuda_lib
    Hk, Hv, dk, dv = 2, 4, 128, 128
    T = sum(lens)
    q, k, v, g, beta = plain.on(plain.rows(T, Hk, Hv, dk, dv, 14))
    pool = torch.randn(5, Hv, dv, dk, generator=torch.Generator().manual_seed(2)).cuda()
    slots, cu = torch.tensor([3, 0, 4], dtype=torch.int32, device="cuda"), torch.tensor([0, lens[0], lens[0] + 7, T], dtype=torch.int32, device="cuda")
    ws = sv.workspace(sv.gdn_chunk_workspace_bytes(3, T, Hk, Hv, dk, dv))

    def once(st, o):
        sv.gdn_chunk(st, slots, q, k, v, g, beta, o, cu, workspace=ws)
        return st, o
    new = lambda: torch.full((T, Hv, dv), 9.0, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    first = once(pool.clone(), new())
    states, o = pool.clone(), new()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once(states, o)
    states.copy_(pool)
    graph.replay()
    assert torch.equal(states, first[0]) and torch.equal(o, first[1])
    slots.copy_(torch.tensor([1, 2, 0])), cu.copy_(torch.tensor([0, 1, 300, T]))
    states.copy_(pool)
    graph.replay()
    again = once(pool.clone(), new())
    assert sv.sv_last_device_error() == sv.SV_OK
    assert torch.equal(states, again[0]) and torch.equal(o, again[1])
