"""gdn_step against the rule in 64 bits, token by token.

fp32 arithmetic: a token's two dot products of dk terms and its update are off
by at most (dk + 8) 2^-24 of sums of absolute values, which pass a row's largest
value by at most sqrt(dk) and carry over from token to token without growing:
tokens * (dk + 8) * 2^-24 * sqrt(dk) of the row's largest, times 4 for rows whose
history was larger; the output's own rounding is half a step."""
import math

import pytest
import torch

import gdn_plain as plain

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8


def bound(tokens, dk):
    return 4 * tokens * (dk + 8) * 2.0 ** -24 * math.sqrt(dk)


def case(sv, B, M, tape_M, Hk, Hv, dk, dv, commit, seed, o_dtype=torch.bfloat16, slots=None, replay=None, stride=0):
    N = B + 3
    gen = torch.Generator().manual_seed(seed)
    pool = torch.randn(N, Hv, dv, dk, generator=gen) * 0.3
    slots = torch.randperm(N, generator=gen)[:B].int() if slots is None else torch.tensor(slots, dtype=torch.int32)
    now, old = plain.rows(B * M, Hk, Hv, dk, dv, seed + 1), plain.rows(B * tape_M, Hk, Hv, dk, dv, seed + 2)
    replay = [int(x) for x in torch.randint(0, tape_M + 1, (B,), generator=gen)] if replay is None else replay
    big = torch.full((N, Hv * dv * dk + stride), 7.0, device="cuda")
    states = big[:, :Hv * dv * dk].view(N, Hv, dv, dk)
    states.copy_(pool)
    o = torch.full((B * M, Hv, dv), 99.0, device="cuda", dtype=o_dtype)
    tape = plain.on(old)[1:] if tape_M else None
    if M == 0:
        o = None
    n = torch.tensor(replay, dtype=torch.int32, device="cuda") if tape_M else None
    args = [None] * 5 if M == 0 else plain.on(now)
    sv.gdn_step(states, slots.cuda(), *args, o, M, tape=tape, n_replay=n, commit=commit)
    assert sv.sv_last_device_error() == sv.SV_OK
    want, out = pool.double().clone(), []
    for b in range(B):
        at = int(slots[b])
        S = pool[at].double() if at >= 0 else torch.zeros(Hv, dv, dk, dtype=torch.float64)
        S, _ = plain.run(S, old, b * tape_M, b * tape_M + (replay[b] if tape_M else 0), False)
        after, got = plain.run(S, now, b * M, (b + 1) * M) if M else (S, None)
        out.append(got)
        if at >= 0:
            want[at] = after if commit else S
    tol = bound(M + tape_M, dk)
    if M:
        plain.close(o, torch.cat(out), tol, BF16 if o_dtype is torch.bfloat16 else 0.0, "o")
    plain.close(states, want, tol, 0.0, "states")
    touched = {int(s) for b, s in enumerate(slots) if s >= 0 and (commit or (tape_M and replay[b]))}
    for s in set(range(N)) - touched:  # equal bits where nothing was to be written
        assert torch.equal(states[s].cpu(), pool[s])
    if stride:
        assert bool((big[:, Hv * dv * dk:] == 7.0).all())


@pytest.mark.parametrize("dk,dv", [(64, 72), (128, 128), (256, 40), (128, 8), (64, 256)])
@pytest.mark.parametrize("commit", [False, True])
def test_shapes(cuda_lib, dk, dv, commit):
    case(cuda_lib, 5, 3, 4, 2, 6, dk, dv, commit, seed=dk + dv)


@pytest.mark.parametrize("B,M,tape_M", [(1, 1, 0), (61, 1, 0), (1, 64, 0), (2, 33, 64), (9, 1, 1), (70, 4, 4)])
def test_counts(cuda_lib, B, M, tape_M):
    case(cuda_lib, B, M, tape_M, 4, 8, 128, 64, True, seed=B + M)


@pytest.mark.parametrize("B,M,tape_M,Hv,dk,dv", [(200, 1, 0, 8, 128, 64), (90, 4, 4, 8, 128, 72), (170, 2, 3, 8, 64, 136),
                                                (110, 3, 0, 8, 256, 40), (160, 1, 2, 8, 128, 8), (160, 0, 5, 8, 128, 64)])
@pytest.mark.parametrize("commit", [False, True])
def test_many_states(cuda_lib, B, M, tape_M, Hv, dk, dv, commit):
    """Enough tiles for every SM to walk over several, some of a few rows only, slots of -1 among them."""
    if M == 0:
        commit = False
    slots = [(b * 7) % B if b % 11 else -1 for b in range(B)]
    slots = [s if s < 0 or s not in slots[:b] else -1 for b, s in enumerate(slots)]
    case(cuda_lib, B, M, tape_M, 4, Hv, dk, dv, commit, seed=B + dk, slots=slots)


def test_fp32_outputs_and_slot_strides(cuda_lib):
    case(cuda_lib, 4, 2, 2, 2, 4, 128, 128, False, seed=3, o_dtype=torch.float32, stride=64)


def test_negative_slots_start_from_zeros_and_are_not_kept(cuda_lib):
    case(cuda_lib, 4, 2, 3, 2, 4, 128, 64, True, seed=5, slots=[-1, 4, -7, 0], replay=[3, 0, 0, 2])


def test_nothing_accepted_leaves_the_state(cuda_lib):
    case(cuda_lib, 3, 2, 2, 2, 4, 128, 64, False, seed=6, replay=[0, 0, 0])


def test_commit_only(cuda_lib):
    """M = 0 is the tape alone; the same tokens through M rows give the same bits."""
    sv = cuda_lib
    B, n, Hk, Hv, dk, dv = 3, 4, 2, 4, 128, 64
    r = plain.rows(B * n, Hk, Hv, dk, dv, 8)
    pool = torch.randn(B, Hv, dv, dk, generator=torch.Generator().manual_seed(9)).cuda()
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    full = torch.full((B,), n, dtype=torch.int32, device="cuda")
    a, b = pool.clone(), pool.clone()
    sv.gdn_step(a, slots, None, None, None, None, None, None, 0, tape=plain.on(r)[1:], n_replay=full)
    o = torch.empty(B * n, Hv, dv, device="cuda", dtype=torch.bfloat16)
    sv.gdn_step(b, slots, *plain.on(r), o, n, commit=True)
    assert sv.sv_last_device_error() == sv.SV_OK
    assert torch.equal(a, b) and not torch.equal(a, pool)


def test_counts_and_slots_out_of_range(cuda_lib):
    """They count as the nearest in range (slots: as negative) and are reported."""
    sv = cuda_lib
    B, M, Hk, Hv, dk, dv = 3, 2, 2, 2, 64, 64
    r, old = plain.rows(B * M, Hk, Hv, dk, dv, 1), plain.rows(B * M, Hk, Hv, dk, dv, 2)
    pool = torch.randn(B, Hv, dv, dk, generator=torch.Generator().manual_seed(3)).cuda()
    states = pool.clone()
    o = torch.empty(B * M, Hv, dv, device="cuda", dtype=torch.bfloat16)
    for slots, n in (([0, 1, 2], [0, 5, 1]), ([0, 1, 2], [-1, 1, 1]), ([0, 3, 2], [1, 1, 1])):
        states.copy_(pool)
        sv.gdn_step(states, torch.tensor(slots, dtype=torch.int32, device="cuda"), *plain.on(r), o, M,
                    tape=plain.on(old)[1:], n_replay=torch.tensor(n, dtype=torch.int32, device="cuda"))
        assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
        for b in range(B):
            S, _ = plain.run(pool[b].cpu(), old, b * M, b * M + min(max(n[b], 0), M), False)
            if slots[b] < B:
                plain.close(states[b], S, bound(4, dk), 0.0, "state")
            else:
                assert torch.equal(states[b], pool[b])
    assert sv.sv_last_device_error() == sv.SV_OK


def test_matches_gdn_verify(cuda_lib):
    """One sequence: the same rule as gdn_verify, to rounding."""
    sv = cuda_lib
    M, Hk, Hv, dk, dv = 4, 4, 8, 128, 128
    now, old = plain.rows(M, Hk, Hv, dk, dv, 1), plain.rows(M, Hk, Hv, dk, dv, 2)
    pool = torch.randn(1, Hv, dv, dk, generator=torch.Generator().manual_seed(3)).cuda()
    a, b = pool.clone(), pool[0].clone()
    oa, ob = (torch.empty(M, Hv, dv, device="cuda", dtype=torch.float32) for _ in range(2))
    zero, n = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 3, dtype=torch.int32, device="cuda")
    sv.gdn_step(a, zero, *plain.on(now), oa, M, tape=plain.on(old)[1:], n_replay=n)
    sv.gdn_verify(b, *plain.on(now), ob, tape=tuple(plain.on(old)[1:]), n_replay=3)
    assert sv.sv_last_device_error() == sv.SV_OK
    tol = bound(7, dk)
    plain.close(a[0], b.cpu(), 2 * tol, 0.0, "state")
    plain.close(oa, ob.cpu(), 2 * tol, 0.0, "o")


def test_captured_call_follows_slots_and_counts(cuda_lib):
    sv = cuda_lib
    B, M, Hk, Hv, dk, dv = 3, 2, 2, 4, 128, 64
    now, old = plain.on(plain.rows(B * M, Hk, Hv, dk, dv, 1)), plain.on(plain.rows(B * M, Hk, Hv, dk, dv, 2))[1:]
    pool = torch.randn(6, Hv, dv, dk, generator=torch.Generator().manual_seed(3)).cuda()
    states, o = pool.clone(), torch.zeros(B * M, Hv, dv, device="cuda", dtype=torch.bfloat16)
    slots, n = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    slots.copy_(torch.tensor([0, 1, 2]))
    call = lambda st, out: sv.gdn_step(st, slots, *now, out, M, tape=old, n_replay=n)  # noqa: E731
    call(states.clone(), o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(states, o)
    for at, count in (([5, 0, 3], [2, 0, 1]), ([-1, 4, 1], [1, 1, 2])):
        slots.copy_(torch.tensor(at)), n.copy_(torch.tensor(count))
        states.copy_(pool)
        graph.replay()
        got, want, out = states.clone(), pool.clone(), torch.zeros_like(o)
        call(want, out)
        assert sv.sv_last_device_error() == sv.SV_OK
        assert torch.equal(got, want) and torch.equal(o, out)
