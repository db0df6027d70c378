"""gdn_chunk over states, values, queries and gates of any size that its contract allows
(GPU), against the rule in 64 bits."""
import pytest
import torch

import gdn_plain as plain

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8
STATE, OUT = 2.0 ** -14, 2.0 ** -8  # of a row's largest value, as in the call's own tests


def compare(sv, r, pool, T):
    _, Hv, dv, dk = pool.shape
    Hk = r["k"].shape[1]
    states, o = pool.cuda(), torch.empty(T, Hv, dv, device="cuda", dtype=torch.bfloat16)
    ws = sv.workspace(sv.gdn_chunk_workspace_bytes(1, T, Hk, Hv, dk, dv))
    sv.gdn_chunk(states, torch.zeros(1, dtype=torch.int32, device="cuda"), *plain.on(r), o,
                 torch.tensor([0, T], dtype=torch.int32, device="cuda"), workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_OK
    S, want = plain.run(pool[0], r, 0, T)
    plain.close(o, want, OUT, BF16, "o")
    plain.close(states[0], S, STATE, 0.0, "state")
    return states[0].double().cpu(), S


def some_rows(T, Hk, Hv, dk, dv, seed, values=1.0, queries=1.0):
    r = plain.rows(T, Hk, Hv, dk, dv, seed)
    r["v"], r["q"] = (r["v"].float() * values).bfloat16(), (r["q"].float() * queries).bfloat16()
    return r


def some_states(Hv, dv, dk, seed, size):
    return torch.randn(1, Hv, dv, dk, generator=torch.Generator().manual_seed(seed)) * size


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("size", [1.0, 1e11, 1e25, 1e36])
def test_tokens_of_no_strength(cuda_lib, dk, size):
    """beta = 0 in whole blocks: they leave the state's decay alone, however large it is."""
    T, Hk, Hv, dv = 150, 1, 2, 40
    for none in (slice(0, T), slice(0, 70), slice(64, 128)):
        r = some_rows(T, Hk, Hv, dk, dv, 71)
        r["beta"][none] = 0.0
        compare(cuda_lib, r, some_states(Hv, dv, dk, 72, size), T)
    r = some_rows(T, Hk, Hv, dk, dv, 71)
    r["beta"][:, 1] = 0.0  # one head of two
    compare(cuda_lib, r, some_states(Hv, dv, dk, 72, size), T)


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("size", [1.0, 1e20, 1e36])
def test_states_that_a_gate_clears(cuda_lib, dk, size):
    """exp(g) = 0 behind a block's updates: an empty state, and what follows starts from it."""
    T, Hk, Hv, dv = 200, 1, 2, 40
    for at in (63, 100, 127):
        r = some_rows(T, Hk, Hv, dk, dv, 73, values=size)
        r["g"][at], r["beta"][at] = -1000.0, 0.0
        compare(cuda_lib, r, some_states(Hv, dv, dk, 74, size), T)


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("size", [1e-36, 1e-30, 1e30, 1e36])
def test_values_and_states_of_any_size(cuda_lib, dk, size):
    T, Hk, Hv, dv = 150, 1, 2, 40
    compare(cuda_lib, some_rows(T, Hk, Hv, dk, dv, 75, values=size), some_states(Hv, dv, dk, 76, size), T)


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("size", [1e-30, 1.0, 1e10, 1e20, 1e36])
@pytest.mark.parametrize("T", [40, 64, 150])
def test_from_an_empty_state(cuda_lib, dk, size, T):
    """A new sequence's state is zeros: nothing about it says how large the values are."""
    Hk, Hv, dv = 1, 2, 40
    compare(cuda_lib, some_rows(T, Hk, Hv, dk, dv, 79, values=size), torch.zeros(1, Hv, dv, dk), T)


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("size", [1e-30, 1e30, 1e38])
def test_queries_of_any_size(cuda_lib, dk, size):
    """Up to the largest bf16 holds, beside states that keep the outputs in range."""
    T, Hk, Hv, dv = 150, 1, 2, 40
    small = 1e-30 if size > 1 else 1.0
    r = some_rows(T, Hk, Hv, dk, dv, 77, values=small, queries=size)
    assert bool(torch.isfinite(r["q"].float()).all())
    compare(cuda_lib, r, some_states(Hv, dv, dk, 78, small), T)


@pytest.mark.parametrize("dk", [64, 128])
def test_keys_of_any_size(cuda_lib, dk):
    """From 1e-30 to the largest bf16 holds, each with a strength to match (none where fp32 has none)."""
    T, Hk, Hv, dv = 150, 1, 2, 40
    r = some_rows(T, Hk, Hv, dk, dv, 80)
    # values go with the keys, so that every token moves the state as much
    size = torch.tensor([1.0, 1e-15, 1e15, 1e38, 1e-30, 1.0, 3e17])[torch.arange(T) % 7]
    r["k"] = (r["k"].float() * size[:, None, None]).bfloat16()
    r["v"] = (r["v"].float() * size[:, None, None]).clamp(-3e38, 3e38).bfloat16()  # finite, as the contract wants them
    assert bool(torch.isfinite(r["k"].float()).all()) and bool(torch.isfinite(r["v"].float()).all())
    r["beta"] = torch.where(size[:, None] > 1e30, torch.zeros(()), (r["beta"].double() / size[:, None].double() ** 2).clamp(max=1e30).float())
    compare(cuda_lib, r, some_states(Hv, dv, dk, 81, 1.0), T)


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("size", [1e6, 1e20, 1e36])
@pytest.mark.parametrize("at", [63, 127])
def test_small_values_behind_a_large_state_that_a_gate_clears(cuda_lib, dk, size, at):
    """At the end of a block of 64, so that no bound of a block holds both: what follows is seen at once."""
    sv, T, Hk, Hv, dv = cuda_lib, 400, 1, 2, 40
    r = some_rows(T, Hk, Hv, dk, dv, 82)
    r["g"][at], r["beta"][at] = -1000.0, 0.0
    pool = some_states(Hv, dv, dk, 83, size)
    states, o = pool.cuda(), torch.empty(T, Hv, dv, device="cuda", dtype=torch.bfloat16)
    sv.gdn_chunk(states, torch.zeros(1, dtype=torch.int32, device="cuda"), *plain.on(r), o,
                 torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                 workspace=sv.workspace(sv.gdn_chunk_workspace_bytes(1, T, Hk, Hv, dk, dv)))
    assert sv.sv_last_device_error() == sv.SV_OK
    S, want = plain.run(pool[0], r, 0, T)
    plain.close(o[:at], want[:at], OUT, BF16, "o before")
    plain.close(o[at:], want[at:], OUT, BF16, "o behind")
    plain.close(states[0], S, STATE, 0.0, "state")
