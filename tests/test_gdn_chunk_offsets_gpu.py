"""gdn_chunk where some offsets are out of order or range (GPU): the sequences that they
spoil are left out and reported, and no other one, its output or its state sees any of it."""
import pytest
import torch

import gdn_plain as plain

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8
STATE, OUT = 2.0 ** -14, 2.0 ** -8  # of a row's largest value, as in the call's own tests


def spoiled(B, each, at, value):
    """Offsets of B sequences of `each` rows, one of them out of range or order."""
    cu = [each * b for b in range(B + 1)]
    cu[at] = value
    return cu


@pytest.mark.parametrize("T,cu", [
    (100, [0, 40, 10000, 60, 100]),          # between two good ones, past the end
    (400, [0, 300, -5, 300, 400]),           # before the beginning
    (400, [300, 400, -1, 0, 200]),           # good ones that do not stand in the rows' order
    (100, [0, 0, 5000, 100]),
    (190, [0, 100000, 90, 190]),
    (4200, [0, 2000, 40000, 2000, 4200]),
    (4200, [2100, 4200, -1000000, 0, 2100]),  # blocks that are prepared beside the chains too
    (1300, spoiled(100, 13, 50, 1 << 30)),
    (2600, spoiled(200, 13, 100, 1 << 30)),
    (2600, spoiled(200, 13, 7, -7)),
    (2600, spoiled(200, 13, 200, 2601)),
    (22500, spoiled(2500, 9, 1500, -1)),
    (22500, spoiled(2500, 9, 1024, 1 << 30)),
], ids=lambda x: str(len(x) - 1) if isinstance(x, list) else None)
def test_sequences_beside_bad_offsets(cuda_lib, T, cu):
    sv, B, Hk, Hv, dk, dv = cuda_lib, len(cu) - 1, 1, 2, 64, 64
    r = plain.rows(T, Hk, Hv, dk, dv, 61)
    pool = torch.randn(B + 1, Hv, dv, dk, generator=torch.Generator().manual_seed(62)) * 0.3
    slots = torch.randperm(B + 1, generator=torch.Generator().manual_seed(63))[:B].int()
    states, o = pool.cuda(), torch.full((T, Hv, dv), 99.0, device="cuda", dtype=torch.bfloat16)
    ws = sv.workspace(sv.gdn_chunk_workspace_bytes(B, T, Hk, Hv, dk, dv))
    ws.fill_(255)  # nothing in it has to be zero; what an earlier call left is not used either
    sv.gdn_chunk(states, slots.cuda(), *plain.on(r), o, torch.tensor(cu, dtype=torch.int32, device="cuda"), workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
    want, written = pool.double().clone(), torch.zeros(T, dtype=torch.bool)
    out = torch.zeros(T, Hv, dv, dtype=torch.float64)
    for b in range(B):
        lo, hi = cu[b], cu[b + 1]
        if 0 <= lo <= hi <= T:
            want[slots[b]], out[lo:hi] = plain.run(pool[slots[b]], r, lo, hi)
            assert not written[lo:hi].any()  # no two of them share rows here
            written[lo:hi] = True
    plain.close(states, want, STATE, 0.0, "states")
    plain.close(o[written.cuda()], out[written], OUT, BF16, "o")
    assert bool((o[~written.cuda()] == 99.0).all())


def test_rows_that_too_many_sequences_name(cuda_lib):
    """Good sequences that share rows have their own states while the blocks of all find places; beyond that
    all are left out."""
    sv, T, Hk, Hv, dk, dv = cuda_lib, 300, 1, 2, 64, 64
    r = plain.rows(T, Hk, Hv, dk, dv, 64)
    pool = torch.randn(5, Hv, dv, dk, generator=torch.Generator().manual_seed(65)) * 0.3
    slots = torch.arange(5, dtype=torch.int32, device="cuda")
    # places: 300 / 64 + 5 = 9 blocks; 3 + 0 + 5, and 5 + 0 + 5 + 0 + 5
    for cu, kept in (([0, 190, 10, 300, 300, 300], True), ([0, 300, 0, 300, 0, 300], False)):
        states, o = pool.cuda(), torch.full((T, Hv, dv), 99.0, device="cuda", dtype=torch.bfloat16)
        ws = sv.workspace(sv.gdn_chunk_workspace_bytes(5, T, Hk, Hv, dk, dv))
        ws.fill_(255)
        sv.gdn_chunk(states, slots, *plain.on(r), o, torch.tensor(cu, dtype=torch.int32, device="cuda"), workspace=ws)
        assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
        want = pool.double().clone()
        for b in range(5):
            if kept and cu[b] <= cu[b + 1]:
                want[b], _ = plain.run(pool[b], r, cu[b], cu[b + 1])
        plain.close(states, want, STATE, 0.0, "states")
        if not kept:
            assert bool((o == 99.0).all())


def test_rows_that_very_many_sequences_name(cuda_lib):
    """The count of their blocks passes every limit; nothing is written, and the next call is right."""
    sv, T, B, Hk, Hv, dk, dv = cuda_lib, 13000, 1500, 1, 1, 64, 16
    r = plain.rows(T, Hk, Hv, dk, dv, 66)
    pool = torch.randn(B, Hv, dv, dk, generator=torch.Generator().manual_seed(67)) * 0.3
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    states, o = pool.cuda(), torch.full((T, Hv, dv), 99.0, device="cuda", dtype=torch.bfloat16)
    ws = sv.workspace(sv.gdn_chunk_workspace_bytes(B, T, Hk, Hv, dk, dv))
    ws.fill_(255)
    cu = torch.tensor([0, T] * (B // 2) + [0], dtype=torch.int32, device="cuda")
    sv.gdn_chunk(states, slots, *plain.on(r), o, cu, workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
    assert torch.equal(states.cpu(), pool) and bool((o == 99.0).all())
    cu = torch.tensor([0] * (B - 2) + [3000, T - 1, T], dtype=torch.int32, device="cuda")
    sv.gdn_chunk(states, slots, *plain.on(r), o, cu, workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_OK
    want, out = pool.double().clone(), []
    for b, lo, hi in ((B - 3, 0, 3000), (B - 2, 3000, T - 1), (B - 1, T - 1, T)):
        want[b], got = plain.run(pool[b], r, lo, hi)
        out.append(got)
    plain.close(states, want, STATE, 0.0, "states")
    plain.close(o, torch.cat(out), OUT, BF16, "o")
