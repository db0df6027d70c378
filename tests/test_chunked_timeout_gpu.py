"""Bounded device waits of paged_chunk_attn and gdn_chunk (GPU): a wait that runs
out is reported, not hung, and the next call is right.

With the test aid SV_LAUNCH_TEST_STALL_COPY the first copy of every CTA's ring never
counts as arrived: the wait for it runs out (about 1.5 s of SM clocks), and with it
those behind it.  All lanes of a warp leave such a wait alike, every named barrier is
still met by all of its warps, and tensor memory is given back; nothing faults or traps."""
import time

import pytest
import torch

import gdn_plain
from test_chunk_attn_gpu import Call

pytestmark = pytest.mark.gpu


def stalled(sv, f):
    old = sv.sv_get_launch_flags()
    assert sv.sv_last_device_error() == sv.SV_OK
    try:
        sv.sv_set_launch_flags(old | sv.SV_LAUNCH_TEST_STALL_COPY)
        t0 = time.monotonic()
        f()
        status = sv.sv_last_device_error()
        elapsed = time.monotonic() - t0
    finally:
        sv.sv_set_launch_flags(old)
    assert status == sv.SV_ERR_TIMEOUT
    assert elapsed < 60.0
    assert sv.sv_last_device_error() == sv.SV_OK


# two tiles a CTA, single tiles, heads of 256; items that are cut and joined; several items a CTA
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("seqs,Hq,Hkv,D", [
    ([(300, 900), (7, 7)], 8, 2, 128), ([(3, 5000)], 16, 2, 128), ([(90, 400), (1, 1)], 12, 2, 256), ([(2, 30)] * 300, 4, 2, 128)])
def test_chunk_attention(cuda_lib, seqs, Hq, Hkv, D, e4m3):
    c = Call(cuda_lib, seqs, Hq, Hkv, D, 32, e4m3=e4m3, dirty=False)
    t = c.tensors()
    stalled(cuda_lib, lambda: c.run(t))
    c.check()


# one chain of several blocks; more CTAs than fit at once; blocks prepared beside the chains
@pytest.mark.parametrize("lens,Hv,dk,dv", [([400], 2, 128, 128), ([70, 3, 90], 4, 64, 200), ([40] * 90, 4, 128, 64), ([2600], 2, 128, 128)])
def test_chunked_rule(cuda_lib, lens, Hv, dk, dv):
    sv, B, T = cuda_lib, len(lens), sum(lens)
    r = gdn_plain.rows(T, 2, Hv, dk, dv, 3)
    rows = gdn_plain.on(r)
    slots = torch.arange(B, device="cuda").int()
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    o = torch.empty(T, Hv, dv, device="cuda", dtype=torch.bfloat16)
    ws = sv.workspace(sv.gdn_chunk_workspace_bytes(B, T, 2, Hv, dk, dv))
    states = torch.zeros(B, Hv, dv, dk, device="cuda")
    stalled(sv, lambda: sv.gdn_chunk(states, slots, *rows, o, cu, workspace=ws))
    states.zero_()
    sv.gdn_chunk(states, slots, *rows, o, cu, workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_OK
    S, want = gdn_plain.run(torch.zeros(Hv, dv, dk), r, 0, lens[0])
    gdn_plain.close(o[:lens[0]], want, 2.0 ** -8, 2.0 ** -8, "o")
    gdn_plain.close(states[0], S, 2.0 ** -14, 0.0, "state")
