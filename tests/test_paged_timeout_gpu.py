"""Bounded device waits of the attention over a paged cache (GPU): a wait that
runs out is reported, not hung, and the next call is right.

With the test aid SV_LAUNCH_TEST_STALL_COPY the first slot of every CTA's ring
never counts as filled, so its consumers' waits run out (about 1.5 s of SM
clocks each) and with them the producers'; nothing faults, traps or spins
unbounded.  All lanes of a warp have to leave such a wait alike, as they go on
to instructions and barriers of the whole warp.
"""
import time

import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


# one tile of rows with pieces of one head in many CTAs, several heads a CTA, two
# tiles with chunks in pairs, eight tiles; streams longer and shorter than the ring
@pytest.mark.parametrize("lens,M,Hq,Hkv,D,e4m3", [
    ([60000], 1, 8, 2, 128, False), ([37] * 200, 2, 4, 2, 128, False), ([3000, 900, 17], 4, 12, 2, 256, True),
    ([500, 2000], 16, 16, 2, 256, False)])
def test_stalled_copy_times_out_and_context_stays_usable(cuda_lib, lens, M, Hq, Hkv, D, e4m3):
    sv, g = cuda_lib, torch.Generator(device=DEV).manual_seed(1)
    page, B = 64, len(lens)
    width = -(-max(lens) // page)
    t = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k, v = (torch.randn(B * width, page, Hkv, D, generator=g, device=DEV).to(t) for _ in range(2))
    cache = sv.PagedKV(k, v)
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    q = torch.randn(B * M, Hq, D, generator=g, device=DEV).bfloat16()
    o = torch.zeros_like(q)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = sv.workspace(sv.paged_attn_workspace_bytes(B, M, Hq, Hkv, D))
    old = sv.sv_get_launch_flags()
    assert sv.sv_last_device_error() == sv.SV_OK
    try:
        sv.sv_set_launch_flags(old | sv.SV_LAUNCH_TEST_STALL_COPY)
        t0 = time.monotonic()
        sv.paged_attn(q, cache, table, n, o, M, D ** -0.5, workspace=ws)
        status = sv.sv_last_device_error()
        elapsed = time.monotonic() - t0
    finally:
        sv.sv_set_launch_flags(old)
    assert status == sv.SV_ERR_TIMEOUT
    assert elapsed < 60.0
    assert sv.sv_last_device_error() == sv.SV_OK
    sv.paged_attn(q, cache, table, n, o, M, D ** -0.5, workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_OK
    b, big = B - 1, float(v.float().abs().max())
    K, V = (x[table[b].long()].view(-1, Hkv, D)[:lens[b]].float().cpu() for x in (k, v))
    want = plain.attend(q[b * M:].cpu(), K, V, lens[b] - M, D ** -0.5, 0, 0)
    assert float((o[b * M:].double().cpu() - want).abs().max()) <= plain.attention_tolerance(big)
