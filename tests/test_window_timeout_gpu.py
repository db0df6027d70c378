"""Bounded device waits of window_attn (GPU): a wait that runs out is reported,
not hung, and the next call is right.

With the test aid SV_LAUNCH_TEST_STALL_COPY the first slot of every CTA's K ring
never counts as filled: the issuing warp's wait runs out (about 1.5 s of SM
clocks), and with it those of the softmax warps, the producers and the queries'.
All lanes of a warp leave such a wait alike, every named barrier is still met by
all of its warps, and tensor memory is given back; nothing faults or traps.
"""
import time

import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


# two tiles a CTA, single tiles at D = 128, at D = 256; several items a CTA; more
# sequences than the prefix sums' place (a smaller ring)
@pytest.mark.parametrize("nq,Hq,Hkv,D", [
    ([2500, 40], 32, 8, 128), ([300, 7], 8, 2, 128), ([900, 130], 12, 2, 256), ([3] * 400 + [50], 4, 2, 128)])
def test_stalled_copy_times_out_and_context_stays_usable(cuda_lib, nq, Hq, Hkv, D):
    sv, g = cuda_lib, torch.Generator(device=DEV).manual_seed(2)
    n = sum(nq)
    q = torch.randn(n, Hq, D, generator=g, device=DEV).bfloat16()
    k, v = (torch.randn(n, Hkv, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    cu = torch.tensor([0] + nq, device=DEV).cumsum(0).int()
    o = torch.zeros_like(q)
    old = sv.sv_get_launch_flags()
    assert sv.sv_last_device_error() == sv.SV_OK
    try:
        sv.sv_set_launch_flags(old | sv.SV_LAUNCH_TEST_STALL_COPY)
        t0 = time.monotonic()
        sv.window_attn(q, k, v, o, cu, cu, D ** -0.5)
        status = sv.sv_last_device_error()
        elapsed = time.monotonic() - t0
    finally:
        sv.sv_set_launch_flags(old)
    assert status == sv.SV_ERR_TIMEOUT
    assert elapsed < 60.0
    assert sv.sv_last_device_error() == sv.SV_OK
    sv.window_attn(q, k, v, o, cu, cu, D ** -0.5)
    assert sv.sv_last_device_error() == sv.SV_OK
    last = nq[-1]
    want = plain.attend(q[-last:].cpu(), k[-last:].cpu(), v[-last:].cpu(), 0, D ** -0.5, 0, 0)
    assert float((o[-last:].double().cpu() - want).abs().max()) <= plain.attention_tolerance(float(v.float().abs().max()))
