"""gdn_step at the most tiles that a call can have streamed (GPU): all are walked over."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_nearly_2_to_the_31_tiles(cuda_lib):
    """42966 sequences of 49981 heads, 2^31 - 2 tiles of eight rows; rows without a state, outputs of 34 GB."""
    sv, B, Hv, dk, dv = cuda_lib, 42966, 49981, 64, 8
    assert B * Hv == 2 ** 31 - 2
    try:
        one = torch.zeros(1, 1, dk, device="cuda", dtype=torch.bfloat16)
        one[0, 0, 0] = 1.0
        v = torch.arange(1, dv + 1, device="cuda", dtype=torch.bfloat16)
        states, slots = torch.zeros(1, Hv, dv, dk, device="cuda"), torch.full((B,), -1, dtype=torch.int32, device="cuda")
        g, beta = torch.zeros(B, Hv, device="cuda"), torch.full((B, Hv), 0.5, device="cuda")
        o = torch.full((B, Hv, dv), 99.0, device="cuda", dtype=torch.bfloat16)
        sv.gdn_step(states, slots, one.expand(B, 1, dk), one.expand(B, 1, dk), v.expand(B, Hv, dv), g, beta, o, 1, commit=True)
        assert sv.sv_last_device_error() == sv.SV_OK
        # from zeros: S = v k^T / 2, o = S q = v / 2
        missed = sum(int((part != v * 0.5).sum()) for part in o.split(2048))
        assert missed == 0
        assert not states.any()
    finally:
        torch.cuda.empty_cache()
