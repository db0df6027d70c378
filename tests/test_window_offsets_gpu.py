"""window_attn over offsets that fall and rise again (GPU): thousands of
sequences over the same rows are reported and nothing is written, instead of
counts that wrap."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def overlapping(n, heads, D):
    """n rows of `heads` heads in little memory: rows and heads 16 bytes apart."""
    flat = torch.zeros(8 * (n + heads) + D, dtype=torch.bfloat16, device=DEV)
    return flat, flat.as_strided((n, heads, D), (8, 8, 1))


# one position an item (128 heads share a key head): 2048 sequences of 2^21 + 2^10
# rows have 2^32 + 2^21 items, a positive count in 32 bits; of 2^20, 2^31 of them
@pytest.mark.parametrize("Tq", [(1 << 21) + (1 << 10), 1 << 20])
def test_counts_that_pass_32_bits(cuda_lib, Tq):
    sv = cuda_lib
    Hq, Hkv, D, pairs = 128, 1, 256, 2048
    _, q = overlapping(Tq, Hq, D)
    flat, o = overlapping(Tq, Hq, D)
    flat.fill_(9.0)
    k = torch.zeros(16, Hkv, D, dtype=torch.bfloat16, device=DEV)
    cu_q = torch.tensor([0, Tq] * pairs, dtype=torch.int32, device=DEV)
    cu_k = torch.tensor([0, 16] * pairs, dtype=torch.int32, device=DEV)
    sv.window_attn(q, k, k, o, cu_q, cu_k, 0.1)
    assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
    assert (flat == 9.0).all()
    assert sv.sv_last_device_error() == sv.SV_OK


def test_rows_named_twice_within_the_bound(cuda_lib):
    """Fewer items than rows and sequences can have: the good sequences are computed."""
    sv = cuda_lib
    q = torch.randn(60, 2, 128, device=DEV).bfloat16()
    k = torch.randn(60, 1, 128, device=DEV).bfloat16()
    o = torch.full_like(q, 9.0)
    cu = torch.tensor([0, 20, 10, 60], dtype=torch.int32, device=DEV)
    sv.window_attn(q, k, k, o, cu, cu, 0.1)
    assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
    want = torch.full_like(q, 9.0)
    c = torch.tensor([10, 60], dtype=torch.int32, device=DEV)
    sv.window_attn(q, k, k, want, c, c, 0.1)
    assert sv.sv_last_device_error() == sv.SV_OK
    assert torch.equal(o[20:], want[20:])


def test_many_sequences_of_no_and_one_row_stay_within_the_bound(cuda_lib):
    sv = cuda_lib
    n = [i % 2 for i in range(4096)]
    cu = torch.tensor([0] + n, device=DEV).cumsum(0).int()
    T = sum(n)
    q = torch.randn(T, 4, 128, device=DEV).bfloat16()
    k, v = (torch.randn(T, 2, 128, device=DEV).bfloat16() for _ in range(2))
    o = torch.zeros_like(q)
    sv.window_attn(q, k, v, o, cu, cu, 0.1)
    assert sv.sv_last_device_error() == sv.SV_OK
    assert torch.equal(o, v.repeat_interleave(2, 1))   # a row's only key is its own
