"""paged_attn where one slot stands far above many others (GPU).

The usual form: a first token with a large score and a small value.  Each other
slot's probability is tiny beside it, but together they are the output, so each
has to keep its relative precision.
"""
import math

import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


def far_case(sv, n, B, orders, e4m3, page=64, M=1, Hq=2, D=128, first_value=0.0):
    """Slot 0 of every sequence scores `orders` binary orders above n others,
    which score alike; their values are of one sign."""
    g = torch.Generator(device=DEV).manual_seed(n + B)
    t = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    width = -(-(n + 1) // page)
    k = torch.zeros(B * width, page, 1, D, device=DEV)
    v = torch.rand(B * width, page, 1, D, generator=g, device=DEV) + 0.5
    table = torch.randperm(B * width, generator=g, device=DEV).int().view(B, width)
    k[table[:, 0].long(), 0, 0, 0] = 16.0
    v[table[:, 0].long(), 0] = first_value
    k, v = k.to(t), v.to(t)
    q = torch.zeros(B * M, Hq, D, dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1.0
    scale = orders * math.log(2.0) / 16.0
    lens = torch.full((B,), n + 1, dtype=torch.int32, device=DEV)
    o = torch.full_like(q, float("nan"))
    ws = sv.workspace(sv.paged_attn_workspace_bytes(B, M, Hq, 1, D))
    sv.paged_attn(q, sv.PagedKV(k, v), table, lens, o, M, scale, workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_OK
    want = torch.empty(B * M, Hq, D, dtype=torch.float64, device=DEV)
    for b in range(B):
        K = k[table[b].long()].view(-1, D)[:n + 1].double()
        V = v[table[b].long()].view(-1, D)[:n + 1].double()
        for i in range(M):
            seen = n + 1 - M + i + 1
            w = torch.softmax(K[:seen] @ q[b * M + i, 0].double() * scale, 0)
            want[b * M + i] = w @ V[:seen]
    return o.double(), want


# The output's own rounding and that of each probability (bf16, or fp16 beside
# e4m3 pages), both relative, and 2^-11 for the fp32 sums: a term of 2^-26 of
# its sum is lost where it is added alone, 2^13 of them a lane at most.
@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("orders", [12, 17, 21, 25, 26])
@pytest.mark.parametrize("n,B,M", [(262144, 1, 1), (32768, 1, 4), (4095, 200, 1)])
def test_many_small_probabilities_beside_a_large_one(cuda_lib, n, B, M, orders, e4m3):
    got, want = far_case(cuda_lib, n, B, float(orders), e4m3, M=M)
    assert torch.isfinite(got).all() and (want > 0).all()
    tol = plain.half_step(torch.bfloat16) + plain.half_step(torch.float16 if e4m3 else torch.bfloat16) + 2.0 ** -11
    err = ((got - want).abs() / want).max()
    assert float(err) <= tol, (float(err), tol)


@pytest.mark.parametrize("orders", [17.0, 25.0])
def test_their_mass_counts_beside_the_large_ones_value(cuda_lib, orders):
    """The large slot's value is 1 and the others' lie about it: the output's
    error is far below what their mass (up to 1/128) would leave out."""
    got, want = far_case(cuda_lib, 262144, 1, orders, True, first_value=1.0)
    tol = plain.attention_tolerance(float(want.max()), roundings=0)
    assert float((got - want).abs().max()) <= tol
