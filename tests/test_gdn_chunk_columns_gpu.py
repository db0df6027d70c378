"""gdn_chunk over states whose columns are of very different size (GPU): the parts that a state's
elements are held in keep small ones beside large ones.

Keys that are single columns leave the columns apart: S_j <- e^g (1 - beta) S_j, each element by
itself.  One block of 64 tokens, each of another column, unit keys (k' = 2^-4 k), beta = 1/2: a state's
row stands below 2^15 in its operands, whose second parts end at 2^-25, 2^-39 of the row's largest
element m or less, and half of that is applied.  R and U~ stand below 2^14 for a bound of 96 m in
units of 2^4 u, so that each is off by 2^-38 * 96 * 2^-4 m = 2^-35.4 m: 2^-34 m in all, beside what is
relative to the element itself: three operands of 2^-22, and fp32's 2^-24 a few times, 2^-20 in all."""
import pytest
import torch

import gdn_plain as plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk", [64, 128])
def test_small_columns_beside_large_ones(cuda_lib, dk):
    sv, T, Hv, dv = cuda_lib, 64, 2, 128
    gen = torch.Generator().manual_seed(91)
    columns = torch.randperm(dk, generator=gen)[:T]
    k = torch.zeros(T, 1, dk)
    k[torch.arange(T), 0, columns] = 1.0
    r = dict(q=k.bfloat16(), k=k.bfloat16(), v=torch.zeros(T, Hv, dv).bfloat16(), g=torch.full((T, Hv), -0.01),
             beta=torch.full((T, Hv), 0.5))
    pool = torch.randn(1, Hv, dv, dk, generator=gen) * torch.exp2(-torch.randint(0, 25, (dk,), generator=gen).float())
    states, o = pool.cuda(), torch.empty(T, Hv, dv, device="cuda", dtype=torch.bfloat16)
    sv.gdn_chunk(states, torch.zeros(1, dtype=torch.int32, device="cuda"), *plain.on(r), o,
                 torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                 workspace=sv.workspace(sv.gdn_chunk_workspace_bytes(1, T, 1, Hv, dk, dv)))
    assert sv.sv_last_device_error() == sv.SV_OK
    S, _ = plain.run(pool[0], r, 0, T)
    off = (states[0].double().cpu() - S).abs()
    most = pool[0].double().abs().amax(-1, keepdim=True)
    assert bool((off <= 2.0 ** -20 * S.abs() + 2.0 ** -34 * most).all()), float((off / most).max())


@pytest.mark.parametrize("dk", [64, 128])
def test_a_state_that_decays_within_a_block(cuda_lib, dk):
    """Values of zero and e^-6.4 over the block: what is left is 2^-9 or 2^-10 of the row's largest element m at
    its beginning.  The inverse's entries are off by 2^-34, and by that again for each of two joins; 64 of
    them meet residuals of at most about m (b S k), in 64 sums, and errors of independent signs grow as the root
    of their number: 3 * 2^-34 * 8 m an update, 3 * 2^-34 * 8 * 2 m in the state, as only the last ten
    updates or so are not decayed themselves.  That is 2^-18.4 of what is left; with 2^-22 for the rest, 2^-18."""
    sv, T, Hv, dv = cuda_lib, 64, 2, 40
    r = plain.rows(T, 1, Hv, dk, dv, 71)
    r["g"][:], r["v"][:] = -0.1, 0.0
    pool = torch.randn(1, Hv, dv, dk, generator=torch.Generator().manual_seed(72))
    states, o = pool.cuda(), torch.empty(T, Hv, dv, device="cuda", dtype=torch.bfloat16)
    sv.gdn_chunk(states, torch.zeros(1, dtype=torch.int32, device="cuda"), *plain.on(r), o,
                 torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                 workspace=sv.workspace(sv.gdn_chunk_workspace_bytes(1, T, 1, Hv, dk, dv)))
    assert sv.sv_last_device_error() == sv.SV_OK
    S, _ = plain.run(pool[0], r, 0, T)
    plain.close(states[0], S, 2.0 ** -18, 0.0, "state")
