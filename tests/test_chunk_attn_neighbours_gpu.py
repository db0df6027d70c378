"""paged_chunk_attn where one sequence's values or queries are not finite (GPU): they reach
no other one's rows, and no other row of their own."""
import pytest
import torch

from test_chunk_attn_gpu import Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hkv,B,e4m3", [
    (128, 1, 900, False), (256, 1, 500, False), (128, 8, 100, False), (256, 6, 60, False), (128, 16, 24, False),
    (128, 1, 900, True), (256, 1, 500, True)])
@pytest.mark.parametrize("page", [16, 64])
def test_values_of_other_sequences(cuda_lib, D, Hkv, B, e4m3, page):
    """Many sequences a CTA, half of them with values, and keys, that are NaN or infinite in every slot."""
    sv, g = cuda_lib, torch.Generator().manual_seed(81)
    lens = torch.tensor([17, 33, 70, 100, 128, 200])[torch.randint(0, 6, (B,), generator=g)].tolist()
    c = Call(sv, [(1, n) for n in lens], 2 * Hkv, Hkv, D, page, e4m3=e4m3, seed=82, dirty=False)
    c.check()
    t = c.tensors()
    good = c.run(t).clone()
    bad = torch.rand(B, generator=g) < 0.5
    for b in bad.nonzero().flatten().tolist():
        pages = c.table[b, :-(-lens[b] // page)].long().cuda()
        t[1].v[pages] = torch.tensor(float("nan") if e4m3 or b % 3 else float("inf")).to(t[1].v.dtype).cuda()
        if b % 2:
            t[1].k[pages] = torch.tensor(float("nan")).to(t[1].k.dtype).cuda()
    o = c.run(t)
    assert sv.sv_last_device_error() == sv.SV_OK
    assert torch.equal(o[~bad.cuda()], good[~bad.cuda()])


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
def test_queries_of_cut_items(cuda_lib, D, e4m3):
    """Long caches, whose items are cut and joined: such a query's own row is NaN, as where nothing is cut."""
    sv = cuda_lib
    c = Call(sv, [(3, 9001), (1, 12345), (2, 1)], 4, 1, D, 64, e4m3=e4m3, seed=87, dirty=False)
    t = c.tensors()
    good = c.run(t).clone()
    t[0][1, 2] = float("nan")
    t[0][2, 1, 5] = float("inf")
    t[0][3, 0, 77] = float("nan")
    t[0][4, 3] = float("nan")          # a row before position 0: it sees nothing
    o = c.run(t)
    assert sv.sv_last_device_error() == sv.SV_OK
    for row, head in ((1, 2), (2, 1), (3, 0)):
        assert bool(o[row, head].isnan().all())
        good[row, head] = o[row, head] = 0
    assert torch.equal(o, good)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("entry", [-1, 0, 1], ids=["below", "next", "beyond"])
def test_a_needed_page_just_outside_the_cache(cuda_lib, D, entry):
    """Its slots count as zeros, and it is reported: the page behind the last one too, and an entry of -1."""
    sv = cuda_lib
    c = Call(sv, [(4, 100)], 4, 2, D, 16, seed=88, dirty=False)
    t = list(c.tensors())
    t[2] = t[2].clone()
    t[2][0, 2] = -1 if entry < 0 else c.k.shape[0] + entry
    o = c.run(t).clone()
    assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
    page = int(c.table[0, 2])
    t = list(c.tensors())
    t[1].k[page], t[1].v[page] = 0.0, 0.0
    assert torch.equal(c.run(t), o)
    assert sv.sv_last_device_error() == sv.SV_OK
