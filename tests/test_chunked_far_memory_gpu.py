"""Pages, rows and states more than 2^32 elements from their tensor's first (GPU):
no offset is 32-bit.  Buffers of 9 to 18 GB, of which little is touched."""
import pytest
import torch

import gdn_plain
import paged_plain as plain
from test_chunk_attn_gpu import attend

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("layout,e4m3", [("NHD", False), ("HND", True)])
def test_pages_far_out(cuda_lib, layout, e4m3):
    sv, g = cuda_lib, torch.Generator().manual_seed(1)
    page, Hq, Hkv, D, nq, n = 16, 8, 2, 128, 45, 150
    pages = (1 << 32) // (page * Hkv * D) + 40           # past 2^32 elements
    typ = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    shape = (pages, page, Hkv, D) if layout == "NHD" else (pages, Hkv, page, D)
    k, v = (torch.empty(shape, dtype=typ, device=DEV) for _ in range(2))
    cache = sv.PagedKV(k, v, layout=layout)
    width = -(-n // page)
    table = (pages - 1 - 3 * torch.arange(width)).int()   # the last pages; every third
    table[0] = 0
    at = torch.arange(n)
    slots = table[at // page].long() * page + at % page
    kn, vn = (torch.randn(n, Hkv, D, generator=g).bfloat16() for _ in range(2))
    sv.paged_kv_append(kn.to(DEV), vn.to(DEV), cache, slots.to(DEV))
    q = torch.randn(nq, Hq, D, generator=g).bfloat16()
    o = torch.full((nq, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = sv.workspace(sv.paged_chunk_attn_workspace_bytes(1, nq, Hq, Hkv, D))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    sv.paged_chunk_attn(q.to(DEV), cache, table[None].to(DEV), ints(n), o, ints(0, nq), D ** -0.5, workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_OK
    K, V = ((x.to(typ) if e4m3 else x).double() for x in (kn, vn))
    want = attend(q, K, V, n - nq, D ** -0.5, 0, 0)
    assert float((o.double().cpu() - want).abs().max()) <= plain.attention_tolerance(float(V.abs().max()))


def test_rows_far_apart(cuda_lib):
    """Query and output rows 2^27 elements apart; the cache is small."""
    sv, g = cuda_lib, torch.Generator().manual_seed(2)
    T, Hq, Hkv, D, step = 37, 4, 2, 128, 1 << 27          # the last row 4.8 * 10^9 elements out
    flat = torch.empty((T - 1) * step + 2 * Hq * D, dtype=torch.bfloat16, device=DEV)
    rows = flat.as_strided((T, 2 * Hq, D), (step, D, 1))
    q = torch.randn(T, Hq, D, generator=g).bfloat16()
    rows[:, :Hq].copy_(q)
    k, v = (torch.randn(3, 16, Hkv, D, generator=g).bfloat16() for _ in range(2))
    cache = sv.PagedKV(k.to(DEV), v.to(DEV))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    sv.paged_chunk_attn(rows[:, :Hq], cache, ints(0, 1, 2)[None], ints(48), rows[:, Hq:], ints(0, T), D ** -0.5,
                        workspace=sv.workspace(sv.paged_chunk_attn_workspace_bytes(1, T, Hq, Hkv, D)))
    assert sv.sv_last_device_error() == sv.SV_OK
    want = attend(q, k.double().view(48, Hkv, D), v.double().view(48, Hkv, D), 48 - T, D ** -0.5, 0, 0)
    got = rows[:, Hq:].double().cpu()
    assert float((got - want).abs().max()) <= plain.attention_tolerance(float(v.float().abs().max()))


def test_states_and_rows_far_out(cuda_lib):
    """States past 2^32 elements, values and outputs too: steps, then a chunk."""
    sv = cuda_lib
    Hk, Hv, dk, dv, n, step = 1, 2, 128, 64, 35, 1 << 27
    slots = 5
    pool = torch.empty((slots - 1) * (1 << 30) + Hv * dv * dk, device=DEV)   # 17 GB
    states = pool.as_strided((slots, Hv, dv, dk), (1 << 30, dv * dk, dk, 1))
    states[4].zero_(), states[0].zero_()
    flat = torch.empty((n - 1) * step + 2 * Hv * dv, dtype=torch.bfloat16, device=DEV)
    rows = flat.as_strided((n, 2 * Hv, dv), (step, dv, 1))
    r = gdn_plain.rows(n, Hk, Hv, dk, dv, 9)
    q, k, v, g, beta = gdn_plain.on(r)
    rows[:, :Hv].copy_(v)
    v, o = rows[:, :Hv], rows[:, Hv:]
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    # three tokens by the step, the rest by a chunk, in the last state
    sv.gdn_step(states, ints(4), q[:3], k[:3], v[:3], g[:3], beta[:3], o[:3], 3, commit=True)
    m = n - 3
    sv.gdn_chunk(states, ints(4), q[3:], k[3:], v[3:], g[3:], beta[3:], o[3:], ints(0, m),
                 workspace=sv.workspace(sv.gdn_chunk_workspace_bytes(1, m, Hk, Hv, dk, dv)))
    assert sv.sv_last_device_error() == sv.SV_OK
    S, want = gdn_plain.run(torch.zeros(Hv, dv, dk), r, 0, n)
    gdn_plain.close(o, want, 2.0 ** -8, 2.0 ** -8, "o")
    gdn_plain.close(states[4], S, 2.0 ** -14, 0.0, "state")
    assert not states[0].any()
