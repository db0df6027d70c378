"""Rows and pages more than 2^32 elements from their tensor's first (GPU): no
offset is 32-bit.  Buffers of 9 to 18 GB, of which little is touched."""
import pytest
import torch

import paged_plain as plain
from test_paged_gpu import assert_rounded

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("layout,e4m3", [("NHD", False), ("HND", True)])
def test_pages_far_out(cuda_lib, layout, e4m3):
    sv, g = cuda_lib, torch.Generator().manual_seed(1)
    page, Hq, Hkv, D, M, n = 16, 8, 2, 128, 2, 150
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
    q = torch.randn(M, Hq, D, generator=g).bfloat16()
    o = torch.full((M, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = sv.workspace(sv.paged_attn_workspace_bytes(1, M, Hq, Hkv, D))
    sv.paged_attn(q.to(DEV), cache, table[None].to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV), o, M,
                  D ** -0.5, workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_OK
    K, V = ((x.to(typ) if e4m3 else x).double() for x in (kn, vn))
    want = plain.attend(q, K, V, n - M, D ** -0.5, 0, 0)
    assert float((o.double().cpu() - want).abs().max()) <= plain.attention_tolerance(float(V.abs().max()))


def test_rows_far_apart(cuda_lib):
    sv, g = cuda_lib, torch.Generator().manual_seed(2)
    T, Hq, Hkv, D, step = 37, 4, 2, 128, 1 << 27          # the last row 4.8 * 10^9 elements out
    flat = torch.empty((T - 1) * step + (Hq + Hkv) * D, dtype=torch.bfloat16, device=DEV)
    rows = flat.as_strided((T, Hq + Hkv, D), (step, D, 1))
    x = torch.randn(T, Hq + Hkv, D, generator=g).bfloat16()
    rows.copy_(x)
    pos = torch.randint(0, 9000, (T,), generator=g, dtype=torch.int32)
    f = plain.inv_freq(D)
    sv.qk_norm_rope(rows[:, :Hq], rows[:, Hq:], rows[:, :Hq], rows[:, Hq:], pos.to(DEV), sv.rope_phases(f))
    assert sv.sv_last_device_error() == sv.SV_OK
    assert_rounded(rows, plain.norm_rope(x, None, 0, 0, pos, f, False))


def test_heads_far_apart(cuda_lib):
    """Keys and values head-major in a long buffer, as a cache of one sequence has them."""
    sv, g = cuda_lib, torch.Generator().manual_seed(3)
    n, Hq, Hkv, D, step = 200, 6, 3, 128, (1 << 31) + 1024
    flat = torch.empty(2 * step + 2 * n * D, dtype=torch.bfloat16, device=DEV)
    k, v = (flat[i * n * D:].as_strided((n, Hkv, D), (D, step, 1)) for i in range(2))
    kn, vn = (torch.randn(n, Hkv, D, generator=g).bfloat16() for _ in range(2))
    k.copy_(kn)
    v.copy_(vn)
    q = torch.randn(n, Hq, D, generator=g).bfloat16()
    out = torch.empty(5 * step + n * D, dtype=torch.bfloat16, device=DEV).as_strided((n, Hq, D), (D, step, 1))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    sv.window_attn(q.to(DEV), k, v, out, cu, cu, D ** -0.5, window=70, sinks=3)
    assert sv.sv_last_device_error() == sv.SV_OK
    want = plain.attend(q, kn, vn, 0, D ** -0.5, 70, 3)
    err = float((out.double().cpu() - want).abs().max())
    assert err <= plain.attention_tolerance(float(vn.float().abs().max()))
