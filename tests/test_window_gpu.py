"""window_attn against the plain 64-bit form (GPU)."""
import math

import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


def prompts(sv, nq, nk, Hq, Hkv, D, window, sinks, seed, gain=1.0, gap=0, fused=False):
    """Packed prompts; `gap` rows of NaN stand between the sequences and after them."""
    g = torch.Generator().manual_seed(seed)
    B = len(nq)
    cu_q, cu_k = [0], [gap]
    for a, b in zip(nq, nk):
        cu_q.append(cu_q[-1] + a)
        cu_k.append(cu_k[-1] + b)
    Tk = cu_k[-1] + gap
    q = torch.randn(cu_q[-1], Hq, D, generator=g).bfloat16()
    kv = torch.full((Tk, 2 * Hkv, D), NAN).bfloat16()
    kv[gap:cu_k[-1]] = (torch.randn(cu_k[-1] - gap, 2 * Hkv, D, generator=g) * gain).bfloat16()
    d = kv.to(DEV)
    k, v = d[:, :Hkv], d[:, Hkv:]
    if not fused:
        k, v = k.contiguous(), v.transpose(0, 1).contiguous().transpose(0, 1)  # head-major values
    dq = q.to(DEV)
    o = torch.full((cu_q[-1], Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    scale = D ** -0.5
    sv.window_attn(dq, k, v, o, torch.tensor(cu_q, dtype=torch.int32, device=DEV),
                   torch.tensor(cu_k, dtype=torch.int32, device=DEV), scale, window=window, sinks=sinks,
                   workspace=sv.workspace(sv.window_attn_workspace_bytes(B, Hq, Hkv, D)))
    assert sv.sv_last_device_error() == sv.SV_OK
    want = torch.zeros(cu_q[-1], Hq, D, dtype=torch.float64)
    for b in range(B):
        K, V = kv[cu_k[b]:cu_k[b + 1], :Hkv].double(), kv[cu_k[b]:cu_k[b + 1], Hkv:].double()
        n, N = nq[b], nk[b]
        if n == 0:
            continue
        p = torch.arange(n)[:, None] + N - n
        j = torch.arange(N)
        seen = (j <= p) & ((j > p - window) | (j < sinks)) if window else j <= p
        x = torch.einsum("ihgd,nhd->hgin", q[cu_q[b]:cu_q[b + 1]].double().view(n, Hkv, -1, D), K) * scale
        x = x.masked_fill(~seen, -math.inf)
        w = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
        want[cu_q[b]:cu_q[b + 1]] = torch.einsum("hgin,nhd->ihgd", w, V).reshape(n, Hq, D)
    big = float(torch.nan_to_num(kv[:, Hkv:].float()).abs().max())
    return o.double().cpu(), want, big


def check(*a, **kw):
    got, want, big = prompts(*a, **kw)
    assert torch.isfinite(got).all()
    err = float((got - want).abs().max()) if got.numel() else 0.0
    assert err <= plain.attention_tolerance(big), (err, plain.attention_tolerance(big))


HEADS = [(8, 2, 128), (6, 1, 256), (3, 3, 128), (2, 2, 256), (10, 2, 128), (32, 1, 256)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 128, 129, 200, 300])
def test_one_prompt(cuda_lib, Hq, Hkv, D, n):
    check(cuda_lib, [n], [n], Hq, Hkv, D, 0, 0, seed=n + D)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS[:4])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (50, 4), (128, 0), (100, 130), (64, 1), (5000, 7)])
def test_ragged_prompts_with_windows(cuda_lib, Hq, Hkv, D, window, sinks):
    nq = [1, 130, 0, 7, 257, 64]
    check(cuda_lib, nq, nq, Hq, Hkv, D, window, sinks, seed=window + sinks, gap=5)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS[:3])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 2)])
def test_more_keys_than_rows_and_fewer(cuda_lib, Hq, Hkv, D, window, sinks):
    """Rows after a past, and rows before the first key, which see nothing."""
    check(cuda_lib, [1, 40, 100, 5, 70], [400, 333, 60, 0, 1], Hq, Hkv, D, window, sinks, seed=3, gap=2, fused=True)


def test_sharp_scores(cuda_lib):
    """Scores of a few tens: the reference maximum rises along a row."""
    check(cuda_lib, [500], [500], 8, 2, 128, 0, 0, seed=1, gain=12.0)
    check(cuda_lib, [500], [500], 6, 1, 256, 0, 0, seed=2, gain=12.0)
    check(cuda_lib, [400], [400], 4, 4, 128, 70, 4, seed=3, gain=12.0)


def test_many_sequences(cuda_lib):
    """More sequences than the shared-memory ring keeps beside five slots, and
    more items than CTAs."""
    nq = [(7 * i) % 23 for i in range(400)]
    check(cuda_lib, nq, nq, 4, 2, 128, 0, 0, seed=4)
    check(cuda_lib, nq, nq, 2, 1, 256, 6, 1, seed=5)


@pytest.mark.parametrize("Hq,Hkv,D,n,window,sinks", [(32, 8, 128, 2500, 0, 0), (24, 4, 256, 2100, 0, 0),
                                                     (16, 16, 128, 3000, 700, 4)])
def test_long_prompt(cuda_lib, Hq, Hkv, D, n, window, sinks):
    """Several rounds of items per CTA, against 64 bits on the GPU."""
    sv, g = cuda_lib, torch.Generator(device=DEV).manual_seed(n)
    q = torch.randn(n, Hq, D, generator=g, device=DEV).bfloat16()
    kv = torch.randn(n, 2 * Hkv, D, generator=g, device=DEV).bfloat16()
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    o = torch.empty_like(q)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    sv.window_attn(q, k, v, o, cu, cu, D ** -0.5, window=window, sinks=sinks,
                   workspace=sv.workspace(sv.window_attn_workspace_bytes(1, Hq, Hkv, D)))
    assert sv.sv_last_device_error() == sv.SV_OK
    j = torch.arange(n, device=DEV)
    seen = j <= j[:, None]
    if window:
        seen &= (j > j[:, None] - window) | (j < sinks)
    for h in range(0, Hq, 5):
        x = (q[:, h].double() @ k[:, h * Hkv // Hq].double().T * D ** -0.5).masked_fill(~seen, -math.inf)
        want = torch.softmax(x, -1) @ v[:, h * Hkv // Hq].double()
        err = float((o[:, h].double() - want).abs().max())
        assert err <= plain.attention_tolerance(float(v.abs().max())), h


def test_bad_offsets_are_reported_and_left_out(cuda_lib):
    sv = cuda_lib
    q = torch.randn(40, 2, 128, device=DEV).bfloat16()
    k = torch.randn(40, 1, 128, device=DEV).bfloat16()
    for cu in ([0, 10, 50], [0, 20, 10], [-4, 10, 20]):
        o = torch.full_like(q, 9.0)
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        sv.window_attn(q, k, k, o, c, c, 0.1, workspace=None)
        assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
        assert torch.isfinite(o).all()
        assert (o[20:] == 9.0).all()     # rows of no good sequence keep their contents
    o = torch.full_like(q, 9.0)
    c = torch.tensor([5, 10, 20], dtype=torch.int32, device=DEV)
    sv.window_attn(q, k, k, o, c, c, 0.1, workspace=None)
    assert sv.sv_last_device_error() == sv.SV_OK
    assert (o[:5] == 9.0).all() and (o[20:] == 9.0).all() and not (o[5:20] == 9.0).any()


def test_strided_output_and_no_rows(cuda_lib):
    sv, g = cuda_lib, torch.Generator().manual_seed(2)
    n, Hq, Hkv, D = 70, 4, 2, 128
    q = torch.randn(n, Hq, D, generator=g).bfloat16()
    k, v = (torch.randn(n, Hkv, D, generator=g).bfloat16() for _ in range(2))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    plain_o = torch.empty(n, Hq, D, dtype=torch.bfloat16, device=DEV)
    wide = torch.full((n, Hq + 3, D + 8), 5.0, dtype=torch.bfloat16, device=DEV)
    for o in (plain_o, wide[:, 1:1 + Hq, :D]):
        sv.window_attn(q.to(DEV), k.to(DEV), v.to(DEV), o, cu, cu, 0.1)
    assert torch.equal(plain_o, wide[:, 1:1 + Hq, :D])
    assert (wide[:, 0] == 5).all() and (wide[:, 1 + Hq:] == 5).all() and (wide[:, :, D:] == 5).all()
    e = plain_o[:0]
    sv.window_attn(e, k.to(DEV), v.to(DEV), e, torch.zeros(2, dtype=torch.int32, device=DEV), cu, 0.1)
    none = k[:0].to(DEV)   # no keys at all: every row sees nothing
    sv.window_attn(q.to(DEV), none, none, plain_o, cu, torch.zeros(2, dtype=torch.int32, device=DEV), 0.1)
    assert sv.sv_last_device_error() == sv.SV_OK and (plain_o == 0).all()


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (6, 1, 256), (3, 3, 128), (2, 2, 256)])
@pytest.mark.parametrize("sinks", [1, 31, 32, 33, 64, 129])
@pytest.mark.parametrize("window", [1, 37, 128, 191])
def test_first_keys_beside_a_far_window(cuda_lib, Hq, Hkv, D, window, sinks):
    """First keys that share the window's first block (up to 32 of them), and that have blocks of their own."""
    check(cuda_lib, [150, 333, 20], [400, 333, 777], Hq, Hkv, D, window, sinks, seed=window + sinks, gap=3)


def test_first_keys_beside_a_far_window_sharp(cuda_lib):
    """The largest scores stand among the first keys, or far from them."""
    check(cuda_lib, [300, 90], [800, 90], 8, 2, 128, 61, 9, seed=5, gain=12.0)
    check(cuda_lib, [300, 90], [800, 90], 12, 2, 256, 61, 9, seed=6, gain=12.0)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 128), (32, 8, 128), (24, 4, 256), (128, 1, 128), (128, 1, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_items_longest_first(cuda_lib, Hq, Hkv, D, window, sinks):
    """Many sequences of very different lengths, pasts and too few keys among them; each row written once."""
    nq = [1, 700, 2, 0, 35, 333, 64, 1, 128, 129, 90, 1, 1, 5, 260, 17]
    nk = [1, 700, 500, 3, 20, 333, 65, 0, 128, 400, 90, 1, 7, 5, 900, 16]
    check(cuda_lib, nq, nk, Hq, Hkv, D, window, sinks, seed=7, gap=1)
