"""The paged-cache operators against their plain 64-bit forms (GPU)."""
import math

import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bf16(*shape, g, gain=1.0):
    return (torch.randn(*shape, generator=g) * gain).bfloat16()


def assert_rounded(got, want, dtype=torch.bfloat16, slack=2.0 ** -18, what=""):
    """got = want rounded once: half a step relative, plus fp32 arithmetic of
    the row (slack times the largest value)."""
    got, want = got.double().cpu(), want.double()
    assert torch.isfinite(got).all(), what
    tol = want.abs() * plain.half_step(dtype) + want.abs().max().clamp(min=1e-30) * slack
    bad = (got - want).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((got - want).abs() / tol).max()))


# ------------------------------------------------------- norm and rotation ----
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,far", [
    (1, 1, 1, 64, 64, False, 10), (1, 24, 4, 256, 64, False, 40000), (3, 5, 1, 128, 128, True, 131072),
    (7, 8, 2, 128, 64, False, 1 << 30), (2, 3, 2, 256, 256, True, 2000000000), (33, 2, 2, 64, 8, False, 5000),
    (5, 4, 4, 128, 24, True, 5000), (9, 7, 3, 256, 40, False, 77), (700, 32, 8, 128, 128, False, 131072),
    (613, 24, 4, 256, 64, True, 9000)])
def test_qk_norm_rope(cuda_lib, T, Hq, Hkv, D, rot, inter, far):
    sv, g = cuda_lib, gen(T + D + rot)
    qkv = bf16(T, Hq + 2 * Hkv, D, g=g, gain=3.0)
    qw, kw = bf16(D, g=g, gain=0.3), bf16(D, g=g, gain=0.3)
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32)
    pos[0] = far - 1
    f = plain.inv_freq(rot)
    ph = sv.rope_phases(f)
    d = qkv.to(DEV)
    q, k = d[:, :Hq], d[:, Hq:Hq + Hkv]   # views of one projection
    for weights, off in (((qw, kw), 1.0), ((None, kw), 0.0), ((None, None), 0.0)):
        qo = torch.full((T, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
        ko = torch.full((Hkv, T, D), NAN, dtype=torch.bfloat16, device=DEV).transpose(0, 1)  # head-major
        sv.qk_norm_rope(q, k, qo, ko, pos.to(DEV), ph, q_weight=None if weights[0] is None else weights[0].to(DEV),
                        k_weight=None if weights[1] is None else weights[1].to(DEV), eps=1e-5, weight_offset=off,
                        interleaved=inter)
        assert sv.sv_last_device_error() == sv.SV_OK
        assert_rounded(qo, plain.norm_rope(qkv[:, :Hq], weights[0], 1e-5, off, pos, f, inter), what="q")
        assert_rounded(ko, plain.norm_rope(qkv[:, Hq:Hq + Hkv], weights[1], 1e-5, off, pos, f, inter), what="k")


def test_norm_without_rotation_in_place_and_negative_positions(cuda_lib):
    sv, g = cuda_lib, gen(3)
    q, k, w = bf16(6, 4, 128, g=g), bf16(6, 2, 128, g=g), bf16(128, g=g)
    dq, dk = q.to(DEV), k.to(DEV)
    sv.qk_norm_rope(dq, dk, dq, dk, q_weight=w.to(DEV), k_weight=w.to(DEV), eps=0.0)
    assert_rounded(dq, plain.norm_rope(q, w, 0.0, 0.0, None, None, False))
    pos = torch.tensor([-1, -7, 0, 1, -100000, 5], dtype=torch.int32)
    f = plain.inv_freq(128)
    dq, dk = q.to(DEV), k.to(DEV)
    sv.qk_norm_rope(dq, dk, dq, dk, pos.to(DEV), sv.rope_phases(f))
    assert_rounded(dq, plain.norm_rope(q, None, 0, 0, pos, f, False))
    assert_rounded(dk, plain.norm_rope(k, None, 0, 0, pos, f, False))


def test_zero_rows_and_no_tokens(cuda_lib):
    sv = cuda_lib
    z = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    o = torch.full_like(z, 5.0)
    sv.qk_norm_rope(z, z, o, o.clone(), q_weight=w, k_weight=w)      # 0 / sqrt(eps)
    assert (o == 0).all()
    e = z[:0]
    sv.qk_norm_rope(e, e, e, e, q_weight=w, k_weight=w)
    assert sv.sv_last_device_error() == sv.SV_OK


def test_keys_straight_into_a_verify_cache(cuda_lib):
    """k_out with a head-major cache's strides is what verify_attn reads."""
    sv, g = cuda_lib, gen(5)
    T, Hkv, D, cap = 5, 2, 128, 40
    k = bf16(T, Hkv, D, g=g)
    cache = torch.zeros(Hkv, cap, D, dtype=torch.bfloat16, device=DEV)
    out = cache[:, 10:10 + T].transpose(0, 1)
    pos = torch.arange(10, 10 + T, dtype=torch.int32)
    f = plain.inv_freq(128)
    sv.qk_norm_rope(k.to(DEV), k.to(DEV), torch.empty_like(k, device=DEV), out, pos.to(DEV), sv.rope_phases(f))
    want = plain.norm_rope(k, None, 0, 0, pos, f, False).transpose(0, 1)
    assert_rounded(cache[:, 10:10 + T], want)
    assert (cache[:, :10] == 0).all() and (cache[:, 10 + T:] == 0).all()


# ------------------------------------------------------------------ append ----
def make_cache(sv, pages, page, Hkv, D, layout, e4m3, fill=0.0, scales=None, pad=0):
    """A cache whose rows are `pad` elements apart from being contiguous."""
    shape = (pages, page, Hkv, D + pad) if layout == "NHD" else (pages, Hkv, page, D + pad)
    t = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k = torch.full(shape, fill, device=DEV).to(t)[..., :D]
    v = torch.full(shape, fill, device=DEV).to(t)[..., :D]
    ks, vs = (None, None) if scales is None else (s.to(DEV) for s in scales)
    return sv.PagedKV(k, v, layout=layout, k_scale=ks, v_scale=vs)


def slot_rows(cache_tensor, layout, slots, page):
    view = cache_tensor if layout == "NHD" else cache_tensor.transpose(1, 2)
    x = view.float().cpu()
    return x[slots // page, slots % page]


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page,pad,with_q", [
    (1, 6, 1, 128, 128, 16, 0, True), (61, 8, 2, 128, 64, 16, 16, True), (40, 6, 1, 256, 64, 48, 0, False),
    (5, 2, 2, 64, 64, 32, 32, True), (900, 16, 4, 128, 128, 64, 0, False)])
def test_append_bf16(cuda_lib, layout, T, Hq, Hkv, D, rot, page, pad, with_q):
    sv, g = cuda_lib, gen(T + D)
    pages = -(-T // page) + 3
    q, k, v = bf16(T, Hq, D, g=g), bf16(T, Hkv, D, g=g, gain=2.0), bf16(T, Hkv, D, g=g)
    qw, kw = bf16(D, g=g), bf16(D, g=g)
    pos = torch.randint(0, 100000, (T,), generator=g, dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g)[:T]
    skipped = torch.zeros(T, dtype=torch.bool)
    if T > 4:
        skipped[3] = True
    given = torch.where(skipped, torch.tensor(-1), slots)
    cache = make_cache(sv, pages, page, Hkv, D, layout, False, fill=7.0, pad=pad)
    f = plain.inv_freq(rot)
    qo = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    extra = dict(q=q.to(DEV), q_out=qo, q_weight=qw.to(DEV)) if with_q else {}
    sv.paged_kv_append(k.to(DEV), v.to(DEV), cache, given.to(DEV), positions=pos.to(DEV), phases=sv.rope_phases(f),
                       k_weight=kw.to(DEV), eps=1e-6, **extra)
    assert sv.sv_last_device_error() == sv.SV_OK
    wk = plain.norm_rope(k, kw, 1e-6, 0.0, pos, f, False)
    assert_rounded(slot_rows(cache.k, layout, slots, page)[~skipped], wk[~skipped], what="k")
    assert torch.equal(slot_rows(cache.v, layout, slots, page)[~skipped], v.float()[~skipped])
    if with_q:
        assert_rounded(qo, plain.norm_rope(q, qw, 1e-6, 0.0, pos, f, False), what="q")
    # everything else keeps what it held
    other = torch.ones(pages * page, dtype=torch.bool)
    other[slots[~skipped]] = False
    rest = torch.arange(pages * page)[other]
    for c in (cache.k, cache.v):
        assert (slot_rows(c, layout, rest, page) == 7.0).all()


@pytest.mark.parametrize("layout,D,page,T", [("NHD", 128, 16, 5), ("HND", 256, 64, 130), ("HND", 128, 32, 1)])
def test_append_e4m3(cuda_lib, layout, D, page, T):
    """Every stored value is one of the two e4m3 neighbours of value / scale,
    the nearer one unless fp32 arithmetic decides (2^-18 of the row's largest)."""
    sv, g = cuda_lib, gen(T + D)
    Hkv, pages = 3, -(-T // page) + 1
    k, v = bf16(T, Hkv, D, g=g, gain=2.0), bf16(T, Hkv, D, g=g, gain=30.0)
    ks, vs = torch.rand(Hkv, generator=g) + 0.01, torch.rand(Hkv, generator=g) * 0.1 + 0.01
    v[0, 0, :4] = torch.tensor([1e30, -1e30, 0.0, 1e-30]).bfloat16()   # saturates; underflows to zero
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g)[:T]
    cache = make_cache(sv, pages, page, Hkv, D, layout, True, scales=(ks, vs))
    f = plain.inv_freq(D)
    sv.paged_kv_append(k.to(DEV), v.to(DEV), cache, slots.to(DEV), positions=pos.to(DEV), phases=sv.rope_phases(f))
    assert sv.sv_last_device_error() == sv.SV_OK
    for c, x, s in ((cache.k, plain.norm_rope(k, None, 0, 0, pos, f, False), ks), (cache.v, v.double(), vs)):
        want = (x / s.double()[None, :, None]).clamp(-448, 448)
        got = slot_rows(c, layout, slots, page).double()
        # half a step: 2^-4 of the value, or 2^-10 among the subnormals (steps of 2^-9)
        tol = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
        tol = tol + want.abs().amax(-1, keepdim=True) * 2.0 ** -18
        assert ((got - want).abs() <= tol).all()
    assert slot_rows(cache.v, layout, slots, page)[0, 0, :4].tolist() == [448.0, -448.0, 0.0, 0.0]


def test_append_slot_out_of_range_is_reported_and_not_written(cuda_lib):
    sv, g = cuda_lib, gen(9)
    cache = make_cache(sv, 2, 16, 1, 128, "NHD", False, fill=3.0)
    k = bf16(3, 1, 128, g=g).to(DEV)
    sv.paged_kv_append(k, k, cache, torch.tensor([32, 5, 1 << 40], device=DEV))
    assert sv.sv_last_device_error() == sv.SV_ERR_INVALID_ARG
    assert sv.sv_last_device_error() == sv.SV_OK
    flat = cache.k.view(32, 128)
    assert torch.equal(flat[5], k[1, 0]) and (flat[:5] == 3).all() and (flat[6:] == 3).all()


# --------------------------------------------------------- paged attention ----
def paged_case(sv, lens, M, Hq, Hkv, D, page, layout, e4m3, window, sinks, seed, poison=True, q_pad=0, gain=1.0):
    """Random pages; slots that no row sees, and unused pages, hold NaN.
    Returns (output, plain output, largest |v|)."""
    g = gen(seed)
    B = len(lens)
    width = max(1, max(-(-n // page) for n in lens))
    table = torch.full((B, width), -1, dtype=torch.int32)
    used = 0
    seen_pos = []
    for b, n in enumerate(lens):
        lo = max(0, n - M - window + 1) if window else 0
        seen = [j for j in range(n) if j >= lo or j < sinks]
        seen_pos.append(seen)
        for pg in sorted({j // page for j in seen}):
            table[b, pg] = used
            used += 1
    pages = used + 2
    order = torch.randperm(pages, generator=g).int()
    table = torch.where(table >= 0, order[table.clamp(min=0).long()], table)
    t = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    shape = (pages, page, Hkv, D) if layout == "NHD" else (pages, Hkv, page, D)
    k = torch.full(shape, NAN if poison else 0.0)
    v = torch.full(shape, NAN if poison else 0.0)
    for b, seen in enumerate(seen_pos):
        for j in seen:
            at = (int(table[b, j // page]), j % page)
            at = at if layout == "NHD" else (at[0], slice(None), at[1])
            k[at], v[at] = torch.randn(Hkv, D, generator=g) * gain, torch.randn(Hkv, D, generator=g)
    k, v = k.to(t), v.to(t)
    ks = vs = None
    if e4m3:
        ks, vs = torch.rand(Hkv, generator=g) + 0.5, torch.rand(Hkv, generator=g) + 0.5
    q = bf16(B * M, Hq, D + q_pad, g=g)[..., :D]
    scale = D ** -0.5
    cache = sv.PagedKV(k.to(DEV), v.to(DEV), layout=layout, k_scale=None if ks is None else ks.to(DEV),
                       v_scale=None if vs is None else vs.to(DEV))
    o = torch.full((B * M, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    dq = torch.empty(B * M, Hq, D + q_pad, dtype=torch.bfloat16, device=DEV)[..., :D]
    dq.copy_(q)
    ws = sv.workspace(sv.paged_attn_workspace_bytes(B, M, Hq, Hkv, D))
    ws.fill_(255)  # nothing in it needs a value beforehand
    sv.paged_attn(dq, cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), o, M, scale,
                  window=window, sinks=sinks, workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_OK
    want = torch.zeros(B * M, Hq, D, dtype=torch.float64)
    big = 0.0
    for b, n in enumerate(lens):
        K = torch.nan_to_num(plain.gather(k.float(), table[b], n, page, layout, ks))
        V = torch.nan_to_num(plain.gather(v.float(), table[b], n, page, layout, vs))
        want[b * M:(b + 1) * M] = plain.attend(q[b * M:(b + 1) * M], K, V, n - M, scale, window, sinks)
        if n:
            big = max(big, float(V.abs().max()))
    return o.double().cpu(), want, big


def check_paged(*a, **kw):
    got, want, big = paged_case(*a, **kw)
    assert torch.isfinite(got).all()
    err = float((got - want).abs().max())
    assert err <= plain.attention_tolerance(big), (err, plain.attention_tolerance(big))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (256, 6, 1), (128, 3, 3)])
@pytest.mark.parametrize("lens", [[1], [16], [17], [0, 5, 1, 33, 0], [300, 2, 129]])
def test_paged_single_token(cuda_lib, D, Hq, Hkv, lens, e4m3):
    check_paged(cuda_lib, lens, 1, Hq, Hkv, D, 16, "NHD", e4m3, 0, 0, seed=sum(lens) + D)


@pytest.mark.parametrize("layout,page", [("NHD", 16), ("HND", 64), ("NHD", 48), ("HND", 128)])
@pytest.mark.parametrize("M,Hq,Hkv,D,e4m3", [
    (2, 8, 2, 128, False), (4, 12, 2, 256, False), (4, 12, 2, 256, True), (5, 8, 1, 128, True),
    (8, 6, 1, 256, False), (16, 16, 2, 128, False), (16, 8, 1, 128, True)])
def test_paged_verify_rows(cuda_lib, layout, page, M, Hq, Hkv, D, e4m3):
    # 8 to 128 query rows per KV head: one to eight tiles
    check_paged(cuda_lib, [200, 77, M, 3, 500], M, Hq, Hkv, D, page, layout, e4m3, 0, 0, seed=M + page)


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (20, 4), (100, 1), (64, 40), (5000, 3)])
@pytest.mark.parametrize("M,Hq,Hkv,D,page,e4m3", [
    (1, 4, 4, 128, 32, False), (4, 6, 1, 256, 16, False), (3, 8, 2, 128, 16, True)])
def test_paged_window_and_sinks(cuda_lib, window, sinks, M, Hq, Hkv, D, page, e4m3):
    check_paged(cuda_lib, [400, 90, 17, 2, 0, 333], M, Hq, Hkv, D, page, "HND", e4m3, window, sinks,
                seed=window + sinks)


def test_paged_sharp_scores_and_strided_queries(cuda_lib):
    """Scores of a few tens: the running maximum moves and single slots win."""
    check_paged(cuda_lib, [700, 64], 2, 8, 2, 128, 16, "NHD", False, 0, 0, seed=4, gain=12.0, q_pad=24)
    check_paged(cuda_lib, [700, 64], 2, 12, 2, 256, 32, "HND", True, 0, 0, seed=5, gain=6.0, q_pad=8)


def test_paged_many_heads_split_at_any_place(cuda_lib):
    """More heads than CTAs (joined by CTA) and one long head among short ones."""
    check_paged(cuda_lib, [40 + 7 * i for i in range(50)], 1, 8, 8, 128, 16, "NHD", False, 0, 0, seed=6)
    check_paged(cuda_lib, [3000] + [5] * 40, 1, 8, 8, 128, 16, "NHD", False, 0, 0, seed=7)


def test_paged_long_sequence_matches_its_halves(cuda_lib):
    """20000 slots over all CTAs against torch in 64 bits on the GPU."""
    sv, g = cuda_lib, torch.Generator(device=DEV).manual_seed(1)
    M, Hq, Hkv, D, page, n = 4, 24, 4, 256, 64, 20011
    pages = -(-n // page)
    k = torch.randn(pages, Hkv, page, D, generator=g, device=DEV).bfloat16()
    v = torch.randn(pages, Hkv, page, D, generator=g, device=DEV).bfloat16()
    table = torch.randperm(pages, generator=g, device=DEV).int()[None]
    q = torch.randn(M, Hq, D, generator=g, device=DEV).bfloat16()
    o = torch.empty_like(q)
    ws = sv.workspace(sv.paged_attn_workspace_bytes(1, M, Hq, Hkv, D))
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    sv.paged_attn(q, sv.PagedKV(k, v, layout="HND"), table, lens, o, M, D ** -0.5, workspace=ws)
    assert sv.sv_last_device_error() == sv.SV_OK
    K = k[table[0].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].double()
    V = v[table[0].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].double()
    for i in range(M):
        x = torch.einsum("hgd,hnd->hgn", q[i].double().view(Hkv, -1, D), K[:, :n - M + i + 1]) * D ** -0.5
        want = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), V[:, :n - M + i + 1]).view(Hq, D)
        err = float((o[i].double() - want).abs().max())
        # outputs here are averages over thousands of slots, well below |v|
        assert err <= plain.half_step(torch.bfloat16) * float(want.abs().max()) * 2 + 2.0 ** -9 * float(V.abs().max()) / math.sqrt(n)


def test_paged_bad_lengths_and_pages_are_reported(cuda_lib):
    sv, g = cuda_lib, gen(11)
    page, Hkv, D = 16, 1, 128
    k = bf16(4, page, Hkv, D, g=g).to(DEV)
    cache = sv.PagedKV(k, k.clone(), layout="NHD")
    q = bf16(2, 2, D, g=g).to(DEV)
    o = torch.full_like(q, NAN)
    ws = sv.workspace(sv.paged_attn_workspace_bytes(2, 1, 2, Hkv, D))

    def call(table, lens):
        sv.paged_attn(q, cache, torch.tensor(table, dtype=torch.int32, device=DEV),
                      torch.tensor(lens, dtype=torch.int32, device=DEV), o, 1, 0.1, workspace=ws)
        return sv.sv_last_device_error()

    assert call([[0, 1], [2, 3]], [33, 20]) == sv.SV_ERR_INVALID_ARG   # past the table
    assert call([[0, 1], [2, 3]], [-5, 20]) == sv.SV_ERR_INVALID_ARG
    assert torch.isfinite(o).all() and (o[0] == 0).all()
    assert call([[0, 9], [2, 3]], [20, 20]) == sv.SV_ERR_INVALID_ARG   # past the cache
    assert call([[0, -1], [2, 3]], [20, 20]) == sv.SV_ERR_INVALID_ARG
    assert torch.isfinite(o).all()
    assert call([[0, 99], [2, -7]], [16, 16]) == sv.SV_OK              # not needed, not read
    with pytest.raises(sv.SvError) as e:
        sv.paged_attn(q, cache, torch.zeros(2, 2, dtype=torch.int32, device=DEV),
                      torch.zeros(2, dtype=torch.int32, device=DEV), o, 1, 0.1, workspace=ws[:64])
    assert e.value.status == sv.SV_ERR_WORKSPACE


def test_paged_graph_follows_lengths_and_side_streams(cuda_lib):
    """A captured append + attention is replayed with other lengths, slots and
    contents, on another stream than the one it was made on."""
    sv, g = cuda_lib, gen(12)
    B, Hq, Hkv, D, page, width = 3, 4, 2, 128, 16, 8
    k = torch.zeros(B * width, page, Hkv, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    cache = sv.PagedKV(k, v)
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    slots = torch.zeros(B, dtype=torch.int64, device=DEV)
    new = torch.zeros(B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    o = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    ws = sv.workspace(sv.paged_attn_workspace_bytes(B, 1, Hq, Hkv, D))

    def step():
        sv.paged_kv_append(new[:, Hq:Hq + Hkv], new[:, Hq + Hkv:], cache, slots)
        sv.paged_attn(new[:, :Hq], cache, table, lens, o, 1, 0.09, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    K, V = [[] for _ in range(B)], [[] for _ in range(B)]
    k.zero_()
    v.zero_()
    for t in range(20):
        x = bf16(B, Hq + 2 * Hkv, D, g=g)
        at = torch.tensor([t, t, t])
        new.copy_(x)
        lens.copy_((at + 1).int())
        slots.copy_(torch.arange(B) * width * page + at)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        for b in range(B):
            K[b].append(x[b, Hq:Hq + Hkv])
            V[b].append(x[b, Hq + Hkv:])
            want = plain.attend(x[b:b + 1, :Hq], torch.stack(K[b]), torch.stack(V[b]), t, 0.09, 0, 0)
            err = float((o[b:b + 1].double().cpu() - want).abs().max())
            assert err <= plain.attention_tolerance(float(torch.stack(V[b]).abs().max())), (t, b, err)
    assert sv.sv_last_device_error() == sv.SV_OK


def test_paged_results_do_not_change_from_call_to_call(cuda_lib):
    sv = cuda_lib
    a = paged_case(sv, [900, 31, 400], 2, 8, 2, 128, 16, "NHD", False, 0, 0, seed=21)[0]
    b = paged_case(sv, [900, 31, 400], 2, 8, 2, 128, 16, "NHD", False, 0, 0, seed=21)[0]
    assert torch.equal(a, b)
