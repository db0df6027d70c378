"""Shapes of the paged-cache calls where their rules change (GPU): more than 64
rows a KV head at D = 256 (eight tiles, four ring slots), e4m3 with more than 32
(pairs of chunks for four and eight tiles), even cuts over 33 to 64 sequences,
more sequences than one step of the scan takes; steps over e4m3 pages against
what the pages hold; the same outputs from call to call."""
import pytest
import torch

import paged_plain as plain
from test_paged_gpu import assert_rounded, check_paged, make_cache, slot_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("M,Hq,Hkv,D,e4m3", [
    (16, 10, 2, 256, False), (8, 16, 1, 256, False), (13, 5, 1, 256, False),    # 80, 128, 65 rows
    (8, 12, 2, 256, True), (11, 3, 1, 256, True), (16, 8, 1, 256, True), (9, 16, 2, 256, True)])  # 48, 33, 128, 72
def test_many_rows_at_256(cuda_lib, M, Hq, Hkv, D, e4m3):
    check_paged(cuda_lib, [200, M - 1, 517, 64], M, Hq, Hkv, D, 32, "HND", e4m3, 0, 0, seed=M + Hq)
    check_paged(cuda_lib, [300, 40], M, Hq, Hkv, D, 16, "NHD", e4m3, 50, 3, seed=M + Hq + 1)


@pytest.mark.parametrize("B,Hkv,window", [(33, 4, 0), (40, 2, 0), (64, 2, 0), (64, 1, 0), (64, 1, 90), (65, 1, 0)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_few_heads_of_many_sequences(cuda_lib, B, Hkv, window, e4m3):
    lens = [(97 * i) % 700 for i in range(B)]   # one of them empty
    check_paged(cuda_lib, lens, 1, 4 * Hkv, Hkv, 128, 16, "NHD", e4m3, window, 2 if window else 0, seed=B)


@pytest.mark.parametrize("B,Hkv,window", [(385, 1, 0), (400, 2, 0), (900, 1, 17)])
def test_more_sequences_than_a_step_of_the_scan(cuda_lib, B, Hkv, window):
    check_paged(cuda_lib, [(7 * i) % 61 for i in range(B)], 1, 2 * Hkv, Hkv, 128, 16, "HND", False, window, 0, seed=B)


def test_e4m3_steps_against_what_the_pages_hold(cuda_lib):
    """Prompts, then verify steps; the pages against the plain rows (half a step
    of e4m3), the outputs against the plain attention over the pages' contents."""
    sv, g = cuda_lib, torch.Generator().manual_seed(3)
    Hq, Hkv, D, M, page, layout, rot, eps = 12, 2, 256, 4, 16, "HND", 64, 1e-6
    lens, B, width = [5, 130, 63], 3, 10
    ks, vs = torch.tensor([0.02, 0.05]), torch.tensor([0.01, 0.03])
    cache = make_cache(sv, B * width, page, Hkv, D, layout, True, scales=(ks, vs))
    table = torch.randperm(B * width, generator=g).int().view(B, width)
    f = plain.inv_freq(rot)
    ph, qw, kw = sv.rope_phases(f), (torch.randn(D, generator=g) * 0.2).bfloat16(), (torch.randn(D, generator=g) * 0.2).bfloat16()
    norm = dict(q_weight=qw.to(DEV), k_weight=kw.to(DEV), eps=eps, weight_offset=1.0)

    def slots_of(b, at):
        return table[b, at // page].long() * page + at % page

    def rows(n):
        return torch.randn(n, Hq + 2 * Hkv, D, generator=g).bfloat16()

    def check_pages(slots, k, v, pos):
        for c, x, s in ((cache.k, plain.norm_rope(k, kw, eps, 1.0, pos, f, False), ks), (cache.v, v.double(), vs)):
            want = (x / s.double()[None, :, None]).clamp(-448, 448)
            tol = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
            got = slot_rows(c, layout, slots, page).double()
            assert ((got - want).abs() <= tol + want.abs().amax(-1, keepdim=True) * 2.0 ** -18).all()

    x = rows(sum(lens))
    d = x.to(DEV)
    pos = torch.cat([torch.arange(n) for n in lens])
    slots = torch.cat([slots_of(b, torch.arange(n)) for b, n in enumerate(lens)])
    sv.paged_kv_append(d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], cache, slots.to(DEV), positions=pos.int().to(DEV), phases=ph,
                       **{n: norm[n] for n in ("k_weight", "eps", "weight_offset")})
    check_pages(slots, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos)
    ws = sv.workspace(sv.paged_attn_workspace_bytes(B, M, Hq, Hkv, D))
    for step in range(3):
        x = rows(B * M)
        d = x.to(DEV)
        at = torch.tensor([[n + i for i in range(M)] for n in lens])
        pos, slots = at.flatten(), torch.cat([slots_of(b, at[b]) for b in range(B)])
        qo, o = (torch.empty(B * M, Hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        now = torch.tensor([n + M for n in lens], dtype=torch.int32)
        sv.paged_kv_append(d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], cache, slots.to(DEV), q=d[:, :Hq], q_out=qo,
                           positions=pos.int().to(DEV), phases=ph, **norm)
        sv.paged_attn(qo, cache, table.to(DEV), now.to(DEV), o, M, D ** -0.5, workspace=ws)
        assert sv.sv_last_device_error() == sv.SV_OK
        check_pages(slots, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos)
        assert_rounded(qo, plain.norm_rope(x[:, :Hq], qw, eps, 1.0, pos, f, False), what="q")
        for b in range(B):
            K = plain.gather(cache.k.float().cpu(), table[b], int(now[b]), page, layout, ks)
            V = plain.gather(cache.v.float().cpu(), table[b], int(now[b]), page, layout, vs)
            r = slice(b * M, (b + 1) * M)
            want = plain.attend(qo[r].cpu(), K, V, lens[b], D ** -0.5, 0, 0)
            err = float((o[r].double().cpu() - want).abs().max())
            assert err <= plain.attention_tolerance(float(V.abs().max())), (step, b, err)
        lens = [n + 1 + (b + step) % M for b, n in enumerate(lens)]


def test_results_are_the_same_from_call_to_call(cuda_lib):
    """Splits, joins and orders depend on the sizes only: two calls give the same bits."""
    sv, g = cuda_lib, torch.Generator(device=DEV).manual_seed(4)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    for D, Hq, Hkv, nq, window in ((128, 32, 8, [2000, 3, 411], 0), (128, 8, 2, [300, 7], 100), (256, 24, 4, [900, 130], 0)):
        n = sum(nq)
        q, k, v = rand(n, Hq, D).bfloat16(), rand(n, Hkv, D).bfloat16(), rand(n, Hkv, D).bfloat16()
        cu = torch.tensor([0] + nq, device=DEV).cumsum(0).int()
        out = [torch.zeros_like(q) for _ in range(4)]
        for o in out:
            sv.window_attn(q, k, v, o, cu, cu, D ** -0.5, window=window)
        assert all(torch.equal(out[0], o) for o in out[1:])
    for D, Hq, Hkv, M, lens, typ in ((128, 32, 8, 1, [9000, 40, 777], torch.bfloat16), (256, 24, 4, 4, [30000], torch.bfloat16),
                                     (256, 24, 4, 4, [5000, 20, 1300], torch.float8_e4m3fn)):
        width = -(-max(lens) // 64)
        k, v = (rand(len(lens) * width, Hkv, 64, D).to(typ) for _ in range(2))
        cache = sv.PagedKV(k, v, layout="HND")
        table = torch.randperm(len(lens) * width, generator=g, device=DEV).int().view(len(lens), width)
        q = rand(len(lens) * M, Hq, D).bfloat16()
        n = torch.tensor(lens, dtype=torch.int32, device=DEV)
        ws = sv.workspace(sv.paged_attn_workspace_bytes(len(lens), M, Hq, Hkv, D))
        out = [torch.zeros_like(q) for _ in range(4)]
        for o in out:
            sv.paged_attn(q, cache, table, n, o, M, D ** -0.5, workspace=ws)
        assert all(torch.equal(out[0], o) for o in out[1:])
    assert sv.sv_last_device_error() == sv.SV_OK
