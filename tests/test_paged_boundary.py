"""The paged-cache entry points on the host: refusals before any launch, the
rotation's phase table, and the plain forms' own pins.  No GPU."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_plain as plain
from speculative_decoding_verify_08_gb300 import build_lib

A = 256  # an aligned stand-in address; never dereferenced


@pytest.fixture(scope="module")
def sv():
    build_lib.build()
    import speculative_decoding_verify_08_gb300 as sv
    sv.load()
    return sv


def rows(sv, ptr=A, ts=1024, hs=128):
    return sv._ROWS.pack(ptr, ts, hs)


def cache(sv, k=A, v=A, ks=0, vs=0, page=16 * 4 * 128, slot=4 * 128, head=128, pages=8, size=16, dtype=0):
    return sv._PAGED_KV.pack(k, v, ks, vs, page, slot, head, pages, size, dtype, 0)


def norm(sv, q=A, k=A, eps=1e-6, offset=0.0):
    return sv._NORM.pack(q, k, eps, offset)


def rotation(sv, phases=A, positions=A, dim=128, inter=0):
    return sv._ROTATION.pack(phases, positions, dim, inter)


def test_qk_norm_rope_refusals(sv):
    f = sv.load().qk_norm_rope
    r, n, t = rows(sv), norm(sv), rotation(sv)

    def call(q=r, k=r, qo=r, ko=r, norm=n, rot=t, T=4, Hq=8, Hkv=2, D=128):
        return f(q, k, qo, ko, norm, rot, T, Hq, Hkv, D, None)

    assert call(q=None) == 1 and call(ko=None) == 1
    assert call(q=rows(sv, ptr=0)) == 1
    assert call(q=rows(sv, ptr=A + 8)) == 1          # not 16-byte aligned
    assert call(k=rows(sv, ts=1028)) == 1            # stride not a multiple of 8
    assert call(k=rows(sv, hs=-128)) == 1
    assert call(k=rows(sv, ts=1 << 40)) == 1
    assert call(T=-1) == 1 and call(Hq=0) == 1 and call(Hkv=0) == 1
    assert call(D=96) == 2 and call(D=512) == 2
    assert call(Hq=5000) == 2
    assert call(T=0x7fffffff, Hq=2) == 2             # rows beyond 31 bits
    assert call(norm=norm(sv, eps=-1.0)) == 1
    assert call(norm=norm(sv, eps=float("nan"))) == 1
    assert call(norm=norm(sv, offset=float("inf"))) == 1
    assert call(norm=norm(sv, q=A + 2)) == 1
    assert call(rot=rotation(sv, positions=0)) == 1
    assert call(rot=rotation(sv, dim=136)) == 1      # beyond D
    assert call(rot=rotation(sv, dim=4)) == 1 and call(rot=rotation(sv, dim=20)) == 1
    assert call(T=0) == 0                            # nothing to do


def test_paged_kv_append_refusals(sv):
    f = sv.load().paged_kv_append
    r, n, t, c = rows(sv), norm(sv), rotation(sv), cache(sv)

    def call(q=None, qo=None, k=r, v=r, cache=c, slots=A, norm=n, rot=t, T=4, Hq=8, Hkv=4, D=128):
        return f(q, qo, k, v, cache, slots, norm, rot, T, Hq, Hkv, D, None)

    assert call(k=None) == 1 and call(v=None) == 1 and call(cache=None) == 1 and call(slots=None) == 1
    assert call(q=r) == 1                            # queries without a place for them
    assert call(slots=A + 4) == 1
    assert call(cache=cache(sv, k=0)) == 1 and call(cache=cache(sv, v=A + 8)) == 1
    assert call(cache=cache(sv, dtype=1)) == 1       # fp32 is no cache type
    assert call(cache=cache(sv, pages=0)) == 1 and call(cache=cache(sv, size=0)) == 1
    assert call(cache=cache(sv, slot=0)) == 1 and call(cache=cache(sv, head=-128)) == 1
    assert call(cache=cache(sv, head=132)) == 1
    assert call(cache=cache(sv, head=136, dtype=2)) == 1   # 8-bit rows start on 16 bytes too
    assert call(cache=cache(sv, ks=A)) == 1          # scales beside bf16
    assert call(cache=cache(sv, size=24)) == 2 and call(cache=cache(sv, size=1 << 17)) == 2
    assert call(cache=cache(sv, dtype=2), D=64) == 2
    assert call(D=32) == 2
    assert call(T=0) == 0


def test_paged_attn_refusals(sv):
    f = sv.load().paged_attn
    r, c = rows(sv), cache(sv)

    def call(q=r, cache=c, table=A, stride=8, width=8, lens=A, o=r, B=2, M=1, Hq=8, Hkv=4, D=128, scale=0.1,
             window=0, sinks=0, ws=None, wsb=0):
        return f(q, cache, table, stride, width, lens, o, B, M, Hq, Hkv, D, scale, window, sinks, ws, wsb, None)

    assert call(q=None) == 1 and call(o=None) == 1 and call(cache=None) == 1
    assert call(table=None) == 1 and call(lens=None) == 1 and call(table=A + 2) == 1
    assert call(M=0) == 1 and call(B=-1) == 1 and call(Hq=6) == 1
    assert call(scale=0.0) == 1 and call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(window=-1) == 1 and call(sinks=-1) == 1
    assert call(width=0) == 1 and call(stride=-1) == 1
    assert call(D=64) == 2 and call(M=65, Hq=8) == 2      # 130 rows per KV head
    assert call(B=5000) == 2
    assert call(width=1 << 27) == 2                       # 2^31 positions
    assert call(B=4096, width=1 << 20) == 2               # chunk line beyond 31 bits
    assert call(B=0) == 0
    if not torch.cuda.is_available():
        assert call() == 3                                # no device to plan for
    assert sv.paged_attn_workspace_bytes(2, 1, 6, 4, 128) == 0
    assert sv.paged_attn_workspace_bytes(2, 1, 8, 4, 64) == 0
    assert sv.paged_attn_workspace_bytes(2, 65, 8, 4, 128) == 0


def test_python_checks(sv):
    """Wrong types, shapes and devices raise before anything reaches the library."""
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(sv.SvError) as e:
        sv.qk_norm_rope(x, x, x, x)                       # CPU memory
    assert e.value.status == sv.SV_ERR_INVALID_ARG
    with pytest.raises(sv.SvError):
        sv.PagedKV(x[None], x[None])                      # CPU memory
    with pytest.raises(sv.SvError):
        sv.PagedKV(x[None], x[None], layout="DHN")


def test_rope_phases_are_the_turns(sv):
    """phase = inv_freq / (2 pi) mod 1 in 2^-64, to the 53 bits of a double."""
    f = [1.0, 0.5, 1e-4, 10000.0 ** -0.37, 7.0, 0.0, 2 * math.pi, 1e-12]
    out = np.empty(len(f), dtype=np.uint64)
    a = np.asarray(f, dtype=np.float64)
    assert sv.load().rope_phases(a.ctypes.data, len(f), out.ctypes.data) == 0
    two_pi = 2 * Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    for x, p in zip(f, out.tolist()):
        t = Fraction(x) / two_pi
        want = (t - (t.numerator // t.denominator)) * 2 ** 64
        # division and 2 pi as doubles: 2^-52 relative to the turns before the whole part is taken
        err = abs(Fraction(p) - want)
        err = min(err, 2 ** 64 - err)
        assert err <= 1 + t * 2 ** 64 * Fraction(1, 2 ** 52), x
    assert sv.load().rope_phases(None, 1, out.ctypes.data) == 1
    assert sv.load().rope_phases(a.ctypes.data, -1, out.ctypes.data) == 1
    bad = np.asarray([float("nan")])
    assert sv.load().rope_phases(bad.ctypes.data, 1, out.ctypes.data) == 1


def test_plain_rotation_keeps_lengths_and_relative_angles():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(2, 1, 64, generator=g, dtype=torch.float64)
    for inter in (False, True):
        f = plain.inv_freq(32)
        a = plain.norm_rope(x, None, 0, 0, torch.tensor([5, 9]), f, inter)
        b = plain.norm_rope(x, None, 0, 0, torch.tensor([105, 109]), f, inter)
        assert torch.allclose(a.norm(dim=-1), x.norm(dim=-1), rtol=1e-12)
        assert torch.equal(a[..., 32:], x[..., 32:])
        # a score depends on the difference of the positions only
        assert math.isclose(float(a[0, 0] @ a[1, 0]), float(b[0, 0] @ b[1, 0]), rel_tol=1e-9)


def test_plain_visibility():
    assert plain.visible(10, 4, 0, 0) == [0, 1, 2, 3, 4]
    assert plain.visible(10, 7, 3, 2) == [0, 1, 5, 6, 7]
    assert plain.visible(10, 1, 3, 4) == [0, 1]
    assert plain.visible(10, -1, 0, 0) == [] and plain.visible(0, 5, 0, 0) == []


def test_window_attn_refusals(sv):
    f = sv.load().window_attn
    r = rows(sv)

    def call(q=r, k=r, v=r, o=r, cu_q=A, cu_k=A, B=2, Tq=9, Tk=9, Hq=8, Hkv=4, D=128, scale=0.1, window=0, sinks=0):
        return f(q, k, v, o, cu_q, cu_k, B, Tq, Tk, Hq, Hkv, D, scale, window, sinks, None, 0, None)

    assert call(q=None) == 1 and call(v=None) == 1 and call(o=rows(sv, ptr=A + 8)) == 1
    assert call(cu_q=None) == 1 and call(cu_k=A + 2) == 1
    assert call(B=-1) == 1 and call(Tq=-1) == 1 and call(Tk=-1) == 1 and call(Hq=6) == 1
    assert call(scale=0.0) == 1 and call(scale=float("nan")) == 1
    assert call(window=-1) == 1 and call(sinks=-1) == 1
    assert call(k=rows(sv, ts=1028)) == 1
    assert call(D=64) == 2 and call(Hq=129 * 4) == 2 and call(B=5000) == 2
    assert call(k=rows(sv, ts=0)) == 2 and call(v=rows(sv, hs=0)) == 2   # repeated rows
    assert call(Tk=(1 << 30) + 1) == 2 and call(window=(1 << 30) + 1) == 2
    assert call(B=0) == 0 and call(Tq=0) == 0


def test_paged_kv_maps_refusals(sv):
    f = sv.load().paged_kv_maps
    out = (ctypes.c_uint64 * 32)()
    assert f(None, 4, 128, out, 256) == 1
    assert f(cache(sv), 4, 128, None, 256) == 1 and f(cache(sv), 4, 128, out, 255) == 1
    assert f(cache(sv), 0, 128, out, 256) == 1
    assert f(cache(sv, k=A + 8), 4, 128, out, 256) == 1
    assert f(cache(sv), 4, 64, out, 256) == 2
    assert sv._PAGED_KV.size == 80
