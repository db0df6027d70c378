"""The calls over packed chunks and pools of states (paged_chunk_attn, gdn_chunk,
gdn_step) on the host: refusals before any launch, operands of another device,
calls with nothing to do, dimensions of one.  No GPU."""
import pytest
import torch

from speculative_decoding_verify_08_gb300 import build_lib

A = 256  # an aligned stand-in address; never dereferenced
BAD, UNSUPPORTED, WORKSPACE = 1, 2, 5


@pytest.fixture
def sv():
    build_lib.build()
    import speculative_decoding_verify_08_gb300 as sv
    sv.load()
    return sv


def rows(sv, ptr=A, ts=1024, hs=128):
    return sv._ROWS.pack(ptr, ts, hs)


def cache(sv, k=A, v=A, ks=0, vs=0, page=16 * 4 * 128, slot=4 * 128, head=128, pages=8, size=16, dtype=0):
    return sv._PAGED_KV.pack(k, v, ks, vs, page, slot, head, pages, size, dtype, 0)


def test_status_values(sv):
    assert (sv.SV_ERR_INVALID_ARG, sv.SV_ERR_UNSUPPORTED, sv.SV_ERR_WORKSPACE) == (BAD, UNSUPPORTED, WORKSPACE)


def test_paged_chunk_attn_refusals(sv):
    f = sv.load().paged_chunk_attn
    r, c = rows(sv), cache(sv)

    def call(q=r, cache=c, table=A, stride=8, width=8, lens=A, o=r, cu=A, B=2, Tq=9, Hq=8, Hkv=4, D=128, scale=0.1,
             window=0, sinks=0, ws=None, wsb=0):
        return f(q, cache, table, stride, width, lens, o, cu, B, Tq, Hq, Hkv, D, scale, window, sinks, ws, wsb, None)

    assert call(q=None) == BAD and call(o=None) == BAD and call(cache=None) == BAD
    assert call(table=None) == BAD and call(lens=None) == BAD and call(cu=None) == BAD
    assert call(table=A + 2) == BAD and call(lens=A + 1) == BAD and call(cu=A + 2) == BAD
    assert call(q=rows(sv, ptr=A + 8)) == BAD and call(o=rows(sv, ts=1028)) == BAD and call(q=rows(sv, hs=-128)) == BAD
    assert call(q=rows(sv, ptr=0)) == BAD
    assert call(B=-1) == BAD and call(Tq=-1) == BAD and call(Hq=6) == BAD and call(Hkv=0) == BAD and call(D=0) == BAD
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == BAD
    assert call(window=-1) == BAD and call(sinks=-1) == BAD and call(width=0) == BAD and call(stride=-1) == BAD
    assert call(cache=cache(sv, k=A + 8)) == BAD and call(cache=cache(sv, pages=0)) == BAD
    assert call(cache=cache(sv, ks=A)) == BAD                  # scales beside bf16
    assert call(cache=cache(sv, size=24)) == UNSUPPORTED
    assert call(D=64) == UNSUPPORTED and call(Hq=129 * 4) == UNSUPPORTED and call(B=4097) == UNSUPPORTED
    assert call(Tq=(1 << 30) + 1) == UNSUPPORTED and call(window=(1 << 30) + 1) == UNSUPPORTED
    assert call(width=1 << 27) == UNSUPPORTED                  # 2^31 positions
    assert call(q=rows(sv, ts=0)) == UNSUPPORTED and call(q=rows(sv, hs=0)) == UNSUPPORTED  # repeated rows
    if not torch.cuda.is_available():
        assert call() == 3                                     # no device to plan for
    w = sv.paged_chunk_attn_workspace_bytes
    assert w(0, 9, 8, 4, 128) == 0 and w(2, 0, 8, 4, 128) == 0 and w(2, 9, 8, 4, 64) == 0


def test_gdn_step_refusals(sv):
    f = sv.load().gdn_step
    r, s = rows(sv), sv._STATES.pack(A, 4 * 16 * 64, 5)

    def call(states=s, slots=A, tk=r, tv=r, tg=A, tb=A, n=A, tape_M=2, q=r, k=r, v=r, g=A, b=A, o=r, odt=sv.SV_BF16,
             B=2, M=3, commit=0, Hk=2, Hv=4, dk=64, dv=16):
        return f(states, slots, tk, tv, tg, tb, n, tape_M, q, k, v, g, b, o, odt, B, M, commit, Hk, Hv, dk, dv, None)

    pack = sv._STATES.pack
    assert call(states=None) == BAD and call(states=pack(0, 4096, 5)) == BAD and call(states=pack(A + 8, 4096, 5)) == BAD
    assert call(states=pack(A, 4095, 5)) == BAD                # not a multiple of four
    assert call(states=pack(A, 4092, 5)) == BAD                # states would overlap
    assert call(states=pack(A, -4096, 5)) == BAD and call(states=pack(A, 4096, 0)) == BAD
    assert call(states=pack(A, 1 << 41, 5)) == UNSUPPORTED and call(states=pack(A, 4096, 1 << 31)) == UNSUPPORTED
    assert call(slots=None) == BAD and call(slots=A + 2) == BAD and call(n=A + 2) == BAD
    for name in ("tk", "tv", "q", "k", "v", "o"):
        for bad in (None, rows(sv, ptr=0), rows(sv, ptr=A + 8), rows(sv, ts=1028), rows(sv, hs=-8)):
            assert call(**{name: bad}) == BAD, name
    for name in ("tg", "tb", "g", "b"):
        assert call(**{name: None}) == BAD and call(**{name: A + 2}) == BAD, name
    assert call(odt=sv.SV_E4M3) == BAD and call(Hv=3) == BAD and call(Hk=0) == BAD and call(dv=0) == BAD
    assert call(B=-1) == BAD and call(M=-1) == BAD and call(tape_M=-1) == BAD and call(dk=0) == BAD
    assert call(dk=96) == UNSUPPORTED and call(dk=512) == UNSUPPORTED
    assert call(M=65) == UNSUPPORTED and call(tape_M=65) == UNSUPPORTED
    assert call(B=65536) == UNSUPPORTED and call(dv=65537) == UNSUPPORTED and call(Hk=65536, Hv=65536) == UNSUPPORTED
    # nothing to do: no sequences, or neither rows nor a tape
    assert call(B=0, slots=None, n=None) == 0 and call(M=0, tape_M=0) == 0
    assert call(M=0, n=None, q=None, k=None, v=None, g=None, b=None, o=None, tk=None, tv=None, tg=None, tb=None) == 0


def test_gdn_chunk_refusals(sv):
    f = sv.load().gdn_chunk
    r, s = rows(sv), sv._STATES.pack(A, 4 * 16 * 64, 5)
    bytes_of = sv.gdn_chunk_workspace_bytes
    need = bytes_of(2, 90, 2, 4, 64, 16)
    assert need > 0

    def call(states=s, slots=A, q=r, k=r, v=r, g=A, b=A, o=r, cu=A, B=2, T=90, Hk=2, Hv=4, dk=64, dv=16, ws=None, wsb=0):
        return f(states, slots, q, k, v, g, b, o, cu, B, T, Hk, Hv, dk, dv, ws, wsb, None)

    pack = sv._STATES.pack
    assert call(states=None) == BAD and call(states=pack(A + 8, 4096, 5)) == BAD and call(states=pack(A, 4092, 5)) == BAD
    assert call(states=pack(A, (1 << 37) + 4, 5)) == UNSUPPORTED
    assert call(slots=None) == BAD and call(cu=None) == BAD and call(slots=A + 2) == BAD and call(cu=A + 2) == BAD
    for name in ("q", "k", "v", "o"):
        for bad in (None, rows(sv, ptr=0), rows(sv, ptr=A + 8), rows(sv, ts=1028), rows(sv, hs=-8)):
            assert call(**{name: bad}) == BAD, name
    for name in ("g", "b"):
        assert call(**{name: None}) == BAD and call(**{name: A + 2}) == BAD, name
    assert call(Hv=3) == BAD and call(Hk=0) == BAD and call(dv=0) == BAD and call(B=-1) == BAD and call(T=-1) == BAD
    assert call(dk=256) == UNSUPPORTED and call(dk=96) == UNSUPPORTED
    assert call(T=(1 << 30) + 1) == UNSUPPORTED and call(B=65536) == UNSUPPORTED
    assert call(dv=65537) == UNSUPPORTED and call(Hk=65536, Hv=65536) == UNSUPPORTED
    assert call(v=rows(sv, ts=0)) == UNSUPPORTED and call(v=rows(sv, hs=0)) == UNSUPPORTED   # repeated values
    assert call() == WORKSPACE and call(ws=A, wsb=need - 1) == WORKSPACE
    assert call(ws=A + 8, wsb=need) == BAD
    assert call(B=0, slots=None, cu=None) == 0 and call(T=0, q=rows(sv, ptr=0)) == 0
    # too many items for a launch's grid, whatever the workspace
    wide = pack(A, 1 << 34, 5)
    assert call(B=65535, Hk=1, Hv=65535, states=wide, ws=A, wsb=1 << 60) == UNSUPPORTED
    assert call(T=1 << 30, Hk=1 << 14, Hv=1 << 14, states=wide, ws=A, wsb=1 << 60) == UNSUPPORTED
    assert bytes_of(0, 9, 1, 1, 64, 64) == 0 and bytes_of(1, 0, 1, 1, 64, 64) == 0 and bytes_of(1, 9, 1, 1, 256, 64) == 0
    # the query grows with what it is given: a larger call's workspace does for a smaller one's
    assert bytes_of(3, 90, 2, 4, 64, 16) > need and bytes_of(2, 190, 2, 4, 64, 16) > need
    assert bytes_of(65535, 1 << 30, 1, 2, 128, 128) > 1 << 33  # past 32 bits


class On:
    """A tensor's description: shape, type and device; contiguous."""
    is_cuda = True

    def __init__(self, device, *shape, dtype=torch.bfloat16):
        self.device_index, self.dtype, self._meta = device, dtype, torch.empty(shape, dtype=dtype, device="meta")
        self.shape = self._meta.shape

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return 256

    def element_size(self):
        return self._meta.element_size()

    def __getattr__(self, name):  # stride, dim, numel, is_contiguous
        return getattr(self._meta, name)


I32, F32 = torch.int32, torch.float32


def calls(sv):
    """Each call with nothing to do, by its operands' devices, and its operands."""
    def attn(q=0, cache=0, table=0, lens=0, o=0, cu=0, ws=0):
        c = sv.PagedKV(On(cache, 4, 16, 2, 128), On(cache, 4, 16, 2, 128))
        sv.paged_chunk_attn(On(q, 0, 8, 128), c, On(table, 0, 3, dtype=I32), On(lens, 0, dtype=I32), On(o, 0, 8, 128),
                            On(cu, 1, dtype=I32), 0.1, workspace=On(ws, 64, dtype=torch.uint8), stream=0)

    def step(states=0, slots=0, q=0, k=0, v=0, g=0, beta=0, o=0, tk=0, tv=0, tg=0, tb=0, n=0):
        sv.gdn_step(On(states, 3, 4, 16, 64, dtype=F32), On(slots, 0, dtype=I32), On(q, 0, 2, 64), On(k, 0, 2, 64),
                    On(v, 0, 4, 16), On(g, 0, 4, dtype=F32), On(beta, 0, 4, dtype=F32), On(o, 0, 4, 16), 2,
                    tape=(On(tk, 0, 2, 64), On(tv, 0, 4, 16), On(tg, 0, 4, dtype=F32), On(tb, 0, 4, dtype=F32)),
                    n_replay=On(n, 0, dtype=I32), stream=0)

    def chunk(states=0, slots=0, q=0, k=0, v=0, g=0, beta=0, o=0, cu=0, ws=0):
        sv.gdn_chunk(On(states, 3, 4, 16, 64, dtype=F32), On(slots, 0, dtype=I32), On(q, 0, 2, 64), On(k, 0, 2, 64),
                     On(v, 0, 4, 16), On(g, 0, 4, dtype=F32), On(beta, 0, 4, dtype=F32), On(o, 0, 4, 16),
                     On(cu, 1, dtype=I32), workspace=On(ws, 64, dtype=torch.uint8), stream=0)

    return attn, step, chunk


@pytest.mark.parametrize("which", [0, 1, 2])
def test_operands_of_another_device(sv, monkeypatch, which):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(sv, "_gpus", 2)
    # no tensor maps without a GPU's driver: the cache's fields as they are
    monkeypatch.setattr(sv.load(), "paged_kv_maps", lambda *a: 0)
    call = calls(sv)[which]
    names = call.__code__.co_varnames[:call.__code__.co_argcount]
    call()
    for n in names:
        with pytest.raises(sv.SvError) as e:
            call(**{n: 1})
        assert e.value.status == BAD, n
    with pytest.raises(sv.SvError):
        call(**{n: 1 for n in names})


class Held(torch.Tensor):
    """CPU memory that says it is a GPU's; calls over it stay on the host."""
    is_cuda = True

    def get_device(self):
        return 0


def held(*shape, dtype=torch.bfloat16, strides=None):
    t = torch.zeros(1 << 16, dtype=dtype)
    return (t[:torch.Size(shape).numel()].view(shape) if strides is None else t.as_strided(shape, strides)).as_subclass(Held)


def step_args(**other):
    a = dict(states=held(3, 4, 16, 64, dtype=F32), slots=held(2, dtype=I32), q=held(4, 2, 64), k=held(4, 2, 64),
             v=held(4, 4, 16), g=held(4, 4, dtype=F32), beta=held(4, 4, dtype=F32), o=held(4, 4, 16), M=2, stream=0)
    a.update(other)
    return a


def chunk_args(**other):
    a = step_args(cu=held(3, dtype=I32), workspace=held(1 << 16, dtype=torch.uint8))
    del a["M"]
    a.update(other)
    return a


@pytest.fixture
def caught(sv, monkeypatch):
    """The library's entry points replaced by ones that keep their arguments."""
    seen = []
    for name in ("gdn_step", "gdn_chunk"):
        monkeypatch.setattr(sv.load(), name, lambda *a: seen.append(a) or 0)
    monkeypatch.setattr(sv, "_gpus", 1)
    return seen


@pytest.mark.parametrize("bad", [
    dict(states=held(3, 4, 16, 64)), dict(states=held(4, 16, 64, dtype=F32)),
    dict(states=held(3, 4, 16, 64, dtype=F32, strides=(8192, 2048, 128, 1))),
    dict(slots=held(2, dtype=torch.int64)), dict(q=held(5, 2, 64)), dict(q=held(4, 2, 128)), dict(k=held(4, 3, 64)),
    dict(q=held(4, 2, 64, dtype=torch.float16)), dict(v=held(4, 2, 16)), dict(g=held(4, 4)), dict(g=held(4, 2, dtype=F32)),
    dict(beta=held(16, dtype=F32)), dict(o=held(4, 4, 17)), dict(q=torch.zeros(4, 2, 64, dtype=torch.bfloat16)),
    dict(states=torch.zeros(3, 4, 16, 64))])
def test_wrong_tensors(sv, caught, bad):
    for f, args in ((sv.gdn_step, step_args), (sv.gdn_chunk, chunk_args)):
        f(**args())
        caught.clear()
        with pytest.raises(sv.SvError) as e:
            f(**args(**bad))
        assert e.value.status == BAD and not caught
    with pytest.raises(sv.SvError):
        sv.gdn_chunk(**chunk_args(cu=held(2, dtype=I32)))
    with pytest.raises(sv.SvError):
        sv.gdn_chunk(**chunk_args(workspace=torch.zeros(64, dtype=torch.uint8)))


def test_tapes(sv, caught):
    tape = (held(6, 2, 64), held(6, 4, 16), held(6, 4, dtype=F32), held(6, 4, dtype=F32))
    sv.gdn_step(**step_args(tape=tape, n_replay=held(2, dtype=I32)))
    assert caught[-1][7] == 3                                  # rows of the tape a sequence
    for bad in (dict(tape=tape), dict(n_replay=held(2, dtype=I32)), dict(tape=tape, n_replay=held(3, dtype=I32)),
                dict(tape=tape[:3], n_replay=held(2, dtype=I32)),
                dict(tape=(held(5, 2, 64),) + tape[1:], n_replay=held(2, dtype=I32)),
                dict(tape=(tape[0], held(4, 4, 16)) + tape[2:], n_replay=held(2, dtype=I32))):
        with pytest.raises(sv.SvError):
            sv.gdn_step(**step_args(**bad))
    caught.clear()
    sv.gdn_step(**step_args(tape=tape, n_replay=held(2, dtype=I32), M=0, q=None, k=None, v=None, g=None, beta=None, o=None))
    assert caught[0][8:14] == (None,) * 6


def test_dimensions_of_one_may_carry_any_stride(sv, caught):
    sv.gdn_step(**step_args(states=held(1, 4, 16, 64, dtype=F32, strides=(7, 1024, 64, 1)), slots=held(2, dtype=I32)))
    assert sv._STATES.unpack(caught[-1][0])[1:] == (4096, 1)
    one = dict(states=held(3, 1, 16, 64, dtype=F32, strides=(1024, 5, 64, 1)), q=held(4, 1, 64, strides=(64, 3, 1)),
               k=held(4, 1, 64, strides=(64, 1, 1)), v=held(4, 1, 16, strides=(16, 9, 1)), g=held(4, 1, dtype=F32),
               beta=held(4, 1, dtype=F32), o=held(4, 1, 16, dtype=F32, strides=(16, 9, 1)))
    sv.gdn_step(**step_args(**one))
    assert all(sv._ROWS.unpack(caught[-1][i])[2] % 8 == 0 for i in (8, 9, 10, 13))
    one["o"] = held(4, 1, 16, strides=(16, 9, 1))
    sv.gdn_chunk(**chunk_args(**one))
    assert all(sv._ROWS.unpack(caught[-1][i])[2] % 8 == 0 for i in (2, 3, 4, 7))
