"""Operands of the paged-cache calls that live on another GPU than the current
one, where the library launches, are refused before anything reaches it.

Stand-ins for tensors carry a device number and no memory; calls that would
pass have no tokens, so nothing is launched.  No GPU."""
import pytest
import torch

from speculative_decoding_verify_08_gb300 import build_lib


@pytest.fixture
def sv(monkeypatch):
    build_lib.build()
    import speculative_decoding_verify_08_gb300 as sv
    sv.load()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(sv, "_gpus", 2)
    return sv


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


def refused(sv, f):
    with pytest.raises(sv.SvError) as e:
        f()
    assert e.value.status == sv.SV_ERR_INVALID_ARG


def each_elsewhere(sv, call, names):
    """The call with everything on the current device, then with one operand
    after the other, and with all of them, on another."""
    call(**{n: 0 for n in names})
    for n in names:
        refused(sv, lambda: call(**{m: 1 if m == n else 0 for m in names}))
    refused(sv, lambda: call(**{n: 1 for n in names}))


def cache_on(sv, device):
    k, v = (On(device, 4, 16, 2, 64) for _ in range(2))
    return sv.PagedKV(k, v)


def test_qk_norm_rope(sv):
    def call(q, k, qo, ko, pos, ph, qw, kw):
        sv.qk_norm_rope(On(q, 0, 8, 64), On(k, 0, 2, 64), On(qo, 0, 8, 64), On(ko, 0, 2, 64),
                        On(pos, 0, dtype=torch.int32), On(ph, 32, dtype=torch.int64), On(qw, 64), On(kw, 64), stream=0)

    each_elsewhere(sv, call, ["q", "k", "qo", "ko", "pos", "ph", "qw", "kw"])


def test_paged_kv_append(sv):
    def call(k, v, cache, slots, q, qo):
        sv.paged_kv_append(On(k, 0, 2, 64), On(v, 0, 2, 64), cache_on(sv, cache), On(slots, 0, dtype=torch.int64),
                           q=On(q, 0, 8, 64), q_out=On(qo, 0, 8, 64), stream=0)

    each_elsewhere(sv, call, ["k", "v", "cache", "slots", "q", "qo"])


def test_paged_attn(sv, monkeypatch):
    # no tensor maps without a GPU's driver: the cache's fields as they are
    monkeypatch.setattr(sv.load(), "paged_kv_maps", lambda *a: 0)

    def call(q, cache, table, lens, o, ws):
        c = sv.PagedKV(On(cache, 4, 16, 2, 128), On(cache, 4, 16, 2, 128))
        sv.paged_attn(On(q, 0, 8, 128), c, On(table, 0, 3, dtype=torch.int32), On(lens, 0, dtype=torch.int32),
                      On(o, 0, 8, 128), 1, 0.1, workspace=On(ws, 64, dtype=torch.uint8), stream=0)

    each_elsewhere(sv, call, ["q", "cache", "table", "lens", "o", "ws"])


def test_window_attn(sv):
    def call(q, k, v, o, cu_q, cu_k):
        sv.window_attn(On(q, 0, 8, 128), On(k, 5, 2, 128), On(v, 5, 2, 128), On(o, 0, 8, 128),
                       On(cu_q, 2, dtype=torch.int32), On(cu_k, 2, dtype=torch.int32), 0.1, stream=0)

    each_elsewhere(sv, call, ["q", "k", "v", "o", "cu_q", "cu_k"])


def test_cache_scales(sv):
    k, v, s = On(1, 4, 16, 2, 64), On(1, 4, 16, 2, 64), On(1, 2, dtype=torch.float32)
    k.dtype = v.dtype = torch.float8_e4m3fn
    refused(sv, lambda: sv.PagedKV(k, v, k_scale=On(0, 2, dtype=torch.float32), v_scale=s))
    refused(sv, lambda: sv.PagedKV(k, v, k_scale=s, v_scale=On(0, 2, dtype=torch.float32)))
    sv.PagedKV(k, v, k_scale=s, v_scale=s)   # a cache may be made while another device is current


def test_one_gpu(sv, monkeypatch):
    """The only GPU is not asked for tensor by tensor; CPU memory is refused all the same."""
    monkeypatch.setattr(sv, "_gpus", 0)
    monkeypatch.setattr(torch._C, "_cuda_getDeviceCount", lambda: 1)
    q, k, cpu = On(0, 0, 8, 64), On(0, 0, 2, 64), torch.empty(0, 2, 64, dtype=torch.bfloat16)
    sv.qk_norm_rope(q, k, q, k, stream=0)
    assert sv._gpus == 1
    sv.qk_norm_rope(q, k, q, k, stream=0)
    for args in ((q, k, q, cpu), (q, cpu, q, k), (torch.empty(0, 8, 64, dtype=torch.bfloat16), k, q, k)):
        refused(sv, lambda: sv.qk_norm_rope(*args, stream=0))
