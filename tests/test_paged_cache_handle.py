"""A PagedKV names its tensors for good: what the calls use was worked out from
them once, so they cannot be exchanged, and a copy works its own out.  No GPU."""
import copy
import pickle

import pytest
import torch

from speculative_decoding_verify_08_gb300 import build_lib


@pytest.fixture
def sv():
    build_lib.build()
    import speculative_decoding_verify_08_gb300 as sv
    sv.load()
    return sv


class Pages(torch.Tensor):
    """CPU memory that says it is a GPU's; calls over it stay on the host."""
    is_cuda = True

    def get_device(self):
        return 0

    def __deepcopy__(self, memo):
        return self.clone()


def pages(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Pages)


def cache_of(sv, **kw):
    return sv.PagedKV(pages(4, 16, 2, 64), pages(4, 16, 2, 64), **kw)


def addresses(sv, cache):
    return sv._PAGED_KV.unpack(cache.packed)[:4]


def test_fields_are_read_only(sv):
    c = cache_of(sv)
    before = dict(k=c.k, v=c.v, packed=c.packed, heads=c.heads)
    for name in ("k", "v", "k_scale", "v_scale", "layout", "page_size", "heads", "D", "device", "packed"):
        with pytest.raises(AttributeError):
            setattr(c, name, pages(4, 16, 2, 64))
        with pytest.raises(AttributeError):
            delattr(c, name)
    assert all(getattr(c, n) is x for n, x in before.items())
    c.k[1, 2, 0, 3] = 5.0   # their contents are another matter
    assert float(c.k[1, 2, 0, 3]) == 5.0


def test_copies_name_their_own_pages(sv):
    c = cache_of(sv, layout="HND")
    other = copy.deepcopy(c)
    assert other.k is not c.k and other.k.data_ptr() != c.k.data_ptr()
    assert addresses(sv, other) == (other.k.data_ptr(), other.v.data_ptr(), 0, 0)
    assert other.layout == c.layout and other.heads == c.heads
    shallow = copy.copy(c)
    assert shallow.k is c.k and addresses(sv, shallow) == addresses(sv, c)


def test_copies_with_scales_and_shared_storage(sv):
    both = pages(4, 32, 2, 64)
    s = pages(2, dtype=torch.float32)
    c = sv.PagedKV(both[:, :16].to(torch.float8_e4m3fn), both[:, 16:].to(torch.float8_e4m3fn), k_scale=s, v_scale=s)
    d = copy.deepcopy(c)
    assert addresses(sv, d) == tuple(t.data_ptr() for t in (d.k, d.v, d.k_scale, d.v_scale))
    assert d.k_scale is d.v_scale and d.k_scale.data_ptr() != s.data_ptr()


def test_a_pickled_cache_names_what_was_loaded(sv):
    c = cache_of(sv)
    d = pickle.loads(pickle.dumps(c))
    assert addresses(sv, d)[:2] == (d.k.data_ptr(), d.v.data_ptr())
    assert d.k.data_ptr() != c.k.data_ptr()
