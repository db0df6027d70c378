"""A cache's dimension of one may carry any stride: PyTorch keeps odd ones there
(a transposed single head counts as contiguous).  No GPU."""
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


def pages(strides, *shape):
    return torch.zeros(1 << 16, dtype=torch.bfloat16).as_strided(shape, strides).as_subclass(Pages)


def strides_of(sv, c):
    """(page, slot, head) strides that the calls get."""
    return sv._PAGED_KV.unpack(c.packed)[4:7]


@pytest.mark.parametrize("odd", [0, 1, 7, 64, 1024])
def test_one_head(sv, odd):
    want = pages((1024, 64, 64, 1), 4, 16, 1, 64)
    c = sv.PagedKV(want, pages((1024, 64, odd, 1), 4, 16, 1, 64))      # k's and v's differ there only
    page, slot, head = strides_of(sv, c)
    assert (page, slot) == (1024, 64) and head > 0 and head % 8 == 0
    c = sv.PagedKV(*(pages((1024, odd, 64, 1), 4, 1, 16, 64) for _ in range(2)), layout="HND")
    page, slot, head = strides_of(sv, c)
    assert (page, slot) == (1024, 64) and head > 0 and head % 8 == 0
    assert c.heads == 1 and c.page_size == 16


@pytest.mark.parametrize("odd", [0, 3, 8192])
def test_one_page(sv, odd):
    c = sv.PagedKV(pages((odd, 128, 64, 1), 1, 16, 2, 64), pages((2048, 128, 64, 1), 1, 16, 2, 64))
    page, slot, head = strides_of(sv, c)
    assert (slot, head) == (128, 64) and page > 0 and page % 8 == 0


def test_a_single_head_seen_the_other_way_round(sv):
    k = torch.zeros(4, 16, 1, 64, dtype=torch.bfloat16).transpose(1, 2).as_subclass(Pages)   # [4, 1, 16, 64]
    v = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16).as_subclass(Pages)
    assert k.is_contiguous() and k.stride() != v.stride()
    assert strides_of(sv, sv.PagedKV(k, v, layout="HND"))[:2] == (1024, 64)


def test_strides_that_count_are_compared(sv):
    for bad in (pages((1024, 64, 64, 1), 4, 16, 2, 64), pages((2048, 128, 128, 1), 4, 16, 2, 64)):
        with pytest.raises(sv.SvError):
            sv.PagedKV(pages((2048, 128, 64, 1), 4, 16, 2, 64), bad)
