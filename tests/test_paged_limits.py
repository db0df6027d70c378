"""The bounds that the header states for paged_attn, on both sides, on the host.
No GPU: a call within them ends at SV_ERR_CUDA, for want of a device."""
import pytest
import torch

from speculative_decoding_verify_08_gb300 import build_lib

A = 256  # an aligned stand-in address; never dereferenced
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a call within the bounds would be launched")


@pytest.fixture(scope="module")
def call():
    build_lib.build()
    import speculative_decoding_verify_08_gb300 as sv
    f, r = sv.load().paged_attn, sv._ROWS.pack(A, 65536, 128)

    def call(cap, B=1, Hkv=1, G=1, M=1, D=128, page=16):
        c = sv._PAGED_KV.pack(A, A, 0, 0, 16 * 4 * 128, 4 * 128, 128, 8, page, 0, 0)
        assert cap % page == 0
        return f(r, c, A, cap // page, cap // page, A, r, B, M, Hkv * G, Hkv, D, 0.1, 0, 0, None, 0, None)

    return call


def test_positions(call):
    assert call(1 << 30) == 3 and call((1 << 30) + 16) == 2


@pytest.mark.parametrize("cap,B,page", [(1 << 30, 1, 16), (1 << 30, 31, 64), (1 << 20, 17, 128), (16, 4096, 16)])
def test_units(call, cap, B, page):
    """B * Hkv * (table_width*page_size / 16 + 12) < 2^31."""
    most = ((1 << 31) - 1) // (B * (cap // 16 + 12))
    assert call(cap, B=B, Hkv=most, page=page) == 3
    assert call(cap, B=B, Hkv=most + 1, page=page) == 2


def test_row_elements(call):
    """M * Hq * D <= 2^33: a sequence's rows are counted in groups of eight, in 31 bits with room for a step."""
    for D, G, M in ((256, 128, 1), (256, 1, 128), (128, 64, 2), (128, 1, 1)):
        most = (1 << 33) // (M * G * D)
        assert call(16, Hkv=min(most, 160000000), G=G, M=M, D=D) == 3
        if most < 160000000:   # (beyond, the units' bound comes first)
            assert call(16, Hkv=most + 1, G=G, M=M, D=D) == 2
