"""The bound on window_attn's items, on the host.  No GPU."""
import pytest
import torch

from speculative_decoding_verify_08_gb300 import build_lib

A = 256  # an aligned stand-in address; never dereferenced


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call within the bound would be launched")
def test_item_bound():
    build_lib.build()
    import speculative_decoding_verify_08_gb300 as sv
    f, r = sv.load().window_attn, sv._ROWS.pack(A, 65536, 128)

    def call(Tq, B, Hq, Hkv):
        return f(r, r, r, r, A, A, B, Tq, 9, Hq, Hkv, 128, 0.1, 0, 0, None, 0, None)

    assert call(0x3fff8000 - 2, 2, 256, 2) == sv.SV_ERR_CUDA          # one position a tile; no device to plan for
    assert call(0x3fff8000 - 1, 2, 256, 2) == sv.SV_ERR_UNSUPPORTED
    assert call(0x3fffffff, 2, 256, 2) == sv.SV_ERR_UNSUPPORTED
    assert call(1 << 30, 4096, 128, 1) == sv.SV_ERR_CUDA
