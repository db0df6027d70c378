"""Calls with nothing to do: empty tensors have no address (PyTorch gives 0),
and no call of theirs may be refused for it.  No GPU."""
import pytest

from speculative_decoding_verify_08_gb300 import build_lib

A = 256  # an aligned stand-in address; never dereferenced


@pytest.fixture(scope="module")
def sv():
    build_lib.build()
    import speculative_decoding_verify_08_gb300 as sv
    sv.load()
    return sv


def test_no_tokens_with_a_rotation(sv):
    r = sv._ROWS.pack(0, 1024, 128)
    turn, norm = sv._ROTATION.pack(A, 0, 128, 0), sv._NORM.pack(A, A, 1e-6, 0.0)
    f = sv.load().qk_norm_rope
    assert f(r, r, r, r, norm, turn, 0, 8, 2, 128, None) == 0
    c = sv._PAGED_KV.pack(A, A, 0, 0, 16 * 4 * 128, 4 * 128, 128, 8, 16, 0, 0)
    f = sv.load().paged_kv_append
    assert f(None, None, r, r, c, None, norm, turn, 0, 0, 4, 128, None) == 0
    assert f(r, r, r, r, c, None, norm, turn, 0, 8, 4, 128, None) == 0
    # with tokens the positions are needed as before, and the table always
    full = sv._ROWS.pack(A, 1024, 128)
    assert sv.load().qk_norm_rope(full, full, full, full, norm, turn, 1, 8, 2, 128, None) == 1
    assert sv.load().qk_norm_rope(r, r, r, r, norm, sv._ROTATION.pack(A, 2, 128, 0), 0, 8, 2, 128, None) == 1
    assert sv.load().qk_norm_rope(r, r, r, r, norm, sv._ROTATION.pack(A, 0, 12, 0), 0, 8, 2, 128, None) == 1


def test_no_sequences(sv):
    r = sv._ROWS.pack(0, 0, 0)
    c = sv._PAGED_KV.pack(A, A, 0, 0, 16 * 4 * 128, 4 * 128, 128, 8, 16, 0, 0)
    f = sv.load().paged_attn
    assert f(r, c, None, 0, 8, None, r, 0, 1, 8, 4, 128, 0.1, 0, 0, None, 0, None) == 0
    assert f(r, c, None, 0, 0, None, r, 0, 1, 8, 4, 128, 0.1, 0, 0, None, 0, None) == 0   # a table of no columns either
    assert f(r, c, None, 0, -1, None, r, 0, 1, 8, 4, 128, 0.1, 0, 0, None, 0, None) == 1
    f = sv.load().window_attn
    assert f(r, r, r, r, None, None, 0, 0, 0, 8, 4, 128, 0.1, 0, 0, None, 0, None) == 0
