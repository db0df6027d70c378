"""paged_chunk_attn over e4m3 pages with key scales and queries so small that all scores are
next to zero (GPU): a row is the plain average of what it sees."""
import pytest
import torch

import paged_plain as plain
from test_chunk_attn_gpu import Call, attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("k_scale", [1.0, 2.0 ** -30, 2.0 ** -60, 2.0 ** -100])
def test_small_queries_and_key_scales(cuda_lib, D, k_scale):
    """Rows of zeros (as a padded batch holds), of 1e-38, 1e-20 and of ones, masked in their last block."""
    seqs = [(60, 200), (5, 3), (7, 9000)]
    c = Call(cuda_lib, seqs, 4, 2, D, 16, e4m3=True, seed=83, dirty=False)
    c.ks = torch.full((2,), k_scale)
    size = torch.tensor([0.0, 1e-38, 1e-20, 1.0])[torch.arange(c.T) % 4]
    c.q = (c.q.float() * size[:, None, None]).bfloat16()
    c.want = []
    for b, (n, L) in enumerate(seqs):
        K, V = (plain.gather(x.float(), c.table[b], L, 16, "NHD", s) for x, s in ((c.k, c.ks), (c.v, c.vs)))
        c.want.append(attend(c.q[int(c.cu[b]):int(c.cu[b + 1]), :4], K, V, L - n, c.scale, 0, 0))
    c.check()
