"""paged_chunk_attn at the sequence and tile counts where the kernel's own bookkeeping
changes (GPU), against softmax attention in 64 bits."""
import pytest
import torch

from test_chunk_attn_gpu import Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [31, 32, 60, 127, 128])
@pytest.mark.parametrize("D,e4m3", [(128, False), (256, False), (128, True), (256, True)])
def test_a_serving_batch(cuda_lib, B, D, e4m3):
    """Prompts' chunks, single tokens and empty rows side by side."""
    g = torch.Generator().manual_seed(B)
    new = torch.tensor([1, 1, 1, 0, 5, 40, 150])[torch.randint(0, 7, (B,), generator=g)].tolist()
    past = torch.randint(0, 300, (B,), generator=g).tolist()
    Call(cuda_lib, [(n, n + p) for n, p in zip(new, past)], 4, 2, D, 16, e4m3=e4m3, seed=84, extra=3).check()


@pytest.mark.parametrize("D,e4m3", [(128, False), (256, False), (128, True), (256, True)])
def test_more_sequences_than_threads(cuda_lib, D, e4m3):
    """A tile a sequence, 700 of them; the CTAs have 384 threads, or 512."""
    Call(cuda_lib, [(1, 1 + 13 * i % 150) for i in range(700)], 2, 1, D, 16, e4m3=e4m3, seed=85).check()


def test_more_tiles_than_threads(cuda_lib):
    """One sequence of 800 rows, two a tile; items are cut and joined too."""
    Call(cuda_lib, [(800, 810)], 64, 1, 256, 64, seed=86, dirty=False).check()
