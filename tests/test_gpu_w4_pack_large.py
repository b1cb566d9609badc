"""w4_pack of more chunks than one launch has threads for (2^32 at 64 a chunk)."""
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu


def test_more_chunks_than_a_launch_holds():
    n, k, gc, L = 16, 128, 128, (1 << 26) + 3          # one chunk a weight, 68 GiB packed
    gen = torch.Generator().manual_seed(1)
    wq = torch.randint(0, 256, (n, k // 2), generator=gen, dtype=torch.uint8).to(DEV)
    s = torch.rand((n, 1), generator=gen).to(DEV)
    if torch.cuda.mem_get_info()[0] < (80 << 30):
        pytest.skip("needs 80 GiB of free device memory")
    one = sg.w4_pack(wq, s, gc)
    say(f"w4 pack of {L} weights")
    many = sg.w4_pack(wq.expand(L, n, k // 2), s.expand(L, n, 1), gc)     # the same weight, distance 0
    assert many.shape == (L, one.numel())
    for at in (0, 1, (1 << 22) - 1, 1 << 22, (1 << 26) - 1, 1 << 26, L - 1):
        assert torch.equal(many[at], one), at
    words = many.view(torch.int64)
    step = 1 << 22
    for i in range(0, L, step):                        # all of it, a part at a time
        assert (words[i:i + step] == one.view(torch.int64)).all(), i
    del many, words
    torch.cuda.empty_cache()
