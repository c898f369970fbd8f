"""GPU tests of the operators around a drafted block at the ends of what their arguments can hold,
and of what a caller's own program does with them."""
import pytest
import torch

from lossless_speculative_sampling_b200 import psispec
from test_gpu_blocks import DEV, Problem, i32, offsets

pytestmark = pytest.mark.gpu
NAN = float("nan")


# --- the commit -------------------------------------------------------------------------------

@pytest.mark.parametrize("path", [None, [[1, 2, 3]] * 3])
@pytest.mark.parametrize("bad", [2**31 - 1, 2**31 - 2, 1 << 30, 1024, 1023, 4, -2, -(2**31)])
def test_commit_tree_accept_lengths_of_any_size(bad, path):
    """An accept length that its request cannot have commits nothing and gives -1, up to the largest
    int, with a path and without one; the requests beside it are committed."""
    g = torch.Generator().manual_seed(61)
    kn, vn = (torch.randn(2, 12, 2, 64, generator=g).bfloat16().to(DEV) for _ in range(2))
    kc, vc = (torch.randn(2, 6, 8, 2, 64, generator=g).bfloat16().to(DEV) for _ in range(2))
    wk, wv = kc.clone(), vc.clone()
    for b, page in ((0, 0), (2, 4)):
        wk[:, page, 3:6], wv[:, page, 3:6] = kn[:, 4 * b:4 * b + 3], vn[:, 4 * b:4 * b + 3]
    new = psispec.commit_tree(kn, vn, offsets([4, 4, 4]), None if path is None else i32(path), i32([2, bad, 2]), kc, vc,
                              i32([[0, 1], [2, 3], [4, 5]]), i32([3, 3, 3]))
    assert new.tolist() == [6, -1, 6]
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
