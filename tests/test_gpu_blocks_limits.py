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


# --- trie attention ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens", [[5, 12], [64, 64, 40]])  # the prefix shared by all rows; read by each request
@pytest.mark.parametrize("length,pages", [(-1, None), (49, None), (2**31 - 1, None), (33, -2), (33, 10**6)])
def test_attend_tree_bad_prefix_leaves_rows_behind_alone(length, pages, lens):
    """A prefix whose length or page is out of range makes every request's rows NaN; the rows behind the
    last request stay as they were, as they do after a good call."""
    p = Problem(lens, [40, 20, 7][:len(lens)], 33, 4, 2, 64, 16, torch.bfloat16, 62)
    n, pad = sum(lens), 7
    p.q, p.kn, p.vn = (torch.cat([t, torch.full_like(t[:pad], NAN)]) for t in (p.q, p.kn, p.vn))
    p.parent += [-5] * pad
    out, lse = torch.full((n + pad, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV), torch.full((n + pad, 4), 3.0, device=DEV)
    table = list(p.prefix_list)
    if pages is not None:
        table[1] = pages
    p.call(prefix_pages=i32(table), prefix_len=i32([length]), out=out, lse=lse)
    assert torch.isnan(out[:n]).all() and torch.isnan(lse[:n]).all()
    assert (out[n:] == 3.0).all() and (lse[n:] == 3.0).all()
    p.off = [0, lens[0] + 1, lens[0]] + p.off[3:]  # bad offsets besides: no row is known to be behind
    p.call(prefix_pages=i32(table), prefix_len=i32([length]), out=out, lse=lse)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


# --- streams ----------------------------------------------------------------------------------

def late(dst, src, stream):
    """Fill dst on `stream`, behind tens of milliseconds of other work."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(1 << 26)
        dst.copy_(src)


@pytest.mark.parametrize("handle", [0, 1, "current", "default", "own"])
def test_streams_by_handle(handle):
    """A call runs on the stream that it is given, as a handle too: the legacy default stream has the
    handles 0 and 1. It sees what was written there before it, and what follows there sees its results."""
    s = torch.cuda.Stream() if handle == "own" else torch.cuda.default_stream()
    h = {"current": torch.cuda.current_stream().cuda_stream, "own": s.cuda_stream, "default": s}.get(handle, handle)
    p = Problem([5, 3], [40, 20], 33, 4, 2, 64, 16, torch.bfloat16, 63)
    args, pre = p.args()
    want = psispec.attend_tree(*args, **pre)
    probs = torch.softmax(torch.randn(3, 500, generator=torch.Generator(DEV).manual_seed(64), device=DEV), -1)
    off, x, ua, ur = i32([0, 2]), probs[:2].argmax(-1).int(), torch.zeros(2, device=DEV), torch.full((3,), 0.5, device=DEV)
    ver = psispec.verify_probs(probs, None, off, x, ua, ur)
    kc, vc = torch.zeros_like(p.kc), torch.zeros_like(p.vc)
    page = (set(range(kc.shape[0])) - set(p.table[0][:3] + p.table[1][:2] + p.prefix_list)).pop()
    table = i32([[page]])
    q, k, rows = torch.zeros_like(args[0]), torch.zeros_like(args[1]), torch.full_like(probs, 1 / 500)
    args[0], args[1], good_q, good_k = q, k, args[0], args[1]
    zero, two = i32([0]), i32([2])
    torch.cuda.synchronize()
    for dst, src in ((q, good_q), (k, good_k), (rows, probs)):
        late(dst, src, s)
    a = psispec.attend_tree(*args, **pre, stream=h)
    v = psispec.verify_probs(rows, None, off, x, ua, ur, stream=h)
    n = psispec.commit_tree(k, args[2], args[3][:2], None, two, kc, vc, table, zero, stream=h)
    with torch.cuda.stream(s):
        got = [t.clone() for t in (a["out"], a["lse"], v["tokens"], v["accept_len"], n, kc[page, :3])]
    torch.cuda.synchronize()
    for g, w in zip(got, (want["out"], want["lse"], ver["tokens"], ver["accept_len"], i32([3]), good_k[:3])):
        assert torch.equal(g, w)


def test_commit_tree_refuses_a_path_without_columns():
    """A path that holds no node is not the linear batch's missing path."""
    kn, kc = torch.randn(4, 2, 64, device=DEV).bfloat16(), torch.zeros(2, 8, 2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        psispec.commit_tree(kn, kn, i32([0, 4]), torch.zeros(1, 0, dtype=torch.int32, device=DEV), i32([2]), kc, kc.clone(),
                            i32([[0]]), i32([0]))
    assert (kc == 0).all()
