"""GPU tests of the operators around a drafted block at the ends of what their arguments can hold,
and of what a caller's own program does with them."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from lossless_speculative_sampling_b200 import build as libbuild
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


def test_a_captured_call_by_handle():
    """The handle of the stream that captures: the call and what it allocates belong to the graph."""
    p = Problem([5, 3], [40, 20], 33, 4, 2, 64, 16, torch.bfloat16, 65)
    args, pre = p.args()
    psispec.attend_tree(*args, **pre)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = psispec.attend_tree(*args, **pre, stream=torch.cuda.current_stream().cuda_stream)
    junk = [torch.full((1 << 20,), NAN, device=DEV) for _ in range(8)]
    for t, seed in ((args[0], 66), (args[1], 67)):
        t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)))
    del junk
    g.replay()
    torch.cuda.synchronize()
    p.check(r)


# --- a user's program ---------------------------------------------------------------------------

def readme_step():
    """The README's decoding step over candidate tries."""
    with open(os.path.join(os.path.dirname(psispec.HEADER), "..", "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)
    return compile([b for b in blocks if "commit_tree(" in b][0], "README.md", "exec")


@pytest.mark.parametrize("temp,top_p", [(0.0, 1.0), (0.7, 0.3), (0.7, 1.0), ("mixed", 0.5)])
def test_the_readme_decodes(temp, top_p):
    """Greedy requests and small top-p leave tries with unused slots, a draft row that is not finite leaves
    none at all. Requests go on in every case but the last, and the last one alone stands still."""
    g = torch.Generator(DEV).manual_seed(71)
    B, K, V, n_prefixes, Hq, Hkv, D, page = 4, 4, 300, 12, 4, 2, 64, 16
    emb = torch.randn(V, Hq * D, generator=g, device=DEV)
    w = torch.randn(Hq * D, (Hq + 2 * Hkv) * D, generator=g, device=DEV) / 16
    last_nodes = []

    def qkv(tokens):
        last_nodes.append(tokens)
        return (emb[tokens.long()] @ w).bfloat16().view(-1, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 1)

    def head(out):  # every node's likeliest next token: its own plus one, which is what is drafted
        return (out.flatten(1).float() @ emb.T * 0.01 + 20.0 * torch.nn.functional.one_hot((last_nodes[-1].long() + 1) % V, V)).contiguous()

    T = torch.tensor([0.0, 0.7, 0.0, 0.7] if temp == "mixed" else [temp] * B, device=DEV)
    ns = dict(torch=torch, psispec=psispec, B=B, K=K, T=T, top_p=torch.full((B,), top_p, device=DEV), n_prefixes=n_prefixes,
              cap=n_prefixes + 1, qkv=qkv, head=head, k_cache=torch.zeros(8, page, Hkv, D, dtype=torch.bfloat16, device=DEV),
              page_table=i32([[2 * b, 2 * b + 1] for b in range(B)]), context_len=i32([0] * B), prompt_pages=None, prompt_len=None,
              last_token=torch.randint(0, V, (B,), generator=g, device=DEV, dtype=torch.int32))
    ns["v_cache"] = torch.zeros_like(ns["k_cache"])
    history, step = [[int(t)] for t in ns["last_token"]], readme_step()
    for it in range(3):
        draft = torch.randn(B, K, V, generator=g, device=DEV)
        for i in range(K):
            draft[torch.arange(B), i, (ns["last_token"].long() + 1 + i) % V] += 12.0
        if it == 2:
            draft[3, 1, 7] = NAN
        u = torch.rand(2, B * ns["cap"], generator=g, device=DEV)
        old = ns["context_len"]
        ns.update(draft=draft, u_acc=u[0], u_res=u[1])
        exec(step, ns)
        accepted, toks = ns["ver"]["accept_len"].tolist(), ns["ver"]["tokens"]
        live = [b for b in range(B) if it < 2 or b != 3]
        assert all(accepted[b] >= 0 for b in live) and (it < 2 or accepted[3] == -1)
        assert ns["context_len"].tolist() == [c + a + 1 for c, a in zip(old.tolist(), accepted)]
        for b in live:
            history[b] += toks[b, :accepted[b] + 1].tolist()
        ns["last_token"] = torch.tensor([h[-1] for h in history], dtype=torch.int32, device=DEV)
    for b in range(B):  # the cache holds every token's keys but the last one's
        n = int(ns["context_len"][b])
        assert n == len(history[b]) - 1
        want = qkv(torch.tensor(history[b][:n], device=DEV))[1]
        got = ns["k_cache"][2 * b:2 * b + 2].flatten(0, 1)[:n]
        # one rounding to bf16 each of sums of 256 products in fp32, in orders of their own
        assert ((got.float() - want.float()).abs() <= 2.0**-7 * want.float().abs() + 2.0**-12).all()
        if float(T[b]) == 0.0:  # greedy: whole blocks are accepted, 5 tokens a step
            assert history[b] == [(history[b][0] + i) % V for i in range(len(history[b]))] and n >= 10


def test_a_step_of_the_tree_sampler_commits_the_right_rows():
    """Four steps of a two-layer model with tries; every row of the cache, in both layers, against the
    keys and values of the whole history run as one chain, and the same comparison with two rows of the cache
    exchanged, which has to fail for every pair of neighbours and every layer.

    Layer 0's keys and values are rows of a table by token: equal bit for bit, in the cache as in the chain.
    Layer 1 sees x = emb + a, a the attention's output, with scores of a few units (a row's weight is
    far from even). Of a, both runs are within u |a| + (1 + u) (u + 4 ds + 2^-20 + (2 n + 16) e) A <= 2.2 u A of the
    exact one (u = 2^-8, |a| <= A = sum p |v| <= max |v|; scale sum |q k| is below 16 in layer 0, so 4 ds and the rest
    are below u / 10), so they differ by 4.4 u max |v| at most, and their keys and values, products in fp64 rounded once,
    by 4.4 u max |v| sum |w| + 2 u |k|. Layer 1's rows are of order 1 and differ by as much."""
    g = torch.Generator(DEV).manual_seed(81)
    B, K, V, Hq, Hkv, D, page, cap = 3, 4, 500, 4, 2, 64, 16, 11
    u, E, dt = 2.0**-8, Hq * D, torch.bfloat16
    emb = torch.randn(V, E, generator=g, device=DEV)
    wq, wk, wv = ([torch.randn(E, h * D, generator=g, device=DEV).double() * (s / 16) for s in (1.0, 1.0)] for h in (Hq, Hkv, Hkv))
    table0 = [(emb.double() @ w[0]).to(dt).view(V, -1, D) for w in (wq, wk, wv)]
    q0, k0 = table0[0].abs().float(), table0[1].abs().float().repeat_interleave(Hq // Hkv, 1)
    assert torch.einsum("ahd,bhd->abh", q0, k0).max() * D**-0.5 < 16

    def run(tokens, off, parent, kc, vc, pages, ctx, pre):
        """Both layers over nodes: the last layer's x, and the layers' keys and values."""
        t, x = tokens.long(), emb[tokens.long()]
        ks, vs = [], []
        for layer in range(2):
            q, k, v = ((tab[t] for tab in table0) if layer == 0 else
                       ((x.double() @ w[1]).to(dt).view(len(t), -1, D) for w in (wq, wk, wv)))
            ks.append(k.contiguous())
            vs.append(v.contiguous())
            r = psispec.attend_tree(q.contiguous(), ks[-1], vs[-1], off, parent, kc[layer], vc[layer], pages, ctx,
                                    prefix_pages=pre[0], prefix_len=pre[1])
            x = x + r["out"].float().reshape(x.shape)
        return x, torch.stack(ks), torch.stack(vs)

    kc, vc = (torch.full((2, 40, page, Hkv, D), NAN, dtype=dt, device=DEV) for _ in range(2))
    prompt, none = torch.randint(0, V, (40,), generator=g, device=DEV), (None, None)
    ppages = i32([[5, 17, 2]])
    _, k, v = run(prompt, i32([0, 40]), None, kc, vc, ppages, i32([0]), none)
    assert psispec.commit_tree(k, v, i32([0, 40]), None, i32([39]), kc, vc, ppages, i32([0])).tolist() == [40]
    pre, pages = (ppages[0].contiguous(), i32([40])), i32([[20 + b, 30 + b] for b in range(B)])
    ctx, root = i32([0] * B), torch.randint(0, V, (B,), generator=g, device=DEV, dtype=torch.int32)
    T, P = torch.full((B,), 0.7, device=DEV), torch.ones(B, device=DEV)
    history = [prompt.tolist() + [int(r)] for r in root]
    for _ in range(4):
        tr = psispec.build_tree((torch.randn(B, K, V, generator=g, device=DEV) * 3).contiguous(), T, P, 4, cap - 1)
        assert tr["nodes"].tolist() == [cap] * B
        tokens = tr["tokens"].clone()
        tokens[:, 0] = root
        off, parent, flat = offsets([cap] * B), tr["parent"].reshape(-1).contiguous(), tokens.reshape(-1)
        _, k, v = run(flat, off, parent, kc, vc, pages, ctx, pre)
        # the model's own logits do not matter here: a node's children are far likelier than other tokens
        logits = torch.randn(B, cap, V, generator=g, device=DEV)
        at = (torch.arange(B, device=DEV)[:, None], tr["parent"][:, 1:].long(), tokens[:, 1:].long())
        logits[at] += 12.0
        logits = logits.view(B * cap, V)
        un = torch.rand(2, B * cap, generator=g, device=DEV)
        out = psispec.verify_tree_det(logits, off, parent, flat.contiguous(), un[0].contiguous(), un[1].contiguous(), T, P, K)
        ctx = psispec.commit_tree(k, v, off, out["path"], out["accept_len"], kc, vc, pages, ctx)
        for b in range(B):
            history[b] += out["tokens"][b, :int(out["accept_len"][b]) + 1].tolist()
        root = out["tokens"].gather(1, out["accept_len"].long()[:, None])[:, 0]
    assert int((ctx - 4).sum()) >= 4  # nodes behind the roots were accepted

    def excess(kc, vc, b):
        """How far each layer's rows of request b, prompt included, are beyond the bound: [2, rows], at most 0."""
        n = 40 + int(ctx[b])
        h = torch.tensor(history[b], device=DEV)
        assert len(h) == n + 1
        _, *want = run(h[:n], i32([0, n]), None, kc, vc, i32([[0]]), i32([0]), none)
        most = want[1][0].float().abs().max()
        worst = torch.full((2, n), -1.0, device=DEV)
        for cache, w1, wt in ((kc, wk, want[0]), (vc, wv, want[1])):
            got = torch.cat([cache[:, ppages[0].long()].flatten(1, 2)[:, :40], cache[:, pages[b].long()].flatten(1, 2)[:, :n - 40]], 1)
            d = (got.float() - wt.float()).abs()
            bound = torch.zeros_like(d)
            bound[1] = 4.4 * u * most * w1[1].abs().sum(0).float().view(Hkv, D) + 2 * u * wt[1].float().abs()
            worst = torch.maximum(worst, (d - bound).flatten(2).amax(-1))
        return worst

    for b in range(B):
        right = excess(kc, vc, b)
        assert (right <= 0).all(), float(right.max())
        own = int(ctx[b])
        for layer in range(2):
            for i in range(own - 1):
                if history[b][40 + i] == history[b][41 + i]:
                    continue
                k2, v2 = kc.clone(), vc.clone()
                at = [(int(pages[b, j // page]), j % page) for j in (i, i + 1)]
                for c2, c in ((k2, kc), (v2, vc)):
                    c2[layer][at[0]], c2[layer][at[1]] = c[layer][at[1]], c[layer][at[0]]
                wrong = excess(k2, v2, b)
                assert (wrong[layer, 40 + i:42 + i] > 0).all() and (wrong[1 - layer] <= 0).all()


# --- what no argument reaches: a library built with other limits ----------------------------------

def limited_library(tmp_path, *defines):
    """The operators built with lower limits, loaded beside the library that the other tests use."""
    so = str(tmp_path / "limited.so")
    subprocess.check_call([libbuild.NVCC] + libbuild.FLAGS + ["-D" + d for d in defines]
                          + ["-o", so, os.path.join(libbuild.CSRC, "blocks.cu")])
    lib, real = ctypes.CDLL(so), psispec.lib()
    for f in ("psispec_attend_tree", "psispec_attend_tree_workspace"):
        getattr(lib, f).argtypes, getattr(lib, f).restype = getattr(real, f).argtypes, getattr(real, f).restype
    return lib


def test_attend_tree_waits_that_run_out(tmp_path, monkeypatch):
    """With node tiles that are never handed over and waits of 2^22 cycles (two milliseconds) the kernels end,
    copies in flight or not, with every row of the requests NaN and the rows behind them as they were, those
    included that were written at once or by CTAs that had no node tile. The next call on the same
    workspace is right."""
    lib = limited_library(tmp_path, "PSISPEC_ATTEND_WAIT_CYCLES=(1ll<<22)", "PSISPEC_ATTEND_HAND_OVER=0")
    for lens, ctx, prefix, heads in (([5, 1, 12], [300, 0, 2000], 33, (4, 2, 64)), ([64, 33, 61], [100, 700, 0], 500, (8, 2, 128)),
                                     ([1] * 9, [3000] * 9, 64, (8, 2, 64)), ([40] * 90, [200] * 90, 0, (8, 2, 64))):
        p = Problem(lens, ctx, prefix, *heads, 16, torch.bfloat16, 91)
        n, pad = sum(lens), 3
        p.q, p.kn, p.vn = (torch.cat([t, torch.full_like(t[:pad], NAN)]) for t in (p.q, p.kn, p.vn))
        p.parent += [0] * pad
        out = torch.full((n + pad, heads[0], heads[2]), 3.0, dtype=torch.bfloat16, device=DEV)
        lse, ws = torch.full((n + pad, heads[0]), 3.0, device=DEV), torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
        with monkeypatch.context() as m:
            m.setattr(psispec, "_lib", lib)
            p.call(out=out, lse=lse, ws=ws)
            torch.cuda.synchronize()
        assert torch.isnan(out[:n]).all() and torch.isnan(lse[:n]).all()
        assert (out[n:] == 3.0).all() and (lse[n:] == 3.0).all()
        p.check(p.call(out=out, lse=lse, ws=ws))
        assert (out[n:] == 3.0).all() and (lse[n:] == 3.0).all()


def test_attend_tree_depth(tmp_path, monkeypatch):
    """A node with more ancestors than the limit is a data error of its rows (here beyond 200, of one chain by
    parents across tiles and of a shallow trie of as many nodes); a chain without parents has no limit."""
    lib = limited_library(tmp_path, "PSISPEC_ATTEND_MAX_DEPTH=200")
    n = 450
    chain = [i - 1 for i in range(n)]
    shallow = [-1] + [(i - 1) // 2 for i in range(1, n)]
    p = Problem([n, n, 40], [30, 0, 300], 50, 4, 2, 64, 16, torch.bfloat16, 92, parents=chain + shallow + chain[:40])
    with monkeypatch.context() as m:
        m.setattr(psispec, "_lib", lib)
        r = p.call()
        torch.cuda.synchronize()
    assert torch.isnan(r["out"][201:n]).all() and torch.isnan(r["lse"][201:n]).all()
    p.check(r, rows={0: slice(0, 201)})
    p.check()
    p.parent = None
    with monkeypatch.context() as m:
        m.setattr(psispec, "_lib", lib)
        p.check()


def test_attend_tree_long_segments_are_waited_for(tmp_path, monkeypatch):
    """Parts of the kernel that run ahead wait while whole segments are worked on, so a wait's limit has to grow
    with the work: with waits of 2^16 cycles, several items of 16384 tokens per block (128 tiles of more than a
    thousand cycles each) are right all the same."""
    lib = limited_library(tmp_path, "PSISPEC_ATTEND_WAIT_CYCLES=(1ll<<16)")
    g = torch.Generator(DEV).manual_seed(93)
    B, Hq, Hkv, D, page, ctx = 111, 16, 8, 64, 64, 16384
    q, k, v = (torch.randn(B, h, D, generator=g, device=DEV).bfloat16() for h in (Hq, Hkv, Hkv))
    kc, vc = (torch.randn(512, page, Hkv, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    table = torch.randint(0, 512, (B, ctx // page), generator=g, device=DEV, dtype=torch.int32)
    args = [q, k, v, offsets([1] * B), None, kc, vc, table, i32([ctx] * B)]
    want = psispec.attend_tree(*args)
    with monkeypatch.context() as m:
        m.setattr(psispec, "_lib", lib)
        got = psispec.attend_tree(*args)
        torch.cuda.synchronize()
    assert torch.isfinite(want["out"]).all()
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
