"""Host-side checks of the operators around a drafted block (verification from probabilities,
trie attention, cache commit): what the entry points refuse before anything reaches a GPU, and the
sizes they ask for. No device needed."""
import ctypes

import pytest
import torch

from lossless_speculative_sampling_b200 import build as libbuild
from lossless_speculative_sampling_b200 import psispec

FAKE = 4096  # aligned, never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return psispec.lib()


def _probs(L, **kw):
    a = dict(t=FAKE, ts=100, d=FAKE, ds=100, dtype=psispec.F32, B=2, N=5, V=100, off=FAKE, x=FAKE, ua=FAKE, ur=FAKE,
             ot=FAKE, ol=FAKE)
    a.update(kw)
    return L.psispec_verify_probs(a["t"], a["ts"], a["d"], a["ds"], a["dtype"], a["B"], a["N"], a["V"], a["off"], a["x"],
                                  a["ua"], a["ur"], a["ot"], a["ol"], None)


@pytest.mark.parametrize("bad", [dict(t=None), dict(off=None), dict(ur=None), dict(ot=None), dict(ol=None), dict(x=None),
                                 dict(ua=None), dict(B=0), dict(N=-1), dict(V=0), dict(ts=99), dict(ds=99), dict(dtype=5),
                                 dict(dtype=psispec.F16), dict(t=FAKE + 2), dict(d=FAKE + 2), dict(off=FAKE + 2),
                                 dict(x=FAKE + 1), dict(ua=FAKE + 2), dict(ur=FAKE + 3), dict(ot=FAKE + 2), dict(ol=FAKE + 2)])
def test_verify_probs_refuses(L, bad):
    assert _probs(L, **bad) == psispec.ERR_INVALID_ARG


@pytest.mark.parametrize("big", [dict(V=(1 << 24) + 1, ts=1 << 25, ds=1 << 25), dict(N=1 << 26),
                                 dict(ts=(1 << 32) + 1)])
def test_verify_probs_limits(L, big):
    assert _probs(L, **big) == psispec.ERR_UNSUPPORTED


def _attend(**kw):
    a = psispec.AttendTreeArgs()
    for k, v in dict(dtype=psispec.BF16, B=2, N=10, Hq=8, Hkv=2, D=64, pages=4, page_size=16, max_pages=2, prefix_pages=0,
                     scale=0.125, q=FAKE, k_nodes=FAKE, v_nodes=FAKE, k_cache=FAKE, v_cache=FAKE, node_offsets=FAKE,
                     parent=FAKE, page_table=FAKE, context_len=FAKE, out=FAKE, out_lse=FAKE).items():
        setattr(a, k, v)
    a.q_stride[:] = (512, 64)
    a.kn_stride[:] = a.vn_stride[:] = (128, 64)
    a.kc_stride[:] = a.vc_stride[:] = (2048, 128, 64)
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(k_nodes=None), dict(v_nodes=None), dict(k_cache=None), dict(v_cache=None), dict(node_offsets=None),
    dict(page_table=None), dict(context_len=None), dict(out=None), dict(dtype=psispec.F32), dict(dtype=7), dict(B=0),
    dict(N=0), dict(Hq=0), dict(Hkv=3), dict(D=0), dict(D=60), dict(pages=0), dict(page_size=12), dict(page_size=0),
    dict(max_pages=0), dict(prefix_pages=-1), dict(prefix_pages=2), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(q=FAKE + 2), dict(v_cache=FAKE + 8), dict(out=FAKE + 4),
    dict(q_stride=(512, 60)), dict(q_stride=(512, 56)), dict(q_stride=(0, 64)), dict(kn_stride=(-128, 64)),
    dict(kc_stride=(2048, 132, 64)), dict(vc_stride=(1 << 39, 128, 64)), dict(out_lse=FAKE + 2), dict(node_offsets=FAKE + 2),
    dict(parent=FAKE + 2), dict(page_table=FAKE + 1), dict(context_len=FAKE + 2),
    dict(prefix_pages=1, prefix_table=FAKE + 2, prefix_len=FAKE), dict(prefix_pages=1, prefix_table=FAKE, prefix_len=FAKE + 2)])
def test_attend_tree_refuses(L, bad):
    a = _attend(**bad)
    assert L.psispec_attend_tree(a, FAKE, 1 << 40, None) == psispec.ERR_INVALID_ARG
    assert L.psispec_attend_tree_workspace(a) == 0


@pytest.mark.parametrize("big", [dict(D=136, q_stride=(2048, 136), kn_stride=(512, 136), vn_stride=(512, 136),
                                      kc_stride=(8192, 512, 136), vc_stride=(8192, 512, 136)),
                                 dict(Hq=258, Hkv=2, q_stride=(1 << 20, 64)), dict(N=1 << 24),
                                 dict(max_pages=1 << 28)])
def test_attend_tree_limits(L, big):
    assert L.psispec_attend_tree(_attend(**big), FAKE, 1 << 40, None) == psispec.ERR_UNSUPPORTED


def test_attend_tree_null_args_and_workspace(L):
    assert L.psispec_attend_tree(None, FAKE, 1 << 40, None) == psispec.ERR_INVALID_ARG
    assert L.psispec_attend_tree_workspace(None) == 0
    a = _attend()
    need = L.psispec_attend_tree_workspace(a)
    assert need > 0
    assert L.psispec_attend_tree(a, None, need, None) == psispec.ERR_WORKSPACE
    assert L.psispec_attend_tree(a, FAKE, need - 1, None) == psispec.ERR_WORKSPACE
    assert L.psispec_attend_tree(a, FAKE + 128, need, None) == psispec.ERR_WORKSPACE


def _commit(**kw):
    a = psispec.CommitTreeArgs()
    for k, v in dict(dtype=psispec.BF16, L=2, B=2, N=10, Hkv=2, D=64, pages=4, page_size=16, max_pages=2, max_depth=4,
                     k_nodes=FAKE, v_nodes=FAKE, k_cache=FAKE, v_cache=FAKE, node_offsets=FAKE, path=FAKE, accept_len=FAKE,
                     page_table=FAKE, context_len=FAKE, out_context_len=2 * FAKE).items():
        setattr(a, k, v)
    a.kn_stride[:] = a.vn_stride[:] = (1280, 128, 64)
    a.kc_stride[:] = a.vc_stride[:] = (8192, 2048, 128, 64)
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(k_nodes=None), dict(v_nodes=None), dict(k_cache=None), dict(v_cache=None), dict(node_offsets=None),
    dict(accept_len=None), dict(page_table=None), dict(context_len=None), dict(out_context_len=None),
    dict(out_context_len=FAKE), dict(dtype=psispec.F32), dict(L=0), dict(B=0), dict(N=0), dict(Hkv=0), dict(D=12),
    dict(pages=0), dict(page_size=0), dict(max_pages=0), dict(max_depth=0), dict(k_cache=FAKE + 2),
    dict(kn_stride=(1280, 128, 60)), dict(vc_stride=(8192, 2048, 0, 64))])
def test_commit_tree_refuses(L, bad):
    assert L.psispec_commit_tree(_commit(**bad), None) == psispec.ERR_INVALID_ARG


def test_commit_tree_limits(L):
    assert L.psispec_commit_tree(None, None) == psispec.ERR_INVALID_ARG
    assert L.psispec_commit_tree(_commit(L=1025), None) == psispec.ERR_UNSUPPORTED
    assert L.psispec_commit_tree(_commit(max_pages=1 << 28), None) == psispec.ERR_UNSUPPORTED


def test_structs_match_the_header():
    """Field names and their order, read from the header's declarations."""
    import re

    with open(psispec.HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    for name, cls in (("psispec_attend_tree_args", psispec.AttendTreeArgs),
                      ("psispec_commit_tree_args", psispec.CommitTreeArgs)):
        body = [m for m in re.findall(r"typedef struct \{(.*?)\} (\w+);", text, flags=re.S) if m[1] == name][0][0]
        got = []
        for line in body.split(";"):
            words = line.replace("const", " ").replace("*", " ").split(None, 1)
            if len(words) == 2:
                got += [re.sub(r"\[\d+\]", "", w).strip() for w in words[1].split(",")]
        assert got == [f[0] for f in cls._fields_]
    assert psispec._ATTEND_PACK.size == ctypes.sizeof(psispec.AttendTreeArgs)
    assert psispec._COMMIT_PACK.size == ctypes.sizeof(psispec.CommitTreeArgs)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(3, 8)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        psispec.verify_probs(x, None, i, i, x, x)
    h = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        psispec.attend_tree(h, h, h, i, None, h, h, i, i)
    with pytest.raises(TypeError):
        psispec.commit_tree(h, h, i, None, i, h, h, i, i)


def test_binding_refuses_a_stream_of_another_device():
    """The kernels would run on that device, with addresses of the tensors' one."""
    class Stream:
        cuda_stream, device = 4096, torch.device("cuda", 1)

    with pytest.raises(ValueError):
        psispec._on(torch.device("cuda", 0), Stream())


@pytest.mark.parametrize("scale", [3.0e38, 2.4e38])
def test_attend_tree_refuses_scales_without_a_finite_logarithm_to_base_2(L, scale):
    """Scores are kept in units of log 2: scale * log2(e) has to be finite too."""
    a = _attend(scale=scale)
    assert L.psispec_attend_tree(a, FAKE, 1 << 40, None) == psispec.ERR_INVALID_ARG
    assert L.psispec_attend_tree_workspace(a) == 0
    assert L.psispec_attend_tree_workspace(_attend(scale=2.0 ** 127)) > 0
