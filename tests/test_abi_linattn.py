"""The linear-attention and group-norm entry points on the CPU: what they
refuse, before anything is launched (fake pointers, launch hook set)."""

import ctypes
import os

import pytest

from gated_delta_rule_79_amd import _lib

A = 0x10000
F32, BF16 = _lib.GDN_F32, _lib.GDN_BF16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libgdn.so not built")
    lib = _lib.load()
    lib.gdn_test_set_fail_launch(1)
    yield lib
    lib.gdn_test_set_fail_launch(0)


def prob(**kw):
    p = _lib.GdnProblem()
    d = dict(B=1, T=640, H=4, dk=128, dv=64, chunk=0, nseq=0, cu_seqlens=None, io_dtype=BF16,
             gate_dtype=7, gate=_lib.GDN_GATE_NONE, seg_chunks=0)
    d.update(kw)
    for k, v in d.items():
        setattr(p, k, v)
    return p


def need(fn, p, *args):
    n = ctypes.c_size_t(0)
    return fn(ctypes.byref(p), *args, ctypes.byref(n)), n.value


FWD = ["q", "k", "v", "log_decay", "s0", "o", "sf"]
BWD = ["q", "k", "v", "log_decay", "s0", "do", "dsf", "dq", "dk", "dv", "ds0"]
STEP = ["q", "k", "v", "log_decay", "state", "o"]


def call(lib, which, p, hq=2, ws=A, short=0, **ptr):
    names, fn = {"fwd": (FWD, lib.gdn_linear_attn_fwd), "bwd": (BWD, lib.gdn_linear_attn_bwd),
                 "step": (STEP, lib.gdn_linear_attn_decode_step)}[which]
    args = [ptr.get(n, A) for n in names]
    if which == "step":
        return fn(ctypes.byref(p), hq, *args, None)
    query = getattr(lib, f"gdn_linear_attn_{which}_workspace")
    _, n = need(query, p, hq)
    return fn(ctypes.byref(p), hq, *args, ws, n - short, None)


@pytest.mark.parametrize("which", ["fwd", "bwd", "step"])
def test_valid_calls_reach_the_launch(lib, which):
    assert call(lib, which, prob()) == _lib.GDN_ERR_HIP
    assert call(lib, which, prob(io_dtype=F32), hq=4) == _lib.GDN_ERR_HIP
    assert call(lib, which, prob(), log_decay=None) == _lib.GDN_ERR_HIP


@pytest.mark.parametrize("kw,hq,status", [
    (dict(gate=_lib.GDN_GATE_SCALAR), 2, _lib.GDN_ERR_UNSUPPORTED),
    (dict(gate=9), 2, _lib.GDN_ERR_UNSUPPORTED),
    (dict(io_dtype=2), 2, _lib.GDN_ERR_DTYPE),
    (dict(dk=48), 2, _lib.GDN_ERR_UNSUPPORTED),
    (dict(dk=256), 2, _lib.GDN_ERR_UNSUPPORTED),
    (dict(dv=24), 2, _lib.GDN_ERR_UNSUPPORTED),
    (dict(dv=272), 2, _lib.GDN_ERR_UNSUPPORTED),
    (dict(B=0), 2, _lib.GDN_ERR_SHAPE),
    (dict(H=0), 1, _lib.GDN_ERR_SHAPE),
    (dict(), 0, _lib.GDN_ERR_SHAPE),
    (dict(), -4, _lib.GDN_ERR_SHAPE),
    (dict(), 3, _lib.GDN_ERR_SHAPE),
    (dict(), 8, _lib.GDN_ERR_SHAPE),
    (dict(H=1 << 18, T=1), 1, _lib.GDN_ERR_UNSUPPORTED),
])
@pytest.mark.parametrize("which", ["fwd", "bwd", "step"])
def test_problem_refusals(lib, which, kw, hq, status):
    assert call(lib, which, prob(**kw), hq=hq) == status
    if which != "step":
        assert need(getattr(lib, f"gdn_linear_attn_{which}_workspace"), prob(**kw), hq)[0] == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), _lib.GDN_ERR_SHAPE),
    (dict(nseq=-1), _lib.GDN_ERR_SHAPE),
    (dict(nseq=2, B=2, cu_seqlens=A), _lib.GDN_ERR_SHAPE),
    (dict(nseq=2), _lib.GDN_ERR_NULL),
    (dict(cu_seqlens=A), _lib.GDN_ERR_SHAPE),
    (dict(nseq=2, cu_seqlens=A + 2), _lib.GDN_ERR_ALIGN),
    (dict(T=(1 << 30) + 1), _lib.GDN_ERR_SHAPE),
    (dict(T=1 << 30, H=4096, B=64), _lib.GDN_ERR_SHAPE),
    (dict(T=1 << 28, H=512, seg_chunks=1), _lib.GDN_ERR_SHAPE),
])
@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_packing_refusals(lib, which, kw, status):
    assert call(lib, which, prob(**kw)) == status


@pytest.mark.parametrize("which,names", [
    ("fwd", ["q", "k", "v", "o"]), ("bwd", ["q", "k", "v", "do", "dq", "dk", "dv"]),
    ("step", ["q", "k", "v", "state", "o"])])
def test_pointer_refusals(lib, which, names):
    for n in names:
        assert call(lib, which, prob(), **{n: None}) == _lib.GDN_ERR_NULL, n
        assert call(lib, which, prob(), **{n: A + 8}) == _lib.GDN_ERR_ALIGN, n
    assert call(lib, which, prob(), log_decay=A + 4) == _lib.GDN_ERR_ALIGN
    for n in {"fwd": ["s0", "sf"], "bwd": ["s0", "dsf", "ds0"], "step": []}[which]:
        assert call(lib, which, prob(), **{n: None}) == _lib.GDN_ERR_HIP, n
        assert call(lib, which, prob(), **{n: A + 4}) == _lib.GDN_ERR_ALIGN, n


def test_null_problem_and_size(lib):
    n = ctypes.c_size_t(0)
    for w in ("fwd", "bwd"):
        q = getattr(lib, f"gdn_linear_attn_{w}_workspace")
        assert q(None, 1, ctypes.byref(n)) == _lib.GDN_ERR_NULL
        assert q(ctypes.byref(prob()), 2, None) == _lib.GDN_ERR_NULL
    assert lib.gdn_linear_attn_decode_step(None, 1, A, A, A, A, A, A, None) == _lib.GDN_ERR_NULL


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_workspace_refusals(lib, which):
    p = prob(seg_chunks=2)
    q = getattr(lib, f"gdn_linear_attn_{which}_workspace")
    assert need(q, p, 2)[1] > 0
    assert call(lib, which, p, ws=None) == _lib.GDN_ERR_WORKSPACE
    assert call(lib, which, p, short=1) == _lib.GDN_ERR_WORKSPACE
    assert call(lib, which, p, ws=A + 8) == _lib.GDN_ERR_ALIGN
    # one walk per sequence and no shared heads: nothing to keep
    assert need(q, prob(seg_chunks=-1), 4) == (_lib.GDN_OK, 0)


def test_empty_sequence_needs_no_rows(lib):
    none = dict(q=None, k=None, v=None, o=None, do=None, dq=None, dk=None, dv=None)
    assert call(lib, "fwd", prob(T=0), **none) == _lib.GDN_ERR_HIP
    assert call(lib, "bwd", prob(T=0), **none) == _lib.GDN_ERR_HIP


def norm(lib, p, bwd, d=64, act=1, eps=1e-5, short=0, ws=A, **ptr):
    names = ["x", "z", "w", "b"] + (["dy", "dx", "dz", "dw", "db"] if bwd else ["y"])
    args = [ptr.get(n, A) for n in names]
    if not bwd:
        return lib.gdn_group_norm_fwd(ctypes.byref(p), d, act, 1, 0, eps, *args, None)
    _, n = need(lib.gdn_group_norm_bwd_workspace, p, d)
    return lib.gdn_group_norm_bwd(ctypes.byref(p), d, act, 1, 0, eps, *args, ws, n - short, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_norm_refusals(lib, bwd):
    hip = _lib.GDN_ERR_HIP
    assert norm(lib, prob(), bwd) == hip
    assert norm(lib, prob(), bwd, d=128) == hip
    assert norm(lib, prob(), bwd, d=32) == _lib.GDN_ERR_SHAPE
    assert norm(lib, prob(dv=24), bwd, d=24) == _lib.GDN_ERR_UNSUPPORTED
    assert norm(lib, prob(dv=512), bwd, d=512) == _lib.GDN_ERR_UNSUPPORTED
    assert norm(lib, prob(io_dtype=5), bwd) == _lib.GDN_ERR_DTYPE
    for kw in (dict(B=0), dict(T=-1), dict(H=0), dict(H=65536), dict(T=1 << 30, B=1 << 20)):
        assert norm(lib, prob(**kw), bwd) == _lib.GDN_ERR_SHAPE, kw
    for a in (-1, 3):
        assert norm(lib, prob(), bwd, act=a) == _lib.GDN_ERR_UNSUPPORTED
    for e in (0.0, -1.0, float("nan"), float("inf")):
        assert norm(lib, prob(), bwd, eps=e) == _lib.GDN_ERR_UNSUPPORTED
    for n in ["x"] + (["dy", "dx", "dz"] if bwd else ["y"]):
        assert norm(lib, prob(), bwd, **{n: None}) == _lib.GDN_ERR_NULL, n
        assert norm(lib, prob(), bwd, **{n: A + 2}) == _lib.GDN_ERR_ALIGN, n
    for n in ["z", "w", "b"] + (["dw", "db"] if bwd else []):
        assert norm(lib, prob(), bwd, **{n: None}) == hip, n
        assert norm(lib, prob(), bwd, **{n: A + 4}) == _lib.GDN_ERR_ALIGN, n
    if bwd:
        assert norm(lib, prob(), True, ws=None) == _lib.GDN_ERR_WORKSPACE
        assert norm(lib, prob(), True, short=1) == _lib.GDN_ERR_WORKSPACE
        assert norm(lib, prob(), True, ws=A + 8) == _lib.GDN_ERR_ALIGN
        assert norm(lib, prob(), True, z=None, dz=None) == hip


def test_log_names_the_calls(lib, capfd, monkeypatch):
    monkeypatch.setenv("GDN_LOG", "1")
    call(lib, "fwd", prob())
    norm(lib, prob(), False)
    err = capfd.readouterr().err
    assert "gdn_linear_attn_fwd: B=1 T=640 H=4 hq=2" in err
    assert "gdn_group_norm_fwd: tokens=640 H=4 d=64" in err


def test_binding_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    import gated_delta_rule_79_amd as gdn
    q, v = torch.zeros(1, 4, 2, 16), torch.zeros(1, 4, 2, 16)
    with pytest.raises(ValueError):
        gdn.linear_attn_fwd(q, q, v)          # host tensors
    with pytest.raises(ValueError):
        gdn.linear_attn_fwd(q[0], q[0], v)    # dimensions
    with pytest.raises(ValueError):
        gdn.linear_attn_decode_step(q, q, v, None, None)
    with pytest.raises(ValueError):
        gdn.group_norm_fwd(q)
    with pytest.raises(ValueError):
        gdn.group_norm_fwd(q[0])


def state_slots(lib, which, p, hq):
    """States for segments that a call's workspace has room for, of a problem
    without shared heads and dv <= 128."""
    n = need(getattr(lib, f"gdn_linear_attn_{which}_workspace"), p, hq)
    assert n[0] == _lib.GDN_OK
    return n[1] / (p.H * p.dk * p.dv * 4) / (1 if which == "fwd" else 2)


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_packed_batches_of_short_sequences_need_little(lib, which):
    # states are kept for the segments of sequences that are cut, none of six
    # chunks or fewer where there are many: a sequence that is cut has one
    # segment more than whole spans, at most twice the spans in all
    for T, nseq, H in ((2000, 24, 32), (16384, 256, 16), (16384, 256, 2), (65536, 1024, 16),
                       (4096, 24, 32), (8192, 24, 16), (900, 30, 2), (32768, 64, 16)):
        p = prob(T=T, H=H, dv=128, nseq=nseq, cu_seqlens=A)
        assert state_slots(lib, which, p, H) <= 2 * (T // (6 * 64)), (T, nseq, H)
    # a handful of chunks in all: one walk
    assert state_slots(lib, which, prob(T=448, H=16, dv=128, nseq=7, cu_seqlens=A), 16) == 0
    # few long sequences are cut as before
    p = prob(T=65536, H=16, dv=128, nseq=7, cu_seqlens=A)
    assert state_slots(lib, which, p, 16) == 28 + 7
    # segments asked for: each long sequence has its own, each short one none
    p = prob(T=640, H=4, dv=128, nseq=100, cu_seqlens=A, seg_chunks=2)
    assert state_slots(lib, which, p, 4) == 5 + 4


SMALL = dict(dk=16, dv=16, H=16, T=1)


@pytest.mark.parametrize("which,kw,hq", [
    # a launch takes fewer than 2^32 threads: 2^20 sequences of 16 heads are
    # one workgroup too many, the backward's three walks reach it earlier
    ("step", dict(SMALL, B=1 << 20), 16), ("fwd", dict(SMALL, B=1 << 20), 16),
    ("bwd", dict(SMALL, B=(1 << 20) // 3 + 1), 16),
    ("fwd", dict(SMALL, nseq=1 << 20, T=1 << 20, cu_seqlens=A), 16),
    # the wide walks of dv = 256 take 512 threads
    ("bwd", dict(SMALL, dk=128, dv=256, B=1 << 18), 16),
    # products of sizes that pass 64 bits
    ("fwd", dict(SMALL, B=1 << 28, T=1 << 28, H=1), 1),
    ("bwd", dict(SMALL, B=1 << 30, T=1 << 30, H=16), 16),
    ("fwd", dict(SMALL, nseq=(1 << 31) - 1, T=1 << 30, H=1 << 19, cu_seqlens=A), 1),
    ("step", dict(SMALL, B=(1 << 31) - 1, H=1 << 19), 1),
])
def test_sizes_past_a_launch_are_refused(lib, which, kw, hq):
    assert call(lib, which, prob(**kw), hq=hq) == _lib.GDN_ERR_SHAPE
    if which != "step":
        query = getattr(lib, f"gdn_linear_attn_{which}_workspace")
        assert need(query, prob(**kw), hq)[0] == _lib.GDN_ERR_SHAPE


@pytest.mark.parametrize("which,kw", [
    ("step", dict(SMALL, B=(1 << 20) - 1)), ("fwd", dict(SMALL, B=(1 << 20) - 1)),
    ("bwd", dict(SMALL, B=(1 << 20) // 3)), ("bwd", dict(SMALL, dk=128, dv=256, B=(1 << 18) - 1))])
def test_the_largest_launches_are_not(lib, which, kw):
    assert call(lib, which, prob(**kw), hq=16) == _lib.GDN_ERR_HIP  # the launch hook's


@pytest.mark.parametrize("which", ["fwd", "bwd"])
@pytest.mark.parametrize("nseq", [1 << 22, (1 << 23) + 1, 1 << 24, 1 << 25, (1 << 31) - 1])
def test_more_sequences_than_tokens(lib, which, nseq):
    # (the plan's own products of the number of sequences stay in 64 bits; a
    # sequence needs a workgroup even if it is empty, so past 2^24 there are
    # too many, in the backward past a third of that)
    p = prob(T=1000, H=1, dk=16, dv=16, nseq=nseq, cu_seqlens=A)
    status, _ = need(getattr(lib, f"gdn_linear_attn_{which}_workspace"), p, 1)
    fits = nseq * (3 if which == "bwd" else 1) < 1 << 24
    assert status == (_lib.GDN_OK if fits else _lib.GDN_ERR_SHAPE)
