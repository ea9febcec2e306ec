"""The selective-scan, short-convolution and draft-acceptance entry points on
the CPU: what they refuse, before anything is launched (fake pointers, launch
hook set)."""

import ctypes
import os

import pytest

from gated_delta_rule_79_amd import _lib

A = 0x10000
F32, BF16 = _lib.GDN_F32, _lib.GDN_BF16
OK, NULL, SHAPE, DTYPE = _lib.GDN_OK, _lib.GDN_ERR_NULL, _lib.GDN_ERR_SHAPE, _lib.GDN_ERR_DTYPE
UNSUPPORTED, ALIGN, WORKSPACE = _lib.GDN_ERR_UNSUPPORTED, _lib.GDN_ERR_ALIGN, _lib.GDN_ERR_WORKSPACE
HIP = _lib.GDN_ERR_HIP


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
    d = dict(B=1, T=640, H=4, dk=16, dv=70, chunk=0, nseq=0, cu_seqlens=None, io_dtype=BF16,
             gate_dtype=7, gate=_lib.GDN_GATE_NONE, seg_chunks=0)
    d.update(kw)
    for k, v in d.items():
        setattr(p, k, v)
    return p


def need(fn, p, *args):
    n = ctypes.c_size_t(0)
    return fn(ctypes.byref(p), *args, ctypes.byref(n)), n.value


IN = ["x", "dt", "a", "b", "c", "d", "bias", "z"]
SCAN = {"fwd": IN + ["s0", "y", "sf"], "step": IN + ["state", "y"],
        "bwd": IN + ["s0", "dy", "dsf", "dx", "ddt", "da", "db", "dc", "dd", "dbias", "dz", "ds0"]}


def scan(lib, which, p, hb=2, ws=A, short=0, **ptr):
    fn = getattr(lib, f"gdn_selective_scan_{which}")
    args = [ptr.get(n, A) for n in SCAN[which]]
    if which == "step":
        return fn(ctypes.byref(p), hb, 1, *args, None)
    _, n = need(getattr(lib, f"gdn_selective_scan_{which}_workspace"), p, hb)
    return fn(ctypes.byref(p), hb, 1, *args, ws, n - short, None)


@pytest.mark.parametrize("which", ["fwd", "bwd", "step"])
def test_scan_valid_calls_reach_the_launch(lib, which):
    assert scan(lib, which, prob()) == HIP
    assert scan(lib, which, prob(io_dtype=F32, dk=64, dv=1), hb=4) == HIP
    for n in ("d", "bias", "s0", "dsf", "dd", "dbias", "ds0"):
        assert scan(lib, which, prob(), **{n: None}) == HIP, n
    assert scan(lib, which, prob(), z=None, dz=None) == HIP


@pytest.mark.parametrize("kw,hb,status", [
    (dict(gate=_lib.GDN_GATE_SCALAR), 2, UNSUPPORTED), (dict(io_dtype=2), 2, DTYPE),
    (dict(dk=0), 2, UNSUPPORTED), (dict(dk=6), 2, UNSUPPORTED), (dict(dk=68), 2, UNSUPPORTED),
    (dict(dv=0), 2, SHAPE), (dict(B=0), 2, SHAPE), (dict(H=0), 1, SHAPE), (dict(), 0, SHAPE),
    (dict(), 3, SHAPE), (dict(), 8, SHAPE), (dict(H=1 << 12, dv=1 << 12), 1, UNSUPPORTED),
    (dict(H=1 << 30, dv=1 << 30), 1, UNSUPPORTED)])
@pytest.mark.parametrize("which", ["fwd", "bwd", "step"])
def test_scan_problem_refusals(lib, which, kw, hb, status):
    assert scan(lib, which, prob(**kw), hb=hb) == status
    if which != "step":
        assert need(getattr(lib, f"gdn_selective_scan_{which}_workspace"), prob(**kw), hb)[0] == status


@pytest.mark.parametrize("which", ["fwd", "bwd", "step"])
def test_scan_rows_of_b_and_c_are_bounded(lib, which):
    # eight of them are addressed with 32 bits
    p = prob(T=1, H=1 << 20, dv=1, dk=16)
    assert scan(lib, which, p, hb=1 << 20) == HIP
    p.dk = 20
    assert scan(lib, which, p, hb=1 << 20) == UNSUPPORTED
    assert scan(lib, which, p, hb=1 << 10) == HIP


def test_sequences_are_bounded(lib):
    p = prob(T=5, H=1, dk=4, dv=1, nseq=(1 << 29) + 1, cu_seqlens=A)
    assert scan(lib, "fwd", p, hb=1) == SHAPE and scan(lib, "bwd", p, hb=1) == SHAPE
    assert conv(lib, "fwd", p) == SHAPE and conv(lib, "bwd", p) == SHAPE


PACKING = [(dict(T=-1), SHAPE), (dict(nseq=-1), SHAPE), (dict(nseq=2, B=2, cu_seqlens=A), SHAPE),
           (dict(nseq=2), NULL), (dict(cu_seqlens=A), SHAPE),
           (dict(nseq=2, cu_seqlens=A + 2), ALIGN), (dict(T=(1 << 30) + 1), SHAPE),
           (dict(T=1 << 30, B=64, H=1 << 10, dv=1 << 10), SHAPE)]


@pytest.mark.parametrize("kw,status", PACKING + [
    (dict(T=1 << 28, H=512, dv=512, seg_chunks=1), SHAPE)])
@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_scan_packing_refusals(lib, which, kw, status):
    assert scan(lib, which, prob(**kw)) == status


@pytest.mark.parametrize("which", ["fwd", "bwd", "step"])
def test_scan_pointer_refusals(lib, which):
    free = {"d", "bias", "z", "s0", "sf", "dsf", "dd", "dbias", "ds0"}
    for n in SCAN[which]:
        assert scan(lib, which, prob(), **{n: A + 8}) == ALIGN, n
        if n not in free:
            assert scan(lib, which, prob(), **{n: None}) == NULL, n


def test_scan_workspace(lib):
    for which in ("fwd", "bwd"):
        p = prob(seg_chunks=2)
        q = getattr(lib, f"gdn_selective_scan_{which}_workspace")
        assert need(q, p, 2)[1] > 0
        assert scan(lib, which, p, ws=None) == WORKSPACE
        assert scan(lib, which, p, short=1) == WORKSPACE
        assert scan(lib, which, p, ws=A + 8) == ALIGN
        assert q(None, 1, ctypes.byref(ctypes.c_size_t(0))) == NULL
        assert q(ctypes.byref(p), 2, None) == NULL
    assert need(lib.gdn_selective_scan_fwd_workspace, prob(seg_chunks=-1), 2) == (OK, 0)


def test_scan_empty_sequences_need_no_rows(lib):
    rows = {n: None for n in ("x", "dt", "b", "c", "z", "y", "dy", "dx", "ddt", "db", "dc", "dz")}
    for which in ("fwd", "bwd"):
        assert scan(lib, which, prob(T=0), **rows) == HIP


CONV = {"fwd": ["x", "taps", "bias", "s0", "y", "sf"], "step": ["x", "taps", "bias", "state", "y"],
        "bwd": ["x", "taps", "bias", "s0", "dy", "dsf", "dx", "dtaps", "dbias", "ds0"]}


def conv(lib, which, p, width=4, act=1, ws=A, short=0, **ptr):
    fn = getattr(lib, f"gdn_short_conv_{which}")
    args = [ptr.get(n, A) for n in CONV[which]]
    if which == "bwd":
        args += [ws, need(lib.gdn_short_conv_bwd_workspace, p, width)[1] - short]
    return fn(ctypes.byref(p), width, act, *args, None)


@pytest.mark.parametrize("which", ["fwd", "bwd", "step"])
def test_conv_refusals(lib, which):
    assert conv(lib, which, prob()) == HIP
    assert conv(lib, which, prob(dk=3, gate=9), width=1, state=None) == HIP
    for kw, status in ((dict(io_dtype=2), DTYPE), (dict(B=0), SHAPE), (dict(H=0), SHAPE),
                       (dict(dv=0), SHAPE), (dict(H=1 << 12, dv=1 << 12), UNSUPPORTED)):
        assert conv(lib, which, prob(**kw)) == status, kw
    for kw in (dict(width=0), dict(width=9), dict(act=-1), dict(act=3)):
        assert conv(lib, which, prob(), **kw) == UNSUPPORTED, kw
    if which != "step":
        for kw, status in PACKING:
            assert conv(lib, which, prob(**kw)) == status, kw
    for n in CONV[which]:
        assert conv(lib, which, prob(), **{n: A + 8}) == ALIGN, n
        free = n in ("bias", "s0", "sf", "dsf", "dbias", "ds0")
        assert conv(lib, which, prob(), **{n: None}) == (HIP if free else NULL), n


def test_conv_workspace(lib):
    p = prob()
    assert conv(lib, "bwd", p, ws=None) == WORKSPACE
    assert conv(lib, "bwd", p, short=1) == WORKSPACE
    assert conv(lib, "bwd", p, ws=A + 8) == ALIGN
    assert lib.gdn_short_conv_bwd_workspace(None, 4, ctypes.byref(ctypes.c_size_t(0))) == NULL
    assert lib.gdn_short_conv_bwd_workspace(ctypes.byref(p), 4, None) == NULL


ACCEPT = ["parent", "tokens", "target", "draft", "uniform", "accepted", "length", "next"]


def accept(lib, p, vocab=1000, ws=A, short=0, **ptr):
    args = [ptr.get(n, A) for n in ACCEPT]
    _, n = need(lib.gdn_draft_accept_workspace, p, vocab, int(args[0] is not None))
    return lib.gdn_draft_accept(ctypes.byref(p), vocab, *args, ws, max(n - short, 0), None)


def test_accept_refusals(lib):
    p = prob(T=64)
    assert accept(lib, p) == HIP and accept(lib, p, parent=None) == HIP
    assert accept(lib, p, draft=None) == HIP
    assert accept(lib, prob(T=0), tokens=None) == HIP
    assert accept(lib, prob(T=1000, nseq=50, cu_seqlens=A)) == HIP
    for kw, status in ((dict(io_dtype=2), DTYPE), (dict(B=0), SHAPE), (dict(T=65), SHAPE),
                       (dict(B=(1 << 20) + 1), SHAPE)):
        assert accept(lib, prob(**{**dict(T=4), **kw})) == status, kw
    for kw, status in PACKING[:7]:
        assert accept(lib, prob(**kw)) == status, kw
    for vocab in (0, -3, (1 << 28) + 1):
        assert accept(lib, p, vocab=vocab) == SHAPE
    for n in ACCEPT:
        assert accept(lib, p, **{n: A + 8}) == ALIGN, n
        assert accept(lib, p, **{n: None}) == (HIP if n in ("parent", "draft") else NULL), n
    assert accept(lib, p, vocab=1001, parent=None, ws=None) == WORKSPACE
    assert accept(lib, p, vocab=1 << 16, parent=None, short=1) == WORKSPACE
    assert accept(lib, p, parent=None, ws=None) == HIP  # nor do chains of rows that fit a CU
    assert accept(lib, p, parent=None, ws=A + 8) == ALIGN
    assert accept(lib, p, ws=None) == HIP  # a tree takes none
    assert lib.gdn_draft_accept_workspace(None, 5, 0, ctypes.byref(ctypes.c_size_t(0))) == NULL
    assert lib.gdn_draft_accept_workspace(ctypes.byref(p), 5, 0, None) == NULL
