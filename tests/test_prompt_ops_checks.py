"""Refusals of gqa_score_decode, gqa_prefill, pages_fork and pages_compact (no GPU: every call fails before any CUDA
call, or does not reach the device)."""
import ctypes

import pytest
import torch

import mqa_decode_attention_paged_gb300 as pkg
from mqa_decode_attention_paged_gb300 import _binding as mqa

FAKE = 0x10000  # aligned, never dereferenced: validation fails first
INV, UNS, SMALL = mqa.ERR_INVALID_ARG, mqa.ERR_UNSUPPORTED, mqa.ERR_WORKSPACE_TOO_SMALL
NAN, INF = float("nan"), float("inf")


def P(v):
    return None if v is None else ctypes.c_void_p(v)


def _score(**kw):
    a = dict(q=FAKE, kv=FAKE, sc=None, bt=FAKE, sl=FAKE, scale=0.1, ks=1.0, vs=1.0, cap=50.0, slopes=FAKE, window=128,
             sinks=4, out=FAKE, lse=None, B=2, L=1, Hq=8, Hkv=2, D=128, nb=10, P=16, maxb=8, G=16, kvd=0, S=1, ws=None,
             wsb=0, st=None)
    a.update(kw)
    return mqa.lib.gqa_score_decode(P(a["q"]), P(a["kv"]), P(a["sc"]), P(a["bt"]), P(a["sl"]), a["scale"], a["ks"],
                                    a["vs"], a["cap"], P(a["slopes"]), a["window"], a["sinks"], P(a["out"]), P(a["lse"]),
                                    a["B"], a["L"], a["Hq"], a["Hkv"], a["D"], a["nb"], a["P"], a["maxb"], a["G"],
                                    a["kvd"], a["S"], P(a["ws"]), a["wsb"], P(a["st"]), None)


CAPS = [(dict(cap=-1.0), INV), (dict(cap=NAN), INV), (dict(cap=INF), INV), (dict(cap=1e-9), INV), (dict(cap=1e20), INV),
        (dict(slopes=FAKE + 2), INV)]


@pytest.mark.parametrize("kw,code", CAPS + [
    (dict(q=None), INV), (dict(out=FAKE + 2), INV), (dict(B=0), INV), (dict(window=0), INV), (dict(D=96), UNS),
    (dict(Hq=34), UNS), (dict(P=24), UNS), (dict(kvd=2), UNS), (dict(kvd=5), INV), (dict(S=4), SMALL)])
def test_score_validation(kw, code):
    assert _score(**kw) == code


def _prefill(**kw):
    a = dict(q=FAKE, kv=FAKE, sc=None, bt=FAKE, sl=FAKE, qs=FAKE, pre=None, scale=0.1, ks=1.0, vs=1.0, cap=0.0,
             slopes=None, window=128, sinks=4, out=FAKE, lse=None, T=5, B=2, Hq=8, Hkv=2, D=128, nb=10, P=16, maxb=8,
             G=16, kvd=0, stride=1024, S=1, ws=None, wsb=0, st=None)
    a.update(kw)
    return mqa.lib.gqa_prefill(P(a["q"]), P(a["kv"]), P(a["sc"]), P(a["bt"]), P(a["sl"]), P(a["qs"]), P(a["pre"]),
                               a["scale"], a["ks"], a["vs"], a["cap"], P(a["slopes"]), a["window"], a["sinks"],
                               P(a["out"]), P(a["lse"]), a["T"], a["B"], a["Hq"], a["Hkv"], a["D"], a["nb"], a["P"],
                               a["maxb"], a["G"], a["kvd"], a["stride"], a["S"], P(a["ws"]), a["wsb"], P(a["st"]), None)


@pytest.mark.parametrize("kw,code", CAPS + [
    (dict(q=None), INV), (dict(kv=None), INV), (dict(bt=None), INV), (dict(sl=None), INV), (dict(qs=None), INV),
    (dict(out=None), INV), (dict(q=FAKE + 8), INV), (dict(kv=FAKE + 8), INV), (dict(out=FAKE + 8), INV),
    (dict(bt=FAKE + 2), INV), (dict(qs=FAKE + 2), INV), (dict(pre=FAKE + 1), INV), (dict(lse=FAKE + 2), INV),
    (dict(st=FAKE + 2), INV), (dict(T=-1), INV), (dict(B=0), INV), (dict(Hq=0), INV), (dict(Hq=9), INV),
    (dict(nb=0), INV), (dict(maxb=0), INV), (dict(P=0), INV), (dict(S=0), INV), (dict(window=0), INV),
    (dict(sinks=-1), INV), (dict(scale=NAN), INV), (dict(kvd=1, ks=INF), INV), (dict(kvd=1, vs=NAN), INV),
    (dict(stride=1020), INV), (dict(stride=1016), INV), (dict(stride=-1024), INV),
    (dict(D=96), UNS), (dict(Hq=129, Hkv=129, stride=1 << 20), UNS), (dict(Hq=129, Hkv=1, stride=1 << 20), UNS),
    (dict(P=24), UNS), (dict(T=(1 << 24) + 1), UNS), (dict(B=8193), UNS), (dict(kvd=2), UNS), (dict(kvd=9), UNS),
    (dict(nb=1 << 26), UNS), (dict(maxb=1 << 26), UNS), (dict(kvd=5), INV), (dict(kvd=6, sc=FAKE, G=0), INV),
    (dict(kvd=6, sc=FAKE, G=24, P=48), UNS), (dict(kvd=6, sc=FAKE, G=32), UNS), (dict(S=2), SMALL)])
def test_prefill_validation(kw, code):
    assert _prefill(**kw) == code


@pytest.mark.parametrize("kw", [
    dict(), dict(out=FAKE + 4 * 2048 + 2032), dict(out=FAKE - 5 * 2048 + 16), dict(out=FAKE + 0x100000, lse=FAKE + 0x100000 + 5 * 2048 - 4),
    dict(out=FAKE + 0x100000, lse=FAKE + 16), dict(out=FAKE + 0x100000, S=2, ws=FAKE + 9216, wsb=1 << 30),
    dict(out=FAKE + 0x100000, stride=2048, lse=FAKE + 4 * 4096 + 2044)])
def test_prefill_overlap(kw):
    """A row of q is read while results of others are written."""
    assert _prefill(**kw) == INV


def test_prefill_workspace_sizes():
    assert mqa.gqa_prefill_workspace_bytes(9, 2, 128) == 0 and mqa.gqa_prefill_workspace_bytes(8, 2, 96) == 0


def _words(*v):
    return (ctypes.c_uint64 * max(1, len(v)))(*v)


def _fork(**kw):
    a = dict(bt=FAKE, sl=FAKE, pa=FAKE, refs=FAKE, nt=FAKE + 0x100000, nl=FAKE + 0x200000, nr=FAKE + 0x300000, R=4, N=8,
             maxb=8, nb=100, P=16, caches=[FAKE + 0x1000000], sizes=[4096], ws=None, wsb=0, st=None)
    a.update(kw)
    return mqa.lib.mqa_pages_fork(P(a["bt"]), P(a["sl"]), P(a["pa"]), P(a["refs"]), P(a["nt"]), P(a["nl"]), P(a["nr"]),
                                  a["R"], a["N"], a["maxb"], a["nb"], a["P"],
                                  None if a["caches"] is None else _words(*a["caches"]), _words(*a["sizes"]),
                                  a.get("n", len(a["sizes"])), P(a["ws"]), a["wsb"], P(a["st"]), None)


def _compact(**kw):
    a = dict(bt=FAKE, sl=FAKE, refs=FAKE, nt=FAKE + 0x100000, nr=FAKE + 0x200000, mv=FAKE + 0x300000, nl=FAKE + 0x400000,
             R=4, maxb=8, nb=100, P=16, caches=[FAKE + 0x1000000], sizes=[4096], ws=None, wsb=0, st=None)
    a.update(kw)
    return mqa.lib.mqa_pages_compact(P(a["bt"]), P(a["sl"]), P(a["refs"]), P(a["nt"]), P(a["nr"]), P(a["mv"]), P(a["nl"]),
                                     a["R"], a["maxb"], a["nb"], a["P"],
                                     None if a["caches"] is None else _words(*a["caches"]), _words(*a["sizes"]),
                                     a.get("n", len(a["sizes"])), P(a["ws"]), a["wsb"], P(a["st"]), None)


CACHES = [
    (dict(caches=None), INV), (dict(caches=[0]), INV), (dict(caches=[FAKE + 0x1000008]), INV), (dict(n=-1), INV),
    (dict(sizes=[0]), INV), (dict(sizes=[4098]), UNS), (dict(sizes=[(1 << 30) + 4]), UNS),
    (dict(caches=[FAKE + 0x1000000] * 257, sizes=[4096] * 257), UNS),
    (dict(caches=[FAKE + 0x1000000, FAKE + 0x1000000], sizes=[4096, 4096]), INV),   # one tensor twice
    (dict(caches=[FAKE + 0x1000000, FAKE + 0x1000000 + 99 * 4096], sizes=[4096, 4096]), INV),
    (dict(caches=[FAKE + 0x1000000, FAKE + 0x1000000 + 100 * 4096], sizes=[4096, 4096]), SMALL)]
SIZES = [(dict(bt=None), INV), (dict(sl=None), INV), (dict(refs=None), INV), (dict(nt=None), INV), (dict(nr=None), INV),
         (dict(bt=FAKE + 2), INV), (dict(st=FAKE + 2), INV), (dict(R=0), INV), (dict(maxb=0), INV), (dict(nb=0), INV),
         (dict(P=0), INV), (dict(P=24), UNS), (dict(R=8193), UNS), (dict(maxb=1 << 27), UNS), (dict(), SMALL),
         (dict(ws=FAKE, wsb=16), SMALL), (dict(ws=FAKE + 4, wsb=1 << 20), INV)]


@pytest.mark.parametrize("kw,code", CACHES + SIZES + [
    (dict(pa=None), INV), (dict(nl=None), INV), (dict(N=0), INV), (dict(N=8193), UNS),
    (dict(nt=FAKE), INV), (dict(nt=FAKE + 64), INV), (dict(nl=FAKE + 4), INV), (dict(nr=FAKE + 4), INV),
    (dict(nr=FAKE), SMALL)])  # in place
def test_fork_validation(kw, code):
    assert _fork(**kw) == code


@pytest.mark.parametrize("kw,code", CACHES + SIZES + [
    (dict(mv=None), INV), (dict(nl=None), INV), (dict(nt=FAKE + 64), INV), (dict(nr=FAKE + 4), INV),
    (dict(mv=FAKE + 4), INV), (dict(nt=FAKE, nr=FAKE), SMALL)])  # in place
def test_compact_validation(kw, code):
    assert _compact(**kw) == code


def test_workspace_sizes():
    assert pkg.pages_fork_workspace_bytes(8) >= 96 and pkg.pages_fork_workspace_bytes(0) == 0
    assert pkg.pages_fork_workspace_bytes(8193) == 0 and pkg.pages_compact_workspace_bytes(0) == 0
    assert pkg.pages_compact_workspace_bytes(1000) >= 12000


# ---- the Python side: shapes, dtypes, strides, devices

def _tensors(T=5, B=2, Hq=8, Hkv=2, D=128):
    return dict(q=torch.zeros(T, Hq, D, dtype=torch.bfloat16), kv=torch.zeros(10, 2, 16, Hkv, D, dtype=torch.bfloat16),
                bt=torch.zeros(B, 4, dtype=torch.int32), sl=torch.zeros(B, dtype=torch.int32),
                qs=torch.zeros(B + 1, dtype=torch.int32))


@pytest.mark.parametrize("change,error", [
    (dict(q=torch.zeros(5, 8, 128)), TypeError), (dict(q=torch.zeros(5, 8, dtype=torch.bfloat16)), ValueError),
    (dict(q=torch.zeros(5, 8, 64, dtype=torch.bfloat16)), ValueError),
    (dict(q=torch.zeros(8, 5, 128, dtype=torch.bfloat16).transpose(0, 1)), ValueError),
    (dict(kv=torch.zeros(10, 2, 16, 2, 128)), TypeError), (dict(kv=torch.zeros(10, 16, 2, 128, dtype=torch.bfloat16)), ValueError),
    (dict(bt=torch.zeros(2, 4, dtype=torch.int64)), TypeError), (dict(sl=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(qs=torch.zeros(2, dtype=torch.int32)), ValueError), (dict(), ValueError)])  # (), on the CPU
def test_prefill_tensors(change, error):
    t = {**_tensors(), **change}
    with pytest.raises(error):
        pkg.gqa_prefill(t["q"], t["kv"], t["bt"], t["sl"], t["qs"], 0.1)


@pytest.mark.parametrize("name,value", [
    ("prefix_lens", torch.zeros(3, dtype=torch.int32)), ("prefix_lens", torch.zeros(2)), ("slopes", torch.zeros(7)),
    ("slopes", torch.zeros(8, dtype=torch.float64)), ("out", torch.zeros(5, 8, 128)), ("lse", torch.zeros(5, 7)),
    ("kv_scales", torch.zeros(10, 2, 1, 2)), ("device_status", torch.zeros(1))])
def test_prefill_optional_tensors(name, value):
    t = _tensors()
    with pytest.raises((TypeError, ValueError)):
        pkg.gqa_prefill(t["q"], t["kv"], t["bt"], t["sl"], t["qs"], 0.1, **{name: value})


def test_no_pages():
    """Caches of no pages reach the call, which refuses them."""
    from mqa_decode_attention_paged_gb300 import _prompt_ops
    assert list(_prompt_ops._pools([torch.zeros(0, 4)], 0, -1)[1]) == [0]
    assert _fork(nb=0) == INV and _compact(nb=0) == INV


def test_score_slopes():
    t = _tensors()
    for slopes in (torch.zeros(7), torch.zeros(8, dtype=torch.bfloat16), torch.zeros(16)[::2]):
        with pytest.raises((TypeError, ValueError)):
            pkg.gqa_score_decode(torch.zeros(2, 8, 128, dtype=torch.bfloat16), t["kv"], t["bt"], t["sl"], 0.1, slopes=slopes)


@pytest.mark.parametrize("change", [
    dict(bt=torch.zeros(2, 4)), dict(bt=torch.zeros(8, dtype=torch.int32)), dict(sl=torch.zeros(3, dtype=torch.int32)),
    dict(refs=torch.zeros(10)), dict(refs=torch.zeros(10, 1, dtype=torch.int32)), dict(caches=[torch.zeros(9, 4)]), dict()])
def test_page_tensors(change):
    t = dict(bt=torch.zeros(2, 4, dtype=torch.int32), sl=torch.zeros(2, dtype=torch.int32),
             refs=torch.zeros(10, dtype=torch.int32), caches=[torch.zeros(10, 4)])
    t.update(change)
    with pytest.raises((TypeError, ValueError)):
        pkg.pages_fork(t["bt"], t["sl"], torch.zeros(3, dtype=torch.int32), t["refs"], t["caches"], 16)
    with pytest.raises((TypeError, ValueError)):
        pkg.pages_compact(t["bt"], t["sl"], t["refs"], t["caches"], 16)
    with pytest.raises((TypeError, ValueError)):
        pkg.pages_fork(t["bt"], t["sl"], torch.zeros(3), t["refs"], t["caches"], 16)


# ---- outputs on other arguments (refused; each call has what it wants but for that)

M = 0x10000000  # so far apart that nothing else overlaps
FORK = dict(bt=M, sl=2 * M, pa=3 * M, refs=4 * M, nt=5 * M, nl=6 * M, nr=7 * M, ws=8 * M, wsb=1 << 20, st=9 * M,
            caches=[10 * M, 11 * M], sizes=[4096, 64])
COMPACT = dict(bt=M, sl=2 * M, refs=4 * M, nt=5 * M, nr=7 * M, mv=12 * M, nl=6 * M, ws=8 * M, wsb=1 << 20, st=9 * M,
               caches=[10 * M, 11 * M], sizes=[4096, 64])
FORK_BYTES = dict(bt=128, sl=16, pa=32, refs=400, nt=256, nl=32, nr=400, ws=(64 + 24) * 4, st=4)
COMPACT_BYTES = dict(bt=128, sl=16, refs=400, nt=128, nr=400, mv=400, nl=4, ws=(64 + 300) * 4, st=4)


def _clashes(sizes, written):
    """Each written argument, each other one, and whether it is to be placed on that one's last or first word."""
    return [(w, o, end) for w in written for o in sizes if o != w for end in (0, 1)]


def _at(start, size, own, end, align):
    """An address, aligned, at which `own` bytes touch the first or last ones of [start, start + size)."""
    return (start + size - 4) // align * align if end else -(-(start + 4 - own) // align) * align


@pytest.mark.parametrize("w,o,end", _clashes(FORK_BYTES, ("nt", "nl", "nr", "ws", "st")))
def test_fork_writes_on_nothing_else(w, o, end):
    at = _at(FORK[o], FORK_BYTES[o], FORK_BYTES[w], end, 16 if w in ("out", "ws") else 4)
    assert _fork(**{**FORK, w: at}) == INV


@pytest.mark.parametrize("w,o,end", _clashes(COMPACT_BYTES, ("nt", "nr", "mv", "nl", "ws", "st")))
def test_compact_writes_on_nothing_else(w, o, end):
    at = _at(COMPACT[o], COMPACT_BYTES[o], COMPACT_BYTES[w], end, 16 if w in ("out", "ws") else 4)
    assert _compact(**{**COMPACT, w: at}) == INV


@pytest.mark.parametrize("name", [*FORK_BYTES, "mv"])
@pytest.mark.parametrize("cache", [0, 1])
def test_pages_of_caches_hold_no_argument(name, cache):
    first, last = FORK["caches"][cache], FORK["caches"][cache] + 100 * FORK["sizes"][cache] - 16
    for at in (first, last):
        if name in FORK_BYTES:
            assert _fork(**{**FORK, name: at}) == INV
        if name in COMPACT_BYTES:
            assert _compact(**{**COMPACT, name: at}) == INV


PREFILL = dict(q=M, kv=2 * M, sc=3 * M, bt=4 * M, sl=5 * M, qs=6 * M, pre=7 * M, slopes=8 * M, out=9 * M, lse=10 * M, st=11 * M,
               ws=12 * M, wsb=0x8000000, S=2, kvd=6, G=16, ks=1.0)
PREFILL_BYTES = dict(q=5 * 2048, kv=10 * 2 * 16 * 2 * 128, sc=10 * 2 * 2 * 4, bt=64, sl=8, qs=12, pre=8, slopes=32, out=5 * 2048,
                     lse=160, st=4, ws=0x8000000)


@pytest.mark.parametrize("w,o,end", _clashes(PREFILL_BYTES, ("out", "lse", "st", "ws")))
def test_prefill_writes_on_nothing_else(w, o, end):
    at = _at(PREFILL[o], PREFILL_BYTES[o], PREFILL_BYTES[w], end, 16 if w in ("out", "ws") else 4)
    assert _prefill(**{**PREFILL, w: at}) == INV
