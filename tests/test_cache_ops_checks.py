"""Refusals and host helpers of the windowed / block-scaled decode and the
cache-append entry points (no GPU: every call fails before any CUDA call, or
does not reach the device)."""
import ctypes

import pytest
import torch

import mqa_decode_attention_paged_gb300 as pkg
from mqa_decode_attention_paged_gb300 import _binding as mqa

FAKE = 0x10000  # aligned, never dereferenced: validation fails first


def P(v):
    return None if v is None else ctypes.c_void_p(v)


def _window(**kw):
    a = dict(q=FAKE, kv=FAKE, sc=None, bt=FAKE, sl=FAKE, scale=0.1, ks=1.0, vs=1.0, window=128, sinks=4, out=FAKE,
             lse=None, B=2, L=1, Hq=8, Hkv=2, D=128, nb=10, P=16, maxb=8, G=16, kvd=0, S=1, ws=None, wsb=0, st=None)
    a.update(kw)
    return mqa.lib.gqa_window_decode(P(a["q"]), P(a["kv"]), P(a["sc"]), P(a["bt"]), P(a["sl"]), a["scale"], a["ks"],
                                     a["vs"], a["window"], a["sinks"], P(a["out"]), P(a["lse"]), a["B"], a["L"],
                                     a["Hq"], a["Hkv"], a["D"], a["nb"], a["P"], a["maxb"], a["G"], a["kvd"], a["S"],
                                     P(a["ws"]), a["wsb"], P(a["st"]), None)


INV, UNS, SMALL = mqa.ERR_INVALID_ARG, mqa.ERR_UNSUPPORTED, mqa.ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INV), (dict(kv=None), INV), (dict(bt=None), INV), (dict(sl=None), INV), (dict(out=None), INV),
    (dict(q=FAKE + 8), INV), (dict(kv=FAKE + 8), INV), (dict(out=FAKE + 2), INV), (dict(bt=FAKE + 2), INV),
    (dict(lse=FAKE + 2), INV), (dict(st=FAKE + 1), INV),
    (dict(B=0), INV), (dict(L=0), INV), (dict(Hq=0), INV), (dict(Hkv=0), INV), (dict(Hq=9), INV), (dict(nb=0), INV),
    (dict(maxb=0), INV), (dict(S=0), INV), (dict(window=0), INV), (dict(window=-5), INV), (dict(sinks=-1), INV),
    (dict(scale=float("nan")), INV), (dict(kvd=1, ks=float("inf")), INV),
    (dict(D=96), UNS), (dict(Hkv=9, Hq=9), UNS), (dict(Hq=34), UNS), (dict(L=33), UNS), (dict(B=2049), UNS),
    (dict(B=257, L=32), UNS),                      # 257 requests x 8 row blocks
    (dict(P=8), UNS), (dict(P=24), UNS), (dict(kvd=2), UNS), (dict(kvd=4), UNS), (dict(kvd=9), UNS),
    (dict(nb=1 << 27, P=16), UNS), (dict(maxb=1 << 27, P=16), UNS),
    (dict(B=2048, maxb=1 << 18), UNS),             # 2048 x (2^18 + 2) boxes of 16 tokens
    (dict(B=2048, maxb=(1 << 18) - 3, S=4), SMALL),  # served as far as this check goes
    (dict(kvd=5), INV), (dict(kvd=6, sc=FAKE + 2), INV), (dict(kvd=6, sc=FAKE, G=0), INV),
    (dict(kvd=6, sc=FAKE, G=24, P=48), UNS), (dict(kvd=5, sc=FAKE, G=32, P=16), UNS),
    (dict(S=4), SMALL),
    (dict(S=4, ws=FAKE, wsb=mqa.gqa_window_decode_workspace_bytes(2, 1, 8, 2, 128, 4) - 1), SMALL),
    (dict(S=4, ws=FAKE + 4, wsb=1 << 30), INV),
])
def test_window_validation(kw, code):
    assert _window(**kw) == code


def _block(**kw):
    a = dict(kvd=5, sc=FAKE, S=1, D=128)
    a.update(kw)
    return mqa.lib.gqa_block_decode(P(FAKE), P(FAKE), P(a["sc"]), P(FAKE), P(FAKE), 0.1, P(FAKE), None, 2, 1, 8, 2,
                                    a["D"], 10, 16, 8, 16, a["kvd"], a["S"], None, 0, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(kvd=0), UNS), (dict(kvd=1), UNS), (dict(kvd=3), UNS), (dict(sc=None), INV), (dict(D=80), UNS),
    (dict(S=2), SMALL)])
def test_block_validation(kw, code):
    assert _block(**kw) == code


def test_existing_decode_refuses_block_formats():
    for kvd in (mqa.KV_FP8_E4M3_BLOCK, mqa.KV_INT8_BLOCK):
        assert mqa.lib.gqa_paged_decode(P(FAKE), P(FAKE), P(FAKE), P(FAKE), 0.1, 1.0, 1.0, P(FAKE), None, 2, 8, 2,
                                        128, 10, 16, 8, kvd, 1, None, 0, None, None) == UNS


def _gqa_append(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, cs=FAKE, qs=FAKE, sl=FAKE, bt=FAKE, qo=FAKE, kv=FAKE, sc=None, ks=1.0, vs=1.0,
             T=4, B=2, Hq=8, Hkv=2, D=128, rot=128, inter=0, maxp=64, nb=10, P=16, maxb=4, G=16, kvd=0,
             sq=1024, sk=256, sv=256, so=1024, st=None)
    a.update(kw)
    return mqa.lib.gqa_rope_append(P(a["q"]), P(a["k"]), P(a["v"]), P(a["cs"]), P(a["qs"]), P(a["sl"]), P(a["bt"]),
                                   P(a["qo"]), P(a["kv"]), P(a["sc"]), a["ks"], a["vs"], a["T"], a["B"], a["Hq"],
                                   a["Hkv"], a["D"], a["rot"], a["inter"], a["maxp"], a["nb"], a["P"], a["maxb"],
                                   a["G"], a["kvd"], a["sq"], a["sk"], a["sv"], a["so"], P(a["st"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(cs=None), INV), (dict(qs=None), INV), (dict(sl=None), INV),
    (dict(bt=None), INV), (dict(kv=None), INV), (dict(qo=None), INV), (dict(q=None), INV),
    (dict(k=FAKE + 8), INV), (dict(v=FAKE + 2), INV), (dict(q=FAKE + 8), INV), (dict(qo=FAKE + 8), INV),
    (dict(kv=FAKE + 8), INV), (dict(cs=FAKE + 4), INV), (dict(qs=FAKE + 2), INV), (dict(st=FAKE + 2), INV),
    (dict(T=-1), INV), (dict(B=0), INV), (dict(Hq=0), INV), (dict(Hkv=0), INV), (dict(nb=0), INV), (dict(maxp=0), INV),
    (dict(rot=0), INV), (dict(rot=8), UNS), (dict(rot=144), INV), (dict(D=96), UNS), (dict(Hkv=9), UNS),
    (dict(P=24), UNS), (dict(kvd=7), UNS), (dict(T=(1 << 24) + 1), UNS), (dict(nb=1 << 27), UNS),
    (dict(sq=1016), INV), (dict(sk=248), INV), (dict(sv=260), INV), (dict(so=1028), INV),
    (dict(kvd=1, ks=0.0), INV), (dict(kvd=1, vs=float("nan")), INV), (dict(kvd=1, ks=1e-39), INV),
    (dict(kvd=1, vs=-2e38), INV), (dict(kvd=1, ks=float("inf")), INV),
    (dict(kvd=5), INV), (dict(kvd=6, sc=FAKE, G=8), UNS), (dict(kvd=6, sc=FAKE, G=32), UNS),
    (dict(kvd=6, sc=FAKE, G=0), INV),
    (dict(T=0), mqa.OK),                           # nothing to append: nothing is enqueued
])
def test_gqa_append_validation(kw, code):
    assert _gqa_append(**kw) == code


def _mla_append(**kw):
    a = dict(c=FAKE, p=FAKE, q=FAKE, cs=FAKE, qs=FAKE, sl=FAKE, bt=FAKE, qo=FAKE, kv=FAKE, ks=1.0, T=4, B=2, H=16,
             D=576, R=512, maxp=64, nb=10, P=16, maxb=4, kvd=0, sc=576, sp=576, sq=16 * 192, sh=192, so=16 * 576,
             soh=576)
    a.update(kw)
    return mqa.lib.mla_rope_append(P(a["c"]), P(a["p"]), P(a["q"]), P(a["cs"]), P(a["qs"]), P(a["sl"]), P(a["bt"]),
                                   P(a["qo"]), P(a["kv"]), a["ks"], a["T"], a["B"], a["H"], a["D"], a["R"], 0,
                                   a["maxp"], a["nb"], a["P"], a["maxb"], a["kvd"], a["sc"], a["sp"], a["sq"],
                                   a["sh"], a["so"], a["soh"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(c=None), INV), (dict(p=None), INV), (dict(q=None), INV), (dict(qo=None), INV), (dict(kv=None), INV),
    (dict(c=FAKE + 8), INV), (dict(p=FAKE + 8), INV), (dict(q=FAKE + 8), INV), (dict(qo=FAKE + 8), INV),
    (dict(H=0), INV), (dict(D=512, R=448), UNS), (dict(kvd=3), UNS), (dict(kvd=5), UNS), (dict(P=20), UNS),
    (dict(sc=504), INV), (dict(sp=60), INV), (dict(sh=60), INV), (dict(soh=68), INV), (dict(kvd=1, ks=0.0), INV),
    (dict(kvd=1, ks=1e-40), INV), (dict(kvd=1, ks=float("nan")), INV), (dict(T=0), mqa.OK)])
def test_mla_append_validation(kw, code):
    assert _mla_append(**kw) == code


def test_workspace_bytes():
    f = mqa.gqa_window_decode_workspace_bytes
    assert f(3, 1, 32, 8, 128, 1) == 0
    assert f(3, 1, 32, 8, 128, 5) == 3 * 5 * 8 * 4 * 129 * 4 + 3 * 8
    assert f(1, 1, 1, 1, 64, 3) == 3 * 64 * 4 + 16 + 8
    # 5 positions x 4 heads = 20 rows of a KV head: one row block; 7 x 4 = 28: two of 14
    assert f(3, 5, 32, 8, 64, 2) == 3 * 2 * 8 * 20 * 65 * 4 + 3 * 8
    assert f(3, 7, 32, 8, 64, 2) == 3 * 2 * 2 * 8 * 14 * 65 * 4 + 6 * 8
    assert f(0, 1, 32, 8, 128, 5) == 0 and f(3, 1, 33, 8, 128, 5) == 0 and f(3, 40, 32, 8, 128, 5) == 0


# ------------------------------------------------------------ binding checks

BF = torch.bfloat16


def _decode_args(**kw):
    a = dict(q=torch.zeros(2, 8, 128, dtype=BF), kv=torch.zeros(4, 2, 16, 2, 128, dtype=torch.int8),
             sc=torch.zeros(4, 2, 1, 2), bt=torch.zeros(2, 2, dtype=torch.int32), sl=torch.zeros(2, dtype=torch.int32))
    a.update(kw)
    return a["q"], a["kv"], a["sc"], a["bt"], a["sl"]


@pytest.mark.parametrize("kw,exc,msg", [
    (dict(), ValueError, "must be a CUDA tensor"),
    (dict(q=torch.zeros(2, 8, 128)), TypeError, "q must have dtype"),
    (dict(q=torch.zeros(8, 128, dtype=BF)), ValueError, "q must be"),
    (dict(q=torch.zeros(2, 8, 64, dtype=BF)), ValueError, "kv_cache must be"),
    (dict(sc=None), TypeError, "kv_cache must be bf16"),
    (dict(sc=torch.zeros(4, 2, 3, 2)), ValueError, "kv_scales must be"),
    (dict(sc=torch.zeros(4, 2, 1, 2, dtype=torch.float64)), TypeError, "kv_scales must have dtype"),
    (dict(kv=torch.zeros(4, 2, 16, 2, 128)), TypeError, "a block-scaled kv_cache is"),
    (dict(sl=torch.zeros(3, dtype=torch.int32)), ValueError, "seq_lens must have shape"),
])
def test_block_decode_argument_checks(kw, exc, msg):
    with pytest.raises(exc, match=msg):
        pkg.gqa_block_decode(*_decode_args(**kw), 0.1)


def test_window_decode_argument_checks():
    q, kv, sc, bt, sl = _decode_args(kv=torch.zeros(4, 2, 16, 2, 128, dtype=BF))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        pkg.gqa_window_decode(q, kv, bt, sl, 0.1, 64)
    with pytest.raises(TypeError, match="a block-scaled kv_cache is"):
        pkg.gqa_window_decode(q, kv, bt, sl, 0.1, 64, kv_scales=sc)
    with pytest.raises(ValueError, match="block-scaled caches"):
        pkg.gqa_block_decode(q, kv, None, bt, sl, 0.1)


def _append_args(**kw):
    a = dict(k=torch.zeros(5, 2, 64, dtype=BF), v=torch.zeros(5, 2, 64, dtype=BF), cs=torch.zeros(32, 64),
             kv=torch.zeros(4, 2, 16, 2, 64, dtype=BF), bt=torch.zeros(2, 2, dtype=torch.int32),
             sl=torch.zeros(2, dtype=torch.int32), qs=torch.zeros(3, dtype=torch.int32))
    a.update(kw)
    return a["k"], a["v"], a["cs"], a["kv"], a["bt"], a["sl"], a["qs"]


@pytest.mark.parametrize("kw,exc,msg", [
    (dict(), ValueError, "must be a CUDA tensor"),
    (dict(k=torch.zeros(5, 2, 64)), TypeError, "k must have dtype"),
    (dict(v=torch.zeros(4, 2, 64, dtype=BF)), ValueError, "v must have shape"),
    (dict(v=torch.zeros(5, 64, 2, dtype=BF).transpose(1, 2)), ValueError, "must be contiguous"),
    (dict(cs=torch.zeros(32, 64, dtype=torch.float64)), TypeError, "cos_sin must have dtype"),
    (dict(kv=torch.zeros(4, 2, 16, 2, 68, dtype=BF)), ValueError, "kv_cache must be"),
    (dict(qs=torch.zeros(2, dtype=torch.int32)), ValueError, "query_start must have shape"),
    (dict(sl=torch.zeros(2, dtype=torch.int64)), TypeError, "seq_lens must have dtype"),
    (dict(bt=torch.zeros(2, dtype=torch.int32)), ValueError, "block_table must be"),
])
def test_gqa_append_argument_checks(kw, exc, msg):
    with pytest.raises(exc, match=msg):
        pkg.gqa_rope_append(*_append_args(**kw))


def test_append_query_checks():
    a = _append_args()
    with pytest.raises(ValueError, match="q_out without q"):
        pkg.gqa_rope_append(*a, q_out=torch.zeros(5, 4, 64, dtype=BF))
    with pytest.raises(ValueError, match="q_out must have shape"):
        pkg.gqa_rope_append(*a, q=torch.zeros(5, 4, 64, dtype=BF), q_out=torch.zeros(5, 2, 64, dtype=BF))
    with pytest.raises(ValueError, match="for the fp8_e4m3_block"):
        pkg.gqa_rope_append(*a, kv_scales=torch.zeros(4, 2, 1, 2), kv_dtype="bf16")
    m = (torch.zeros(5, 512, dtype=BF), torch.zeros(5, 64, dtype=BF), torch.zeros(32, 64),
         torch.zeros(4, 16, 576, dtype=BF), a[4], a[5], a[6])
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        pkg.mla_rope_append(*m)
    with pytest.raises(ValueError, match="kv_cache must be"):
        pkg.mla_rope_append(m[0][:, :256], *m[1:])
    with pytest.raises(ValueError, match="q_pe_out without q_pe"):
        pkg.mla_rope_append(*m, q_pe_out=torch.zeros(5, 4, 64, dtype=BF))
    with pytest.raises(ValueError, match="cos_sin must be"):
        pkg.mla_rope_append(m[0], m[1], torch.zeros(32, 32), *m[3:])


def test_row_strides():
    x = torch.zeros(7, 12, 64, dtype=BF)
    assert mqa._check_rows(x[:, 2:6], "k", (7, 4, 64), 2) == (768,)
    assert mqa._check_rows(x[:1, 2:6], "k", (1, 4, 64), 2) == (256,)    # one token: no stride of its own
    assert mqa._check_rows(x[..., :64].transpose(0, 1), "q_pe", (12, 7, 64), 1) == (64, 768)


def test_mla_append_refuses_overlapping_output_rows():
    # two heads' or two tokens' rows of q_pe_out in the same place: which one stays would be left to chance
    assert _mla_append(so=64, soh=64) == INV
    assert _mla_append(so=576, soh=576) == INV
    assert _mla_append(T=3, H=2, so=64, soh=128) == INV  # the third token meets the second head
