"""gqa_score_decode against attention in 64 bits (attention_reference.py)."""
import pytest
import torch

import mqa_decode_attention_paged_gb300 as mqa
from attention_reference import NO_WINDOW, Paged, attention, judge

pytestmark = pytest.mark.gpu


def run(lens, L=1, Hq=8, Hkv=2, D=128, page=16, kv="bf16", group=0, window=None, sinks=0, cap=0.0, slopes=False, splits=None,
        size=1.0, seed=3, scale=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (len(lens), Hq, D) if L == 1 else (len(lens), L, Hq, D)
    q = (torch.randn(*shape, generator=g, device="cuda") * size).to(torch.bfloat16)
    c = Paged(lens, Hkv, D, page, kv, seed, group)
    sl = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq).float() if slopes else None
    if isinstance(slopes, list):
        sl = torch.tensor(slopes, device="cuda")
    scale = D ** -0.5 if scale is None else scale
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = mqa.gqa_score_decode(q, c.cache, c.table, c.seq_lens, scale, softcap=cap, slopes=sl, window=window,
                                    sinks=sinks, kv_scales=c.scales, k_scale=c.k_scale, v_scale=c.v_scale,
                                    num_kv_splits=splits, device_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and out.shape == q.shape and lse.shape == q.shape[:-1]
    for b, n in enumerate(lens):
        ref = attention(q[b].view(L, Hq, D), c.K[b], c.V[b], n - L, scale, cap, sl,
                        NO_WINDOW if window is None else window, sinks, half_codes=c.codes[b])
        judge(out[b].view(L, Hq, D), lse[b].view(L, Hq), ref, f"request {b}")
    return q, c, out, lse


@pytest.mark.parametrize("splits", [1, None])
@pytest.mark.parametrize("cap,slopes", [(50.0, False), (0.0, True), (15.0, True), (0.0, False)])
@pytest.mark.parametrize("kv,group", [("bf16", 0), ("fp8_e4m3", 0), ("fp8_e4m3_block", 16), ("int8_block", 16)])
@pytest.mark.parametrize("D", [64, 128])
def test_formats(kv, group, cap, slopes, D, splits):
    run([1, 37, 300, 2000, 0], kv=kv, group=group, cap=cap, slopes=slopes, D=D, splits=splits, size=3.0)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (7, 1), (32, 8), (15, 5), (16, 1), (36, 3)])
@pytest.mark.parametrize("L", [1, 2, 5])
def test_heads_and_positions(Hq, Hkv, L):
    run([L, 400, 3, 77], L=L, Hq=Hq, Hkv=Hkv, cap=30.0, slopes=True, size=3.0)
    run([L, 400, 3, 77], L=L, Hq=Hq, Hkv=Hkv, cap=30.0, slopes=True, size=3.0, kv="int8_block", D=64)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (100, 4), (1000, 0), (1 << 33, 0)])
def test_windows(window, sinks):
    run([1, 99, 100, 5000], window=window, sinks=sinks, cap=20.0, slopes=True, L=3, size=3.0)
    run([1, 99, 100, 5000], window=window, sinks=sinks, cap=20.0, slopes=True, kv="fp8_e4m3_block", size=3.0)


@pytest.mark.parametrize("cap", [1e-3, 50.0, 1e4, 1e9])
@pytest.mark.parametrize("size", [0.1, 30.0, 300.0])
def test_caps_over_the_range(size, cap):
    run([300, 70], cap=cap, size=size)
    run([300, 70], cap=cap, size=size, kv="fp8_e4m3", L=4)


def test_without_shaping_it_is_the_windowed_call():
    q, c, out, lse = run([300, 2000], window=500, sinks=4)
    o, l = mqa.gqa_window_decode(q, c.cache, c.table, c.seq_lens, 128 ** -0.5, 500, 4)
    assert torch.equal(o, out) and torch.equal(l, lse)


def test_captured_and_replayed():
    q, c, out, lse = run([300, 9000, 1], cap=50.0, slopes=True)
    sl = torch.exp2(-8.0 * torch.arange(1, 9, device="cuda") / 8).float()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = mqa.gqa_score_decode(q, c.cache, c.table, c.seq_lens, 128 ** -0.5, softcap=50.0, slopes=sl)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)


@pytest.mark.parametrize("cap,scale", [(4e-6, 4.4e-10), (2.0 ** -20, 0.1), (2.0 ** 60, 0.1), (2.0 ** 60, 2.0 ** 48), (30.0, -0.2), (30.0, 0.0)])
def test_ends_of_the_range_of_caps(cap, scale):
    run([300, 70], cap=cap, scale=scale)
    run([300, 70], cap=cap, scale=scale, slopes=True, kv="int8_block", L=3)


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "int8_block"])
def test_slopes_of_any_size_and_sign(kv, cap):
    run([300, 70, 3000], slopes=[0.0, -0.05, 5.0, 1e4, 1.4, 1.5, -3.0, 1e-6], cap=cap, kv=kv)
