"""gqa_prefill against attention in 64 bits (attention_reference.py): formats, head layouts, page sizes, ragged
lengths from no token to long ones, windows, sinks, prefixes, caps and biases, cut and uncut."""
import itertools
import os

import pytest
import torch

import mqa_decode_attention_paged_gb300 as mqa
from attention_reference import NO_WINDOW, Paged, attention, judge

pytestmark = pytest.mark.gpu


def slopes_of(Hq):
    return torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq).float()


def batch(new, old, Hq, D, pad=0, seed=1, size=1.0, fused=False, lead=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(new) + pad + lead
    if fused:
        q = (torch.randn(T, Hq + 4, D, generator=g, device="cuda") * size).to(torch.bfloat16)[:, 2:2 + Hq]
    else:
        q = (torch.randn(T, Hq, D, generator=g, device="cuda") * size).to(torch.bfloat16)
    starts = torch.tensor([lead] + [lead + s for s in itertools.accumulate(new)], dtype=torch.int32, device="cuda")
    return q, starts, [a + b for a, b in zip(new, old)]


def run(new, old, Hq=8, Hkv=2, D=128, page=16, kv="bf16", group=0, window=NO_WINDOW, sinks=0, prefix=None, cap=0.0,
        slopes=False, splits=None, pad=0, size=1.0, fused=False, lead=0, value=1.0, scale=None, seed=1):
    q, starts, lens = batch(new, old, Hq, D, pad, seed, size, fused, lead)
    c = Paged(lens, Hkv, D, page, kv, seed, group, value=value)
    scale = D ** -0.5 if scale is None else scale
    sl = slopes_of(Hq) if slopes else None
    if isinstance(slopes, list):
        sl = torch.tensor(slopes, device="cuda")
    pre = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device="cuda")
    out = torch.full((q.shape[0], Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], Hq), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, scale, softcap=cap, slopes=sl, window=window, sinks=sinks,
                    prefix_lens=pre, kv_scales=c.scales, k_scale=c.k_scale, v_scale=c.v_scale, out=out, lse=lse,
                    num_kv_splits=splits, device_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    at = lead
    for b, k in enumerate(new):
        if k:
            ref = attention(q[at:at + k], c.K[b], c.V[b], lens[b] - k, scale, cap, sl, window, sinks,
                            min(max(prefix[b], 0), lens[b]) if prefix else 0)
            judge(out[at:at + k], lse[at:at + k], ref, f"request {b}")
        at += k
    for x in (out[:lead], out[at:], lse[:lead], lse[at:]):
        assert bool((x == 7.0).all()), "padding rows are left as they were"
    return out, lse


@pytest.mark.parametrize("splits", [1, None])
@pytest.mark.parametrize("kv,group", [("bf16", 0), ("fp8_e4m3", 0), ("fp8_e4m3_block", 16), ("int8_block", 32)])
@pytest.mark.parametrize("D", [64, 128])
def test_formats(kv, group, D, splits):
    run([37, 1, 300, 0, 129], [0, 500, 70, 10, 1], D=D, page=32, kv=kv, group=group, splits=splits, pad=3)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (6, 2), (7, 1), (32, 8), (10, 5), (16, 1), (48, 3), (71, 1), (128, 1), (40, 40)])
def test_heads(Hq, Hkv):
    run([1, 150, 3], [5, 40, 0], Hq=Hq, Hkv=Hkv, pad=1)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 144, 256, 1024])
def test_pages(page):
    run([200, 5], [90, 700], page=page)
    run([200, 5], [90, 700], page=page, kv="int8_block", D=64)


@pytest.mark.parametrize("new,old", [([1], [0]), ([1], [127]), ([1], [128]), ([32], [0]), ([33], [0]), ([64], [64]),
                                     ([65], [63]), ([127, 128, 129], [1, 0, 255]), ([1] * 40, list(range(40))),
                                     ([0, 0, 5, 0], [0, 3, 0, 9]), ([2000], [3000]), ([3], [9000])])
def test_lengths(new, old):
    for splits in (1, None):
        run(new, old, splits=splits)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 5), (16, 0), (100, 4), (128, 128), (129, 130), (333, 1), (1000, 17)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (2, 2)])
def test_windows(window, sinks, Hq, Hkv):
    run([300, 1, 40], [200, 700, 0], Hq=Hq, Hkv=Hkv, window=window, sinks=sinks)
    run([300, 1, 40], [200, 700, 0], Hq=Hq, Hkv=Hkv, window=window, sinks=sinks, kv="fp8_e4m3_block", group=16, D=64)


@pytest.mark.parametrize("window", [NO_WINDOW, 90])
@pytest.mark.parametrize("slopes", [False, True])
def test_prefixes(slopes, window):
    run([300, 1, 40, 200], [0, 700, 100, 50], prefix=[250, 0, 1000, -4], slopes=slopes, window=window)
    run([300, 40], [0, 100], prefix=[129, 110], Hq=4, Hkv=4, slopes=slopes, window=window, sinks=3, kv="int8_block")


@pytest.mark.parametrize("cap", [5.0, 15.0, 50.0, 1e4, 1e9])
@pytest.mark.parametrize("size", [0.5, 4.0, 40.0])
def test_caps(cap, size):
    run([200, 1], [60, 300], cap=cap, size=size)
    run([200, 1], [60, 300], cap=cap, size=size, slopes=True, kv="fp8_e4m3", D=64)


@pytest.mark.parametrize("kv", ["bf16", "int8_block"])
def test_distance_bias(kv):
    run([200, 1, 5], [60, 3000, 9], slopes=True, kv=kv)
    run([200, 1, 5], [60, 3000, 9], slopes=True, kv=kv, window=70, sinks=2, Hq=6, Hkv=3)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-6, 3.0])
def test_scales(scale):
    run([150], [30], scale=scale)


def test_large_logits_move_the_reference():
    # logits of hundreds: rows' references move often, in both tiles
    run([260], [500], size=20.0, scale=1.0)
    run([260], [500], size=20.0, scale=1.0, kv="fp8_e4m3_block", D=64)


def test_fused_projection_and_padding():
    run([70, 1, 9], [10, 90, 0], fused=True, pad=9, lead=5)
    run([1], [90], Hq=1, Hkv=1, fused=True)


def test_values_of_unlike_magnitude():
    run([200], [60], value=1e-6)
    run([200], [60], value=1e4, scale=1e-9)


def test_many_requests():
    run([1 + i % 3 for i in range(700)], [i % 90 for i in range(700)], Hq=4, Hkv=1, D=64)


def test_queries_before_the_first_position():
    # fewer tokens in the sequence than new ones: the first queries see nothing
    q, starts, _ = batch([6], [0], 8, 128)
    c = Paged([4], 2, 128, 16, "bf16")
    out, lse = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1, prefix_lens=torch.tensor([3], dtype=torch.int32, device="cuda"))
    judge(out, lse, attention(q, c.K[0], c.V[0], -2, 0.1, prefix=3))
    assert bool((out[:2] == 0).all()) and bool((lse[:2] == -float("inf")).all())


def test_an_empty_sequence_and_an_empty_batch():
    q, starts, _ = batch([3], [0], 8, 128)
    c = Paged([0], 2, 128, 16, "bf16")
    for splits in (1, None):
        out, lse = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1, num_kv_splits=splits)
        assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, lse = mqa.gqa_prefill(q[:0], c.cache, c.table, c.seq_lens, none, 0.1)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)


def test_uncut_results_do_not_depend_on_the_batch():
    q, starts, lens = batch([37, 200, 90], [10, 300, 5], 8, 128)
    c = Paged(lens, 2, 128, 16, "bf16")
    out, lse = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1, num_kv_splits=1)
    one = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    o1, l1 = mqa.gqa_prefill(q[37:237].contiguous(), c.cache, c.table[1:2].contiguous(), c.seq_lens[1:2].contiguous(), one, 0.1,
                             num_kv_splits=1)
    assert torch.equal(out[37:237], o1) and torch.equal(lse[37:237], l1)


def test_reproducible():
    q, starts, lens = batch([64, 1, 700], [9000, 4000, 0], 32, 128)
    c = Paged(lens, 8, 128, 64, "bf16")
    ref = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1)
    for _ in range(5):
        got = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_bad_block_ids_and_lengths():
    q, starts, lens = batch([40, 40], [100, 100], 8, 128)
    c = Paged(lens, 2, 128, 16, "bf16")
    for bad in (-1, c.cache.shape[0], 2 ** 31 - 1):
        table = c.table.clone()
        table[0, 3] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = mqa.gqa_prefill(q, c.cache, table, c.seq_lens, starts, 0.1, device_status=status)
        assert int(status) == 5
        judge(out[40:], lse[40:], attention(q[40:], c.K[1], c.V[1], 100, 0.1))
        # the block's tokens are not seen
        K, V = (torch.cat([x[:48], x[64:]]) for x in (c.K[0], c.V[0]))
        ref = attention(q[:40], K, V, 84, 0.1)
        judge(out[:40], lse[:40], ref)
    for lengths, start in (([10 ** 6, 140], None), ([-5, 140], None), ([140, 140], [0, 90, 80]), ([140, 140], [-3, 40, 80]),
                           ([140, 140], [0, 40, 1000])):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        st = starts if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
        mqa.gqa_prefill(q, c.cache, c.table, torch.tensor(lengths, dtype=torch.int32, device="cuda"), st, 0.1,
                        device_status=status)
        assert int(status) == 5


def test_captured_and_replayed_on_two_streams():
    q, starts, lens = batch([64, 3], [3000, 100], 32, 128)
    c = Paged(lens, 8, 128, 64, "bf16")
    want = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1)
    outs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1)
        outs.append((g, s, got))
    for g, s, got in outs:
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    for _, _, got in outs:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_wait_that_runs_out(monkeypatch):
    import ctypes
    from mqa_decode_attention_paged_gb300 import _binding as b
    monkeypatch.setenv("MQA_ENABLE_TEST_HOOKS", "1")
    q, starts, lens = batch([64, 64], [200, 100], 8, 128)
    c = Paged(lens, 2, 128, 16, "bf16")
    out = torch.zeros_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P = ctypes.c_void_p
    fn = b.lib.mqa_test_gqa_prefill_withheld
    fn.argtypes = [P] * 5 + [ctypes.c_float, P] + [ctypes.c_int] * 8 + [ctypes.c_longlong, P, P, ctypes.c_int]
    rc = fn(q.data_ptr(), c.cache.data_ptr(), c.table.data_ptr(), c.seq_lens.data_ptr(), starts.data_ptr(), 0.1,
            out.data_ptr(), 128, 2, 8, 2, 128, c.cache.shape[0], 16, c.table.shape[1], q.stride(0), status.data_ptr(),
            torch.cuda.current_stream().cuda_stream, 1)
    torch.cuda.synchronize()
    assert rc == 0 and int(status) == 6
    run([37], [10])  # the context goes on


@pytest.mark.parametrize("kv", ["fp8_e4m3_block", "int8_block"])
@pytest.mark.parametrize("shape", [dict(), dict(window=50, sinks=3), dict(cap=30.0), dict(slopes=True), dict(cap=30.0, slopes=True)])
@pytest.mark.parametrize("D", [64, 128])
def test_unusual_block_scales(kv, shape, D):
    """Scales of 0, far below and far above what caches hold, in blocks of their own and among others."""
    new, old = [300, 40], [170, 300]
    q, starts, lens = batch(new, old, 8, D)
    c = Paged(lens, 2, D, 16, kv, 1, 16)
    cap, window, sinks = shape.get("cap", 0.0), shape.get("window", NO_WINDOW), shape.get("sinks", 0)
    sl = slopes_of(8) if shape.get("slopes") else None
    for b, group, plane, h, factor in [(0, 0, 1, 0, 0.0), (0, 3, 0, 1, 0.0), (0, 9, 1, 1, 2.0 ** -60), (0, 12, 0, 0, 2.0 ** -110),
                                       (0, 17, 1, 0, 2.0 ** 50), (0, 20, 1, 1, 2.0 ** -39), (0, 28, 1, 1, 0.0),
                                       *((1, k, 1, 0, 0.0) for k in range(22)), (1, 5, 1, 1, 2.0 ** 39)]:
        c.scales[int(c.table[b, group]), plane, 0, h] *= factor
        (c.V if plane else c.K)[b][16 * group:16 * group + 16, h] *= factor
    for splits in (1, None):
        out, lse = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, D ** -0.5, softcap=cap, slopes=sl, window=window,
                                   sinks=sinks, kv_scales=c.scales, num_kv_splits=splits)
        for b, at in ((0, 0), (1, 300)):
            k = new[b]
            judge(out[at:at + k], lse[at:at + k], attention(q[at:at + k], c.K[b], c.V[b], old[b], D ** -0.5, cap, sl, window, sinks, 0),
                  f"request {b}")


@pytest.mark.parametrize("kv,what", [(kv, what) for kv in ("bf16", "fp8_e4m3", "fp8_e4m3_block") for what in ("key", "value")]
                         + [("fp8_e4m3_block", "scale"), ("int8_block", "scale")])  # (int8 codes are finite)
@pytest.mark.parametrize("shape", [dict(), dict(window=50, sinks=3), dict(prefix=[130, 0]), dict(cap=30.0), dict(slopes=True)])
def test_non_finite_tokens_reach_those_that_see_them_alone(kv, what, shape):
    new, old = [150, 40], [70, 300]
    q, starts, lens = batch(new, old, 8, 128)
    c = Paged(lens, 2, 128, 16, kv, 1, 16)
    cap, window, sinks = shape.get("cap", 0.0), shape.get("window", NO_WINDOW), shape.get("sinks", 0)
    sl = slopes_of(8) if shape.get("slopes") else None
    pre = shape.get("prefix")
    kw = dict(softcap=cap, slopes=sl, window=window, sinks=sinks, kv_scales=c.scales, k_scale=c.k_scale, v_scale=c.v_scale,
              prefix_lens=torch.tensor(pre, dtype=torch.int32, device="cuda") if pre else None)
    spots = [1, 90, 131, 200]  # tokens of the first request
    codes = c.cache.view(torch.int16 if kv == "bf16" else torch.uint8)
    for t in spots:
        block, slot = int(c.table[0, t // 16]), t % 16
        if what == "scale":
            c.scales[block, :, 0, 1] = float("nan")
        else:
            codes[block, 0 if what == "key" else 1, slot, 1, 5] = (0x7f80 if t % 2 else 0x7fc0) if kv == "bf16" else 0x7f
    for splits in (1, None):
        out, lse = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1, num_kv_splits=splits, **kw)
        ref = attention(q[150:], c.K[1], c.V[1], 300, 0.1, cap, sl, window, sinks, 0)
        judge(out[150:], lse[150:], ref, "the other request")
        p = 70 + torch.arange(150, device="cuda")[:, None]
        t = torch.tensor(sum(([*range(s // 16 * 16, s // 16 * 16 + 16)] for s in spots), []) if what == "scale" else spots, device="cuda")
        sees = (((t <= p) | (t < (pre[0] if pre else 0))) & ((t < sinks) | (t > p - window))).any(1)
        ref = attention(q[:150], c.K[0], c.V[0], 70, 0.1, cap, sl, window, sinks, pre[0] if pre else 0)
        for heads in (slice(0, 4), slice(4, 8)):  # the first KV head is clean
            rows = ~sees if heads.start else torch.ones_like(sees)
            judge(out[:150][rows][:, heads], lse[:150][rows][:, heads], tuple(x[rows][:, heads] for x in ref), f"{heads}")
        if what != "key" or kv != "bf16":  # (of an infinite key the logit may be -inf: no weight at all)
            assert not bool(torch.isfinite(out[:150][sees][:, 4:].float()).all(-1).any()), "rows that see one say so"


@pytest.mark.parametrize("cap,scale", [(4e-6, 4.4e-10), (4e-6, 1e-6), (2.0 ** -20, 0.1), (2.0 ** 60, 0.1), (2.0 ** 60, 2.0 ** 48)])
def test_ends_of_the_range_of_caps(cap, scale):
    run([200, 1], [60, 300], cap=cap, scale=scale, window=150)
    run([200, 1], [60, 300], cap=cap, scale=scale, slopes=True, kv="int8_block")


def test_replayed_with_other_lengths():
    """A captured call reads lengths and starts when it runs; the workspace holds what the run before left."""
    lens = [[300, 40, 700], [20, 600, 1], [700, 700, 700]]
    new = [[300, 0, 64], [20, 90, 0], [1, 200, 129]]
    c = Paged([700] * 3, 2, 128, 16, "bf16")
    q = batch([400], [0], 8, 128)[0]
    sl, starts = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(400, 8, device="cuda")
    workspace = torch.full((mqa.gqa_prefill_workspace_bytes(8, 2, 128),), 0xff, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mqa.gqa_prefill(q, c.cache, c.table, sl, starts, 0.1, out=out, lse=lse, workspace=workspace)
    for n, k in zip(lens, new):
        sl.copy_(torch.tensor(n, dtype=torch.int32))
        starts.copy_(torch.tensor([0, *itertools.accumulate(k)], dtype=torch.int32))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        at = 0
        for b in range(3):
            if k[b]:
                judge(out[at:at + k[b]], lse[at:at + k[b]],
                      attention(q[at:at + k[b]], c.K[b][:n[b]], c.V[b][:n[b]], n[b] - k[b], 0.1), f"request {b}")
            at += k[b]
        assert bool((out[at:] == 7.0).all())


@pytest.mark.parametrize("splits", [1, None])
def test_results_at_odd_addresses(splits):
    q, starts, lens = batch([150, 7], [40, 900], 6, 64)
    c = Paged(lens, 3, 64, 16, "bf16")
    want = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1, num_kv_splits=splits)
    buffer = torch.zeros(q.numel() + 16, dtype=torch.bfloat16, device="cuda")
    words = torch.zeros(157 * 6 + 3, device="cuda")
    room = torch.zeros(mqa.gqa_prefill_workspace_bytes(6, 3, 64) + 16, dtype=torch.uint8, device="cuda")
    got = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1, num_kv_splits=splits,
                          out=buffer[8:8 + q.numel()].view(q.shape), lse=words[1:1 + 157 * 6].view(157, 6), workspace=room[16:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((buffer[:8] == 0).all()) and bool((buffer[-8:] == 0).all()) and float(words[0]) == float(words[-1]) == 0


@pytest.mark.parametrize("kv", ["bf16", "int8_block"])
def test_pages_far_into_a_large_cache(kv):
    """Pages whose addresses lie past 2^32 bytes, and past 2^31 values, of their cache."""
    new, old, page, Hkv, D = [70, 5], [100, 300], 16, 8, 128
    q, starts, lens = batch(new, old, 8, D)
    c = Paged(lens, Hkv, D, page, kv, 1, 16 if "block" in kv else 0)
    small = c.cache.shape[0]
    nb = 2 ** 31 // (2 * page * Hkv * D) + 1000
    big = torch.empty((nb, *c.cache.shape[1:]), dtype=c.cache.dtype, device="cuda")
    big[-small:] = c.cache
    scales = None
    if c.scales is not None:
        scales = torch.ones(nb, *c.scales.shape[1:], device="cuda")
        scales[-small:] = c.scales
    table = torch.where((c.table >= 0) & (c.table < small), c.table + (nb - small), c.table)
    want = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1, kv_scales=c.scales)
    got = mqa.gqa_prefill(q, big, table, c.seq_lens, starts, 0.1, kv_scales=scales)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "int8_block"])
def test_slopes_of_any_size_and_sign(kv, cap):
    run([200, 1, 5], [60, 3000, 9], slopes=[0.0, -0.05, 5.0, 1e4, 1.4, 1.5, -3.0, 1e-6], cap=cap, kv=kv)
    run([200, 40], [60, 0], slopes=[1.42, 0.3, 2.0, -1.0, 0.0, 0.0, 64.0, 1.0], cap=cap, kv=kv, Hq=8, Hkv=8, window=50, sinks=3, D=64)


# ---- rows that see nothing among others that do: each of their (cell, KV head) pairs is a piece without blocks

@pytest.mark.parametrize("splits", [1, None])
@pytest.mark.parametrize("kv,D", [("bf16", 128), ("bf16", 64), ("fp8_e4m3", 128), ("fp8_e4m3_block", 64), ("int8_block", 128)])
@pytest.mark.parametrize("empty", ["last 4", "last 16", "last 64", "every other", "all but one"])
def test_single_tokens_some_without_a_sequence(empty, kv, D, splits):
    none = {"last 4": range(252, 256), "last 16": range(240, 256), "last 64": range(192, 256), "every other": range(1, 256, 2),
            "all but one": [i for i in range(256) if i != 77]}[empty]
    run([1] * 256, [-1 if i in none else 199 for i in range(256)], Hq=32, Hkv=8, D=D, page=32, kv=kv, splits=splits)


@pytest.mark.parametrize("splits", [1, None])
@pytest.mark.parametrize("at", [0, 11, 23])
@pytest.mark.parametrize("shape", [dict(), dict(kv="int8_block", D=64), dict(window=100, sinks=3, kv="fp8_e4m3"),
                                   dict(cap=20.0, slopes=True)])
def test_prompts_one_of_them_longer_than_its_sequence(shape, at, splits):
    new = [100 + 20 * i for i in range(24)]
    new[at] = 500
    run(new, [-460 if i == at else i % 3 * 40 for i in range(24)], Hq=32, Hkv=8, splits=splits, pad=2, **shape)


def test_pieces_without_blocks_in_runs_of_any_length():
    """Between requests with keys 0 to 11 requests without, several heads each, in an order of their own for each share."""
    new, old = [], []
    for k in range(12):
        for i in range(12):
            new += [1 + (7 * i + k) % 300] + [1 + j % 3 for j in range(k)]
            old += [(50 * i + 11 * k) % 400] + [-(1 + j % 3) for j in range(k)]
    for Hkv in (1, 3):
        for splits in (1, None):
            run(new, old, Hq=2 * Hkv, Hkv=Hkv, splits=splits, D=64 if Hkv == 3 else 128)


@pytest.mark.parametrize("kv", ["fp8_e4m3", "bf16", "fp8_e4m3_block"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_bad_value_of_the_second_tiles_block_stays_there(kv, D):
    """Cells of two tiles of 128 tokens: the first one is done a block before the second, in whose block values are NaN."""
    B, H = 48, 4
    q, starts, lens = batch([256] * B, [0] * B, H, D)
    c = Paged(lens, H, D, 64, kv)
    codes = c.cache.view(torch.int16 if kv == "bf16" else torch.uint8)
    kw = dict(kv_scales=c.scales, k_scale=c.k_scale, v_scale=c.v_scale, num_kv_splits=1)
    want = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1, **kw)
    for t in (130, 170, 230, 255):
        codes[c.table[:, t // 64].long(), 1, t % 64, :, 5] = 0x7fc0 if kv == "bf16" else 0x7f
    sees = (torch.arange(256, device="cuda") >= 130).repeat(B)
    for i in range(40):
        out, lse = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1, **kw)
        assert torch.equal(out[~sees], want[0][~sees]) and torch.equal(lse[~sees], want[1][~sees]), f"call {i}"
        assert bool(torch.isnan(out[sees].float()).any(-1).all())


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 64), (16, 2, 128), (128, 1, 64)])
def test_starts_that_go_up_and_down(Hq, Hkv, D):
    """Every second request claims all tokens: no work is done for them, and the call says so."""
    T, B = 3000, 8192
    q, _, _ = batch([T], [0], Hq, D)
    c = Paged([T], Hkv, D, 64, "bf16")
    starts = torch.tensor([0, T] * (B // 2) + [0], dtype=torch.int32, device="cuda")
    for splits in (1, None):
        out, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
        mqa.gqa_prefill(q, c.cache, c.table.expand(B, -1).contiguous(), c.seq_lens.expand(B).contiguous(), starts, 0.1, out=out,
                        num_kv_splits=splits, device_status=status)
        assert int(status) == 5 and bool((out == 7.0).all())
    run([37], [10])


@pytest.mark.parametrize("scale", [2.0 ** -39, 2.0 ** -42, 2.0 ** -60, 2.0 ** -120])
@pytest.mark.parametrize("kv,D", [("int8_block", 64), ("fp8_e4m3_block", 128)])
@pytest.mark.parametrize("shape", [dict(), dict(slopes=True), dict(cap=30.0)])
def test_tiny_scales_over_blocks_whose_keys_scale_is_zero(shape, kv, D, scale):
    new, old = [300, 40], [170, 300]
    q, starts, lens = batch(new, old, 8, D)
    c = Paged(lens, 2, D, 16, kv, 1, 16)
    for b in (0, 1):
        for group in (0, 3, 4, 10, 20):
            c.scales[int(c.table[b, group]), 0, 0, :] = 0.0
            c.K[b][16 * group:16 * group + 16] = 0.0
    sl = slopes_of(8) if shape.get("slopes") else None
    out, lse = mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, scale, softcap=shape.get("cap", 0.0), slopes=sl,
                               window=150, sinks=3, kv_scales=c.scales)
    for b, at in ((0, 0), (1, 300)):
        k = new[b]
        judge(out[at:at + k], lse[at:at + k], attention(q[at:at + k], c.K[b], c.V[b], old[b], scale, shape.get("cap", 0.0), sl, 150, 3, 0),
              f"request {b}")


def test_splits_beyond_a_c_int_are_taken_at_their_value():
    q, starts, lens = batch([64, 1], [9000, 4000], 32, 128)
    c = Paged(lens, 8, 128, 64, "bf16")
    call = lambda n: mqa.gqa_prefill(q, c.cache, c.table, c.seq_lens, starts, 0.1, num_kv_splits=n)  # noqa: E731
    want = call(2)
    for n in (2 ** 32, 2 ** 32 + 1):
        out, lse = call(n)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(mqa.MqaError):
        call(1 - 2 ** 32)


@pytest.mark.parametrize("cap", [20.0, 34.0, 36.0, 50.0, 57.0, 58.0, 59.0, 60.0, 90.0])
@pytest.mark.parametrize("size", [1.0, 8.0])
def test_caps_over_small_scales_of_the_cache(cap, size):
    """scale k_scale / cap from 1.8e-4 to 3.9e-5, either side of where its ninth power times the cap stops being normal."""
    run([200, 1], [60, 300], cap=cap, size=size, kv="fp8_e4m3")
    run([200, 1], [60, 300], cap=cap, size=size, kv="fp8_e4m3", slopes=True, window=150)


@pytest.mark.parametrize("cap", [1e2, 1e3, 1e5, 3e5, 1e9])
@pytest.mark.parametrize("size", [0.1, 1.0, 30.0])
@pytest.mark.parametrize("D", [64, 128])
def test_caps_far_above_the_scale_of_the_cache(cap, size, D, monkeypatch):
    run([200, 1], [60, 300], cap=cap, size=size, kv="fp8_e4m3", D=D, window=200, sinks=3)
    # With a scale of 1e-5 all weights are alike, and a row's denominator is a sum of up to 300 numbers of one size in four
    # fp32 chains: 75 additions, each rounded by up to 2^-24 of the sum, 300 2^-26 in lse beside what judge() counts.
    monkeypatch.setitem(globals(), "judge", lambda out, lse, ref, what, plain=judge: plain(out, lse, (*ref[:3], ref[3] + 300 * 2.0 ** -26), what))
    run([150, 300], [60, 0], cap=cap, size=size, kv="fp8_e4m3", D=D, prefix=[90, 0], scale=1e-5)
