"""The append and decode operators run together, as a serving loop runs them:
prompts appended, then tokens one at a time (or a few at once), each step's
decode reading what the appends wrote; also captured into a graph and
replayed.  The reference attends, in 64 bits, over the cache as it stands."""
import pytest
import torch

import cache_reference as ref
import mqa_decode_attention_paged_gb300 as mqa
from test_gpu_append import BF, table

pytestmark = pytest.mark.gpu


def attend(q, cache, scales, bt, lens, page, window, sinks, D, kv):
    for b, n in enumerate(lens):
        codes = [ref.gather(cache, bt, b, n, page, i) for i in (0, 1)]
        s = [ref.token_scales(scales, bt, b, n, page, i) if scales is not None
             else torch.ones(n, cache.shape[3], dtype=torch.float64) for i in (0, 1)]
        yield ref.window_decode(q[b].double(), codes[0] * s[0][..., None], codes[1] * s[1][..., None], n, D ** -0.5,
                                window, sinks, code_v=codes[1], s_v=s[1], half_p=kv != "bf16")


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3_block", "int8_block"])
@pytest.mark.parametrize("L", [1, 3])
def test_prefill_then_steps(kv, L):
    torch.manual_seed(0)
    B, Hq, Hkv, D, page, window, sinks = 3, 8, 2, 64, 32, 40, 4
    prompts, steps = [37, 1, 70], 6
    bt = torch.randperm(15)[:15].view(B, 5).to(torch.int32)
    cs = table(200, D).cuda()
    dtype = {"bf16": BF, "fp8_e4m3_block": torch.float8_e4m3fn, "int8_block": torch.int8}[kv]
    cache = torch.zeros(15, 2, page, Hkv, D, dtype=torch.uint8 if kv != "bf16" else BF, device="cuda").view(dtype)
    scales = None if kv == "bf16" else torch.zeros(15, 2, 2, Hkv, device="cuda")
    dbt = bt.cuda()

    qkv = torch.randn(sum(prompts), Hq + 2 * Hkv, D).to(BF).cuda()
    starts = torch.tensor([0, 37, 38, 108], dtype=torch.int32, device="cuda")
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    mqa.gqa_rope_append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], cs, cache, dbt, lens, starts, q=qkv[:, :Hq],
                        q_out=qkv[:, :Hq], kv_scales=scales)

    # one step, captured: append L tokens of each request, then decode them
    x = torch.zeros(B * L, Hq + 2 * Hkv, D, dtype=BF, device="cuda")
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * L

    def step():
        q = mqa.gqa_rope_append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cs, cache, dbt, lens, starts, q=x[:, :Hq],
                                kv_scales=scales)
        q = q.view(B, L, Hq, D)
        win = mqa.gqa_window_decode(q, cache, dbt, lens, D ** -0.5, window, sinks, kv_scales=scales)
        full = mqa.gqa_block_decode(q, cache, scales, dbt, lens, D ** -0.5) if scales is not None else None
        return q, win, full

    keep = cache.clone(), None if scales is None else scales.clone()
    lens += L
    step()  # warm-up, undone
    torch.cuda.synchronize()
    cache.copy_(keep[0])
    if scales is not None:
        scales.copy_(keep[1])
    lens -= L
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for i in range(steps):
        x.copy_(torch.randn(x.shape).to(BF))
        lens += L
        if i % 2:
            graph.replay()
            got = res
        else:
            got = step()
        torch.cuda.synchronize()
        q, (out, lse), full = got
        n = lens.tolist()
        c, s = cache.cpu(), None if scales is None else scales.cpu()
        for w, sk, pair in ((window, sinks, (out, lse)), (1 << 30, 0, full)):
            if pair is None:
                continue
            o, l = pair[0].cpu().double(), pair[1].cpu().double()
            for b, (ro, rl, to, tl) in enumerate(attend(q.cpu(), c, s, bt, n, page, w, sk, D, kv)):
                assert ((o[b] - ro).abs() <= to).all(), (kv, i, b, w)
                assert ((l[b] - rl).abs() <= tl).all(), (kv, i, b, w)


def test_mla_append_feeds_the_decode():
    # rows written by mla_rope_append, read by mla_decode
    torch.manual_seed(1)
    B, H, R, page = 2, 16, 512, 16
    lens = [20, 5]
    bt = torch.tensor([[2, 0], [1, 3]], dtype=torch.int32)
    cs = table(64, 64).cuda()
    cache = torch.zeros(4, page, R + 64, dtype=BF, device="cuda")
    a = torch.randn(25, R + 64).to(BF).cuda()
    q = torch.randn(25, H, R + 64).to(BF).cuda()
    starts = torch.tensor([0, 20, 25], dtype=torch.int32, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    mqa.mla_rope_append(a[:, :R], a[:, R:], cs, cache, bt.cuda(), sl, starts, q_pe=q[..., R:], q_pe_out=q[..., R:])
    last = q[[19, 24]].contiguous()
    out, lse = mqa.mla_decode(last, cache, bt.cuda(), sl, 192 ** -0.5)
    torch.cuda.synchronize()
    rows = cache.cpu().double()
    for b, n in enumerate(lens):
        k = torch.cat([rows[int(j)] for j in bt[b]])[:n]
        x = last[b].cpu().double() @ k.T * 192 ** -0.5
        p = torch.softmax(x, -1)
        o = p @ k[:, :R]
        # P and the output rounded to bf16 (2^-8 each), P.V a convex sum
        bound = 2 ** -8 * (p @ k[:, :R].abs()) + 2 ** -8 * o.abs() + 1e-4
        assert ((out[b].cpu().double() - o).abs() <= bound).all()
        assert (lse[b].cpu().double() - torch.logsumexp(x, -1)).abs().max() <= 1e-3
