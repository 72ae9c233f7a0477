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


def half_step(x, kv, s):
    """What a value x may lose in a cache of scale s: half a step of its code, and the rounding of the quotient."""
    if kv.startswith("fp8"):
        return torch.maximum(x.abs() * 2 ** -4, s * 2 ** -10) + x.abs() * 2 ** -20
    return s / 2 + x.abs() * 2 ** -20


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "fp8_e4m3_pth", "int8_pth", "int4_pth"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (32, 8, 128), (3, 3, 128)])
def test_appended_rows_read_back_by_the_decode(kv, Hq, Hkv, D):
    # requests of one token: out is the value, lse the key's column that a query of a single one picks (scale 1)
    torch.manual_seed(2)
    B, page, grp = 40, 16, Hq // Hkv
    row, dtype = {"bf16": (D, BF), "fp8_e4m3": (D, torch.uint8), "int4_pth": (D // 2 + 4, torch.uint8)}.get(
        kv, (D + 4, torch.uint8))
    cache = torch.zeros(B, 2, page, Hkv, row, dtype=dtype, device="cuda")
    if kv == "fp8_e4m3":
        cache = cache.view(torch.float8_e4m3fn)
    name = kv if kv.endswith("pth") else None
    ks, vs = (0.05, 0.03) if kv == "fp8_e4m3" else (1.0, 1.0)
    cs = table(9, D)[8:]  # one angle row, not that of position 0
    bt = torch.randperm(B).to(torch.int32)[:, None]
    k, v = torch.randn(B, Hkv, D).to(BF), torch.randn(B, Hkv, D).to(BF)
    ones = torch.ones(B, dtype=torch.int32, device="cuda")
    mqa.gqa_rope_append(k.cuda(), v.cuda(), cs.cuda(), cache, bt.cuda(), ones,
                        torch.arange(B + 1, dtype=torch.int32, device="cuda"), k_scale=ks, v_scale=vs, kv_dtype=name)
    col = (torch.arange(B)[:, None] * 5 + torch.arange(Hq) * 3) % D
    q = torch.zeros(B, Hq, D).scatter_(2, col[..., None], 1.0).to(BF)
    out, lse = mqa.gqa_paged_decode(q.cuda(), cache, bt.cuda(), ones, 1.0, ks, vs, kv_dtype=name)
    torch.cuda.synchronize()
    out, lse = out.cpu().double(), lse.cpu().double()
    for b in range(B):
        kr, mag = ref.rotate(k[b].double(), cs[0].double(), False)
        for h in range(Hq):
            kk, vv, m = kr[h // grp], v[b, h // grp].double(), mag[h // grp]
            if kv == "bf16":
                ek, ev = kk.abs() * 2 ** -8, torch.zeros_like(vv)
            elif kv == "fp8_e4m3":
                ek, ev = half_step(kk, kv, torch.tensor(ks)), half_step(vv, kv, torch.tensor(vs))
            else:
                ek, ev = (half_step(x, kv, x.abs().max() / ref.Q_MAX[kv] * (1 + 2 ** -20)) for x in (kk, vv))
            assert ((out[b, h] - vv).abs() <= ev + (vv.abs() + ev) * 2 ** -8).all(), (kv, b, h)
            c = int(col[b, h])
            assert abs(lse[b, h] - kk[c]) <= ek[c] + m[c] * 2 ** -21 + kk[c].abs() * 2 ** -20 + 1e-6, (kv, b, h)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("R,H", [(512, 16), (512, 128), (256, 16)])
def test_appended_latent_rows_read_back_by_the_decode(fp8, R, H):
    torch.manual_seed(3)
    B, page, ks = 24, 16, 0.05 if fp8 else 1.0
    cache = torch.zeros(B, page, R + 64, dtype=torch.uint8 if fp8 else BF, device="cuda")
    if fp8:
        cache = cache.view(torch.float8_e4m3fn)
    cs = table(9, 64)[8:]
    bt = torch.randperm(B).to(torch.int32)[:, None]
    a = torch.randn(B, R + 64).to(BF)
    ones = torch.ones(B, dtype=torch.int32, device="cuda")
    da = a.cuda()
    mqa.mla_rope_append(da[:, :R], da[:, R:], cs.cuda(), cache, bt.cuda(), ones,
                        torch.arange(B + 1, dtype=torch.int32, device="cuda"), k_scale=ks)
    col = (torch.arange(B)[:, None] * 5 + torch.arange(H) * 37) % (R + 64)
    q = torch.zeros(B, H, R + 64).scatter_(2, col[..., None], 1.0).to(BF)
    out, lse = mqa.mla_decode(q.cuda(), cache, bt.cuda(), ones, 1.0, ks)
    torch.cuda.synchronize()
    out, lse = out.cpu().double(), lse.cpu().double()
    for b in range(B):
        turned, mag = ref.rotate(a[b, None, R:].double(), cs[0].double(), False)
        x = torch.cat([a[b, :R].double(), turned[0]])
        m = torch.cat([torch.zeros(R, dtype=torch.float64), mag[0]])
        e = half_step(x, "fp8_e4m3", torch.tensor(ks)) if fp8 else x.abs() * 2 ** -8
        e += m * 2 ** -21
        assert ((out[b] - x[:R]).abs() <= e[:R] + (x[:R].abs() + e[:R]) * 2 ** -8).all(), b
        assert ((lse[b] - x[col[b]]).abs() <= e[col[b]] + x[col[b]].abs() * 2 ** -20 + 1e-6).all(), b
