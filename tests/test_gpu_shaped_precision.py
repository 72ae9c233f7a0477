"""How exact attention with shaped logits is where biases are steep and caps far from the logits: a key's error counts by
the key's own weight, so that a head whose bias leaves a few keys is held to those; where logits are so large that only
their order counts, results are held to lie among the values."""
import math

import pytest
import torch

import mqa_decode_attention_paged_gb300 as mqa
from attention_reference import NO_WINDOW, Paged

pytestmark = pytest.mark.gpu


def logits(q, K, first, scale, cap, slopes, window, sinks):
    """Logits x [w, Hkv, grp, n] in 64 bits (-inf: not seen) and bounds d of their errors in the kernels: D products summed
    in fp32 (D 2^-24 of their absolute sum); the cap (2^-18 of the logit, 2^-21 of the cap at most); slope and bias rounded
    (2^-22 of the bias), a bias put together from that of 32 keys (of slopes up to 64 ln 2 / 31, steeper ones are not);
    the logit less a reference (2^-23 of both; a reference may be a bound, 64 above the largest)."""
    w, Hq, D = q.shape
    n, Hkv = K.shape[:2]
    p = first + torch.arange(w, device=q.device)[:, None]
    t = torch.arange(n, device=q.device)[None]
    seen = ((t <= p) & ((t < sinks) | (t > p - window)) & (p >= 0))[:, None, None]
    qd = q.double().view(w, Hkv, Hq // Hkv, D)
    x = torch.einsum("whgd,nhd->whgn", qd, K) * scale
    d = torch.einsum("whgd,nhd->whgn", qd.abs(), K.abs()) * (abs(scale) * D * 2.0 ** -24)
    if cap:
        x = cap * torch.tanh(x / cap)
        d = d + torch.clamp(x.abs() * 2.0 ** -18, max=cap * 2.0 ** -21)
    if slopes is not None:
        sl = slopes.double().view(1, Hkv, Hq // Hkv, 1)
        bias = sl * (p - t).abs().double()[:, None, None]
        x = x - bias
        d = d + bias.abs() * 2.0 ** -22 + sl.abs().clamp(max=1.5) * 32 * 2.0 ** -22
    x = x.masked_fill(~seen, -math.inf)
    return x, torch.where(seen, d + (x.abs() + x.amax(-1, keepdim=True).abs() + 64) * 2.0 ** -23, 0.0)


def judge(out, lse, x, d, V, codes, what):
    """lse is off by at most ln sum P_t e^{d_t}, P_t then by the factor e^{d_t} times that; sums of k fp32 numbers by k 2^-26
    of themselves (four or more chains of them; k: keys that are not lost beside the largest), exponential and logarithm by
    2^-20.  P and the output are rounded to bf16 (2^-8 each), with a tenth of that for fp32 sums of up to 6000 products.
    codes: those of a kernel that keeps numerators in f16 (2^-25 of the largest, times each code)."""
    w, Hkv, grp, n = x.shape
    want = torch.logsumexp(x, -1, keepdim=True)
    P = torch.exp(x - want)
    lse_tol = torch.logsumexp(x - want + d, -1, keepdim=True) + (P > 2.0 ** -25).sum(-1, keepdim=True) * 2.0 ** -26 + 2.0 ** -20
    y, mass, off = (torch.einsum("whgn,nhd->whgd", a, b) for a, b in ((P, V), (P, V.abs()), (torch.exp(x - want + d + lse_tol) - P, V.abs())))
    tol = (y.abs() + 1.1 * mass) * 2.0 ** -8 + 1.1 * off + 1e-30
    if codes is not None:
        code, s_v = codes
        largest = (P * s_v.T.view(1, Hkv, 1, n)).amax(-1, keepdim=True)
        tol = tol + 2.0 ** -25 * largest * torch.einsum("whgn,nhd->whgd", (x > -math.inf).double(), code)
    for got, ref, t, name in ((out.view(y.shape), y, tol, "outputs"), (lse.view(w, Hkv, grp, 1), want, lse_tol, "lse")):
        bad = ~((got.double() - ref).abs() <= t)
        assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} {name} off, first at {bad.nonzero()[0].tolist()}: "
                               f"{got[bad][:4].tolist()} for {ref[bad][:4].tolist()} within {t[bad][:4].tolist()}")


def decode(c, lens, q, scale, cap, slopes, window, sinks):
    out, lse = mqa.gqa_score_decode(q, c.cache, c.table, c.seq_lens, scale, softcap=cap, slopes=slopes, window=window, sinks=sinks,
                                    kv_scales=c.scales, k_scale=c.k_scale, v_scale=c.v_scale)
    return [(q[b], out[b], lse[b], n - q.shape[1], c.codes[b]) for b, n in enumerate(lens)]


def prompt(c, lens, q, scale, cap, slopes, window, sinks):
    B, L = q.shape[:2]
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * L
    flat = q.view(B * L, *q.shape[2:])
    out, lse = mqa.gqa_prefill(flat, c.cache, c.table, c.seq_lens, starts, scale, softcap=cap, slopes=slopes, window=window,
                               sinks=sinks, kv_scales=c.scales, k_scale=c.k_scale, v_scale=c.v_scale)
    return [(q[b], out.view(q.shape)[b], lse.view(q.shape[:3])[b], n - L, None) for b, n in enumerate(lens)]


SLOPES = [[0.0, -0.05, 5.0, 1e4, 1.4, 1.5, -3.0, 1e-6], [1.42, 0.3, 2.0, -1.0, 0.0, 0.5, 64.0, 1.0], [1e7, 1e-3, 1.43, 1.44, 0.7, 9.0, 30.0, 0.1]]


@pytest.mark.parametrize("call,L", [(decode, 1), (decode, 5), (prompt, 5), (prompt, 150)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("kv,group,D", [("bf16", 0, 128), ("bf16", 0, 64), ("fp8_e4m3", 0, 128), ("fp8_e4m3_block", 16, 64),
                                        ("int8_block", 16, 128)])
def test_steep_biases(kv, group, D, cap, call, L):
    lens = [300, L, 3000, 777]
    c = Paged(lens, 2, D, 16, kv, 5, group)
    g = torch.Generator(device="cuda").manual_seed(6)
    q = torch.randn(len(lens), L, 8, D, generator=g, device="cuda").to(torch.bfloat16)
    for slopes in SLOPES:
        for window, sinks in ((NO_WINDOW, 0), (70, 2)):
            sl = torch.tensor(slopes, device="cuda")
            for b, (qb, out, lse, first, codes) in enumerate(call(c, lens, q, D ** -0.5, cap, sl, window, sinks)):
                x, d = logits(qb, c.K[b], first, D ** -0.5, cap, sl, window, sinks)
                judge(out, lse, x, d, c.V[b], codes, f"request {b}, slopes {slopes}, window {window}")


@pytest.mark.parametrize("call,L", [(decode, 1), (decode, 3), (prompt, 3), (prompt, 150)])
@pytest.mark.parametrize("cap,scale,biased", [(2.0 ** 60, 2.0 ** 48, False), (2.0 ** 60, 2.0 ** 30, False), (2.0 ** 60, 2.0 ** 30, True),
                                              (0.0, 2.0 ** 18, False), (0.0, 2.0 ** 15, True), (0.0, 2.0 ** 8, True)])
@pytest.mark.parametrize("kv", ["bf16", "int8_block"])
def test_logits_whose_order_alone_counts(kv, cap, scale, biased, call, L):
    """Which key is the largest may be a matter of rounding here: lse is as exact as the logits, outputs lie among the
    values that are seen (2^-8 of them for the rounding of each of P and the output).  Without a cap logits are within the
    2^30 that the contract allows, with slopes 2^26: they are up to 1690 times the scale (over these int8 blocks), so a scale
    of 2^20 is beyond it.

    The decode kernel adds the logarithm of V's scale to the exponent of codes, beside two references of the logit's size:
    four roundings of 2^-24 of the largest logit, by which the outputs as a whole are off (over codes and with the larger
    scales here that says no more than that they are finite)."""
    lens = [300, 160]
    c = Paged(lens, 2, 128, 16, kv, 7, 16)
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn(2, L, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    sl = torch.tensor(SLOPES[1], device="cuda") if biased else None
    for b, (qb, out, lse, first, _) in enumerate(call(c, lens, q, scale, cap, sl, NO_WINDOW, 0)):
        x, d = logits(qb, c.K[b], first, scale, cap, sl, NO_WINDOW, 0)
        want, tol = torch.logsumexp(x, -1), d.amax(-1) + math.log(lens[b])
        assert bool(((lse.view(want.shape).double() - want).abs() <= tol).all()), f"request {b}: lse"
        for i in range(L):
            V = c.V[b][:first + i + 1]
            lo, hi = V.amin(0)[:, None], V.amax(0)[:, None]
            y, slack = out[i].double().view(2, 4, 128), 2 * 2.0 ** -8
            if call is decode and kv != "bf16":
                slack = slack + torch.expm1((x[i].abs().masked_fill(x[i] == -math.inf, 0.0).amax(-1, keepdim=True) * 2.0 ** -22).clamp(max=50))
            slack = slack * V.abs().amax(0)[:, None]
            assert bool(((y >= lo - slack) & (y <= hi + slack)).all()), f"request {b}, query {i}"
