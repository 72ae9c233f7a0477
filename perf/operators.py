"""The cases on which the cache-append and the windowed / block-scaled decode operators are measured.

Four operators of a serving step over paged caches:

  gqa_append   new keys and values of a ragged batch, rotated to their positions, into a paged GQA cache
               (and the rotated queries beside them);
  mla_append   new latent rows [kv_c | k_pe], k_pe rotated, into a paged MLA cache (and the rotated q_pe
               into the absorbed query);
  window       GQA decode over a sliding window and the first `sinks` tokens, 1 or more new positions;
  block        GQA decode over an 8-bit cache with one scale per block of tokens and head.

A case is a dict of plain values; lengths come from its own "lens_seed", values from the seed given to prepare().
"""
import math

import numpy as np
import torch

own = False

Q_MAX = {"fp8_e4m3_block": 448.0, "int8_block": 127.0}
TINY = 2.0 ** -126  # block scales are zero or normal fp32 numbers


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a full batch: a new token for each of 256 requests, heads and pages of the GQA benchmark
        dict(name="append decode bf16", op="gqa_append", B=256, new="1,1", old="1,2000", pad=0, Hq=32, Hkv=8, D=128,
             page=16, kv="bf16", group=0, rot=128, inter=False, fused=True, lens_seed=1),
        # prefill of a few prompts at once, from the slices of a fused projection, padded to a captured size
        dict(name="append prefill e4m3 blocks", op="gqa_append", B=6, new="500,2600", old="0,100", pad=13, Hq=32,
             Hkv=8, D=128, page=64, kv="fp8_e4m3_block", group=64, rot=128, inter=False, fused=True, lens_seed=2),
        # a few speculative tokens per request, small heads, half of each rotated, pairs side by side
        dict(name="append few int8 blocks", op="gqa_append", B=7, new="1,9", old="0,900", pad=2, Hq=12, Hkv=4, D=64,
             page=32, kv="int8_block", group=16, rot=32, inter=True, fused=False, lens_seed=3),
        # one decode step of the V3-like MLA batch: 128 requests, 128 heads, e4m3 latent rows
        dict(name="mla append decode e4m3", op="mla_append", B=128, new="1,1", old="4096,9000", pad=0, H=128, R=512,
             page=64, kv="fp8_e4m3", inter=True, lens_seed=4),
        # prompts of the V2-Lite-like shape (16 heads, bf16 latent rows)
        dict(name="mla append prefill bf16", op="mla_append", B=3, new="700,1500", old="0,50", pad=5, H=16, R=512,
             page=64, kv="bf16", inter=True, lens_seed=5),
        # the smallest call: one request, one token, a short window; latency
        dict(name="window one request", op="window", B=1, L=1, lens="300,300", W=128, S=4, Hq=32, Hkv=8, D=128,
             page=16, kv="bf16", group=0, lens_seed=6),
        # streaming decode of an ordinary batch: 4 sinks and the last 1024 tokens of long and short contexts
        dict(name="window 1024 bf16", op="window", B=64, L=1, lens="1,16384", W=1024, S=4, Hq=32, Hkv=8, D=128,
             page=16, kv="bf16", group=0, lens_seed=7),
        # verification of 4 positions under a long window, 8-bit cache with a scale per 64-token page and head
        dict(name="window 4096 x4 e4m3 blocks", op="window", B=32, L=4, lens="500,20000", W=4096, S=128, Hq=32,
             Hkv=8, D=128, page=64, kv="fp8_e4m3_block", group=64, lens_seed=8),
        # a large batch of short windows, 8 query heads to a KV head, head size 64
        dict(name="window 128 int8 blocks", op="window", B=256, L=1, lens="1,5000", W=128, S=1, Hq=64, Hkv=8, D=64,
             page=32, kv="int8_block", group=32, lens_seed=9),
        # the tiny batch of the tests: two short requests
        dict(name="block tiny e4m3", op="block", B=2, L=1, lens="37,100", Hq=8, Hkv=2, D=128, page=16,
             kv="fp8_e4m3_block", group=16, lens_seed=10),
        # the GQA benchmark's batch (256 requests, lognormal lengths) over block-scaled e4m3
        dict(name="block batch e4m3", op="block", B=256, L=1, lens="lognormal 2048,16384", Hq=32, Hkv=8, D=128,
             page=16, kv="fp8_e4m3_block", group=16, lens_seed=11),
        # four very long contexts
        dict(name="block long int8", op="block", B=4, L=1, lens="65536,131072", Hq=32, Hkv=8, D=128, page=64,
             kv="int8_block", group=32, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gqa_append", "mla_append", "window", "block"])
    c = dict(op=op, lens_seed=rng.randrange(1 << 30))
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    if op in ("gqa_append", "mla_append"):
        if rng.random() < 0.5:
            c.update(B=_log_int(rng, 1, 256), new="1,%d" % rng.choice([1, 1, 4, 7]))
        else:
            c.update(B=rng.randint(1, 8), new="1,%d" % _log_int(rng, 20, 1500))
        c.update(old="0,%d" % _log_int(rng, 10, 3000), pad=rng.choice([0, 0, 1, 9]), page=page,
                 inter=rng.random() < 0.5)
        if op == "mla_append":
            c.update(H=_log_int(rng, 1, 128), R=rng.choice([256, 512]), kv=rng.choice(["bf16", "fp8_e4m3"]))
        else:
            kv = rng.choice(["bf16", "fp8_e4m3_block", "int8_block"])
            c.update(Hq=Hkv * rng.choice([1, 3, 4, 8]), Hkv=Hkv, D=D, kv=kv, rot=rng.choice([D, D, D // 2]),
                     fused=rng.random() < 0.5, group=0 if kv == "bf16" else rng.choice([16, page]))
        return c
    kv = rng.choice(["fp8_e4m3_block", "int8_block"] + (["bf16"] if op == "window" else []))
    L = rng.choice([1, 1, 2, 5])
    B = _log_int(rng, 1, 128)
    hi = min(_log_int(rng, 16, 30000), max(16, 250000 // B))
    c.update(B=B, L=L, lens="%d,%d" % (rng.choice([1, hi // 2 + 1, hi]), hi), Hq=Hkv * rng.choice([1, 2, 4, 7, 8, 16]),
             Hkv=Hkv, D=D, page=page, kv=kv, group=0 if kv == "bf16" else rng.choice([16, page]))
    if op == "window":
        c.update(W=_log_int(rng, 1, 4096), S=rng.choice([0, 1, 4, 17, 64]))
    return c


def _range(text, rng, B):
    if text.startswith("lognormal"):
        median, top = (int(x) for x in text.split()[1].split(","))
        return np.clip(np.ceil(np.exp(rng.normal(math.log(median), 1.0, B))), 1, top).astype(np.int64)
    lo, hi = (int(x) for x in text.split(","))
    return rng.integers(lo, hi + 1, B)


def _lengths(c):
    """(new tokens of each request, lengths with them) as numpy."""
    rng = np.random.default_rng(c["lens_seed"])
    if c["op"].endswith("append"):
        new = _range(c["new"], rng, c["B"])
        return new, new + _range(c["old"], rng, c["B"])
    n = _range(c["lens"], rng, c["B"])
    if c["B"] == 2 and c["lens"] == "37,100":
        n = np.array([37, 100])
    return np.full(c["B"], c["L"]), n


def _elt(kv):
    return 2 if kv == "bf16" else 1


def work(c):
    new, n = _lengths(c)
    T = int(new.sum())
    if c["op"].endswith("append"):
        rows = len(np.unique(np.concatenate([np.arange(b - a, b) for a, b in zip(new, n)])))
        if c["op"] == "mla_append":
            b = T * ((c["R"] + 64) * (2 + _elt(c["kv"])) + 2 * c["H"] * 64 * 2) + rows * 64 * 4
            return {"bytes": b, "flops": T * (c["H"] + 1) * 64 * 3}
        b = T * (2 * c["Hq"] * c["D"] * 2 + 2 * c["Hkv"] * c["D"] * (2 + _elt(c["kv"]))) + rows * c["rot"] * 4
        if c["group"]:
            blocks = int(((n + c["group"] - 1) // c["group"] - (n - new) // c["group"]).sum())
            b += blocks * 2 * c["Hkv"] * 4
        return {"bytes": b, "flops": T * (c["Hq"] + c["Hkv"]) * c["rot"] * 3}
    L, seen, pairs = c["L"], 0, 0
    for m in n.tolist():
        W, S = (c["W"], c["S"]) if c["op"] == "window" else (m + 1, 0)
        lo = max(0, m - L - W + 1)
        seen += m - lo + min(S, lo)
        for i in range(L):
            p = m - L + i
            if p >= 0:
                first = max(0, p - W + 1)
                pairs += p + 1 - first + min(S, first)
    b = seen * 2 * c["Hkv"] * c["D"] * _elt(c["kv"]) + 2 * c["B"] * L * c["Hq"] * c["D"] * 2 + c["B"] * L * c["Hq"] * 4
    if c["group"]:
        b += seen // c["group"] * 2 * c["Hkv"] * 4
    return {"bytes": b, "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---------------------------------------------------------------------------- inputs

def _quantised(x, kv):
    """Codes and scales of values [blocks, 2, groups, tokens, heads, D]: one scale for each group and head."""
    s = x.abs().amax(dim=(3, 5), keepdim=True).float() / Q_MAX[kv]
    y = x.float().div_(s)
    if kv == "int8_block":
        return y.round_().to(torch.int8), s
    return y.clamp_(-448, 448).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    new, n = _lengths(c)
    page, B, kv = c["page"], c["B"], c["kv"]
    pages = -(-n // page)
    nb = int(pages.sum()) + 3
    perm = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    width = max(1, int(pages.max()))
    first = np.concatenate([[0], np.cumsum(pages)])
    cols = torch.arange(width, device=dev)
    at = torch.from_numpy(first[:-1]).to(dev)[:, None] + cols
    has = cols < torch.from_numpy(pages).to(dev)[:, None]
    bt = torch.where(has, perm[at.clamp(max=nb - 1)], -1).to(torch.int32).contiguous()
    s = dict(case=c, bt=bt, lens=torch.from_numpy(n.astype(np.int32)).to(dev), nb=nb, max_len=int(n.max()))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    if c["op"] == "mla_append":
        cache = randn(nb, page, c["R"] + 64)
        s["k_scale"] = 0.05 if kv == "fp8_e4m3" else 1.0
        s["cache"] = cache if kv == "bf16" else cache.div_(0.05).clamp_(-448, 448).to(torch.float8_e4m3fn)
    elif c["group"]:
        G = c["group"]
        x = randn(nb, 2, page // G, G, c["Hkv"], c["D"])
        x *= torch.exp(0.5 * randn(nb, 2, page // G, 1, c["Hkv"], 1))  # blocks and heads of unlike magnitude
        codes, scales = _quantised(x, kv)
        s["cache"] = codes.view(nb, 2, page, c["Hkv"], c["D"])
        s["scales"] = scales.view(nb, 2, page // G, c["Hkv"]).contiguous()
    else:
        s["cache"], s["scales"] = randn(nb, 2, page, c["Hkv"], c["D"]), None

    if not c["op"].endswith("append"):
        s["q"] = randn(B, c["L"], c["Hq"], c["D"])
        s["scale"] = 1.0 / math.sqrt(c["D"])
        return s

    T = int(new.sum()) + c["pad"]
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s.update(T=int(new.sum()), max_new=int(new.max()), query_start=torch.from_numpy(starts).to(dev))
    rot = 64 if c["op"] == "mla_append" else c["rot"]
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
    angle = torch.arange(int(n.max()) + 8, device=dev, dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    if c["op"] == "mla_append":
        R, H = c["R"], c["H"]
        kv_a = randn(T, R + 64)  # one projection gives both parts of the row
        s.update(kv_c=kv_a[:, :R], k_pe=kv_a[:, R:], q_pe=randn(T, H, 192)[..., 128:], q=torch.zeros(T, H, R + 64, dtype=torch.bfloat16, device=dev))
        s["q_pe_out"] = s["q"][..., R:]
        return s
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["fused"]:
        qkv = randn(T, Hq + 2 * Hkv, D)
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:])
    else:
        s.update(q=randn(T, Hq, D), k=randn(T, Hkv, D), v=randn(T, Hkv, D))
    s["q_out"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------------------- plain forms

def _positions(s):
    """Request and position of each new token."""
    t = torch.arange(s["T"], device=s["bt"].device)
    b = torch.searchsorted(s["query_start"][1:].long(), t, right=True)
    return b, s["lens"].long()[b] - s["query_start"].long()[b + 1] + t


def _rotated(x, cs, inter):
    """x [T, heads, D] in fp32, its first cs.shape[1] columns rotated by the tokens' cos | sin rows."""
    r = cs.shape[1]
    cos, sin = cs[:, None, :r // 2], cs[:, None, r // 2:]
    if inter:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _codes(x, kv):
    if kv == "int8_block":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _bytes(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _cells(cache, *at):
    """The cells of a cache at advanced indices, whatever its type."""
    return _bytes(cache)[at].view(cache.dtype)


def _plain_mla_append(s):
    c, T = s["case"], s["T"]
    b, pos = _positions(s)
    cs = s["cos_sin"][pos]
    row = torch.cat([s["kv_c"][:T].float(), _rotated(s["k_pe"][:T, None].float(), cs, c["inter"])[:, 0]], -1)
    blk = s["bt"].long()[b, pos // c["page"]]
    row = row.to(torch.bfloat16) if c["kv"] == "bf16" else _codes(row / s["k_scale"], "e4m3")
    _bytes(s["cache"])[blk, pos % c["page"]] = _bytes(row)
    s["q_pe_out"][:T] = _rotated(s["q_pe"][:T].float(), cs, c["inter"]).to(torch.bfloat16)
    return s["q_pe_out"], s["cache"]


def _plain_gqa_append(s):
    c, T, page, G, kv = s["case"], s["T"], s["case"]["page"], s["case"]["group"], s["case"]["kv"]
    b, pos = _positions(s)
    cs = s["cos_sin"][pos]
    s["q_out"][:T] = _rotated(s["q"][:T].float(), cs, c["inter"]).to(torch.bfloat16)
    x = torch.stack([_rotated(s["k"][:T].float(), cs, c["inter"]), s["v"][:T].float()], 1)  # [T, 2, Hkv, D]
    blk, slot = s["bt"].long()[b, pos // page], pos % page
    cache = s["cache"]
    if not G:
        cache[blk, :, slot] = x.to(torch.bfloat16)
        return s["q_out"], cache
    # one scale for each group of G tokens: it grows to hold the new tokens, a group that starts anew forgets its own
    per = page // G
    scales = s["scales"].permute(0, 2, 1, 3).reshape(-1, 2, c["Hkv"])
    gid = blk * per + slot // G
    anew = torch.zeros(scales.shape[0], dtype=torch.bool, device=x.device).index_fill_(0, gid[pos % G == 0], True)
    top = torch.zeros_like(scales).index_reduce_(0, gid, x.abs().amax(-1), "amax") / Q_MAX[kv]
    held = torch.where(anew[:, None, None], 0.0, scales)
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=x.device).index_fill_(0, gid, True)
    grown = torch.maximum(held, torch.where(top < TINY, 0.0, top))
    final = torch.where(touched[:, None, None], grown, scales)
    # the tokens that a request's first group held before
    start = s["lens"].long() - (s["query_start"][1:] - s["query_start"][:-1]).long()
    blk0 = s["bt"].long().gather(1, (start // page)[:, None])[:, 0]
    gid0 = blk0 * per + start % page // G
    at = (start % page // G * G)[:, None] + torch.arange(G, device=x.device)
    was = torch.arange(G, device=x.device) < (start % G)[:, None]
    old = _cells(cache, blk0[:, None], slice(None), at)  # [B, G, 2, Hkv, D]
    ratio = torch.where(final[gid0] > 0, scales[gid0] / final[gid0], 0.0)[:, None, :, :, None]
    moved = _codes(old.float() * ratio, kv)
    _bytes(cache)[blk0[:, None], :, at] = torch.where(was[:, :, None, None, None], _bytes(moved), _bytes(old))
    f = final[gid][..., None]
    _bytes(cache)[blk, :, slot] = _bytes(_codes(torch.where(f > 0, x / f, 0.0), kv))
    s["scales"].copy_(final.view(s["nb"], per, 2, c["Hkv"]).permute(0, 2, 1, 3))
    return _appended(s)


def _appended(s):
    """What an append into a block-scaled cache leaves: e4m3 codes and scales, or int8 codes as the values they stand for."""
    if s["case"]["kv"] == "fp8_e4m3_block":
        return s["q_out"], s["cache"], s["scales"]
    per_token = s["scales"].repeat_interleave(s["case"]["group"], 2)[..., None]
    return s["q_out"], (s["cache"] * per_token).to(torch.bfloat16), s["scales"]


def _plain_decode(s):
    c = s["case"]
    B, L, Hq, Hkv, D, page, G = c["B"], c["L"], c["Hq"], c["Hkv"], c["D"], c["page"], c["group"]
    dev = s["bt"].device
    n = s["lens"].long()[:, None]
    S, W = (c["S"], c["W"]) if c["op"] == "window" else (0, s["max_len"] + 1)
    wide = min(W + L - 1, s["max_len"])
    lo = (n - wide).clamp(min=0)
    pos = torch.cat([torch.arange(S, device=dev).expand(B, S), lo + torch.arange(wide, device=dev)], 1)
    first = torch.cat([torch.ones(S, dtype=torch.bool, device=dev), torch.zeros(wide, dtype=torch.bool, device=dev)])
    ok = (pos < n) & (first | (pos >= S) | (S == 0))
    at = torch.where(ok, pos, 0)
    blk, slot = s["bt"].long().gather(1, at // page), at % page
    qp = n - L + torch.arange(L, device=dev)
    seen = ok[:, None] & (pos[:, None] <= qp[..., None]) & ((pos[:, None] < S) | (pos[:, None] > qp[..., None] - W))

    def plane(i):
        x = _cells(s["cache"], blk, i, slot).float()  # [B, keys, Hkv, D]
        if G:
            x *= s["scales"][blk, i, slot // G][..., None]
        return x.masked_fill_(~ok[..., None, None], 0.0).transpose(1, 2)

    q = s["q"].float().view(B, L, Hkv, Hq // Hkv, D).transpose(1, 2).reshape(B, Hkv, -1, D)
    x = (q @ plane(0).transpose(-1, -2)).view(B, Hkv, L, Hq // Hkv, -1) * s["scale"]
    x = x.masked_fill(~seen[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ plane(1)).view(B, Hkv, L, Hq // Hkv, D)
    out = torch.where(total > 0, o / total, 0.0).transpose(1, 2).reshape(B, L, Hq, D).to(torch.bfloat16)
    return out, (m + torch.log(total))[..., 0].transpose(1, 2).reshape(B, L, Hq)


# ---------------------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"gqa_append": _plain_gqa_append, "mla_append": _plain_mla_append}.get(c["op"], _plain_decode)(s)
    import mqa_decode_attention_paged_gb300 as mqa
    if c["op"] == "mla_append":
        mqa.mla_rope_append(s["kv_c"], s["k_pe"], s["cos_sin"], s["cache"], s["bt"], s["lens"], s["query_start"],
                            q_pe=s["q_pe"], q_pe_out=s["q_pe_out"], k_scale=s["k_scale"], interleaved=c["inter"])
        return s["q_pe_out"], s["cache"]
    if c["op"] == "gqa_append":
        mqa.gqa_rope_append(s["k"], s["v"], s["cos_sin"], s["cache"], s["bt"], s["lens"], s["query_start"], q=s["q"],
                            q_out=s["q_out"], kv_scales=s["scales"], interleaved=c["inter"])
        return _appended(s) if c["group"] else (s["q_out"], s["cache"])
    if "out" not in s:  # a serving program keeps its outputs and workspace from step to step
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:3], dtype=torch.float32, device=s["q"].device)
        s["splits"] = mqa.gqa_window_num_kv_splits(c["B"], c["L"], c["Hq"], c["Hkv"])
        need = mqa.gqa_window_decode_workspace_bytes(c["B"], c["L"], c["Hq"], c["Hkv"], c["D"], s["splits"])
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=s["q"].device)
    kept = dict(out=s["out"], lse=s["lse"], num_kv_splits=s["splits"], workspace=s["workspace"])
    if c["op"] == "window":
        return mqa.gqa_window_decode(s["q"], s["cache"], s["bt"], s["lens"], s["scale"], c["W"], c["S"],
                                     kv_scales=s["scales"], **kept)
    return mqa.gqa_block_decode(s["q"], s["cache"], s["scales"], s["bt"], s["lens"], s["scale"], **kept)


# ---------------------------------------------------------------------------- the definition in 64 bits

def _grid_e4m3(y):
    """The nearest e4m3 value (ties to even), in 64 bits."""
    y = y.clamp(-448.0, 448.0)
    e = torch.frexp(y.abs())[1].double() - 1.0
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.round(y / step) * step


def _grid(y, kv):
    return torch.round(y).clamp(-127.0, 127.0) if kv == "int8_block" else _grid_e4m3(y)


def _turn(x, table, inter):
    """x [n, heads, D] in 64 bits turned pair by pair as complex numbers."""
    r = table.shape[1]
    w = torch.complex(table[:, :r // 2], table[:, r // 2:])[:, None]
    head = x[..., :r].unflatten(-1, (r // 2, 2) if inter else (2, r // 2))
    z = (torch.complex(head[..., 0], head[..., 1]) if inter else torch.complex(head[..., 0, :], head[..., 1, :])) * w
    y = torch.stack([z.real, z.imag], -1 if inter else -2).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    bt, page = s["bt"].cpu().numpy().astype(np.int64), c["page"]
    new, n = _lengths(c)
    dev = s["bt"].device

    def cells(b, p):  # physical block and slot of positions p (numpy)
        return torch.from_numpy(bt[b][p // page]).to(dev), torch.from_numpy(p % page).to(dev)

    if c["op"].endswith("append"):
        table = s["cos_sin"].double()
        cache = s["cache"].double()
        out = (s["q_pe_out"] if c["op"] == "mla_append" else s["q_out"]).double().clone()
        scales = s["scales"].double() if c.get("group") else None
        t = 0
        for b in range(c["B"]):
            m, p = int(new[b]), np.arange(n[b] - new[b], n[b])
            blk, slot = cells(b, p)
            cs = table[int(p[0]):int(p[0]) + m]
            if c["op"] == "mla_append":
                out[t:t + m] = _turn(s["q_pe"][t:t + m].double(), cs, c["inter"])
                row = torch.cat([s["kv_c"][t:t + m].double(), _turn(s["k_pe"][t:t + m, None].double(), cs, c["inter"])[:, 0]], 1)
                cache[blk, slot] = row if c["kv"] == "bf16" else _grid_e4m3(row / s["k_scale"])
                t += m
                continue
            out[t:t + m] = _turn(s["q"][t:t + m].double(), cs, c["inter"])
            x = torch.stack([_turn(s["k"][t:t + m].double(), cs, c["inter"]), s["v"][t:t + m].double()], 1)
            t += m
            if not c["group"]:
                cache[blk, :, slot] = x
                continue
            G = c["group"]
            for k in range(int(p[0]) // G, int(p[-1]) // G + 1):
                inside = torch.from_numpy(p // G == k).to(dev)
                y, had = x[inside], max(0, int(p[0]) - k * G)
                block, off = int(bt[b][k * G // page]), k * G % page
                was = scales[block, :, off // G].clone()
                now = torch.maximum(was if had else torch.zeros_like(was), y.abs().amax((0, 3)) / Q_MAX[c["kv"]])
                f = now[:, None, :, None]
                if had:
                    held = cache[block, :, off:off + had]
                    cache[block, :, off:off + had] = _grid(held * (was[:, None, :, None] / f), c["kv"])
                at = off + had
                cache[block, :, at:at + y.shape[0]] = _grid(y.transpose(0, 1) / f, c["kv"])
                scales[block, :, off // G] = now
        if not c.get("group"):
            return out, cache
        if c["kv"] == "int8_block":
            cache = cache * scales.repeat_interleave(c["group"], 2)[..., None]
        return out, cache, scales

    L, Hkv, grp = c["L"], c["Hkv"], c["Hq"] // c["Hkv"]
    out = torch.zeros(c["B"], L, c["Hq"], c["D"], dtype=torch.float64, device=dev)
    lse = torch.full((c["B"], L, c["Hq"]), -math.inf, dtype=torch.float64, device=dev)
    for b in range(c["B"]):
        W, S = (c["W"], c["S"]) if c["op"] == "window" else (int(n[b]) + 1, 0)
        for i in range(L):
            top = int(n[b]) - L + i
            if top < 0:
                continue
            p = np.arange(top + 1)
            p = p[(p < S) | (p > top - W)]
            blk, slot = cells(b, p)
            k, v = _cells(s["cache"], blk, 0, slot).double(), _cells(s["cache"], blk, 1, slot).double()
            if c["group"]:
                k = k * s["scales"][blk, 0, slot // c["group"]].double()[..., None]
                v = v * s["scales"][blk, 1, slot // c["group"]].double()[..., None]
            q = s["q"][b, i].double().view(Hkv, grp, -1)
            x = torch.einsum("hgd,nhd->hgn", q, k) * s["scale"]
            lse[b, i] = torch.logsumexp(x, -1).flatten()
            out[b, i] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v).flatten(0, 1)
    return out, lse
