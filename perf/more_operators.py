"""The cases on which attention with shaped scores (decode and prompts) and the page operations are measured.

Four operators of a serving program over paged caches:

  score    GQA decode whose logits are capped by a tanh and biased by the distance of query and key, under a
           sliding window with sink tokens or none, 1 or more new positions per request;
  prefill  GQA attention of a ragged batch of prompt chunks over a paged cache that already holds their keys:
           causal or with a bidirectional prefix, with the same caps, biases, windows and sinks;
  fork     new rows of a block table from parents (beam search, several samples of a prompt, requests that end):
           full pages shared by count, a partly filled last page copied, in the caches of several layers;
  compact  live pages moved to the lowest ids, tables and counts renamed.

A case is a dict of plain values; lengths come from its own "lens_seed", values from the seed given to prepare().
"""
import math

import numpy as np
import torch

own = False

Q_MAX = {"fp8_e4m3_block": 448.0, "int8_block": 127.0}
NO_WINDOW = 1 << 30


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest decode: one short request, capped logits; latency
        dict(name="score one request", op="score", B=1, L=1, lens="300,300", W=0, S=0, cap=50.0, alibi=False, Hq=32,
             Hkv=8, D=128, page=16, kv="bf16", group=0, lens_seed=21),
        # the GQA benchmark's batch (256 requests, lognormal lengths) with capped logits
        dict(name="score batch bf16 cap", op="score", B=256, L=1, lens="lognormal 2048,16384", W=0, S=0, cap=50.0,
             alibi=False, Hq=32, Hkv=8, D=128, page=16, kv="bf16", group=0, lens_seed=22),
        # verification of 4 positions, distance bias, long window, 8-bit cache with a scale per page and head
        dict(name="score x4 e4m3 blocks distance", op="score", B=32, L=4, lens="500,20000", W=4096, S=0, cap=0.0,
             alibi=True, Hq=32, Hkv=8, D=128, page=64, kv="fp8_e4m3_block", group=64, lens_seed=23),
        # two short prompts with the heads of the tests; latency
        dict(name="prefill tiny", op="prefill", B=2, new="37,100", old="0,0", pad=0, pre="", W=0, S=0, cap=50.0,
             alibi=False, Hq=8, Hkv=2, D=128, page=16, kv="bf16", group=0, lens_seed=24),
        # a few prompts at once, from a fused projection padded to a captured size: capped logits, sliding window
        dict(name="prefill prompts window cap", op="prefill", B=6, new="500,2600", old="0,100", pad=13, pre="",
             W=1024, S=0, cap=50.0, alibi=False, Hq=32, Hkv=8, D=128, page=16, kv="bf16", group=0, lens_seed=25),
        # one long document, causal
        dict(name="prefill long", op="prefill", B=1, new="15999,15999", old="0,0", pad=0, pre="", W=0, S=0, cap=0.0,
             alibi=False, Hq=32, Hkv=8, D=128, page=64, kv="bf16", group=0, lens_seed=26),
        # chunks of 64 tokens behind long contexts in an e4m3 cache, distance bias: few rows, long axis
        dict(name="prefill chunks e4m3 distance", op="prefill", B=3, new="64,64", old="20000,40000", pad=0, pre="",
             W=0, S=0, cap=0.0, alibi=True, Hq=32, Hkv=8, D=128, page=64, kv="fp8_e4m3", group=0, lens_seed=27),
        # prompts with bidirectional prefixes beside single tokens of running requests, int8 blocks, small heads
        dict(name="prefill prefix int8 blocks", op="prefill", B=24, new="1,700", old="0,900", pad=5, pre="0,500", W=0,
             S=0, cap=0.0, alibi=False, Hq=64, Hkv=8, D=64, page=32, kv="int8_block", group=32, lens_seed=28),
        # one step of beam search: 8 requests of 4 beams, one layer's cache
        dict(name="fork beams", op="fork", groups=8, beams=4, each=4, lens="37,2000", page=16, layers=1, Hkv=8, D=128,
             kv="bf16", spare=40, lens_seed=29),
        # 8 samples of each of 64 prompts, several layers of an e4m3 cache with block scales
        dict(name="fork samples", op="fork", groups=64, beams=1, each=8, lens="100,3000", page=64, layers=6, Hkv=8,
             D=128, kv="fp8_e4m3_block", spare=500, lens_seed=30),
        # a small pool after some requests have ended
        dict(name="compact small", op="compact", rows=8, lens="1,200", live=0.5, page=16, layers=1, Hkv=2, D=128,
             kv="bf16", lens_seed=31),
        # a pool of several layers, half of its pages free
        dict(name="compact pool", op="compact", rows=256, lens="1,600", live=0.5, page=16, layers=2, Hkv=8, D=128,
             kv="bf16", lens_seed=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "prefill", "prefill", "fork", "compact"])
    c = dict(op=op, lens_seed=rng.randrange(1 << 30))
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "fork":
        c.update(groups=_log_int(rng, 1, 64), beams=rng.choice([1, 1, 3, 4]), each=rng.choice([1, 4, 5, 8]),
                 lens="%d,%d" % (rng.choice([0, 1, 100]), _log_int(rng, 100, 2500)), page=page,
                 layers=rng.choice([1, 2, 5]), Hkv=rng.choice([1, 2, 4]), D=D,
                 kv=rng.choice(["bf16", "fp8_e4m3_block"]), spare=rng.choice([520, 700]))
        return c
    if op == "compact":
        c.update(rows=_log_int(rng, 1, 200), lens="%d,%d" % (rng.choice([0, 1]), _log_int(rng, 20, 600)),
                 live=rng.choice([0.1, 0.5, 0.9]), page=page, layers=rng.choice([1, 2]), Hkv=rng.choice([1, 2, 4]),
                 D=D, kv=rng.choice(["bf16", "fp8_e4m3_block"]))
        return c
    shape = rng.choice(["cap", "distance", "both", "none"])
    kv = rng.choice(["bf16", "fp8_e4m3", "fp8_e4m3_block", "int8_block"])
    c.update(cap=rng.choice([15.0, 30.0, 50.0]) if shape in ("cap", "both") else 0.0,
             alibi=shape in ("distance", "both"), Hkv=Hkv, D=D, page=page, kv=kv,
             group=rng.choice([16, page]) if kv.endswith("block") else 0)
    windowed = rng.random() < 0.5
    c.update(W=_log_int(rng, 1, 4096) if windowed else 0, S=rng.choice([0, 1, 4, 17, 64]) if windowed else 0)
    if op == "score":
        B = _log_int(rng, 1, 128)
        hi = min(_log_int(rng, 16, 30000), max(16, 250000 // B))
        c.update(B=B, L=rng.choice([1, 1, 2, 5]), lens="%d,%d" % (rng.choice([1, hi // 2 + 1, hi]), hi),
                 Hq=Hkv * rng.choice([1, 2, 4, 7, 8, 16]))
        return c
    kind = rng.choice(["prompts", "prompts", "chunks", "mixed"])
    if kind == "prompts":
        hi = _log_int(rng, 3, 5000)
        c.update(B=rng.randint(1, max(1, min(12, 12000 // hi))), new="%d,%d" % (hi // 3 + 1, hi),
                 old="0,%d" % rng.choice([0, 90]))
    elif kind == "chunks":
        c.update(B=rng.randint(1, 4), new="1,%d" % _log_int(rng, 2, 400), old="100,%d" % _log_int(rng, 200, 20000))
    else:
        c.update(B=_log_int(rng, 2, 40), new="1,%d" % _log_int(rng, 2, 300), old="0,%d" % _log_int(rng, 1, 1500))
    c.update(pad=rng.choice([0, 0, 1, 9]), pre=rng.choice(["", "", "0,%d" % _log_int(rng, 1, 1000)]),
             Hq=Hkv * rng.choice([1, 2, 3, 4, 7, 8, 16]))
    return c


def _range(text, rng, B):
    if text.startswith("lognormal"):
        median, top = (int(x) for x in text.split()[1].split(","))
        return np.clip(np.ceil(np.exp(rng.normal(math.log(median), 1.0, B))), 1, top).astype(np.int64)
    lo, hi = (int(x) for x in text.split(","))
    return rng.integers(lo, hi + 1, B)


def _lengths(c):
    """(new tokens of each request, lengths with them, prefix lengths) as numpy."""
    rng = np.random.default_rng(c["lens_seed"])
    if c["op"] == "score":
        n = _range(c["lens"], rng, c["B"])
        return np.full(c["B"], c["L"]), n, np.zeros(c["B"], np.int64)
    new = np.array([37, 100]) if c["new"] == "37,100" else _range(c["new"], rng, c["B"])
    n = new + _range(c["old"], rng, c["B"])
    return new, n, _range(c["pre"], rng, c["B"]) if c["pre"] else np.zeros(c["B"], np.int64)


def _elt(kv):
    return 2 if kv == "bf16" else 1


def _page_bytes(c):
    return c["layers"] * (2 * c["page"] * c["Hkv"] * c["D"] * _elt(c["kv"]) + (0 if c["kv"] == "bf16" else 8 * c["Hkv"]))


def work(c):
    if c["op"] == "fork":
        r = _rows(c)
        rows = r["table"].size + len(r["parents"]) * r["table"].shape[1]
        copies = int(_fork_needs(r, c["page"]).sum())
        return {"bytes": 4 * (rows + 2 * r["nb"]) + 2 * copies * _page_bytes(c), "flops": rows + r["nb"]}
    if c["op"] == "compact":
        r = _rows(c)
        live = int((r["refs"] > 0).sum())
        moves = int((r["refs"][live:] > 0).sum())
        return {"bytes": 4 * (2 * r["table"].size + 3 * r["nb"]) + 2 * moves * _page_bytes(c), "flops": r["table"].size + r["nb"]}
    new, n, pre = _lengths(c)
    W, S = (c["W"], c["S"]) if c["W"] else (NO_WINDOW, 0)
    seen, pairs = 0, 0
    for m, k, x in zip(n.tolist(), new.tolist(), pre.tolist()):
        p = np.arange(max(0, m - k), m)
        if not p.size:
            continue
        hi = np.maximum(p + 1, min(x, m))
        lo = np.maximum(0, p - W + 1)
        pairs += int((hi - lo + np.minimum(S, lo)).sum())
        seen += int(hi.max() - lo.min() + min(S, lo.min()))
    b = seen * 2 * c["Hkv"] * c["D"] * _elt(c["kv"]) + 2 * int(new.sum()) * c["Hq"] * c["D"] * 2 + int(new.sum()) * c["Hq"] * 4
    if c["group"]:
        b += seen // c["group"] * 2 * c["Hkv"] * 4
    return {"bytes": b, "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---------------------------------------------------------------------------- inputs

def _rows(c):
    """Block table, lengths, counts and parents of a page operation, as numpy: a program's state between steps."""
    rng = np.random.default_rng(c["lens_seed"])
    page = c["page"]
    if c["op"] == "compact":
        lens = _range(c["lens"], rng, c["rows"])
        pages = -(-lens // page)
        used = int(pages.sum())
        nb = max(2, int(used / c["live"]) + 1)
        ids = rng.permutation(nb)[:used]
        table = np.full((c["rows"], max(1, int(pages.max()) + 1)), -1, np.int32)
        at = 0
        for b, k in enumerate(pages):
            table[b, :k] = ids[at:at + k]
            at += k
        refs = np.zeros(nb, np.int32)
        refs[ids] = 1
        for b in range(1, c["rows"], 5):  # some requests share the first pages of the one before
            k = int(min(pages[b], pages[b - 1]) // 2)
            refs[table[b, :k]] -= 1
            table[b, :k] = table[b - 1, :k]
            refs[table[b, :k]] += 1
        return dict(nb=nb, table=table, lens=lens, refs=refs, parents=None)
    G, beams, each = c["groups"], c["beams"], c["each"]
    first = _range(c["lens"], rng, G)
    lens = np.repeat(first, beams)  # beams of a request are equally long
    pages = -(-lens // page)
    shared = first // 2 // page  # full pages that a request's beams have in common
    used = int((pages - np.repeat(shared, beams)).sum() + shared.sum())
    nb = used + c["spare"]
    ids = rng.permutation(nb)
    table = np.full((G * beams, max(1, int(pages.max()) + 1)), -1, np.int32)
    refs = np.zeros(nb, np.int32)
    at = 0
    for g in range(G):
        common, at = ids[at:at + shared[g]], at + shared[g]
        for r in range(g * beams, (g + 1) * beams):
            tail, at = ids[at:at + pages[r] - shared[g]], at + pages[r] - shared[g]
            table[r, :pages[r]] = np.concatenate([common, tail])
            refs[table[r, :pages[r]]] += 1
    parents = np.repeat(np.arange(G) * beams, each) + rng.integers(0, beams, G * each)
    if beams > 1:
        parents[rng.random(G * each) < 0.1] = -1  # beams that end
    return dict(nb=nb, table=table, lens=lens, refs=refs, parents=parents.astype(np.int32))


def _fork_needs(r, page):
    """Which new rows get a page of their own: all children but a parent's first, where its last page is not full."""
    p, needs, met = r["parents"], np.zeros(len(r["parents"]), bool), set()
    for i, q in enumerate(p.tolist()):
        if q >= 0:
            needs[i] = q in met and r["lens"][q] % page != 0
            met.add(q)
    return needs


def _quantised(x, kv):
    """Codes and scales of values [blocks, 2, groups, tokens, heads, D]: one scale for each group and head."""
    s = x.abs().amax(dim=(3, 5), keepdim=True).float() / Q_MAX[kv]
    y = x.float().div_(s)
    if kv == "int8_block":
        return y.round_().to(torch.int8), s
    return y.clamp_(-448, 448).to(torch.float8_e4m3fn), s


def _cache(c, nb, randn):
    """A cache of the case's format and its block scales, or None."""
    page, kv, Hkv, D = c["page"], c["kv"], c["Hkv"], c["D"]
    if kv == "bf16":
        return randn(nb, 2, page, Hkv, D), None
    if kv == "fp8_e4m3":
        return randn(nb, 2, page, Hkv, D).div_(0.05).clamp_(-448, 448).to(torch.float8_e4m3fn), None
    G = c.get("group") or page
    x = randn(nb, 2, page // G, G, Hkv, D)
    x *= torch.exp(0.5 * randn(nb, 2, page // G, 1, Hkv, 1))  # blocks and heads of unlike magnitude
    codes, scales = _quantised(x, kv)
    return codes.view(nb, 2, page, Hkv, D), scales.view(nb, 2, page // G, Hkv).contiguous()


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    if c["op"] in ("fork", "compact"):
        r = _rows(c)
        perm = torch.randperm(r["nb"], generator=g, device=dev)
        table = torch.from_numpy(r["table"]).to(dev)
        table = torch.where(table >= 0, perm[table.long().clamp(min=0)].int(), -1).contiguous()
        refs = torch.empty(r["nb"], dtype=torch.int32, device=dev)
        refs[perm] = torch.from_numpy(r["refs"]).to(dev)
        caches = []
        for _ in range(c["layers"]):
            caches += [t for t in _cache(c, r["nb"], randn) if t is not None]
        s = dict(case=c, table=table, lens=torch.from_numpy(r["lens"].astype(np.int32)).to(dev), refs=refs, caches=caches)
        if c["op"] == "fork":
            s["parents"] = torch.from_numpy(r["parents"]).to(dev)
        return s

    new, n, pre = _lengths(c)
    page, B, Hq, Hkv, D = c["page"], c["B"], c["Hq"], c["Hkv"], c["D"]
    pages = -(-n // page)
    nb = int(pages.sum()) + 3
    perm = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    first = np.concatenate([[0], np.cumsum(pages)])
    cols = torch.arange(max(1, int(pages.max())), device=dev)
    at = torch.from_numpy(first[:-1]).to(dev)[:, None] + cols
    has = cols < torch.from_numpy(pages).to(dev)[:, None]
    bt = torch.where(has, perm[at.clamp(max=nb - 1)], -1).to(torch.int32).contiguous()
    s = dict(case=c, bt=bt, lens=torch.from_numpy(n.astype(np.int32)).to(dev), nb=nb, max_len=int(n.max()),
             scale=1.0 / math.sqrt(D), k_scale=0.05 if c["kv"] == "fp8_e4m3" else 1.0)
    s["cache"], s["scales"] = _cache(c, nb, randn)
    # slopes of a geometric series over the heads
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=dev) / Hq).float() if c["alibi"] else None
    wide = 3.0 if c["cap"] else 1.0  # logits that a cap is there for
    if c["op"] == "score":
        s["q"] = randn(B, c["L"], Hq, D) * wide
        return s
    T = int(new.sum()) + c["pad"]
    s["query_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(dev)
    s["prefix"] = torch.from_numpy(pre.astype(np.int32)).to(dev) if c["pre"] else None
    if c["pad"]:  # the queries of a fused projection
        s["q"] = (randn(T, Hq + 2 * Hkv, D) * wide)[:, :Hq]
    else:
        s["q"] = randn(T, Hq, D) * wide
    s["out"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.zeros(T, Hq, dtype=torch.float32, device=dev)
    return s


# ---------------------------------------------------------------------------- plain forms

def _bytes(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _cells(cache, *at):
    """The cells of a cache at advanced indices, whatever its type."""
    return _bytes(cache)[at].view(cache.dtype)


def _window(c):
    return (c["W"], c["S"]) if c["W"] else (NO_WINDOW, 0)


def _shaped(x, c, slopes, far):
    """Logits x capped and biased; slopes and far (the distance of query and key) broadcast against x."""
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if slopes is not None:
        x = x - slopes * far
    return x


def _softmax_sum(x, v):
    """sum softmax(x) v and the logsumexp of x over its last dimension; 0 and -inf where x is -inf throughout."""
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, (p @ v) / total, 0.0), (m + torch.log(total))[..., 0]


def _plain_score(s):
    c = s["case"]
    B, L, Hq, Hkv, D, page, G = c["B"], c["L"], c["Hq"], c["Hkv"], c["D"], c["page"], c["group"]
    dev = s["bt"].device
    n = s["lens"].long()[:, None]
    W, S = _window(c)
    wide = min(W + L - 1, s["max_len"])
    lo = (n - wide).clamp(min=0)
    pos = torch.cat([torch.arange(S, device=dev).expand(B, S), lo + torch.arange(wide, device=dev)], 1)
    first = torch.cat([torch.ones(S, dtype=torch.bool, device=dev), torch.zeros(wide, dtype=torch.bool, device=dev)])
    ok = (pos < n) & (first | (pos >= S))
    at = torch.where(ok, pos, 0)
    blk, slot = s["bt"].long().gather(1, at // page), at % page
    qp = n - L + torch.arange(L, device=dev)
    seen = ok[:, None] & (pos[:, None] <= qp[..., None]) & ((pos[:, None] < S) | (pos[:, None] > qp[..., None] - W))

    def plane(i):
        x = _cells(s["cache"], blk, i, slot).float()  # [B, keys, Hkv, D]
        if G:
            x *= s["scales"][blk, i, slot // G][..., None]
        return x.mul_(s["k_scale"]).masked_fill_(~ok[..., None, None], 0.0).transpose(1, 2)

    q = s["q"].float().view(B, L, Hkv, Hq // Hkv, D).transpose(1, 2).reshape(B, Hkv, -1, D)
    x = (q @ plane(0).transpose(-1, -2)).view(B, Hkv, L, Hq // Hkv, -1) * s["scale"]
    slopes = None if s["slopes"] is None else s["slopes"].view(Hkv, 1, Hq // Hkv, 1)
    x = _shaped(x, c, slopes, (qp[..., None] - pos[:, None]).abs().float()[:, None, :, None])
    x = x.masked_fill(~seen[:, None, :, None], -math.inf).flatten(2, 3)
    out, lse = _softmax_sum(x, plane(1))
    return (out.view(B, Hkv, L, Hq // Hkv, D).transpose(1, 2).reshape(B, L, Hq, D).to(torch.bfloat16),
            lse.view(B, Hkv, L, -1).transpose(1, 2).reshape(B, L, Hq))


def _plain_prefill(s):
    c = s["case"]
    Hq, Hkv, D, page, G = c["Hq"], c["Hkv"], c["D"], c["page"], c["group"]
    grp = Hq // Hkv
    dev = s["bt"].device
    W, S = _window(c)
    new, n, pre = _lengths(c)
    slopes = None if s["slopes"] is None else s["slopes"].view(Hkv, 1, grp, 1)
    start = 0
    for b in range(c["B"]):
        m, k = int(n[b]), int(new[b])
        t = torch.arange(m, device=dev)
        blk, slot = s["bt"][b].long()[t // page], t % page

        def plane(i):
            x = _cells(s["cache"], blk, i, slot).float()
            if G:
                x *= s["scales"][blk, i, slot // G][..., None]
            return x.mul_(s["k_scale"]).transpose(0, 1)  # [Hkv, m, D]

        keys, values = plane(0), plane(1)
        step = max(1, min(k, (1 << 28) // (Hq * m)))
        for at in range(0, k, step):
            w = min(step, k - at)
            p = m - k + at + torch.arange(w, device=dev)[:, None]
            hi = max(m - k + at + w, min(int(pre[b]), m))  # no row of this piece sees a key from here on
            seen = ((t[:hi] <= p) | (t[:hi] < int(pre[b]))) & ((t[:hi] < S) | (t[:hi] > p - W))
            q = s["q"][start + at:start + at + w].float().view(w, Hkv, grp, D).transpose(0, 1).reshape(Hkv, w * grp, D)
            x = (q @ keys[:, :hi].transpose(-1, -2)).view(Hkv, w, grp, hi) * s["scale"]
            x = _shaped(x, c, slopes, (p - t[:hi]).abs().float()[None, :, None])
            x = x.masked_fill(~seen[None, :, None], -math.inf).flatten(1, 2)
            out, lse = _softmax_sum(x, values[:, :hi])
            s["out"][start + at:start + at + w] = out.view(Hkv, w, grp, D).transpose(0, 1).reshape(w, Hq, D).to(torch.bfloat16)
            s["lse"][start + at:start + at + w] = lse.view(Hkv, w, grp).transpose(0, 1).reshape(w, Hq)
        start += k
    return s["out"], s["lse"]


def _plain_fork(s):
    page, table, lens, parents = s["case"]["page"], s["table"].long(), s["lens"].long(), s["parents"].long()
    dev = table.device
    R, N, width = table.shape[0], parents.shape[0], table.shape[1]
    cols = torch.arange(width, device=dev)
    alive, p = parents >= 0, parents.clamp(min=0)
    n2 = torch.where(alive, lens[p], 0)
    pages2 = (n2 + page - 1) // page
    table2 = torch.where(cols < pages2[:, None], table[p], -1)
    count = torch.zeros(R, dtype=torch.long, device=dev).scatter_add_(0, p, alive.long())
    pages = ((lens + page - 1) // page)[:, None]
    partial = (cols == pages - 1) & (lens % page != 0)[:, None]
    change = torch.where(partial, (count > 0).long()[:, None], count[:, None]) - 1
    held = cols < pages
    refs2 = s["refs"].long().scatter_add(0, torch.where(held, table, 0).flatten(), torch.where(held, change, 0).flatten())
    row = torch.arange(N, device=dev)
    first = torch.full((R,), N, device=dev).scatter_reduce_(0, p, torch.where(alive, row, N), "amin")
    needs = (alive & (n2 % page != 0) & (row != first[p])).nonzero()[:, 0]
    fresh = (refs2 == 0).nonzero()[:needs.shape[0], 0]  # the lowest free pages, in the order of the rows
    last = table2[needs, pages2[needs] - 1]
    for x in s["caches"]:
        _bytes(x)[fresh] = _bytes(x)[last]
    table2[needs, pages2[needs] - 1] = fresh
    refs2[fresh] = 1
    return table2.int(), n2.int(), refs2.int(), *s["caches"]


def _plain_compact(s):
    page, refs, table = s["case"]["page"], s["refs"], s["table"]
    ids = torch.arange(refs.shape[0], device=refs.device, dtype=torch.int32)
    live = refs > 0
    count = live.sum(dtype=torch.int32)
    src, dst = (live & (ids >= count)).nonzero()[:, 0], (~live & (ids < count)).nonzero()[:, 0]
    moved = torch.where(live, ids, -1)
    moved[src] = dst.int()
    refs2 = refs.clone()
    refs2[dst] = refs[src]
    refs2[src] = 0
    held = torch.arange(table.shape[1], device=refs.device) < ((s["lens"] + page - 1) // page)[:, None]
    table2 = torch.where(held, moved[torch.where(held, table, 0).long()], table)
    for x in s["caches"]:
        _bytes(x)[dst] = _bytes(x)[src]
    return table2, refs2, moved, count.view(1), *s["caches"]


# ---------------------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"score": _plain_score, "prefill": _plain_prefill, "fork": _plain_fork, "compact": _plain_compact}[c["op"]](s)
    import mqa_decode_attention_paged_gb300 as mqa
    if c["op"] == "fork":
        return *mqa.pages_fork(s["table"], s["lens"], s["parents"], s["refs"], s["caches"], c["page"]), *s["caches"]
    if c["op"] == "compact":
        return *mqa.pages_compact(s["table"], s["lens"], s["refs"], s["caches"], c["page"]), *s["caches"]
    W, S = _window(c)
    shape = dict(softcap=c["cap"], slopes=s["slopes"], window=W, sinks=S, kv_scales=s["scales"], k_scale=s["k_scale"],
                 v_scale=s["k_scale"])
    if "workspace" not in s:  # a serving program keeps its outputs and workspace from step to step
        if c["op"] == "score":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:3], dtype=torch.float32, device=s["q"].device)
            s["splits"] = mqa.gqa_window_num_kv_splits(c["B"], c["L"], c["Hq"], c["Hkv"])
            need = mqa.gqa_window_decode_workspace_bytes(c["B"], c["L"], c["Hq"], c["Hkv"], c["D"], s["splits"])
        else:
            need = mqa.gqa_prefill_workspace_bytes(c["Hq"], c["Hkv"], c["D"])
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=s["q"].device)
    if c["op"] == "score":
        return mqa.gqa_score_decode(s["q"], s["cache"], s["bt"], s["lens"], s["scale"], out=s["out"], lse=s["lse"],
                                    num_kv_splits=s["splits"], workspace=s["workspace"], **shape)
    return mqa.gqa_prefill(s["q"], s["cache"], s["bt"], s["lens"], s["query_start"], s["scale"], prefix_lens=s["prefix"],
                           out=s["out"], lse=s["lse"], workspace=s["workspace"], **shape)


# ---------------------------------------------------------------------------- the definition in 64 bits

def _exact_attention(c, s):
    new, n, pre = _lengths(c)
    page, Hkv, grp = c["page"], c["Hkv"], c["Hq"] // c["Hkv"]
    dev = s["bt"].device
    W, S = _window(c)
    bt = s["bt"].cpu().numpy().astype(np.int64)
    flat = s["q"].reshape(-1, c["Hq"], c["D"]) if c["op"] == "score" else s["q"]
    out = torch.zeros(flat.shape[0], c["Hq"], c["D"], dtype=torch.float64, device=dev)
    lse = torch.zeros(flat.shape[0], c["Hq"], dtype=torch.float64, device=dev)
    row = 0
    for b in range(c["B"]):
        m, k = int(n[b]), int(new[b])
        p = np.arange(m)
        blk, slot = torch.from_numpy(bt[b][p // page]).to(dev), torch.from_numpy(p % page).to(dev)
        kv = [_cells(s["cache"], blk, i, slot).double() for i in (0, 1)]
        if c["group"]:
            kv = [x * s["scales"][blk, i, slot // c["group"]].double()[..., None] for i, x in enumerate(kv)]
        kv = [x * s["k_scale"] for x in kv]
        step = max(1, min(k, 40_000_000 // (c["Hq"] * m)))
        for at in range(0, k, step):
            w = min(step, k - at)
            top = torch.arange(m - k + at, m - k + at + w, device=dev)
            end = min(m, max(m - k + at + w, int(pre[b])))
            t = torch.arange(end, device=dev)
            near = (t[None] <= top[:, None]) | (t[None] < int(pre[b]))
            near &= (t[None] < S) | (t[None] > top[:, None] - W)
            q = flat[row + at:row + at + w].double().view(w, Hkv, grp, -1)
            x = torch.einsum("whgd,nhd->whgn", q, kv[0][:end]) * s["scale"]
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if s["slopes"] is not None:
                x -= s["slopes"].double().view(1, Hkv, grp, 1) * (top[:, None] - t[None]).abs()[:, None, None]
            x.masked_fill_(~near[:, None, None], -math.inf)
            some = near.any(1)
            lse[row + at:row + at + w] = torch.logsumexp(x, -1).flatten(1)
            y = torch.einsum("whgn,nhd->whgd", torch.softmax(x, -1), kv[1][:end]).flatten(1, 2)
            out[row + at:row + at + w] = torch.where(some[:, None, None], y, 0.0)
        row += k
    if c["op"] == "score":
        return out.view(s["q"].shape), lse.view(s["q"].shape[:3])
    return out, lse


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("score", "prefill"):
        return _exact_attention(c, s)
    page, dev = c["page"], s["table"].device
    table, lens, refs = s["table"].cpu().numpy(), s["lens"].cpu().numpy(), s["refs"].cpu().numpy().copy()
    held = [table[b, :-(-int(n) // page)] for b, n in enumerate(lens)]
    src, dst = [], []
    if c["op"] == "fork":
        parents = s["parents"].cpu().numpy()
        table2 = np.full((len(parents), table.shape[1]), -1, np.int32)
        lens2 = np.zeros(len(parents), np.int32)
        for h in held:  # every old row lets its pages go, every new one takes them up
            refs[h] -= 1
        own_page = []
        for r, q in enumerate(parents):
            if q < 0:
                continue
            lens2[r] = lens[q]
            table2[r, :len(held[q])] = held[q]
            kept = held[q]
            if lens[q] % page and (parents[:r] == q).any():
                own_page.append(r)
                kept = kept[:-1]
            refs[kept] += 1
        free = np.flatnonzero(refs == 0)
        for r, f in zip(own_page, free):
            last = len(held[parents[r]]) - 1
            src.append(int(table2[r, last]))
            dst.append(int(f))
            table2[r, last] = f
            refs[f] = 1
        first = (table2, lens2, refs)
    else:
        count = int((refs > 0).sum())
        src = [i for i in range(count, len(refs)) if refs[i] > 0]
        dst = [i for i in range(count) if refs[i] <= 0]
        moved = np.where(refs > 0, np.arange(len(refs)), -1).astype(np.int32)
        moved[src] = dst
        refs2 = refs.copy()
        refs2[dst], refs2[src] = refs[src], 0
        table2 = table.copy()
        for b, h in enumerate(held):
            table2[b, :len(h)] = moved[h]
        first = (table2, refs2, moved, np.array([count], np.int32))
    caches = []
    for x in s["caches"]:
        y = x.double()
        y[torch.tensor(dst, device=dev, dtype=torch.long)] = x.double()[torch.tensor(src, device=dev, dtype=torch.long)]
        caches.append(y)
    return *(torch.from_numpy(np.ascontiguousarray(x)).to(dev) for x in first), *caches
