"""Paged caches of every format with poisoned spare bytes, and attention over them in 64 bits, for the tests of
attention with shaped logits.

The reference is the definition: logits of every query and key, masks as truth values, softmax, product.  It shares
nothing with the kernels but the meaning of the arguments."""
import math

import torch

Q_MAX = {"fp8_e4m3_block": 448.0, "int8_block": 127.0}
NO_WINDOW = 1 << 30


class Paged:
    """A cache of the given lengths: tensors for the calls, and K and V of each request in 64 bits.  Spare blocks,
    tokens behind a request's last one and table entries behind its last page hold what must not be used."""

    def __init__(self, lens, Hkv, D, page, kv, seed=0, group=0, spare=3, value=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        pages = [-(-n // page) for n in lens]
        nb, width = sum(pages) + spare, max(pages + [1]) + 2
        perm = torch.randperm(nb, generator=g, device="cuda").tolist()
        self.kv, self.page, self.lens, self.k_scale, self.v_scale, self.scales = kv, page, list(lens), 1.0, 1.0, None
        x = torch.randn(nb, 2, page, Hkv, D, generator=g, device="cuda") * value
        if kv == "bf16":
            self.cache = x.to(torch.bfloat16)
            values = self.cache.double()
        elif kv == "fp8_e4m3":
            self.k_scale, self.v_scale = 0.04, 0.03
            x[:, 0] /= self.k_scale
            x[:, 1] /= self.v_scale
            self.cache = x.clamp(-448, 448).to(torch.float8_e4m3fn)
            values = self.cache.double()
            values[:, 0] *= self.k_scale
            values[:, 1] *= self.v_scale
        else:
            G = group or page
            x = x.view(nb, 2, page // G, G, Hkv, D)
            x *= torch.exp(torch.randn(nb, 2, page // G, 1, Hkv, 1, generator=g, device="cuda"))
            s = x.abs().amax((3, 5), keepdim=True) / Q_MAX[kv]
            y = x / s
            y = y.round().to(torch.int8) if kv == "int8_block" else y.to(torch.float8_e4m3fn)
            values = (y.double() * s.double()).view(nb, 2, page, Hkv, D)
            self.cache = y.view(nb, 2, page, Hkv, D)
            self.scales = s.view(nb, 2, page // G, Hkv).contiguous()
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        self.K, self.V, self.codes = [], [], []  # codes: magnitudes of V's codes and their scales
        used, at = torch.zeros(nb, page, dtype=torch.bool, device="cuda"), 0
        for b, n in enumerate(lens):
            ids = perm[at:at + pages[b]]
            at += pages[b]
            table[b, :pages[b]] = torch.tensor(ids, dtype=torch.int32)
            table[b, pages[b]:] = torch.tensor([-1, 2 ** 31 - 1] * width, dtype=torch.int32)[:width - pages[b]]
            rows = values[ids]  # [pages, 2, page, Hkv, D]
            self.K.append(rows[:, 0].reshape(-1, Hkv, D)[:n])
            self.V.append(rows[:, 1].reshape(-1, Hkv, D)[:n])
            if kv == "bf16":
                self.codes.append(None)
            else:
                s_v = torch.full((n, Hkv), self.v_scale, dtype=torch.float64, device="cuda")
                if self.scales is not None:
                    s_v = self.scales[ids, 1].double().repeat_interleave(group or page, 1).reshape(-1, Hkv)[:n]
                self.codes.append((self.cache[ids, 1].double().abs().reshape(-1, Hkv, D)[:n], s_v))
            flat = torch.zeros(pages[b] * page, dtype=torch.bool, device="cuda")
            flat[:n] = True
            used[ids] = flat.view(-1, page)
        raw = self.cache.view(torch.int16 if kv == "bf16" else torch.uint8)
        poison = 0x7fc0 if kv == "bf16" else 0x7f
        raw.masked_fill_(~used[:, None, :, None, None], poison)
        if self.scales is not None:  # scales of blocks without a token
            G = group or page
            idle = ~used.view(nb, page // G, G).any(-1)
            self.scales.masked_fill_(idle[:, None, :, None], float("nan"))
        self.table, self.seq_lens = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def attention(q, K, V, first, scale, cap=0.0, slopes=None, window=NO_WINDOW, sinks=0, prefix=0, half_codes=None):
    """half_codes: Paged.codes of a kernel that multiplies f16 numerators and codes.  Returns out and lse in 64 bits of queries q [w, Hq, D] at positions first, first + 1, .., and the bounds of their
    errors by which a kernel is judged: (out, lse, out_tol, lse_tol)."""
    w, Hq, D = q.shape
    n, Hkv = K.shape[:2]
    grp = Hq // Hkv
    p = first + torch.arange(w, device=q.device)[:, None]
    t = torch.arange(n, device=q.device)[None]
    seen = ((t <= p) | (t < prefix)) & ((t < sinks) | (t > p - window)) & (p >= 0)
    qd = q.double().view(w, Hkv, grp, D)
    x = torch.einsum("whgd,nhd->whgn", qd, K) * scale
    size = torch.einsum("whgd,nhd->whgn", qd.abs(), K.abs()) * abs(scale)
    if cap:
        x = cap * torch.tanh(x / cap)
    far = (p - t).abs().double()[:, None, None]
    bias = torch.zeros_like(x) if slopes is None else slopes.double().view(1, Hkv, grp, 1) * far
    x = (x - bias).masked_fill(~seen[:, None, None], -math.inf)
    some = seen.any(1)[:, None, None]
    lse = torch.logsumexp(x, -1)
    P = torch.where(some[..., None], torch.exp(x - lse[..., None]), 0.0).nan_to_num(0.0)
    out = torch.einsum("whgn,nhd->whgd", P, V)
    mass = torch.einsum("whgn,nhd->whgd", P, V.abs())
    # Logits: D products summed in fp32 (D 2^-24 of their absolute sum), a cap within 2^-21 of it or 2^-18 of the
    # logit, whichever is less (a polynomial's errors), a bias of two fp32
    # roundings, exp and log within 2^-21.  Numerators and, of scaled codes, values rounded to bf16 (2^-8 each of the
    # weighted absolute sum, which logits' errors change by as much again), the output to bf16 (2^-8).
    capped = torch.minimum((x + bias).abs() * 2.0 ** -18, torch.tensor(abs(cap) * 2.0 ** -21, device=q.device))
    dx = torch.where(seen[:, None, None], D * 2.0 ** -24 * size + bias.abs() * 2.0 ** -22 + capped, 0.0)
    dx = (P * dx).sum(-1) * 4 + (dx.amax(-1) if n else 0.0) * 0.25 + 2.0 ** -20
    out_tol = out.abs() * 2.0 ** -8 + mass * (2 * 2.0 ** -8 + 2 * dx[..., None]) + 1e-30
    if half_codes is not None:
        # f16 numerators P s_v are kept relative to one that is at most the largest, so those below 2^-14 of it are off
        # by 2^-25 of it at most, each times its code: absolute errors, which stand out where the large ones' codes are 0
        code, s_v = half_codes
        largest = (P * s_v.transpose(0, 1).view(1, Hkv, 1, n)).amax(-1, keepdim=True) if n else 0.0
        codes = torch.einsum("whgn,nhd->whgd", seen[:, None, None].double().expand_as(P), code)
        out_tol = out_tol + 2.0 ** -25 * largest * codes
    return out.reshape(w, Hq, D), lse.reshape(w, Hq), out_tol.reshape(w, Hq, D), dx.reshape(w, Hq)


def judge(out, lse, ref, what=""):
    want, want_lse, tol, lse_tol = ref
    bad = ~((out.double() - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outputs off, first at {bad.nonzero()[0].tolist()}: "
                           f"{out[bad][:4].tolist()} for {want[bad][:4].tolist()} within {tol[bad][:4].tolist()}")
    if lse is not None:
        none = want_lse == -math.inf
        assert torch.equal(lse == -math.inf, none), f"{what}: rows without a key"
        bad = ~((lse.double() - want_lse).abs() <= lse_tol) & ~none
        assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} lse off, first at {bad.nonzero()[0].tolist()}: "
                               f"{lse[bad][:4].tolist()} for {want_lse[bad][:4].tolist()} within {lse_tol[bad][:4].tolist()}")
