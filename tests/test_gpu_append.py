"""GPU parity of the cache-append entry points against a 64-bit reference.

Bounds: a rotated value is an fp32 sum of two products, off by at most 2^-22
(|x| + |y|) of its pair; a bf16 store adds 2^-8 relative; a code must be one
that a value within that distance (and 2^-21 relative, for the division)
rounds to; a scale is off by 2^-21 relative and the distance of its largest
value.  Everything that is not written must keep its bytes."""
import numpy as np
import pytest
import torch

import cache_reference as ref
import mqa_decode_attention_paged_gb300 as mqa

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def table(positions, rot):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


class Batch:
    def __init__(self, new, old, page, pad=0, seed=0, rot=64, extra=2):
        self.g = torch.Generator().manual_seed(seed)
        self.new, self.lens, self.page, self.pad = new, [a + b for a, b in zip(new, old)], page, pad
        pages = [-(-n // page) for n in self.lens]
        self.nb = sum(pages) + extra
        perm = torch.randperm(self.nb, generator=self.g)
        self.bt = torch.full((len(new), max(1, max(pages)) + 1), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(pages):
            self.bt[b, :m] = perm[at:at + m].to(torch.int32)
            at += m
        self.T = sum(new) + pad
        self.qs = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.cs = table(max(self.lens) + 1, rot)

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g)

    def tokens(self):
        """(token row, request, position) of each new token."""
        for b, m in enumerate(self.new):
            for i in range(m):
                yield int(self.qs[b]) + i, b, self.lens[b] - m + i

    def where(self, b, p):
        return int(self.bt[b, p // self.page]), p % self.page

    def dev(self):
        return self.cs.cuda(), self.bt.cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda"), self.qs.cuda()


def fused(batch, Hq, Hkv, D, dense):
    T = batch.T
    if dense:
        return [batch.randn(T, h, D).to(BF) for h in (Hq, Hkv, Hkv)]
    x = batch.randn(T, Hq + 2 * Hkv + 1, D).to(BF)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:Hq + 2 * Hkv]


def check_rows(got, x, row, inter, what):
    y, mag = ref.rotate(x.double(), row.double(), inter)
    err = (got.double() - y).abs()
    assert (err <= y.abs() * 2 ** -8 + mag * 2 ** -22 * 1.01).all(), what
    return y, mag


def check_codes(code, x, mag, s, kv, what):
    """codes of values x (off by mag 2^-22) at scale s."""
    if s == 0:
        assert (code == 0).all(), what
        return
    y = x / s
    lo, hi = ref.code_range(y, y.abs() * 2 ** -21 + mag * (2 ** -22 / s), kv)
    assert ((lo <= code) & (code <= hi)).all(), what


def check_scale(s, x, mag, kv, what, least=0.0):
    want = max(float(x.abs().max()) / ref.Q_MAX[kv], least)
    assert abs(s - want) <= want * 2 ** -21 + float(mag.max()) * 2 ** -22 / ref.Q_MAX[kv], what


def run(batch, q, k, v, cache, *, inter=False, scales=None, kv=None, status=None, ks=1.0, vs=1.0, dense_views=None):
    cs, bt, sl, qs = batch.dev()
    base = None
    if not q.is_contiguous():  # the slices of one projection stay slices on the device
        base = q._base.cuda()
        q = base[:, :q.shape[1]]
        k, v = (base[:, q.shape[1] + i * k.shape[1]:q.shape[1] + (i + 1) * k.shape[1]] for i in (0, 1))
    dq, dk, dv, dc = (t.cuda() if not t.is_cuda else t for t in (q, k, v, cache))
    out = torch.full((batch.T,) + tuple(q.shape[1:]), 7.0, dtype=BF, device="cuda")
    dsc = None if scales is None else scales.cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mqa.gqa_rope_append(dk, dv, cs, dc, bt, sl, qs, q=dq, q_out=out, kv_scales=dsc, k_scale=ks, v_scale=vs,
                              interleaved=inter, kv_dtype=kv, device_status=st)
    torch.cuda.synchronize()
    assert got is out
    return out.cpu(), dc.cpu(), None if dsc is None else dsc.cpu(), int(st.item())


def untouched(before, after, written):
    """Cells outside `written` [blocks, page] keep their bytes."""
    a, b = before.view(torch.uint8), after.view(torch.uint8)
    keep = ~written[:, None, :]
    return torch.equal(a[keep.expand(a.shape[:3])], b[keep.expand(b.shape[:3])])


SHAPES = [(32, 8, 128, 128), (8, 2, 128, 64), (12, 4, 64, 64), (3, 3, 64, 32), (1, 1, 128, 16), (35, 5, 128, 112),
          (48, 8, 64, 48)]
RAGGED = ([1, 0, 5, 16, 33, 1, 2], [0, 9, 11, 0, 40, 15, 100])


@pytest.mark.parametrize("Hq,Hkv,D,rot", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
def test_bf16(Hq, Hkv, D, rot, inter):
    for dense, pad in ((True, 0), (False, 3)):
        bt = Batch(*RAGGED, page=16, pad=pad, seed=1, rot=rot)
        q, k, v = fused(bt, Hq, Hkv, D, dense)
        cache = bt.randn(bt.nb, 2, 16, Hkv, D).to(BF)
        out, got, _, status = run(bt, q, k, v, cache, inter=inter)
        assert status == 0
        written = torch.zeros(bt.nb, 16, dtype=torch.bool)
        for t, b, p in bt.tokens():
            blk, slot = bt.where(b, p)
            written[blk, slot] = True
            check_rows(out[t], q[t], bt.cs[p], inter, f"q token {t}")
            check_rows(got[blk, 0, slot], k[t], bt.cs[p], inter, f"k token {t}")
            assert torch.equal(got[blk, 1, slot], v[t])
        assert untouched(cache, got, written)
        assert (out[sum(bt.new):] == 7.0).all()  # padding


def decode_row(row, kv, D):
    """(codes float64, scale) of a per-token-head row of bytes."""
    n = D // 2 if kv == "int4_pth" else D
    s = float(row[n:].contiguous().view(torch.float32)[0])
    c = row[:n]
    if kv == "fp8_e4m3_pth":
        return c.contiguous().view(torch.float8_e4m3fn).double(), s
    if kv == "int8_pth":
        return c.contiguous().view(torch.int8).double(), s
    x = torch.stack([c & 15, c >> 4], 1).flatten().double()
    return torch.where(x > 7, x - 16, x), s


@pytest.mark.parametrize("kv", ["fp8_e4m3_pth", "int8_pth", "int4_pth"])
@pytest.mark.parametrize("Hq,Hkv,D,rot", SHAPES[1:])
def test_per_token_head(kv, Hq, Hkv, D, rot):
    bt = Batch(*RAGGED, page=16, pad=2, seed=2, rot=rot)
    q, k, v = fused(bt, Hq, Hkv, D, False)
    k[3] = 0.0  # a row of zeros
    v[4] = 1e-40
    row = (D // 2 if kv == "int4_pth" else D) + 4
    cache = torch.randint(0, 256, (bt.nb, 2, 16, Hkv, row), generator=bt.g, dtype=torch.uint8)
    out, got, _, status = run(bt, q, k, v, cache, kv=kv)
    assert status == 0
    written = torch.zeros(bt.nb, 16, dtype=torch.bool)
    for t, b, p in bt.tokens():
        blk, slot = bt.where(b, p)
        written[blk, slot] = True
        check_rows(out[t], q[t], bt.cs[p], False, f"q token {t}")
        kr, mag = ref.rotate(k[t].double(), bt.cs[p].double(), False)
        for plane, x, m in ((0, kr, mag), (1, v[t].double(), torch.zeros_like(mag))):
            for h in range(Hkv):
                code, s = decode_row(got[blk, plane, slot, h], kv, D)
                if float(x[h].abs().max()) < 1e-30:
                    assert s == 0 and (code == 0).all()
                    continue
                check_scale(s, x[h], m[h], kv, f"{kv} scale of token {t} plane {plane}")
                check_codes(code, x[h], m[h], s, kv, f"{kv} codes of token {t} plane {plane}")
    assert untouched(cache, got, written)


def test_per_tensor_e4m3():
    bt = Batch(*RAGGED, page=32, seed=3, rot=128)
    q, k, v = fused(bt, 8, 2, 128, True)
    k[5] *= 100  # saturates
    cache = torch.zeros(bt.nb, 2, 32, 2, 128).to(torch.float8_e4m3fn)
    out, got, _, status = run(bt, q, k, v, cache, ks=0.05, vs=0.25)
    assert status == 0
    for t, b, p in bt.tokens():
        blk, slot = bt.where(b, p)
        kr, mag = ref.rotate(k[t].double(), bt.cs[p].double(), False)
        check_codes(got[blk, 0, slot].double(), kr, mag, float(np.float32(0.05)), "fp8_e4m3", f"k {t}")
        check_codes(got[blk, 1, slot].double(), v[t].double(), torch.zeros_like(mag), 0.25, "fp8_e4m3", f"v {t}")


def block_case(bt, Hkv, D, kv, group):
    """A block-scaled cache with content in every cell."""
    x = bt.randn(bt.nb, 2, bt.page // group, group, Hkv, D)
    s = x.abs().amax(dim=(3, 5), keepdim=True) / ref.Q_MAX[kv]
    y = x / s
    code = y.round().to(torch.int8) if kv == "int8_block" else y.clamp(-448, 448).to(torch.float8_e4m3fn)
    return code.view(bt.nb, 2, bt.page, Hkv, D), s.view(bt.nb, 2, bt.page // group, Hkv).contiguous()


def check_block_append(bt, k, v, inter, kv, group, cache, scales, got, got_s):
    """Every cell and scale after one append, against the definition."""
    written = torch.zeros(bt.nb, bt.page, dtype=torch.bool)
    touched = torch.zeros(bt.nb, bt.page // group, dtype=torch.bool)
    for b, m in enumerate(bt.new):
        if m == 0:
            continue
        p0, p1 = bt.lens[b] - m, bt.lens[b]
        for first in range(p0 // group * group, p1, group):
            pa, pe = max(p0, first), min(p1, first + group)
            blk, slot = bt.where(b, first)
            gi = slot // group
            touched[blk, gi] = True
            written[blk, slot:slot + pe - first] = True
            rows = [int(bt.qs[b]) + p - p0 for p in range(pa, pe)]
            kr, mag = zip(*(ref.rotate(k[t].double(), bt.cs[p].double(), inter)
                            for t, p in zip(rows, range(pa, pe))))
            had = pa - first
            for plane, x, mg in ((0, torch.stack(kr), torch.stack(mag)),
                                 (1, v[rows].double(), torch.zeros(len(rows), *v.shape[1:], dtype=torch.float64))):
                for h in range(k.shape[1]):
                    s_old = float(scales[blk, plane, gi, h]) if had else 0.0
                    s = float(got_s[blk, plane, gi, h])
                    what = f"{kv} request {b} block at {first} plane {plane} head {h}"
                    check_scale(s, x[:, h], mg[:, h], kv, what, least=s_old)
                    at = slot + had
                    check_codes(got[blk, plane, at:at + len(rows), h].double(), x[:, h], mg[:, h], s, kv, what)
                    old = cache[blk, plane, slot:slot + had, h].double()
                    new = got[blk, plane, slot:slot + had, h].double()
                    if s == s_old:
                        assert torch.equal(old, new), what
                    elif had:
                        check_codes(new, old * s_old, torch.zeros_like(old), s, kv, what + " held")
    assert untouched(cache, got, written)
    keep = ~touched[:, None].expand(scales.shape[:3])
    assert torch.equal(scales[keep], got_s[keep])


@pytest.mark.parametrize("kv", ["fp8_e4m3_block", "int8_block"])
@pytest.mark.parametrize("page,group", [(16, 16), (48, 16), (64, 64), (32, 32)])
@pytest.mark.parametrize("Hq,Hkv,D,rot,inter", [(8, 8, 128, 128, False), (6, 3, 64, 32, True), (5, 5, 128, 64, False)])
def test_block_scaled(kv, page, group, Hq, Hkv, D, rot, inter):
    bt = Batch([1, 0, 5, 16, 70, 1, 2, 15], [0, 9, 11, 0, 40, 15, 100, 1], page, pad=2, seed=4, rot=rot)
    q, k, v = fused(bt, Hq, Hkv, D, False)
    k[2] *= 4  # the scale grows: the held codes move
    v[2] *= 0.01
    k[10] *= 50
    cache, scales = block_case(bt, Hkv, D, kv, group)
    out, got, got_s, status = run(bt, q, k, v, cache, inter=inter, scales=scales)
    assert status == 0
    for t, b, p in bt.tokens():
        check_rows(out[t], q[t], bt.cs[p], inter, f"q token {t}")
    assert (out[sum(bt.new):] == 7.0).all()
    check_block_append(bt, k, v, inter, kv, group, cache, scales, got, got_s)


@pytest.mark.parametrize("kv", ["fp8_e4m3_block", "int8_block"])
def test_block_scaled_degenerate_values(kv):
    # zeros, values below any normal scale, and a stale block of NaN codes and scales that starts anew
    bt = Batch([3, 2, 16], [0, 4, 0], 16, seed=5, rot=64)
    q, k, v = fused(bt, 2, 2, 64, True)
    k[:3], v[:3] = 0.0, 1e-39
    cache, scales = block_case(bt, 2, 64, kv, 16)
    blk = int(bt.bt[2, 0])
    cache.view(torch.uint8)[blk] = 0x7f
    scales[blk] = float("nan")
    scales[int(bt.bt[1, 0]), :, :, 0] = 0.0  # a block of zeros that grows
    cache.view(torch.uint8)[int(bt.bt[1, 0]), :, :, 0] = 0
    out, got, got_s, status = run(bt, q, k, v, cache, scales=scales)
    assert status == 0
    b0 = int(bt.bt[0, 0])
    assert (got_s[b0] == 0).all() and (got.view(torch.uint8)[b0, :, :3] == 0).all()
    bt.new[0], bt.lens[0] = 0, 0  # checked; the rest by the definition
    cache.view(torch.uint8)[b0], scales[b0] = got.view(torch.uint8)[b0], got_s[b0]
    check_block_append(bt, k, v, False, kv, 16, cache, scales, got, got_s)


def test_block_scaled_token_by_token_then_read_back():
    # 40 single-token appends: every value stays within its codes' error at the final scale, one more half step for
    # each time the scale grew
    for kv in ("fp8_e4m3_block", "int8_block"):
        bt = Batch([1], [0], 16, seed=6, rot=64, extra=4)
        bt.bt = torch.tensor([[3, 1, 0, 2]], dtype=torch.int32)
        bt.cs = table(64, 64)
        n = 40
        k, v = bt.randn(n, 2, 64).to(BF), bt.randn(n, 2, 64).to(BF)
        cs, tb, _, qs = bt.dev()
        code = torch.zeros(5, 2, 16, 2, 64, dtype=torch.int8 if kv == "int8_block" else torch.uint8, device="cuda")
        cache = code if kv == "int8_block" else code.view(torch.float8_e4m3fn)
        scales = torch.zeros(5, 2, 1, 2, device="cuda")
        grew = torch.zeros(n, 2, 2)
        prev = torch.zeros(2, 2)
        for p in range(n):
            sl = torch.tensor([p + 1], dtype=torch.int32, device="cuda")
            mqa.gqa_rope_append(k[p:p + 1].cuda(), v[p:p + 1].cuda(), cs, cache, tb, sl, qs, kv_scales=scales)
            now = scales[int(bt.bt[0, p // 16]), :, 0].cpu()
            if p % 16 == 0:
                prev = now
            grew[p // 16 * 16:p] += (now > prev).float()
            prev = now
        for p in range(n):
            blk = int(bt.bt[0, p // 16])
            kr, _ = ref.rotate(k[p].double(), bt.cs[p].double(), False)
            for plane, x in ((0, kr), (1, v[p].double())):
                s = scales[blk, plane, 0].cpu().double()[:, None]
                val = cache[blk, plane, p % 16].cpu().double() * s
                step = 0.5 * s if kv == "int8_block" else x.abs() * 2 ** -4 * 1.2 + s * 2 ** -10
                err = (val - x).abs()
                assert (err <= step * (1.001 + grew[p, plane].double()[:, None])).all(), (kv, p, plane)


@pytest.mark.parametrize("R,H", [(512, 128), (512, 1), (256, 5)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_mla(R, H, fp8, inter):
    bt = Batch([1, 3, 0, 20, 2], [0, 30, 7, 0, 47], 16, pad=2, seed=7)
    a = bt.randn(bt.T, R + 64).to(BF)
    qp = bt.randn(bt.T, H, 192).to(BF)
    cache = bt.randn(bt.nb, 16, R + 64).to(torch.float8_e4m3fn if fp8 else BF)
    cs, tb, sl, qs = bt.dev()
    da, dq, dc = a.cuda(), qp.cuda(), cache.cuda()
    q = torch.full((bt.T, H, R + 64), 7.0, dtype=BF, device="cuda")
    ks = 0.05 if fp8 else 1.0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mqa.mla_rope_append(da[:, :R], da[:, R:], cs, dc, tb, sl, qs, q_pe=dq[..., 128:], q_pe_out=q[..., R:],
                        k_scale=ks, interleaved=inter, device_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    got, q = dc.cpu(), q.cpu()
    assert (q[..., :R] == 7.0).all() and (q[sum(bt.new):] == 7.0).all()
    written = torch.zeros(bt.nb, 16, dtype=torch.bool)
    for t, b, p in bt.tokens():
        blk, slot = bt.where(b, p)
        written[blk, slot] = True
        check_rows(q[t, :, R:], qp[t, :, 128:], bt.cs[p], inter, f"q token {t}")
        y, mag = ref.rotate(a[t, None, R:].double(), bt.cs[p].double(), inter)
        if fp8:
            s = float(np.float32(ks))
            check_codes(got[blk, slot, R:].double(), y[0], mag[0], s, "fp8_e4m3", f"k_pe {t}")
            check_codes(got[blk, slot, :R].double(), a[t, :R].double(), torch.zeros(R, dtype=torch.float64), s,
                        "fp8_e4m3", f"kv_c {t}")
        else:
            check_rows(got[blk, slot, None, R:], a[t, None, R:], bt.cs[p], inter, f"k_pe {t}")
            assert torch.equal(got[blk, slot, :R], a[t, :R])
    assert torch.equal(cache.view(torch.uint8).view(bt.nb, 16, -1)[~written],
                       got.view(torch.uint8).view(bt.nb, 16, -1)[~written])


def test_in_place_and_without_queries():
    bt = Batch([2, 5], [3, 0], 16, seed=8)
    q, k, v = fused(bt, 4, 2, 64, True)
    cs, tb, sl, qs = bt.dev()
    cache = torch.zeros(bt.nb, 2, 16, 2, 64, dtype=BF, device="cuda")
    want = mqa.gqa_rope_append(k.cuda(), v.cuda(), cs, cache, tb, sl, qs, q=q.cuda())
    dq, c2 = q.cuda(), torch.zeros_like(cache)
    got = mqa.gqa_rope_append(k.cuda(), v.cuda(), cs, c2, tb, sl, qs, q=dq, q_out=dq)
    assert got is dq and torch.equal(got, want) and torch.equal(c2, cache)
    c3 = torch.zeros_like(cache)
    assert mqa.gqa_rope_append(k.cuda(), v.cuda(), cs, c3, tb, sl, qs) is None
    assert torch.equal(c3, cache)
    none = mqa.gqa_rope_append(k[:0].cuda(), v[:0].cuda(), cs, c3, tb, sl, torch.zeros_like(qs), q=q[:0].cuda())
    assert none.shape == (0, 4, 64) and torch.equal(c3, cache)


@pytest.mark.parametrize("kv", ["bf16", "int8_block"])
def test_bad_places_are_reported_and_skipped(kv):
    bt = Batch([2, 3, 1, 4], [14, 0, 20, 5], 16, seed=9)
    q, k, v = fused(bt, 4, 2, 64, True)
    if kv == "bf16":
        cache, scales = bt.randn(bt.nb, 2, 16, 2, 64).to(BF), None
    else:
        cache, scales = block_case(bt, 2, 64, kv, 16)
    lens, table_, cs = list(bt.lens), bt.bt.clone(), bt.cs
    for what in ("length", "negative", "block", "negative block", "table", "angles"):
        bt.lens, bt.bt, bt.cs = list(lens), table_.clone(), cs
        if what == "length":
            bt.lens[1] = 2           # three new tokens in a length of two
        elif what == "negative":
            bt.lens[1] = -5
        elif what == "block":
            bt.bt[1, 0] = bt.nb
        elif what == "negative block":
            bt.bt[1, 0] = -1
        elif what == "table":
            bt.lens[1] = 16 * bt.bt.shape[1] + 3   # wholly behind the table
        else:
            bt.cs = cs[:21]          # request 2 sits at position 20: the last angle; others fit
            bt.lens[1] = 40
        out, got, got_s, status = run(bt, q, k, v, cache, scales=scales)
        assert status == 5, what
        keep = torch.ones(bt.nb, dtype=torch.bool)
        for b in (0, 2, 3):
            for p in range(lens[b] - bt.new[b], lens[b]):
                keep[bt.where(b, p)[0]] = False
                check_rows(out[int(bt.qs[b]) + p - lens[b] + bt.new[b]], q[int(bt.qs[b]) + p - lens[b] + bt.new[b]],
                           bt.cs[p], False, what)
                if kv == "bf16":
                    blk, slot = bt.where(b, p)
                    assert torch.equal(got[blk, 1, slot], v[int(bt.qs[b]) + p - lens[b] + bt.new[b]])
        assert torch.equal(got.view(torch.uint8)[keep], cache.view(torch.uint8)[keep]), what


def test_large_batches_and_offsets():
    # 700 requests (the search over query_start takes several rounds) in a cache whose offsets pass 32 bits
    rng = np.random.default_rng(1)
    new = rng.integers(0, 4, 700).tolist()
    bt = Batch(new, rng.integers(0, 30, 700).tolist(), 16, pad=1, seed=10, rot=128)
    q, k, v = fused(bt, 8, 8, 128, False)
    shift = (5 << 30) // (2 * 16 * 8 * 128 * 2)
    bt.bt = torch.where(bt.bt >= 0, bt.bt + shift, bt.bt)
    cache = torch.zeros(bt.nb + shift, 2, 16, 8, 128, dtype=BF, device="cuda")
    cs, tb, sl, qs = bt.dev()
    base = q._base.cuda()
    out = mqa.gqa_rope_append(base[:, 8:16], base[:, 16:24], cs, cache, tb, sl, qs, q=base[:, :8])
    got, out = cache[shift:].cpu(), out.cpu()
    assert not cache[:shift].any()
    for t, b, p in bt.tokens():
        blk, slot = bt.where(b, p)
        assert torch.equal(got[blk - shift, 1, slot], v[t])
        if t % 29 == 0:
            check_rows(out[t], q[t], bt.cs[p], False, f"q {t}")
            check_rows(got[blk - shift, 0, slot], k[t], bt.cs[p], False, f"k {t}")


@pytest.mark.parametrize("kv", ["fp8_e4m3_block", "int8_block"])
def test_block_scaled_many_requests(kv):
    rng = np.random.default_rng(2)
    new = rng.choice([0, 1, 1, 1, 2, 9], 150).tolist()
    bt = Batch(new, rng.integers(0, 40, 150).tolist(), 32, pad=1, seed=11, rot=64)
    q, k, v = fused(bt, 2, 1, 64, False)
    cache, scales = block_case(bt, 1, 64, kv, 16)
    _, got, got_s, status = run(bt, q, k, v, cache, scales=scales)
    assert status == 0
    check_block_append(bt, k, v, False, kv, 16, cache, scales, got, got_s)


@pytest.mark.parametrize("page,group", [(16, 16), (64, 32)])
def test_block_scaled_batches_of_short_runs(page, group):
    # more than 32 x 32 requests of a few tokens each: several rounds of search, by number and by token
    rng = np.random.default_rng(6)
    for counts in ([3, 4, 5, 17], [0, 1, 1, 2]):
        new = rng.choice(counts, 1100).tolist()
        bt = Batch(new, rng.integers(0, 70, 1100).tolist(), page, pad=3, seed=12, rot=64)
        q, k, v = fused(bt, 1, 1, 64, False)
        cache, scales = block_case(bt, 1, 64, "int8_block", group)
        _, got, got_s, status = run(bt, q, k, v, cache, scales=scales)
        assert status == 0
        check_block_append(bt, k, v, False, "int8_block", group, cache, scales, got, got_s)


def test_block_scaled_bad_requests_are_reported_by_number():
    # long runs (shares found by number): one request shorter than its new tokens, one beyond its pages
    for bad in (0, 1):
        bt = Batch([40, 50, 45], [5, 0, 20], 16, seed=13, rot=64)
        q, k, v = fused(bt, 2, 1, 64, False)
        cache, scales = block_case(bt, 1, 64, "int8_block", 16)
        lens = list(bt.lens)
        bt.lens[1] = 49 if bad == 0 else 16 * bt.bt.shape[1] + 1
        bt.cs = table(16 * bt.bt.shape[1] + 2, 64)
        _, got, got_s, status = run(bt, q, k, v, cache, scales=scales)
        assert status == 5
        bt.lens = lens
        ok = torch.zeros(bt.nb, dtype=torch.bool)
        ok[bt.bt[[0, 2]][bt.bt[[0, 2]] >= 0].long()] = True
        for b in (0, 2):
            p0 = bt.lens[b] - bt.new[b]
            for p in range(p0, bt.lens[b]):
                blk, slot = bt.where(b, p)
                t = int(bt.qs[b]) + p - p0
                s = float(got_s[blk, 1, 0, 0])
                check_codes(got[blk, 1, slot, 0].double(), v[t, 0].double(), torch.zeros(64, dtype=torch.float64), s,
                            "int8_block", f"request {b} position {p}")
        if bad == 0:  # its pages keep their bytes
            own = bt.bt[1][bt.bt[1] >= 0].long()
            assert torch.equal(got[own], cache[own]) and torch.equal(got_s[own], scales[own])
        assert torch.equal(got[~ok & ~torch.isin(torch.arange(bt.nb), bt.bt[1].long())],
                           cache[~ok & ~torch.isin(torch.arange(bt.nb), bt.bt[1].long())])


def test_mla_query_rows_in_any_order():
    # q_pe_out with a token's heads side by side, and with a head's tokens side by side; inputs that overlap
    bt = Batch([1, 4], [3, 30], 16, seed=14)
    R, H = 512, 3
    cs, tb, sl, qs = bt.dev()
    a = bt.randn(bt.T, R + 64).to(BF).cuda()
    base = bt.randn(H + bt.T, 64).to(BF).cuda()
    q = base.as_strided((bt.T, H, 64), (64, 64, 1))
    want = None
    for out in (torch.zeros(bt.T, H, 64, dtype=BF, device="cuda"),
                torch.zeros(H, bt.T, 64, dtype=BF, device="cuda").transpose(0, 1),
                torch.zeros(bt.T, H, R + 64, dtype=BF, device="cuda")[..., R:]):
        cache = torch.zeros(bt.nb, 16, R + 64, dtype=BF, device="cuda")
        got = mqa.mla_rope_append(a[:, :R], a[:, R:], cs, cache, tb, sl, qs, q_pe=q, q_pe_out=out)
        torch.cuda.synchronize()
        assert got is out
        if want is None:
            want = out.clone()
            for t, _, p in bt.tokens():
                check_rows(out.cpu()[t], q.cpu()[t], bt.cs[p], False, f"q token {t}")
        assert torch.equal(out, want)
    with pytest.raises(mqa.MqaError):
        mqa.mla_rope_append(a[:, :R], a[:, R:], cs, cache, tb, sl, qs, q_pe=q, q_pe_out=q)
