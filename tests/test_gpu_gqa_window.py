"""GPU parity of windowed and block-scaled GQA decode (C ABI -> sm_103a
kernels) against a 64-bit reference on the same values, with bounds derived
from the kernels' roundings (cache_reference.py)."""
import numpy as np
import pytest
import torch

import cache_reference as ref
import mqa_decode_attention_paged_gb300 as mqa

pytestmark = pytest.mark.gpu

NONE = 1 << 30
KINDS = ["bf16", "fp8_e4m3", "fp8_e4m3_block", "int8_block"]


class Case:
    """A paged batch on the CPU; every byte that no query may see is poisoned, and the block-table entries of pages
    without a visible key hold invalid ids."""

    def __init__(self, lens, Hq, Hkv, D, page, kv, L=1, window=NONE, sinks=0, group=16, seed=0, poison=True,
                 extra=2):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.L, self.page, self.kv, self.window, self.sinks = lens, L, page, kv, window, sinks
        B = len(lens)
        pages = [-(-n // page) for n in lens]
        nb = sum(pages) + extra
        self.nb = nb
        perm = torch.randperm(nb, generator=g)
        width = max(1, max(pages)) + 1
        bt = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(pages):
            bt[b, :m] = perm[at:at + m].to(torch.int32)
            at += m
        self.q = torch.randn(B, L, Hq, D, generator=g).to(torch.bfloat16)
        x = torch.randn(nb, 2, page, Hkv, D, generator=g)
        self.scales, self.ks, self.vs = None, 1.0, 1.0
        if kv == "bf16":
            self.cache = x.to(torch.bfloat16)
        elif kv == "fp8_e4m3":
            self.ks, self.vs = 0.05, 0.03
            self.cache = (x / 0.05).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            x = x.view(nb, 2, page // group, group, Hkv, D)
            x *= torch.exp(torch.randn(nb, 2, page // group, 1, Hkv, 1, generator=g))
            s = x.abs().amax(dim=(3, 5), keepdim=True) / ref.Q_MAX[kv]
            y = x / s
            codes = y.round().to(torch.int8) if kv == "int8_block" else y.clamp(-448, 448).to(torch.float8_e4m3fn)
            self.cache = codes.view(nb, 2, page, Hkv, D)
            self.scales = s.view(nb, 2, page // group, Hkv).contiguous()
        self.group = group
        self.scale = D ** -0.5
        self.bt_ref = bt.clone()
        if poison:
            raw = self.cache.view(torch.uint8) if kv.startswith("fp8") else self.cache
            bad = float("nan") if kv == "bf16" else 0x7f
            seen = torch.zeros(nb, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                ok = torch.zeros(max(1, pages[b]) * page, dtype=torch.bool)
                for p in range(max(0, n - L), n):
                    t = torch.arange(p + 1)
                    ok[t[(t < sinks) | (t > p - window)]] = True
                for j in range(pages[b]):
                    part = ok[j * page:(j + 1) * page]
                    seen[bt[b, j]] = part
                    if not part.any():
                        bt[b, j] = (-1, nb, 1 << 30)[j % 3]
            raw.masked_fill_(~seen[:, None, :, None, None], bad)
            if self.scales is not None:
                dead = ~seen.view(nb, page // group, group).any(-1)
                self.scales.masked_fill_(dead[:, None, :, None], float("nan"))
        self.bt = bt

    def dev(self):
        return [None if t is None else t.cuda() for t in (self.q, self.cache, self.bt, self.scales)] + [
            torch.tensor(self.lens, dtype=torch.int32, device="cuda")]

    def values(self, b, plane):
        """(values, codes, per-token scales) of request b's tokens, float64, poisoned bytes as zeros."""
        n = self.lens[b]
        codes = ref.gather(self.cache, self.bt_ref, b, n, self.page, plane).nan_to_num(0.0, 0.0, 0.0)
        Hkv = self.cache.shape[3]
        if self.scales is not None:
            s = ref.token_scales(self.scales, self.bt_ref, b, n, self.page, plane).nan_to_num(0.0)
        else:
            s = torch.full((n, Hkv), self.ks if plane == 0 else self.vs, dtype=torch.float64)
        return codes * s[..., None], codes, s

    def reference(self, rows=None):
        for b in rows if rows is not None else range(len(self.lens)):
            k, _, _ = self.values(b, 0)
            v, code, s = self.values(b, 1)
            yield b, ref.window_decode(self.q[b].double(), k, v, self.lens[b], self.scale, self.window, self.sinks,
                                       code_v=code, s_v=s, half_p=self.kv != "bf16")

    def run(self, splits=None, dev=None, **kw):
        q, kv, bt, sc, sl = dev or self.dev()
        B, L, Hq, D = q.shape
        Hkv = kv.shape[3]
        out = torch.full_like(q, float("nan"))
        lse = torch.full(q.shape[:3], float("nan"), device="cuda")
        n = splits or mqa.gqa_window_num_kv_splits(B, L, Hq, Hkv)
        ws = torch.full((max(16, mqa.gqa_window_decode_workspace_bytes(B, L, Hq, Hkv, D, n)),), 0xFF,
                        dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = dict(out=out, lse=lse, num_kv_splits=n, workspace=ws, device_status=status, **kw)
        if self.window >= NONE and self.sinks == 0 and sc is not None:
            mqa.gqa_block_decode(q, kv, sc, bt, sl, self.scale, **kw)
        else:
            mqa.gqa_window_decode(q, kv, bt, sl, self.scale, self.window, self.sinks, kv_scales=sc, k_scale=self.ks,
                                  v_scale=self.vs, **kw)
        torch.cuda.synchronize()
        return out.cpu().double(), lse.cpu().double(), int(status.item())


def check(case, out, lse, rows=None, what=""):
    for b, (o, l, tol_o, tol_l) in case.reference(rows):
        dead = torch.isneginf(l)
        assert torch.equal(torch.isneginf(lse[b]), dead), f"{what}: lse -inf pattern, request {b}"
        assert (out[b][dead] == 0).all(), f"{what}: rows without a key, request {b}"
        err = (out[b] - o).abs()
        assert (err <= tol_o).all(), f"{what}: request {b} out off by {float((err / tol_o).max()):.2f} x its bound"
        e2 = (lse[b] - l)[~dead].abs()
        assert (e2 <= tol_l[~dead]).all(), f"{what}: request {b} lse off by {float((e2 / tol_l[~dead]).max()):.2f} x"


def run_and_check(case, splits, what=""):
    dev = case.dev()
    for s in splits:
        out, lse, status = case.run(s, dev)
        assert status == 0, f"{what}: status {status}"
        check(case, out, lse, what=f"{what} splits={s}")


RAGGED = [1, 15, 16, 17, 40, 0, 100, 333]
HEADS = [(32, 8, 128), (8, 8, 64), (16, 1, 64), (12, 4, 128), (6, 3, 128), (10, 5, 64), (14, 2, 64), (64, 8, 64)]


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_window_shapes(kv, Hq, Hkv, D):
    for window, sinks in ((1, 0), (16, 1), (33, 4), (100, 40)):
        case = Case(RAGGED, Hq, Hkv, D, 16, kv, window=window, sinks=sinks, seed=1)
        run_and_check(case, (1, 2, None), f"{kv} {Hq}/{Hkv}x{D} W={window} S={sinks}")


@pytest.mark.parametrize("kv", ["fp8_e4m3_block", "int8_block"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_block_shapes(kv, Hq, Hkv, D):
    run_and_check(Case(RAGGED, Hq, Hkv, D, 16, kv, seed=2), (1, 3, None), f"{kv} {Hq}/{Hkv}x{D}")


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("page,group", [(16, 16), (32, 16), (48, 48), (64, 32), (128, 64), (256, 256)])
def test_pages_and_scale_blocks(kv, page, group):
    for Hkv in (8, 2, 1):
        case = Case([1, 47, 129, 300, 700], 4 * Hkv, Hkv, 64, page, kv, window=200, sinks=20, group=group, seed=3)
        run_and_check(case, (1, None), f"{kv} page={page} G={group} Hkv={Hkv}")


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("L,Hq,Hkv,D", [(2, 8, 2, 128), (5, 32, 8, 64), (3, 7, 1, 128), (4, 32, 8, 128),
                                        (8, 16, 1, 64), (128, 2, 2, 64), (17, 14, 2, 128)])
def test_several_positions(kv, L, Hq, Hkv, D):
    # fewer cached tokens than positions: the first rows see nothing
    for window, sinks in ((1, 0), (24, 3), (NONE, 0)):
        case = Case([0, 1, L - 1, L, L + 15, 130], Hq, Hkv, D, 16, kv, L=L, window=window, sinks=sinks, seed=4)
        run_and_check(case, (1, None), f"{kv} L={L} {Hq}/{Hkv}x{D} W={window}")


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3_block"])
@pytest.mark.parametrize("bad", ["inf", "nan"])
def test_non_finite_value_reaches_only_the_queries_that_see_it(kv, bad):
    # the last token's V is seen by the last position only, the token that the
    # window drops next by the first position only
    L, n, W = 4, 90, 32
    case = Case([n], 8, 2, 64, 16, kv, L=L, window=W, sinks=0, seed=5)
    raw = case.cache if kv == "bf16" else case.cache.view(torch.uint8)
    value = (float(bad) if kv == "bf16" else 0x7f)  # e4m3 has no Inf: NaN in both cases
    for t in (n - 1, n - L - W + 1):
        raw[case.bt[0, t // 16], 1, t % 16] = value
    out, lse, _ = case.run(1)

    # the reference takes non-finite values as zeros: right for the rows that do not see them
    (_, (o, l, tol_o, tol_l)), = case.reference()
    for i in (1, 2):
        assert ((out[0, i] - o[i]).abs() <= tol_o[i]).all(), f"row {i}"
    assert not torch.isfinite(out[0, 0]).any() and not torch.isfinite(out[0, 3]).any()
    assert ((lse[0] - l).abs() <= tol_l).all()


def test_scales_of_unlike_magnitude():
    for kv in ("fp8_e4m3_block", "int8_block"):
        case = Case([300, 90, 40], 8, 2, 128, 16, kv, seed=6, poison=False)
        bt = case.bt
        case.scales[bt[1, :6].long(), 1] *= 1e-7       # a whole request of tiny values
        case.scales[bt[0, 15:18].long(), 1] *= 3e4     # late jumps
        case.scales[bt[2, 1].long(), 1] *= 1e-20       # one tiny block between ordinary ones
        case.scales[bt[2, 2].long(), :] = 0.0          # and one of zeros
        case.scales[bt[0, 0].long(), 0] *= 20.0        # large logits
        run_and_check(case, (1, 4, None), kv)


def test_all_values_zero_and_zero_scales():
    case = Case([50], 8, 2, 64, 16, "int8_block", seed=7, poison=False)
    case.scales.zero_()
    out, lse, status = case.run(None)
    assert status == 0 and (out == 0).all()
    assert (lse - np.log(50)).abs().max() < 1e-5


@pytest.mark.parametrize("kv", KINDS)
def test_reproducible_and_batch_invariant(kv):
    case = Case([700, 20, 333, 1, 512, 90], 32, 8, 128, 16, kv, window=256, sinks=4, seed=8)
    dev = case.dev()
    for s in (1, None):
        a, b = case.run(s, dev), case.run(s, dev)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one = case.run(1, dev)
    q, cache, bt, sc, sl = dev
    part = case.run(1, [q[[4, 1]].contiguous(), cache, bt[[4, 1]].contiguous(), sc, sl[[4, 1]].contiguous()])
    assert torch.equal(part[0], one[0][[4, 1]]) and torch.equal(part[1], one[1][[4, 1]])


def test_bad_block_id_and_lengths_are_reported():
    case = Case([40, 70, 33], 8, 2, 128, 16, "int8_block", seed=9, poison=False)
    case.bt[1, 2] = case.nb + 5
    for s in (1, None):
        out, lse, status = case.run(s)
        assert status == 5 and torch.isfinite(out).all()
        check(case, out, lse, rows=[0, 2])
    case = Case([40, 70], 8, 2, 128, 16, "bf16", window=20, seed=9, poison=False)
    q, kv, bt, sc, sl = case.dev()
    for n, want in ((-3, 0), (10 ** 6, bt.shape[1] * 16)):
        sl[1] = n
        out, lse, status = case.run(None, [q, kv, bt, sc, sl])
        assert status == 5
        check(case, out, lse, rows=[0])


def test_layouts_of_the_call():
    case = Case([90, 7], 8, 2, 64, 16, "bf16", window=40, sinks=2, seed=10)
    q, kv, bt, _, sl = case.dev()
    want, lse, _ = case.run(1)
    o3, l3 = mqa.gqa_window_decode(q[:, 0].contiguous(), kv, bt, sl, case.scale, 40, 2, num_kv_splits=1)
    assert o3.shape == (2, 8, 64) and l3.shape == (2, 8)
    assert torch.equal(o3.cpu().double(), want[:, 0]) and torch.equal(l3.cpu().double(), lse[:, 0])
    o, none = mqa.gqa_window_decode(q, kv, bt, sl, case.scale, 40, 2, num_kv_splits=1, return_lse=False)
    assert none is None and torch.equal(o.cpu().double(), want)
    # a window wider than any length is no window
    wide = Case([90, 7], 8, 2, 64, 16, "int8_block", window=10 ** 9, sinks=0, seed=10)
    run_and_check(wide, (1, None))


def test_full_batches():
    # as many virtual requests as a call takes: single tokens and short lengths
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 40, 2048).tolist()
    case = Case(lens, 2, 1, 64, 16, "int8_block", seed=11, poison=False)
    out, lse, status = case.run(None)
    assert status == 0
    check(case, out, lse, rows=[0, 1, 2, 1023, 1024, 2046, 2047])
    one, l1, _ = case.run(1)
    check(case, one, l1, rows=[3, 5, 2047])


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3_block"])
def test_cells_behind_four_gigabytes(kv):
    # blocks at the far end of a cache whose byte offsets pass 32 bits
    small = Case([200, 33], 8, 8, 128, 16, kv, window=150, sinks=3, seed=12, poison=False)
    per = 2 * 16 * 8 * 128 * (2 if kv == "bf16" else 1)
    shift = (5 << 30) // per
    q, cache, bt, sc, sl = small.dev()
    big = torch.zeros((shift + small.nb,) + tuple(cache.shape[1:]), dtype=torch.uint8 if kv != "bf16" else cache.dtype,
                      device="cuda")
    big[shift:] = cache.view(torch.uint8) if kv != "bf16" else cache
    if sc is not None:
        far = torch.zeros((shift + small.nb,) + tuple(sc.shape[1:]), device="cuda")
        far[shift:] = sc
        sc = far
    bt = torch.where(bt >= 0, bt + shift, bt)
    out, lse, status = small.run(None, [q, big.view(cache.dtype), bt, sc, sl])
    assert status == 0
    check(small, out, lse)


def test_streams_and_graphs():
    # captured once and replayed with other lengths and queries; two graphs with workspaces of their own; a call on
    # another stream than the current one
    case = Case([300, 20, 150], 8, 2, 128, 16, "fp8_e4m3_block", window=64, sinks=4, seed=13, poison=False)
    q, kv, bt, sc, sl = case.dev()
    call = lambda **kw: mqa.gqa_window_decode(q, kv, bt, sl, case.scale, 64, 4, kv_scales=sc, **kw)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = call()
        graphs.append((g, res))
    for lens in ([300, 20, 150], [17, 1, 149], [0, 20, 64]):
        case.lens = lens
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, (out, lse) in graphs:
            check(case, out.cpu().double(), lse.cpu().double(), what=f"replay {lens}")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    results = [call(stream=s) for _ in range(3)]
    raw = call(stream=s.cuda_stream)
    s.synchronize()
    for out, lse in results + [raw]:
        check(case, out.cpu().double(), lse.cpu().double(), what="other stream")


@pytest.mark.parametrize("kv,Hkv", [("bf16", 8), ("int8_block", 2), ("fp8_e4m3_block", 1)])
def test_a_wait_that_runs_out_is_reported(kv, Hkv, monkeypatch):
    # one unit copies nothing: its bounded waits (2 s) run out, every block returns (also where warps of a head meet
    # to hand over their sums, and where requests are cut and merged), the status says so, and the context goes on
    monkeypatch.setenv("MQA_ENABLE_TEST_HOOKS", "1")
    import ctypes
    from mqa_decode_attention_paged_gb300 import _binding as binding
    P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    fn = binding.lib.mqa_test_gqa_window_withheld
    fn.restype = I
    fn.argtypes = [P, P, P, P, P, F, I, I, P, P, I, I, I, I, I, I, I, I, I, I, I, P, SZ, P, P, I]
    case = Case([900, 300, 40], 4 * Hkv, Hkv, 64, 16, kv, window=700, sinks=4, seed=16, poison=False)
    q, cache, bt, sc, sl = case.dev()
    B, L, Hq, D = q.shape
    code = binding._KV_NAMES[kv]
    for splits in (1, 3):
        out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda")
        ws = torch.full((max(16, mqa.gqa_window_decode_workspace_bytes(B, L, Hq, Hkv, D, splits)),), 0xFF,
                        dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        rc = fn(q.data_ptr(), cache.data_ptr(), None if sc is None else sc.data_ptr(), bt.data_ptr(), sl.data_ptr(),
                case.scale, 700, 4, out.data_ptr(), lse.data_ptr(), B, L, Hq, Hkv, D, case.nb, 16, bt.shape[1], 16,
                code, splits, ws.data_ptr(), ws.numel(), status.data_ptr(), torch.cuda.current_stream().cuda_stream, 0)
        assert rc == binding.OK
        torch.cuda.synchronize()
        assert int(status.item()) == binding.ERR_DEVICE_TIMEOUT
        if splits == 1:
            check(case, out.cpu().double(), lse.cpu().double(), rows=[1, 2])
    run_and_check(case, (1, None))


def test_two_calls_at_once():
    cases = [Case([400, 90, 33], 32, 8, 128, 16, kv, window=100, sinks=4, seed=14) for kv in ("bf16", "int8_block")]
    devs = [c.dev() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    res = []
    for c, d, s in zip(cases, devs, streams):
        with torch.cuda.stream(s):
            for _ in range(4):
                res.append((c, mqa.gqa_window_decode(d[0], d[1], d[2], d[4], c.scale, 100, 4, kv_scales=d[3])))
    torch.cuda.synchronize()
    for c, (out, lse) in res:
        check(c, out.cpu().double(), lse.cpu().double())


def test_random_shapes():
    rng = np.random.default_rng(3)
    for _ in range(40):
        Hkv = int(rng.integers(1, 9))
        grp, L = int(rng.integers(1, 17)), int(rng.integers(1, 8))
        kv = KINDS[int(rng.integers(0, 4))]
        page = int(rng.choice([16, 32, 48, 64]))
        case = Case([int(x) for x in rng.integers(0, 500, int(rng.integers(1, 6)))], Hkv * grp, Hkv,
                    int(rng.choice([64, 128])), page, kv, L=L, window=int(rng.choice([1, 7, 64, 300, NONE])),
                    sinks=int(rng.choice([0, 1, 5, 70])), group=int(rng.choice([16, page])), seed=int(rng.integers(1 << 30)))
        run_and_check(case, (1, int(rng.integers(2, 9)), None),
                      f"{kv} Hkv={Hkv} grp={grp} L={L} page={page} lens={case.lens} W={case.window} S={case.sinks}")


def widen(case, columns=2048):
    """The same batch under a block table made for far longer requests: nothing says that they are short."""
    case.bt = torch.cat([case.bt, torch.full((len(case.lens), columns), -1, dtype=torch.int32)], 1)
    return case


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("L,Hq,Hkv,D", [(1, 32, 8, 128), (1, 16, 1, 64), (1, 12, 4, 128), (4, 32, 8, 128),
                                        (5, 32, 8, 64), (17, 14, 2, 128), (3, 6, 3, 64)])
def test_short_requests_that_are_cut(kv, L, Hq, Hkv, D):
    # nothing but the lengths on the device says that requests are short: they are cut and merged
    for window, sinks in ((NONE, 0), (3000, 7)):
        case = widen(Case([0, 1, L + 1, L + 15, 130, 333, 700], Hq, Hkv, D, 16, kv, L=L, window=window, sinks=sinks,
                          seed=17))
        run_and_check(case, (2, 3, None), f"{kv} L={L} {Hq}/{Hkv}x{D} W={window}")


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (32, 2, 128)])
def test_more_requests_than_blocks(kv, Hq, Hkv, D):
    # units that hold several requests and parts of others, under a small window
    lens = np.random.default_rng(5).integers(0, 120, 330).tolist()
    for window, sinks in ((1, 0), (24, 3)):
        case = Case(lens, Hq, Hkv, D, 16, kv, window=window, sinks=sinks, seed=18)
        for s in (2, None):
            out, lse, status = case.run(s)
            assert status == 0
            check(case, out, lse, rows=[*range(0, 330, 7), 328, 329], what=f"{kv} W={window} splits={s}")


def test_graphs_of_cut_requests():
    # two captured calls over one batch, each with its own partials, replayed together on two streams
    case = widen(Case([700, 20, 1500], 8, 2, 128, 16, "int8_block", seed=19, poison=False))
    q, kv, bt, sc, sl = case.dev()
    graphs = []
    for _ in range(2):
        mqa.gqa_block_decode(q, kv, sc, bt, sl, case.scale)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = mqa.gqa_block_decode(q, kv, sc, bt, sl, case.scale)
        graphs.append((g, res, torch.cuda.Stream()))
    for lens in ([700, 20, 1500], [1, 0, 900], [333, 20, 17]):
        case.lens = lens
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for g, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for _, (out, lse), _ in graphs:
            check(case, out.cpu().double(), lse.cpu().double(), what=f"replay {lens}")


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("L,Hq,Hkv,D", [(5, 32, 8, 128), (12, 2, 1, 128), (5, 7, 1, 128), (9, 10, 5, 64), (24, 1, 1, 64),
                                        (25, 4, 4, 128), (7, 28, 4, 64)])
def test_blocks_of_many_rows(kv, L, Hq, Hkv, D):
    # 17 to 24 rows in one block, more in blocks of unlike sizes; whole and cut, with values that some rows must not see
    for window, sinks in ((9, 2), (NONE, 0)):
        case = Case([0, L - 1, L + 2, 60, 500], Hq, Hkv, D, 32, kv, L=L, window=window, sinks=sinks, group=16, seed=20)
        run_and_check(case, (1, None), f"{kv} L={L} {Hq}/{Hkv}x{D} W={window}")
        run_and_check(widen(case), (3,), f"{kv} L={L} {Hq}/{Hkv}x{D} W={window} cut")


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3_block"])
def test_non_finite_value_among_many_rows(kv):
    # 20 rows of a block: the last token's V is NaN and seen by the last position only
    L, n = 5, 90
    case = Case([n], 8, 2, 64, 16, kv, L=L, window=32, sinks=0, seed=21)
    raw = case.cache if kv == "bf16" else case.cache.view(torch.uint8)
    raw[case.bt[0, (n - 1) // 16], 1, (n - 1) % 16] = float("nan") if kv == "bf16" else 0x7f
    out, lse, _ = case.run(1)
    (_, (o, l, tol_o, tol_l)), = case.reference()
    assert ((out[0, :L - 1] - o[:L - 1]).abs() <= tol_o[:L - 1]).all()
    assert not torch.isfinite(out[0, L - 1]).any()
    assert ((lse[0] - l).abs() <= tol_l).all()


@pytest.mark.parametrize("kv", ["fp8_e4m3_block", "int8_block"])
@pytest.mark.parametrize("bad", ["inf", "nan"])
@pytest.mark.parametrize("L,Hq,Hkv,D", [(4, 8, 2, 64), (4, 8, 2, 128), (4, 8, 4, 128), (5, 40, 8, 128), (9, 8, 1, 64),
                                        (3, 20, 2, 64)])
def test_non_finite_value_scale_reaches_only_the_queries_that_see_it(kv, bad, L, Hq, Hkv, D):
    # the last token starts a scale block whose V scale (of the first head) is Inf or NaN: the last position alone
    # sees it; the first positions of the batch see no key at all or keys of that block only
    n = 97
    grp = Hq // Hkv
    for lens, cut in (([n], False), ([n, 40, 1], True)):
        case = Case(lens, Hq, Hkv, D, 16, kv, L=L, seed=22, poison=False)
        want = dict(case.reference())  # (before the scale is planted: rows that do not see it)
        case.scales[case.bt[0, 6], 1, :, 0] = float(bad)
        if cut:
            widen(case)
        for splits in ((1,) if not cut else (3, None)):
            out, lse, status = case.run(splits)
            assert status == 0
            for b, (o, l, tol_o, tol_l) in want.items():
                ok = torch.ones(L, Hq, dtype=torch.bool)
                if b == 0:
                    ok[L - 1, :grp] = False
                    assert not torch.isfinite(out[0, L - 1, :grp]).any(), f"{kv} {bad} splits={splits}"
                assert ((out[b] - o).abs() <= tol_o)[ok].all(), f"{kv} {bad} splits={splits} request {b}"
                dead = torch.isneginf(l)
                assert torch.equal(torch.isneginf(lse[b]), dead) and (out[b][dead] == 0).all()
                assert ((lse[b] - l).abs() <= tol_l)[~dead].all(), f"{kv} {bad} splits={splits} request {b}"


@pytest.mark.parametrize("kv", ["fp8_e4m3_block", "int8_block"])
def test_appended_infinity_reaches_only_the_queries_that_see_it(kv):
    # the scale as gqa_rope_append stores it: of four new tokens the last starts a scale block and holds an Inf
    from test_gpu_append import table
    L, old, Hq, Hkv, D = 4, 13, 8, 2, 64
    case = Case([old + L - 1], Hq, Hkv, D, 16, kv, L=L, seed=23, poison=False)
    q, cache, bt, sc, _ = case.dev()
    bt[0, 1] = case.nb - 1 if int(bt[0, 0]) != case.nb - 1 else case.nb - 2
    k, v = torch.randn(L, Hkv, D).to(torch.bfloat16), torch.randn(L, Hkv, D).to(torch.bfloat16)
    v[L - 1, 0, 5] = float("inf")
    lens = torch.tensor([old + L], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    rq = mqa.gqa_rope_append(k.cuda(), v.cuda(), table(32, D).cuda(), cache, bt, lens, starts,
                             q=q[0].contiguous(), kv_scales=sc)
    torch.cuda.synchronize()
    assert torch.isinf(sc[bt[0, 1].item(), 1, 0, 0]) and torch.isfinite(sc[bt[0, 1].item(), 1, 0, 1])
    case.cache, case.scales, case.q, case.lens = cache.cpu(), sc.cpu(), rq.cpu()[None], [old + L]
    case.bt = case.bt_ref = bt.cpu()
    grp = Hq // Hkv
    case.scales[bt[0, 1].item(), 1, 0, 0] = 1.0  # for the rows that do not see it
    (_, (o, l, tol_o, tol_l)), = case.reference()
    for splits in (1, None):
        out, lse, status = case.run(splits, [rq[None], cache, bt, sc, lens])
        assert status == 0
        assert ((out[0] - o).abs() <= tol_o)[:L - 1].all() and ((out[0] - o).abs() <= tol_o)[:, grp:].all()
        assert not torch.isfinite(out[0, L - 1, :grp]).any()
        assert ((lse[0] - l).abs() <= tol_l).all()


def test_no_window_beyond_two_to_the_thirty_keys():
    # one request of 2^30 + 2^16 tokens through a table that repeats a page: the first page holds the keys that count
    page, columns, D = 1 << 16, (1 << 14) + 1, 64
    cache = torch.zeros(2, 2, page, 1, D, dtype=torch.int8, device="cuda")
    cache[0, 0], cache[0, 1] = 1, 100  # logits 25, values 100; the other page: logits 0, values 0
    sc = torch.ones(2, 2, 1, 1, device="cuda")
    bt = torch.ones(1, columns, dtype=torch.int32, device="cuda")
    bt[0, 0] = 0
    n = columns * page
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.ones(1, 1, D, dtype=torch.bfloat16, device="cuda")
    # the weight of the first page's keys is 1 - 2.3e-7; lse is off by a few thousand fp32 additions
    want = 25 + np.log(page + (n - page) * np.exp(-25.0))
    for call in (lambda: mqa.gqa_block_decode(q, cache, sc, bt, sl, 25 / D),
                 lambda: mqa.gqa_window_decode(q, cache, bt, sl, 25 / D, NONE, kv_scales=sc),
                 lambda: mqa.gqa_window_decode(q, cache, bt, sl, 25 / D, (1 << 31) - 1, kv_scales=sc)):
        out, lse = call()
        assert (out.cpu().double() - 100).abs().max() <= 100 * 2 ** -8
        assert abs(float(lse) - want) <= 4096 * 2 ** -24 + 2 ** -20 * want


def test_windows_and_sinks_wider_than_an_int():
    case = Case([90, 7, 300], 8, 2, 64, 16, "bf16", seed=24, poison=False)
    q, kv, bt, _, sl = case.dev()
    want = mqa.gqa_window_decode(q, kv, bt, sl, case.scale, NONE)
    for window, sinks in (((1 << 32) + 5, 0), ((1 << 63) + 1, 0), ((1 << 33) + 1, 3), (1, (1 << 32) + 2),
                          (1, (1 << 31) - 1)):
        got = mqa.gqa_window_decode(q, kv, bt, sl, case.scale, window, sinks, num_kv_splits=1)
        check(case, got[0].cpu().double(), got[1].cpu().double(), what=f"W={window} S={sinks}")
    check(case, want[0].cpu().double(), want[1].cpu().double())
    for window, sinks in ((-(1 << 32) + 5, 0), (5, -(1 << 32) + 5), (0, 0), (5, -1)):
        with pytest.raises(mqa.MqaError):
            mqa.gqa_window_decode(q, kv, bt, sl, case.scale, window, sinks)


@pytest.mark.parametrize("kv,Hkv,L", [("bf16", 8, 3), ("bf16", 1, 5), ("fp8_e4m3_block", 1, 3), ("int8_block", 2, 5),
                                      ("fp8_e4m3_block", 4, 5)])
def test_a_wait_that_runs_out_among_cut_requests(kv, Hkv, L, monkeypatch):
    # two and three row groups, requests that are cut and merged: the first unit, inside request 0, copies nothing;
    # the others are exact, and so is the next call
    monkeypatch.setenv("MQA_ENABLE_TEST_HOOKS", "1")
    import ctypes
    from mqa_decode_attention_paged_gb300 import _binding as binding
    P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    fn = binding.lib.mqa_test_gqa_window_withheld
    fn.restype = I
    fn.argtypes = [P, P, P, P, P, F, I, I, P, P, I, I, I, I, I, I, I, I, I, I, I, P, SZ, P, P, I]
    case = widen(Case([6000, 300, 40], 4 * Hkv, Hkv, 64, 16, kv, L=L, window=5000, sinks=4, seed=25, poison=False))
    q, cache, bt, sc, sl = case.dev()
    B, _, Hq, D = q.shape
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda")
    ws = torch.full((mqa.gqa_window_decode_workspace_bytes(B, L, Hq, Hkv, D, 3),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rc = fn(q.data_ptr(), cache.data_ptr(), None if sc is None else sc.data_ptr(), bt.data_ptr(), sl.data_ptr(),
            case.scale, 5000, 4, out.data_ptr(), lse.data_ptr(), B, L, Hq, Hkv, D, case.nb, 16, bt.shape[1], 16,
            binding._KV_NAMES[kv], 3, ws.data_ptr(), ws.numel(), status.data_ptr(),
            torch.cuda.current_stream().cuda_stream, 0)
    assert rc == binding.OK
    torch.cuda.synchronize()
    assert int(status.item()) == binding.ERR_DEVICE_TIMEOUT
    units = ws.cpu()[-8 * B:].view(torch.int32).view(B, 2)  # each request's first and last unit
    assert units[0, 0] == 0 and units[0, 1] > 0 and units[1, 0] > 0
    check(case, out.cpu().double(), lse.cpu().double(), rows=[1, 2])
    run_and_check(case, (3,))
