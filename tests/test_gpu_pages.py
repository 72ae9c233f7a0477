"""pages_fork and pages_compact against plain loops over rows and pages."""
import pytest
import torch

import mqa_decode_attention_paged_gb300 as mqa

pytestmark = pytest.mark.gpu
I32 = torch.int32


def caches_of(nb, page, kinds, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for k in kinds:
        if k == "bf16":
            out.append(torch.randn(nb, 2, page, 2, 64, generator=g, device="cuda").to(torch.bfloat16))
        elif k == "mla":
            out.append(torch.randn(nb, page, 576, generator=g, device="cuda").to(torch.bfloat16))
        elif k == "pth":
            out.append(torch.randint(0, 256, (nb, 2, page, 3, 68), generator=g, device="cuda", dtype=torch.uint8))
        elif k == "scale":
            out.append(torch.rand(nb, 2, 1, 1, generator=g, device="cuda"))
        elif k == "wide":
            out.append(torch.randn(nb, 5003, 3, generator=g, device="cuda"))
    return out


def state(lens, page, spare, share=(), seed=0, extra=2):
    """Table, lengths and counts of rows; share: (row, other, pages) shares the first pages of another row."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // page) for n in lens]
    nb = max(1, sum(pages) + spare)
    perm = torch.randperm(nb, generator=g).tolist()
    table = torch.full((len(lens), max(pages + [1]) + extra), 12345678, dtype=I32)  # what is behind a row is not read
    refs, at = torch.zeros(nb, dtype=I32), 0
    for r, k in enumerate(pages):
        table[r, :k] = torch.tensor(perm[at:at + k], dtype=I32)
        at += k
    for r, o, k in share:
        table[r, :k] = table[o, :k]
    for r, k in enumerate(pages):
        for i in table[r, :k].tolist():
            refs[i] += 1
    return table, torch.tensor(lens, dtype=I32), refs


def plain_fork(table, lens, refs, parents, page, caches):
    W = table.shape[1]
    refs, used = refs.tolist(), [-(-n // page) for n in lens.tolist()]
    for r, k in enumerate(used):
        for i in table[r, :k].tolist():
            refs[i] -= 1
    rows, waiting = [], []
    for r, p in enumerate(parents):
        row = [] if p < 0 else table[p, :used[p]].tolist()
        if p >= 0 and lens[p] % page and p in parents[:r]:
            waiting.append((r, row[-1]))
            for i in row[:-1]:
                refs[i] += 1
        else:
            for i in row:
                refs[i] += 1
        rows.append(row)
    free, short = [i for i, c in enumerate(refs) if c == 0], False
    for r, src in waiting:
        if not free:
            rows[r][-1], short = -1, True
            continue
        f = free.pop(0)
        rows[r][-1] = f
        refs[f] = 1
        for x in caches:
            x[f] = x[src]
    out = torch.full((len(parents), W), -1, dtype=I32)
    for r, row in enumerate(rows):
        out[r, :len(row)] = torch.tensor(row, dtype=I32)
    return out, torch.tensor([0 if p < 0 else int(lens[p]) for p in parents], dtype=I32), torch.tensor(refs, dtype=I32), short


def check_fork(lens, parents, page=16, spare=20, share=(), kinds=("bf16",), seed=0, in_place=False):
    table, n, refs = state(lens, page, spare, share, seed)
    caches = caches_of(len(refs), page, kinds)
    want_caches = [x.clone() for x in caches]
    want = plain_fork(table, n, refs, parents, page, want_caches)
    status = torch.zeros(1, dtype=I32, device="cuda")
    d_refs = refs.cuda()
    got = mqa.pages_fork(table.cuda(), n.cuda(), torch.tensor(parents, dtype=I32, device="cuda"), d_refs, caches, page,
                         new_refs=d_refs if in_place else None, device_status=status)
    torch.cuda.synchronize()
    for a, b, name in zip(got, want, ("table", "lens", "refs")):
        assert torch.equal(a.cpu(), b), name
    for a, b in zip(caches, want_caches):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert int(status) == (5 if want[3] else 0)


@pytest.mark.parametrize("kinds", [("bf16",), ("bf16", "scale", "mla", "pth"), ("scale",), (), ("wide", "bf16")])
def test_fork_formats(kinds):
    check_fork([40, 17, 100], [0, 0, 1, 2, 2, 2, 0], kinds=kinds)


@pytest.mark.parametrize("count", [16, 17, 61, 256])
def test_caches_of_many_layers(count):
    kinds = (("bf16", "scale", "mla", "pth") * 64)[:count]
    check_fork([40, 17, 100], [0, 0, 1, 2, 2, 2, 0], kinds=kinds)
    check_compact([40, 17, 100], kinds=kinds)


@pytest.mark.parametrize("lens,parents", [
    ([5], [0]), ([5], [0, 0, 0, 0]), ([16], [0, 0]), ([0], [0, 0]), ([5], [-1]), ([1, 2, 3], [-1, 2, -1, 2, 0]),
    ([33, 47], [1, 0]), ([33, 47], [1, 1]), ([15, 16, 17], [2, 2, 1, 1, 0, 0, -1]), ([300], [0] * 50)])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork_parents(lens, parents, in_place):
    check_fork(lens, parents, spare=60, in_place=in_place)


def test_fork_of_shared_prefixes():
    # beams that share full pages; freed beams' pages are taken in the same call
    check_fork([70, 70, 70, 70], [1, 1, 1, 3], share=((1, 0, 3), (2, 0, 3), (3, 0, 3)), spare=0)
    check_fork([70, 70, 70, 70], [-1, -1, -1, -1], share=((1, 0, 3), (2, 0, 4), (3, 0, 3)), spare=0)


def test_fork_without_enough_pages():
    check_fork([5, 20], [0, 0, 0, 1, 1, 1], spare=2)
    check_fork([5, 20], [0, 0, 0, 1, 1, 1], spare=0)


@pytest.mark.parametrize("seed", range(4))
def test_fork_of_large_batches(seed):
    g = torch.Generator().manual_seed(seed)
    R, N, page = [(300, 1500, 32), (2000, 2000, 16), (1, 3000, 16), (8192, 8192, 16)][seed]
    lens = torch.randint(0, 200 if R < 5000 else 40, (R,), generator=g).tolist()
    parents = torch.randint(-1, R, (N,), generator=g).tolist()
    check_fork(lens, parents, page=page, spare=3000, seed=seed, kinds=("scale", "pth") if R > 1000 else ("bf16", "scale"))


def test_fork_reports_bad_rows():
    table, n, refs = state([40, 17], 16, 5)
    caches = caches_of(len(refs), 16, ("bf16",))
    for what in range(4):
        t, m, p = table.clone(), n.clone(), [0, 1, 1]
        if what == 0:
            t[1, 1] = len(refs)
        elif what == 1:
            m[1] = 10 ** 6
            t[1] = table[1, 0]
        elif what == 2:
            m[1] = -3
        else:
            p = [0, 1, 7]
        status = torch.zeros(1, dtype=I32, device="cuda")
        before = caches[0].clone()
        nt, nl, nr = mqa.pages_fork(t.cuda(), m.cuda(), torch.tensor(p, dtype=I32, device="cuda"), refs.cuda(), caches, 16,
                                    device_status=status)
        torch.cuda.synchronize()
        assert int(status) == 5
        assert torch.equal(nt[0, :3].cpu(), table[0, :3]) and int(nl[0]) == 40
        if what == 0:  # the entry is kept, nothing is copied
            assert nt[1, 1] == len(refs) and nt[2, 1] == len(refs) and torch.equal(before, caches[0])
        if what == 2:
            assert int(nl[1]) == 0 and bool((nt[1] == -1).all())
        if what == 3:
            assert int(nl[2]) == 0 and bool((nt[2] == -1).all())


def check_compact(lens, page=16, spare=30, share=(), kinds=("bf16",), seed=0, held=(), in_place=False):
    table, n, refs = state(lens, page, spare, share, seed)
    for i in held:  # pages that something else holds
        free = (refs == 0).nonzero()[:, 0]
        refs[free[i]] = 3
    caches = caches_of(len(refs), page, kinds)
    L = int((refs > 0).sum())
    src = [i for i in range(L, len(refs)) if refs[i] > 0]
    dst = [i for i in range(L) if refs[i] <= 0]
    moved = torch.where(refs > 0, torch.arange(len(refs), dtype=I32), -1)
    moved[src] = torch.tensor(dst, dtype=I32)
    r2, t2 = refs.clone(), table.clone()
    r2[dst], r2[src] = refs[src], 0
    for b, m in enumerate(lens):
        k = -(-m // page)
        t2[b, :k] = moved[table[b, :k].long()]
    want = [x.clone() for x in caches]
    for x in want:
        x[dst] = x[src]
    status = torch.zeros(1, dtype=I32, device="cuda")
    dt, dr = table.cuda(), refs.cuda()
    got = mqa.pages_compact(dt, n.cuda(), dr, caches, page, device_status=status, new_table=dt if in_place else None,
                            new_refs=dr if in_place else None)
    torch.cuda.synchronize()
    for a, b, name in zip(got, (t2, r2, moved, torch.tensor([L], dtype=I32)), ("table", "refs", "moved", "live")):
        assert torch.equal(a.cpu(), b), name
    for a, b in zip(caches, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert int(status) == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kinds", [("bf16",), ("bf16", "scale", "mla", "pth"), (), ("wide",)])
def test_compact_formats(kinds, in_place):
    check_compact([40, 0, 17, 100], kinds=kinds, share=((3, 0, 2),), held=(1, 5), in_place=in_place)


@pytest.mark.parametrize("lens,spare", [([0], 0), ([0], 50), ([16], 0), ([1], 1), ([500], 0), ([5] * 300, 1),
                                        ([37] * 200, 5000), ([3] * 8000, 3000)])
def test_compact_sizes(lens, spare):
    check_compact(lens, spare=spare, kinds=("scale",) if len(lens) > 1000 else ("bf16",))


def test_compact_reports_entries_that_are_no_pages():
    table, n, refs = state([40, 17], 16, 5)
    table[0, 1], table[1, 0] = len(refs) + 7, int((refs == 0).nonzero()[0])
    status = torch.zeros(1, dtype=I32, device="cuda")
    t2 = mqa.pages_compact(table.cuda(), n.cuda(), refs.cuda(), [], 16, device_status=status)[0]
    assert int(status) == 5 and t2[0, 1] == table[0, 1] and t2[1, 0] == table[1, 0]


def test_captured_and_replayed():
    table, n, refs = (x.cuda() for x in state([40, 17, 100], 16, 20))
    caches = caches_of(len(refs), 16, ("bf16", "scale"))
    parents = torch.tensor([0, 0, 2, 2], dtype=I32, device="cuda")
    want = mqa.pages_fork(table, n, parents, refs, caches, 16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = mqa.pages_fork(table, n, parents, refs, caches, 16)
        more = mqa.pages_compact(got[0], got[1], got[2], caches, 16)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert int(more[3]) == int((want[2] > 0).sum())


def test_pages_far_into_a_large_cache():
    """Copies between pages on both sides of 2^32 bytes of their cache."""
    nb, words = 140000, 32768 // 4
    cache = torch.empty(nb, words, dtype=I32, device="cuda")
    row = torch.arange(words, dtype=I32, device="cuda")
    refs = torch.ones(nb, dtype=I32, device="cuda")
    refs[[5, nb - 2]] = 0
    cache[[nb - 1, 7]] = torch.stack([row + 1, row + 2])
    table = torch.tensor([[nb - 1], [7]], dtype=I32, device="cuda")
    got, lens, after = mqa.pages_fork(table, torch.tensor([3, 3], dtype=I32, device="cuda"),
                                      torch.tensor([0, 0, 1, 1], dtype=I32, device="cuda"), refs, [cache], 16)
    assert got.tolist() == [[nb - 1], [5], [7], [nb - 2]] and lens.tolist() == [3] * 4
    assert torch.equal(cache[5], row + 1) and torch.equal(cache[nb - 2], row + 2) and int(after.sum()) == nb
    after[:nb - 4] = 0  # live: the last four
    got, after, moved, live = mqa.pages_compact(got[[0, 3]].contiguous(), lens[:2].contiguous(), after, [cache], 16)
    assert int(live) == 4 and got.tolist() == [[3], [2]]
    assert torch.equal(cache[3], row + 1) and torch.equal(cache[2], row + 2)


@pytest.mark.parametrize("bad", [-1, -7, "nb", 2 ** 31 - 1])
@pytest.mark.parametrize("lens,at", [([40, 17], (1, 0)), ([40, 17], (1, 1)), ([40, 32], (1, 1)), ([40, 17], (0, 2))])
@pytest.mark.parametrize("parents", [[0, 1], [1, 0], [0, 1, -1], [0, 1, 0], [0, 1, 1]])
def test_fork_reports_bad_ids_whatever_the_number_of_children(parents, lens, at, bad):
    table, n, refs = state(lens, 16, 6)
    held = table.clone()
    bad = len(refs) if bad == "nb" else bad
    table[at] = bad
    cache = caches_of(len(refs), 16, ("scale",))[0]
    before, status = cache.clone(), torch.zeros(1, dtype=I32, device="cuda")
    nt, nl, nr = mqa.pages_fork(table.cuda(), n.cuda(), torch.tensor(parents, dtype=I32, device="cuda"), refs.cuda(), [cache], 16,
                                device_status=status)
    assert int(status) == 5
    count = [parents.count(r) for r in range(2)]
    want = refs.clone()
    for r in range(2):
        for j in range(-(-lens[r] // 16)):
            tail = lens[r] % 16 and j == lens[r] // 16
            if (r, j) != at:
                want[held[r, j]] += (count[r] > 0) - 1 if tail else count[r] - 1
    copied = [(parents.index(p), r) for r, p in enumerate(parents) if p >= 0 and p in parents[:r] and lens[p] % 16 and at != (p, lens[p] // 16)]
    free = [i for i, c in enumerate(want.tolist()) if c == 0]
    for (first, r), f in zip(copied, free):
        want[f] = 1
        before[f] = before[int(nt[first, lens[parents[r]] // 16])]
        assert int(nt[r, lens[parents[r]] // 16]) == f
    assert torch.equal(nr.cpu(), want) and torch.equal(cache, before)
    for r, p in enumerate(parents):
        if p >= 0 and r not in [x for _, x in copied]:
            assert torch.equal(nt[r, :-(-lens[p] // 16)].cpu(), table[p, :-(-lens[p] // 16)])


@pytest.mark.parametrize("given", [False, True])
def test_fork_without_new_rows(given):
    """Every row ends: the counts fall, pages that something else holds stay."""
    table, n, refs = state([40, 16, 0, 17], 16, 5, share=((3, 0, 1),))
    refs[table[0, 1]] += 1
    want = refs.clone()
    for r, k in enumerate((3, 1, 0, 2)):
        for i in table[r, :k].tolist():
            want[i] -= 1
    cache = caches_of(len(refs), 16, ("scale",))[0]
    before, status = cache.clone(), torch.zeros(1, dtype=I32, device="cuda")
    none, d_refs, W = torch.zeros(0, dtype=I32, device="cuda"), refs.cuda(), table.shape[1]
    kw = dict(new_table=torch.zeros(0, W, dtype=I32, device="cuda"), new_lens=none.clone(), new_refs=d_refs,
              workspace=torch.zeros(mqa.pages_fork_workspace_bytes(0), device="cuda")) if given else {}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    nt, nl, nr = mqa.pages_fork(table.cuda(), n.cuda(), none, d_refs, [cache], 16, device_status=status, stream=stream, **kw)
    stream.synchronize()
    assert nt.shape == (0, W) and nl.shape == (0,) and int(status) == 0
    assert torch.equal(nr.cpu(), want) and torch.equal(cache, before) and torch.equal(d_refs.cpu(), want if given else refs)


def test_page_sizes_beyond_a_c_int_are_taken_at_their_value():
    table, n, refs = (x.cuda() for x in state([40, 17], 16, 5))
    parents = torch.tensor([0, 1], dtype=I32, device="cuda")
    for page in (2 ** 32 + 16, -2 ** 32 + 16, 2 ** 33):
        with pytest.raises(mqa.MqaError):
            mqa.pages_fork(table, n, parents, refs, [], page)
        with pytest.raises(mqa.MqaError):
            mqa.pages_compact(table, n, refs, [], page)


@pytest.mark.parametrize("parents", [[0], [0, 0, 0], [-1], [1, 0, 1]])
def test_fork_of_a_partly_filled_page_that_something_else_holds(parents):
    """The page stays with the first child, further ones get copies; the other holder keeps its count."""
    table, n, refs = state([40, 21], 16, 6)
    tail = int(table[0, 2])
    refs[tail] += 2
    caches = caches_of(len(refs), 16, ("bf16",))
    want_caches = [x.clone() for x in caches]
    want = plain_fork(table, n, refs, parents, 16, want_caches)
    got = mqa.pages_fork(table.cuda(), n.cuda(), torch.tensor(parents, dtype=I32, device="cuda"), refs.cuda(), caches, 16)
    for a, b in zip(got, want[:3]):
        assert torch.equal(a.cpu(), b)
    assert torch.equal(caches[0], want_caches[0]) and int(got[2][tail]) == 2 + (0 in parents)
    if 0 in parents:
        assert int(got[0][parents.index(0), 2]) == tail
