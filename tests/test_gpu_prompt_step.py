"""A run of the operators together, as a serving program would: prompts appended and attended, forked into several
samples, decoded with their own tokens, some of them ended, the pool compacted, decoded on.  Every attention is held
to the definition in 64 bits on the values that a plain model of the cache says are there."""
import pytest
import torch

import mqa_decode_attention_paged_gb300 as mqa
from attention_reference import NO_WINDOW, attention, judge

pytestmark = pytest.mark.gpu
I32 = torch.int32
HQ, HKV, D, PAGE, LAYERS = 8, 2, 128, 16, 2


def dev(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Program:
    """Two layers of caches, one block table; `values`: the tokens of each row and layer by the caches' own contents."""

    def __init__(self, kv, blocks=200):
        self.kv = kv
        shape = (blocks, 2, PAGE, HKV, D)
        if kv == "bf16":
            self.caches = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)]
            self.scales = [None] * LAYERS
        else:
            dtype = torch.int8 if kv == "int8_block" else torch.float8_e4m3fn
            self.caches = [torch.zeros(shape, dtype=torch.int8, device="cuda").view(dtype) for _ in range(LAYERS)]
            self.scales = [torch.zeros(blocks, 2, 1, HKV, device="cuda") for _ in range(LAYERS)]
        self.refs = torch.zeros(blocks, dtype=I32, device="cuda")
        angle = torch.arange(512.0)[:, None] * 10000.0 ** (-torch.arange(0, D, 2) / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).cuda()
        self.slopes = torch.exp2(-torch.arange(1, HQ + 1, device="cuda").float())
        self.generator = torch.Generator(device="cuda").manual_seed(5)

    def pools(self):
        return [t for t in self.caches + self.scales if t is not None]

    def token_values(self, layer, row, n):
        ids = self.table[row, :-(-n // PAGE)].long()
        x = self.caches[layer][ids].double()
        if self.scales[layer] is not None:
            x = x * self.scales[layer][ids].double()[..., None]
        return x[:, 0].reshape(-1, HKV, D)[:n], x[:, 1].reshape(-1, HKV, D)[:n]

    def grow(self, new):
        """Takes free pages for `new` tokens of each row, as the program's allocator would."""
        lens = self.lens.tolist()
        free = (self.refs == 0).nonzero()[:, 0].tolist()
        for r, k in enumerate(new):
            for j in range(-(-lens[r] // PAGE), -(-(lens[r] + k) // PAGE)):
                self.table[r, j] = f = free.pop(0)
                self.refs[f] = 1
        self.lens = self.lens + dev(new)

    def step(self, new, attend):
        """Appends `new` random tokens to each row, layer by layer, and attends."""
        self.grow(new)
        starts = [0]
        for k in new:
            starts.append(starts[-1] + k)
        T = starts[-1]
        status = dev([0])
        for layer in range(LAYERS):
            qkv = torch.randn(T, HQ + 2 * HKV, D, generator=self.generator, device="cuda").to(torch.bfloat16)
            q = mqa.gqa_rope_append(qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], self.cos_sin, self.caches[layer], self.table,
                                    self.lens, dev(starts), q=qkv[:, :HQ], kv_scales=self.scales[layer], device_status=status)
            attend(layer, q, starts, status)
        assert int(status) == 0

    def prompts(self, new, prefix):
        def attend(layer, q, starts, status):
            out, lse = mqa.gqa_prefill(q, self.caches[layer], self.table, self.lens, dev(starts), D ** -0.5, softcap=30.0,
                                       slopes=self.slopes, prefix_lens=dev(prefix), kv_scales=self.scales[layer], device_status=status)
            for r, n in enumerate(self.lens.tolist()):
                k = starts[r + 1] - starts[r]
                if k:
                    K, V = self.token_values(layer, r, n)
                    at = slice(starts[r], starts[r + 1])
                    judge(out[at], lse[at], attention(q[at], K, V, n - k, D ** -0.5, 30.0, self.slopes, NO_WINDOW, 0,
                                                      min(prefix[r], n)), f"layer {layer}, row {r}")
        self.step(new, attend)

    def decode(self, window=None):
        def attend(layer, q, starts, status):
            out, lse = mqa.gqa_score_decode(q, self.caches[layer], self.table, self.lens, D ** -0.5, softcap=30.0, slopes=self.slopes,
                                            window=window, kv_scales=self.scales[layer], device_status=status)
            # a prompt chunk of one token is a decode step
            out2, lse2 = mqa.gqa_prefill(q, self.caches[layer], self.table, self.lens, dev(starts), D ** -0.5, softcap=30.0,
                                         slopes=self.slopes, window=window, kv_scales=self.scales[layer])
            for r, n in enumerate(self.lens.tolist()):
                K, V = self.token_values(layer, r, n)
                ref = attention(q[r:r + 1], K, V, n - 1, D ** -0.5, 30.0, self.slopes, window or NO_WINDOW)
                judge(out[r:r + 1], lse[r:r + 1], ref, f"layer {layer}, row {r}")
                judge(out2[r:r + 1], lse2[r:r + 1], ref, f"layer {layer}, row {r}, as a prompt")
        self.step([1] * len(self.lens), attend)


@pytest.mark.parametrize("kv", ["bf16", "int8_block", "fp8_e4m3_block"])
def test_prompts_samples_and_compaction(kv):
    p = Program(kv)
    p.table = torch.full((3, 32), -1, dtype=I32, device="cuda")
    p.lens = dev([0, 0, 0])
    p.prompts([100, 37, 64], [20, 0, 64])       # the prompts, the last of them bidirectional throughout
    p.prompts([5, 0, 33], [20, 0, 0])           # a second chunk of two of them
    # samples: three of the first prompt, two of the second (its last page is full: none is copied), one of the third
    before = [p.token_values(1, r, n) for r, n in enumerate(p.lens.tolist())]
    parents = [0, 1, 0, 2, 0, 1]
    p.table, p.lens, p.refs = mqa.pages_fork(p.table, p.lens, dev(parents), p.refs, p.pools(), PAGE)
    for r, q in enumerate(parents):
        for a, b in zip(p.token_values(1, r, int(p.lens[r])), before[q]):
            assert torch.equal(a, b)
    for _ in range(3):
        p.decode()
    # two samples end, one is doubled; then the pool is packed
    p.table, p.lens, p.refs = mqa.pages_fork(p.table, p.lens, dev([2, -1, 4, 3, 3]), p.refs, p.pools(), PAGE)
    keep = dev([0, 2, 3, 4])
    p.table, p.lens = p.table[keep.long()].contiguous(), p.lens[keep.long()].contiguous()
    before = [p.token_values(0, r, n) for r, n in enumerate(p.lens.tolist())]
    p.table, p.refs, moved, live = mqa.pages_compact(p.table, p.lens, p.refs, p.pools(), PAGE)
    assert int(live) == int((p.refs > 0).sum()) and bool((p.refs[int(live):] == 0).all())
    held = torch.bincount(torch.cat([p.table[r, :-(-n // PAGE)] for r, n in enumerate(p.lens.tolist())]).long(), minlength=len(p.refs))
    assert torch.equal(held.int(), p.refs)
    for r, n in enumerate(p.lens.tolist()):
        for a, b in zip(p.token_values(0, r, n), before[r]):
            assert torch.equal(a, b)
    p.decode(window=40)
    p.prompts([9, 1, 0, 20], [0, 0, 0, 0])
