"""The paged append with rotation, the rotation of queries, the sparse decode
and the group attention over a shared context, run together by a LayerGroup.

Own parts are compared bit by bit with the same library call on rotated rows;
the joined outputs with the softmax over own part and shared entries in 64
bits. The tolerances are those of the group attention alone (its own test
module derives them); the own part enters it as the fp32 tensors that it reads."""
import math

import pytest
import torch

from test_gpu_group_attn import Case
from test_gpu_rope import freqs, lib, rotate      # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu

H, DIM, KD, PAGE = 16, 576, 64, 64
SCALE = 1.0 / math.sqrt(DIM)


class Batch:
    """B sequences and shared prompts in the caches of a group's Full layers, all from raw latents."""

    def __init__(self, lib, B, Sq, lens, prompts, tokens, modes, top_k, seed):
        from compressed_sparse_attention_quant_b200.group import LayerGroup, SharedContext
        self.lib, self.B, self.Sq, self.modes = lib, B, Sq, modes
        self.g = torch.Generator().manual_seed(seed)
        self.inv = freqs(32)
        self.rope, self.krope = lib.Rope(self.inv.cuda(), 512, True), lib.Rope(self.inv.cuda(), 0, True)
        W = max(-(-t // PAGE) for t in lens)
        P = max(max(-(-t // PAGE) for t in prompts), 1)
        pages = B * W + len(prompts) * P
        perm = torch.randperm(pages, generator=self.g).to(torch.int32)
        self.table, self.prompt_table = perm[:B * W].view(B, W), perm[B * W:].view(len(prompts), P)
        self.lens, self.prompts, self.tokens = lens, prompts, tokens
        self.group = LayerGroup(modes, B, Sq, W, pages, top_k, rope=self.rope, idx_rope=self.krope)
        for cache in self.group.caches.values():
            for table, at, n in [(self.table, b, t - Sq) for b, t in enumerate(lens)] + [
                    (self.prompt_table, i, t) for i, t in enumerate(prompts)]:
                if n == 0:
                    continue
                pos = torch.arange(n)
                lib.append_kv_rope(self.rand(n, DIM).cuda(), pos.int().cuda(), lib.slot_mapping(table, at, pos).cuda(),
                                   cache, self.rope, self.rand(n, KD).cuda(), self.krope)
        self.shared = SharedContext(self.prompt_table.cuda(), torch.tensor(prompts, dtype=torch.int32).cuda(), tokens)
        n = B * Sq
        self.pos = torch.cat([torch.arange(t - Sq, t) for t in lens]).int()
        slots = torch.cat([lib.slot_mapping(self.table, b, torch.arange(t - Sq, t)) for b, t in enumerate(lens)])
        L = len(modes)
        self.q = [self.rand(B, Sq, H, DIM) for _ in range(L)]
        self.swa = [self.rand(B, 127 + Sq, DIM).cuda() for _ in range(L)]
        self.q_idx = {i: torch.randint(0, 0x70, (B, Sq, lib.IDX_HEADS, KD), generator=self.g, dtype=torch.uint8).cuda()
                      for i in range(L) if modes[i] in ("F", "R")}
        self.w = {i: torch.rand(B, Sq, lib.IDX_HEADS, generator=self.g).cuda() for i in self.q_idx}
        self.raw = {i: (self.rand(n, DIM).cuda(), self.pos.cuda(), slots.cuda(), self.rand(n, KD).cuda())
                    for i in range(L) if modes[i] == "F"}
        self.q_dev = [t.cuda() for t in self.q]
        self.lens_dev = torch.tensor(lens, dtype=torch.int32).cuda()
        self.table_dev = self.table.cuda()

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g).to(torch.bfloat16)

    def args(self):
        return (self.table_dev, self.lens_dev, self.q_dev, self.swa, self.q_idx, self.w), dict(
            positions=self.pos.cuda(), raw_append=self.raw, shared=self.shared)

    def check(self):
        n, lib = self.B * self.Sq, self.lib
        assert lib.last_device_error() == 0
        for i, q in enumerate(self.q):
            cache = self.group.cache(i)
            rot = rotate(q.view(n, H, DIM), self.pos, self.inv, 512, True)
            o, lse = lib.sparse_attn_decode(rot.view(self.B, self.Sq, H, DIM).cuda(), cache, self.table_dev,
                                            self.lens_dev, self.group.index(i), self.swa[i], SCALE)
            assert torch.equal(o, self.group.out[i]) and torch.equal(lse, self.group.lse[i])
            c = Case.__new__(Case)
            c.lib, c.cache, c.lens, c.table, c.q = lib, cache, self.prompts, self.prompt_table, rot
            c.offs = self.shared.q_offsets.tolist()
            c.own = (o.cpu().view(n, H, DIM), lse.cpu().view(n, H))
            c.check(self.group.joined[i].view(n, H, DIM), self.group.joined_lse[i].view(n, H))


SHAPES = [
    (1, 1, [129], [65], [1], ("F",), 16),
    (3, 2, [200, 131, 640], [150, 0], [4, 2], ("F", "R", "U"), 64),
    (4, 4, [300, 900, 257, 512], [1, 640, 77], [9, 0, 7], ("F", "U", "F"), 200),
]


@pytest.mark.parametrize("B,Sq,lens,prompts,tokens,modes,k", SHAPES)
def test_step_with_raw_rows_and_shared_context(lib, B, Sq, lens, prompts, tokens, modes, k):
    b = Batch(lib, B, Sq, lens, prompts, tokens, modes, k, seed=B)
    args, kw = b.args()
    b.group.step(*args, **kw)
    b.check()


def test_captured_step_on_refreshed_inputs(lib):
    """The whole step as a CUDA graph: new queries, another prompt length and another split of pages between replays;
    the bits are those of an eager step."""
    from compressed_sparse_attention_quant_b200.group import StepGraph
    B, Sq, lens, prompts, tokens, modes, k = SHAPES[1]
    b = Batch(lib, B, Sq, lens, prompts, tokens, modes, k, seed=5)
    args, kw = b.args()
    graph = StepGraph(b.group, *args, **kw)
    for new_lens in ([150, 0], [20, 3]):
        b.q = [b.rand(B, Sq, H, DIM) for _ in modes]
        for d, v in zip(b.q_dev, b.q):
            d.copy_(v)
        b.prompts = new_lens
        b.shared.lens.copy_(torch.tensor(new_lens, dtype=torch.int32))
        for t in b.group.joined + b.group.joined_lse + b.group.out:
            t.fill_(7.0)
        graph.replay()
        b.check()
        got = [t.clone() for t in b.group.joined + b.group.joined_lse]
        b.group.step(*args, **kw)
        assert all(torch.equal(x, y) for x, y in zip(got, b.group.joined + b.group.joined_lse))
    del graph


@pytest.mark.parametrize("captured", [False, True])
def test_rotated_queries_reach_the_kernel_behind(lib, captured):
    """The sparse decode starts before its predecessor ends and must still see the queries that the predecessor
    rotates, however often the buffer changes hands."""
    n, k, turns = 64, 64, 40
    g = torch.Generator().manual_seed(30)
    cache = lib.PagedCache(n * 2)
    slots = torch.arange(n * 2 * PAGE, dtype=torch.int32).cuda()
    lib.quant_kv_fp4(torch.randn(n * 2 * PAGE, DIM, generator=g).to(torch.bfloat16).cuda(), slots, cache)
    table = torch.arange(n * 2, dtype=torch.int32).view(n, 2).cuda()
    lens = torch.full((n,), 2 * PAGE, dtype=torch.int32).cuda()
    idx = torch.arange(k, dtype=torch.int32).view(1, 1, k).expand(n, 1, k).contiguous().cuda()
    rope = lib.Rope(freqs(32).cuda(), 512, True)
    pos = torch.arange(n, dtype=torch.int32).cuda()
    qs = [torch.randn(n, H, DIM, generator=g).to(torch.bfloat16).cuda() for _ in range(turns)]
    out = [torch.zeros(n, 1, H, DIM).cuda() for _ in range(turns)]
    lse = torch.empty(n, 1, H).cuda()
    ws = lib.workspace(lib.sparse_attn_workspace_bytes(n, 1, k))
    ref = []
    for q in qs:
        rot = lib.rope_rows(q, pos, rope)
        torch.cuda.synchronize()
        ref.append(lib.sparse_attn_decode(rot.view(n, 1, H, DIM), cache, table, lens, idx, None, SCALE)[0])
    buf = torch.empty(n, H, DIM, dtype=torch.bfloat16).cuda()

    def run():
        for q, o in zip(qs, out):
            lib.rope_rows(q, pos, rope, out=buf)
            lib.sparse_attn_decode(buf.view(n, 1, H, DIM), cache, table, lens, idx, None, SCALE, out=o, lse=lse, ws=ws)

    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        run = graph.replay
    for _ in range(10):
        for o in out:
            o.zero_()
        run()
        assert all(torch.equal(o, r) for o, r in zip(out, ref))
    assert lib.last_device_error() == 0
