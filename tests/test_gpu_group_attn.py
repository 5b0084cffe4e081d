"""K12 / K13: attention of groups of query tokens over shared FP4 entries,
against the formula in 64 bits.

Tolerances, per output element o with A = sum_t w_t |v_t| (the same softmax
weights w over the magnitudes): the result is rounded to bf16 (2^-8 |o|, half
a step of the type), each probability to f16 (2^-11 of its weight: 2^-11 A),
and a score s carries an error of at most d = 576 * 2^-24 * scale * sum |q k|
(576 fp32 additions) plus 2^-21 |s| (the exponent's fp32 argument), which moves
every weight by at most 2 d relatively (2 d A). f16 queries add 2^-25 of a
row's largest magnitude per channel, covered by d. Below 2^-14 f16 has a fixed
step of 2^-24: a probability exp(s - max) below that errs by 2^-25 absolutely
instead (the sum they are divided by is at least 1, the largest entry's own
probability): 2^-25 / sum times the |v| of those entries. lse moves by d, by the
exponentials (2^-21 of each) and by the fp32 sum of T of them: positive terms,
so each addition errs by at most 2^-24 of the final sum, and a term passes
through at most 64 additions inside a block of 64 entries and one for each of
the T / 64 blocks: (64 + T / 64) 2^-24. lse itself is fp32 (2^-22 |lse| with
the change of base)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

H, DIM, PAGE = 16, 576, 64
SCALE = 1.0 / math.sqrt(DIM)


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from compressed_sparse_attention_quant_b200 import lib as L
    return L


class Case:
    """A cache of quantised rows in shuffled pages and a batch of query tokens in groups."""

    def __init__(self, lib, tokens, lens, seed=0, before=0, after=0, k_gain=1.0, q_gain=1.0, spare_pages=3,
                 poison=True):
        g = torch.Generator().manual_seed(seed)
        self.lib, self.tokens, self.lens = lib, tokens, lens
        self.N = before + sum(tokens) + after
        offs = [before]
        for t in tokens:
            offs.append(offs[-1] + t)
        self.offs = offs
        per = [-(-t // PAGE) for t in lens]
        self.max_pages = max(max(per), 1)
        self.pages = sum(per) + spare_pages
        perm = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), self.max_pages), -5, dtype=torch.int32)
        at = 0
        self.cache = lib.PagedCache(self.pages)
        if poison:                                       # whatever is not written: NaN scales, the largest codes
            self.cache.kv_fp4.fill_(0xFF)
            self.cache.kv_scale.fill_(0x7F)
        self.rows = []
        for i, (p, t) in enumerate(zip(per, lens)):
            self.table[i, :p] = perm[at:at + p]
            at += p
            x = (torch.randn(t, DIM, generator=g) * k_gain).to(torch.bfloat16)
            pos = torch.arange(t)
            if t:
                lib.quant_kv_fp4(x.cuda(), lib.slot_mapping(self.table, i, pos).cuda(), self.cache)
        assert lib.last_device_error() == 0
        self.q = (torch.randn(self.N, H, DIM, generator=g) * q_gain).to(torch.bfloat16)
        self.own = None

    def with_own(self, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.own = (torch.randn(self.N, H, DIM, generator=g), torch.randn(self.N, H, generator=g) + 5.0)
        return self

    def call(self, out=None, lse=None, scale=SCALE, ws=None, q=None):
        own = (None, None) if self.own is None else tuple(t.cuda() for t in self.own)
        return self.lib.group_attn((self.q if q is None else q).cuda(), self.cache, self.table.cuda(),
                                   torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                                   torch.tensor(self.offs, dtype=torch.int32, device="cuda"), scale, o_own=own[0],
                                   lse_own=own[1], out=out, lse=lse, ws=ws)

    def keys(self, g, drop=()):
        """Dequantised entries of group g in 64 bits (without those of the dropped pages)."""
        lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
        kv, sc = self.cache.kv_fp4.cpu(), self.cache.kv_scale.cpu().view(torch.float8_e4m3fn)
        parts = [torch.zeros(0, DIM, dtype=torch.float64)]
        for p in range(-(-self.lens[g] // PAGE)):
            if p in drop:
                continue
            n = min(PAGE, self.lens[g] - p * PAGE)
            page = int(self.table[g, p])
            c = torch.stack((kv[page, :n] & 15, kv[page, :n] >> 4), -1).flatten(-2).long()
            parts.append((lut[c].view(n, 36, 16) * sc[page, :n].double()[..., None]).view(n, DIM))
        return torch.cat(parts)

    def check(self, out, lse, scale=SCALE, drop=(), rows=None, q=None):
        out, lse = out.cpu().double(), lse.cpu().double()
        q = (self.q if q is None else q).double()
        for g in range(len(self.lens)):
            a, b = self.offs[g], self.offs[g + 1]
            if a == b:
                continue
            k = self.keys(g, drop)
            s = torch.einsum("nhc,tc->nht", q[a:b], k) * scale
            mag = torch.einsum("nhc,tc->nht", q[a:b].abs(), k.abs()) * abs(scale)
            d = (576 * 2.0 ** -24 * mag + 2.0 ** -21 * s.abs())
            d = d.amax(-1) if s.shape[-1] else torch.zeros(s.shape[:2], dtype=torch.float64)
            v = k
            low = torch.zeros(1, dtype=torch.float64)
            if s.shape[-1]:
                e = torch.exp(s - s.amax(-1, keepdim=True))
                low = torch.einsum("nht,tc->nhc", (e < 2.0 ** -14).double(), v.abs()) / e.sum(-1, keepdim=True)
            if self.own is not None:
                s = torch.cat([s, self.own[1][a:b].double()[..., None]], -1)
            m = s.amax(-1, keepdim=True) if s.shape[-1] else torch.full((b - a, H, 1), -math.inf)
            m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
            p = torch.exp(s - m)
            l = p.sum(-1, keepdim=True)
            w = torch.where(l > 0, p / l.clamp(min=1e-300), torch.zeros_like(p))
            T = len(v)
            o = torch.einsum("nht,tc->nhc", w[..., :T], v)
            A = torch.einsum("nht,tc->nhc", w[..., :T], v.abs())
            if self.own is not None:
                o = o + w[..., T:] * self.own[0][a:b].double()
                A = A + w[..., T:] * self.own[0][a:b].double().abs()
            L = torch.where(l[..., 0] > 0, m[..., 0] + torch.log(l[..., 0].clamp(min=1e-300)), -math.inf)
            tol = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * d[..., None]) * A + 2.0 ** -25 * low + 1e-30
            err = (out[a:b] - o).abs()
            sel = slice(None) if rows is None else rows
            assert bool((err <= tol)[sel].all()), f"group {g}: off by {float((err / tol)[sel].max()):.2f} tolerances"
            dead = torch.isinf(L)
            assert torch.equal(torch.isinf(lse[a:b])[sel], dead[sel])
            dl = torch.where(dead, torch.zeros_like(L), (lse[a:b] - L).abs())
            tl = d + 2.0 ** -21 + (64 + T / 64) * 2.0 ** -24 + 2.0 ** -22 * torch.where(dead, torch.zeros_like(L), L).abs()
            assert bool((dl <= tl)[sel].all()), f"group {g}: lse off by {float((dl / tl)[sel].max()):.2f} tolerances"


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("tokens,lens", [
    ([1], [1]), ([1], [64]), ([1], [65]), ([3], [63]), ([8], [128]), ([9], [1000]), ([20], [4097]),
    ([1, 0, 9, 17, 3], [0, 1, 64, 700, 129]), ([0, 2, 0], [70, 0, 10]), ([1] * 40, [17 * (i % 7) + i for i in range(40)]),
    ([64], [20000]), ([5, 30], [9000, 300])])
def test_against_64_bits(lib, tokens, lens, own):
    c = Case(lib, tokens, lens, seed=len(tokens) + lens[0])
    if own:
        c.with_own()
    out, lse = c.call()
    assert lib.last_device_error() == 0
    c.check(out, lse)


def test_tokens_of_no_group_keep_their_rows(lib):
    c = Case(lib, [3, 9], [100, 200], before=5, after=11).with_own()
    out = torch.full((c.N, H, DIM), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.N, H), -2.0, device="cuda")
    c.call(out, lse)
    assert lib.last_device_error() == 0
    c.check(out, lse)
    for part in (slice(0, 5), slice(c.N - 11, c.N)):
        assert (out[part] == 3.0).all() and (lse[part] == -2.0).all()


def test_own_part_without_keys(lib):
    """lse_own = -inf takes no part (whatever o_own holds); no entries and no own key give zeros."""
    c = Case(lib, [4, 3], [150, 0]).with_own()
    c.own[1][:2] = -math.inf
    c.own[1][4:6, 3] = -math.inf
    c.check(*c.call())
    c.own[0][:2] = math.nan
    out, lse = c.call()
    assert torch.isfinite(out.float()).all()
    ref = Case(lib, [4, 3], [150, 0])
    ref_out, ref_lse = ref.call()
    assert torch.equal(out[:2], ref_out[:2]) and torch.equal(lse[:2], ref_lse[:2])
    assert (out[4:6, 3] == 0).all() and torch.isinf(lse[4:6, 3]).all()


@pytest.mark.parametrize("scale,q_gain", [(3.0, 1.0), (-0.7, 1.0), (0.0, 1.0), (SCALE, 1e-6), (1e-6, 1e5), (SCALE, 0.0)])
def test_scales_and_magnitudes(lib, scale, q_gain):
    """Sharp softmaxes whose maximum rises from block to block, reversed and flat ones, tiny and huge queries."""
    c = Case(lib, [11], [1500], seed=3, q_gain=q_gain)
    c.check(*c.call(scale=scale), scale=scale)


def test_rising_maximum(lib):
    """Every block of entries beats the one before by more than the running reference lets pass."""
    c = Case(lib, [10], [64 * 24], seed=4)
    c.q = c.q.abs()
    for p in range(24):
        page = int(c.table[0, p])
        x = torch.full((PAGE, DIM), (p + 1) * 0.25, dtype=torch.bfloat16)
        lib.quant_kv_fp4(x.cuda(), (page * PAGE + torch.arange(PAGE)).to(torch.int32).cuda(), c.cache)
    c.check(*c.call(scale=0.3), scale=0.3)


def test_extreme_scales_of_entries(lib):
    """Entries under the smallest and the largest block scales."""
    for gain in (2.0 ** -8, 400.0):
        c = Case(lib, [9], [300], seed=6, k_gain=gain)
        c.check(*c.call(scale=SCALE / gain), scale=SCALE / gain)


def test_a_row_with_nan_keeps_to_itself(lib):
    c = Case(lib, [9], [700], seed=7)
    ref, ref_lse = c.call()
    q = c.q.clone()
    q[2, 5, 100] = math.nan
    q[8, 0, 0] = math.inf
    out, lse = c.call(q=q)
    bad = torch.zeros(9, H, dtype=torch.bool)
    bad[2, 5] = bad[8, 0] = True
    assert torch.equal(out.cpu()[~bad], ref.cpu()[~bad]) and torch.equal(lse.cpu()[~bad], ref_lse.cpu()[~bad])
    assert torch.isnan(out.cpu()[2, 5].float()).all()


@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_bad_page_is_left_out(lib, bad):
    c = Case(lib, [10], [400], seed=8)
    c.table[0, 2] = bad
    out, lse = c.call()
    assert lib.status_string(lib.last_device_error()) == "CSA2_ERR_DEVICE_BOUNDS"
    c.check(out, lse, drop=(2,))


def test_bad_lengths_and_offsets(lib):
    c = Case(lib, [4, 5, 6], [100, 200, 300], seed=9)
    out = torch.full((c.N, H, DIM), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.N, H), -2.0, device="cuda")
    lens = c.lens
    for wrong in (-1, c.max_pages * PAGE + 1):
        c.lens = [100, wrong, 300]
        c.call(out, lse)
        assert lib.status_string(lib.last_device_error()) == "CSA2_ERR_DEVICE_BOUNDS"
        c.lens = [100, 0, 300]                            # counts as empty
        c.check(out, lse)
        assert (out[4:9] == 0).all()
    c.lens = lens
    offs = c.offs
    for wrong in ([0, -4, 9, 15], [0, 20, 9, 15], [7, 4, 9, 15]):
        out.fill_(3.0)
        c.offs = wrong
        c.call(out, lse)
        assert lib.status_string(lib.last_device_error()) == "CSA2_ERR_DEVICE_BOUNDS"
        c.offs = [9, 9, 9, 15]                            # the last group is whole
        c.check(out, lse)
    c.offs = offs


def test_bounds_that_go_back_and_forth_stay_inside(lib):
    """Offsets 0, N, 0, N, ...: half of the groups are refused, the other half claim the same tokens; nothing is
    written past the workspace and the rows are those of one such group."""
    c = Case(lib, [16], [128], seed=10)
    G = 64
    c.table = c.table.expand(G, -1).contiguous()
    c.lens = [128] * G
    c.offs = [0 if i % 2 == 0 else 16 for i in range(G + 1)]
    need = lib.group_attn_workspace_bytes(c.N, G)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros(c.N, H, DIM, dtype=torch.bfloat16).cuda(), torch.zeros(c.N, H).cuda()
    own = lib.group_attn(c.q.cuda(), c.cache, c.table.cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda(),
                         torch.tensor(c.offs, dtype=torch.int32).cuda(), SCALE, out=out, lse=lse, ws=ws[:need])
    assert lib.status_string(lib.last_device_error()) == "CSA2_ERR_DEVICE_BOUNDS"
    assert own[0] is out and (ws[need:] == 0x5A).all()
    c.table, c.lens, c.offs = c.table[:1], [128], [0, 16]
    c.check(out, lse)


def test_same_bits_again_and_on_two_streams(lib):
    """Two calls at once with workspaces of their own, and the same call again, give the same bits."""
    c = Case(lib, [30, 5], [3000, 900], seed=11).with_own()
    ref, ref_lse = c.call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([c.call() for _ in range(3)])
    torch.cuda.synchronize()
    for per in got:
        for out, lse in per:
            assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_captured_and_replayed(lib):
    """One graph serves other lengths, offsets, pages and queries of the same shapes."""
    c = Case(lib, [30, 5], [3000, 900], seed=12).with_own()
    q, table = c.q.cuda(), c.table.cuda()
    lens, offs = torch.tensor(c.lens, dtype=torch.int32).cuda(), torch.tensor(c.offs, dtype=torch.int32).cuda()
    own = [t.cuda() for t in c.own]
    ws = lib.workspace(lib.group_attn_workspace_bytes(c.N, 2))
    out, lse = torch.empty(c.N, H, DIM, dtype=torch.bfloat16).cuda(), torch.empty(c.N, H).cuda()

    def call():
        lib.group_attn(q, c.cache, table, lens, offs, SCALE, *own, out=out, lse=lse, ws=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new_lens, new_offs in (([3000, 900], [0, 30, 35]), ([64, 777], [0, 1, 35]), ([1, 0], [0, 34, 35])):
        c.lens, c.offs = new_lens, new_offs
        lens.copy_(torch.tensor(new_lens, dtype=torch.int32))
        offs.copy_(torch.tensor(new_offs, dtype=torch.int32))
        c.q = torch.randn(c.N, H, DIM, generator=torch.Generator().manual_seed(new_lens[0])).to(torch.bfloat16)
        q.copy_(c.q)
        graph.replay()
        assert lib.last_device_error() == 0
        c.check(out, lse)


def test_agrees_with_the_sparse_decode(lib):
    """A shared prefix as one group joined with each sequence's own entries and window equals one sparse decode
    over both (every prefix entry selected)."""
    B, P = 6, 256
    g = torch.Generator().manual_seed(13)
    own_len = 128
    pages = P // PAGE + B * (own_len // PAGE)
    cache = lib.PagedCache(pages)
    table = torch.zeros(B, (P + own_len) // PAGE, dtype=torch.int32)
    table[:, :P // PAGE] = torch.arange(P // PAGE)
    for b in range(B):
        table[b, P // PAGE:] = P // PAGE + b * (own_len // PAGE) + torch.arange(own_len // PAGE)
    n = pages * PAGE
    lib.quant_kv_fp4(torch.randn(n, DIM, generator=g).to(torch.bfloat16).cuda(),
                     torch.arange(n, dtype=torch.int32).cuda(), cache)
    q = torch.randn(B, 1, H, DIM, generator=g).to(torch.bfloat16).cuda()
    swa = torch.randn(B, 128, DIM, generator=g).to(torch.bfloat16).cuda()
    full = torch.full((B,), P + own_len, dtype=torch.int32).cuda()
    every = torch.arange(P + own_len, dtype=torch.int32).view(1, 1, -1).expand(B, 1, -1).contiguous().cuda()
    ref, ref_lse = lib.sparse_attn_decode(q, cache, table.cuda(), full, every, swa, SCALE)
    tail = torch.arange(own_len, dtype=torch.int32).view(1, 1, -1).expand(B, 1, -1).contiguous().cuda()
    o_own, lse_own = lib.sparse_attn_decode(q, cache, table[:, P // PAGE:].contiguous().cuda(), full - P, tail, swa, SCALE)
    out, lse = lib.group_attn(q.view(B, H, DIM), cache, table[:1, :P // PAGE].contiguous().cuda(),
                              torch.tensor([P], dtype=torch.int32).cuda(), torch.tensor([0, B], dtype=torch.int32).cuda(),
                              SCALE, o_own.view(B, H, DIM), lse_own.view(B, H))
    assert lib.last_device_error() == 0
    # both sides round probabilities to f16 (2^-11 of sum w |v|, |v| <= 4.5 here) and one rounds the result to bf16
    err = (out.double() - ref.view(B, H, DIM).double()).abs().cpu()
    assert bool((err <= 2.0 ** -8 * ref.view(B, H, DIM).abs().cpu().double() + 2 * 2.0 ** -11 * 4.5).all())
    np.testing.assert_allclose(lse.cpu(), ref_lse.view(B, H).cpu(), atol=2 * 2.0 ** -11, rtol=0)
