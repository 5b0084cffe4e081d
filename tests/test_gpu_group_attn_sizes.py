"""K12 / K13 at the ends of their ranges: more groups than a batch of the offsets' scan holds, one token and no entry,
pages behind the 4 GiB mark, one page many times, a batch much longer than its entries. Against the formula in
64 bits, with the tolerances of the group attention's own test module."""
import math

import pytest
import torch

from test_gpu_group_attn import DIM, H, PAGE, SCALE, Case, lib      # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("groups", [511, 512, 513, 1300])
def test_many_groups(lib, groups, own):
    c = Case(lib, [(i * 7) % 4 for i in range(groups)], [(i * 37) % 150 if i % 5 else 0 for i in range(groups)],
             seed=groups)
    if own:
        c.with_own()
    out, lse = c.call()
    assert lib.last_device_error() == 0
    c.check(out, lse)


def test_one_long_group_among_many_short_ones(lib):
    tokens, lens = [1] * 300, [3] * 300
    tokens[150], lens[150] = 17, 30000
    tokens[299], lens[299] = 8, 5000
    c = Case(lib, tokens, lens, seed=20).with_own()
    out, lse = c.call()
    assert lib.last_device_error() == 0
    c.check(out, lse)


@pytest.mark.parametrize("tokens,length", [(1, 0), (8, 1), (1, 148 * 64 + 1), (500, 70), (1100, 1)])
def test_sizes(lib, tokens, length):
    c = Case(lib, [tokens], [length], seed=tokens)
    c.check(*c.call())
    c.with_own()
    c.check(*c.call())
    assert lib.last_device_error() == 0


def test_the_same_page_again(lib):
    """Groups that share pages with one another, and a page that a group names twice."""
    c = Case(lib, [5, 9, 1], [300, 260, 640], seed=21)
    c.table[1, :5] = c.table[0, :5]
    c.table[2, 4], c.table[2, 7] = c.table[0, 0], c.table[0, 0]
    out, lse = c.call()
    assert lib.last_device_error() == 0
    c.check(out, lse)


def test_pages_behind_four_gib(lib):
    """18,432 B of codes a page: byte offsets of these pages need more than 32 bits. The append writes them there."""
    from test_gpu_rope import freqs, rotate, held
    pages, n = 240000, 200
    cache = lib.PagedCache(pages)
    table = torch.tensor([[pages - 1, 5, pages - 7, 233100]], dtype=torch.int32)
    g = torch.Generator().manual_seed(22)
    x, k = torch.randn(n, DIM, generator=g).to(torch.bfloat16), torch.randn(n, 64, generator=g).to(torch.bfloat16)
    inv, pos = freqs(32), torch.arange(n)
    slots = lib.slot_mapping(table, 0, pos)
    lib.append_kv_rope(x.cuda(), pos.int().cuda(), slots.cuda(), cache, lib.Rope(inv.cuda(), 512, True), k.cuda(),
                       lib.Rope(inv.cuda(), 0, True))
    small = lib.PagedCache(4)
    small_slots = torch.arange(n, dtype=torch.int32)
    lib.append_kv_rope(x.cuda(), pos.int().cuda(), small_slots.cuda(), small, lib.Rope(inv.cuda(), 512, True), k.cuda(),
                       lib.Rope(inv.cuda(), 0, True))
    assert lib.last_device_error() == 0
    s = slots.long().cuda()
    for name, width in (("kv_fp4", 288), ("kv_scale", 36)):
        assert torch.equal(getattr(cache, name).view(-1, width)[s], getattr(small, name).view(-1, width)[:n])
    assert torch.equal(cache.kidx_scale.view(-1)[s], small.kidx_scale.view(-1)[:n])
    for at in range(4):
        page, m = int(table[0, at]), min(PAGE, n - at * PAGE)
        got, ref = (t.view(8, 4, 8, 16).permute(0, 2, 1, 3).reshape(PAGE, 64) for t in (cache.kidx[page], small.kidx[at]))
        assert torch.equal(got[:m], ref[:m])
    q = torch.randn(3, H, DIM, generator=g).to(torch.bfloat16).cuda()
    lens, offs = torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor([0, 3], dtype=torch.int32).cuda()
    far = lib.group_attn(q, cache, table.cuda(), lens, offs, SCALE)
    near = lib.group_attn(q, small, torch.arange(4, dtype=torch.int32)[None].cuda(), lens, offs, SCALE)
    assert lib.last_device_error() == 0
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])


def test_infinite_and_missing_own_parts(lib):
    """lse_own of -inf leaves the entries alone, of +inf or NaN makes that row NaN and no other."""
    c = Case(lib, [6], [200], seed=23).with_own()
    ref, ref_lse = c.call()
    c.own[1][1, 2], c.own[1][4, 15] = math.inf, math.nan
    out, lse = c.call()
    bad = torch.zeros(6, H, dtype=torch.bool)
    bad[1, 2] = bad[4, 15] = True
    assert torch.equal(out.cpu()[~bad], ref.cpu()[~bad]) and torch.equal(lse.cpu()[~bad], ref_lse.cpu()[~bad])
    assert torch.isnan(lse.cpu()[bad]).all()


def test_two_graphs_in_turn(lib):
    """Two captured calls with workspaces of their own, replayed at once on two streams."""
    cases = [Case(lib, [9, 2], [2000, 65], seed=24).with_own(), Case(lib, [40], [700], seed=25)]
    runs, refs = [], []
    for c in cases:
        refs.append(c.call())
        args = (c.q.cuda(), c.cache, c.table.cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda(),
                torch.tensor(c.offs, dtype=torch.int32).cuda(), SCALE) + (
                    (None, None) if c.own is None else tuple(t.cuda() for t in c.own))
        out, lse = torch.zeros(c.N, H, DIM, dtype=torch.bfloat16).cuda(), torch.zeros(c.N, H).cuda()
        ws = lib.workspace(lib.group_attn_workspace_bytes(c.N, len(c.lens)))
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            lib.group_attn(*args, out=out, lse=lse, ws=ws)
        runs.append((graph, out, lse, args, ws))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                r[0].replay()
    torch.cuda.synchronize()
    for (ref, ref_lse), r in zip(refs, runs):
        assert torch.equal(ref, r[1]) and torch.equal(ref_lse, r[2])
    assert lib.last_device_error() == 0


def test_no_group_has_tokens(lib):
    c = Case(lib, [0, 0, 0], [100, 0, 70], before=2, after=3).with_own()
    out = torch.full((c.N, H, DIM), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.N, H), -2.0, device="cuda")
    for _ in range(2):
        c.call(out, lse)
    assert lib.last_device_error() == 0
    assert (out == 3.0).all() and (lse == -2.0).all()


def test_most_groups(lib):
    tokens, lens = [0] * 65535, [0] * 65535
    for g, (t, n) in {0: (1, 65), 511: (2, 300), 512: (1, 1), 40000: (7, 1000), 65534: (1, 64)}.items():
        tokens[g], lens[g] = t, n
    c = Case(lib, tokens, lens, seed=26).with_own()
    out, lse = c.call()
    assert lib.last_device_error() == 0
    c.check(out, lse)
