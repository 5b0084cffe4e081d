"""The group attention over long groups: a flat tail behind one dominant entry, where the tail's weights are far below
f16's normal numbers, and a million entries. Pages are named many times, so that the exact values are sums over few
distinct entries.

Tolerances, with A = sum_t w_t |v_t| of the exact weights w: the result is rounded to bf16 (2^-8 |o|, half a step of the
type); a score s is off by d (see test_gpu_group_attn.py), which moves every weight by at most 2 d; a probability is
rounded to f16 after it was raised by 2^7: 2^-11 of itself, or where f16 has its fixed step 2^-24 by half of that,
2^-32 of the largest weight, T of them together T 2^-32 max |v|. The products are added up in fp32 16 entries at a time;
the tensor cores cut off what does not fit, at each of at most 4 additions 2^-23 of the sum so far, so n entries under one
accumulator give n / 16 2^-21 A; n is 32,768 at most, then the sum is moved out and added up with rounding (T / 28672
times at most, 2^-24 A each, the shorter of the two forms' distances). Joining the ranges (at most 160) gives
160 2^-24 A. lse as in test_gpu_group_attn.py."""
import math

import pytest
import torch

from test_gpu_group_attn import DIM, H, PAGE, SCALE, lib      # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu

ONE, HALF_STEP, AT_ONCE = 0x38, 2.0 ** -32, 32768                       # E4M3's 1.0


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def call(lib, cache, q, table, T, groups, own=None, scale=SCALE):
    """Every group has the same entries and an equal share of the tokens."""
    n = q.shape[0]
    return lib.group_attn(q, cache, table[None].expand(groups, -1).contiguous().cuda(),
                          torch.full((groups,), T, dtype=torch.int32).cuda(),
                          (torch.arange(groups + 1) * (n // groups)).int().cuda(), scale,
                          *((None, None) if own is None else own))


def expect(v, count, s, own=None):
    """Softmax over entries v [U, 576] with scores s [..., U], each there count times, joined with an own part."""
    s = s + torch.log(count)
    m = s.amax(-1, keepdim=True)
    if own is not None:
        m = torch.maximum(m, own[1][..., None])
    w = torch.exp(s - m)
    l = w.sum(-1, keepdim=True)
    o, A = w @ v, w @ v.abs()
    if own is not None:
        e = torch.exp(own[1][..., None] - m)
        l, o, A = l + e, o + e * own[0], A + e * own[0].abs()
    return o / l, A / l, (m + torch.log(l))[..., 0]


def close(out, lse, o, A, L, d, T, at_once, top):
    sums = min(at_once, AT_ONCE) / 16 * 2.0 ** -21 + (T / 28672 + 160) * 2.0 ** -24
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * d + sums) * A + T * HALF_STEP * top
    err = (out.double() - o).abs()
    assert bool((err <= tol).all()), f"off by {float((err / tol).max()):.2f} tolerances"
    tl = d[..., 0] + 2.0 ** -21 + (64 + T / 64) * 2.0 ** -24 + 2.0 ** -22 * L.abs()
    dl = (lse.double() - L).abs()
    assert bool((dl <= tl).all()), f"lse off by {float((dl / tl).max()):.2f} tolerances"


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("few", [False, True])
def test_flat_tail_behind_a_dominant_entry(lib, few, at, own):
    """A CTA walks 131,072 entries under one reference: one leads the others by 16 to 21 (a different lead for every
    head). The tail is up to a seventh of the output in the channels that it alone has, all of it in others."""
    T, pages = 131072, 2
    cache = lib.PagedCache(pages)
    cache.kv_scale.fill_(ONE)
    kv = torch.zeros(pages, PAGE, DIM, dtype=torch.uint8)
    kv[..., 192:] = 2                                    # the tail is 1 in channels 192 on
    sink = {"first": 0, "middle": 37, "last": 63}[at]
    kv[0, sink] = 0
    kv[0, sink, 0] = 7                                   # 6 in channel 0, the only one that the queries have
    kv[0, sink, 64:320] = 1                              # and 0.5 in channels 64 to 319
    cache.kv_fp4.copy_((kv[..., 0::2] | kv[..., 1::2] << 4).cuda())
    table = torch.ones(T // PAGE, dtype=torch.int32)
    table[{"first": 0, "middle": T // PAGE // 2, "last": T // PAGE - 1}[at]] = 0
    groups, tokens = (sms(), 4) if few else (1, 8)       # as many row tiles as CTAs, each a whole range
    n = sms() * tokens
    q = torch.zeros(n, H, DIM, dtype=torch.bfloat16)
    q[..., 0] = (64 + 1.25 * torch.arange(H)).to(torch.bfloat16)
    v = torch.zeros(2, DIM, dtype=torch.float64)
    v[0, 0], v[0, 64:320], v[1, 192:] = 6.0, 0.5, 1.0
    s = torch.stack((q[0, :, 0].double() * 6 * SCALE, torch.zeros(H, dtype=torch.float64)), -1)
    count = torch.tensor([1, T - 1], dtype=torch.float64)
    part = None
    if own:
        g = torch.Generator().manual_seed(1)
        part = (torch.randn(H, DIM, generator=g), torch.linspace(10, 20, H))
    o, A, L = expect(v, count, s, None if part is None else (part[0].double(), part[1].double()))
    d = (576 * 2.0 ** -24 + 2.0 ** -21) * s[:, :1]
    gpu = None if part is None else tuple(t.cuda()[None].expand(n, *t.shape).contiguous() for t in part)
    out, lse = call(lib, cache, q.cuda(), table, T, groups, gpu)
    assert lib.last_device_error() == 0
    close(out, lse, *(t.cuda() for t in (o, A, L, d)), T, T, 1.0)


@pytest.mark.parametrize("tiles,T", [(1, 1 << 20), (2.5, 131072), (2.5, 70000)])
@pytest.mark.parametrize("few", [False, True])
def test_sums_of_one_sign(lib, few, tiles, T):
    """Equal values, joined with an own part that takes all of them away again, so that the result is the error of the
    sum; two weights, so that no sum is exact. Row tiles that are a range each, and ranges of two and a half tiles."""
    cache = lib.PagedCache(1)
    cache.kv_scale.fill_(ONE)
    cache.kv_fp4.fill_(0x22)                             # 1.0
    cache.kv_fp4[0, ::2, 0] = 0x24                       # 2.0 in channel 0 of every other entry
    n, tokens = int(tiles * sms()), 4 if few else 8
    groups = n if few else 1
    n *= tokens
    q = torch.zeros(n, H, DIM, dtype=torch.bfloat16)
    q[..., 0] = (1 + torch.arange(H) * 2.0).to(torch.bfloat16)
    s = q[0, :, :1].double() * torch.tensor([2.0, 1.0]) * SCALE
    count = torch.tensor([-(-T // 2), T // 2], dtype=torch.float64)
    v = torch.ones(2, DIM, dtype=torch.float64)
    v[0, 0] = 2.0
    o, _, L = expect(v, count, s)
    own = (-o.float().cuda()[None].expand(n, H, DIM).contiguous(), L.float().cuda()[None].expand(n, H).contiguous())
    out, lse = call(lib, cache, q.cuda(), torch.zeros(-(-T // PAGE), dtype=torch.int32), T, groups, own)
    assert lib.last_device_error() == 0
    exact = expect(v, count, s, (own[0][0].double().cpu(), own[1][0].double().cpu()))
    d = (576 * 2.0 ** -24 + 2.0 ** -21) * s[:, :1]
    close(out, lse, *(t.cuda() for t in exact + (d,)), T, T, 2.0)


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("tokens,groups,gain", [(4, 1, 1.0), (4, 1, 5.0), (9, 1, 1.0), (9, 1, 5.0), (3, 3, 1.0)])
def test_a_million_entries(lib, tokens, groups, gain, own):
    T, pages = (1 << 20) - 29, 256
    g = torch.Generator().manual_seed(tokens)
    cache = lib.PagedCache(pages)
    n = pages * PAGE
    lib.quant_kv_fp4(torch.randn(n, DIM, generator=g).to(torch.bfloat16).cuda(), torch.arange(n, dtype=torch.int32).cuda(),
                     cache)
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64).cuda()
    codes = torch.stack((cache.kv_fp4 & 15, cache.kv_fp4 >> 4), -1).flatten(-2).long()
    v = (lut[codes].view(n, 36, 16) * cache.kv_scale.view(torch.float8_e4m3fn).double().view(n, 36, 1)).view(n, DIM)
    table = torch.randint(0, pages, (-(-T // PAGE),), generator=g, dtype=torch.int32)
    count = torch.bincount(table.long()[:-1], minlength=pages).double()[:, None].repeat(1, PAGE)
    count[int(table[-1]), :T - (len(table) - 1) * PAGE] += 1
    assert int(count.sum()) == T
    q = (torch.randn(tokens, H, DIM, generator=g) * gain).to(torch.bfloat16).cuda()
    s = q.double() @ v.t() * SCALE
    d = (576 * 2.0 ** -24 * SCALE * (q.double().abs() @ v.abs().t()) + 2.0 ** -21 * s.abs()).amax(-1, keepdim=True)
    part = None
    if own:
        part = (torch.randn(tokens, H, DIM, generator=g).cuda(), torch.randn(tokens, H, generator=g).cuda() + 14)
    o, A, L = expect(v, count.view(-1).cuda(), s, None if part is None else (part[0].double(), part[1].double()))
    out, lse = call(lib, cache, q, table, T, groups, part)
    assert lib.last_device_error() == 0
    close(out, lse, o, A, L, d, T, T * max(groups, -(-tokens // 8)) / sms() + 128, float(v.abs().max()))


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("few", [False, True])
def test_groups_about_the_distance_of_moving_out(lib, few, own):
    """Groups whose row tiles are cut anywhere, of lengths about the distances at which outputs leave tensor memory, with
    pages that are left out, entries whose scores grow half-way, and a workspace that holds anything."""
    lens = [32768, 32769, 0, 28672, 28673, 65536, 65537, 57345, 200, 140001] * (10 if few else 1)
    share = [3, 4, 2, 5, 1, 4, 0, 7, 4, 4] if few else [90, 64, 9, 130, 61, 40, 0, 77, 8, 210]
    tokens = share * (10 if few else 1)
    N, G, pages = sum(tokens), len(lens), 24
    assert few == (N <= 4 * G)
    g = torch.Generator().manual_seed(8)
    cache = lib.PagedCache(pages)
    n = pages * PAGE
    x = torch.randn(n, DIM, generator=g) + 0.25
    x[n // 2:, 0] += 6
    lib.quant_kv_fp4(x.to(torch.bfloat16).cuda(), torch.arange(n, dtype=torch.int32).cuda(), cache)
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64).cuda()
    codes = torch.stack((cache.kv_fp4 & 15, cache.kv_fp4 >> 4), -1).flatten(-2).long()
    v = (lut[codes].view(n, 36, 16) * cache.kv_scale.view(torch.float8_e4m3fn).double().view(n, 36, 1)).view(n, DIM)
    W = max(-(-t // PAGE) for t in lens)
    table = torch.randint(0, pages, (G, W), generator=g)
    table[:, :W // 4] %= pages // 2
    table[torch.rand(G, W, generator=g) < 0.02] = -1
    q = torch.randn(N, H, DIM, generator=g)
    q[:, ::2, 0] += 8
    q = q.to(torch.bfloat16).cuda()
    part = (None, None) if not own else (torch.randn(N, H, DIM, generator=g).cuda(), torch.randn(N, H, generator=g).cuda() + 11)
    offs = [sum(tokens[:i]) for i in range(G + 1)]
    got = []
    for fill in (0, 0xFF):
        ws = torch.full((lib.group_attn_workspace_bytes(N, G),), fill, dtype=torch.uint8, device="cuda")
        got.append(lib.group_attn(q, cache, table.int().cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                  torch.tensor(offs, dtype=torch.int32).cuda(), SCALE, *part, ws=ws))
    assert lib.status_string(lib.last_device_error()) == "CSA2_ERR_DEVICE_BOUNDS"
    (out, lse), again = got
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    for i, T in enumerate(lens):
        a, b = offs[i], offs[i + 1]
        if a == b:
            continue
        mine = None if not own else (part[0][a:b].double(), part[1][a:b].double())
        t = torch.arange(T)
        page = table[i][t // PAGE]
        count = torch.bincount((page * PAGE + t % PAGE)[page >= 0], minlength=n).double().cuda()
        if T == 0:
            o = mine[0] if own else torch.zeros(b - a, H, DIM, dtype=torch.float64).cuda()
            assert torch.equal(out[a:b], o.to(torch.bfloat16))
            assert torch.equal(lse[a:b], part[1][a:b]) if own else bool((lse[a:b] == -math.inf).all())
            continue
        s = q[a:b].double() @ v.t() * SCALE
        d = (576 * 2.0 ** -24 * SCALE * (q[a:b].double().abs() @ v.abs().t()) + 2.0 ** -21 * s.abs()).amax(-1, keepdim=True)
        o, A, L = expect(v, count, s, mine)
        close(out[a:b], lse[a:b], o, A, L, d, T, T, float(v.abs().max()))


@pytest.mark.parametrize("power,scale", [(-130, SCALE), (20, SCALE), (24, -SCALE), (-100, 2.0 ** 98), (-62, 2.0 ** 60),
                                         (70, 2.0 ** -69), (80, -2.0 ** -80), (113, 2.0 ** -113), (127, 2.0 ** -124)])
@pytest.mark.parametrize("tokens,groups", [(9, 1), (4, 1)])
def test_queries_of_any_finite_magnitude(lib, tokens, groups, power, scale):
    """Queries of magnitude 2^power, from bf16's subnormal numbers to its largest, under scales that keep the scores below
    2^23. Entries of two kinds, 1 and 0.5 in channel 0, the only one that the queries have."""
    T, pages = 200, 4
    g = torch.Generator().manual_seed(power + 200)
    cache = lib.PagedCache(pages)
    cache.kv_scale.fill_(ONE)
    kv = torch.randint(0, 16, (pages, PAGE, DIM), generator=g, dtype=torch.uint8)
    kv[..., 0] = 2                                       # 1.0, in every third entry 0.5
    kv[:, ::3, 0] = 1
    cache.kv_fp4.copy_((kv[..., 0::2] | kv[..., 1::2] << 4).cuda())
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    v = lut[kv.view(-1, DIM)[:T].long()]
    q = torch.zeros(tokens, H, DIM, dtype=torch.bfloat16)
    q[..., 0] = 2.0 ** power * 1.25
    s = q[0, :, :1].double() * v[:, 0] * scale
    o, A, L = expect(v, torch.ones(T, dtype=torch.float64), s)
    out, lse = call(lib, cache, q.cuda(), torch.arange(pages, dtype=torch.int32), T, groups, scale=scale)
    assert lib.last_device_error() == 0
    # the kinds' distance (64 at most where both weigh) is off by 2^-22 of itself for the scale and 2^-19 for the
    # exponent's argument; lse by five roundings of its magnitude
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2.0 ** -15) * A + T * HALF_STEP * 6
    assert bool(((out.cpu().double() - o).abs() <= tol).all())
    assert bool(((lse.cpu().double() - L).abs() <= 2.0 ** -21 * s.abs().amax() + 2.0 ** -18).all())
