"""K10 / K11: the paged append with the position rotation, and the rotation of
query rows. The rotation is checked against angles, sines and products in 64
bits (NumPy), the quantised bytes against the oracle on the rotated rows."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DIM, KD, PAGE = 576, 64, 64


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from compressed_sparse_attention_quant_b200 import lib as L
    return L


def freqs(pairs, base=10000.0):
    return torch.from_numpy((base ** (-np.arange(pairs) / pairs)).astype(np.float32))


def rotate(x, pos, inv_freq, offset, interleaved):
    """x [n, ..., D] bf16 (CPU) -> rotated bf16: 64 bits, then binary32, then bf16."""
    half = len(inv_freq)
    ang = pos.numpy().astype(np.float64)[:, None] * inv_freq.numpy().astype(np.float64)
    c, s = np.cos(ang), np.sin(ang)
    for _ in range(x.dim() - 2):
        c, s = c[:, None], s[:, None]
    y = x.double().numpy().copy()
    i = np.arange(half)
    ia, ib = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + half + i)
    a, b = y[..., ia], y[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return torch.from_numpy(y.astype(np.float32)).to(torch.bfloat16)


def slots_of(n, pages, seed):
    return torch.randperm(pages * PAGE, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32)


def held(cache, slots):
    """The cache's bytes at the slots: codes, scales, keys, sigma."""
    s = slots.long().cuda()
    logical = cache.kidx_logical().reshape(-1, KD)
    return (cache.kv_fp4.view(-1, 288)[s].cpu().numpy(), cache.kv_scale.view(-1, 36)[s].cpu().numpy(),
            logical[s].cpu().numpy(), cache.kidx_scale.view(-1)[s].cpu().numpy())


def fill(cache, byte=0xA5):
    for t in (cache.kv_fp4, cache.kv_scale, cache.kidx):
        t.fill_(byte)
    cache.kidx_scale.fill_(-7.0)


def strided(x, stride):
    wide = torch.full((x.shape[0], stride), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :x.shape[1]] = x.cuda()
    return wide[:, :x.shape[1]]


CASES = [  # n, pairs, offset, interleaved, x stride, key: (pairs, offset, interleaved) or None, far
    (1, 32, 512, True, 576, (32, 0, True), 1 << 20),
    (7, 32, 512, False, 584, (32, 0, False), 131072),
    (8, 1, 574, True, 576, None, 100),
    (9, 3, 10, False, 640, (3, 58, True), 1 << 16),
    (64, 288, 0, True, 576, (16, 32, False), 4096),
    (65, 288, 0, False, 1152, None, 1 << 29),
    (130, 48, 480, True, 576, (32, 0, True), 1 << 29),
    (515, 8, 20, False, 576, (8, 2, False), 1 << 24),
]


@pytest.mark.parametrize("n,pairs,offset,inter,stride,key,far", CASES)
@pytest.mark.parametrize("same_freqs", [True, False])
def test_append_bytes(lib, n, pairs, offset, inter, stride, key, far, same_freqs):
    g = torch.Generator().manual_seed(n + pairs)
    x = (torch.randn(n, DIM, generator=g) * torch.exp2(torch.randint(-20, 20, (n, 1), generator=g).float())
         ).to(torch.bfloat16)
    pos = torch.randint(0, far, (n,), generator=g, dtype=torch.int32)
    pos[-1] = far - 1
    pos[0] = 0 if n > 1 else pos[0]
    inv = freqs(pairs)
    inv_dev = inv.cuda()
    pages = n // PAGE + 2
    slots = slots_of(n, pages, n)
    cache = lib.PagedCache(pages)
    fill(cache)
    k = kr = kinv = None
    if key is not None:
        kp, ko, ki = key
        k = torch.randn(n, KD, generator=g).to(torch.bfloat16)
        # the latent's own table when it is long enough (one angle for both rows), else a table of its own
        shared = same_freqs and kp <= pairs
        kinv = inv[:kp] if shared else freqs(kp, 160000.0)
        kr = lib.Rope(inv_dev[:kp] if shared else kinv.cuda(), ko, ki)
    lib.append_kv_rope(strided(x, stride), pos.cuda(), slots.cuda(), cache, lib.Rope(inv_dev, offset, inter),
                       None if k is None else strided(k, KD + 8), kr)
    assert lib.last_device_error() == 0
    codes, scales, keys, sigma = held(cache, slots)
    rc, rs = oracle.quant_fp4(oracle.bf16_bits(rotate(x, pos, inv, offset, inter)))
    np.testing.assert_array_equal(scales, rs)
    np.testing.assert_array_equal(codes, rc)
    if k is not None:
        ok, osg = oracle.quant_index_fp8(oracle.bf16_bits(rotate(k, pos, kinv, key[1], key[2])))
        np.testing.assert_array_equal(sigma, osg)
        np.testing.assert_array_equal(keys, ok)
    else:
        assert (keys == 0xA5).all() and (sigma == -7.0).all()
    # every other slot as it was
    rest = torch.ones(pages * PAGE, dtype=torch.bool)
    rest[slots.long()] = False
    codes, scales, keys, sigma = held(cache, rest.nonzero()[:, 0])
    assert (codes == 0xA5).all() and (scales == 0xA5).all() and (keys == 0xA5).all() and (sigma == -7.0).all()


def test_append_unrotated_key_and_padding(lib):
    n, inv = 37, freqs(32)
    g = torch.Generator().manual_seed(5)
    x, k = (torch.randn(n, c, generator=g).to(torch.bfloat16) for c in (DIM, KD))
    pos = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32)
    slots = slots_of(n, 3, 1)
    slots[::5] = -1
    pos[::5] = -9                                          # a skipped token's position is not looked at
    cache = lib.PagedCache(3)
    fill(cache)
    lib.append_kv_rope(x.cuda(), pos.cuda(), slots.cuda(), cache, lib.Rope(inv.cuda(), 512, True), k.cuda())
    assert lib.last_device_error() == 0
    keep = slots >= 0
    codes, scales, keys, sigma = held(cache, slots[keep])
    rc, rs = oracle.quant_fp4(oracle.bf16_bits(rotate(x[keep], pos[keep], inv, 512, True)))
    ok, osg = oracle.quant_index_fp8(oracle.bf16_bits(k[keep]))
    for got, ref in ((codes, rc), (scales, rs), (keys, ok), (sigma, osg)):
        np.testing.assert_array_equal(got, ref)
    assert int((cache.kidx_scale != -7.0).sum()) == int(keep.sum())


def test_append_bad_slots_and_positions_are_skipped(lib):
    n, inv = 12, freqs(32)
    x = torch.randn(n, DIM, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    pos = torch.arange(n, dtype=torch.int32)
    slots = slots_of(n, 2, 3)
    for bad in ("slot", "low", "high"):
        cache = lib.PagedCache(2)
        fill(cache)
        p, s = pos.clone(), slots.clone()
        if bad == "slot":
            s[4] = 2 * PAGE
        else:
            p[4] = -1 if bad == "low" else 1 << 29
        lib.append_kv_rope(x.cuda(), p.cuda(), s.cuda(), cache, lib.Rope(inv.cuda(), 512, True))
        assert lib.status_string(lib.last_device_error()) == "CSA2_ERR_DEVICE_BOUNDS"
        keep = torch.arange(n) != 4
        codes, scales, _, _ = held(cache, s[keep])
        rc, rs = oracle.quant_fp4(oracle.bf16_bits(rotate(x[keep], p[keep], inv, 512, True)))
        np.testing.assert_array_equal(codes, rc)
        np.testing.assert_array_equal(scales, rs)
        assert int((cache.kv_scale.view(-1, 36) != 0xA5).any(-1).sum()) <= n - 1
        if bad != "slot":
            assert (held(cache, s[4:5])[0] == 0xA5).all()


def test_append_at_position_zero_is_the_plain_append(lib):
    """No rotation at position 0, so the bytes are csa2_quant_kv_fp4's and csa2_quant_indexer_fp8's: every bf16
    value up to 6s under every E4M3 scale s, and rows of every magnitude."""
    e4m3 = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    every = every[torch.isfinite(every.float())]
    groups = []
    for s in e4m3:
        v = every[every.double().abs() <= 6 * s]
        v = torch.cat([v, torch.zeros((-len(v)) % 15, dtype=torch.bfloat16)]).view(-1, 15)
        groups.append(torch.cat([torch.full((len(v), 1), float(6 * s)).to(torch.bfloat16), v], 1))
    big = every.double().abs() > 6 * e4m3[-1]
    v = every[big]
    groups.append(torch.cat([v, torch.zeros((-len(v)) % 16, dtype=torch.bfloat16)]).view(-1, 16))
    groups = torch.cat(groups)
    pad = (-len(groups)) % 36
    x = torch.cat([groups, torch.zeros(pad, 16, dtype=torch.bfloat16)]).view(-1, DIM).cuda()
    n = x.shape[0]
    g = torch.Generator().manual_seed(9)
    k = (torch.randn(n, KD, generator=g) * torch.exp2(torch.randint(-100, 100, (n, 1), generator=g).float())
         ).to(torch.bfloat16).cuda()
    pages = n // PAGE + 1
    slots = slots_of(n, pages, 4).cuda()
    a, b = lib.PagedCache(pages), lib.PagedCache(pages)
    zero = torch.zeros(n, dtype=torch.int32, device="cuda")
    inv = freqs(32).cuda()
    lib.append_kv_rope(x, zero, slots, a, lib.Rope(inv, 512, True), k, lib.Rope(inv, 0, False))
    codes, sigma = lib.quant_indexer_fp8(k)
    lib.quant_kv_fp4(x, slots, b, codes, sigma)
    assert lib.last_device_error() == 0
    for t in ("kv_fp4", "kv_scale", "kidx", "kidx_scale"):
        assert torch.equal(getattr(a, t), getattr(b, t)), t


@pytest.mark.parametrize("n,heads,dim,pairs,offset,inter", [
    (1, 16, 576, 32, 512, True), (3, 16, 576, 32, 512, False), (64, 4, 64, 32, 0, True), (9, 4, 64, 16, 32, False),
    (17, 1, 576, 288, 0, True), (5, 1, 576, 288, 0, False), (33, 3, 72, 5, 6, False), (130, 2, 8, 1, 2, True),
    (2, 1024, 16, 8, 0, False), (257, 16, 576, 24, 100, True)])
def test_rope_rows(lib, n, heads, dim, pairs, offset, inter):
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, heads, dim, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 29, (n,), generator=g, dtype=torch.int32)
    pos[0] = (1 << 29) - 1
    inv = freqs(pairs)
    ref = rotate(x, pos, inv, offset, inter)
    rope = lib.Rope(inv.cuda(), offset, inter)
    got = lib.rope_rows(x.cuda(), pos.cuda(), rope)
    assert torch.equal(got.cpu(), ref)
    # in place, and from and to slices of wider rows (the rest of which stays)
    y = x.cuda()
    assert lib.rope_rows(y, pos.cuda(), rope, out=y) is y
    assert torch.equal(y.cpu(), ref)
    wide_in = torch.full((n, heads * dim + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    wide_out = torch.full((n, heads * dim + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    src = wide_in[:, 8:8 + heads * dim].view(n, heads, dim)
    dst = wide_out[:, :heads * dim].view(n, heads, dim)
    src.copy_(x)
    lib.rope_rows(src, pos.cuda(), rope, out=dst)
    assert lib.last_device_error() == 0
    assert torch.equal(dst.cpu(), ref)
    assert (wide_out[:, heads * dim:] == 3.0).all() and torch.equal(src.cpu(), x)


def test_rope_rows_bad_position_leaves_the_row(lib):
    x = torch.randn(20, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    pos = torch.arange(20, dtype=torch.int32)
    pos[7], pos[19] = -1, 1 << 29
    inv = freqs(32)
    out = torch.full_like(x, 9.0).cuda()
    lib.rope_rows(x.cuda(), pos.cuda(), lib.Rope(inv.cuda()), out=out)
    assert lib.status_string(lib.last_device_error()) == "CSA2_ERR_DEVICE_BOUNDS"
    keep = (pos >= 0) & (pos < 1 << 29)
    assert torch.equal(out.cpu()[keep], rotate(x[keep], pos[keep], inv, 0, False))
    assert (out.cpu()[~keep] == 9.0).all()


def test_rotation_captured_and_on_another_stream(lib):
    """The append and the query rotation in one CUDA graph, replayed on refreshed inputs."""
    n, inv = 40, freqs(32)
    rope, krope = lib.Rope(inv.cuda(), 512, True), lib.Rope(inv.cuda(), 0, True)
    x, k = torch.zeros(n, DIM, dtype=torch.bfloat16).cuda(), torch.zeros(n, KD, dtype=torch.bfloat16).cuda()
    q = torch.zeros(n, 16, DIM, dtype=torch.bfloat16).cuda()
    out = torch.empty_like(q)
    pos, slots = torch.zeros(n, dtype=torch.int32).cuda(), slots_of(n, 2, 0).cuda()
    cache = lib.PagedCache(2)

    def step():
        lib.append_kv_rope(x, pos, slots, cache, rope, k, krope)
        lib.rope_rows(q, pos, rope, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        xs, ks, qs = (torch.randn(s, generator=g).to(torch.bfloat16) for s in ((n, DIM), (n, KD), (n, 16, DIM)))
        ps = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32)
        for d, v in ((x, xs), (k, ks), (q, qs), (pos, ps)):
            d.copy_(v)
        graph.replay()
        assert lib.last_device_error() == 0
        codes, scales, keys, sigma = held(cache, slots.cpu())
        rc, rs = oracle.quant_fp4(oracle.bf16_bits(rotate(xs, ps, inv, 512, True)))
        ok, osg = oracle.quant_index_fp8(oracle.bf16_bits(rotate(ks, ps, inv, 0, True)))
        for got, ref in ((codes, rc), (scales, rs), (keys, ok), (sigma, osg)):
            np.testing.assert_array_equal(got, ref)
        assert torch.equal(out.cpu(), rotate(qs, ps, inv, 512, True))
