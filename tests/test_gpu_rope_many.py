"""K10 / K11 with enough tokens that a warp (K10) or a CTA (K11) takes several, ragged ends included, and K11 with
many heads of few tokens shared out over CTAs. Bytes and bits as in the small cases: no tolerance."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_rope import DIM, KD, PAGE, fill, freqs, held, lib, rotate, slots_of      # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [5921, 8883, 11841, 12001, 14209, 15003])
@pytest.mark.parametrize("keys", [False, True])
def test_append_many(lib, n, keys):
    g = torch.Generator().manual_seed(n)
    x, k = torch.randn(n, DIM, generator=g).to(torch.bfloat16), torch.randn(n, KD, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32)
    inv = freqs(32)
    pages = n // PAGE + 2
    slots = slots_of(n, pages, n)
    drop = torch.randperm(n, generator=g)[:100]
    slots[drop[:50]] = -1                                # skipped, not an error
    keep = torch.ones(n, dtype=torch.bool)
    keep[drop[:50]] = False
    cache = lib.PagedCache(pages)
    fill(cache)
    lib.append_kv_rope(x.cuda(), pos.cuda(), slots.cuda(), cache, lib.Rope(inv.cuda(), 512, True),
                       k.cuda() if keys else None, lib.Rope(inv.cuda(), 0, False) if keys else None)
    assert lib.last_device_error() == 0
    codes, scales, kc, sigma = held(cache, slots[keep])
    rc, rs = oracle.quant_fp4(oracle.bf16_bits(rotate(x[keep], pos[keep], inv, 512, True)))
    np.testing.assert_array_equal(scales, rs)
    np.testing.assert_array_equal(codes, rc)
    if keys:
        ok, osg = oracle.quant_index_fp8(oracle.bf16_bits(rotate(k[keep], pos[keep], inv, 0, False)))
        np.testing.assert_array_equal(sigma, osg)
        np.testing.assert_array_equal(kc, ok)
    rest = torch.ones(pages * PAGE, dtype=torch.bool)    # slots of nobody keep their bytes
    rest[slots[keep].long()] = False
    idx = rest.nonzero()[:, 0].int()
    codes, scales, kc, sigma = held(cache, idx)
    assert (codes == 0xA5).all() and (scales == 0xA5).all() and (sigma == -7.0).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,heads,dim,pairs,offset", [
    (1, 16, 576, 32, 512), (1, 1024, 64, 32, 0), (3, 7, 136, 8, 8), (3, 7, 136, 8, 20), (300, 5, 64, 4, 56),
    (2401, 2, 64, 32, 0), (4737, 1, 72, 12, 48), (9477, 1, 64, 16, 16), (9500, 3, 40, 10, 6), (1200, 2, 576, 288, 0)])
def test_rows_many(lib, n, heads, dim, pairs, offset, inter):
    g = torch.Generator().manual_seed(n + heads)
    x = torch.randn(n, heads, dim, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32)
    inv = freqs(pairs)
    rope = lib.Rope(inv.cuda(), offset, inter)
    ref = rotate(x, pos, inv, offset, inter)
    src = x.cuda()
    out = lib.rope_rows(src, pos.cuda(), rope)
    assert torch.equal(out.cpu(), ref) and torch.equal(src.cpu(), x)
    assert lib.rope_rows(src, pos.cuda(), rope, out=src) is src      # in place
    assert torch.equal(src.cpu(), ref) and lib.last_device_error() == 0
