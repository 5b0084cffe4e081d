"""Refusals of the append with rotation, the query rotation and the group
attention (CPU): every argument error is found on the host, with its own
status, before anything is enqueued."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from compressed_sparse_attention_quant_b200 import _build
    _build.build()
    from compressed_sparse_attention_quant_b200 import lib as L
    return L


INVALID, UNSUPPORTED, WORKSPACE, ALIGNMENT = 1, 2, 7, 8


def rope(lib, inv=16, dim=64, offset=0, interleaved=0):
    return ctypes.byref(lib._Rope(inv, dim, offset, interleaved))


def test_append_refusals(lib):
    cache = lib._Cache(16, 16, 16, 16, 4)

    def call(x=16, xs=576, n=4, dim=576, pos=16, slots=16, r="ok", k=16, ks=64, kr="ok", c=cache):
        r = rope(lib) if r == "ok" else r
        kr = rope(lib) if kr == "ok" else kr
        return lib._L.csa2_append_kv_rope(x, xs, n, dim, pos, slots, r, k, ks, kr,
                                          None if c is None else ctypes.byref(c), None)

    n0 = lib.launch_count()
    assert call(n=0) == 0 and call(n=0, x=None, k=None, kr=None) == 0
    for bad in (dict(n=-1), dict(c=None), dict(r=None), dict(x=None), dict(pos=None), dict(slots=None),
                dict(xs=568), dict(ks=56), dict(k=None), dict(c=lib._Cache(16, 16, 16, 16, 0)),
                dict(c=lib._Cache(None, 16, 16, 16, 4)), dict(c=lib._Cache(16, None, 16, 16, 4)),
                dict(c=lib._Cache(16, 16, None, 16, 4)), dict(c=lib._Cache(16, 16, 16, None, 4)),
                dict(r=rope(lib, inv=None)), dict(r=rope(lib, dim=0)), dict(r=rope(lib, dim=63)),
                dict(r=rope(lib, dim=578)), dict(r=rope(lib, offset=514)), dict(r=rope(lib, offset=-2)),
                dict(r=rope(lib, offset=1)), dict(r=rope(lib, interleaved=2)), dict(kr=rope(lib, offset=2)),
                dict(kr=rope(lib, dim=128)), dict(r=rope(lib, dim=2, offset=2147483646))):
        assert call(**bad) == INVALID, bad
    assert call(dim=512) == UNSUPPORTED and call(n=(1 << 31) + 1) == UNSUPPORTED
    assert call(xs=(1 << 31) + 8) == UNSUPPORTED
    for bad in (dict(x=24), dict(xs=580), dict(k=24), dict(ks=68), dict(pos=18), dict(slots=18),
                dict(r=rope(lib, inv=18)), dict(kr=rope(lib, inv=18)), dict(c=lib._Cache(24, 16, 16, 16, 4)),
                dict(c=lib._Cache(16, 16, 24, 16, 4)), dict(c=lib._Cache(16, 16, 16, 20, 4))):
        assert call(**bad) == ALIGNMENT, bad
    assert lib.launch_count() == n0


def test_rope_rows_refusals(lib):
    def call(x=16, xs=256, n=4, heads=4, dim=64, pos=16, r="ok", out=32, os=256):
        return lib._L.csa2_rope_rows(x, xs, n, heads, dim, pos, rope(lib) if r == "ok" else r, out, os, None)

    n0 = lib.launch_count()
    assert call(n=0) == 0
    for bad in (dict(n=-1), dict(heads=0), dict(dim=0), dict(r=None), dict(x=None), dict(pos=None), dict(out=None),
                dict(xs=248), dict(os=248), dict(out=16, os=264), dict(r=rope(lib, offset=2)),
                dict(r=rope(lib, dim=66)), dict(xs=(1 << 31) + 8)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dim=584, xs=1 << 13, os=1 << 13), dict(dim=60), dict(heads=1025), dict(n=(1 << 31) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(x=24), dict(out=24), dict(xs=260), dict(os=260), dict(pos=18), dict(r=rope(lib, inv=18))):
        assert call(**bad) == ALIGNMENT, bad
    assert lib.launch_count() == n0


def test_group_attn_refusals(lib):
    cache = lib._Cache(16, 16, None, None, 4)            # the indexer's arrays are not read

    def call(q=16, N=4, H=16, D=576, c=cache, pt=16, G=1, mp=2, lens=16, offs=16, scale=0.1, o=None, l=None, out=16,
             lse=16, ws=256, nb=1 << 40):
        return lib._L.csa2_group_attn(q, N, H, D, None if c is None else ctypes.byref(c), pt, G, mp, lens, offs, scale,
                                      o, l, out, lse, ws, nb, None)

    n0 = lib.launch_count()
    for bad in (dict(N=0), dict(G=0), dict(mp=0), dict(c=None), dict(q=None), dict(pt=None), dict(lens=None),
                dict(offs=None), dict(out=None), dict(lse=None), dict(o=16), dict(l=16), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(c=lib._Cache(None, 16, None, None, 4)),
                dict(c=lib._Cache(16, None, None, None, 4)), dict(c=lib._Cache(16, 16, None, None, -1))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(H=8), dict(D=512), dict(N=(1 << 20) + 1), dict(G=65536), dict(mp=(1 << 24) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(q=24), dict(out=24), dict(lse=18), dict(pt=18), dict(lens=18), dict(offs=18), dict(o=24, l=16),
                dict(o=16, l=18), dict(c=lib._Cache(24, 16, None, None, 4)), dict(c=lib._Cache(16, 24, None, None, 4))):
        assert call(**bad) == ALIGNMENT, bad
    assert lib.launch_count() == n0
    for N, G in ((0, 1), (1, 0), (-1, 1), ((1 << 20) + 1, 1), (1, 65536)):
        assert lib.group_attn_workspace_bytes(N, G) == 0


def test_binding_refusals(lib):
    bf = torch.zeros(4, 576, dtype=torch.bfloat16)
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        lib.Rope(torch.ones(32))                          # frequencies on the CPU
    with pytest.raises(TypeError):
        lib.Rope(torch.ones(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        lib.append_kv_rope(bf, i32, i32, None, None)      # rows on the CPU
    with pytest.raises(TypeError):
        lib.append_kv_rope(bf.float(), i32, i32, None, None)
    with pytest.raises(ValueError):
        lib.rope_rows(bf, i32, None)                      # no head dimension
    with pytest.raises(ValueError):
        lib.group_attn(bf.view(4, 1, 576), None, i32, i32, i32, 0.1)
