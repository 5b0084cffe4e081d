"""Host checks (CPU) of the rotation and the group attention: outputs that share bytes with an input or the workspace
are refused, neighbours are not. A call that passes every check ends with CSA2_ERR_CUDA here, for want of a GPU;
addresses are numbers that nothing reads."""
import ctypes

import pytest
import torch

from compressed_sparse_attention_quant_b200 import lib

INVALID, CUDA, WORKSPACE = 1, 3, 7
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would launch")
M = 1 << 20


def rows(x, xs, out, os, n=4, heads=2, dim=64):
    r = lib._Rope(16, 64, 0, 1)
    return lib._L.csa2_rope_rows(x, xs, n, heads, dim, 16, ctypes.byref(r), out, os, None)


@pytest.mark.parametrize("x,xs,out,os,ok", [
    (M, 128, M, 128, True),                              # in place
    (M, 128, M + 4 * 256, 128, True),                    # one after the other
    (M, 128, M + 3 * 256, 128, False),                   # the last row is the first
    (M, 128, M + 16, 128, False),
    (M, 256, M + 256, 256, True),                        # columns side by side in one wide tensor
    (M + 256, 256, M, 256, True),
    (M, 256, M + 240, 256, False),
    (M, 256, M + 272, 256, False),                       # reaches into the next row
    (M, 248, M + 256, 248, False),
    (M, 256, M + 256, 512, False),                       # two strides, ranges that cross
    (M, 256, M + 4 * 512, 512, True),
])
def test_rows(x, xs, out, os, ok):
    assert rows(x, xs, out, os) == (CUDA if ok else INVALID)
    if x != out and xs == os:
        assert rows(out, os, x, xs) == (CUDA if ok else INVALID)


def test_one_row():
    assert rows(M, 1 << 20, M + 256, 128, n=1) == CUDA and rows(M, 128, M + 240, 128, n=1) == INVALID


def test_group_attn():
    cache, N = lib._Cache(16, 16, None, None, 4), 3
    need = lib.group_attn_workspace_bytes(N, 1)
    q, o = N * 16 * 576 * 2, N * 16 * 576 * 4
    at, place = 1 << 32, {}
    for name, size in (("q", q), ("o", o), ("l", N * 64), ("out", q), ("lse", N * 64), ("ws", need)):
        place[name] = (at, size)
        at += (size + 255) // 256 * 256                  # neighbours

    def call(own=True, nb=need, scale=0.1, **moved):
        a = {k: moved.get(k, v[0]) for k, v in place.items()}
        return lib._L.csa2_group_attn(a["q"], N, 16, 576, ctypes.byref(cache), 16, 1, 2, 16, 16, scale,
                                      a["o"] if own else None, a["l"] if own else None, a["out"], a["lse"], a["ws"],
                                      nb, None)

    assert call() == CUDA and call(own=False) == CUDA
    for out in ("out", "lse", "ws"):
        step = 256 if out == "ws" else 16
        for other, (base, size) in place.items():
            if other == out:
                continue
            assert call(**{out: base}) == INVALID, (out, other)
            last = base + (size - 1) // step * step
            assert call(**{out: last}) == INVALID, (out, other)
    assert call(own=False, out=place["o"][0]) == CUDA    # without an own part nothing is there
    assert call(nb=need - 1) == WORKSPACE and call(ws=0) == WORKSPACE and call(ws=place["ws"][0] + 128) == WORKSPACE
    assert call(scale=3e38) == INVALID                   # infinite in the base-2 domain
