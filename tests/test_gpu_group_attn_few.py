"""K12b: the form of the group attention for few tokens per group (a mean of 4 or less), and the border between the
forms. Against the formula in 64 bits, with the tolerances of the group attention's own test module: the additions of
a row's sum are counted there for blocks of 64 entries, (64 + T / 64) 2^-24. Here a key's sum takes one addition per
block of 112 and the 112 keys' sums eight more (five steps inside a warp, three over the quarters): T / 112 + 8,
fewer."""
import math

import pytest
import torch

from test_gpu_group_attn import DIM, H, PAGE, SCALE, Case, lib      # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("tokens,lens", [
    ([1], [111]), ([2], [112]), ([3], [113]), ([4], [224]), ([4], [225]), ([1], [48 + 112]), ([1, 2, 3, 4], [1, 15, 16, 17]),
    ([16, 0, 0, 0], [700, 5, 0, 0]),                     # more tokens than a row tile in this form
    ([4, 5, 3, 0, 7], [337, 1200, 0, 64, 2300]), ([3] * 60, [13 * i for i in range(60)]), ([4], [30000]), ([2, 1], [9000, 20000]),
    ([5, 4], [300, 500]), ([30, 1, 1], [300, 500, 10]), ([5], [600])])       # the other form: a mean above 4
def test_against_64_bits(lib, tokens, lens, own):
    c = Case(lib, tokens, lens, seed=sum(tokens) + lens[0])
    if own:
        c.with_own()
    out, lse = c.call()
    assert lib.last_device_error() == 0
    c.check(out, lse)


@pytest.mark.parametrize("scale,q_gain", [(3.0, 1.0), (-0.7, 1.0), (0.0, 1.0), (SCALE, 1e-6), (1e-6, 1e5), (SCALE, 0.0)])
@pytest.mark.parametrize("tokens", [1, 3, 4])
def test_scales_and_magnitudes(lib, scale, q_gain, tokens):
    c = Case(lib, [tokens], [1500], seed=3, q_gain=q_gain)
    c.check(*c.call(scale=scale), scale=scale)


@pytest.mark.parametrize("tokens", [1, 2, 3, 4])
def test_rising_maximum(lib, tokens):
    """Every page of entries beats the one before by more than the running reference lets pass, for some rows; the
    others see their maximum in the first entries."""
    c = Case(lib, [tokens], [PAGE * 24], seed=4)
    c.q = c.q.abs()
    c.q[:, 1::2] *= -1
    for p in range(24):
        page = int(c.table[0, p])
        x = torch.full((PAGE, DIM), (p + 1) * 0.25, dtype=torch.bfloat16)
        lib.quant_kv_fp4(x.cuda(), (page * PAGE + torch.arange(PAGE)).to(torch.int32).cuda(), c.cache)
    c.check(*c.call(scale=0.3), scale=0.3)


def test_a_row_with_nan_keeps_to_itself(lib):
    c = Case(lib, [4], [700], seed=7)
    ref, ref_lse = c.call()
    q = c.q.clone()
    q[2, 5, 100] = math.nan
    q[3, 0, 0] = math.inf
    out, lse = c.call(q=q)
    bad = torch.zeros(4, H, dtype=torch.bool)
    bad[2, 5] = bad[3, 0] = True
    assert torch.equal(out.cpu()[~bad], ref.cpu()[~bad]) and torch.equal(lse.cpu()[~bad], ref_lse.cpu()[~bad])
    assert torch.isnan(out.cpu()[2, 5].float()).all()


@pytest.mark.parametrize("bad", [-1, 1 << 20])
@pytest.mark.parametrize("at", [0, 2, 6])
def test_bad_page_is_left_out(lib, bad, at):
    c = Case(lib, [3], [400], seed=8)
    c.table[0, at] = bad
    out, lse = c.call()
    assert lib.status_string(lib.last_device_error()) == "CSA2_ERR_DEVICE_BOUNDS"
    c.check(out, lse, drop=(at,))


def test_every_page_bad(lib):
    """Rows without a key: zeros, or the own part."""
    c = Case(lib, [3], [400], seed=9)
    c.table[:] = -1
    out, lse = c.call()
    assert (out == 0).all() and torch.isinf(lse).all()
    c.with_own()
    out, lse = c.call()
    assert torch.equal(out.cpu(), c.own[0].to(torch.bfloat16))
    torch.testing.assert_close(lse.cpu(), c.own[1], rtol=2.0 ** -21, atol=0)     # once to base 2 and back
    lib.last_device_error()


def test_rows_behind_the_last_sequence(lib):
    c = Case(lib, [3, 1, 0], [100, 200, 50], before=2, after=3).with_own()
    out = torch.full((c.N, H, DIM), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.N, H), -2.0, device="cuda")
    c.call(out, lse)
    assert lib.last_device_error() == 0
    c.check(out, lse)
    for part in (slice(0, 2), slice(c.N - 3, c.N)):
        assert (out[part] == 3.0).all() and (lse[part] == -2.0).all()


def test_same_bits_in_a_graph(lib):
    c = Case(lib, [1, 4, 2], [3000, 0, 900], seed=12).with_own()
    q, table = c.q.cuda(), c.table.cuda()
    lens, offs = torch.tensor(c.lens, dtype=torch.int32).cuda(), torch.tensor(c.offs, dtype=torch.int32).cuda()
    own = [t.cuda() for t in c.own]
    ws = lib.workspace(lib.group_attn_workspace_bytes(c.N, 3))
    out, lse = torch.empty(c.N, H, DIM, dtype=torch.bfloat16).cuda(), torch.empty(c.N, H).cuda()
    ref, ref_lse = c.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.group_attn(q, c.cache, table, lens, offs, SCALE, *own, out=out, lse=lse, ws=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    lens.copy_(torch.tensor([10, 2900, 113], dtype=torch.int32))
    c.table[1] = c.table[0]
    table.copy_(c.table)
    c.lens = [10, 2900, 113]
    graph.replay()
    c.check(out, lse)
