"""LayerGroup's optional parts on the host (CPU): raw latents, unrotated queries and a shared context. The device
calls are replaced by recorders; the plan comes from the real library's csa2_plan."""
import pytest
import torch

from compressed_sparse_attention_quant_b200 import group, lib


class _Cache:
    def __init__(self, num_pages, device="cpu"):
        self.num_pages = num_pages


@pytest.fixture
def rec(monkeypatch):
    calls = []
    monkeypatch.setattr(lib, "PagedCache", _Cache)
    monkeypatch.setattr(lib, "workspace", lambda n, device="cpu": torch.empty(max(int(n), 256), dtype=torch.uint8))
    monkeypatch.setattr(lib, "sparse_attn_workspace_bytes", lambda B, Sq, k: 1024)
    monkeypatch.setattr(lib, "indexer_topk", lambda *a, out=None, ws=None: calls.append(("topk", a)))
    monkeypatch.setattr(lib, "sparse_attn_decode",
                        lambda q, *a, out=None, lse=None, ws=None: calls.append(("attn", q, out, lse)))
    monkeypatch.setattr(lib, "append_kv_rope", lambda *a: calls.append(("append",) + a))
    monkeypatch.setattr(lib, "rope_rows", lambda x, pos, rope, out=None: calls.append(("rope", x, pos, rope, out)))
    monkeypatch.setattr(lib, "group_attn", lambda *a, **k: calls.append(("group", a, k)))
    return calls


ROPE, IDX_ROPE = object(), object()


def _group(modes=("F", "U"), B=2, Sq=3, **kw):
    return group.LayerGroup(modes, B, Sq, 4, 8, top_k=4, device="cpu", **kw)


def _args(B=2, Sq=3, layers=2):
    q = [torch.zeros(B, Sq, lib.HEADS, lib.DIM, dtype=torch.bfloat16) for _ in range(layers)]
    return (None, None, q, [None] * layers, {0: None}, {0: None})


def _shared(tokens, pages=2):
    return group.SharedContext(torch.zeros(len(tokens), pages, dtype=torch.int32),
                               torch.zeros(len(tokens), dtype=torch.int32), tokens)


def test_order_and_tensors(rec):
    g = _group(rope=ROPE, idx_rope=IDX_ROPE)
    args, pos, sh = _args(), torch.arange(6, dtype=torch.int32), _shared([4, 0, 2])
    x, xp, slots, k = (torch.zeros(1) for _ in range(4))
    g.step(*args, positions=pos, raw_append={0: (x, xp, slots, k)}, shared=sh)
    assert [c[0] for c in rec] == ["append", "topk", "rope", "attn", "group", "rope", "attn", "group"]
    assert rec[0][1] is x and rec[0][4] is g.caches[0] and rec[0][5] is ROPE and rec[0][7] is IDX_ROPE
    rope, attn, grp = rec[2], rec[3], rec[4]
    assert rope[2] is pos and rope[3] is ROPE and rope[1].shape == (6, lib.HEADS, lib.DIM)
    # both attentions read the rotated rows, never the caller's
    assert attn[1] is g._q_rot and rope[4].data_ptr() == g._q_rot.data_ptr() == grp[1][0].data_ptr()
    assert attn[1].data_ptr() != args[2][0].data_ptr()
    # the group attention joins this layer's own part, from its own cache
    kw = grp[2]
    assert grp[1][1] is g.caches[0] and grp[1][2] is sh.page_table and grp[1][3] is sh.lens
    assert kw["o_own"].data_ptr() == g.out[0].data_ptr() == attn[2].data_ptr()
    assert kw["lse_own"].data_ptr() == g.lse[0].data_ptr()
    assert kw["out"].data_ptr() == g.joined[0].data_ptr() and kw["lse"].data_ptr() == g.joined_lse[0].data_ptr()
    assert rec[7][2]["out"].data_ptr() == g.joined[1].data_ptr() != g.joined[0].data_ptr()
    assert rec[7][2]["o_own"].data_ptr() == g.out[1].data_ptr()
    assert g.joined[0].dtype == torch.bfloat16 and sh.q_offsets.tolist() == [0, 4, 4, 6]


def test_without_options_nothing_new_is_called(rec):
    g = _group()
    args = _args()
    g.step(*args)
    assert [c[0] for c in rec] == ["topk", "attn", "attn"] and rec[1][1] is args[2][0] and g.joined == []


def test_raw_append_without_keys(rec):
    g = _group(rope=ROPE, idx_rope=IDX_ROPE)
    t = torch.zeros(1)
    g.step(*_args(), raw_append={0: (t, t, t, None)})
    assert rec[0][0] == "append" and rec[0][6] is None and rec[0][7] is None


def test_buffers_stay_where_they_are(rec):
    """A captured step holds their addresses."""
    g = _group(rope=ROPE)
    args, pos = _args(), torch.arange(6, dtype=torch.int32)
    g.step(*args, positions=pos, shared=_shared([6]))
    first = [g._q_rot.data_ptr(), g.joined[0].data_ptr(), rec[-1][2]["ws"].data_ptr()]
    g.step(*args, positions=pos, shared=_shared([1, 5]))
    g.step(*args, positions=pos, shared=_shared([6]))
    assert [g._q_rot.data_ptr(), g.joined[0].data_ptr(), rec[-1][2]["ws"].data_ptr()] == first


def test_refusals(rec):
    args, pos = _args(), torch.arange(6, dtype=torch.int32)
    with pytest.raises(ValueError, match="without a rope"):
        _group().step(*args, positions=pos)
    with pytest.raises(ValueError, match="without a rope"):
        _group().step(*args, raw_append={0: (None,) * 4})
    for tokens in ([5], [6, 1], [0]):
        with pytest.raises(ValueError, match="query tokens"):
            _group().step(*args, shared=_shared(tokens))
    with pytest.raises(ValueError, match="negative"):
        _shared([7, -1])
    with pytest.raises(ValueError, match="one of each per group"):
        group.SharedContext(torch.zeros(2, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), [3, 3])
    assert rec == []
