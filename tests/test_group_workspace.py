"""The workspace of a LayerGroup's shared context (CPU): one for every number of groups that its steps see."""
import torch

from compressed_sparse_attention_quant_b200 import group, lib
from test_group_options import _args, _group, _shared, rec      # noqa: F401 (rec is a fixture)


def test_size_does_not_depend_on_the_groups():
    for n in (1, 3, 8, 64, 1 << 20):
        assert len({lib.group_attn_workspace_bytes(n, g) for g in (1, 2, 17, 512, 65535)}) == 1


def test_one_for_any_number_of_groups(rec, monkeypatch):
    made = []
    monkeypatch.setattr(lib, "workspace", lambda n, device="cpu": made.append(n) or torch.empty(n, dtype=torch.uint8))
    monkeypatch.setattr(lib, "group_attn_workspace_bytes", lambda N, G: 512 if G <= 65535 else 0)
    g = _group()
    made.clear()
    g.step(*_args(), shared=group.SharedContext(torch.zeros(65536, 1, dtype=torch.int32),
                                                torch.zeros(65536, dtype=torch.int32), [6] + [0] * 65535))   # refused later
    used = set()
    for tokens in ([6], [1, 5], [2, 2, 2], [1] * 6, [0, 6, 0], [6]):
        g.step(*_args(), shared=_shared(tokens))
        used.add(rec[-1][2]["ws"].data_ptr())
        assert rec[-1][2]["ws"].numel() >= 512
    assert len(used) == 1 and made == [0, 512]
