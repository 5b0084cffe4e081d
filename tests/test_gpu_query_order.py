"""A query (or a query's weights) that the kernel right in front writes reaches the sparse decode and the pool selection
whole, also when that kernel lets its successor start before its own end, as the joining kernels do: here their outputs
are the next kernel's queries or weights, in one buffer that changes hands every turn."""
import pytest
import torch

pytestmark = pytest.mark.gpu

H, DIM, PAGE = 16, 576, 64


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("n,T,k", [(64, 4096, 64), (5, 1000, 200), (1, 4096, 0)])
def test_joined_outputs_as_queries(n, T, k, captured):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from compressed_sparse_attention_quant_b200 import lib
    turns = 30
    g = torch.Generator().manual_seed(n)
    pages = T // PAGE + 1
    cache = lib.PagedCache(pages)
    lib.quant_kv_fp4(torch.randn(pages * PAGE, DIM, generator=g).to(torch.bfloat16).cuda(),
                     torch.arange(pages * PAGE, dtype=torch.int32).cuda(), cache)
    table = torch.arange(pages, dtype=torch.int32)[None].cuda()
    tables, lens = table.expand(n, -1).contiguous(), torch.full((n,), T, dtype=torch.int32).cuda()
    idx = torch.arange(k, dtype=torch.int32).view(1, 1, k).expand(n, 1, k).contiguous().cuda()
    swa = None if k else torch.randn(n, 128, DIM, generator=g).to(torch.bfloat16).cuda()
    offs = torch.tensor([0, n], dtype=torch.int32).cuda()
    qs = [(torch.randn(n, H, DIM, generator=g) * 3).to(torch.bfloat16).cuda() for _ in range(turns)]
    buf, lse = torch.empty(n, H, DIM, dtype=torch.bfloat16).cuda(), torch.empty(n, H).cuda()
    out, out_lse = [torch.zeros(n, 1, H, DIM).cuda() for _ in qs], torch.empty(n, 1, H).cuda()
    ws_g = lib.workspace(lib.group_attn_workspace_bytes(n, 1))
    ws = lib.workspace(max(256, lib.sparse_attn_workspace_bytes(n, 1, k)))

    def turn(q, o, between=lambda: None):
        lib.group_attn(q, cache, table, lens[:1], offs, 0.2, out=buf, lse=lse, ws=ws_g)
        between()
        lib.sparse_attn_decode(buf.view(n, 1, H, DIM), cache, tables, lens, idx, swa, 0.2, out=o, lse=out_lse, ws=ws)

    same_back_to_back(turn, qs, out, captured)
    assert lib.last_device_error() == 0


@pytest.mark.parametrize("captured", [False, True])
def test_merged_values_as_weights(captured):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from compressed_sparse_attention_quant_b200 import lib
    R, T, C, k, turns, parts = 16, 512, 256, 32, 30, 64
    B = 4 * R
    g = torch.Generator().manual_seed(3)
    pages = B * T // PAGE
    n = pages * PAGE
    cache = lib.PagedCache(pages)
    keys, sigma = lib.quant_indexer_fp8(torch.randn(n, 64, generator=g).to(torch.bfloat16).cuda())
    lib.quant_kv_fp4(torch.zeros(n, DIM, dtype=torch.bfloat16).cuda(), torch.arange(n, dtype=torch.int32).cuda(), cache,
                     keys, sigma)
    table = torch.arange(pages, dtype=torch.int32).view(B, -1).cuda()
    lens = torch.full((B,), T, dtype=torch.int32).cuda()
    pool = torch.arange(0, 2 * C, 2, dtype=torch.int32).view(1, 1, C).expand(B, 1, C).contiguous().cuda()
    q_idx, _ = lib.quant_indexer_fp8(torch.randn(B, 1, lib.IDX_HEADS, 64, generator=g).to(torch.bfloat16).cuda())
    o_parts = torch.randn(parts, R, H, DIM, generator=g).cuda()
    lses = [torch.randn(parts, R, H, generator=g).cuda() * 3 for _ in range(turns)]
    o, lse = torch.empty(R, H, DIM).cuda(), torch.empty(R, H).cuda()
    out = [torch.zeros(B, 1, k, dtype=torch.int32).cuda() for _ in lses]

    def turn(l, i, between=lambda: None):
        lib.lse_merge(o_parts, l, out=o, lse=lse)
        between()
        lib.indexer_pool_topk(q_idx, lse.view(B, 1, 4), cache, table, lens, pool, k, out=i)

    same_back_to_back(turn, lses, out, captured)
    assert lib.last_device_error() == 0


def same_back_to_back(turn, ins, outs, captured):
    """The turns one after the other on a stream give what each gives with a synchronisation in its middle."""
    for i, o in zip(ins, outs):
        turn(i, o, torch.cuda.synchronize)
    ref = [o.clone() for o in outs]

    def run():
        for i, o in zip(ins, outs):
            turn(i, o)

    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        run = graph.replay
    for _ in range(10):
        for o in outs:
            o.zero_()
        run()
        assert all(torch.equal(o, r) for o, r in zip(outs, ref))
