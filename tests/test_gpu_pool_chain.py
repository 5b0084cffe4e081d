"""Query quantisation and the candidate pool's selection back to back in one buffer: the selection starts before its
predecessor ends and must still see the codes that it writes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_quantised_queries_reach_the_selection():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from compressed_sparse_attention_quant_b200 import lib
    B, T, C, k, turns = 64, 512, 256, 32, 40
    g = torch.Generator().manual_seed(1)
    pages = B * T // 64
    cache = lib.PagedCache(pages)
    n = pages * 64
    keys, sigma = lib.quant_indexer_fp8(torch.randn(n, 64, generator=g).to(torch.bfloat16).cuda())
    lib.quant_kv_fp4(torch.zeros(n, 576, dtype=torch.bfloat16).cuda(), torch.arange(n, dtype=torch.int32).cuda(), cache,
                     keys, sigma)
    table = torch.arange(pages, dtype=torch.int32).view(B, -1).cuda()
    lens = torch.full((B,), T, dtype=torch.int32).cuda()
    pool = torch.arange(0, 2 * C, 2, dtype=torch.int32).view(1, 1, C).expand(B, 1, C).contiguous().cuda()
    w = torch.rand(B, 1, lib.IDX_HEADS, generator=g).cuda()
    qs = [torch.randn(B, 1, lib.IDX_HEADS, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(turns)]
    ref = []
    for q in qs:
        codes, _ = lib.quant_indexer_fp8(q)
        torch.cuda.synchronize()
        ref.append(lib.indexer_pool_topk(codes, w, cache, table, lens, pool, k))
    codes, sig = torch.zeros_like(codes), torch.zeros(B, 1, lib.IDX_HEADS).cuda()
    out = [torch.zeros(B, 1, k, dtype=torch.int32).cuda() for _ in qs]

    def run():
        for q, o in zip(qs, out):
            lib.quant_indexer_fp8(q, codes, sig)
            lib.indexer_pool_topk(codes, w, cache, table, lens, pool, k, out=o)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for call in (run, graph.replay):
        for _ in range(10):
            call()
            assert all(torch.equal(o, r) for o, r in zip(out, ref))
    assert lib.last_device_error() == 0
