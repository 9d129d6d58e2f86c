"""The decode attention over a cache in 4 bits where calls and numbers are at their ends: scratch that a call does not
use, sizes of queries, scales and factors from one end of fp32 to the other."""
import numpy as np
import pytest
import torch

import fp4_ref as ref
import invariant_bi_gemm_gb300 as bg
from test_gpu_r_cache4 import attention64, case, i32, random_cache, rows_of, table_of, tolerance

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ scratch

@pytest.mark.parametrize("Hq,Hkv,D,lengths", [(32, 8, 128, [700]), (32, 8, 128, [2000]), (8, 1, 128, [1000] * 60),
                                              (8, 2, 64, [1, 1500, 600, 0, 513])])
def test_calls_that_merge_in_clusters_take_no_scratch(Hq, Hkv, D, lengths):
    """Their first call may be a captured one, and workspace_size says 0."""
    q, seq, pos, four, table = case(Hq, Hkv, D, 16, lengths)
    bound = max(lengths) - 1
    want = bg.BiAttention4(Hq, Hkv, D, 16).run(q, seq, pos, *four, table, 9000)
    att = bg.BiAttention4(Hq, Hkv, D, 16)
    assert att.workspace_size(len(lengths), bound) == 0 and att.workspace_size(len(lengths), 9000) > 0
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att.run(q, seq, pos, *four, table, bound, o=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert att.device_error() == bg.BI_GEMM_OK


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (8, 2, 64), (8, 1, 128), (16, 16, 64)])
def test_scratch_is_what_the_call_uses(Hq, Hkv, D):
    """Nothing for a single split or in clusters, and bytes of the first 512 tokens else; a call of them works on a
    handle that has that much, captured too."""
    att = bg.BiAttention4(Hq, Hkv, D, 16)
    slot = Hq * (D + 2) * 4
    small = 0
    for T in (1, 3, 20, 60, 200, 512, 600, 3000):
        for bound in (0, 511, 512, 1023, 1024, 2047, 2048, 40000):
            splits, got = bound // 512 + 1, att.workspace_size(T, bound)
            assert got in ((0,) if splits == 1 else (0, min(T, 512) * splits * slot))
            assert splits <= 4 or got > 0
            small += splits > 1 and got == 0
    assert small > 0 and att.workspace_size(3000, 600) == 512 * 2 * slot
    table, pages = table_of([64] * 4)
    four = random_cache(pages, 16, Hkv, D, 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((600, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    seq = (torch.arange(600, device="cuda") % 4).to(torch.int32)
    pos = (torch.arange(600, device="cuda") * 5 % 1024).to(torch.int32)
    want = att.run(q, seq, pos, *four, table, 1023)
    fresh = bg.BiAttention4(Hq, Hkv, D, 16)
    torch.cuda.synchronize()
    with pytest.raises(bg.BiGemmError) as e:
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            fresh.run(q, seq, pos, *four, table, 1023)
    assert e.value.code == bg.BI_GEMM_ERR_SCRATCH_LIMIT
    torch.cuda.synchronize()
    fresh.run(q[:512], seq[:512], pos[:512], *four, table, 1023)
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(want)
    with torch.cuda.graph(graph):
        fresh.run(q, seq, pos, *four, table, 1023, o=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
