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


# ------------------------------------------------------------------ sizes

# The query's size, k_scale and the softmax's scale, whose product leaves scores of ordinary size; the last two
# queries are below the smallest factor's range, the last one of denormals.
SIZES = [(2.0 ** 100, 2.0 ** -64, 2.0 ** -34), (2.0 ** 120, 2.0 ** -60, 2.0 ** -58), (2.0 ** -100, 2.0 ** 64, 2.0 ** 38),
         (2.0 ** 60, 2.0 ** -1, 2.0 ** -57), (2.0 ** -120, 2.0 ** 64, 2.0 ** 58), (2.0 ** -128, 2.0 ** 64, 2.0 ** 62)]


@pytest.mark.parametrize("spread,ks,scale", SIZES)
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 4, 128), (8, 1, 64)])
def test_ordinary_scores_of_extreme_factors(spread, ks, scale, Hq, Hkv, D):
    q, seq, pos, four, table = case(Hq, Hkv, D, 16, [900, 2500, 37], 5, spread, lo=0x08, hi=0x10)
    att = bg.BiAttention4(Hq, Hkv, D, 16, scale=scale, k_scale=ks)
    o = att.run(q, seq, pos, *four, table, 2499)
    want, a, e, total = attention64(q, seq, pos, four, table, 16, scale, ks, 1.0)
    # (scores are of ordinary size, so that the weights' part of the tolerance is small)
    assert 0.25 < float(e.max()) < 256.0
    off = (o.double() - want).abs() - tolerance(want, a, e, total, D)
    assert off.max() <= 0, float(off.max())


def planted(q, four, table, n, page, seed):
    """Gives each query head of the first request a key of its own that all its dimensions agree with, at 6, among the
    n: [Hq] positions."""
    Hq, D = q.shape[1:]
    Hkv = four[0].shape[2]
    G = Hq // Hkv
    at = torch.from_numpy(np.random.default_rng(seed).permutation(n)[:Hq].copy()).cuda()
    for h in range(Hq):
        code = torch.where(torch.signbit(q[0, h]), 15, 7).to(torch.uint8)
        page_of, row = int(table[0, int(at[h]) // page]), int(at[h]) % page
        four[0][page_of, row, h // G] = code[0::2] | (code[1::2] << 4)
        four[1][page_of, row, h // G] = 0x40
    return at


@pytest.mark.parametrize("spread,ks,scale", [(1e30, 2.0 ** -60, None), (2.0 ** 125, 2.0 ** -40, None),
                                             (1e-30, 2.0 ** 64, 2.0 ** 50), (64.0, 1.0, 8.0),
                                             (2.0 ** 40, 2.0 ** 40, 2.0 ** 20)])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 4, 128), (8, 1, 64), (2, 2, 128)])
def test_one_key_takes_all_of_extreme_scores(spread, ks, scale, Hq, Hkv, D):
    """A key above the others by 1e2 to 1e37: the output is its value, rounded once to bf16 (2^-8) behind fp32 steps."""
    q, seq, pos, four, table = case(Hq, Hkv, D, 16, [2500], 7, spread, lo=0x30, hi=0x38)
    at = planted(q, four, table, 2500, 16, 1)
    att = bg.BiAttention4(Hq, Hkv, D, 16, scale=scale, k_scale=ks, v_scale=0.37)
    k, v = rows_of(four, table, 0, 2500, 16, ks, 0.37)
    for h in range(Hq):                      # the next score is below by far more than any rounding of either
        s = (k[:, h * Hkv // Hq] @ q[0, h].double()) * att.scale
        top, second = s.topk(2).values.tolist()
        size = float((k[:, h * Hkv // Hq].abs() @ q[0, h].double().abs()).max()) * att.scale
        assert s.argmax() == at[h] and top - second > 60 + 2.0 ** -16 * size
    o = att.run(q, seq, pos, *four, table, 2499)
    want = torch.stack([v[at[h], h * Hkv // Hq] for h in range(Hq)])
    assert ((o[0].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs()).all()


def test_a_factor_beyond_fp32():
    """Queries whose largest element meets keys of 0 and whose others, 2^-24 of it, decide: scores are finite, the
    factor from the products to them (2^129) is not."""
    Hq, Hkv, D, n = 8, 2, 64, 700
    table, pages = table_of([-(-n // 16)])
    four = random_cache(pages, 16, Hkv, D, 3, 0x30, 0x38)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = (torch.randn((1, Hq, D), generator=g, device="cuda").sign() * 2.0 ** 102).to(torch.bfloat16)
    at = planted(q, four, table, n, 16, 4)
    q[0, :, 0] = 2.0 ** 126
    four[0][..., 0] &= 0xF0                  # every key's element 0
    att = bg.BiAttention4(Hq, Hkv, D, 16, scale=2.0 ** -50, k_scale=2.0 ** 64)
    o = att.run(q, i32([0]), i32([n - 1]), *four, table, n - 1)
    _, v = rows_of(four, table, 0, n, 16, 1.0, 1.0)
    want = torch.stack([v[at[h], h * Hkv // Hq] for h in range(Hq)])
    assert ((o[0].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs()).all()
