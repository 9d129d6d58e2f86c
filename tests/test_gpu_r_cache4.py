"""The paged cache in 4 bits (include/bi_attention4.h, bi_qkrope_run4): the append against the bf16 append bit by bit,
attention against 64-bit sums over the values that the cache stands for, bits across batches and pages, places
that nothing may see, expansion, and the operators together."""
import ctypes
import math

import numpy as np
import pytest
import torch

import fp4_ref as ref
import invariant_bi_gemm_gb300 as bg
from gpu_util import Controls, stream_ptr
from test_gpu_p_streams import owner

pytestmark = pytest.mark.gpu
CPU = torch.device("cpu")


def host(t):
    return t.cpu().numpy()


def cos_sin(positions, rot):
    rate = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    a = torch.arange(positions, dtype=torch.float64)[:, None] * rate
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def table_of(counts, seed=0, spare=2):
    """Page tables with pages handed out in random order, -1 behind; and the number of pages."""
    r = np.random.default_rng(seed)
    total = sum(counts)
    order = r.permutation(total + spare).astype(np.int32)
    t = np.full((len(counts), max(max(counts), 1)), -1, np.int32)
    at = 0
    for i, n in enumerate(counts):
        t[i, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(t).cuda(), total + spare


def empty_cache4(pages, page, Hkv, D, fill=0xEE):
    return [torch.full((pages, page, Hkv, w), fill, dtype=torch.uint8, device="cuda") for w in (D // 2, D // 16) * 2]


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("Hq,Hkv,D,page,rot,inter,norm,T", [
    (64, 8, 128, 16, 128, False, True, 800), (64, 8, 128, 16, 64, True, False, 1300),
    (32, 8, 128, 16, 128, False, True, 1), (32, 8, 128, 16, 128, False, False, 70), (32, 8, 128, 12, 128, True, True, 33),
    (16, 2, 64, 5, 32, False, True, 77), (16, 2, 64, 16, 64, True, False, 9), (4, 4, 128, 8, 64, False, True, 40),
    (8, 1, 128, 32, 16, False, True, 21), (8, 8, 64, 64, 48, False, False, 130), (4, 4, 128, 7, 96, False, True, 50),
    (32, 8, 128, 16, 128, False, True, 4500), (8, 8, 64, 16, 32, False, True, 14000), (16, 2, 64, 12, 64, True, True, 20000),
])
def test_append_is_the_quantised_bf16_append(Hq, Hkv, D, page, rot, inter, norm, T):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").mul_(
        torch.exp2(torch.randint(-6, 6, (T, 1), generator=g, device="cuda").float())).to(torch.bfloat16)
    gq, gk = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)] if norm else (None, None)
    seqs = -(-T // 300)
    q_seq = (torch.arange(T, device="cuda") // 300).to(torch.int32)
    q_pos = (torch.arange(T, device="cuda") % 300 + 11).to(torch.int32)
    table, pages = table_of([-(-312 // page)] * seqs)
    rope = bg.BiQkRope(Hq, Hkv, D, page, rot, interleaved=inter)
    cs = cos_sin(320, rot)
    k, v = (torch.zeros((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = rope.run(qkv, gq, gk, cs, q_seq, q_pos, k, v, table)
    four = empty_cache4(pages, page, Hkv, D)
    q4 = rope.run4(qkv, gq, gk, cs, q_seq, q_pos, *four, table, k_scale=0.25, v_scale=0.37)
    assert rope.device_error() == bg.BI_GEMM_OK
    assert torch.equal(q4, q)
    slot = (table[q_seq.long(), q_pos.long() // page].long() * page + q_pos.long() % page)
    for cache, codes, scales, s in ((k, four[0], four[1], 0.25), (v, four[2], four[3], 0.37)):
        rows = host(cache.view(-1, Hkv, D)[slot].reshape(-1, D).float())
        want, byte = ref.quantise(rows, "nvfp4", s)
        assert np.array_equal(host(codes.view(-1, Hkv, D // 2)[slot]).reshape(-1, D // 2), ref.pack(want))
        assert np.array_equal(host(scales.view(-1, Hkv, D // 16)[slot]).reshape(-1, D // 16), byte)
        other = torch.ones(pages * page, dtype=torch.bool, device="cuda")
        other[slot] = False
        assert (codes.view(-1, Hkv, D // 2)[other] == 0xEE).all() and (scales.view(-1, Hkv, D // 16)[other] == 0xEE).all()


def test_append_of_infinities_and_denormals():
    Hq, Hkv, D, page = 2, 2, 64, 16
    x = torch.zeros((4, 6 * 64), dtype=torch.bfloat16, device="cuda")
    x[0, 128 + 3], x[1, 256 + 40], x[2, 128:] = float("inf"), float("nan"), 1e-39
    x[3] = 3e38
    table, pages = table_of([1])
    four = empty_cache4(pages, page, Hkv, D)
    rope = bg.BiQkRope(Hq, Hkv, D, page)
    cs = torch.cat([torch.ones(8, 32), torch.zeros(8, 32)], 1).cuda()     # no turn
    rope.run4(x, None, None, cs, i32([0] * 4), i32([0, 1, 2, 3]), *four, table)
    rows = table[0, 0].long() * page + torch.arange(4, device="cuda")
    for name, lo, codes, scales in (("k", 128, *four[:2]), ("v", 256, *four[2:])):
        want, byte = ref.quantise(host(x[:, lo:lo + 128].reshape(-1, 64).float()), "nvfp4")
        if name == "k":      # an infinity times a sine of zero is NaN in its partner as well
            ex = host(x[:, lo:lo + 128].reshape(-1, 64).float())
            ex[0, 35] = np.nan
            want, byte = ref.quantise(ex, "nvfp4")
        assert np.array_equal(host(codes.view(-1, Hkv, D // 2)[rows]).reshape(-1, D // 2), ref.pack(want)), name
        assert np.array_equal(host(scales.view(-1, Hkv, D // 16)[rows]).reshape(-1, D // 16), byte), name


def test_append_catches_bad_places():
    Hq, Hkv, D, page = 4, 2, 128, 16
    rope = bg.BiQkRope(Hq, Hkv, D, page)
    cs = cos_sin(64, D)
    table = i32([[0, -1, 9], [1, 2, 3]])
    qkv = torch.randn((6, 8 * D), device="cuda").to(torch.bfloat16)
    seq, pos = i32([0, 0, 0, 2, 1, 1]), i32([3, 17, 33, 0, -1, 64])     # fine, no page, page 9 of 4, no request, no position
    for T, bad in ((1, False), (6, True)):
        four = empty_cache4(4, page, Hkv, D)
        q = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        rope.run4(qkv[:T], None, None, cs, seq[:T], pos[:T], *four, table, q_out=q)
        assert rope.device_error() == (bg.BI_GEMM_ERR_INVALID_ARG if bad else bg.BI_GEMM_OK)
        assert (q[1:] == 7.0).all() and not (q[0] == 7.0).all()
        assert int((four[0].view(-1, Hkv, D // 2) != 0xEE).any(-1).any(-1).sum()) == 1
    for bad in (0.0, float("nan"), 2.0 ** 65):
        with pytest.raises(bg.BiGemmError):
            rope.run4(qkv, None, None, cs, seq, pos, *empty_cache4(4, page, Hkv, D), table, k_scale=bad)
    with pytest.raises(ValueError):
        rope.run4(qkv, None, None, cs, seq, pos, *empty_cache4(4, page, Hkv, 64), table)


# ------------------------------------------------------------------ attention

def random_cache(pages, page, Hkv, D, seed, lo=0x28, hi=0x44):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(2):
        out.append(torch.randint(0, 256, (pages, page, Hkv, D // 2), generator=g, device="cuda", dtype=torch.uint8))
        out.append(torch.randint(lo, hi, (pages, page, Hkv, D // 16), generator=g, device="cuda", dtype=torch.uint8))
    return out


def rows_of(four, table, b, n, page, ks, vs):
    """Keys and values of a request's first n positions, 64 bits [n, Hkv, D]."""
    pages = table[b, :-(-n // page)].long()
    out = []
    for codes, scales, s in ((four[0], four[1], ks), (four[2], four[3], vs)):
        c, sc = (a[pages].flatten(0, 1)[:n] for a in (codes, scales))
        grid = torch.tensor(np.concatenate([ref.GRID, -ref.GRID]), device="cuda")
        val = torch.stack([grid[(c & 15).long()], grid[(c >> 4).long()]], -1).flatten(-2)
        e4 = torch.tensor(ref.e4m3_value(np.arange(128)), device="cuda")
        out.append(val * e4[sc.long()].repeat_interleave(16, -1) * float(np.float32(s)))
    return out


def attention64(q, q_seq, q_pos, four, table, page, scale, ks, vs):
    """(result, sum of weighted sizes, largest sum of sizes of a score's products, sum of sizes of the values)"""
    T, Hq, D = q.shape
    o, a, e, total = (torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda") for _ in range(4))
    for t in range(T):
        n = int(q_pos[t]) + 1
        if n <= 0:
            continue
        k, v = rows_of(four, table, int(q_seq[t]), n, page, ks, vs)
        G = Hq // k.shape[1]
        k, v = k.repeat_interleave(G, 1).transpose(0, 1), v.repeat_interleave(G, 1).transpose(0, 1)
        x = q[t].double()[:, :, None]
        w = torch.softmax((k @ x)[..., 0] * scale, 1)
        o[t], a[t] = (w[:, None] @ v)[:, 0], (w[:, None] @ v.abs())[:, 0]
        e[t] = ((k.abs() @ x.abs())[..., 0] * scale).amax(1, keepdim=True)
        total[t] = v.abs().sum(1)
    return o, a, e, total


def tolerance(o, a, e, total, D):
    """Keys, values and queries are exact in f16 (the inputs below); a score's D / 16 products of sixteen and the factor
    are within (D / 16 + 4) 2^-22 of the sum of sizes, natural units, and so is a weight twice (it and the sum) with
    2^-21 for exp2 and its argument's roundings of at most 2^-23 |s| log2(e); weights round to f16, half a step 2^-11, or
    2^-25 against a largest one of 2^7 at least; sums of a split's quarter in 32-position steps, of four warps and of the
    splits: 2^-16 covers 2^-22 for each of up to 64 additions.  bf16 at the end, half a step 2^-8."""
    return 2.0 ** -8 * o.abs() + a * (2.0 ** -11 + 2 * ((D / 16 + 8) * 2.0 ** -22 * e) + 2.0 ** -16) + 2.0 ** -32 * total


def case(Hq, Hkv, D, page, lengths, seed=1, spread=1.0, **kw):
    table, pages = table_of([-(-n // page) for n in lengths], seed)
    four = random_cache(pages, page, Hkv, D, seed, **kw)
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    q = (torch.randn((len(lengths), Hq, D), generator=g, device="cuda") * spread).to(torch.bfloat16)
    return q, i32(list(range(len(lengths)))), i32([n - 1 for n in lengths]), four, table


SETS = [
    (32, 8, 128, 16, [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129]),
    (32, 8, 128, 16, [511, 512, 513, 0, 1023, 1024, 1025, 700, 5000]),
    (16, 2, 64, 12, [1, 0, 0, 100, 333, 2049, 4097]),
    (8, 1, 128, 5, [77, 640, 1281, 3]),
    (8, 8, 64, 64, [600, 64, 65]),
    (4, 4, 128, 8, [2000, 9]),
    (16, 8, 128, 32, [1500, 31, 0]),
    (2, 1, 64, 1, [40, 530]),
    (8, 1, 64, 1000, [999, 1000, 1001, 2100]),
]


@pytest.mark.parametrize("Hq,Hkv,D,page,lengths", SETS)
@pytest.mark.parametrize("split", [0, 128, 1024])
def test_attention(Hq, Hkv, D, page, lengths, split):
    q, seq, pos, four, table = case(Hq, Hkv, D, page, lengths)
    ks, vs = 0.25, 0.37
    att = bg.BiAttention4(Hq, Hkv, D, page, k_scale=ks, v_scale=vs, split_size=split)
    o = att.run(q, seq, pos, *four, table, max(lengths) - 1)
    assert att.device_error() == bg.BI_GEMM_OK
    want, a, e, total = attention64(q, seq, pos, four, table, page, att.scale, ks, vs)
    off = (o.double() - want).abs() - tolerance(want, a, e, total, D)
    assert off.max() <= 0, (float(off.max()), [int(i) for i in (off > 0).nonzero()[0]])
    for t, n in enumerate(lengths):
        if n == 0:
            assert (o[t] == 0).all()


@pytest.mark.parametrize("spread,lo,hi", [(8.0, 0x38, 0x50), (1e-3, 0x01, 0x20), (1e30, 0x08, 0x10), (1.0, 0x70, 0x7E)])
def test_attention_of_peaked_flat_and_extreme_scores(spread, lo, hi):
    """Scores that differ by thousands (one weight), by nothing, and scales at the ends of E4M3."""
    q, seq, pos, four, table = case(16, 4, 128, 16, [900, 2500, 37], 5, spread, lo=lo, hi=hi)
    ks = 2.0 ** -60 if spread > 1e20 else 2.0 ** -8 if lo >= 0x70 else 1.0
    att = bg.BiAttention4(16, 4, 128, 16, k_scale=ks)
    o = att.run(q, seq, pos, *four, table, 2499)
    want, a, e, total = attention64(q, seq, pos, four, table, 16, att.scale, ks, 1.0)
    assert torch.isfinite(o).all()
    off = (o.double() - want).abs() - tolerance(want, a, e, total, 128)
    if float(e.max()) * (128 / 16 + 8) * 2.0 ** -22 < 0.25:
        assert off.max() <= 0, float(off.max())


def test_growing_scores_move_the_reference():
    """Keys whose scores climb all along the context, by more and by less than the slack at a time."""
    Hq, Hkv, D, page, n = 4, 1, 64, 16, 3000
    table, pages = table_of([-(-n // page)])
    four = random_cache(pages, page, Hkv, D, 3)
    flat = table[0].long().repeat_interleave(page) * page + torch.arange(page, device="cuda").repeat(table.shape[1])
    at = torch.arange(flat.numel(), device="cuda")
    four[0].view(-1, Hkv, D // 2)[flat] = 0x22                                       # every element 1
    four[1].view(-1, Hkv, D // 16)[flat] = (1 + at // 25).clamp(max=126).to(torch.uint8)[:, None, None].expand(-1, 1, 4)
    q = torch.ones((1, Hq, D), dtype=torch.bfloat16, device="cuda") * torch.tensor([1.0, 0.25, -1.0, 4.0], device="cuda").to(
        torch.bfloat16)[None, :, None]
    att = bg.BiAttention4(Hq, Hkv, D, page)
    o = att.run(q, i32([0]), i32([n - 1]), *four, table, n - 1)
    want, a, e, total = attention64(q, i32([0]), i32([n - 1]), four, table, page, att.scale, 1.0, 1.0)
    assert ((o.double() - want).abs() <= tolerance(want, a, e, total, D)).all()


@pytest.mark.parametrize("Hq,Hkv,D,page", [(32, 8, 128, 16), (16, 2, 64, 12), (8, 1, 128, 5)])
def test_a_tokens_bits_do_not_depend_on_the_call(Hq, Hkv, D, page):
    """Alone, in any batch, at another index, with another bound, on other pages of another size."""
    lengths = [1300, 1, 513, 0, 700, 2600, 64, 1024, 33]
    q, seq, pos, four, table = case(Hq, Hkv, D, page, lengths)
    att = bg.BiAttention4(Hq, Hkv, D, page)
    whole = att.run(q, seq, pos, *four, table, 2599)
    for t, n in enumerate(lengths):
        one = att.run(q[t:t + 1], seq[t:t + 1], pos[t:t + 1], *four, table, max(n - 1, 0) + 5000 * (t % 2))
        assert torch.equal(one[0], whole[t]), t
    back = torch.arange(len(lengths) - 1, -1, -1, device="cuda")
    assert torch.equal(att.run(q[back], seq[back], pos[back], *four, table, 2599)[back], whole)
    # the same rows in pages of another size
    other = 24
    t2, pages2 = table_of([-(-n // other) for n in lengths], 9)
    moved = empty_cache4(pages2, other, Hkv, D, 0x7F)
    for b, n in enumerate(lengths):
        j = torch.arange(n, device="cuda")
        src = table[b, j // page].long() * page + j % page
        dst = t2[b, j // other].long() * other + j % other
        for a, c in zip(four, moved):
            c.view(-1, Hkv, c.shape[-1])[dst] = a.view(-1, Hkv, a.shape[-1])[src]
    assert torch.equal(bg.BiAttention4(Hq, Hkv, D, other).run(q, seq, pos, *moved, t2, 2599), whole)


@pytest.mark.parametrize("Hq,Hkv,page,split", [(32, 8, 16, 0), (8, 8, 12, 0), (64, 8, 16, 128), (48, 12, 64, 0), (32, 16, 1, 256)])
def test_large_calls_have_the_bits_of_small_ones(Hq, Hkv, page, split):
    """Batches whose blocks take four KV heads: ragged contexts, empty places, a token that cannot be served."""
    D = 128
    lengths = [1 + (37 * i * i) % 1500 for i in range(68)] + [0, 1501]
    q, seq, pos, four, table = case(Hq, Hkv, D, page, lengths, 3)
    att = bg.BiAttention4(Hq, Hkv, D, page, split_size=split)
    whole = att.run(q, seq, pos, *four, table, 1500)
    assert att.device_error() == bg.BI_GEMM_OK
    for t in (0, 1, 5, 13, 31, 40, 66, 67, 68, 69):
        one = att.run(q[t:t + 1], seq[t:t + 1], pos[t:t + 1], *four, table, max(lengths[t] - 1, 0))
        assert torch.equal(one[0], whole[t]), t
    some = torch.tensor([1, 40, 69], device="cuda")
    want, a, e, total = attention64(q[some], seq[some], pos[some], four, table, page, att.scale, 1.0, 1.0)
    assert ((whole[some].double() - want).abs() <= tolerance(want, a, e, total, D)).all()
    seq2, pos2 = seq.clone(), pos.clone()
    seq2[7], pos2[11] = 1000, 1501
    o = att.run(q, seq2, pos2, *four, table, 1500)
    assert att.device_error() == bg.BI_GEMM_ERR_INVALID_ARG
    served = torch.tensor([t for t in range(70) if t not in (7, 11)], device="cuda")
    assert torch.equal(o[served], whole[served])


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 64, 12), (16, 2, 128, 16), (4, 4, 128, 5), (8, 1, 64, 16), (2, 2, 64, 64)])
@pytest.mark.parametrize("longest", [1000, 2048])
def test_splits_that_merge_in_clusters(Hq, Hkv, D, page, longest):
    """Small calls of two to four splits, a block each: ragged contexts, empty places, tokens that cannot be served; the
    bits of calls with a larger bound, which merge in a second kernel, and of a captured call."""
    lengths = [longest, 1, 0, 512, 513, min(1025, longest), 37, 700, min(1536, longest), 2, 511, 999]
    q, seq, pos, four, table = case(Hq, Hkv, D, page, lengths, 6)
    att = bg.BiAttention4(Hq, Hkv, D, page)
    o = att.run(q, seq, pos, *four, table, longest - 1)
    assert att.device_error() == bg.BI_GEMM_OK
    assert torch.equal(o, att.run(q, seq, pos, *four, table, 9000))
    for t, n in enumerate(lengths):
        assert torch.equal(att.run(q[t:t + 1], seq[t:t + 1], pos[t:t + 1], *four, table, longest - 1)[0], o[t]), t
    want, a, e, total = attention64(q, seq, pos, four, table, page, att.scale, 1.0, 1.0)
    assert ((o.double() - want).abs() <= tolerance(want, a, e, total, D)).all()
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(o)
    with torch.cuda.graph(graph):
        att.run(q, seq, pos, *four, table, longest - 1, o=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, o)
    seq2, pos2 = seq.clone(), pos.clone()
    seq2[0], pos2[7] = -3, longest
    got = att.run(q, seq2, pos2, *four, table, longest - 1)
    assert att.device_error() == bg.BI_GEMM_ERR_INVALID_ARG
    served = torch.tensor([t for t in range(len(lengths)) if t not in (0, 7)], device="cuda")
    assert torch.equal(got[served], o[served])


def test_many_tokens_of_few_requests():
    """More tokens than one launch serves, several of one request at consecutive positions, empty places between."""
    Hq, Hkv, D, page = 8, 2, 64, 16
    table, pages = table_of([-(-900 // page)] * 3)
    four = random_cache(pages, page, Hkv, D, 2)
    T = 2500
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randn((T, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    seq = (torch.arange(T, device="cuda") % 3).to(torch.int32)
    pos = (torch.arange(T, device="cuda") % 850).to(torch.int32)
    pos[::7], seq[::7] = -1, -5
    att = bg.BiAttention4(Hq, Hkv, D, page)
    o = att.run(q, seq, pos, *four, table, 899)
    assert att.device_error() == bg.BI_GEMM_OK
    assert (o[::7] == 0).all()
    some = torch.tensor([1, 500, 1023, 1024, 1025, 2047, 2048, 2499], device="cuda")
    for t in some.tolist():
        assert torch.equal(att.run(q[t:t + 1], seq[t:t + 1], pos[t:t + 1], *four, table, 899)[0], o[t])
    want, a, e, total = attention64(q[some], seq[some], pos[some], four, table, page, att.scale, 1.0, 1.0)
    assert ((o[some].double() - want).abs() <= tolerance(want, a, e, total, D)).all()


def test_many_tokens_in_blocks_of_four_heads():
    """Three launches of such blocks, a captured call of them, and two handles at once on two streams."""
    Hq, Hkv, D, page, T = 16, 8, 128, 16, 1100
    table, pages = table_of([-(-1400 // page)] * 3)
    four = random_cache(pages, page, Hkv, D, 4)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((T, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    seq = (torch.arange(T, device="cuda") % 3).to(torch.int32)
    pos = (torch.arange(T, device="cuda") * 7 % 1399).to(torch.int32)
    pos[::11], seq[::11] = -1, 77
    att, other = (bg.BiAttention4(Hq, Hkv, D, page) for _ in range(2))
    o = att.run(q, seq, pos, *four, table, 1399)
    assert att.device_error() == bg.BI_GEMM_OK
    assert (o[::11] == 0).all()
    for t in (1, 300, 511, 512, 513, 1023, 1024, 1025, 1099):
        assert torch.equal(att.run(q[t:t + 1], seq[t:t + 1], pos[t:t + 1], *four, table, 1399)[0], o[t]), t
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(o)
    with torch.cuda.graph(graph):
        att.run(q, seq, pos, *four, table, 1399, o=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, h in enumerate((att, other)):
            with torch.cuda.stream(streams[k]):
                got[k].append(h.run(q, seq, pos, *four, table, 1399))
    torch.cuda.synchronize()
    assert all(torch.equal(x, o) for xs in got for x in xs)


def test_what_lies_behind_a_position_is_not_seen():
    """NaN scales in the same page behind the position, and in other pages."""
    q, seq, pos, four, table = case(32, 8, 128, 16, [100, 513, 7])
    att = bg.BiAttention4(32, 8, 128, 16)
    o = att.run(q, seq, pos, *four, table, 512)
    slot = torch.ones((four[0].shape[0] * 16,), dtype=torch.bool, device="cuda")
    for b, n in enumerate([100, 513, 7]):
        j = torch.arange(n, device="cuda")
        slot[table[b, j // 16].long() * 16 + j % 16] = False
    for a in (four[1], four[3]):
        a.view(-1, 8, 8)[slot] = 0x7F
    assert torch.equal(att.run(q, seq, pos, *four, table, 512), o)


@pytest.mark.parametrize("which", [1, 3])
def test_a_nan_block_reaches_its_tokens_alone(which):
    q, seq, pos, four, table = case(32, 8, 128, 16, [600, 600])
    att = bg.BiAttention4(32, 8, 128, 16)
    clean = att.run(q, seq, pos, *four, table, 599)
    four[which].view(-1, 8, 8)[int(table[0, 20]) * 16 + 3, 5, 2] = 0x7F     # position 323, KV head 5, dimensions 32 .. 47
    o = att.run(q, seq, pos, *four, table, 599)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, 20:24, slice(None) if which == 1 else slice(32, 48)] = True
    assert torch.equal(torch.isnan(o), hit)
    assert torch.equal(o[~hit], clean[~hit])


def test_queries_that_are_not_finite_and_zero_queries():
    q, seq, pos, four, table = case(8, 2, 64, 16, [50, 50])
    q[0, 3, 7], q[0, 6] = float("nan"), 0.0
    att = bg.BiAttention4(8, 2, 64, 16)
    o = att.run(q, seq, pos, *four, table, 49)
    assert torch.isnan(o[0, 3]).all() and not torch.isnan(o[1]).any() and not torch.isnan(o[0, 4:]).any()
    _, v = rows_of(four, table, 0, 50, 16, 1.0, 1.0)
    assert ((o[0, 6].double() - v[:, 1].mean(0)).abs() <= 2.0 ** -7 * v[:, 1].abs().mean(0)).all()
    tiny = bg.BiAttention4(8, 2, 64, 16, k_scale=2.0 ** -64)       # a factor that underflows
    assert torch.equal(tiny.run(q, seq, pos, *four, table, 49)[0, 6], o[0, 6])


def test_bad_places_are_reported():
    q, seq, pos, four, table = case(8, 2, 64, 16, [50, 40])
    att = bg.BiAttention4(8, 2, 64, 16)
    good = att.run(q, seq, pos, *four, table, 49)
    for s, p, tab, bound in (([0, 2], [49, 0], table, 49), ([0, 1], [49, -2], table, 49), ([0, 1], [49, 39], table, 40),
                             ([0, 1], [49, 64], table, 64), ([0, -1], [49, 3], table, 49)):
        o = att.run(q, i32(s), i32(p), *four, tab, bound)
        assert att.device_error() == bg.BI_GEMM_ERR_INVALID_ARG
        if bound >= 49:
            assert torch.equal(o[0], good[0])
        assert att.device_error() == bg.BI_GEMM_OK
    worse = table.clone()
    worse[1, 1], worse[1, 2] = -1, 1 << 30
    o = att.run(q, seq, pos, *four, worse, 49)
    assert att.device_error() == bg.BI_GEMM_ERR_INVALID_ARG and torch.equal(o[0], good[0])


def test_caches_past_32_bit_offsets():
    Hq, Hkv, D, page = 8, 2, 128, 64
    pages = (1 << 33) // (page * Hkv * D // 2) + 7                  # 8.6 GB of codes each
    four = [torch.empty((pages, page, Hkv, w), dtype=torch.uint8, device="cuda") for w in (D // 2, D // 16) * 2]
    n = 500
    used = torch.arange(pages - 8, pages, device="cuda", dtype=torch.int32)
    small = random_cache(8, page, Hkv, D, 4)
    for a, c in zip(four, small):
        a[used.long()] = c
    table = used[None].contiguous()
    q = torch.randn((1, Hq, D), device="cuda").to(torch.bfloat16)
    att = bg.BiAttention4(Hq, Hkv, D, page)
    want = att.run(q, i32([0]), i32([n - 1]), *small, i32([list(range(8))]), n - 1)
    assert torch.equal(att.run(q, i32([0]), i32([n - 1]), *four, table, n - 1), want)
    k, v = att.expand(*four, used)
    k2, v2 = att.expand(*small, i32(list(range(8))))
    assert torch.equal(k, k2) and torch.equal(v, v2)
    rope = bg.BiQkRope(Hq, Hkv, D, page)
    qkv = torch.randn((3, 12 * D), device="cuda").to(torch.bfloat16)
    seq, pos = i32([0] * 3), i32([60, 130, n])
    rope.run4(qkv, None, None, cos_sin(512, D), seq, pos, *four, table)
    rope.run4(qkv, None, None, cos_sin(512, D), seq, pos, *small, i32([list(range(8))]))
    for a, c in zip(four, small):
        assert torch.equal(a[used.long()], c)


# ------------------------------------------------------------------ expansion

@pytest.mark.parametrize("Hkv,D,page", [(8, 128, 16), (2, 64, 12), (1, 64, 5)])
def test_expand(Hkv, D, page):
    four = random_cache(9, page, Hkv, D, 1, 0, 0x7F)
    att = bg.BiAttention4(Hkv, Hkv, D, page, k_scale=0.5, v_scale=0.37)
    pages = i32([8, 0, 3, 3, -1, 5])
    k = torch.full((6, page, Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    att.expand(*four, pages, k, v)
    assert att.device_error() == bg.BI_GEMM_OK
    for out, codes, scales, s in ((k, four[0], four[1], 0.5), (v, four[2], four[3], 0.37)):
        assert (out[4] == 9.0).all()
        use = [0, 1, 2, 3, 5]
        c, sc = host(codes[pages[use].long()]), host(scales[pages[use].long()])
        unit = (ref.e4m3_value(sc).astype(np.float32) * np.float32(s)).astype(np.float32)
        val = np.concatenate([ref.GRID, -ref.GRID])[ref.unpack(c)].astype(np.float32) * np.repeat(unit, 16, -1)
        assert torch.equal(out[use].cpu(), torch.from_numpy(val).to(torch.bfloat16))
    att.expand(*four, i32([9, -2, 1]))
    assert att.device_error() == bg.BI_GEMM_ERR_INVALID_ARG


# ------------------------------------------------------------------ together

def test_a_prompt_a_chunk_and_decode_steps():
    """A prompt is attended in bf16 and cached in 4 bits; a second chunk attends its expanded pages; decode steps run
    on the codes, each against the bf16 decode attention over the expanded cache."""
    Hq, Hkv, D, page, n1, n2, steps = 32, 8, 128, 16, 200, 90, 6
    rope, att4 = bg.BiQkRope(Hq, Hkv, D, page), bg.BiAttention4(Hq, Hkv, D, page, k_scale=0.5, v_scale=0.5)
    pre, att = bg.BiPromptAttention(Hq, Hkv, D, page), bg.BiAttention(Hq, Hkv, D, page)
    total = n1 + n2 + steps
    table, pages = table_of([-(-total // page)])
    four = empty_cache4(pages, page, Hkv, D, 0)
    cs = cos_sin(total, D)
    g = torch.Generator(device="cuda").manual_seed(0)
    qkv = torch.randn((total, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(torch.bfloat16)
    compact = torch.arange(table.shape[1], device="cuda", dtype=torch.int32)[None].contiguous()
    for first, n in ((0, n1), (n1, n2)):
        pos = torch.arange(first, first + n, device="cuda", dtype=torch.int32)
        q = rope.run4(qkv[first:first + n], None, None, cs, torch.zeros_like(pos), pos, *four, table, 0.5, 0.5)
        k, v = att4.expand(*four, table[0])
        o = pre.run(q, i32([0, n]), i32([first]), k, v, compact, first + n - 1)
        for t in (0, n // 2, n - 1):       # the same tokens by the decode attentions
            one = (q[t:t + 1], i32([0]), pos[t:t + 1])
            a = att.run(*one, k, v, compact, first + n - 1)
            b = att4.run(*one, *four, table, first + n - 1)
            want, size, e, tot = attention64(*one, four, table, page, att4.scale, 0.5, 0.5)
            tol = tolerance(want, size, e, tot, D)
            assert ((b.double() - want).abs() <= tol).all()
            assert ((a.double() - want).abs() <= tol).all()
            assert ((o[t:t + 1].double() - want).abs() <= tol + 2.0 ** -8 * size).all()
    for i in range(steps):
        p = i32([n1 + n2 + i])
        q = rope.run4(qkv[n1 + n2 + i:n1 + n2 + i + 1], None, None, cs, i32([0]), p, *four, table, 0.5, 0.5)
        o = att4.run(q, i32([0]), p, *four, table, total - 1)
        want, size, e, tot = attention64(q, i32([0]), p, four, table, page, att4.scale, 0.5, 0.5)
        assert ((o.double() - want).abs() <= tolerance(want, size, e, tot, D)).all()
    assert rope.device_error() == att4.device_error() == bg.BI_GEMM_OK


def test_a_layers_step_in_4_bits():
    """Quantise, project, append, attend, quantise, project: the whole step captured into a graph and replayed on
    other inputs, with the bits of the calls one by one."""
    Hq, Hkv, D, page, d, T = 16, 4, 64, 16, 512, 5
    width = (Hq + 2 * Hkv) * D
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, d), generator=g, device="cuda").to(torch.bfloat16)
    qd, qo = bg.BiQuant4(d), bg.BiQuant4(Hq * D)
    wq = qd.run((torch.randn((width, d), generator=g, device="cuda") * 0.05).to(torch.bfloat16))
    wo = qo.run((torch.randn((d, Hq * D), generator=g, device="cuda") * 0.05).to(torch.bfloat16))
    up, down = bg.BiGemm4(d, width), bg.BiGemm4(Hq * D, d)
    rope, att = bg.BiQkRope(Hq, Hkv, D, page), bg.BiAttention4(Hq, Hkv, D, page)
    lengths = [700, 3, 1030, 64, 17]
    table, pages = table_of([-(-n // page) for n in lengths])
    four = random_cache(pages, page, Hkv, D, 6)
    cs = cos_sin(2048, D)
    seq, pos = i32(list(range(T))), i32([n - 1 for n in lengths])

    def step(x, four):
        qkv = up.run(*qd.run(x), *wq)
        q = rope.run4(qkv, None, None, cs, seq, pos, *four, table)
        o = att.run(q, seq, pos, *four, table, 1029)
        return down.run(*qo.run(o.view(T, Hq * D)), *wo)

    kept = [a.clone() for a in four]
    want = step(x, [a.clone() for a in kept])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(x, four)
    for f in (1.0, -0.5):
        x.mul_(f)
        for a, k in zip(four, kept):
            a.copy_(k)
        graph.replay()
        torch.cuda.synchronize()
        now = [a.clone() for a in kept]
        assert torch.equal(y, step(x, now))
        assert all(torch.equal(a, b) for a, b in zip(four, now))
    assert not torch.equal(y, want) and torch.isfinite(y).all()
    # a row's result does not depend on the rows around it
    full = step(x, [a.clone() for a in kept])
    seq_all, pos_all, T_all = seq, pos, T
    for t in range(T_all):
        seq, pos, T = seq_all[t:t + 1].contiguous(), pos_all[t:t + 1].contiguous(), 1
        assert torch.equal(step(x[t:t + 1].contiguous(), [a.clone() for a in kept])[0], full[t])


def test_workspace_graphs_and_streams():
    Hq, Hkv, D, page = 8, 2, 64, 16
    lengths = [3000, 20, 1500]
    q, seq, pos, four, table = case(Hq, Hkv, D, page, lengths)
    want = bg.BiAttention4(Hq, Hkv, D, page).run(q, seq, pos, *four, table, 2999)
    att = bg.BiAttention4(Hq, Hkv, D, page)
    assert att.workspace_size(3, 511) == 0 and att.workspace_size(3, 2999) > 0 and att.workspace_size(0, 10) == 0
    torch.cuda.synchronize()
    with pytest.raises(bg.BiGemmError) as e:           # a captured call that nothing made room for
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            att.run(q, seq, pos, *four, table, 2999)
    assert e.value.code == bg.BI_GEMM_ERR_SCRATCH_LIMIT
    torch.cuda.synchronize()
    att.run(q, seq, pos, *four, table, 2999)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = att.run(q, seq, pos, *four, table, 2999)
    att.run(q, seq, pos, *four, table, 200000)         # grows the workspace behind the graph's back
    for _ in range(3):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = att.run(q, seq, pos, *four, table, 2999, stream=s)
    s.synchronize()
    assert torch.equal(other, want)


def test_a_handle_dropped_right_behind_its_call():
    """Its workspace outlives the call: the results are those of a handle that stays."""
    Hq, Hkv, D, page = 8, 2, 64, 16
    lengths = [6000, 20, 5000, 6000]
    q, seq, pos, four, table = case(Hq, Hkv, D, page, lengths)
    att, pre = bg.BiAttention4(Hq, Hkv, D, page), bg.BiPromptAttention(Hq, Hkv, D, page)
    k, v = att.expand(*four, torch.arange(four[0].shape[0], device="cuda", dtype=torch.int32))
    keep = bg.BiAttention(Hq, Hkv, D, page)
    start, first = i32([0, 4]), i32([5996])
    calls = (lambda h: h.run(q, seq, pos, *four, table, 5999), lambda h: h.run(q, seq, pos, k, v, table, 5999),
             lambda h: h.run(q, start, first, k, v, table[:1].contiguous(), 5999))
    for call, handle, make in zip(calls, (att, keep, pre), (bg.BiAttention4, bg.BiAttention, bg.BiPromptAttention)):
        want = call(handle)
        torch.cuda.synchronize()
        for _ in range(5):
            assert torch.equal(call(make(Hq, Hkv, D, page)), want)


def test_steps_back_to_back_without_a_wait():
    """Appends and attentions queued right behind one another, with one split and with several: each step's result is
    that of the step on its own."""
    Hq, Hkv, D, page = 8, 2, 128, 16
    for n0 in (5, 600):
        rope, att = bg.BiQkRope(Hq, Hkv, D, page), bg.BiAttention4(Hq, Hkv, D, page)
        table, pages = table_of([-(-(n0 + 64) // page)])
        first = random_cache(pages, page, Hkv, D, 2)
        qkv = torch.randn((64, 12 * D), device="cuda").to(torch.bfloat16)
        cs = cos_sin(n0 + 64, D)
        out = []
        for wait in (False, True):
            four, got = [a.clone() for a in first], []
            torch.cuda.synchronize()
            for i in range(64):
                p = i32([n0 + i])
                q = rope.run4(qkv[i:i + 1], None, None, cs, i32([0]), p, *four, table)
                if wait:
                    torch.cuda.synchronize()
                got.append(att.run(q, i32([0]), p, *four, table, n0 + 63))
                if wait:
                    torch.cuda.synchronize()
            out.append(torch.cat(got))
        assert torch.equal(out[0], out[1])


def test_sizes_of_nothing_and_refusals():
    Hq, Hkv, D, page = 8, 2, 64, 16
    q, seq, pos, four, table = case(Hq, Hkv, D, page, [50, 40])
    att = bg.BiAttention4(Hq, Hkv, D, page)
    assert att.run(q[:0], seq[:0], pos[:0], *four, table, 49).shape == (0, Hq, D)
    assert (att.run(q, seq, i32([-1, -1]), *four, table, -1) == 0).all()
    assert att.device_error() == bg.BI_GEMM_OK
    k, v = att.expand(*four, i32([]))
    assert k.shape == (0, page, Hkv, D)
    good = dict(q=q, q_seq=seq, q_pos=pos, k_codes=four[0], k_scales=four[1], v_codes=four[2], v_scales=four[3],
                page_table=table, max_pos=49)
    for bad in (dict(q=q.float()), dict(q_seq=seq.long()), dict(k_scales=four[1][:1]), dict(v_codes=four[2].cpu()),
                dict(page_table=table[0]), dict(k_codes=four[0].view(torch.int8))):
        with pytest.raises(ValueError):
            att.run(**{**good, **bad})
    with pytest.raises(bg.BiGemmError):
        att.run(**{**good, "max_pos": -2})
    assert math.isclose(att.scale, D ** -0.5)


def test_the_appends_waits_end():
    """Failure injection (test controls): block 0 of the form for many tokens loads nothing; its waits end after 50 ms."""
    Hq, Hkv, D, page = 16, 8, 128, 16
    L, P, I64 = Controls().L, ctypes.c_void_p, ctypes.c_int64
    L.bi_ctl_qkrope_create.argtypes = [ctypes.POINTER(P), I64, I64, I64, I64, I64, ctypes.c_int32, ctypes.c_float]
    L.bi_ctl_qkrope_stall4.argtypes = [P, P, I64, I64, P, P, P, I64, P, P, P, P, P, P, ctypes.c_float, ctypes.c_float, I64, P,
                                       I64, I64, P, ctypes.c_uint64, P]
    L.bi_ctl_qkrope_get_device_error.argtypes, L.bi_ctl_qkrope_destroy.argtypes = [P, P], [P]
    rope = bg.BiQkRope(Hq, Hkv, D, page)
    T = rope.config["ring_from"] + 5
    table, pages = table_of([-(-T // page)])
    four = empty_cache4(pages, page, Hkv, D)
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), device="cuda").to(torch.bfloat16)
    cs, seq, pos = cos_sin(T, D), torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    q = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    h = P()
    assert L.bi_ctl_qkrope_create(ctypes.byref(h), Hq, Hkv, D, page, D, 0, 1e-6) == 0
    assert L.bi_ctl_qkrope_stall4(h, qkv.data_ptr(), T, qkv.shape[1], None, None, cs.data_ptr(), T, seq.data_ptr(),
                                  pos.data_ptr(), *[a.data_ptr() for a in four], 1.0, 1.0, pages, table.data_ptr(), 1,
                                  table.shape[1], q.data_ptr(), 50_000_000, stream_ptr()) == 0
    assert L.bi_ctl_qkrope_get_device_error(h, stream_ptr()) == bg.BI_GEMM_ERR_TIMEOUT
    assert L.bi_ctl_qkrope_get_device_error(h, stream_ptr()) == 0
    assert L.bi_ctl_qkrope_destroy(h) == 0
    assert torch.equal(rope.run4(qkv, None, None, cs, seq, pos, *four, table), rope.run4(qkv, None, None, cs, seq, pos, *four, table))
    assert rope.device_error() == bg.BI_GEMM_OK


def test_tensors_of_another_device_are_refused():
    """Pointers of another GPU never reach a kernel of the handle's."""
    q, seq, pos, four, table = case(8, 2, 64, 16, [50, 40])
    att, rope, quant, gemm = bg.BiAttention4(8, 2, 64, 16), bg.BiQkRope(8, 2, 64, 16), bg.BiQuant4(128), bg.BiGemm4(128, 64)
    codes, scales = quant.run(torch.zeros((3, 128), dtype=torch.bfloat16, device="cuda"))
    for op in (att, rope, quant, gemm):
        op._device += 1                        # (as if it had been made there)
    qkv = torch.zeros((2, 12 * 64), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: att.run(q, seq, pos, *four, table, 49), lambda: att.expand(*four, i32([0])),
                 lambda: rope.run4(qkv, None, None, cos_sin(64, 64), seq, pos, *four, table),
                 lambda: quant.run(torch.zeros((3, 128), dtype=torch.bfloat16, device="cuda")),
                 lambda: quant.expand(codes, scales), lambda: gemm.run(codes, scales, codes, scales)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("as_number", [False, True])
@pytest.mark.parametrize("which", ["quant", "expand", "gemm", "append", "attend", "pages"])
def test_outputs_belong_to_the_stream_that_writes_them(which, as_number):
    """Outputs that a call makes itself, on a stream that is not the current one: memory of that stream."""
    q, seq, pos, four, table = case(8, 2, 64, 16, [700, 40])
    att, rope, quant, gemm = bg.BiAttention4(8, 2, 64, 16), bg.BiQkRope(8, 2, 64, 16), bg.BiQuant4(256), bg.BiGemm4(256, 96)
    x = torch.randn((5, 256), device="cuda").to(torch.bfloat16)
    codes, scales = quant.run(x)
    w, sw = quant.run(torch.randn((96, 256), device="cuda").to(torch.bfloat16))
    qkv, cs = torch.randn((2, 12 * 64), device="cuda").to(torch.bfloat16), cos_sin(704, 64)
    calls = {"quant": lambda s: quant.run(x, stream=s)[:1], "expand": lambda s: [quant.expand(codes, scales, stream=s)],
             "gemm": lambda s: [gemm.run(codes, scales, w, sw, stream=s)],
             "append": lambda s: [rope.run4(qkv, None, None, cs, seq, pos, *four, table, stream=s)],
             "attend": lambda s: [att.run(q, seq, pos, *four, table, 699, stream=s)],
             "pages": lambda s: att.expand(*four, table[1, :3].contiguous(), stream=s)}
    call = calls[which]
    want = [o.clone() for o in call(None)]
    torch.cuda.synchronize()
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    for o in [*call(None), *call(current), *call(current.cuda_stream)]:
        assert owner(o) == current.cuda_stream
    torch.cuda.synchronize()
    got = call(side.cuda_stream if as_number else side)
    side.synchronize()
    for o, was in zip(got, want):
        assert owner(o) == side.cuda_stream and torch.equal(o, was)
