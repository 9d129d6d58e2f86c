"""A batch of fixed size with empty places through the whole step in 4 bits: append, attention, product."""
import pytest
import torch

import invariant_bi_gemm_gb300 as bg
from test_gpu_r_cache4 import cos_sin, empty_cache4, i32, random_cache, table_of

pytestmark = pytest.mark.gpu


def blank(t, places):
    t = t.clone()
    t[places] = -1
    return t


@pytest.mark.parametrize("Hq,Hkv,D,page,inter,T", [(32, 8, 128, 16, False, 1), (32, 8, 128, 16, False, 37),
                                                   (16, 2, 64, 12, True, 90), (64, 8, 128, 16, False, 900),
                                                   (8, 8, 64, 16, True, 14000)])
def test_append_leaves_empty_places_alone(Hq, Hkv, D, page, inter, T):
    """Every third place is empty, requests out of range among them: the other tokens' rows and slots are those of a
    call without the empty ones, everything else stays, and nothing is reported.  Both forms of the append."""
    g = torch.Generator(device="cuda").manual_seed(T)
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(torch.bfloat16)
    qkv[::3] = float("nan")
    seq = (torch.arange(T, device="cuda") // 300).to(torch.int32)
    pos = (torch.arange(T, device="cuda") % 300).to(torch.int32)
    table, pages = table_of([-(-300 // page)] * -(-T // 300))
    rope, cs = bg.BiQkRope(Hq, Hkv, D, page, interleaved=inter), cos_sin(300, D)
    empty = torch.arange(T, device="cuda") % 3 == 0
    seq2, pos2 = seq.clone(), blank(pos, empty)
    seq2[::6], seq2[3::6] = 1 << 30, -7
    four = empty_cache4(pages, page, Hkv, D)
    q = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    rope.run4(qkv, None, None, cs, seq2, pos2, *four, table, q_out=q)
    assert rope.device_error() == bg.BI_GEMM_OK
    assert (q[empty] == 7.0).all()
    alone = empty_cache4(pages, page, Hkv, D)
    if T > 1:
        rows = (qkv[~empty], None, None, cs, seq[~empty], pos[~empty])
        assert torch.equal(q[~empty], rope.run4(*rows, *alone, table))
    assert all(torch.equal(a, b) for a, b in zip(four, alone))


def test_other_bad_places_beside_empty_ones_are_reported():
    Hq, Hkv, D, page, T = 4, 2, 64, 16, 6
    rope, cs = bg.BiQkRope(Hq, Hkv, D, page), cos_sin(64, D)
    qkv = torch.randn((T, 8 * D), device="cuda").to(torch.bfloat16)
    table = i32([[0, 1, -1, -1]])
    for seq, pos, bad in (([0] * 6, [-1, 0, -1, 1, 2, -1], False), ([0] * 6, [-1, 0, -2, 1, 2, -1], True),
                          ([0] * 6, [-1, 0, 40, 1, 2, -1], True), ([0, 1, 0, 0, 0, 0], [-1, 0, -1, 1, 2, 3], True)):
        rope.run4(qkv, None, None, cs, i32(seq), i32(pos), *empty_cache4(2, page, Hkv, D), table)
        assert rope.device_error() == (bg.BI_GEMM_ERR_INVALID_ARG if bad else bg.BI_GEMM_OK)
    # the append in bf16 has no empty places
    k, v = (torch.zeros((2, page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rope.run(qkv, None, None, cs, i32([0] * 6), i32([-1, 0, 3, 1, 2, 4]), k, v, table)
    assert rope.device_error() == bg.BI_GEMM_ERR_INVALID_ARG


def test_a_captured_step_of_a_padded_batch():
    """One graph of a fixed size serves batches with different places empty: the rows that are there have the bits of a
    call of their own, the empty ones project zeros, and nothing is reported."""
    Hq, Hkv, D, page, d, T = 16, 4, 64, 16, 512, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    qo = bg.BiQuant4(Hq * D)
    wo = qo.run((torch.randn((d, Hq * D), generator=g, device="cuda") * 0.05).to(torch.bfloat16))
    down = bg.BiGemm4(Hq * D, d)
    rope, att = bg.BiQkRope(Hq, Hkv, D, page), bg.BiAttention4(Hq, Hkv, D, page)
    lengths = [700, 3, 1030, 64, 17, 512, 1, 1500]
    table, pages = table_of([-(-n // page) for n in lengths])
    kept = random_cache(pages, page, Hkv, D, 6)
    cs = cos_sin(2048, D)
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(torch.bfloat16)
    full_seq, full_pos = i32(list(range(T))), i32([n - 1 for n in lengths])

    def step(qkv, seq, pos, four):
        q = rope.run4(qkv, None, None, cs, seq, pos, *four, table)
        o = att.run(q, seq, pos, *four, table, 1499)
        return down.run(*qo.run(o.view(-1, Hq * D)), *wo)

    want = step(qkv, full_seq, full_pos, [a.clone() for a in kept])
    seq, pos, four = full_seq.clone(), full_pos.clone(), [a.clone() for a in kept]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(qkv, seq, pos, four)
    for empty in ([], [0], [7, 2], [1, 3, 4, 5, 6], list(range(T))):
        there = [t for t in range(T) if t not in empty]
        pos.copy_(blank(full_pos, empty))
        for a, k in zip(four, kept):
            a.copy_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y[there], want[there]), empty
        assert (y[empty] == 0).all()
    assert rope.device_error() == att.device_error() == bg.BI_GEMM_OK
