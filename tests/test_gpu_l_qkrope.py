"""Per-head norm, rotation and cache append (include/bi_qkrope.h) on the GPU against the
definition in fp64, every element: head shapes, partial rotation, both pairings, with and without
weights, strided rows, page sizes, one token and many; independence of the batch; bad inputs;
untouched slots; streams and graphs.

Tolerance: the output is one bf16 rounding (2^-8 of the value) of fp32 arithmetic.  Before it, with
u = 2^-24: the sum of squares is off by at most 12 u (eight fma, four adds), the division, the
added eps and the reciprocal square root leave 9 u on r, two products 2 u more, the rotation's
product and fma 2 u of each of its two terms: under 16 u (|y_a| + |y_b|) = 2^-20 (|y_a| + |y_b|)."""
import numpy as np
import pytest
import torch

import invariant_bi_gemm_gb300 as bg
from invariant_bi_gemm_gb300 import BiQkRope

pytestmark = pytest.mark.gpu
EPS = float(np.float32(1e-6))


def make(T, Hq, Hkv, D, page, rot, seed=1, far=700, pad=0, norm=True, seqs=3):
    """T tokens spread over `seqs` requests at distinct random positions below `far`."""
    g = torch.Generator().manual_seed(seed)
    W = (Hq + 2 * Hkv) * D
    qkv = (3 * torch.randn(T, W + pad, generator=g)).to(torch.bfloat16).cuda()[:, :W]
    pick = torch.randperm(seqs * far, generator=g)[:T]
    q_seq, q_pos = (pick // far).to(torch.int32).cuda(), (pick % far).to(torch.int32).cuda()
    per = -(-far // page)
    table = torch.randperm(seqs * per + 2, generator=g)[:seqs * per].view(seqs, per).to(torch.int32).cuda()
    rate = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    ang = torch.arange(far, dtype=torch.float64)[:, None] * rate
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    kc = torch.randn(seqs * per + 2, page, Hkv, D, generator=g).to(torch.bfloat16).cuda()
    vc = torch.randn(seqs * per + 2, page, Hkv, D, generator=g).to(torch.bfloat16).cuda()
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() if norm else None for _ in range(2)]
    return dict(qkv=qkv, gq=w[0], gk=w[1], cos_sin=cs, q_seq=q_seq, q_pos=q_pos, k_cache=kc, v_cache=vc,
                page_table=table)


def reference(a, Hq, Hkv, D, page, rot, interleaved):
    """(value, bound) of the query rows and of the key rows, in fp64, and the slots."""
    x = a["qkv"].double().reshape(-1, Hq + 2 * Hkv, D)
    pos = a["q_pos"].long()
    cs = a["cos_sin"].double()[pos]
    co, si = cs[:, None, :rot // 2], cs[:, None, rot // 2:]

    def head(y, g):
        if g is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * g.double()
        v, size = y.clone(), y.abs()
        ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
        ib = ia + 1 if interleaved else ia + rot // 2
        v[..., ia], v[..., ib] = y[..., ia] * co - y[..., ib] * si, y[..., ib] * co + y[..., ia] * si
        both = y[..., ia].abs() + y[..., ib].abs()
        size[..., ia], size[..., ib] = both, both
        return v, 2.0**-8 * v.abs() + 2.0**-20 * size

    slot = a["page_table"][a["q_seq"].long(), pos // page].long() * page + pos % page
    return head(x[:, :Hq], a["gq"]), head(x[:, Hq:Hq + Hkv], a["gk"]), a["qkv"].reshape(x.shape)[:, Hq + Hkv:], slot


@pytest.mark.parametrize("T,Hq,Hkv,D,page,rot,inter,norm,pad", [
    (1, 32, 8, 128, 16, 128, False, True, 0),
    (37, 32, 8, 128, 16, 128, False, True, 64),
    (700, 32, 8, 128, 16, 64, True, True, 0),
    (333, 16, 2, 64, 7, 64, False, True, 8),
    (65, 16, 2, 64, 32, 32, True, False, 0),
    (64, 8, 1, 128, 5, 16, False, True, 0),
    (5, 1, 1, 64, 1, 16, True, True, 0),
    (130, 40, 40, 128, 64, 96, False, True, 0),          # more heads than a block holds at once
    (9, 3, 1, 64, 12, 48, False, False, 24),
    (6001, 16, 4, 64, 16, 64, False, True, 8),           # many tokens, and the form for them
    (5000, 8, 2, 128, 7, 64, True, True, 0),
    (4001, 2, 1, 64, 32, 32, True, False, 0),
    (8900, 16, 4, 64, 16, 64, False, True, 8),
    (8903, 8, 2, 128, 7, 64, True, True, 0),
    (2500, 32, 8, 128, 16, 128, False, True, 0),
    (49001, 2, 1, 64, 32, 32, True, False, 0),
])
def test_every_element(T, Hq, Hkv, D, page, rot, inter, norm, pad):
    a = make(T, Hq, Hkv, D, page, rot, norm=norm, pad=pad, far=max(2500, T // 3 + 1))
    kc0, vc0 = a["k_cache"].clone(), a["v_cache"].clone()
    h = BiQkRope(Hq, Hkv, D, page, rot_dim=rot, eps=EPS, interleaved=inter)
    q = h.run(**a)
    assert h.device_error() == 0
    (vq, tq), (vk, tk), v, slot = reference(a, Hq, Hkv, D, page, rot, inter)
    flat_k, flat_v = a["k_cache"].view(-1, Hkv, D), a["v_cache"].view(-1, Hkv, D)
    assert bool(((q.double() - vq).abs() <= tq).all())
    assert bool(((flat_k[slot].double() - vk).abs() <= tk).all())
    assert torch.equal(flat_v[slot], v)
    # every other slot as it was
    rest = torch.ones(flat_k.shape[0], dtype=torch.bool, device="cuda")
    rest[slot] = False
    assert torch.equal(flat_k[rest], kc0.view(-1, Hkv, D)[rest])
    assert torch.equal(flat_v[rest], vc0.view(-1, Hkv, D)[rest])
    h.close()


def test_token_independent_of_its_batch():
    """Each token alone gives the bits it has among 300 others."""
    a = make(300, 32, 8, 128, 16, 128)
    h = BiQkRope(32, 8, 128, 16, eps=EPS)
    q = h.run(**a)
    kc = a["k_cache"].clone()
    for t in (0, 1, 77, 299):
        b = dict(a, qkv=a["qkv"][t:t + 1], q_seq=a["q_seq"][t:t + 1], q_pos=a["q_pos"][t:t + 1])
        assert torch.equal(h.run(**b)[0].view(torch.int16), q[t].view(torch.int16))
    assert torch.equal(a["k_cache"].view(torch.int16), kc.view(torch.int16))
    h.close()


def test_token_independent_of_the_form():
    """Tokens of a call large enough for the form for many tokens, alone and in calls on both sides of
    the border between the forms: the same bits; bad tokens among them are reported and left out."""
    h = BiQkRope(16, 2, 64, 16, eps=EPS)
    border = h.config["ring_from"]
    a = make(border + 3, 16, 2, 64, 16, 64, far=4000)
    q = h.run(**a).clone()
    kc = a["k_cache"].clone()
    cut = lambda lo, hi: dict(a, qkv=a["qkv"][lo:hi], q_seq=a["q_seq"][lo:hi], q_pos=a["q_pos"][lo:hi])
    for lo, hi in ((0, 1), (border, border + 3), (3, border + 2), (3, border + 3)):
        assert torch.equal(h.run(**cut(lo, hi)).view(torch.int16), q[lo:hi].view(torch.int16)), (lo, hi)
    assert torch.equal(a["k_cache"].view(torch.int16), kc.view(torch.int16)) and h.device_error() == 0
    bad = dict(a, q_seq=a["q_seq"].clone())
    bad["q_seq"][[5, border]] = -1
    out = torch.full_like(q, 7.0)
    h.run(**bad, q_out=out)
    assert h.device_error() == bg.BI_GEMM_ERR_INVALID_ARG
    keep = torch.ones(border + 3, dtype=torch.bool)
    keep[[5, border]] = False
    assert bool((out[~keep] == 7).all()) and torch.equal(out[keep].view(torch.int16), q[keep].view(torch.int16))
    h.close()


def test_infinities_and_nan_stay_in_their_head():
    a = make(20, 8, 2, 64, 16, 64)
    h = BiQkRope(8, 2, 64, 16, eps=EPS)
    clean = h.run(**a).clone()
    a["qkv"].view(20, 12, 64)[3, 1, 5] = float("nan")
    a["qkv"].view(20, 12, 64)[3, 2, 6] = float("inf")
    a["qkv"].view(20, 12, 64)[4, 0] = 0.0
    q = h.run(**a)
    assert bool(q[3, 1].isnan().all()) and bool(q[3, 2].isnan().any())
    assert bool((q[4, 0] == 0).all())
    keep = torch.ones(20, 8, dtype=torch.bool)
    keep[3, 1] = keep[3, 2] = keep[4, 0] = False
    assert torch.equal(q[keep], clean[keep])
    h.close()


@pytest.mark.parametrize("what", ["seq", "negative", "far", "page", "pages"])
def test_bad_tokens_are_reported_and_write_nothing(what):
    a = make(40, 8, 2, 64, 16, 64)
    good = dict(a, q_seq=a["q_seq"].clone(), q_pos=a["q_pos"].clone(), page_table=a["page_table"].clone())
    if what == "seq":
        good["q_seq"][7] = 3
    elif what == "negative":
        good["q_pos"][7] = -1
    elif what == "far":
        good["q_pos"][7] = 700                        # behind the angles
    elif what == "pages":
        good["page_table"] = good["page_table"][:, :int(a["q_pos"].max()) // 16].contiguous()
    else:
        good["page_table"][a["q_seq"][7].long(), a["q_pos"][7].long() // 16] = -1
    h = BiQkRope(8, 2, 64, 16, eps=EPS)
    kc0 = a["k_cache"].clone()
    marked = torch.full((40, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q = h.run(**good, q_out=marked)
    assert h.device_error() == bg.BI_GEMM_ERR_INVALID_ARG and h.device_error() == 0
    if what != "pages":
        assert bool((q[7] == 7).all()) and not bool((q[8] == 7).all())
        (_, _), (_, _), _, slot = reference(a, 8, 2, 64, 16, 64, False)
        assert torch.equal(a["k_cache"].view(-1, 2, 64)[slot[7]], kc0.view(-1, 2, 64)[slot[7]])
    h.close()


def test_refusals():
    a = make(4, 8, 2, 64, 16, 64)
    h = BiQkRope(8, 2, 64, 16)
    for change in (dict(gq=None), dict(cos_sin=a["cos_sin"][:, :32]), dict(q_pos=a["q_pos"].long()),
                   dict(qkv=a["qkv"].float()), dict(k_cache=a["k_cache"][:, :8]), dict(q_seq=a["q_seq"][:3]),
                   dict(page_table=a["page_table"].t()), dict(v_cache=a["v_cache"].cpu())):
        with pytest.raises(ValueError):
            h.run(**dict(a, **change))
    wide = torch.zeros(4, 12 * 64 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bg.BiGemmError):
        h.run(**dict(a, qkv=wide[:, :12 * 64]))        # row pitch not 16 bytes
    with pytest.raises(bg.BiGemmError):
        h.run(**dict(a, qkv=torch.zeros(4 * 12 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, -1)))
    assert h.run(**dict(a, qkv=a["qkv"][:0], q_seq=a["q_seq"][:0], q_pos=a["q_pos"][:0])).shape == (0, 8, 64)
    h.close()


def test_stream_and_graph():
    """On a stream of its own, and captured and replayed on new contents: the bits of a plain call."""
    a = make(50, 32, 8, 128, 16, 128)
    h = BiQkRope(32, 8, 128, 16, eps=EPS)
    want = h.run(**a).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = h.run(**a)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    new = a["qkv"].flip(0).contiguous()
    kc, vc = a["k_cache"].clone(), a["v_cache"].clone()
    want2 = h.run(**dict(a, qkv=new, k_cache=kc, v_cache=vc)).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.run(**a, q_out=out)
    a["qkv"].copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2) and torch.equal(a["k_cache"], kc) and torch.equal(a["v_cache"], vc)
    assert h.device_error() == 0
    h.close()
