"""Prompt attention (include/bi_prompt.h) on the GPU: every element against fp64 softmax attention
within a derived bound, over head shapes, lengths, chunks and page sizes; rows bitwise independent
of the packing, the chunk they came in, page placement and page size; values that are not finite
only where they are seen; bad inputs; untouched rows; streams and graphs.

Bound on |o - v| (w the exact weights, a = sum w |value|, e = max |score|, L keys, u = 2^-24):
bf16 rounding of the output 2^-8 |v|; each weight rounded to bf16 for the product but not in the
sum, 2^-9 relative at random and 2^-8 at most: 2^-8 a; fp32 before it, as for the decode
attention: 4 (D + 8) u e a + 2 (L + 160) u a (L + 32 there; here the weights of up to 2^8 and the
rescalings of the sums add a rounding per block, at most L / 128 + 1, and 128 terms' order)."""
import numpy as np
import pytest
import torch

import invariant_bi_gemm_gb300 as bg
from invariant_bi_gemm_gb300 import BiPromptAttention

pytestmark = pytest.mark.gpu


class Pack:
    """Sequences (id, tokens, context before them): contents from (seed, id) alone, packed queries, a
    paged cache with shuffled pages whose unused slots hold NaN."""

    def __init__(self, seqs, Hq, Hkv, D, page, seed=5, page_seed=1, lead=0, tail=0):
        self.seqs, self.dims, self.page = seqs, (Hq, Hkv, D), page
        self.K, self.V, qs = [], [], []
        for sid, n, ctx in seqs:
            g = torch.Generator().manual_seed(seed * 1000 + sid)
            total = n + ctx
            self.K.append(torch.randn(total, Hkv, D, generator=g).to(torch.bfloat16))
            self.V.append(torch.randn(total, Hkv, D, generator=g).to(torch.bfloat16))
            q = torch.randn(total, Hq, D, generator=g).to(torch.bfloat16)
            qs.append(q[ctx:])
        counts = [-(-k.shape[0] // page) for k in self.K]
        order = torch.randperm(sum(counts) + 2, generator=torch.Generator().manual_seed(page_seed))
        self.kc = torch.full((len(order), page, Hkv, D), float("nan"), dtype=torch.bfloat16)
        self.vc = self.kc.clone()
        self.table = torch.full((len(seqs), max(max(counts), 1)), -1, dtype=torch.int32)
        at = 0
        for b, c in enumerate(counts):
            ids = order[at:at + c]
            self.table[b, :c] = ids.to(torch.int32)
            at += c
            for i, pg in enumerate(ids.tolist()):
                part = slice(i * page, min((i + 1) * page, self.K[b].shape[0]))
                self.kc[pg, :part.stop - part.start] = self.K[b][part]
                self.vc[pg, :part.stop - part.start] = self.V[b][part]
        fill = torch.zeros(1, Hq, D, dtype=torch.bfloat16)
        self.q = torch.cat([fill.expand(lead, -1, -1)] + qs + [fill.expand(tail, -1, -1)])
        starts = np.cumsum([lead] + [n for _, n, _ in seqs])
        self.q_start = torch.tensor(starts, dtype=torch.int32)
        self.q_pos0 = torch.tensor([c for _, _, c in seqs], dtype=torch.int32)
        self.max_pos = max(max(n + c for _, n, c in seqs) - 1, 0)

    def args(self):
        return [x.cuda() for x in (self.q, self.q_start, self.q_pos0, self.kc, self.vc, self.table)] + [self.max_pos]

    def run(self, h, o=None):
        out = h.run(*self.args(), o=o)
        assert h.device_error() == 0
        return out

    def check(self, o, scale):
        Hq, Hkv, D = self.dims
        worst = 0.0
        for b, (_, n, ctx) in enumerate(self.seqs):
            if n == 0:
                continue
            lo = int(self.q_start[b])
            k, v = (x.cuda().double() for x in (self.K[b], self.V[b]))
            for h0 in range(Hkv):
                G = Hq // Hkv
                q = self.q[lo:lo + n, h0 * G:(h0 + 1) * G].cuda().double()
                s = torch.einsum("ngd,ld->ngl", q, k[:, h0]) * scale
                seen = torch.arange(n + ctx, device="cuda")[None] <= torch.arange(ctx, ctx + n, device="cuda")[:, None]
                s = s.masked_fill(~seen[:, None], -float("inf"))
                w = torch.softmax(s, -1)
                val = torch.einsum("ngl,ld->ngd", w, v[:, h0])
                a = torch.einsum("ngl,ld->ngd", w, v[:, h0].abs())
                e = s.masked_fill(~seen[:, None], 0).abs().amax(-1, keepdim=True)
                L = torch.arange(ctx + 1, ctx + n + 1, device="cuda").double()[:, None, None]
                u = 2.0**-24
                tol = 2.0**-8 * val.abs() + (2.0**-8 + 4 * (D + 8) * u * e + 2 * (L + 160) * u) * a
                err = (o[lo:lo + n, h0 * G:(h0 + 1) * G].double() - val).abs()
                assert bool((err <= tol).all()), (b, h0, float((err / tol).max()))
                worst = max(worst, float((err / tol).max()))
        return worst


def bits(x):
    return x.view(torch.int16)


@pytest.mark.parametrize("Hq,Hkv,D,page", [
    (32, 8, 128, 16), (8, 8, 64, 8), (16, 2, 64, 32), (8, 1, 128, 64), (4, 4, 128, 128), (16, 8, 128, 256),
    (8, 4, 64, 7), (8, 2, 128, 5), (4, 1, 64, 1), (2, 2, 128, 12), (8, 1, 64, 1000),
])
def test_every_element(Hq, Hkv, D, page):
    """Whole prompts of one token to several blocks, and chunks whose context ends anywhere."""
    seqs = [(0, 1, 0), (1, 37, 0), (2, 128, 0), (3, 129, 0), (4, 300, 0), (5, 1, 127), (6, 1, 128), (7, 5, 250),
            (8, 200, 77), (9, 64, 640), (10, 0, 30), (11, 257, 255)]
    pk = Pack(seqs, Hq, Hkv, D, page)
    h = BiPromptAttention(Hq, Hkv, D, page)
    worst = pk.check(pk.run(h), h.scale)
    h.close()
    print(f"prompt Hq={Hq} Hkv={Hkv} D={D} page={page}: max err/tol {worst:.3g}")


@pytest.mark.parametrize("Hq,Hkv,D,seqs", [
    (32, 8, 128, [(0, 2000, 0), (1, 1500, 3000)]),
    (16, 2, 64, [(0, 700, 9000), (1, 3000, 0), (2, 1, 12000)]),
    (4, 4, 128, [(0, 2500, 0)]),
])
def test_long(Hq, Hkv, D, seqs):
    pk = Pack(seqs, Hq, Hkv, D, 16)
    h = BiPromptAttention(Hq, Hkv, D, 16)
    pk.check(pk.run(h), h.scale)
    h.close()


@pytest.mark.parametrize("scale", [1e-3, 4.0])
def test_flat_and_sharp_scores(scale):
    """Scores near zero and scores of hundreds, whose running maximum climbs many times."""
    pk = Pack([(0, 700, 0), (1, 40, 400)], 8, 2, 128, 16)
    h = BiPromptAttention(8, 2, 128, 16, scale=scale)
    pk.check(pk.run(h), scale)
    h.close()


def test_climbing_maximum():
    """Keys that grow with their position: every block passes the reference and rescales."""
    pk = Pack([(0, 900, 0)], 8, 2, 64, 16)
    ramp = (1 + torch.arange(900) / 100)[:, None, None]
    pk.K[0] = (pk.K[0].float() * ramp).to(torch.bfloat16)
    for i in range(-(-900 // 16)):
        part = pk.K[0][16 * i:16 * i + 16]
        pk.kc[pk.table[0, i].long(), :len(part)] = part
    h = BiPromptAttention(8, 2, 64, 16, scale=0.5)
    pk.check(pk.run(h), 0.5)
    h.close()


def test_rows_independent_of_packing_pages_and_page_size():
    Hq, Hkv, D = 16, 4, 128
    target = (50, 333, 100)
    h16, h32, h7 = (BiPromptAttention(Hq, Hkv, D, ps) for ps in (16, 32, 7))
    golden = bits(Pack([target], Hq, Hkv, D, 16).run(h16))
    others = [(i, 1 + 97 * i % 500, 61 * i % 300) for i in range(9)]
    for at in (0, 4, 9):
        seqs = others[:at] + [target] + others[at:]
        for h, ps in ((h16, 16), (h32, 32), (h7, 7)):
            pk = Pack(seqs, Hq, Hkv, D, ps, page_seed=at + ps, lead=3, tail=5)
            lo = int(pk.q_start[at])
            assert torch.equal(bits(pk.run(h))[lo:lo + 333], golden), (at, ps)
    for h in (h16, h32, h7):
        h.close()


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (4, 4, 128), (8, 1, 64)])
def test_rows_independent_of_chunks(Hq, Hkv, D):
    """A prompt of 700 in one call, in uneven chunks and token by token at its ends: the same bits."""
    h = BiPromptAttention(Hq, Hkv, D, 16)
    whole = bits(Pack([(0, 700, 0)], Hq, Hkv, D, 16).run(h))
    for cut in ((0, 1, 2, 130, 384, 389, 698, 699, 700), (0, 64, 256, 700)):
        for lo, hi in zip(cut[:-1], cut[1:]):
            pk = Pack([(0, 700, 0)], Hq, Hkv, D, 16)
            # the cache as it is after this chunk: later positions hold NaN
            for i in range(-(-700 // 16)):
                for k in range(16):
                    if i * 16 + k >= hi:
                        pk.kc[pk.table[0, i].long(), k] = float("nan")
                        pk.vc[pk.table[0, i].long(), k] = float("nan")
            pk.q = pk.q[lo:hi].contiguous()
            pk.q_start, pk.q_pos0 = torch.tensor([0, hi - lo], dtype=torch.int32), torch.tensor([lo], dtype=torch.int32)
            assert torch.equal(bits(pk.run(h)), whole[lo:hi]), (lo, hi)
    h.close()


def test_values_that_are_not_finite_count_where_they_are_seen():
    """One infinite and one NaN value, in a block that is the diagonal for some rows and a whole
    block for others: rows before them are untouched, rows that see them carry them in that
    dimension of that KV head alone.  A NaN key spoils the rows that see it."""
    Hq, Hkv, D, n = 8, 2, 64, 400
    pk = Pack([(0, n, 0)], Hq, Hkv, D, 16)
    h = BiPromptAttention(Hq, Hkv, D, 16)
    clean = pk.run(h)
    at = lambda p: (pk.table[0, p // 16].long(), p % 16)
    pk.vc[at(150)[0], at(150)[1], 1, 7] = float("inf")
    pk.vc[at(200)[0], at(200)[1], 1, 9] = float("nan")
    pk.vc[at(210)[0], at(210)[1], 1, 7] = float("-inf")
    o = pk.run(h)
    want_inf = torch.zeros(n, Hq, D, dtype=torch.bool)
    want_nan = want_inf.clone()
    want_inf[150:210, 4:, 7] = True
    want_nan[200:, 4:, 9] = True
    want_nan[210:, 4:, 7] = True
    assert torch.equal(o.cpu() == float("inf"), want_inf)
    assert torch.equal(o.cpu().isnan(), want_nan)
    rest = ~(want_inf | want_nan)
    assert torch.equal(bits(o.cpu()[rest]), bits(clean.cpu()[rest]))
    pk.kc[at(300)[0], at(300)[1], 0, 3] = float("nan")
    o = pk.run(h).cpu()
    assert bool(o[300:, :4].isnan().all()) and not bool(o[:300, :4].isnan().any())
    h.close()


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 128), (4, 2, 64), (8, 2, 128), (8, 1, 64), (8, 1, 128), (2, 2, 64)])
@pytest.mark.parametrize("page", [16, 12])
def test_infinite_values_in_whole_and_cut_tiles(Hq, Hkv, D, page):
    """An infinite value now and then, each in a dimension of its own, so that the rows of a warp add
    back different numbers of them, in tiles that leave whole and in tiles cut by the chunk's ends."""
    pk = Pack([(0, 300, 0), (1, 70, 45), (2, 33, 300)], Hq, Hkv, D, page)
    h = BiPromptAttention(Hq, Hkv, D, page)
    clean = pk.run(h).cpu()
    want = torch.zeros(clean.shape, dtype=torch.bool)
    for b, (_, n, ctx) in enumerate(pk.seqs):
        lo = int(pk.q_start[b])
        for k, p in enumerate(range(0, n + ctx, 37)):
            d = (29 * k) % D
            pk.vc[pk.table[b, p // page].long(), p % page, Hkv - 1, d] = float("inf")
            want[lo + max(p - ctx, 0):lo + n, Hq - Hq // Hkv:, d] = True
    o = pk.run(h).cpu()
    assert torch.equal(o == float("inf"), want)
    assert torch.equal(bits(o[~want]), bits(clean[~want]))
    h.close()


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 128), (2, 2, 64), (4, 2, 128), (8, 1, 64)])
def test_infinite_values_under_weights_of_zero_do_not_show_the_chunk(Hq, Hkv, D):
    """Scores so sharp that most weights underflow to zero, and infinite values of both signs and NaN
    under them: a row's bits are those of the whole prompt in every chunk, one that begins in a unit's
    second tile (position 130 of units of 256) among them."""
    n = 700
    pk = Pack([(0, n, 0)], Hq, Hkv, D, 16)
    for p, d, x in ((50, 7, "inf"), (127, 8, "-inf"), (128, 9, "inf"), (200, 10, "nan"), (300, 11, "-inf"),
                    (383, 12, "inf"), (390, 13, "inf"), (640, 14, "-inf")):
        pk.vc[pk.table[0, p // 16].long(), p % 16, :, d] = float(x)
    h = BiPromptAttention(Hq, Hkv, D, 16, scale=4.0)
    whole = pk.run(h)
    assert bool(whole.isinf().any()) and bool(whole.isnan().any())
    q = pk.q
    for lo, hi in ((130, 256), (130, 700), (1, 140), (128, 129), (127, 128), (255, 512), (385, 390), (300, 700), (641, 642)):
        pk.q = q[lo:hi].contiguous()
        pk.q_start, pk.q_pos0 = torch.tensor([0, hi - lo], dtype=torch.int32), torch.tensor([lo], dtype=torch.int32)
        assert torch.equal(bits(pk.run(h)), bits(whole[lo:hi])), (lo, hi)
    h.close()


def test_zeros_of_both_signs_do_not_show_the_chunk():
    """Values of minus zero, and values of either sign behind a row: the sign of a row's zeros does not
    depend on what stands in the cache behind it."""
    Hq, Hkv, D, n = 4, 4, 64, 200
    pk = Pack([(0, n, 0)], Hq, Hkv, D, 16)
    h = BiPromptAttention(Hq, Hkv, D, 16)
    at = lambda p: (pk.table[0, p // 16].long(), p % 16)
    got = []
    for sign in (1.0, -1.0):
        for p in range(n):
            pk.vc[at(p)[0], at(p)[1], :, 3] = -0.0 if p < 100 else sign
            pk.vc[at(p)[0], at(p)[1], :, 4] = 0.0 if p < 100 else sign
        got.append(bits(pk.run(h))[:100].clone())
    assert torch.equal(got[0], got[1])
    h.close()


def test_rows_outside_the_sequences_and_empty_calls():
    pk = Pack([(0, 70, 0), (1, 0, 0), (2, 30, 5)], 8, 2, 128, 16, lead=11, tail=23)
    h = BiPromptAttention(8, 2, 128, 16)
    o = torch.full_like(pk.q, 3.0).cuda()
    pk.check(pk.run(h, o), h.scale)
    assert bool((o[:11] == 3).all()) and bool((o[-23:] == 3).all())
    a = pk.args()
    assert h.run(a[0][:0], torch.zeros(4, dtype=torch.int32, device="cuda"), *a[2:]).shape[0] == 0
    h.close()


@pytest.mark.parametrize("what", ["descending", "past the end", "negative start", "negative position", "max_pos",
                                  "page", "pages"])
def test_bad_inputs_are_reported(what):
    """The bad sequence is reported; the others keep their bits and the handle goes on."""
    pk = Pack([(0, 70, 0), (1, 90, 64), (2, 30, 5)], 8, 2, 128, 16)
    h = BiPromptAttention(8, 2, 128, 16)
    good = bits(pk.run(h))
    q, qs, q0, kc, vc, table, mp = pk.args()
    if what == "descending":
        qs[2] = 60
    elif what == "past the end":
        qs[3] = 191
    elif what == "negative start":
        qs[0] = -1
    elif what == "negative position":
        q0[1] = -3
    elif what == "max_pos":
        mp = 100
    elif what == "page":
        table[1, 4] = 10**6
    else:
        table = table[:, :9].contiguous()
    o = torch.zeros_like(q)
    h.run(q, qs, q0, kc, vc, table, mp, o=o)
    assert h.device_error() == bg.BI_GEMM_ERR_INVALID_ARG and h.device_error() == 0
    if what in ("negative position", "max_pos", "page", "pages"):
        assert torch.equal(bits(o)[:70], good[:70]) and torch.equal(bits(o)[160:], good[160:])
    if what == "past the end":
        assert torch.equal(bits(o)[:160], good[:160]) and bool((o[160:] == 0).all())
    if what == "descending":                   # sequences that overlap: none is computed
        assert bool((o == 0).all())
    assert torch.equal(bits(pk.run(h)), good)
    h.close()


@pytest.mark.parametrize("num_seqs", [1, 3, 31, 33, 70])
def test_empty_sequences_around_and_the_plan(num_seqs):
    """A sequence keeps its bits among empty ones, in calls so small that no plan is made and in calls
    with one, wherever it stands."""
    rows = [(i, 0, 0) for i in range(num_seqs)]
    for at in {0, num_seqs // 2, num_seqs - 1}:
        for others in (0, 40):
            seqs = list(rows)
            seqs[at] = (at, 75, 30)
            pk = Pack(seqs + [(num_seqs + i, 90, 11 * i) for i in range(others)], 8, 1, 64, 16)
            one = Pack([(at, 75, 30)], 8, 1, 64, 16)
            h = BiPromptAttention(8, 1, 64, 16)
            q, qs, q0, kc, vc, table, mp = pk.args()
            got = bits(h.run(q, qs, q0, kc, vc, table, mp))
            lo, hi = int(pk.q_start[at]), int(pk.q_start[at + 1])
            alone = h.run(q[lo:hi].contiguous(), torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"),
                          q0[at:at + 1].contiguous(), kc, vc, table[at:at + 1].contiguous(), mp)
            assert h.device_error() == 0
            assert torch.equal(got[lo:hi], bits(alone)) and hi - lo == 75
            one.check(one.run(h), h.scale)
            h.close()


def test_refusals():
    pk = Pack([(0, 7, 0), (1, 9, 4)], 8, 2, 64, 16)
    h = BiPromptAttention(8, 2, 64, 16)
    a = pk.args()
    for i, bad in ((0, a[0].float()), (0, a[0][:, :4]), (0, a[0].transpose(0, 1)), (1, a[1][:2]), (1, a[1].long()),
                   (2, a[2][:1]), (3, a[3][:, :, :1]), (4, a[4].half()), (5, a[5].cpu()), (5, a[5][0])):
        with pytest.raises(ValueError):
            h.run(*(a[:i] + [bad] + a[i + 1:]))
    with pytest.raises(ValueError):
        h.run(*a, o=torch.zeros_like(a[0], dtype=torch.float32))
    with pytest.raises(bg.BiGemmError):
        h.run(torch.zeros(16 * 8 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(16, 8, 64), *a[1:])
    with pytest.raises(bg.BiGemmError):
        h.run(*a[:-1], -1)
    with pytest.raises(bg.BiGemmError):
        h.run(*a[:-1], 1 << 30)
    h.close()


def test_repeat_stream_and_graph():
    pk = Pack([(i, 50 + 31 * i, 17 * i) for i in range(12)], 32, 8, 128, 16)
    h = BiPromptAttention(32, 8, 128, 16)
    a = pk.args()
    want = bits(h.run(*a)).clone()
    for _ in range(20):
        assert torch.equal(bits(h.run(*a)), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = h.run(*a)
    side.synchronize()
    assert torch.equal(bits(got), want)
    # captured, then replayed with other lengths and other queries in the same buffers
    out = torch.zeros_like(a[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.run(*a, o=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), want)
    a[0].copy_(a[0].flip(0).contiguous())
    a[1][3:].copy_(a[1][3:] - 20)
    a[2][2] = 0
    fresh = BiPromptAttention(32, 8, 128, 16)
    want2 = torch.zeros_like(out)
    fresh.run(*a, o=want2)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(want2))
    assert h.device_error() == 0 and fresh.device_error() == 0
    h.close()
    fresh.close()
