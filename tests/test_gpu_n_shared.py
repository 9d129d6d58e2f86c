"""Decode attention over groups that share a prefix (bi_attention_run_shared) on the GPU: for every
call the bits of bi_attention_run on the same tokens (whose values the decode attention's tests hold
to the oracle), and fp64 attention for one call of each head dimension; groups of all sizes and
lengths, several tokens of one request, page and split sizes, values that are not finite, zeros of
both signs; bad groups; streams and graphs."""
import numpy as np
import pytest
import torch

import invariant_bi_gemm_gb300 as bg
from invariant_bi_gemm_gb300 import BiAttention

pytestmark = pytest.mark.gpu


class Groups:
    """groups: [(prefix, [own tokens of each request])]; pages of the prefix's whole pages in common,
    its rest copied; one query token per request at its last position; `more`: further (request,
    position) tokens placed at the end, outside every group."""

    def __init__(self, groups, Hq, Hkv, D, page, seed=3, more=()):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
        tables, lens, start, share = [], [], [0], []
        pages_k, pages_v = [], []
        order_at = 0

        def add(k, v):
            """Pages holding rows k, v; returns their ids."""
            nonlocal order_at
            n = -(-k.shape[0] // page)
            ids = list(range(order_at, order_at + n))
            order_at += n
            for i in range(n):
                for dst, src in ((pages_k, k), (pages_v, v)):
                    pg = torch.full((page, Hkv, D), float("nan"), dtype=torch.bfloat16)
                    part = src[i * page:(i + 1) * page]
                    pg[:len(part)] = part
                    dst.append(pg)
            return ids

        for prefix, owns in groups:
            k, v = rn(prefix, Hkv, D), rn(prefix, Hkv, D)
            whole = prefix // page
            common = add(k[:whole * page], v[:whole * page])
            for own in owns:
                mk, mv = rn(own, Hkv, D), rn(own, Hkv, D)
                rest = add(torch.cat([k[whole * page:], mk]), torch.cat([v[whole * page:], mv]))
                tables.append(common + rest)
                lens.append(prefix + own)
            start.append(start[-1] + len(owns))
            share.append(whole * page)
        perm = torch.randperm(order_at + 2, generator=g)
        self.kc = torch.full((order_at + 2, page, Hkv, D), float("nan"), dtype=torch.bfloat16)
        self.vc = self.kc.clone()
        self.kc[perm[:order_at]], self.vc[perm[:order_at]] = torch.stack(pages_k), torch.stack(pages_v)
        self.table = torch.full((len(tables), max(map(len, tables))), -1, dtype=torch.int32)
        for b, ids in enumerate(tables):
            self.table[b, :len(ids)] = perm[torch.tensor(ids, dtype=torch.long)].to(torch.int32)
        tokens = [(b, n - 1) for b, n in enumerate(lens)] + list(more)
        self.q_seq = torch.tensor([b for b, _ in tokens], dtype=torch.int32)
        self.q_pos = torch.tensor([p for _, p in tokens], dtype=torch.int32)
        self.q = rn(len(tokens), Hq, D)
        self.start, self.len = torch.tensor(start, dtype=torch.int32), torch.tensor(share, dtype=torch.int32)
        # (a bound that is loose enough for a call of few tokens to share as well)
        self.max_pos = max(int(self.q_pos.max()), 1024 * (1024 // (len(tokens) * Hkv) + 1))

    def args(self):
        return [x.cuda() for x in (self.q, self.q_seq, self.q_pos, self.kc, self.vc, self.table)] + [self.max_pos]

    def both(self, h):
        a = self.args()
        plain = h.run(*a)
        assert h.device_error() == 0
        shared = h.run_shared(*a, self.start.cuda(), self.len.cuda())
        assert h.device_error() == 0
        return bits(plain), bits(shared)


def bits(x):
    return x.view(torch.int16)


@pytest.mark.parametrize("Hq,Hkv,D,page,split", [
    (32, 8, 128, 16, 0), (32, 8, 128, 16, 128), (32, 8, 128, 64, 1024), (8, 1, 128, 32, 256), (4, 4, 128, 8, 512),
    (16, 8, 128, 128, 384), (16, 2, 64, 16, 0), (8, 8, 64, 32, 256), (8, 4, 64, 8, 1024), (16, 4, 64, 256, 128),
    (32, 8, 128, 5, 0), (16, 2, 64, 12, 128), (4, 4, 64, 1, 256), (8, 1, 128, 7, 640),
])
def test_bits_of_run(Hq, Hkv, D, page, split):
    """Groups of one, few and many tokens, prefixes below, at and above split borders, own tails over a
    border, and tokens in no group."""
    s = split or 512
    groups = [(2 * s + 37, [1, 5, s + 3, 40]), (s - 1, [1, 2]), (s, [1, 2, 3]), (3 * s, [7]),
              (s + page, [1 + 3 * i for i in range(37)]), (10, [4, 5])]
    gr = Groups(groups, Hq, Hkv, D, page, more=[(0, 2 * s + 30), (3, 5)])
    h = BiAttention(Hq, Hkv, D, page, split_size=split)
    plain, shared = gr.both(h)
    assert torch.equal(plain, shared)
    h.close()


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (16, 2, 64)])
def test_long_prefix_and_fp64(Hq, Hkv, D):
    gr = Groups([(9000, [1 + 17 * i for i in range(70)])], Hq, Hkv, D, 16)
    h = BiAttention(Hq, Hkv, D, 16)
    plain, shared = gr.both(h)
    assert torch.equal(plain, shared)
    o = shared.view(torch.bfloat16).double().cpu()
    for t in (0, 31, 69):
        L = int(gr.q_pos[t]) + 1
        slot = gr.table[t, torch.arange(L) // 16].long() * 16 + torch.arange(L) % 16
        k, v = (x.view(-1, Hkv, D)[slot].double().repeat_interleave(Hq // Hkv, 1) for x in (gr.kc, gr.vc))
        sc = torch.einsum("hd,lhd->hl", gr.q[t].double(), k) * D**-0.5
        w = torch.softmax(sc, 1)
        val, a = torch.einsum("hl,lhd->hd", w, v), torch.einsum("hl,lhd->hd", w, v.abs())
        u = 2.0**-24       # the decode attention's bound
        tol = 2.0**-8 * val.abs() + (4 * (D + 8) * u * sc.abs().amax(1, keepdim=True) + 2 * (L + 32) * u) * a
        assert bool(((o[t] - val).abs() <= tol).all())
    h.close()


def _page_factors(gr, page, f):
    """Multiplies every page's keys by f(position of its first slot)."""
    k = gr.kc.float()
    done = set()
    for row in gr.table.tolist():
        for i, pg in enumerate(row):
            if pg >= 0 and pg not in done:
                done.add(pg)
                k[pg] *= f(i * page)
    gr.kc = k.to(torch.bfloat16)


@pytest.mark.parametrize("what", ["scale 4", "scale 16", "growing keys", "wide", "cancelling", "denormal", "far splits"])
@pytest.mark.parametrize("Hq,Hkv,D,split", [(8, 8, 64, 128), (16, 2, 64, 1024), (4, 4, 128, 512), (8, 1, 128, 128),
                                            (8, 1, 64, 512), (4, 4, 128, 1024), (32, 8, 128, 512)])
def test_bits_of_run_on_harsh_inputs(Hq, Hkv, D, split, what):
    """Scores of hundreds, whose weights underflow or are denormal; keys that grow with their position;
    keys and values over many powers of two; sums that cancel; denormal inputs; splits whose maxima lie
    hundreds of powers of two apart: the bits of run, none of them a NaN."""
    page = 16
    g = torch.Generator().manual_seed(11)
    gr = Groups([(2 * split + 77, [1 + 29 * i for i in range(21)]), (split + 16, [3, 40])], Hq, Hkv, D, page)
    power = lambda x, lo, hi: (x.float() * torch.exp2(torch.randint(lo, hi + 1, x.shape, generator=g).float())).to(
        torch.bfloat16)
    scale = D**-0.5
    if what.startswith("scale"):
        scale = float(what.split()[1])
    elif what == "growing keys":
        _page_factors(gr, page, lambda p: 1 + p / 200)
        scale = 0.5
    elif what == "wide":
        gr.kc, gr.vc, gr.q = power(gr.kc, -12, 6), power(gr.vc, -60, 60), power(gr.q, -6, 2)
    elif what == "cancelling":
        gr.kc[..., 1::2] = gr.kc[..., ::2]                       # (pairs of equal keys under opposite queries)
        gr.q[..., 1::2] = -gr.q[..., ::2] * (1 + 2.0**-7 * (gr.q[..., ::2] > 0))
        gr.vc[:, 1::2] = -gr.vc[:, ::2]                          # (neighbours of opposite values)
        gr.kc, gr.vc = power(gr.kc, 0, 6), power(gr.vc, 0, 8)
    elif what == "denormal":
        tiny = lambda x: torch.where(x.isnan(), x, torch.randint(-127, 128, x.shape, generator=g).to(torch.bfloat16) * 2.0**-133)
        gr.vc = tiny(gr.vc)
        gr.kc[..., ::2] = tiny(gr.kc)[..., ::2]
        gr.q[0] = tiny(gr.q[0])
    else:
        gr.q[..., 0] = 16.0
        apart = {0: 0.0, 1: 120.0, 2: -120.0, 3: 60.0}
        k = gr.kc.clone()
        for row in gr.table.tolist():
            for i, pg in enumerate(row):
                if pg >= 0:
                    k[pg, :, :, 0] = apart[i * page // split % 4]
        gr.kc = k
    h = BiAttention(Hq, Hkv, D, page, scale=scale, split_size=split)
    plain, shared = gr.both(h)
    assert not bool(plain.view(torch.bfloat16).isnan().any())
    assert torch.equal(plain, shared)
    h.close()


def test_tokens_of_one_request_and_positions_inside_the_prefix():
    """A group may hold a chunk of a request and tokens whose position lies inside the prefix: each
    shares the splits before its own."""
    Hq, Hkv, D = 16, 4, 128
    base = Groups([(2000, [10, 20])], Hq, Hkv, D, 16)
    tokens = [(0, p) for p in (3, 511, 512, 700, 1023, 1024, 1999, 2009)] + [(1, p) for p in (1, 600, 1500, 2019)]
    base.q_seq = torch.tensor([b for b, _ in tokens], dtype=torch.int32)
    base.q_pos = torch.tensor([p for _, p in tokens], dtype=torch.int32)
    base.q = torch.randn(12, Hq, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    base.start = torch.tensor([0, 12], dtype=torch.int32)
    h = BiAttention(Hq, Hkv, D, 16)
    plain, shared = base.both(h)
    assert torch.equal(plain, shared)
    h.close()


def test_zeros_infinities_and_nan():
    """Zeros of both signs as queries, keys and values; infinities and NaN in the prefix: the bits of
    run (any NaN for a NaN)."""
    Hq, Hkv, D = 8, 2, 64
    gr = Groups([(1100, [3, 4, 5])], Hq, Hkv, D, 16)
    gr.q[0, 0] = 0.0
    gr.q[1, 1] = -0.0
    flat_k, flat_v = gr.kc.view(-1, Hkv, D), gr.vc.view(-1, Hkv, D)
    slot = lambda p: int(gr.table[0, p // 16]) * 16 + p % 16
    for p in range(1100 // 16 * 16):
        flat_v[slot(p), 0, 3] = -0.0
        flat_v[slot(p), 0, 4] = 0.0
    flat_k[slot(100), 1, 5] = float("inf")
    flat_v[slot(700), 0, 9] = float("-inf")
    flat_v[slot(701), 0, 10] = float("nan")
    h = BiAttention(Hq, Hkv, D, 16)
    plain, shared = (x.view(torch.bfloat16) for x in gr.both(h))
    assert torch.equal(plain.isnan(), shared.isnan())
    fine = ~plain.isnan()
    assert torch.equal(bits(plain[fine]), bits(shared[fine]))
    assert bool(plain.isnan().any()) and bool(plain.isinf().any())
    h.close()


def test_independent_of_grouping():
    """The same 20 tokens as one group, as groups of 7, 1 and 12, and with a shorter common length."""
    gr = Groups([(3000, [1 + 9 * i for i in range(20)])], 32, 8, 128, 16)
    h = BiAttention(32, 8, 128, 16)
    want, got = gr.both(h)
    assert torch.equal(want, got)
    for start, lens in (([0, 7, 8, 20], [2992, 2992, 2992]), ([0, 20], [1024]), ([0, 20], [0]), ([3, 11], [2000]),
                        ([0, 0, 20, 20], [5, 2992, 7])):
        gr.start, gr.len = torch.tensor(start, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
        assert torch.equal(gr.both(h)[1], want), start
    h.close()


@pytest.mark.parametrize("what", ["descending", "past the end", "negative length", "other pages", "position", "page"])
def test_bad_groups_are_reported(what):
    gr = Groups([(1100, [3, 40, 5]), (1500, [1, 2])], 8, 2, 64, 16)
    h = BiAttention(8, 2, 64, 16)
    good = gr.both(h)[0]
    start, length, mp = gr.start.clone(), gr.len.clone(), gr.max_pos
    table, pos = gr.table.clone(), gr.q_pos.clone()
    if what == "descending":
        gr.start[1] = 6
    elif what == "past the end":
        gr.start[2] = 9
    elif what == "negative length":
        gr.len[1] = -1
    elif what == "other pages":
        gr.table[1, 5] = gr.table[1, 6]
    elif what == "position":
        gr.q_pos[4] = -1
    else:
        gr.table[3:, 2] = -1
    a = gr.args()
    o = h.run_shared(*a, gr.start.cuda(), gr.len.cuda())
    assert h.device_error() == bg.BI_GEMM_ERR_INVALID_ARG and h.device_error() == 0
    if what in ("past the end", "negative length", "page"):
        assert torch.equal(bits(o)[:3], good[:3])
    if what in ("descending", "past the end", "negative length"):      # nothing is shared
        assert torch.equal(bits(o), good)
    gr.start, gr.len, gr.table, gr.q_pos = start, length, table, pos
    assert torch.equal(gr.both(h)[1], good)
    h.close()


@pytest.mark.parametrize("page", [16, 12])
def test_both_sides_of_the_rule(page):
    """Calls whose units all run at once are not shared, the next larger ones are: the same bits, and a
    bad table of groups is only looked at where it is used."""
    gr = Groups([(1100, [3, 40, 5, 9])], 8, 2, 64, page)
    h = BiAttention(8, 2, 64, page)
    want = gr.both(h)[0]
    a, good, bad = gr.args()[:-1], gr.start.cuda(), (gr.start + 1).cuda()
    seen = []
    for bound in (1200, 512 * 56, 512 * 75, 512 * 76, 512 * 110, 512 * 400):
        assert torch.equal(bits(h.run_shared(*a, bound, good, gr.len.cuda())), want)
        assert h.device_error() == 0
        assert torch.equal(bits(h.run_shared(*a, bound, bad, gr.len.cuda())), want)
        seen.append(h.device_error())
    assert seen[0] == 0 and seen[-1] == bg.BI_GEMM_ERR_INVALID_ARG and sorted(seen, reverse=True) == seen
    h.close()


@pytest.mark.parametrize("Hq,Hkv,D,page,T,splits", [(16, 2, 64, 12, 4, 94), (16, 2, 64, 12, 16, 22), (8, 8, 64, 12, 16, 5)])
def test_what_run_serves_in_one_round_is_not_shared(Hq, Hkv, D, page, T, splits):
    """For pages that are copied by rows the rule counts the blocks of the kernel that run takes (five per
    SM here, 760 for 640 to 752 units), so that no call is shared whose units those hold at once."""
    h = BiAttention(Hq, Hkv, D, page)
    assert 608 < T * Hkv * splits <= 760
    assert h.shared_workspace_size(T, 512 * splits - 1, 1) == h.workspace_size(T, 512 * splits - 1)
    assert h.shared_workspace_size(T, 512 * 2 * splits - 1, 1) > h.workspace_size(T, 512 * 2 * splits - 1)
    h.close()


def test_overlapping_groups():
    """Groups that climb, fall back and climb again claim the same tokens twice: reported, and every
    token is served by units of its own."""
    gr = Groups([(1100, [3, 40, 5]), (1500, [1, 2, 7, 9])], 8, 2, 64, 16)
    h = BiAttention(8, 2, 64, 16)
    good = gr.both(h)[0]
    for starts, lens in (([0, 3, 0, 7, 3, 7], [1100, 5, 0, 5, 1500]), ([3, 7, 0, 3], [1500, 0, 1100]),
                         ([0, 7, 6, 7], [1100, 0, 700]), ([0] + [7, 0] * 40, [600] * 80)):
        start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        o = h.run_shared(*gr.args(), start, torch.tensor(lens, dtype=torch.int32, device="cuda"))
        assert h.device_error() == bg.BI_GEMM_ERR_INVALID_ARG and h.device_error() == 0
        assert torch.equal(bits(o), good)
    h.close()


@pytest.mark.parametrize("groups", [1, 5, 31, 33, 1023, 1024, 1025, 1500])
def test_many_groups(groups):
    """Group tables and batches on both sides of what the plan keeps in shared memory, some groups empty."""
    rng = np.random.default_rng(groups)
    gr = Groups([(260, [int(rng.integers(1, 200)) for _ in range(int(rng.integers(1, 4)))]) for _ in range(groups)],
                4, 2, 64, 16)
    h = BiAttention(4, 2, 64, 16, split_size=128)
    got = gr.both(h)
    assert torch.equal(got[0], got[1]) and h.device_error() == 0
    h.close()


def test_a_long_table_of_empty_groups():
    """Groups that hold no two tokens share nothing and need no room: a table padded with 2^18 of them
    is served like the one without, and asks for no more workspace than the tokens can fill."""
    gr = Groups([(1100, [3, 40, 5]), (1500, [1, 2, 7, 9])], 8, 2, 64, 16)
    h = BiAttention(8, 2, 64, 16)
    want = gr.both(h)[0]
    n = 1 << 18
    start = torch.full((n + 1,), 7, dtype=torch.int32)
    length = torch.zeros(n, dtype=torch.int32)
    start[:3], length[:2] = gr.start, gr.len
    assert torch.equal(bits(h.run_shared(*gr.args(), start.cuda(), length.cuda())), want)
    assert h.device_error() == 0
    # one token, under a bound that would have more of them share
    one = [x[:1].contiguous() for x in gr.args()[:3]] + gr.args()[3:-1]
    assert torch.equal(bits(h.run_shared(*one, 1 << 20, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                                         gr.len[:1].cuda())), want[:1])
    assert h.device_error() == 0
    # (seven tokens make at most three groups of two or more)
    assert h.shared_workspace_size(7, 1 << 20, n) == h.shared_workspace_size(7, 1 << 20, 3)
    bound = (1 << 29) - 1                      # 2^20 splits: room for a unit of every group was refused
    assert h.shared_workspace_size(7, bound, n) == h.shared_workspace_size(7, bound, 3)
    h.close()


def test_refusals_and_empty_calls():
    gr = Groups([(600, [3, 4])], 8, 2, 64, 16)
    h = BiAttention(8, 2, 64, 16)
    a, s, n = gr.args(), gr.start.cuda(), gr.len.cuda()
    want = bits(h.run(*a))
    for bad in ((s[:1], n), (s.long(), n), (s, n.cpu()), (s, n.float())):
        with pytest.raises(ValueError):
            h.run_shared(*a, *bad)
    with pytest.raises(bg.BiGemmError):
        h.run_shared(*a[:-1], -1, s, n)
    assert torch.equal(bits(h.run_shared(*a, s[:1], n[:0])), want)          # no group
    empty = [a[0][:0], a[1][:0], a[2][:0]] + a[3:]
    assert h.run_shared(*empty, torch.zeros(2, dtype=torch.int32, device="cuda"), n).shape[0] == 0
    assert h.shared_workspace_size(2, 600, 1) == h.workspace_size(2, 600)          # (nothing is shared)
    assert h.shared_workspace_size(200, 9000, 1) > h.workspace_size(200, 9000)
    h.close()


def test_repeat_stream_and_graph():
    gr = Groups([(2600, [1 + 11 * i for i in range(40)]), (700, [2, 3])], 32, 8, 128, 16)
    h = BiAttention(32, 8, 128, 16)
    want, got = gr.both(h)
    assert torch.equal(want, got)
    a, s, n = gr.args(), gr.start.cuda(), gr.len.cuda()
    for _ in range(20):
        assert torch.equal(bits(h.run_shared(*a, s, n)), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = h.run_shared(*a, s, n)
    side.synchronize()
    assert torch.equal(bits(got), want)
    out = torch.zeros_like(a[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.run_shared(*a, s, n, o=out)
    a[2].copy_(a[2] - 1)                       # replayed with other positions and queries
    a[0].copy_(a[0].flip(0).contiguous())
    other = BiAttention(32, 8, 128, 16)
    want2 = bits(other.run(*a))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), want2)
    assert h.device_error() == 0 and other.device_error() == 0
    h.close()
    other.close()
