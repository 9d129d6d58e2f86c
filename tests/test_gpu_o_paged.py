"""The operators around the paged cache together on the GPU, as a serving loop uses them: a prompt's
projection normalised, rotated and appended (BiQkRope), attended (BiPromptAttention), its cache forked
for several samples and decoded behind the shared prefix (BiAttention.run_shared); caches past 32-bit
offsets; handles on streams of their own at once; workspaces and graphs; and waits that run out."""
import ctypes

import pytest
import torch

import invariant_bi_gemm_gb300 as bg
from gpu_util import Controls, stream_ptr
from invariant_bi_gemm_gb300 import BiAttention, BiPromptAttention, BiQkRope
from test_gpu_l_qkrope import make as make_rope
from test_gpu_m_prompt import Pack
from test_gpu_n_shared import Groups

pytestmark = pytest.mark.gpu


def bits(x):
    return x.view(torch.int16)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def attention64(q, k, v, scale):
    """q [n, H, D] at the last n positions of k, v [L, Hkv, D]: (value, sum of weights times |v|, largest score)."""
    n, H, D = q.shape
    L, G = k.shape[0], H // k.shape[1]
    k, v = (x.double().repeat_interleave(G, 1) for x in (k, v))
    s = torch.einsum("nhd,lhd->nhl", q.double(), k) * scale
    seen = torch.arange(L, device=q.device)[None] <= torch.arange(L - n, L, device=q.device)[:, None]
    s = s.masked_fill(~seen[:, None], -float("inf"))
    w = torch.softmax(s, -1)
    e = s.masked_fill(~seen[:, None], 0).abs().amax(-1, keepdim=True)
    return torch.einsum("nhl,lhd->nhd", w, v), torch.einsum("nhl,lhd->nhd", w, v.abs()), e


@pytest.mark.parametrize("Hq,Hkv,D,page,n", [(32, 8, 128, 16, 1300), (16, 2, 64, 32, 700)])
def test_prompt_then_forked_samples(Hq, Hkv, D, page, n):
    """Each step against fp64 on the very caches it read (the bounds of the operators' own tests), for
    a prompt in two chunks and three decode steps of four samples."""
    g = torch.Generator(device="cuda").manual_seed(9)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    samples, steps, width = 4, 3, (Hq + 2 * Hkv) * D
    per = -(-(n + steps) // page)
    pages = per + samples * 2 + 1
    kc, vc = rn(pages, page, Hkv, D), rn(pages, page, Hkv, D)
    rate = 10000.0 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
    ang = torch.arange(n + steps, device="cuda", dtype=torch.float64)[:, None] * rate
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    gq, gk = rn(D), rn(D)
    rope, prompt, att = BiQkRope(Hq, Hkv, D, page), BiPromptAttention(Hq, Hkv, D, page), BiAttention(Hq, Hkv, D, page)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    mine = table[:per].view(1, per).contiguous()
    flat = lambda c, row, length: c.view(-1, Hkv, D)[
        row[torch.arange(length, device="cuda") // page].long() * page + torch.arange(length, device="cuda") % page]
    u = 2.0**-24
    done = 0
    for m in (n - n // 3, n // 3):
        q = rope.run(rn(m, width), gq, gk, cs, torch.zeros(m, dtype=torch.int32, device="cuda"),
                     torch.arange(done, done + m, dtype=torch.int32, device="cuda"), kc, vc, mine)
        o = prompt.run(q, i32(0, m), i32(done), kc, vc, mine, n - 1)
        done += m
        val, a, e = attention64(q, flat(kc, mine[0], done), flat(vc, mine[0], done), prompt.scale)
        tol = 2.0**-8 * val.abs() + (2.0**-8 + 4 * (D + 8) * u * e + 2 * (done + 160) * u) * a
        assert bool(((o.double() - val).abs() <= tol).all())
    # the fork: whole pages in common, the last one copied
    whole = n // page
    tables = mine.repeat(samples, 1)
    for b in range(samples):
        own = table[per + 2 * b:per + 2 * b + per - whole]
        if n % page:
            kc[own[0].long()], vc[own[0].long()] = kc[mine[0, whole].long()], vc[mine[0, whole].long()]
        tables[b, whole:] = own[:per - whole]
    seqs = torch.arange(samples, dtype=torch.int32, device="cuda")
    for t in range(steps):
        pos = torch.full((samples,), n + t, dtype=torch.int32, device="cuda")
        q = rope.run(rn(samples, width), gq, gk, cs, seqs, pos, kc, vc, tables)
        args = (q, seqs, pos, kc, vc, tables, n + t)
        # (as it is, and under a bound so loose that the few samples share)
        o = att.run_shared(*args[:-1], 1 << 17, i32(0, samples), i32(whole * page))
        assert torch.equal(bits(o), bits(att.run_shared(*args, i32(0, samples), i32(whole * page))))
        assert torch.equal(bits(o), bits(att.run(*args)))
        for b in range(samples):
            val, a, e = attention64(q[b:b + 1], flat(kc, tables[b], n + t + 1), flat(vc, tables[b], n + t + 1), att.scale)
            tol = 2.0**-8 * val.abs() + (4 * (D + 8) * u * e + 2 * (n + t + 33) * u) * a
            assert bool(((o[b:b + 1].double() - val).abs() <= tol).all())
    for h in (rope, prompt, att):
        assert h.device_error() == 0
        h.close()


@pytest.mark.parametrize("page", [16, 12])
def test_caches_past_32_bit_offsets(page):
    """Pages behind 2^32 bytes (and 2^31 elements) of a cache give the bits of the same pages near its
    start, for both attentions, and take the appended keys and values."""
    Hq, Hkv, D = 4, 4, 64
    pages = ((1 << 32) // (Hkv * D * 2 * page)) + 400
    kc = torch.empty(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    n = 1400
    per = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(2)
    for c in (kc, vc):
        c[:per] = torch.randn(per, page, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
        c[pages - per:] = c[:per]
    near = torch.arange(per, dtype=torch.int32, device="cuda").view(1, per)
    far = near + (pages - per)
    q = torch.randn(n, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    prompt, att, rope = BiPromptAttention(Hq, Hkv, D, page), BiAttention(Hq, Hkv, D, page), BiQkRope(Hq, Hkv, D, page)
    o = [prompt.run(q, i32(0, n), i32(0), kc, vc, t, n - 1) for t in (near, far)]
    assert torch.equal(bits(o[0]), bits(o[1]))
    two = [torch.cat([t, t]) for t in (near, far)]
    pos, seq = i32(n - 1, n - 2), i32(0, 1)
    # (the bound is loose, so that two tokens share)
    s = [att.run_shared(q[:2].contiguous(), seq, pos, kc, vc, t, 1 << 17, i32(0, 2), i32(1024)) for t in two]
    assert torch.equal(bits(s[0]), bits(s[1]))
    assert torch.equal(bits(s[0]), bits(att.run(q[:2].contiguous(), seq, pos, kc, vc, two[0], n - 1)))
    qkv = torch.randn(n, 3 * Hq * D, generator=g, device="cuda").to(torch.bfloat16)
    cs = torch.rand(n, D, generator=g, device="cuda")
    z, at = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    r = [rope.run(qkv, None, None, cs, z, at, kc, vc, t) for t in (near, far)]
    assert torch.equal(bits(r[0]), bits(r[1]))
    assert torch.equal(bits(kc[:per]), bits(kc[pages - per:])) and torch.equal(bits(vc[:per]), bits(vc[pages - per:]))
    assert torch.equal(vc[:per].view(-1, Hkv, D)[:n], qkv.view(n, 3 * Hq, D)[:, 2 * Hq:])
    for h in (prompt, att, rope):
        assert h.device_error() == 0
        h.close()


def test_handles_on_streams_of_their_own_at_once():
    """Two handles of each operator, each on a stream of its own, many calls in flight: the bits of calls one by one."""
    pk = [Pack([(i, 300 + 40 * i, 90 * i)], 16, 4, 64, 16) for i in range(2)]
    gr = [Groups([(1500, [1 + 7 * i for i in range(10 + 5 * k)])], 16, 4, 64, 16, seed=k) for k in range(2)]
    ro = [make_rope(600 + 300 * k, 16, 4, 64, 16, 64, seed=k) for k in range(2)]
    hs = [(BiPromptAttention(16, 4, 64, 16), BiAttention(16, 4, 64, 16), BiQkRope(16, 4, 64, 16)) for _ in range(2)]
    pa, ga = [p.args() for p in pk], [x.args() + [x.start.cuda(), x.len.cuda()] for x in gr]
    call = [lambda k: hs[k][0].run(*pa[k]), lambda k: hs[k][1].run_shared(*ga[k]), lambda k: hs[k][2].run(**ro[k])]
    want = [[bits(f(k)).clone() for f in call] for k in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k] += [(j, call[j](k)) for j in range(3)]
    torch.cuda.synchronize()
    for k in range(2):
        for j, o in got[k]:
            assert torch.equal(bits(o), want[k][j])
        for h in hs[k]:
            assert h.device_error() == 0
            h.close()


def test_graphs_outlive_the_growth_of_their_workspace():
    """A graph captured with a small workspace replays to the same bits after a larger eager call has
    grown it; a capture that would have to grow it is refused and the handle goes on."""
    small, large = Pack([(0, 60, 0)], 8, 2, 64, 16), Pack([(i, 200 + i, 0) for i in range(40)], 8, 2, 64, 16)
    gs, gl = Groups([(600, [3, 4])], 8, 2, 64, 16), Groups([(3000, [1 + i for i in range(60)])], 8, 2, 64, 16)
    middle = Pack([(i, 100, 7 * i) for i in range(24)], 8, 2, 64, 16)
    prompt, second, att = BiPromptAttention(8, 2, 64, 16), BiPromptAttention(8, 2, 64, 16), BiAttention(8, 2, 64, 16)
    assert prompt.workspace_size(60, 1) == 0 < prompt.workspace_size(2400, 24) < prompt.workspace_size(8780, 40)
    runs = []
    for h, x, y in ((prompt.run, small.args(), large.args()), (second.run, middle.args(), large.args()),
                    (att.run_shared, gs.args() + [gs.start.cuda(), gs.len.cuda()],
                     gl.args() + [gl.start.cuda(), gl.len.cuda()])):
        want = bits(h(*x)).clone()
        out = torch.zeros_like(x[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            h(*x, o=out)
        refused = torch.cuda.CUDAGraph()
        big = torch.zeros_like(y[0])
        with torch.cuda.graph(refused):
            with pytest.raises(bg.BiGemmError) as e:
                h(*y, o=big)
        assert e.value.code == bg.BI_GEMM_ERR_SCRATCH_LIMIT
        runs.append((h, x, y, want, out, graph))
    for h, x, y, want, out, graph in runs:
        big = bits(h(*y)).clone()
        junk = [torch.full((1 << 22,), 0x7F7F7F7F, dtype=torch.int32, device="cuda") for _ in range(8)]
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), want)
        assert torch.equal(bits(h(*y)), big)
        del junk
    for h in (prompt, second, att):
        assert h.device_error() == 0
        h.close()


def _held(f):
    """Device memory that f() left allocated outside torch."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.mem_get_info()[0]
    f()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    return before - torch.cuda.mem_get_info()[0]


def test_growth_holds_no_more_than_its_step():
    """A bound that climbs call by call: the handle ends up with the workspace that the last call needs
    and one step of growth (64 MiB, and what the driver rounds up), not with every earlier one."""
    gr = Groups([(600, [3 + i for i in range(64)])], 32, 8, 128, 16)
    att, a = BiAttention(32, 8, 128, 16), gr.args()[:-1]
    extra = (gr.start.cuda(), gr.len.cuda())
    out = torch.empty_like(a[0])
    att.run_shared(*a, 8191, *extra, o=out)
    bounds = [512 * n - 1 for n in range(40, 321, 40)]
    need = att.shared_workspace_size(64, bounds[-1], 1)
    assert need > 300 << 20
    held = _held(lambda: [att.run_shared(*a, b, *extra, o=out) for b in bounds])
    assert held <= need + (64 << 20) + (64 << 20), (held, need)
    want = bits(att.run(*a, 8191))
    assert torch.equal(bits(att.run_shared(*a, bounds[-1], *extra)), want) and att.device_error() == 0
    att.close()


def test_growth_keeps_what_captured_calls_use():
    """Large workspaces: one that a captured call uses outlives the growth, and the graph its bits."""
    gr = Groups([(600, [3 + i for i in range(64)])], 32, 8, 128, 16)
    att, a = BiAttention(32, 8, 128, 16), gr.args()[:-1]
    extra = (gr.start.cuda(), gr.len.cuda())
    want = bits(att.run_shared(*a, 512 * 100, *extra)).clone()
    out = torch.zeros_like(a[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att.run_shared(*a, 512 * 100, *extra, o=out)
    for n in (150, 250, 350):
        assert torch.equal(bits(att.run_shared(*a, 512 * n, *extra)), want)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), want) and att.device_error() == 0
    att.close()


def test_captured_runs_and_the_workspace_of_run():
    """BiAttention.run captured by a handle that has not run before, captured again after smaller calls,
    and grown between the replays: graphs and calls give the bits of a handle that is never captured."""
    gr = Groups([(3000, [3 + 5 * i for i in range(40)])], 8, 2, 64, 16)
    few, many = [x[:5].contiguous() for x in gr.args()[:3]] + gr.args()[3:], gr.args()
    plain, att = BiAttention(8, 2, 64, 16), BiAttention(8, 2, 64, 16)
    want = [bits(plain.run(*a)).clone() for a in (few, many)]
    out = [torch.zeros_like(a[0]) for a in (few, many, few)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(3)]

    def replay(k):
        out[k].zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        return torch.equal(bits(out[k]), want[k % 2])

    with torch.cuda.graph(graphs[0]):
        att.run(*few, o=out[0])                       # nothing has run: the graph's own memory
    assert torch.equal(bits(att.run(*few)), want[0])
    assert replay(0) and replay(0)
    with torch.cuda.graph(graphs[1]):
        att.run(*many, o=out[1])                      # more than there is
    with torch.cuda.graph(graphs[2]):
        att.run(*few, o=out[2])                       # what there is
    assert replay(1) and replay(2) and replay(1)
    for _ in range(2):
        assert torch.equal(bits(att.run(*many)), want[1])                # grows past what graph 2 uses
        junk = [torch.full((1 << 22,), 0x7F7F7F7F, dtype=torch.int32, device="cuda") for _ in range(8)]
        assert replay(2) and replay(0) and replay(1)
        del junk
    assert torch.equal(bits(att.run(*few)), want[0]) and att.device_error() == 0
    att.close()
    plain.close()


def test_waits_that_run_out_are_reported_and_the_handles_survive():
    """Failure injection (test controls): block 0 of each kernel loads nothing, its waits end after
    50 ms, the call reports BI_GEMM_ERR_TIMEOUT, and the next ordinary call gives the golden bits."""
    L, P, V = Controls().L, ctypes.c_void_p, ctypes.c_void_p
    I64, U64 = ctypes.c_int64, ctypes.c_uint64
    ptr = lambda t: V(t.data_ptr())
    # prompt
    pk = Pack([(i, 200, 100) for i in range(3)], 8, 2, 128, 16)
    product = BiPromptAttention(8, 2, 128, 16)
    golden = bits(pk.run(product))
    q, qs, q0, kc, vc, table, mp = pk.args()
    o = torch.zeros_like(q)
    h = P()
    L.bi_ctl_prompt_create.argtypes = [ctypes.POINTER(P), I64, I64, I64, I64, ctypes.c_float]
    L.bi_ctl_prompt_run.argtypes = [P, P, I64, P, P, I64, P, P, I64, P, I64, I64, P, P]
    L.bi_ctl_prompt_stall.argtypes = [P, P, I64, P, P, I64, P, P, I64, P, I64, I64, P, U64, P]
    L.bi_ctl_prompt_get_device_error.argtypes = L.bi_ctl_qkrope_get_device_error.argtypes = [P, P]
    L.bi_ctl_prompt_destroy.argtypes = L.bi_ctl_qkrope_destroy.argtypes = [P]
    assert L.bi_ctl_prompt_create(ctypes.byref(h), 8, 2, 128, 16, product.scale) == 0
    args = (ptr(q), q.shape[0], ptr(qs), ptr(q0), 3, ptr(kc), ptr(vc), kc.shape[0], ptr(table), table.shape[1], mp, ptr(o))
    assert L.bi_ctl_prompt_stall(h, *args, 50_000_000, stream_ptr()) == 0
    assert L.bi_ctl_prompt_get_device_error(h, stream_ptr()) == bg.BI_GEMM_ERR_TIMEOUT
    assert L.bi_ctl_prompt_run(h, *args, stream_ptr()) == 0
    assert L.bi_ctl_prompt_get_device_error(h, stream_ptr()) == 0
    assert torch.equal(bits(o), golden)
    assert L.bi_ctl_prompt_destroy(h) == 0
    product.close()
    # the groups of a shared prefix
    gr = Groups([(1200, [3, 9, 70])], 8, 2, 128, 16)
    a, gs, gl = gr.args(), gr.start.cuda(), gr.len.cuda()
    h = P()
    assert L.bi_ctl_attention_create(ctypes.byref(h), 8, 2, 128, 16, ctypes.c_float(128**-0.5), 0) == 0
    L.bi_ctl_attention_shared_stall.argtypes = [P, P, I64, P, P, P, P, I64, P, I64, I64, I64, P, P, I64, P, U64, P]
    o = torch.zeros_like(a[0])
    args = (ptr(a[0]), 3, ptr(a[1]), ptr(a[2]), ptr(a[3]), ptr(a[4]), a[3].shape[0], ptr(a[5]), 3, a[5].shape[1], a[6])
    assert L.bi_ctl_attention_shared_stall(h, *args, ptr(gs), ptr(gl), 1, ptr(o), 50_000_000, stream_ptr()) == 0
    assert L.bi_ctl_attention_get_device_error(h, stream_ptr()) == bg.BI_GEMM_ERR_TIMEOUT
    assert L.bi_ctl_attention_run(h, *args, ptr(o), stream_ptr()) == 0
    assert L.bi_ctl_attention_get_device_error(h, stream_ptr()) == 0
    plain = BiAttention(8, 2, 128, 16)
    assert torch.equal(bits(o), bits(plain.run_shared(*a, gs, gl)))
    L.bi_ctl_attention_destroy(h)
    # the form for many tokens of the append
    rope = BiQkRope(16, 8, 128, 16)
    T = rope.config["ring_from"]
    r = make_rope(T, 16, 8, 128, 16, 128, far=2500)
    h = P()
    L.bi_ctl_qkrope_create.argtypes = [ctypes.POINTER(P), I64, I64, I64, I64, I64, ctypes.c_int32, ctypes.c_float]
    L.bi_ctl_qkrope_stall.argtypes = [P, P, I64, I64, P, P, P, I64, P, P, P, P, I64, P, I64, I64, P, U64, P]
    assert L.bi_ctl_qkrope_create(ctypes.byref(h), 16, 8, 128, 16, 128, 0, 1e-6) == 0
    q = torch.zeros(T, 16, 128, dtype=torch.bfloat16, device="cuda")
    assert L.bi_ctl_qkrope_stall(h, ptr(r["qkv"]), T, 32 * 128, ptr(r["gq"]), ptr(r["gk"]), ptr(r["cos_sin"]), 2500,
                                 ptr(r["q_seq"]), ptr(r["q_pos"]), ptr(r["k_cache"]), ptr(r["v_cache"]),
                                 r["k_cache"].shape[0], ptr(r["page_table"]), 3, r["page_table"].shape[1], ptr(q),
                                 50_000_000, stream_ptr()) == 0
    assert L.bi_ctl_qkrope_get_device_error(h, stream_ptr()) == bg.BI_GEMM_ERR_TIMEOUT
    assert L.bi_ctl_qkrope_get_device_error(h, stream_ptr()) == 0
    assert L.bi_ctl_qkrope_destroy(h) == 0
    assert rope.run(**r).shape == (T, 16, 128) and rope.device_error() == 0
    rope.close()
    plain.close()


def test_tensors_of_another_device_are_refused():
    """Pointers of another GPU never reach a kernel of the handle's."""
    rope, prompt, att = BiQkRope(8, 2, 64, 16), BiPromptAttention(8, 2, 64, 16), BiAttention(8, 2, 64, 16)
    for op in (rope, prompt, att):
        op._device += 1                        # (as if it had been made there)
    gr, pk, x = Groups([(600, [3, 4])], 8, 2, 64, 16), Pack([(0, 7, 0)], 8, 2, 64, 16), torch.zeros
    with pytest.raises(ValueError):
        att.run_shared(*gr.args(), gr.start.cuda(), gr.len.cuda())
    with pytest.raises(ValueError):
        prompt.run(*pk.args())
    with pytest.raises(ValueError):
        rope.run(x(1, 768, dtype=torch.bfloat16, device="cuda"), None, None, x(1, 64, device="cuda"), i32(0), i32(0),
                 *[t.cuda() for t in (pk.kc, pk.vc, pk.table)])


@pytest.mark.parametrize("bound", [511, 4000])
def test_appends_right_behind_a_call_that_merges_nothing(bound):
    """Contexts of one split, whose outputs need no merge: keys and values appended over them by the next
    kernel of the stream, which starts as early as it may, change nothing that was asked before."""
    Hq, Hkv, D, page, T = 32, 8, 128, 16, 2048
    g = torch.Generator(device="cuda").manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    att, rope = BiAttention(Hq, Hkv, D, page), BiQkRope(Hq, Hkv, D, page)
    pages = T * 512 // page
    kc, vc, q = rn(pages, page, Hkv, D), rn(pages, page, Hkv, D), rn(T, Hq, D)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(T, -1).contiguous()
    seq = torch.arange(T, dtype=torch.int32, device="cuda")
    last = torch.full((T,), 511, dtype=torch.int32, device="cuda")
    qkv, cs = rn(T, (Hq + 2 * Hkv) * D), torch.rand(512, D, generator=g, device="cuda")
    want = bits(att.run(q, seq, last, kc, vc, table, bound)).clone()
    old = [c.clone() for c in (kc, vc)]
    for step in range(6):
        o = att.run(q, seq, last, kc, vc, table, bound)
        rope.run(qkv, None, None, cs, seq, last - 100 * (step % 2), kc, vc, table)      # inside the contexts
        assert torch.equal(bits(o), want), step
        for c, was in zip((kc, vc), old):
            c.copy_(was)
    assert att.device_error() == 0 and rope.device_error() == 0
    att.close()
    rope.close()
