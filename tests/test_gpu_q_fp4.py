"""Matrices in 4 bits (include/bi_fp4.h): quantisation against the format's definition bit by bit, the values
back, the product against 64-bit sums, and batch invariance of both."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_ref as ref
import invariant_bi_gemm_gb300 as bg
from gpu_util import Controls, stream_ptr

pytestmark = pytest.mark.gpu
KINDS = ("mxfp4", "nvfp4")


def bf16(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def host(t: torch.Tensor) -> np.ndarray:
    return t.cpu().numpy()


def rows(M, K, seed):
    """bf16 rows whose blocks cover the format: ordinary values, ties of every code, tiny and huge blocks, zeros of
    either sign, infinities and NaN."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((M, K)).astype(np.float32) * np.exp2(r.integers(-12, 12, (M, 1))).astype(np.float32)
    x = x.reshape(M, -1, 16)
    pick = r.integers(0, 16, x.shape[:2])
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6], np.float32)
    unit = np.exp2(r.integers(-6, 6, x.shape[:2])).astype(np.float32) * r.choice([1, 1.125, 1.25, 1.5, 1.875], x.shape[:2])
    x = np.where((pick < 4)[..., None], ties * unit[..., None].astype(np.float32), x)
    x = np.where((pick == 4)[..., None], np.float32(0) * x, x)                       # zeros of both signs
    x = np.where((pick == 5)[..., None], x * np.float32(2.0 ** -126), x)             # denormals and what is lost
    x = np.where((pick == 6)[..., None], x * np.float32(2.0 ** 110), x)              # beyond E4M3's range
    odd = np.where(r.random(x.shape) < 0.1, r.choice([np.inf, -np.inf, np.nan], x.shape), x)
    x = np.where((pick == 7)[..., None], odd, x).reshape(M, K).astype(np.float32)
    return host(bf16(x).float())


@pytest.mark.parametrize("kind,g", [("mxfp4", 1.0), ("nvfp4", 1.0), ("nvfp4", 0.25), ("nvfp4", 0.37), ("nvfp4", 2.0 ** -60)])
@pytest.mark.parametrize("M,K", [(1, 128), (3, 256), (37, 384), (130, 4096), (300, 128)])
def test_quantisation_has_the_definitions_bits(kind, g, M, K):
    x = rows(M, K, M * 7 + K)
    codes, scales = bg.BiQuant4(K, kind, g).run(bf16(x))
    want, byte = ref.quantise(x, kind, g)
    got_s = ref.from_tiles(host(scales), M)
    assert np.array_equal(got_s, byte), np.argwhere(got_s != byte)[:5]
    got = ref.unpack(host(codes))
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("kind", KINDS)
def test_every_bf16_value_of_a_block(kind):
    """Each of the 65536 patterns beside a block maximum of 1.0 and of 3.0."""
    bits = np.arange(65536, dtype=np.uint32)
    v = ref.bf16_values(bits)
    v = v[np.isfinite(v) & (np.abs(v) <= 1)]
    v = np.concatenate([v, np.zeros(-len(v) % 15, np.float32)]).reshape(-1, 15)
    for top in (1.0, 3.0):
        x = np.concatenate([np.full((len(v), 1), top, np.float32), v * np.float32(top)], 1)
        x = host(bf16(x).float())
        x = x if kind == "nvfp4" else np.repeat(x, 2, 1)
        x = np.pad(x.reshape(-1), (0, -x.size % 1024)).reshape(-1, 1024)
        codes, scales = bg.BiQuant4(1024, kind).run(bf16(x))
        want, byte = ref.quantise(x, kind)
        assert np.array_equal(ref.from_tiles(host(scales), len(x)), byte)
        assert np.array_equal(ref.unpack(host(codes)), want)


@pytest.mark.parametrize("kind", KINDS)
def test_strided_rows_and_bytes_of_rows_that_are_not_there(kind):
    K, M = 256, 70
    wide = bf16(rows(M, K + 64, 3))
    q = bg.BiQuant4(K, kind)
    scales = torch.full((1, K // (4 * q.block), 32, 4, 4), 0xAB, dtype=torch.uint8, device="cuda")
    codes, _ = q.run(wide[:, 8:8 + K], scales=scales)
    again, s2 = q.run(wide[:, 8:8 + K].contiguous())
    assert torch.equal(codes, again)
    assert np.array_equal(ref.from_tiles(host(scales), M), ref.from_tiles(host(s2), M))
    assert (ref.from_tiles(host(scales), 128)[M:] == 0xAB).all()


@pytest.mark.parametrize("g", [1.0, 0.37, 2.0 ** 64, 2.0 ** -64, 1.7 * 2.0 ** -60])
@pytest.mark.parametrize("top", [3.3e38, 3000.0])
def test_every_bf16_value_of_a_block_beyond_the_largest_scale(g, top):
    """Each finite pattern of either sign in blocks whose largest element asks for a scale above 448 (top: as it is, or
    3000 g, just above 448 * 6 g)."""
    big = np.float32(min(top * g, 3.3e38) if top < 1e30 else top)
    v = ref.bf16_values(np.arange(65536, dtype=np.uint32))
    v = v[np.isfinite(v) & (np.abs(v) <= big)]
    v = np.concatenate([v, np.zeros(-len(v) % 15, np.float32)]).reshape(-1, 15)
    x = host(bf16(np.concatenate([np.full((len(v), 1), big, np.float32), v], 1)).float())
    x = np.pad(x.reshape(-1), (0, -x.size % 1024)).reshape(-1, 1024)
    codes, scales = bg.BiQuant4(1024, "nvfp4", g).run(bf16(x))
    want, byte = ref.quantise(x, "nvfp4", g)
    got_s = ref.from_tiles(host(scales), len(x))
    assert np.array_equal(got_s, byte) and (got_s.reshape(-1)[:len(v)] == 0x7E).all()
    got = ref.unpack(host(codes))
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("kind,g", [("mxfp4", 1.0), ("nvfp4", 0.5), ("nvfp4", 0.37)])
def test_expand_gives_the_values(kind, g):
    r = np.random.default_rng(5)
    M, K = 77, 384
    packed = r.integers(0, 256, (M, K // 2), dtype=np.uint8)
    byte = r.integers(60, 190, (M, K // ref.BLOCK[kind]), dtype=np.uint8) if kind == "mxfp4" else \
        r.integers(0, 127, (M, K // 16), dtype=np.uint8)
    byte[3, 1], byte[5, 2] = (255, 0) if kind == "mxfp4" else (0x7F, 0)
    y = bg.BiQuant4(K, kind, g).expand(torch.from_numpy(packed).cuda(), torch.from_numpy(ref.to_tiles(byte, 0x7F)).cuda())
    want = torch.from_numpy(ref.values(packed, byte, kind, g)).float().to(torch.bfloat16)
    if kind == "nvfp4":        # fl32(scale g), then fl32(code x that), then bf16
        s = (ref.e4m3_value(byte).astype(np.float32) * np.float32(g)).astype(np.float32)
        v = np.concatenate([ref.GRID, -ref.GRID])[ref.unpack(packed)].astype(np.float32) * np.repeat(s, 16, -1)
        want = torch.from_numpy(v).to(torch.bfloat16)
    y = y.cpu()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))


@pytest.mark.parametrize("kind", KINDS)
def test_a_rows_codes_do_not_depend_on_the_batch(kind):
    K = 1024
    x = bf16(rows(257, K, 11))
    q = bg.BiQuant4(K, kind)
    codes, scales = q.run(x)
    s = ref.from_tiles(host(scales), 257)
    for i in (0, 5, 128, 256):
        c1, s1 = q.run(x[i:i + 1])
        assert torch.equal(c1[0], codes[i]) and np.array_equal(ref.from_tiles(host(s1), 1)[0], s[i])


# ------------------------------------------------------------------ product

def operand(M, K, kind, seed, lo=-3, hi=3):
    """Codes and scales of a matrix, and its values in 64 bits."""
    r = np.random.default_rng(seed)
    packed = r.integers(0, 256, (M, K // 2), dtype=np.uint8)
    C = K // ref.BLOCK[kind]
    byte = (127 + r.integers(lo, hi + 1, (M, C))).astype(np.uint8) if kind == "mxfp4" else \
        (r.integers(0x38 + 8 * lo, 0x38 + 8 * hi, (M, C))).astype(np.uint8)
    return (torch.from_numpy(packed).cuda(), torch.from_numpy(ref.to_tiles(byte, 0x7F if kind == "nvfp4" else 255)).cuda(),
            torch.from_numpy(ref.values(packed, byte, kind)).cuda())


def bound(vx, vw, K, out, want):
    """Products are exact; each of the K / 64 instructions adds its 64 products and the running sum, aligned to the
    largest and rounded to 24 bits: at most 2^-22 of the sum of sizes.  Then one rounding for alpha, one to bf16."""
    size = vx.abs() @ vw.abs().T
    return (K / 64 + 8) * 2.0 ** -22 * size + want.abs() * (2.0 ** -8 if out == "bf16" else 2.0 ** -22)


SHAPES = [(1, 128, 8), (7, 256, 24), (64, 384, 256), (65, 640, 264), (129, 128, 1000), (256, 1024, 512), (300, 2176, 520),
          (513, 512, 2048), (1000, 4096, 776)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_product(kind, out, M, K, N):
    x, sx, vx = operand(M, K, kind, M + K)
    w, sw, vw = operand(N, K, kind, N + 1)
    g = bg.BiGemm4(K, N, kind, out)
    y = g.run(x, sx, w, sw, alpha=0.75)
    assert g.device_error() == bg.BI_GEMM_OK
    want = 0.75 * (vx @ vw.T)
    off = (y.double() - want).abs() - bound(vx, vw, K, out, want)
    assert off.max() <= 0, (float(off.max()), int((off > 0).sum()))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K,N", [(1024, 264), (4096, 1024), (384, 2056)])
def test_a_rows_bits_do_not_depend_on_the_batch(kind, K, N):
    """Every M, every place, in both outputs: the bits of the row alone."""
    x, sx, _ = operand(600, K, kind, 1, -6, 6)
    w, sw, _ = operand(N, K, kind, 2, -6, 6)
    raw = ref.from_tiles(host(sx), 600)
    for out in ("bf16", "f32"):
        g = bg.BiGemm4(K, N, kind, out)
        whole = g.run(x, sx, w, sw)
        few = g.config["few_rows"]
        for M in sorted({1, 2, 7, 8, 9, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 599, max(1, few), few + 1}):
            for first in (0, 600 - M):
                part = torch.from_numpy(ref.to_tiles(raw[first:first + M], 0x11)).cuda()
                y = g.run(x[first:first + M].contiguous(), part, w, sw)
                assert torch.equal(y.view(torch.uint8), whole[first:first + M].contiguous().view(torch.uint8)), (M, first)


@pytest.mark.parametrize("out", ("bf16", "f32"))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K,N", [(5760, 4104), (2176, 4104), (1152, 9736)])
def test_large_and_small_tiles_have_the_same_bits(kind, K, N, out):
    """700 rows in tiles of 256 x 256 on CTA pairs; 1 to 128 of them in the smaller tiles, in stages of four and of two
    slots whose last ones are not full."""
    x, sx, _ = operand(700, K, kind, 3, -6, 6)
    w, sw, _ = operand(N, K, kind, 4, -6, 6)
    raw = ref.from_tiles(host(sx), 700)
    g = bg.BiGemm4(K, N, kind, out)
    assert -(-700 // 128) * -(-N // 128) > torch.cuda.get_device_properties(0).multi_processor_count
    whole = g.run(x, sx, w, sw)
    for M in (1, 20, 64, 100, 128):
        for first in (0, 700 - M):
            part = torch.from_numpy(ref.to_tiles(raw[first:first + M], 0x11)).cuda()
            y = g.run(x[first:first + M].contiguous(), part, w, sw)
            assert torch.equal(y.view(torch.uint8), whole[first:first + M].contiguous().view(torch.uint8)), (M, first)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [5, 200])
def test_a_nan_stays_in_its_row_and_column(kind, M):
    K, N = 512, 320
    x, sx, _ = operand(M, K, kind, 1)
    w, sw, _ = operand(N, K, kind, 2)
    g = bg.BiGemm4(K, N, kind)
    clean = g.run(x, sx, w, sw)
    a, b = ref.from_tiles(host(sx), M).copy(), ref.from_tiles(host(sw), N).copy()
    nan = 255 if kind == "mxfp4" else 0x7F
    a[3, 2], b[300, 0] = nan, nan
    y = g.run(x, torch.from_numpy(ref.to_tiles(a, nan)).cuda(), w, torch.from_numpy(ref.to_tiles(b, nan)).cuda())
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[3], hit[:, 300] = True, True
    assert torch.equal(torch.isnan(y), hit)
    assert torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("kind", KINDS)
def test_quantised_product_is_near_the_product(kind):
    """The two together: the quantiser's own output through the product, against its values in 64 bits."""
    K, N, M = 2048, 512, 190
    r = np.random.default_rng(0)
    xb, wb = bf16(r.standard_normal((M, K))), bf16(r.standard_normal((N, K)) * 0.02)
    gx, gw = (0.5, 0.01) if kind == "nvfp4" else (1.0, 1.0)
    qx, qw = bg.BiQuant4(K, kind, gx), bg.BiQuant4(K, kind, gw)
    (x, sx), (w, sw) = qx.run(xb), qw.run(wb)
    y = bg.BiGemm4(K, N, kind).run(x, sx, w, sw, alpha=gx * gw)
    vx, vw = (torch.from_numpy(ref.values(host(c), ref.from_tiles(host(s), n), kind, g)).cuda()
              for c, s, n, g in ((x, sx, M, gx), (w, sw, N, gw)))
    want = vx @ vw.T
    # (g rounds to fp32 in alpha and in the values alike: 2^-22 more)
    assert ((y.double() - want).abs() <= bound(vx, vw, K, "bf16", want) + 2.0 ** -22 * want.abs()).all()
    # and an element's own error is at most half a step of its block: 1/6 of the block's maximum
    bl = ref.BLOCK[kind]
    top = xb.double().abs().view(M, -1, bl).amax(-1, keepdim=True).expand(-1, -1, bl).reshape(M, K)
    limit = top / 6 * (1 + 2.0 ** -4) if kind == "nvfp4" else top / 4
    assert ((vx - xb.double()).abs() <= limit).all()


@pytest.mark.parametrize("M", [3, 300])
def test_graphs_and_streams(M):
    K, N = 1024, 512
    x = bf16(np.random.default_rng(1).standard_normal((M, K)))
    q, g = bg.BiQuant4(K), bg.BiGemm4(K, N)
    w, sw, _ = operand(N, K, "nvfp4", 2)
    codes, scales = q.run(x)
    want = g.run(codes, scales, w, sw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c2, s2 = q.run(x, stream=s)
    y = g.run(c2, s2, w, sw, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.run(x, codes, scales)
        g.run(codes, scales, w, sw, y=out)
    for scale in (1.0, -2.0):
        x.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        c3, s3 = q.run(x)
        assert torch.equal(out, g.run(c3, s3, w, sw))


def test_sizes_of_nothing_and_refusals():
    K, N = 256, 64
    q, g = bg.BiQuant4(K), bg.BiGemm4(K, N)
    codes, scales = q.run(torch.empty((0, K), dtype=torch.bfloat16, device="cuda"))
    assert codes.shape == (0, K // 2) and scales.shape[0] == 0
    w, sw, _ = operand(N, K, "nvfp4", 2)
    assert g.run(codes, scales, w, sw).shape == (0, N)
    x, sx, _ = operand(5, K, "nvfp4", 1)
    for bad in (dict(x=x[:, :64].contiguous()), dict(sx=sx[:, :1].contiguous()), dict(w=w[:32].contiguous()), dict(x=x.cpu()),
                dict(sw=sw.view(torch.int8)), dict(y=torch.empty((5, N), device="cuda"))):
        with pytest.raises(ValueError):
            g.run(**{**dict(x=x, sx=sx, w=w, sw=sw), **bad})
    with pytest.raises(bg.BiGemmError):
        g.run(x, sx, w, sw, alpha=float("nan"))
    xb = torch.zeros((4, K + 4), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bg.BiGemmError):          # rows 8-byte apart
        q.run(xb[:, :K])
    with pytest.raises(ValueError):
        q.run(xb[:, :K].t())


@pytest.mark.parametrize("M", [20, 700])
def test_waits_of_both_forms_end(M):
    """Failure injection (test controls): nothing is loaded, every wait ends after 50 ms, and the handle serves the next
    call as if nothing had been."""
    K, N = 1024, 4096
    x, sx, _ = operand(M, K, "nvfp4", 1)
    w, sw, _ = operand(N, K, "nvfp4", 2)
    g = bg.BiGemm4(K, N)
    assert (M > g.config["few_rows"]) == (M == 700)
    want = g.run(x, sx, w, sw)
    L, P, I64, I32, F = Controls().L, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    L.bi_ctl_gemm4_create.argtypes = [ctypes.POINTER(P), I64, I64, I32, I32]
    L.bi_ctl_gemm4_run.argtypes = [P, P, P, I64, P, P, F, P, P]
    L.bi_ctl_gemm4_stall.argtypes = [P, P, P, I64, P, P, F, P, ctypes.c_uint64, P]
    L.bi_ctl_gemm4_get_device_error.argtypes, L.bi_ctl_gemm4_destroy.argtypes = [P, P], [P]
    h, y = P(), torch.zeros_like(want)
    assert L.bi_ctl_gemm4_create(ctypes.byref(h), K, N, bg.BI_NVFP4, 0) == 0
    a = (h, x.data_ptr(), sx.data_ptr(), M, w.data_ptr(), sw.data_ptr(), 1.0, y.data_ptr())
    for _ in range(2):
        assert L.bi_ctl_gemm4_stall(*a, 50_000_000, stream_ptr()) == 0
        assert L.bi_ctl_gemm4_get_device_error(h, stream_ptr()) == bg.BI_GEMM_ERR_TIMEOUT
        assert L.bi_ctl_gemm4_run(*a, stream_ptr()) == 0
        assert L.bi_ctl_gemm4_get_device_error(h, stream_ptr()) == 0
        assert torch.equal(y, want)
        y.zero_()
    assert L.bi_ctl_gemm4_destroy(h) == 0
