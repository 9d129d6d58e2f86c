"""The product in 4 bits in every form that a call can take: each row against 64-bit sums and, between the forms, bit
for bit.  Which form a shape takes on this device is read through the test controls."""
import pytest
import torch

import fp4_ref as ref
import invariant_bi_gemm_gb300 as bg
from test_gemm4_forms_cpu import form
from test_gpu_q_fp4 import KINDS, bound, host, operand

pytestmark = pytest.mark.gpu


def form_of(K, N, kind, out, M):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return form(K, N, bg.BI_NVFP4 if kind == "nvfp4" else bg.BI_MXFP4, int(out == "f32"), M, sms)


def bits(y):
    return y.contiguous().view(torch.uint8)


def slice_of(x, raw, first, n):
    """Rows first .. first + n - 1 as an operand of their own; the scales of rows that are not there are NaN."""
    return x[first:first + n].contiguous(), torch.from_numpy(ref.to_tiles(raw[first:first + n], 0xFF)).cuda()


def check_rows(y, vx, vw, K, out):
    """y against 64-bit sums, in blocks of columns (64-bit copies of a wide w would not fit otherwise)."""
    for c in range(0, vw.shape[0], 16384):
        w = vw[c:c + 16384]
        want = vx @ w.T
        off = (y[:, c:c + 16384].double() - want).abs() - bound(vx, w, K, out, want)
        assert off.max() <= 0, (c, float(off.max()), int((off > 0).sum()))


# Rows past a tile's first half, past none of it (one CTA of the last pair has no rows), more M tiles than a raster's
# group.
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(257, 384, 10000), (300, 2176, 10248), (513, 128, 10000), (700, 640, 16392),
                                   (4225, 256, 1000), (4104, 1152, 776)])
def test_pairs_against_64_bits_and_the_smaller_tiles(kind, out, M, K, N):
    assert form_of(K, N, kind, out, M)[0] == 0
    x, sx, vx = operand(M, K, kind, M + K)
    w, sw, vw = operand(N, K, kind, N + 1)
    g = bg.BiGemm4(K, N, kind, out)
    y = g.run(x, sx, w, sw)
    assert g.device_error() == bg.BI_GEMM_OK
    check_rows(y, vx, vw, K, out)
    raw = ref.from_tiles(host(sx), M)
    for first in range(0, M, 128):
        n = min(128, M - first)
        assert form_of(K, N, kind, out, n)[0] > 0
        assert torch.equal(bits(g.run(*slice_of(x, raw, first, n), w, sw)), bits(y[first:first + n])), first


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_a_nan_stays_in_its_row_and_column_of_the_pairs(kind, out):
    M, K, N = 700, 512, 10000
    assert form_of(K, N, kind, out, M)[0] == 0
    x, sx, _ = operand(M, K, kind, 1)
    w, sw, _ = operand(N, K, kind, 2)
    g = bg.BiGemm4(K, N, kind, out)
    clean = g.run(x, sx, w, sw)
    a, b = ref.from_tiles(host(sx), M).copy(), ref.from_tiles(host(sw), N).copy()
    nan = 255 if kind == "mxfp4" else 0x7F
    rows, cols = [3, 200, 255, 256, 640, 699], [0, 129, 5000, 9999]
    for i, r in enumerate(rows):
        a[r, (5 * i) % a.shape[1]] = nan
    for i, c in enumerate(cols):
        b[c, (7 * i) % b.shape[1]] = nan
    y = g.run(x, torch.from_numpy(ref.to_tiles(a, nan)).cuda(), w, torch.from_numpy(ref.to_tiles(b, nan)).cuda())
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[rows], hit[:, cols] = True, True
    assert torch.equal(torch.isnan(y), hit)
    assert torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("K,N", [(640, 19464), (1280, 20480), (256, 32008), (384, 128256)])
def test_few_rows_by_a_vocabulary(kind, out, K, N):
    """More tiles of w's rows than SMs, so that a CTA takes several: 64-bit sums and the bits of the pairs."""
    M = 300
    assert form_of(K, N, kind, out, M)[0] == 0
    x, sx, vx = operand(M, K, kind, 5)
    w, sw, vw = operand(N, K, kind, 6)
    g = bg.BiGemm4(K, N, kind, out)
    whole = g.run(x, sx, w, sw)
    check_rows(whole, vx, vw, K, out)
    raw = ref.from_tiles(host(sx), M)
    taken = set()
    for n in (1, 8, 16, 17, 31, 32, 33, 64, 65, 128):
        rows, per_sm, _, _ = form_of(K, N, kind, out, n)
        taken.add((rows, per_sm))
        for first in (0, M - n):
            y = g.run(*slice_of(x, raw, first, n), w, sw)
            assert torch.equal(bits(y), bits(whole[first:first + n])), (n, first)
    assert g.device_error() == bg.BI_GEMM_OK
    assert taken == {(128, 1), (128, 2)}
