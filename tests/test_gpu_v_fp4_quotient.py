"""The one divisor at which a corrected quotient could miss the rounded one (tests/test_fp4_quotient_cpu.py has the
proof): mantissa 2^24 - 1, at a quarter of a unit.  On the device the reciprocal has to be the one that does not."""
import numpy as np
import pytest
import torch

import fp4_ref as ref
import invariant_bi_gemm_gb300 as bg
from test_gpu_r_cache4 import empty_cache4, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [0, 1, -7, 30, -50, 63, -63])
def test_a_divisor_of_ones(k):
    """Blocks whose scale is a power of two, times g = 2^k (1 - 2^-24): elements of a quarter of a unit and around."""
    g = (1 - 2.0 ** -24) * 2.0 ** k                         # (exact in 24 bits)
    unit = np.exp2(np.arange(-6, 9)).astype(np.float64) * g
    part = np.array([6, .25, -.25, .5, .25 * (1 + 2 ** -7), .25 * (1 - 2 ** -8), .75, 1.25, 1.75, 2.5, 3.5, 5, -5, -.75, 0,
                     -0.0])
    x = torch.from_numpy(np.pad(unit[:, None] * part, ((0, 0), (0, 112)))).float().to(torch.bfloat16).cuda()
    want, byte = ref.quantise(x.float().cpu().numpy(), "nvfp4", g)
    assert (byte[:, 0] % 8 == 0).all()                       # powers of two: the divisor keeps g's mantissa
    codes, scales = bg.BiQuant4(128, "nvfp4", g).run(x)
    assert np.array_equal(ref.from_tiles(scales.cpu().numpy(), len(x)), byte)
    got = ref.unpack(codes.cpu().numpy())
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    # the append's
    rope, four = bg.BiQkRope(1, 1, 128, 16), empty_cache4(1, 16, 1, 128)
    cs = torch.cat([torch.ones(16, 64), torch.zeros(16, 64)], 1).cuda()
    n = len(x)
    rope.run4(x.repeat(1, 3).contiguous(), None, None, cs, i32([0] * n), i32(list(range(n))), *four, i32([[0]]), g, g)
    for c, s in (four[:2], four[2:]):
        assert np.array_equal(c[0, :n, 0].cpu().numpy(), ref.pack(want))
        assert np.array_equal(s[0, :n, 0].cpu().numpy(), byte)
