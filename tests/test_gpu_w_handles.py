"""Handles with a workspace that are dropped right behind their call: its results are those of a handle that stays."""
import pytest
import torch

import inputgen as ig
import invariant_bi_gemm_gb300 as bg
from gpu_util import dev_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("make", [lambda K, N: bg.BiPreNorm(K, N), lambda K, N: bg.BiGemm(K, N, "bf16_f32")])
def test_a_dropped_handles_workspace_outlives_its_call(make):
    K, N, M = 16384, 24, 4096
    x, w = dev_bf16(ig.scaled_rows_bf16(ig.SEED_X, M, K)), dev_bf16(ig.normal_bf16(ig.SEED_W, K, N, std=0.02))
    keep = make(K, N)
    want = keep(x, w)
    torch.cuda.synchronize()
    for _ in range(5):
        got = make(K, N)(x, w)                  # (dropped here; what follows takes memory of its size)
        again = make(K, N)(x.flip(0), w)
        assert torch.equal(got, want) and torch.equal(again, want.flip(0))
