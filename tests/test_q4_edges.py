"""Rows, weights, streams and buffers at the edges of what the 4-bit and expert calls take.

Bounds as in test_q4.py: one bf16 rounding is 2^-8 of the value; fp32 sums are within
2^-12 of the sum of magnitudes S; weights rounded to fp16 (many rows, on the tensor cores)
add 2^-11 S.
"""
import numpy as np
import pytest
import torch

from bit_weight_only_ternary_b200 import synth


@pytest.fixture(scope="module")
def L():
    from bit_weight_only_ternary_b200 import build
    build.build()
    from bit_weight_only_ternary_b200 import lbq
    return lbq


def _us(f, n=8):
    """The fastest of n runs in us, on the device."""
    f()
    best = float("inf")
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b))
    return best


# ------------------------------------------------------- what a row of activations holds

@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 1, 6, 7])
@pytest.mark.parametrize("experts", [False, True])
def test_the_smallest_value_of_all_counts(L, at, experts):
    """A row of ones with one 2^-133 beside a zero, on weights that are zero everywhere but
    there: fp16 cannot hold both, so the row is recomputed in fp32."""
    K, N, M = 256, 40, 70
    q = torch.full((N, K), 8, dtype=torch.int32)
    q[:, at] = 15
    word = torch.zeros(N, K // 8, dtype=torch.int32)
    for i in range(8):
        word |= q[:, i::8] << (4 * ((i >> 1) + 4 * (i & 1)))
    codes = word.view(N // 4, 4, K // 8).transpose(1, 2).contiguous().view(torch.uint8).view(N // 4, 2 * K)
    scales = torch.full((N // 4, 32), 65504.0, dtype=torch.float16).view(torch.int16)
    X = torch.ones(M, K, dtype=torch.bfloat16)
    X[:, at ^ 1], X[:, at] = 0.0, 2.0 ** -133
    if experts:
        ew = L.ExpertWeights(5, K, N, 1, codes[None].cuda(), scales[None].cuda())
        Y = L.lbq_expert_gemm(ew, X.cuda(), torch.tensor([0, M], dtype=torch.int32, device="cuda"))
    else:
        Y = L.lbq_gemm(L.PackedWeights(5, K, N, codes.cuda(), scales.cuda()), X.cuda())
    want = 7 * 65504.0 * 2.0 ** -133  # (a normal bf16 value's range; exact in fp32)
    assert ((Y.double() - want).abs() <= 2.0 ** -8 * want).all(), Y[0, :2].tolist()
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("experts", [False, True])
def test_rows_of_zeros_take_no_longer(L, experts):
    """Padding tokens are ordinary rows (recomputed apart, they took 130 times as long)."""
    K, N, M, E = 2048, 2048, 1024, 4
    gen = torch.Generator("cuda").manual_seed(3)
    W = torch.randn(E if experts else 1, N, K, device="cuda", generator=gen) * 0.02
    X = torch.randn(M, K, device="cuda", generator=gen).to(torch.bfloat16)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    if experts:
        w = L.pack_experts(6, W)
        off = torch.arange(0, M + 1, M // E, dtype=torch.int32, device="cuda")
        ws = L.workspace_for_experts(w, M)
        run = lambda: L.lbq_expert_gemm(w, X, off, Y=Y, workspace=ws)  # noqa: E731
    else:
        w = L.lbq_pack(6, W[0])
        ws = L.workspace_for(w, M)
        run = lambda: L.lbq_gemm(w, X, Y=Y, workspace=ws)  # noqa: E731
    ordinary = _us(run)
    full = Y.clone()
    X[::2] = 0
    zeros = _us(run)
    assert (Y[::2] == 0).all() and torch.equal(Y[1::2], full[1::2])
    assert zeros <= 2 * ordinary, f"{zeros:.1f} us, {ordinary:.1f} without rows of zeros"
