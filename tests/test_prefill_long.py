"""Prefill products: those whose activations exceed an XCD's L2 (M * K over 4 MiB), where workgroups take their tiles in
another order (sampled rows against 64 bits, and every row against the product of fewer rows), and outputs that are aligned
to 4 bytes only."""
import numpy as np
import pytest
import torch

import bit_quantized_matvec_q1_amd.lowbit as L
import weights_ref as W
from gpu_util import dev, host, say


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [L.Q1_0, L.Q2_0_G64, L.Q4_0])
@pytest.mark.parametrize("M,N,K", [(600, 1300, 8064), (1030, 1290, 4224), (2300, 450, 1920)])
def test_sampled_rows(fmt, M, N, K):
    say(f"case long prefill fmt={fmt} M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K)
    w, d = W.random_codes(rng, fmt, N, K), W.random_scales(rng, fmt, N, K)
    q, s = W.random_rows(rng, M, K)
    p = torch.zeros(L.lowbit_weight_bytes(fmt, N, K), dtype=torch.uint8, device="cuda")
    L.lowbit_pack_weights(fmt, dev(W.blocks(fmt, w, d).reshape(-1)), N, K, p)
    y = torch.full((M + 1, N), 5.0, device="cuda")
    L.lowbit_gemm(fmt, p, N, K, 1.0, L.ACT_Q8_0, dev(q), dev(s), M, y)
    assert (host(y)[M] == 5).all()
    rows = [0, 1, 127, 128, 255, 256, M // 2, M - 2, M - 1]
    want, mags = W.product(fmt, w, d, q[rows], s[rows])
    off = np.abs(host(y)[rows] - want) / W.allowance(mags, K)
    say(f"  worst error {off.max():.3g} of what is allowed")
    assert (off <= 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [L.Q1_0, L.Q2_0_G64, L.Q8_0, L.TERNARY_PLANAR])
@pytest.mark.parametrize("M,N,K", [(700, 70, 6272), (1300, 1000, 3584), (600, 200, 7232)])
def test_rows_as_with_fewer(fmt, M, N, K):
    """A row's result does not depend on the tiles' order: parts of 384 rows have less than 4 MiB.  (Both the whole and the
    parts have few tiles, so that both divide K alike.)"""
    if fmt in (L.Q1_0, L.Q8_0) and K % 128:
        K -= K % 128
    say(f"case long prefill in parts fmt={fmt} M={M} N={N} K={K}")
    g = torch.Generator(device="cuda").manual_seed(M + K)
    planar = fmt == L.TERNARY_PLANAR
    w = torch.randint(0, 60, (L.lowbit_weight_bytes(fmt, N, K),), dtype=torch.uint8, generator=g, device="cuda")
    q = torch.randint(-127, 128, (M, K), dtype=torch.int8, generator=g, device="cuda")
    s = torch.rand(M, 1 if planar else K // 32, generator=g, device="cuda") * 0.1 + 0.01
    s = s.flatten() if planar else s.half()
    act = L.ACT_I8_ROW if planar else L.ACT_Q8_0
    whole, parts = torch.full((M + 1, N), 5.0, device="cuda"), torch.zeros(M, N, device="cuda")
    assert M * K > 1 << 22
    L.lowbit_gemm(fmt, w, N, K, 1.0, act, q, s, M, whole)
    for a in range(0, M, 384):
        n = min(384, M - a)
        L.lowbit_gemm(fmt, w, N, K, 1.0, act, q[a:a + n].contiguous(), s[a:a + n].contiguous(), n, parts[a:a + n])
    assert (whole[M] == 5).all() and torch.isfinite(parts).all()
    assert torch.equal(whole[:M], parts)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [L.Q1_0, L.Q2_0_G64, L.Q8_0, L.Q4_0, L.TERNARY_PLANAR])
def test_outputs_that_lie_on_4_bytes(fmt):
    """Outputs one to three elements off 16 bytes, rows of every remainder: the values of aligned ones, and nothing beside."""
    planar = fmt == L.TERNARY_PLANAR
    for M, N, K in ((300, 16001, 128), (129, 130, 384), (40, 67, 256), (600, 2600, 128)):
        say(f"case outputs on 4 bytes fmt={fmt} M={M} N={N} K={K}")
        g = torch.Generator(device="cuda").manual_seed(N)
        w = torch.randint(0, 60, (L.lowbit_weight_bytes(fmt, N, K),), dtype=torch.uint8, generator=g, device="cuda")
        q = torch.randint(-127, 128, (M, K), dtype=torch.int8, generator=g, device="cuda")
        s = torch.rand(M, device="cuda") if planar else torch.rand(M, K // 32, device="cuda").half()
        act = L.ACT_I8_ROW if planar else L.ACT_Q8_0
        want = torch.zeros(M, N, device="cuda")
        L.lowbit_gemm(fmt, w, N, K, 1.0, act, q, s, M, want)
        for off in (1, 2, 3):
            buf = torch.full((off + M * N + 5,), 5.0, device="cuda")
            L.lowbit_gemm(fmt, w, N, K, 1.0, act, q, s, M, buf[off:off + M * N])
            assert torch.equal(buf[off:off + M * N].view(M, N), want)
            assert (buf[:off] == 5).all() and (buf[off + M * N:] == 5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [L.Q1_0, L.Q2_0_G64, L.Q4_0])
@pytest.mark.parametrize("pairs", [30, 250])
def test_experts_outputs_that_lie_on_4_bytes(fmt, pairs):
    E, N, K = 3, 333, 384
    say(f"case experts' outputs on 4 bytes fmt={fmt} pairs={pairs}")
    g = torch.Generator(device="cuda").manual_seed(pairs)
    w = torch.randint(0, 60, (L.lowbit_experts_weight_bytes(fmt, E, N, K),), dtype=torch.uint8, generator=g, device="cuda")
    e = torch.randint(-1, E, (pairs,), dtype=torch.int32, generator=g, device="cuda")
    q = torch.randint(-127, 128, (pairs, K), dtype=torch.int8, generator=g, device="cuda")
    s = torch.rand(pairs, K // 32, generator=g, device="cuda").half()
    plan = torch.zeros(L.lowbit_experts_plan_bytes(pairs, E), dtype=torch.uint8, device="cuda")
    L.lowbit_experts_plan(e, pairs, E, plan)
    want = torch.full((pairs, N), 5.0, device="cuda")
    L.lowbit_experts_matmul(fmt, w, E, N, K, q, s, e, pairs, 1, want, plan=plan)
    for off in (1, 2, 3):
        buf = torch.full((off + pairs * N + 5,), 5.0, device="cuda")
        L.lowbit_experts_matmul(fmt, w, E, N, K, q, s, e, pairs, 1, buf[off:off + pairs * N], plan=plan)
        assert torch.equal(buf[off:off + pairs * N].view(pairs, N), want)
        assert (buf[:off] == 5).all() and (buf[off + pairs * N:] == 5).all() and (want[e < 0] == 5).all()
