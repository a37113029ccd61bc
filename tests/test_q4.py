"""4-bit weights (Q4_0): layout, exact block sums, products of one row and of many, work lists, against 64 bits."""
import numpy as np
import pytest
import torch

import bit_quantized_matvec_q1_amd.lowbit as L
import weights_ref as W
from gpu_util import dev, host, say

A16 = 1 << 20
Q4 = L.Q4_0


def test_sizes_and_refusals():
    assert L.lowbit_weight_bytes(Q4, 4096, 4096) == 4096 * 4096 // 32 * 18
    assert L.lowbit_weight_bytes(Q4, 3, 32) == 54
    assert L.lowbit_weight_bytes(Q4, 3, 48) == -1 and L.lowbit_weight_bytes(Q4, -1, 32) == -1
    call = lambda N, K, **a: L.lib.lowbit_matvec(Q4, a.get("W", A16), N, K, 1.0, a.get("afmt", L.ACT_Q8_0), a.get("x", A16), A16, A16, None)  # noqa: E731
    assert call(8, 48) == L.LB_ESHAPE and call(8, 16384 + 32) == L.LB_ESHAPE and call(-1, 32) == L.LB_ESHAPE
    assert call(1 << 22, 16384) == L.LB_ESHAPE  # 4 GiB and more
    assert call(8, 32, afmt=L.ACT_I8_ROW) == L.LB_EINVAL and call(8, 32, W=None) == L.LB_EINVAL
    assert call(8, 32, W=A16 + 8) == L.LB_EALIGN and call(8, 32, x=A16 + 8) == L.LB_EALIGN
    assert call(0, 32, W=None) == L.LB_OK
    gemm = lambda K, M: L.lib.lowbit_gemm(Q4, A16, 8, K, 1.0, L.ACT_Q8_0, A16, A16, M, A16, None)  # noqa: E731
    assert gemm(96, 4) == L.LB_ESHAPE and gemm(160, 2) == L.LB_ESHAPE and gemm(128, -1) == L.LB_ESHAPE
    assert L.lib.lowbit_block_sums(Q4, A16, 8, 96, L.ACT_Q8_0, A16, A16, 2, A16, None) == L.LB_ESHAPE
    assert L.lib.lowbit_pack_weights(Q4, A16, 2, 48, A16, None) == L.LB_ESHAPE


def test_binding_checks_extents():
    w = torch.zeros(L.lowbit_weight_bytes(Q4, 8, 64), dtype=torch.uint8)
    xq, xs, y = torch.zeros(64, dtype=torch.int8), torch.zeros(2, dtype=torch.float16), torch.zeros(8)
    for bad in (dict(w=w[:-1]), dict(xq=xq[:-1]), dict(xs=xs[:1]), dict(y=y[:7]), dict(xs=xs.float())):
        a = dict(w=w, xq=xq, xs=xs, y=y) | bad
        with pytest.raises(ValueError):
            L.lowbit_matvec(Q4, a["w"], 8, 64, 1.0, L.ACT_Q8_0, a["xq"], a["xs"], a["y"])


def case(N, K, M=1, seed=0):
    rng = np.random.default_rng(seed + 7 * N + K)
    w, d = W.random_codes(rng, Q4, N, K), W.random_scales(rng, Q4, N, K)
    w[0], w[-1] = -8, 7  # the ends of the range
    if N > 2:
        w[1] = 0
        d[2, ::3] = -d[2, ::3]
    q, s = W.random_rows(rng, M, K)
    q[0, :32], q[-1, -32:] = -128, 127
    return w, d, q, s


def packed(w, d):
    N, K = w.shape
    out = torch.zeros(L.lowbit_weight_bytes(Q4, N, K), dtype=torch.uint8, device="cuda")
    L.lowbit_pack_weights(Q4, dev(W.blocks(Q4, w, d).reshape(-1)), N, K, out)
    return out


def close(got, w, d, q, s, what):
    want, mags = W.product(Q4, w, d, q, s)
    off = np.abs(got - want) / W.allowance(mags, w.shape[1])
    say(f"  {what}: worst error {off.max():.3g} of what is allowed")
    assert (off <= 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(1, 32), (5, 96), (33, 4096)])
def test_layout(N, K):
    w, d, _, _ = case(N, K)
    p = packed(w, d)
    assert np.array_equal(host(p), W.layout(Q4, w, d))
    back = torch.zeros_like(p)
    L.lowbit_unpack_weights(Q4, p, N, K, back)
    assert np.array_equal(host(back), W.blocks(Q4, w, d).reshape(-1))


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(1, 32), (3, 64), (130, 96), (7, 800), (517, 2560), (300, 4096), (65, 6912), (129, 11008), (20, 16384), (9, 16352)])
def test_one_row(N, K):
    say(f"case one row N={N} K={K}")
    w, d, q, s = case(N, K)
    p = packed(w, d)
    z = torch.full((N + 1, K // 32), 5, dtype=torch.int32, device="cuda")
    L.lowbit_block_sums(Q4, p, N, K, L.ACT_Q8_0, dev(q), dev(s), 1, z)
    assert np.array_equal(host(z)[:N], W.sums(w, q)[0]) and (host(z)[N] == 5).all()
    y = torch.full((N + 1,), 5.0, device="cuda")
    L.lowbit_matvec(Q4, p, N, K, 1.0, L.ACT_Q8_0, dev(q), dev(s), y)
    assert host(y)[N] == 5
    close(host(y)[None, :N], w, d, q, s, f"{N}x{K}")


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(2, 1, 128), (3, 65, 256), (70, 130, 384), (128, 64, 4096), (129, 300, 640), (260, 1000, 1408),
                                   (16, 4100, 2048), (33, 8200, 1152), (17, 1030, 16384), (5, 20, 896), (193, 4100, 256), (300, 2500, 128),
                                   (1, 77, 512), (4100, 70, 384)])
def test_many_rows(M, N, K):
    say(f"case many rows M={M} N={N} K={K}")
    w, d, q, s = case(N, K, M)
    p = packed(w, d)
    z = torch.zeros(M, N, K // 32, dtype=torch.int32, device="cuda")
    L.lowbit_block_sums(Q4, p, N, K, L.ACT_Q8_0, dev(q), dev(s), M, z)
    assert np.array_equal(host(z), W.sums(w, q))
    y = torch.full((M + 1, N), 5.0, device="cuda")
    L.lowbit_gemm(Q4, p, N, K, 1.0, L.ACT_Q8_0, dev(q), dev(s), M, y)
    assert (host(y)[M] == 5).all()
    close(host(y)[:M], w, d, q, s, f"{M}x{N}x{K}")


@pytest.mark.gpu
def test_empty_products():
    y = torch.full((4,), 5.0, device="cuda")
    L.lowbit_matvec(Q4, None, 0, 64, 1.0, L.ACT_Q8_0, None, None, None, stream=0)
    L.lowbit_matvec(Q4, y, 3, 0, 1.0, L.ACT_Q8_0, torch.zeros(16, dtype=torch.int8, device="cuda"), torch.zeros(8, dtype=torch.float16, device="cuda"), y)
    assert host(y).tolist() == [0, 0, 0, 5]


@pytest.mark.gpu
def test_scales_that_are_not_finite_stay_in_their_rows():
    w, d, q, s = case(40, 256)
    d[7, 3], d[9, 0], d[20, 5] = np.inf, np.nan, 0
    y = torch.zeros(40, device="cuda")
    L.lowbit_matvec(Q4, packed(w, d), 40, 256, 1.0, L.ACT_Q8_0, dev(q), dev(s), y)
    got = host(y)
    assert not np.isfinite(got[7]) and np.isnan(got[9])
    ok = np.setdiff1d(np.arange(40), [7, 9])
    close(got[None, ok], w[ok], d[ok], q, s, "the others")


@pytest.mark.gpu
def test_work_lists_agree_with_single_products():
    """Lists of several sizes, activations in bytes and in fp32, both kinds of list, captured and replayed: the same bits
    as one call each (a row's lanes and their order depend on K alone)."""
    rng = np.random.default_rng(5)
    shapes = [(300, 1024), (64, 96), (1, 32), (1000, 4096), (129, 9216), (77, 16384)]
    descs, outs, want = [], [], []
    for i, (N, K) in enumerate(shapes):
        w, d, q, s = case(N, K, seed=i)
        p, y = packed(w, d), torch.zeros(N, device="cuda")
        one = torch.zeros(N, device="cuda")
        if i % 2:
            x = dev(rng.standard_normal(K).astype(np.float32))
            xq, xs = torch.zeros(K, dtype=torch.int8, device="cuda"), torch.zeros(K // 32, dtype=torch.float16, device="cuda")
            L.lowbit_quantize_act(L.ACT_Q8_0, x, 1, K, xq, xs)
            descs.append(L.desc(Q4, p, N, K, None, None, y, x=x))
        else:
            xq, xs = dev(q[0]), dev(s[0])
            descs.append(L.desc(Q4, p, N, K, xq, xs, y))
        L.lowbit_matvec(Q4, p, N, K, 1.0, L.ACT_Q8_0, xq, xs, one)
        outs.append(y)
        want.append(host(one))
    batch = L.Batch(descs)

    def same(what):
        for (N, K), y, ref in zip(shapes, outs, want):
            assert np.array_equal(host(y), ref), (what, N, K)
            y.fill_(7)

    batch.run()
    same("batch")
    arr = (L.lb_matvec_desc * len(descs))(*descs)
    L._check(L.lib.lowbit_matvec_batched_static(arr, len(descs), torch.cuda.current_stream().cuda_stream), "static")
    same("static")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        batch.run()
    for i in range(3):
        g.replay()
        same(f"replay {i}")
    batch.close()
