"""The experts' products of routed pairs: the plan, the products in every format, the sum over a token's experts, and a
whole layer, against 64 bits."""
import numpy as np
import pytest
import torch

import bit_quantized_matvec_q1_amd.lowbit as L
import test_route
import weights_ref as W
from gpu_util import dev, host, say

A = 1 << 20
FMTS = [L.Q1_0, L.Q2_0_G64, L.Q4_0]
TYPES = {"f32": (L.F32, torch.float32), "bf16": (L.BF16, torch.bfloat16), "f16": (L.F16, torch.float16)}


def test_sizes():
    assert L.lowbit_experts_weight_bytes(L.Q4_0, 3, 5, 128) == 3 * 368  # 5 * 4 * 18 = 360, padded
    assert L.lowbit_experts_weight_bytes(L.Q2_0_G64, 0, 5, 128) == 0
    assert L.lowbit_experts_weight_bytes(L.Q4_0, 1, 1 << 22, 16384) == -1 and L.lowbit_experts_weight_bytes(9, 1, 1, 128) == -1
    assert L.lowbit_experts_weight_bytes(L.Q1_0, 1, 1, 64) == -1 and L.lowbit_experts_weight_bytes(L.Q1_0, 1025, 1, 128) == -1
    for pairs, E in ((0, 1), (1, 1), (7, 1024), (2**30, 1024)):
        assert L.lowbit_experts_plan_bytes(pairs, E) >= 4 * pairs
    for pairs, E in ((-1, 4), (2**30 + 1, 4), (4, 0), (4, 1025)):
        assert L.lowbit_experts_plan_bytes(pairs, E) == -1


def test_refusals():
    lib = L.lib
    plan = lambda e=A, n=8, E=4, p=A: lib.lowbit_experts_plan(e, n, E, p, None)  # noqa: E731
    assert plan(n=-1) == L.LB_ESHAPE and plan(E=0) == L.LB_ESHAPE and plan(E=1025) == L.LB_ESHAPE and plan(n=2**31 - 1) == L.LB_ESHAPE
    assert plan(e=None) == L.LB_EINVAL and plan(p=None) == L.LB_EINVAL and plan(e=A + 2) == L.LB_EALIGN and plan(p=A + 8) == L.LB_EALIGN
    assert plan(n=0, e=None, p=None) == L.LB_OK

    def mm(fmt=L.Q2_0_G64, w=A, E=4, N=8, K=128, xq=A, xs=A, e=A, n=8, per=2, p=A, y=A):
        return lib.lowbit_experts_matmul(fmt, w, E, N, K, xq, xs, e, n, per, p, y, None)

    assert mm(fmt=0) == L.LB_EINVAL and mm(fmt=7) == L.LB_EINVAL
    for fmt in (L.TERNARY_PLANAR, L.Q8_0, L.TERNARY_B3):
        assert mm(fmt=fmt) == L.LB_EUNSUPPORTED
    for bad in (dict(N=-1), dict(K=0), dict(K=96), dict(fmt=L.Q1_0, K=192), dict(fmt=L.Q4_0, K=64), dict(fmt=L.Q4_0, K=16384 + 128), dict(K=32768 + 64),
                dict(E=0), dict(E=1025), dict(n=-1), dict(per=0), dict(fmt=L.Q4_0, N=1 << 22, K=16384), dict(n=1 << 30, K=128, per=1),
                dict(N=1 << 26, n=1 << 10)):
        assert mm(**bad) == L.LB_ESHAPE, bad
    for name in ("w", "xq", "xs", "y"):
        assert mm(**{name: None}) == L.LB_EINVAL
    assert mm(e=None, p=None) == L.LB_EINVAL
    assert mm(w=A + 8) == L.LB_EALIGN and mm(xq=A + 8) == L.LB_EALIGN and mm(p=A + 8) == L.LB_EALIGN and mm(y=A + 2) == L.LB_EALIGN
    assert mm(N=0, w=None) == L.LB_OK and mm(n=0, xq=None) == L.LB_OK

    def co(dtype=0, y=A, e=A, w=A, T=4, k=2, E=4, N=8, o=A, so=8):
        return lib.lowbit_experts_combine(dtype, y, e, w, T, k, E, N, o, so, None)

    assert co(dtype=5) == L.LB_EINVAL and co(T=-1) == L.LB_ESHAPE and co(k=0) == L.LB_ESHAPE and co(E=0) == L.LB_ESHAPE and co(so=7) == L.LB_ESHAPE
    assert co(T=1 << 20, N=1 << 14, so=1 << 14) == L.LB_ESHAPE
    for name in ("y", "e", "w", "o"):
        assert co(**{name: None}) == L.LB_EINVAL and co(**{name: A + 2}) == L.LB_EALIGN
    assert co(T=0, y=None) == L.LB_OK


def test_binding_checks_extents():
    t = dict(W=torch.zeros(L.lowbit_experts_weight_bytes(L.Q4_0, 2, 8, 128), dtype=torch.uint8), xq=torch.zeros(3, 128, dtype=torch.int8),
             xs=torch.zeros(3, 4, dtype=torch.float16), e=torch.zeros(6, dtype=torch.int32), y=torch.zeros(6, 8),
             plan=torch.zeros(L.lowbit_experts_plan_bytes(6, 2), dtype=torch.uint8))
    bad = dict(W=t["W"][:-1], xq=t["xq"][:2], xs=t["xs"].float(), e=t["e"][:5], y=t["y"][:5], plan=t["plan"][:-16])
    for name, x in bad.items():
        a = t | {name: x}
        with pytest.raises(ValueError):
            L.lowbit_experts_matmul(L.Q4_0, a["W"], 2, 8, 128, a["xq"], a["xs"], a["e"], 6, 2, a["y"], plan=a["plan"])
    with pytest.raises(ValueError):
        L.lowbit_experts_plan(t["e"], 6, 2, t["plan"][:-16])
    with pytest.raises(ValueError):
        L.lowbit_experts_combine(L.F32, t["y"], t["e"], torch.zeros(5), 3, 2, 2, 8, torch.zeros(3, 8))


def planned(e, E):
    plan = torch.full((L.lowbit_experts_plan_bytes(len(e), E) + 16,), 0x55, dtype=torch.uint8, device="cuda")
    L.lowbit_experts_plan(dev(e), len(e), E, plan[:-16])
    assert (host(plan)[-16:] == 0x55).all()
    return plan[:-16]


@pytest.mark.gpu
@pytest.mark.parametrize("pairs,E", [(1, 1), (7, 3), (64, 64), (300, 60), (1025, 7), (5000, 1024), (5000, 8), (70001, 128)])
def test_plan(pairs, E):
    """Pairs by expert, in their order, in tiles of one expert; pairs without one are in none."""
    say(f"case plan {pairs} pairs {E} experts")
    rng = np.random.default_rng(pairs)
    e = (rng.random(pairs) ** 2 * E).astype(np.int32)
    e[rng.random(pairs) < 0.1] = -1
    e[pairs // 2] = [E, 2**31 - 1, -2**31][pairs % 3]
    for which in (e, np.full(pairs, E - 1, np.int32), np.full(pairs, -1, np.int32)):
        p = host(planned(which, E)).view(np.int32)
        ok = (which >= 0) & (which < E)
        want = np.argsort(np.where(ok, which, E), kind="stable")[:ok.sum()]
        assert p[1] == ok.sum()
        size = 128 if pairs >= 64 * E else 16  # rows a tile
        n = pairs // size + min(pairs, E)
        tiles, places = p[4:4 + 2 * n].reshape(-1, 2), p[4 + (2 * n + 3) // 4 * 4:][:n * size].reshape(n, size)
        assert (tiles[p[0]:, 1] == 0).all() and (tiles[:, 1] >= 0).all()
        at = 0
        for (x, rows), pair in zip(tiles, places):
            if rows:  # they cover the order one after another
                assert np.array_equal(pair[:rows], want[at:at + rows]) and (which[pair[:rows]] == x).all() and (pair[rows:] == -1).all()
                at += rows
        assert at == p[1]
        used = tiles[tiles[:, 1] != 0]
        for a, b in zip(used, used[1:]):  # and are full but for each expert's last
            assert a[0] != b[0] or a[1] == size


class Layer:
    """E experts of N x K in `fmt`."""

    def __init__(self, fmt, E, N, K, seed=0):
        rng = np.random.default_rng(seed + N + K)
        self.fmt, self.E, self.N, self.K = fmt, E, N, K
        self.w = [W.random_codes(rng, fmt, N, K) for _ in range(E)]
        self.d = [W.random_scales(rng, fmt, N, K) for _ in range(E)]
        step = L.lowbit_experts_weight_bytes(fmt, 1, N, K)
        self.packed = torch.full((L.lowbit_experts_weight_bytes(fmt, E, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
        n = L.lowbit_weight_bytes(fmt, N, K)
        for i in range(E):
            L.lowbit_pack_weights(fmt, dev(W.blocks(fmt, self.w[i], self.d[i]).reshape(-1)), N, K, self.packed[i * step:i * step + n])

    def check(self, e, per, plan, seed=1, stream=None):
        rng = np.random.default_rng(seed)
        n = len(e)
        q, s = W.random_rows(rng, -(-n // per), self.K)
        y = torch.full((n + 1, self.N), 7.0, device="cuda")
        xq, xs, ed = dev(q), dev(s), dev(e)
        torch.cuda.synchronize()
        L.lowbit_experts_matmul(self.fmt, self.packed, self.E, self.N, self.K, xq, xs, ed if plan is None else None, n, per, y, plan=plan, stream=stream)
        got = host(y)
        assert (got[n] == 7).all() and (got[:n][(e < 0) | (e >= self.E)] == 7).all()  # rows of pairs that are left out
        worst = 0.0
        for x in range(self.E):
            p = np.flatnonzero(e == x)
            if len(p):
                want, mags = W.product(self.fmt, self.w[x], self.d[x], q[p // per], s[p // per])
                worst = max(worst, (np.abs(got[p] - want) / W.allowance(mags, self.K)).max())
        say(f"  worst error {worst:.3g} of what is allowed")
        assert worst <= 1
        return got


def some_pairs(rng, n, E):
    e = (rng.random(n) ** 2 * E).astype(np.int32)
    if n > 3:
        e[n // 2], e[n // 3] = -1, E
    return e


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS, ids=W.NAMES.get)
@pytest.mark.parametrize("E,N,K,n,per", [
    (1, 1, 128, 1, 1), (4, 33, 128, 8, 8), (5, 130, 384, 3, 1), (8, 65, 640, 40, 4), (16, 300, 768, 100, 1), (3, 17, 1408, 11, 2), (6, 40, 2048, 30, 3),
    (4, 23, 7168, 9, 1), (2, 5, 16384, 7, 1)])
def test_few_rows(fmt, E, N, K, n, per):
    """Without a plan, each pair by itself, and with one."""
    say(f"case few rows {W.NAMES[fmt]} E={E} N={N} K={K} pairs={n} per={per}")
    layer = Layer(fmt, E, N, K)
    e = some_pairs(np.random.default_rng(n), n, E)
    alone = layer.check(e, per, None)
    layer.check(e, per, planned(e, E))
    q, s = W.random_rows(np.random.default_rng(1), -(-n // per), K)
    step, y = L.lowbit_experts_weight_bytes(fmt, 1, N, K), torch.zeros(N, device="cuda")
    for p in {0, n - 1}:
        if 0 <= e[p] < E:
            L.lowbit_matvec(fmt, layer.packed[e[p] * step:], N, K, 1.0, L.ACT_Q8_0, dev(q[p // per]), dev(s[p // per]), y)
            assert np.array_equal(host(y), alone[p])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS, ids=W.NAMES.get)
@pytest.mark.parametrize("E,N,K,n,per", [
    (1, 1, 128, 17, 1), (2, 65, 256, 200, 2), (8, 130, 384, 700, 7), (8, 130, 384, 400, 7), (3, 300, 2048, 600, 1), (60, 64, 128, 1000, 4),
    (40, 1000, 1152, 500, 1), (20, 1000, 1408, 150, 2)])
def test_many_rows(fmt, E, N, K, n, per):
    say(f"case many rows {W.NAMES[fmt]} E={E} N={N} K={K} pairs={n} per={per}")
    layer = Layer(fmt, E, N, K)
    rng = np.random.default_rng(n)
    layer.check(some_pairs(rng, n, E), per, planned(some_pairs(np.random.default_rng(n), n, E), E))
    e = np.full(n, E - 1, np.int32)  # all to one expert
    layer.check(e, per, planned(e, E))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS, ids=W.NAMES.get)
@pytest.mark.parametrize("N,K", [(20, 1152), (600, 384), (1500, 2304), (1700, 1152), (50, 6912), (1700, 128)])
def test_every_number_of_rows(fmt, N, K):
    """Experts with one pair to 19: tiles of every number of rows, in each of the product's forms."""
    E = 19
    if fmt == L.Q2_0_G64 and K > 1000:
        K += 64 * (1 + N % 3)  # rows of every remainder of blocks
    say(f"case every number of rows {W.NAMES[fmt]} N={N} K={K}")
    layer = Layer(fmt, E, N, K)
    e = np.repeat(np.arange(E, dtype=np.int32), np.arange(1, E + 1))
    np.random.default_rng(N).shuffle(e)
    layer.check(e, 1, planned(e, E))


@pytest.mark.gpu
def test_odd_numbers_of_blocks():
    """Q2_0_g64 rows of an odd number of 64-weight blocks, few and many."""
    for n in (5, 90):
        layer = Layer(L.Q2_0_G64, 3, 70, 64 * 11)
        e = some_pairs(np.random.default_rng(n), n, 3)
        layer.check(e, 1, planned(e, 3))


@pytest.mark.gpu
def test_long_rows():
    for fmt in (L.Q1_0, L.Q2_0_G64):
        layer = Layer(fmt, 2, 3, 32768)
        e = np.int32([1, 0, 1, 1, 1, 1, 0])
        layer.check(e, 1, planned(e, 2))
        layer.check(e, 1, None)


@pytest.mark.gpu
def test_a_plan_of_other_pairs_stays_inside():
    """A buffer that is no plan of these pairs: nothing is read or written out of range."""
    layer = Layer(L.Q2_0_G64, 4, 40, 256)
    n = 30
    q, s = W.random_rows(np.random.default_rng(0), n, 256)
    for pairs in (n, 70, 300):  # few and many rows an expert
        q, s = W.random_rows(np.random.default_rng(0), pairs, 256)
        for fill in (0x7F, 0xFF, 0x01, 0x00):
            plan = torch.full((L.lowbit_experts_plan_bytes(pairs, 4),), fill, dtype=torch.uint8, device="cuda")
            y = torch.full((pairs + 2, 40), 7.0, device="cuda")
            L.lowbit_experts_matmul(L.Q2_0_G64, layer.packed, 4, 40, 256, dev(q), dev(s), None, pairs, 1, y[1:-1], plan=plan)
            got = host(y)
            assert (got[0] == 7).all() and (got[-1] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 8, 65), (33, 6, 2048), (5, 2, 1027), (2, 64, 12)])
def test_combine(kind, T, k, N):
    say(f"case combine {kind} T={T} k={k} N={N}")
    rng = np.random.default_rng(N)
    E = 16
    y = rng.standard_normal((T * k, N)).astype(np.float32)
    e = rng.integers(0, E, (T, k)).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    if T > 1:
        e[0, 0], e[-1], e[1, -1] = -1, E, 2**31 - 1
        y[(e.reshape(-1) < 0) | (e.reshape(-1) >= E)] = np.nan  # not written by a product, and not read here
    ok = (e >= 0) & (e < E)
    t = np.where(ok[..., None], np.where(ok.reshape(-1)[:, None], y, 0).reshape(T, k, N) * w[..., None].astype(np.float64), 0)
    want, mags = t.sum(1), np.abs(t).sum(1)
    eps = torch.finfo(TYPES[kind][1]).eps / 2
    for pad in (0, 4, 3):
        out = torch.full((T + 1, N + pad), 7.0, dtype=TYPES[kind][1], device="cuda")
        L.lowbit_experts_combine(TYPES[kind][0], dev(y), dev(e), dev(w), T, k, E, N, out[:, :N])
        got = out.double().cpu().numpy()
        assert (got[T] == 7).all() and (got[:, N:] == 7).all()
        # one rounding to the type, and one to fp32 for each of the k additions
        assert (np.abs(got[:T, :N] - want) <= eps * np.abs(want) * (1 + 2.0**-10) + k * 2.0**-24 * mags * 1.001 + 2.0**-25).all()


@pytest.mark.gpu
def test_values_that_are_not_finite_stay_in_their_rows():
    for n, E in ((6, 3), (60, 3)):
        layer = Layer(L.Q4_0, E, 20, 256)
        q, s = W.random_rows(np.random.default_rng(0), n, 256)
        s[2, 1], s[4, 7] = np.inf, np.nan
        e = (np.arange(n) % E).astype(np.int32)
        y = torch.zeros(n, 20, device="cuda")
        L.lowbit_experts_matmul(L.Q4_0, layer.packed, E, 20, 256, dev(q), dev(s), None, n, 1, y, plan=planned(e, E))
        got = host(y)
        fine = np.isfinite(got).all(1)
        assert not fine[2] and not fine[4] and fine[[0, 1, 3, 5]].all() and fine[6:].all()


def exact_layer(x, first, last, e, w):
    """The layer of one token in 64 bits, with its activations quantised as lowbit_quantize_act does."""
    def q8(v):
        v = v.astype(np.float32).reshape(-1, 32)
        a = np.abs(v).max(1, keepdims=True)
        i = np.where(a > 0, np.float32(127) / np.where(a > 0, a, 1), 0).astype(np.float32)
        return np.rint(v * i).astype(np.int8).reshape(1, -1), (a / np.float32(127)).astype(np.float16).reshape(1, -1)

    out = 0.0
    for x_e, weight in zip(e, w):
        gu = W.product(first.fmt, first.w[x_e], first.d[x_e], *q8(x))[0][0]
        h = last.K
        act = gu[:h] / (1 + np.exp(-gu[:h])) * gu[h:]
        out = out + weight * W.product(last.fmt, last.w[x_e], last.d[x_e], *q8(act))[0][0]
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("T,fmts", [(1, (L.Q2_0_G64, L.Q4_0)), (9, (L.Q4_0, L.Q4_0)), (120, (L.Q1_0, L.Q2_0_G64))])
def test_a_layer_of_experts(T, fmts):
    """Routing, the plan, both products and their sum as they are used: eagerly, and captured and replayed with other
    tokens, some of them padding, and eager calls between the replays."""
    say(f"case layer T={T}")
    E, k, D, H = 12, 3, 256, 128
    first, last = Layer(fmts[0], E, 2 * H, D), Layer(fmts[1], E, D, H, seed=3)
    g = torch.Generator(device="cuda").manual_seed(T)
    n = T * k
    x, logits = torch.zeros(T, D, device="cuda"), torch.zeros(T, E, device="cuda")
    count = torch.full((1,), T, dtype=torch.int32, device="cuda")

    class Run:
        def __init__(self):
            z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
            self.e, self.w, self.plan = z(T, k, t=torch.int32), z(T, k), z(L.lowbit_experts_plan_bytes(n, E), t=torch.uint8)
            self.xq, self.xs, self.gu = z(T, D, t=torch.int8), z(T, D // 32, t=torch.float16), z(n, 2 * H)
            self.hq, self.hs, self.y, self.out = z(n, H, t=torch.int8), z(n, H // 32, t=torch.float16), z(n, D), z(T, D)

        def __call__(self):
            L.lowbit_route(L.F32, logits, T, E, k, self.e, self.w, score=L.SCORE_SIGMOID, count=count)
            plan = None
            if T > 1:
                plan = self.plan
                L.lowbit_experts_plan(self.e, n, E, plan)
            L.lowbit_quantize_act(L.ACT_Q8_0, x, T, D, self.xq, self.xs)
            L.lowbit_experts_matmul(first.fmt, first.packed, E, 2 * H, D, self.xq, self.xs, self.e, n, k, self.gu, plan=plan)
            h = torch.nn.functional.silu(self.gu[:, :H]) * self.gu[:, H:]
            L.lowbit_quantize_act(L.ACT_Q8_0, h.contiguous(), n, H, self.hq, self.hs)
            L.lowbit_experts_matmul(last.fmt, last.packed, E, D, H, self.hq, self.hs, self.e, n, 1, self.y, plan=plan)
            L.lowbit_experts_combine(L.F32, self.y, self.e, self.w, T, k, E, D, self.out)

    held, eager = Run(), Run()
    held()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held()
    for i in range(3):
        x.copy_(torch.randn(T, D, generator=g, device="cuda"))
        logits.copy_(torch.randn(T, E, generator=g, device="cuda"))
        real = max(1, T - 2 * i)
        count.fill_(real)
        torch.cuda.synchronize()
        graph.replay()
        eager()
        torch.cuda.synchronize()
        assert torch.equal(held.out, eager.out) and torch.equal(held.e, eager.e)
        assert (held.out[real:] == 0).all()
        we, ww = test_route.reference(host(logits).astype(np.float64), k, True)
        assert np.array_equal(host(held.e)[:real], we[:real])
        for t in {0, real // 2, real - 1}:
            want = exact_layer(host(x)[t], first, last, we[t], ww[t])
            got = host(held.out)[t]
            # a hidden value a rounding away from a border between two of its 255 steps may fall to the other: its block's
            # largest / 127 times the weight; of all k * H of them hardly more than a few do (fp32 is right to 2^-20 of a
            # step's 2^-7), and 1 % of the result's size is over 10 of the largest such steps
            assert np.abs(got - want).max() <= 0.01 * np.abs(want).max(), (t, np.abs(got - want).max(), np.abs(want).max())


@pytest.mark.gpu
@pytest.mark.parametrize("pairs,N", [(150, 16_000_000), (3000, 800_000)])
def test_outputs_past_32_bits(pairs, N):
    """Rows of 16 and of 128 a tile, and every pair by itself, at sampled places; then the sum over pairs of rows."""
    say(f"case outputs past 32 bits {pairs} x {N}")
    fmt, E, K = L.Q1_0, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    step = L.lowbit_experts_weight_bytes(fmt, 1, N, K)
    w = torch.randint(0, 256, (E, step), dtype=torch.uint8, generator=g, device="cuda")
    w[:, 16 * N:18 * N] = (torch.rand(E, N, generator=g, device="cuda") * 0.02 + 0.005).half().view(torch.uint8)
    q, s = W.random_rows(np.random.default_rng(0), pairs, K)
    e = (np.arange(pairs) % 3 == 0).astype(np.int32)
    y = torch.zeros(pairs * N, device="cuda")
    at_p, at_n = [0, pairs // 2, pairs - 2, pairs - 1], [0, 5, N // 3, N - 1]
    want, mags = np.zeros((4, 4)), np.zeros((4, 4))
    for i, p in enumerate(at_p):
        for j, n in enumerate(at_n):
            rec = w[e[p], 16 * n:16 * n + 16].cpu().numpy()
            bits = np.array([rec[(32 * (k % 32 // 8) + 4 * (k % 8) + k // 32) // 8] >> ((4 * (k % 8) + k // 32) % 8) & 1 for k in range(128)])
            d = w[e[p], 16 * N + 2 * n:16 * N + 2 * n + 2].cpu().numpy().view(np.float16)
            a, b = W.product(fmt, (2 * bits.astype(np.int64) - 1)[None], d[None], q[p:p + 1], s[p:p + 1])
            want[i, j], mags[i, j] = a[0, 0], b[0, 0]

    def check():
        got = y.view(pairs, N)[at_p][:, at_n].cpu().numpy()
        assert (np.abs(got - want) <= W.allowance(mags, K)).all()
        y.zero_()

    xq, xs, ed = dev(q), dev(s), dev(e)
    L.lowbit_experts_matmul(fmt, w.view(-1), E, N, K, xq, xs, ed, pairs, 1, y)
    check()
    L.lowbit_experts_matmul(fmt, w.view(-1), E, N, K, xq, xs, ed, pairs, 1, y, plan=planned(e, E))
    got = y.view(pairs, N)[at_p][:, at_n].cpu().numpy()
    assert (np.abs(got - want) <= W.allowance(mags, K)).all()
    out = torch.zeros(pairs // 2, N, dtype=torch.bfloat16, device="cuda")
    ones = torch.ones(pairs, device="cuda")
    L.lowbit_experts_combine(L.BF16, y, ed, ones, pairs // 2, 2, E, N, out)
    both = y.view(pairs, N)
    assert torch.equal(out[-1], (both[pairs - 2 - pairs % 2] + both[pairs - 1 - pairs % 2]).bfloat16()) and torch.equal(out[0], (both[0] + both[1]).bfloat16())


@pytest.mark.gpu
def test_experts_past_32_bits():
    """The last expert of tensors that together pass 4 GiB."""
    fmt, E, N, K = L.Q4_0, 1000, 2048, 4096
    step = L.lowbit_experts_weight_bytes(fmt, 1, N, K)
    assert E * step > 2**32
    packed = torch.zeros(E * step, dtype=torch.uint8, device="cuda")
    layer = Layer(fmt, 1, N, K)
    packed[(E - 1) * step:] = layer.packed
    e = np.full(5, E - 1, np.int32)
    q, s = W.random_rows(np.random.default_rng(2), 5, K)
    want, mags = W.product(fmt, layer.w[0], layer.d[0], q, s)
    for plan in (None, planned(e, E)):
        y = torch.zeros(5, N, device="cuda")
        L.lowbit_experts_matmul(fmt, packed, E, N, K, dev(q), dev(s), dev(e), 5, 1, y, plan=plan)
        assert (np.abs(host(y) - want) <= W.allowance(mags, K)).all()


@pytest.mark.gpu
def test_on_another_stream_and_two_at_once():
    """Two products with plans of their own on two streams at once, against one after another."""
    layer = Layer(L.Q2_0_G64, 6, 300, 512)
    rng = np.random.default_rng(3)
    runs = []
    for i in range(2):
        n = 60 + 700 * i
        e = some_pairs(rng, n, 6)
        q, s = W.random_rows(rng, n, 512)
        runs.append((n, dev(e), dev(q), dev(s), torch.zeros(L.lowbit_experts_plan_bytes(n, 6), dtype=torch.uint8, device="cuda"),
                     torch.zeros(n, 300, device="cuda"), torch.zeros(n, 300, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def go(n, e, q, s, plan, y, stream):
        L.lowbit_experts_plan(e, n, 6, plan, stream=stream)
        L.lowbit_experts_matmul(L.Q2_0_G64, layer.packed, 6, 300, 512, q, s, e, n, 1, y, plan=plan, stream=stream)

    for n, e, q, s, plan, y, _, stream in runs:
        go(n, e, q, s, plan, y, stream)
    torch.cuda.synchronize()
    for n, e, q, s, plan, y, z, _ in runs:
        go(n, e, q, s, plan, z, None)
        torch.cuda.synchronize()
        assert torch.equal(y, z)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS, ids=W.NAMES.get)
@pytest.mark.parametrize("E,N,K,n,per,rows", [(128, 70, 256, 5000, 4, 16), (20, 130, 384, 9000, 1, 128)])
def test_products_on_a_plan_with_gaps(fmt, E, N, K, n, per, rows):
    """Past 4096 pairs an expert's tiles begin at a number that the pairs before it give, with tiles without rows between:
    both sizes of tile on such a table, with experts that have no pair, and all pairs of one expert."""
    say(f"case a plan with gaps {W.NAMES[fmt]} E={E} N={N} K={K} pairs={n} per={per}")
    layer = Layer(fmt, E, N, K)
    e = some_pairs(np.random.default_rng(n), n, E)
    e[np.isin(e, [1, E // 2, E - 1])] = 0
    for which in (e, np.full(n, E - 1, np.int32)):
        plan = planned(which, E)
        p, tiles = host(plan).view(np.int32), n // rows + E
        assert len(p) == -(-(4 + (2 * tiles + 3) // 4 * 4 + tiles * rows) // 4) * 4  # the size for tiles of so many rows
        assert (p[4:4 + 2 * p[0]].reshape(-1, 2)[:, 1] == 0).any()
        layer.check(which, per, plan)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS, ids=W.NAMES.get)
@pytest.mark.parametrize("pairs,rows", [(30, 16), (300, 128)])
@pytest.mark.parametrize("place", [-1, None, 2**31 - 1, -2**31])
def test_pairs_past_the_end_count_as_the_last(fmt, pairs, rows, place):
    """Tiles of an expert that is there, whose pairs are not (`place`; None: the number of pairs, the first past the end):
    rows of x and y are those of the last pair, and nothing else is read or written."""
    say(f"case pairs past the end {W.NAMES[fmt]} {pairs} pairs, {rows} rows a tile, place {place}")
    E, N, K = 4, 40, 256
    layer, tiles = Layer(fmt, E, N, K), pairs // rows + E
    plan = np.zeros(L.lowbit_experts_plan_bytes(pairs, E) // 4, np.int32)
    at = 4 + (2 * tiles + 3) // 4 * 4
    assert len(plan) == -(-(at + tiles * rows) // 4) * 4  # the size for tiles of so many rows
    q, s = W.random_rows(np.random.default_rng(0), pairs, K)
    want, mags = W.product(fmt, layer.w[2], layer.d[2], q[-1:], s[-1:])
    for used in (1, 5, rows - 1, rows):  # in the forms for few and for many rows
        plan[0], plan[1], plan[4:at] = tiles, tiles * used, np.resize(np.int32([2, used]), at - 4)
        plan[at:] = pairs if place is None else place
        y = torch.full((pairs + 2, N), 7.0, device="cuda")
        L.lowbit_experts_matmul(fmt, layer.packed, E, N, K, dev(q), dev(s), None, pairs, 1, y[1:-1], plan=dev(plan))
        got = host(y)
        assert (np.abs(got[pairs] - want[0]) <= W.allowance(mags[0], K)).all()
        got[pairs] = 7
        assert (got == 7).all()


@pytest.mark.gpu
def test_outputs_of_16_row_tiles_past_32_bits():
    """Rows past 2^32 outputs, from a full tile and from one of few rows, at sampled places."""
    fmt, E, K, pairs, N = L.Q1_0, 3, 128, 150, 31_000_000
    say(f"case outputs of 16-row tiles past 32 bits {pairs} x {N}")
    tiles = pairs // 16 + E
    assert L.lowbit_experts_plan_bytes(pairs, E) == -(-4 * (4 + (2 * tiles + 3) // 4 * 4 + 16 * tiles) // 16) * 16
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(0, 256, (E, L.lowbit_experts_weight_bytes(fmt, 1, N, K)), dtype=torch.uint8, generator=g, device="cuda")
    w[:, 16 * N:18 * N] = (torch.rand(E, N, generator=g, device="cuda") * 0.02 + 0.005).half().view(torch.uint8)
    q, s = W.random_rows(np.random.default_rng(0), pairs, K)
    e = (np.arange(pairs) % E).astype(np.int32)  # 50 pairs each: three tiles of 16, the last two in one of their own
    y = torch.full((pairs * N + 64,), 7.0, device="cuda")
    L.lowbit_experts_matmul(fmt, w.view(-1), E, N, K, dev(q), dev(s), dev(e), pairs, 1, y, plan=planned(e, E))
    assert (y[pairs * N:] == 7).all()
    at_n = [0, 63, 64, N // 3, N - 1]
    assert 143 * N > 2**32
    for p in (0, 2, 75, 143, 144, 149):
        got = y[p * N:(p + 1) * N][at_n].cpu().numpy()
        x = w[e[p]]
        rec = np.stack([x[16 * n:16 * n + 16].cpu().numpy() for n in at_n])
        d = np.stack([x[16 * N + 2 * n:16 * N + 2 * n + 2].cpu().numpy().view(np.float16) for n in at_n])
        i = np.arange(128)
        bit = 32 * (i % 32 // 8) + 4 * (i % 8) + i // 32
        signs = 2 * (rec[:, bit // 8] >> (bit % 8) & 1).astype(np.int64) - 1
        want, mags = W.product(fmt, signs, d, q[p:p + 1], s[p:p + 1])
        assert (np.abs(got - want[0]) <= W.allowance(mags[0], K)).all(), p
