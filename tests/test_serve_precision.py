"""Attention over blocks of very different sizes: keys, queries and values whose 32-element blocks lie far apart, against
64 bits, with bounds derived for each kernel."""
import numpy as np
import pytest

import serve_ref as R
from gpu_util import say
from test_serve_attention import Case

pytestmark = pytest.mark.gpu

# heads (over one kv head) and new tokens that take the kernel for few rows, the one for up to 64, and a prompt's
FORMS = {"few": (4, 1), "some": (8, 2), "many": (4, 40)}


def scales_of(c, which):
    """The keys' (0) or values' (1) scales as an array [pages, hk, P / 4, blocks, 4] that writes through."""
    n = c.P * c.D // 32 * 2
    steps = (c.cache.strides[0], c.cache.strides[1], c.D // 32 * 8, 8, 2)
    return np.ndarray((c.pages, c.hk, c.P // 4, c.D // 32, 4), np.float16, c.cache, c.P * c.D + which * n, steps)


def rows(c, t):
    """Keys, values and value scales that query token t of the (single) request sees."""
    z = c.lens[0] - c.news[0] + t + 1
    got = [R.load(c.cache, c.P, c.D, int(c.table[0, j // c.P]) * c.P + j % c.P, 0) for j in range(z)]
    return [np.array([g[i] for g in got]) for i in range(3)]


@pytest.mark.parametrize("kind,form", [("f32", "few"), ("f32", "some"), ("f32", "many"), ("bf16", "few"), ("bf16", "some"), ("f16", "few"),
                                       ("f16", "some")])
def test_small_query_elements_against_large_keys(kind, form):
    """Queries whose second block is 2^-20 of the first, keys where it is 2^20 times the first: both count alike.

    The score's error, beside what serve_ref counts (a chain of 32 products, the block sums and scalings, fp32 queries
    in 22 bits): queries are held as binary16 numbers up to 2^15, so what is small there is off by half its least step,
    2^-25, that is 2^-39 of the row's largest (fp32 rows' second number ends at the same step)."""
    hq, new = FORMS[form]
    say(f"case small queries {kind} {form}")
    c = Case(71, kind, 128, 16, hq, 1, [57], [new], extra=0)
    f = 2.0**-10
    d = scales_of(c, 0)
    d[:, :, :, 0] *= np.float16(f)
    d[:, :, :, 1] /= np.float16(f)
    d[:, :, :, 2:] *= np.float16(f)
    c.q[:, :, 32:64] *= f * f
    c.q *= 2.0**7  # scores of about one
    got = c.gpu()
    worst = 0.0
    for t in range(new):
        k, v, dv = rows(c, t)
        for h in range(hq):
            x = c.q[t, h].double().numpy()
            s = k @ x * c.scale
            w = np.exp(s - s.max())
            w /= w.sum()
            want, A, m = w @ v, w @ np.abs(v), len(w)
            size = c.scale * (np.abs(k) @ np.abs(x)).max()
            few = c.scale * np.abs(k).sum(-1).max() * np.abs(x).max() * 2.0**-39
            ds = size * (52 * 2.0**-24 + (2.0**-22 if kind == "f32" else 0.0)) + few + 2.0**-22 + np.abs(s).max() * 2.0**-23
            dp = 2.0**-21 if kind == "f32" else R.EPS["f16"] / 2
            tol = np.abs(want) * R.EPS[kind] / 2 + A * (2 * ds + dp + (m + 64) * 2.0**-24) + m * 6 * 2.0**-31 * (w * dv.max(-1)).max() + 1e-37
            if kind == "f16":
                tol += 2.0**-25
            worst = max(worst, float((np.abs(got[t, h] - want) / tol).max()))
    say(f"  worst {worst:.3g} of the bound")
    assert worst <= 1.0


@pytest.mark.parametrize("kind,form", [("f32", "few"), ("f32", "some"), ("f32", "many"), ("bf16", "few"), ("bf16", "some"), ("bf16", "many"),
                                       ("f16", "few"), ("f16", "some"), ("f16", "many")])
@pytest.mark.parametrize("ratio", [2.0**-10, 2.0**-17])
def test_blocks_of_small_values(kind, form, ratio):
    """One block's values a small fraction of the others', and one block's keys.

    Weights times value scales end at binary16's least step: half of it, 2^-25, a key, times a code of at most 6, where
    the largest such product is at least 2^6: of the block's own products in the kernel for few rows, of all blocks'
    in the one for some (and fp32's many).  The kernel for many rows rounds the weights alone (2^-25 where the largest
    is 2^7, taken as 2^6), and keys and values, code times scale, to 2^-11, and where the largest scale is 2^8 or more
    to half the least step, 2^-25, for the scale (times 6) and once more for the product: 7 * 2^-33 of it."""
    hq, new = FORMS[form]
    say(f"case small values {kind} {form} {ratio}")
    c = Case(72, kind, 128, 16, hq, 1, [90], [new], extra=0)
    scales_of(c, 1)[:, :, :, 2] *= np.float16(ratio)
    scales_of(c, 0)[:, :, :, 1] *= np.float16(ratio)
    got = c.gpu()
    many = form == "many" and kind != "f32"
    worst = 0.0
    kd, vd = (float(scales_of(c, i).max()) for i in (0, 1))
    for t in range(new):
        k, v, dv = rows(c, t)
        for h in range(hq):
            x = c.q[t, h].double().numpy()
            s = k @ x * c.scale
            w = np.exp(s - s.max())
            w /= w.sum()
            want, A, m = w @ v, w @ np.abs(v), len(w)
            size = c.scale * (np.abs(k) @ np.abs(x)).max()
            few = c.scale * np.abs(k).sum(-1).max() * np.abs(x).max() * 2.0**-39
            ds = size * (52 * 2.0**-24 + (2.0**-22 if kind == "f32" else 0.0)) + few + 2.0**-22 + np.abs(s).max() * 2.0**-23
            dp = 2.0**-21 if kind == "f32" else R.EPS["f16"] / 2
            if many:
                ds += size * R.EPS["f16"] / 2 + c.scale * np.abs(x).sum() * 7 * 2.0**-33 * kd
                dp += R.EPS["f16"] / 2
                floor = 2.0**-31 * w.max() * np.abs(v).sum(0) + 7 * 2.0**-33 * vd
            elif form == "few":
                floor = m * 6 * 2.0**-31 * np.repeat((w[:, None] * dv).max(0), 32)
            else:
                floor = m * 6 * 2.0**-31 * (w[:, None] * dv).max()
            tol = np.abs(want) * R.EPS[kind] / 2 + A * (2 * ds + dp + (m + 64) * 2.0**-24) + floor + 1e-37
            if kind == "f16":
                tol += 2.0**-25
            worst = max(worst, float((np.abs(got[t, h] - want) / tol).max()))
    say(f"  worst {worst:.3g} of the bound")
    assert worst <= 1.0


def expect(c, got, t, h, blocks, form):
    """Query t, head h against 64 bits in the elements of `blocks`: the worst error over its bound.  The bounds are those
    of test_blocks_of_small_values; largest products over all keys that are finite."""
    k, v, dv = rows(c, t)
    dv = np.where(np.isfinite(dv), dv, 0.0)
    x = c.q[t, h].double().numpy()
    s = k @ x * c.scale
    w = np.exp(s - s.max())
    w /= w.sum()
    m = len(w)
    size = c.scale * (np.abs(k) @ np.abs(x)).max()
    ds = size * (52 * 2.0**-24 + (2.0**-22 if c.kind == "f32" else 0.0)) + c.scale * np.abs(k).sum(-1).max() * np.abs(x).max() * 2.0**-39
    ds += 2.0**-22 + np.abs(s).max() * 2.0**-23
    dp = 2.0**-21 if c.kind == "f32" else R.EPS["f16"] / 2
    largest = (w[:, None] * dv).max(0) if form == "few" else np.full(c.D // 32, (w[:, None] * dv).max())
    worst = 0.0
    for b in blocks:
        e = slice(32 * b, 32 * b + 32)
        want, A = w @ v[:, e], w @ np.abs(v[:, e])
        tol = np.abs(want) * R.EPS[c.kind] / 2 + A * (2 * ds + dp + (m + 64) * 2.0**-24) + m * 6 * 2.0**-31 * largest[b] + 1e-37
        if c.kind == "f16":
            tol += 2.0**-25
        err = np.abs(got[t, h, e] - want)
        assert np.isfinite(err).all()
        worst = max(worst, float((err / tol).max()))
    return worst


SMALL = [("f32", "few"), ("f32", "some"), ("f32", "many"), ("bf16", "few"), ("bf16", "some")]


@pytest.mark.parametrize("kind,form", SMALL)
@pytest.mark.parametrize("zero", [[37], [5, 37, 60], "tiny"])
def test_the_heaviest_keys_have_no_values(kind, form, zero):
    """Keys that take nearly all of the weight, and values that are zero there (or all values below binary16's normal
    range): what is left has its own size."""
    hq, new = FORMS[form]
    say(f"case zero values {kind} {form} {zero}")
    c = Case(73, kind, 64, 16, hq, 1, [90], [new], extra=0)
    c.scale = 2.0 if zero != "tiny" else 0.125
    if zero == "tiny":
        scales_of(c, 1)[:] *= np.float16(2.0**-20)
    else:
        scales_of(c, 0)[:] *= np.float16(0.125)
        for j in zero:
            page, o = c.table[0, j // 16], j % 16
            scales_of(c, 0)[page, 0, o // 4, :, o % 4] *= np.float16(8)
            scales_of(c, 1)[page, 0, o // 4, :, o % 4] = 0
            rec = c.cache[page, 0]
            rec[o * 32:(o + 1) * 32] = 0x22  # all elements 1 times the scale
        c.q = c.q.abs()  # scores there: about 2 * 64 * 0.8 * 0.4, the others' a few
    got = c.gpu()
    worst = max(expect(c, got, t, h, range(2), form) for t in range(max(0, new - 10), new) for h in range(hq))
    say(f"  worst {worst:.3g} of the bound")
    assert worst <= 1.0


@pytest.mark.parametrize("kind,form", SMALL)
def test_a_block_that_is_not_finite_leaves_the_others(kind, form):
    hq, new = FORMS[form]
    say(f"case NaN block {kind} {form}")
    c = Case(74, kind, 128, 16, hq, 1, [90], [new], extra=0)
    for j in (3, 40):
        scales_of(c, 1)[c.table[0, j // 16], 0, j % 16 // 4, 2, j % 4] = np.nan
    got = c.gpu()
    assert np.isnan(got[:, :, 64:96]).all()
    worst = max(expect(c, got, t, h, (0, 1, 3), form) for t in range(max(0, new - 10), new) for h in range(hq))
    say(f"  worst {worst:.3g} of the bound")
    assert worst <= 1.0


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("form", list(FORMS))
def test_the_largest_scores(kind, form):
    """Scores of 2^24 and less, two keys' equal and far above the others': the mean of their values is the result.

    The other keys' scores are over 2^23 below, so their weights are 0; the values are codes times their scales, for
    16-bit rows of many tokens rounded to binary16 (2^-11), weighed and divided by the same weight (2^-11 for the
    weight's rounding against the sum's, 2^-21 in fp32 rows), and rounded."""
    hq, new = FORMS[form]
    say(f"case largest scores {kind} {form}")
    c = Case(75, kind, 64, 16, hq, 1, [90], [new], extra=0)
    scales_of(c, 0)[:] = np.float16(0.5)
    for j in range(90):
        rec = c.cache[c.table[0, j // 16], 0]
        rec[j % 16 * 32:(j % 16 + 1) * 32] = 0x77 if j in (20, 50) else 0x11  # 6 * 0.5, twice the same, and 0.5 * 0.5
    c.q = (c.q * 0 + 2.0**10)
    c.scale = 2.0**24 / (64 * 3 * 2.0**10)
    j = 90 - new  # the first query's position
    got = c.gpu()
    k, v, _ = rows(c, new - 1)
    assert abs((k @ c.q[0, 0].double().numpy()).max() * c.scale - 2.0**24) < 2.0
    assert j >= 50
    want = (v[20] + v[50]) / 2
    tol = np.abs(want) * R.EPS[kind] / 2 + (np.abs(v[20]) + np.abs(v[50])) / 2 * (2.0**-20 if kind == "f32" else 3 * 2.0**-11) + 1e-6
    assert (np.abs(got - want) <= tol).all()
