"""The attention kernel for many new tokens: its forms, padded batches, and sizes that only it meets, against the 64-bit
reference."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_matvec_q1_amd.lowbit as L
import serve_ref as R
from gpu_util import dev, say
from test_serve_attention import TYPES, Case

pytestmark = pytest.mark.gpu


def check_rows(c, got, tokens, heads, rounded=True):
    """Query rows of a Case (token of the step, kv head) against the reference, each as a request of its own: the last
    token of what it sees.  got: [T, hq, D], a tensor or an array."""
    G, worst = c.hq // c.hk, 0.0
    for t in tokens:
        b = int(np.searchsorted(c.cu, t, side="right")) - 1
        length = c.lens[b] - int(c.cu[b + 1] - t) + 1  # up to its own token
        for h in heads:
            q = c.q[t, h * G:(h + 1) * G].double().cpu().numpy()[None]
            ref, tol = R.attention(c.cache[:, h:h + 1], c.P, c.D, q, [0, 1], [length], c.table[b:b + 1], 1, c.scale, c.window, c.kind, rounded=rounded)
            rows = got[t, h * G:(h + 1) * G]
            err = np.abs((rows.double().cpu().numpy() if isinstance(rows, torch.Tensor) else rows) - ref[0])
            ratio = float((err / tol[0]).max())
            assert np.isfinite(err).all() and ratio <= 1.0, f"token {t}, kv head {h}: {ratio} of the bound"
            worst = max(worst, ratio)
    say(f"  worst of {len(tokens) * len(heads)} sampled groups: {worst:.3g} of the bound")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,news", [([700], [40]), ([300, 900], [64, 17]), ([400, 20], [300, 5])])
def test_a_padded_batch(D, lens, news):
    # a captured step's rows: many more than its requests may bring, which choose neither the tiles' size nor the parts'
    Case(40 + D, "bf16", D, 16, 32, 8, lens, news, extra=4200 - sum(news)).check(f"padded D={D} {news}")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_more_than_2_23_query_rows(kind):
    """One prompt of 131077 tokens of 64 heads, a window of 40 so that it is quick: rows from all over it."""
    say(f"case long prompt {kind}")
    T, hq, hk, D = 131077, 64, 8, 64
    rng = np.random.default_rng(50)
    c = Case.__new__(Case)
    c.kind, c.D, c.P, c.hq, c.hk, c.lens, c.window, c.scale = kind, D, 64, hq, hk, [T], 40, 1 / math.sqrt(D)
    c.pages = -(-T // 64)
    c.table, c.cu = rng.permutation(c.pages).astype(np.int32)[None], np.array([0, T], np.int32)
    c.cache = R.random_cache(rng, c.pages, hk, 64, D)
    g = torch.Generator(device="cuda")
    g.manual_seed(50)
    c.q = torch.randn(T, hq, D, device="cuda", generator=g).to(TYPES[kind][1])
    out = torch.full_like(c.q, 7.0)
    L.lowbit_kv_attention(TYPES[kind][0], c.q, T, 1, hq, hk, D, dev(c.cu), dev(np.array([T], np.int32)), dev(c.table), c.pages, dev(c.cache),
                          c.pages, 64, T, T, c.scale, out, window=40)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    check_rows(c, out, [0, 1, 33, 39, 40, 41, 65535, 65536, 131000, 131071, 131072, T - 1], [0, 3, 7], rounded=kind != "f32")


# Batches of 128 or 64 query heads that take each form of the kernel at head sizes 64 and 128 (at 256 there is one), with
# what the host counts: slots (rows / tile + requests) times kv heads, and the tiles that the rows fill.
FORMS = {
    # 16 or more tiles of 256 rows and 32 heads: at least 512
    "256 rows": dict(hq=128, hk=32, lens=[600, 333, 70, 5, 140], news=[500, 333, 70, 5, 129]),
    "256 rows, a request a tile": dict(hq=128, hk=32, lens=[64, 65, 200, 90] * 4, news=[64, 64, 64, 64] * 4),
    "256 rows, window": dict(hq=128, hk=32, lens=[600, 700, 5, 1], news=[500, 530, 5, 1], window=50),
    # (6 + 2) * 32 = 256 workgroups for 224 full tiles, none split
    "halves": dict(hq=128, hk=32, lens=[300, 260], news=[130, 70]),
    "halves, window": dict(hq=128, hk=32, lens=[900, 500], news=[130, 70], window=300),
    # (16 + 3) * 16 = 304 for 272, requests of 260, 160 and 100 rows
    "halves, uneven": dict(hq=64, hk=16, lens=[1100, 400, 300], news=[260, 160, 100]),
    # (16 + 1) * 16 = 272
    "halves, one prompt": dict(hq=64, hk=16, lens=[521], news=[521]),
    # 256 workgroups of short requests, 384 for two rounds of equal ones, and parts of split tiles
    "four waves, short": dict(hq=128, hk=32, lens=[200, 150], news=[130, 70]),
    "four waves, equal": dict(hq=64, hk=16, lens=[300] * 6, news=[96] * 6),
    "four waves, split": dict(hq=32, hk=8, lens=[900, 130], news=[90, 130]),
}


def sample(c):
    """The first and last tokens of every request, and some on the way (every sixteenth of the larger ones)."""
    t = set()
    for b, n in enumerate(c.news):
        for i in {0, 1, 31, 32, 33, 63, 64, n // 2, n // 2 + 17, n - 2, n - 1}:
            if 0 <= i < n and (b < 4 or i in (0, n - 1)):
                t.add(int(c.cu[b]) + i)
    return sorted(t)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", list(FORMS))
def test_forms(form, D, kind):
    say(f"case {form} {kind} D={D}")
    c = Case(80 + D, kind, D, 16, **FORMS[form], pad=8)
    if c.window:  # pages before every query's window may be gone
        for b in range(c.B):
            c.table[b, :max(0, c.lens[b] - c.news[b] + 1 - c.window) // 16] = -1
    got = c.gpu()
    rows = c.cu[-1]
    assert (got[rows:] == 7).all() and np.isfinite(got[:rows]).all()
    check_rows(c, got, sample(c), [0, c.hk // 2 + 1, c.hk - 1])
    assert np.array_equal(c.gpu(), got)  # and the same bits again


@pytest.mark.parametrize("form", ["256 rows", "halves", "halves, one prompt", "four waves, short"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("first", ["keys", "values"])
def test_forms_with_scales_that_grow_on_the_way(first, D, form):
    # tokens 70 and 135 of the first request pass the scales seen before by far: the tile is unpacked again
    say(f"case growing {first} {form} D={D}")
    c = Case(81, "bf16", D, 16, **FORMS[form])
    heads = [1, c.hk - 1]
    for j, f in ((70, 300.0), (135, 20000.0)):
        for h in heads:
            rec = c.cache[c.table[0, j // 16], h]
            for s in R.places(16, D, j % 16)[4 if first == "keys" else 5]:
                d = rec[s:s + 2].view(np.float16)
                d[:] = np.float16(float(d[0]) * f)
    if first == "keys":
        c.q = c.q * 2.0**-12  # scores of some tens
    check_rows(c, c.gpu(), sample(c), heads)


@pytest.mark.parametrize("form", ["256 rows", "halves", "halves, one prompt", "four waves, short"])
@pytest.mark.parametrize("D", [64, 128])
def test_forms_see_what_is_not_finite_and_no_more(D, form):
    say(f"case NaN {form} D={D}")
    c = Case(82, "f16", D, 16, **FORMS[form])
    clean = c.gpu()
    n, first, h, G = c.news[0], c.lens[0] - c.news[0], c.hk - 2, c.hq // c.hk
    nan = np.float16(np.nan).view(np.uint16)
    a, b, z = first + n // 3, first + n // 2, c.lens[0] - 1  # a value block, a key block, and the last token's first value block
    for j, which, block in ((a, 5, 1), (b, 4, 0), (z, 5, 0)):
        rec = c.cache[c.table[0, j // 16], h]
        s = R.places(16, D, j % 16)[which][block]
        rec[s], rec[s + 1] = nan & 255, nan >> 8
    tail = c.cache[c.table[0, z // 16], h]
    for o in range(z % 16 + 1, 16):  # behind the end
        for s in R.places(16, D, o)[4:]:
            tail[s], tail[s + 1] = nan & 255, nan >> 8
    got = c.gpu()
    at = first + np.arange(n)
    bad = np.zeros((c.T, c.hq, D), bool)
    mine = bad[:n, h * G:(h + 1) * G]
    mine[at >= a, :, 32:64] = True
    mine[at >= b] = True
    mine[at >= z, :, :32] = True
    assert np.array_equal(np.isnan(got), bad)
    # scales that are not finite are left out of the tile's power of two, and that changes no bit of the others
    assert np.array_equal(got[~bad], clean[~bad])
    c.table[0, 1] = c.pages + 5  # a page that is none: the request's rows from its first token on see it
    got, sees = c.gpu(), np.zeros(c.T, bool)
    sees[:n] = at >= 16
    assert np.isnan(got[sees]).all() and np.array_equal(got[~sees], clean[~sees])


@pytest.mark.parametrize("kind,D,hq,hk,lens,news", [
    ("f32", 128, 40, 2, [30, 50], [1, 3]), ("bf16", 128, 10, 2, [70, 20, 5], [2, 3, 5]), ("f16", 256, 12, 3, [40], [1]),  # 16-row tiles
    ("f32", 64, 4, 4, [100, 30], [40, 30]), ("bf16", 128, 16, 4, [200, 90], [130, 40]), ("f16", 64, 14, 2, [600], [70]),  # and a prompt's
    ("bf16", 64, 16, 4, [40, 300], [1, 1]), ("f16", 128, 128, 32, [300, 260], [130, 70])])
@pytest.mark.parametrize("first", [1, 5, 100])
def test_a_step_behind_other_rows(first, kind, D, hq, hk, lens, news):
    """A step's rows from `first` on: what lies before them is not its own."""
    say(f"case rows from {first} on {kind} D={D} {hq}/{hk} {news}")
    c = Case(90, kind, D, 16, hq, hk, lens, news, extra=first + 3, pad=8)
    c.q = torch.cat([c.q[-first - 3:-3], c.q[:-first - 3], c.q[-3:]])
    c.cu = c.cu + np.int32(first)
    got = c.gpu()
    assert (got[:first] == 7).all() and (got[c.cu[-1]:] == 7).all()
    check_rows(c, got, sample(c), sorted({0, 1 % hk, hk - 1}), rounded=kind != "f32" and c.max_q * hq // hk > 64)
