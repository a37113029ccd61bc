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
    token of what it sees.  got: [T, hq, D] on the GPU."""
    G, worst = c.hq // c.hk, 0.0
    for t in tokens:
        b = int(np.searchsorted(c.cu, t, side="right")) - 1
        length = c.lens[b] - int(c.cu[b + 1] - t) + 1
        for h in heads:
            q = c.q[t, h * G:(h + 1) * G].double().cpu().numpy()[None]
            ref, tol = R.attention(c.cache[:, h:h + 1], c.P, c.D, q, [0, 1], [length], c.table[b:b + 1], 1, c.scale, c.window, c.kind, rounded=rounded)
            err = np.abs(got[t, h * G:(h + 1) * G].double().cpu().numpy() - ref[0])
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
