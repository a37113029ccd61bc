"""Logits that are not finite (infinities, NaN) at tokens that nothing touches, and at penalised, biased and masked ones."""
import numpy as np
import pytest
import torch

import bit_quantized_matvec_q1_amd.lowbit as L
from gpu_util import dev, host, say

pytestmark = pytest.mark.gpu

TYPES = {"f32": (L.F32, torch.float32), "bf16": (L.BF16, torch.bfloat16), "f16": (L.F16, torch.float16)}
INF, NAN = np.inf, np.nan
VALUES = (INF, -INF, NAN)
# the first of three tokens with the three values
NOTHING, PROMPT, OUTPUT, BOTH, BIASED, ALL, BANNED, FORCED = range(40, 120, 10)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("B,V", [(1, 200), (3, 1500), (130, 16385), (600, 3001)])  # the stretches of all sizes
def test_values_that_are_not_finite(kind, B, V):
    say(f"case logits not finite {kind} B={B} V={V}")
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.standard_normal((B, V)) * 4).to(TYPES[kind][1])
    triple = lambda *firsts: [f + i for f in firsts for i in range(3)]  # noqa: E731
    for f in range(40, 120, 10):
        for i, v in enumerate(VALUES):
            x[:, f + i] = v
    tokens = np.array([triple(PROMPT, BOTH, ALL) + triple(OUTPUT, BOTH, ALL) * 2] * B, np.int32)
    biases = [(t, v) for t, v in zip(triple(BIASED, ALL), [5.0, -7.0, 2.0] * 2)] + [(t, -INF) for t in triple(BANNED)] + [(t, INF) for t in triple(FORCED)]
    biases += [(BIASED, 1.0), (150, -INF), (151, INF), (152, NAN), (153, INF), (153, -INF)]
    a = dict(tokens=tokens, total_lens=np.full(B, tokens.shape[1], np.int32), prompt_lens=np.full(B, 9, np.int32),
             repetition=np.full(B, 1.5, np.float32), presence=np.full(B, 0.25, np.float32), frequency=np.full(B, 0.5, np.float32),
             bias_tokens=np.array([[t for t, _ in biases]] * B, np.int32), bias_values=np.array([[v for _, v in biases]] * B, np.float32),
             bias_lens=np.full(B, len(biases), np.int32), mask=np.full((B, -(-V // 32)), -1, np.int32))
    masked = triple(NOTHING, BOTH, FORCED) + [152, 7]
    for t in masked:  # in every second row
        a["mask"][1::2, t // 32] &= ~np.int32(np.uint32(1 << t % 32).view(np.int32))
    want = x.double().numpy().copy()  # penalties and finite biases leave infinities and NaN as they are
    with np.errstate(invalid="ignore"):
        for t, v in biases:
            want[:, t] += v
    want[1::2, masked] = -INF
    out = torch.full_like(x.cuda(), 7.0)
    L.lowbit_logits_process(TYPES[kind][0], x.cuda(), B, V, out, **{k: dev(v) for k, v in a.items()})
    got = host(out.double())
    special = [t for f in range(40, 120, 10) for t in (f, f + 1, f + 2)] + [150, 151, 152, 153, 7]
    for t in special:
        assert np.array_equal(got[:, t], want[:, t], equal_nan=True), (t, got[:2, t], want[:2, t])
    assert np.isnan(got[0, [BANNED, FORCED + 1, 152, 153]]).all() and np.isneginf(got[0, [BANNED + 1, 150]]).all() and got[0, 151] == INF
    rest = np.setdiff1d(np.arange(V), special)
    assert np.array_equal(got[:, rest], x.double().numpy()[:, rest])


@pytest.mark.parametrize("kind", list(TYPES))
def test_a_row_without_any_allowed_token(kind):
    say(f"case logits nothing allowed {kind}")
    V = 1111
    x = torch.randn(3, V, generator=torch.Generator().manual_seed(1)).to(TYPES[kind][1])
    x[1, :3] = torch.tensor(VALUES)
    mask = np.full((3, -(-V // 32)), -1, np.int32)
    mask[1] = 0
    out = torch.full_like(x.cuda(), 7.0)
    L.lowbit_logits_process(TYPES[kind][0], x.cuda(), 3, V, out, mask=dev(mask))
    torch.cuda.synchronize()
    assert torch.isneginf(out[1]).all() and torch.equal(out[::2].cpu(), x[::2])
