"""The dependency-ordered token with a 4-bit key/value cache (bench.py's LayeredGraph): every layer's attention
against the 64-bit reference on the products' own outputs, and the captured token's replays against the eager one."""
import numpy as np
import pytest
import torch

import serve_ref as R
import synth
from bench import DecodeToken, LayeredGraph
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,layer,fused,context", [(synth.Q2_0_G64, synth.QWEN3_8B_LAYER, True, 300), (synth.TERNARY_PLANAR, synth.BITNET_2B_GQA_LAYER, False, 127)],
                         ids=["Q2_0_g64", "planar"])
def test_token_after_a_context(fmt, layer, fused, context):
    say(f"case token after {context} tokens, format {fmt}")
    tok = DecodeToken(fmt, layer, 2, seed=8100 + fmt)
    lg = LayeredGraph(tok, fused=fused, context=context)
    c = lg.cache
    lg.eager()
    torch.cuda.synchronize()
    assert c.status.tolist()[0] == 0 and c.lens_out.tolist() == [context + 1] and c.lens.tolist() == [context]
    table, slot = c.table.cpu().numpy(), int(c.slots)
    assert slot == table[0, context // c.PAGE] * c.PAGE + context % c.PAGE
    for l in range(2):
        cache = c.caches[l].cpu().numpy().reshape(c.pages, c.hk, -1)
        q, k, v = (c.y[l, n].cpu().numpy().reshape(-1, c.D) for n in ("attn_q", "attn_k", "attn_v"))
        for h in range(c.hk):  # the token's own rows are in the cache
            gk, gv, _ = R.load(cache, c.PAGE, c.D, slot, h)
            assert np.array_equal(gk, R.values(*R.quantise(k[h]))) and np.array_equal(gv, R.values(*R.quantise(v[h])))
        ref, tol = R.attention(cache, c.PAGE, c.D, q[None], [0, 1], [context + 1], table, c.hk, c.D ** -0.5, 0, "f32")
        K, r = tok.row_of[l, 1]
        got = tok.x[K][r].cpu().numpy().reshape(1, c.hq, c.D)
        assert (np.abs(got - ref) <= tol).all()
    kept = [p["y"].clone() for p in tok.products]
    for _ in range(3):
        for p in tok.products:
            p["y"].fill_(float("nan"))
        lg.graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p["y"], y) for p, y in zip(tok.products, kept))
        lg.eager()  # eager work between replays
        torch.cuda.synchronize()
    lg.close()
    tok.batch.close()
