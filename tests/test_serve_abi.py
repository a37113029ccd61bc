"""The serving entry points on the host: every documented refusal, before a device is touched, and the binding's
own checks of tensors."""
import pytest
import torch

import bit_quantized_matvec_q1_amd.lowbit as L

A = 1 << 20  # an aligned stand-in address; never dereferenced (every call below fails validation)
lib = L.lib


def plan(new=A, B=2, P=16, lens=A, lens_out=A, table=A, stride=4, free=A, cap=8, count=A, count_out=A, cu=A, cup=A, slots=A, pos=A, n=8,
         status=A):
    return lib.lowbit_kv_plan(new, B, P, lens, lens_out, table, stride, free, cap, count, count_out, cu, cup, slots, pos, n, status, None)


def test_plan():
    for bad in (dict(B=-1), dict(stride=-1), dict(cap=-1), dict(n=-1), dict(B=2**31), dict(P=8), dict(P=48), dict(P=2048), dict(P=0), dict(P=-16)):
        assert plan(**bad) == L.LB_ESHAPE, bad
    for k in ("new", "lens", "lens_out", "table", "free", "count", "count_out", "cu", "cup", "slots", "pos", "status"):
        assert plan(**{k: None}) == L.LB_EINVAL, k
        assert plan(**{k: A + 2}) == L.LB_EALIGN, k
    assert plan(slots=A + 4) == L.LB_EALIGN
    assert plan(B=0, new=None) == L.LB_OK


def release(done=A, B=2, P=16, lens=A, table=A, stride=4, free=A, cap=8, count=A, status=A):
    return lib.lowbit_kv_release(done, B, P, lens, table, stride, free, cap, count, status, None)


def test_release():
    for bad in (dict(B=-1), dict(B=1 << 24), dict(stride=-1), dict(cap=-1), dict(P=24)):
        assert release(**bad) == L.LB_ESHAPE, bad
    for k in ("done", "lens", "table", "free", "count", "status"):
        assert release(**{k: None}) == L.LB_EINVAL, k
        assert release(**{k: A + 1}) == L.LB_EALIGN, k
    assert release(B=0, done=None) == L.LB_OK


def append(dtype=L.BF16, k=A, ks=256, v=A, vs=256, T=3, H=2, D=128, slots=A, cache=A, pages=4, P=16):
    return lib.lowbit_kv_append(dtype, k, ks, v, vs, T, H, D, slots, cache, pages, P, None)


def read(dtype=L.BF16, k=A, ks=256, v=A, vs=256, T=3, H=2, D=128, slots=A, cache=A, pages=4, P=16):
    return lib.lowbit_kv_read(dtype, cache, pages, P, T, H, D, slots, k, ks, v, vs, None)


@pytest.mark.parametrize("call", [append, read])
def test_append_and_read(call):
    assert call(dtype=3) == call(dtype=-1) == L.LB_EINVAL
    for bad in (dict(T=-1), dict(H=0), dict(H=-2), dict(D=96), dict(D=0), dict(P=20), dict(pages=-1), dict(ks=255), dict(vs=128),
                dict(T=2**30)):
        assert call(**bad) == L.LB_ESHAPE, bad
    for k in ("k", "v", "slots", "cache"):
        assert call(**{k: None}) == L.LB_EINVAL, k
        assert call(**{k: A + 4}) == L.LB_EALIGN, k
    assert call(ks=257) == L.LB_EALIGN and call(dtype=L.F32, vs=258) == L.LB_EALIGN
    assert call(T=0, k=None, cache=None) == L.LB_OK


def attn(dtype=L.F16, q=A, qs=1024, T=3, B=2, hq=8, hk=2, D=128, cu=A, lens=A, table=A, stride=4, cache=A, pages=8, P=16, max_q=2,
         max_kv=64, scale=0.1, window=0, out=A, os=1024, ws=None, wsb=0):
    return lib.lowbit_kv_attention(dtype, q, qs, T, B, hq, hk, D, cu, lens, table, stride, cache, pages, P, max_q, max_kv, scale, window,
                                   out, os, ws, wsb, None)


def test_attention():
    assert attn(dtype=7) == L.LB_EINVAL
    for bad in (dict(T=-1), dict(B=-1), dict(hq=0), dict(hq=7), dict(hk=0), dict(hk=3), dict(D=112), dict(P=8), dict(P=17), dict(pages=-1),
                dict(pages=0), dict(max_q=-1), dict(max_kv=-1), dict(window=-1), dict(stride=-1), dict(qs=1016), dict(os=512),
                dict(T=2**29), dict(max_kv=2**31 - 1), dict(B=1 << 24, T=1 << 24),
                dict(B=1 << 23, T=1 << 23, hq=1, hk=1, max_q=1)):
        assert attn(**bad) == L.LB_ESHAPE, bad
    for k in ("q", "out", "cu", "lens", "table", "cache"):
        assert attn(**{k: None}) == L.LB_EINVAL, k
        assert attn(**{k: A + 2}) == L.LB_EALIGN, k
    assert attn(qs=1025) == L.LB_EALIGN and attn(ws=A + 8, wsb=64) == L.LB_EALIGN
    assert attn(T=0, q=None) == L.LB_OK and attn(B=0, cu=None) == L.LB_OK
    need = L.lowbit_kv_attention_workspace(1, 1, 8, 2, 128, 1, 100000)
    assert need > 0
    long = dict(T=1, B=1, max_q=1, max_kv=100000, stride=10000)
    assert attn(**long) == L.LB_EINVAL and attn(ws=A, wsb=need - 1, **long) == L.LB_ESHAPE


def test_workspace_and_cache_bytes():
    assert L.lowbit_kv_cache_bytes(10, 8, 16, 128) == 10 * 8 * 2304
    assert L.lowbit_kv_cache_bytes(1 << 20, 8, 64, 128) == (1 << 20) * 8 * 9216  # past 32 bits
    for bad in ((-1, 8, 16, 128), (1, 0, 16, 128), (1, 8, 24, 128), (1, 8, 16, 80)):
        assert L.lowbit_kv_cache_bytes(*bad) == -1
    ws = L.lowbit_kv_attention_workspace
    assert ws(0, 4, 8, 2, 128, 1, 1000) == 0 and ws(4, 0, 8, 2, 128, 1, 1000) == 0
    assert ws(-1, 4, 8, 2, 128, 1, 1000) == ws(4, 4, 8, 3, 128, 1, 1000) == ws(4, 4, 8, 2, 100, 1, 1000) == -1
    # a window bounds what a request reads, and with it the parts to join
    assert ws(1, 1, 8, 2, 128, 1, 1 << 20, 512) < ws(1, 1, 8, 2, 128, 1, 1 << 20, 0)
    assert ws(1, 1, 8, 2, 128, 1, 1000, 1000) == ws(1, 1, 8, 2, 128, 1, 1000, 0)


def logits(dtype=L.F32, x=A, xs=100, B=2, V=100, tok=None, ts=0, pl=None, tl=None, rep=None, pres=None, freq=None, bt=None, bv=None, bs=0,
           bl=None, mask=None, ms=0, out=A, os=100):
    return lib.lowbit_logits_process(dtype, x, xs, B, V, tok, ts, pl, tl, rep, pres, freq, bt, bv, bs, bl, mask, ms, out, os, None)


def test_logits():
    assert logits(dtype=9) == L.LB_EINVAL
    for bad in (dict(B=-1), dict(V=-1), dict(ts=-1), dict(bs=-1), dict(bs=16385), dict(xs=99), dict(os=99), dict(mask=A, ms=3),
                dict(out=A, os=101), dict(B=1 << 20, V=1 << 20)):
        assert logits(**bad) == L.LB_ESHAPE, bad
    for bad in (dict(x=None), dict(out=None), dict(tok=A), dict(rep=A), dict(pres=A), dict(freq=A), dict(bt=A, bl=A), dict(bt=A, bv=A)):
        assert logits(**bad) == L.LB_EINVAL, bad
    for bad in (dict(x=A + 2, out=A + 2), dict(dtype=L.BF16, out=A + 1), dict(tok=A + 2, tl=A), dict(mask=A + 2, ms=4),
                dict(tok=A, tl=A, rep=A + 1)):
        assert logits(**bad) == L.LB_EALIGN, bad
    assert logits(B=0, x=None) == L.LB_OK and logits(V=0, x=None) == L.LB_OK


def test_binding_refuses_short_and_foreign_tensors():
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    cache, slots = torch.zeros(4 * 2 * 2304, dtype=torch.uint8), torch.zeros(3, dtype=torch.int64)

    def app(**o):
        a = dict(k=k, v=k, T=3, slots=slots, cache=cache)
        a.update(o)
        L.lowbit_kv_append(L.BF16, a["k"], a["v"], a["T"], 2, 128, a["slots"], a["cache"], 4, 16)

    with pytest.raises(ValueError, match="device tensor required"):
        app()
    with pytest.raises(ValueError, match="k: dtype"):
        app(k=k.float())
    with pytest.raises(ValueError, match="v: shape"):
        app(v=torch.zeros(3, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="k: needs at least"):
        app(k=k[:2])
    with pytest.raises(ValueError, match="k: a row's elements"):
        app(k=torch.zeros(3, 128, 2, dtype=torch.bfloat16).transpose(1, 2))
    with pytest.raises(ValueError, match="k: a row's elements"):
        app(k=k[:1].expand(3, 2, 128))
    with pytest.raises(ValueError, match="slots: needs at least"):
        app(slots=slots[:2])
    with pytest.raises(ValueError, match="slots: dtype"):
        app(slots=slots.int())
    with pytest.raises(ValueError, match="cache: needs at least"):
        app(cache=cache[1:])
    with pytest.raises(ValueError, match="cache: contiguous"):
        app(cache=torch.zeros(2 * cache.numel(), dtype=torch.uint8)[::2])
    with pytest.raises(ValueError, match="block_table: needs at least"):
        L.lowbit_kv_plan(i32(2), 2, 16, i32(2), i32(2), i32(7), 4, i32(8), i32(1), i32(1), i32(3), i32(3), slots, i32(3), 3, i32(3))
    with pytest.raises(ValueError, match="status: needs at least"):
        L.lowbit_kv_plan(i32(2), 2, 16, i32(2), i32(2), i32(8), 4, i32(8), i32(1), i32(1), i32(3), i32(3), slots, i32(3), 3, i32(2))
    with pytest.raises(ValueError, match="free_pages: needs at least"):
        L.lowbit_kv_release(i32(2), 2, 16, i32(2), i32(8), 4, i32(8), i32(1), i32(2), free_capacity=9)
    q = torch.zeros(3, 8, 128, dtype=torch.float16)

    def att(**o):
        a = dict(q=q, out=q, cu=i32(3), lens=i32(2), table=i32(8), ws=None, max_kv=64)
        a.update(o)
        L.lowbit_kv_attention(L.F16, a["q"], 3, 2, 8, 2, 128, a["cu"], a["lens"], a["table"], 4, cache, 4, 16, 2, a["max_kv"], 0.1,
                              a["out"], workspace=a["ws"])

    for o, what in ((dict(q=q[:2]), "q: needs at least"), (dict(out=q.float()), "out: dtype"), (dict(cu=i32(2)), "cu_q: needs at least"),
                    (dict(lens=i32(1)), "kv_lens: needs"), (dict(table=i32(7)), "block_table: needs"), ({}, "device tensor required")):
        with pytest.raises(ValueError, match=what):
            att(**o)
    x = torch.zeros(2, 100)
    lo = lambda **o: L.lowbit_logits_process(L.F32, o.pop("x", x), 2, 100, o.pop("out", x), **o)  # noqa: E731
    for o, what in ((dict(x=x[:, :99]), "logits: shape"), (dict(out=x.half()), "out: a tensor"), (dict(mask=torch.zeros(2, 3, dtype=torch.int32)), "mask: shape"),
                    (dict(tokens=torch.zeros(1, 5, dtype=torch.int32)), "tokens: shape"), (dict(repetition=torch.zeros(1)), "repetition: needs"),
                    (dict(bias_tokens=torch.zeros(2, 5, dtype=torch.int32), bias_values=torch.zeros(2, 4)), "bias_values: the shape"),
                    (dict(x=x.T.contiguous().T), "logits: dense rows"), (dict(x=x[:1].expand(2, 100)), "logits: rows must not overlap"),
                    ({}, "device tensor required")):
        with pytest.raises(ValueError, match=what):
            lo(**o)
