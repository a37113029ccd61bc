"""The serving operators in 64 bits, written from their definitions: quantised rows and the cache's records, the
page plan, attention over the cache, and the processing of logits.  numpy on the host; no code of the library."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EPS = {"f32": 2.0**-23, "bf16": 2.0**-7, "f16": 2.0**-10}  # twice the most that a rounding is off by


def record_bytes(P, D):
    return P * D * 9 // 8


def quantise(x):
    """[..., D] -> codes (uint8) [..., D], scales (fp16) [..., D/32]."""
    x = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    a = np.abs(x)
    amax = a.max(-1)
    fine = np.isfinite(x).all(-1)
    with np.errstate(over="ignore", invalid="ignore"):
        q = np.where(fine, amax, 0.0).astype(np.float32) * (np.float32(1) / np.float32(6))  # as the format defines it
        d = np.where(fine, np.minimum(q, np.float32(65504)), np.float32(np.nan)).astype(np.float16)
    codes = np.zeros(x.shape, np.uint8)
    live = fine & (d > 0)
    dd = np.where(live, d.astype(np.float64), 1.0)[..., None]
    far = np.abs(np.minimum(np.where(fine[..., None], a, 0.0), 6 * dd)[..., None] - dd[..., None] * GRID)  # past 6: 6
    best = far.min(-1, keepdims=True)
    even = (far == best) & (np.arange(8) % 2 == 0)
    c = np.where(even.any(-1), even.argmax(-1), (far == best).argmax(-1)).astype(np.uint8)
    codes = np.where(live[..., None], c | np.where(x < 0, 8, 0).astype(np.uint8), 0).astype(np.uint8)
    return codes.reshape(*codes.shape[:-2], -1), d


def values(codes, d):
    v = np.where(codes & 8, -GRID[codes & 7], GRID[codes & 7])
    return v * np.repeat(d.astype(np.float64), 32, -1)


def places(P, D, o):
    """Byte and shift of every element of token o's key and value, and the bytes of its scales, in a record."""
    e, b, nb = np.arange(D), np.arange(D // 32), D // 32
    k = o * (D // 2) + (e % 32) // 8 * (D // 8) + e // 32 * 4 + e % 8 // 2
    v = P * D // 2 + ((o // 4) * 16 + e % 16) * 4 * nb + (o % 4) * nb + e // 32
    s = P * D + ((o // 4) * nb * 4 + b * 4 + o % 4) * 2
    return k, e % 2 * 4, v, e // 16 % 2 * 4, s, s + 2 * P * nb


def store(cache, P, D, slot, head, k, v):
    """One token's key and value rows into the cache [pages][heads][record] (uint8)."""
    rec = cache[slot // P, head]
    at = places(P, D, slot % P)
    for row, byte, shift, sc in ((k, at[0], at[1], at[4]), (v, at[2], at[3], at[5])):
        c, d = quantise(row)
        for i in range(D):
            rec[byte[i]] = (rec[byte[i]] & (0xF0 >> shift[i])) | (c[i] << shift[i])
        bits = d.view(np.uint16)
        rec[sc] = bits & 255
        rec[sc + 1] = bits >> 8


def load(cache, P, D, slot, head):
    """(key, value, value scales) of a slot, in 64 bits."""
    rec = cache[slot // P, head]
    kb, ks, vb, vs, sk, sv = places(P, D, slot % P)
    dk = (rec[sk].astype(np.uint16) | rec[sk + 1].astype(np.uint16) << 8).view(np.float16)
    dv = (rec[sv].astype(np.uint16) | rec[sv + 1].astype(np.uint16) << 8).view(np.float16)
    with np.errstate(invalid="ignore"):
        return values((rec[kb] >> ks) & 15, dk), values((rec[vb] >> vs) & 15, dv), dv.astype(np.float64)


def random_cache(rng, pages, heads, P, D, scale=1.0):
    """Codes at random, scales as rows of unit variance have them, times `scale`."""
    rec = rng.integers(0, 256, (pages, heads, record_bytes(P, D)), dtype=np.uint8)
    d = (rng.uniform(0.25, 0.55, (pages, heads, P * D // 16)) * scale).astype(np.float16)
    rec[:, :, P * D:] = d.view(np.uint8)
    return rec


def attention(cache, P, D, q, cu, lens, table, hk, scale, window, dtype, rounded=False):
    """Outputs [T, hq, D] and how far off a kernel of 32-bit sums may be, element by element.

    The weights' relative error (twice, for the numerator and for the sum): the score's, scale times
    sum |q||k| times the roundings of a chain of 32 products, nb scaled sums and three scalings, the query row's
    own (2^-24 of its largest element for elements far below that; fp32 queries are held in 22 bits), and the
    exponential's 2^-22.  Then the rounding of weight times value scale (fp16: 2^-11, fp32 rows: two of them,
    2^-21), with what is lost below binary16's range: half its least step, 2^-25, a key, times a code of at most 6,
    where the row's largest such product is at least 2^6 (the kernel aims it at 2^7 and knows it within a factor of
    2; fp32 rows' second number ends at the same step); sums over the keys in fp32, and the result's rounding.

    rounded: keys and values are code times scale rounded to binary16 (the kernel for many rows), each off by at most
    half a step, 2^-11 of its size: the scores by 2^-11 scale sum |q||k|, the outputs by 2^-11 sum w |v|."""
    T, hq, _ = q.shape
    G = hq // hk
    out, tol = np.full((T, hq, D), np.nan), np.zeros((T, hq, D))
    nb = D // 32
    for b in range(len(lens)):
        n, kv = cu[b + 1] - cu[b], lens[b]
        if n == 0:
            continue
        if kv <= 0:
            out[cu[b]:cu[b + 1]] = 0.0
            continue
        lo = max(0, kv - n + 1 - window) if window else 0
        slots = [int(table[b][j // P]) * P + j % P for j in range(lo, kv)]
        for h in range(hk):
            rows = [load(cache, P, D, s, h) for s in slots]
            k, v, dv = (np.array([r[i] for r in rows]).reshape(len(rows), -1) for i in range(3))
            for i in range(n):
                pos = kv - n + i
                a, z = (max(0, pos - window + 1) if window else 0), pos + 1
                for g in range(G):
                    t, hh = cu[b] + i, h * G + g
                    if z <= a:
                        out[t, hh] = 0.0
                        continue
                    kk, vv, dd = k[a - lo:z - lo], v[a - lo:z - lo], dv[a - lo:z - lo]
                    x = q[t, hh].astype(np.float64)
                    s = kk @ x * scale
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[t, hh] = w @ vv
                    size = np.abs(scale) * (np.abs(kk) @ np.abs(x)).max()
                    few = np.abs(scale) * np.abs(kk).sum(-1).max() * np.abs(x).max() * 2.0**-24
                    ds = size * ((48 + nb) * 2.0**-24 + (2.0**-22 if dtype == "f32" else 0.0)) + few + 2.0**-22 + np.abs(s).max() * 2.0**-23
                    dp = 2.0**-21 if dtype == "f32" else EPS["f16"] / 2
                    if rounded:
                        ds, dp = ds + size * EPS["f16"] / 2, dp + EPS["f16"] / 2
                    m = len(w)
                    A = w @ np.abs(vv)
                    floor = m * 6 * 2.0**-31 * (w * dd.max(-1)).max()
                    tol[t, hh] = np.abs(out[t, hh]) * EPS[dtype] / 2 + A * (2 * ds + dp + (m + 64) * 2.0**-24) + floor + 1e-37
                    if dtype == "f16":
                        tol[t, hh] += 2.0**-25  # below binary16's normal range
    return out, tol


def plan(new, P, lens, table, free, count, max_tokens, capacity):
    """The step's results as a dict (table: a new one)."""
    B, stride = len(lens), len(table[0])
    ok_len = all(o >= 0 and a >= 0 and -(-(o + a) // P) <= stride and o + a < 2**31 for o, a in zip(lens, new))
    need = [-(-(o + a) // P) - -(-o // P) if o >= 0 and a >= 0 else 0 for o, a in zip(lens, new)]
    toks = sum(a for o, a in zip(lens, new) if o >= 0 and a >= 0)
    st = (sum(need) > count) + 2 * (toks > max_tokens) + 4 * (not ok_len) + 8 * (not 0 <= count <= capacity)
    table = [list(r) for r in table]
    r = dict(status=[st, sum(need), toks], slots=[-1] * max_tokens, positions=[0] * max_tokens, cu=[0] * (B + 1), pages=[0] * (B + 1),
             lens=list(lens), count=[count], table=table)
    if st:
        return r
    t = took = 0
    for b in range(B):
        for k in range(need[b]):
            table[b][-(-lens[b] // P) + k] = free[count - 1 - took]
            took += 1
        for i in range(new[b]):
            p = lens[b] + i
            r["slots"][t] = table[b][p // P] * P + p % P
            r["positions"][t] = p
            t += 1
        r["cu"][b + 1], r["pages"][b + 1] = t, took
        r["lens"][b] += new[b]
    r["count"] = [count - took]
    return r


def logits(x, tokens=None, prompt=None, total=None, rep=None, pres=None, freq=None, btok=None, bval=None, blen=None, mask=None):
    """[B, V] in 64 bits, and the size of what went into each value (for the tolerance)."""
    x = np.array(x, np.float64)
    B, V = x.shape
    size = np.abs(x)
    for b in range(B):
        if tokens is not None:
            n = min(max(int(total[b]), 0), tokens.shape[1])
            p = min(max(int(prompt[b]), 0), n) if prompt is not None else 0
            inside = lambda a: a[(a >= 0) & (a < V)].astype(np.int64)  # noqa: E731
            seen = np.unique(inside(tokens[b, :n]))
            count = np.bincount(inside(tokens[b, p:n]), minlength=V).astype(np.float64)
            if rep is not None:
                with np.errstate(invalid="ignore"):
                    x[b, seen] = np.where(x[b, seen] > 0, x[b, seen] / np.float64(rep[b]), x[b, seen] * np.float64(rep[b]))
                size[b, seen] = np.maximum(size[b, seen], np.abs(x[b, seen]))
            if freq is not None:
                x[b] -= np.where(count > 0, np.float64(freq[b]) * count, 0.0)
                size[b] += np.abs(np.float64(freq[b]) * count)
            if pres is not None:
                x[b] -= np.where(count > 0, np.float64(pres[b]), 0.0)
                size[b] += np.abs(np.float64(pres[b])) * (count > 0)
        if btok is not None:
            for t, v in zip(btok[b, :max(0, min(int(blen[b]), btok.shape[1]))], bval[b]):
                if 0 <= t < V:
                    x[b, t] += np.float64(v)
                    size[b, t] += abs(np.float64(v))
        if mask is not None:
            bits = (mask[b].view(np.uint32)[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
            x[b, bits == 0] = -np.inf
    return x, size
