"""The 64-bit reference of the serving operators against hand-made values and itself (CPU)."""
import numpy as np

import serve_ref as R


def test_codes_of_exact_values_and_ties():
    # a block whose largest value is 6 has scale 1: the grid's own numbers, and the borders between them, which
    # go to the even code
    x = np.array([6, -6, 0.5, -1.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, 0.2500001, 4.999, 0, -0.2] + [0.0] * 16)
    c, d = R.quantise(x)
    assert d[0] == 1.0
    assert c[:16].tolist() == [7, 15, 1, 11, 0, 2, 2, 4, 4, 6, 6, 14, 1, 6, 0, 8]


def test_scales_of_six_times_a_binary16_are_exact():
    m = np.arange(1, 31744, dtype=np.uint16).view(np.float16).astype(np.float64)  # every one above 0
    m = m[m <= 65504 / 2]
    x = np.zeros((m.size, 32))
    x[:, 3] = -6 * m
    _, d = R.quantise(x)
    assert np.array_equal(d[:, 0].astype(np.float64), m)


def test_nearest_by_brute_force():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 64)).astype(np.float32)
    c, d = R.quantise(x)
    v = R.values(c, d)
    dd = np.repeat(d.astype(np.float64), 32, -1)
    every = np.abs(x[..., None].astype(np.float64)) - dd[..., None] * R.GRID
    assert np.allclose(np.abs(np.abs(x) - np.abs(v)), np.abs(every).min(-1), rtol=0, atol=0)
    assert np.abs(x - v).max() <= dd.max() * (1 + 2**-10)  # the widest gap is 2, and 6 is the largest value


def test_scales_at_the_ends():
    big, tiny = np.full(32, 3.0e38), np.full(32, 1e-9)
    c, d = R.quantise(np.concatenate([big, tiny, np.full(32, np.nan), np.full(32, 6e-8 * 6)]))
    assert d[0] == 65504 and (c[:32] == 7).all()
    assert d[1] == 0 and (c[32:64] == 0).all()
    assert np.isnan(d[2]) and (c[64:96] == 0).all()
    assert d[3] > 0


def test_records_hold_every_row_apart():
    rng = np.random.default_rng(2)
    for P, D in ((16, 64), (32, 128), (16, 256)):
        cache = np.zeros((2, 1, R.record_bytes(P, D)), np.uint8)
        rows = {s: (rng.standard_normal(D), rng.standard_normal(D)) for s in range(2 * P)}
        for s in rng.permutation(2 * P):
            R.store(cache, P, D, int(s), 0, *rows[int(s)])
        for s, (k, v) in rows.items():
            gk, gv, _ = R.load(cache, P, D, s, 0)
            assert np.array_equal(gk, R.values(*R.quantise(k))) and np.array_equal(gv, R.values(*R.quantise(v)))


def test_every_byte_of_a_record_is_used_once():
    for P, D in ((16, 64), (16, 128), (32, 256)):
        seen = np.zeros(R.record_bytes(P, D) * 2, int)
        for o in range(P):
            kb, ks, vb, vs, sk, sv = R.places(P, D, o)
            for byte, shift in ((kb, ks), (vb, vs)):
                np.add.at(seen, 2 * byte + shift // 4, 1)
            for s in (sk, sv):
                for n in range(4):
                    np.add.at(seen, 2 * s + n, 1)
        assert (seen == 1).all()


def test_plan_by_hand():
    r = R.plan([3, 0, 17], 16, [15, 0, 0], [[9, -1], [-1, -1], [-1, -1]], [1, 2, 3, 4, 5], 5, 24, 5)
    assert r["status"] == [0, 3, 20] and r["table"] == [[9, 5], [-1, -1], [4, 3]] and r["count"] == [2]
    assert r["slots"][:4] == [9 * 16 + 15, 80, 81, 64] and r["slots"][19] == 48 and r["slots"][20:] == [-1] * 4
    assert r["positions"][:4] == [15, 16, 17, 0] and r["cu"] == [0, 3, 3, 20]
