"""Release of many requests' pages at once: more requests than the launch has workgroups."""
import numpy as np
import pytest
import torch

import bit_quantized_matvec_q1_amd.lowbit as L
from gpu_util import dev, host, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,stride", [(1024, 5), (1025, 5), (5000, 9), (100_003, 3), (1 << 22, 1)])
def test_release_of_many_requests(B, stride):
    say(f"case release B={B}")
    rng = np.random.default_rng(B)
    P = 32
    lens = rng.integers(0, stride * P + 1, B).astype(np.int32)
    done = (rng.random(B) < 0.6).astype(np.int32)
    done[B // 2:B // 2 + 40] = 0  # a workgroup's run may hold nothing
    table = rng.integers(0, 1 << 30, (B, stride)).astype(np.int32)
    held = np.where(done != 0, -(-lens // P), 0)
    pages = table[np.arange(stride)[None, :] < held[:, None]]  # in order of requests and blocks
    count = 7
    free = np.full(count + len(pages) + 3, -9, np.int32)
    want = free.copy()
    want[count:count + len(pages)] = pages
    dl, dc, st, df = dev(lens), dev(np.array([count], np.int32)), dev(np.array([-7, -7], np.int32)), dev(free)
    # too little room: nothing but what lies above the count may change
    L.lowbit_kv_release(dev(done), B, P, dl, dev(table), stride, df, dc, st, free_capacity=count + len(pages) - 1)
    assert host(st).tolist() == [8, len(pages)] and host(dc).tolist() == [count] and np.array_equal(host(dl), lens)
    assert np.array_equal(host(df)[:count], free[:count]) and (host(df)[count + len(pages) - 1:] == -9).all()
    # one length beyond its table, in the last run
    bad = lens.copy()
    bad[-1], done[-1] = stride * P + 1, 1
    db = dev(bad)
    L.lowbit_kv_release(dev(done), B, P, db, dev(table), stride, df, dc, st)
    assert host(st)[0] & 4 and host(dc).tolist() == [count] and np.array_equal(host(db), bad) and np.array_equal(host(df)[:count], free[:count])
    done[-1] = int(held[-1] > 0)
    L.lowbit_kv_release(dev(done), B, P, dl, dev(table), stride, df, dc, st)
    assert host(st).tolist() == [0, len(pages)] and host(dc).tolist() == [count + len(pages)]
    assert np.array_equal(host(df)[:count + len(pages)], want[:count + len(pages)])
    assert np.array_equal(host(dl), np.where(done != 0, 0, lens))
    torch.cuda.synchronize()
