"""A batch served over several steps with the serving operators together: pages and slots, rows into the cache,
attention, the head, and the logits, eagerly and as one captured step replayed."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_matvec_q1_amd.lowbit as L
import serve_ref as R
import synth
from gpu_util import dev, host, say

pytestmark = pytest.mark.gpu

HQ, HK, D, P = 4, 2, 64, 16
WIDTH = (HQ + 2 * HK) * D


class Server:
    """The state of a batch, on the device, and one step over it; every buffer is kept, so a step can be captured."""

    def __init__(self, B, stride, pages, max_tokens, max_q):
        i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.B, self.stride, self.pages, self.max_tokens, self.max_q = B, stride, pages, max_tokens, max_q
        self.new, self.lens, self.table = i32(B), i32(B), torch.full((B, stride), -1, dtype=torch.int32, device="cuda")
        self.free, self.count = torch.arange(pages, dtype=torch.int32, device="cuda"), torch.full((1,), pages, dtype=torch.int32, device="cuda")
        self.cu, self.cup, self.positions, self.status = i32(B + 1), i32(B + 1), i32(max_tokens), i32(3)
        self.slots = torch.zeros(max_tokens, dtype=torch.int64, device="cuda")
        self.cache = torch.randint(0, 256, (L.lowbit_kv_cache_bytes(pages, HK, P, D),), dtype=torch.uint8, device="cuda")
        self.qkv = torch.zeros(max_tokens, WIDTH, device="cuda")
        self.out = torch.zeros(max_tokens, HQ, D, device="cuda")
        need = L.lowbit_kv_attention_workspace(max_tokens, B, HQ, HK, D, max_q, stride * P)
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def step(self):
        n = self.max_tokens
        L.lowbit_kv_plan(self.new, self.B, P, self.lens, self.lens, self.table, self.stride, self.free, self.count, self.count, self.cu, self.cup,
                         self.slots, self.positions, n, self.status)
        q, k, v = (self.qkv[:, a * D:z * D] for a, z in ((0, HQ), (HQ, HQ + HK), (HQ + HK, HQ + 2 * HK)))
        L.lowbit_kv_append(L.F32, k, v, n, HK, D, self.slots, self.cache, self.pages, P)
        L.lowbit_kv_attention(L.F32, q, n, self.B, HQ, HK, D, self.cu, self.lens, self.table, self.stride, self.cache, self.pages, P, self.max_q,
                              self.stride * P, 1 / math.sqrt(D), self.out, workspace=self.ws)


class Follower:
    """The same on the host, in 64 bits: every request's quantised rows."""

    def __init__(self, B):
        self.k, self.v = [[] for _ in range(B)], [[] for _ in range(B)]

    def step(self, news, qkv):
        outs, t = [], 0
        for b, n in enumerate(news):
            for i in range(n):
                row = qkv[t + i].astype(np.float64).reshape(-1, D)
                self.k[b].append(np.array([R.values(*R.quantise(x)) for x in row[HQ:HQ + HK]]))
                self.v[b].append(np.array([R.values(*R.quantise(x)) for x in row[HQ + HK:]]))
            for i in range(n):
                held = len(self.k[b]) - n + i + 1
                row = qkv[t + i].astype(np.float64).reshape(-1, D)
                o = []
                for h in range(HQ):
                    kk, vv = (np.array([x[h // (HQ // HK)] for x in c[b][:held]]) for c in (self.k, self.v))
                    s = kk @ row[h] / math.sqrt(D)
                    w = np.exp(s - s.max())
                    o.append(w @ vv / w.sum())
                outs.append(np.array(o))
            t += n
        return np.array(outs)


# fp32 rows: 22-bit operands and sums of a few hundred products, on outputs of about 1 and scores of about 10:
# 2 * (10 + sum |q||k| scale = 60) * 50 * 2^-24 at the very most
TOL = 5e-4


def test_steps_of_a_batch_with_requests_coming_and_going():
    rng = np.random.default_rng(0)
    B = 5
    s, f = Server(B, 12, 40, 64, 40), Follower(B)
    steps = [[20, 0, 7, 1, 16], [1, 1, 1, 1, 1], [1, 30, 0, 1, 1], [1, 1, 1, 1, 1], "done 2 4", [1, 1, 33, 1, 17], [1, 1, 1, 1, 1]]
    for news in steps:
        say(f"case step {news}")
        if isinstance(news, str):
            done = torch.zeros(B, dtype=torch.int32, device="cuda")
            for b in map(int, news.split()[1:]):
                done[b] = 1
                f.k[b], f.v[b] = [], []
            st = torch.zeros(2, dtype=torch.int32, device="cuda")
            L.lowbit_kv_release(done, B, P, s.lens, s.table, s.stride, s.free, s.count, st)
            assert host(st)[0] == 0
            continue
        n = sum(news)
        qkv = rng.standard_normal((64, WIDTH)).astype(np.float32)
        s.new.copy_(torch.tensor(news, dtype=torch.int32))
        s.qkv.copy_(torch.from_numpy(qkv))
        s.out.fill_(7.0)
        s.step()
        want = f.step(news, qkv[:n])
        assert host(s.status).tolist()[0] == 0 and host(s.lens).tolist() == [len(k) for k in f.k]
        got = host(s.out)
        assert np.abs(got[:n] - want).max() < TOL and (got[n:] == 7).all()
        # what the cache holds at the new slots is the quantised rows
        k, v = torch.empty(64, HK, D, device="cuda"), torch.empty(64, HK, D, device="cuda")
        L.lowbit_kv_read(L.F32, s.cache, s.pages, P, 64, HK, D, s.slots, k, v)
        rows = qkv[:n].reshape(n, -1, D)
        assert np.array_equal(host(k)[:n], R.values(*R.quantise(rows[:, HQ:HQ + HK])).astype(np.float32))
        assert np.array_equal(host(v)[:n], R.values(*R.quantise(rows[:, HQ + HK:])).astype(np.float32)) and (host(v)[n:] == 0).all()
    # no two requests share a page, and none is lost
    used = [p for b in range(B) for p in host(s.table)[b][:-(-len(f.k[b]) // P)].tolist()]
    assert sorted(used + host(s.free)[:int(host(s.count)[0])].tolist()) == list(range(40))


def test_a_step_that_does_not_fit_changes_nothing():
    s = Server(2, 4, 3, 64, 64)
    s.new.copy_(torch.tensor([20, 17], dtype=torch.int32))  # four pages of three
    s.out.fill_(7.0)
    before = s.cache.clone()
    s.step()
    assert host(s.status).tolist() == [1, 4, 37] and host(s.lens).tolist() == [0, 0] and int(host(s.count)[0]) == 3
    assert torch.equal(s.cache, before) and (s.out == 7).all()


def test_a_captured_step_replayed_goes_on_where_the_last_one_ended():
    say("case captured step")
    rng = np.random.default_rng(1)
    B = 3
    s, e = Server(B, 80, 250, B, 1), Server(B, 80, 250, B, 1)  # long enough for the attention to be split
    e.cache.copy_(s.cache)
    assert L.lowbit_kv_attention_workspace(B, B, HQ, HK, D, 1, 80 * P) > 0
    for srv in (s, e):
        srv.new.fill_(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.new.zero_()
        s.step()  # nothing new: nothing changes
        s.new.fill_(1)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    f = Follower(B)
    for turn in range(40):
        qkv = rng.standard_normal((B, WIDTH)).astype(np.float32)
        for srv in (s, e):
            srv.qkv.copy_(torch.from_numpy(qkv))
        graph.replay()
        e.step()
        if turn % 8 == 0:
            torch.cuda.synchronize()
        want = f.step([1] * B, qkv)
        assert torch.equal(s.out, e.out) and torch.equal(s.lens, e.lens) and torch.equal(s.slots, e.slots) and torch.equal(s.cache, e.cache)
        assert np.abs(host(s.out) - want).max() < TOL
    assert host(s.lens).tolist() == [40] * B


def test_head_and_logits():
    say("case head, penalties and mask")
    V, K = 1000, 256
    W, x = synth.head_weights(V, K, 5), synth.activations(synth.rng(6), 1, K)[0]
    y = torch.empty(V, device="cuda")
    L.dense_head_matvec(dev(W), V, K, dev(x), y)
    rng = np.random.default_rng(2)
    a = dict(tokens=rng.integers(0, V, (1, 50)).astype(np.int32), total_lens=np.array([50], np.int32), prompt_lens=np.array([30], np.int32),
             repetition=np.array([1.3], np.float32), frequency=np.array([0.1], np.float32), presence=np.array([0.2], np.float32),
             mask=rng.integers(-2**31, 2**31, (1, 32), dtype=np.int64).astype(np.int32))
    before = host(y).copy()
    row = y.view(1, V)
    L.lowbit_logits_process(L.F32, row, 1, V, row, **{k: dev(v) for k, v in a.items()})
    want, size = R.logits(before[None], a["tokens"], a["prompt_lens"], a["total_lens"], a["repetition"], a["presence"], a["frequency"], mask=a["mask"])
    got = host(y).astype(np.float64)
    fine = np.isfinite(want[0])
    assert np.array_equal(np.isneginf(got), ~fine) and (np.abs(got[fine] - want[0][fine]) <= (size[0] * 6 * 2.0**-24 + np.abs(want[0]) * 2.0**-24)[fine]).all()
