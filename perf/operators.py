"""The serving operators around the low-bit products, as they are timed: block tables and slot maps from request
lengths, rows quantised into a 4-bit cache, attention over that cache, and penalties, biases and masks on logits.

With `own` false, run() computes an operator in elementary torch operations; with `own` true it calls the library.

The cache (one layer): pages of P tokens, one record per page and kv head.  32 consecutive values of a token's
head share a binary16 scale d = fp16(amax / 6); a code is the E2M1 number (sign and 0 .5 1 1.5 2 3 4 6) nearest to
x / d, ties to the even code.  A record holds, with nb = D / 32 blocks a row:
  K codes  [P][4][nb][4 bytes]      byte (g, b, i): elements 32b + 8g + 2i (low nibble) and 32b + 8g + 2i + 1
  V codes  [P/4][16][4][nb bytes]   quad, c, token of the quad, byte i: elements 32i + c (low) and 32i + 16 + c
  K scales [P/4][nb][4] binary16    quad, block, token of the quad;   V scales alike
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
CODE = {"f32": 0, "bf16": 1, "f16": 2}  # the library's lb_dtype


def listed():
    return [
        # attention: one token of one short chat, in the library's own activation type: latency
        dict(name="attn_one_f32", op="attn", t="f32", B=1, hq=32, hk=8, D=128, P=16, kv=37, ragged=False, new=1, window=0),
        # the ordinary decode step of a server: a few dozen ragged requests
        dict(name="attn_decode_bf16", op="attn", t="bf16", B=32, hq=20, hk=5, D=128, P=64, kv=4000, ragged=True, new=1, window=0),
        # one request with a very long context: the work has to be split over its length
        dict(name="attn_long_f16", op="attn", t="f16", B=1, hq=32, hk=8, D=128, P=16, kv=131071, ragged=False, new=1, window=0),
        # a full server: the cache of many long requests, several times the memory-side cache
        dict(name="attn_full_bf16", op="attn", t="bf16", B=64, hq=32, hk=8, D=128, P=32, kv=12345, ragged=True, new=1, window=0),
        # chunks of several prompts appended to what is cached already
        dict(name="attn_chunk_bf16", op="attn", t="bf16", B=4, hq=20, hk=5, D=128, P=64, kv=2600, ragged=True, new=777, window=0),
        # one long prompt
        dict(name="attn_prefill_f16", op="attn", t="f16", B=1, hq=32, hk=8, D=128, P=32, kv=8192, ragged=False, new=8192, window=0),
        # the rows of one decode step of a batch, as the products leave them (fp32)
        dict(name="append_decode_f32", op="append", t="f32", T=32, hk=8, D=128, P=16),
        # the rows of a prompt
        dict(name="append_prompt_bf16", op="append", t="bf16", T=16384, hk=8, D=128, P=32),
        # one decode step's slots and the few pages it needs
        dict(name="plan_decode", op="plan", B=64, P=16, kv=4000, new=1),
        # many prompts arriving at once
        dict(name="plan_prompts", op="plan", B=512, P=16, kv=500, new=400),
        # one request's logits
        dict(name="logits_one_f32", op="logits", t="f32", B=1, V=128256, hist=700, bias=16, mask=True),
        # a batch with long histories
        dict(name="logits_batch_f32", op="logits", t="f32", B=96, V=151669, hist=6000, bias=64, mask=True),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["attn", "attn", "attn", "append", "plan", "logits"])
    if op == "attn":
        hk = rng.choice([1, 2, 4, 5, 8])
        c = dict(op=op, t=rng.choice(["f32", "bf16", "f16"]), hk=hk, hq=hk * rng.choice([1, 2, 4, 5, 7, 8]),
                 D=rng.choice([64, 128, 128, 256]), P=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7,
                 window=rng.choice([0, 0, 0, 500]))
        if rng.random() < 0.6:
            c["B"], c["kv"], c["new"] = log(1, 64), log(1, 8000), rng.choice([1, 1, 1, 2, 5])
        else:
            c["B"], c["new"] = log(1, 4), log(6, 1500)
            c["kv"] = c["new"] + log(1, 1500)
        c["kv"] = max(c["kv"], c["new"])
        return c
    if op == "append":
        return dict(op=op, t=rng.choice(["f32", "bf16", "f16"]), T=log(1, 8000), hk=rng.choice([1, 2, 4, 5, 8]),
                    D=rng.choice([64, 128, 128, 256]), P=rng.choice([16, 32, 64, 128]))
    if op == "plan":
        return dict(op=op, B=log(1, 512), P=rng.choice([16, 32, 64, 128]), kv=log(1, 4000), new=rng.choice([1, 1, log(2, 400)]))
    return dict(op=op, t=rng.choice(["f32", "bf16", "f16"]), B=log(1, 64), V=rng.choice([128256, 151669, log(1000, 150000)]),
                hist=log(1, 8000), bias=rng.choice([0, log(1, 300)]), mask=rng.random() < 0.5)


# ---- what the caller has in hand ----------------------------------------------------------------

def record_bytes(P, D):
    return P * D * 9 // 8


def lengths(case, g):
    """Cached lengths (new tokens included) and new tokens of each request, on the host."""
    B, kv, new = case["B"], case["kv"], case["new"]
    if not case.get("ragged"):
        return [kv] * B, [new] * B
    f = torch.rand(B, generator=g).tolist()
    kvs = [max(1, int(kv * (0.1 + 0.9 * x))) for x in f]
    kvs[-1] = kv
    news = [max(1, int(new * (0.3 + 0.7 * (b * 0.618 % 1)))) for b in range(B)]  # the same rows in all from seed to seed
    return [max(k, n) for k, n in zip(kvs, news)], news


def random_cache(pages, hk, P, D, g):
    """Random codes, and the scales that rows of unit variance have (amax of 32 over 6)."""
    rec = torch.randint(0, 256, (pages, hk, record_bytes(P, D)), dtype=torch.uint8, device=DEV, generator=g)
    sc = torch.rand(pages, hk, P * D // 16, device=DEV, generator=g).mul_(0.3).add_(0.25).to(torch.float16)
    rec[:, :, P * D:] = sc.view(torch.uint8)
    return rec


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed)
    s = dict(case)
    op = case["op"]

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    if op == "attn":
        B, hq, hk, D, P = (case[k] for k in ("B", "hq", "hk", "D", "P"))
        kvs, news = lengths(case, h)
        blocks = [-(-k // P) for k in kvs]
        pages = sum(blocks) + 3
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        stride = max(blocks)
        table = torch.full((B, stride), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b in range(B):
            table[b, :blocks[b]] = order[at:at + blocks[b]]
            at += blocks[b]
        cu = [0]
        for n in news:
            cu.append(cu[-1] + n)
        s.update(T=cu[-1], pages=pages, table=table, stride=stride, cache=random_cache(pages, hk, P, D, g), cu=i32(cu), lens=i32(kvs),
                 max_q=max(news), max_kv=max(kvs), scale=1.0 / math.sqrt(D),
                 q=torch.randn(cu[-1], hq, D, generator=g, device=DEV).to(TYPES[case["t"]]))
    elif op == "append":
        T, hk, D, P = (case[k] for k in ("T", "hk", "D", "P"))
        pages = max(T, 4) if T <= 64 else -(-T // P) + 4
        order = torch.randperm(pages, generator=g, device=DEV)
        t = torch.arange(T, device=DEV)
        if T <= 64:  # a decode step: each row at the end of its own request's page
            slots = order[:T] * P + torch.randint(0, P, (T,), generator=g, device=DEV)
        else:  # prompts: rows one after another, through pages in any order
            slots = order[t // P] * P + t % P
        s.update(pages=pages, slots=slots,
                 cache=torch.zeros(pages, hk, record_bytes(P, D), dtype=torch.uint8, device=DEV))
        for n in ("k", "v"):
            s[n] = torch.randn(T, hk, D, generator=g, device=DEV).to(TYPES[case["t"]])
    elif op == "plan":
        B, P = case["B"], case["P"]
        kvs = torch.randint(0, case["kv"] + 1, (B,), generator=h)
        news = torch.randint(0 if case["new"] > 1 else 1, case["new"] + 1, (B,), generator=h)
        used, want = (kvs + P - 1) // P, (kvs + news + P - 1) // P
        stride = -(-(case["kv"] + case["new"]) // P) + 1
        pages = int(want.sum()) + 8
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((B, stride), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b in range(B):
            n = int(used[b])
            table[b, :n] = order[at:at + n]
            at += n
        free = torch.zeros(pages, dtype=torch.int32, device=DEV)
        free[:pages - at] = order[at:]
        s.update(lens=kvs.to(torch.int32).to(DEV), new_lens=news.to(torch.int32).to(DEV), table=table, stride=stride, free=free,
                 count=i32([pages - at]), max_tokens=B * case["new"] + 5)  # the bound that a captured step is padded to
    else:
        B, V, H, n = case["B"], case["V"], case["hist"], case["bias"]
        total = [max(1, int(H * f)) for f in torch.rand(B, generator=h).mul_(0.7).add_(0.3).tolist()]
        prompt = [int(t * f) for t, f in zip(total, torch.rand(B, generator=h).tolist())]
        u = torch.rand(B, H, generator=g, device=DEV)
        s.update(logits=(3 * torch.randn(B, V, generator=g, device=DEV)).to(TYPES[case["t"]]),
                 tokens=(u ** 3 * V).to(torch.int32).clamp_(max=V - 1),  # a few tokens come often
                 prompt=i32(prompt), total=i32(total),
                 rep=1.0 + 0.5 * torch.rand(B, generator=g, device=DEV), pres=torch.rand(B, generator=g, device=DEV),
                 freq=torch.rand(B, generator=g, device=DEV))
        if n:
            s.update(btok=torch.randint(0, V, (B, n), dtype=torch.int32, generator=g, device=DEV),
                     bval=5 * torch.randn(B, n, generator=g, device=DEV),
                     blen=torch.randint(0, n + 1, (B,), dtype=torch.int32, generator=g, device=DEV))
        if case["mask"]:
            s["bits"] = torch.randint(-2**31, 2**31, (B, -(-V // 32)), generator=g, device=DEV).to(torch.int32)
    return s


# ---- one pass -----------------------------------------------------------------------------------

def run(s):
    if own:
        return {"attn": own_attn, "append": own_append, "plan": own_plan, "logits": own_logits}[s["op"]](s)
    return {"attn": plain_attn, "append": plain_append, "plan": plain_plan, "logits": plain_logits}[s["op"]](s)


def own_attn(s):
    import bit_quantized_matvec_q1_amd.lowbit as L

    out = torch.empty_like(s["q"])
    L.lowbit_kv_attention(CODE[s["t"]], s["q"], s["T"], s["B"], s["hq"], s["hk"], s["D"], s["cu"], s["lens"], s["table"],
                          s["stride"], s["cache"], s["pages"], s["P"], s["max_q"], s["max_kv"], s["scale"], out, window=s["window"])
    return out


def own_append(s):
    import bit_quantized_matvec_q1_amd.lowbit as L

    T, hk, D = s["T"], s["hk"], s["D"]
    L.lowbit_kv_append(CODE[s["t"]], s["k"], s["v"], T, hk, D, s["slots"], s["cache"], s["pages"], s["P"])
    k, v = (torch.empty(T, hk, D, dtype=torch.float32, device=s["k"].device) for _ in range(2))
    L.lowbit_kv_read(CODE["f32"], s["cache"], s["pages"], s["P"], T, hk, D, s["slots"], k, v)
    return k, v


def own_plan(s):
    import bit_quantized_matvec_q1_amd.lowbit as L

    B, n, dev = s["B"], s["max_tokens"], s["lens"].device
    new = {k: torch.empty(c, dtype=torch.int32, device=dev) for k, c in
           (("lens", B), ("count", 1), ("cu", B + 1), ("pages", B + 1), ("positions", n), ("status", 3))}
    slots = torch.empty(n, dtype=torch.int64, device=dev)
    L.lowbit_kv_plan(s["new_lens"], B, s["P"], s["lens"], new["lens"], s["table"], s["stride"], s["free"], s["count"], new["count"],
                     new["cu"], new["pages"], slots, new["positions"], n, new["status"])
    return dict(new, slots=slots, table=s["table"])


def own_logits(s):
    import bit_quantized_matvec_q1_amd.lowbit as L

    out = torch.empty_like(s["logits"])
    L.lowbit_logits_process(CODE[s["t"]], s["logits"], s["B"], s["V"], out, tokens=s["tokens"], prompt_lens=s["prompt"],
                            total_lens=s["total"], repetition=s["rep"], presence=s["pres"], frequency=s["freq"],
                            bias_tokens=s.get("btok"), bias_values=s.get("bval"), bias_lens=s.get("blen"), mask=s.get("bits"))
    return out


# the values of a byte's two codes
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def byte_values(device):
    v = torch.tensor(E2M1 + [-x for x in E2M1], device=device)
    b = torch.arange(256, device=device)
    return torch.stack([v[b & 15], v[b >> 4]], -1)  # [256][2]


def scales(rec, at, P, nb):
    """[..., record] bytes -> the scales from byte `at` on: [..., P, nb] fp32."""
    d = rec[..., at:at + P * nb * 2].contiguous().view(torch.float16).float()
    return d.view(*d.shape[:-1], P // 4, nb, 4).transpose(-1, -2).reshape(*d.shape[:-1], P, nb)


def plain_keys(rec, P, D):
    """[..., record] bytes -> [..., P, D] fp32 keys."""
    nb, lead = D // 32, rec.shape[:-1]
    c = byte_values(rec.device)[rec[..., :P * D // 2].int()]  # [..., bytes, 2]
    c = c.view(*lead, P, 4, nb, 8).transpose(-3, -2)  # [..., P, nb, 4, 8]
    d = scales(rec, P * D, P, nb)
    return (c.reshape(*lead, P, nb, 32) * d[..., None]).view(*lead, P, D)


def plain_values(rec, P, D):
    """[..., record] bytes -> [..., P, D] fp32 values."""
    nb, lead, n = D // 32, rec.shape[:-1], rec.dim() - 1
    c = byte_values(rec.device)[rec[..., P * D // 2:P * D].int()].view(*lead, P // 4, 16, 4, nb, 2)
    c = c.permute(*range(n), n, n + 2, n + 3, n + 4, n + 1).reshape(*lead, P, nb, 32)  # [quad, token, block, half, c]
    d = scales(rec, P * D + P * nb * 2, P, nb)
    return (c * d[..., None]).view(*lead, P, D)


def plain_attn(s):
    B, hq, hk, D, P, T = (s[k] for k in ("B", "hq", "hk", "D", "P", "T"))
    G, nq, nblk, dev = hq // hk, s["max_q"], s["stride"], s["q"].device
    rec = s["cache"][s["table"].clamp(min=0)].transpose(1, 2)  # [B, hk, blocks, record]
    L = nblk * P
    k = plain_keys(rec, P, D).view(B, hk, L, D)
    n = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(nq, device=dev)
    row = (s["cu"][:-1, None] + i).clamp(max=T - 1)  # padded query rows
    q = s["q"].float()[row].view(B, nq, hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, hk, nq * G, D)
    sc = torch.matmul(q, k.transpose(-1, -2).contiguous()).view(B, hk, nq, G, L) * s["scale"]
    del k
    pos = (s["lens"] - n)[:, None] + i  # [B, nq]
    j = torch.arange(L, device=dev)
    see = (j <= pos[..., None]) & (j < s["lens"][:, None, None])
    if s["window"]:
        see &= j > pos[..., None] - s["window"]
    see = see[:, None, :, None, :]
    sc.masked_fill_(~see, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    v = plain_values(rec, P, D).view(B, hk, L, D)
    o = torch.matmul(p.view(B, hk, nq * G, L), v).view(B, hk, nq, G, D) / torch.where(z > 0, z, torch.ones_like(z))
    o = o.permute(0, 2, 1, 3, 4).reshape(B * nq, hq, D)
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(s["cu"], t, right=True, out_int32=True) - 1
    return o[b * nq + (t - s["cu"][b])].to(s["q"].dtype)


def plain_codes(x, D):
    """[T, hk, D] rows -> codes [T, hk, nb, 32] (uint8) and scales [T, hk, nb] (fp16)."""
    x = x.float().view(*x.shape[:-1], D // 32, 32)
    a = x.abs()
    d = (a.amax(-1) / 6).clamp(max=65504).to(torch.float16)
    b = d.float()[..., None]
    c = (a > b * 0.25).to(torch.uint8) + (a >= b * 0.75) + (a > b * 1.25) + (a >= b * 1.75) + (a > b * 2.5) + (a >= b * 3.5) + (a > b * 5)
    return torch.where(b > 0, c | ((x < 0).to(torch.uint8) << 3), torch.zeros_like(c)), d


def plain_append(s):
    T, hk, D, P, nb = s["T"], s["hk"], s["D"], s["P"], s["D"] // 32
    rec, page, off = s["cache"], s["slots"] // s["P"], s["slots"] % s["P"]
    quad, lane, h = off // 4, off % 4, P * D // 2
    c, d = plain_codes(s["k"], D)
    c = c.view(T, hk, nb, 4, 8).transpose(2, 3).reshape(T, hk, D // 2, 2)
    rec[:, :, :h].view(-1, hk, P, D // 2)[page, :, off] = c[..., 0] | (c[..., 1] << 4)
    halves = rec.view(torch.float16)  # the same bytes, two at a time
    halves[:, :, h:h + P * nb].view(-1, hk, P // 4, nb, 4)[page, :, quad, :, lane] = d
    c, d = plain_codes(s["v"], D)
    c = c.view(T, hk, nb, 2, 16).permute(0, 1, 4, 2, 3)  # [T, hk, 16, nb, 2]
    rec[:, :, h:2 * h].view(-1, hk, P // 4, 16, 4, nb)[page, :, quad, :, lane] = c[..., 0] | (c[..., 1] << 4)
    halves[:, :, h + P * nb:].view(-1, hk, P // 4, nb, 4)[page, :, quad, :, lane] = d
    # and back: the rows as the cache holds them
    val = byte_values(rec.device)
    k = val[rec[:, :, :h].view(-1, hk, P, D // 2)[page, :, off].int()].view(T, hk, 4, nb, 8).transpose(2, 3).reshape(T, hk, nb, 32)
    k = k * halves[:, :, h:h + P * nb].view(-1, hk, P // 4, nb, 4)[page, :, quad, :, lane].float()[..., None]
    v = val[rec[:, :, h:2 * h].view(-1, hk, P // 4, 16, 4, nb)[page, :, quad, :, lane].int()].permute(0, 1, 3, 4, 2).reshape(T, hk, nb, 32)
    v = v * halves[:, :, h + P * nb:].view(-1, hk, P // 4, nb, 4)[page, :, quad, :, lane].float()[..., None]
    return k.view(T, hk, D), v.view(T, hk, D)


def plain_plan(s):
    B, P, n, dev = s["B"], s["P"], s["max_tokens"], s["lens"].device
    old, add = s["lens"].long(), s["new_lens"].long()
    zero = torch.zeros(1, dtype=torch.long, device=dev)
    have, want = (old + P - 1) // P, (old + add + P - 1) // P
    cu = torch.cat([zero, add.cumsum(0)])
    cup = torch.cat([zero, (want - have).cumsum(0)])
    status = torch.cat([(cup[-1:] > s["count"]) + 2 * (cu[-1:] > n) + 4 * ((want > s["stride"]) | (add < 0)).any().view(1), cup[-1:], cu[-1:]])
    ok = status[0] == 0
    cu, cup = cu * ok, cup * ok
    # new pages: the i-th of all, in order of requests and blocks, is the i-th from the top of the free list
    blk = torch.arange(s["stride"], device=dev)
    take = ok & (blk >= have[:, None]) & (blk < want[:, None])
    i = s["count"].long() - 1 - (cup[:-1, None] + blk - have[:, None])
    table = s["table"]
    table.copy_(torch.where(take, s["free"][i.clamp(0, s["free"].numel() - 1)], table))
    t = torch.arange(n, device=dev)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=B - 1)
    pos = old[b] + t - cu[b]
    real = t < cu[-1]
    pos = torch.where(real, pos, torch.zeros_like(pos))
    slots = torch.where(real, table[b, pos // P].long() * P + pos % P, torch.full_like(pos, -1))
    i32 = torch.int32
    return dict(lens=(old + add * ok).to(i32), count=(s["count"] - cup[-1]).to(i32), cu=cu.to(i32), pages=cup.to(i32), positions=pos.to(i32),
                status=status.to(i32), slots=slots, table=table)


def plain_logits(s):
    x = s["logits"].float()
    B, V, H, dev = s["B"], s["V"], s["tokens"].shape[1], x.device
    at = torch.arange(H, device=dev)
    tok = s["tokens"].long()
    live = at < s["total"][:, None]
    written = live & (at >= s["prompt"][:, None])
    seen = torch.zeros(B, V, dtype=torch.int32, device=dev).scatter_add_(1, tok, live.int())
    count = torch.zeros(B, V, dtype=torch.int32, device=dev).scatter_add_(1, tok, written.int())
    r = s["rep"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - s["freq"][:, None] * count
    x = x - s["pres"][:, None] * (count > 0)
    if "btok" in s:
        n = torch.arange(s["btok"].shape[1], device=dev) < s["blen"][:, None]
        x = x.scatter_add(1, s["btok"].long(), torch.where(n, s["bval"], torch.zeros_like(s["bval"])))
    if "bits" in s:
        t = torch.arange(V, device=dev)
        x = x.masked_fill(((s["bits"][:, t >> 5] >> (t & 31)) & 1) == 0, -math.inf)
    return x.to(s["logits"].dtype)


# ---- what a pass cannot do without --------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "attn":
        h = torch.Generator()
        h.manual_seed(0)  # ragged lengths differ from seed to seed, their sums little
        kvs, news = lengths(case, h)
        w = case["window"]
        pairs = touched = 0
        for kv, n in zip(kvs, news):
            if w:
                a = max(0, min(n, w - (kv - n)))  # query rows whose window reaches back to the first key
                pairs += a * (kv - n) + a * (a + 1) // 2 + (n - a) * w
                touched += min(kv, n + w - 1)
            else:
                pairs += n * (kv - n) + n * (n + 1) // 2
                touched += kv
        rows = sum(news)
        return {"bytes": touched * case["hk"] * case["D"] * 9 // 8 + 2 * rows * case["hq"] * case["D"] * SIZE[case["t"]] + 4 * touched // case["P"],
                "flops": 4 * case["D"] * case["hq"] * pairs}
    if op == "append":  # the rows in, the cache written and read, the rows out in fp32
        n = 2 * case["T"] * case["hk"] * case["D"]
        return {"bytes": n * SIZE[case["t"]] + 2 * (n * 9 // 16) + 4 * n + 8 * case["T"], "flops": 10 * n}
    if op == "plan":
        B, P, n = case["B"], case["P"], case["B"] * (1 if case["new"] == 1 else case["new"] / 2)
        return {"bytes": 20 * B + 12 * n + 12 * (n / P + B / 2), "flops": 10 * (n + B)}
    n = case["B"] * case["V"]
    return {"bytes": 2 * n * SIZE[case["t"]] + (n // 8 if case["mask"] else 0) + case["B"] * (4 * case["hist"] * 0.65 + 4 * case["bias"] + 20),
            "flops": 4 * n}


# ---- the definition in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"attn": exact_attn, "append": exact_append, "logits": exact_logits}[case["op"]](s)


def exact_rows(s, b, h, length):
    """Keys and values [length, D] of request b, kv head h, in fp64, element by element from the record's layout."""
    P, D = s["P"], s["D"]
    nb, dev = D // 32, s["q"].device
    t = torch.arange(length, device=dev)
    flat = s["cache"].view(-1)
    base = (s["table"][b].long()[t // P] * s["hk"] + h) * (P * D * 9 // 8)
    o, e = (t % P)[:, None], torch.arange(D, device=dev)[None, :]
    mag = torch.tensor(E2M1, dtype=torch.float64, device=dev)

    def value(byte, high, scale_at):
        raw = flat[base[:, None] + byte].to(torch.int64)
        c = torch.where(high, raw >> 4, raw & 15)
        at = base[:, None] + scale_at + 2 * ((o // 4) * nb * 4 + (e // 32) * 4 + o % 4)
        bits = flat[at].to(torch.int64) | (flat[at + 1].to(torch.int64) << 8)
        d = bits.to(torch.int16).view(torch.float16).double()
        return torch.where(c >= 8, -mag[c & 7], mag[c & 7]) * d

    k = value(o * (D // 2) + ((e % 32) // 8) * (D // 8) + (e // 32) * 4 + (e % 8) // 2, (e % 2 == 1).expand(length, D), P * D)
    v = value(P * D // 2 + (o // 4) * (2 * D) + (e % 16) * (4 * nb) + (o % 4) * nb + e // 32, ((e // 16) % 2 == 1).expand(length, D),
              P * D + 2 * P * nb)
    return k, v


def exact_attn(s):
    G, w = s["hq"] // s["hk"], s["window"]
    out = torch.zeros(s["T"], s["hq"], s["D"], dtype=torch.float64, device=s["q"].device)
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    for b in range(s["B"]):
        n, kv = cu[b + 1] - cu[b], lens[b]
        pos = kv - n + torch.arange(n, device=out.device)[:, None]
        j = torch.arange(kv, device=out.device)[None, :]
        hide = (j > pos) | ((j <= pos - w) if w else torch.zeros_like(j, dtype=torch.bool))
        for h in range(s["hk"]):
            k, v = exact_rows(s, b, h, kv)
            for i in range(G):
                a = (s["q"][cu[b]:cu[b + 1], h * G + i].double() @ k.T) * s["scale"]
                out[cu[b]:cu[b + 1], h * G + i] = torch.softmax(a.masked_fill(hide, -math.inf), -1) @ v
    return out


def exact_append(s):
    def held(x):
        x = x.double().view(s["T"], s["hk"], -1, 32)
        d = (x.abs().amax(-1, keepdim=True).float() / 6).to(torch.float16).double()  # the scale as the format holds it
        grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
        far = (x.abs()[..., None] - d[..., None] * grid).abs()
        best = far.amin(-1, keepdim=True)
        tie = far == best
        even = tie & (torch.arange(8, device=x.device) % 2 == 0)
        c = torch.where(even.any(-1), even.int().argmax(-1), tie.int().argmax(-1))
        return (grid[c] * d * x.sign()).view(s["T"], s["hk"], s["D"])

    return held(s["k"]), held(s["v"])


def exact_logits(s):
    x = s["logits"].double()
    out = x.clone()
    total, prompt = s["total"].tolist(), s["prompt"].tolist()
    for b in range(s["B"]):
        tok = s["tokens"][b, :total[b]].long()
        seen, said = torch.unique(tok), torch.bincount(tok[prompt[b]:], minlength=s["V"]).double()
        r = s["rep"][b].double()
        out[b, seen] = torch.where(x[b, seen] > 0, x[b, seen] / r, x[b, seen] * r)
        out[b] -= s["freq"][b].double() * said + s["pres"][b].double() * (said > 0)
        if "btok" in s:
            n = int(s["blen"][b])
            out[b].index_add_(0, s["btok"][b, :n].long(), s["bval"][b, :n].double())
        if "bits" in s:
            word = s["bits"][b].long() & 0xFFFFFFFF
            allowed = ((word[:, None] >> torch.arange(32, device=x.device)) & 1).view(-1)[:s["V"]].bool()
            out[b, ~allowed] = -math.inf
    return out
