"""More operators around the low-bit products, as they are timed: products with 4-bit weights (Q4_0), routing of tokens to
experts, the experts' products of the routed tokens, and keys and values appended to the 4-bit cache with the position
rotation applied on the way.

Weights, as the products read them (one tensor of N x K; the experts' tensors lie one after another, each padded to a
multiple of 16 bytes): all 16-byte code records row by row, then all binary16 scales row by row.  A record is
  q4   32 weights: byte j holds weights 2j (low nibble) and 2j + 1, as 4-bit two's complement; weight = d * nibble
  q2   64 weights: byte j holds weights 4j .. 4j + 3, lowest bits first; weight = d * (code - 1)
  q1  128 weights: the sign of weight 32r + 8m + k at bit 4k + r of dword m; weight = d * (bit ? 1 : -1)
Activations are q8_0: signed bytes and one binary16 scale per 32.

The cache: pages of P tokens, one record per page and kv head.  32 consecutive values of a token's head share a binary16
scale d = fp16(amax * fp32(1/6)); a code is the E2M1 number (sign and 0 .5 1 1.5 2 3 4 6) nearest to x / d, ties to the
even code.  A record holds, with nb = D / 32 blocks a row:
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
BLOCK = {"q1": 128, "q2": 64, "q4": 32}  # weights a record
FORMAT = {"q1": 1, "q2": 2, "q4": 6}  # the library's lb_wfmt


def listed():
    return [
        # 4-bit products: the smallest projection of a small model's token, where latency counts
        dict(name="q4_projection", op="q4", M=1, N=640, K=2560),
        # a feed-forward product of a token
        dict(name="q4_feed_forward", op="q4", M=1, N=12288, K=4096),
        # the head of a token, an odd number of rows
        dict(name="q4_head", op="q4", M=1, N=151669, K=4096),
        # a prompt's rows
        dict(name="q4_prompt", op="q4", M=512, N=4096, K=12288),
        # routing: one token of one chat
        dict(name="route_token_f32", op="route", t="f32", T=1, E=64, k=8, score="softmax", bias=False, groups=1, kept=1, best=1, renorm=True),
        # a long prompt, with groups and a bias for balance
        dict(name="route_prompt_bf16", op="route", t="bf16", T=8191, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4, best=2,
             renorm=True),
        # experts' first products (gate and up together): one token
        dict(name="experts_token_q2", op="experts", fmt="q2", T=1, E=64, k=8, N=1536, K=2048, down=False, t="f32"),
        # experts' last products with the sum over a token's experts: a decode step of a few dozen requests, most experts with few rows
        dict(name="experts_decode_q4", op="experts", fmt="q4", T=45, E=128, k=8, N=2048, K=768, down=True, t="bf16"),
        # a prompt of single-bit experts
        dict(name="experts_prompt_q1", op="experts", fmt="q1", T=4096, E=64, k=6, N=2816, K=2048, down=False, t="f32"),
        # a chunk's last products and their sum
        dict(name="experts_chunk_q2", op="experts", fmt="q2", T=1000, E=32, k=4, N=2560, K=1408, down=True, t="f16"),
        # rotation and cache: the rows of one decode step, far into their requests
        dict(name="rotary_decode_f32", op="rotary", t="f32", T=32, hq=32, hk=8, D=128, P=16, rd=128, pairs=False, far=131071),
        # the rows of a prompt
        dict(name="rotary_prompt_bf16", op="rotary", t="bf16", T=16384, hq=32, hk=8, D=128, P=32, rd=128, pairs=False, far=0),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["q4", "route", "experts", "experts", "rotary"])
    if op == "q4":
        if rng.random() < 0.7:
            return dict(op=op, M=1, N=log(1, 150000), K=32 * log(2, 128))
        return dict(op=op, M=log(2, 512), N=log(16, 4096), K=128 * log(1, 90))
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
        groups = rng.choice([1, 1, 2, 4])
        kept = rng.randint(1, groups)
        best = rng.choice([1, 2]) if groups > 1 else 1
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, t=rng.choice(["f32", "f32", "bf16", "f16"]), T=log(1, 8000), E=E, k=rng.randint(1, min(10, E // groups * kept)),
                    score=score, bias=rng.random() < (0.7 if score == "sigmoid" else 0.3), groups=groups, kept=kept, best=best,
                    renorm=rng.random() < 0.7)
    if op == "experts":
        E = rng.choice([8, 16, 32, 60, 64, 128])
        return dict(op=op, fmt=rng.choice(["q1", "q2", "q4"]), T=log(1, 2000), E=E, k=rng.randint(1, min(8, E)), N=log(100, 2500),
                    K=128 * log(2, 16), down=rng.random() < 0.5, t=rng.choice(["f32", "bf16", "f16"]))
    hk = rng.choice([1, 2, 4, 5, 8])
    D = rng.choice([64, 128, 128, 256])
    return dict(op=op, t=rng.choice(["f32", "bf16", "f16"]), T=log(1, 8000), hq=hk * rng.choice([1, 2, 4, 5, 7]), hk=hk, D=D,
                P=rng.choice([16, 32, 64, 128]), rd=rng.choice([D, D, D // 2, 16]), pairs=rng.random() < 0.4,
                far=rng.choice([0, log(1, 1000000)]))


# ---- what the caller has in hand ----------------------------------------------------------------

def record_bytes(P, D):
    return P * D * 9 // 8


def tensor_bytes(fmt, N, K):
    return N * (K // BLOCK[fmt]) * 18


def stride_bytes(fmt, N, K):
    return -(-tensor_bytes(fmt, N, K) // 16) * 16


def random_weights(fmt, E, N, K, g):
    """E tensors of random codes, with scales of the size that trained weights have."""
    w = torch.zeros(E, stride_bytes(fmt, N, K), dtype=torch.uint8, device=DEV)
    n = N * (K // BLOCK[fmt])
    w[:, :16 * n] = torch.randint(0, 256, (E, 16 * n), dtype=torch.uint8, device=DEV, generator=g)
    d = torch.rand(E, n, device=DEV, generator=g).mul_(0.02).add_(0.005).to(torch.float16)
    w[:, 16 * n:18 * n] = d.view(torch.uint8)
    return w


def random_rows(M, K, g):
    """q8_0 rows: the bytes of normal values whose largest of 32 is 127, and scales to match."""
    x = torch.randn(M, K // 32, 32, device=DEV, generator=g)
    a = x.abs().amax(-1)
    q = (x * (127 / a)[..., None]).round().to(torch.int8)
    return q.view(M, K), (a / 127).to(torch.float16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "q4":
        s["W"] = random_weights("q4", 1, case["N"], case["K"], g)[0]
        s["xq"], s["xs"] = random_rows(case["M"], case["K"], g)
    elif op == "route":
        T, E = case["T"], case["E"]
        skew = 0.7 * torch.randn(E, device=DEV, generator=g)  # some experts are liked better
        s["logits"] = (1.5 * torch.randn(T, E, device=DEV, generator=g) + skew).to(TYPES[case["t"]])
        s["b"] = 0.1 * torch.randn(E, device=DEV, generator=g) if case["bias"] else None
    elif op == "experts":
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        s["W"] = random_weights(case["fmt"], E, N, K, g)
        s["xq"], s["xs"] = random_rows(T * k if case["down"] else T, K, g)
        like = torch.randn(T, E, device=DEV, generator=g) + 0.5 * torch.randn(E, device=DEV, generator=g)
        top = like.topk(k, -1)
        s["experts"] = top.indices.to(torch.int32)
        s["weights"] = torch.softmax(top.values, -1)
        s["most"] = int(torch.bincount(s["experts"].flatten().long(), minlength=E).max())  # rows of the busiest expert
    else:
        T, hq, hk, D, P, far = (case[n] for n in ("T", "hq", "hk", "D", "P", "far"))
        step = far > 0 and T <= 64  # a decode step: each row at the end of its own request's page
        pages = max(T, 4) if step else -(-T // P) + 4
        order = torch.randperm(pages, generator=g, device=DEV)
        t = torch.arange(T, device=DEV)
        if step:
            s["slots"] = order[:T] * P + torch.randint(0, P, (T,), generator=g, device=DEV)
            s["positions"] = torch.randint(0, far + 1, (T,), generator=g, device=DEV).to(torch.int32)
        else:  # rows one after another, through pages in any order
            s["slots"] = order[t // P] * P + t % P
            s["positions"] = (t + far).to(torch.int32)
        i = torch.arange(case["rd"] // 2, device=DEV, dtype=torch.float64)
        s["freq"] = (1e6 ** (-2 * i / case["rd"])).to(torch.float32)
        s.update(pages=pages, cache=torch.zeros(pages, hk, record_bytes(P, D), dtype=torch.uint8, device=DEV))
        # queries, keys and values as a product leaves them: parts of one wide row
        wide = torch.randn(T, (hq + 2 * hk) * D, generator=g, device=DEV).to(TYPES[case["t"]])
        s["q"], s["k"], s["v"] = (x.view(T, -1, D) for x in wide.split([hq * D, hk * D, hk * D], -1))
    return s


# ---- one pass -----------------------------------------------------------------------------------

def run(s):
    if own:
        return {"q4": own_q4, "route": own_route, "experts": own_experts, "rotary": own_rotary}[s["op"]](s)
    return {"q4": plain_q4, "route": plain_route, "experts": plain_experts, "rotary": plain_rotary}[s["op"]](s)


def own_q4(s):
    import bit_quantized_matvec_q1_amd.lowbit as L

    y = torch.empty(s["M"], s["N"], dtype=torch.float32, device=s["xq"].device)
    if s["M"] == 1:
        L.lowbit_matvec(L.Q4_0, s["W"], s["N"], s["K"], 1.0, L.ACT_Q8_0, s["xq"], s["xs"], y)
    else:
        L.lowbit_gemm(L.Q4_0, s["W"], s["N"], s["K"], 1.0, L.ACT_Q8_0, s["xq"], s["xs"], s["M"], y)
    return y


def own_route(s):
    import bit_quantized_matvec_q1_amd.lowbit as L

    T, k, dev = s["T"], s["k"], s["logits"].device
    experts = torch.empty(T, k, dtype=torch.int32, device=dev)
    weights = torch.empty(T, k, dtype=torch.float32, device=dev)
    L.lowbit_route(CODE[s["t"]], s["logits"], T, s["E"], k, experts, weights,
                   score=L.SCORE_SIGMOID if s["score"] == "sigmoid" else L.SCORE_SOFTMAX, bias=s["b"], groups=s["groups"],
                   groups_kept=s["kept"], group_best=s["best"], renormalise=s["renorm"])
    return experts, weights


def own_experts(s):
    import bit_quantized_matvec_q1_amd.lowbit as L

    T, E, k, N, K, dev = s["T"], s["E"], s["k"], s["N"], s["K"], s["xq"].device
    plan = None
    if T > 1:
        plan = torch.empty(L.lowbit_experts_plan_bytes(T * k, E), dtype=torch.uint8, device=dev)
        L.lowbit_experts_plan(s["experts"], T * k, E, plan)
    y = torch.empty(T * k, N, dtype=torch.float32, device=dev)
    L.lowbit_experts_matmul(FORMAT[s["fmt"]], s["W"], E, N, K, s["xq"], s["xs"], s["experts"], T * k, 1 if s["down"] else k, y, plan=plan)
    if not s["down"]:
        return y
    out = torch.empty(T, N, dtype=TYPES[s["t"]], device=dev)
    L.lowbit_experts_combine(CODE[s["t"]], y, s["experts"], s["weights"], T, k, E, N, out)
    return out


def own_rotary(s):
    import bit_quantized_matvec_q1_amd.lowbit as L

    T, hq, hk, D = s["T"], s["hq"], s["hk"], s["D"]
    q = torch.empty(T, hq, D, dtype=s["q"].dtype, device=s["q"].device)
    L.lowbit_kv_append_rotary(CODE[s["t"]], s["q"], q, s["k"], s["v"], T, hq, hk, D, s["positions"], s["freq"], s["rd"],
                              L.ROTARY_PAIRS if s["pairs"] else L.ROTARY_HALVES, s["slots"], s["cache"], s["pages"], s["P"])
    k, v = (torch.empty(T, hk, D, dtype=torch.float32, device=s["k"].device) for _ in range(2))
    L.lowbit_kv_read(CODE["f32"], s["cache"], s["pages"], s["P"], T, hk, D, s["slots"], k, v)
    return q, k, v


def split(w, fmt, N, K):
    """[..., bytes] -> code bytes [..., N, K / block, 16] and scales [..., N, K / block] in fp32."""
    n = K // BLOCK[fmt]
    d = w[..., 16 * N * n:18 * N * n].contiguous().view(torch.float16).float()
    return w[..., :16 * N * n].reshape(*w.shape[:-1], N, n, 16), d.view(*w.shape[:-1], N, n)


def plain_weights(w, fmt, N, K):
    """[..., bytes] -> [..., N, K] weights in fp32."""
    c, d = split(w, fmt, N, K)
    b = torch.arange(256, device=w.device)[:, None]
    if fmt == "q4":
        v = ((b >> torch.tensor([0, 4], device=w.device) & 15) ^ 8) - 8
        v = v.float()[c.int()].flatten(-2)  # [..., n, 32]
    elif fmt == "q2":
        v = ((b >> torch.tensor([0, 2, 4, 6], device=w.device)) & 3) - 1
        v = v.float()[c.int()].flatten(-2)  # [..., n, 64]
    else:
        at = torch.arange(8, device=w.device) * 4 + torch.arange(4, device=w.device)[:, None]  # [r][k]
        m = c.contiguous().view(torch.int32)  # [..., n, 4]
        v = (m[..., None, :, None] >> at[:, None, :]) & 1  # [..., n, r, m, k]
        v = (2 * v - 1).float().flatten(-3)
    return (v * d[..., None]).flatten(-2)


def plain_rows(xq, xs):
    return (xq.float().view(*xs.shape, 32) * xs.float()[..., None]).flatten(-2)


def plain_q4(s):
    w = plain_weights(s["W"], "q4", s["N"], s["K"])
    return plain_rows(s["xq"], s["xs"]) @ w.t()


def plain_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    x = s["logits"].double()
    p = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.exp(x - x.amax(-1, keepdim=True))
    if s["score"] == "softmax":
        p = p / p.sum(-1, keepdim=True)
    sel = p if s["b"] is None else p + s["b"].double()
    if G > 1:
        per = sel.view(T, G, E // G)
        top = per.sort(dim=-1, descending=True).values[..., :s["best"]].sum(-1)
        keep = top.sort(dim=-1, descending=True, stable=True).indices[:, :s["kept"]]
        use = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, keep, torch.ones_like(keep, dtype=torch.bool))
        sel = per.masked_fill(~use[..., None], -math.inf).view(T, E)
    at = sel.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, at)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return at.to(torch.int32), w.float()


def plain_experts(s):
    T, E, k, N, K, most = (s[n] for n in ("T", "E", "k", "N", "K", "most"))
    dev, n = s["xq"].device, T * k
    e = s["experts"].flatten().long()
    order = torch.argsort(e, stable=True)
    count = torch.zeros(E, dtype=torch.long, device=dev).scatter_add_(0, e, torch.ones_like(e))
    at = torch.empty_like(e)
    at[order] = torch.arange(n, device=dev) - (count.cumsum(0) - count)[e[order]]  # place among the rows of its expert
    p = torch.arange(n, device=dev)
    x = plain_rows(s["xq"], s["xs"])[p if s["down"] else p // k]
    if n <= E // 2:  # few rows: the weights of each one's expert
        y = (plain_weights(s["W"][e], s["fmt"], N, K) * x[:, None]).sum(-1)
    else:  # the rows of each expert together, up to those of the busiest
        rows = torch.zeros(E, most, K, device=dev)
        rows[e, at] = x
        y = torch.bmm(rows, plain_weights(s["W"], s["fmt"], N, K).transpose(1, 2).contiguous())[e, at]
    if not s["down"]:
        return y
    return (y.view(T, k, N) * s["weights"][..., None]).sum(1).to(TYPES[s["t"]])


# the values of a byte's two codes
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def byte_values(device):
    v = torch.tensor(E2M1 + [-x for x in E2M1], device=device)
    b = torch.arange(256, device=device)
    return torch.stack([v[b & 15], v[b >> 4]], -1)  # [256][2]


def plain_codes(x, D):
    """[T, hk, D] rows -> codes [T, hk, nb, 32] (uint8) and scales [T, hk, nb] (fp16)."""
    x = x.float().view(*x.shape[:-1], D // 32, 32)
    a = x.abs()
    d = (a.amax(-1) * torch.tensor(1 / 6, dtype=torch.float32, device=x.device)).clamp(max=65504).to(torch.float16)
    b = d.float()[..., None]
    c = (a > b * 0.25).to(torch.uint8) + (a >= b * 0.75) + (a > b * 1.25) + (a >= b * 1.75) + (a > b * 2.5) + (a >= b * 3.5) + (a > b * 5)
    return torch.where(b > 0, c | ((x < 0).to(torch.uint8) << 3), torch.zeros_like(c)), d


def plain_turn(s, x):
    """Rows [T, heads, D] turned by their positions: angles, sines and products in 64 bits, rounded to 32 and to the type."""
    rd = s["rd"]
    a = s["positions"].double()[:, None] * s["freq"].double()
    c, n = a.cos()[:, None], a.sin()[:, None]
    w = x[..., :rd].double()
    if s["pairs"]:
        w = w.unflatten(-1, (-1, 2))
        w = torch.stack([w[..., 0] * c - w[..., 1] * n, w[..., 1] * c + w[..., 0] * n], -1).flatten(-2)
    else:
        lo, hi = w[..., :rd // 2], w[..., rd // 2:]
        w = torch.cat([lo * c - hi * n, hi * c + lo * n], -1)
    return torch.cat([w.float().to(x.dtype), x[..., rd:]], -1)


def plain_rotary(s):
    T, hk, D, P, nb = s["T"], s["hk"], s["D"], s["P"], s["D"] // 32
    rec, page, off = s["cache"], s["slots"] // s["P"], s["slots"] % s["P"]
    quad, lane, h = off // 4, off % 4, P * D // 2
    c, d = plain_codes(plain_turn(s, s["k"]), D)
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
    return plain_turn(s, s["q"]), k.view(T, hk, D), v.view(T, hk, D)


# ---- what a pass cannot do without --------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "q4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": tensor_bytes("q4", N, K) + M * K * 17 // 16 + 4 * M * N, "flops": 2 * M * N * K}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * SIZE[case["t"]] + 8 * T * k + (4 * E if case["bias"] else 0), "flops": T * E * 10}
    if op == "experts":
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        touched = E * (1 - (1 - k / E) ** T)  # experts with a row
        rows = T * k if case["down"] else T
        out = T * N * SIZE[case["t"]] if case["down"] else 4 * T * k * N
        return {"bytes": int(touched * tensor_bytes(case["fmt"], N, K)) + rows * K * 17 // 16 + out + 8 * T * k, "flops": 2 * T * k * N * K}
    T, hq, hk, D, z = case["T"], case["hq"], case["hk"], case["D"], SIZE[case["t"]]
    n = 2 * T * hk * D  # the rows in, queries out, the cache written and read, keys and values out in fp32
    return {"bytes": 2 * T * hq * D * z + n * z + 2 * (n * 9 // 16) + 4 * n + 12 * T, "flops": 10 * n + 3 * T * (hq + hk) * case["rd"]}


# ---- the definition in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"q4": exact_q4, "route": exact_route, "experts": exact_experts, "rotary": exact_rotary}[case["op"]](s)


def exact_matrix(w, fmt, N, K, rows):
    """Rows `rows` of one tensor in fp64, weight by weight from the layout."""
    b = BLOCK[fmt]
    r, i = rows[:, None], torch.arange(K, device=w.device)[None, :]
    rec, j = r * (K // b) + i // b, i % b
    if fmt == "q4":
        c = w[16 * rec + j // 2].long() >> (4 * (j % 2)) & 15
        v = torch.where(c >= 8, c - 16, c)
    elif fmt == "q2":
        v = (w[16 * rec + j // 4].long() >> (2 * (j % 4)) & 3) - 1
    else:
        bit = 4 * (j % 8) + j // 32  # of dword m
        v = 2 * (w[16 * rec + 4 * (j % 32 // 8) + bit // 8].long() >> (bit % 8) & 1) - 1
    at = 16 * N * (K // b) + 2 * rec
    d = (w[at].to(torch.int32) | w[at + 1].to(torch.int32) << 8).to(torch.int16).view(torch.float16).double()
    return v.double() * d


def exact_x(s):
    return s["xq"].double() * s["xs"].double().repeat_interleave(32, -1)


def exact_q4(s):
    x = exact_x(s)
    parts = [x @ exact_matrix(s["W"], "q4", s["N"], s["K"], r).T for r in torch.arange(s["N"], device=x.device).split(16384)]
    return torch.cat(parts, 1)


def exact_experts(s):
    T, E, k, N, K = (s[n] for n in ("T", "E", "k", "N", "K"))
    x, e = exact_x(s), s["experts"].flatten()
    y = torch.zeros(T * k, N, dtype=torch.float64, device=x.device)
    for i in range(E):
        p = (e == i).nonzero().flatten()
        if p.numel():
            y[p] = x[p if s["down"] else p // k] @ exact_matrix(s["W"][i], s["fmt"], N, K, torch.arange(N, device=x.device)).T
    return torch.einsum("tkn,tk->tn", y.view(T, k, N), s["weights"].double()) if s["down"] else y


def exact_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    x = s["logits"].double()
    p = 1 / (1 + (-x).exp()) if s["score"] == "sigmoid" else torch.softmax(x, -1)
    sel = p.clone() if s["b"] is None else p + s["b"].double()
    if G > 1:
        left = sel.view(T, G, E // G).clone()
        score = torch.zeros(T, G, dtype=torch.float64, device=x.device)
        for _ in range(s["best"]):
            m, i = left.max(-1)
            score += m
            left.scatter_(-1, i[..., None], -math.inf)
        drop = torch.ones(T, G, dtype=torch.bool, device=x.device)
        for _ in range(s["kept"]):
            best = (score == score.amax(-1, keepdim=True)).int().argmax(-1, keepdim=True)
            drop.scatter_(1, best, False)
            score.scatter_(1, best, -math.inf)
        sel[drop.repeat_interleave(E // G, 1)] = -math.inf
    w = torch.zeros(T, k, dtype=torch.float64, device=x.device)
    for j in range(k):
        i = (sel == sel.amax(-1, keepdim=True)).int().argmax(-1, keepdim=True)
        w[:, j:j + 1] = p.gather(1, i)
        sel.scatter_(1, i, -math.inf)
    return None, w / w.sum(-1, keepdim=True) if s["renorm"] else w


def exact_rotary(s):
    rd, dev = s["rd"], s["q"].device
    i = torch.arange(rd, device=dev)
    pair = i // 2 if s["pairs"] else i % (rd // 2)
    first = i % 2 == 0 if s["pairs"] else i < rd // 2
    other = torch.where(first, i + (1 if s["pairs"] else rd // 2), i - (1 if s["pairs"] else rd // 2))
    z = torch.polar(torch.ones((), dtype=torch.float64, device=dev), s["positions"].double()[:, None] * s["freq"].double()[pair])[:, None]

    def turn(x):
        x = x.double()
        w = x.clone()
        w[..., :rd] = x[..., :rd] * z.real + torch.where(first, -x[..., other], x[..., other]) * z.imag
        return w

    def held(x):  # fp32 values as the cache holds them
        x = x.double().view(s["T"], s["hk"], -1, 32)
        d = (x.abs().amax(-1, keepdim=True).float() * torch.tensor(1 / 6, device=dev)).to(torch.float16).double()  # as the format has it
        grid = torch.tensor(E2M1, dtype=torch.float64, device=dev)
        far = (x.abs()[..., None] - d[..., None] * grid).abs()
        tie = far == far.amin(-1, keepdim=True)
        even = tie & (torch.arange(8, device=dev) % 2 == 0)
        c = torch.where(even.any(-1), even.int().argmax(-1), tie.int().argmax(-1))
        return (grid[c] * d * x.sign()).view(s["T"], s["hk"], s["D"])

    return turn(s["q"]), held(turn(s["k"]).float().to(s["k"].dtype)), held(s["v"])
