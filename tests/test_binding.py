"""The binding's refusals by name: each argument's size, type and layout by itself, where everything else is in order."""
import pytest
import torch

import bit_quantized_matvec_q1_amd.lowbit as L

U8, I8, I32, I64, F16, F32 = torch.uint8, torch.int8, torch.int32, torch.int64, torch.float16, torch.float32
RIGHT = "device tensor required"  # all that is wrong with right arguments on the host


def zeros(device, **shapes):
    return {name: torch.zeros(shape, dtype=dtype, device=device) for name, (shape, dtype) in shapes.items()}


def refuse(call, args, **bad):
    """Each (argument, what the message says) by itself."""
    for name, (x, says) in bad.items():
        with pytest.raises(ValueError, match=says):
            call(**(args | {name: x}))


def product(device):
    a = zeros(device, W=(L.lowbit_weight_bytes(L.Q4_0, 8, 64), U8), xq=(64, I8), xs=(2, F16), y=(8, F32))
    call = lambda W, xq, xs, y: L.lowbit_matvec(L.Q4_0, W, 8, 64, 1.0, L.ACT_Q8_0, xq, xs, y)  # noqa: E731
    bad = dict(W=(a["W"][:-1], "^W: needs at least 288 bytes, has 287"), xq=(a["xq"][:-1], "^xq: needs at least 64"), xs=(a["xs"][:1], "^xscale: needs at least 2"),
               y=(a["y"][:7], "^y: needs at least 8"))
    return call, a, bad, dict(xq=(a["xq"].to(U8), "^xq: dtype"), xs=(a["xs"].float(), "^xscale: dtype"), y=(a["y"].double(), "^y: dtype"))


def many(device):
    a = zeros(device, W=(L.lowbit_weight_bytes(L.Q4_0, 8, 128), U8), xq=((3, 128), I8), xs=((3, 4), F16), y=((3, 8), F32))
    call = lambda W, xq, xs, y: L.lowbit_gemm(L.Q4_0, W, 8, 128, 1.0, L.ACT_Q8_0, xq, xs, 3, y)  # noqa: E731
    bad = dict(W=(a["W"][:-1], "^W: needs at least"), xq=(a["xq"][:2], "^Xq: needs at least 384"), xs=(a["xs"][:2], "^Xscale: needs at least 12"),
               y=(a["y"][:2], "^Y: needs at least 24"))
    return call, a, bad, dict(xq=(a["xq"].to(U8), "^Xq: dtype"), xs=(a["xs"].float(), "^Xscale: dtype"), y=(a["y"].double(), "^Y: dtype"))


def experts(device):
    a = zeros(device, W=(L.lowbit_experts_weight_bytes(L.Q4_0, 2, 8, 128), U8), xq=((3, 128), I8), xs=((3, 4), F16), e=(6, I32), y=((6, 8), F32),
              plan=(L.lowbit_experts_plan_bytes(6, 2), U8))
    call = lambda W, xq, xs, e, y, plan: L.lowbit_experts_matmul(L.Q4_0, W, 2, 8, 128, xq, xs, e, 6, 2, y, plan=plan)  # noqa: E731
    bad = dict(W=(a["W"][:-1], "^W: needs at least"), xq=(a["xq"][:2], "^xq: needs at least 384"), xs=(a["xs"][:2], "^xscale: needs at least 24 bytes"),
               e=(a["e"][:5], "^experts: needs at least 6"), y=(a["y"][:5], "^y: needs at least 48"), plan=(a["plan"][:-16], "^plan: needs at least"))
    return call, a, bad, dict(xq=(a["xq"].to(U8), "^xq: dtype"), xs=(a["xs"].float(), "^xscale: dtype"), e=(a["e"].long(), "^experts: dtype"),
                              y=(a["y"].double(), "^y: dtype"))


def plan(device):
    a = zeros(device, e=(6, I32), plan=(L.lowbit_experts_plan_bytes(6, 2), U8))
    call = lambda e, plan: L.lowbit_experts_plan(e, 6, 2, plan)  # noqa: E731
    return call, a, dict(e=(a["e"][:5], "^experts: needs at least 6"), plan=(a["plan"][:-1], "^plan: needs at least")), dict(e=(a["e"].long(), "^experts: dtype"))


def combine(device):
    a = zeros(device, y=((6, 8), F32), e=(6, I32), w=(6, F32), out=((3, 8), F32))
    call = lambda y, e, w, out: L.lowbit_experts_combine(L.F32, y, e, w, 3, 2, 2, 8, out)  # noqa: E731
    bad = dict(y=(a["y"][:5], "^y: needs at least 48"), e=(a["e"][:5], "^experts: needs at least 6"), w=(a["w"][:5], "^weights: needs at least 6"),
               out=(a["out"][:2], "^out: needs at least 3 rows"))
    return call, a, bad, dict(y=(a["y"].double(), "^y: dtype"), e=(a["e"].long(), "^experts: dtype"), w=(a["w"].half(), "^weights: dtype"),
                              out=(a["out"].half(), "^out: dtype"))


def route(device):
    a = zeros(device, x=((4, 64), F32), bias=(64, F32), count=(1, I32), e=((4, 8), I32), w=((4, 8), F32))
    call = lambda x, bias, count, e, w: L.lowbit_route(L.F32, x, 4, 64, 8, e, w, bias=bias, count=count)  # noqa: E731
    bad = dict(x=(a["x"][:3], "^logits: shape"), bias=(a["bias"][:63], "^bias: needs at least 64"), count=(a["count"][:0], "^count: needs at least 1"),
               e=(a["e"][:3], "^experts: needs at least 32"), w=(a["w"][:3], "^weights: needs at least 32"))
    return call, a, bad, dict(x=(a["x"].half(), "^logits: a tensor of"), bias=(a["bias"].half(), "^bias: dtype"), count=(a["count"].long(), "^count: dtype"),
                              e=(a["e"].long(), "^experts: dtype"), w=(a["w"].double(), "^weights: dtype"))


def rotary(device):
    a = zeros(device, q=((4, 8, 64), F32), qo=((4, 8, 64), F32), k=((4, 2, 64), F32), v=((4, 2, 64), F32), pos=(4, I32), freq=(32, F32), slots=(4, I64),
              cache=(L.lowbit_kv_cache_bytes(4, 2, 16, 64), U8))
    a["slots"] += torch.arange(4, device=device)

    def call(q, qo, k, v, pos, freq, slots, cache):
        L.lowbit_kv_append_rotary(L.F32, q, qo, k, v, 4, 8, 2, 64, pos, freq, 64, L.ROTARY_HALVES, slots, cache, 4, 16)

    bad = dict(q=(a["q"][:3], "^q: needs at least 4 rows"), qo=(a["qo"][:, :7], "^q_out: shape"), k=(torch.zeros(4, 3, 64, device=device), "^k: shape"),
               v=(a["v"][:, :1], "^v: shape"), pos=(a["pos"][:3], "^positions: needs at least 4"), freq=(a["freq"][:31], "^inv_freq: needs at least 32"),
               slots=(a["slots"][:3], "^slots: needs at least 4"), cache=(a["cache"][:-1], "^cache: needs at least"))
    return call, a, bad, dict(q=(a["q"].half(), "^q: dtype"), qo=(a["qo"].half(), "^q_out: dtype"), k=(a["k"].half(), "^k: dtype"), v=(a["v"].half(), "^v: dtype"),
                              pos=(a["pos"].long(), "^positions: dtype"), freq=(a["freq"].double(), "^inv_freq: dtype"), slots=(a["slots"].int(), "^slots: dtype"))


CALLS = [product, many, experts, plan, combine, route, rotary]


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_sizes_and_types_of_host_tensors(make):
    call, args, sizes, types = make("cpu")
    with pytest.raises(ValueError, match=RIGHT):
        call(**args)
    refuse(call, args, **sizes)
    refuse(call, args, **types)


def spread(t):
    """The same values, every other element of a buffer twice as large."""
    return torch.stack([t, t], -1)[..., 0]


@pytest.mark.gpu
@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_device_tensors(make):
    """Right arguments are taken, and of one that is short, of another type, spread or on the host the call is refused
    before anything is launched."""
    call, args, sizes, types = make("cuda")
    call(**args)  # zeros: every product is zero, every token the first experts'
    torch.cuda.synchronize()
    for t in args.values():
        t.fill_(1)  # which no call would leave
    kept = {name: t.clone() for name, t in args.items()}
    refuse(call, args, **sizes)
    refuse(call, args, **types)
    strided = "contiguous|dense"
    refuse(call, args, **{name: (spread(t), strided) for name, t in args.items() if t.numel() > 1})
    refuse(call, args, **{name: (t.cpu(), RIGHT) for name, t in args.items()})
    torch.cuda.synchronize()
    assert all(torch.equal(t, kept[name]) for name, t in args.items())
