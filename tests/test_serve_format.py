"""The cache's format: rows that it holds already keep their values."""
import pytest
import torch

import bit_quantized_matvec_q1_amd.lowbit as L
import serve_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_read_back_and_appended_again(D):
    """Scales from 2^-14 (the least normal binary16) to its largest, saturated ones among them; a block's largest value
    is 6 times its scale then, and 6 d * fp32(1/6) is within 2^-23 of d, which rounds to d."""
    say(f"case again D={D}")
    T, H, P = 300, 3, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    pages = 2 * -(-T // P)
    cache = torch.zeros(pages, H, R.record_bytes(P, D), dtype=torch.uint8, device="cuda")
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:2 * T]
    k, v = (torch.randn(T, H, D, generator=g, device="cuda") * torch.exp2(torch.rand(T, H, D // 32, 1, generator=g, device="cuda") * 30 - 11)
            .expand(T, H, D // 32, 32).reshape(T, H, D) for _ in range(2))
    rows = [k, v]
    for at in (slots[:T].contiguous(), slots[T:].contiguous()):
        L.lowbit_kv_append(L.F32, *rows, T, H, D, at, cache, pages, P)
        out = [torch.empty(T, H, D, device="cuda") for _ in range(2)]
        L.lowbit_kv_read(L.F32, cache, pages, P, T, H, D, at, *out)
        if rows[0] is not k:
            assert torch.equal(out[0], rows[0]) and torch.equal(out[1], rows[1])
        rows = out
    assert float(rows[0].abs().max()) == 6 * 65504 and float(rows[1].abs().max()) == 6 * 65504
