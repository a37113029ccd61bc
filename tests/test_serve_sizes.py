"""Sizes at the entry points' limits, on the host: what is refused, and what is not."""
import pytest

import bit_quantized_matvec_q1_amd.lowbit as L
from test_serve_abi import attn, plan

WS = L.lowbit_kv_attention_workspace


@pytest.mark.parametrize("T,hq,hk", [(131072, 64, 8), (262144, 32, 8), (65536, 128, 8), (131072, 64, 64), ((1 << 20) + 1, 64, 8)])
def test_long_prompts_are_not_refused(T, hq, hk):
    # 2^23 query rows and more: some 2^16 to 2^22 tiles of any row type, none of them split
    assert WS(T, 1, hq, hk, 128, T, T) == 0
    for dtype in (L.F32, L.BF16, L.F16):  # the sizes pass: the missing pointer is what is left to say
        assert attn(dtype=dtype, T=T, B=1, hq=hq, hk=hk, max_q=T, max_kv=T, qs=hq * 128, os=hq * 128, q=None) == L.LB_EINVAL


def test_the_largest_steps():
    # T * 16 rows: a tile for every 16 of fp32 (T tiles and one), for every 256 of the others; then 2^31 rows
    size = dict(B=1, hq=16, hk=1, qs=2048, os=2048, q=None, max_kv=1 << 24)
    for T, f32, f16 in (((1 << 23) - 2, L.LB_EINVAL, L.LB_EINVAL), ((1 << 23) - 1, L.LB_ESHAPE, L.LB_EINVAL),
                        ((1 << 27) - 17, L.LB_ESHAPE, L.LB_EINVAL), ((1 << 27) - 16, L.LB_ESHAPE, L.LB_ESHAPE), (1 << 27, L.LB_ESHAPE, L.LB_ESHAPE)):
        assert attn(dtype=L.F32, T=T, max_q=T, **size) == f32, T
        assert attn(dtype=L.F16, T=T, max_q=T, **size) == f16, T
        assert attn(dtype=L.BF16, T=T, max_q=T, **size) == f16, T
        assert WS(T, 1, 16, 1, 128, T, 1 << 24) == (-1 if f16 == L.LB_ESHAPE else 0)
    # many requests of a token: a tile each, whatever the type
    for B, want in (((1 << 23) - 1, L.LB_EINVAL), (1 << 23, L.LB_ESHAPE)):
        for dtype in (L.F32, L.F16):
            assert attn(dtype=dtype, T=B, B=B, hq=1, hk=1, max_q=1, q=None) == want
        assert WS(B, B, 1, 1, 128, 1, 64) == (0 if want == L.LB_EINVAL else -1)
    # few tiles in many parts
    assert WS(64, 64, 8, 8, 128, 1, 1 << 24) > 0 and WS(64, 64, 8, 8, 128, 1, (1 << 31) - (1 << 13)) == -1


def test_what_a_type_cannot_take_does_not_refuse_the_others():
    # 8 requests of 65 rows after 2^27 tokens: fp32 in 320 tiles of 16 rows and parts of some 2000 tokens (2^24 of
    # them), the others in 64 tiles of 128 rows and 12 parts
    size = dict(T=520, B=8, hq=8, hk=8, max_q=65, max_kv=1 << 27, qs=1024, os=1024, q=None)
    assert WS(520, 8, 8, 8, 128, 65, 1 << 27) == 64 * 12 * (128 * 128 + 256) * 4
    assert attn(dtype=L.F32, **size) == L.LB_ESHAPE and attn(dtype=L.BF16, **size) == L.LB_EINVAL


def test_the_most_requests_of_a_plan():
    # beyond 2^30 the sum of two request numbers passes 31 bits in the kernels' bisection
    assert plan(B=(1 << 30) + 1, new=None) == plan(B=(1 << 31) - 1, new=None) == L.LB_ESHAPE
    assert plan(B=1 << 30, new=None) == L.LB_EINVAL


def test_cache_bytes_of_pages_that_nothing_takes():
    # 2^31 pages of 65536 heads' records would pass 2^63; a page of 2^32 bytes is refused by every entry point
    assert L.lowbit_kv_cache_bytes((1 << 31) - 1, 65536, 1024, 256) == -1
    assert L.lowbit_kv_cache_bytes(1, 65536, 1024, 256) == -1
    assert L.lowbit_kv_cache_bytes((1 << 31) - 1, 65536, 16, 256) == ((1 << 31) - 1) * 65536 * 16 * 288
    assert L.lowbit_kv_cache_bytes(1, 65536, 512, 64) == 65536 * 512 * 72
