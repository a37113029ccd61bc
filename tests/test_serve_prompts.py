"""The attention kernel for many new tokens: its forms, padded batches, and sizes that only it meets, against the 64-bit
reference."""
import pytest

from test_serve_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,news", [([700], [40]), ([300, 900], [64, 17]), ([400, 20], [300, 5])])
def test_a_padded_batch(D, lens, news):
    # a captured step's rows: many more than its requests may bring, which choose neither the tiles' size nor the parts'
    Case(40 + D, "bf16", D, 16, 32, 8, lens, news, extra=4200 - sum(news)).check(f"padded D={D} {news}")
