"""The cached decoding example: projections, append, attention, weights and
eviction together, against attention over the unquantized keys and values of
the tokens still cached.

Bound.  An E4M3 code is within 2^-4 of its value (relative, normal range), with
a root mean square of about 2^-4 / sqrt(3) / sqrt(2); keys of 128 dims put an
error of |q| |k| scale * 0.026 on a score of unit size, and values 0.026 on the
output, plus one more rounding of either where a page's scale grew or its
tokens moved.  0.1 covers the sum three times over; an output that misses a
token or takes a stale one is off by far more.
"""

import pytest

from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_gpu()


@pytest.mark.parametrize("batch,prompt,steps,dim,page", [(3, 100, 40, 128, 16), (2, 300, 20, 64, 64)])
def test_serving_matches_unquantized_attention(batch, prompt, steps, dim, page):
    from examples import cached_decode
    print(f"example batch={batch} prompt={prompt} steps={steps} dim={dim} page={page}", flush=True)
    _, err, lens = cached_decode.serve(batch, prompt, steps, hidden=256, q_heads=8, heads=2, dim=dim, page=page)
    assert max(lens) <= prompt + steps // 2 + 1
    assert err < 0.1, err
