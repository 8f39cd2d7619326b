"""Gradient norm and clipping where the rounding of the sums is one-sided, and
where the quotient max_norm / (norm + eps) has no value.

Tolerance of the norm, fixed before the first run: a thread adds up to 64
squares (and single elements at the ends) in two fp32 chains of at most 33
additions, each rounded by 2^-24 of a partial sum that is on average half
of the whole, and joins them: 17.5 * 2^-24 of the sum of squares; fp64 from
there on.  The root halves it, and fp32 rounds it once: 10 * 2^-24.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CHAIN = 10 * 2.0 ** -24


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("value", [1.0, 1.1, 0.7, 1.9, 1.3333])
@pytest.mark.parametrize("n", [64 * 256, 300_001])
def test_norm_of_equal_values(fg, kind, value, n):
    t = torch.full((n,), value, device="cuda").to(kind)
    want = math.sqrt(n) * float(t[0].double())
    assert abs(float(fg.grad_norm([t])) - want) <= CHAIN * want


def clipped(fg, values, max_norm, eps):
    t = torch.tensor(values, device="cuda")
    out = torch.full_like(t, 7.0)
    norm = fg.clip_grad_norm([t], max_norm, out=[out], eps=eps)
    again = t.clone()
    fg.clip_grad_norm([again], max_norm, eps=eps)
    assert torch.equal(again.nan_to_num(9.0), out.nan_to_num(9.0))
    return float(norm), out.tolist()


def test_nothing_to_clip_stays_zero(fg):
    for max_norm in (0.0, 1.0, math.inf):
        for eps in (0.0, 1e-6):
            assert clipped(fg, [0.0] * 40, max_norm, eps) == (0.0, [0.0] * 40)


def test_an_infinite_norm_scales_by_zero(fg):
    for max_norm in (0.0, 1.0, math.inf):
        norm, out = clipped(fg, [math.inf] + [1.0] * 40, max_norm, 1e-6)
        assert norm == math.inf and out[1:] == [0.0] * 40 and math.isnan(out[0])


def test_no_bound(fg):
    assert clipped(fg, [3.0, 4.0], math.inf, 1e-6) == (5.0, [3.0, 4.0])
    norm, out = clipped(fg, [3.0, math.nan], math.inf, 1e-6)
    assert math.isnan(norm) and all(map(math.isnan, out))
