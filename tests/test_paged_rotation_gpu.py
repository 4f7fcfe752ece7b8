"""Rotation over part of a head: what does not turn does not mix."""
import math

import pytest
import torch

import dit_token_b200 as dit
from _paged import Batch, check_rotation, reference_rotation

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["interleaved", "half", "none"])
@pytest.mark.parametrize("d,rotary", [(64, 32), (128, 64), (128, 120), (256, 72)])
@pytest.mark.parametrize("what", ["row", "weight"])
def test_an_infinity_that_does_not_turn_stays_alone(mode, d, rotary, what):
    """y = x * rsqrt(mean(x^2) + eps) * w: an infinite element makes its head's
    factor 0, itself NaN and every other element of the head 0; a NaN among the
    weights is seen in its own elements only.  Elements behind ``rotary`` (all,
    without rotation) keep y, one by one."""
    x = Batch([9], [0], 2, 1, d, seed=d + rotary)
    first = 0 if mode == "none" else rotary
    freqs, gain = dit.dit_rope_frequencies(rotary)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    at = first + 3
    if what == "row":
        x.q[4, d + at] = math.inf
        x.k[5, at] = -math.inf
    else:
        w[at] = math.nan
    q_out, k_out = (torch.full((x.rows, h * d), 7.0, dtype=torch.bfloat16, device="cuda") for h in (2, 1))
    dit.dit_qk_rope_scaled(x.q, x.k, x.cs, x.cp, num_q_heads=2, num_k_heads=1, head_dim=d, q_out=q_out, k_out=k_out,
                           freqs=None if mode == "none" else freqs, q_weight=w, k_weight=w, rope_mode=mode)
    for t, out, heads in ((x.q, q_out, 2), (x.k, k_out, 1)):
        want, size = reference_rotation(t, x.chunks, x.first, heads, d, rotary=rotary, mode=mode, freqs=freqs, gain=1.0,
                                        starts=[0], weight=w)
        want, size, got = want[:9], size[:9], out[:9].view(9, heads, d)
        nan = want.isnan()
        assert bool(nan.any()) and torch.equal(got.isnan(), nan)
        check_rotation(torch.where(nan, 0, got), torch.where(nan, 0, want), torch.where(nan, 0, size), what)
