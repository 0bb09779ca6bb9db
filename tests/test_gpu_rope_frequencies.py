"""Frequencies set by hand, below zero among them, near both ends of the positions."""
import math
from fractions import Fraction

import pytest
import torch

import grouped_query_decode_gb300 as gq
import ragged_model as model

pytestmark = pytest.mark.gpu

TWO_PI = Fraction(62831853071795864769252867665590057683943387987502, 10 ** 49)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("t", [(1 << 31) - 1, -(1 << 31)])
@pytest.mark.parametrize("size", [3.1e-7, 1.3e-4, 0.02])
def test_angles_of_2_to_the_minus_22(size, t, sign):
    """Frequencies whose angle at t is nearly whole turns: the second of the pair (1, 0) becomes sin, a small
    number, of which bf16 holds the angle's error."""
    rope = gq.gqa_rope_init(64)
    angles = []
    for i in range(32):
        turns = round(size * (1 + i / 64) * abs(t) / (2 * math.pi))
        f = sign * float(turns * TWO_PI / abs(t))
        rope.inv_freq[i] = f
        x = Fraction(f) * t / TWO_PI
        angles.append(float((x - round(x)) * TWO_PI))
    assert max(abs(a) for a in angles) < 1e-4
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[..., :32] = 1
    out = torch.empty_like(q)
    gq.gqa_rope(rope, q, None, torch.tensor([t], dtype=torch.int32, device="cuda"), out, None)
    got, want = out.double().cpu()[0, 0], torch.tensor(angles, dtype=torch.float64)
    assert torch.equal(got[:32], torch.ones(32, dtype=torch.float64))
    assert ((got[32:] - torch.sin(want)).abs() <= 2.0 ** -22 + model.BF16_HALF * want.abs()).all()
