"""kda.qk_rope's angles, looked at where a cosine or sine is nearly nothing, so that a bf16 output shows them.

Tolerance. An output x cos t (its partner is 0) is off by its bf16 rounding, 2^-8 of it, by 2^-20 of it for the cosine and
the product in fp32, and by what the angle is off: for positions below 2^32 and frequencies up to 1 at most 2^-31 turns,
2 pi 2^-31 of x. The true cosine and sine come from integers: the position times the frequency's 24 bits times 1 / (2 pi) to
200 bits, the rest of the turn reduced to the nearest quarter before it is a float."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
BITS = 200


def _arctan_inverse(n, one):
    total = term = one // n
    k, sign = 1, -1
    while term:
        term //= n * n
        total += sign * (term // (2 * k + 1))
        k, sign = k + 1, -sign
    return total


ONE = 1 << (BITS + 20)
PI = 4 * (4 * _arctan_inverse(5, ONE) - _arctan_inverse(239, ONE))  # pi 2^220
TURNS = ONE * (1 << BITS) // (2 * PI)                              # 2^200 / (2 pi)


def cos_sin(position, f):
    """Cosine and sine of position f, and the distance of the angle from a multiple of a quarter in turns."""
    num, den = f.as_integer_ratio()
    t = position * num * TURNS // den % (1 << BITS)
    n = (t + (1 << (BITS - 3))) >> (BITS - 2)
    r = (t - (n << (BITS - 2))) / (1 << BITS)
    c, s = math.cos(2 * math.pi * r), math.sin(2 * math.pi * r)
    for _ in range(n % 4):
        c, s = -s, c
    return c, s, abs(r)


def near_quarters(f, start, count):
    """The positions of a range whose angles are nearest to multiples of a quarter, by their fractions of 2^-64 turns."""
    num, den = f.as_integer_ratio()
    step = (num * TURNS // den >> (BITS - 64)) % (1 << 64)
    at = np.arange(start, start + (1 << 20), dtype=np.int64)
    t = at.view(np.uint64) * np.uint64(step) << np.uint64(2)  # of a quarter
    away = np.minimum(t, np.uint64(0) - t)
    return at[np.argsort(away, kind="stable")[:count]].tolist()


@pytest.mark.parametrize("start", [0, 100000, (1 << 31) - (1 << 20), (1 << 32) - (1 << 20), -(1 << 20)])
@pytest.mark.parametrize("i", [0, 3, 17])
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_rope_angles_near_quarter_turns(start, i, interleaved):
    import gated_linear_attention_kda_gb300 as kda
    f = float(torch.tensor(500000.0 ** (-2 * i / 64), dtype=torch.float32))
    positions = near_quarters(f, start, 32)
    q = torch.zeros(32, 2, 64, dtype=BF16, device="cuda")
    first, second = (0, 1) if interleaved else (0, 8)
    q[:, 0, first], q[:, 1, second] = 1.0, 1.0
    out = torch.empty_like(q)
    freq = torch.zeros(8, device="cuda")
    freq[0] = f
    kda.qk_rope(q, None, out, None, torch.tensor(positions, device="cuda"), freq, norm=False, interleaved=interleaved)
    kda.check_device_status()
    out = out.double().cpu()
    for row, p in enumerate(positions):
        c, s, _ = cos_sin(p, f)
        for head, ch, want in ((0, first, c), (0, second, s), (1, first, -s), (1, second, c)):
            got = float(out[row, head, ch])
            assert abs(got - want) <= (2.0 ** -8 + 2.0 ** -20) * abs(want) + 2 * math.pi * 2.0 ** -31, (p, head, ch, got, want)
