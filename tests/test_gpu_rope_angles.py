"""Angles of dsa_rope far from the usual ones: positions times frequencies that are tiny, or frequencies well above one.

The reference takes pos * inv_freq (both exact) modulo 2 pi in integers, with 2 pi to 120 digits.

Tolerances.  The phase is a 64-bit fraction of a turn: off by 2^-64 turns of the frequency times the position, at most
2^-33 turns, which is 2^-30 rad; its conversion to fp32 and sincospif are off by 2^-24 and 2^-22 of their value or, near a
zero other than at angle 0, of 1.  The output is a fused multiply-add and a product in fp32 (2^-23 of |x0| + |x1|), then
rounded to bf16 (2^-8 of it).  With x = (1, 0), y1 = sin(theta): for tiny angles 2^-8 + 2^-21 of it is all."""
import decimal

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_sparse_attention_gb300 import build

    build.build()
    import top_sparse_attention_gb300 as m

    torch.cuda.set_device(0)
    yield m
    torch.cuda.synchronize()
    assert m.dsa_get_device_error() == 0


def _two_pi():
    """2 pi to 120 digits, by Machin's formula in integers."""
    one = 10 ** 130

    def arctan_inv(n):
        total, term, k, sign = 0, one // n, 1, 1
        while term:
            total += sign * (term // k)
            term //= n * n
            k += 2
            sign = -sign
        return total

    return decimal.Decimal(2 * 4 * (4 * arctan_inv(5) - arctan_inv(239))).scaleb(-130)


def _angles(pos, f):
    """pos[i] * f modulo 2 pi, in (-pi, pi], for each pos and the fp32 value f."""
    with decimal.localcontext() as ctx:
        ctx.prec = 120
        two_pi, f = _two_pi(), decimal.Decimal(float(f))
        out = []
        for p in pos:
            a = decimal.Decimal(int(p)) * f
            out.append(float(a - (a / two_pi).to_integral_value() * two_pi))
    return np.array(out)


def _turn(dsa, pos, f, style, inverse):
    """y of x = (1, 0) and of x = (0, 1) in 16 pairs of the same frequency."""
    n = len(pos)
    x = torch.zeros(n, 2, 32, dtype=torch.bfloat16)
    x[:, 0, :16 if style == "half" else None:1 if style == "half" else 2] = 1
    x[:, 1] = 1 - x[:, 0]
    y = dsa.dsa_rope(x.cuda(), torch.tensor(pos, dtype=torch.int64).to(torch.int32).cuda(), torch.full((16,), float(f), device="cuda"),
                     style=style, inverse=inverse).double().cpu().numpy()
    y = y.reshape(n, 2, 2, 16) if style == "half" else y.reshape(n, 2, 16, 2).swapaxes(2, 3)
    assert np.all(y == y[..., :1])  # every pair alike
    return y[..., 0]


@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("f", [1e-4, 1e-6, 1e-7, 1e-8, 1e-10])
def test_small_angles_keep_their_digits(dsa, f, inverse, style):
    pos = [1, 2, 3, 5, 17, 100, -1, -2, -100, 4096]
    f = np.float32(f)
    theta = np.array(pos) * float(f) * (-1 if inverse else 1)
    y = _turn(dsa, pos, f, style, inverse)
    tol = (2.0**-8 + 2.0**-21) * np.abs(np.sin(theta))
    assert np.all(np.abs(y[:, 0, 1] - np.sin(theta)) <= tol)
    assert np.all(np.abs(y[:, 1, 0] + np.sin(theta)) <= tol)
    assert np.all(np.abs(y[:, 0, 0] - np.cos(theta)) <= 2.0**-8)


@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("f", [0.0, 0.75, 1.0, 3.0, 1000.0, 12345.678, 2.0**20 + 1, 3.0e9, 2.0**40, -1.0, -777.7])
def test_frequencies_above_one(dsa, f, style):
    pos = [0, 1, -1, 7, 4097, -65535, (1 << 20) + 3, (1 << 24) - 1, 1 << 24, (1 << 31) - 1, -(1 << 31), -(1 << 31) + 5]
    f = np.float32(f)
    theta = _angles(pos, f)
    for inverse in (False, True):
        y = _turn(dsa, pos, f, style, inverse)
        sin, cos = np.sin(-theta if inverse else theta), np.cos(theta)
        for got, want in ((y[:, 0, 0], cos), (y[:, 0, 1], sin), (y[:, 1, 0], -sin), (y[:, 1, 1], cos)):
            assert np.all(np.abs(got - want) <= 2.0**-8 * np.abs(want) + 2.0**-21)


@pytest.mark.parametrize("f", [1e-8, 1e-6, 1.0, 12345.678, 2.0**20 + 1])
@pytest.mark.parametrize("rows", [3, 40000])
def test_the_append_turns_by_the_same_angles(dsa, f, rows):
    # every form of the append (few rows, many rows, any alignment) against dsa_rope, bit for bit, in bf16; the latent row
    rng = np.random.default_rng(rows)
    x = torch.from_numpy(rng.standard_normal((rows, 576))).bfloat16().cuda()
    pos = torch.from_numpy(rng.integers(-(1 << 31), 1 << 31, rows)).to(torch.int32).cuda()
    pos[:3] = torch.tensor([1, -2, 3])
    freq = torch.full((32,), float(np.float32(f)), device="cuda")
    want = dsa.dsa_rope(x, pos, freq, rot_off=512)
    cache = torch.zeros(rows, 576, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_rope_append(x, pos, freq, cache, rot_off=512)
    assert torch.equal(cache, want)
    odd = torch.zeros(rows, 577, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_rope_append(x, pos, freq, odd[:, 1:], rot_off=512)
    assert torch.equal(odd[:, 1:], want)
