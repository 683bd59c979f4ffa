"""GPU test that starts of sequences outside of the rows, or that decrease, are recorded by dsa_expanded_attn, with nothing written outside
of what the call was given; the other sequences are right."""
import numpy as np
import pytest
import torch

from test_gpu_expanded import Packed, _i32, dsa  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu


def call(dsa, c, q_start, kv_start, guard=256):  # noqa: F811
    """Outputs with rows before and behind them that nobody may touch."""
    T, H = c.q.shape[:2]
    out = torch.full((T + 2 * guard, H, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 2 * guard, H), 6.0, device="cuda")
    mine = slice(guard, guard + T)
    dsa.dsa_expanded_attn(c.q, c.kv[..., :128], c.k_rope, c.kv[..., 128:], _i32(q_start), _i32(kv_start), sm_scale=192**-0.5, out=out[mine],
                          lse=lse[mine])
    err = dsa.dsa_get_device_error()
    for rows in (slice(0, guard), slice(guard + T, None)):
        assert bool((out[rows] == 5.0).all()) and bool((lse[rows] == 6.0).all())
    return out[mine], lse[mine], err


@pytest.mark.parametrize("H", [1, 16])
@pytest.mark.parametrize("q_start,kv_start", [
    ([0, 200, 600], [0, 300, 900]),      # queries behind the last row
    ([0, 200, 500], [0, 300, 1000]),     # positions behind the last row
    ([0, 200, 100], [0, 300, 900]),      # decreasing
    ([0, 200, 500], [0, 300, 200]),
])
def test_the_second_of_two_sequences(dsa, q_start, kv_start, H):  # noqa: F811
    c = Packed(1, [200, 300], [300, 600], H)
    out, lse, err = call(dsa, c, q_start, kv_start)
    assert err == 1
    c.new, c.lens = c.new[:1], c.lens[:1]
    c.check(out, lse)


@pytest.mark.parametrize("H", [1, 16])
@pytest.mark.parametrize("q_start,kv_start", [([-7, 200, 500], [0, 300, 900]), ([0, 200, 500], [-1, 300, 900])])
def test_a_negative_start(dsa, q_start, kv_start, H):  # noqa: F811
    c = Packed(2, [200, 300], [300, 600], H)
    out, lse, err = call(dsa, c, q_start, kv_start)
    assert err == 1
    c.new, c.lens, c.q_start, c.kv_start = c.new[1:], c.lens[1:], c.q_start[1:], c.kv_start[1:]
    c.check(out, lse)


@pytest.mark.parametrize("H", [1, 16])
def test_many_that_overlap(dsa, H):  # noqa: F811
    # more blocks than T rows of that many sequences can have
    c = Packed(3, [1000], [1200], H)
    _, _, err = call(dsa, c, np.array([0, 1000] * 40), np.array([0, 1200] * 40))
    assert err == 1


def test_starts_within_the_rows_are_not_recorded(dsa):  # noqa: F811
    c = Packed(4, [0, 200, 0, 300], [9, 300, 0, 600], 3, q_first=5, k_first=8, spare=3)
    out, lse, err = call(dsa, c, c.q_start, c.kv_start)
    assert err == 0
    c.check(out, lse)
