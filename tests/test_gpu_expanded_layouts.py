"""GPU test of dsa_expanded_attn at the largest number of heads and over keys and values whose rows and heads lie apart."""
import pytest
import torch

from test_gpu_expanded import Packed, dsa  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H", [127, 128])
@pytest.mark.parametrize("new,lens", [([1, 300], [1, 520]), ([700, 0, 3], [900, 40, 2000])])
def test_as_many_heads_as_there_may_be(dsa, new, lens, H, causal):  # noqa: F811
    c = Packed(H, new, lens, H)
    out, lse = c.call(dsa, causal=causal)
    some = [0, 1, 63, H - 2, H - 1]
    c.q, c.kv, c.H = c.q[:, some], c.kv[:, some], len(some)
    c.check(out[:, some], lse[:, some], causal=causal)


@pytest.mark.parametrize("pad", [8, 24, 136])
def test_heads_and_rows_apart(dsa, pad):  # noqa: F811
    c = Packed(pad, [150, 20], [400, 20], 3)
    want = c.call(dsa)
    apart = torch.full((c.kv.shape[0] + 1, 4, 256 + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    apart[1:, 1:, :256] = c.kv
    c.kv = apart[1:, 1:, :256]
    got = c.call(dsa)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
