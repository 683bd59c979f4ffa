"""GPU test that dsa_expanded_attn repeats to the bit where many blocks are equally long and some of them are cut into parts: which
ones are cut goes by their numbers."""
import pytest
import torch

from test_gpu_expanded import Packed, dsa  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu

CASES = [  # new, lens, heads, causal: blocks of 256 queries x heads, dealt to 152 CTAs
    ([40 * 256], [8192], 16, False),          # 640: 32 behind four rounds, cut four ways
    ([256] * 33, [4352] * 33, 16, True),      # 528: 72 behind three rounds, cut in two
    ([300] * 200, [4200] * 200, 2, False),    # 800: 40 behind five, blocks of 256 and of 44 queries
    ([40 * 256], [70000], 16, False),         # in stretches, lengths sorted by fours of tiles
]


@pytest.mark.parametrize("new,lens,H,causal", CASES)
def test_equally_long_blocks(dsa, new, lens, H, causal):  # noqa: F811
    c = Packed(len(new), new, lens, H)
    out, lse = c.call(dsa, causal=causal)
    junk = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    for k in range(24):
        with torch.cuda.stream(side):  # other work beside it, so that the warps of the plan run at other speeds
            junk[: 1 << (14 + k % 15)].fill_(k)
        again = c.call(dsa, causal=causal)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse), k
    torch.cuda.synchronize()
    # a few sequences against 64 bits
    keep = [0, len(new) // 2, len(new) - 1][: len(new)]
    keep = sorted(set(keep))
    if max(lens) <= 16384:
        c.q_start, c.kv_start, c.new, c.lens = c.q_start[keep], c.kv_start[keep], c.new[keep], c.lens[keep]
        c.check(out, lse, causal=causal)
