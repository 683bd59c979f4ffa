"""GPU test of dsa_latent_expand where a pair of CTAs goes from a whole tile of 256 rows to one that the sequences fill in part: the
copies of the whole tile's last columns leave while the rest is read out, and what either holds has to be what it is in a call whose
rows fill every tile (the same products in the same order: equal bits)."""
import pytest
import torch

from test_gpu_expanded import FORMATS, Rows, dsa, weights  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("tiles,H", [
    (77, 16),   # a unit of the last whole tile before the partial one, units of 256 columns
    (144, 16),  # fifteen of them
    (4, 28),    # units of 128 columns, three before it
])
@pytest.mark.parametrize("rest", [1, 31, 33, 100, 129, 255])
def test_whole_tiles_before_a_partial_one(dsa, kv, tiles, H, rest):  # noqa: F811
    rows, whole = 256 * tiles + rest, 256 * (tiles + 1)
    r, w = Rows(tiles + rest, [whole], kv, 64), weights(H, rest)
    want, want_rope = r.call(dsa, w, [0, whole], rows=whole)
    last = Rows.__new__(Rows)  # the values of the last 512 rows against 64 bits
    last.kv_kind, last.val, last.at = kv, r.val[r.at()[whole - 512:]], lambda: slice(None)
    last.check(want[whole - 512:], want_rope[whole - 512:], w)
    for _ in range(6):
        out = torch.full((whole, H, 256), 3.0, dtype=torch.bfloat16, device="cuda")
        rope = torch.full((whole, 64), 4.0, dtype=torch.bfloat16, device="cuda")
        r.call(dsa, w, [0, rows], out=out, rope_out=rope)
        assert torch.equal(out[:rows], want[:rows]) and torch.equal(rope[:rows], want_rope[:rows])
        assert bool((out[rows:] == 3.0).all()) and bool((rope[rows:] == 4.0).all())


@pytest.mark.parametrize("kv", FORMATS)
def test_rows_before_the_first_sequence(dsa, kv):  # noqa: F811
    # the same at the other end: partial tiles first, then whole ones
    whole, first = 256 * 80, 300
    r, w = Rows(5, [whole], kv), weights(16)
    want, want_rope = r.call(dsa, w, [0, whole], rows=whole)
    for _ in range(6):
        out = torch.full((first + whole, 16, 256), 3.0, dtype=torch.bfloat16, device="cuda")
        rope = torch.full((first + whole, 64), 4.0, dtype=torch.bfloat16, device="cuda")
        r.call(dsa, w, [first, first + whole], out=out, rope_out=rope)
        assert torch.equal(out[first:], want) and torch.equal(rope[first:], want_rope)
        assert bool((out[:first] == 3.0).all()) and bool((rope[:first] == 4.0).all())
