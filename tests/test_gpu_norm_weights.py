"""GPU test that weights and biases may lie at any 4-byte address (slices of a packed parameter) without changing what a call gives:
the same form of the kernel takes them, to the same bits."""
import pytest
import torch

from test_gpu_norm_rope import Case, check_bf16, check_rows, dsa, pools  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu


def shifted(t, by):
    """The same numbers, `by` floats behind a 16-byte boundary."""
    if t is None:
        return None
    packed = torch.full((len(t) + 8,), float("nan"), device="cuda")
    out = packed[by:by + len(t)]
    out.copy_(t)
    assert out.data_ptr() % 16 == 4 * by
    return out


@pytest.mark.parametrize("by", [1, 2, 3])
@pytest.mark.parametrize("norm,bias", [("rms", False), ("layer", True)])
@pytest.mark.parametrize("rows,heads,width,nd,ro", [(2000, 16, 192, 192, 128), (700, 3, 64, 64, 0), (300, 2, 576, 512, 512), (40, 1, 1024, 1024, 0)])
def test_heads(dsa, rows, heads, width, nd, ro, norm, bias, by):  # noqa: F811
    c = Case(width + by, rows, heads, width, norm, 0, nd, ro, 64, bias=bias)
    want = dsa.dsa_norm_rope(c.x, c.pos, c.freq, **c.kw)
    check_bf16(want, *c.want())
    c.kw.update(weight=shifted(c.w, by), bias=shifted(c.b, by))
    assert torch.equal(dsa.dsa_norm_rope(c.x, c.pos, c.freq, **c.kw), want)


@pytest.mark.parametrize("by", [1, 2, 3])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "t128", "mx"])
@pytest.mark.parametrize("rows", [129, 9000])
def test_rows_into_a_cache(dsa, kind, rows, by):  # noqa: F811
    c = Case(rows + by, rows, 1, 576, "rms", 0, 512, 512, 64)
    kv, scale = pools(kind, rows, 576)
    dsa.dsa_norm_rope_append(c.x[:, 0], c.pos, c.freq, kv, scale=scale, **c.kw)
    want, err = c.want()
    check_rows(kind, kv, scale, want[:, 0], err[:, 0])
    c.kw.update(weight=shifted(c.w, by))
    kv2, scale2 = pools(kind, rows, 576)
    dsa.dsa_norm_rope_append(c.x[:, 0], c.pos, c.freq, kv2, scale=scale2, **c.kw)
    assert torch.equal(kv2, kv) and (scale is None or torch.equal(scale2, scale))
