"""GPU parity of dsa_norm_rope and dsa_norm_rope_append with the formula in 64 bits.

Tolerances, per element.  With M_c = |w_c| (|x_c| + |mean|) r + |b_c| (the terms that make up a normed value; |x_c| for a
column that is not normed):
 * the sums of n squares, the mean and the products are fp32: a relative error of at most (n + 16) 2^-24 of M_c;
 * a turned column is cos or sin times two of those, the sines off by 2^-22 (an angle right to fp32 and sincospif's ulps);
 * bf16 is off by 2^-8 of the value; E4M3 by 2^-4 of it, or by half of its smallest step, 2^-10 of the scale (448 codes
   a scale's largest value, so the scale itself, and the quotient, are off by as much as the values and 2^-23)."""
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


class Case:
    def __init__(self, seed, rows, heads, width, norm="rms", norm_off=0, norm_dim=None, rot_off=0, rot=64, style="half", weight=True, bias=False,
                 axes=1, eps=1e-6, offset=0.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        norm_dim = width - norm_off if norm_dim is None else norm_dim
        self.x = ((torch.randn(rows, heads, width, generator=g) + offset) * torch.exp(torch.randn(rows, heads, 1, generator=g))).bfloat16().cuda()
        self.w = (1 + 0.3 * torch.randn(norm_dim, generator=g)).cuda() if weight else None
        self.b = (0.3 * torch.randn(norm_dim, generator=g)).cuda() if bias else None
        pos = rng.integers(0, 1 << 20, (rows, axes)).astype(np.int32)
        self.pos = torch.from_numpy(pos).cuda()
        self.freq = torch.from_numpy((10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)).cuda()
        self.axis = bytes(int(a) for a in rng.integers(0, axes, rot // 2)) if axes > 1 else None
        self.kw = dict(norm=norm, weight=self.w, bias=self.b, eps=eps, norm_off=norm_off, norm_dim=norm_dim, rot_off=rot_off, rot_dim=rot,
                       style=style, pair_axis=self.axis)

    def want(self):
        """(values, bound on the error before the last rounding), fp64 [rows, heads, width]."""
        k = self.kw
        x = self.x.double().cpu().numpy()
        a, n = k["norm_off"], k["norm_dim"]
        part = x[..., a:a + n]
        mean = part.mean(-1, keepdims=True) if k["norm"] == "layer" else np.zeros(part.shape[:-1] + (1,))
        r = 1.0 / np.sqrt(((part - mean) ** 2).mean(-1, keepdims=True) + k["eps"])
        w = 1.0 if self.w is None else self.w.double().cpu().numpy()
        b = 0.0 if self.b is None else self.b.double().cpu().numpy()
        y, mag = x.copy(), np.abs(x)
        y[..., a:a + n] = (part - mean) * r * w + b
        mag[..., a:a + n] = np.abs(w) * (np.abs(part) + np.abs(mean)) * r + np.abs(b)
        err = (n + 16) * 2.0**-24 * mag
        p, off = k["rot_dim"] // 2, k["rot_off"]
        axis = np.zeros(p, int) if self.axis is None else np.frombuffer(self.axis, np.uint8).astype(int)
        theta = self.pos.double().cpu().numpy()[:, axis] * self.freq.double().cpu().numpy()
        cos, sin = np.cos(theta)[:, None], np.sin(theta)[:, None]
        c0 = off + (np.arange(p) if k["style"] == "half" else 2 * np.arange(p))
        c1 = c0 + (p if k["style"] == "half" else 1)
        y0, y1, e = y[..., c0].copy(), y[..., c1].copy(), err[..., c0] + err[..., c1] + 2.0**-21 * (mag[..., c0] + mag[..., c1])
        y[..., c0], y[..., c1] = y0 * cos - y1 * sin, y1 * cos + y0 * sin
        err[..., c0] = err[..., c1] = e
        return y, err


def check_bf16(got, want, err):
    got = got.double().cpu().numpy()
    tol = 2.0**-8 * np.abs(want) + 1.01 * err
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


SHAPES = [  # rows, heads, width, norm_off, norm_dim, rot_off, rot
    (1, 1, 64, 0, 64, 0, 64), (5, 3, 64, 0, 64, 32, 32), (3, 64, 128, 0, 128, 0, 64), (130, 17, 128, 0, 128, 64, 64), (7, 16, 192, 0, 192, 128, 64),
    (33, 5, 256, 0, 256, 0, 256), (9, 2, 576, 0, 512, 512, 64), (301, 1, 576, 0, 512, 512, 64), (2, 3, 1024, 512, 512, 0, 128), (65, 1, 128, 0, 128, 0, 64),
    (11, 1, 48, 16, 32, 0, 16),
    # not whole 16-byte chunks: any column, any number of pairs
    (4, 3, 100, 3, 77, 5, 62), (3, 2, 63, 0, 63, 1, 2), (2, 1, 1023, 1, 1000, 700, 254), (6, 2, 72, 0, 72, 0, 40),
]


@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("shape", SHAPES)
def test_heads(dsa, shape, norm, style):
    rows, heads, width, no, nd, ro, rd = shape
    c = Case(width + rows, rows, heads, width, norm, no, nd, ro, rd, style, bias=norm == "layer", offset=1.0 if norm == "layer" else 0.0)
    check_bf16(dsa.dsa_norm_rope(c.x, c.pos, c.freq, **c.kw), *c.want())


@pytest.mark.parametrize("rows,width,nd,ro,rd", [
    (65, 128, 128, 0, 128), (2500, 128, 128, 0, 128), (3, 64, 64, 0, 64), (40, 256, 256, 0, 256), (70, 192, 192, 48, 96), (61, 128, 128, 56, 72),
    (2600, 576, 512, 320, 256), (2600, 576, 512, 448, 128), (2600, 576, 512, 440, 136), (5, 640, 640, 0, 256),
])
@pytest.mark.parametrize("style", ["half", "pairs"])
def test_one_head_that_turns_many_columns(dsa, rows, width, nd, ro, rd, style):
    # rows whose pairs are more than a table of turns holds for several rows of a warp
    c = Case(rows + rd, rows, 1, width, "rms", 0, nd, ro, rd, style)
    check_bf16(dsa.dsa_norm_rope(c.x, c.pos, c.freq, **c.kw), *c.want())
    want, err = c.want()
    for kind in ("fp8", "t128", "mx"):
        kv, scale = pools(kind, rows, width)
        dsa.dsa_norm_rope_append(c.x[:, 0], c.pos, c.freq, kv, scale=scale, **c.kw)
        check_rows(kind, kv, scale, want[:, 0], err[:, 0])


@pytest.mark.parametrize("weight,bias", [(False, False), (True, True), (False, True)])
@pytest.mark.parametrize("axes", [1, 3])
def test_without_weights_and_with_axes(dsa, weight, bias, axes):
    c = Case(3, 40, 4, 128, weight=weight, bias=bias, axes=axes)
    check_bf16(dsa.dsa_norm_rope(c.x, c.pos, c.freq, **c.kw), *c.want())


@pytest.mark.parametrize("width,rot_off", [(192, 128), (100, 36)])
def test_strides_in_place_and_wider_outputs(dsa, width, rot_off):
    c = Case(4, 50, 6, width, rot_off=rot_off)
    want, err = c.want()
    wide = torch.full((50, 9, width + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    view = wide[:, 1:7, 8:8 + width]
    view.copy_(c.x)
    out = torch.full((50, 7, 2 * width), 3.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_norm_rope(view, c.pos, c.freq, out=out[:, :6, width:], **c.kw)
    check_bf16(out[:, :6, width:], want, err)
    assert bool((out[:, 6] == 3.0).all()) and bool((out[:, :6, :width] == 3.0).all())
    dsa.dsa_norm_rope(view, c.pos, c.freq, out=view, **c.kw)  # in place
    check_bf16(view, want, err)
    keep = torch.ones_like(wide, dtype=torch.bool)
    keep[:, 1:7, 8:8 + width] = False
    assert bool((wide[keep] == 7.0).all())
    rows = Case(5, 33, 1, width, rot_off=rot_off)  # [rows, width], rows apart
    x = torch.zeros(33, width + 24, dtype=torch.bfloat16, device="cuda")[:, :width]
    x.copy_(rows.x[:, 0])
    check_bf16(dsa.dsa_norm_rope(x, rows.pos[:, 0], rows.freq, **rows.kw)[:, None], *rows.want())


def test_small_and_large_values(dsa):
    c = Case(6, 64, 4, 128, eps=1e-5)
    c.x = (c.x.double() * torch.ldexp(torch.ones(64, 4, 1), torch.arange(256).view(64, 4, 1) // 4 - 40).double().cuda()).bfloat16()
    c.x[3, 2] = 0.0  # eps keeps a vector of zeros
    check_bf16(dsa.dsa_norm_rope(c.x, c.pos, c.freq, **c.kw), *c.want())


def pools(kind, count, width):
    if kind == "bf16":
        return torch.full((count, width), 5.0, dtype=torch.bfloat16, device="cuda"), None
    kv = torch.full((count, width), 9, dtype=torch.uint8, device="cuda")
    if kind == "mx":
        return kv, torch.full((count, width // 32), 11, dtype=torch.uint8, device="cuda")
    return kv, torch.full((count,) if kind == "fp8" else (count, -(-width // 128)), 2.0, device="cuda")


def check_rows(kind, kv, scale, want, err):
    if len(want) == 0:
        return
    if kind == "bf16":
        check_bf16(kv, want, err)
        return
    code = kv.view(torch.float8_e4m3fn).double().cpu().numpy()
    width = want.shape[-1]
    if kind == "mx":
        s = np.repeat(np.ldexp(1.0, scale.cpu().numpy().astype(int) - 127), 32, -1)
        top = np.abs(want).reshape(len(want), -1, 32)
        limit = np.repeat(np.where(top.max(-1) > 0, np.exp2(np.floor(np.log2(np.maximum(top.max(-1), 1e-300))) - 8), 1.0), 32, -1)
        slack = np.repeat(err.reshape(top.shape).max(-1) / np.maximum(top.max(-1), 1e-300), 32, -1)
        # the exponent is that of the largest value, which may round over a power of two
        ok = (s == limit) | ((slack > 0) & ((s == 2 * limit) | (2 * s == limit)))
        assert np.all(ok)
        sat = np.abs(want) >= 448 * s  # saturated: the largest codes stand for all that is above them
        assert np.all(np.abs(code[sat]) == 448)
        tol = np.where(sat, np.inf, 2.0**-4 * np.abs(want) + 2.0**-10 * s + 2 * err)
    else:
        tile = width if kind == "fp8" else 128
        s = np.repeat(scale.double().cpu().numpy().reshape(len(want), -(-width // tile)), tile, -1)[:, :width]
        for lo in range(0, width, tile):
            top, e = np.abs(want[:, lo:lo + tile]).max(-1), err[:, lo:lo + tile].max(-1)
            assert np.all(np.abs(s[:, lo] - np.where(top > 0, top / 448, 1.0)) <= 2.0**-23 * top + e / 448 + 1e-38)
            err = err.copy()
            err[:, lo:lo + tile] += (e / np.maximum(top, 1e-300) + 2.0**-22)[:, None] * np.abs(want[:, lo:lo + tile])
        tol = 2.0**-4 * np.abs(want) + 2.0**-10 * s + 2 * err
    assert np.all(np.abs(code * s - want) <= tol), np.max(np.abs(code * s - want) / tol)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "t128", "mx"])
@pytest.mark.parametrize("rows,width,norm,no,nd,ro,rd,style", [
    (1, 576, "rms", 0, 512, 512, 64, "half"), (129, 576, "rms", 0, 512, 512, 64, "pairs"), (2600, 576, "rms", 0, 512, 512, 64, "half"),
    (77, 128, "layer", 0, 128, 0, 64, "half"), (2501, 64, "layer", 0, 64, 0, 64, "pairs"), (30, 1024, "rms", 0, 1024, 0, 256, "half"),
    (12, 96, "rms", 5, 80, 3, 60, "half"), (12, 992, "layer", 1, 991, 100, 254, "pairs"),
])
def test_rows_into_a_cache(dsa, kind, rows, width, norm, no, nd, ro, rd, style):
    c = Case(rows, rows, 1, width, norm, no, nd, ro, rd, style, bias=norm == "layer")
    want, err = c.want()
    want, err = want[:, 0], err[:, 0]
    count = rows + 40
    dst = np.random.default_rng(rows).permutation(count)[:rows].astype(np.int64)
    dst[::7] = -1
    kv, scale = pools(kind, count, width)
    before = kv.clone(), None if scale is None else scale.clone()
    dsa.dsa_norm_rope_append(c.x[:, 0], c.pos, c.freq, kv, scale=scale, dst_rows=torch.from_numpy(dst).cuda(), **c.kw)
    live = dst >= 0
    at = torch.from_numpy(dst[live]).cuda()
    check_rows(kind, kv[at], None if scale is None else scale[at], want[live], err[live])
    rest = torch.from_numpy(np.setdiff1d(np.arange(count), dst[live])).cuda()
    assert torch.equal(kv[rest], before[0][rest]) and (scale is None or torch.equal(scale[rest], before[1][rest]))
    kv, scale = pools(kind, count, width)  # without a list: row r
    dsa.dsa_norm_rope_append(c.x[:, 0], c.pos, c.freq, kv, scale=scale, **c.kw)
    check_rows(kind, kv[:rows], None if scale is None else scale[:rows], want, err)


@pytest.mark.parametrize("width", [576, 100])
def test_rows_past_the_pool_are_dropped_and_recorded(dsa, width):
    c = Case(8, 9, 1, width, rot_off=0)
    kv, _ = pools("bf16", 6, width)
    dst = torch.tensor([0, 6, 5, 1 << 40, -3, 1, 2, 7, 3], device="cuda")
    dsa.dsa_norm_rope_append(c.x[:, 0], c.pos, c.freq, kv, dst_rows=dst, **c.kw)
    assert dsa.dsa_get_device_error() == 1
    want, err = c.want()
    at = [0, 2, 5, 6, 8]
    check_bf16(kv[dst[at]], want[at, 0], err[at, 0])
    assert bool((kv[4] == 5.0).all())


def test_the_normed_query_equals_the_same_row_in_a_cache(dsa):
    # the same arithmetic in both entries: equal bits
    c = Case(9, 300, 1, 576, norm_dim=512, rot_off=512)
    kv, _ = pools("bf16", 300, 576)
    dsa.dsa_norm_rope_append(c.x[:, 0], c.pos, c.freq, kv, **c.kw)
    assert torch.equal(kv, dsa.dsa_norm_rope(c.x[:, 0], c.pos, c.freq, **c.kw))


def test_no_rows_and_a_captured_call(dsa):
    c = Case(10, 20, 4, 128)
    assert dsa.dsa_norm_rope(c.x[:0], c.pos[:0], c.freq, **c.kw).shape == (0, 4, 128)
    out = torch.empty_like(c.x)
    dsa.dsa_norm_rope(c.x, c.pos, c.freq, out=out, **c.kw)
    want = out.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_norm_rope(c.x, c.pos, c.freq, out=out, **c.kw)
    out.zero_()
    g.replay()
    assert torch.equal(out, want)
