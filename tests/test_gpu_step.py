"""GPU parity of the block plan, the rotary positions and the rotated cache append with the oracle."""
import numpy as np
import pytest
import torch

import oracle

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


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


# ---------------------------------------------------------------------------------------------
# block plan: whole numbers, equal

def _plan_case(seed, n_seq, new, ctx, block, spare=5):
    rng = np.random.default_rng(seed)
    c, m = rng.integers(0, ctx + 1, n_seq), rng.integers(0, new + 1, n_seq)
    max_blocks = -(-(ctx + new) // block)
    have, total = -(-c // block), -(-(c + m) // block)
    num = int(total.sum()) + spare
    ids = rng.permutation(num)
    table = np.full((n_seq, max_blocks), -1)
    table[np.arange(max_blocks)[None, :] < have[:, None]] = ids[: int(have.sum())]
    return c, m, ids[int(have.sum()):], table, num


def _check_plan(dsa, c, m, free, table, num, *, block, rows, q=0, n_free=None, out=None):
    want = oracle.block_plan(c, m, free, table, block_size=block, num_blocks=num, rows=rows, q_per_seq=q, n_free=n_free)
    t = _i32(table)
    p = dsa.dsa_block_plan(_i32(c), _i32(m), _i32(free), t, block_size=block, num_blocks=num, rows=rows, q_per_seq=q,
                           n_free=None if n_free is None else _i32([n_free]), out=out)
    for name in ("dst_rows", "pos", "seq", "row_start", "n_placed", "taken"):
        np.testing.assert_array_equal(getattr(p, name).cpu().numpy(), want[name], err_msg=name)
    np.testing.assert_array_equal(t.cpu().numpy(), want["table"])
    assert (dsa.dsa_get_device_error() == 0) == want["ok"]
    return want


@pytest.mark.parametrize("n_seq,new,ctx,block", [(1, 1, 0, 64), (1, 1, 64, 64), (3, 200, 500, 64), (33, 7, 1000, 192),
                                                 (1000, 1, 4096, 64), (1025, 3, 300, 128), (5000, 4, 100, 1), (7, 5000, 9, 33)])
@pytest.mark.parametrize("padded", [False, True])
def test_block_plan_equals_the_oracle(dsa, n_seq, new, ctx, block, padded):
    c, m, free, table, num = _plan_case(n_seq + new, n_seq, new, ctx, block)
    rows = n_seq * new + 3 if padded else int(m.sum()) + 37
    _check_plan(dsa, c, m, free, table, num, block=block, rows=rows, q=new if padded else 0)


def test_block_plan_largest_batch(dsa):
    c, m, free, table, num = _plan_case(3, 16384, 2, 256, 64)
    _check_plan(dsa, c, m, free, table, num, block=64, rows=int(m.sum()))


def test_block_plan_no_sequences_and_no_tokens(dsa):
    none = np.zeros(0, np.int64)
    _check_plan(dsa, none, none, np.arange(3), np.zeros((0, 4)), 3, block=64, rows=5)
    _check_plan(dsa, [0, 64, 3], [0, 0, 0], np.arange(3), np.full((3, 2), 1), 3, block=64, rows=0)


def test_block_plan_repeats_and_negative_lengths_count_as_zero(dsa):
    c, m, free, table, num = _plan_case(9, 20, 70, 300, 64)
    c[3], m[4], c[5] = -7, -2, 0
    for _ in range(2):
        _check_plan(dsa, c, m, free, table, num, block=64, rows=int(np.maximum(m, 0).sum()) + 80)


@pytest.mark.parametrize("keep", [0, 1, 10, 39])
def test_block_plan_short_free_list(dsa, keep):
    # sequences in order until the list runs out; those that need no block are placed all the same
    c, m, free, table, num = _plan_case(11, 40, 60, 500, 64)
    want = _check_plan(dsa, c, m, free, table, num, block=64, rows=int(m.sum()), n_free=keep)
    need = int((-(-(c + m) // 64) - -(-c // 64)).sum())
    assert want["ok"] == (keep >= need) and want["taken"][0] <= keep
    _check_plan(dsa, c, m, free[:keep], table, num, block=64, rows=int(m.sum()))


def test_block_plan_sequence_past_its_table_and_rows_past_their_number(dsa):
    c, m, free, table, num = _plan_case(12, 6, 100, 200, 64, spare=40)
    m[2] = 64 * table.shape[1]  # cannot fit beside what is cached
    c[2] = 1
    table[2, 0] = 0
    want = _check_plan(dsa, c, m, free, table, num, block=64, rows=int(m.sum()))
    assert want["n_placed"][2] == 0
    _check_plan(dsa, c, m, free, table, num, block=64, rows=int(m[:2].sum()) + 1)


def test_block_plan_bad_block_ids_get_no_row(dsa):
    c, m, free, table, num = _plan_case(13, 6, 100, 200, 64, spare=10)
    c[0], m[0] = 30, 5
    table[0, 0] = num + 3       # the partly filled block of sequence 0
    free[1] = -5
    want = oracle.block_plan(c, m, free, table, block_size=64, num_blocks=num, rows=int(m.sum()))
    t = _i32(table)
    p = dsa.dsa_block_plan(_i32(c), _i32(m), _i32(free), t, block_size=64, num_blocks=num, rows=int(m.sum()))
    np.testing.assert_array_equal(p.dst_rows.cpu().numpy(), want["dst_rows"])
    np.testing.assert_array_equal(t.cpu().numpy(), want["table"])
    assert (want["dst_rows"][:5] == -1).all()
    assert dsa.dsa_get_device_error() == 1


def test_block_plan_graph_replay_follows_the_lengths(dsa):
    c, m, free, table, num = _plan_case(14, 50, 9, 700, 64, spare=60)
    tc, tm, tf, tt = _i32(c), _i32(m), _i32(free), _i32(table)
    rows = 50 * 9
    call = lambda out: dsa.dsa_block_plan(tc, tm, tf, tt, block_size=64, num_blocks=num, rows=rows, out=out)  # noqa: E731
    p = call(None)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(p)
    m2 = np.minimum(m[::-1].copy(), 5)
    tm.copy_(_i32(m2))
    tt.copy_(_i32(table))
    g.replay()
    want = oracle.block_plan(c, m2, free, table, block_size=64, num_blocks=num, rows=rows)
    np.testing.assert_array_equal(p.dst_rows.cpu().numpy(), want["dst_rows"])
    np.testing.assert_array_equal(tt.cpu().numpy(), want["table"])


# ---------------------------------------------------------------------------------------------
# rotary positions.  y0 = x0 cos - x1 sin: sin and cos are off by at most 2^-22 (their argument's and
# their own rounding in fp32), the products and the sum add three fp32 roundings of values up to
# |x0| + |x1|: (|x0| + |x1|) 2^-21 covers both; then bf16 rounds by at most 2^-8 |y|.

def _inv_freq(n):
    return (1.0 / 10000.0 ** (np.arange(n) / n)).astype(np.float32)


def _pair_sum(x, rot_off, rot_dim, style):
    """|x0| + |x1| at both columns of every pair."""
    y = np.zeros_like(x)
    p = rot_dim // 2
    r = np.abs(x[..., rot_off:rot_off + rot_dim])
    s = r[..., :p] + r[..., p:] if style == "half" else r[..., 0::2] + r[..., 1::2]
    y[..., rot_off:rot_off + rot_dim] = np.concatenate([s, s], -1) if style == "half" else np.repeat(s, 2, -1)
    return y


CASES = [  # rows, heads, width, rot_off, rot_dim, axis of each pair
    (1, 1, 64, 0, 64, None), (5, 16, 64, 0, 64, None), (33, 16, 576, 512, 64, None), (7, 3, 128, 64, 64, "three"),
    (9, 17, 96, 8, 48, "two"), (4, 5, 70, 3, 22, "two"), (3, 2, 256, 0, 256, "three"), (300, 128, 64, 0, 64, None),
    (2, 1, 2, 0, 2, None), (6, 20, 80, 16, 64, "four"),
]


def _axes(kind, pairs):
    n = {None: 1, "two": 2, "three": 3, "four": 4}[kind]
    return n, None if n == 1 else [(i * 7 // 3) % n for i in range(pairs)]


@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("rows,heads,width,rot_off,rot_dim,kind", CASES)
def test_rope_against_the_oracle(dsa, rows, heads, width, rot_off, rot_dim, kind, style):
    rng = np.random.default_rng(rows * width + rot_dim)
    n_axes, axis = _axes(kind, rot_dim // 2)
    x = torch.from_numpy(rng.standard_normal((rows, heads, width))).bfloat16()
    pos = rng.integers(0, 1 << 20, (rows, n_axes))
    pos[0, 0] = (1 << 24) - 1
    f = _inv_freq(rot_dim // 2)
    kw = dict(rot_off=rot_off, rot_dim=rot_dim, pair_axis=axis, style=style)
    xd = x.double().numpy()
    for inverse in (False, True):
        want = oracle.rotate(xd, pos, f, inverse=inverse, **kw)
        tol = np.abs(want) * 2.0**-8 + _pair_sum(xd, rot_off, rot_dim, style) * 2.0**-21
        tol[..., :rot_off] = 0
        tol[..., rot_off + rot_dim:] = 0
        gx = x.cuda()
        got = dsa.dsa_rope(gx, _i32(pos), torch.from_numpy(f).cuda(), inverse=inverse, **kw)
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
        assert torch.equal(gx.cpu(), x)
        # in place, and into the middle of a wider buffer whose other columns stay as they were
        dsa.dsa_rope(gx, _i32(pos), torch.from_numpy(f).cuda(), inverse=inverse, out=gx, **kw)
        assert torch.equal(gx, got)
        wide = torch.full((rows, heads, width + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        dsa.dsa_rope(x.cuda(), _i32(pos), torch.from_numpy(f).cuda(), inverse=inverse, out=wide[..., 8:8 + width], **kw)
        assert torch.equal(wide[..., 8:8 + width], got)
        assert torch.all(wide[..., :8] == 7) and torch.all(wide[..., 8 + width:] == 7)


def test_rope_strided_heads_and_two_axes_of_x(dsa):
    # [heads, rows, width] seen as [rows, heads, width], odd pitches, and x without a head axis
    rng = np.random.default_rng(5)
    f = torch.from_numpy(_inv_freq(32)).cuda()
    pos = _i32(rng.integers(0, 5000, 9))
    base = torch.from_numpy(rng.standard_normal((4, 9, 64))).bfloat16().cuda()
    want = dsa.dsa_rope(base.transpose(0, 1).contiguous(), pos, f)
    assert torch.equal(dsa.dsa_rope(base.transpose(0, 1), pos, f), want)
    odd = torch.zeros(9, 4, 67, dtype=torch.bfloat16, device="cuda")
    odd[..., 1:65] = base.transpose(0, 1)
    assert torch.equal(dsa.dsa_rope(odd[..., 1:65], pos, f), want)
    assert torch.equal(dsa.dsa_rope(base[2], pos, f), want[:, 2])


def test_rope_negative_and_far_positions(dsa):
    # the angle of the largest positions: its error there is fp32's own, 2^-24 turns
    f = _inv_freq(32)
    pos = np.array([0, -1, -(1 << 20), (1 << 31) - 1, -(1 << 31), 1 << 24])
    x = torch.ones(6, 64, dtype=torch.bfloat16)
    want = oracle.rotate(x.double().numpy(), pos, f, rot_off=0, rot_dim=64)
    got = dsa.dsa_rope(x.cuda(), _i32(pos), torch.from_numpy(f).cuda()).double().cpu().numpy()
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0**-8 + 2 * (2.0**-21 + 2 * np.pi * 2.0**-23))
    assert np.array_equal(got[0], np.ones(64))  # position 0 leaves the row as it is


def test_rope_inverse_is_the_gradient(dsa):
    # L = <w, rope(x)>: dL/dx = rope^-1(w), against central differences of the oracle
    rng = np.random.default_rng(8)
    f, pos = _inv_freq(8), rng.integers(0, 50, (2, 2))
    axis = [0, 1] * 4
    x, w = rng.standard_normal((2, 3, 20)), torch.from_numpy(rng.standard_normal((2, 3, 20))).bfloat16()
    kw = dict(rot_off=2, rot_dim=16, pair_axis=axis, style="pairs")
    got = dsa.dsa_rope(w.cuda(), _i32(pos), torch.from_numpy(f).cuda(), inverse=True, **kw).double().cpu().numpy()
    wd, h = w.double().numpy(), 1e-4
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        d = (np.sum(wd * oracle.rotate(x + e, pos, f, **kw)) - np.sum(wd * oracle.rotate(x - e, pos, f, **kw))) / (2 * h)
        assert abs(got[at] - d) <= abs(d) * 2.0**-8 + 1e-5


# ---------------------------------------------------------------------------------------------
# rotated append.  Codes stand for code * s: E4M3 rounds x / s by at most 2^-4 of it, or half its
# smallest step 2^-10 below 2^-6; the scale by 2^-22; the rotation as above.

def _append(dsa, fmt, x, pos, f, dst, pool, pitch=None, scale_fill=-7.0, **kw):
    width = x.shape[1]
    pitch = pitch or width
    if fmt == "bf16":
        cache, scale = torch.full((pool, pitch), 3.0, dtype=torch.bfloat16, device="cuda"), None
    else:
        cache = torch.full((pool, pitch), 0xEF, dtype=torch.uint8, device="cuda")
        shape = {"fp8": (pool,), "t128": (pool, -(-width // 128)), "mx": (pool, width // 32)}[fmt]
        scale = torch.full(shape, 0xCD, dtype=torch.uint8, device="cuda") if fmt == "mx" else \
            torch.full(shape, scale_fill, dtype=torch.float32, device="cuda")
    dsa.dsa_rope_append(x, pos, f, cache[:, :width], scale=scale, dst_rows=dst, **kw)
    return cache, scale


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "t128", "mx"])
@pytest.mark.parametrize("rows,width,rot_off,rot_dim,kind,style,pitch", [
    (1, 576, 512, 64, None, "half", 576), (130, 576, 512, 64, "three", "half", 592), (67, 576, 512, 64, "two", "pairs", 576),
    (50, 128, 64, 64, None, "half", 128), (50, 128, 0, 64, "three", "pairs", 136), (41, 160, 30, 44, "two", "half", 163),
    (9, 1024, 0, 256, None, "half", 1024), (5, 1056, 512, 64, None, "pairs", 1056),
])
def test_rope_append_against_the_oracle(dsa, fmt, rows, width, rot_off, rot_dim, kind, style, pitch):
    rng = np.random.default_rng(rows + width)
    n_axes, axis = _axes(kind, rot_dim // 2)
    x = torch.from_numpy(rng.standard_normal((rows, width)) * np.ldexp(1.0, rng.integers(-12, 12, (rows, 1)))).bfloat16()
    pos = rng.integers(0, 1 << 18, (rows, n_axes))
    f = _inv_freq(rot_dim // 2)
    pool = rows + 20
    dst = rng.permutation(pool)[:rows].astype(np.int64)
    if rows > 4:
        dst[3] = -1
        x[4] = 0
    kw = dict(rot_off=rot_off, rot_dim=rot_dim, pair_axis=axis, style=style)
    cache, scale = _append(dsa, fmt, x.cuda(), _i32(pos), torch.from_numpy(f).cuda(), torch.from_numpy(dst).cuda(), pool,
                           pitch, **kw)
    xd = x.double().numpy()
    y = oracle.rotate(xd, pos, f, **kw)
    slack = _pair_sum(xd, rot_off, rot_dim, style) * 2.0**-21
    live = dst >= 0
    y, slack, at = y[live], slack[live], dst[live]
    raw = cache.cpu()
    got = raw[at, :width]
    if fmt == "bf16":
        assert np.all(np.abs(got.double().numpy() - y) <= np.abs(y) * 2.0**-8 + slack)
        untouched = raw == 3.0
    else:
        group = {"fp8": width, "t128": 128, "mx": 32}[fmt]
        sc = scale.cpu().numpy()[at].reshape(len(at), -1)
        s = (np.ldexp(1.0, sc.astype(int) - 127) if fmt == "mx" else sc.astype(np.float64)).repeat(group, 1)[:, :width]
        v = oracle.e4m3_to_f64(got.numpy()) * s
        # the shared exponent of a group of 32 puts its largest value in [256, 512) steps of s, and E4M3
        # ends at 448, where the format saturates: the value to stand for is y clipped to 448 s
        y_all = y
        if fmt == "mx":
            y = np.clip(y, -448.0 * s, 448.0 * s)
        assert np.all(np.abs(v - y) <= np.maximum(np.abs(y) * 2.0**-4, s * 2.0**-10) * (1 + 2.0**-20) + slack * 1.1)
        for g in range(-(-width // group)):  # each scale against its group's largest value
            sl = slice(g * group, min((g + 1) * group, width))
            amax, most = np.abs(y_all[:, sl]).max(1), slack[:, sl].max(1)
            if fmt == "mx":
                lo = np.where(amax > most, np.floor(np.log2(np.maximum(amax - most, 1e-300))), 8) - 8
                hi = np.where(amax > 0, np.floor(np.log2(np.maximum(amax + most, 1e-300))), 8) - 8
                e = sc[:, g].astype(int) - 127
                assert np.all((e >= np.maximum(lo, -127)) & (e <= hi))
            else:
                want = np.where(amax > 0, amax / 448.0, 1.0)
                assert np.all(np.abs(sc[:, g] - want) <= want * 2.0**-22 + most / 448.0)
        untouched = raw == 0xEF
    rest = np.setdiff1d(np.arange(pool), at)
    assert bool(untouched[rest].all()) and bool(untouched[:, width:].all())
    if scale is not None:
        fill = 0xCD if fmt == "mx" else -7.0
        assert bool((scale.cpu()[rest] == fill).all())


@pytest.mark.parametrize("fmt", ["fp8", "t128", "mx"])
def test_rope_append_at_position_zero_is_the_quantiser(dsa, fmt):
    # no rotation: codes and scales are those of dsa_quantize_*, bit for bit
    x = torch.randn(77, 576, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    f = torch.from_numpy(_inv_freq(32)).cuda()
    cache, scale = _append(dsa, fmt, x, _i32(np.zeros(77)), f, None, 77, rot_off=512)
    want = {"fp8": dsa.dsa_quantize_fp8_rows, "t128": dsa.dsa_quantize_fp8_tiles, "mx": dsa.dsa_quantize_mxfp8}[fmt](x)
    assert torch.equal(cache, want[0]) and torch.equal(scale, want[1])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "t128", "mx"])
@pytest.mark.parametrize("width,rot_off,rot_dim,kind,style,pitch", [
    (576, 512, 64, "three", "half", 576), (576, 512, 64, None, "pairs", 592), (640, 0, 32, "two", "pairs", 640),
    (160, 96, 64, "two", "half", 168), (704, 64, 64, None, "half", 704),
])
def test_rope_append_of_many_rows_is_that_of_few(dsa, fmt, width, rot_off, rot_dim, kind, style, pitch):
    # one call of so many rows that a warp may take two at a time, against calls of few: bit for bit, also at quotients
    # that are rounding midpoints (small integers, scales that are 7 times a power of two over 448)
    rows = 32768 + 777
    rng = np.random.default_rng(width + rot_dim)
    n_axes, axis = _axes(kind, rot_dim // 2)
    x = torch.from_numpy(rng.standard_normal((rows, width)) * np.ldexp(1.0, rng.integers(-12, 12, (rows, 1)))).bfloat16()
    x[1000:3000] = torch.from_numpy(rng.integers(-28, 29, (2000, width)).astype(np.float32)).bfloat16()
    x[4000:4010] = 0
    pos = rng.integers(0, 1 << 18, (rows, n_axes))
    pos[1000:3000] = 0
    pool = rows + 20
    dst = rng.permutation(pool)[:rows].astype(np.int64)
    dst[[3, 4000, rows - 1]] = -1
    x, pos, dst, f = x.cuda(), _i32(pos), torch.from_numpy(dst).cuda(), torch.from_numpy(_inv_freq(rot_dim // 2)).cuda()
    kw = dict(rot_off=rot_off, rot_dim=rot_dim, pair_axis=axis, style=style)
    cache, scale = _append(dsa, fmt, x, pos, f, dst, pool, pitch, **kw)
    few = torch.full_like(cache, 3.0 if fmt == "bf16" else 0xEF)
    few_scale = None if scale is None else torch.full_like(scale, 0xCD if fmt == "mx" else -7.0)
    for i in range(0, rows, 3001):
        dsa.dsa_rope_append(x[i:i + 3001], pos[i:i + 3001], f, few[:, :width], scale=few_scale, dst_rows=dst[i:i + 3001], **kw)
    assert torch.equal(cache, few) and (scale is None or torch.equal(scale, few_scale))
    big = dst.clone()
    big[77] = pool  # past the cache: dropped and reported
    if fmt == "t128" and width == 576:
        dsa.dsa_rope_append(x, pos, f, cache[:, :width], scale=scale, dst_rows=big, **kw)
        assert dsa.dsa_get_device_error() == 1
        assert torch.equal(cache, few) and torch.equal(scale, few_scale)


def test_rope_append_row_past_the_cache_is_dropped(dsa):
    x = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(6, 64, dtype=torch.bfloat16, device="cuda")
    dst = torch.tensor([1, 4, 1 << 40], device="cuda")
    dsa.dsa_rope_append(x, _i32([0, 0, 0]), torch.from_numpy(_inv_freq(32)).cuda(), cache[:4], dst_rows=dst, rot_off=0)
    assert dsa.dsa_get_device_error() == 1
    assert cache.float().sum(1).tolist() == [0, 64, 0, 0, 0, 0]


def test_step_operators_refuse_what_does_not_fit(dsa):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    f, pos = torch.zeros(32, device="cuda"), _i32(np.zeros(4))
    with pytest.raises(TypeError):
        dsa.dsa_rope(x.float(), pos, f)
    with pytest.raises(TypeError):
        dsa.dsa_rope(x, pos.long(), f)
    with pytest.raises(ValueError):
        dsa.dsa_rope(x, pos[:3], f)
    with pytest.raises(ValueError):
        dsa.dsa_rope(x, pos, f[:16])
    with pytest.raises(ValueError):
        dsa.dsa_rope(x, pos, f, style="other")
    with pytest.raises(ValueError):
        dsa.dsa_rope(x, torch.stack([pos, pos], 1), f, sections=(32,))
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rope(x, torch.stack([pos, pos], 1).contiguous(), f)
    with pytest.raises(ValueError):
        dsa.dsa_rope(x, pos, f, out=torch.zeros(4, 65, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        dsa.dsa_rope(x, pos.cpu(), f)
    cache = torch.zeros(4, 64, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        dsa.dsa_rope_append(x, pos, f, cache, rot_off=0)                                  # no scales
    with pytest.raises(ValueError):
        dsa.dsa_rope_append(x, pos, f, cache, scale=torch.zeros(3, device="cuda"), rot_off=0)
    with pytest.raises(ValueError):
        dsa.dsa_rope_append(x, pos, f, cache[:, :32], scale=torch.zeros(4, device="cuda"), rot_off=0)
    with pytest.raises(ValueError):
        dsa.dsa_block_plan(pos, pos, pos, pos.view(2, 2), block_size=64, num_blocks=4, rows=4)
    with pytest.raises(ValueError):
        dsa.dsa_block_plan(pos, pos, pos, pos.view(4, 1), block_size=64, num_blocks=4)


def test_rope_runs_on_the_given_stream(dsa):
    # the input is made on a side stream; the call on that stream follows it without a synchronisation
    s = torch.cuda.Stream()
    f, pos = torch.from_numpy(_inv_freq(32)).cuda(), _i32(np.arange(4096))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x = torch.randn(4096, 16, 64, device="cuda").bfloat16()
        got = dsa.dsa_rope(x, pos, f)
        again = dsa.dsa_rope(x, pos, f, stream=s)
    s.synchronize()
    want = dsa.dsa_rope(x, pos, f)
    assert torch.equal(got, want) and torch.equal(again, want)
