"""dsa_tree_attn over contexts that a pair of CTAs walks for thousands of tiles.

Tolerances, per output element, with A = sum_p softmax_p |v_p| and ds the logits' error as for short contexts
(2^-22 (d + 2) sm_scale max |q| |k|):
 * the second product truncates its sums, four to a tile of 64 positions, by at most 2^-23 of the sum each.  Where L is
   65536 at most they run over 1024 tiles or fewer: 4 * 1024 * 2^-23 = 2^-11 A; elsewhere over 512 before they are added up
   in fp32: 2^-12 A;
 * one fp32 rounding per 512 tiles: 2^-24 each, 2^-14 A up to 1024 of them, with the exponentials and the merge;
 * the weights' rounding to bf16 2^-8 A, the output's 2^-8 |out|, the logits' 2 ds A.
The sums of weights take one fp32 addition per tile, over 1024 tiles at most (2^-14 of the sum), or over 512 and then one
per 512 (2^-15 + 2^-17 for 65536 tiles), so lse is off by ds + 2^-14 + 2^-20 (|lse| + 1)."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

D, DV, SM = 576, 512, 1 / 24
FORMATS = ["bf16", "fp8", "t128"]
BREAKS = 65536  # positions up to which a walk is not broken


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


def _encode(x, kv):
    """(cache rows, scales or None, the values they hold in fp64)"""
    if kv == "bf16":
        return x.bfloat16().cuda(), None, x.bfloat16().double().numpy()
    tiles = [x] if kv == "fp8" else list(x.split(128, 1))
    sc = torch.stack([t.abs().amax(1) / 448.0 for t in tiles], 1)
    wide = sc.repeat_interleave(D if kv == "fp8" else 128, 1)[:, :D]
    raw = (x / wide).to(torch.float8_e4m3fn).view(torch.uint8)
    val = oracle.e4m3_to_f64(raw.numpy()) * wide.double().numpy()
    return raw.cuda(), (sc[:, 0] if kv == "fp8" else sc).contiguous().cuda(), val


def _check(out, lse, q, rows, times=1, L=BREAKS + 1):
    """out [H, DV], lse [H] against the attention of q [H, D] over `rows`, each of them there `times` times."""
    q = q.double().cpu().numpy()
    x = SM * q @ rows.T
    m = x.max(1, keepdims=True)
    e = np.exp(x - m)
    w = e / e.sum(1, keepdims=True)
    want, A = w @ rows[:, :DV], w @ np.abs(rows[:, :DV])
    ds = 2.0**-22 * (D + 2) * SM * (np.abs(q) @ np.abs(rows).T).max(1)
    tol = 2.0**-8 * np.abs(want) + (2.0**-8 + (2.0**-12 if L > BREAKS else 2.0**-11) + 2.0**-14 + 2 * ds[:, None]) * A
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= tol), np.max(err / tol)
    want_lse = m[:, 0] + np.log(e.sum(1)) + np.log(times)
    assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= ds + 2.0**-14 + 2.0**-20 * (np.abs(want_lse) + 1))


def _one_sided(seed, rows, kv):
    # values of one sign: the sums only grow, which is where truncation shows
    g = torch.Generator().manual_seed(seed)
    cache, scale, val = _encode(torch.randn(rows, D, generator=g).abs(), kv)
    return cache, scale, val, (torch.randn(1, 8, D, generator=g) * 0.05).bfloat16().cuda()


@pytest.mark.parametrize("kv", FORMATS)
def test_four_million_positions_in_one_walk(dsa, kv):
    # more row tiles than are split (609 sequences): one pair of CTAs walks the only long context, 65536 tiles
    rows, times = 8192, 512
    cache, scale, val, q = _one_sided(1, rows, kv)
    n = 609
    ctx, new = np.zeros(n), np.zeros(n)
    ctx[0], new[0] = rows * times, 1
    out, lse = dsa.dsa_tree_attn(q.expand(n, -1, -1).contiguous(), cache, _i32(ctx), sm_scale=SM, q_per_seq=1, n_new=_i32(new),
                                 kv_scale=scale, block_table=_i32(np.zeros((n, times))), block_size=rows, L=rows * times)
    _check(out[0], lse[0], q[0], val, times)
    assert not out[1:].any() and bool((lse[1:] == -np.inf).all())


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("times", [1, 256, 1024])
def test_split_walks_of_any_length(dsa, kv, times):
    # one sequence of 256 tiles, of 65536 and of 262144 (3450 for each pair of CTAs)
    rows = 16384
    cache, scale, val, q = _one_sided(2, rows, kv)
    L = rows * times
    out, lse = dsa.dsa_tree_attn(q, cache, _i32([L]), sm_scale=SM, q_per_seq=1, n_new=_i32([1]), kv_scale=scale,
                                 block_table=_i32(np.zeros((1, times))), block_size=rows, L=L)
    _check(out[0], lse[0], q[0], val, times, L)


def _table(n, block, limit):
    return np.zeros((n, -(-limit // block)))  # entries past a sequence's end are not read


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("tiles,limit", [(511, 0), (513, 0), (1023, 0), (1024, 0)] +
                         [(t, BREAKS + 64) for t in (3, 511, 512, 513, 700, 1024, 1025)])
def test_walks_that_end_around_a_break(dsa, kv, tiles, limit):
    # no split: 609 sequences, two of them long; drafted tokens in the tile behind the context.  Without a limit the cache
    # ends with the context, and the walk is not broken
    rng = np.random.default_rng(tiles)
    n, N, H = 609, 2, 4
    g = torch.Generator().manual_seed(tiles)
    L = tiles * 64
    cache, scale, val = _encode(torch.randn(2 * L, D, generator=g), kv)
    q = torch.randn(n * N, H, D, generator=g).bfloat16().cuda()
    ctx, new = rng.integers(0, 3, n), np.zeros(n, int)
    ctx[[5, 600]], new[[5, 600]] = [L - 2, L - 65], [2, 1]
    limit = max(limit, L)
    table = _table(n, L, limit)
    table[600, 0] = 1
    out, lse = dsa.dsa_tree_attn(q, cache, _i32(ctx), sm_scale=SM, q_per_seq=N, n_new=_i32(new), kv_scale=scale,
                                 block_table=_i32(table), block_size=L, L=limit)
    out, lse, q = out.view(n, N, H, DV), lse.view(n, N, H), q.view(n, N, H, D)
    for i in range(2):
        _check(out[5, i], lse[5, i], q[5, i], val[:L - 2 + i + 1], 1, limit)
    _check(out[600, 0], lse[600, 0], q[600, 0], val[L:2 * L - 64], 1, limit)
    assert not out[600, 1].any()


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("rising", [True, False])
def test_a_maximum_that_moves_between_breaks(dsa, kv, rising):
    # rows that grow (or shrink) with their position, over 1100 tiles that one pair of CTAs walks
    n, L = 609, 1100 * 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn(L, D, generator=g) * torch.linspace(0.05, 4.0, L)[:, None]
    cache, scale, val = _encode(x if rising else x.flip(0), kv)
    q = torch.randn(n, 4, D, generator=g).bfloat16().cuda()
    ctx, new = np.zeros(n), np.zeros(n)
    ctx[7], new[7] = L - 1, 1
    out, lse = dsa.dsa_tree_attn(q, cache, _i32(ctx), sm_scale=SM, q_per_seq=1, n_new=_i32(new), kv_scale=scale,
                                 block_table=_i32(_table(n, L, L)), block_size=L, L=L)
    _check(out[7], lse[7], q[7], val)


@pytest.mark.parametrize("kv", FORMATS)
def test_nothing_seen_before_a_break(dsa, kv):
    # the first 40960 positions (640 tiles) lie in blocks outside of the pool: reported, and not seen
    n, block, L = 609, 4096, 14 * 4096
    limit = BREAKS + 1
    g = torch.Generator().manual_seed(4)
    cache, scale, val = _encode(torch.randn(4 * block, D, generator=g), kv)
    q = torch.randn(n, 4, D, generator=g).bfloat16().cuda()
    ctx, new = np.zeros(n), np.zeros(n)
    ctx[0], new[0] = L - 1, 1
    table = np.full((n, -(-limit // block)), -1)
    table[0, 10:14] = [2, 0, 3, 1]
    out, lse = dsa.dsa_tree_attn(q, cache, _i32(ctx), sm_scale=SM, q_per_seq=1, n_new=_i32(new), kv_scale=scale,
                                 block_table=_i32(table), block_size=block, L=limit)
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_error() == 1
    _check(out[0], lse[0], q[0], val)
