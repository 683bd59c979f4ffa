"""GPU parity of dsa_tree_attn with the oracle (fp64), for all cache formats and layouts.

Tolerances, per output element.  With A = sum_p softmax_p |v_p| and G = sm_scale max_p sum_j |q_j k_pj|:
 * the logits are fp32 sums of d = 576 products: off by at most ds = 2^-22 (d + 2) G (twice the unit
   roundoff, for accumulators that truncate), to first order 2 ds A on the output;
 * the weights are rounded to bf16 for the second product, by at most 2^-8 of each: 2^-8 A;
 * the exponentials, the running sums and the merge are fp32: under 2^-14 A together;
 * the output is rounded to bf16: 2^-8 |out|.
lse is off by ds and fp32 roundings of values up to |lse| + 1."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

D, DV = 576, 512


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


def tree_bits(rng, n_seq, N, kind):
    if kind == "chain":
        return np.broadcast_to(np.tril(np.ones((N, N), bool)), (n_seq, N, N)).copy()
    if kind == "any":       # any set of nodes, later ones and none at all included
        bits = rng.random((n_seq, N, N)) < 0.4
        bits[:, N // 2] = False
        return bits
    anc = np.zeros((n_seq, N, N), bool)
    for s in range(n_seq):
        for i in range(N):
            parent = int(rng.integers(-1, i)) if i else -1
            if parent >= 0:
                anc[s, i] = anc[s, parent]
            anc[s, i, i] = True
    return anc


def pack(bits):
    n_seq, N, _ = bits.shape
    W = -(-N // 32)
    words = np.zeros((n_seq * N, W), np.uint32)
    for j in range(N):
        words[:, j // 32] |= bits.reshape(-1, N)[:, j].astype(np.uint32) << np.uint32(j % 32)
    return torch.from_numpy(words.view(np.int32)).cuda()


class Case:
    """Inputs on the device, and the rows of each sequence in fp64, in position order."""

    def __init__(self, seed, ctx, N, H, kv="bf16", block=0, new=None, mask="tree", L=None, pitch=D, spread=1.0, pool_extra=3):
        rng = np.random.default_rng(seed)
        self.N, self.H, self.kv_kind, self.block = N, H, kv, block
        self.ctx = np.asarray(ctx)
        n = len(self.ctx)
        self.n = n
        self.new = np.full(n, N) if new is None else np.asarray(new)
        self.L = int(max(0, self.ctx.max()) + N) if L is None else L
        self.bits = tree_bits(rng, n, N, mask)
        self.mask = None if mask == "chain" else pack(self.bits)
        per = -(-self.L // block) if block else 0
        if block:
            ids = rng.permutation(n * per + pool_extra)
            self.table = ids[: n * per].reshape(n, per).astype(np.int32)
            rows = (n * per + pool_extra) * block
        else:
            self.table, rows = None, n * self.L
        g = torch.Generator().manual_seed(seed)
        x = torch.randn(rows, D, generator=g) * spread
        self.q = torch.randn(n * N, H, D, generator=g).bfloat16().cuda()
        self.scale = None
        if kv == "bf16":
            raw = x.bfloat16()
            val = raw.double().numpy()
        else:
            tiles = [x] if kv == "fp8" else list(x.split(128, 1))
            sc = torch.stack([t.abs().amax(1).clamp(min=1e-30) / 448.0 for t in tiles], 1)
            wide = sc.repeat_interleave(D if kv == "fp8" else 128, 1)[:, :D]
            raw = (x / wide).to(torch.float8_e4m3fn).view(torch.uint8)
            val = oracle.e4m3_to_f64(raw.numpy()) * wide.double().numpy()
            self.scale = (sc[:, 0] if kv == "fp8" else sc).contiguous().cuda()
        cache = torch.zeros(rows, pitch, dtype=raw.dtype)
        cache[:, :D] = raw
        self.cache = cache.cuda()[:, :D]
        self.val, self.rows = val, rows

    def row_of(self, s, p):
        return int(self.table[s, p // self.block]) * self.block + p % self.block if self.block else s * self.L + p

    def call(self, dsa, sm_scale, **kw):
        kv, scale = self.cache, self.scale
        if not self.block:
            kv = kv.unflatten(0, (self.n, self.L))
            scale = None if scale is None else scale.unflatten(0, (self.n, self.L))
        args = dict(sm_scale=sm_scale, q_per_seq=self.N, n_new=_i32(self.new), tree_mask=self.mask, kv_scale=scale,
                    block_table=_i32(self.table) if self.block else None, block_size=self.block,
                    L=self.L if self.block else None)
        args.update(kw)
        return dsa.dsa_tree_attn(self.q, kv, _i32(self.ctx), **args)

    def check(self, out, lse, sm_scale, nodes=None):
        out = out.double().cpu().numpy().reshape(self.n, self.N, self.H, DV)
        lse = lse.double().cpu().numpy().reshape(self.n, self.N, self.H)
        q = self.q.double().cpu().numpy().reshape(self.n, self.N, self.H, D)
        for s in range(self.n):
            c = min(max(int(self.ctx[s]), 0), self.L)
            m = min(max(int(self.new[s]), 0), self.N, self.L - c)
            kv = self.val[[self.row_of(s, p) for p in range(c + m)]]
            sees = self.bits[s].copy()
            live = min(max(int(self.new[s]), 0), self.N)
            for i in range(self.N) if nodes is None else nodes:
                at = list(range(c)) + [c + j for j in range(m) if sees[i, j]] if i < live else []
                if not at:
                    assert np.all(out[s, i] == 0) and np.all(lse[s, i] == -np.inf), (s, i)
                    continue
                want, want_lse = oracle.tree_attention(q[s, i:i + 1], kv[at], len(at), 1, np.zeros((1, 1), bool), sm_scale, DV)
                A, _ = oracle.tree_attention(q[s, i:i + 1], np.concatenate([kv[at], np.zeros((1, D))]), len(at), 1,
                                             np.zeros((1, 1), bool), sm_scale, DV)
                x = sm_scale * q[s, i] @ kv[at].T
                w = np.exp(x - want_lse[0][:, None])
                A = w @ np.abs(kv[at][:, :DV])
                ds = 2.0**-22 * (D + 2) * sm_scale * (np.abs(q[s, i]) @ np.abs(kv[at]).T).max(1)
                tol = 2.0**-8 * np.abs(want[0]) + (2.0**-8 + 2.0**-14 + 2 * ds[:, None]) * A
                assert np.all(np.abs(out[s, i] - want[0]) <= tol), (s, i, np.max(np.abs(out[s, i] - want[0]) / tol))
                assert np.all(np.abs(lse[s, i] - want_lse[0]) <= ds + 2.0**-20 * (np.abs(want_lse[0]) + 1)), (s, i)

    def run(self, dsa, sm_scale=1 / 24, **kw):
        out, lse = self.call(dsa, sm_scale, **kw)
        self.check(out, lse, sm_scale)
        return out, lse


FORMATS = ["bf16", "fp8", "t128"]


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("block", [0, 64, 192])
def test_trees_over_caches_of_every_format(dsa, kv, block):
    Case(1, [100, 257, 64], 7, 16, kv, block).run(dsa)


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("N,H", [(1, 1), (1, 16), (1, 128), (2, 5), (4, 16), (5, 20), (3, 64), (33, 4), (64, 2), (70, 1)])
def test_nodes_and_heads(dsa, kv, N, H):
    Case(N * H, [130, 3], N, H, kv, 0 if N % 2 else 64).run(dsa)


@pytest.mark.parametrize("kv", FORMATS)
def test_lengths_from_nothing_to_several_tiles(dsa, kv):
    ctx = [0, 1, 2, 31, 32, 63, 64, 65, 127, 128, 129, 191, 320, 500, 0, 7]
    new = [4, 4, 3, 4, 0, 4, 4, 1, 4, 2, 4, 4, 0, 4, 0, -3]
    for block in (0, 64):
        Case(5, ctx, 4, 16, kv, block, new=new).run(dsa)


@pytest.mark.parametrize("mask", ["chain", "any", "tree"])
@pytest.mark.parametrize("N,ctx", [(6, [0, 60]), (40, [0, 90]), (130, [5, 64])])
def test_masks_that_leave_nothing_or_look_ahead(dsa, mask, N, ctx):
    Case(6, ctx, N, 3, "bf16", 64, mask=mask, new=[N, N - 1]).run(dsa)


def test_without_node_counts(dsa):
    Case(7, [90, 20], 5, 16, "bf16").run(dsa, n_new=None)


def test_positions_past_the_cache_do_not_exist(dsa):
    # n_ctx + n_new beyond L: the drafted rows past the end are not there; n_ctx beyond L is L; below 0 is 0
    Case(8, [62, 70, 64, -5, 1000], 4, 16, "bf16", L=64).run(dsa)
    Case(8, [62, 70, 64, -5, 1000], 4, 16, "fp8", 64, L=64).run(dsa)


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("pitch", [592, 704])
def test_row_pitch(dsa, kv, pitch):
    Case(9, [100, 33], 4, 16, kv, 64, pitch=pitch).run(dsa)
    Case(9, [100, 33], 4, 16, kv, 0, pitch=pitch).run(dsa)


@pytest.mark.parametrize("kv", FORMATS)
def test_more_row_tiles_than_fill_the_device_evenly(dsa, kv):
    # 26 row tiles of each of three sequences: their tiles are shared out end to end, and a row tile's parts merged
    c = Case(20, [1200, 1310, 1150], 104, 32, kv)
    out, lse = c.call(dsa, 1 / 24)
    c.check(out, lse, 1 / 24, nodes=[4 * k + k % 4 for k in range(26)])


@pytest.mark.parametrize("kv", FORMATS)
def test_row_tiles_of_padding_nodes_beside_shared_out_ones(dsa, kv):
    # 3 row tiles per sequence, of which two to none hold nodes, over contexts of 20 to 60 tiles
    rng = np.random.default_rng(24)
    ctx = rng.integers(1280, 3800, 24)
    new = rng.choice([12, 11, 8, 5, 4, 1, 0], 24)
    ctx[3], new[3] = 0, 0
    c = Case(24, ctx, 12, 32, kv, 64, new=new)
    out, lse = c.call(dsa, 1 / 24)
    c.check(out, lse, 1 / 24, nodes=[0, 3, 7, 10, 11])


@pytest.mark.parametrize("n", [300, 700])
def test_many_short_sequences(dsa, n):
    rng = np.random.default_rng(n)
    Case(n, rng.integers(0, 150, n), 2, 16, "bf16", new=rng.integers(0, 3, n)).run(dsa)


@pytest.mark.parametrize("kv", FORMATS)
def test_a_context_of_hundreds_of_millions_of_positions(dsa, kv):
    # a table that names the same two blocks again and again: the softmax is theirs, lse that of `times` copies; the
    # scales' number (five per position) passes 2^31.  Sums: 7.0e6 tiles over 76 pairs of CTAs (92500 each), an fp32
    # rounding of the sum per tile and of the output per 16 positions (truncated: an ulp), so 92500 * 2^-24 = 0.6 % and
    # 4 * 92500 * 2^-23 = 4.4 % at the very worst
    times = 3_515_625  # 450 million positions
    c = Case(25, [128 * times], 1, 3, kv, 64, mask="chain", new=[0], L=128)
    table = torch.from_numpy(c.table[0, :2].copy()).cuda().repeat(times)[None].contiguous()
    out, lse = dsa.dsa_tree_attn(
        c.q, c.cache, torch.tensor([128 * times - 1], dtype=torch.int32, device="cuda"), sm_scale=1 / 24, q_per_seq=1,
        kv_scale=c.scale, block_table=table, block_size=64, L=128 * times)
    kv64 = c.val[[c.row_of(0, p) for p in range(128)]]
    q = c.q.double().cpu().numpy().reshape(1, 3, D)
    want, want_lse = oracle.tree_attention(q, kv64, 128, 1, np.zeros((1, 1), bool), 1 / 24, DV)
    x = q[0] @ kv64.T / 24
    A = np.exp(x - want_lse[0][:, None]) @ np.abs(kv64[:, :DV])
    assert np.all(np.abs(lse.double().cpu().numpy()[0] - want_lse[0] - np.log(times)) <= 0.006 + 2.0**-10)
    assert np.all(np.abs(out.double().cpu().numpy()[0] - want[0]) <= (0.05 + 2.0**-7) * A)


@pytest.mark.parametrize("kv", FORMATS)
def test_halves_of_the_values_whose_logits_round_apart(dsa, kv):
    # 2^25 + 1.5 - 2^25 + 8 is 8 or 9.5 in fp32, by the order of the columns, and a row's reference maximum moves at
    # more than 8: the CTAs that take the two halves of the values may go either way.  All rows hold the same values in
    # the columns looked at, so those are the output whatever the weights, also where the parts of a context are merged
    n_tiles = 400
    c = Case(26, [64 * n_tiles], 1, 2, kv, mask="chain", new=[0], L=64 * n_tiles)
    const = torch.from_numpy(np.random.default_rng(26).choice([1.0, -0.5, 2.0, 3.5, -1.25], D)).float()
    odd = (torch.arange(c.rows) // 64) % 2 == 1
    rows = const.repeat(c.rows, 1)
    used = [5, 130, 300, 301]
    rows[:, used] = 0.0
    rows[odd, 5], rows[odd, 130], rows[odd, 300], rows[odd, 301] = 256.0, 1.0, -256.0, 8.0
    q = torch.zeros(D)
    q[5], q[130], q[300], q[301] = 2.0**17, 1.5, 2.0**17, 1.0
    c.q = q.repeat(1, 2, 1).bfloat16().cuda()
    if kv == "bf16":
        c.cache.copy_(rows.bfloat16())
    else:
        c.cache.copy_(rows.to(torch.float8_e4m3fn).view(torch.uint8))
        c.scale.fill_(1.0)
    out, _ = dsa.dsa_tree_attn(c.q, c.cache.unflatten(0, (1, c.L)), torch.tensor([c.L], dtype=torch.int32, device="cuda"),
                               sm_scale=float(np.log(2.0)), q_per_seq=1, n_new=torch.zeros(1, dtype=torch.int32, device="cuda") + 1,
                               kv_scale=None if kv == "bf16" else c.scale.unflatten(0, (1, c.L)))
    keep = np.setdiff1d(np.arange(DV), used)
    want = const[keep].double().numpy()
    # each weight is rounded to bf16 for the product and not in the sum (2^-8), the output once more (2^-8)
    assert np.all(np.abs(out.double().cpu().numpy()[0][:, keep] - want) <= np.abs(want) * 2.0**-6.9)


@pytest.mark.parametrize("kv", ["fp8", "t128"])
def test_queries_of_a_wide_range(dsa, kv):
    # E4M3 rows: a query row enters as E4M3 plus E5M2, exact from 2^-13 of its largest value on, to 2^-20 of it below
    c = Case(21, [150, 20], 4, 16, kv, 64)
    rng = np.random.default_rng(21)
    f = np.ldexp(1.0, -rng.integers(0, 30, tuple(c.q.shape)))
    f *= np.ldexp(1.0, rng.integers(-60, 40, (c.q.shape[0], c.q.shape[1], 1)))  # rows of any size
    f[1, 3] = 0.0
    c.q = (c.q.double() * torch.from_numpy(f).cuda()).bfloat16()
    q = c.q.double().cpu().numpy().reshape(2, 4, 16, D)
    big = np.abs(q).max(-1, keepdims=True)
    sm = 1 / 24
    out, lse = c.call(dsa, sm)
    out, lse = out.double().cpu().numpy().reshape(2, 4, 16, DV), lse.double().cpu().numpy().reshape(2, 4, 16)
    for s in range(2):
        ctx = int(c.ctx[s])
        for i in range(4):
            at = list(range(ctx)) + [ctx + j for j in range(4) if c.bits[s, i, j]]
            kv64 = c.val[[c.row_of(s, p) for p in at]]
            want, want_lse = oracle.tree_attention(q[s, i:i + 1], kv64, len(at), 1, np.zeros((1, 1), bool), sm, DV)
            x = sm * q[s, i] @ kv64.T
            A = np.exp(x - want_lse[0][:, None]) @ np.abs(kv64[:, :DV])
            # the fp32 sums' part as in `check`, and 2^-20 of the row's largest value per product
            ds = sm * (2.0**-22 * (D + 2) * (np.abs(q[s, i]) @ np.abs(kv64).T) + 2.0**-20 * big[s, i] * np.abs(kv64).sum(1)).max(1)
            ok = ds < 0.25  # (rows whose logits are far beyond that have a single winner)
            tol = 2.0**-8 * np.abs(want[0]) + (2.0**-8 + 2.0**-14 + 2 * np.expm1(np.minimum(ds, 1.0))[:, None]) * A
            assert np.all((np.abs(out[s, i] - want[0]) <= tol)[ok]), (s, i)
            assert np.all((np.abs(lse[s, i] - want_lse[0]) <= ds + 2.0**-20 * (np.abs(want_lse[0]) + 1))[ok]), (s, i)
            assert ok.sum() >= 8  # (exponents below 12 or so of the 100 drawn)


@pytest.mark.parametrize("kv", ["fp8", "t128"])
def test_a_query_row_that_is_not_finite(dsa, kv):
    c = Case(22, [100, 40], 2, 16, kv)
    c.q[1, 5, 77] = float("inf")
    c.q[2, 0, 3] = float("nan")
    out, _ = c.call(dsa, 1 / 24)
    bad = torch.zeros(4, 16, dtype=torch.bool, device="cuda")
    bad[1, 5] = bad[2, 0] = True
    assert bool(torch.isnan(out.view(4, 16, DV)[bad]).all()) and bool(torch.isfinite(out.view(4, 16, DV)[~bad]).all())


@pytest.mark.parametrize("kv", ["fp8", "t128"])
@pytest.mark.parametrize("block", [0, 64])
def test_hidden_codes_do_not_matter(dsa, kv, block):
    c = Case(23, [70, 128, 5], 6, 16, kv, block, new=[6, 3, 2], L=200)
    used = [c.row_of(s, p) for s in range(3) for p in range(int(c.ctx[s] + c.new[s]))]
    c.cache[torch.from_numpy(np.setdiff1d(np.arange(c.rows), used)).cuda()] = 0x7F  # E4M3's NaN
    c.run(dsa)


@pytest.mark.parametrize("kv", FORMATS)
def test_sharp_softmax_and_a_maximum_that_keeps_rising(dsa, kv):
    c = Case(10, [700, 300], 4, 16, kv)
    c.run(dsa, sm_scale=0.7)
    # rows that grow with their position: every tile raises the running maximum of many query rows
    c = Case(11, [900], 2, 16, kv, spread=1.0)
    grow = torch.linspace(0.05, 3.0, c.rows)
    if kv == "bf16":
        c.cache.copy_((c.cache.float() * grow.cuda()[:, None]).bfloat16())
        c.val = c.cache.double().cpu().numpy()
    else:
        old = c.scale.clone()
        c.scale.mul_(grow.cuda() if kv == "fp8" else grow.cuda()[:, None])
        ratio = (c.scale.double() / old.double()).cpu().numpy()
        c.val = c.val * (ratio[:, None] if kv == "fp8" else ratio.repeat(128, 1)[:, :D])
    c.run(dsa, sm_scale=1.0)


@pytest.mark.parametrize("kv", ["fp8", "t128"])
def test_scales_zero_negative_and_far_apart(dsa, kv):
    c = Case(12, [200, 64], 4, 16, kv, 64)
    rng = np.random.default_rng(12)
    f = np.ldexp(1.0, rng.integers(-20, 2, c.scale.shape)) * rng.choice([-1.0, 1.0, 1.0, 0.0], c.scale.shape)
    c.scale.mul_(torch.from_numpy(f).float().cuda())
    c.val = c.val * (f[:, None] if kv == "fp8" else f.repeat(128, 1)[:, :D])
    c.run(dsa)


def _poison(c, rows):
    """NaN (or infinities, or NaN scales) in the given cache rows."""
    if c.kv_kind == "bf16":
        c.cache[rows[0::2]] = float("nan")
        c.cache[rows[1::2]] = float("inf")
    else:
        c.scale[rows] = float("nan")


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("block", [0, 64])
def test_hidden_rows_do_not_matter(dsa, kv, block):
    # rows past each sequence's end, rows of unused blocks
    c = Case(13, [70, 128, 5], 6, 16, kv, block, new=[6, 3, 2], L=200)
    used = [c.row_of(s, p) for s in range(3) for p in range(int(c.ctx[s] + c.new[s]))]
    rest = np.setdiff1d(np.arange(c.rows), used)
    _poison(c, torch.from_numpy(rest).cuda())
    c.run(dsa)


@pytest.mark.parametrize("kv", FORMATS)
def test_a_bad_row_reaches_only_the_nodes_that_see_it(dsa, kv):
    c = Case(14, [70, 3], 8, 16, kv, 64, mask="tree")
    bad_node = 2
    rows = torch.tensor([c.row_of(s, int(c.ctx[s]) + bad_node) for s in range(2)]).cuda()
    _poison(c, rows)
    out, lse = c.call(dsa, 1 / 24)
    o = out.view(2, 8, 16, DV)
    for s in range(2):
        for i in range(8):
            if c.bits[s, i, bad_node]:
                # an infinity gives infinite or undefined logits; a NaN makes everything NaN
                if kv != "bf16" or s == 0:
                    assert bool(torch.isnan(o[s, i]).all())
                else:
                    assert not bool(torch.isfinite(o[s, i]).all())
    clean = [i for i in range(8) if not c.bits[:, i, bad_node].any()]
    assert clean
    c.val[rows.cpu().numpy()] = 0
    c.check(out, lse, 1 / 24, nodes=clean)


def test_bad_block_ids_are_not_seen(dsa):
    c = Case(15, [200, 100], 4, 16, "bf16", 64)
    good = c.run(dsa)[0]
    c.table[0, 1] = c.rows // 64 + 5
    out, lse = c.call(dsa, 1 / 24)
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_error() == 1
    assert torch.equal(out[4:], good[4:])
    # the same as a sequence without those 64 positions
    keep = np.r_[0:64, 128:204]
    kv = c.val[[c.row_of(0, p) if p // 64 != 1 else 0 for p in range(204)]][keep]
    q = c.q.double().cpu().numpy()[:4]
    want, _ = oracle.tree_attention(q, kv, 136, 4, c.bits[0], 1 / 24, DV)
    assert np.max(np.abs(out[:4].double().cpu().numpy() - want)) <= 2e-2
    # entries past a sequence's end are never read
    c = Case(16, [100, 10], 4, 16, "fp8", 64, L=640)
    c.table[:, 2:] = -7
    c.run(dsa)


def test_offsets_past_32_bits(dsa):
    # a pool of 4.9 GB: rows beyond 2^32 bytes
    block, blocks = 64, 66000
    pool = torch.empty(blocks * block, D, dtype=torch.bfloat16, device="cuda")
    c = Case(17, [150], 3, 16, "bf16", 64, pool_extra=0)
    ids = [blocks - 1, 3, blocks - 7]
    for j, b in enumerate(ids):
        pool[b * block:(b + 1) * block] = c.cache[int(c.table[0, j]) * block:(int(c.table[0, j]) + 1) * block]
    out, lse = dsa.dsa_tree_attn(c.q, pool, _i32(c.ctx), sm_scale=1 / 24, q_per_seq=3, n_new=_i32(c.new),
                                 tree_mask=c.mask, block_table=_i32([ids]), block_size=block, L=c.L)
    c.check(out, lse, 1 / 24)
    # one contiguous sequence of that size, the last positions of which are drafted
    L = blocks * block
    ctx = L - 3
    pool.normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    q = c.q[:3]
    out, lse = dsa.dsa_tree_attn(q, pool.view(1, L, D), _i32([ctx]), sm_scale=1 / 24, q_per_seq=3)
    # rows by position in fp32 pieces on the device
    parts = []
    for lo in range(0, L, 1 << 18):
        x = (q.reshape(48, D).float() @ pool[lo:lo + (1 << 18)].float().T / 24).double()
        pos = torch.arange(lo, min(L, lo + (1 << 18)), device="cuda")
        node = torch.arange(48, device="cuda") // 16
        x.masked_fill_(pos[None, :] > ctx + node[:, None], -float("inf"))
        lse_p = torch.logsumexp(x, 1)
        v = pool[lo:lo + (1 << 18), :DV].float()
        parts.append((lse_p, torch.softmax(x, 1).float() @ v, torch.softmax(x, 1).float() @ v.abs()))
    lses = torch.stack([p[0] for p in parts])
    w = torch.softmax(lses, 0)
    want = sum(w[k][:, None] * p[1].double() for k, p in enumerate(parts))
    A = sum(w[k][:, None] * p[2].double() for k, p in enumerate(parts))
    assert torch.all((lse.view(48) - torch.logsumexp(lses, 0)).abs() <= 1e-3)
    # the bound above: A is about 0.8 here (the mean size of a value) and out about q / 24, so the weights'
    # rounding, 2^-8 A, is more than 2^-8 |out|; logits with |q| |k| = 576 / 24 give ds = 2^-22 578 24 at most
    ds = 2.0**-22 * (D + 2) * 24 * 1.5
    assert torch.all((out.view(48, DV) - want).abs() <= 2.0**-8 * want.abs() + (2.0**-8 + 2.0**-14 + 2 * ds) * A)


def test_given_buffers_streams_and_graphs(dsa):
    c = Case(18, [300, 90, 0, 64], 5, 16, "fp8", 64, new=[5, 2, 5, 5])
    want, want_lse = c.run(dsa)
    # the same inputs twice give the same bits
    again, again_lse = c.call(dsa, 1 / 24)
    assert torch.equal(again, want) and torch.equal(again_lse, want_lse)
    # on another stream, into given buffers, with a workspace full of NaN
    s = torch.cuda.Stream()
    out = torch.full_like(want, 9.0)
    ws = torch.full((1 << 27,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    c.call(dsa, 1 / 24, out=out, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    # captured; replayed with other lengths in the same tensors, beside a second graph on another stream
    ctx, new = _i32(c.ctx), _i32(c.new)
    kw = dict(sm_scale=1 / 24, q_per_seq=c.N, n_new=new, tree_mask=c.mask, kv_scale=c.scale, block_table=_i32(c.table),
              block_size=64, L=c.L)
    graphs, outs, wss = [], [], []
    for k in range(2):
        outs.append((torch.zeros_like(want), torch.zeros_like(want_lse)))
        wss.append(torch.empty(1 << 27, dtype=torch.uint8, device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dsa.dsa_tree_attn(c.q, c.cache, ctx, out=outs[k][0], lse=outs[k][1], ws=wss[k], **kw)
        graphs.append(g)
    c.ctx, c.new = np.array([64, 300, 130, 1]), np.array([0, 5, 1, 4])
    ctx.copy_(_i32(c.ctx))
    new.copy_(_i32(c.new))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0])
    c.check(*outs[0], 1 / 24)


def test_refusals(dsa):
    c = Case(19, [64], 2, 4, "fp8", 64)
    with pytest.raises(ValueError):
        c.call(dsa, 1.0, q_per_seq=3)
    with pytest.raises(ValueError):
        c.call(dsa, 1.0, tree_mask=torch.zeros(2, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        c.call(dsa, 1.0, tree_mask=torch.zeros(2, 1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        c.call(dsa, 1.0, kv_scale=None)
    with pytest.raises(ValueError):
        c.call(dsa, 1.0, kv_scale=c.scale[:-1])
    with pytest.raises(ValueError):
        c.call(dsa, 1.0, L=None)
    with pytest.raises(dsa.DsaError):
        c.call(dsa, 1.0, block_size=48)
    with pytest.raises(dsa.DsaError):
        c.call(dsa, 1.0, L=10000)
    with pytest.raises(ValueError):
        c.call(dsa, 1.0, out=torch.zeros(2, 4, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        c.call(dsa, 1.0, n_new=torch.tensor([2], device="cuda"))


def test_a_step_of_the_serving_path(dsa):
    # plan -> rotated append -> attention: three requests draft a tree of six tokens each in a paged FP8 cache
    rng = np.random.default_rng(20)
    N, H, block, num = 6, 16, 64, 24
    ctx, max_blocks = np.array([62, 0, 130]), 4
    table = np.full((3, max_blocks), -1, np.int32)
    table[0, 0], table[2, :3] = 5, [9, 1, 20]
    free = np.array([7, 3, 11, 2, 8, 0])
    t, n_ctx, n_new = _i32(table), _i32(ctx), _i32([N, N, N])
    inv_freq = torch.from_numpy((1e4 ** -(np.arange(32) / 32)).astype(np.float32)).cuda()
    cache = torch.zeros(num * block, D, dtype=torch.uint8, device="cuda")
    scale = torch.ones(num * block, device="cuda")
    g = torch.Generator().manual_seed(20)
    # the cached rows, as earlier steps wrote them
    old = torch.randn(int(ctx.sum()), D, generator=g).bfloat16()
    plan = dsa.dsa_block_plan(_i32([0, 0, 0]), n_ctx, _i32(np.array([5, 9, 1, 20])), t.clone(), block_size=block, num_blocks=num,
                              rows=int(ctx.sum()))
    dsa.dsa_rope_append(old.cuda(), plan.pos, inv_freq, cache, scale=scale, dst_rows=plan.dst_rows, rot_off=512)
    # the step
    bits = tree_bits(rng, 3, N, "tree")
    depth = bits.sum(2) - 1
    x = torch.randn(3 * N, D, generator=g).bfloat16()
    q = torch.randn(3 * N, H, D, generator=g).bfloat16()
    plan = dsa.dsa_block_plan(n_ctx, n_new, _i32(free), t, block_size=block, num_blocks=num, q_per_seq=N)
    pos = n_ctx.repeat_interleave(N) + _i32(depth.reshape(-1))
    dsa.dsa_rope_append(x.cuda(), pos, inv_freq, cache, scale=scale, dst_rows=plan.dst_rows, rot_off=512)
    qr = dsa.dsa_rope(q.cuda(), pos, inv_freq, rot_off=512)
    out, lse = dsa.dsa_tree_attn(qr, cache, n_ctx, sm_scale=1 / 24, q_per_seq=N, n_new=plan.n_placed, tree_mask=pack(bits),
                                 kv_scale=scale, block_table=t, block_size=block, L=max_blocks * block)
    # the oracle from the unrotated inputs: FP8 rounds the rows (2^-4 of an element at most), so the outputs
    # are compared with the stored rows exactly and with the unrounded rows loosely
    assert plan.taken.item() == 2 and t.cpu().numpy()[0, 1] == 7 and t.cpu().numpy()[1, 0] == 3
    val = oracle.e4m3_to_f64(cache.cpu().numpy()) * scale.double().cpu().numpy()[:, None]
    tb = t.cpu().numpy()
    start = np.concatenate([[0], np.cumsum(ctx)])
    p64 = pos.cpu().numpy().reshape(3, N)
    for s in range(3):
        rows = val[[int(tb[s, p // block]) * block + p % block for p in range(ctx[s] + N)]]
        want, want_lse = oracle.tree_attention(qr.double().cpu().numpy().reshape(3, N, H, D)[s], rows, ctx[s], N, bits[s], 1 / 24, DV)
        assert np.max(np.abs(out.double().cpu().numpy().reshape(3, N, H, DV)[s] - want)) <= 2.0**-7 * np.abs(rows[:, :DV]).max()
        raw = np.concatenate([old.double().numpy()[start[s]:start[s + 1]], x.double().numpy()[s * N:(s + 1) * N]])
        turned = oracle.rotate(raw, np.r_[np.arange(ctx[s]), p64[s]], inv_freq.cpu().numpy(), rot_off=512, rot_dim=64)
        assert np.all(np.abs(rows - turned) <= np.abs(turned) * 2.0**-4 + 2.0**-10 * np.abs(turned).max(1, keepdims=True) / 448 * 1.01 + 1e-5)
