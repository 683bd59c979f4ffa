"""GPU parity of the expanded form (dsa_latent_expand, dsa_expanded_attn) with the formulas in 64 bits.

Expansion, per output: fp32 sums of d = 512 products of bf16 values are off by at most 2^-22 (d + 2) S (twice the unit roundoff,
for accumulators that truncate), S = sum_c |row_c w_c|; with a scale per 128 columns each code times its scale is rounded to bf16
before, 2^-8 S; the output 2^-8 of itself.

Attention: as for the attention of drafted tokens.  With A = sum_p softmax_p |v_p| and G = sm_scale max_p sum_j |q_j k_pj|: the
logits (fp32 sums of d = 192 products) are off by at most ds = 2^-22 (d + 2) G, to first order 2 ds A on the output; the weights
are rounded to bf16, 2^-8 A; exponentials, running sums and the merge are fp32 and the second product truncates, under
2^-13 A together for contexts up to 16384 positions; the output is rounded, 2^-8 |out|."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

D = 576


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


def _starts(lens, first=0):
    return np.concatenate([[0], np.cumsum(lens)]) + first


# ----------------------------------------------------------------------------------------------
# expansion

class Rows:
    """A latent cache, and its values in fp64."""

    def __init__(self, seed, lens, kv="bf16", block=0, pitch=D, L=None):
        rng, g = np.random.default_rng(seed), torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.kv_kind, self.block = np.asarray(lens), kv, block
        n = len(lens)
        self.L = int(max([1, *lens])) if L is None else L
        per = -(-self.L // block) if block else 0
        rows = (n * per + 3) * block if block else n * self.L
        self.table = rng.permutation(n * per + 3)[: n * per].reshape(n, per) if block else None
        x = torch.randn(rows, D, generator=g, device="cuda")
        self.scale = None
        if kv == "bf16":
            raw = x.bfloat16()
            self.val = raw.double()
        else:
            tiles = [x] if kv == "fp8" else list(x.split(128, 1))
            sc = torch.stack([t.abs().amax(1).clamp(min=1e-30) / 448.0 for t in tiles], 1)
            wide = sc.repeat_interleave(D if kv == "fp8" else 128, 1)[:, :D]
            raw = (x / wide).to(torch.float8_e4m3fn).view(torch.uint8)
            self.val = raw.view(torch.float8_e4m3fn).double() * wide.double()
            self.scale = (sc[:, 0] if kv == "fp8" else sc).contiguous()
        cache = torch.zeros(rows, pitch, dtype=raw.dtype, device="cuda")
        cache[:, :D] = raw
        self.cache, self.rows = cache[:, :D], rows

    def at(self):
        """The cache row of every packed position."""
        out = []
        for s, m in enumerate(self.lens):
            p = np.arange(m)
            out.append(self.table[s, p // self.block] * self.block + p % self.block if self.block else s * self.L + p)
        return torch.from_numpy(np.concatenate(out + [np.zeros(0, np.int64)]).astype(np.int64)).cuda()

    def call(self, dsa, w, start, **kw):
        kv, scale = self.cache, self.scale
        if not self.block:
            kv = kv.unflatten(0, (len(self.lens), self.L))
            scale = None if scale is None else scale.unflatten(0, (len(self.lens), self.L))
        return dsa.dsa_latent_expand(kv, w, _i32(start), kv_scale=scale, block_table=_i32(self.table) if self.block else None,
                                     block_size=self.block, **kw)

    def check(self, out, rope, w):
        x, wide = self.val[self.at()], w.double().view(-1, 512)
        want = x[:, :512] @ wide.t()
        S = x[:, :512].abs() @ wide.abs().t()
        tol = 2.0**-8 * want.abs() + (2.0**-22 * 514 + (2.0**-8 if self.kv_kind == "t128" else 0.0)) * S
        err = (out.double().view(len(x), -1) - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        assert bool(((rope.double() - x[:, 512:]).abs() <= (0.0 if self.kv_kind == "bf16" else 2.0**-8 + 2.0**-22) * x[:, 512:].abs()).all())


def weights(H, seed=0):
    return (torch.randn(H, 256, 512, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") / 22).bfloat16()


FORMATS = ["bf16", "fp8", "t128"]


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("block", [0, 64, 192])
@pytest.mark.parametrize("lens", [[1], [127, 0, 2, 300], [256], [257, 511, 1]])
def test_expansion_of_caches_of_every_format(dsa, kv, block, lens):
    r, w = Rows(1, lens, kv, block), weights(3)
    out, rope = r.call(dsa, w, _starts(lens), rows=int(sum(lens)))
    r.check(out, rope, w)


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("H,lens", [(1, [700]), (16, [5000, 3000, 2100]), (20, [2000]), (128, [300, 40]), (7, [20000])])
def test_expansion_for_heads_and_many_rows(dsa, kv, H, lens):
    r, w = Rows(2, lens, kv, 64), weights(H)
    r.check(*r.call(dsa, w, _starts(lens), rows=int(sum(lens))), w)


@pytest.mark.parametrize("kv", FORMATS)
def test_expansion_leaves_other_rows_alone(dsa, kv):
    lens = [70, 0, 100]
    r, w = Rows(3, lens, kv, 0, pitch=592, L=128), weights(2)
    out = torch.full((400, 2, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    rope = torch.full((400, 64), 4.0, dtype=torch.bfloat16, device="cuda")
    r.call(dsa, w, _starts(lens, 30), out=out, rope_out=rope)
    r.check(out[30:200], rope[30:200], w)
    assert bool((out[:30] == 3.0).all()) and bool((out[200:] == 3.0).all())
    assert bool((rope[:30] == 4.0).all()) and bool((rope[200:] == 4.0).all())
    # the outputs hold fewer rows than there are positions
    out, rope = r.call(dsa, w, _starts(lens), rows=130)
    full = r.call(dsa, w, _starts(lens), rows=170)
    assert torch.equal(out, full[0][:130]) and torch.equal(rope, full[1][:130])


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("block", [0, 64])
def test_positions_outside_the_cache_are_zeros_and_recorded(dsa, kv, block):
    r, w = Rows(4, [100, 90], kv, block, L=128), weights(2)
    if block:
        r.table[1, 1] = 1 << 20
        start, bad = [0, 100, 190], slice(164, 190)
    else:
        start, bad = [0, 100, 100 + 140], slice(100 + 128, 240)
    out, rope = r.call(dsa, w, start, rows=start[-1])
    assert dsa.dsa_get_device_error() == 1
    assert bool((out[bad] == 0).all()) and bool((rope[bad] == 0).all())
    assert bool((out[100:164].abs().amax((1, 2)) > 0).all())


def test_expansion_of_nothing(dsa):
    r, w = Rows(5, [0, 0], "bf16"), weights(2)
    out, rope = r.call(dsa, w, [0, 0, 0], rows=0)
    assert out.shape == (0, 2, 256) and rope.shape == (0, 64)
    out, rope = torch.ones(5, 2, 256, device="cuda").bfloat16(), torch.ones(5, 64, device="cuda").bfloat16()
    r.call(dsa, w, [0, 0, 0], out=out, rope_out=rope)
    assert bool((out == 1).all()) and bool((rope == 1).all())


# ----------------------------------------------------------------------------------------------
# attention

class Packed:
    def __init__(self, seed, new, lens, H, q_first=0, k_first=0, spare=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.lens, self.H = np.asarray(new), np.asarray(lens), H
        self.q_start, self.kv_start = _starts(new, q_first), _starts(lens, k_first)
        T, N = int(self.q_start[-1]) + spare, int(self.kv_start[-1]) + spare
        self.q = torch.randn(T, H, 192, generator=g, device="cuda").bfloat16()
        self.kv = torch.randn(N, H, 256, generator=g, device="cuda").bfloat16()
        self.k_rope = torch.randn(N, 64, generator=g, device="cuda").bfloat16()

    def call(self, dsa, sm=192**-0.5, **kw):
        return dsa.dsa_expanded_attn(self.q, self.kv[..., :128], self.k_rope, self.kv[..., 128:], _i32(self.q_start), _i32(self.kv_start),
                                     sm_scale=sm, **kw)

    def check(self, out, lse, sm=192**-0.5, causal=True, more=0.0):
        for s in range(len(self.new)):
            m, n = int(self.new[s]), int(self.lens[s])
            qa, ka = int(self.q_start[s]), int(self.kv_start[s])
            for h in range(self.H):
                k = torch.cat([self.kv[ka:ka + n, h, :128], self.k_rope[ka:ka + n]], 1).double()
                v = self.kv[ka:ka + n, h, 128:].double()
                for lo in range(0, m, 2048):
                    r = min(2048, m - lo)
                    q = self.q[qa + lo:qa + lo + r, h].double()
                    x, G = sm * q @ k.t(), sm * q.abs() @ k.abs().t()
                    if causal:
                        hide = torch.arange(n, device="cuda")[None] > (n - m + lo + torch.arange(r, device="cuda"))[:, None]
                        x, G = x.masked_fill(hide, -torch.inf), G.masked_fill(hide, 0.0)
                    o, l = out[qa + lo:qa + lo + r, h].double(), lse[qa + lo:qa + lo + r, h].double()
                    none = torch.isinf(x).all(1) if n else torch.ones(r, dtype=torch.bool, device="cuda")
                    assert bool((o[none] == 0).all()) and bool((l[none] == -torch.inf).all()), (s, h)
                    if not n or bool(none.all()):
                        continue
                    live = ~none
                    w = torch.softmax(x[live], 1)
                    want, A, want_l = w @ v, w @ v.abs(), torch.logsumexp(x[live], 1)
                    ds = 2.0**-22 * 194 * G[live].amax(1)
                    tol = 2.0**-8 * want.abs() + (2.0**-8 + 2.0**-13 + more + 2 * ds[:, None]) * A
                    err = (o[live] - want).abs()
                    assert bool((err <= tol).all()), (s, h, float((err / tol).max()))
                    assert bool(((l[live] - want_l).abs() <= ds + 2.0**-20 * (want_l.abs() + 1)).all()), (s, h)


@pytest.mark.parametrize("H", [1, 3, 16])
@pytest.mark.parametrize("m", [1, 2, 127, 128, 129, 255, 256, 257, 700])
def test_a_prompt(dsa, H, m):
    c = Packed(m, [m], [m], H)
    c.check(*c.call(dsa))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 1000), (1, 20000), (5, 128), (130, 1100), (300, 4000), (1000, 1001), (256, 16384)])
def test_a_chunk_over_its_context(dsa, m, n, causal):
    c = Packed(m + n, [m], [n], 2)
    c.check(*c.call(dsa, causal=causal), causal=causal)


@pytest.mark.parametrize("causal", [True, False])
def test_ragged_sequences_with_empty_ones(dsa, causal):
    new, lens = [0, 1, 300, 17, 0, 256, 5, 128, 64], [0, 1, 300, 1000, 50, 256, 700, 128, 64]
    c = Packed(1, new, lens, 5, q_first=3, k_first=7, spare=11)
    out = torch.full((len(c.q), 5, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((len(c.q), 5), 8.0, device="cuda")
    c.call(dsa, causal=causal, out=out, lse=lse)
    c.check(out, lse, causal=causal)
    for a, b in ((0, 3), (int(c.q_start[-1]), len(c.q))):  # rows of no sequence
        assert bool((out[a:b] == 9.0).all()) and bool((lse[a:b] == 8.0).all())


def test_queries_that_see_nothing(dsa):
    # more queries than positions: the first ones come before every position
    c = Packed(2, [400, 10, 3], [150, 0, 1], 2)
    c.check(*c.call(dsa))


@pytest.mark.parametrize("n_seq", [300, 4096])
def test_many_short_sequences(dsa, n_seq):
    rng = np.random.default_rng(n_seq)
    new = rng.integers(0, 4, n_seq)
    c = Packed(3, new, new + rng.integers(0, 9, n_seq), 1)
    out, lse = c.call(dsa)
    c.new, keep = c.new[::7], np.arange(0, n_seq, 7)
    c.lens, c.q_start, c.kv_start = c.lens[keep], c.q_start[keep], c.kv_start[keep]
    c.check(out, lse)


def test_chunks_of_positions_are_merged(dsa):
    # few blocks of queries over long contexts: each is cut into spans of positions
    c = Packed(4, [3, 260, 1], [9000, 12000, 60], 2)
    c.check(*c.call(dsa))
    c.check(*c.call(dsa, max_len=12000))


def test_a_context_longer_than_a_chunk_may_be(dsa):
    # 65536 positions a chunk at most; the values have one sign, so that what a truncating sum loses adds up: 2^-23 per step
    # of 16 positions, 4096 steps of a chunk
    c = Packed(5, [40], [140000], 1)
    c.kv[..., 128:] = c.kv[..., 128:].abs()
    c.check(*c.call(dsa), more=4096 * 2.0**-23)


@pytest.mark.parametrize("new,lens,H", [
    ([31 * 256 - 9, 100], [9000, 100], 16),  # 512 blocks: 56 behind three rounds of 152, 16 of them too short to be cut in two
    ([8192], [9300], 24),                    # 768 blocks: 8 behind five rounds, for at most 19 CTAs each
])
def test_what_is_left_behind_whole_rounds_is_cut(dsa, new, lens, H):
    c = Packed(9, new, lens, H)
    out, lse = c.call(dsa)
    c.check(out, lse)
    again = c.call(dsa)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("new,lens", [
    ([29 * 256], [131072 - 128 + 29 * 256]),              # a block a CTA: 464 of 16 heads
    ([14 * 256 - 3, 40], [131072 - 128 + 14 * 256 - 3, 70000]),  # spans of more than 512 tiles
])
def test_long_contexts_of_many_blocks(dsa, new, lens):
    # blocks are walked in stretches of 65536 positions, 4096 steps, whose sums are added up in fp32; of the first block's 256
    # queries the first 128 end where a stretch does
    c = Packed(8, new, lens, 16, q_first=2, k_first=1, spare=5)
    c.kv[..., 128:] = c.kv[..., 128:].abs()
    T, N = c.q.shape[0], c.kv.shape[0]
    first, last = torch.full((T, 16, 128), 3.0, device="cuda").bfloat16(), torch.full((T, 16), 3.0, device="cuda")
    out, lse = c.call(dsa, out=first, lse=last)
    for rows in (slice(0, 2), slice(T - 5, T)):
        assert bool((out[rows] == 3).all()) and bool((lse[rows] == 3).all())
    for s, (m, n) in enumerate(zip(new, lens)):
        qa, ka = int(c.q_start[s]), int(c.kv_start[s])
        for lo, r, h in ((0, 3, 0), (126, 4, 15), (m // 2, 3, 7), (m - 2, 2, 1), (255, 2, 14)):
            lo = min(lo, m - r)
            part = Packed(0, [r], [n - m + lo + r], 1)
            part.q = c.q[qa + lo:qa + lo + r, h:h + 1]
            part.kv, part.k_rope = c.kv[ka:ka + n - m + lo + r, h:h + 1], c.k_rope[ka:ka + n - m + lo + r]
            part.check(out[qa + lo:qa + lo + r, h:h + 1], lse[qa + lo:qa + lo + r, h:h + 1], more=4096 * 2.0**-23)
    again = c.call(dsa)
    assert torch.equal(again[0][2:T - 5], out[2:T - 5]) and torch.equal(again[1][2:T - 5], lse[2:T - 5])
    # a hidden infinity changes nothing, a seen one shows up whichever stretch holds it
    c.kv[1 + lens[0] - 1, 3, 128 + 9] = float("inf")
    c.kv[1 + 65536 + 100, 4, 128 + 10] = float("inf")
    o = c.call(dsa)[0]
    qa, end = 2, 2 + new[0]
    same = torch.ones_like(o[qa:end], dtype=torch.bool)
    same[-1, 3, 9] = False
    same[:, 4, 10] = False
    assert bool((o[qa:end] == out[qa:end])[same].all())
    assert bool(torch.isinf(o[end - 1, 3, 9])) and bool(torch.isinf(o[qa:end, 4, 10]).all())


@pytest.mark.parametrize("sm", [0.9, 1e-4])
def test_sharp_and_flat_softmax(dsa, sm):
    c = Packed(6, [300], [900], 2)
    c.check(*c.call(dsa, sm=sm), sm=sm)
    # keys that grow with their position: the running maximum keeps rising
    c.kv[..., :128] = (c.kv[..., :128].float() * torch.linspace(0.1, 6.0, 900, device="cuda")[:, None, None]).bfloat16()
    c.check(*c.call(dsa, sm=sm), sm=sm)


@pytest.mark.parametrize("m,n", [(300, 300), (130, 1000), (520, 2000), (2, 129)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_what_a_hidden_position_holds_does_not_matter(dsa, m, n, bad):
    c = Packed(7, [m, 5], [n, 5], 2, spare=200)
    clean = c.call(dsa)
    end = int(c.kv_start[-1])
    # rows of no sequence
    c.kv[end:], c.k_rope[end:] = bad, bad
    got = c.call(dsa)
    assert all(torch.equal(a[: m + 5], b[: m + 5]) for a, b in zip(got, clean))
    # a value among the chunk's positions: the queries before it do not see it, the others have it in that column
    p = n - m + m // 2
    c.kv[p, 0, 128 + 5] = bad
    out, lse = c.call(dsa)
    hit = torch.zeros(m + 5, 2, 128, dtype=torch.bool, device="cuda")
    hit[m // 2:m, 0, 5] = True
    assert bool((out[: m + 5] == clean[0][: m + 5])[~hit].all()) and torch.equal(lse[: m + 5], clean[1][: m + 5])
    assert not bool(torch.isfinite(out[: m + 5][hit]).any())
    # a key: NaN for the queries that see it (an infinity may also win the softmax or lose it)
    c.kv[p, 0, 128 + 5] = 0.0
    base = c.call(dsa)
    c.kv[p, 1, 3] = float("nan")
    out, lse = c.call(dsa)
    rows = torch.zeros(m + 5, 2, dtype=torch.bool, device="cuda")
    rows[m // 2:m, 1] = True
    assert bool((out[: m + 5] == base[0][: m + 5]).all(-1)[~rows].all()) and bool(torch.isnan(out[: m + 5][rows]).all())
    # a query row
    c.kv[p, 1, 3] = 0.0
    base = c.call(dsa)
    c.q[1, 0, 0] = bad
    out, _ = c.call(dsa)
    same = (out[: m + 5] == base[0][: m + 5]).all(-1)
    assert not bool(same[1, 0]) and bool(same.view(-1)[torch.arange(2 * (m + 5), device="cuda") != 2].all())


def test_other_layouts(dsa):
    c = Packed(8, [200, 90], [350, 90], 4)
    want = c.call(dsa)
    k, v = c.kv[..., :128].contiguous(), c.kv[..., 128:].contiguous()
    args = (c.k_rope, v, _i32(c.q_start), _i32(c.kv_start))
    got = dsa.dsa_expanded_attn(c.q, k, *args, sm_scale=192**-0.5)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)  # [H][N] in memory
    got = dsa.dsa_expanded_attn(c.q, kt, *args, sm_scale=192**-0.5)
    assert torch.equal(got[0], want[0])
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        got = c.call(dsa, ws=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_longer_sequence_than_announced_is_recorded(dsa):
    c = Packed(9, [10, 20], [600, 900], 2)
    c.call(dsa, max_len=700)
    assert dsa.dsa_get_device_error() == 1
    c.check(*c.call(dsa, max_len=900))


def test_no_queries_and_no_positions(dsa):
    c = Packed(10, [0, 0], [5, 9], 2)
    out, lse = c.call(dsa)
    assert out.shape == (0, 2, 128) and lse.shape == (0, 2)
    c = Packed(11, [3, 140], [0, 0], 2)
    out, lse = c.call(dsa)
    assert bool((out == 0).all()) and bool((lse == -torch.inf).all())


def test_a_captured_call_follows_its_inputs(dsa):
    c = Packed(12, [260, 40], [900, 600], 2)
    qs, ks = _i32(c.q_start), _i32(c.kv_start)
    out, lse = torch.zeros(300, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(300, 2, device="cuda")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")

    def call():
        dsa.dsa_expanded_attn(c.q, c.kv[..., :128], c.k_rope, c.kv[..., 128:], qs, ks, sm_scale=192**-0.5, out=out, lse=lse, ws=ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    c.new, c.lens = np.array([100, 200]), np.array([1000, 333])
    c.q_start, c.kv_start = _starts(c.new), _starts(c.lens)
    qs.copy_(_i32(c.q_start))
    ks.copy_(_i32(c.kv_start))
    g.replay()
    c.check(out, lse)


def test_a_prompt_through_the_whole_expanded_form(dsa):
    # the rows' norm, rotation and append, their expansion, the queries' norm and rotation, attention, together
    T, H = 333, 4
    g = torch.Generator(device="cuda").manual_seed(13)
    latent = torch.randn(T, 576, generator=g, device="cuda").bfloat16()
    q = torch.randn(T, H, 192, generator=g, device="cuda").bfloat16()
    w, pos = weights(H), _i32(np.arange(T))
    freq = torch.from_numpy((10000.0 ** (-np.arange(32) / 32)).astype(np.float32)).cuda()
    kv = torch.zeros(512, 576, dtype=torch.bfloat16, device="cuda")
    table = _i32([[5, 0, 3, 6, 1, 7]])
    p = np.arange(T)
    dst = torch.from_numpy(table.cpu().numpy()[0][p // 64].astype(np.int64) * 64 + p % 64).cuda()
    dsa.dsa_norm_rope_append(latent, pos, freq, kv, dst_rows=dst, norm_dim=512, rot_off=512)
    qt = dsa.dsa_norm_rope(q, pos, freq, rot_off=128)
    start = _i32([0, T])
    kv_exp, rope = dsa.dsa_latent_expand(kv, w, start, rows=T, block_table=table, block_size=64)
    out, lse = dsa.dsa_expanded_attn(qt, kv_exp[..., :128], rope, kv_exp[..., 128:], start, start, sm_scale=192**-0.5)
    # each step from the step before it, as the steps' own tests have it; then the whole against 64 bits throughout
    c = Packed(0, [T], [T], H)
    c.q, c.kv, c.k_rope = qt, kv_exp, rope
    c.check(out, lse)

    def rms(x):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)

    def turn(x):
        a = (torch.arange(T, device="cuda")[:, None].double() * freq.double()).view((T,) + (1,) * (x.dim() - 2) + (32,))
        x0, x1 = x[..., :32], x[..., 32:]
        return torch.cat([x0 * a.cos() - x1 * a.sin(), x1 * a.cos() + x0 * a.sin()], -1)

    x64 = latent.double()
    lat, kr = rms(x64[:, :512]), turn(x64[:, 512:])
    q64 = rms(q.double())
    q64 = torch.cat([q64[..., :128], turn(q64[..., 128:])], -1)
    e = torch.einsum("nc,hjc->nhj", lat, w.double())
    x = (torch.einsum("nhd,lhd->hnl", q64[..., :128], e[..., :128]) + torch.einsum("nhd,ld->hnl", q64[..., 128:], kr)) * 192**-0.5
    x = x.masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
    sm = torch.softmax(x, 2)
    want, A = torch.einsum("hnl,lhd->nhd", sm, e[..., 128:]), torch.einsum("hnl,lhd->nhd", sm, e[..., 128:].abs())
    # bf16 roundings on the way: q, k (of the row and of the expansion) move a logit by at most dl, the values, weights and
    # output by 2^-8 each of A
    G = (torch.einsum("nhd,lhd->hnl", q64[..., :128].abs(), e[..., :128].abs()) + torch.einsum("nhd,ld->hnl", q64[..., 128:].abs(), kr.abs())) * 192**-0.5
    S = torch.einsum("nc,hjc->nhj", lat.abs(), w.double().abs())  # what the rounding of the normed row's values is relative to
    GS = torch.einsum("nhd,lhd->hnl", q64[..., :128].abs(), S[..., :128]) * 192**-0.5
    dl = (2.0**-8 * 2.02 * G + 2.0**-8 * GS).masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1), 0.0).amax(2).t()[..., None]
    AS = torch.einsum("hnl,lhd->nhd", sm, S[..., 128:])
    tol = (torch.expm1(2 * dl) + 3.1 * 2.0**-8) * A + 2.0**-8 * 1.01 * AS
    assert bool(((out.double() - want).abs() <= tol).all())
