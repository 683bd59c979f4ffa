"""GPU parity of dsa_prefix_attn with the oracle (fp64): groups of sequences with a shared prefix, over every cache format
and layout.  Tolerances are those of the attention of drafted tokens (test_gpu_tree.py): the sums are the same ones, split
elsewhere."""
import numpy as np
import pytest
import torch

from test_gpu_tree import FORMATS, Case, _i32, dsa  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu


def share(c, group_start, n_shared):
    """Makes the first n_shared[g] positions of every sequence of group g the same rows as its first sequence's."""
    c.group_start, c.n_shared = np.asarray(group_start), np.asarray(n_shared)
    for g, m in enumerate(c.n_shared):
        lo, hi = int(c.group_start[g]), int(c.group_start[g + 1])
        for s in range(lo + 1, hi):
            m_s = min(max(int(m), 0), max(int(c.ctx[s]), 0), max(int(c.ctx[lo]), 0), c.L)
            if c.block:  # whole blocks by the table, the rest of the last one as a copy
                c.table[s, : m_s // c.block] = c.table[lo, : m_s // c.block]
            at = [(c.row_of(s, p), c.row_of(lo, p)) for p in range(m_s) if c.row_of(s, p) != c.row_of(lo, p)]
            if at:
                to, frm = np.array(at).T
                c.val[to] = c.val[frm]
                to, frm = torch.from_numpy(to).cuda(), torch.from_numpy(frm).cuda()
                c.cache[to] = c.cache[frm]
                if c.scale is not None:
                    c.scale[to] = c.scale[frm]
    return c


def call(dsa, c, sm_scale=1 / 24, **kw):  # noqa: F811
    kv, scale = c.cache, c.scale
    if not c.block:
        kv = kv.unflatten(0, (c.n, c.L))
        scale = None if scale is None else scale.unflatten(0, (c.n, c.L))
    args = dict(sm_scale=sm_scale, q_per_seq=c.N, n_new=_i32(c.new), tree_mask=c.mask, kv_scale=scale, group_start=_i32(c.group_start),
                n_shared=_i32(c.n_shared), block_table=_i32(c.table) if c.block else None, block_size=c.block, L=c.L if c.block else None)
    args.update(kw)
    return dsa.dsa_prefix_attn(c.q, kv, _i32(c.ctx), **args)


def run(dsa, c, nodes=None, **kw):  # noqa: F811
    out, lse = call(dsa, c, **kw)
    c.check(out, lse, 1 / 24, nodes)
    return out, lse


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("block", [0, 64, 192])
def test_two_groups_and_a_sequence_of_its_own(dsa, kv, block):  # noqa: F811
    c = Case(1, [300, 257, 264, 64, 500, 450], 3, 16, kv, block)
    run(dsa, share(c, [0, 3, 4, 6], [257, 64, 449]))


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("N,H,n", [(1, 1, 2), (1, 16, 9), (1, 128, 3), (2, 5, 13), (5, 20, 4), (9, 16, 2), (33, 4, 3), (1, 3, 100)])
def test_nodes_heads_and_row_tiles(dsa, kv, N, H, n):  # noqa: F811
    rng = np.random.default_rng(N * H)
    c = Case(N * H + n, 700 + rng.integers(0, 200, n), N, H, kv, 0 if N % 2 else 64)
    run(dsa, share(c, [0, n], [700]))


@pytest.mark.parametrize("shared", [0, 1, 63, 64, 65, 127, 128, 320, 5000, -7])
def test_shared_lengths(dsa, shared):  # noqa: F811
    # beyond the contexts: clamped to the shortest; a whole context may be shared
    c = Case(3, [320, 400, 321], 4, 16, "bf16", 64)
    run(dsa, share(c, [0, 3], [shared]))


@pytest.mark.parametrize("kv", FORMATS)
def test_sequences_without_queries_have_no_say(dsa, kv):  # noqa: F811
    # sequences 0 and 3 hold nothing and ask nothing: the group's prefix is the others', read from sequence 1
    c = Case(4, [0, 400, 390, 0, 410], 4, 16, kv, 64, new=[0, 4, 2, 0, 3])
    c.group_start, c.n_shared = np.array([0, 5]), np.array([384])
    for s in (2, 4):
        c.table[s, :6] = c.table[1, :6]
    c.table[0], c.table[3] = 1 << 24, -1  # (their blocks are not looked at)
    run(dsa, c)


def test_groups_of_one_of_none_and_gaps(dsa):  # noqa: F811
    c = Case(5, [200, 130, 0, 64, 90, 70], 2, 16, "bf16")
    run(dsa, share(c, [1, 2, 2, 5], [130, 9, 64]))
    run(dsa, share(c, [6, 6], [4]))
    c.group_start, c.n_shared = np.array([0]), np.zeros(0, int)
    run(dsa, c)


@pytest.mark.parametrize("mask", ["chain", "any", "tree"])
def test_masks_of_drafted_tokens(dsa, mask):  # noqa: F811
    c = Case(6, [130, 191, 128, 150], 40, 3, "bf16", 64, mask=mask, new=[40, 39, 7, 1])
    run(dsa, share(c, [0, 4], [128]))


@pytest.mark.parametrize("kv", FORMATS)
def test_long_prefixes_are_split_and_merged(dsa, kv):  # noqa: F811
    rng = np.random.default_rng(7)
    c = Case(7, 6000 + rng.integers(0, 300, 12), 2, 16, kv, 64)
    run(dsa, share(c, [0, 7, 12], [5950, 6000]))
    # many groups of different lengths, more units of work than pairs of CTAs
    n = 160
    ctx = 64 + rng.integers(0, 400, n)
    c = Case(8, ctx, 1, 16, kv, 64)
    start = np.concatenate([[0], np.sort(rng.choice(np.arange(1, n), 40, replace=False)), [n]])
    run(dsa, share(c, start, rng.integers(0, 400, 41)))


def test_contexts_in_caches_longer_than_65536(dsa):  # noqa: F811
    # the form whose walks are broken into stretches: two sequences' tables name the same blocks again and again
    times = 700
    c = Case(9, [128 * times + 70, 128 * times + 9], 2, 4, "bf16", 64, L=128 * times + 128)
    c.table[1, : 2 * times] = c.table[0, : 2 * times] = np.tile(c.table[0, :2], times)
    c.group_start, c.n_shared = np.array([0, 2]), np.array([128 * times])
    run(dsa, c, nodes=[1])


def test_agrees_with_the_sequences_alone_and_repeats(dsa):  # noqa: F811
    c = share(Case(10, [3000, 3100, 3050], 4, 16, "bf16", 64), [0, 3], [2944])
    out, lse = call(dsa, c)
    alone, alone_lse = c.call(dsa, 1 / 24)
    # (both are within their tolerance of the truth; with logits and values of a few units that is well below this)
    assert float((out.float() - alone.float()).abs().max()) < 2e-2 and float((lse - alone_lse).abs().max()) < 1e-3
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda").random_(0, 256)
    for _ in range(3):
        again = call(dsa, c, ws=ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("kv", FORMATS)
def test_hidden_rows_do_not_matter(dsa, kv):  # noqa: F811
    c = share(Case(11, [200, 150, 190], 4, 16, kv, 64, new=[4, 2, 1], L=256), [0, 3], [150])
    used = [c.row_of(s, p) for s in range(3) for p in range(int(c.ctx[s] + c.new[s]))]
    rest = torch.from_numpy(np.setdiff1d(np.arange(c.rows), used)).cuda()
    c.cache[rest] = float("nan") if kv == "bf16" else 0x7F
    if c.scale is not None:
        c.scale[rest] = float("nan")
    run(dsa, c)


def test_a_block_outside_the_pool_is_recorded(dsa):  # noqa: F811
    c = share(Case(12, [200, 210], 1, 16, "bf16", 64), [0, 2], [192])
    c.table[0, 1] = 1 << 20  # of the prefix, read from sequence 0: its positions are not seen
    out, _ = call(dsa, c)
    assert dsa.dsa_get_device_error() == 1
    assert bool(torch.isfinite(out).all())


def test_without_node_counts_on_another_stream_and_captured(dsa):  # noqa: F811
    c = share(Case(13, [500, 520], 2, 16, "fp8"), [0, 2], [450])
    want = run(dsa, c, n_new=None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(dsa, c, n_new=None, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0])
    gs, ns, ctx = _i32([0, 2]), _i32([450]), _i32(c.ctx)
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    kv, scale = c.cache.unflatten(0, (2, c.L)), c.scale.unflatten(0, (2, c.L))

    def step():
        dsa.dsa_prefix_attn(c.q, kv, ctx, sm_scale=1 / 24, q_per_seq=2, kv_scale=scale, group_start=gs, n_shared=ns, tree_mask=c.mask,
                            out=out, lse=lse, ws=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    c.ctx, c.n_shared = np.array([460, 333]), np.array([200])
    c.new[:] = 2
    share(c, [0, 2], [200])
    ctx.copy_(_i32(c.ctx))
    ns.copy_(_i32([200]))
    g.replay()
    c.check(out, lse, 1 / 24)
