"""Host-side checks of the serving-step operators (no GPU): argument refusals before any launch, and
the oracle's pins by hand-worked values and library routines."""
import numpy as np
import pytest
import torch

import oracle

F = 16  # a fake, aligned device address: every call here is refused before it is used


@pytest.fixture(scope="module")
def lib():
    from top_sparse_attention_gb300 import build

    build.build()
    from top_sparse_attention_gb300 import _native

    return _native.lib


# (n_ctx, n_new, n_seq, q_per_seq, block_size, free, n_free, num_free, num_blocks, table, max_blocks, rows,
#  dst_rows, pos, seq, row_start, n_placed, taken, stream)
PLAN = [F, F, 4, 0, 64, F, None, 8, 64, F, 16, 100, F, F, F, F, F, F, None]


@pytest.mark.parametrize("at,value,status", [
    (0, None, 1), (1, None, 1), (9, None, 1), (12, None, 1), (5, None, 1),   # missing arrays
    (2, -1, 1), (3, -1, 1), (4, 0, 1), (7, -1, 1), (8, -1, 1), (10, -1, 1), (11, -1, 1),  # sizes
    (3, 26, 1),           # padded rows do not fit: 4 * 26 > 100
    (2, 16385, 2),        # more sequences than supported
    (10, 1 << 26, 2),     # max_blocks * block_size leaves 31 bits
])
def test_block_plan_refusals(lib, at, value, status):
    args = list(PLAN)
    args[at] = value
    assert lib.dsa_block_plan(*args) == status


def test_block_plan_with_nothing_to_do(lib):
    assert lib.dsa_block_plan(None, None, 0, 0, 64, None, None, 0, 0, None, 0, 0, None, None, None, None, None, None, None) == 0


# (x, row stride, head stride, rows, heads, width, rot_off, rot_dim, pos, n_axes, pair_axis, inv_freq, style,
#  inverse, out, out row stride, out head stride, stream)
ROPE = [F, 1024, 64, 8, 16, 64, 0, 64, F, 1, None, F, 0, 0, 4096, 1024, 64, None]
# (x, row stride, rows, width, rot_off, rot_dim, pos, n_axes, pair_axis, inv_freq, style, dtype, dst, dst row
#  bytes, dst_count, scale, dst_rows, stream)
APPEND = [F, 576, 8, 576, 512, 64, F, 1, None, F, 0, 1, F, 576, 100, F, F, None]


@pytest.mark.parametrize("at,value,status", [
    (0, None, 1), (8, None, 1), (11, None, 1), (14, None, 1), (0, 17, 1), (14, 17, 1),
    (3, -1, 1), (4, 0, 1), (5, 0, 1), (6, -1, 1), (6, 8, 1), (7, 0, 1), (7, 63, 1), (9, 0, 1),
    (9, 2, 1),            # two axes without a table
    (9, 5, 2), (12, 2, 1),
    (1, 32, 1), (2, 32, 1), (15, 32, 1), (16, 0, 1),     # rows or heads that overlap
])
def test_rope_refusals(lib, at, value, status):
    args = list(ROPE)
    args[at] = value
    assert lib.dsa_rope(*args) == status


def test_rope_refuses_other_combinations(lib):
    args = list(ROPE)
    args[5], args[2], args[16], args[7] = 512, 512, 512, 258   # more than 128 pairs
    args[1] = args[15] = 16 * 512
    assert lib.dsa_rope(*args) == 2
    args = list(ROPE)
    args[9], args[10] = 2, bytes([0] * 31 + [2])               # an axis that does not exist
    assert lib.dsa_rope(*args) == 1
    args = list(ROPE)
    args[14], args[15] = args[0], 2048                         # in place under another layout
    assert lib.dsa_rope(*args) == 1
    args = list(ROPE)
    args[3], args[0], args[8] = 0, None, None                  # no rows
    assert lib.dsa_rope(*args) == 0


@pytest.mark.parametrize("at,value,status", [
    (0, None, 1), (6, None, 1), (9, None, 1), (12, None, 1), (15, None, 1), (0, 17, 1), (15, 18, 1),
    (2, -1, 1), (3, 0, 1), (4, 520, 1), (5, 62 + 3, 1), (11, 9, 2), (13, 575, 1), (14, -1, 1), (1, 500, 1),
    (14, 4, None),
])
def test_rope_append_refusals(lib, at, value, status):
    args = list(APPEND)
    args[at] = value
    if status is None:  # fewer destination rows than rows, without a list of them
        args[16], status = None, 1
    assert lib.dsa_rope_append(*args) == status


def test_rope_append_mxfp8_needs_whole_groups(lib):
    args = list(APPEND)
    args[11], args[3], args[4], args[5] = 2, 120, 56, 64
    assert lib.dsa_rope_append(*args) == 1


def test_python_refuses_host_tensors_and_wrong_types():
    import top_sparse_attention_gb300 as dsa

    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_block_plan(i, i, i, i.view(2, 1), block_size=64, num_blocks=2, rows=2)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_rope(torch.zeros(2, 64, dtype=torch.bfloat16), i, torch.zeros(32))
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_rope_append(torch.zeros(2, 64, dtype=torch.bfloat16), i, torch.zeros(32),
                            torch.zeros(2, 64, dtype=torch.bfloat16), rot_off=0)


# ---------------------------------------------------------------------------------------------
# pins of the oracle

def test_oracle_block_plan_by_hand():
    # blocks of 4; sequence 0 has 3 of 4 positions used and adds 3 (one new block), sequence 1 is full
    # at 4 and adds 1 (one), sequence 2 adds none, sequence 3 is new and adds 5 (two: one block too many)
    table = np.array([[7, -1], [5, -1], [6, -1], [-1, -1]])
    got = oracle.block_plan([3, 4, 2, 0], [3, 1, 0, 5], [9, 8, 3], table, block_size=4, num_blocks=10, rows=10)
    assert got["dst_rows"].tolist() == [7 * 4 + 3, 36, 37, 32, -1, -1, -1, -1, -1, -1]
    assert got["pos"].tolist() == [3, 4, 5, 4] + [-1] * 6
    assert got["row_start"].tolist() == [0, 3, 4, 4, 9] and got["n_placed"].tolist() == [3, 1, 0, 0]
    assert got["taken"].tolist() == [2] and not got["ok"]
    assert got["table"].tolist() == [[7, 9], [5, 8], [6, -1], [-1, -1]]


def test_oracle_rotation_by_hand_and_as_complex_numbers():
    y = oracle.rotate([[3.0, 4.0]], [1], [np.pi / 2], rot_off=0, rot_dim=2)
    np.testing.assert_allclose(y, [[-4.0, 3.0]], atol=1e-15)
    rng = np.random.default_rng(0)
    x, pos, f = rng.standard_normal((5, 3, 12)), rng.integers(0, 100, (5, 2)), rng.random(4)
    axis = [0, 1, 1, 0]
    for style in ("half", "pairs"):
        y = oracle.rotate(x, pos, f, rot_off=2, rot_dim=8, pair_axis=axis, style=style)
        theta = pos[:, axis] * f
        r = x[..., 2:10]
        z = r[..., :4] + 1j * r[..., 4:] if style == "half" else r[..., 0::2] + 1j * r[..., 1::2]
        z = z * np.exp(1j * theta)[:, None]
        want = np.concatenate([z.real, z.imag], -1) if style == "half" else np.stack([z.real, z.imag], -1).reshape(r.shape)
        np.testing.assert_allclose(y[..., 2:10], want, atol=1e-12)
        np.testing.assert_array_equal(y[..., :2], x[..., :2])
        np.testing.assert_array_equal(y[..., 10:], x[..., 10:])
        back = oracle.rotate(y, pos, f, rot_off=2, rot_dim=8, pair_axis=axis, style=style, inverse=True)
        np.testing.assert_allclose(back, x, atol=1e-12)


def test_oracle_tree_attention_is_masked_attention():
    rng = np.random.default_rng(1)
    N, H, D, DV, c, m = 5, 3, 24, 16, 11, 4
    q, rows = rng.standard_normal((N, H, D)), rng.standard_normal((c + N, D))
    sees = np.tril(rng.random((N, N)) < 0.5) | np.eye(N, dtype=bool)
    out, lse = oracle.tree_attention(q, rows, c, m, sees, 0.2, DV)
    mask = np.zeros((N, c + m), bool)
    mask[:, :c] = True
    mask[:, c:] = sees[:, :m]
    t = torch.from_numpy
    want = torch.nn.functional.scaled_dot_product_attention(
        t(q).transpose(0, 1), t(rows[: c + m]).expand(H, -1, -1), t(rows[: c + m, :DV]).expand(H, -1, -1),
        attn_mask=t(mask)[None], scale=0.2).transpose(0, 1)
    np.testing.assert_allclose(out[:m], want.numpy()[:m], atol=1e-12)
    assert np.all(out[m:] == 0) and np.all(lse[m:] == -np.inf)
    # no context and an empty mask row: nothing is seen
    out, lse = oracle.tree_attention(q, rows, 0, N, np.zeros((N, N), bool), 0.2, DV)
    assert np.all(out == 0) and np.all(lse == -np.inf)


# ---------------------------------------------------------------------------------------------
# tree attention: refusals, and the argument struct

def _tree_args(**kw):
    from top_sparse_attention_gb300 import _native as N

    a = N.DsaTreeArgs()
    base = dict(n_seq=2, q_per_seq=4, L=128, H=16, D_qk=576, D_v=512, sm_scale=0.04, kv_dtype=0, n_ctx=F, q=F, kv=F, out=F,
                kv_row_stride=1152, kv_seq_stride=1152 * 128)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(n_seq=-1), 1), (dict(q_per_seq=0), 1), (dict(L=-1), 1), (dict(H=0), 1), (dict(n_ctx=None), 1), (dict(q=None), 1),
    (dict(out=None), 1), (dict(kv=None), 1), (dict(q=24), 1), (dict(kv=24), 1), (dict(out=24), 1),
    (dict(D_qk=512), 2), (dict(D_v=256), 2), (dict(H=129), 2), (dict(q_per_seq=1025), 2), (dict(n_seq=4097), 2), (dict(kv_dtype=2), 2),
    (dict(kv_row_stride=1 << 40, kv_seq_stride=1 << 48), 2), (dict(n_seq=2, kv_seq_stride=1 << 40), 2),
    (dict(kv_row_stride=1150), 1), (dict(kv_row_stride=1136), 1), (dict(kv_seq_stride=1000), 1),
    (dict(kv_dtype=1, kv_row_stride=576, kv_seq_stride=576 * 128), 1),       # no scales
    (dict(block_table=F, block_size=48, max_blocks=4, num_blocks=8), 1), (dict(block_table=F, block_size=64, max_blocks=1, num_blocks=8), 1),
    (dict(block_table=F, block_size=64, max_blocks=2, num_blocks=0), 1), (dict(block_table=F, block_size=64, max_blocks=2, num_blocks=1 << 25), 2),
])
def test_tree_attn_refusals(lib, kw, status):
    import ctypes

    a, n = _tree_args(**kw), ctypes.c_size_t(0)
    assert lib.dsa_tree_attn_workspace_size(ctypes.byref(a), ctypes.byref(n)) == status
    assert lib.dsa_tree_attn(ctypes.byref(a), F, 1 << 40, None) == status


def test_tree_attn_nothing_to_do_and_missing_arguments(lib):
    import ctypes

    a, n = _tree_args(n_seq=0, n_ctx=None, q=None, kv=None, out=None), ctypes.c_size_t(7)
    assert lib.dsa_tree_attn_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value == 0
    assert lib.dsa_tree_attn(ctypes.byref(a), None, 0, None) == 0
    assert lib.dsa_tree_attn(None, None, 0, None) == 1
    assert lib.dsa_tree_attn_workspace_size(ctypes.byref(a), None) == 1


def test_tree_args_layout_matches_c(tmp_path, lib):
    import ctypes
    import os
    import subprocess

    from top_sparse_attention_gb300 import _native as N

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [f for f, _ in N.DsaTreeArgs._fields_]
    body = "\n".join(f'  printf("%zu\\n", offsetof(dsa_tree_args, {f}));' for f in fields)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dsa.h"\nint main(void){\n'
                   f'  printf("%zu\\n", sizeof(dsa_tree_args));\n{body}\n  return 0;\n}}\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o",
                    str(tmp_path / "layout")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(N.DsaTreeArgs)] + [getattr(N.DsaTreeArgs, f).offset for f in fields]


def test_tree_attn_workspace_holds_accumulators_of_long_contexts(lib):
    import ctypes

    def size(**kw):
        a, n = _tree_args(**kw), ctypes.c_size_t(0)
        assert lib.dsa_tree_attn_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
        return n.value

    def contiguous(L, n_seq, **kw):
        return size(L=L, n_seq=n_seq, kv_seq_stride=1152 * L, **kw)

    # up to 1024 tiles of 64 positions: partial results only, and those only where row tiles are split
    row = 128 * (2 * 8 + 512 * 4)
    parts = contiguous(65536, 2)
    assert parts >= 228 * row and contiguous(64, 2) == parts and contiguous(65536, 609) == 0
    # beyond: 128 rows of sums, half of the values, for each of 152 CTAs
    sums = 152 * 128 * (2 * 8 + 256 * 4)
    assert contiguous(65537, 2) == parts + sums
    assert contiguous(65537, 609) == sums
    a = _tree_args(L=65537, n_seq=609, kv_seq_stride=1152 * 65537)
    assert lib.dsa_tree_attn(ctypes.byref(a), None, 0, None) == 3  # workspace
    assert lib.dsa_tree_attn(ctypes.byref(a), F, sums - 1, None) == 3


@pytest.mark.parametrize("sections,ok", [((16, 16), True), ((0, 32), True), ((32, 0), True), ((-8, 32), False), ((32, -1), False),
                                         ((40, -8), False), ((16, 15), False), ((32,), False)])
def test_sections_are_numbers_of_pairs(sections, ok):
    # a negative count used to be taken for none: (-8, 32) turned all 32 pairs by the second axis
    from top_sparse_attention_gb300 import api

    x, pos, f = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(32)
    args = ("dsa_rope", x.device, x, pos, f, 0, None, sections, None, "half")
    if ok:
        assert api._rope_args(*args)[2] == b"\0" * sections[0] + b"\1" * sections[1]
    else:
        with pytest.raises(ValueError):
            api._rope_args(*args)
