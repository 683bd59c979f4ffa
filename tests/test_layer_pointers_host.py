"""Host-side checks (no GPU): device pointers that a kernel reads as 4- or 8-byte words are refused where they lie between those, before
any launch."""
import ctypes

import pytest

from test_layer_host import APPEND, F, ROPE, attn_args, expand, native, norm, tree  # noqa: F401  (native: the fixture)


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("field", ["q_start", "kv_start", "lse"])
def test_expanded_attn(native, field, off):  # noqa: F811
    n = ctypes.c_size_t(0)
    a = attn_args(native, **{field: F + off})
    assert native.lib.dsa_expanded_attn(a, F, 1 << 40, None) == 1
    assert native.lib.dsa_expanded_attn_workspace_size(a, ctypes.byref(n)) == 1
    b = attn_args(native, **{field: F + 4})  # (4-byte aligned ones are taken)
    assert native.lib.dsa_expanded_attn_workspace_size(b, ctypes.byref(n)) == 0


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("field", ["kv_start", "block_table"])
def test_expand(native, field, off):  # noqa: F811
    paged = dict(block_table=F, block_size=64, max_blocks=1, num_blocks=4)
    assert expand(native, **{**paged, field: F + off}) == 1


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("at", [0, 1])
def test_prefix(native, at, off):  # noqa: F811
    groups = [F, F, 1]
    groups[at] += off
    n = ctypes.c_size_t(0)
    assert native.lib.dsa_prefix_attn_workspace_size(tree(native), *groups, ctypes.byref(n)) == 1
    assert native.lib.dsa_prefix_attn(tree(native), *groups, F, 1 << 40, None) == 1
    groups[at] += 4 - off
    assert native.lib.dsa_prefix_attn_workspace_size(tree(native), *groups, ctypes.byref(n)) == 0


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("at", [9, 12])  # pos, inv_freq
def test_norm_rope(native, at, off):  # noqa: F811
    args = list(ROPE)
    args[6] = norm(native)
    args[at] = F + off
    assert native.lib.dsa_norm_rope(*args) == 1


@pytest.mark.parametrize("at,off", [(7, 1), (7, 2), (10, 2), (10, 3), (17, 1), (17, 2), (17, 4)])  # pos, inv_freq, dst_rows
def test_norm_rope_append(native, at, off):  # noqa: F811
    args = list(APPEND)
    args[4] = norm(native, dim=512)
    args[at] = F + off
    assert native.lib.dsa_norm_rope_append(*args) == 1


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("field", ["n_ctx", "n_new", "tree_mask", "lse", "kv_scale", "block_table"])
def test_tree(native, field, off):  # noqa: F811
    n = ctypes.c_size_t(0)
    paged = dict(kv_dtype=1, kv_scale=F, block_table=F, block_size=64, max_blocks=4, num_blocks=4)
    assert native.lib.dsa_tree_attn_workspace_size(tree(native, **{**paged, field: F + 4}), ctypes.byref(n)) == 0
    assert native.lib.dsa_tree_attn_workspace_size(tree(native, **{**paged, field: F + off}), ctypes.byref(n)) == 1
    assert native.lib.dsa_tree_attn(tree(native, **{**paged, field: F + off}), F, 1 << 40, None) == 1


@pytest.mark.parametrize("at,off", [(8, 1), (8, 2), (11, 3)])  # pos, inv_freq
def test_rope(native, at, off):  # noqa: F811
    args = [F, 1024, 64, 8, 16, 64, 0, 64, F, 1, None, F, 0, 0, 8192, 1024, 64, None]
    args[at] = F + off
    assert native.lib.dsa_rope(*args) == 1


@pytest.mark.parametrize("at,off", [(6, 1), (6, 2), (9, 3), (16, 4)])  # pos, inv_freq, dst_rows
def test_rope_append(native, at, off):  # noqa: F811
    args = [F, 576, 8, 576, 512, 64, F, 1, None, F, 0, 1, F, 576, 100, F, F, None]
    args[at] = F + off
    assert native.lib.dsa_rope_append(*args) == 1
