"""Host-side checks of the latent-layer operators (no GPU): argument refusals before any launch, struct layouts, and what the
Python entries refuse."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = 4096  # a fake, aligned device address: every call here is refused before it is used


@pytest.fixture(scope="module")
def native():
    from top_sparse_attention_gb300 import build

    build.build()
    from top_sparse_attention_gb300 import _native

    return _native


@pytest.mark.parametrize("name,struct", [("DsaNorm", "dsa_norm"), ("DsaExpandArgs", "dsa_expand_args"),
                                         ("DsaExpandedAttnArgs", "dsa_expanded_attn_args"), ("DsaTreeArgs", "dsa_tree_args")])
def test_struct_layouts_match_c(tmp_path, native, name, struct):
    cls = getattr(native, name)
    fields = [f for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    body = "\n".join(f'  printf("{f} %zu\\n", offsetof({struct}, {f}));' for f in fields)
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dsa.h"\nint main(void){\n'
                   f'  printf("sizeof %zu\\n", sizeof({struct}));\n{body}\n  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n") if line)
    assert int(got["sizeof"]) == ctypes.sizeof(cls)
    for f in fields:
        assert int(got[f]) == getattr(cls, f).offset, f


def norm(native, **kw):
    a = dict(kind=0, off=0, dim=64, eps=1e-6, weight=F, bias=None)
    a.update(kw)
    return ctypes.byref(native.DsaNorm(*(a[f] for f, _ in native.DsaNorm._fields_)))


# (x, row stride, head stride, rows, heads, width, norm, rot_off, rot_dim, pos, n_axes, pair_axis, inv_freq, style, out, out row stride,
#  out head stride, stream)
ROPE = [F, 1024, 64, 8, 16, 64, None, 0, 64, F, 1, None, F, 0, 8192, 1024, 64, None]
# (x, row stride, rows, width, norm, rot_off, rot_dim, pos, n_axes, pair_axis, inv_freq, style, dtype, dst, dst row bytes, dst_count, scale,
#  dst_rows, stream)
APPEND = [F, 576, 8, 576, None, 512, 64, F, 1, None, F, 0, 1, F, 576, 100, F, F, None]

NORMS = [(dict(kind=2), 1), (dict(kind=-1), 1), (dict(off=-1), 1), (dict(dim=0), 1), (dict(off=1), 1), (dict(dim=65), 1), (dict(eps=-1e-9), 1),
         (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(weight=F + 2), 1), (dict(bias=F + 1), 1)]


@pytest.mark.parametrize("kw,status", NORMS)
def test_norm_refusals(native, kw, status):
    args = list(ROPE)
    args[6] = norm(native, **kw)
    assert native.lib.dsa_norm_rope(*args) == status
    args = list(APPEND)
    args[3], args[1], args[5], args[6] = 64, 64, 0, 64
    args[4] = norm(native, **kw)
    assert native.lib.dsa_norm_rope_append(*args) == status


@pytest.mark.parametrize("at,value,status", [
    (0, None, 1), (6, None, 1), (9, None, 1), (12, None, 1), (14, None, 1), (0, F + 1, 1), (14, 8193, 1),
    (3, -1, 1), (4, 0, 1), (5, 0, 1), (7, -1, 1), (7, 8, 1), (8, 0, 1), (8, 63, 1), (10, 0, 1), (10, 2, 1), (10, 5, 2), (13, 2, 1),
    (1, 32, 1), (2, 32, 1), (15, 32, 1), (16, 0, 1),     # rows or heads that overlap
])
def test_norm_rope_refusals(native, at, value, status):
    args = list(ROPE)
    args[6] = norm(native)
    args[at] = value
    assert native.lib.dsa_norm_rope(*args) == status


def test_norm_rope_refuses_other_combinations(native):
    args = list(ROPE)
    args[6], args[5], args[1], args[2], args[15], args[16] = norm(native, dim=1025), 1025, 16 * 1025, 1025, 16 * 1025, 1025
    assert native.lib.dsa_norm_rope(*args) == 2                # wider than supported
    args = list(ROPE)
    args[6], args[14], args[15] = norm(native), F, 2048       # in place under another layout
    assert native.lib.dsa_norm_rope(*args) == 1
    args = list(ROPE)
    args[6], args[3], args[0], args[9] = norm(native), 0, None, None  # no rows
    assert native.lib.dsa_norm_rope(*args) == 0


@pytest.mark.parametrize("at,value,status", [
    (0, None, 1), (4, None, 1), (7, None, 1), (10, None, 1), (13, None, 1), (16, None, 1), (0, F + 1, 1), (16, F + 2, 1),
    (2, -1, 1), (3, 0, 1), (5, 520, 1), (6, 63, 1), (12, 9, 2), (14, 575, 1), (15, -1, 1), (1, 500, 1), (15, 4, None),
])
def test_norm_rope_append_refusals(native, at, value, status):
    args = list(APPEND)
    args[4] = norm(native, dim=512)
    args[at] = value
    if status is None:  # fewer destination rows than rows, without a list of them
        args[17], status = None, 1
    assert native.lib.dsa_norm_rope_append(*args) == status


def expand(native, **kw):
    a = native.DsaExpandArgs(n_seq=2, rows=100, L=64, H=4, kv_dtype=0, kv_start=F, kv=F, kv_scale=None, kv_row_stride=1152, kv_seq_stride=64 * 1152,
                             w=F, out=F, rope_out=F)
    for k, v in kw.items():
        setattr(a, k, v)
    return native.lib.dsa_latent_expand(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_seq=-1), 1), (dict(rows=-1), 1), (dict(L=-1), 1), (dict(H=0), 1), (dict(H=129), 2), (dict(n_seq=4097), 2), (dict(kv_dtype=2), 2),
    (dict(kv_dtype=7), 2), (dict(kv_start=None), 1), (dict(kv=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(kv=F + 8), 1),
    (dict(w=F + 8), 1), (dict(out=F + 8), 1), (dict(rope_out=F + 8), 1), (dict(kv_row_stride=1144), 1), (dict(kv_row_stride=1136), 1),
    (dict(kv_seq_stride=63 * 1152), 1), (dict(kv_seq_stride=64 * 1152 + 8), 1), (dict(kv_dtype=1), 1),
    (dict(kv_dtype=1, kv_scale=F + 2, kv_row_stride=576), 1), (dict(kv_dtype=3, kv_scale=F, kv_row_stride=560), 1),
    (dict(block_table=F, block_size=0, max_blocks=1, num_blocks=4), 1), (dict(block_table=F, block_size=96, max_blocks=1, num_blocks=4), 1),
    (dict(block_table=F, block_size=64, max_blocks=0, num_blocks=4), 1), (dict(block_table=F, block_size=64, max_blocks=1, num_blocks=0), 1),
    (dict(block_table=F, block_size=64, max_blocks=1, num_blocks=1 << 25), 2), (dict(L=2**31 - 1), 2),
    (dict(n_seq=0, kv=None), 0), (dict(rows=0, out=None), 0),
])
def test_expand_refusals(native, kw, status):
    assert expand(native, **kw) == status


def attn_args(native, **kw):
    a = native.DsaExpandedAttnArgs(n_seq=2, T=100, N=200, H=4, max_len=0, causal=1, sm_scale=0.07, q_start=F, kv_start=F, q=F, k=F, k_rope=F, v=F,
                                   k_row_stride=1024, k_head_stride=256, v_row_stride=1024, v_head_stride=256, out=F, lse=F)
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


REFUSED = [
    (dict(n_seq=-1), 1), (dict(T=-1), 1), (dict(N=-1), 1), (dict(H=0), 1), (dict(max_len=-1), 1), (dict(sm_scale=0.0), 1), (dict(sm_scale=-1.0), 1),
    (dict(sm_scale=float("nan")), 1), (dict(sm_scale=float("inf")), 1), (dict(H=129), 2), (dict(n_seq=4097), 2), (dict(T=1 << 24), 2),
    (dict(N=1 << 24), 2), (dict(q_start=None), 1), (dict(kv_start=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(k_rope=None), 1),
    (dict(v=None), 1), (dict(out=None), 1), (dict(q=F + 8), 1), (dict(k=F + 8), 1), (dict(v=F + 8), 1), (dict(k_rope=F + 8), 1), (dict(out=F + 8), 1),
    (dict(k_row_stride=1020), 1), (dict(v_head_stride=64), 1), (dict(k_head_stride=0), 1), (dict(v_row_stride=1 << 39), 2),
]


@pytest.mark.parametrize("kw,status", REFUSED)
def test_expanded_attn_refusals(native, kw, status):
    n = ctypes.c_size_t(0)
    assert native.lib.dsa_expanded_attn_workspace_size(attn_args(native, **kw), ctypes.byref(n)) == status
    assert native.lib.dsa_expanded_attn(attn_args(native, **kw), F, 1 << 40, None) == status


def test_expanded_attn_workspaces(native):
    lib, n = native.lib, ctypes.c_size_t(0)
    assert lib.dsa_expanded_attn_workspace_size(attn_args(native), None) == 1
    assert lib.dsa_expanded_attn_workspace_size(attn_args(native), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.dsa_expanded_attn(attn_args(native), None, n.value, None) == 3
    assert lib.dsa_expanded_attn(attn_args(native), F, n.value - 1, None) == 3
    assert lib.dsa_expanded_attn(attn_args(native), F + 16, n.value, None) == 3
    for kw in (dict(n_seq=0), dict(T=0)):
        assert lib.dsa_expanded_attn_workspace_size(attn_args(native, **kw), ctypes.byref(n)) == 0 and n.value == 0
        assert lib.dsa_expanded_attn(attn_args(native, **kw), None, 0, None) == 0
    # partial results: two for each SM at most, and one of blocks in stretches where contexts may be longer than 65536 positions
    sizes = []
    for kw in (dict(T=8192, N=8192, n_seq=1, H=16), dict(T=1 << 23, N=1 << 23, n_seq=1, H=128), dict(T=8192, N=131072, n_seq=4, H=16, max_len=65536)):
        assert lib.dsa_expanded_attn_workspace_size(attn_args(native, **kw), ctypes.byref(n)) == 0
        sizes.append(n.value)
    assert sizes[0] < 50 << 20 and sizes[1] < 80 << 20 and sizes[2] < 50 << 20


def tree(native, **kw):
    a = native.DsaTreeArgs(n_seq=4, q_per_seq=2, L=256, H=16, D_qk=576, D_v=512, sm_scale=0.04, kv_dtype=0, n_ctx=F, n_new=F, tree_mask=None, q=F, kv=F,
                           kv_row_stride=1152, kv_seq_stride=256 * 1152, out=F, lse=F)
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


@pytest.mark.parametrize("kw,groups,status", [
    ({}, (None, F, 1), 1), ({}, (F, None, 1), 1), ({}, (F, F, -1), 1), ({}, (F, F, 4097), 2), (dict(n_ctx=None), (F, F, 1), 1),
    (dict(q=F + 8), (F, F, 1), 1), (dict(D_qk=64), (F, F, 1), 2), (dict(H=129), (F, F, 1), 2), (dict(kv_row_stride=1100), (F, F, 1), 1),
    (dict(n_seq=4096, q_per_seq=1024, H=128), (F, F, 1), 2),                      # more rows than supported
    (dict(n_seq=4096, q_per_seq=8, H=128, L=1 << 30, kv_seq_stride=1152 << 30), (F, F, 1), 2),  # costs beyond 31 bits
])
def test_prefix_refusals(native, kw, groups, status):
    n = ctypes.c_size_t(0)
    assert native.lib.dsa_prefix_attn_workspace_size(tree(native, **kw), *groups, ctypes.byref(n)) == status
    assert native.lib.dsa_prefix_attn(tree(native, **kw), *groups, F, 1 << 40, None) == status


def test_prefix_workspaces(native):
    lib, n = native.lib, ctypes.c_size_t(0)
    assert lib.dsa_prefix_attn_workspace_size(tree(native), F, F, 1, None) == 1
    assert lib.dsa_prefix_attn_workspace_size(tree(native), F, F, 1, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.dsa_prefix_attn(tree(native), F, F, 1, None, n.value, None) == 3
    assert lib.dsa_prefix_attn(tree(native), F, F, 1, F, n.value - 1, None) == 3
    assert lib.dsa_prefix_attn(tree(native), F, F, 1, F + 16, n.value, None) == 3
    assert lib.dsa_prefix_attn_workspace_size(tree(native, n_seq=0), F, F, 1, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.dsa_prefix_attn(tree(native, n_seq=0), F, F, 1, None, 0, None) == 0


def test_python_refuses_host_tensors_and_wrong_arguments():
    import top_sparse_attention_gb300 as dsa

    i, x, f = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(32)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_norm_rope(x, i, f)
    with pytest.raises(ValueError, match="norm must be"):
        dsa.dsa_norm_rope(x, i, f, norm="l2")
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_norm_rope_append(x, i, f, x, rot_off=0)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_latent_expand(x.view(1, 2, 64), x, i)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_expanded_attn(x, x, x, x, i, i, sm_scale=1.0)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_prefix_attn(x, x, i, sm_scale=1.0, q_per_seq=1, group_start=i, n_shared=i)
