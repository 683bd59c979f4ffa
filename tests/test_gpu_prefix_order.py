"""GPU test that a group_start that decreases (groups that would overlap) is recorded, shares nothing and writes nothing outside of
what the call was given."""
import ctypes

import numpy as np
import pytest
import torch

from test_gpu_prefix import call
from test_gpu_tree import Case, _i32, dsa  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu


def workspace(c, n_groups):
    """Bytes that the library asks for."""
    from top_sparse_attention_gb300 import _native as N

    a = N.DsaTreeArgs(n_seq=c.n, q_per_seq=c.N, L=c.L, H=c.H, D_qk=576, D_v=512, sm_scale=1 / 24, kv_dtype=0, n_ctx=4096, q=4096, kv=4096,
                      kv_row_stride=1152, kv_seq_stride=c.L * 1152, out=4096, lse=4096)
    n = ctypes.c_size_t(0)
    assert N.lib.dsa_prefix_attn_workspace_size(ctypes.byref(a), 4096, 4096, n_groups, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("n,H,start", [
    (4, 16, [4, 0]), (5, 16, [0, 3, 1, 5]), (6, 5, [0, 6, -3, 6]), (6, 4, [2, 9, 5, 5]), (100, 16, [0, 100, 0, 100]),
    (100, 16, [0, 100] * 50), (40, 16, [0, 40] * 1000),
])
def test_groups_that_overlap(dsa, n, H, start):  # noqa: F811
    c = Case(n, 130 + np.arange(n), 1, H, "bf16", 0)
    c.group_start, c.n_shared = np.asarray(start), np.full(len(start) - 1, 128)
    need = workspace(c, len(start) - 1)
    ws = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = call(dsa, c, ws=ws[:need])
    # (in the caches' bounds either way: [2, 9, 5, 5] is [2, 6, 5, 5])
    assert dsa.dsa_get_device_error() == 1
    assert bool((ws[need:] == 0xA5).all())
    c.check(out, lse, 1 / 24, None)
    want = call(dsa, c, group_start=_i32(np.zeros(len(start))))
    assert dsa.dsa_get_device_error() == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_groups_clamped_to_the_sequences(dsa):  # noqa: F811
    # not decreasing once they are clamped: taken as they are
    c = Case(3, [200, 210, 190], 2, 16, "bf16", 0)
    c.group_start, c.n_shared = np.array([-5, -7, 3, 9, 8]), np.full(4, 64)
    for s in (1, 2):
        c.val[s * c.L:s * c.L + 64] = c.val[:64]
        c.cache[s * c.L:s * c.L + 64] = c.cache[:64]
    out, lse = call(dsa, c)
    assert dsa.dsa_get_device_error() == 0
    c.check(out, lse, 1 / 24, None)
