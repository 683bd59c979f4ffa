"""Oracle (TEST INFRASTRUCTURE ONLY) of the serving step around the chain: block plan, rotary
positions, attention of drafted tokens over a latent cache.  Plain numpy, fp64, Python loops over
sequences; shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

__all__ = ["block_plan", "rotate", "tree_attention"]


def block_plan(n_ctx, n_new, free, table, *, block_size, num_blocks, rows, q_per_seq=0, n_free=None):
    """One sequence after another: blocks popped from the front of the free list, one row per token.
    Returns the outputs by name, the updated table and whether every token found a place."""
    b = block_size
    free = [int(f) for f in free]
    avail = len(free) if n_free is None else min(max(int(n_free), 0), len(free))
    table = np.array(table, dtype=np.int64)
    n_seq, max_blocks = len(n_ctx), table.shape[1]
    dst, pos, seq = (np.full(rows, -1, np.int64) for _ in range(3))
    start, placed_out = [], []
    used = demand = row = 0
    ok = True
    for s in range(n_seq):
        c, m = max(int(n_ctx[s]), 0), max(int(n_new[s]), 0)
        if q_per_seq:
            m = min(m, q_per_seq)
        have, total = -(-c // b), -(-(c + m) // b)
        r0 = s * q_per_seq if q_per_seq else row
        start.append(r0)
        placed = total <= max_blocks
        if placed:
            need = total - have
            demand += need
            placed = (need == 0 or demand <= avail) and (m == 0 or r0 + m <= rows)
            if placed:
                for j in range(have, total):
                    if 0 <= free[used + j - have] < num_blocks:
                        table[s, j] = free[used + j - have]
                for i in range(m):
                    j = (c + i) // b
                    block = int(table[s, j]) if j < have else free[used + j - have]
                    if 0 <= block < num_blocks:
                        dst[r0 + i] = block * b + (c + i) % b
                        pos[r0 + i] = c + i
                        seq[r0 + i] = s
                used += need
        ok = ok and (placed or m == 0)
        placed_out.append(m if placed else 0)
        row += m
    end = n_seq * q_per_seq if q_per_seq else row
    return {"dst_rows": dst, "pos": pos, "seq": seq, "row_start": np.array(start + [end]), "n_placed": np.array(placed_out),
            "taken": np.array([used]), "table": table, "ok": ok}


def rotate(x, pos, inv_freq, *, rot_off, rot_dim, pair_axis=None, style="half", inverse=False):
    """x [rows, ..., width] with columns [rot_off, rot_off + rot_dim) turned (fp64)."""
    y = np.array(x, dtype=np.float64)
    pos = np.asarray(pos, dtype=np.float64).reshape(len(y), -1)
    pairs = rot_dim // 2
    for i in range(pairs):
        a = 0 if pair_axis is None else pair_axis[i]
        theta = pos[:, a] * float(inv_freq[i]) * (-1.0 if inverse else 1.0)
        c0 = rot_off + (i if style == "half" else 2 * i)
        c1 = rot_off + (i + pairs if style == "half" else 2 * i + 1)
        shape = (len(y),) + (1,) * (y.ndim - 2)
        cos, sin = np.cos(theta).reshape(shape), np.sin(theta).reshape(shape)
        x0, x1 = y[..., c0].copy(), y[..., c1].copy()
        y[..., c0] = x0 * cos - x1 * sin
        y[..., c1] = x1 * cos + x0 * sin
    return y


def tree_attention(q, rows, n_ctx, n_new, sees, sm_scale, D_v):
    """One sequence: q [N, H, D]; rows [>= n_ctx + n_new, D] (positions in order); sees [N, N] truth
    values (node i attends to drafted node j).  Returns out [N, H, D_v], lse [N, H]; nodes at or past
    n_new, and nodes that see nothing, give 0 and -inf."""
    N, H, _ = q.shape
    out, lse = np.zeros((N, H, D_v)), np.full((N, H), -np.inf)
    for i in range(min(N, n_new)):
        at = list(range(n_ctx)) + [n_ctx + j for j in range(n_new) if sees[i, j]]
        if not at:
            continue
        kv = rows[at]
        logit = sm_scale * (q[i] @ kv.T)
        m = logit.max(axis=1, keepdims=True)
        e = np.exp(logit - m)
        lse[i] = m[:, 0] + np.log(e.sum(1))
        out[i] = (e / e.sum(1, keepdims=True)) @ kv[:, :D_v]
    return out, lse
