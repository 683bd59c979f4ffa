"""The serving-step operators of the latent cache, as a user calls them, beside their plain forms.

Four operators, which one decode or draft-verification step runs in this order:

* ``plan``   dsa_block_plan: request lengths -> new cache blocks, block-table entries, destination rows;
* ``rope``   dsa_rope: rotary positions (one axis, or time / height / width) on the queries' rope part;
* ``append`` dsa_rope_append: the new latent rows rotated, encoded in the cache's format and written to
  their destination rows;
* ``tree``   dsa_tree_attn: attention of the drafted tokens of each request over its latent cache.

``own`` chooses between the library's kernels and the plain form in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
D_QK, D_V, ROPE = 576, 512, 64
SM_SCALE = 1.0 / math.sqrt(D_QK)


# ----------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one decode step of a large batch: one new token per request
        {"name": "plan_decode_256", "op": "plan", "n_seq": 256, "new": 1, "ctx": 32768, "block": 64, "padded": False, "vary": False},
        # chunked prefill of a mixed batch: ragged chunks, rows packed one request after another
        {"name": "plan_prefill_ragged", "op": "plan", "n_seq": 61, "new": 2048, "ctx": 16384, "block": 64, "padded": False, "vary": True},
        # draft verification over many requests: a fixed number of rows per request, some unused
        {"name": "plan_drafts_4096", "op": "plan", "n_seq": 4096, "new": 16, "ctx": 8192, "block": 128, "padded": True, "vary": True},
        # the queries' rope part of a small decode batch, written into the 576-wide queries
        {"name": "rope_q_decode", "op": "rope", "rows": 64, "heads": 16, "axes": 1, "style": "half"},
        # a long prompt with video frames: three axes, neighbouring pairs
        {"name": "rope_q_video", "op": "rope", "rows": 32768, "heads": 16, "axes": 3, "style": "pairs"},
        # the new rows of a decode batch into an FP8 cache with one scale per row
        {"name": "append_fp8_decode", "op": "append", "rows": 129, "kv": "fp8", "axes": 1, "style": "half"},
        # a prompt's rows into a bf16 cache
        {"name": "append_bf16_prompt", "op": "append", "rows": 16384, "kv": "bf16", "axes": 1, "style": "half"},
        # a large batch of prompts into an FP8 cache with one scale per 128 columns, three axes
        {"name": "append_t128_prompts", "op": "append", "rows": 131072, "kv": "t128", "axes": 3, "style": "half"},
        # one request, one token: latency
        {"name": "tree_one_token_l2k", "op": "tree", "n_seq": 1, "nodes": 1, "heads": 16, "ctx": 2048, "vary": False, "kv": "bf16", "block": 0, "mask": "chain"},
        # a batch that verifies a tree of eight drafted tokens each, bf16 caches
        {"name": "tree_b8_n8_l32k_bf16", "op": "tree", "n_seq": 8, "nodes": 8, "heads": 16, "ctx": 32768, "vary": False, "kv": "bf16", "block": 0, "mask": "tree"},
        # requests of different lengths in a paged cache with 128-column scales, some drafts shorter
        {"name": "tree_b16_n13_paged_t128", "op": "tree", "n_seq": 16, "nodes": 13, "heads": 16, "ctx": 16384, "vary": True, "kv": "t128", "block": 64, "mask": "tree"},
        # wide trees over long contexts in a paged FP8 cache: bound by the matrix products
        {"name": "tree_b8_n64_l32k_fp8", "op": "tree", "n_seq": 8, "nodes": 64, "heads": 16, "ctx": 32768, "vary": False, "kv": "fp8", "block": 128, "mask": "tree"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "tree", "tree"])
    if op == "plan":
        n_seq = _log(rng, 1, 4096)
        new = _log(rng, 1, max(1, min(4096, 131072 // n_seq)))
        return {"op": op, "n_seq": n_seq, "new": new, "ctx": _log(rng, 16, 32768), "block": 64 * rng.randint(1, 4),
                "padded": rng.random() < 0.5, "vary": rng.random() < 0.7}
    if op == "rope":
        return {"op": op, "rows": _log(rng, 1, 32768), "heads": rng.choice([1, 8, 16, 16, 16]), "axes": rng.choice([1, 2, 3]),
                "style": rng.choice(["half", "pairs"])}
    if op == "append":
        return {"op": op, "rows": _log(rng, 1, 131072), "kv": rng.choice(["bf16", "fp8", "t128"]), "axes": rng.choice([1, 2, 3]),
                "style": rng.choice(["half", "pairs"])}
    nodes, heads = _log(rng, 1, 64), rng.choice([8, 16, 16, 16, 20, 32, 128])
    n_seq = _log(rng, 1, max(1, min(64, 8192 // (nodes * heads))))
    ctx = _log(rng, 64, max(65, min(32768, (1 << 28) // (n_seq * nodes * heads), (1 << 18) // n_seq)))
    return {"op": op, "n_seq": n_seq, "nodes": nodes, "heads": heads, "ctx": ctx, "vary": rng.random() < 0.6,
            "kv": rng.choice(["bf16", "fp8", "t128"]), "block": rng.choice([0, 64, 128, 192]),
            "mask": rng.choice(["chain", "tree", "tree"])}


# ----------------------------------------------------------------------------------------------
# inputs

def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _inv_freq():
    return (1.0 / (10000.0 ** (torch.arange(0, ROPE, 2, dtype=torch.float64) / ROPE))).float().to(DEV)


def _sections(axes):
    """Pairs of the 32 that each axis turns, in order."""
    return {1: (32,), 2: (16, 16), 3: (8, 12, 12)}[axes]


def _axis_of_pair(axes):
    return torch.tensor([a for a, n in enumerate(_sections(axes)) for _ in range(n)], device=DEV)


def _positions(rng, rows, axes):
    pos = np.empty((rows, axes), np.int64)
    pos[:, 0] = rng.integers(0, 4096) + np.arange(rows)  # running time, in a context that may be long
    pos[:, 0] += int(rng.integers(0, 1 << 20)) if rng.random() < 0.5 else 0
    for a in range(1, axes):
        pos[:, a] = rng.integers(0, 128, rows)
    return _i32(pos)


def _lengths(rng, n, mean_to, vary, least=0):
    return rng.integers(least, mean_to + 1, n) if vary else np.full(n, mean_to)


def _prepare_plan(c, rng):
    n, b = c["n_seq"], c["block"]
    ctx = rng.integers(0, c["ctx"] + 1, n)
    new = _lengths(rng, n, c["new"], c["vary"])
    rows = n * c["new"]
    if c["vary"] and not c["padded"]:  # a step's budget of rows; requests behind it wait
        rows = max(1, rows * 5 // 8)
        new = np.minimum(new, np.maximum(rows - (np.cumsum(new) - new), 0))
    max_blocks = -(-(c["ctx"] + c["new"]) // b)
    have = -(-ctx // b)
    need = -(-(ctx + new) // b) - have
    num = int(have.sum() + need.sum()) + 64
    ids = rng.permutation(num).astype(np.int32)
    table = np.full((n, max_blocks), -1, np.int32)
    used = np.arange(max_blocks)[None, :] < have[:, None]
    table[used] = ids[: int(have.sum())]
    free = ids[int(have.sum()):]
    return {"n_ctx": _i32(ctx), "n_new": _i32(new), "free": _i32(free), "table": _i32(table), "rows": rows, "num": num}


def _prepare_rope(c, rng, seed):
    x = torch.randn(c["rows"], c["heads"], ROPE, generator=_gen(seed), device=DEV).bfloat16()
    q = torch.randn(c["rows"], c["heads"], D_QK, generator=_gen(seed + 1), device=DEV).bfloat16()
    return {"x": x, "q": q, "pos": _positions(rng, c["rows"], c["axes"]), "inv_freq": _inv_freq(), "axis": _axis_of_pair(c["axes"])}


def _prepare_append(c, rng, seed):
    rows = c["rows"]
    x = torch.randn(rows, D_QK, generator=_gen(seed), device=DEV).bfloat16()
    pool = -(-(rows + rows // 4 + 64) // 64) * 64
    dst = rng.permutation(pool // 64)[: -(-rows // 64)].astype(np.int64)  # whole blocks in any order, the last one partly
    dst = (dst[:, None] * 64 + np.arange(64)[None, :]).reshape(-1)[:rows]
    dst[rng.random(rows) < 0.01] = -1  # rows of the batch that hold no token
    s = {"x": x, "dst": torch.from_numpy(dst).to(DEV), "pos": _positions(rng, rows, c["axes"]), "inv_freq": _inv_freq(),
         "axis": _axis_of_pair(c["axes"]), "pool": pool}
    # the pools carry one spare row, which the plain form writes dropped rows to
    if c["kv"] == "bf16":
        s["kv"], s["scale"] = torch.zeros(pool + 1, D_QK, dtype=torch.bfloat16, device=DEV), None
    else:
        s["kv"] = torch.zeros(pool + 1, D_QK, dtype=torch.uint8, device=DEV)
        s["scale"] = torch.ones((pool + 1,) if c["kv"] == "fp8" else (pool + 1, 5), dtype=torch.float32, device=DEV)
    return s


def _tree_bits(rng, n_seq, nodes, kind):
    """[n_seq, nodes, nodes] truth values: node i attends to drafted node j (its ancestors and itself)."""
    if kind == "chain":
        return np.broadcast_to(np.tril(np.ones((nodes, nodes), bool)), (n_seq, nodes, nodes))
    anc = np.zeros((n_seq, nodes, nodes), bool)
    at = np.arange(n_seq)
    for i in range(nodes):
        parent = rng.integers(-1, i, n_seq) if i else np.full(n_seq, -1)
        anc[:, i] = np.where((parent >= 0)[:, None], anc[at, np.maximum(parent, 0)], False)
        anc[:, i, i] = True
    return anc


def _pack_bits(bits):
    n_seq, nodes, _ = bits.shape
    words = -(-nodes // 32)
    full = np.zeros((n_seq, nodes, words * 32), np.uint64)
    full[..., :nodes] = bits
    packed = (full.reshape(n_seq, nodes, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return packed.reshape(n_seq * nodes, words).view(np.int32)


def _prepare_tree(c, rng, seed):
    n, nodes, b = c["n_seq"], c["nodes"], c["block"]
    ctx = _lengths(rng, n, c["ctx"], c["vary"], c["ctx"] // 8)
    new = _lengths(rng, n, nodes, c["vary"], nodes // 2)
    bits = _tree_bits(rng, n, nodes, c["mask"])
    L = c["ctx"] + nodes
    s = {"n_ctx": _i32(ctx), "n_new": _i32(new), "L": L, "block": b,
         "mask": None if c["mask"] == "chain" else _i32(_pack_bits(bits)),
         "bits": torch.from_numpy(np.ascontiguousarray(bits)).to(DEV)}
    if b:
        per = -(-L // b)
        rows = (n * per + 3) * b
        s["table"] = _i32(rng.permutation(n * per + 3)[: n * per].reshape(n, per))
    else:
        rows, s["table"] = n * L, None
    g = _gen(seed)
    s["q"] = torch.randn(n * nodes, c["heads"], D_QK, generator=g, device=DEV).bfloat16()
    if c["kv"] == "bf16":
        kv, s["scale"] = torch.empty(rows, D_QK, dtype=torch.bfloat16, device=DEV), None
    else:
        kv = torch.empty(rows, D_QK, dtype=torch.uint8, device=DEV)
        s["scale"] = torch.empty((rows,) if c["kv"] == "fp8" else (rows, 5), dtype=torch.float32, device=DEV)
    for lo in range(0, rows, 65536):  # made in pieces: the caches are large
        x = torch.randn(min(65536, rows - lo), D_QK, generator=g, device=DEV)
        if c["kv"] == "bf16":
            kv[lo:lo + 65536] = x.bfloat16()
        elif c["kv"] == "fp8":
            sc = x.abs().amax(1) / 448.0
            kv[lo:lo + 65536] = (x / sc[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            s["scale"][lo:lo + 65536] = sc
        else:
            sc = torch.cat([x[:, :512].view(-1, 4, 128).abs().amax(2), x[:, 512:].abs().amax(1, keepdim=True)], 1) / 448.0
            kv[lo:lo + 65536] = (x / sc.repeat_interleave(128, 1)[:, :D_QK]).to(torch.float8_e4m3fn).view(torch.uint8)
            s["scale"][lo:lo + 65536] = sc
    if not b:
        kv = kv.view(n, L, D_QK)
        if s["scale"] is not None:
            s["scale"] = s["scale"].view((n, L) + tuple(s["scale"].shape[1:]))
    s["kv"] = kv
    return s


def prepare(case, seed):
    rng = np.random.default_rng([int(seed), 77])
    c = dict(case)
    op = c["op"]
    s = (_prepare_plan(c, rng) if op == "plan" else _prepare_rope(c, rng, 2 * int(seed)) if op == "rope"
         else _prepare_append(c, rng, int(seed)) if op == "append" else _prepare_tree(c, rng, int(seed)))
    s["case"] = c
    return s


# ----------------------------------------------------------------------------------------------
# one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return {"plan": _plain_plan, "rope": _plain_rope, "append": _plain_append, "tree": _plain_tree}[op](state)


def _own_plan(s):
    import top_sparse_attention_gb300 as dsa

    c = s["case"]
    p = dsa.dsa_block_plan(s["n_ctx"], s["n_new"], s["free"], s["table"], block_size=c["block"], num_blocks=s["num"],
                           rows=s["rows"], q_per_seq=c["new"] if c["padded"] else 0)
    return {"dst_rows": p.dst_rows, "pos": p.pos, "seq": p.seq, "row_start": p.row_start, "n_placed": p.n_placed,
            "taken": p.taken, "table": s["table"]}


def _own_rope(s):
    import top_sparse_attention_gb300 as dsa

    c = s["case"]
    dsa.dsa_rope(s["x"], s["pos"], s["inv_freq"], sections=_sections(c["axes"]), style=c["style"], out=s["q"][..., D_V:])
    return s["q"]


def _own_append(s):
    import top_sparse_attention_gb300 as dsa

    c, pool = s["case"], s["pool"]
    kv, scale = s["kv"][:pool], None if s["scale"] is None else s["scale"][:pool]
    dsa.dsa_rope_append(s["x"], s["pos"], s["inv_freq"], kv, scale=scale, dst_rows=s["dst"], rot_off=D_V, rot_dim=ROPE,
                        sections=_sections(c["axes"]), style=c["style"])
    return {"kv": kv} if scale is None else {"kv": kv.view(torch.float8_e4m3fn), "scale": scale}


def _own_tree(s):
    import top_sparse_attention_gb300 as dsa

    c = s["case"]
    return dsa.dsa_tree_attn(s["q"], s["kv"], s["n_ctx"], n_new=s["n_new"], tree_mask=s["mask"], kv_scale=s["scale"],
                             q_per_seq=c["nodes"], sm_scale=SM_SCALE, block_table=s["table"], block_size=s["block"],
                             L=s["L"] if s["block"] else None)


_OWN = {"plan": _own_plan, "rope": _own_rope, "append": _own_append, "tree": _own_tree}


# ----------------------------------------------------------------------------------------------
# plain forms

def _plain_plan(s):
    c = s["case"]
    b, rows, table = c["block"], s["rows"], s["table"]
    ctx, new = s["n_ctx"].clamp(min=0).long(), s["n_new"].clamp(min=0).long()
    n_seq = ctx.numel()
    have = (ctx + b - 1) // b
    total = (ctx + new + b - 1) // b
    fits = total <= table.shape[1]
    need = torch.where(fits, total - have, 0)
    upto = torch.cumsum(need, 0)
    placed = fits & ((need == 0) | (upto <= s["free"].numel()))
    first = upto - need
    row_start = torch.zeros(n_seq + 1, dtype=torch.int64, device=DEV)
    row_start[1:] = torch.cumsum(new, 0)
    r = torch.arange(rows, device=DEV)
    if c["padded"]:
        row_start = torch.arange(n_seq + 1, device=DEV) * c["new"]
        seq, i = r // c["new"], r % c["new"]
    else:
        seq = torch.searchsorted(row_start, r, right=True) - 1
        seq = seq.clamp(max=n_seq - 1)
        i = r - row_start[seq]
    live = (i < new[seq]) & placed[seq]
    p = ctx[seq] + i
    j = p // b
    fresh = j >= have[seq]
    at = (first[seq] + j - have[seq]).clamp(0, s["free"].numel() - 1)
    jc = j.clamp(max=table.shape[1] - 1)
    block = torch.where(fresh, s["free"][at], table[seq, jc])
    dst = torch.where(live, block.long() * b + p % b, -1)
    wide = torch.nn.functional.pad(table, (0, 1))  # a spare column takes what rows without a token write
    wide[seq, torch.where(live, jc, table.shape[1])] = block
    table.copy_(wide[:, :-1])
    return {"dst_rows": dst, "pos": torch.where(live, p, -1).int(), "seq": torch.where(live, seq, -1).int(),
            "row_start": row_start.int(), "n_placed": torch.where(placed, new, 0).int(),
            "taken": torch.where(placed, need, 0).sum().int().view(1), "table": table}


def _plain_angles(s):
    """cos, sin [rows, 32]: the angle in 64 bits (far positions lose it in 32), reduced to one turn."""
    a = torch.remainder(s["pos"][:, s["axis"]].double() * s["inv_freq"].double(), 2 * math.pi).float()
    return torch.cos(a), torch.sin(a)


def _plain_rotate(x, cos, sin, style):
    """x [..., 64] fp32 with cos / sin that broadcast over [..., 32]."""
    if style == "half":
        x0, x1 = x[..., :32], x[..., 32:]
        return torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)


def _plain_rope(s):
    c = s["case"]
    cos, sin = _plain_angles(s)
    s["q"][..., D_V:] = _plain_rotate(s["x"].float(), cos[:, None], sin[:, None], c["style"]).bfloat16()
    return s["q"]


def _plain_append(s):
    c, pool = s["case"], s["pool"]
    cos, sin = _plain_angles(s)
    x = s["x"].float()
    x = torch.cat([x[:, :D_V], _plain_rotate(x[:, D_V:], cos, sin, c["style"])], 1)
    dst = torch.where(s["dst"] < 0, pool, s["dst"])
    if c["kv"] == "bf16":
        s["kv"][dst] = x.bfloat16()
        return {"kv": s["kv"][:pool]}
    if c["kv"] == "fp8":
        scale = x.abs().amax(1) / 448.0
        scale = torch.where(scale > 0, scale, 1.0)
        wide = scale[:, None]
    else:
        scale = torch.cat([x[:, :512].view(-1, 4, 128).abs().amax(2), x[:, 512:].abs().amax(1, keepdim=True)], 1) / 448.0
        scale = torch.where(scale > 0, scale, 1.0)
        wide = scale.repeat_interleave(128, 1)[:, :D_QK]
    s["kv"][dst] = (x / wide).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    s["scale"][dst] = scale
    return {"kv": s["kv"][:pool].view(torch.float8_e4m3fn), "scale": s["scale"][:pool]}


def _cache_rows(s):
    """The cache row of each position, [n_seq, L] (paged caches: through the block table)."""
    n, L, b = s["n_ctx"].numel(), s["L"], s["block"]
    p = torch.arange(L, device=DEV)
    if not b:
        return torch.arange(n, device=DEV)[:, None] * L + p[None, :]
    return s["table"][:, p // b].long() * b + p % b


def _plain_tree(s):
    c = s["case"]
    n, N, H, L = c["n_seq"], c["nodes"], c["heads"], s["L"]
    rows = _cache_rows(s)
    kv = s["kv"].reshape(-1, D_QK)[rows]
    if c["kv"] != "bf16":
        sc = s["scale"].reshape((-1,) + tuple(s["scale"].shape[1 if s["block"] else 2:]))[rows]
        sc = sc[..., None] if c["kv"] == "fp8" else sc.repeat_interleave(128, -1)[..., :D_QK]
        kv = kv.view(torch.float8_e4m3fn).float() * sc
    kv = kv.float()
    ctx, new = s["n_ctx"].long(), s["n_new"].long()
    # node i of each request sees the context and the drafted rows of its mask
    p = torch.arange(L, device=DEV)
    j = (p[None, :] - ctx[:, None])
    drafted = torch.gather(s["bits"], 2, j.clamp(0, N - 1)[:, None, :].expand(n, N, L))
    sees = (j < 0)[:, None, :] | (drafted & ((j >= 0) & (j < new[:, None]))[:, None, :])
    sees = sees & (torch.arange(N, device=DEV)[None, :] < new[:, None])[:, :, None]
    sees = sees[:, :, None, :].expand(n, N, H, L).reshape(n, N * H, L)
    x = torch.matmul(s["q"].view(n, N * H, D_QK).float(), kv.transpose(1, 2)) * SM_SCALE
    x = torch.where(sees, x, -math.inf)
    m = x.amax(2, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    total = e.sum(2, keepdim=True)
    out = torch.matmul(e, kv[..., :D_V]) / torch.where(total > 0, total, 1.0)
    lse = m + torch.log(total)
    return out.view(n * N, H, D_V).bfloat16(), lse.view(n * N, H)


# ----------------------------------------------------------------------------------------------
# work of one pass: inputs read once, outputs written once

def work(case):
    c = case
    if c["op"] == "plan":
        rows = c["n_seq"] * c["new"] * (0.625 if c["vary"] and not c["padded"] else 1.0)
        tokens = c["n_seq"] * c["new"] * (0.5 if c["vary"] else 1.0)
        return {"bytes": 16.0 * rows + 20.0 * c["n_seq"] + 8.0 * tokens / c["block"], "flops": 0.0}
    if c["op"] == "rope":
        n = c["rows"] * c["heads"] * ROPE
        return {"bytes": 4.0 * n + 4.0 * c["rows"] * c["axes"], "flops": 3.0 * n}
    if c["op"] == "append":
        out = {"bf16": 1152, "fp8": 580, "t128": 596}[c["kv"]]
        return {"bytes": float(c["rows"]) * (1152 + out + 8 + 4 * c["axes"]), "flops": float(c["rows"]) * 6 * D_QK}
    share = 0.5625 if c["vary"] else 1.0  # mean context of a varying batch
    live = 0.75 if c["vary"] else 1.0
    row = {"bf16": 1152, "fp8": 580, "t128": 596}[c["kv"]]
    rows, q = c["n_seq"] * (c["ctx"] * share + c["nodes"] * live), c["n_seq"] * c["nodes"] * c["heads"]
    return {"bytes": rows * row + q * (1152 + 1028.0), "flops": 2.0 * (D_QK + D_V) * q * live * c["ctx"] * share}


# ----------------------------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    if op in ("rope", "append"):
        return _exact_turn(s, case)
    return _exact_tree(s, case)


def _exact_turn(s, c):
    """Rotation as a product of complex numbers."""
    axis = [a for a, n in enumerate(_sections(c["axes"])) for _ in range(n)]
    angle = s["pos"].double()[:, axis] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)

    def rotated(x):
        z = torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous()) if c["style"] == "half" else torch.view_as_complex(x.reshape(x.shape[:-1] + (32, 2)))
        z = z * (turn[:, None] if x.dim() == 3 else turn)
        return torch.cat([z.real, z.imag], -1) if c["style"] == "half" else torch.view_as_real(z).reshape(x.shape)

    if c["op"] == "rope":
        q = s["q"].double()
        q[..., D_V:] = rotated(s["x"].double())
        return q
    x = s["x"].double()
    x[:, D_V:] = rotated(x[:, D_V:].contiguous())
    keep = s["dst"] >= 0
    kv = torch.zeros(s["pool"], D_QK, dtype=torch.float64, device=DEV)
    if c["kv"] == "bf16":
        kv[s["dst"][keep]] = x[keep]
        return {"kv": kv}
    parts = [x] if c["kv"] == "fp8" else list(x.split(128, 1))
    scales = torch.stack([y.abs().max(1).values / 448.0 for y in parts], 1)
    coded = torch.cat([y / scales[:, k:k + 1] for k, y in enumerate(parts)], 1)
    scale = torch.ones(s["pool"], len(parts), dtype=torch.float64, device=DEV)
    kv[s["dst"][keep]] = coded[keep]
    scale[s["dst"][keep]] = scales[keep]
    return {"kv": kv, "scale": scale.view(s["scale"][:-1].shape)}


def _exact_tree(s, c):
    n, N, H = c["n_seq"], c["nodes"], c["heads"]
    out = torch.zeros(n, N, H, D_V, dtype=torch.float64, device=DEV)
    lse = torch.full((n, N, H), -math.inf, dtype=torch.float64, device=DEV)
    ctx, new, bits = s["n_ctx"].tolist(), s["n_new"].tolist(), s["bits"]
    flat = s["kv"].reshape(-1, D_QK)
    rows = _cache_rows(s)
    for k in range(n):
        if not new[k]:
            continue
        at = rows[k, : ctx[k] + new[k]]
        if c["kv"] == "bf16":
            v = flat[at].double()
        else:
            v = flat[at].view(torch.float8_e4m3fn).to(torch.float64)
            if c["kv"] == "fp8":
                v = v * s["scale"].reshape(-1)[at].double()[:, None]
            else:
                sc = s["scale"].reshape(-1, 5)[at].double()
                v = torch.cat([v[:, 128 * t:128 * t + 128] * sc[:, t:t + 1] for t in range(5)], 1)
        logit = torch.einsum("nhd,ld->nhl", s["q"].view(n, N, H, D_QK)[k, : new[k]].double(), v) * SM_SCALE
        hidden = ~bits[k, : new[k], : new[k]]
        logit[:, :, ctx[k]:] = logit[:, :, ctx[k]:].masked_fill(hidden[:, None, :], -math.inf)
        lse[k, : new[k]] = torch.logsumexp(logit, 2)
        out[k, : new[k]] = torch.einsum("nhl,ld->nhd", torch.softmax(logit, 2), v[:, :D_V])
    return out.view(n * N, H, D_V), lse.view(n * N, H)
