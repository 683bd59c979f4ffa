"""The operators around a latent-attention layer, as a user calls them, beside their plain forms.

* ``norm``    dsa_norm_rope: norm of each head's query (or key) and its rotary positions in one pass;
* ``append``  dsa_norm_rope_append: the new latent rows (or indexer keys) normed, rotated, encoded in the
  cache's format and written to their destination rows;
* ``prefix``  dsa_prefix_attn: attention of a decode (or draft-verification) batch over the latent cache, whose
  sequences share long prefixes in groups;
* ``expand``  dsa_latent_expand: cached latent rows expanded to every head's key and value;
* ``attn``    dsa_expanded_attn: causal attention of prompts, or chunks of them, over expanded keys and values.

``own`` chooses between the library's kernels and the plain form in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
LATENT, D_V, ROPE = 576, 512, 64  # a cached row: 512 latent columns (which are also the values), 64 rotary ones
NOPE, VALUE = 128, 128            # a head's expanded key without its rotary part, and its value
EPS = 1e-6


# ----------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # the indexer's queries of a decode batch, 64 heads of 128 each, half of the columns rotary
        {"name": "norm_q_decode", "op": "norm", "rows": 64, "heads": 64, "width": 128, "kind": "rms", "rot_off": 0, "rot": 64, "style": "half"},
        # a prompt's queries with a norm for each head, the rotary part last
        {"name": "norm_q_prompt", "op": "norm", "rows": 16384, "heads": 16, "width": 192, "kind": "rms", "rot_off": 128, "rot": 64, "style": "pairs"},
        # the new latent rows of a decode batch into a cache with one scale per row
        {"name": "append_fp8_decode", "op": "append", "rows": 129, "what": "latent", "kv": "fp8", "style": "half"},
        # a large batch of prompts into a cache with one scale per 128 columns
        {"name": "append_t128_prompts", "op": "append", "rows": 65536, "what": "latent", "kv": "t128", "style": "half"},
        # a few requests behind a short system prompt: latency
        {"name": "prefix_b4_l1k", "op": "prefix", "n_seq": 4, "groups": 1, "nodes": 1, "heads": 16, "shared": 1024, "tail": 64, "vary": False, "kv": "bf16", "block": 0, "mask": "chain"},
        # three system prompts, a chain of four drafted tokens each, tails of different lengths, 128-column scales
        {"name": "prefix_g3_n4_paged_t128", "op": "prefix", "n_seq": 48, "groups": 3, "nodes": 4, "heads": 16, "shared": 8192, "tail": 1500, "vary": True, "kv": "t128", "block": 64, "mask": "chain"},
        # one long document, 64 questions about it, one token each
        {"name": "prefix_b64_l32k_paged_fp8", "op": "prefix", "n_seq": 64, "groups": 1, "nodes": 1, "heads": 16, "shared": 32768, "tail": 512, "vary": True, "kv": "fp8", "block": 64, "mask": "chain"},
        # the rows of a few short prompts
        {"name": "expand_short_bf16", "op": "expand", "n_seq": 5, "len": 97, "heads": 16, "vary": True, "kv": "bf16", "block": 0},
        # the cached contexts of a chunked prefill, from a paged cache
        {"name": "expand_ctx_paged_fp8", "op": "expand", "n_seq": 3, "len": 16384, "heads": 16, "vary": True, "kv": "fp8", "block": 64},
        # a batch of short prompts
        {"name": "attn_ragged_short", "op": "attn", "n_seq": 7, "new": 200, "ctx": 0, "heads": 16, "vary": True},
        # one prompt
        {"name": "attn_prompt_8k", "op": "attn", "n_seq": 1, "new": 8192, "ctx": 0, "heads": 16, "vary": False},
        # chunks of long prompts over what is cached of them
        {"name": "attn_chunks_ctx", "op": "attn", "n_seq": 2, "new": 1500, "ctx": 16384, "heads": 16, "vary": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "prefix", "prefix", "expand", "attn", "attn"])
    if op == "norm":
        width = rng.choice([64, 128, 128, 192, 256, 576])
        rot = rng.choice([r for r in (32, 64, 64, 128) if r <= width])
        heads = rng.choice([1, 4, 8, 16, 16, 64])
        return {"op": op, "rows": _log(rng, 1, max(1, min(32768, (50 << 20) // (heads * width)))), "heads": heads, "width": width,
                "kind": rng.choice(["rms", "rms", "layer"]), "rot_off": rng.choice([0, width - rot]), "rot": rot,
                "style": rng.choice(["half", "pairs"])}
    if op == "append":
        what = rng.choice(["latent", "latent", "key"])
        return {"op": op, "rows": _log(rng, 1, 65536), "what": what, "kv": rng.choice(["bf16", "fp8", "t128"]) if what == "latent" else "bf16",
                "style": rng.choice(["half", "pairs"])}
    if op == "prefix":
        nodes, heads = _log(rng, 1, 16), rng.choice([8, 16, 16, 16, 20, 128])
        n_seq = _log(rng, 2, max(2, min(64, 2048 // (nodes * heads))))
        shared = _log(rng, 64, max(65, min(32768, (1 << 26) // (n_seq * nodes * heads))))
        return {"op": op, "n_seq": n_seq, "groups": rng.randint(1, max(1, min(4, n_seq // 2))), "nodes": nodes, "heads": heads, "shared": shared,
                "tail": _log(rng, 1, 1024), "vary": rng.random() < 0.6, "kv": rng.choice(["bf16", "fp8", "t128"]),
                "block": rng.choice([0, 64, 128]), "mask": rng.choice(["chain", "tree"])}
    heads = rng.choice([1, 8, 16, 16, 16, 20, 32])
    if op == "expand":
        n_seq = _log(rng, 1, 32)
        return {"op": op, "n_seq": n_seq, "len": _log(rng, 1, max(2, min(16384, 400000 // (n_seq * heads)))), "heads": heads, "vary": rng.random() < 0.6,
                "kv": rng.choice(["bf16", "fp8", "t128"]), "block": rng.choice([0, 64, 128])}
    n_seq = _log(rng, 1, 32)
    new = _log(rng, 1, max(2, 4096 // n_seq))
    ctx = rng.choice([0, _log(rng, 1, max(2, min(16384, (1 << 29) // (n_seq * new * heads))))])
    return {"op": op, "n_seq": n_seq, "new": new, "ctx": ctx, "heads": heads, "vary": rng.random() < 0.6}


# ----------------------------------------------------------------------------------------------
# inputs

def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _inv_freq(rot):
    return (1.0 / (10000.0 ** (torch.arange(0, rot, 2, dtype=torch.float64) / rot))).float().to(DEV)


def _positions(rng, rows):
    first = int(rng.integers(0, 1 << 20)) if rng.random() < 0.5 else int(rng.integers(0, 4096))
    return _i32(first + np.arange(rows))


def _lengths(rng, n, most, vary, least=0):
    return rng.integers(least, most + 1, n) if vary else np.full(n, most)


def _ragged(rng, n, most, vary):
    """Lengths between a half of `most` and the whole, whose sum is the same for every seed."""
    if not vary:
        return np.full(n, most)
    a, total = rng.integers(most // 2, most + 1, n), -(-n * most * 3 // 4)
    while a.sum() != total:
        k = np.flatnonzero(a > most // 2 if a.sum() > total else a < most)
        k = k[: abs(int(a.sum()) - total)]
        a[k] += 1 if a.sum() < total else -1
    return a


def _starts(lengths):
    return np.concatenate([[0], np.cumsum(lengths)])


def _weights(n, g, bias):
    w = 1.0 + 0.2 * torch.randn(n, generator=g, device=DEV)
    return w, 0.2 * torch.randn(n, generator=g, device=DEV) if bias else None


def _prepare_norm(c, rng, seed):
    g = _gen(seed)
    x = (torch.randn(c["rows"], c["heads"], c["width"], generator=g, device=DEV) * 2.0).bfloat16()
    w, b = _weights(c["width"], g, c["kind"] == "layer")
    return {"x": x, "w": w, "b": b, "pos": _positions(rng, c["rows"]), "inv_freq": _inv_freq(c["rot"])}


def _prepare_append(c, rng, seed):
    rows, g = c["rows"], _gen(seed)
    width = LATENT if c["what"] == "latent" else 128
    x = (torch.randn(rows, width, generator=g, device=DEV) * 2.0).bfloat16()
    w, b = _weights(D_V if c["what"] == "latent" else 128, g, c["what"] == "key")
    pool = -(-(rows + rows // 4 + 64) // 64) * 64
    dst = rng.permutation(pool // 64)[: -(-rows // 64)].astype(np.int64)  # whole blocks in any order, the last one partly
    dst = (dst[:, None] * 64 + np.arange(64)[None, :]).reshape(-1)[:rows]
    dst[rng.random(rows) < 0.01] = -1  # rows of the batch that hold no token
    s = {"x": x, "w": w, "b": b, "dst": torch.from_numpy(dst).to(DEV), "pos": _positions(rng, rows), "inv_freq": _inv_freq(ROPE), "pool": pool}
    # the pools carry one spare row, which the plain form writes dropped rows to
    if c["kv"] == "bf16":
        s["kv"], s["scale"] = torch.zeros(pool + 1, width, dtype=torch.bfloat16, device=DEV), None
    else:
        s["kv"] = torch.zeros(pool + 1, width, dtype=torch.uint8, device=DEV)
        s["scale"] = torch.ones((pool + 1,) if c["kv"] == "fp8" else (pool + 1, 5), dtype=torch.float32, device=DEV)
    return s


def _cache(rows, kind, g):
    """Random latent rows in the cache's format: (kv [rows, 576], scale)."""
    if kind == "bf16":
        kv, scale = torch.empty(rows, LATENT, dtype=torch.bfloat16, device=DEV), None
    else:
        kv = torch.empty(rows, LATENT, dtype=torch.uint8, device=DEV)
        scale = torch.empty((rows,) if kind == "fp8" else (rows, 5), dtype=torch.float32, device=DEV)
    for lo in range(0, rows, 65536):  # made in pieces: the caches are large
        x = torch.randn(min(65536, rows - lo), LATENT, generator=g, device=DEV)
        if kind == "bf16":
            kv[lo:lo + 65536] = x.bfloat16()
        elif kind == "fp8":
            sc = x.abs().amax(1) / 448.0
            kv[lo:lo + 65536] = (x / sc[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            scale[lo:lo + 65536] = sc
        else:
            sc = torch.cat([x[:, :512].view(-1, 4, 128).abs().amax(2), x[:, 512:].abs().amax(1, keepdim=True)], 1) / 448.0
            kv[lo:lo + 65536] = (x / sc.repeat_interleave(128, 1)[:, :LATENT]).to(torch.float8_e4m3fn).view(torch.uint8)
            scale[lo:lo + 65536] = sc
    return kv, scale


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


def _groups(c):
    """First sequence of each group, then the number of sequences."""
    return np.array([c["n_seq"] * g // c["groups"] for g in range(c["groups"] + 1)])


def _prepare_prefix(c, rng, seed):
    n, nodes, b = c["n_seq"], c["nodes"], c["block"]
    start = _groups(c)
    shared = _lengths(rng, c["groups"], c["shared"], c["vary"] and c["groups"] > 1, -(-c["shared"] // 2))
    if b:
        shared = np.maximum(shared // b, 1) * b  # whole blocks are shared
    of = np.repeat(np.arange(c["groups"]), np.diff(start))  # the group of each sequence
    ctx = shared[of] + _lengths(rng, n, c["tail"], c["vary"])
    new = _lengths(rng, n, nodes, c["vary"], (nodes + 1) // 2)
    bits = _tree_bits(rng, n, nodes, c["mask"])
    L = int(max(c["shared"], shared.max())) + c["tail"] + nodes
    s = {"n_ctx": _i32(ctx), "n_new": _i32(new), "L": L, "block": b, "group_start": _i32(start), "n_shared": _i32(shared),
         "mask": None if c["mask"] == "chain" else _i32(_pack_bits(bits)),
         "bits": torch.from_numpy(np.ascontiguousarray(bits)).to(DEV)}
    g = _gen(seed)
    s["q"] = torch.randn(n * nodes, c["heads"], LATENT, generator=g, device=DEV).bfloat16()
    lead = start[of]  # the sequence that a sequence's prefix is the same as
    if b:
        per = -(-L // b)
        table = rng.permutation(n * per + 3)[: n * per].reshape(n, per)
        for k in range(n):
            m = shared[of[k]] // b
            table[k, :m] = table[lead[k], :m]
        s["table"] = _i32(table)
        s["kv"], s["scale"] = _cache((n * per + 3) * b, c["kv"], g)
    else:
        s["table"] = None
        kv, scale = _cache(n * L, c["kv"], g)
        s["kv"], s["scale"] = kv.view(n, L, LATENT), None if scale is None else scale.view((n, L) + tuple(scale.shape[1:]))
        for k in range(n):
            m = int(shared[of[k]])
            if lead[k] != k:
                s["kv"][k, :m] = s["kv"][lead[k], :m]
                if scale is not None:
                    s["scale"][k, :m] = s["scale"][lead[k], :m]
    return s


def _prepare_expand(c, rng, seed):
    n, b = c["n_seq"], c["block"]
    lens = _ragged(rng, n, c["len"], c["vary"])
    L, g = c["len"], _gen(seed)
    s = {"kv_start": _i32(_starts(lens)), "rows": int(lens.sum()), "block": b, "L": L, "lens": torch.from_numpy(lens).to(DEV)}
    if b:
        per = -(-L // b)
        s["table"] = _i32(rng.permutation(n * per + 3)[: n * per].reshape(n, per))
        s["kv"], s["scale"] = _cache((n * per + 3) * b, c["kv"], g)
    else:
        s["table"] = None
        kv, scale = _cache(n * L, c["kv"], g)
        s["kv"], s["scale"] = kv.view(n, L, LATENT), None if scale is None else scale.view((n, L) + tuple(scale.shape[1:]))
    s["w"] = (torch.randn(c["heads"], NOPE + VALUE, D_V, generator=g, device=DEV) / math.sqrt(D_V)).bfloat16()
    return s


def _prepare_attn(c, rng, seed):
    n, H = c["n_seq"], c["heads"]
    new, ctx = _ragged(rng, n, c["new"], c["vary"]), _ragged(rng, n, c["ctx"], c["vary"])
    g = _gen(seed)
    T, N = int(new.sum()), int((new + ctx).sum())

    def make(*shape):
        return torch.randn(*shape, generator=g, device=DEV).bfloat16()

    return {"q": make(T, H, NOPE + ROPE), "kv": make(N, H, NOPE + VALUE), "k_rope": make(N, ROPE),
            "q_start": _i32(_starts(new)), "kv_start": _i32(_starts(new + ctx)), "new": new.tolist(), "len": (new + ctx).tolist()}


_PREPARE = {"norm": _prepare_norm, "append": _prepare_append, "prefix": _prepare_prefix, "expand": _prepare_expand, "attn": _prepare_attn}


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, np.random.default_rng([int(seed), 78]), int(seed))
    s["case"] = dict(case)
    return s


# ----------------------------------------------------------------------------------------------
# one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _own_norm(s):
    import top_sparse_attention_gb300 as dsa

    c = s["case"]
    return dsa.dsa_norm_rope(s["x"], s["pos"], s["inv_freq"], norm=c["kind"], weight=s["w"], bias=s["b"], eps=EPS, rot_off=c["rot_off"],
                             rot_dim=c["rot"], style=c["style"])


def _own_append(s):
    import top_sparse_attention_gb300 as dsa

    c, pool = s["case"], s["pool"]
    kv, scale = s["kv"][:pool], None if s["scale"] is None else s["scale"][:pool]
    latent = c["what"] == "latent"
    dsa.dsa_norm_rope_append(s["x"], s["pos"], s["inv_freq"], kv, scale=scale, dst_rows=s["dst"], norm="rms" if latent else "layer",
                             weight=s["w"], bias=s["b"], eps=EPS, norm_dim=D_V if latent else 128, rot_off=D_V if latent else 0,
                             rot_dim=ROPE, style=c["style"])
    return {"kv": kv} if scale is None else {"kv": kv.view(torch.float8_e4m3fn), "scale": scale}


def _own_prefix(s):
    import top_sparse_attention_gb300 as dsa

    c = s["case"]
    return dsa.dsa_prefix_attn(s["q"], s["kv"], s["n_ctx"], group_start=s["group_start"], n_shared=s["n_shared"], n_new=s["n_new"],
                               tree_mask=s["mask"], kv_scale=s["scale"], q_per_seq=c["nodes"], sm_scale=1.0 / math.sqrt(LATENT),
                               block_table=s["table"], block_size=s["block"], L=s["L"] if s["block"] else None)


def _own_expand(s):
    import top_sparse_attention_gb300 as dsa

    return dsa.dsa_latent_expand(s["kv"], s["w"], s["kv_start"], rows=s["rows"], kv_scale=s["scale"], block_table=s["table"], block_size=s["block"])


def _own_attn(s):
    import top_sparse_attention_gb300 as dsa

    kv = s["kv"]
    return dsa.dsa_expanded_attn(s["q"], kv[..., :NOPE], s["k_rope"], kv[..., NOPE:], s["q_start"], s["kv_start"],
                                 sm_scale=1.0 / math.sqrt(NOPE + ROPE))


_OWN = {"norm": _own_norm, "append": _own_append, "prefix": _own_prefix, "expand": _own_expand, "attn": _own_attn}


# ----------------------------------------------------------------------------------------------
# plain forms

def _plain_norm_of(x, kind, w, b):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return x if b is None else x + b


def _plain_turn(x, s, off, rot, style):
    """Columns [off, off + rot) of x turned; angles in 64 bits (far positions lose them in 32), reduced to one turn."""
    a = torch.remainder(s["pos"][:, None].double() * s["inv_freq"].double(), 2 * math.pi).float()
    cos, sin = torch.cos(a), torch.sin(a)
    if x.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    t = x[..., off:off + rot]
    if style == "half":
        x0, x1 = t[..., :rot // 2], t[..., rot // 2:]
        t = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
    else:
        x0, x1 = t[..., 0::2], t[..., 1::2]
        t = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
    return torch.cat([x[..., :off], t, x[..., off + rot:]], -1)


def _plain_norm(s):
    c = s["case"]
    return _plain_turn(_plain_norm_of(s["x"].float(), c["kind"], s["w"], s["b"]), s, c["rot_off"], c["rot"], c["style"]).bfloat16()


def _plain_append(s):
    c, pool = s["case"], s["pool"]
    x = s["x"].float()
    if c["what"] == "latent":
        x = torch.cat([_plain_norm_of(x[:, :D_V], "rms", s["w"], None), x[:, D_V:]], 1)
        x = _plain_turn(x, s, D_V, ROPE, c["style"])
    else:
        x = _plain_turn(_plain_norm_of(x, "layer", s["w"], s["b"]), s, 0, ROPE, c["style"])
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
        wide = scale.repeat_interleave(128, 1)[:, :LATENT]
    s["kv"][dst] = (x / wide).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    s["scale"][dst] = scale
    return {"kv": s["kv"][:pool].view(torch.float8_e4m3fn), "scale": s["scale"][:pool]}


def _cache_rows(s, n):
    """The cache row of each position, [n_seq, L] (paged caches: through the block table)."""
    L, b = s["L"], s["block"]
    p = torch.arange(L, device=DEV)
    if not b:
        return torch.arange(n, device=DEV)[:, None] * L + p[None, :]
    return s["table"][:, p // b].long() * b + p % b


def _plain_rows(s, rows):
    """The cache rows `rows` as 32-bit values."""
    kind = s["case"]["kv"]
    kv = s["kv"].reshape(-1, LATENT)[rows]
    if kind == "bf16":
        return kv.float()
    sc = s["scale"].reshape((-1,) if kind == "fp8" else (-1, 5))[rows]
    sc = sc[..., None] if kind == "fp8" else sc.repeat_interleave(128, -1)[..., :LATENT]
    return kv.view(torch.float8_e4m3fn).float() * sc


def _plain_prefix(s):
    c = s["case"]
    n, N, H, L = c["n_seq"], c["nodes"], c["heads"], s["L"]
    kv = _plain_rows(s, _cache_rows(s, n))
    ctx, new = s["n_ctx"].long(), s["n_new"].long()
    # node i of each request sees the context and the drafted rows of its mask
    j = torch.arange(L, device=DEV)[None, :] - ctx[:, None]
    drafted = torch.gather(s["bits"], 2, j.clamp(0, N - 1)[:, None, :].expand(n, N, L))
    sees = (j < 0)[:, None, :] | (drafted & ((j >= 0) & (j < new[:, None]))[:, None, :])
    sees = sees & (torch.arange(N, device=DEV)[None, :] < new[:, None])[:, :, None]
    sees = sees[:, :, None, :].expand(n, N, H, L).reshape(n, N * H, L)
    x = torch.matmul(s["q"].view(n, N * H, LATENT).float(), kv.transpose(1, 2)) * (1.0 / math.sqrt(LATENT))
    x = torch.where(sees, x, -math.inf)
    m = x.amax(2, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    total = e.sum(2, keepdim=True)
    out = torch.matmul(e, kv[..., :D_V]) / torch.where(total > 0, total, 1.0)
    lse = m + torch.log(total)
    return out.view(n * N, H, D_V).bfloat16(), lse.view(n * N, H)


def _expand_rows(s):
    """The cache row of each expanded row."""
    n = s["case"]["n_seq"]
    rows = _cache_rows(s, n)
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), s["lens"], output_size=s["rows"])
    return rows[seq, torch.arange(s["rows"], device=DEV) - s["kv_start"].long()[seq]]


def _plain_expand(s):
    H = s["case"]["heads"]
    x = _plain_rows(s, _expand_rows(s))
    out = torch.matmul(x[:, :D_V], s["w"].view(H * (NOPE + VALUE), D_V).float().t()).bfloat16()
    return out.view(-1, H, NOPE + VALUE), x[:, D_V:].bfloat16()


def _plain_attn(s):
    H, scale = s["case"]["heads"], 1.0 / math.sqrt(NOPE + ROPE)
    outs, lses, qa, ka = [], [], 0, 0
    for m, n in zip(s["new"], s["len"]):
        k = torch.cat([s["kv"][ka:ka + n, :, :NOPE].float(), s["k_rope"][ka:ka + n, None].float().expand(n, H, ROPE)], 2).permute(1, 2, 0)
        v = s["kv"][ka:ka + n, :, NOPE:].float().transpose(0, 1)
        for lo in range(0, m, 1024):  # in pieces: the logits are large
            r = min(1024, m - lo)
            x = torch.matmul(s["q"][qa + lo:qa + lo + r].float().transpose(0, 1), k) * scale
            sees = torch.arange(n, device=DEV)[None, :] <= (n - m + lo + torch.arange(r, device=DEV))[:, None]
            x = torch.where(sees, x, -math.inf)
            top = x.amax(2, keepdim=True)
            e = torch.exp(x - top)
            total = e.sum(2, keepdim=True)
            outs.append((torch.matmul(e, v) / total).transpose(0, 1).bfloat16())
            lses.append((top + torch.log(total))[..., 0].t())
        qa, ka = qa + m, ka + n
    if not outs:
        return torch.empty(0, H, VALUE, dtype=torch.bfloat16, device=DEV), torch.empty(0, H, device=DEV)
    return torch.cat(outs), torch.cat(lses).contiguous()


_PLAIN = {"norm": _plain_norm, "append": _plain_append, "prefix": _plain_prefix, "expand": _plain_expand, "attn": _plain_attn}


# ----------------------------------------------------------------------------------------------
# work of one pass: inputs read once, outputs written once

def work(case):
    c = case
    row = {"bf16": 1152, "fp8": 580, "t128": 596}
    if c["op"] == "norm":
        n = c["rows"] * c["heads"] * c["width"]
        return {"bytes": 4.0 * n + 4.0 * c["rows"] + 8.0 * c["width"], "flops": 7.0 * n}
    if c["op"] == "append":
        if c["what"] == "latent":
            return {"bytes": float(c["rows"]) * (1152 + row[c["kv"]] + 12), "flops": float(c["rows"]) * 8 * LATENT}
        return {"bytes": float(c["rows"]) * (512 + 12), "flops": float(c["rows"]) * 8 * 128}
    mean = 0.75 if c["vary"] else 1.0  # of lengths between a half and the whole
    if c["op"] == "prefix":
        shared = c["shared"] * (mean if c["groups"] > 1 else 1.0)
        tail, live = c["tail"] * (0.5 if c["vary"] else 1.0) + c["nodes"] * mean, mean if c["nodes"] > 1 else 1.0
        q = c["n_seq"] * c["nodes"] * c["heads"]
        return {"bytes": (c["groups"] * shared + c["n_seq"] * tail) * row[c["kv"]] + q * (1152 + 1028.0),
                "flops": 2.0 * (LATENT + D_V) * q * live * (shared + tail)}
    if c["op"] == "expand":
        rows = c["n_seq"] * c["len"] * mean
        return {"bytes": rows * (row[c["kv"]] + 512 * c["heads"] + 128) + c["heads"] * 262144.0, "flops": rows * c["heads"] * 262144.0}
    new, ctx = c["new"] * mean, c["ctx"] * mean
    seen = new * ctx + new * (new + 1) / 2
    return {"bytes": c["n_seq"] * (new * c["heads"] * (384 + 260.0) + (new + ctx) * (c["heads"] * 512 + 128)),
            "flops": 2.0 * (NOPE + ROPE + VALUE) * c["n_seq"] * c["heads"] * seen}


# ----------------------------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s, case)


def _exact_turned(x, s, off, rot, style):
    """Rotation as a product of complex numbers."""
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()[None, :]
    turn = torch.polar(torch.ones_like(angle), angle)
    turn = turn[:, None] if x.dim() == 3 else turn
    part = x[..., off:off + rot].contiguous()
    if style == "half":
        z = torch.complex(part[..., :rot // 2].contiguous(), part[..., rot // 2:].contiguous()) * turn
        part = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(part.view(part.shape[:-1] + (rot // 2, 2))) * turn
        part = torch.view_as_real(z).reshape(part.shape)
    x = x.clone()
    x[..., off:off + rot] = part
    return x


def _exact_normed(x, kind, w, b):
    if kind == "layer":
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        return (x - mean) * torch.rsqrt(var + EPS) * w.double() + b.double()
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double() + (0.0 if b is None else b.double())


def _exact_norm(s, c):
    return _exact_turned(_exact_normed(s["x"].double(), c["kind"], s["w"], s["b"]), s, c["rot_off"], c["rot"], c["style"])


def _exact_append(s, c):
    x = s["x"].double()
    latent = c["what"] == "latent"
    n = D_V if latent else 128
    x[:, :n] = _exact_normed(x[:, :n], "rms" if latent else "layer", s["w"], s["b"])
    x = _exact_turned(x, s, D_V if latent else 0, ROPE, c["style"])
    keep = s["dst"] >= 0
    kv = torch.zeros(s["pool"], x.shape[1], dtype=torch.float64, device=DEV)
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


def _exact_rows(s, at):
    flat, kind = s["kv"].reshape(-1, LATENT), s["case"]["kv"]
    if kind == "bf16":
        return flat[at].double()
    v = flat[at].view(torch.float8_e4m3fn).to(torch.float64)
    if kind == "fp8":
        return v * s["scale"].reshape(-1)[at].double()[:, None]
    sc = s["scale"].reshape(-1, 5)[at].double()
    return torch.cat([v[:, 128 * t:128 * t + 128] * sc[:, t:t + 1] for t in range(5)], 1)


def _exact_prefix(s, c):
    n, N, H = c["n_seq"], c["nodes"], c["heads"]
    out = torch.zeros(n, N, H, D_V, dtype=torch.float64, device=DEV)
    lse = torch.full((n, N, H), -math.inf, dtype=torch.float64, device=DEV)
    ctx, new, bits = s["n_ctx"].tolist(), s["n_new"].tolist(), s["bits"]
    rows = _cache_rows(s, n)
    for k in range(n):
        if not new[k]:
            continue
        v = _exact_rows(s, rows[k, : ctx[k] + new[k]])
        logit = torch.einsum("nhd,ld->nhl", s["q"].view(n, N, H, LATENT)[k, : new[k]].double(), v) / math.sqrt(LATENT)
        hidden = ~bits[k, : new[k], : new[k]]
        logit[:, :, ctx[k]:] = logit[:, :, ctx[k]:].masked_fill(hidden[:, None, :], -math.inf)
        lse[k, : new[k]] = torch.logsumexp(logit, 2)
        out[k, : new[k]] = torch.einsum("nhl,ld->nhd", torch.softmax(logit, 2), v[:, :D_V])
    return out.view(n * N, H, D_V), lse.view(n * N, H)


def _exact_expand(s, c):
    at = _expand_rows(s)
    H, w = c["heads"], s["w"].double()
    out = torch.empty(s["rows"], H, NOPE + VALUE, dtype=torch.float64, device=DEV)
    rope = torch.empty(s["rows"], ROPE, dtype=torch.float64, device=DEV)
    for lo in range(0, s["rows"], 8192):
        x = _exact_rows(s, at[lo:lo + 8192])
        out[lo:lo + 8192] = torch.einsum("nc,hjc->nhj", x[:, :D_V], w)
        rope[lo:lo + 8192] = x[:, D_V:]
    return out, rope


def _exact_attn(s, c):
    if 1e-12 * work(c)["flops"] > 10.0:
        return None
    H, T = c["heads"], s["q"].shape[0]
    out = torch.empty(T, H, VALUE, dtype=torch.float64, device=DEV)
    lse = torch.empty(T, H, dtype=torch.float64, device=DEV)
    qa = ka = 0
    for m, n in zip(s["new"], s["len"]):
        for h in range(H):
            key = torch.cat([s["kv"][ka:ka + n, h, :NOPE], s["k_rope"][ka:ka + n]], 1).double()
            for lo in range(0, m, 4096):
                r = min(4096, m - lo)
                last = n - m + lo + r  # positions that the piece's last query sees
                logit = s["q"][qa + lo:qa + lo + r, h].double() @ key[:last].t() / math.sqrt(NOPE + ROPE)
                logit = logit.masked_fill(torch.ones(r, last, dtype=torch.bool, device=DEV).triu(n - m + lo + 1), -math.inf)
                lse[qa + lo:qa + lo + r, h] = torch.logsumexp(logit, 1)
                out[qa + lo:qa + lo + r, h] = torch.softmax(logit, 1) @ s["kv"][ka:ka + last, h, NOPE:].double()
        qa, ka = qa + m, ka + n
    return out, lse


_EXACT = {"norm": _exact_norm, "append": _exact_append, "prefix": _exact_prefix, "expand": _exact_expand, "attn": _exact_attn}
