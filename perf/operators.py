"""The serving operators around a shared prompt, case by case: their inputs, their plain forms and their values in 64 bits.

Four operators of one path, requests that continue a common prefix:

  prefix   attention of a packed step whose sequences form groups, each group sharing the cache pages of its prefix
  rope     RMS norm of each query and key head and the position rotation, with the append of keys and values to the paged cache
  fork     child sequences that share their parent's full pages and get a copy of its last, partial one
  compact  live pages of the pool moved to its lowest ids, block tables rewritten

`run` computes an operator in elementary torch operations in fp32, or, where `own` is true, through the library's entry points."""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_ROPE_BASE = 10000.0


def _api():
    from continuous_batching_ragged_gb300 import api
    return api


def _prefix_case(name, groups, members, prefix, suffix, q_len, heads, kv_heads, block):
    """groups x members sequences; prefix and suffix are the longest ones, drawn per group and per sequence."""
    return {"name": name, "op": "prefix", "groups": groups, "members": members, "prefix": prefix, "suffix": suffix,
            "q_len": q_len, "heads": heads, "kv_heads": kv_heads, "block": block}


def listed():
    return [
        # one request sampled four times: the smallest decode step, where latency counts
        _prefix_case("prefix 4 samples", 1, 4, 512, 64, 1, 32, 8, 16),
        # 64 chats behind one system prompt, one key/value head per query head
        _prefix_case("prefix 64 chats, 32 heads", 1, 64, 2048, 512, 1, 32, 32, 16),
        # a full decode step of 256 requests over one long document
        _prefix_case("prefix 256 on a document", 1, 256, 8192, 1024, 1, 32, 8, 16),
        # many prompts, each sampled a few times: odd group sizes and prefix lengths, pages of 32
        _prefix_case("prefix 24 prompts, sampled", 24, 7, 4096, 300, 1, 32, 4, 32),
        # prompts that continue a system prompt: chunks of their own tokens behind the shared pages
        _prefix_case("prefix 12 prompt chunks", 1, 12, 4096, 661, 200, 32, 8, 16),
        # the rows of one small decode step
        {"name": "rope 4 tokens", "op": "rope", "tokens": 4, "heads": 32, "kv_heads": 8, "head_dim": 128, "rot_dim": 128,
         "norm": True, "interleaved": False, "packed": True, "dtype": "bf16", "block": 16, "positions": 4096},
        # a chunk in fp32, rotating half of each head, pairs side by side
        {"name": "rope 661 tokens, fp32", "op": "rope", "tokens": 661, "heads": 4, "kv_heads": 4, "head_dim": 64, "rot_dim": 32,
         "norm": True, "interleaved": True, "packed": False, "dtype": "f32", "block": 4, "positions": 4096},
        # a whole step's token budget
        {"name": "rope 2048 tokens", "op": "rope", "tokens": 2048, "heads": 32, "kv_heads": 32, "head_dim": 128, "rot_dim": 128,
         "norm": True, "interleaved": False, "packed": True, "dtype": "bf16", "block": 16, "positions": 32768},
        # one prompt forked into eight samples, a few layers
        {"name": "fork 8 of 1", "op": "fork", "forks": 8, "parents": 1, "context": 700, "layers": 4, "kv_heads": 8,
         "head_dim": 128, "block": 16, "dtype": "bf16"},
        # 16 prompts forked into 256 samples over every layer of a deep stack
        {"name": "fork 256 of 16", "op": "fork", "forks": 256, "parents": 16, "context": 1000, "layers": 16, "kv_heads": 8,
         "head_dim": 128, "block": 32, "dtype": "bf16"},
        # a small pool after a few requests left
        {"name": "compact 200 pages", "op": "compact", "blocks": 200, "seqs": 12, "live": 0.5, "shared": 0.3, "layers": 2,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "bf16"},
        # the serving trace's pool, fragmented
        {"name": "compact 10240 pages", "op": "compact", "blocks": 10240, "seqs": 200, "live": 0.6, "shared": 0.2, "layers": 6,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "rope", "fork", "compact"])
    if op == "prefix":
        heads, kv_heads = rng.choice([(32, 32), (32, 8), (32, 4), (32, 1), (16, 4), (8, 8), (12, 4), (24, 8)])
        q_len = rng.choice([1, 1, 1, 2, 5, _log_int(rng, 2, 200)])
        prefix = _log_int(rng, 16, 8192)
        suffix = max(q_len, _log_int(rng, 1, 1024))
        # sequences so that the step reads no more than the largest listed one's gathered keys
        most = int(256 * 9216 * 8 / (kv_heads * (prefix + suffix)))
        most = max(2, min(256, most, int(12 * 200 * 4757 / (q_len * (prefix + suffix)))))
        seqs = _log_int(rng, 2, most) if most > 2 else 2
        groups = min(seqs, rng.choice([1, 1, 2, 3, 7, 24]))
        return {"op": "prefix", "groups": groups, "members": max(1, seqs // groups), "prefix": prefix, "suffix": suffix,
                "q_len": q_len, "heads": heads, "kv_heads": kv_heads, "block": rng.choice([16, 16, 32, 64, 128])}
    if op == "rope":
        heads, kv_heads = rng.choice([(32, 32), (32, 8), (32, 4), (32, 1), (16, 4), (4, 4), (12, 4), (5, 1)])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        head_dim = rng.choice([64, 128, 128] if dtype == "f32" else [64, 128, 128, 256])
        rot = rng.choice([head_dim, head_dim, head_dim // 2])
        tokens = _log_int(rng, 1, 2048)
        while tokens * (heads + 2 * kv_heads) * head_dim * (4 if dtype == "f32" else 2) > 2048 * 96 * 256:
            tokens = tokens // 2 + 1
        return {"op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "rot_dim": rot,
                "norm": rng.random() < 0.8, "interleaved": rng.random() < 0.3, "packed": rng.random() < 0.5, "dtype": dtype,
                "block": rng.choice([4, 16, 16, 32, 64]), "positions": rng.choice([512, 4096, 32768])}
    if op == "fork":
        forks = _log_int(rng, 1, 256)
        return {"op": "fork", "forks": forks, "parents": rng.randint(1, min(forks, 16)), "context": _log_int(rng, 1, 1000),
                "layers": rng.randint(1, 16), "kv_heads": rng.choice([1, 4, 8]), "head_dim": 128,
                "block": rng.choice([16, 16, 32]), "dtype": "bf16"}
    blocks = _log_int(rng, 8, 10240)
    return {"op": "compact", "blocks": blocks, "seqs": min(200, max(1, blocks // rng.choice([5, 20, 50]))),
            "live": round(rng.uniform(0.05, 0.95), 3), "shared": round(rng.uniform(0.0, 0.6), 3), "layers": rng.randint(1, 6),
            "kv_heads": rng.choice([1, 4, 8]), "head_dim": 128, "block": 16, "dtype": "bf16"}


# ------------------------------------------------------------------------------------------------ inputs
# Lengths follow from the case alone, so that every seed gives outputs of the same shape; which pages and rows hold them, and all
# values, follow from the seed.

def _lengths():
    return torch.Generator().manual_seed(20)


def _randint(g, lo, hi, n=None):
    """Whole numbers in [lo, hi]: one as an int, or a list of n."""
    v = torch.randint(lo, hi + 1, (1 if n is None else n,), generator=g).tolist()
    return v[0] if n is None else v


def _values(shape, seed, dtype, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _pools(shape, seed, dtype):
    """Page pools, filled in slices so that no fp32 copy of the whole is held."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda", dtype=torch.float32))
    return out


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _prefix_layout(case, seed):
    """Lengths and pages of a prefix case: plain lists."""
    g = _lengths()
    B, n, m = case["block"], case["groups"], case["members"]
    cu_groups, prefix, q_len, ctx = [0], [], [], []
    for i in range(n):
        # sizes around the case's own: the first group has all of them, later ones one to `members`
        size = m if i == 0 else _randint(g, max(1, m // 2), m)
        p = case["prefix"] if i == 0 else _randint(g, max(1, case["prefix"] // 4), case["prefix"])
        prefix.append(p)
        cu_groups.append(cu_groups[-1] + size)
        for j in range(size):
            q = case["q_len"] if j == 0 else _randint(g, max(1, case["q_len"] // 3), case["q_len"])
            q_len.append(q)
            ctx.append(p + (case["suffix"] if j == 0 else _randint(g, q, max(q, case["suffix"]))))
    pages = [-(-c // B) for c in ctx]
    again = sum((cu_groups[i + 1] - cu_groups[i] - 1) * (p // B) for i, p in enumerate(prefix))
    perm = torch.randperm(sum(pages) - again + 8, generator=torch.Generator().manual_seed(seed)).tolist()     # a few pages belong to nobody
    tables, at = [], 0
    width = max(pages)
    for i in range(n):
        common = perm[at:at + prefix[i] // B]      # whole pages of the prefix are the group's
        at += len(common)
        for s in range(cu_groups[i], cu_groups[i + 1]):
            mine = perm[at:at + pages[s] - len(common)]
            at += len(mine)
            tables.append(common + mine + [-1] * (width - pages[s]))
    cu = [0]
    for q in q_len:
        cu.append(cu[-1] + q)
    return {"cu_groups": cu_groups, "prefix": prefix, "q_len": q_len, "ctx": ctx, "tables": tables, "cu": cu,
            "blocks": len(perm)}


def _prepare_prefix(case, seed):
    lay = _prefix_layout(case, seed)
    A = 128
    dt = torch.bfloat16
    T, S = lay["cu"][-1], len(lay["ctx"])
    shape = (lay["blocks"], case["kv_heads"], case["block"], A)
    k, v = _pools(shape, seed * 4 + 1, dt), _pools(shape, seed * 4 + 2, dt)
    # the partly filled page behind the shared ones is each sequence's own copy: it holds the same prefix keys
    B = case["block"]
    for i, p in enumerate(lay["prefix"]):
        if p % B:
            first = lay["tables"][lay["cu_groups"][i]][p // B]
            rest = [lay["tables"][s][p // B] for s in range(lay["cu_groups"][i] + 1, lay["cu_groups"][i + 1])]
            if rest:
                rest = torch.tensor(rest, device="cuda")
                k[rest, :, :p % B] = k[first, :, :p % B]
                v[rest, :, :p % B] = v[first, :, :p % B]
    state = {"case": case, "q": _values((T, case["heads"], A), seed * 4, dt, 2.0), "k": k, "v": v,
             "cu": _int32(lay["cu"]), "ctx": _int32(lay["ctx"]), "tables": _int32(lay["tables"]),
             "cu_groups": _int32(lay["cu_groups"]), "prefix": _int32(lay["prefix"]), "max_q": max(lay["q_len"]),
             "max_ctx": max(lay["ctx"]), "scale": 1.0 / math.sqrt(A), "out": torch.empty((T, case["heads"], A), dtype=dt, device="cuda")}
    if own:                                        # the workspace that a serving program keeps
        api = state["api"] = _api()
        state["cache"] = api.KVCache(k, v)
        n = api.cb_shared_prefix_workspace_size(state["cache"], case["heads"], S, T, len(lay["prefix"]), state["max_ctx"])
        state["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return state


def _cos_sin(positions, rot):
    """fp32 table [positions][rot]: cosines of each pair's angle, then sines; the angles in 64 bits."""
    inv = _ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _prepare_rope(case, seed):
    g = torch.Generator().manual_seed(seed)
    dt, A, T = _DTYPES[case["dtype"]], case["head_dim"], case["tokens"]
    H, K, B = case["heads"], case["kv_heads"], case["block"]
    if case["packed"]:                             # one projection's output: q | k | v of a token side by side
        qkv = _values((T, H + 2 * K, A), seed * 4, dt)
        q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    else:
        q, k, v = (_values((T, h, A), seed * 4 + i, dt) for i, h in enumerate((H, K, K)))
    blocks = T // B + 3
    pools = _pools((2, blocks, K, B, A), seed * 4 + 3, dt)
    slots = torch.randperm(blocks * B, generator=g)[:T]
    if T > 8:
        slots[T // 2] = -1                         # a token that is not cached
    state = {"case": case, "q": q, "k": k, "v": v, "pools": pools, "slots": slots.to(torch.int64).cuda(),
             "positions": _int32(_randint(g, 0, case["positions"] - 1, T)), "eps": 1e-6,
             "cos_sin": _cos_sin(case["positions"], case["rot_dim"]), "q_out": torch.empty((T, H, A), dtype=dt, device="cuda"),
             "wq": None, "wk": None}
    if case["norm"]:
        state["wq"], state["wk"] = ((1 + 0.2 * _values((A,), seed * 8 + i, torch.float32)).to(dt) for i in (4, 5))
    if own:
        state["api"] = _api()
        state["cache"] = state["api"].KVCache(pools[0], pools[1])
    return state


def _fork_layout(case, seed):
    g, pick = _lengths(), torch.Generator().manual_seed(seed)
    B, F, P = case["block"], case["forks"], case["parents"]
    ctx = [case["context"]] + _randint(g, max(1, case["context"] // 2), case["context"], P - 1) if P > 1 else [case["context"]]
    pages = [-(-c // B) for c in ctx]
    width = max(pages) + 2
    perm = torch.randperm(sum(pages) + F + 4, generator=pick).tolist()
    tables, at = [], 0
    for n in pages:
        tables.append(perm[at:at + n] + [-1] * (width - n))
        at += n
    rows = torch.randperm(P + F, generator=pick).tolist()   # parents and children sit anywhere in the table
    parents = list(range(P)) + _randint(g, 0, P - 1, F - P) if F > P else list(range(F))
    return {"ctx": ctx, "tables": tables, "width": width, "parent_rows": rows[:P], "parents": [rows[p] for p in parents],
            "children": rows[P:P + F], "new": perm[at:at + F], "blocks": len(perm)}


def _prepare_fork(case, seed):
    lay = _fork_layout(case, seed)
    rows = case["parents"] + case["forks"]
    tables, ctx = [[-1] * lay["width"] for _ in range(rows)], [0] * rows
    for r, c, t in zip(lay["parent_rows"], lay["ctx"], lay["tables"]):
        tables[r], ctx[r] = t, c
    pools = _pools((case["layers"], 2, lay["blocks"], case["kv_heads"], case["block"], case["head_dim"]), seed * 4 + 1, _DTYPES[case["dtype"]])
    state = {"case": case, "pools": pools, "tables": _int32(tables), "ctx": _int32(ctx), "parents": _int32(lay["parents"]),
             "children": _int32(lay["children"]), "new": _int32(lay["new"])}
    if own:
        state["api"] = _api()
        state["caches"] = state["api"].KVCacheStack([state["api"].KVCache(p[0], p[1]) for p in pools])
    return state


def _compact_layout(case, seed):
    """Block tables of a fragmented pool: random pages, a share of them in two sequences' tables."""
    g = _lengths()
    B, S = case["block"], case["seqs"]
    n_live = max(1, min(case["blocks"], int(case["blocks"] * case["live"])))
    perm = torch.randperm(case["blocks"], generator=torch.Generator().manual_seed(seed))[:n_live].tolist()
    cuts = sorted(_randint(g, 0, n_live, S - 1)) if S > 1 else []
    tables, ctx = [], []
    for a, b in zip([0] + cuts, cuts + [n_live]):
        mine = perm[a:b]
        if tables and torch.rand(1, generator=g).item() < case["shared"]:   # behind another sequence's first pages
            other = tables[_randint(g, 0, len(tables) - 1)]
            mine = other[:_randint(g, 0, len(other))] + mine
        tables.append(mine)
        ctx.append(max(0, len(mine) * B - _randint(g, 0, B - 1)))
    return tables, ctx


def _prepare_compact(case, seed):
    tables, ctx = _compact_layout(case, seed)
    width = max(max(len(t) for t in tables), 1) + 1
    pools = _pools((case["layers"], 2, case["blocks"], case["kv_heads"], case["block"], case["head_dim"]), seed * 4 + 1, _DTYPES[case["dtype"]])
    state = {"case": case, "pools": pools, "tables": _int32([t + [-1] * (width - len(t)) for t in tables]), "ctx": _int32(ctx)}
    state["new_tables"] = torch.empty_like(state["tables"])
    state["remap"] = torch.empty(case["blocks"], dtype=torch.int32, device="cuda")
    state["num_live"] = torch.empty(1, dtype=torch.int32, device="cuda")
    if own:                                        # the workspace that a serving program keeps
        api = state["api"] = _api()
        state["caches"] = api.KVCacheStack([api.KVCache(p[0], p[1]) for p in pools])
        state["workspace"] = torch.empty(api.cb_compact_workspace_size(case["blocks"]), dtype=torch.uint8, device="cuda")
    return state


def prepare(case, seed):
    return {"prefix": _prepare_prefix, "rope": _prepare_rope, "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](case, seed)


# ------------------------------------------------------------------------------------------------ one pass

def _run_prefix(s):
    if own:
        s["api"].cb_shared_prefix_attention(s["q"], s["cache"], s["cu"], s["ctx"], s["tables"], s["cu_groups"], s["prefix"],
                                          max_q_len=s["max_q"], max_context_len=s["max_ctx"], scale=s["scale"], out=s["out"],
                                          workspace=s["workspace"])
        return s["out"]
    # every sequence's keys and values, padded to the longest, against its padded query rows
    q, cu, ctx = s["q"], s["cu"].long(), s["ctx"].long()
    B, (T, H, A) = s["k"].shape[2], q.shape
    K, S, C, Q = s["k"].shape[1], ctx.numel(), s["max_ctx"], s["max_q"]
    pages = s["tables"].long().clamp(min=0)[:, :-(-C // B)]
    k = s["k"][pages].permute(0, 2, 1, 3, 4).reshape(S, K, -1, A)[:, :, :C].float()
    v = s["v"][pages].permute(0, 2, 1, 3, 4).reshape(S, K, -1, A)[:, :, :C].float()
    q_len = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=q.device)
    real = i[None] < q_len[:, None]                                     # [S, Q]
    rows = (cu[:-1, None] + i[None]).clamp(max=T - 1)
    qp = q[rows].float().view(S, Q, K, H // K, A).permute(0, 2, 3, 1, 4).reshape(S, K, (H // K) * Q, A) * s["scale"]
    j = torch.arange(C, device=q.device)
    seen = j[None, None] <= (ctx - q_len)[:, None, None] + i[None, :, None]     # row i sees keys up to p + i
    seen &= (j[None] < ctx[:, None])[:, None]
    score = (qp @ k.transpose(2, 3)).view(S, K, H // K, Q, C).masked_fill_(~seen[:, None, None], -math.inf)
    score = (score - score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    o = (score.view(S, K, -1, C) @ v).view(S, K, H // K, Q, A) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(S, Q, H, A)
    s["out"].copy_(o[real])
    return s["out"]


def _norm_rotate(x, w, eps, cos, sin, rot, interleaved):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _run_rope(s):
    c = s["case"]
    if own:
        s["api"].cb_norm_rope_append(s["q"], s["k"], s["v"], s["slots"], s["cache"], positions=s["positions"], q_out=s["q_out"],
                                   cos_sin=s["cos_sin"], q_weight=s["wq"], k_weight=s["wk"], eps=s["eps"], interleaved=c["interleaved"])
        return {"q": s["q_out"], "pools": s["pools"]}
    half = c["rot_dim"] // 2
    cs = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = cs[..., :half], cs[..., half:]
    s["q_out"].copy_(_norm_rotate(s["q"], s["wq"], s["eps"], cos, sin, c["rot_dim"], c["interleaved"]))
    k = _norm_rotate(s["k"], s["wk"], s["eps"], cos, sin, c["rot_dim"], c["interleaved"]).to(s["k"].dtype)
    slots = s["slots"]
    kept = slots >= 0
    blk, off = slots[kept] // c["block"], slots[kept] % c["block"]
    s["pools"][0][blk, :, off] = k[kept]
    s["pools"][1][blk, :, off] = s["v"][kept]
    return {"q": s["q_out"], "pools": s["pools"]}


def _run_fork(s):
    if own:
        s["api"].cb_fork_sequences(s["caches"], s["tables"], s["ctx"], s["parents"], s["children"], s["new"])
        return {"tables": s["tables"], "ctx": s["ctx"], "pools": s["pools"]}
    B = s["case"]["block"]
    parents, children = s["parents"].long(), s["children"].long()
    n = s["ctx"][parents].long()
    col = torch.arange(s["tables"].shape[1], device=n.device)[None]
    full, part = (n // B)[:, None], (n % B > 0)[:, None]
    rows = torch.where(col < full, s["tables"][parents], -1)
    rows = torch.where((col == full) & part, s["new"][:, None], rows)
    copy = part[:, 0]
    src = s["tables"][parents].gather(1, full.clamp(max=col.shape[1] - 1))[:, 0].long()[copy]
    dst = s["new"].long()[copy]
    held = (torch.arange(B, device=n.device)[None] < (n % B)[copy][:, None])[None, None, :, None, :, None]
    s["pools"][:, :, dst] = torch.where(held, s["pools"][:, :, src], s["pools"][:, :, dst])
    s["tables"][children] = rows
    s["ctx"][children] = n.int()
    return {"tables": s["tables"], "ctx": s["ctx"], "pools": s["pools"]}


def _run_compact(s):
    if own:
        s["api"].cb_compact_blocks(s["caches"], s["tables"], s["ctx"], new_block_tables=s["new_tables"], remap=s["remap"],
                                 num_live=s["num_live"], workspace=s["workspace"])
        return {"tables": s["new_tables"], "remap": s["remap"], "live": s["num_live"], "pools": s["pools"]}
    N, B = s["case"]["blocks"], s["case"]["block"]
    t = s["tables"].long()
    used = torch.arange(t.shape[1], device=t.device)[None] < ((s["ctx"].long() + B - 1) // B)[:, None]
    live = torch.zeros(N, dtype=torch.bool, device=t.device)
    live[t[used]] = True
    n = live.sum()
    ids = torch.arange(N, device=t.device)
    movers, holes = ids[live & (ids >= n)], ids[~live & (ids < n)]      # as many of the one as of the other
    remap = torch.where(live, ids, -1)
    remap[movers] = holes
    s["pools"][:, :, holes] = s["pools"][:, :, movers]
    s["remap"].copy_(remap)
    s["num_live"].copy_(n)
    s["new_tables"].copy_(torch.where(used, remap[t.clamp(min=0)], -1))
    return {"tables": s["new_tables"], "remap": s["remap"], "live": s["num_live"], "pools": s["pools"]}


def run(state):
    return {"prefix": _run_prefix, "rope": _run_rope, "fork": _run_fork, "compact": _run_compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    item = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "prefix":
        lay = _prefix_layout(case, 1)
        A, H, K, B = 128, case["heads"], case["kv_heads"], case["block"]
        keys = flops = 0
        for i, p in enumerate(lay["prefix"]):
            shared = p // B * B
            keys += shared
            for s in range(lay["cu_groups"][i], lay["cu_groups"][i + 1]):
                n, c = lay["q_len"][s], lay["ctx"][s]
                keys += c - shared
                flops += 4 * A * H * (n * (c - n) + n * (n + 1) // 2)
        return {"bytes": keys * 2 * K * A * 2 + 2 * lay["cu"][-1] * H * A * 2, "flops": flops}
    if case["op"] == "rope":
        row = case["head_dim"] * item
        T, H, K = case["tokens"], case["heads"], case["kv_heads"]
        return {"bytes": T * (2 * (H + 2 * K) * row + case["rot_dim"] * 4 + 12), "flops": T * (H + K) * case["head_dim"] * 8}
    page = case["layers"] * 2 * case["kv_heads"] * case["head_dim"] * item     # bytes of one token slot over all layers
    if case["op"] == "fork":
        lay = _fork_layout(case, 1)
        rest = dict(zip(lay["parent_rows"], [c % case["block"] for c in lay["ctx"]]))
        return {"bytes": page * (sum(rest[p] for p in set(lay["parents"])) + sum(rest[p] for p in lay["parents"]))
                + 8 * case["forks"] * lay["width"], "flops": 0}
    tables, _ = _compact_layout(case, 1)
    live = {b for t in tables for b in t}
    moves = sum(b >= len(live) for b in live)
    return {"bytes": 2 * moves * page * case["block"] + 8 * sum(map(len, tables)) + 4 * case["blocks"], "flops": 0}


# ------------------------------------------------------------------------------------------------ values in 64 bits

def _exact_prefix(case, seed):
    """softmax(q K^T) V of each sequence over its own table, one sequence after the other."""
    s, lay = _prepare_prefix(case, seed), _prefix_layout(case, seed)
    B, H, K = case["block"], case["heads"], case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for n, (c, q) in enumerate(zip(lay["ctx"], lay["q_len"])):
        pages = torch.tensor(lay["tables"][n][:-(-c // B)], device="cuda")
        k, v = (s[x][pages].transpose(1, 2).reshape(-1, K, 128)[:c].double() for x in ("k", "v"))
        x = s["q"][lay["cu"][n]:lay["cu"][n + 1]].double().view(q, K, H // K, 128)
        for h in range(K):
            w = torch.einsum("igd,jd->gij", x[:, h], k[:, h]) * s["scale"]
            late = torch.arange(c, device="cuda")[None] > torch.arange(c - q, c, device="cuda")[:, None]
            w = torch.softmax(w.masked_fill(late, -math.inf), -1)
            out[lay["cu"][n]:lay["cu"][n + 1], h * (H // K):(h + 1) * (H // K)] = torch.einsum("gij,jd->igd", w, v[:, h])
    return out


def _exact_rope(case, seed):
    s = _prepare_rope(case, seed)
    rot, A = case["rot_dim"], case["head_dim"]
    at = s["positions"].cpu().tolist()
    c, d = s["cos_sin"][at, :rot // 2].double(), s["cos_sin"][at, rot // 2:].double()

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.square().sum(-1, keepdim=True) / A + s["eps"]).sqrt() * w.double()
        y = x.clone()
        for p in range(rot // 2):
            i, j = (2 * p, 2 * p + 1) if case["interleaved"] else (p, p + rot // 2)
            y[..., i] = x[..., i] * c[:, None, p] - x[..., j] * d[:, None, p]
            y[..., j] = x[..., i] * d[:, None, p] + x[..., j] * c[:, None, p]
        return y

    k, pools = turned(s["k"], s["wk"]), s["pools"].double()
    for t, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            pools[0, slot // case["block"], :, slot % case["block"]] = k[t]
            pools[1, slot // case["block"], :, slot % case["block"]] = s["v"][t].double()
    return {"q": turned(s["q"], s["wq"]), "pools": pools}


def _exact_fork(case, seed):
    s, lay = _prepare_fork(case, seed), _fork_layout(case, seed)
    B = case["block"]
    tables, ctx = s["tables"].tolist(), s["ctx"].tolist()
    for p, c, new in zip(lay["parents"], lay["children"], lay["new"]):
        n = ctx[p]
        row = tables[p][:n // B]
        if n % B:
            s["pools"][:, :, new, :, :n % B] = s["pools"][:, :, tables[p][n // B], :, :n % B]
            row = row + [new]
        tables[c], ctx[c] = row + [-1] * (lay["width"] - len(row)), n
    return {"tables": _int32(tables), "ctx": _int32(ctx), "pools": s["pools"]}


def _exact_compact(case, seed):
    s = _prepare_compact(case, seed)
    tables, _ = _compact_layout(case, seed)
    live = sorted({b for t in tables for b in t})
    n = len(live)
    to = {b: b for b in live}
    held = set(live)
    to.update(zip([b for b in live if b >= n], [b for b in range(n) if b not in held]))
    for a, b in to.items():
        if a != b:
            s["pools"][:, :, b] = s["pools"][:, :, a]
    width = s["tables"].shape[1]
    return {"tables": _int32([[to[b] for b in t] + [-1] * (width - len(t)) for t in tables]),
            "remap": _int32([to.get(b, -1) for b in range(case["blocks"])]), "live": _int32([n]), "pools": s["pools"]}


def exact(case, seed):
    return {"prefix": _exact_prefix, "rope": _exact_rope, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](case, seed)
