"""The paged cache in 8 bits, case by case: inputs, plain forms and values in 64 bits.

Pages of e4m3 numbers with a fp32 scale for each page and key/value head (keys and values apart), and three operators:

  append   quantise a step's keys and values into the pages; a page that gets a larger token is scaled anew
  gather   read sequences' cached keys and values back, as rows of bf16 or fp32
  attend   attention of a packed step (decode rows and prompt chunks) over such a cache, prompts shared or not

A page's scale is the least power of two with which its largest number is at most 448, e4m3's largest; no page's falls while
tokens are added to it.  `run` computes an operator in elementary torch operations in fp32, or, where `own` is true, through the
library's entry points."""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_E4M3 = torch.float8_e4m3fn
_LEAST = -100          # exponent of the smallest scale


def _api():
    from continuous_batching_ragged_gb300 import api
    return api


def _attend_case(name, decodes, context, chunks, chunk, before, heads, kv_heads, block, prefix=0):
    """`decodes` sequences of one query token with up to `context` keys, then `chunks` prompt chunks of about `chunk` tokens, the
    last with `before` keys cached before it.  prefix > 0: all of them share that many keys."""
    return {"name": name, "op": "attend", "decodes": decodes, "context": context, "chunks": chunks, "chunk": chunk, "before": before,
            "heads": heads, "kv_heads": kv_heads, "block": block, "prefix": prefix}


def listed():
    return [
        # a small decode step's new rows, parts of one projection: latency
        {"name": "append 64 decode tokens", "op": "append", "decodes": 64, "chunks": 0, "chunk": 0, "kv_heads": 8, "head_dim": 128,
         "block": 16, "dtype": "bf16", "packed": True},
        # one prompt chunk in fp32, from the middle of a page on
        {"name": "append 661 tokens, fp32", "op": "append", "decodes": 0, "chunks": 1, "chunk": 661, "kv_heads": 4, "head_dim": 64,
         "block": 32, "dtype": "f32", "packed": False},
        # a whole step's token budget: decode rows and three prompt chunks, one key/value head per query head
        {"name": "append 2048-token step", "op": "append", "decodes": 64, "chunks": 3, "chunk": 662, "kv_heads": 32, "head_dim": 128,
         "block": 16, "dtype": "bf16", "packed": False},
        # one request's keys and values read back, to move it to another cache
        {"name": "gather 700 keys", "op": "gather", "seqs": 1, "keys": 700, "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "bf16"},
        # a batch read back, not from its first token on
        {"name": "gather 24 sequences", "op": "gather", "seqs": 24, "keys": 4096, "kv_heads": 32, "head_dim": 128, "block": 32, "dtype": "bf16"},
        # the smallest decode step, where latency counts
        _attend_case("attend 4 decode rows", 4, 512, 0, 0, 0, 32, 8, 16),
        # a full decode step, one key/value head per query head
        _attend_case("attend 256 decode rows, 32 heads", 256, 4096, 0, 0, 0, 32, 32, 16),
        # the same with grouped heads, an odd batch and pages of 32
        _attend_case("attend 201 decode rows, 32/8", 201, 4096, 0, 0, 0, 32, 8, 32),
        # one key/value head for all query heads
        _attend_case("attend 140 decode rows, 32/1", 140, 4096, 0, 0, 0, 32, 1, 64),
        # decode rows and prompt chunks in one step
        _attend_case("attend mixed step, 32/8", 64, 4096, 3, 662, 2048, 32, 8, 16),
        # the last chunk of a long prompt: the matrix products count
        _attend_case("attend 2048-token chunk", 0, 0, 1, 2048, 30720, 32, 32, 16),
        # chats behind one system prompt, whose pages they share
        _attend_case("attend 64 chats of one prompt", 64, 512, 0, 0, 0, 32, 8, 16, prefix=2048),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "gather", "attend", "attend"])
    if op == "append":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        c = {"op": op, "decodes": rng.choice([0, 1, _log_int(rng, 1, 256)]), "chunks": rng.randint(0, 4), "chunk": _log_int(rng, 2, 662),
             "kv_heads": rng.choice([1, 4, 8, 12, 32]), "head_dim": rng.choice([64, 128, 128]), "block": rng.choice([16, 16, 32, 64, 128]),
             "dtype": dtype, "packed": rng.random() < 0.5}
        if c["decodes"] + c["chunks"] == 0:
            c["decodes"] = 1
        if c["chunks"] == 0:
            c["chunk"] = 0
        if dtype == "f32" and c["kv_heads"] == 32:
            c["kv_heads"] = 16
        return c
    if op == "gather":
        c = {"op": op, "seqs": _log_int(rng, 1, 64), "keys": _log_int(rng, 1, 4096), "kv_heads": rng.choice([1, 4, 8, 12, 32]),
             "head_dim": rng.choice([64, 128, 128]), "block": rng.choice([16, 16, 32, 64, 128]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
        while c["seqs"] * c["keys"] * c["kv_heads"] * (2 if c["dtype"] == "f32" else 1) > 24 * 4096 * 24:
            c["seqs"] = c["seqs"] // 2 + 1
            c["keys"] = c["keys"] * 3 // 4
        return c
    heads, kv_heads = rng.choice([(32, 32), (32, 8), (32, 8), (32, 4), (32, 1), (16, 4), (8, 8), (12, 4), (24, 8)])
    kind = rng.choice(["decode", "decode", "mixed", "chunk"])
    decodes, context = (_log_int(rng, 1, 256), _log_int(rng, 1, 4096)) if kind != "chunk" else (0, 0)
    chunks = {"decode": 0, "mixed": rng.randint(1, 4), "chunk": rng.randint(1, 3)}[kind]
    chunk = _log_int(rng, 2, 662 if kind == "mixed" or chunks > 1 else 2048) if chunks else 0
    before = rng.choice([0, _log_int(rng, 1, 4096 if kind == "mixed" or chunks > 1 else 30720)]) if chunks else 0
    prefix = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])
    # no more than the largest listed ones: padded keys, and padded scores
    longest = prefix + max(context, before + chunk)
    while (decodes + chunks) * longest * kv_heads > 256 * 4096 * 32 or (decodes + chunks) * heads * max(1, chunk) * longest > 32 * 2048 * 32768:
        decodes, context, before, prefix = decodes // 2 + (chunks == 0), context * 3 // 4 + 1, before * 3 // 4, prefix * 3 // 4
        longest = prefix + max(context, before + chunk)
        if decodes <= 1:
            chunk = max(2, chunk * 3 // 4) if chunks else 0
    return {"op": "attend", "decodes": decodes, "context": context, "chunks": chunks, "chunk": chunk, "before": before,
            "heads": heads, "kv_heads": kv_heads, "block": rng.choice([16, 16, 32, 64, 128]), "prefix": prefix}


# ------------------------------------------------------------------------------------------------ inputs
# Lengths follow from the case alone, so that every seed gives outputs of the same shape; which pages and rows hold them, and all
# values, follow from the seed.

def _lengths():
    return torch.Generator().manual_seed(20)


def _randint(g, lo, hi, n=None):
    """Whole numbers in [lo, hi]: one as an int, or a list of n."""
    v = torch.randint(lo, max(lo, hi) + 1, (1 if n is None else n,), generator=g).tolist()
    return v[0] if n is None else v


def _values(shape, seed, dtype, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(blocks, heads, block, dim, seed):
    """A filled pool of e4m3 pages and its scales: numbers of about 1, of another size in each page and head; in slices, so that no
    fp32 copy of the whole is held."""
    q = torch.empty((blocks, heads, block, dim), dtype=_E4M3, device="cuda")
    s = torch.empty((blocks, heads), dtype=torch.float32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    step = max(1, (1 << 26) // (heads * block * dim))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        x = torch.randn((n, heads, block, dim), generator=g, device="cuda")
        x *= torch.exp2(2 * torch.rand((n, heads, 1, 1), generator=g, device="cuda") - 1)
        m, e = torch.frexp(x.abs().amax((2, 3)))
        s[i:i + n] = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875))
        q[i:i + n] = (x / s[i:i + n, :, None, None]).to(_E4M3)
    return q, s


def _append_layout(case, seed):
    """Tokens cached before the step and new ones, per sequence; its pages; the slots of all new tokens."""
    g = _lengths()
    B = case["block"]
    new = [1] * case["decodes"] + ([case["chunk"]] + _randint(g, max(1, case["chunk"] - 1), case["chunk"], case["chunks"] - 1) if case["chunks"] > 1
                                   else [case["chunk"]] * case["chunks"])
    old = _randint(g, 0, 2 * B, len(new))
    if len(old) > 1:
        old[1] = B                                 # one that begins a page
    # pages that the step writes to, and the ones before them
    pages = [-(-(o + n) // B) for o, n in zip(old, new)]
    perm = torch.randperm(sum(pages) + 3, generator=torch.Generator().manual_seed(seed)).tolist()
    slots, at = [], 0
    for o, n, p in zip(old, new, pages):
        mine = perm[at:at + p]
        at += p
        slots += [mine[j // B] * B + j % B for j in range(o, o + n)]
    if len(slots) > 8:
        slots[len(slots) // 2] = -1                # a token that is not cached
    return {"old": old, "new": new, "slots": slots, "blocks": len(perm)}


def _prepare_append(case, seed):
    lay = _append_layout(case, seed)
    T, K, A, dt = len(lay["slots"]), case["kv_heads"], case["head_dim"], _DTYPES[case["dtype"]]
    if case["packed"]:                             # parts of one projection's output: the query heads, then k, then v
        qkv = _values((T, 6 * K, A), seed * 4, dt, 1.5)
        k, v = qkv[:, 4 * K:5 * K], qkv[:, 5 * K:]
    else:
        k, v = (_values((T, K, A), seed * 4 + i, dt, 1.5) for i in range(2))
    pk, sk = _pool(lay["blocks"], K, case["block"], A, seed * 4 + 2)
    pv, sv = _pool(lay["blocks"], K, case["block"], A, seed * 4 + 3)
    state = {"case": case, "k_new": k, "v_new": v, "slots": torch.tensor(lay["slots"], dtype=torch.int64, device="cuda"),
             "k": pk, "v": pv, "k_scale": sk, "v_scale": sv}
    if own:
        state["api"] = _api()
        state["cache"] = state["api"].QuantKVCache(pk, pv, sk, sv)
    return state


def _gather_layout(case, seed):
    g = _lengths()
    B, S = case["block"], case["seqs"]
    keys = [case["keys"]] + (_randint(g, max(1, case["keys"] // 8), case["keys"], S - 1) if S > 1 else [])
    starts = [0] + (_randint(g, 0, min(3 * B, max(1, case["keys"] // 16)), S - 1) if S > 1 else [])
    pages = [-(-(a + n) // B) for a, n in zip(starts, keys)]
    perm = torch.randperm(sum(pages) + 2, generator=torch.Generator().manual_seed(seed)).tolist()
    tables, at = [], 0
    for p in pages:
        tables.append(perm[at:at + p] + [-1] * (max(pages) - p))
        at += p
    cu = [0]
    for n in keys:
        cu.append(cu[-1] + n)
    return {"starts": starts, "cu": cu, "tables": tables, "blocks": len(perm)}


def _prepare_gather(case, seed):
    lay = _gather_layout(case, seed)
    K, A = case["kv_heads"], case["head_dim"]
    pk, sk = _pool(lay["blocks"], K, case["block"], A, seed * 4 + 2)
    pv, sv = _pool(lay["blocks"], K, case["block"], A, seed * 4 + 3)
    k_out, v_out = (torch.empty((lay["cu"][-1], K, A), dtype=_DTYPES[case["dtype"]], device="cuda") for _ in range(2))
    state = {"case": case, "k": pk, "v": pv, "k_scale": sk, "v_scale": sv, "tables": _int32(lay["tables"]), "cu": _int32(lay["cu"]),
             "starts": _int32(lay["starts"]), "k_out": k_out, "v_out": v_out}
    if own:
        state["api"] = _api()
        state["cache"] = state["api"].QuantKVCache(pk, pv, sk, sv)
    return state


def _attend_layout(case, seed):
    g = _lengths()
    B, p = case["block"], case["prefix"]
    q_len, ctx = [], []
    if case["decodes"]:
        q_len += [1] * case["decodes"]
        ctx += [p + case["context"]] + [p + c for c in _randint(g, max(1, case["context"] // 8), case["context"], case["decodes"] - 1)] \
            if case["decodes"] > 1 else [p + case["context"]]
    for i in range(case["chunks"]):
        n = case["chunk"] if i == case["chunks"] - 1 else _randint(g, max(1, case["chunk"] - 1), case["chunk"])
        q_len.append(n)
        ctx.append(p + n + case["before"] * (i + 1) // case["chunks"])
    shared = p // B                                # whole pages of the prefix are everybody's
    pages = [-(-c // B) for c in ctx]
    perm = torch.randperm(sum(n - shared for n in pages) + shared + 4, generator=torch.Generator().manual_seed(seed)).tolist()
    tables, at = [], shared
    for n in pages:
        mine = perm[at:at + n - shared]
        at += len(mine)
        tables.append(perm[:shared] + mine + [-1] * (max(pages) - n))
    cu = [0]
    for n in q_len:
        cu.append(cu[-1] + n)
    return {"q_len": q_len, "ctx": ctx, "tables": tables, "cu": cu, "blocks": len(perm)}


def _prepare_attend(case, seed):
    lay = _attend_layout(case, seed)
    A, H, K = 128, case["heads"], case["kv_heads"]
    T, S = lay["cu"][-1], len(lay["ctx"])
    pk, sk = _pool(lay["blocks"], K, case["block"], A, seed * 4 + 2)
    pv, sv = _pool(lay["blocks"], K, case["block"], A, seed * 4 + 3)
    state = {"case": case, "q": _values((T, H, A), seed * 4, torch.bfloat16, 1.5), "k": pk, "v": pv, "k_scale": sk, "v_scale": sv,
             "cu": _int32(lay["cu"]), "ctx": _int32(lay["ctx"]), "tables": _int32(lay["tables"]), "max_q": max(lay["q_len"]),
             "max_ctx": max(lay["ctx"]), "scale": 1.0 / math.sqrt(A), "out": torch.empty((T, H, A), dtype=torch.bfloat16, device="cuda"),
             "groups": _int32([0, S]) if case["prefix"] else None, "prefix": _int32([case["prefix"]]) if case["prefix"] else None}
    if own:                                        # the workspace that a serving program keeps
        api = state["api"] = _api()
        state["cache"] = api.QuantKVCache(pk, pv, sk, sv)
        n = api.cb_ragged_attention_q8_workspace_size(state["cache"], H, S, T, state["max_ctx"], num_groups=1 if case["prefix"] else 0)
        state["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return state


def prepare(case, seed):
    return {"append": _prepare_append, "gather": _prepare_gather, "attend": _prepare_attend}[case["op"]](case, seed)


# ------------------------------------------------------------------------------------------------ one pass

def _pages(pool, *at):
    """pool[at] in fp32."""
    return pool.view(torch.uint8)[at].view(_E4M3).float()


def _append_one(new, slots, pool, scale, B):
    """Keys or values: rows new [T, K, A] of the tokens that are cached, into pool and scale."""
    page, off = slots // B, slots % B
    first = torch.full((pool.shape[0],), B, dtype=torch.int64, device=pool.device).scatter_reduce_(0, page, off, "amin")
    amax = torch.zeros_like(scale).index_reduce_(0, page, new.abs().amax(2), "amax")
    m, e = torch.frexp(amax)
    needed = torch.ldexp(torch.ones_like(m), (e - 9 + (m > 0.875)).clamp(min=_LEAST))
    lead = torch.ones_like(page, dtype=torch.bool)
    lead[1:] = page[1:] != page[:-1]               # a page's tokens follow one another
    pages = page[lead]
    old = scale[pages]
    held = first[pages] > 0                        # the page has tokens before the first new one: their scale counts
    s = torch.where(held[:, None], torch.maximum(old, needed[pages]), needed[pages])
    x = _pages(pool, pages)
    before = torch.arange(B, device=pool.device) < first[pages][:, None]
    x = torch.where(before[:, None, :, None], x * (old / s)[:, :, None, None], x).to(_E4M3)
    pool.view(torch.uint8)[pages] = x.view(torch.uint8)
    scale[pages] = s
    pool.view(torch.uint8)[page, :, off] = (new / scale[page][:, :, None]).to(_E4M3).view(torch.uint8)


def _run_append(s):
    if own:
        s["api"].cb_append_kv_q8(s["k_new"], s["v_new"], s["slots"], s["cache"])
    else:
        kept = s["slots"] >= 0
        _append_one(s["k_new"].float()[kept], s["slots"][kept], s["k"], s["k_scale"], s["case"]["block"])
        _append_one(s["v_new"].float()[kept], s["slots"][kept], s["v"], s["v_scale"], s["case"]["block"])
    return {"k": s["k"], "k_scale": s["k_scale"], "v": s["v"], "v_scale": s["v_scale"]}


def _run_gather(s):
    if own:
        s["api"].cb_gather_kv_q8(s["cache"], s["tables"], s["cu"], k_out=s["k_out"], v_out=s["v_out"], starts=s["starts"])
        return {"k": s["k_out"], "v": s["v_out"]}
    B, cu = s["case"]["block"], s["cu"].long()
    row = torch.arange(s["k_out"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    at = s["starts"].long()[seq] + row - cu[seq]
    page, off = s["tables"].long()[seq, at // B], at % B
    s["k_out"].copy_(_pages(s["k"], page, slice(None), off) * s["k_scale"][page][:, :, None])
    s["v_out"].copy_(_pages(s["v"], page, slice(None), off) * s["v_scale"][page][:, :, None])
    return {"k": s["k_out"], "v": s["v_out"]}


def _run_attend(s):
    if own:
        s["api"].cb_ragged_attention_q8(s["q"], s["cache"], s["cu"], s["ctx"], s["tables"], max_q_len=s["max_q"], max_context_len=s["max_ctx"],
                                        scale=s["scale"], out=s["out"], workspace=s["workspace"], cu_groups=s["groups"], prefix_lens=s["prefix"])
        return s["out"]
    # every sequence's keys and values, padded to the longest, against its padded query rows
    q, cu, ctx = s["q"], s["cu"].long(), s["ctx"].long()
    B, (T, H, A) = s["case"]["block"], q.shape
    K, S, C, Q = s["k"].shape[1], ctx.numel(), s["max_ctx"], s["max_q"]
    pages = s["tables"].long().clamp(min=0)[:, :-(-C // B)]
    k = (_pages(s["k"], pages) * s["k_scale"][pages][..., None, None]).transpose(1, 2).reshape(S, K, -1, A)[:, :, :C]
    q_len = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=q.device)
    real = i[None] < q_len[:, None]                                     # [S, Q]
    rows = (cu[:-1, None] + i[None]).clamp(max=T - 1)
    qp = q[rows].float().view(S, Q, K, H // K, A).permute(0, 2, 3, 1, 4).reshape(S, K, (H // K) * Q, A) * s["scale"]
    j = torch.arange(C, device=q.device)
    seen = j[None, None] <= (ctx - q_len)[:, None, None] + i[None, :, None]     # row i sees keys up to p + i
    seen &= (j[None] < ctx[:, None])[:, None]
    score = (qp @ k.transpose(2, 3)).view(S, K, H // K, Q, C).masked_fill_(~seen[:, None, None], -math.inf)
    del k
    score = (score - score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    v = (_pages(s["v"], pages) * s["v_scale"][pages][..., None, None]).transpose(1, 2).reshape(S, K, -1, A)[:, :, :C]
    o = (score.view(S, K, -1, C) @ v).view(S, K, H // K, Q, A) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(S, Q, H, A)
    s["out"].copy_(o[real])
    return s["out"]


def run(state):
    return {"append": _run_append, "gather": _run_gather, "attend": _run_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    K = case["kv_heads"]
    if case["op"] == "append":
        lay = _append_layout(case, 1)
        item, T = 4 if case["dtype"] == "f32" else 2, len(lay["slots"])
        pages = len({x // case["block"] for x in lay["slots"] if x >= 0})
        return {"bytes": T * (2 * K * case["head_dim"] * (item + 1) + 8) + pages * 2 * K * 8, "flops": 4 * T * K * case["head_dim"]}
    if case["op"] == "gather":
        lay = _gather_layout(case, 1)
        item, R = 4 if case["dtype"] == "f32" else 2, lay["cu"][-1]
        pages = sum(-(-(a + n) // case["block"]) - a // case["block"] for a, n in zip(lay["starts"], (b - c for b, c in zip(lay["cu"][1:], lay["cu"]))))
        return {"bytes": R * 2 * K * case["head_dim"] * (1 + item) + pages * (4 + 8 * K), "flops": R * 2 * K * case["head_dim"]}
    lay = _attend_layout(case, 1)
    A, H, B = 128, case["heads"], case["block"]
    shared = case["prefix"] // B * B if len(lay["ctx"]) > 1 else 0
    keys, flops = shared, 0
    for n, c in zip(lay["q_len"], lay["ctx"]):
        keys += c - shared
        flops += 4 * A * H * (n * (c - n) + n * (n + 1) // 2)
    return {"bytes": keys * 2 * K * A + -(-keys // B) * 8 * K + 2 * lay["cu"][-1] * H * A * 2, "flops": flops}


# ------------------------------------------------------------------------------------------------ values in 64 bits

def _grid(x):
    """64-bit numbers, at most 448, to the nearest e4m3 ones (four significant bits, the step 2^-9 below 2^-6), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_append(case, seed):
    s, lay = _prepare_append(case, seed), _append_layout(case, seed)
    B = case["block"]
    out = {}
    for name in ("k", "v"):
        q, scale, new = s[name].double(), s[name + "_scale"].double(), s[name + "_new"].double()
        by_page = {}
        for t, slot in enumerate(lay["slots"]):
            if slot >= 0:
                by_page.setdefault(slot // B, []).append((t, slot % B))
        for page, toks in by_page.items():
            t, off = [a for a, _ in toks], [b for _, b in toks]
            x = new[t].transpose(0, 1)             # [K, n, A]
            # the logarithm of a power of two may come out a last bit too large; the next numbers' are 1e-7 away
            need = torch.exp2(torch.ceil(torch.log2(x.abs().amax((1, 2)) / 448) - 1e-9).clamp(min=_LEAST))
            if off[0] > 0:
                need = torch.maximum(need, scale[page])
                q[page, :, :off[0]] = _grid(q[page, :, :off[0]] * scale[page, :, None, None] / need[:, None, None])
            scale[page] = need
            q[page][:, off] = _grid(x / need[:, None, None])
        out[name], out[name + "_scale"] = q, scale
    return out


def _exact_gather(case, seed):
    s, lay = _prepare_gather(case, seed), _gather_layout(case, seed)
    B = case["block"]
    out = {"k": [], "v": []}
    for n, table in enumerate(lay["tables"]):
        a, keys = lay["starts"][n], lay["cu"][n + 1] - lay["cu"][n]
        pages = torch.tensor(table[:-(-(a + keys) // B)], device="cuda")
        for name in ("k", "v"):
            x = _pages(s[name], pages).double() * s[name + "_scale"][pages].double()[:, :, None, None]
            out[name].append(x.transpose(1, 2).reshape(-1, case["kv_heads"], case["head_dim"])[a:a + keys])
    return {name: torch.cat(x) for name, x in out.items()}


def _exact_attend(case, seed):
    """softmax(q K^T) V of each sequence over its own table, one sequence and head after the other."""
    s, lay = _prepare_attend(case, seed), _attend_layout(case, seed)
    B, H, K = case["block"], case["heads"], case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for n, (c, q) in enumerate(zip(lay["ctx"], lay["q_len"])):
        pages = torch.tensor(lay["tables"][n][:-(-c // B)], device="cuda")
        x = s["q"][lay["cu"][n]:lay["cu"][n + 1]].double().view(q, K, H // K, 128)
        k, v = ((_pages(s[y], pages) * s[y + "_scale"][pages][:, :, None, None]).transpose(0, 1).reshape(K, -1, 128)[:, :c].double()
                for y in ("k", "v"))
        late = torch.arange(c, device="cuda")[None] > torch.arange(c - q, c, device="cuda")[:, None]
        for h in range(0, K, K if q == 1 else 1):  # all heads of a decode row at once, one of a chunk
            hs = slice(h, h + (K if q == 1 else 1))
            w = torch.einsum("ihgd,hjd->hgij", x[:, hs], k[hs]) * s["scale"]
            w = torch.softmax(w.masked_fill_(late, -math.inf), -1)
            y = torch.einsum("hgij,hjd->ihgd", w, v[hs])
            out[lay["cu"][n]:lay["cu"][n + 1], hs.start * (H // K):hs.stop * (H // K)] = y.reshape(q, -1, 128)
    return out


def exact(case, seed):
    return {"append": _exact_append, "gather": _exact_gather, "attend": _exact_attend}[case["op"]](case, seed)
