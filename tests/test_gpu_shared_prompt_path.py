"""Samples of prompts through the operators together, as a serving loop uses them:
the prompt is appended (norm, rotation, cache) and attended, forked into samples,
every sample decodes tokens of its own over the shared pages, some finish, the pool
is compacted and the others go on.  After each step the cached rows are compared
with norm and rotation in 64 bits, and the attention with softmax(q K^T) V in 64
bits over the rows that the cache holds."""
import math

import pytest
import torch

from test_gpu_norm_rope import close, turned

pytestmark = pytest.mark.gpu

A, B, LAYERS, H, K = 128, 16, 2, 16, 8
SCALE = 1 / math.sqrt(A)


class Loop:
    """Tables and lengths as a serving program keeps them, on the host; rows are never reused."""

    def __init__(self, num_blocks, max_rows, width, seed):
        from continuous_batching_ragged_gb300 import api
        self.api = api
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        nan = lambda: torch.full((num_blocks, K, B, A), float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.stack = api.KVCacheStack([api.KVCache(nan(), nan()) for _ in range(LAYERS)])
        self.tables = torch.full((max_rows, width), -1, dtype=torch.int32, device="cuda")
        self.ctx = torch.zeros(max_rows, dtype=torch.int32, device="cuda")
        self.free = list(range(num_blocks))
        ang = torch.arange(8192, dtype=torch.float64, device="cuda")[:, None] * 1e4 ** (
            -torch.arange(0, A, 2, dtype=torch.float64, device="cuda") / A)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        self.w = [(1 + 0.2 * torch.randn(A, generator=self.g, device="cuda")).bfloat16() for _ in range(2)]
        self.expected = {}                           # (layer, row) -> [(position, exact k, magnitude, v), ...]

    def step(self, rows, n_new, cu_groups, prefix):
        """n_new tokens for each row, through every layer; checks caches and outputs."""
        api, ctx0, tables = self.api, self.ctx.tolist(), self.tables.tolist()
        cu, slots, pos = [0], [], []
        for r, n in zip(rows, n_new):
            for p in range(ctx0[r], ctx0[r] + n):
                if p % B == 0:
                    tables[r][p // B] = self.free.pop(0)
                slots.append(tables[r][p // B] * B + p % B)
                pos.append(p)
            cu.append(cu[-1] + n)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.tables.copy_(i32(tables))
        self.ctx[rows] += i32(n_new)
        T, S, ctx = cu[-1], len(rows), self.ctx[rows].contiguous()
        step_tables, max_ctx = self.tables[rows].contiguous(), int(ctx.max())
        pos, slots = i32(pos), torch.tensor(slots, dtype=torch.int64, device="cuda")
        q_out = torch.empty((T, H, A), dtype=torch.bfloat16, device="cuda")
        for layer, cache in enumerate(self.stack.caches):
            qkv = torch.randn((T, H + 2 * K, A), generator=self.g, device="cuda").bfloat16()
            q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
            api.cb_norm_rope_append(q, k, v, slots, cache, q_out=q_out, positions=pos, cos_sin=self.cos_sin,
                                    q_weight=self.w[0], k_weight=self.w[1], eps=1e-5)
            out = torch.full_like(q_out, float("nan"))
            if cu_groups is None:
                ws = api.cb_attention_workspace_size_gqa(cache, H, S, T, max_ctx)
                api.cb_ragged_attention_gqa(q_out, cache, i32(cu), ctx, step_tables, max_q_len=max(n_new), max_context_len=max_ctx,
                                            scale=SCALE, out=out, workspace=torch.empty(ws, dtype=torch.uint8, device="cuda"))
            else:
                ws = api.cb_shared_prefix_workspace_size(cache, H, S, T, len(prefix), max_ctx)
                api.cb_shared_prefix_attention(q_out, cache, i32(cu), ctx, step_tables, i32(cu_groups), i32(prefix),
                                               max_q_len=max(n_new), max_context_len=max_ctx, scale=SCALE, out=out,
                                               workspace=torch.empty(ws, dtype=torch.uint8, device="cuda"))
            api.cb_check_device_errors()
            close(q_out, *turned(q, self.w[0], 1e-5, self.cos_sin, pos, False))
            exact, mag = turned(k, self.w[1], 1e-5, self.cos_sin, pos, False)
            for i, r in enumerate(rows):
                a, b = cu[i], cu[i + 1]
                self.expected.setdefault((layer, r), []).append((exact[a:b], mag[a:b], v[a:b].clone()))
                self.check(cache, layer, r, q_out[a:b], out[a:b])

    def check(self, cache, layer, r, q, out):
        n, j = int(self.ctx[r]), torch.arange(int(self.ctx[r]), device="cuda")
        page = self.tables[r].long()[j // B]
        k, v = cache.k[page, :, j % B], cache.v[page, :, j % B]
        exact, mag, value = (torch.cat(x) for x in zip(*self.expected[layer, r]))
        close(k, exact, mag)
        assert torch.equal(v, value)
        m, G = len(q), H // K
        late = j[None] > torch.arange(n - m, n, device="cuda")[:, None]
        s = torch.einsum("ihgd,jhd->hgij", q.double().view(m, K, G, A), k.double()) * SCALE
        p = torch.softmax(s.masked_fill(late, -math.inf), -1)
        want = torch.einsum("hgij,jhd->ihgd", p, v.double()).reshape(m, H, A)
        size = torch.einsum("hgij,jhd->ihgd", p, v.double().abs()).reshape(m, H, A)
        # P and the output rounded to bf16, each by half a step, 2^-8; and 2^-10 of P for scores summed in fp32: 128
        # products of at most 40 in all are off by 128 * 2^-24 * 40, so the ratio of two exponentials by twice that, 2^-10.6
        off, lim = (out.double() - want).abs(), (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -8 * want.abs()
        assert bool((off <= lim).all()), float((off - lim).max())

    def fork(self, parent, children):
        new = [self.free.pop(0) for _ in children]
        self.api.cb_fork_sequences(self.stack, self.tables, self.ctx, *(
            torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([parent] * len(children), children, new)))
        self.api.cb_check_device_errors()
        for c in children:
            for layer in range(LAYERS):
                self.expected[layer, c] = list(self.expected[layer, parent])
        if int(self.ctx[parent]) % B == 0:            # ends on a page border: no copies were needed
            self.free = new + self.free

    def compact(self, rows):
        n = self.stack.caches[0].num_blocks
        live, remap = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
        tables, ctx = self.tables[rows].contiguous(), self.ctx[rows].contiguous()
        self.api.cb_compact_blocks(self.stack, tables, ctx, new_block_tables=tables, remap=remap, num_live=live,
                                   workspace=torch.empty(self.api.cb_compact_workspace_size(n), dtype=torch.uint8, device="cuda"))
        self.api.cb_check_device_errors()
        self.tables.fill_(-1)
        self.tables[rows] = tables
        self.free = list(range(int(live), n))
        for cache in self.stack.caches:               # what is free holds nothing that anyone needs
            cache.k[int(live):] = float("nan")
            cache.v[int(live):] = float("nan")
        return int(live)


@pytest.mark.parametrize("long", [300, 5000])          # of 8 heads: shared reads would save 13 MB, and do save 205 MB
def test_samples_of_two_prompts(native_lib, long):
    short, samples = 37, 12
    loop = Loop(num_blocks=700, max_rows=32, width=330, seed=1)
    loop.step([0, 20], [long, short], None, None)                       # both prompts
    loop.fork(0, list(range(1, samples)))
    loop.fork(20, [21, 22])
    group = list(range(samples)) + [20, 21, 22]
    for n in (1, 1, 1, 3):                                              # samples decode, one step with three tokens each
        loop.step(group, [n] * len(group), [0, samples, samples + 3], [long, short])
    kept = [0, 2, 3, 5, 6, 7, 8, 9, 10, 11, 20, 22]                     # three samples finish
    used = {b for r in kept for b in loop.tables[r, :-(-int(loop.ctx[r]) // B)].tolist()}
    assert loop.compact(kept) == len(used)
    for _ in range(14):                                                 # past the next page border
        loop.step(kept, [1] * len(kept), [0, 10, 12], [long, short])
    loop.fork(5, [12, 13])                                              # a sample branches again
    kept = kept[:4] + [12, 13] + kept[4:]
    loop.step(kept, [1, 30] + [1] * (len(kept) - 2), [0, 12, 14], [long, short])
