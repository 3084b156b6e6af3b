"""cb_append_kv_q8 and cb_gather_kv_q8 against their rules restated in 64 bits.

Scales are powers of two, so dividing by one is exact and each number is rounded
once, to the nearest e4m3 number: the comparisons of e4m3 numbers and scales are
exact.  What is read back is number * scale, exact in fp32 (four significant bits)
and in bf16, wherever the scale is a power of two; with other scales, rounded once."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def grid(x):
    """The nearest e4m3 numbers to 64-bit numbers of magnitude up to 448, ties to even; NaN for what is not finite."""
    m, e = torch.frexp(x.abs().clamp(min=2.0 ** -6))
    step = torch.ldexp(torch.ones_like(m), e - 4)
    y = torch.round(x / step) * step
    return torch.where(torch.isfinite(x), y, float("nan"))


def need(amax):
    """The least power of two, 2^-100 or more, with amax <= 448 of it."""
    e = -100
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append_plain(new, slots, q, scale):
    """One token run after the other; q, scale: 64-bit copies, written in place."""
    B = q.shape[2]
    runs = []
    for t, s in enumerate(slots):
        if s < 0 or s >= q.shape[0] * B:
            continue
        if runs and runs[-1][0] == s // B:
            runs[-1][1].append((t, s % B))
        else:
            runs.append((s // B, [(t, s % B)]))
    for page, toks in runs:
        first = toks[0][1]
        for h in range(q.shape[1]):
            x = new[[t for t, _ in toks], h]
            fine = x[torch.isfinite(x)].abs()
            s = need(float(fine.max()) if fine.numel() else 0.0)
            if first > 0:
                s = max(s, float(scale[page, h]))
                if s > float(scale[page, h]):
                    q[page, h, :first] = grid(q[page, h, :first] * float(scale[page, h]) / s)
            scale[page, h] = s
            for (t, o), row in zip(toks, x):
                q[page, h, o] = grid(row / s)


def same(a, b):
    """Equal numbers, NaN where NaN."""
    a, b = a.double().cpu(), b.double().cpu()
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


class Pool:
    def __init__(self, blocks, K, B, A, seed=0):
        from continuous_batching_ragged_gb300 import api
        g = torch.Generator().manual_seed(seed)
        self.k, self.v = (torch.randn((blocks, K, B, A), generator=g).mul(60).clamp(-448, 448).to(E4M3).cuda() for _ in range(2))
        self.ks, self.vs = (torch.exp2(torch.randint(-9, -5, (blocks, K), generator=g).float()).cuda() for _ in range(2))
        self.cache = api.QuantKVCache(self.k, self.v, self.ks, self.vs)
        self.want = [x.double().cpu() for x in (self.k, self.v, self.ks, self.vs)]

    def append(self, k, v, slots, **kw):
        from continuous_batching_ragged_gb300 import api
        api.cb_append_kv_q8(k, v, torch.tensor(slots, dtype=torch.int64, device="cuda"), self.cache, **kw)

    def plain(self, k, v, slots):
        wk, wv, ws, wt = self.want
        append_plain(k.double().cpu(), slots, wk, ws)
        append_plain(v.double().cpu(), slots, wv, wt)

    def check(self):
        for name, got, want in zip(("k", "v", "k_scale", "v_scale"), (self.k, self.v, self.ks, self.vs), self.want):
            assert same(got, want), name


def rows(T, K, A, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K, A), generator=g) * scale
    return (x * torch.exp2(4 * torch.rand((T, K, 1), generator=g) - 2)).to(DT[dtype]).cuda()


def chunk_slots(page_ids, B, start, n):
    return [page_ids[j // B] * B + j % B for j in range(start, start + n)]


SHAPES = [(1, 16, 128, "bf16"), (8, 16, 128, "bf16"), (3, 32, 64, "bf16"), (5, 8, 256, "bf16"), (4, 64, 64, "f32"), (2, 128, 128, "f32"),
          (32, 16, 128, "bf16"), (3, 1, 128, "bf16"), (2, 256, 64, "bf16")]


@pytest.mark.parametrize("K,B,A,dtype", SHAPES)
def test_append(native_lib, K, B, A, dtype):
    """Decode rows at every kind of place in a page, and chunks that begin and end inside pages, begin one, fill one,
    and span several; skipped tokens between; numbers of widely different size."""
    from continuous_batching_ragged_gb300 import api
    n = 3 * B + 3
    p = Pool(40, K, B, A)
    ids = torch.randperm(40, generator=torch.Generator().manual_seed(1)).tolist()
    slots = [ids[0] * B, ids[1] * B + B - 1, ids[2] * B + B // 2]                      # decode rows
    slots += chunk_slots(ids[20:30], B, B // 3, n)
    slots += [-1, -1]
    slots += chunk_slots(ids[8:12], B, 0, B)
    slots += chunk_slots(ids[12:14], B, B - 1, 1)
    tail = chunk_slots(ids[14:20], B, 0, 2 * B + 1)
    tail[len(tail) // 2] = -1                                                          # a token that is not cached, inside a page
    slots += tail + [-5]
    k, v = (rows(len(slots), K, A, dtype, s) for s in (2, 3))
    p.append(k, v, slots)
    api.cb_check_device_errors()
    p.plain(k, v, slots)
    p.check()


@pytest.mark.parametrize("growth", [0.25, 1.0, 3.0, 100.0])
def test_token_by_token(native_lib, growth):
    """A page filled one token a call, the tokens shrinking, alike and growing: scales that stay and that grow at every token."""
    from continuous_batching_ragged_gb300 import api
    K, B, A = 4, 16, 128
    p = Pool(5, K, B, A, seed=4)
    slots = chunk_slots([3, 0, 4], B, 0, 35)
    for i, s in enumerate(slots):
        k, v = (rows(1, K, A, "bf16", 10 + 2 * i + j, growth ** (i % 16)) for j in range(2))
        p.append(k, v, [s])
        p.plain(k, v, [s])
    api.cb_check_device_errors()
    p.check()


def test_scale_borders(native_lib):
    """Largest numbers just below, at and above 448 of a power of two, zeros, the smallest and the largest numbers of bf16."""
    from continuous_batching_ragged_gb300 import api
    K, B, A = 1, 16, 64
    tops = [0.0, 3.5, 3.515625, 3.484375, 448.0, 450.0, 1.75, 2.0, 2.0 ** -126, 2.0 ** -133, 3e38, 1.1 * 2.0 ** -92, 1.75 * 2.0 ** -92, 1e-20]
    p = Pool(len(tops), K, B, A)
    x = rows(len(tops), K, A, "bf16", 5).clamp(-1, 1)
    x *= torch.tensor(tops, device="cuda")[:, None, None].bfloat16()
    x[:, :, 7] = torch.tensor(tops, device="cuda")[:, None].bfloat16()
    slots = [i * B for i in range(len(tops))]
    p.append(x, -x, slots)
    api.cb_check_device_errors()
    p.plain(x, -x, slots)
    p.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_not_finite(native_lib, dtype):
    """Infinities and NaN become NaN, spare the scale, and stay NaN when the page is scaled anew; a row of nothing else too."""
    from continuous_batching_ragged_gb300 import api
    K, B, A = 2, 16, 64
    p = Pool(4, K, B, A)
    k, v = (rows(6, K, A, dtype, s) for s in (6, 7))
    k[0, 0, 5], k[0, 1, 6], k[1, 0, 7], v[2, 0] = math.inf, -math.inf, math.nan, math.inf
    slots = [0, 1, 2, 16, 17, 40]
    for a, b in ((0, 4), (4, 6)):
        p.append(k[a:b], v[a:b], slots[a:b])
        p.plain(k[a:b], v[a:b], slots[a:b])
    big = rows(1, K, A, dtype, 8, 1e4)
    p.append(big, big, [3])
    p.plain(big, big, [3])
    api.cb_check_device_errors()
    p.check()
    assert bool(p.k[0, 0, 0, 5].float().isnan()) and bool(p.v[0, 0, 2].float().isnan().all())


@pytest.mark.parametrize("T,dtype", [(300, "bf16"), (2500, "f32")])
def test_strided_tokens_and_many(native_lib, T, dtype):
    """Parts of one projection's output; more tokens than a CTA has threads, decode rows behind a long gap of skipped tokens."""
    from continuous_batching_ragged_gb300 import api
    K, B, A = 3, 16, 64
    p = Pool(T // B + 70, K, B, A, seed=9)
    ids = torch.randperm(T // B + 70, generator=torch.Generator().manual_seed(2)).tolist()
    qkv = rows(T, 5 * K, A, dtype, 11)
    k, v = qkv[:, 3 * K:4 * K], qkv[:, 4 * K:]
    gap = T // 2
    slots = chunk_slots(ids[:T // B + 2], B, 5, T - gap - 40) + [-1] * gap + [i * B + 3 for i in ids[-40:]]
    p.append(k, v, slots)
    api.cb_check_device_errors()
    p.plain(k, v, slots)
    p.check()


def test_bad_slots(native_lib):
    """Slots past the pool are skipped, slots that fall or repeat leave their page as it was; the others are written."""
    from continuous_batching_ragged_gb300 import api, native
    K, B, A = 2, 16, 128
    p = Pool(6, K, B, A)
    slots = [5, 6, 6 * 16, 7, 16 + 4, 16 + 4, 2 * 16 + 9, 2 * 16 + 8, 1 << 40, 3 * 16]
    k, v = (rows(len(slots), K, A, "bf16", s) for s in (12, 13))
    p.append(k, v, slots)
    with pytest.raises(native.CBError) as e:
        api.cb_check_device_errors()
    assert e.value.status == native.CB_ERR_BOUNDS
    good = [s if i in (0, 1, 3, 9) else -1 for i, s in enumerate(slots)]
    p.plain(k, v, good)
    p.check()
    p.append(k[4:6], v[4:6], slots[4:6])
    with pytest.raises(native.CBError) as e:
        api.cb_check_device_errors()
    assert e.value.status == native.CB_ERR_INVALID
    p.check()


def test_dims(native_lib):
    """The token count on the device: fewer, none, and more than the capacity."""
    from continuous_batching_ragged_gb300 import api, native
    K, B, A = 2, 16, 128
    p = Pool(6, K, B, A)
    k, v = (rows(20, K, A, "bf16", s) for s in (14, 15))
    slots = chunk_slots([4, 2], B, 3, 20)
    for n in (7, 0, 20):
        p.append(k, v, slots, dims=torch.tensor([1, n, 1, 1], dtype=torch.int32, device="cuda"))
        p.plain(k[:n], v[:n], slots[:n])
        api.cb_check_device_errors()
        p.check()
    p.append(k, v, slots, dims=torch.tensor([1, 21, 1, 1], dtype=torch.int32, device="cuda"))
    with pytest.raises(native.CBError):
        api.cb_check_device_errors()
    p.check()


def gather_plain(p, tables, cu, starts, total):
    q = [(p.k.double() * p.ks.double()[..., None, None]).cpu(), (p.v.double() * p.vs.double()[..., None, None]).cpu()]
    B = p.k.shape[2]
    out = [torch.full((total, p.k.shape[1], p.k.shape[3]), float("nan"), dtype=torch.float64) for _ in range(2)]
    for s in range(len(tables)):
        for r in range(cu[s], cu[s + 1]):
            pos = starts[s] + r - cu[s]
            for o, x in zip(out, q):
                o[r] = x[tables[s][pos // B], :, pos % B]
    return out


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("K,B,A,dtype", [(1, 16, 128, "bf16"), (8, 16, 128, "f32"), (3, 32, 64, "bf16"), (32, 1, 256, "bf16"), (2, 256, 64, "f32")])
@pytest.mark.parametrize("with_starts", [False, True])
def test_gather(native_lib, K, B, A, dtype, with_starts):
    """Sequences of no, one and many keys, from inside pages on; rows behind the last sequence stay."""
    from continuous_batching_ragged_gb300 import api
    p = Pool(60, K, B, A, seed=20)
    n = [0, 1, B, B + 1, 2 * B - 1, 0, 5]
    starts = [0, 1, B // 2, 0, B - 1, 3, B] if with_starts else [0] * 7
    perm = torch.randperm(60, generator=torch.Generator().manual_seed(3)).tolist()
    tables = [perm[6 * s:6 * s + 6] + [-1] for s in range(7)]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    k, v = (torch.full((cu[-1] + 3, K, A), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
    api.cb_gather_kv_q8(p.cache, ints(tables), ints(cu), k_out=k, v_out=v, starts=ints(starts) if with_starts else None)
    api.cb_check_device_errors()
    for got, want in zip((k, v), gather_plain(p, tables, cu, starts, cu[-1] + 3)):
        assert same(got, want)
    again = torch.full_like(v, float("nan"))
    api.cb_gather_kv_q8(p.cache, ints(tables), ints(cu), k_out=None, v_out=again, starts=ints(starts) if with_starts else None)
    assert same(again, v)


def test_gather_other_scales(native_lib):
    """Scales that are no powers of two: the product is rounded once."""
    from continuous_batching_ragged_gb300 import api
    p = Pool(4, 2, 16, 128, seed=21)
    p.ks.copy_(torch.rand(4, 2) + 0.1)
    k = torch.empty((40, 2, 128), dtype=torch.bfloat16, device="cuda")
    api.cb_gather_kv_q8(p.cache, ints([[2, 0, 3]]), ints([0, 40]), k_out=k, v_out=None)
    want = gather_plain(p, [[2, 0, 3]], [0, 40], [0], 40)[0]
    assert same(k, want.to(torch.bfloat16))          # the product of 4 and 24 bits is exact in 64


def test_gather_bad_metadata(native_lib):
    """Rows outside their table or with a negative start, and pages outside the pool, are left as they were and reported;
    rows past the outputs are not written."""
    from continuous_batching_ragged_gb300 import api, native
    p = Pool(8, 2, 16, 64, seed=22)

    def run(tables, cu, starts, rows_, status):
        k = torch.full((rows_, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        api.cb_gather_kv_q8(p.cache, ints(tables), ints(cu), k_out=k, v_out=None, starts=ints(starts))
        if status is None:
            api.cb_check_device_errors()
        else:
            with pytest.raises(native.CBError) as e:
                api.cb_check_device_errors()
            assert e.value.status == status
        return k

    a = run([[1, 9], [3, 4]], [0, 20, 40], [0, 0], 40, native.CB_ERR_BOUNDS)
    want = gather_plain(p, [[1, 1], [3, 4]], [0, 20, 40], [0, 0], 40)[0]
    want[16:20] = float("nan")
    assert same(a, want)
    a = run([[1, 2], [3, 4]], [0, 20, 40], [-1, 30], 40, native.CB_ERR_INVALID)
    want = torch.full_like(want, float("nan"))
    want[20:22] = gather_plain(p, [[1, 2], [3, 4]], [0, 20, 22], [0, 30], 40)[0][20:22]
    assert same(a, want)
    a = run([[1, 2], [3, 4]], [0, 20, 40], [0, 0], 25, None)
    assert same(a, gather_plain(p, [[1, 2], [3, 4]], [0, 20, 25], [0, 0], 25)[0])


def test_append_then_gather_on_streams(native_lib):
    """Calls on a stream of the caller's, one behind the other without a wait between; and captured, replayed over new values."""
    from continuous_batching_ragged_gb300 import api
    K, B, A = 4, 16, 128
    p = Pool(10, K, B, A, seed=23)
    slots = chunk_slots([7, 2, 5], B, 0, 41)
    k, v = (rows(41, K, A, "bf16", s) for s in (24, 25))
    ko, vo = (torch.empty_like(k) for _ in range(2))
    sl, tables, cu = torch.tensor(slots, device="cuda"), ints([[7, 2, 5]]), ints([0, 41])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(stream):
        api.cb_append_kv_q8(k, v, sl, p.cache, stream=stream)
        api.cb_gather_kv_q8(p.cache, tables, cu, k_out=ko, v_out=vo, stream=stream)

    step(side)
    side.synchronize()
    p.plain(k, v, slots)
    p.check()
    want = gather_plain(p, [[7, 2, 5]], [0, 41], [0], 41)
    assert same(ko, want[0]) and same(vo, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for seed in (30, 31):
        k.copy_(rows(41, K, A, "bf16", seed, 4.0))
        v.copy_(rows(41, K, A, "bf16", seed + 5, 0.1))
        graph.replay()
        torch.cuda.synchronize()
        p.plain(k, v, slots)
        p.check()
        want = gather_plain(p, [[7, 2, 5]], [0, 41], [0], 41)
        assert same(ko, want[0]) and same(vo, want[1])
    api.cb_check_device_errors()


def test_wide_offsets(native_lib):
    """Pages whose numbers begin behind 2^31 and 2^32 bytes of their pools, and gathered rows behind 2^31 bytes of the output."""
    from continuous_batching_ragged_gb300 import api
    K, B, A = 8, 128, 128
    p = Pool(5, K, B, A, seed=26)
    far_ids = [0, 2 ** 31 // (K * B * A) - 1, 2 ** 31 // (K * B * A), 2 ** 32 // (K * B * A) - 1, 2 ** 32 // (K * B * A) + 3]
    at = torch.tensor(far_ids, device="cuda")
    far = [torch.zeros((far_ids[-1] + 1, K, B, A), dtype=torch.uint8, device="cuda") for _ in range(2)]
    far_scales = [torch.ones((far_ids[-1] + 1, K), device="cuda") for _ in range(2)]
    for x, y in zip(far, (p.k, p.v)):
        x[at] = y.view(torch.uint8)
    for x, y in zip(far_scales, (p.ks, p.vs)):
        x[at] = y
    cache = api.QuantKVCache(*(x.view(E4M3) for x in far), *far_scales)
    for n, order in ((300, [1, 4, 3]), (1, [2]), (1, [4])):
        slots = chunk_slots(order, B, 70, n)
        k, v = (rows(n, K, A, "bf16", s) for s in (27, 28))
        api.cb_append_kv_q8(k, v, torch.tensor([far_ids[s // B] * B + s % B for s in slots], device="cuda"), cache)
        api.cb_check_device_errors()
        p.plain(k, v, slots)
    for x, y in zip(far, (p.k, p.v)):
        y.copy_(x[at].view(E4M3))
        x[at] = 0
        assert not bool(x.any())                     # nothing elsewhere
        x[at] = y.view(torch.uint8)
    for x, y in zip(far_scales, (p.ks, p.vs)):
        y.copy_(x[at])
    p.check()
    T = 2 ** 31 // (K * A * 4) + 40
    ko = torch.full((T, K, A), float("nan"), device="cuda")
    vo = torch.full((T, K, A), float("nan"), device="cuda")
    long = [4, 2, 3, 1, 0] * (T // B // 5 + 1)
    tables = torch.tensor([[far_ids[i] for i in long], [far_ids[i] for i in (0, 1, 4)] + [-1] * (len(long) - 3)])
    cu = [0, T - 300, T - 5]
    api.cb_gather_kv_q8(cache, tables.int().cuda(), ints(cu), k_out=ko, v_out=vo)
    api.cb_check_device_errors()
    first = (T - 300) // (5 * B) * 5 * B              # of the long sequence's last rows
    want = gather_plain(p, [long, [0, 1, 4]], [0, T - 300 - first, T - 5 - first], [0, 0], T - first)
    for got, w in zip((ko, vo), want):
        assert same(got[first:], w)
        assert same(got[:5 * B], got[first - 5 * B:first])
        assert same(got[:5 * B], gather_plain(p, [long], [0, 5 * B], [0], 5 * B)[0 if got is ko else 1])


@pytest.mark.parametrize("B", [16, 128])
@pytest.mark.parametrize("tail", [2900, 64_800])
def test_few_tokens_of_many(native_lib, B, tail):
    """A padded batch: most slots are skipped, before, between and behind the tokens."""
    from continuous_batching_ragged_gb300 import api
    K, A = 3, 64
    p = Pool(30, K, B, A, seed=29)
    ids = torch.randperm(30, generator=torch.Generator().manual_seed(30)).tolist()
    slots = [-1] * 70 + [ids[i] * B + 5 for i in range(9)] + [-1] * (tail // 2) + chunk_slots(ids[10:16], B, 3, 4 * B)
    slots += [-1] * 33 + [ids[20] * B] + [-1] * (tail - tail // 2)
    k, v = (rows(len(slots), K, A, "bf16", s) for s in (31, 32))
    p.append(k, v, slots)
    api.cb_check_device_errors()
    p.plain(k, v, slots)
    p.check()


def test_captured_append_with_a_count(native_lib):
    """A captured append replayed with other counts and slots on the device."""
    from continuous_batching_ragged_gb300 import api
    K, B, A = 4, 16, 128
    p = Pool(12, K, B, A, seed=33)
    k, v = (rows(60, K, A, "bf16", s) for s in (34, 35))
    slots = torch.full((60,), -1, dtype=torch.int64, device="cuda")
    dims = torch.tensor([1, 0, 1, 1], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        api.cb_append_kv_q8(k, v, slots, p.cache, dims=dims, stream=side)
    for n, ids, start in ((0, [0, 1, 2, 3, 4], 0), (60, [9, 3, 1, 7, 0], 2), (17, [5, 2], 0), (1, [5], 1), (2, [2, 5], 15)):
        mine = chunk_slots(ids, B, start, n)
        slots.copy_(torch.tensor(mine + [ids[0] * B] * (60 - n)))   # those behind the count are not read
        dims[1] = n
        graph.replay()
        api.cb_check_device_errors()
        p.plain(k[:n], v[:n], mine)
        p.check()


@pytest.mark.parametrize("blocks,K,B,A", [(12, 2, 16, 128), (12, 1, 64, 64), (70_000, 1, 1, 64), (66_000, 2, 2, 64)])
def test_pages_that_come_again(native_lib, blocks, K, B, A):
    """A page whose tokens do not follow one another is left as it was and reported, whether at other slots, at the same one or as
    decode rows; the pages between are written, and pages of a large pool that only look alike to the check."""
    from continuous_batching_ragged_gb300 import api, native
    p = Pool(blocks, K, B, A, seed=30)
    far = 65_536 if blocks > 65_536 else 0         # pages 3 and 3 + far, and so on
    run = list(range(min(B, 3)))
    parts = [(3, run, False), (5, [0], True), (3 + far // 2, [B - 1], True), (3, [B - 1], False), (7, run, True), (4, [0], False),
             (6, run, True), (4, [0], False), (4, [0], False), (8, [B - 1], True)]
    if far:
        parts += [(7 + far, [0], True), (9 + far, [0], True), (9, [B - 1], True), (4 + far, [0], True), (10 + far, [0], False), (10, [0], True),
                  (10 + far, [B - 1], False)]
    else:
        parts[2] = (2, [B - 1], True)
    slots = [page * B + o for page, offs, _ in parts for o in offs]
    good = [page * B + o if ok else -1 for page, offs, ok in parts for o in offs]
    k, v = (rows(len(slots), K, A, "bf16", s) for s in (31, 32))
    p.append(k, v, slots)
    with pytest.raises(native.CBError) as e:
        api.cb_check_device_errors()
    assert e.value.status == native.CB_ERR_INVALID
    p.plain(k, v, good)
    p.check()
    p.append(k, v, good)
    api.cb_check_device_errors()
    p.plain(k, v, good)
    p.check()


def test_many_pages_that_come_again(native_lib):
    """More runs than a CTA has threads, half of them of pages that another run is of."""
    from continuous_batching_ragged_gb300 import api, native
    p = Pool(1500, 1, 16, 64, seed=33)
    perm = torch.randperm(1500, generator=torch.Generator().manual_seed(34)).tolist()
    once, twice = perm[:600], perm[600:900]
    slots = [x * 16 for i in range(600) for x in [once[i]] + [twice[i // 2]] * (i % 2)] + [x * 16 + 1 for x in twice]
    k, v = (rows(len(slots), 1, 64, "f32", s) for s in (35, 36))
    p.append(k, v, slots)
    with pytest.raises(native.CBError) as e:
        api.cb_check_device_errors()
    assert e.value.status == native.CB_ERR_INVALID
    keep = set(once)
    p.plain(k, v, [s if s // 16 in keep else -1 for s in slots])
    p.check()


def bf16_once(x):
    """64-bit numbers in bf16's normal range to the nearest bf16 ones, ties to even (a conversion by way of fp32 rounds twice)."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256), e - 8)


def tie_scales(f, n, top, seed):
    """n fp32 scales, 2^top and more, whose product with f rounds in fp32 to a number halfway between two bf16 ones without being it."""
    g = torch.Generator().manual_seed(seed)
    tie = torch.randint(128, 256, (40 * n,), generator=g) * 2 + 1
    s = (tie.double() * 2.0 ** (top - 8) / f).float()
    p = s.double() * f
    near = p.float().double()
    half = torch.frexp(near)[0] * 512
    s = s[(half == torch.round(half)) & (half % 2 == 1) & (near != p)]
    assert s.numel() >= n
    return s[:n]


@pytest.mark.parametrize("top", [0, -60, -95, -115, 100])
def test_gather_rounds_once(native_lib, top):
    """Products that fp32 would first round to a tie of bf16, and the scales' own neighbours; whatever the scales' size."""
    from continuous_batching_ragged_gb300 import api
    K, B, A = 2, 16, 128
    for f in (1.125, 1.375, 1.625, 1.75, 1.875):
        s = tie_scales(f, 6, top, 40)
        s = torch.cat([s, s.nextafter(torch.tensor(0.0)), s.nextafter(torch.tensor(math.inf))])
        p = Pool(18, K, B, A, seed=41)
        x = torch.tensor([f, -f, 8 * f, f / 8])[torch.randint(0, 4, (18, K, B, A), generator=torch.Generator().manual_seed(42))]
        p.k.copy_(x.to(E4M3))
        p.ks.copy_(s[:, None].expand(18, K))
        k = torch.empty((18 * B, K, A), dtype=torch.bfloat16, device="cuda")
        api.cb_gather_kv_q8(p.cache, ints([list(range(18))]), ints([0, 18 * B]), k_out=k, v_out=None)
        api.cb_check_device_errors()
        want = gather_plain(p, [list(range(18))], [0, 18 * B], [0], 18 * B)[0]
        assert same(k, bf16_once(want))
        twice = want.float().bfloat16().double()
        assert bool((twice != bf16_once(want)).any())  # the numbers tell the two apart


def near_ties(K, A, dtype, seed, low):
    """Scales [K], 2^low and more, and numbers [40, K, A] of `dtype` whose quotients lie on, just above or just below ties of e4m3."""
    g = torch.Generator().manual_seed(seed)
    tie = (torch.randint(8, 16, (K,), generator=g) * 2 + 1).double() / 16        # between two numbers of four bits
    x = 1 + torch.randint(1, 128, (K,), generator=g).double() / 128
    s = (x / tie).float() * 2.0 ** (low + 1)
    rows_ = (x * 2.0 ** (low + 1))[None, :, None] * torch.exp2(torch.randint(-5, 8, (40, K, A), generator=g).double())
    rows_ = rows_ * (2 * torch.randint(0, 2, (40, K, A), generator=g) - 1)
    if dtype == "f32":
        rows_ = rows_.float()
        to = torch.randint(0, 3, rows_.shape, generator=g)
        rows_ = torch.where(to == 1, rows_.nextafter(torch.tensor(math.inf)), torch.where(to == 2, rows_.nextafter(torch.tensor(-math.inf)), rows_))
    return s, rows_.to(DT[dtype]).cuda()


@pytest.mark.parametrize("K,B,A,dtype", [(8, 16, 128, "bf16"), (3, 64, 128, "bf16"), (5, 8, 256, "bf16"), (4, 64, 64, "f32"), (7, 16, 128, "f32")])
@pytest.mark.parametrize("low", [0, -7, -60, -99, 90])
def test_kept_scales_of_any_kind(native_lib, K, B, A, dtype, low):
    """A page keeps a scale that is no power of two: quotients near ties are rounded once, for single tokens, runs, runs longer than a
    warp holds and among infinities; the page is scaled anew by one larger number."""
    from continuous_batching_ragged_gb300 import api
    p = Pool(12, K, B, A, seed=50)
    (ks, k), (vs, v) = (near_ties(K, A, dtype, s + 51, low) for s in range(2))
    for i, (to, s) in enumerate(((p.ks, ks), (p.vs, vs), (p.want[2], ks), (p.want[3], vs))):
        to.copy_(s.to(to.dtype)[None].expand(12, K))
    k[4, 0, 3], v[6, K - 1, 5] = math.inf, -math.inf
    n = min(B - 1, 40)
    slots = [0 * B + 1, 3 * B + B - 1] + [5 * B + o for o in range(1, 1 + min(n, 4))]
    slots += [7 * B + o for o in range(B - n, B)][:40 - len(slots)]
    tie = k[:len(slots)], v[:len(slots)]
    p.append(*tie, slots)
    p.plain(*tie, slots)
    api.cb_check_device_errors()
    p.check()
    assert float(p.ks[0, 0]) == float(ks[0])          # kept
    # old numbers, scaled anew by 2^4 / the kept scale and more
    big = [x[:2].clone() for x in (k, v)]
    for x in big:
        x.fill_(448.0 * 2.0 ** (low + 4) if low < 90 else 2.0 ** 105)
    at = [7 * B + B - 1, 9 * B + 2 % B]
    p.append(*big, at)
    p.plain(*big, at)
    api.cb_check_device_errors()
    p.check()


@pytest.mark.parametrize("top", [0, -60])
def test_scaled_anew_rounds_once(native_lib, top):
    """Old numbers whose product with the ratio of the scales fp32 would round to a tie of e4m3."""
    from continuous_batching_ragged_gb300 import api
    K, B, A = 6, 16, 128
    g = torch.Generator().manual_seed(60)
    for f in (9.0, 11.0, 13.0, 15.0):
        tie = (torch.randint(8, 16, (400,), generator=g) * 2 + 1).double()
        s = (tie / f).float()
        p_ = s.double() * f
        s = s[(p_.float().double() == tie) & (p_ != tie)][:12 * K]
        assert s.numel() == 12 * K
        p = Pool(12, K, B, A, seed=61)
        x = torch.tensor([f, -f, 2 * f, f / 8, 16.0, 1.0])[torch.randint(0, 6, (12, K, B, A), generator=g)]
        s = s.reshape(12, K) * 2.0 ** top
        for to in (p.k, p.v):
            to.copy_(x.to(E4M3))
        for to in (p.ks, p.vs):
            to.copy_(s)
        p.want = [t.double().cpu() for t in (p.k, p.v, p.ks, p.vs)]
        k = torch.full((12, K, A), 448 * 2.0 ** (top + 5), device="cuda").bfloat16()
        slots = [i * B + B - 1 - i % 3 for i in range(10)] + [10 * B + B - 2, 10 * B + B - 1]   # decode rows, and a run
        p.append(k, k, slots)
        p.plain(k, k, slots)
        api.cb_check_device_errors()
        p.check()


@pytest.mark.parametrize("again", [False, True])
def test_the_most_tokens(native_lib, again):
    """65,536 tokens: chunks over thousands of pages and decode rows among them; with one page that comes again at the very end."""
    from continuous_batching_ragged_gb300 import api, native
    B, T, blocks = 16, 65_536, 5700
    p = Pool(blocks, 1, B, 64, seed=70)
    perm = torch.randperm(blocks, generator=torch.Generator().manual_seed(71)).tolist()
    singles = perm[4100:4100 + 1536]
    slots = chunk_slots(perm, B, 7, 40_000) + [x * B + x % B for x in singles] + chunk_slots(perm[2600:], B, 0, T - 41_536)
    good = list(slots)
    if again:
        slots[-1] = slots[40_000]                  # the first decode row's page, and slot
        good[-1] = good[40_000] = -1
    assert len(slots) == T
    k, v = (rows(T, 1, 64, "bf16", s) for s in (72, 73))
    p.append(k, v, slots)
    if again:
        with pytest.raises(native.CBError) as e:
            api.cb_check_device_errors()
        assert e.value.status == native.CB_ERR_INVALID
    else:
        api.cb_check_device_errors()
    p.plain(k, v, good)
    p.check()
