"""Page operations: forks and compaction against a plain restatement of their rules.
Every result is whole pages, rows and numbers, so all comparisons are exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def stack(layers, blocks, heads, block, A, dtype=torch.bfloat16, seed=0):
    from continuous_batching_ragged_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(seed)
    pools = torch.randn((layers, 2, blocks, heads, block, A), generator=g, device="cuda").to(dtype)
    return pools, api.KVCacheStack([api.KVCache(p[0], p[1]) for p in pools])


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def fork_plain(pools, tables, ctx, parents, children, new, block):
    """The valid forks one after the other (none touches what another reads)."""
    pools, tables, ctx = pools.clone(), tables.tolist(), ctx.tolist()
    width = len(tables[0])
    for p, c, b in zip(parents, children, new):
        n = ctx[p]
        row = tables[p][:n // block]
        if n % block:
            pools[:, :, b, :, :n % block] = pools[:, :, tables[p][n // block], :, :n % block]
            row = row + [b]
        tables[c], ctx[c] = row + [-1] * (width - len(row)), n
    return pools, ints(tables), ints(ctx)


def run_fork(pools, caches, tables, ctx, parents, children, new, stream=None):
    from continuous_batching_ragged_gb300 import api
    api.cb_fork_sequences(caches, tables, ctx, ints(parents), ints(children), ints(new), stream=stream)


CTX = [0, 1, 15, 16, 17, 100, 128]


@pytest.mark.parametrize("heads,block,A,dtype,layers", [(8, 16, 128, torch.bfloat16, 3), (1, 16, 128, torch.bfloat16, 1),
                                                        (32, 32, 128, torch.bfloat16, 2), (4, 1, 64, torch.float32, 2),
                                                        (3, 5, 24, torch.bfloat16, 2), (2, 128, 128, torch.bfloat16, 2)])
def test_forks(native_lib, heads, block, A, dtype, layers):
    """Parents of every length around page borders, each forked once or several times."""
    from continuous_batching_ragged_gb300 import api
    width = 128 // block + 2 if block < 128 else 3
    width = max(width, 130) if block == 1 else width
    pages = [-(-n // block) for n in CTX]
    total = sum(pages) + 12
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(1)).tolist()
    tables, at = [], 0
    for n in pages:
        tables.append(perm[at:at + n] + [-1] * (width - n))
        at += n
    children = [7, 9, 8, 10, 16, 11, 12, 15, 13, 14]
    tables = ints(tables + [[77] * width] * 10)          # child rows hold anything before
    ctx = ints(CTX + [99] * 10)
    pools, caches = stack(layers, total, heads, block, A, dtype)
    parents = [0, 1, 2, 3, 4, 5, 6, 5, 5, 2]
    new = perm[at:at + 10]
    want = fork_plain(pools, tables, ctx, parents, children, new, block)
    run_fork(pools, caches, tables, ctx, parents, children, new)
    api.cb_check_device_errors()
    assert torch.equal(tables, want[1]) and torch.equal(ctx, want[2]) and torch.equal(pools, want[0])


def test_many_forks_and_layers(native_lib):
    """More layers than one launch takes, more forks than a block has threads."""
    from continuous_batching_ragged_gb300 import api
    F = 300
    pools, caches = stack(130, F + 8, 1, 4, 8)
    tables = ints([[0, 1, -1], [2, 3, -1]] + [[-1] * 3] * F)
    ctx = ints([7, 8] + [0] * F)
    parents, children, new = [i % 2 for i in range(F)], list(range(2, F + 2)), list(range(8, F + 8))
    want = fork_plain(pools, tables, ctx, parents, children, new, 4)
    run_fork(pools, caches, tables, ctx, parents, children, new)
    api.cb_check_device_errors()
    assert torch.equal(tables, want[1]) and torch.equal(ctx, want[2]) and torch.equal(pools, want[0])


@pytest.mark.parametrize("fault,error", [("child is a parent", "INVALID"), ("child twice", "INVALID"), ("new page twice", "INVALID"),
                                         ("new page is a source", "INVALID"), ("parent row", "INVALID"), ("child row", "INVALID"),
                                         ("new page id", "BOUNDS"), ("source page id", "BOUNDS"), ("length", "INVALID"),
                                         ("child is its own parent", "INVALID")])
def test_bad_forks_are_left_out(native_lib, fault, error):
    """The forks at fault do nothing and are reported; the others are done."""
    from continuous_batching_ragged_gb300 import api, native
    pools, caches = stack(2, 32, 2, 8, 16, seed=2)
    tables = ints([[0, 1, -1, -1], [2, -1, -1, -1], [3, 4, 5, -1]] + [[-1] * 4] * 5)
    ctx = ints([12, 3, 20] + [0] * 5)
    parents, children, new = [0, 0, 1, 2, 2], [3, 4, 5, 6, 7], [10, 11, 12, 13, 14]
    bad = [1]
    if fault == "child is a parent":
        children[1] = 2
    elif fault == "child is its own parent":
        children[1] = 0
    elif fault == "child twice":
        children[1], bad = 6, [1, 3]
    elif fault == "new page twice":
        new[1], bad = 13, [1, 3]
    elif fault == "new page is a source":
        new[1] = 5
    elif fault == "parent row":
        parents[1] = 8
    elif fault == "child row":
        children[1] = -1
    elif fault == "new page id":
        new[1] = 32
    elif fault == "source page id":
        tables[1, 0], bad = 500, [2]
    elif fault == "length":
        ctx[1], bad = 33, [2]
    keep = [i for i in range(5) if i not in bad]
    want = fork_plain(pools, tables, ctx, *([x[i] for i in keep] for x in (parents, children, new)), 8)
    run_fork(pools, caches, tables, ctx, parents, children, new)
    with pytest.raises(native.CBError, match=error):
        api.cb_check_device_errors()
    assert torch.equal(tables, want[1]) and torch.equal(ctx, want[2]) and torch.equal(pools, want[0])


def test_fork_offsets_past_32_bits(native_lib):
    from continuous_batching_ragged_gb300 import api
    block, heads, A = 16, 8, 128
    nb = (1 << 32) // (block * heads * A) + 8
    k, v = (torch.empty((nb, heads, block, A), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[nb - 2], v[nb - 2] = torch.randn_like(k[0]), torch.randn_like(v[0])
    tables, ctx = ints([[nb - 2, -1], [-1, -1], [-1, -1]]), ints([11, 0, 0])
    api.cb_fork_sequences([api.KVCache(k, v)], tables, ctx, ints([0, 0]), ints([1, 2]), ints([nb - 1, 3]))
    api.cb_check_device_errors()
    for b in (nb - 1, 3):
        assert torch.equal(k[b, :, :11], k[nb - 2, :, :11]) and torch.equal(v[b, :, :11], v[nb - 2, :, :11])
    assert tables.tolist() == [[nb - 2, -1], [nb - 1, -1], [3, -1]] and ctx.tolist() == [11, 11, 11]


def compact_plain(pools, tables, ctx, block, blocks):
    pools, tables = pools.clone(), tables.tolist()
    used = [t[:-(-c // block)] for t, c in zip(tables, ctx.tolist())]
    live = sorted({b for t in used for b in t})
    n = len(live)
    to = {b: b for b in live if b < n}
    free = [b for b in range(n) if b not in to]
    for b in live:
        if b >= n:
            to[b] = free.pop(0)
            pools[:, :, to[b]] = pools[:, :, b]
    width = len(tables[0]) if tables else 0
    return pools, [[to[b] for b in t] + [-1] * (width - len(t)) for t in used], [to.get(b, -1) for b in range(blocks)], n


def run_compact(caches, tables, ctx, blocks, in_place=False, stream=None):
    from continuous_batching_ragged_gb300 import api
    new = tables if in_place else torch.full_like(tables, 555)
    remap, live = torch.full((blocks,), 555, dtype=torch.int32, device="cuda"), ints([555])
    ws = torch.empty(api.cb_compact_workspace_size(blocks), dtype=torch.uint8, device="cuda")
    api.cb_compact_blocks(caches, tables, ctx, new_block_tables=new, remap=remap, num_live=live, workspace=ws, stream=stream)
    return new, remap, live, ws


def fragmented(blocks, seqs, share, block, seed, shared=True):
    """Tables over a random `share` of the pool, some rows behind another row's pages, some rows empty."""
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(blocks, generator=g)[:int(round(blocks * share))].tolist()
    cuts = [0] + sorted(torch.randint(0, len(perm) + 1, (seqs - 1,), generator=g).tolist()) + [len(perm)]
    rows = [perm[a:b] for a, b in zip(cuts, cuts[1:])]
    if shared:
        for i in range(2, seqs, 3):
            rows[i] = rows[i - 1][:3] + rows[i]
    width = max(map(len, rows)) + 2
    ctx = [max(0, len(r) * block - int(torch.randint(0, block, (1,), generator=g))) for r in rows]
    junk = torch.randint(-5, blocks + 5, (seqs, width), generator=g).tolist()   # entries behind a row's pages hold anything
    return ints([r + j[len(r):] for r, j in zip(rows, junk)]), ints(ctx)


@pytest.mark.parametrize("blocks,seqs,share,block", [(1, 1, 1.0, 16), (1, 1, 0.0, 16), (33, 3, 0.5, 16), (200, 12, 0.5, 16),
                                                     (1000, 40, 0.05, 4), (1000, 40, 0.97, 4), (64, 5, 1.0, 8), (70, 7, 0.0, 1),
                                                     (2500, 300, 0.6, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compaction(native_lib, blocks, seqs, share, block, in_place):
    from continuous_batching_ragged_gb300 import api
    pools, caches = stack(2, blocks, 2, block, 16, seed=blocks)
    tables, ctx = fragmented(blocks, seqs, share, block, blocks + seqs)
    want = compact_plain(pools, tables, ctx, block, blocks)
    new, remap, live, _ = run_compact(caches, tables, ctx, blocks, in_place)
    api.cb_check_device_errors()
    assert live.tolist() == [want[3]] and new.tolist() == want[1] and remap.tolist() == want[2]
    assert torch.equal(pools, want[0])
    # what is compact stays as it is
    again, remap, live2, _ = run_compact(caches, new, ctx, blocks)
    api.cb_check_device_errors()
    assert torch.equal(live, live2) and torch.equal(again, new) and torch.equal(pools, want[0])


def test_compaction_keeps_what_every_sequence_reads(native_lib):
    """f32 pages of 3 heads and 40 bytes a row: each sequence reads the same values through its new table."""
    from continuous_batching_ragged_gb300 import api
    pools, caches = stack(3, 150, 3, 4, 12, torch.float32, seed=5)
    tables, ctx = fragmented(150, 10, 0.4, 4, 9)
    held = [pools[:, :, t[:-(-c // 4)]].clone() for t, c in zip(tables.tolist(), ctx.tolist())]
    new, _, live, _ = run_compact(caches, tables, ctx, 150)
    api.cb_check_device_errors()
    for t, c, h in zip(new.tolist(), ctx.tolist(), held):
        mine = t[:-(-c // 4)]
        assert torch.equal(pools[:, :, mine], h) and all(0 <= b < int(live) for b in mine)


@pytest.mark.parametrize("blocks", [400_000, 1 << 20])
def test_large_pools(native_lib, blocks):
    """Pools whose bitmap is larger than the default shared memory."""
    from continuous_batching_ragged_gb300 import api
    pools, caches = stack(1, blocks, 1, 1, 8, seed=6)
    g = torch.Generator().manual_seed(2)
    rows = torch.randperm(blocks, generator=g)[:blocks // 10 * 4].view(4, -1)
    tables, ctx = rows.to(torch.int32).cuda(), ints([rows.shape[1]] * 3 + [rows.shape[1] - 7])
    before = pools.clone()
    new, remap, live, _ = run_compact(caches, tables, ctx, blocks)
    api.cb_check_device_errors()
    n = rows.numel() - 7
    assert int(live) == n
    used = torch.ones_like(tables, dtype=torch.bool)
    used[3, -7:] = False
    assert bool((new[used] < n).all()) and bool((new[~used] == -1).all())
    assert torch.equal(new[used].sort().values, torch.arange(n, dtype=torch.int32, device="cuda"))
    assert torch.equal(pools[:, :, new[used].long()], before[:, :, tables[used].long()])
    assert torch.equal(remap[tables[used].long()], new[used]) and int((remap >= 0).sum()) == n


@pytest.mark.parametrize("fault,error", [("page id", "BOUNDS"), ("negative page id", "BOUNDS"), ("length", "INVALID"),
                                         ("negative length", "INVALID")])
def test_bad_tables_change_nothing(native_lib, fault, error):
    from continuous_batching_ragged_gb300 import api, native
    pools, caches = stack(2, 100, 2, 4, 16, seed=7)
    tables, ctx = fragmented(100, 6, 0.5, 4, 3)
    s = int(ctx.argmax())
    if "page" in fault:
        tables[s, 0] = 100 if fault == "page id" else -1
    else:
        ctx[s] = tables.shape[1] * 4 + 1 if fault == "length" else -1
    before, t0 = pools.clone(), tables.clone()
    new, remap, live, _ = run_compact(caches, tables, ctx, 100)
    with pytest.raises(native.CBError, match=error):
        api.cb_check_device_errors()
    assert live.tolist() == [-1] and torch.equal(pools, before) and torch.equal(tables, t0)
    assert bool((new == 555).all()) and bool((remap == 555).all())


def test_no_sequences(native_lib):
    from continuous_batching_ragged_gb300 import api
    pools, caches = stack(1, 20, 1, 4, 8, seed=8)
    before = pools.clone()
    new, remap, live, _ = run_compact(caches, torch.empty((0, 4), dtype=torch.int32, device="cuda"), ints([]), 20)
    api.cb_check_device_errors()
    assert live.tolist() == [0] and bool((remap == -1).all()) and torch.equal(pools, before)


def test_captured_forks_and_compaction(native_lib):
    """Both calls captured in one graph and replayed over new tables, on a side stream."""
    from continuous_batching_ragged_gb300 import api
    blocks, block = 60, 4
    pools, caches = stack(2, blocks, 2, block, 16, seed=9)
    tables, ctx = ints([[50, 41, -1, -1], [30, -1, -1, -1], [-1] * 4, [-1] * 4]), ints([6, 4, 0, 0])
    parents, children, new_pages = ints([0, 1]), ints([2, 3]), ints([44, 45])
    t0, c0, p0 = tables.clone(), ctx.clone(), pools.clone()
    new, remap, live = torch.empty_like(tables), torch.empty(blocks, dtype=torch.int32, device="cuda"), ints([0])
    ws = torch.empty(api.cb_compact_workspace_size(blocks), dtype=torch.uint8, device="cuda")

    def both():
        api.cb_fork_sequences(caches, tables, ctx, parents, children, new_pages)
        api.cb_compact_blocks(caches, tables, ctx, new_block_tables=new, remap=remap, num_live=live, workspace=ws)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    t1 = ints([[7, 58, 59, -1], [30, 2, -1, -1], [-1] * 4, [-1] * 4])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t, c in ((t0, c0), (t1, ints([9, 7, 0, 0]))):
        with torch.cuda.stream(side):
            tables.copy_(t)
            ctx.copy_(c)
            pools.copy_(p0)
            graph.replay()
        side.synchronize()
        api.cb_check_device_errors(side)
        f = fork_plain(p0, t, c, [0, 1], [2, 3], [44, 45], block)
        want = compact_plain(f[0], f[1], f[2], block, blocks)
        assert torch.equal(tables, f[1]) and new.tolist() == want[1] and remap.tolist() == want[2]
        assert live.tolist() == [want[3]] and torch.equal(pools, want[0])
