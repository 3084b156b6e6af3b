"""cb_shared_prefix_attention against softmax(q K^T) V of every sequence over its
own keys, in 64 bits.

Tolerance.  An output is sum_j p_j v_j with sum p_j = 1.  P is rounded to bf16
for the tensor core, half a step (2^-8) of each p_j, so the sum moves by at most
2^-8 * a, a = sum_j p_j |v_j|; the output's own rounding by 2^-8 of its value.
In fp32 a score is a sum of 128 products: off by at most 128 * 2^-24 * r, r the
row's largest sum of |q_d k_d| in the exp2 domain, which moves p_j by ln 2 times
that, relatively; the sums over up to 2^16 keys are trees and tensor-core
chains below 2^-12 relative.  Both count for numerator and denominator."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

A = 128


class Step:
    """Groups of sequences over one pool: [(prefix, [(own keys, query tokens), ...]), ...]; own keys include the query tokens."""

    def __init__(self, groups, H, K, B, seed=0, q_scale=1.0, k_slope=0.0, extra_blocks=3, num_blocks=None, width=None,
                 ballast=True, force=False):
        from continuous_batching_ragged_gb300 import api
        # a step shares only where that saves some 190 MB: one more group that does, whatever the others are
        self.real = sum(len(members) for _, members in groups)
        if ballast:
            n = 2 + 200_000_000 // (2048 * 4 * A * K)
            groups = list(groups) + [(2048, [(1, 1)] * max(n, force * (64 // (H // K) + 1)))]
        g = torch.Generator(device="cuda").manual_seed(seed)
        pick = torch.Generator().manual_seed(seed)
        self.H, self.K, self.B, self.groups = H, K, B, groups
        seqs = [(p, own, n) for p, members in groups for own, n in members]
        self.ctx_l, self.q_l = [p + own for p, own, _ in seqs], [n for _, _, n in seqs]
        need = sum(-(-c // B) for c in self.ctx_l) + sum(p // B for p, members in groups if not members) + extra_blocks
        nb = num_blocks or need
        ids = torch.randperm(nb, generator=pick)[:need].tolist() if nb < 1 << 20 else \
            (nb - 1 - torch.randperm(need, generator=pick)).tolist()
        shape = (nb, K, B, A)
        if num_blocks is None:
            k, v = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        else:
            k, v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        rnd = lambda n, h: torch.randn((n, h, A), generator=g, device="cuda")  # noqa: E731
        width = width or max(-(-c // B) for c in self.ctx_l) + 2
        self.tables_l, self.keys, at, s, self.cu_groups_l = [], [], 0, 0, [0]
        for p, members in groups:
            common = ids[at:at + p // B]
            at += len(common)
            pk, pv = (rnd(p, K) for _ in range(2))
            for own, _ in members:
                c = p + own
                mine = ids[at:at + -(-c // B) - len(common)]
                at += len(mine)
                sk, sv = torch.cat([pk, rnd(own, K)]), torch.cat([pv, rnd(own, K)])
                if k_slope:                        # scores climb along the keys, so the running maximum keeps moving
                    sk = sk + k_slope * torch.arange(c, device="cuda")[:, None, None] / math.sqrt(A)
                sk, sv = sk.bfloat16(), sv.bfloat16()
                row = torch.tensor(common + mine, device="cuda")
                j = torch.arange(c, device="cuda")
                k[row[j // B], :, j % B] = sk
                v[row[j // B], :, j % B] = sv
                self.keys.append((sk, sv))
                self.tables_l.append(common + mine + [-1] * (width - len(common) - len(mine)))
                s += 1
            self.cu_groups_l.append(s)
        self.cu_l = [0]
        for n in self.q_l:
            self.cu_l.append(self.cu_l[-1] + n)
        self.q = (rnd(self.cu_l[-1], H) * q_scale + (k_slope > 0) * 1.0).bfloat16()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cache = api.KVCache(k, v)
        self.cu, self.ctx, self.tables = i32(self.cu_l), i32(self.ctx_l), i32(self.tables_l)
        self.cu_groups, self.prefix = i32(self.cu_groups_l), i32([p for p, _ in groups])
        self.max_q, self.max_ctx, self.scale = max(self.q_l), max(self.ctx_l), 1 / math.sqrt(A)
        if force:                                  # where there may be chunks, even small groups share
            self.max_q = max(self.max_q, 64 // (H // K) + 1)
        self.out = torch.full_like(self.q, float("nan"))
        n = api.cb_shared_prefix_workspace_size(self.cache, H, len(seqs), self.cu_l[-1], len(groups), self.max_ctx)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")   # contents need no initialisation

    def run(self, stream=None):
        from continuous_batching_ragged_gb300 import api
        api.cb_shared_prefix_attention(self.q, self.cache, self.cu, self.ctx, self.tables, self.cu_groups, self.prefix,
                                       max_q_len=self.max_q, max_context_len=self.max_ctx, scale=self.scale, out=self.out,
                                       workspace=self.ws, stream=stream)
        return self.out

    def check(self, sequences=None):
        G = self.H // self.K
        for s in range(min(self.real + 2, len(self.q_l))) if sequences is None else sequences:
            k, v = (x.double() for x in self.keys[s])
            a, b = self.cu_l[s], self.cu_l[s + 1]
            q = self.q[a:b].double().view(b - a, self.K, G, A)
            late = torch.arange(len(k), device="cuda")[None] > torch.arange(len(k) - (b - a), len(k), device="cuda")[:, None]
            for h in range(self.K):
                sc = torch.einsum("igd,jd->igj", q[:, h], k[:, h]) * self.scale
                p = torch.softmax(sc.masked_fill(late[:, None], -math.inf), -1)
                want, mag = p @ v[:, h], p @ v[:, h].abs()
                r = (torch.einsum("igd,jd->igj", q[:, h].abs(), k[:, h].abs()) * self.scale * math.log2(math.e)).amax(-1, keepdim=True)
                rel = 2.0 ** -8 + 2 * (math.log(2) * 128 * 2.0 ** -24 * r + 2.0 ** -12)
                off = (self.out[a:b, h * G:(h + 1) * G].double() - want).abs()
                lim = rel * mag + 2.0 ** -8 * (want.abs() + rel * mag)
                assert bool((off <= lim).all()), (s, h, float((off - lim).max()))


def run_checked(*args, **kw):
    from continuous_batching_ragged_gb300 import api
    st = Step(*args, **kw)
    st.run()
    api.cb_check_device_errors()
    st.check()
    return st


HEADS = [(8, 8, 16), (8, 2, 16), (4, 1, 64), (12, 4, 32), (16, 1, 16), (5, 1, 128), (6, 2, 16), (32, 1, 32)]


@pytest.mark.parametrize("H,K,B", HEADS)
@pytest.mark.parametrize("force", [False, True])
def test_prefix_lengths(native_lib, H, K, B, force):
    """Prefixes around blocks and KV tiles, from none to several tiles; suffixes of one key and more."""
    own = [(1, 1), (5, 1), (130, 1)]
    run_checked([(p, own) for p in (0, 1, B - 1, B, B + 1, 127, 128, 129, 256, 257, 640, 1000)], H, K, B, seed=H + K, force=force)


@pytest.mark.parametrize("H,K,B", HEADS)
@pytest.mark.parametrize("force", [False, True])
def test_group_sizes(native_lib, H, K, B, force):
    """Groups of one sequence to more rows than two tiles hold: the one-tile mode with its
    last rows, exactly one tile, one row more, two tiles, and a third."""
    tt = 128 // (H // K)
    sizes = sorted({1, 2, 3, tt - 1, tt, tt + 1, 2 * tt, 2 * tt + 1} - {0})
    sizes = [n for n in sizes if n <= 257]
    run_checked([(300, [(1 + i % 7, 1) for i in range(n)]) for n in sizes], H, K, B, seed=50 + H, force=force)


@pytest.mark.parametrize("H,K,B", [(8, 8, 16), (8, 2, 32), (16, 2, 16), (12, 4, 64)])
@pytest.mark.parametrize("q", [2, 17, 150])
def test_several_query_tokens(native_lib, H, K, B, q):
    """Chunks of query tokens behind the prefix, with their causal mask, among single ones."""
    run_checked([(500, [(q, q), (q + 40, q), (3, 1), (q, q)]), (77, [(q, q), (9, 2)]), (1100, [(1, 1), (q + 300, q)])],
                H, K, B, seed=70 + q)


@pytest.mark.parametrize("H,K,tokens", [(32, 8, 4), (32, 1, 2), (8, 8, 3), (32, 32, 64), (32, 8, 256)])
def test_long_prefix(native_lib, H, K, tokens):
    """Prefixes cut into many KV segments (few rows) and into few (many rows)."""
    st = run_checked([(20_000 if tokens < 64 else 5000, [(1 + 3 * (i % 5), 1) for i in range(tokens)])], H, K, 16, seed=tokens,
                     ballast=tokens < 64)
    first = st.out.clone()
    st.ws.fill_(7)
    st.out.fill_(float("nan"))
    st.run()
    torch.cuda.synchronize()
    assert torch.equal(first, st.out)                # the same bits from call to call


@pytest.mark.parametrize("force", [False, True])
def test_many_groups(native_lib, force):
    """More groups than the plan has threads, sizes and prefixes mixed, some empty or without a prefix."""
    g = torch.Generator().manual_seed(3)
    r = lambda a, b: int(torch.randint(a, b + 1, (1,), generator=g))  # noqa: E731
    groups = [(r(0, 400) if i % 5 else 0, [(r(1, 60), 1) for _ in range(r(0, 4))]) for i in range(300)]
    run_checked(groups, 8, 2, 16, seed=4, force=force)


@pytest.mark.parametrize("force", [False, True])
def test_growing_scores(native_lib, force):
    """The running maximum is overtaken again and again, in the prefix and behind it."""
    run_checked([(900, [(40, 1), (300, 1), (70, 30)]), (600, [(2, 1)] * 20)], 8, 2, 16, seed=5, q_scale=0.5, k_slope=0.2, force=force)


@pytest.mark.parametrize("force", [False, True])
def test_peaked_rows(native_lib, force):
    """Scores of tens: nearly all weight on single keys."""
    run_checked([(1500, [(3, 1), (200, 1)] * 5)], 8, 8, 16, seed=6, q_scale=8.0, force=force)


def test_without_sharing(native_lib):
    """Groups of one sequence share nothing: every sequence reads its own pages, single rows and chunks."""
    run_checked([(300, [(7, 1)]), (900, [(1, 1)]), (0, [(200, 150)]), (64, [(30, 5)]), (5000, [(1, 1)]), (0, [(1, 1)])],
                8, 2, 16, seed=7, ballast=False)


@pytest.mark.parametrize("H,K", [(8, 8), (32, 4)])
@pytest.mark.parametrize("q", [1, 3, 70])
def test_small_steps(native_lib, H, K, q):
    """Groups too small for sharing to pay: the same rows, through each sequence's own table."""
    run_checked([(300, [(q, q)] * 3), (40, [(q + 9, q), (1, 1)]), (513, [(2, 1)] * 2)], H, K, 16, seed=8 + q, ballast=False)


@pytest.mark.parametrize("H,K", [(8, 8), (32, 8), (16, 1), (32, 1)])
def test_long_own_keys(native_lib, H, K):
    """Own keys cut into chunks (several records a row), with and without a prefix, one and several query tokens."""
    run_checked([(40, [(9000, 1), (5, 1), (700, 3)]), (0, [(4000, 1), (2500, 40)]), (2000, [(6000, 2)])], H, K, 16, seed=30 + H + K)


def test_infinite_and_nan_keys_of_others(native_lib):
    """NaN and infinities in one group's prefix or one sequence's own keys reach no other."""
    from continuous_batching_ragged_gb300 import api
    groups = [(400, [(9, 1)] * 5), (400, [(9, 1)] * 5)]
    st = Step(groups, 8, 2, 16, seed=8, force=True)
    st.cache.k[st.tables_l[0][3], 1] = float("nan")          # group 0, key/value head 1
    st.cache.v[st.tables_l[6][25], 0, 0] = float("inf")      # sequence 6, head 0, a key of its own
    st.run()
    api.cb_check_device_errors()
    bad = st.out.isnan().any(-1) | st.out.isinf().any(-1)
    want = torch.zeros_like(bad)
    want[:5, 4:] = True
    want[6, :4] = True
    assert torch.equal(bad, want)
    st.check([5, 7, 8, 9, 10, 11])


@pytest.mark.parametrize("fault", ["prefix too long", "negative prefix", "gap", "overlap", "not all", "start", "page", "first page",
                                   "context"])
def test_bad_metadata(native_lib, fault):
    """What is wrong is reported; sequences that do not depend on it keep their results."""
    from continuous_batching_ragged_gb300 import api, native
    st = Step([(300, [(5, 1)] * 4), (200, [(8, 1)] * 3), (50, [(40, 1)] * 2)], 8, 2, 16, seed=9, force=True)
    good, error, n = range(9), "INVALID", len(st.q_l)
    if fault == "prefix too long":
        st.ctx[5], good = 200, [0, 1, 2, 3, 4, 6, 7, 8]   # its cached keys end before the prefix does
    elif fault == "negative prefix":
        st.prefix[1], good = -3, [0, 1, 2, 3, 7, 8]
    elif fault == "gap":
        st.cu_groups[1], good = n + 1, []
    elif fault == "overlap":
        st.cu_groups[2], good = 3, []
    elif fault == "not all":
        st.cu_groups[4], good = n - 1, []
    elif fault == "start":
        st.cu_groups[0], good = 1, []
    elif fault == "page":
        st.tables[8, 4], good, error = st.cache.num_blocks, range(8), "BOUNDS"
    elif fault == "first page":
        st.tables[4, 2], good, error = -1, [0, 1, 2, 3, 7, 8], "BOUNDS"
    elif fault == "context":
        st.ctx[0], good = st.max_ctx + 1, [1, 2, 3, 4, 5, 6, 7, 8]
    st.run()
    with pytest.raises(native.CBError, match=error):
        api.cb_check_device_errors()
    st.check(good)
    if not good:
        assert bool(st.out.isnan().all())


def test_rows_behind_the_step_stay(native_lib):
    """q and out with rows behind the last sequence: the metadata's token count rules, the rest is not written."""
    from continuous_batching_ragged_gb300 import api
    st = Step([(300, [(5, 1)] * 4)], 8, 2, 16, seed=10, force=True)
    rows = len(st.q)
    more = torch.full((7, 8, A), float("nan"), dtype=torch.bfloat16, device="cuda")
    st.q, st.out = torch.cat([st.q, more]), torch.cat([st.out, more])
    n = api.cb_shared_prefix_workspace_size(st.cache, 8, len(st.q_l), rows + 7, 2, st.max_ctx)
    st.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    st.run()
    api.cb_check_device_errors()
    st.check()
    assert bool(st.out[rows:].isnan().all())


def test_captured_and_replayed(native_lib):
    """A captured call replays over new groups, lengths and pages of the same sizes; two graphs share a workspace."""
    from continuous_batching_ragged_gb300 import api
    sizes = dict(width=200, num_blocks=2000)
    first = Step([(300, [(5, 1)] * 4), (500, [(60, 1)] * 6)], 8, 2, 16, seed=11, force=True, **sizes)
    other = Step([(0, [(9, 1)] * 1), (540, [(25, 1)] * 9)], 8, 2, 16, seed=12, force=True, **sizes)
    for st in (first, other):
        st.max_ctx = 2500
    n = api.cb_shared_prefix_workspace_size(first.cache, 8, len(first.q_l), len(first.q), 3, 2500)
    first.ws = other.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    first.run()
    graphs = []
    for st in (first, other):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            st.run()
        graphs.append(graph)
    for _ in range(2):
        for st, graph in ((first, graphs[0]), (other, graphs[1])):
            st.out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            st.check()
    # new metadata and values in the first graph's buffers
    for name in ("q", "cu", "ctx", "tables", "cu_groups", "prefix"):
        getattr(first, name).copy_(getattr(other, name))
    first.cache.k.copy_(other.cache.k)
    first.cache.v.copy_(other.cache.v)
    graphs[0].replay()
    api.cb_check_device_errors()
    assert torch.equal(first.out, other.out)


def test_on_another_stream_back_to_back(native_lib):
    """Calls in a row over one workspace on a side stream, without waiting between them."""
    from continuous_batching_ragged_gb300 import api
    steps = [Step([(300 + 50 * i, [(5 + i, 1)] * (3 + i)), (17, [(60, 20)] * 2)], 8, 2, 16, seed=20 + i) for i in range(4)]
    n = max(st.ws.numel() for st in steps)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for st in steps * 3:
        st.ws = ws
        st.run(stream=side)
    side.synchronize()
    api.cb_check_device_errors(side)
    for st in steps:
        st.check()


def test_pages_past_32_bit_offsets(native_lib):
    nb = (1 << 32) // (8 * 16 * A) + 500
    run_checked([(500, [(3, 1), (40, 1), (90, 50)]), (100, [(1, 1)] * 2)], 8, 8, 16, seed=13, num_blocks=nb)


@pytest.mark.parametrize("q", [1, 90])
def test_more_sequences_than_the_plan_caches(native_lib, q):
    """More groups and sequences than the plan keeps in shared memory; with chunks, more jobs too."""
    g = torch.Generator().manual_seed(q)
    r = lambda a, b: int(torch.randint(a, b + 1, (1,), generator=g))  # noqa: E731
    groups = [(r(0, 200), [(q + r(0, 9), q) if i % 40 == 0 else (r(1, 40), 1)] * r(0, 3)) for i in range(700)]
    run_checked(groups, 4, 2, 16, seed=90 + q)


@pytest.mark.parametrize("H,K", [(128, 1), (100, 1), (66, 1), (240, 2)])
@pytest.mark.parametrize("force", [False, True])
def test_many_query_heads_of_one_key_head(native_lib, H, K, force):
    """One token, or few, fill a row tile: 128 rows, and tiles with rows of no token."""
    run_checked([(300, [(5, 1)] * 3), (700, [(40, 1), (9, 3)]), (50, [(200, 30)] if force else [(200, 1)])], H, K, 32, seed=H, force=force)


def test_two_calls_at_once(native_lib):
    """Two streams, a workspace each."""
    from continuous_batching_ragged_gb300 import api
    steps = [Step([(400, [(90 + i, 1)] * 20), (100, [(300, 70)])], 8, 2, 16, seed=40 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, stream in zip(steps, streams):
            st.run(stream=stream)
    for st, stream in zip(steps, streams):
        api.cb_check_device_errors(stream)
        st.check()


@pytest.mark.parametrize("fault", ["prefix too long", "negative prefix", "gap", "overlap", "not all", "start", "page", "context",
                                   "no query", "tokens"])
def test_bad_metadata_of_a_small_step(native_lib, fault):
    """The same of steps that every CTA plans for itself."""
    from continuous_batching_ragged_gb300 import api, native
    st = Step([(300, [(5, 1)] * 4), (200, [(8, 1)] * 3), (50, [(40, 1)] * 2)], 8, 2, 16, seed=9, ballast=False)
    good, error, n = [0, 1, 2, 3, 4, 6, 7, 8], "INVALID", 9
    if fault == "prefix too long":
        st.ctx[5] = 200
    elif fault == "negative prefix":
        st.prefix[1], good = -3, [0, 1, 2, 3, 7, 8]
    elif fault == "gap":
        st.cu_groups[1], good = n + 1, []
    elif fault == "overlap":
        st.cu_groups[2], good = 3, []
    elif fault == "not all":
        st.cu_groups[3], good = n - 1, []
    elif fault == "start":
        st.cu_groups[0], good = 1, []
    elif fault == "page":
        st.tables[5, 4], error = st.cache.num_blocks, "BOUNDS"
    elif fault == "context":
        st.ctx[5] = st.max_ctx + 1
    elif fault == "no query":
        st.cu[6], good = 5, [0, 1, 2, 3, 4, 7, 8]      # sequence 5 has no row, sequence 6 two: more than max_q_len
    elif fault == "tokens":
        st.cu[9], good = 10, range(8)
    st.run()
    with pytest.raises(native.CBError, match=error):
        api.cb_check_device_errors()
    st.check(good)
    if not good:
        assert bool(st.out.isnan().all())
    elif error == "INVALID" and fault not in ("no query", "tokens"):
        for s in set(range(9)) - set(good):
            assert bool(st.out[s].isnan().all())


@pytest.mark.parametrize("S", [1, 32, 33, 255, 256, 257])
@pytest.mark.parametrize("H,K,q", [(8, 2, 1), (8, 8, 3), (128, 1, 1), (100, 1, 1)])
def test_few_sequences(native_lib, S, H, K, q):
    """Steps on both sides of what a CTA's threads plan, in groups of three, with rows behind the last sequence."""
    from continuous_batching_ragged_gb300 import api
    groups = [(40 * i % 300, [(q + 37 * j % 200, q if j % 2 else 1) for j in range(i, min(i + 3, S))]) for i in range(0, S, 3)]
    st = Step(groups, H, K, 16, seed=S, ballast=False)
    rows = len(st.q)
    more = torch.full((7, H, A), float("nan"), dtype=torch.bfloat16, device="cuda")
    st.q, st.out = torch.cat([st.q, more]), torch.cat([st.out, more])
    n = api.cb_shared_prefix_workspace_size(st.cache, H, S, rows + 7, len(groups), st.max_ctx)
    st.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    st.run()
    api.cb_check_device_errors()
    st.check()
    assert bool(st.out[rows:].isnan().all())
    first = st.out[:rows].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    for _ in range(2):
        st.out.fill_(float("nan"))
        graph.replay()
    api.cb_check_device_errors()
    assert torch.equal(first, st.out[:rows])


def test_one_long_sequence(native_lib):
    """More units than warps, for one row."""
    run_checked([(100, [(70_000, 1)])], 16, 16, 16, seed=14, ballast=False)


@pytest.mark.parametrize("S,H,K,q,longest", [(3, 8, 8, 1, 128), (3, 8, 8, 1, 129), (90, 8, 4, 1, 384), (90, 8, 4, 1, 385),
                                             (50, 16, 8, 9, 300)])
def test_short_contexts(native_lib, S, H, K, q, longest):
    """Rows of one chunk, which no join follows, on both sides of their lengths."""
    from continuous_batching_ragged_gb300 import api
    own = [max(q, 1 + 53 * i % (longest - 33)) for i in range(S - 1)] + [longest - 33]
    st = run_checked([(33, [(n, q if i % 2 else 1) for i, n in enumerate(own)])], H, K, 16, seed=S, ballast=False)
    assert st.max_ctx == longest
    st.ctx[1] = longest + 1                            # left out, and its rows as they were
    st.out.fill_(float("nan"))
    st.run()
    from continuous_batching_ragged_gb300 import native
    with pytest.raises(native.CBError, match="INVALID"):
        api.cb_check_device_errors()
    assert bool(st.out[st.cu_l[1]:st.cu_l[2]].isnan().all())
    st.check([s for s in range(S) if s != 1])


def pieces(st):
    """Pieces that the last call's plan listed; -1 where its CTAs planned the step themselves, without sharing."""
    return int(st.ws[:4].view(torch.int32))


@pytest.mark.parametrize("H,K", [(8, 1), (16, 2)])
@pytest.mark.parametrize("prefix", [0, 400])
@pytest.mark.parametrize("ballast", [False, True])
@pytest.mark.parametrize("singles,empty", [(7, 8), (3, 6)])
def test_sequences_without_tokens_beside_a_chunk(native_lib, H, K, prefix, ballast, singles, empty):
    """Sequences that have no row leave room for a chunk among no more tokens than sequences, or hardly more: they are
    left out and reported, and the others run."""
    from continuous_batching_ragged_gb300 import api, native
    chunk = 64 // (H // K) + 1
    st = Step([(prefix, [(20, chunk)] + [(5 + i, 1) for i in range(singles)] + [(9, 0)] * empty)], H, K, 16, seed=15, ballast=ballast)
    assert (len(st.q) - len(st.q_l) + 1) * (H // K) <= 64
    st.run()
    with pytest.raises(native.CBError, match="INVALID"):
        api.cb_check_device_errors()
    st.check([s for s, n in enumerate(st.q_l) if n > 0])


@pytest.mark.parametrize("chunk", [False, True])
def test_small_groups_beside_a_chunk_read_their_own(native_lib, chunk):
    """Pairs whose pieces take longer than the reads they save do not share, whatever the bound on query tokens allows
    for and whatever chunk runs beside them."""
    pairs = [(96, [(1 + i % 9, 1), (20, 1)]) for i in range(150)]
    st = run_checked(pairs + [(0, [(100, 100)] if chunk else [(7, 2)] * 16)], 32, 8, 16, seed=16, force=True)
    assert 0 < pieces(st) < len(pairs) * 8           # the other group's, and the chunk's


@pytest.mark.parametrize("H,K,B", HEADS)
def test_prefix_lengths_of_groups_with_a_chunk(native_lib, H, K, B):
    """Prefixes around blocks and KV tiles, whatever sharing them saves: a chunk's rows are pieces either way."""
    c = 64 // (H // K) + 1
    prefixes = (0, 1, B - 1, B, B + 1, 127, 128, 129, 256, 257, 640, 1000)
    st = run_checked([(p, [(1, 1), (c + 3, c), (130, 1)]) for p in prefixes], H, K, B, seed=17 + H + K)
    assert pieces(st) >= K * (len(prefixes) + sum(p >= B for p in prefixes) + 1)


@pytest.mark.parametrize("H,K,B", HEADS)
def test_sizes_of_groups_with_a_chunk(native_lib, H, K, B):
    """From the chunk's rows alone behind the prefix to more rows than two tiles hold."""
    c, tt = 64 // (H // K) + 1, 128 // (H // K)
    sizes = sorted({c + 1, c + 2, tt - 1, tt, tt + 1, 2 * tt, 2 * tt + 1} - set(range(c + 1)))
    st = run_checked([(300, [(c, c)] + [(1 + i % 7, 1) for i in range(n - c)]) for n in sizes], H, K, B, seed=18 + H)
    assert pieces(st) >= K * (2 * len(sizes) + 1)


@pytest.mark.parametrize("fault", ["first page", "own page", "length"])
def test_bad_pages_of_groups_with_a_chunk(native_lib, fault):
    """A bad page that the whole group reads costs the group, any other its own sequence."""
    from continuous_batching_ragged_gb300 import api, native
    st = Step([(300, [(5, 1)] * 2 + [(40, 33)]), (200, [(8, 1)] * 2 + [(50, 17)])], 8, 2, 16, seed=19)
    good, error = [0, 1, 2], "BOUNDS"
    if fault == "first page":
        st.tables[3, 2] = -1
    elif fault == "own page":
        st.tables[5, 14], good = st.cache.num_blocks, [0, 1, 2, 3, 4]
    else:
        st.ctx[4], good, error = 150, [0, 1, 2, 3, 5], "INVALID"
    st.run()
    with pytest.raises(native.CBError, match=error):
        api.cb_check_device_errors()
    st.check(good)
    assert pieces(st) >= 2 * 5


@pytest.mark.parametrize("empty", [25, 200])
def test_empty_groups_do_not_stop_sharing(native_lib, empty):
    """Reads that one group saves are saved whatever the number of empty groups around it, captured too."""
    from continuous_batching_ragged_gb300 import api
    group = [(2048, [(1 + i % 7, 1) for i in range(26)])]
    st = run_checked([(0, [])] * (empty // 2) + group + [(0, [])] * (empty - empty // 2), 32, 8, 16, seed=20, ballast=False)
    assert pieces(st) > 0
    alone = Step(group, 32, 8, 16, seed=20, ballast=False)
    assert torch.equal(alone.run(), st.out) and pieces(alone) == pieces(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    st.out.fill_(float("nan"))
    graph.replay()
    api.cb_check_device_errors()
    assert torch.equal(alone.out, st.out)


def test_captured_among_small_and_shared_steps(native_lib):
    """One captured call over groups that leave the step small, then over one group, then back; rows behind stay."""
    from continuous_batching_ragged_gb300 import api
    sizes = dict(width=200, num_blocks=4200, ballast=False)
    apart = Step([(2000 - 30 * i, [(9 + i, 1)]) for i in range(28)], 32, 8, 16, seed=21, **sizes)
    shared = Step([(0, [])] * 20 + [(1984, [(30 - i, 1) for i in range(28)])] + [(7, [])] * 7, 32, 8, 16, seed=22, **sizes)
    assert len(apart.groups) == len(shared.groups) == len(apart.q_l)
    calls = [{n: getattr(st, n).clone() for n in ("q", "cu", "ctx", "tables", "cu_groups", "prefix")} for st in (apart, shared)]
    pools = [(st.cache.k.clone(), st.cache.v.clone()) for st in (apart, shared)]
    run = apart
    run.max_ctx = 2048
    run.out = torch.full((31, 32, A), float("nan"), dtype=torch.bfloat16, device="cuda")
    run.q = torch.cat([run.q, torch.zeros_like(run.q[:3])])
    n = api.cb_shared_prefix_workspace_size(run.cache, 32, 28, 31, 28, 2048)
    run.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    run.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run.run()
    for i in (0, 1, 0, 1):
        for name, t in calls[i].items():
            getattr(run, name)[:len(t)].copy_(t)
        run.cache.k.copy_(pools[i][0])
        run.cache.v.copy_(pools[i][1])
        run.out.fill_(float("nan"))
        graph.replay()
        api.cb_check_device_errors()
        st = (apart, shared)[i]
        st.out = run.out
        st.check()
        assert bool(run.out[28:].isnan().all()) and (pieces(run) > 0) == (i == 1)


@pytest.mark.parametrize("fault", ["prefix too long", "gap", "page", "no query"])
@pytest.mark.parametrize("shared", [False, True])
def test_bad_metadata_where_the_groups_decide(native_lib, fault, shared):
    from continuous_batching_ragged_gb300 import api, native
    members = [(9 + i, 1) for i in range(30)]
    groups = [(0, [])] * 29 + [(2000, members)] if shared else [(2000, [m]) for m in members]
    st = Step(groups, 8, 8, 16, seed=23, ballast=False)
    good, error = [s for s in range(30) if s != 5], "INVALID"
    if fault == "prefix too long":
        st.ctx[5] = 1200
    elif fault == "gap":
        st.cu_groups[29], good = 31, []
    elif fault == "page":
        st.tables[5, 125], error = st.cache.num_blocks, "BOUNDS"
    elif fault == "no query":
        st.cu[6], good = 5, [s for s in range(30) if s not in (5, 6)]
    st.run()
    with pytest.raises(native.CBError, match=error):
        api.cb_check_device_errors()
    st.check(good)
    if not good:
        assert bool(st.out.isnan().all())
