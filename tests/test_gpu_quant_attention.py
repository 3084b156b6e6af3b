"""cb_ragged_attention_q8 against softmax(q K^T) V of every sequence over its own
keys and values, number * scale, in 64 bits.

Tolerance.  An output is sum_j p_j v_j with sum p_j = 1.  Weights are rounded for
the tensor core to f16, by half a step 2^-11 of each, or by 2^-25 of the largest weight
(times the value scale) where a weight is too small for f16's normal numbers.  So an
output moves by at most 2^-11 a + 2^-25 b, a = sum_j p_j |v_j|, b = max_j(p_j s_j) sum_j
|n_j|, v_j = s_j n_j; the output's own rounding by 2^-8 of its value.  In fp32 a score is
a sum of 128 products: off by at most 128 * 2^-24 * r, r the row's largest sum of
|q_d k_d| in the exp2 domain (and by 2^-38 of the largest |q_d| times sum |k_d|,
where a query number is below f16's normal numbers), which moves p_j by ln 2 times
that, relatively; the sums over up to 2^16 keys are trees and tensor-core chains
below 2^-12 relative.  Both count for numerator and denominator."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

A = 128
E4M3 = torch.float8_e4m3fn


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Step:
    """Sequences (own keys, query tokens), own keys with the query tokens; or groups of them, [(prefix, [...]), ...], that share
    whole pages of their prefix."""

    def __init__(self, seqs, H, K, B, groups=False, seed=0, q_scale=1.0, k_slope=0.0, spread=2.0, extra=3):
        from continuous_batching_ragged_gb300 import api
        self.groups = seqs if groups else [(0, [m]) for m in seqs]
        g = torch.Generator(device="cuda").manual_seed(seed)
        flat = [(p, own, n) for p, members in self.groups for own, n in members]
        self.H, self.K, self.B = H, K, B
        self.ctx_l, self.q_l = [p + own for p, own, _ in flat], [n for _, _, n in flat]
        shared = [p // B if members else 0 for p, members in self.groups]
        need = sum(-(-c // B) for c in self.ctx_l) - sum((len(m) - 1) * s for (_, m), s in zip(self.groups, shared) if m) + extra
        ids = torch.randperm(need, generator=torch.Generator().manual_seed(seed)).tolist()
        width = max(-(-c // B) for c in self.ctx_l) + 2
        # numbers in use are finite, all others NaN: the slots behind a context, the pages in no table, their scales
        self.k, self.v = (torch.full((need, K, B, A), float("nan"), device="cuda").to(E4M3) for _ in range(2))
        self.ks, self.vs = (torch.full((need, K), float("nan"), device="cuda") for _ in range(2))
        self.tables_l, self.cu_groups_l, at, self.keys = [], [0], 0, []
        for (p, members), n_shared in zip(self.groups, shared):
            common = ids[at:at + n_shared]
            at += len(common)
            for i, (own, _) in enumerate(members):
                c = p + own
                mine = ids[at:at + -(-c // B) - len(common)]
                at += len(mine)
                row = common + mine
                self.tables_l.append(row + [-1] * (width - len(row)))
                for j0 in range(0 if i == 0 else len(common), len(row)):
                    n = min(B, c - j0 * B)
                    for pool, scale, slope in ((self.k, self.ks, k_slope), (self.v, self.vs, 0.0)):
                        x = torch.randn((K, n, A), generator=g, device="cuda")
                        x = x * torch.exp2(spread * (2 * torch.rand((K, 1, 1), generator=g, device="cuda") - 1))
                        if slope:                  # scores climb along the keys, so the running maximum keeps moving
                            x = x + slope * (j0 * B + torch.arange(n, device="cuda")[None, :, None]) / math.sqrt(A)
                        m, e = torch.frexp(x.abs().amax((1, 2)))
                        s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875))
                        pool[row[j0], :, :n] = (x / s[:, None, None]).to(E4M3)
                        scale[row[j0]] = s
            self.cu_groups_l.append(self.cu_groups_l[-1] + len(members))
        self.cu_l = [0]
        for n in self.q_l:
            self.cu_l.append(self.cu_l[-1] + n)
        self.q = (torch.randn((self.cu_l[-1], H, A), generator=g, device="cuda") * q_scale + (k_slope > 0) * 1.0).bfloat16()
        self.cache = api.QuantKVCache(self.k, self.v, self.ks, self.vs)
        self.cu, self.ctx, self.tables = ints(self.cu_l), ints(self.ctx_l), ints(self.tables_l)
        self.cu_groups, self.prefix = (ints(self.cu_groups_l), ints([p for p, _ in self.groups])) if groups else (None, None)
        self.max_q, self.max_ctx, self.scale = max(self.q_l), max(self.ctx_l), 1 / math.sqrt(A)
        self.out = torch.full_like(self.q, float("nan"))
        n = api.cb_ragged_attention_q8_workspace_size(self.cache, H, len(flat), self.cu_l[-1], self.max_ctx,
                                                      num_groups=len(self.groups) if groups else 0)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")   # contents need no initialisation

    def run(self, stream=None):
        from continuous_batching_ragged_gb300 import api
        api.cb_ragged_attention_q8(self.q, self.cache, self.cu, self.ctx, self.tables, max_q_len=self.max_q,
                                   max_context_len=self.max_ctx, scale=self.scale, out=self.out, workspace=self.ws,
                                   cu_groups=self.cu_groups, prefix_lens=self.prefix, stream=stream)
        return self.out

    def check(self, sequences=None):
        G = self.H // self.K
        for s in range(len(self.q_l)) if sequences is None else sequences:
            c, a, b = self.ctx_l[s], self.cu_l[s], self.cu_l[s + 1]
            pages = torch.tensor(self.tables_l[s][:-(-c // self.B)], device="cuda")

            def rows(x):
                return x.transpose(0, 1).reshape(self.K, -1, A)[:, :c]

            def numbers(pool):
                return pool.view(torch.uint8)[pages].view(E4M3).double()

            k = rows(numbers(self.k) * self.ks[pages].double()[..., None, None])
            n = rows(numbers(self.v))
            vs = self.vs[pages].double()[..., None, None].expand(-1, -1, self.B, 1).transpose(0, 1).reshape(self.K, -1)[:, :c]
            q = self.q[a:b].double().view(b - a, self.K, G, A)
            late = torch.arange(c, device="cuda")[None] > torch.arange(c - (b - a), c, device="cuda")[:, None]
            for h in range(self.K):
                v, to_log2 = n[h] * vs[h, :, None], self.scale * math.log2(math.e)
                sc = torch.einsum("igd,jd->igj", q[:, h], k[h]) * self.scale
                p = torch.softmax(sc.masked_fill(late[:, None], -math.inf), -1)
                want, mag = p @ v, p @ v.abs()
                small = 2.0 ** -25 * (p * vs[h]).amax(-1, keepdim=True) * n[h].abs().sum(0)
                r = (torch.einsum("igd,jd->igj", q[:, h].abs(), k[h].abs()) * to_log2).amax(-1, keepdim=True)
                tiny = 2.0 ** -38 * q[:, h].abs().amax(-1, keepdim=True) * k[h].abs().sum(-1).amax() * to_log2
                rel = 2.0 ** -11 + 2 * (math.log(2) * (128 * 2.0 ** -24 * r + tiny) + 2.0 ** -12)
                off = (self.out[a:b, h * G:(h + 1) * G].double() - want).abs()
                lim = rel * mag + small + 2.0 ** -8 * (want.abs() + rel * mag + small)
                assert bool((off <= lim).all()), (s, h, float((off - lim).max()))


def run_checked(*args, sequences=None, **kw):
    from continuous_batching_ragged_gb300 import api
    st = Step(*args, **kw)
    st.run()
    api.cb_check_device_errors()
    st.check(sequences)
    return st


HEADS = [(8, 8, 16), (8, 2, 16), (4, 1, 64), (12, 4, 32), (16, 1, 16), (5, 1, 128), (6, 2, 16), (32, 1, 32), (128, 1, 16)]


@pytest.mark.parametrize("H,K,B", HEADS)
def test_decode_lengths(native_lib, H, K, B):
    """Contexts around tiles and pages, from one key on; some cut into several chunks."""
    run_checked([(c, 1) for c in (1, 2, 15, 16, 17, 31, 33, B - 1, B, B + 1, 2 * B + 1, 127, 128, 129, 511, 640, 1000, 3001)],
                H, K, B, seed=H + K)


@pytest.mark.parametrize("H,K,B", HEADS)
@pytest.mark.parametrize("q", [1, 2, 3])
def test_few_short_streams(native_lib, H, K, B, q):
    """Few sequences of few tokens and short contexts, which take a CTA each; with a larger bound on the contexts they are
    dealt out to all warps.  A sequence whose length does not hold has no rows of its own, before or behind others."""
    from continuous_batching_ragged_gb300 import api, native
    for seqs in ([(q, q)], [(16 * i + q, q) for i in (0, 1, 15, 16)], [(q + 30, q), (500, q)], [(300, q), (17 + q, 1), (512, q)]):
        st = run_checked(seqs, H, K, B, seed=5 + q)
        few = st.out.clone()
        st.tables = torch.nn.functional.pad(st.tables, (0, -(-6000 // B)), value=-1)
        st.max_ctx = 6000
        n = api.cb_ragged_attention_q8_workspace_size(st.cache, H, len(seqs), st.cu_l[-1], st.max_ctx)
        st.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        st.out.fill_(float("nan"))
        st.run()
        api.cb_check_device_errors()
        st.check()
        if len(seqs) > 1:
            for max_ctx in (512, 6000):
                for bad in (0, len(seqs) - 1):
                    st.max_ctx = max_ctx
                    st.ctx[bad] = -1
                    st.out.fill_(float("nan"))
                    st.run()
                    with pytest.raises(native.CBError) as e:
                        api.cb_check_device_errors()
                    assert e.value.status == native.CB_ERR_INVALID
                    assert bool(st.out[st.cu_l[bad]:st.cu_l[bad + 1]].isnan().all())
                    st.check([s for s in range(len(seqs)) if s != bad])
                    st.ctx[bad] = st.ctx_l[bad]
        st.max_ctx = max(st.ctx_l)
        st.run()
        torch.cuda.synchronize()
        assert torch.equal(few, st.out)


@pytest.mark.parametrize("H,K,B", HEADS)
def test_many_decode_rows(native_lib, H, K, B):
    """More sequences than a CTA has threads: the step is planned by a kernel of its own."""
    run_checked([(1 + (37 * i) % 450, 1) for i in range(300)], H, K, B, seed=10 + H, sequences=range(0, 300, 7))


@pytest.mark.parametrize("H,K,B", [(8, 8, 16), (8, 2, 32), (16, 2, 16), (12, 4, 64), (32, 1, 128)])
@pytest.mark.parametrize("q", [2, 5, 17, 64, 150, 300])
def test_chunks(native_lib, H, K, B, q):
    """Chunks with their causal mask, at the beginning of their sequence and behind cached keys, among decode rows."""
    run_checked([(q, q), (q + 40, q), (3, 1), (q + 1, q), (700, 1), (q + 1111, q), (1, 1)], H, K, B, seed=20 + q)


def test_one_long_chunk(native_lib):
    """More query rows than one pair of tiles and more keys than one segment."""
    run_checked([(2900, 700)], 4, 2, 16, seed=30)


def test_long_context(native_lib):
    st = run_checked([(40_000, 1), (9000, 1), (13, 1)], 8, 2, 16, seed=31)
    first = st.out.clone()
    st.ws.fill_(7)
    st.out.fill_(float("nan"))
    st.run()
    torch.cuda.synchronize()
    assert torch.equal(first, st.out)                # the same bits from call to call


@pytest.mark.parametrize("members", [1, 3, 40, 200])
@pytest.mark.parametrize("H,K,B", [(8, 8, 16), (32, 8, 16), (16, 1, 64)])
def test_shared_prefixes(native_lib, members, H, K, B):
    """Groups that share pages: none, a few and all of their keys but one; chunks among them; a group without sequences."""
    big = (2050, [(1 + (29 * i) % 70, 1) for i in range(members)])
    run_checked([big, (B - 1, [(5, 1), (9, 2)]), (77, []), (B, [(1, 1)] * 3), (300, [(90, 70), (3, 3), (1, 1)]), (0, [(33, 1)])],
                H, K, B, groups=True, seed=40 + members, sequences=list(range(0, members, 13)) + list(range(members, members + 9)))


@pytest.mark.parametrize("q", [1, 130])
def test_growing_scores(native_lib, q):
    """The running maximum is overtaken again and again."""
    run_checked([(max(q, 900), q), (q + 600, q), (300, 1)], 8, 2, 16, seed=50, q_scale=0.5, k_slope=0.2)


@pytest.mark.parametrize("q", [1, 130])
def test_peaked_rows(native_lib, q):
    """Scores of tens: nearly all weight on single keys."""
    run_checked([(1500, q), (200, 1)] * 2, 8, 8, 16, seed=51, q_scale=8.0)


@pytest.mark.parametrize("q", [1, 130])
@pytest.mark.parametrize("spread", [0.0, 8.0])
def test_scales_apart(native_lib, q, spread):
    """Blocks whose numbers differ by factors of up to 2^16: the largest weight times scale is not at the largest score."""
    run_checked([(900, q), (q + 30, q), (500, 1)], 8, 2, 16, seed=52, spread=spread, q_scale=0.2)


@pytest.mark.parametrize("q", [1, 130])
def test_value_scales_of_any_size(native_lib, q):
    """Value scales from 2^-90 to 2^60, the larger ones at keys without weight, and key scales that are no powers of two."""
    from continuous_batching_ragged_gb300 import api
    st = Step([(700, q), (333, 1)], 4, 2, 16, seed=53, q_scale=0.3)
    e = (torch.arange(st.vs.shape[0], device="cuda") * 37) % 151 - 90
    st.vs.copy_(torch.exp2(e.float())[:, None].expand_as(st.vs))
    st.ks.mul_(1.37)
    st.run()
    api.cb_check_device_errors()
    st.check()


@pytest.mark.parametrize("q", [1, 130])
def test_query_magnitudes(native_lib, q):
    """Query rows of zeros, of the smallest and largest numbers, and with numbers far apart in one row."""
    from continuous_batching_ragged_gb300 import api
    st = Step([(200, q), (130, 1)], 8, 8, 16, seed=54)
    st.q[:, 0] = 0
    st.q[:, 1] *= 2.0 ** -120
    st.q[:, 2] *= 2.0 ** -60
    st.q[:, 3, ::2] *= 2.0 ** -20
    st.q[:, 4, 1:] *= 2.0 ** -35
    st.q[:, 5] *= 2.0 ** 7
    st.run()
    api.cb_check_device_errors()
    st.check()


@pytest.mark.parametrize("H,K", [(8, 2), (12, 4)])
@pytest.mark.parametrize("q", [1, 3, 130])
@pytest.mark.parametrize("far", [2.0 ** 16, 2.0 ** 40, math.inf])
def test_enormous_scores(native_lib, H, K, q, far):
    """Scores up to 2^20 are weighed like others; beyond fp32's reach, or infinite queries, they end, and leave other sequences'
    rows alone."""
    from continuous_batching_ragged_gb300 import api
    st = Step([(q + 300, q), (q + 77, q), (900, 1)], H, K, 16, seed=63)
    st.q[st.cu_l[1]:st.cu_l[2], ::2] *= far
    st.run()
    api.cb_check_device_errors()
    st.check([0, 1, 2] if far == 2.0 ** 16 else [0, 2])


@pytest.mark.parametrize("q", [1, 130])
def test_not_finite_keys_behind_the_mask(native_lib, q):
    """A NaN among the keys of a chunk's last token leaves the rows before it alone."""
    from continuous_batching_ragged_gb300 import api
    st = Step([(q + 20, q), (50, 1)], 4, 4, 16, seed=55)
    c = st.ctx_l[0] - 1
    page = st.tables_l[0][c // 16]
    good = st.k[page, :, c % 16].clone()
    st.k[page, :, c % 16] = torch.full((4, A), float("nan"), device="cuda").to(E4M3)
    st.run()
    api.cb_check_device_errors()
    st.k[page, :, c % 16] = good
    last = st.out[q - 1].clone()
    assert bool(last.isnan().all())
    st2 = Step([(q + 20, q), (50, 1)], 4, 4, 16, seed=55)
    st2.run()
    st.out[q - 1] = st2.out[q - 1]
    st.check()


def test_packed_equals_alone(native_lib):
    """A sequence's rows do not depend, beyond rounding, on what is packed with it; nothing leaks between sequences."""
    st = run_checked([(517, 1), (90, 30), (2, 1), (300, 1)], 8, 2, 16, seed=56)
    before = st.out.clone()
    for s in (0, 1, 3):                              # other values in one sequence change its rows alone
        st.q[st.cu_l[s]:st.cu_l[s + 1]] *= -1
        st.run()
        torch.cuda.synchronize()
        for o in range(4):
            a, b = st.cu_l[o], st.cu_l[o + 1]
            assert torch.equal(st.out[a:b], before[a:b]) == (o != s)
        st.q[st.cu_l[s]:st.cu_l[s + 1]] *= -1


@pytest.mark.parametrize("seqs", [[(40, 1), (50, 1), (60, 1)], [(40, 1)] * 300, [(300, 130), (50, 1), (60, 1)]])
def test_bad_metadata(native_lib, seqs):
    """Sequences whose lengths contradict the bounds are left out and reported, pages outside the pool too; the others are right."""
    from continuous_batching_ragged_gb300 import api, native
    st = Step(seqs, 8, 2, 16, seed=57)
    others = [s for s in range(min(len(seqs), 9)) if s != 1]

    def run(status):
        st.out.fill_(float("nan"))
        st.run()
        with pytest.raises(native.CBError) as e:
            api.cb_check_device_errors()
        assert e.value.status == status
        st.check(others)

    a, b = st.cu_l[1], st.cu_l[2]
    for bad in (0, -3, st.max_ctx + 1):
        st.ctx[1] = bad
        run(native.CB_ERR_INVALID)
        assert bool(st.out[a:b].isnan().all())
    st.ctx[1] = st.ctx_l[1]
    for bad in (-1, st.k.shape[0], 2 ** 31 - 1):
        st.tables[1, 0] = bad
        run(native.CB_ERR_BOUNDS)
    st.tables[1, 0] = st.tables_l[1][0]
    st.run()
    api.cb_check_device_errors()
    st.check(range(min(len(seqs), 9)))


@pytest.mark.parametrize("members,q", [(3, 1), (200, 1), (5, 140)])
def test_bad_groups(native_lib, members, q):
    """Groups that do not cover the sequences in order leave the whole step out; a prefix that its sequences do not have leaves
    them out.  Both are reported, with the plan kernel and without it."""
    from continuous_batching_ragged_gb300 import api, native
    groups = [(64, [(10 + i % 50, 1) for i in range(members)]), (200, [(q + 5, q), (20, 1)])]
    st = Step(groups, 8, 2, 16, groups=True, seed=61)
    S = members + 2

    def run():
        st.out.fill_(float("nan"))
        st.run()
        with pytest.raises(native.CBError) as e:
            api.cb_check_device_errors()
        assert e.value.status == native.CB_ERR_INVALID

    for bad in ([0, members, S - 1], [0, S + 1, S], [1, members, S], [-5, members, S], [0, members, 2 ** 31 - 1]):
        st.cu_groups.copy_(ints(bad))
        run()
        assert bool(st.out.isnan().all())
    st.cu_groups.copy_(ints(st.cu_groups_l))
    for bad in (-1, 207, 2 ** 31 - 1):               # of its sequences' 205 + q and 220 keys, q and 1 are new
        st.prefix[1] = bad
        run()
        st.check(range(0, members, 7))
        if bad != 207:
            assert bool(st.out[st.cu_l[members]:].isnan().all())
    st.prefix[1] = 200
    st.run()
    api.cb_check_device_errors()
    st.check()


def test_wide_offsets(native_lib):
    """Pages whose numbers begin behind 2^31 and 2^32 bytes of their pools."""
    from continuous_batching_ragged_gb300 import api
    st = Step([(150, 1), (300, 140), (40, 1)], 8, 8, 128, seed=62)
    blocks = 2 ** 32 // (8 * 128 * A) + 40
    at = [2 ** 31 // (8 * 128 * A) + i // 2 if i % 2 else blocks - 1 - i for i in range(st.k.shape[0])]
    to = torch.tensor(at, device="cuda")
    pools = []
    for x in (st.k, st.v):
        far = torch.full((blocks, 8, 128, A), 0x7f, dtype=torch.uint8, device="cuda")
        far[to] = x.view(torch.uint8)
        pools.append(far.view(E4M3))
    scales = []
    for x in (st.ks, st.vs):
        far = torch.full((blocks, 8), float("nan"), device="cuda")
        far[to] = x
        scales.append(far)
    near, near_tables = st.cache, st.tables.clone()
    st.cache = api.QuantKVCache(*pools, *scales)
    st.tables = torch.where(near_tables >= 0, to.int()[near_tables.clamp(min=0).long()], near_tables)
    for cu in (slice(0, 3), slice(0, 1)):            # with a chunk, by the plan; one decode row, without it
        st.out.fill_(float("nan"))
        q, seqs = (st.q, 3) if cu.stop == 3 else (st.q[:1], 1)
        api.cb_ragged_attention_q8(q, st.cache, st.cu[:seqs + 1], st.ctx[:seqs], st.tables[:seqs], max_q_len=st.max_q if seqs == 3 else 1,
                                   max_context_len=st.max_ctx, scale=st.scale, out=st.out[:q.shape[0]], workspace=st.ws)
        api.cb_check_device_errors()
        st.check(range(seqs))


@pytest.mark.parametrize("seqs", [[(400, 1), (50, 1), (333, 1)], [(300 + i % 60, 1) for i in range(270)], [(400, 140), (50, 1)]])
def test_streams_and_graphs(native_lib, seqs):
    """On another stream; two at once with workspaces of their own; captured and replayed over new contents."""
    from continuous_batching_ragged_gb300 import api
    a, b = Step(seqs, 8, 2, 16, seed=58), Step(seqs, 8, 2, 16, seed=59)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(sa)
        b.run(sb)
    torch.cuda.synchronize()
    a.check(range(0, len(seqs), 9))
    b.check(range(0, len(seqs), 9))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=sa):
        a.run(sa)
    a.q.copy_(b.q)
    for x, y in ((a.k, b.k), (a.v, b.v)):
        x.view(torch.uint8).copy_(y.view(torch.uint8))
    a.ks.copy_(b.ks)
    a.vs.copy_(b.vs)
    a.tables.copy_(b.tables)
    a.ctx[0] = a.ctx_l[0] = 290                      # shorter: the same sizes on the host
    b.ctx_l[0] = 290
    a.tables_l = b.tables_l
    for _ in range(2):
        a.out.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    api.cb_check_device_errors()
    a.check(range(0, len(seqs), 9))


@pytest.mark.parametrize("H,K", [(4, 4), (8, 2)])
def test_serving_steps(native_lib, H, K):
    """Steps as a server runs them, on one stream: prompts appended in chunks, then tokens, attended over the cache in 8 bits and
    read back from it; the attention of the numbers read back is the attention."""
    from continuous_batching_ragged_gb300 import api
    B, blocks = 16, 60
    cache = api.QuantKVCache.empty(blocks, K, B, A)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x7f)
    cache.k_scale.fill_(float("nan"))
    cache.v_scale.fill_(float("nan"))
    g = torch.Generator(device="cuda").manual_seed(60)
    perm = torch.randperm(blocks, generator=torch.Generator().manual_seed(60)).tolist()
    tables_l = [perm[20 * s:20 * s + 20] for s in range(3)]
    tables = ints(tables_l)
    held = [0, 0, 0]
    for step in range(9):
        new = [[30, 5, 70], [1, 40, 1], [140, 1, 1]][step] if step < 3 else [1, 1, 1]
        T = sum(new)
        scale = 2.0 ** (step % 3)
        q, k, v = (torch.randn((T, h, A), generator=g, device="cuda").mul(scale if h == K else 1).bfloat16() for h in (H, K, K))
        ctx_l = [a + n for a, n in zip(held, new)]
        slots = [tables_l[s][j // B] * B + j % B for s in range(3) for j in range(held[s], ctx_l[s])]
        cu = [0, new[0], new[0] + new[1], T]
        out = torch.full_like(q, float("nan"))
        n = api.cb_ragged_attention_q8_workspace_size(cache, H, 3, T, max(ctx_l))
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        api.cb_append_kv_q8(k, v, torch.tensor(slots, device="cuda"), cache)
        api.cb_ragged_attention_q8(q, cache, ints(cu), ints(ctx_l), tables, max_q_len=max(new), max_context_len=max(ctx_l),
                                   scale=1 / math.sqrt(A), out=out, workspace=ws)
        cu_keys = [0, ctx_l[0], ctx_l[0] + ctx_l[1], sum(ctx_l)]
        ko, vo = (torch.empty((sum(ctx_l), K, A), device="cuda") for _ in range(2))
        api.cb_gather_kv_q8(cache, tables, ints(cu_keys), k_out=ko, v_out=vo)
        api.cb_check_device_errors()
        assert bool(ko.isfinite().all()) and bool(vo.isfinite().all())
        for s in range(3):                           # this step's tokens, as far as 8 bits hold them
            a, n = cu[s], new[s]
            for x, o in ((k, ko), (v, vo)):
                off = (o[cu_keys[s + 1] - n:cu_keys[s + 1]] - x[a:a + n].float()).abs()
                assert bool((off <= x[a:a + n].float().abs() * 2.0 ** -4 + 2.0 ** -10 * 0.25).all())
            st = Step.__new__(Step)
            st.H, st.K, st.B, st.scale = H, K, B, 1 / math.sqrt(A)
            st.q, st.out, st.k, st.v, st.ks, st.vs = q, out, cache.k, cache.v, cache.k_scale, cache.v_scale
            st.cu_l, st.ctx_l, st.q_l, st.tables_l = cu, ctx_l, new, tables_l
            st.check([s])
        held = ctx_l


def run_repeated(*args, sequences=None, **kw):
    """Checked, and the same bits three times over: what one piece of a CTA leaves in shared memory is not the next one's."""
    st = run_checked(*args, sequences=sequences, **kw)
    first = st.out.clone()
    for _ in range(3):
        st.out.fill_(float("nan"))
        st.run()
        torch.cuda.synchronize()
        assert torch.equal(first, st.out)
    return st


# One pair of row tiles and one token: of such a chunk's two pieces one has both row tiles, one exactly one; and a prompt of one KV
# tile whose rows are pieces and fit one row tile (no such prompt with 128 heads on one).
TILES = [(8, 8, 16), (8, 2, 16), (32, 8, 16), (12, 4, 32), (16, 2, 64), (32, 1, 16), (128, 1, 16)]


def tile_sizes(H, K):
    G = H // K
    return 2 * (128 // G) + 1, (min(128 // G, 64 // G + 6) if G < 64 else 2)


@pytest.mark.parametrize("H,K,B", TILES)
@pytest.mark.parametrize("before", [0, 40, 600])
@pytest.mark.parametrize("kind", ["chunks", "prompts", "mixed"])
def test_pieces_in_turn(native_lib, H, K, B, before, kind):
    """More pieces than SMs, each CTA with several in turn: pieces whose second row tile is empty, and prompts of one KV tile, whose
    second slot is; a piece's queries stay until its last scores have read them."""
    odd, short = tile_sizes(H, K)
    n = -(-460 // (2 * K))
    chunk, prompt = (before + odd, odd), (short + min(before, 20), short)
    seqs = {"chunks": [chunk] * n, "prompts": [prompt] * (2 * n), "mixed": [chunk, prompt, (before + 3 * odd + 1, odd - 1), prompt, prompt] * (n // 2)}[kind]
    run_repeated(seqs, H, K, B, seed=70 + H + before, sequences=range(0, len(seqs), max(1, len(seqs) // 40)))


@pytest.mark.parametrize("H,K,B", TILES)
def test_group_pieces_in_turn(native_lib, H, K, B):
    """The same for groups whose members' rows are one pair of row tiles and one token, behind prefixes of several KV tiles."""
    odd, _ = tile_sizes(H, K)
    n = -(-320 // (2 * K))
    groups = [(640, [(1 + (7 * i + g) % 40, 1) for i in range(odd)]) for g in range(n)]
    S = n * odd
    run_repeated(groups, H, K, B, groups=True, seed=71 + H, sequences=range(0, S, max(1, S // 60)))


@pytest.mark.parametrize("q", [1, 3, 130])
@pytest.mark.parametrize("down", [100, 113, 114, 120])
def test_smallest_queries_and_largest_keys(native_lib, q, down):
    """Query numbers down to 2^-122, and key scales that bring their scores back to ones of about 1."""
    from continuous_batching_ragged_gb300 import api
    st = Step([(q + 200, q), (130, 1)], 8, 2, 16, seed=64)
    st.q *= 2.0 ** -down
    st.ks *= 2.0 ** (down - 1)
    st.run()
    api.cb_check_device_errors()
    st.check()


@pytest.mark.parametrize("more", [1, 70])
@pytest.mark.parametrize("seqs,groups", [([(40, 1), (700, 1)], False), ([(40, 1), (7, 3)], False), ([(30 + i % 50, 1) for i in range(600)], False),
                                         ([(300, 140), (50, 1)], False), ([(2000, [(9 + i, 1) for i in range(90)])], True)])
def test_rows_behind_the_last_sequence(native_lib, seqs, groups, more):
    """Rows of q and out that no sequence has stay as they were; with many heads on one, where a spare row counts as 128."""
    from continuous_batching_ragged_gb300 import api
    for H, K in ((8, 2), (128, 1)):
        st = Step(seqs, H, K, 16, groups=groups, seed=65)
        T = st.cu_l[-1]
        st.q = torch.cat([st.q, torch.randn((more, H, A), device="cuda").bfloat16()])
        st.out = torch.full_like(st.q, float("nan"))
        n = api.cb_ragged_attention_q8_workspace_size(st.cache, H, len(st.ctx_l), T + more, st.max_ctx, num_groups=len(seqs) if groups else 0)
        st.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        st.run()
        api.cb_check_device_errors()
        st.check(range(0, len(st.ctx_l), 1 + len(st.ctx_l) // 20))
        assert bool(st.out[T:].isnan().all()) and bool(st.out[:T].isfinite().all())
