"""cb_norm_rope_append against its formula in 64 bits.

Tolerance.  The kernel works in fp32 and rounds once.  A norm's relative error
is at most the sum's (a lane's chunk in order, then a tree: under 16 roundings)
halved by the square root, plus the reciprocal root's 2 steps and two products:
under 14 * 2^-24 in all; a turned element adds two products and a sum to the
errors of its two terms.  So an element is off by at most 16 * 2^-24 times
|y_a cos| + |y_b sin|, and by half a step of its type, relative to its value,
at the store."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def turned(x, w, eps, cos_sin, pos, interleaved):
    """(exact rows, sum of the magnitudes of each element's terms), fp64."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    y, mag = x.clone(), x.abs()
    if cos_sin is not None:
        half = cos_sin.shape[1] // 2
        c, s = (t.double()[:, None] for t in cos_sin[pos.long()].split(half, 1))
        i = torch.arange(half, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, mag


def close(got, exact, mag):
    half = torch.finfo(got.dtype).eps / 2
    off = (got.double() - exact).abs()
    lim = half * exact.abs() + (1 + half) * 16 * 2.0 ** -24 * mag
    assert bool((off <= lim).all()), float((off - lim).max())


class Step:
    def __init__(self, T, H, K, A, rot, *, dtype="bf16", interleaved=False, norm=(True, True), packed=False, block=16,
                 seed=0, positions=500, num_blocks=None):
        from continuous_batching_ragged_gb300 import api
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = DT[dtype]
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
        if packed:
            qkv = rnd(T, H + 2 * K, A)
            self.q, self.k, self.v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
        else:
            self.q, self.k, self.v = rnd(T, H, A), rnd(T, K, A), rnd(T, K, A)
        nb = num_blocks or T // block + 2
        self.cache = api.KVCache(rnd(nb, K, block, A), rnd(nb, K, block, A))
        self.before = (self.cache.k.clone(), self.cache.v.clone())
        self.slots = torch.randperm(nb * block, generator=g, device="cuda")[:T].to(torch.int64)
        self.pos = torch.randint(0, positions, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.wq = (1 + 0.3 * rnd(A).float()).to(dt) if norm[0] else None
        self.wk = (1 + 0.3 * rnd(A).float()).to(dt) if norm[1] else None
        self.cs = None
        if rot:
            ang = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * 1e4 ** (
                -torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
            self.cs = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        self.interleaved, self.block, self.eps = interleaved, block, 1e-5
        self.q_out = torch.full((T, H, A), float("nan"), dtype=dt, device="cuda")

    def run(self, dims=None, stream=None):
        from continuous_batching_ragged_gb300 import api
        api.cb_norm_rope_append(self.q, self.k, self.v, self.slots, self.cache, q_out=self.q_out,
                                positions=self.pos if self.cs is not None else None, cos_sin=self.cs, q_weight=self.wq,
                                k_weight=self.wk, eps=self.eps, interleaved=self.interleaved, dims=dims, stream=stream)

    def check(self, tokens=None, q_in=None):
        """`tokens`: those that the call processed (default all); every other row and slot is untouched."""
        T = self.q.shape[0]
        done = torch.ones(T, dtype=torch.bool, device="cuda") if tokens is None else tokens
        exact, mag = turned(self.q if q_in is None else q_in, self.wq, self.eps, self.cs,
                            self.pos.clamp(0, self.cs.shape[0] - 1) if self.cs is not None else None, self.interleaved)
        close(self.q_out[done], exact[done], mag[done])
        exact, mag = turned(self.k, self.wk, self.eps, self.cs,
                            self.pos.clamp(0, self.cs.shape[0] - 1) if self.cs is not None else None, self.interleaved)
        n_slots = self.cache.num_blocks * self.block
        kept = done & (self.slots >= 0) & (self.slots < n_slots)
        b, o = self.slots[kept] // self.block, self.slots[kept] % self.block
        close(self.cache.k[b, :, o], exact[kept], mag[kept])
        assert torch.equal(self.cache.v[b, :, o], self.v[kept])
        untouched = torch.ones(n_slots, dtype=torch.bool, device="cuda")
        untouched[self.slots[kept]] = False
        u = untouched.nonzero()[:, 0]
        for pool, old in zip((self.cache.k, self.cache.v), self.before):
            assert torch.equal(pool[u // self.block, :, u % self.block], old[u // self.block, :, u % self.block])


@pytest.mark.parametrize("dtype,A", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("part", [0, 1, 2])
def test_types_heads_and_pairs(native_lib, dtype, A, interleaved, part):
    from continuous_batching_ragged_gb300 import api
    rot = (A, A // 2, 16)[part]
    st = Step(37, *((4, 4), (5, 1), (12, 4))[part], A, rot, dtype=dtype, interleaved=interleaved, packed=part != 1,
              block=(16, 4, 1)[part], seed=part)
    st.run()
    api.cb_check_device_errors()
    st.check()


@pytest.mark.parametrize("T", [1, 2, 255, 2048])
@pytest.mark.parametrize("H,K", [(32, 32), (32, 8), (32, 1)])
def test_lengths(native_lib, T, H, K):
    from continuous_batching_ragged_gb300 import api
    st = Step(T, H, K, 128, 128, packed=True, seed=T)
    st.run()
    api.cb_check_device_errors()
    st.check()


@pytest.mark.parametrize("norm,rot", [((False, False), 64), ((True, False), 0), ((False, True), 64), ((False, False), 0)])
def test_parts_left_out(native_lib, norm, rot):
    """No norm of one or both, no rotation; with neither the rows come through bit for bit."""
    from continuous_batching_ragged_gb300 import api
    st = Step(40, 8, 2, 128, rot, norm=norm, seed=3)
    st.run()
    api.cb_check_device_errors()
    st.check()
    if norm == (False, False) and rot == 0:
        assert torch.equal(st.q_out, st.q)


def test_equals_append_without_norm_and_rotation(native_lib):
    """With nothing to compute the cache holds what cb_append_kv writes, bit for bit."""
    from continuous_batching_ragged_gb300 import api
    st = Step(70, 8, 2, 128, 0, norm=(False, False), seed=4)
    st.slots[5] = -1
    st.run()
    other = api.KVCache(st.before[0].clone(), st.before[1].clone())
    api.cb_append_kv(st.k, st.v, st.slots, other)
    api.cb_check_device_errors()
    assert torch.equal(other.k, st.cache.k) and torch.equal(other.v, st.cache.v)


def test_in_place_queries(native_lib):
    from continuous_batching_ragged_gb300 import api
    st = Step(50, 8, 2, 128, 128, seed=5)
    q_in = st.q.clone()
    st.q_out = st.q
    st.run()
    api.cb_check_device_errors()
    st.check(q_in=q_in)


def test_skipped_and_bad_tokens(native_lib):
    """A negative slot caches nothing; a slot past the pool or a position outside the
    table is reported, and every other token is written."""
    from continuous_batching_ragged_gb300 import api, native
    st = Step(64, 8, 2, 128, 128, seed=6)
    st.slots[3] = -1
    st.slots[10] = -(1 << 40)
    st.run()
    api.cb_check_device_errors()
    st.check()
    st = Step(64, 8, 2, 128, 128, seed=7)
    st.slots[9] = st.cache.num_blocks * 16
    st.run()
    with pytest.raises(native.CBError, match="BOUNDS"):
        api.cb_check_device_errors()
    st.check()
    for bad in (-1, 500, 2 ** 31 - 1):
        st = Step(64, 8, 2, 128, 128, seed=8)
        st.pos[20] = bad
        st.run()
        with pytest.raises(native.CBError, match="BOUNDS"):
            api.cb_check_device_errors()
        done = torch.ones(64, dtype=torch.bool, device="cuda")
        done[20] = False
        st.check(tokens=done)
        assert bool(st.q_out[20].isnan().all())


def test_values_stay_in_their_head(native_lib):
    """Infinities and NaN of one head and token reach no other row."""
    from continuous_batching_ragged_gb300 import api
    st = Step(33, 6, 3, 128, 128, seed=9)
    st.run()
    clean_q, clean_k = st.q_out.clone(), st.cache.k.clone()
    st.q[7, 2, 5] = float("nan")
    st.q[8, 0, :] = float("inf")
    st.k[9, 1, 100] = float("-inf")
    st.run()
    api.cb_check_device_errors()
    same = (st.q_out == clean_q).all(-1)
    assert not same[7, 2] and not same[8, 0] and int((~same).sum()) == 2
    same = (st.cache.k == clean_k).all(-1)
    b, o = int(st.slots[9]) // 16, int(st.slots[9]) % 16
    assert not same[b, 1, o] and int((~same).sum()) == 1


def test_zero_rows_and_eps(native_lib):
    """A row of zeros stays zero for eps > 0; tiny and huge rows keep their norm."""
    from continuous_batching_ragged_gb300 import api
    st = Step(8, 4, 4, 128, 64, seed=10)
    st.q[0] = 0
    st.k[1] = 0
    st.q[2] *= 1e-6
    st.q[3] *= 1e12
    st.run()
    api.cb_check_device_errors()
    assert not st.q_out[0].any()
    st.check()


@pytest.mark.parametrize("tokens", [0, 1, 40, 64])
def test_token_count_on_the_device(native_lib, tokens):
    """dims[1] tokens of a larger capacity; the rows behind stay as they were."""
    from continuous_batching_ragged_gb300 import api
    st = Step(64, 8, 2, 128, 128, packed=True, seed=11)
    dims = torch.tensor([3, tokens, 1, 1], dtype=torch.int32, device="cuda")
    st.run(dims=dims)
    api.cb_check_device_errors()
    done = torch.arange(64, device="cuda") < tokens
    st.check(tokens=done)
    assert bool(st.q_out[~done].isnan().all())


def test_token_count_beyond_the_capacity(native_lib):
    from continuous_batching_ragged_gb300 import api, native
    st = Step(16, 4, 4, 128, 128, seed=12)
    st.run(dims=torch.tensor([1, 17, 1, 1], dtype=torch.int32, device="cuda"))
    with pytest.raises(native.CBError, match="INVALID"):
        api.cb_check_device_errors()
    st.check(tokens=torch.zeros(16, dtype=torch.bool, device="cuda"))


def test_captured_and_on_another_stream(native_lib):
    """A captured call replays with new values in the same buffers; a call on a side stream is ordered by that stream."""
    from continuous_batching_ragged_gb300 import api
    st = Step(100, 8, 2, 128, 128, packed=True, seed=13)
    st.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    st.q.copy_(torch.randn_like(st.q))
    st.k.copy_(torch.randn_like(st.k))
    graph.replay()
    api.cb_check_device_errors()
    st.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st.q.mul_(-1.5)
        st.q_out.zero_()
        st.run(stream=side)
    side.synchronize()
    api.cb_check_device_errors(side)
    st.check()


def test_slots_past_32_bit_offsets(native_lib):
    """Slots whose element offset in the pool passes 2^31 and 2^32."""
    from continuous_batching_ragged_gb300 import api
    block, K, A = 16, 8, 128
    nb = (1 << 32) // (block * K * A) + 40
    k, v = (torch.empty((nb, K, block, A), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = Step(6, 8, K, A, A, seed=14)
    st.cache = api.KVCache(k, v)
    st.slots = torch.tensor([(nb - 1) * block + 15, nb // 2 * block + 3, 7, (nb - 30) * block, -1, nb // 2 * block + 700],
                            dtype=torch.int64, device="cuda")
    st.run()
    api.cb_check_device_errors()
    exact, mag = turned(st.k, st.wk, st.eps, st.cs, st.pos, False)
    for t, s in enumerate(st.slots.tolist()):
        if s >= 0:
            close(k[s // block, :, s % block], exact[t], mag[t])
            assert torch.equal(v[s // block, :, s % block], st.v[t])
