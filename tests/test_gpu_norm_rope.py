"""Norm and rotation of q and K heads with the cache write, against 64-bit numpy (needs a GB300)."""

import numpy as np
import pytest
import torch

import block_scale_reference as R
from paged_kv_cache_55_gb300 import binding as B
from paged_kv_cache_55_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
MAX_POSITION = 300


class Case:
    def __init__(self, T, H, Hkv, D, rot, dtype, cache, bs=16, seed=0, scale=2.0, pad=True):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.Hkv, self.D, self.rot, self.dtype, self.cache = T, H, Hkv, D, rot, dtype, cache
        dt = DT[dtype]
        qkv = torch.from_numpy(rng.standard_normal((T, H + 2 * Hkv, D)) * scale).to(dt).cuda()
        self.q, self.key, self.value = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        self.qw = torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).to(dt).cuda()
        self.kw = torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).to(dt).cuda()
        self.table = torch.from_numpy(W.rope_cos_sin_cache(MAX_POSITION, rot)).cuda()
        self.positions = torch.from_numpy(rng.integers(0, MAX_POSITION, T)).cuda()
        self.nb, self.bs = (T + bs - 1) // bs + 2, bs
        slots = rng.permutation(self.nb * bs)[:T].astype(np.int64)
        if pad and T > 3:
            slots[rng.permutation(T)[:max(1, T // 7)]] = -1
        self.slots = torch.from_numpy(slots).cuda()
        self.q_out = torch.full((T, H, D), float("nan"), dtype=dt, device="cuda")
        if cache == "rows":
            self.key_out = torch.full((T, Hkv, D), float("nan"), dtype=dt, device="cuda")
        elif cache == "16":
            self.kc0 = torch.from_numpy(rng.standard_normal((self.nb, bs, Hkv, D))).to(dt).cuda()
            self.vc0 = torch.from_numpy(rng.standard_normal((self.nb, bs, Hkv, D))).to(dt).cuda()
        else:
            self.k_scale, self.v_scale = 0.03, 0.021
            self.kc0 = torch.from_numpy(rng.integers(0, 256, (self.nb, bs, Hkv, D)).astype(np.uint8)).cuda()
            self.vc0 = torch.from_numpy(rng.integers(0, 256, (self.nb, bs, Hkv, D)).astype(np.uint8)).cuda()
        if cache != "rows":
            self.kc, self.vc = self.kc0.clone(), self.vc0.clone()

    def run(self, neox=True, qw="own", kw="own", q_out=None, stream=None):
        qw, kw = (self.qw if qw == "own" else qw), (self.kw if kw == "own" else kw)
        q_out = self.q_out if q_out is None else q_out
        if self.cache == "rows":
            B.pa_norm_rope(self.q, self.key, qw, kw, EPS, self.positions, self.table, q_out, self.key_out,
                           is_neox=neox, stream=stream)
        elif self.cache == "16":
            B.pa_norm_rope_reshape_and_cache(self.q, self.key, self.value, qw, kw, EPS, self.kc, self.vc, self.slots,
                                             self.positions, self.table, q_out, is_neox=neox, stream=stream)
        else:
            B.pa_norm_rope_reshape_and_cache_fp8(self.q, self.key, self.value, qw, kw, EPS, self.kc, self.vc,
                                                 self.slots, self.positions, self.table, self.k_scale, self.v_scale,
                                                 q_out, is_neox=neox, stream=stream)

    def check(self, neox=True, qw="own", kw="own"):
        qw, kw = (self.qw if qw == "own" else qw), (self.kw if kw == "own" else kw)
        pos, table = self.positions.cpu().numpy(), self.table.cpu().numpy()
        f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        refs = [R.norm_rope(f64(x), None if w is None else f64(w), EPS, pos, table, self.rot, neox)
                for x, w in ((self.q, qw), (self.key, kw))]
        assert_within(f64(self.q_out), refs[0][0], R.norm_rope_bound(*refs[0], self.dtype), "q_out")
        kref, kmag = refs[1]
        if self.cache == "rows":
            assert_within(f64(self.key_out), kref, R.norm_rope_bound(kref, kmag, self.dtype), "key_out")
            return
        slots = self.slots.cpu().numpy()
        live = slots >= 0
        rows = lambda c: c.reshape(self.nb * self.bs, self.Hkv, self.D).cpu()  # noqa: E731
        kc, vc, kc0, vc0 = rows(self.kc), rows(self.vc), rows(self.kc0), rows(self.vc0)
        rest = np.setdiff1d(np.arange(self.nb * self.bs), slots[live])
        assert torch.equal(bits(kc[rest]), bits(kc0[rest])) and torch.equal(bits(vc[rest]), bits(vc0[rest]))
        if self.cache == "16":
            assert torch.equal(bits(vc[slots[live]]), bits(self.value.cpu()[live]))
            assert_within(f64(kc[slots[live]]), kref[live], R.norm_rope_bound(kref, kmag, self.dtype)[live], "K")
            return
        quotient = self.value.float().cpu().numpy()[live] / np.float32(self.v_scale)
        assert np.array_equal(vc.numpy()[slots[live]], R.encode(quotient))
        got = R.decode(kc.numpy()[slots[live]]) * self.k_scale
        ref = kref[live]
        sat = np.clip(ref, -448 * self.k_scale, 448 * self.k_scale)
        row = R.norm_rope_bound(kref, kmag, self.dtype)[live]
        # then one rounding to a code: half a step 2^-4 of the value, 2^-10 of the scale among the subnormals
        assert_within(got, sat, row * (1 + 2.0 ** -4) + 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * self.k_scale, "K codes")


def bits(t):
    return t.contiguous().view(torch.uint8)


def assert_within(got, ref, bound, what):
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside the bound, worst ratio "
                           f"{float(np.nanmax(err / bound))}, first {np.argwhere(bad)[:3].tolist()}")


SHAPES = [  # (T, H, Hkv, D, rotary_dim, bs)
    (1, 32, 8, 128, 128, 16),
    (5, 4, 1, 64, 64, 8),
    (37, 16, 4, 96, 64, 16),
    (300, 8, 8, 80, 80, 32),
    (11, 6, 3, 256, 16, 16),
    (700, 32, 8, 128, 64, 16),
    (3, 2, 1, 16, 16, 16),
    (9, 5, 5, 512, 512, 16),
    (2, 1, 1, 48, 32, 8),
]


@pytest.mark.parametrize("cache", ["rows", "16", "8"])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_matches_the_definition(shape, dtype, neox, cache):
    T, H, Hkv, D, rot, bs = shape
    c = Case(T, H, Hkv, D, rot, dtype, cache, bs=bs, seed=T)
    c.run(neox)
    torch.cuda.synchronize()
    assert B.pa_debug_status() == 0
    c.check(neox)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rows_of_eight_element_multiples(dtype):
    """head_dim 24 and 40: an odd number of 16-byte chunks (rows and 16-bit caches only)."""
    for D, rot in ((24, 16), (40, 32), (40, 16), (8 * 63, 16)):
        for cache in ("rows", "16"):
            for neox in (True, False):
                c = Case(6, 3, 2, D, rot, dtype, cache, seed=D)
                c.run(neox)
                torch.cuda.synchronize()
                c.check(neox)


@pytest.mark.parametrize("cache", ["rows", "16", "8"])
def test_without_weights_it_is_the_rotation(cache):
    """No norm on one side or both; both None must agree with pa_rope_reshape_and_cache bit for bit."""
    c = Case(50, 8, 2, 128, 64, "bf16", cache, seed=4)
    for qw, kw in ((None, "own"), ("own", None), (None, None)):
        c.run(True, qw, kw)
        torch.cuda.synchronize()
        c.check(True, qw, kw)
    if cache == "16":
        q, kc, vc = c.q.clone(), c.kc0.clone(), c.vc0.clone()
        B.pa_rope_reshape_and_cache(q, c.key, c.value, kc, vc, c.slots, c.positions, c.table)
        torch.cuda.synchronize()
        assert torch.equal(q, c.q_out) and torch.equal(kc, c.kc) and torch.equal(vc, c.vc)


@pytest.mark.parametrize("neox", [True, False])
def test_in_place_equals_out_of_place(neox):
    c = Case(200, 8, 2, 128, 96, "bf16", "rows", seed=6)
    c.run(neox)
    q, key = c.q, c.key  # slices of one fused buffer
    want_q, want_k = c.q_out.clone(), c.key_out.clone()
    B.pa_norm_rope(q, key, c.qw, c.kw, EPS, c.positions, c.table, q, key, is_neox=neox)
    torch.cuda.synchronize()
    assert torch.equal(q, want_q) and torch.equal(key, want_k)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_zero_tiny_and_huge_rows(dtype):
    """A zero row, rows whose squares underflow, and (bf16) rows whose squares overflow fp32."""
    c = Case(8, 4, 2, 128, 128, dtype, "rows", seed=7)
    c.q[0] = 0
    c.q[1] *= 2.0 ** -20
    if dtype == "bf16":
        c.q[2] *= 2.0 ** 100
        c.key[3] *= 2.0 ** 64
        c.q[4] *= 2.0 ** -100
        c.q[5, 0, 5] = 3.0e38
    else:
        c.q[2] *= 2.0 ** 12
    c.run()
    torch.cuda.synchronize()
    assert torch.isfinite(c.q_out.float()).all() and torch.isfinite(c.key_out.float()).all()
    c.check()


def test_nonfinite_heads_stay_apart():
    c = Case(4, 4, 2, 128, 128, "bf16", "rows", seed=8)
    c.run()
    clean_q, clean_k = c.q_out.clone(), c.key_out.clone()
    c.q[1, 2, 7] = float("nan")
    c.key[2, 0, 3] = float("inf")
    c.run()
    torch.cuda.synchronize()
    same_q, same_k = torch.ones(4, 4, dtype=torch.bool), torch.ones(4, 2, dtype=torch.bool)
    same_q[1, 2] = same_k[2, 0] = False
    assert torch.equal(c.q_out[same_q.cuda()], clean_q[same_q.cuda()])
    assert torch.equal(c.key_out[same_k.cuda()], clean_k[same_k.cuda()])
    assert c.q_out[1, 2].isnan().all()
    assert c.key_out[2, 0, 3].isnan() and c.key_out[2, 0, 67].isnan()  # inf / inf and its rotation partner
    others = [i for i in range(128) if i not in (3, 67)]
    assert (c.key_out[2, 0, others] == 0).all()


def test_out_of_range_positions_and_slots():
    c = Case(6, 4, 2, 64, 64, "bf16", "16", seed=9, pad=False)
    before = c.q_out.clone()
    c.positions[1], c.positions[2] = -1, MAX_POSITION
    c.slots[3] = c.nb * c.bs
    c.run()
    torch.cuda.synchronize()
    assert B.pa_debug_status() == B.FLAG_POSITION_RANGE | B.FLAG_SLOT_RANGE
    assert torch.equal(bits(c.q_out[1:3]), bits(before[1:3]))       # skipped tokens: nothing written
    rows, rows0 = c.kc.view(-1, 2, 64), c.kc0.view(-1, 2, 64)
    assert torch.equal(rows[c.slots[1:3]], rows0[c.slots[1:3]])
    assert torch.isfinite(c.q_out[[0, 3, 4, 5]].float()).all()      # a bad slot still rotates q
    untouched = torch.ones(c.nb * c.bs, dtype=torch.bool, device="cuda")
    untouched[c.slots[[0, 4, 5]]] = False
    assert torch.equal(rows[untouched], rows0[untouched])


def test_no_tokens_and_single_tokens_of_a_wide_buffer():
    c = Case(4, 4, 2, 64, 64, "bf16", "16", seed=10)
    n = B.pa_launch_count()
    B.pa_norm_rope_reshape_and_cache(c.q[:0], c.key[:0], c.value[:0], c.qw, c.kw, EPS, c.kc, c.vc, c.slots[:0],
                                     c.positions[:0], c.table, c.q_out[:0])
    assert B.pa_launch_count() == n
    c.run()
    want = c.q_out.clone()
    c.q_out.zero_()
    for t in range(4):
        B.pa_norm_rope_reshape_and_cache(c.q[t:t + 1], c.key[t:t + 1], c.value[t:t + 1], c.qw, c.kw, EPS, c.kc, c.vc,
                                         c.slots[t:t + 1], c.positions[t:t + 1], c.table, c.q_out[t:t + 1])
    torch.cuda.synchronize()
    assert torch.equal(c.q_out, want)


def test_captured_and_on_another_stream():
    c = Case(64, 8, 2, 128, 128, "bf16", "16", seed=11)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    side.synchronize()
    c.check()
    c.q_out.zero_()
    c.run(stream=side)
    side.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    c.q.mul_(-1.5)
    c.kc.copy_(c.kc0)
    g.replay()
    torch.cuda.synchronize()
    c.check()


def test_many_tokens_take_every_warp_through_several_tokens():
    c = Case(9000, 4, 1, 64, 64, "bf16", "16", seed=12)
    c.run()
    torch.cuda.synchronize()
    c.check()
