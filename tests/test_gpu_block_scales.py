"""8-bit caches with a scale per (block, KV head): the scatter bit for bit and
attention within its derived bound, against 64-bit numpy (needs a GB300)."""

import numpy as np
import pytest
import torch

import block_scale_reference as R
from paged_kv_cache_55_gb300 import binding as B
from paged_kv_cache_55_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Step:
    """Block-scaled caches of a step: context rows hold codes, everything unowned NaN codes and NaN scales."""

    def __init__(self, context_lens, query_lens, num_heads, num_kv_heads, head_dim, bs=16, dtype="bf16", seed=0,
                 q_scale=1.0, v_exp=(-7, -4), k_exp=(-7, -5), spread=1.0):
        rng = np.random.default_rng(seed)
        self.H, self.Hkv, self.D, self.bs, self.dtype = num_heads, num_kv_heads, head_dim, bs, dtype
        ctx, ql = np.asarray(context_lens), np.asarray(query_lens)
        self.lens = (ctx + ql).astype(np.int32)
        self.starts = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
        self.B, self.T = len(ql), int(ql.sum())
        need = -(-self.lens // bs)
        self.nb = int(need.sum()) + 3
        ids = rng.permutation(self.nb)
        self.tables = np.full((self.B, int(need.max()) + 2), -2147483648, dtype=np.int32)
        at = 0
        shape = (self.nb, bs, num_kv_heads, head_dim)
        self.kc, self.vc = np.full(shape, 0x7F, np.uint8), np.full(shape, 0x7F, np.uint8)
        self.ks = np.full((self.nb, num_kv_heads), np.nan)
        self.vs = np.full((self.nb, num_kv_heads), np.nan)
        for b in range(self.B):
            n = int(need[b])
            self.tables[b, :n] = ids[at:at + n]
            at += n
            for i in range(n):
                held = min(bs, int(ctx[b]) - i * bs)
                if held <= 0:
                    continue
                p = self.tables[b, i]
                self.ks[p] = 2.0 ** rng.integers(k_exp[0], k_exp[1] + 1, num_kv_heads)
                self.vs[p] = 2.0 ** rng.integers(v_exp[0], v_exp[1] + 1, num_kv_heads)
                for c in (self.kc, self.vc):
                    c[p, :held] = R.encode(np.clip(rng.standard_normal((held, num_kv_heads, head_dim)) * 64, -448, 448))
        dt = DT[dtype]
        rows = rng.standard_normal((self.T, 2 * num_kv_heads, head_dim))
        rows *= np.exp(spread * rng.standard_normal((self.T, 2 * num_kv_heads, 1)))
        rows = torch.from_numpy(rows).to(dt)
        self.rows = rows.cuda()
        self.key, self.value = self.rows[:, :num_kv_heads], self.rows[:, num_kv_heads:]
        self.q = (torch.from_numpy(rng.standard_normal((self.T, num_heads, head_dim))) * q_scale).to(dt).cuda()
        self.scale = float(np.float32(head_dim ** -0.5))
        self.upload()

    def upload(self):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.d_kc, self.d_vc = dev(self.kc), dev(self.vc)
        self.d_ks, self.d_vs = dev(self.ks.astype(np.float32)), dev(self.vs.astype(np.float32))
        self.d_tables, self.d_lens, self.d_starts = dev(self.tables), dev(self.lens), dev(self.starts)
        self.max_q, self.max_len = int(np.diff(self.starts).max()), int(self.lens.max())
        self.out = torch.full((self.T, self.H, self.D), float("nan"), dtype=DT[self.dtype], device="cuda")
        n = B.pa_attention_workspace_size(self.B, self.T, self.max_q, self.max_len, self.H, self.Hkv, self.D, self.bs)
        self.workspace = torch.empty(n, dtype=torch.uint8, device="cuda")

    def scatter(self, stream=None):
        B.pa_reshape_and_cache_fp8_block(self.key, self.value, self.d_kc, self.d_vc, self.d_ks, self.d_vs,
                                         self.d_tables, self.d_lens, self.d_starts, self.max_q, stream=stream)

    def attention(self, stream=None):
        B.pa_attention_varlen_fp8_block(self.q, self.d_kc, self.d_vc, self.d_ks, self.d_vs, self.d_tables, self.d_lens,
                                        self.d_starts, self.max_q, self.max_len, self.scale, self.out, self.workspace,
                                        stream=stream)

    def scatter_reference(self):
        for rows, cache, scales in ((self.key, self.kc, self.ks), (self.value, self.vc, self.vs)):
            R.block_scatter(rows.double().cpu().numpy(), cache, scales, self.tables, self.lens, self.starts, self.bs)

    def check_scatter(self):
        torch.cuda.synchronize()
        assert B.pa_debug_status() == 0
        for got, want in ((self.d_ks, self.ks), (self.d_vs, self.vs)):
            assert np.array_equal(got.cpu().numpy(), want.astype(np.float32), equal_nan=True)
        for got, want in ((self.d_kc, self.kc), (self.d_vc, self.vc)):
            g = got.cpu().numpy()
            nan = (want & 0x7F) == 0x7F
            assert np.array_equal(g[~nan], want[~nan]) and ((g[nan] & 0x7F) == 0x7F).all()

    def check_attention(self):
        torch.cuda.synchronize()
        assert B.pa_debug_status() == 0
        ref, bound = R.attention(self.q.double().cpu().numpy(), self.d_kc.cpu().numpy(), self.d_vc.cpu().numpy(),
                                 self.d_ks.double().cpu().numpy(), self.d_vs.double().cpu().numpy(), self.tables,
                                 self.lens, self.starts, self.bs, self.scale)
        got = self.out.double().cpu().numpy()
        bound = bound + R.EPS[self.dtype] * (np.abs(ref) + bound) + R.TINY[self.dtype]
        err = np.abs(got - ref)
        bad = ~(err <= bound)
        assert not bad.any(), (f"{int(bad.sum())} of {bad.size} outside the bound, worst ratio "
                               f"{float(np.nanmax(err / bound))}, first {np.argwhere(bad)[:3].tolist()}")


# ---- scatter ---------------------------------------------------------------

SCATTER = {
    "decode": dict(context_lens=[0, 6, 15, 16, 31, 100, 7], query_lens=[1] * 7, num_heads=8, num_kv_heads=2,
                   head_dim=128),
    "mixed": dict(context_lens=[0, 37, 15, 20, 64, 5, 0, 9], query_lens=[40, 2, 1, 129, 0, 7, 300, 32], num_heads=8,
                  num_kv_heads=8, head_dim=128),
    "d64_one_head": dict(context_lens=[3, 0, 30], query_lens=[5, 17, 2], num_heads=1, num_kv_heads=1, head_dim=64),
    "d80": dict(context_lens=[3, 0, 30], query_lens=[50, 17, 1], num_heads=6, num_kv_heads=3, head_dim=80),
    "d96": dict(context_lens=[13, 40], query_lens=[50, 17], num_heads=4, num_kv_heads=2, head_dim=96),
    "d256": dict(context_lens=[13, 0, 63], query_lens=[50, 17, 1], num_heads=4, num_kv_heads=2, head_dim=256),
    "many_requests": dict(context_lens=[(7 * i) % 41 for i in range(1500)], query_lens=[i % 4 for i in range(1500)],
                          num_heads=1, num_kv_heads=1, head_dim=64),
    "decode_and_idle": dict(context_lens=[4] * 70, query_lens=[i % 2 for i in range(70)], num_heads=1,
                            num_kv_heads=1, head_dim=64),
}


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("name", sorted(SCATTER))
def test_scatter_bit_for_bit(name, dtype, bs):
    s = Step(bs=bs, dtype=dtype, seed=3, **SCATTER[name])
    s.scatter()
    s.scatter_reference()
    s.check_scatter()


def test_scatter_of_special_values():
    """Zero rows, tiny and huge magnitudes, infinities and NaN: neither of the last two enters a scale."""
    s = Step([0, 5, 20, 16, 0], [16, 3, 12, 1, 16], 2, 2, 64, seed=5)
    k = s.rows
    k[0:16, 0] = 0                      # all zero: the smallest scale
    k[3, 1, 5] = float("inf")
    k[4, 1, 6] = float("-inf")
    k[5, 1, 7] = float("nan")
    k[16:19, 2] = float("nan")          # nothing finite
    k[19:31, 3] *= 2.0 ** 100
    k[19:31, 0] *= 2.0 ** -90           # below the smallest scale's codes
    k[31, 1] = 3.3e38
    k[32:48, 0, :] = 448.0              # exactly the largest code
    k[32:48, 1, :] = 450.0
    s.scatter()
    s.scatter_reference()
    s.check_scatter()


def test_appending_row_by_row_keeps_one_scale_per_block():
    """40 decode steps of three requests whose magnitudes grow and shrink: each step bit for bit."""
    s = Step([0, 3, 14], [1, 1, 1], 2, 2, 128, seed=6)
    rng = np.random.default_rng(7)
    s.tables = rng.permutation(15).reshape(3, 5).astype(np.int32)
    s.nb = 15
    s.kc, s.vc = (rng.integers(0, 0x7F, (15, 16, 2, 128)).astype(np.uint8) for _ in range(2))
    s.ks, s.vs = (2.0 ** rng.integers(-8, -3, (15, 2)).astype(np.float64) for _ in range(2))
    s.upload()
    for step in range(40):
        s.rows.copy_(torch.from_numpy(rng.standard_normal((3, 4, 128)) * np.exp(2 * rng.standard_normal((3, 4, 1)))))
        s.scatter()
        s.scatter_reference()
        s.check_scatter()
        s.lens += 1
        s.d_lens += 1


def test_a_growing_scale_keeps_nan_codes_and_a_bad_scale_counts_as_zero():
    s = Step([5, 5, 5], [1, 1, 1], 1, 1, 64, seed=8)
    p = s.tables[:, 0]
    s.kc[p[0], 2, 0, :8] = 0x7F
    s.kc[p[0], 3, 0, :8] = 0xFF
    s.ks[p[1], 0], s.vs[p[1], 0] = np.nan, np.inf
    s.ks[p[2], 0], s.vs[p[2], 0] = -1.0, 0.0
    s.rows *= 1000.0
    s.upload()
    s.scatter()
    s.scatter_reference()
    s.check_scatter()


def test_appending_under_a_scale_that_is_no_power_of_two():
    """A cache made elsewhere: its larger scale stays, new rows take E4M3(x / scale) of the fp32 quotient, old
    rows keep their codes."""
    s = Step([5, 20, 9], [3, 1, 60], 2, 2, 128, seed=28, spread=0.3)
    firsts = [int(s.tables[0, 0]), int(s.tables[1, 1]), int(s.tables[2, 0])]
    for p in firsts:
        s.ks[p], s.vs[p] = np.float32([0.7, 1.1]), np.float32([0.9, 0.3])
    s.upload()
    kc, vc = s.kc.copy(), s.vc.copy()
    s.scatter()
    torch.cuda.synchronize()
    for b, p in enumerate(firsts):
        held = int(s.lens[b] - (s.starts[b + 1] - s.starts[b])) % 16
        n = min(16 - held, int(s.starts[b + 1] - s.starts[b]))
        t0 = int(s.starts[b])
        for rows, codes, old, scales, d_scales in ((s.key, s.d_kc, kc, s.ks, s.d_ks),
                                                   (s.value, s.d_vc, vc, s.vs, s.d_vs)):
            got = codes[p].cpu().numpy()
            assert np.array_equal(d_scales[p].cpu().numpy(), scales[p].astype(np.float32))
            assert np.array_equal(got[:held], old[p, :held])
            quotient = rows[t0:t0 + n].float().cpu().numpy() / scales[p].astype(np.float32)[None, :, None]
            assert np.array_equal(got[held:held + n], R.encode(quotient.astype(np.float64)))
    assert B.pa_debug_status() == 0


def test_scatter_refuses_on_the_device_and_leaves_the_rest():
    s = Step([0, 20, 5, 9], [4, 4, 4, 4], 2, 2, 64, seed=9)
    s.tables[1, 1] = s.nb                # block id out of range
    s.lens[2] = 2                        # shorter than its query
    s.lens[3] = 1 + s.tables.shape[1] * 16
    s.upload()
    kc, ks = s.kc.copy(), s.ks.copy()
    s.scatter()
    torch.cuda.synchronize()
    assert B.pa_debug_status() == B.FLAG_BLOCK_RANGE | B.FLAG_LENGTHS
    s.lens[1:] = 0
    s.starts[1:] = 4
    R.block_scatter(s.key.double().cpu().numpy(), kc, ks, s.tables, s.lens, s.starts, 16)
    assert np.array_equal(s.d_ks.cpu().numpy(), ks.astype(np.float32), equal_nan=True)
    assert np.array_equal(s.d_kc.cpu().numpy(), kc)
    s = Step([0, 20], [4, 4], 2, 2, 64, seed=9)
    s.d_starts[2] = 7                    # does not end at the token count
    s.scatter()
    torch.cuda.synchronize()
    assert B.pa_debug_status() & B.FLAG_QUERY_LOC


def test_copy_block_scales():
    rng = np.random.default_rng(1)
    ks, vs = (rng.random((50, 5)).astype(np.float32) for _ in range(2))
    d_ks, d_vs = torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda()
    ids = rng.permutation(50)
    pairs = np.stack([ids[:20], ids[20:40]], 1).astype(np.int64)
    B.pa_copy_block_scales(d_ks, d_vs, torch.from_numpy(pairs).cuda())
    torch.cuda.synchronize()
    ks[pairs[:, 1]], vs[pairs[:, 1]] = ks[pairs[:, 0]], vs[pairs[:, 0]]
    assert np.array_equal(d_ks.cpu().numpy(), ks) and np.array_equal(d_vs.cpu().numpy(), vs)
    assert B.pa_debug_status() == 0
    B.pa_copy_block_scales(d_ks, d_vs, torch.tensor([[3, 50], [-1, 4]]).cuda())
    torch.cuda.synchronize()
    assert B.pa_debug_status() == B.FLAG_BLOCK_RANGE
    assert np.array_equal(d_ks.cpu().numpy(), ks) and np.array_equal(d_vs.cpu().numpy(), vs)


# ---- attention -------------------------------------------------------------

ATTENTION = {
    "decode_g4_d128": dict(context_lens=[0, 6, 15, 16, 511, 512, 513, 1100, 1535, 40, 3], query_lens=[1] * 11,
                           num_heads=8, num_kv_heads=2, head_dim=128),
    "decode_g8_d128_split": dict(context_lens=[4999, 700, 32], query_lens=[1] * 3, num_heads=8, num_kv_heads=1,
                                 head_dim=128),
    "decode_g1_d64": dict(context_lens=[100, 1, 900, 513], query_lens=[1] * 4, num_heads=2, num_kv_heads=2,
                          head_dim=64),
    "drafts_g2_d64": dict(context_lens=[30, 1400, 7, 50], query_lens=[4, 1, 3, 0], num_heads=4, num_kv_heads=2,
                          head_dim=64),
    "drafts_g1_d96": dict(context_lens=[0, 300, 64, 800], query_lens=[8, 1, 5, 7], num_heads=2, num_kv_heads=2,
                          head_dim=96),
    "mixed_g4_d128": dict(context_lens=[0, 37, 600, 20, 1000, 5, 0], query_lens=[40, 2, 1, 129, 1, 7, 300],
                          num_heads=8, num_kv_heads=2, head_dim=128),
    "chunks_g1_d64": dict(context_lens=[0, 700, 5], query_lens=[300, 260, 129], num_heads=2, num_kv_heads=2,
                          head_dim=64),
    "chunks_g8_d64": dict(context_lens=[10, 800, 0], query_lens=[5, 1, 24], num_heads=8, num_kv_heads=1, head_dim=64),
    "mixed_g4_d80": dict(context_lens=[0, 700, 33, 1500, 20], query_lens=[1, 1, 2, 1, 150], num_heads=4,
                         num_kv_heads=1, head_dim=80),
    "mixed_g2_d96": dict(context_lens=[1030, 3, 260, 0], query_lens=[1, 4, 1, 300], num_heads=4, num_kv_heads=2,
                         head_dim=96),
    "mixed_g4_d256": dict(context_lens=[0, 700, 33, 1500, 20], query_lens=[1, 1, 2, 1, 150], num_heads=4,
                          num_kv_heads=1, head_dim=256),
    "chunks_g1_d256": dict(context_lens=[0, 500, 900], query_lens=[300, 130, 1], num_heads=2, num_kv_heads=2,
                           head_dim=256),
    "sharp_g4_d128": dict(context_lens=[300, 900, 17], query_lens=[1, 2, 150], num_heads=8, num_kv_heads=2,
                          head_dim=128, q_scale=8.0),
    "chunks_of_many_tiles": dict(context_lens=[100, 0, 300, 40, 5, 130], query_lens=[400] * 6, num_heads=32,
                                 num_kv_heads=16, head_dim=64),
    "one_chunk_long_context": dict(context_lens=[5000], query_lens=[40], num_heads=8, num_kv_heads=2, head_dim=128),
    "one_chunk_long_context_d256": dict(context_lens=[3000], query_lens=[40], num_heads=4, num_kv_heads=1,
                                        head_dim=256),
    "chunk_whose_halves_end_apart": dict(context_lens=[100], query_lens=[700], num_heads=1, num_kv_heads=1,
                                         head_dim=64),
    "scales_far_apart": dict(context_lens=[300, 900, 17, 400], query_lens=[1, 2, 150, 200], num_heads=8,
                             num_kv_heads=2, head_dim=128, v_exp=(-20, 4), k_exp=(-12, -5)),
    "scales_far_apart_d256": dict(context_lens=[300, 17, 400], query_lens=[1, 150, 200], num_heads=4, num_kv_heads=2,
                                  head_dim=256, v_exp=(-20, 4), k_exp=(-12, -5)),
    "tiny_values": dict(context_lens=[300, 17], query_lens=[1, 150], num_heads=4, num_kv_heads=1, head_dim=64,
                        v_exp=(-64, -60), dtype_only="bf16"),
    "huge_values": dict(context_lens=[300, 17], query_lens=[1, 150], num_heads=4, num_kv_heads=1, head_dim=64,
                        v_exp=(80, 84), dtype_only="bf16"),
}


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("name", sorted(ATTENTION))
def test_attention_after_the_scatter(name, bs):
    kw = dict(ATTENTION[name])
    only = kw.pop("dtype_only", None)
    for dtype in ("bf16", "fp16"):
        if only and dtype != only:
            continue
        s = Step(bs=bs, dtype=dtype, seed=11, spread=0.3, **kw)
        s.scatter()
        s.attention()
        s.check_attention()


@pytest.mark.parametrize("q_scale", [3.0e4, 2.0e9])
def test_queries_beyond_fp16(q_scale):
    """bf16 queries that the fp16 operand cannot hold are scaled by a power of two on the way in."""
    s = Step([40, 900, 3, 700], [1, 2, 1, 150], 8, 2, 128, seed=12, q_scale=q_scale, spread=0.3)
    s.scatter()
    s.attention()
    s.check_attention()


@pytest.mark.parametrize("head_dim", [64, 80, 128, 256])
def test_some_queries_beyond_fp16(head_dim):
    """Only the rows that need it are scaled; their neighbours in the tile are not."""
    s = Step([40, 900], [150, 1], 8, 2, head_dim, seed=29, spread=0.3)
    s.q[::7, 3] *= 5.0e5
    s.q[5, 1, 11] = 3.0e5
    s.scatter()
    s.attention()
    s.check_attention()


@pytest.mark.parametrize("head_dim", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_query_rows_at_any_even_stride_and_offset(dtype, head_dim):
    """q 4-byte aligned only, its rows apart: the bits of contiguous rows."""
    s = Step([40, 900, 3], [150, 1, 2], 8, 2, head_dim, dtype=dtype, seed=30, spread=0.3)
    s.scatter()
    s.attention()
    torch.cuda.synchronize()
    want = s.out.clone()
    n = 8 * head_dim
    for offset, stride in ((2, n + 2), (8, n + 8), (0, n + 4)):
        buf = torch.full((s.T * stride + offset,), float("nan"), dtype=s.q.dtype, device="cuda")
        rows = buf[offset:].view(s.T, stride)[:, :n].view(s.T, 8, head_dim)
        rows.copy_(s.q)
        contiguous, s.q = s.q, rows
        s.out.fill_(float("nan"))
        s.attention()
        torch.cuda.synchronize()
        assert torch.equal(s.out, want)
        s.q = contiguous
    assert B.pa_debug_status() == 0


def test_any_positive_scale_is_read_exactly():
    """Scales that are no powers of two (a cache made elsewhere)."""
    s = Step([300, 900, 17], [1, 2, 150], 8, 2, 128, seed=13, spread=0.3)
    s.scatter()
    torch.cuda.synchronize()
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (s.d_ks, s.d_vs):
        t.mul_(0.6 + torch.rand(t.shape, generator=g, device="cuda"))
    s.attention()
    s.check_attention()


def test_one_scale_everywhere_agrees_with_the_per_cache_call():
    s = Step([300, 900, 17, 5], [1, 2, 150, 40], 8, 2, 128, seed=14, v_exp=(-5, -5), k_exp=(-6, -6), spread=0.0)
    s.scatter()
    s.d_ks.fill_(2.0 ** -6)
    s.d_vs.fill_(2.0 ** -5)
    s.attention()
    s.check_attention()
    out = torch.empty_like(s.out)
    B.pa_attention_varlen_fp8(s.q, s.d_kc, s.d_vc, s.d_tables, s.d_lens, s.d_starts, s.max_q, s.max_len, s.scale,
                              2.0 ** -6, 2.0 ** -5, out, s.workspace)
    torch.cuda.synchronize()
    diff = (out.float() - s.out.float()).abs()
    assert (diff <= 2.0 ** -7 * s.out.float().abs() + 2.0 ** -9).all()


@pytest.mark.parametrize("lens", [([2000, 40], [1, 1]), ([700, 40], [40, 3])])
def test_a_nan_reaches_only_its_own_rows(lens):
    """A NaN value code of a visible key, a NaN scale, or a NaN query: NaN in the rows that see it (through
    the split partials too), the other requests and KV heads untouched."""
    s = Step(*lens, 4, 2, 64, seed=26, spread=0.3)
    s.scatter()
    s.attention()
    torch.cuda.synchronize()
    clean = s.out.clone()
    s.d_vc[int(s.tables[0, 3]), 5, 1, 7] = 0x7F       # request 0, KV head 1 (query heads 2, 3), d 7
    s.q[int(s.starts[1]), 0, 0] = float("nan")        # request 1's first row, query head 0
    s.attention()
    torch.cuda.synchronize()
    n0 = int(s.starts[1])
    assert s.out[:n0, 2:, 7].isnan().all() and s.out[n0, 0].isnan().all()
    keep = torch.ones_like(s.out, dtype=torch.bool)
    keep[:n0, 2:, 7] = False
    keep[n0, 0] = False
    assert torch.equal(s.out[keep], clean[keep])


def test_one_long_request():
    s = Step([70000], [1], 8, 1, 128, seed=15, spread=0.3)
    s.scatter()
    s.attention()
    s.check_attention()


@pytest.mark.parametrize("lens", [[1], [1, 1, 1], [8], [9], [16, 17], [128], [129], [255], [256, 257]])
def test_first_steps_of_new_requests(lens):
    """No context: the whole request is this step's rows, at lengths around the tile edges."""
    for bs in (8, 16, 32):
        s = Step([0] * len(lens), lens, 4, 1, 128, bs=bs, seed=16, spread=0.3)
        s.scatter()
        s.attention()
        s.scatter_reference()
        s.check_scatter()
        s.check_attention()


def test_many_requests_use_the_two_pass_planner():
    n = 1300
    s = Step([(5 * i) % 60 for i in range(n)], [1 + (i % 97 == 0) * 20 for i in range(n)], 4, 1, 64, seed=17,
             spread=0.3)
    s.scatter()
    s.attention()
    s.check_attention()


def test_repeated_and_permuted_steps_give_the_same_bits():
    s = Step([300, 900, 17, 2000], [1, 2, 150, 1], 8, 2, 128, seed=18, spread=0.3)
    s.scatter()
    s.attention()
    torch.cuda.synchronize()
    first = s.out.clone()
    for _ in range(5):
        s.out.fill_(float("nan"))
        s.attention()
        torch.cuda.synchronize()
        assert torch.equal(s.out, first)


def test_bad_block_ids_are_flagged():
    s = Step([300, 40], [1, 100], 8, 2, 128, seed=19, spread=0.3)
    s.scatter()
    torch.cuda.synchronize()
    s.d_tables[0, 3] = -5
    s.d_tables[1, 2] = s.nb
    s.attention()
    torch.cuda.synchronize()
    assert B.pa_debug_status() & B.FLAG_BLOCK_RANGE


# ---- a layer's step --------------------------------------------------------

def layer_step(s, qkv, weights, table, positions, q_out, key_out):
    q, key = qkv[:, :s.H], qkv[:, s.H:s.H + s.Hkv]
    B.pa_norm_rope(q, key, weights[0], weights[1], 1e-6, positions, table, q_out, key_out)
    B.pa_reshape_and_cache_fp8_block(key_out, qkv[:, s.H + s.Hkv:], s.d_kc, s.d_vc, s.d_ks, s.d_vs, s.d_tables,
                                     s.d_lens, s.d_starts, s.max_q)
    B.pa_attention_varlen_fp8_block(q_out, s.d_kc, s.d_vc, s.d_ks, s.d_vs, s.d_tables, s.d_lens, s.d_starts, s.max_q,
                                    s.max_len, s.scale, s.out, s.workspace)


@pytest.mark.parametrize("captured", [False, True])
def test_norm_scatter_attention_as_one_step(captured):
    s = Step([0, 37, 600, 20, 1000, 0], [40, 1, 1, 129, 1, 0], 8, 2, 128, seed=20)
    rng = np.random.default_rng(21)
    dt = torch.bfloat16
    qkv = torch.empty(s.T, 12, 128, dtype=dt, device="cuda")
    w = [torch.from_numpy(1 + 0.2 * rng.standard_normal(128)).to(dt).cuda() for _ in range(2)]
    table = torch.from_numpy(W.rope_cos_sin_cache(1100, 128)).cuda()
    pos = np.concatenate([np.arange(L - n, L) for L, n in zip(s.lens, np.diff(s.starts))]).astype(np.int64)
    positions = torch.from_numpy(pos).cuda()
    q_out, key_out = torch.empty(s.T, 8, 128, dtype=dt, device="cuda"), torch.empty(s.T, 2, 128, dtype=dt, device="cuda")
    args = (s, qkv, w, table, positions, q_out, key_out)
    if captured:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            qkv.normal_()
            layer_step(*args)
        side.synchronize()
        s.upload()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer_step(*args)
    kc0, vc0, ks0, vs0 = s.kc.copy(), s.vc.copy(), s.ks.copy(), s.vs.copy()
    for _ in range(2):
        s.kc, s.vc, s.ks, s.vs = kc0.copy(), vc0.copy(), ks0.copy(), vs0.copy()
        for d, h in ((s.d_kc, s.kc), (s.d_vc, s.vc), (s.d_ks, s.ks.astype(np.float32)),
                     (s.d_vs, s.vs.astype(np.float32))):
            d.copy_(torch.from_numpy(h))
        qkv.copy_(torch.from_numpy(rng.standard_normal(qkv.shape) * 3))
        s.out.fill_(float("nan"))
        if captured:
            g.replay()
        else:
            layer_step(*args)
        torch.cuda.synchronize()
        for x, got, wt in ((qkv[:, :8], q_out, w[0]), (qkv[:, 8:10], key_out, w[1])):
            ref, mag = R.norm_rope(x.double().cpu().numpy(), wt.double().cpu().numpy(), 1e-6, pos,
                                   table.cpu().numpy(), 128, True)
            assert (np.abs(got.double().cpu().numpy() - ref) <= R.norm_rope_bound(ref, mag, "bf16")).all()
        s.key, s.value, s.q = key_out, qkv[:, 10:], q_out
        s.scatter_reference()
        s.check_scatter()
        s.check_attention()


def test_two_steps_on_two_streams_with_their_own_workspaces():
    a = Step([300, 900], [1, 60], 8, 2, 128, seed=22, spread=0.3)
    b = Step([700, 20, 5], [1, 1, 90], 8, 2, 128, seed=23, spread=0.3)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, st in zip((a, b), streams):
            s.scatter(stream=st)
            s.attention(stream=st)
    torch.cuda.synchronize()
    a.check_attention()
    b.check_attention()


def test_copy_on_write_of_a_shared_block():
    """A block copied with its scales serves a second request that then grows it."""
    s = Step([20, 20], [1, 1], 4, 1, 64, seed=24)
    src, dst = int(s.tables[0, 1]), int(s.tables[1, 1])
    s.upload()
    pairs = torch.tensor([[src, dst], [int(s.tables[0, 0]), int(s.tables[1, 0])]]).cuda()
    B.pa_copy_blocks(s.d_kc, s.d_vc, pairs)
    B.pa_copy_block_scales(s.d_ks, s.d_vs, pairs)
    for a, c in pairs.cpu().tolist():
        for x in (s.kc, s.vc, s.ks, s.vs):
            x[c] = x[a]
    s.rows[1] *= 50.0
    s.scatter()
    s.attention()
    s.scatter_reference()
    s.check_scatter()
    s.check_attention()
