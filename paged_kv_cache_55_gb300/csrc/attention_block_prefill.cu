// Chunked-prefill attention over 8-bit caches with a scale per (block, KV
// head), on the 5th-generation tensor cores (tcgen05 + TMEM).
//
// The pipeline of attention_prefill_tc.cu over 8-bit caches (one CTA per SM; a
// producer, an MMA, two converter and sixteen softmax warps handing K/V ranges
// of 128 keys over through mbarriers; tiles of two 128-row halves), with two
// things of its own:
//   * block scales. With ks_j, vs_j the scales of key j's block, the softmax
//     takes P'_j = 2^(s_j ks_j scale log2 e + log2 vs_j - m) against the running
//     maximum m of those exponents, so P' carries the V scale into O = sum P'_j
//     code_j and stays an fp16 value whatever the scales are, and the row sum
//     takes P'_j / vs_j, the plain weight. The producer stages a range's
//     scales (K factor, log2 and inverse of V's) per group of GRP keys that
//     share a block: 16, or 8 for 8-token blocks. A group costs a few
//     operations, a key none;
//   * parts. The planner splits tiles over their keys when there are too few
//     to fill the SMs; a part writes its rows' normalised fp32 outputs and
//     log2-sum-exps to a slot, and the merge kernel joins them.
// Bound by the chain of a half: the tensor core takes 1000 cycles for P V of a
// range and S of the next, the softmax 3000 to 4000 (two TMEM reads, the
// maxima's exchange, 64 exponents a thread), and P lies over S, so neither runs
// under the other of its own half; with two halves the tensor core is 41 % busy.
// Measured (a step of 16 chunks of 512 and 48 decode requests over 8-bit
// caches, 188 GFLOP): 241 us, of which the tiles 214 under a counter. What
// brought it there, in turn: Q loaded along rows and not a lane per row (325 ->
// 280), q sent towards L2 by the producer (275), MMAs issued by an elected
// thread with broadcast descriptors (263), no masks where all keys are visible
// (241).
// Tried and not kept: P handed over in two halves (2 % slower: the issuing
// thread then waits inside a product while the other half is ready), the next
// tile's record read before the last range (3 % slower, registers), ring
// slots counted instead of divided, one arrival per warp at the exchange, and
// the loop over P unrolled in full (no difference).
#include <type_traits>

#include "attention_tile.cuh"

namespace pa {

namespace {

// Block scales of a range in shared memory: groups of GRP keys in 128 bytes.
// 16-key groups: (K scale times the softmax scale, log2 V scale, 1 / V scale, -);
// 8-key groups: the first two.
constexpr int kScaleSlotBytes = 128;

// Scale slots and their barriers behind a layout's other parts; `Slots` of
// them, taken in turn.
template <typename Base, int Slots>
struct WithScales : Base {
  static constexpr int SCALE_SLOTS = Slots;
  static constexpr int SC_BAR_OFF = (Base::BYTES + 15) / 16 * 16;
  static constexpr int SC_OFF = SC_BAR_OFF + (8 * Slots + 15) / 16 * 16;
  static constexpr int BYTES = SC_OFF + Slots * kScaleSlotBytes;
  // more than half an SM's, so that a second CTA (which would wait for TMEM)
  // never lands on the same SM
  static constexpr int REQUEST = BYTES > 116 * 1024 ? BYTES : 116 * 1024;
};
// The producer writes range g's scales once the ring slot of K(g) is free,
// that is, once load 2 g - SLOTS has been used up: V of range g - (SLOTS + 1) / 2
// (odd SLOTS; its P is written) or K of range g - SLOTS / 2 (even; S of a range
// is issued only after both halves' P of the range before it). So the softmax
// warps have finished with range g - (SLOTS / 2 + 1).
template <int D>
using BlockLayout = WithScales<TcLayout<D>, TcLayout<D>::SLOTS / 2 + 1>;
static_assert(BlockLayout<128>::BYTES <= 227 * 1024, "shared memory of one CTA");

// Block scales of 16 keys: (K factor, log2 V scale, 1 / V scale, -) of a
// 16-key group, or (K factor, log2 V scale) of two 8-key groups.
__device__ __forceinline__ float4 ld_scales(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// One thread of the converged warp, the same every time. With the operands
// broadcast, the compiler keeps an MMA's descriptors in uniform registers
// instead of moving each there from a thread's.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n .reg .b32 l;\n elect.sync l|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Row maximum of 32 scores under block scales (at shared address sc): s *
// (rowf * kf) + lv per group, as separately rounded operations. kf and rowf are
// positive, so a group's largest raw score gives its largest scaled one.
template <int GRP, bool MASK>
__device__ __forceinline__ float scaled_max32(const uint32_t (&s)[32], int ck0, int lim, float rowf, uint32_t sc) {
  float m = -INFINITY;
  float4 v;
#pragma unroll
  for (int g = 0; g < 32 / GRP; ++g) {
    constexpr int PER16 = 16 / GRP;  // groups per 16 keys
    if (g % PER16 == 0) v = ld_scales(sc + 16 * (g / PER16));
    const float kf = g % PER16 == 0 ? v.x : v.z, lv = g % PER16 == 0 ? v.y : v.w;
    float t;
    if (!MASK || ck0 + 32 <= lim) {
      t = max3(__uint_as_float(s[GRP * g]), __uint_as_float(s[GRP * g + 1]), __uint_as_float(s[GRP * g + 2]));
      float u = max3(__uint_as_float(s[GRP * g + 3]), __uint_as_float(s[GRP * g + 4]), __uint_as_float(s[GRP * g + 5]));
#pragma unroll
      for (int i = 6; i < GRP; i += 4) {
        t = max3(t, __uint_as_float(s[GRP * g + i]), __uint_as_float(s[GRP * g + i + 1]));
        if (i + 3 < GRP) u = max3(u, __uint_as_float(s[GRP * g + i + 2]), __uint_as_float(s[GRP * g + i + 3]));
      }
      t = fmaxf(t, u);
    } else {
      t = -INFINITY;
#pragma unroll
      for (int i = 0; i < GRP; ++i) t = ck0 + GRP * g + i < lim ? fmaxf(t, __uint_as_float(s[GRP * g + i])) : t;
    }
    m = fmaxf(m, __fadd_rn(__fmul_rn(t, __fmul_rn(rowf, kf)), lv));
  }
  return m;
}

// P for the 16 keys of one UMMA K step under block scales `c` (scores s[0..16), key
// k0 + i visible while k0 + i < lim), one fp16 value per key, summed into *sum and
// stored at TMEM column `col` of this thread's lane (8 columns):
// P' = 2^(s * kf + lv - ms) carries the V scale 2^lv, so O accumulates P' times
// codes; the row sum takes P' / 2^lv. RARE: the row's factor (1 otherwise),
// every operation rounded by itself, and the mask; without it all 16 keys are
// visible (or the row is none of the tile's and is never stored).
template <int GRP, bool RARE>
__device__ __forceinline__ void probs16_scaled_store(const uint32_t *s, int k0, int lim, float rowf, float ms,
                                                     float &sum, uint32_t col, const float4 &c) {
  uint32_t hv[8];
#pragma unroll
  for (int g = 0; g < 16 / GRP; ++g) {
    const float kf = g == 0 ? c.x : c.z, lv = g == 0 ? c.y : c.w;
    const float f = RARE ? __fmul_rn(rowf, kf) : kf, add = lv - ms;
    float acc0 = 0.f, acc1 = 0.f;
#pragma unroll
    for (int j = 0; j < GRP / 2; ++j) {
      const int i = GRP / 2 * g + j;
      float x0 = __uint_as_float(s[2 * i]), x1 = __uint_as_float(s[2 * i + 1]);
      if (RARE) {
        x0 = k0 + 2 * i < lim ? x0 : -INFINITY;
        x1 = k0 + 2 * i + 1 < lim ? x1 : -INFINITY;
      }
      float e0, e1;
      if (RARE) {
        e0 = __fsub_rn(__fadd_rn(__fmul_rn(x0, f), lv), ms);
        e1 = __fsub_rn(__fadd_rn(__fmul_rn(x1, f), lv), ms);
      } else {
        fma2(e0, e1, x0, x1, f, f, add, add);
      }
      const float p0 = ex2_approx(e0), p1 = ex2_approx(e1);
      add2(acc0, acc1, acc0, acc1, p0, p1);
      hv[i] = ElemFp16::pack(p0, p1);
    }
    sum = fmaf(acc0 + acc1, GRP == 16 ? c.z : ex2_approx(-lv), sum);
  }
  tmem_st8u(col, hv);
}

// A published unit, or the end of the stream: a tile of one request and one KV
// head, or a part of its keys (kv_begin a multiple of 128) whose rows go to
// partial slot `slot` (-1: the output).
struct TileUnit {
  int b, row0, npos, pos0, kv_end, kvh, stop, kv_begin, slot;
};

// The key range of a unit with block scales: a whole tile's keys, or a part of
// them with a partial slot that exists.
__device__ __forceinline__ bool part_sane(const TileUnit &r, const BlockTileParams &p, int item) {
  if (r.kv_begin < 0 || r.kv_begin % kKeyTile != 0 || r.kv_begin >= r.kv_end || r.kv_end > r.pos0 + r.npos) return false;
  return r.slot < 0 ? r.kv_begin == 0 && r.kv_end == r.pos0 + r.npos : item < p.max_part_items;
}

// Block scales of the group that starts at `key` (this KV head); left as
// they are past the last key or for a block id out of range. p.k_scales and
// p.v_scales may have been written shortly before: not an invariant load.
__device__ __forceinline__ void block_scales_of(const BlockTileParams &p, const int32_t *table, int key, int kv_end, int kvh,
                                                float &ks, float &vs) {
  if (key >= kv_end) return;
  const int phys = __ldg(table + (key >> p.block_shift));
  if (phys < 0 || phys >= p.num_blocks) return;
  const int64_t at = static_cast<int64_t>(phys) * p.num_kv_heads + kvh;
  ks = ld_cg(p.k_scales + at);
  vs = ld_cg(p.v_scales + at);
}
template <int GRP>
__device__ __forceinline__ void st_scales(uint32_t slot, int group, float kf, float vs) {
  const float lv = __log2f(vs);
  if (GRP == 16)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %3};\n" ::"r"(slot + 16 * group), "f"(kf), "f"(lv),
                 "f"(__fdividef(1.f, vs))
                 : "memory");
  else
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};\n" ::"r"(slot + 8 * group), "f"(kf), "f"(lv) : "memory");
}

// Sixteen rows of a unit's Q, row0 .. row0 + 15 of the tile (or half) whose
// first position is `pos_base` of the unit (row r = (position, head), K-major),
// to shared memory as fp16 or as they are, chunk c of a row at at(row, c).
// Consecutive lanes take consecutive 16-byte chunks. Returns (lanes 0..15) the
// softmax factor of row row0 + lane: 2^e, e > 0 for a scaled bf16 row. Measured
// (16 chunks of 512, 6.7 tiles a CTA): a lane per row instead, 32 lines an
// instruction, cost 36000 cycles between two tiles; at head_dim 256 (8 chunks of
// 600, 16 / 4 heads) the step took 223 us against 199.
template <int D, int G, typename E, typename At>
__device__ __forceinline__ float load_q_rows(const BlockTileParams &p, const TileUnit &u, int pos_base, int row0,
                                             int lane, At at) {
  constexpr bool kBf16 = std::is_same<E, ElemBf16>::value;
  constexpr int CPR = D / 8, NL = 16 * CPR / 32;  // chunks per row, and per lane
  auto valid = [&](int row) { return pos_base + row / G < u.npos; };
  auto q_row = [&](int row) {
    return p.q + static_cast<int64_t>(u.row0 + pos_base + row / G) * p.q_stride +
           static_cast<int64_t>(u.kvh * G + row % G) * D;
  };
  auto put = [&](int row, int c, uint4 w, float qmul) {
    if constexpr (kBf16) {
      w = make_uint4(ElemFp16::pack(ElemBf16::lo(w.x) * qmul, ElemBf16::hi(w.x) * qmul),
                     ElemFp16::pack(ElemBf16::lo(w.y) * qmul, ElemBf16::hi(w.y) * qmul),
                     ElemFp16::pack(ElemBf16::lo(w.z) * qmul, ElemBf16::hi(w.z) * qmul),
                     ElemFp16::pack(ElemBf16::lo(w.w) * qmul, ElemBf16::hi(w.w) * qmul));
    }
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(at(row, c)), "r"(w.x), "r"(w.y), "r"(w.z),
                 "r"(w.w)
                 : "memory");
  };
  // q is only required to be 4-byte aligned: 16-byte loads when rows allow them
  const bool q16 = (reinterpret_cast<uintptr_t>(p.q) & 15u) == 0 && (p.q_stride & 7) == 0;
  uint4 w[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int row = row0 + (32 * i + lane) / CPR, c = (32 * i + lane) % CPR;
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (q16 && valid(row)) w[i] = __ldg(reinterpret_cast<const uint4 *>(q_row(row)) + c);
  }
  bool rare = !q16;  // or an element of magnitude 2^15 or more (or NaN) that fp16 may not hold
  if constexpr (kBf16) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      m = __vimax3_u16x2(m, w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu);
      m = __vimax3_u16x2(m, w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu);
    }
    rare = rare || __any_sync(0xffffffffu, max(m & 0xffffu, m >> 16) >= 0x4700u);  // bf16 2^15
  }
  float rowf = 1.f;
  if (!rare) {
#pragma unroll
    for (int i = 0; i < NL; ++i) put(row0 + (32 * i + lane) / CPR, (32 * i + lane) % CPR, w[i], 1.f);
  } else if (lane < 16) {  // a lane per row
    const int row = row0 + lane;
    auto ldq = [&](int c) {
      if (!valid(row)) return make_uint4(0u, 0u, 0u, 0u);
      const uint32_t *q32 = reinterpret_cast<const uint32_t *>(q_row(row)) + 4 * c;
      return make_uint4(__ldg(q32), __ldg(q32 + 1), __ldg(q32 + 2), __ldg(q32 + 3));
    };
    float qmul = 1.f;
    if constexpr (kBf16) {
      // 2^-e, e > 0 only when the row's largest |q| reaches 2^15
      float amax = 0.f;
#pragma unroll 1
      for (int c = 0; c < CPR; ++c) {
        const uint4 x = ldq(c);
        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          amax = fmaxf(amax, fmaxf(fabsf(ElemBf16::lo(v[k])), fabsf(ElemBf16::hi(v[k]))));
      }
      const int ex = static_cast<int>((__float_as_uint(amax) >> 23) & 0xffu) - 127;  // floor(log2(amax))
      const int e = ex >= 15 ? min(ex - 14, 120) : 0;
      qmul = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      rowf = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    }
#pragma unroll 1
    for (int c = 0; c < CPR; ++c) put(row, c, ldq(c), qmul);
  }
  return rowf;
}

template <int D, int G, typename E, int GRP>
// Twenty warps, one CTA per SM.
__global__ void __launch_bounds__(kTileThreads8, 1)
    block_tile_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const BlockTileParams p) {
  using Lay = BlockLayout<D>;
  using Tm = TcTmem<D>;
  constexpr int RAW_ROW = D <= 64 ? 64 : 128;      // bytes per staged row of codes (padded past head_dim)
  constexpr int RAW_BYTES = kKeyTile * RAW_ROW;    // 8-bit codes of one range
  constexpr uint32_t RAW_OFF = Lay::KV_BYTES / 2;  // staged in the back half of the slot
  static_assert(RAW_BYTES == Lay::KV_BYTES / 2, "a range's codes fill half of its 16-bit slot");
  constexpr int KSTEPS_S = D / 16;         // UMMA K steps of S = Q K^T
  constexpr int KSTEPS_O = kKeyTile / 16;  // UMMA K steps of O = P V
  constexpr int POS_PER_HALF = kHalfRows / G;
  constexpr int PART_KEYS = kKeyTile / kParts;  // keys of a range per softmax warp
  constexpr int NCH = (D + 31) / 32;            // 32-column chunks of O (head_dim 80: 16 padding columns)
  constexpr uint32_t IDESC_S = f16_idesc(kHalfRows, kKeyTile, 0, ElemFp16::kUmmaFormat);
  constexpr uint32_t IDESC_O = f16_idesc(kHalfRows, D, 1, ElemFp16::kUmmaFormat);
  // O stays in TMEM and is rescaled only when a row's running maximum grows
  // by more than 2^8 (log2 domain); in between, probabilities are taken
  // against the older maximum and stay below 256.
  constexpr float kRescaleLog2 = 8.f;
  constexpr unsigned FULL = 0xffffffffu;

  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = smem_u32(smem_raw);
  if (base & 1023u) {  // the swizzled tiles need 1024-byte alignment; never touch misaligned tiles
    if (tid == 0) flag_error(p.status, PA_FLAG_LENGTHS);
    griddep_wait();  // completion still implies the decode kernel's
    return;
  }
  constexpr int SLOTS = Lay::SLOTS;
  const uint32_t sQ0 = base + Lay::Q_OFF, sRing = base + Lay::RING_OFF;
  auto bar = [&](int i) { return base + Lay::BAR_OFF + 8u * static_cast<uint32_t>(i); };
  auto sc_bar = [&](uint32_t i) { return base + Lay::SC_BAR_OFF + 8u * i; };  // a range's scales are written
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(smem_raw + Lay::TMEM_OFF);
  volatile int *units = reinterpret_cast<volatile int *>(smem_raw + Lay::UNIT_OFF);
  volatile float *xch = reinterpret_cast<volatile float *>(smem_raw + Lay::XCH_OFF);

  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_base_s), kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(bar(Lay::B_FULL + i), kConvWarps);
      mbar_init(bar(Lay::B_EMPTY + i), 1);  // the MMA warp's commit after the range's last product
      mbar_init(bar(Lay::B_RAW + i), 1);
      mbar_init(bar(Lay::B_CONV + i), 32 * kConvWarps);
    }
    for (int h = 0; h < kHalves; ++h) {
      mbar_init(bar(Lay::B_S + h), 1);
      mbar_init(bar(Lay::B_P + h), 4 * kParts);  // the half's softmax warps
      mbar_init(bar(Lay::B_O + h), 1);
      mbar_init(bar(Lay::B_QF + h), 4 * kParts);
      mbar_init(bar(Lay::B_QE + h), 1);
    }
    for (int i = 0; i < kUnitSlots; ++i) {
      mbar_init(bar(Lay::B_UF + i), 1);
      mbar_init(bar(Lay::B_UE + i), 1 + kSoftmaxWarps + kConvWarps);
    }
    for (int i = 0; i < 4 * kHalves; ++i) mbar_init(bar(Lay::B_X + i), 32 * kParts);
    for (int i = 0; i < Lay::SCALE_SLOTS; ++i) mbar_init(sc_bar(i), 1);
    mbar_init(bar(Lay::B_DRAIN), 1);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  fence_mbar_init();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // No griddepcontrol.wait here: this kernel follows the split-KV decode
  // kernel, which lets it start as its CTAs exit; it reads only what the
  // kernels before that one wrote (the plan's tiles, q, the caches), all
  // complete before the decode kernel let it start. It waits for the decode
  // kernel at its end, so its own completion still orders later work.
  const uint32_t tmem = *tmem_base_s;

  const int Hkv = p.num_kv_heads;
  const int bs = p.block_size;
  bool failed = false;
  uint32_t issued = 0;  // producer: loads issued (the final drain waits for them)

  // Record j of the stream sits in slot j % kUnitSlots; every consumer warp
  // reads each record once and releases the slot.
  auto read_unit = [&](uint32_t j, TileUnit &r) {
    const uint32_t s = j % kUnitSlots;
    wait_warp(bar(Lay::B_UF + s), (j / kUnitSlots) & 1u, failed);
    r.stop = 1;
    if (!failed) {
      const volatile int *u = units + 8 * s;
      r.slot = u[0];
      r.row0 = u[1];
      r.npos = u[2];
      r.pos0 = u[3];
      r.kv_end = u[4];
      r.kvh = u[5];
      r.stop = u[6];
      r.kv_begin = u[7];
    }
    __syncwarp();
    if (lane == 0 && !failed) mbar_arrive(bar(Lay::B_UE + s));
  };
  // key ranges of the unit, and of each half: up to its last valid position (0 = no valid rows)
  auto ranges = [&](const TileUnit &r, int (&nh)[kHalves]) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int last = min(r.npos, (h + 1) * POS_PER_HALF);  // positions [h * POS_PER_HALF, last)
      nh[h] = last > h * POS_PER_HALF
                  ? max((min(r.pos0 + last, r.kv_end) - r.kv_begin + kKeyTile - 1) / kKeyTile, 0)
                  : 0;
    }
    return (r.kv_end - r.kv_begin + kKeyTile - 1) / kKeyTile;
  };
  if (warp == kTmaWarp) {
    // ---------------- producer: unit records, then K(j), V(j) of each range ----------------
    const int total_units = min(max(ld_cg(p.tile_count), 0), p.max_tiles) * Hkv;
    const int box_rows = bs < kRawBoxRows ? bs : kRawBoxRows;
    const int nbk = kKeyTile / box_rows;                // 4 .. 16
    constexpr int LINES = (G * D * 2 + 127) / 128;      // of a position's q heads
    uint32_t j = 0, g = 0;
    for (;;) {
      int u = 0;
      if (lane == 0) u = atomicAdd(p.tile_counter, 1);
      u = __shfl_sync(FULL, u, 0);
      TileUnit r{0, 0, 0, 0, 0, 0, u >= total_units ? 1 : 0, 0, -1};
      if (!r.stop) {
        const int item = u / Hkv;
        r.kvh = u - item * Hkv;
        const int4 r0 = ld_cg(p.tiles + 2 * item);
        const int4 r1 = ld_cg(p.tiles + 2 * item + 1);
        r.b = r0.x;
        r.row0 = r0.y;
        r.npos = r0.z;
        r.pos0 = r0.w;
        r.kv_end = r1.y;
        r.kv_begin = r1.x;
        r.slot = r1.z >= 0 ? item * Hkv + r.kvh : -1;
        const bool sane = r.b >= 0 && r.b < p.num_seqs && r.npos >= 1 && r.npos <= kPrefillTileRows / G &&
                          r.row0 >= 0 && r.row0 + r.npos <= p.total_q && r.pos0 >= 0 &&
                          part_sane(r, p, item) &&
                          r.kv_end <= static_cast<int64_t>(p.max_blocks_per_seq) * bs;
        if (!sane) {
          if (lane == 0) flag_error(p.status, PA_FLAG_LENGTHS);
          continue;
        }
      }
      const uint32_t s = j % kUnitSlots;
      if (j >= kUnitSlots) wait_warp(bar(Lay::B_UE + s), (j / kUnitSlots - 1) & 1u, failed);
      if (failed) break;
      if (lane == 0) {
        volatile int *d = units + 8 * s;
        d[0] = r.slot;
        d[1] = r.row0;
        d[2] = r.npos;
        d[3] = r.pos0;
        d[4] = r.kv_end;
        d[5] = r.kvh;
        d[6] = r.stop;
        d[7] = r.kv_begin;
        mbar_arrive(bar(Lay::B_UF + s));  // release: the record is visible to whoever sees the phase
      }
      __syncwarp();
      ++j;
      if (r.stop) break;
      // its q rows towards L2, ahead of the softmax warps that load them: a
      // position's G heads are contiguous
      for (int i = lane; i < r.npos * LINES; i += 32) {
        const int pos = i / LINES;
        const char *row = reinterpret_cast<const char *>(p.q + static_cast<int64_t>(r.row0 + pos) * p.q_stride +
                                                         static_cast<int64_t>(r.kvh * G) * D);
        asm volatile("prefetch.global.L2 [%0];\n" ::"l"(row + (i - pos * LINES) * 128));
      }
      const int32_t *table = p.block_tables + static_cast<int64_t>(r.b) * p.max_blocks_per_seq;
      // First cache row of the box of `rows` keys starting at `key`: a block-table
      // lookup (block sizes are powers of two); keys past the end, or a block id
      // out of range, read at -rows (zero fill).
      auto box_z = [&](int key, int rows) {
        if (key >= r.kv_end) return -rows;
        const int phys = __ldg(table + (key >> p.block_shift));
        if (phys < 0 || phys >= p.num_blocks) {
          flag_error(p.status, PA_FLAG_BLOCK_RANGE);
          return -rows;
        }
        return (phys << p.block_shift) + (key & (bs - 1));
      };
      int dummy[kHalves];
      const int nkt = ranges(r, dummy);
      for (int kt = 0; kt < nkt && !failed; ++kt) {
        // lane i computes the row coordinate of K box i and V box i of this
        // range, and issues those boxes itself once lane 0 has set the byte count
        const int key0 = r.kv_begin + kt * kKeyTile;  // first key of the range
        const int zk = lane < nbk ? box_z(key0 + lane * box_rows, box_rows) : 0;
        float gks = 1.f, gvs1 = 1.f;  // block scales of group `lane` (1 past the last key)
        if (lane < kKeyTile / GRP) block_scales_of(p, table, key0 + GRP * lane, r.kv_end, r.kvh, gks, gvs1);
        for (int v = 0; v < 2 && !failed; ++v) {
          const uint32_t slot = g % SLOTS, use = g / SLOTS;
          if (use > 0) wait_warp(bar(Lay::B_EMPTY + slot), (use - 1) & 1u, failed);
          if (failed) break;
          if (v == 0) {
            const uint32_t fi = (g / 2) % Lay::SCALE_SLOTS;
            if (lane < kKeyTile / GRP)
              st_scales<GRP>(base + Lay::SC_OFF + fi * kScaleSlotBytes, lane, gks * p.scale_log2, gvs1);
            __syncwarp();
            if (lane == 0) mbar_arrive(sc_bar(fi));  // release: the range's scales
          }
          const void *map = v ? static_cast<const void *>(&vmap) : static_cast<const void *>(&kmap);
          const uint32_t dst = sRing + slot * Lay::KV_BYTES;
          // the range's codes: boxes of box_rows x D bytes into the back half of the slot
          const uint32_t b8 = bar(Lay::B_RAW + slot);
          if (lane == 0) mbar_arrive_expect_tx(b8, RAW_BYTES);
          __syncwarp();
          if (lane < nbk) tma_load_3d(dst + RAW_OFF + lane * box_rows * RAW_ROW, map, b8, 0, r.kvh, zk);
          __syncwarp();
          issued = ++g;
        }
      }
      if (failed) break;
    }
  } else if (warp >= kConvWarp && warp < kSoftmaxWarp0) {
    // ---------------- 8-bit caches: widen staged codes to fp16 in place ----------------
    // Lane l of converter warp w takes 16-byte code chunk c of rows
    // r0 + l % 8, so the eight lanes of one shared-memory phase touch eight
    // rows at one chunk: distinct bank groups in both swizzled layouts.
    constexpr int CPR = RAW_ROW / 16;         // code chunks per staged row (zeros past head_dim)
    constexpr int ROWS_PASS = 8 * (8 / CPR);  // rows per pass of the 64 threads
    constexpr int PASSES = kKeyTile / ROWS_PASS;
    const int ct = (warp - kConvWarp) * 32 + lane;
    const int q8 = ct >> 3, c = q8 % CPR, rsub = (q8 / CPR) * 8 + (ct & 7);
    uint32_t j = 0, g = 0;
    for (;;) {
      TileUnit r;
      read_unit(j++, r);
      if (failed || r.stop) break;
      int dummy[kHalves];
      const int nkt = ranges(r, dummy);
      for (int i = 0; i < 2 * nkt && !failed; ++i, ++g) {
        const uint32_t slot = g % SLOTS, use = g / SLOTS;
        wait_warp(bar(Lay::B_RAW + slot), use & 1u, failed);
        if (failed) break;
        const uint32_t sbase = sRing + slot * Lay::KV_BYTES;
        uint4 codes[PASSES];
#pragma unroll
        for (int i2 = 0; i2 < PASSES; ++i2) {
          const int rr = i2 * ROWS_PASS + rsub;
          const uint32_t a = sbase + RAW_OFF + (RAW_ROW == 128 ? rr * 128 + (((c ^ rr) & 7) << 4)
                                                                : rr * 64 + (((c ^ (rr >> 1)) & 3) << 4));
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                       : "=r"(codes[i2].x), "=r"(codes[i2].y), "=r"(codes[i2].z), "=r"(codes[i2].w)
                       : "r"(a));
        }
        // every code of the slot is in registers (both warps) before any fp16 row overwrites them
        mbar_arrive(bar(Lay::B_CONV + slot));
        wait_warp(bar(Lay::B_CONV + slot), use & 1u, failed);
        if (failed) break;
#pragma unroll
        for (int i2 = 0; i2 < PASSES; ++i2) {
          const int rr = i2 * ROWS_PASS + rsub;
          const uint32_t w[4] = {codes[i2].x, codes[i2].y, codes[i2].z, codes[i2].w};
          uint32_t hh[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
                " cvt.rn.f16x2.e4m3x2 %1, u;\n}\n"
                : "=r"(hh[2 * k]), "=r"(hh[2 * k + 1])
                : "r"(w[k]));
          }
          // codes d = 16c .. 16c + 15 -> fp16 chunks 2c (d .. d + 7) and 2c + 1
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(sbase + Lay::off(rr, 2 * c, Lay::KV_ATOM)),
                       "r"(hh[0]), "r"(hh[1]), "r"(hh[2]), "r"(hh[3])
                       : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(
                           sbase + Lay::off(rr, 2 * c + 1, Lay::KV_ATOM)),
                       "r"(hh[4]), "r"(hh[5]), "r"(hh[6]), "r"(hh[7])
                       : "memory");
        }
        fence_proxy_async_smem();  // the MMA reads the slot through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Lay::B_FULL + slot));
      }
      if (failed) break;
    }
  } else if (warp == kMmaWarp) {
    // ---------------- MMA issue ----------------
    // The whole warp follows the loops (it zeroes the tail of the last V
    // range); lane 0 alone issues tensor-core work and commits. Range r of a
    // unit is read by the halves with r < nkt_h: the first of them waits for
    // the K/V loads, the last one's commit releases the buffers.
    constexpr uint32_t DHI = desc_hi(1024);
    const uint32_t utmem = uniform(tmem);
    const uint32_t q_lo0 = uniform(desc_lo(sQ0, 16)), q_lo1 = uniform(desc_lo(sQ0 + Lay::Q_BYTES, 16));
    const uint32_t k_lo = desc_lo(sRing, 16);  // slot 0
    // V (MN-major): LBO = distance between the two 64-element atoms along d,
    // SBO = distance between 8-key groups along K; K step ks at byte 2048 ks
    const uint32_t v_lo = desc_lo(sRing, Lay::KV_ATOM);
    constexpr uint32_t SLOT_STEP = Lay::KV_BYTES >> 4;  // per slot
    uint32_t ph[kHalves] = {0, 0};  // ranges each half has run so far (phases of its s, p, o barriers)
    uint32_t ring0 = 0;             // loads of earlier units
    for (uint32_t j = 0;; ++j) {
      TileUnit r;
      read_unit(j, r);
      if (failed || r.stop) break;
      int nkt_h[kHalves];
      const int nkt = ranges(r, nkt_h);
      auto first_reader = [&](int kt) { return kt < nkt_h[0] ? 0 : 1; };
      auto last_reader = [&](int kt) { return kt < nkt_h[1] ? 1 : 0; };
      // ring slot of K(kt) (v = 0) or V(kt) (v = 1), and the parity of its full barrier
      auto slot_of = [&](int kt, int v) { return (ring0 + 2 * kt + v) % SLOTS; };
      auto full_parity = [&](int kt, int v) { return ((ring0 + 2 * kt + v) / SLOTS) & 1u; };
      auto mma_s = [&](int kt, int h) {
        const uint32_t klo = uniform(k_lo + slot_of(kt, 0) * SLOT_STEP), qlo = h ? q_lo1 : q_lo0;
        const uint32_t d = utmem + h * Tm::HALF + Tm::SP;
        if (elect_one()) {
          tc_fence_after();
          mma_ss<0>(d, qlo, DHI, klo, DHI, IDESC_S);
#pragma unroll
          for (int ks = 1; ks < KSTEPS_S; ++ks) {
            const uint32_t qo = ((ks >> 2) * Lay::Q_ATOM + (ks & 3) * 32) >> 4;
            const uint32_t ko = ((ks >> 2) * Lay::KV_ATOM + (ks & 3) * 32) >> 4;
            mma_ss<1>(d, qlo + qo, DHI, klo + ko, DHI, IDESC_S);
          }
          tc_commit(bar(Lay::B_S + h));
          if (h == last_reader(kt)) tc_commit(bar(Lay::B_EMPTY + slot_of(kt, 0)));
        }
        __syncwarp();
      };
      // this unit's Q in both halves (the softmax warps store it); qe lets them store the next one
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        wait_warp(bar(Lay::B_QF + h), j & 1u, failed);
        if (lane == 0 && !failed) mbar_arrive(bar(Lay::B_QE + h));
      }
      if (failed) break;
      if (nkt > 0) {
        wait_warp(bar(Lay::B_FULL + slot_of(0, 0)), full_parity(0, 0), failed);
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          if (nkt_h[h] > 0 && !failed) mma_s(0, h);
      }
      for (int kt = 0; kt < nkt && !failed; ++kt) {
        const uint32_t vslot = slot_of(kt, 1);
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          if (kt >= nkt_h[h]) continue;
          wait_warp(bar(Lay::B_P + h), (ph[h] + kt) & 1u, failed);  // P(kt) is in place
          if (failed) break;
          if (h == first_reader(kt)) {
            wait_warp(bar(Lay::B_FULL + vslot), full_parity(kt, 1), failed);
            if (failed) break;
            const int key0 = r.kv_begin + kt * kKeyTile;
            if (key0 + kKeyTile > r.kv_end) {
              // rows of keys past kv_end may hold anything (even NaN): zero them in V
              const uint32_t sV = sRing + vslot * Lay::KV_BYTES;
              const int vr0 = r.kv_end - key0;
              const int n = (kKeyTile - vr0) * (D / 8);
              for (int i = lane; i < n; i += 32) {
                const int rr = vr0 + i / (D / 8), c = i % (D / 8);
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(sV + Lay::off(rr, c, Lay::KV_ATOM)), "r"(0u)
                             : "memory");
              }
              fence_proxy_async_smem();
            }
            __syncwarp();
          }
          const uint32_t vlo = uniform(v_lo + vslot * SLOT_STEP);
          const uint32_t t = utmem + h * Tm::HALF;
          if (elect_one()) {
            tc_fence_after();
            // one fp16 P per key: K step ks at column 8 ks (+ 32 for the second part's keys)
            auto pcol = [](int ks) { return 8 * ks + (ks >= 4 ? 32 : 0); };
            if (kt == 0)
              mma_ts<0>(t + Tm::O, t + Tm::SP, vlo, DHI, IDESC_O);  // the unit's first product overwrites O
            else
              mma_ts<1>(t + Tm::O, t + Tm::SP, vlo, DHI, IDESC_O);
#pragma unroll
            for (int ks = 1; ks < KSTEPS_O; ++ks)
              mma_ts<1>(t + Tm::O, t + Tm::SP + pcol(ks), vlo + ((ks * 2048) >> 4), DHI, IDESC_O);
            tc_commit(bar(Lay::B_O + h));
            if (h == last_reader(kt)) tc_commit(bar(Lay::B_EMPTY + vslot));
          }
          __syncwarp();
          if (kt + 1 < nkt_h[h]) {
            if (h == first_reader(kt + 1))
              wait_warp(bar(Lay::B_FULL + slot_of(kt + 1, 0)), full_parity(kt + 1, 0), failed);
            if (failed) break;
            mma_s(kt + 1, h);
          }
        }
      }
      if (failed) break;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) ph[h] += nkt_h[h];
      ring0 += 2 * nkt;
    }
  } else {
    // ---------------- softmax: one row per thread (its TMEM lane), 64 keys per range ----------------
    const int sw = warp - kSoftmaxWarp0;  // softmax warp index
    const int quad = sw & 3, h = (sw >> 2) & 1, part = sw / (4 * kHalves);
    const int r = quad * 32 + lane;  // row within the half = TMEM lane
    const uint32_t t_lane = tmem + h * Tm::HALF + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t bx = bar(Lay::B_X + h * 4 + quad);  // exchange with the other warp of these rows
    volatile float *x_mine = xch + (h * kParts + part) * kHalfRows + r;
    volatile float *x_other = xch + (h * kParts + (kParts - 1 - part)) * kHalfRows + r;
    uint32_t nx = 0;  // exchanges so far
    // my value out, the other warp's value in (both warps of the rows call it alike)
    auto exchange = [&](float v) -> float {
      *x_mine = v;
      mbar_arrive(bx);  // every thread: release of its own store
      wait_warp(bx, nx & 1u, failed);
      ++nx;
      return failed ? v : *x_other;
    };
    // both warps of the rows have reached this point (no data)
    auto pair_sync = [&]() {
      mbar_arrive(bx);
      wait_warp(bx, nx & 1u, failed);
      ++nx;
    };
    const int ch0 = part ? (NCH + 1) / 2 : 0, ch1 = part ? NCH : (NCH + 1) / 2;  // this warp's O chunks
    // the factors of this warp's 32 rows, from the lanes that stored their Q
    // (lane l < 16: row 16 part + l); the values exchanged before have been read
    auto row_factors = [&](float mine) -> float {
      if (lane < 16) xch[(h * kParts + part) * kHalfRows + quad * 32 + part * 16 + lane] = mine;
      pair_sync();
      const float v = xch[(h * kParts + (lane >> 4)) * kHalfRows + r];
      pair_sync();
      return v;
    };
    const int g = r % G;
    uint32_t phh = 0;  // ranges this half has run so far
    uint32_t gvs = 0;  // ranges of the CTA's earlier units (both halves)

    // Q of the half for unit `u`: this warp's 16 rows; returns their factors (lanes 0..15)
    auto load_q = [&](const TileUnit &u) -> float {
      const uint32_t sQ = sQ0 + h * Lay::Q_BYTES;
      const float mine = load_q_rows<D, G, E>(p, u, h * POS_PER_HALF, quad * 32 + part * 16, lane,
                                              [&](int row, int c) { return sQ + Lay::off(row, c, Lay::Q_ATOM); });
      fence_proxy_async_smem();  // the MMA reads Q through the async proxy
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Lay::B_QF + h));
      return mine;
    };

    TileUnit cur;
    read_unit(0, cur);
    // the row's score factor (> 0: the max of raw scores gives the max of scaled ones)
    float rowf = 1.f;
    if (!failed && !cur.stop) rowf = row_factors(load_q(cur));
    for (uint32_t j = 0; !failed && !cur.stop; ++j) {
      int nkt_h[kHalves];
      const int nkt_all = ranges(cur, nkt_h);
      const int nk = nkt_h[h];
      const int qi = h * POS_PER_HALF + r / G;
      const bool row_valid = qi < cur.npos;
      const int lim = row_valid ? cur.pos0 + qi + 1 : 0;  // keys j < lim are visible to this row
      float m_used = -INFINITY, l = 0.f;
      for (int kt = 0; kt < nk; ++kt) {
        const int ck0 = cur.kv_begin + kt * kKeyTile + part * PART_KEYS;  // this warp's first key of the range
        const uint32_t sp = t_lane + Tm::SP + part * PART_KEYS;
        wait_warp(bar(Lay::B_S + h), (phh + kt) & 1u, failed);
        if (failed) break;
        uint32_t sc = 0;  // block scales: this warp's keys of the range
        // (already there: they were written before the K that S came from)
        const uint32_t gv = gvs + kt, fi = gv % Lay::SCALE_SLOTS;
        wait_warp(sc_bar(fi), (gv / Lay::SCALE_SLOTS) & 1u, failed);
        if (failed) break;
        sc = base + Lay::SC_OFF + fi * kScaleSlotBytes + part * (kScaleSlotBytes / kParts);
        tc_fence_after();
        uint32_t s0[32], s1[32];
        tmem_ld32x2_wait(sp, s0, s1);
        // The range's maximum over both warps' keys, then its growth over
        // m_used, as separately rounded operations (no contraction into one
        // fused multiply-add): the exponents below are bounded by exactly this
        // difference. The other warp reads its scores before either writes P.
        float mx;
        // (64 keys a warp and range; a row that is none of the tile's is not stored, and needs no mask)
        const bool masked = __any_sync(FULL, row_valid && ck0 + 64 > lim);
        if (masked)
          mx = fmaxf(scaled_max32<GRP, true>(s0, ck0, lim, rowf, sc),
                     scaled_max32<GRP, true>(s1, ck0 + 32, lim, rowf, sc + 32));
        else
          mx = fmaxf(scaled_max32<GRP, false>(s0, ck0, lim, rowf, sc),
                     scaled_max32<GRP, false>(s1, ck0 + 32, lim, rowf, sc + 32));
        const float mo = exchange(mx);
        if (failed) break;
        const float cm = fmaxf(mx, mo);
        const bool grow = cm > -INFINITY && (m_used == -INFINITY || __fsub_rn(cm, m_used) > kRescaleLog2);
        float alpha = 1.f;  // factor owed by O and l for the growth
        if (grow) {
          alpha = m_used > -INFINITY ? ex2_approx(__fsub_rn(m_used, cm)) : 1.f;
          m_used = cm;
        }
        const float ms = m_used == -INFINITY ? 0.f : m_used;
        float sum = 0.f;
        const bool rare = masked || __any_sync(FULL, fabsf(ms) > 4096.f || rowf != 1.f);
        // P over the scores it came from, one UMMA K step (16 keys) at a
        // time, the scores read again from TMEM: a loop unrolled twice, not
        // four times (the hot code of twenty warps shares the instruction
        // cache; measured 5 % faster over bf16 caches than four steps inline
        // on scores kept in registers), no score registers live across it.
        // P of step ks (8 columns at 8 ks) covers only scores read by
        // earlier steps. Rare cases stay out of the loop (inside it, as a
        // branch per step, they cost 2 %).
        if (rare) {
#pragma unroll 1
          for (int ks = 0; ks < PART_KEYS / 16; ++ks) {
            const float4 c = ld_scales(sc + 16 * ks);
            uint32_t t[16];
            tmem_ld16_wait(sp + 16 * ks, t);
            probs16_scaled_store<GRP, true>(t, ck0 + 16 * ks, lim, rowf, ms, sum, sp + 8 * ks, c);
          }
        } else {
#pragma unroll 2
          for (int ks = 0; ks < PART_KEYS / 16; ++ks) {
            const float4 c = ld_scales(sc + 16 * ks);
            uint32_t t[16];
            tmem_ld16_wait(sp + 16 * ks, t);
            probs16_scaled_store<GRP, false>(t, ck0 + 16 * ks, lim, rowf, ms, sum, sp + 8 * ks, c);
          }
        }
        // O holds P V(0 .. kt-1), all complete (they were issued before S(kt),
        // whose completion the wait above observed); each warp rescales its
        // own columns.
        if (kt > 0 && __any_sync(FULL, alpha != 1.f)) {
#pragma unroll 1
          for (int ch = ch0; ch < ch1; ++ch) {
            uint32_t t[32];
            tmem_ld32_wait(t_lane + Tm::O + ch * 32, t);
#pragma unroll
            for (int i = 0; i < 32; ++i) t[i] = __float_as_uint(__uint_as_float(t[i]) * alpha);
            tmem_st32u(t_lane + Tm::O + ch * 32, t);
          }
        }
        l = l * alpha + sum;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Lay::B_P + h));
      }
      if (failed) break;
      // the next unit's record and Q (overlapping this unit's last products)
      float next_mine = 1.f;
      TileUnit nxt;
      read_unit(j + 1, nxt);
      if (!failed && !nxt.stop) {
        wait_warp(bar(Lay::B_QE + h), j & 1u, failed);  // the MMA warp has taken this unit's Q
        if (!failed) next_mine = load_q(nxt);
      }
      if (failed) break;
      if (nk > 0) {
        // epilogue: the row sum over both warps' keys, then this warp's columns
        // of the half's last P V product, normalised
        pair_sync();  // both warps are past their last read of the maxima
        const float lt = l + exchange(l);
        pair_sync();  // both have read the sums
        wait_warp(bar(Lay::B_O + h), (phh + nk - 1) & 1u, failed);
        if (failed) break;
        tc_fence_after();
        const float inv = lt != 0.f ? 1.f / lt : 0.f;
        bf16 *dst = p.out + static_cast<int64_t>(cur.row0 + (row_valid ? qi : 0)) * p.num_heads * D +
                    static_cast<int64_t>(cur.kvh * G + g) * D;
        float *pdst = nullptr;  // the row's partial, for a part of the tile's keys
        if (cur.slot >= 0) {
          const int64_t prow = static_cast<int64_t>(cur.slot) * kPrefillTileRows + h * kHalfRows + r;
          pdst = p.part_o + prow * D;
          if (part == 0 && row_valid) p.part_lse[prow] = lt != 0.f ? m_used + __log2f(lt) : -INFINITY;
        }
#pragma unroll 1
        for (int ch = ch0; ch < ch1; ++ch) {
          uint32_t t[32];
          tmem_ld32_wait(t_lane + Tm::O + ch * 32, t);
          if (pdst) {
            if (row_valid) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                if (32 * ch + 4 * c >= D) continue;
                const float *f = reinterpret_cast<const float *>(&t[4 * c]);
                *reinterpret_cast<float4 *>(pdst + ch * 32 + 4 * c) =
                    make_float4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
              }
            }
          } else if (row_valid) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (32 * ch + 8 * c >= D) continue;  // head_dim 80: the last 16 columns are padding
              const float *f = reinterpret_cast<const float *>(&t[8 * c]);
              const uint4 v = make_uint4(E::pack(f[0] * inv, f[1] * inv), E::pack(f[2] * inv, f[3] * inv),
                                         E::pack(f[4] * inv, f[5] * inv), E::pack(f[6] * inv, f[7] * inv));
              *reinterpret_cast<uint4 *>(dst + ch * 32 + 8 * c) = v;
            }
          }
        }
        tc_fence_before();  // O is overwritten by a later unit's first product
      } else if (cur.slot >= 0 && part == 0 && row_valid) {
        // the half sees none of this part's keys
        p.part_lse[static_cast<int64_t>(cur.slot) * kPrefillTileRows + h * kHalfRows + r] = -INFINITY;
      }
      phh += nk;
      gvs += nkt_all;
      if (!nxt.stop) rowf = row_factors(next_mine);
      cur = nxt;
    }
  }

  // Every warp has left its loop (normally at the end of the stream, or after
  // a timeout). Before tensor memory and shared memory go away, wait (bounded)
  // for work still in flight: the MMA thread's products (one last commit)
  // and the producer's loads (loads into a buffer complete in order, so
  // waiting for the last SLOTS issued suffices).
  if (warp == kMmaWarp && elect_one()) {  // the thread that issued them
    tc_commit(bar(Lay::B_DRAIN));
    if (!mbar_wait_bounded(bar(Lay::B_DRAIN), 0, kTcWaitTimeoutNs)) failed = true;
  }
  if (warp == kTmaWarp && lane == 0) {
    const int landed = Lay::B_RAW;  // where the loads' completion is counted
    for (uint32_t g = issued > SLOTS ? issued - SLOTS : 0; g < issued; ++g)
      if (!mbar_wait_bounded(bar(landed + static_cast<int>(g % SLOTS)), (g / SLOTS) & 1u, kTcWaitTimeoutNs))
        failed = true;
  }
  if (failed) flag_error(p.status, PA_FLAG_TIMEOUT);
  griddep_wait();  // the decode kernel before this one has completed
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------
// head_dim 256: one 128-row half per tile, two score buffers, a K or V range as
// two units of 128 keys x 128 elements (the one-half kernel of
// attention_prefill_tc.cu, with block scales and parts).
// ---------------------------------------------------------------------------
constexpr int kWideD = 256;
constexpr int kWideSoftmaxWarps = 8;
constexpr int kWideThreads = 32 * (kSoftmaxWarp0 + kWideSoftmaxWarps);

struct WideTmem {
  static constexpr uint32_t SP0 = 0, O = 2 * kKeyTile;  // score buffers at 0 and 128, O at [256, 512)
};

struct WideLayout {
  static constexpr int Q_ATOM = kHalfRows * 128;   // 128 rows x 128 B
  static constexpr int Q_BYTES = 4 * Q_ATOM;       // one half, four 64-element atoms
  static constexpr int KV_ATOM = kKeyTile * 128;   // 128 keys x 128 B
  static constexpr int UNIT_BYTES = 2 * KV_ATOM;   // 128 keys x 128 elements: a ring slot
  // mbarriers: per ring slot full, empty, raw, conv; per score buffer s, p;
  // o, qf, qe; per record slot uf, ue; per lane quadrant x1 (values
  // written), x2 (values read); drain
  static constexpr int B_FULL = 0, B_EMPTY = kMaxSlots, B_RAW = 2 * kMaxSlots, B_CONV = 3 * kMaxSlots;
  static constexpr int B_S = 4 * kMaxSlots, B_P = B_S + 2, B_O = B_P + 2, B_QF = B_O + 1, B_QE = B_QF + 1;
  static constexpr int B_UF = B_QE + 1, B_UE = B_UF + kUnitSlots, B_X1 = B_UE + kUnitSlots, B_X2 = B_X1 + 4;
  static constexpr int B_DRAIN = B_X2 + 4, NBARS = B_DRAIN + 1;
  static constexpr int XCH_BYTES = kWideSoftmaxWarps * 32 * 4;
  static constexpr int REC_BYTES = kUnitSlots * 32;
  static constexpr int FIXED = Q_BYTES + XCH_BYTES + REC_BYTES + 8 * NBARS + 16;
  static constexpr int FIT = (227 * 1024 - FIXED) / UNIT_BYTES;
  static constexpr int SLOTS = FIT < kMaxSlots ? FIT : kMaxSlots;
  static_assert(SLOTS >= 5, "the ring holds a range's four loads and the next one's first");
  static constexpr int RING_OFF = Q_BYTES;
  static constexpr int XCH_OFF = RING_OFF + SLOTS * UNIT_BYTES;
  static constexpr int REC_OFF = XCH_OFF + XCH_BYTES;
  static constexpr int BAR_OFF = REC_OFF + REC_BYTES;
  static constexpr int TMEM_OFF = BAR_OFF + 8 * NBARS;
  static constexpr int BYTES = TMEM_OFF + 16;
};
// Range g's scales are written once load 4 g - 5 (V of range g - 2) has been used up: two slots.
static_assert(WideLayout::SLOTS == 5, "two scale slots");
using BlockWideLayout = WithScales<WideLayout, 2>;
static_assert(BlockWideLayout::BYTES <= 227 * 1024, "shared memory of one CTA");

template <int G, typename E, int GRP>
__global__ void __launch_bounds__(kWideThreads, 1)
    block_tile_wide_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                             const BlockTileParams p) {
  using Lay = BlockWideLayout;
  using Tm = WideTmem;
  using TL = TcLayout<128>;  // a ring slot: the layout of a head_dim-128 range
  constexpr int D = kWideD;
  constexpr int RAW_ROW = 128;
  constexpr int RAW_BYTES = kKeyTile * RAW_ROW;    // 8-bit codes of one unit
  constexpr uint32_t RAW_OFF = Lay::UNIT_BYTES / 2;
  constexpr int LPR = 4;                           // loads per range: K lo, K hi, V lo, V hi
  constexpr int KSTEPS_S = D / 16;
  constexpr int KSTEPS_O = kKeyTile / 16;
  constexpr int POS = kHalfRows / G;               // positions per tile
  constexpr uint32_t IDESC_S = f16_idesc(kHalfRows, kKeyTile, 0, ElemFp16::kUmmaFormat);
  constexpr uint32_t IDESC_O = f16_idesc(kHalfRows, 128, 1, ElemFp16::kUmmaFormat);
  constexpr float kRescaleLog2 = 8.f;
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int SLOTS = Lay::SLOTS;

  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = smem_u32(smem_raw);
  if (base & 1023u) {
    if (tid == 0) flag_error(p.status, PA_FLAG_LENGTHS);
    griddep_wait();
    return;
  }
  const uint32_t sQ = base, sRing = base + Lay::RING_OFF;
  auto bar = [&](int i) { return base + Lay::BAR_OFF + 8u * static_cast<uint32_t>(i); };
  auto sc_bar = [&](uint32_t i) { return base + Lay::SC_BAR_OFF + 8u * i; };  // a range's scales are written
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(smem_raw + Lay::TMEM_OFF);
  volatile int *units = reinterpret_cast<volatile int *>(smem_raw + Lay::REC_OFF);
  volatile float *xch = reinterpret_cast<volatile float *>(smem_raw + Lay::XCH_OFF);

  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_base_s), kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(bar(Lay::B_FULL + i), kConvWarps);
      mbar_init(bar(Lay::B_EMPTY + i), 1);
      mbar_init(bar(Lay::B_RAW + i), 1);
      mbar_init(bar(Lay::B_CONV + i), 32 * kConvWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(Lay::B_S + b), 1);
      mbar_init(bar(Lay::B_P + b), kWideSoftmaxWarps);
    }
    mbar_init(bar(Lay::B_O), 1);
    mbar_init(bar(Lay::B_QF), kWideSoftmaxWarps);
    mbar_init(bar(Lay::B_QE), 1);
    for (int i = 0; i < kUnitSlots; ++i) {
      mbar_init(bar(Lay::B_UF + i), 1);
      mbar_init(bar(Lay::B_UE + i), 1 + kWideSoftmaxWarps + kConvWarps);
    }
    for (int q = 0; q < 4; ++q) {
      mbar_init(bar(Lay::B_X1 + q), 64);  // the two softmax warps of a lane quadrant
      mbar_init(bar(Lay::B_X2 + q), 64);
    }
    for (int i = 0; i < Lay::SCALE_SLOTS; ++i) mbar_init(sc_bar(i), 1);
    mbar_init(bar(Lay::B_DRAIN), 1);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  fence_mbar_init();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // No griddepcontrol.wait here: this kernel follows the split-KV decode
  // kernel, which lets it start as its CTAs exit; it reads only what the
  // kernels before that one wrote (the plan's tiles, q, the caches), all
  // complete before the decode kernel let it start. It waits for the decode
  // kernel at its end, so its own completion still orders later work.
  const uint32_t tmem = *tmem_base_s;

  const int Hkv = p.num_kv_heads;
  const int bs = p.block_size;
  bool failed = false;
  uint32_t issued = 0;

  auto read_unit = [&](uint32_t j, TileUnit &r) {
    const uint32_t s = j % kUnitSlots;
    wait_warp(bar(Lay::B_UF + s), (j / kUnitSlots) & 1u, failed);
    r.stop = 1;
    if (!failed) {
      const volatile int *u = units + 8 * s;
      r.slot = u[0];
      r.row0 = u[1];
      r.npos = u[2];
      r.pos0 = u[3];
      r.kv_end = u[4];
      r.kvh = u[5];
      r.stop = u[6];
      r.kv_begin = u[7];
    }
    __syncwarp();
    if (lane == 0 && !failed) mbar_arrive(bar(Lay::B_UE + s));
  };
  auto nranges = [&](const TileUnit &r) { return (r.kv_end - r.kv_begin + kKeyTile - 1) / kKeyTile; };

  if (warp == kTmaWarp) {
    // ---------------- producer ----------------
    const int total_units = min(max(ld_cg(p.tile_count), 0), p.max_tiles) * Hkv;
    constexpr int MAXROWS = kRawBoxRows;
    const int box_rows = bs < MAXROWS ? bs : MAXROWS;
    const int nbk = kKeyTile / box_rows;
    uint32_t j = 0, g = 0;
    for (;;) {
      int u = 0;
      if (lane == 0) u = atomicAdd(p.tile_counter, 1);
      u = __shfl_sync(FULL, u, 0);
      TileUnit r{0, 0, 0, 0, 0, 0, u >= total_units ? 1 : 0, 0, -1};
      if (!r.stop) {
        const int item = u / Hkv;
        r.kvh = u - item * Hkv;
        const int4 r0 = ld_cg(p.tiles + 2 * item);
        const int4 r1 = ld_cg(p.tiles + 2 * item + 1);
        r.b = r0.x;
        r.row0 = r0.y;
        r.npos = r0.z;
        r.pos0 = r0.w;
        r.kv_end = r1.y;
        r.kv_begin = r1.x;
        r.slot = r1.z >= 0 ? item * Hkv + r.kvh : -1;
        const bool sane = r.b >= 0 && r.b < p.num_seqs && r.npos >= 1 && r.npos <= POS && r.row0 >= 0 &&
                          r.row0 + r.npos <= p.total_q && r.pos0 >= 0 &&
                          part_sane(r, p, item) &&
                          r.kv_end <= static_cast<int64_t>(p.max_blocks_per_seq) * bs;
        if (!sane) {
          if (lane == 0) flag_error(p.status, PA_FLAG_LENGTHS);
          continue;
        }
      }
      const uint32_t s = j % kUnitSlots;
      if (j >= kUnitSlots) wait_warp(bar(Lay::B_UE + s), (j / kUnitSlots - 1) & 1u, failed);
      if (failed) break;
      if (lane == 0) {
        volatile int *d = units + 8 * s;
        d[0] = r.slot;
        d[1] = r.row0;
        d[2] = r.npos;
        d[3] = r.pos0;
        d[4] = r.kv_end;
        d[5] = r.kvh;
        d[6] = r.stop;
        d[7] = r.kv_begin;
        mbar_arrive(bar(Lay::B_UF + s));
      }
      __syncwarp();
      ++j;
      if (r.stop) break;
      const int32_t *table = p.block_tables + static_cast<int64_t>(r.b) * p.max_blocks_per_seq;
      auto box_z = [&](int key, int rows) {
        if (key >= r.kv_end) return -rows;
        const int phys = __ldg(table + (key >> p.block_shift));
        if (phys < 0 || phys >= p.num_blocks) {
          flag_error(p.status, PA_FLAG_BLOCK_RANGE);
          return -rows;
        }
        return (phys << p.block_shift) + (key & (bs - 1));
      };
      const int nkt = nranges(r);
      for (int kt = 0; kt < nkt && !failed; ++kt) {
        const int key0 = r.kv_begin + kt * kKeyTile;  // first key of the range
        const int z = lane < nbk ? box_z(key0 + lane * box_rows, box_rows) : 0;
        float gks = 1.f, gvs1 = 1.f;  // block scales of group `lane` (1 past the last key)
        if (lane < kKeyTile / GRP) block_scales_of(p, table, key0 + GRP * lane, r.kv_end, r.kvh, gks, gvs1);
        for (int v = 0; v < LPR && !failed; ++v) {
          const uint32_t slot = g % SLOTS, use = g / SLOTS;
          if (use > 0) wait_warp(bar(Lay::B_EMPTY + slot), (use - 1) & 1u, failed);
          if (failed) break;
          if (v == 0) {
            const uint32_t fi = (g / LPR) % Lay::SCALE_SLOTS;
            if (lane < kKeyTile / GRP)
              st_scales<GRP>(base + Lay::SC_OFF + fi * kScaleSlotBytes, lane, gks * p.scale_log2, gvs1);
            __syncwarp();
            if (lane == 0) mbar_arrive(sc_bar(fi));  // release: the range's scales
          }
          const void *map = v >= 2 ? static_cast<const void *>(&vmap) : static_cast<const void *>(&kmap);
          const int x0 = (v & 1) * 128;  // first element of the unit's half of d
          const uint32_t dst = sRing + slot * Lay::UNIT_BYTES;
          const uint32_t b8 = bar(Lay::B_RAW + slot);
          if (lane == 0) mbar_arrive_expect_tx(b8, RAW_BYTES);
          __syncwarp();
          if (lane < nbk) tma_load_3d(dst + RAW_OFF + lane * box_rows * RAW_ROW, map, b8, x0, r.kvh, z);
          __syncwarp();
          issued = ++g;
        }
      }
      if (failed) break;
    }
  } else if (warp >= kConvWarp && warp < kSoftmaxWarp0) {
    // ---------------- 8-bit caches: widen staged codes to fp16 in place (unit by unit) ----------------
    constexpr int CPR = RAW_ROW / 16;
    constexpr int ROWS_PASS = 8 * (8 / CPR);
    constexpr int PASSES = kKeyTile / ROWS_PASS;
    const int ct = (warp - kConvWarp) * 32 + lane;
    const int q8 = ct >> 3, c = q8 % CPR, rsub = (q8 / CPR) * 8 + (ct & 7);
    uint32_t j = 0, g = 0;
    for (;;) {
      TileUnit r;
      read_unit(j++, r);
      if (failed || r.stop) break;
      const int nkt = nranges(r);
      for (int i = 0; i < LPR * nkt && !failed; ++i, ++g) {
        const uint32_t slot = g % SLOTS, use = g / SLOTS;
        wait_warp(bar(Lay::B_RAW + slot), use & 1u, failed);
        if (failed) break;
        const uint32_t sbase = sRing + slot * Lay::UNIT_BYTES;
        uint4 codes[PASSES];
#pragma unroll
        for (int i2 = 0; i2 < PASSES; ++i2) {
          const int rr = i2 * ROWS_PASS + rsub;
          const uint32_t a = sbase + RAW_OFF + rr * 128 + (((c ^ rr) & 7) << 4);
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                       : "=r"(codes[i2].x), "=r"(codes[i2].y), "=r"(codes[i2].z), "=r"(codes[i2].w)
                       : "r"(a));
        }
        mbar_arrive(bar(Lay::B_CONV + slot));
        wait_warp(bar(Lay::B_CONV + slot), use & 1u, failed);
        if (failed) break;
#pragma unroll
        for (int i2 = 0; i2 < PASSES; ++i2) {
          const int rr = i2 * ROWS_PASS + rsub;
          const uint32_t w[4] = {codes[i2].x, codes[i2].y, codes[i2].z, codes[i2].w};
          uint32_t hh[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
                " cvt.rn.f16x2.e4m3x2 %1, u;\n}\n"
                : "=r"(hh[2 * k]), "=r"(hh[2 * k + 1])
                : "r"(w[k]));
          }
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(sbase + TL::off(rr, 2 * c, TL::KV_ATOM)),
                       "r"(hh[0]), "r"(hh[1]), "r"(hh[2]), "r"(hh[3])
                       : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(
                           sbase + TL::off(rr, 2 * c + 1, TL::KV_ATOM)),
                       "r"(hh[4]), "r"(hh[5]), "r"(hh[6]), "r"(hh[7])
                       : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Lay::B_FULL + slot));
      }
      if (failed) break;
    }
  } else if (warp == kMmaWarp) {
    // ---------------- MMA issue ----------------
    // Ranges run S(0), S(1), then per range r: P V(r) (once P(r) is written)
    // and S(r + 2) into the score buffer P V(r) read (the products one thread
    // issues execute in issue order). Range number gr = (ranges of earlier
    // units) + r counts across units: its score buffer is gr % 2 and that
    // buffer's barriers complete once per use, phase gr / 2.
    constexpr uint32_t DHI = desc_hi(1024);
    const uint32_t q_lo = desc_lo(sQ, 16);
    const uint32_t k_lo = desc_lo(sRing, 16), v_lo = desc_lo(sRing, Lay::KV_ATOM);
    constexpr uint32_t SLOT_STEP = Lay::UNIT_BYTES >> 4;
    uint32_t ph = 0, ring0 = 0;
    for (uint32_t j = 0;; ++j) {
      TileUnit r;
      read_unit(j, r);
      if (failed || r.stop) break;
      const int nkt = nranges(r);
      auto slot_of = [&](int kt, int u) { return (ring0 + LPR * kt + u) % SLOTS; };
      auto full_parity = [&](int kt, int u) { return ((ring0 + LPR * kt + u) / SLOTS) & 1u; };
      auto mma_s = [&](int kt) {
        wait_warp(bar(Lay::B_FULL + slot_of(kt, 0)), full_parity(kt, 0), failed);
        wait_warp(bar(Lay::B_FULL + slot_of(kt, 1)), full_parity(kt, 1), failed);
        if (failed) return;
        if (lane == 0) {
          tc_fence_after();
          const uint32_t gr = ph + kt;
          const uint32_t d = tmem + Tm::SP0 + (gr & 1u) * kKeyTile;
          const uint32_t klo0 = k_lo + slot_of(kt, 0) * SLOT_STEP, klo1 = k_lo + slot_of(kt, 1) * SLOT_STEP;
#pragma unroll
          for (int ks = 0; ks < KSTEPS_S; ++ks) {
            const uint32_t qo = ((ks >> 2) * Lay::Q_ATOM + (ks & 3) * 32) >> 4;
            const uint32_t ko = (((ks >> 2) & 1) * Lay::KV_ATOM + (ks & 3) * 32) >> 4;
            const uint32_t kb = ks < 8 ? klo0 : klo1;
            if (ks == 0)
              mma_ss<0>(d, q_lo + qo, DHI, kb + ko, DHI, IDESC_S);
            else
              mma_ss<1>(d, q_lo + qo, DHI, kb + ko, DHI, IDESC_S);
          }
          tc_commit(bar(Lay::B_S + (gr & 1u)));
          tc_commit(bar(Lay::B_EMPTY + slot_of(kt, 0)));
          tc_commit(bar(Lay::B_EMPTY + slot_of(kt, 1)));
        }
        __syncwarp();
      };
      wait_warp(bar(Lay::B_QF), j & 1u, failed);
      if (lane == 0 && !failed) mbar_arrive(bar(Lay::B_QE));
      if (failed) break;
      if (nkt > 0) mma_s(0);
      if (nkt > 1) mma_s(1);
      for (int kt = 0; kt < nkt && !failed; ++kt) {
        const uint32_t gr = ph + kt;
        wait_warp(bar(Lay::B_P + (gr & 1u)), (gr >> 1) & 1u, failed);  // P(kt) is in place
        const uint32_t vs0 = slot_of(kt, 2), vs1 = slot_of(kt, 3);
        wait_warp(bar(Lay::B_FULL + vs0), full_parity(kt, 2), failed);
        wait_warp(bar(Lay::B_FULL + vs1), full_parity(kt, 3), failed);
        if (failed) break;
        const int key0 = r.kv_begin + kt * kKeyTile;
        if (key0 + kKeyTile > r.kv_end) {
          // rows of keys past kv_end may hold anything (even NaN): zero them in both V units
          const int vr0 = r.kv_end - key0;
          const int n = (kKeyTile - vr0) * 16;  // 16 chunks of 16 bytes per row and unit
          for (int i = lane; i < 2 * n; i += 32) {
            const int unit = i / n, ii = i - unit * n;
            const int rr = vr0 + ii / 16, c = ii % 16;
            const uint32_t sV = sRing + (unit ? vs1 : vs0) * Lay::UNIT_BYTES;
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(sV + TL::off(rr, c, TL::KV_ATOM)),
                         "r"(0u)
                         : "memory");
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          tc_fence_after();
          const uint32_t sp = tmem + Tm::SP0 + (gr & 1u) * kKeyTile;
          const uint32_t v0 = v_lo + vs0 * SLOT_STEP, v1 = v_lo + vs1 * SLOT_STEP;
          // P of K step ks at column 8 ks (+ 32 for the second warp's keys)
          auto pcol = [](int ks) { return 8 * ks + (ks >= 4 ? 32 : 0); };
#pragma unroll
          for (int ks = 0; ks < KSTEPS_O; ++ks) {
            const uint32_t vo = (ks * 2048) >> 4;
            const uint32_t a = sp + pcol(ks);
            if (kt == 0 && ks == 0) {  // the unit's first products overwrite O
              mma_ts<0>(tmem + Tm::O, a, v0 + vo, DHI, IDESC_O);
              mma_ts<0>(tmem + Tm::O + 128, a, v1 + vo, DHI, IDESC_O);
            } else {
              mma_ts<1>(tmem + Tm::O, a, v0 + vo, DHI, IDESC_O);
              mma_ts<1>(tmem + Tm::O + 128, a, v1 + vo, DHI, IDESC_O);
            }
          }
          tc_commit(bar(Lay::B_O));
          tc_commit(bar(Lay::B_EMPTY + vs0));
          tc_commit(bar(Lay::B_EMPTY + vs1));
        }
        __syncwarp();
        if (kt + 2 < nkt) mma_s(kt + 2);
      }
      if (failed) break;
      ph += nkt;
      ring0 += LPR * nkt;
    }
  } else if (warp >= kSoftmaxWarp0) {
    // ---------------- softmax: one row per thread, 64 keys of each range per warp ----------------
    const int sw = warp - kSoftmaxWarp0;
    const int quad = sw & 3, part = sw >> 2;
    const int r = quad * 32 + lane;  // row = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t bx1 = bar(Lay::B_X1 + quad), bx2 = bar(Lay::B_X2 + quad);
    volatile float *x_mine = xch + (part * 4 + quad) * 32 + lane;
    volatile float *x_other = xch + ((1 - part) * 4 + quad) * 32 + lane;
    uint32_t nx = 0;
    // my value out, the other warp's value in; x2 (its read of the last
    // exchange) is waited for only before the next write
    auto exchange = [&](float v) -> float {
      if (nx > 0) wait_warp(bx2, (nx - 1) & 1u, failed);
      *x_mine = v;
      mbar_arrive(bx1);
      wait_warp(bx1, nx & 1u, failed);
      const float o = failed ? v : *x_other;
      mbar_arrive(bx2);
      ++nx;
      return o;
    };
    const int g = r % G;
    const int qi = r / G;
    // Q of unit `u`: this warp's 16 rows; returns their factors (lanes 0..15)
    auto load_q = [&](const TileUnit &u) -> float {
      const float mine = load_q_rows<D, G, E>(p, u, 0, quad * 32 + part * 16, lane,
                                              [&](int row, int c) { return sQ + TL::off(row, c, Lay::Q_ATOM); });
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Lay::B_QF));
      return mine;
    };
    // the factors of this warp's 32 rows, from the lanes that stored their Q
    auto row_factors = [&](float mine) -> float {
      const float other = exchange(mine);
      const float own = __shfl_sync(FULL, mine, lane & 15), got = __shfl_sync(FULL, other, lane & 15);
      return (lane >> 4) == part ? own : got;
    };

    uint32_t ph = 0;
    TileUnit cur;
    read_unit(0, cur);
    float rowf = 1.f;  // the row's score factor: 2^e for a scaled bf16 row
    if (!failed && !cur.stop) rowf = row_factors(load_q(cur));
    for (uint32_t j = 0; !failed && !cur.stop; ++j) {
      const int nk = nranges(cur);
      const bool row_valid = qi < cur.npos;
      const int lim = row_valid ? cur.pos0 + qi + 1 : 0;
      float m_used = -INFINITY, l = 0.f;
      for (int kt = 0; kt < nk; ++kt) {
        const uint32_t gr = ph + kt;
        const int ck0 = cur.kv_begin + kt * kKeyTile + part * 64;
        const uint32_t sp = tmem + lane_off + Tm::SP0 + (gr & 1u) * kKeyTile + part * 64;
        wait_warp(bar(Lay::B_S + (gr & 1u)), (gr >> 1) & 1u, failed);
        if (failed) break;
        tc_fence_after();
        uint32_t s0[32], s1[32];
        tmem_ld32x2_wait(sp, s0, s1);
        uint32_t sc = 0;  // block scales: this warp's keys of the range
        float mx;
        const uint32_t fi = gr % Lay::SCALE_SLOTS;
        wait_warp(sc_bar(fi), (gr / Lay::SCALE_SLOTS) & 1u, failed);
        if (failed) break;
        sc = base + Lay::SC_OFF + fi * kScaleSlotBytes + part * 64;
        // (64 keys a warp and range; a row that is none of the tile's is not stored, and needs no mask)
        const bool masked = __any_sync(FULL, row_valid && ck0 + 64 > lim);
        if (masked)
          mx = fmaxf(scaled_max32<GRP, true>(s0, ck0, lim, rowf, sc),
                     scaled_max32<GRP, true>(s1, ck0 + 32, lim, rowf, sc + 32));
        else
          mx = fmaxf(scaled_max32<GRP, false>(s0, ck0, lim, rowf, sc),
                     scaled_max32<GRP, false>(s1, ck0 + 32, lim, rowf, sc + 32));
        const float mo = exchange(mx);
        if (failed) break;
        const float cm = fmaxf(mx, mo);
        const bool grow = cm > -INFINITY && (m_used == -INFINITY || __fsub_rn(cm, m_used) > kRescaleLog2);
        float alpha = 1.f;
        if (grow) {
          alpha = m_used > -INFINITY ? ex2_approx(__fsub_rn(m_used, cm)) : 1.f;
          m_used = cm;
        }
        const float ms = m_used == -INFINITY ? 0.f : m_used;
        float sum = 0.f;
        const bool rare = masked || __any_sync(FULL, fabsf(ms) > 4096.f || rowf != 1.f);
#pragma unroll 1
        for (int ks = 0; ks < 4; ++ks) {
          const float4 c = ld_scales(sc + 16 * ks);
          uint32_t t[16];
          tmem_ld16_wait(sp + 16 * ks, t);
          if (rare)
            probs16_scaled_store<GRP, true>(t, ck0 + 16 * ks, lim, rowf, ms, sum, sp + 8 * ks, c);
          else
            probs16_scaled_store<GRP, false>(t, ck0 + 16 * ks, lim, rowf, ms, sum, sp + 8 * ks, c);
        }
        // O holds P V(0 .. kt-1) once P V(kt-1) completes (S(kt) may have been
        // issued before it): wait for it only when O must be rescaled
        if (kt > 0 && __any_sync(FULL, alpha != 1.f)) {
          wait_warp(bar(Lay::B_O), (gr - 1) & 1u, failed);
          if (failed) break;
          tc_fence_after();
#pragma unroll 1
          for (int ch = part * 4; ch < part * 4 + 4; ++ch) {
            uint32_t t[32];
            tmem_ld32_wait(tmem + lane_off + Tm::O + ch * 32, t);
#pragma unroll
            for (int i = 0; i < 32; ++i) t[i] = __float_as_uint(__uint_as_float(t[i]) * alpha);
            tmem_st32u(tmem + lane_off + Tm::O + ch * 32, t);
          }
        }
        l = l * alpha + sum;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Lay::B_P + (gr & 1u)));
      }
      if (failed) break;
      TileUnit nxt;
      read_unit(j + 1, nxt);
      float next_mine = 1.f;
      if (!failed && !nxt.stop) {
        wait_warp(bar(Lay::B_QE), j & 1u, failed);
        if (!failed) next_mine = load_q(nxt);
      }
      if (failed) break;
      if (nk > 0) {
        const float lt = l + exchange(l);
        wait_warp(bar(Lay::B_O), (ph + nk - 1) & 1u, failed);
        if (failed) break;
        tc_fence_after();
        const float inv = lt != 0.f ? 1.f / lt : 0.f;
        bf16 *dst = p.out + static_cast<int64_t>(cur.row0 + (row_valid ? qi : 0)) * p.num_heads * D +
                    static_cast<int64_t>(cur.kvh * G + g) * D;
        float *pdst = nullptr;  // the row's partial, for a part of the tile's keys
        if (cur.slot >= 0) {
          const int64_t prow = static_cast<int64_t>(cur.slot) * kPrefillTileRows128 + r;
          pdst = p.part_o + prow * D;
          if (part == 0 && row_valid) p.part_lse[prow] = lt != 0.f ? m_used + __log2f(lt) : -INFINITY;
        }
#pragma unroll 1
        for (int ch = part * 4; ch < part * 4 + 4; ++ch) {
          uint32_t t[32];
          tmem_ld32_wait(tmem + lane_off + Tm::O + ch * 32, t);
          if (pdst) {
            if (row_valid) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float *f = reinterpret_cast<const float *>(&t[4 * c]);
                *reinterpret_cast<float4 *>(pdst + ch * 32 + 4 * c) =
                    make_float4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
              }
            }
          } else if (row_valid) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float *f = reinterpret_cast<const float *>(&t[8 * c]);
              const uint4 v = make_uint4(E::pack(f[0] * inv, f[1] * inv), E::pack(f[2] * inv, f[3] * inv),
                                         E::pack(f[4] * inv, f[5] * inv), E::pack(f[6] * inv, f[7] * inv));
              *reinterpret_cast<uint4 *>(dst + ch * 32 + 8 * c) = v;
            }
          }
        }
        tc_fence_before();
      }
      ph += nk;
      if (!nxt.stop) rowf = row_factors(next_mine);
      cur = nxt;
    }
  }

  if (warp == kMmaWarp && lane == 0) {
    tc_commit(bar(Lay::B_DRAIN));
    if (!mbar_wait_bounded(bar(Lay::B_DRAIN), 0, kTcWaitTimeoutNs)) failed = true;
  }
  if (warp == kTmaWarp && lane == 0) {
    const int landed = Lay::B_RAW;
    for (uint32_t g = issued > SLOTS ? issued - SLOTS : 0; g < issued; ++g)
      if (!mbar_wait_bounded(bar(landed + static_cast<int>(g % SLOTS)), (g / SLOTS) & 1u, kTcWaitTimeoutNs))
        failed = true;
  }
  if (failed) flag_error(p.status, PA_FLAG_TIMEOUT);
  griddep_wait();  // the decode kernel before this one has completed
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

template <int D, int G, typename E>
cudaError_t launch_block_tiles(const CUtensorMap &kmap, const CUtensorMap &vmap, const BlockTileParams &tp, int sm_count,
                               cudaStream_t stream) {
  constexpr bool WIDE = D == kWideD;
  int smem = 0, threads = 0;
  void (*kern)(CUtensorMap, CUtensorMap, BlockTileParams) = nullptr;
  if constexpr (WIDE) {
    smem = BlockWideLayout::BYTES;
    threads = kWideThreads;
    kern = tp.block_size >= 16 ? block_tile_wide_kernel<G, E, 16> : block_tile_wide_kernel<G, E, 8>;
  } else {
    smem = BlockLayout<D>::REQUEST;
    threads = kTileThreads8;
    kern = tp.block_size >= 16 ? block_tile_kernel<D, G, E, 16> : block_tile_kernel<D, G, E, 8>;
  }
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (err != cudaSuccess) return err;
  int64_t grid = sm_count;  // one CTA per SM: it holds all of the SM's tensor memory
  const int64_t units = static_cast<int64_t>(tp.max_tiles) * tp.num_kv_heads;
  if (grid > units) grid = units;
  if (grid < 1) grid = 1;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(threads), smem, stream, kmap, vmap, tp);
}

#define PA_TILE_INST1(DD, GG, EE)                                                                                   \
  template cudaError_t launch_block_tiles<DD, GG, EE>(const CUtensorMap &, const CUtensorMap &,                     \
                                                      const BlockTileParams &, int, cudaStream_t);
#define PA_TILE_INST(DD)                                                                                            \
  PA_TILE_INST1(DD, 1, ElemBf16)                                                                                    \
  PA_TILE_INST1(DD, 1, ElemFp16)                                                                                    \
  PA_TILE_INST1(DD, 2, ElemBf16)                                                                                    \
  PA_TILE_INST1(DD, 2, ElemFp16)                                                                                    \
  PA_TILE_INST1(DD, 4, ElemBf16)                                                                                    \
  PA_TILE_INST1(DD, 4, ElemFp16)                                                                                    \
  PA_TILE_INST1(DD, 8, ElemBf16)                                                                                    \
  PA_TILE_INST1(DD, 8, ElemFp16)
PA_TILE_INST(64)
PA_TILE_INST(80)
PA_TILE_INST(96)
PA_TILE_INST(128)
PA_TILE_INST(256)
#undef PA_TILE_INST
#undef PA_TILE_INST1

}  // namespace pa
