// Shared by the tensor-core prefill-tile kernels (sm_103a): shared-memory and
// tensor-memory layouts, descriptors, tcgen05 issue and tensor-memory access.
#pragma once

#include "attention_internal.cuh"

namespace pa {

constexpr int kHalfRows = 128;  // UMMA M: rows per half
constexpr int kHalves = kPrefillTileRows / kHalfRows;
static_assert(kHalves == 2, "the pipeline interleaves exactly two halves");
constexpr int kParts = 2;        // softmax warps per TMEM lane quadrant and half (64 keys of a range each)
constexpr int kKeyTile = 128;    // keys per range (UMMA N of S, K of P V)
constexpr int kMaxSlots = 8;     // K/V ring slots (as many as shared memory holds)
constexpr int kUnitSlots = 2;    // published unit records
// Warp roles. The MMA warp is warp 0: its issue rate sets the tensor cores'
// (they queue only a couple of products) and it shares a scheduler with
// softmax warps; the schedulers favour lower-numbered warps when several are
// ready. Warp 1 loads K/V; warps 2 and 3 widen 8-bit codes (idle otherwise);
// warps 4 .. 19 run the softmax (warp % 4 is their TMEM lane quadrant).
constexpr int kSoftmaxWarps = 4 * kHalves * kParts, kMmaWarp = 0, kTmaWarp = 1, kSoftmaxWarp0 = 4;
constexpr int kTileThreads = 32 * (kSoftmaxWarp0 + kSoftmaxWarps);
// 8-bit caches: two more warps widen each staged range to fp16 in place.
constexpr int kConvWarp = 2, kConvWarps = 2;
constexpr int kTileThreads8 = kTileThreads;
constexpr int kRawBoxRows = 32;  // 8-bit boxes: min(block_size, 32) rows
constexpr uint64_t kTcWaitTimeoutNs = 2000000000;
constexpr uint32_t kTmemCols = 512;

// Tensor memory columns of half A: the score buffer SP [0, 128) and O
// [128, 128 + D); half B's are the same plus HALF. SP holds S (fp32, column
// = key) and then P. With P as a bf16 hi + lo pair, the 16 keys of UMMA K
// step k occupy columns [16k, 16k + 16) (8 columns of hi pairs, then 8 of lo
// pairs); with one 16-bit P per key, K step k occupies 8 columns at 8k for
// k < 4 and at 8k + 32 for k >= 4, so that each softmax warp's probabilities
// stay inside the 64 score columns it reads (the other warp of its row may
// still be reading its own).
template <int D>
struct TcTmem {
  static constexpr uint32_t SP = 0, O = kKeyTile;
  static constexpr uint32_t HALF = kTmemCols / kHalves;
  static_assert(O + D <= HALF, "a half's columns must fit its share of TMEM");
};

template <int D>
struct TcLayout {
  // 64-element swizzle atoms along D; head_dim 80 or 96 is padded to two, the
  // columns past it zero-filled by TMA (K, V) and never read (Q)
  static constexpr int ATOMS = (D + 63) / 64;
  static constexpr int Q_ATOM = kHalfRows * 128;   // 128 rows x 128 B
  static constexpr int KV_ATOM = kKeyTile * 128;   // 128 keys x 128 B
  static constexpr int Q_BYTES = ATOMS * Q_ATOM;   // Q of one half
  static constexpr int KV_BYTES = ATOMS * KV_ATOM;             // one K or V range: a ring slot
  // mbarriers (8 bytes each): per ring slot full, empty, raw (8-bit codes
  // landed; bf16 caches: V range g % kMaxSlots put back to bf16) and conv
  // (8-bit caches: both converter warps hold a slot's codes; bf16 caches: V
  // range g % kMaxSlots rewritten); per half s
  // (S complete), p (P written), o (P V complete), qf (Q stored), qe (the MMA
  // warp has seen qf); per unit slot uf (record published), ue (record read);
  // per (half, lane quadrant) the softmax pair's exchange; drain
  static constexpr int B_FULL = 0, B_EMPTY = kMaxSlots, B_RAW = 2 * kMaxSlots, B_CONV = 3 * kMaxSlots;
  static constexpr int B_S = 4 * kMaxSlots, B_P = B_S + kHalves, B_O = B_P + kHalves, B_QF = B_O + kHalves;
  static constexpr int B_QE = B_QF + kHalves, B_UF = B_QE + kHalves, B_UE = B_UF + kUnitSlots;
  static constexpr int B_X = B_UE + kUnitSlots, B_DRAIN = B_X + 4 * kHalves, NBARS = B_DRAIN + 1;
  static constexpr int XCH_BYTES = kHalves * kParts * kHalfRows * 4;  // one float per (half, part, row)
  static constexpr int UNIT_BYTES = kUnitSlots * 32;                  // records of eight ints
  static constexpr int VF_BYTES = kMaxSlots * 8;                      // per V range and converter warp: kept bf16
  static constexpr int FIXED = kHalves * Q_BYTES + XCH_BYTES + UNIT_BYTES + VF_BYTES + 8 * NBARS + 16;
  static constexpr int FIT = (227 * 1024 - FIXED) / KV_BYTES;
  static constexpr int SLOTS = FIT < kMaxSlots ? FIT : kMaxSlots;
  static_assert(SLOTS >= 4, "the ring holds at least K and V of two ranges");
  static constexpr int Q_OFF = 0;                                // Q of halves A and B
  static constexpr int RING_OFF = Q_OFF + kHalves * Q_BYTES;     // K(0), V(0), K(1), V(1), ... in SLOTS slots
  static constexpr int XCH_OFF = RING_OFF + SLOTS * KV_BYTES;    // the softmax pairs' exchange
  static constexpr int UNIT_OFF = XCH_OFF + XCH_BYTES;           // unit records
  static constexpr int VF_OFF = UNIT_OFF + UNIT_BYTES;           // V range flags (bf16 V rewritten as fp16)
  static constexpr int BAR_OFF = VF_OFF + VF_BYTES;
  static constexpr int TMEM_OFF = BAR_OFF + 8 * NBARS;
  static constexpr int BYTES = TMEM_OFF + 16;
  // Shared memory requested per CTA: more than half an SM's, so that a second
  // CTA (which would wait for TMEM) never lands on the same SM.
  static constexpr int REQUEST = BYTES > 116 * 1024 ? BYTES : 116 * 1024;
  // byte offset of 16-byte chunk c of row r in a swizzled tile with `atom` bytes per atom column
  static __device__ __forceinline__ uint32_t off(int r, int c, int atom) {
    return (c >> 3) * atom + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  }
};
static_assert(TcLayout<128>::BYTES <= 227 * 1024, "shared memory of one CTA");
static_assert(TcLayout<128>::SLOTS >= 5, "loads run two ranges ahead at head_dim 128");

// Bounded wait by a whole warp; the outcome is made warp-uniform, so a warp
// that gives up leaves its loops together (no lane is left inside a
// warp-collective instruction). A warp waits out at most one timeout.
__device__ __forceinline__ void wait_warp(uint32_t bar, uint32_t parity, bool &failed) {
  if (!failed) failed = !mbar_wait_bounded(bar, parity, kTcWaitTimeoutNs);
  failed = __any_sync(0xffffffffu, failed);
}

// The two 32-bit words of a 128-byte-swizzle shared-memory descriptor (the
// layout sw128_desc builds). The low word holds the start address >> 4 in
// bits 0-13, so a tile's descriptors differ from its first one by adding the
// byte offset >> 4 to the low word (shared addresses stay below 256 KB: no
// carry out of the field). Building them once per unit keeps the issuing
// thread at two additions per MMA: it shares its scheduler with two softmax
// warps, and the tensor core queues only a couple of instructions.
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr, uint32_t lbo) {
  return ((smem_addr & 0x3FFFFu) >> 4) | (((lbo >> 4) & 0x3FFFu) << 16);
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) {
  return ((sbo >> 4) & 0x3FFFu) | (1u << 14) | (2u << 29);  // SBO, version (bit 46), 128-byte swizzle (61-63)
}
// D[tmem] (+)= A[smem] * B[smem] with descriptors given as words; ACC = 0 overwrites D.
template <int ACC>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n mov.b64 a, {%1, %2};\n"
      " mov.b64 b, {%3, %4};\n tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(ACC)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem].
template <int ACC>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(ACC)
      : "memory");
}

// 32 consecutive 32-bit columns of this thread's TMEM lane; the wait is in
// the same statement, so no use of the registers can be scheduled before it.
__device__ __forceinline__ void tmem_ld32_wait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// The same for 16 columns.
__device__ __forceinline__ void tmem_ld16_wait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Packed pairs of fp32 operations (one instruction for two lanes of data).
__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float &d0, float &d1, float a0, float a1, float b0, float b1) {
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void sub2(float &d0, float &d1, float a0, float a1, float b0, float b1) {
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n sub.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Row maximum of 32 raw scores, key ck0 + i visible while ck0 + i < lim.
__device__ __forceinline__ float masked_max32(const uint32_t (&s)[32], int ck0, int lim) {
  float m = -INFINITY;
  if (ck0 + 32 <= lim) {
    // a tree of depth 4 (a chain of 16 three-input maxima would be 16 deep)
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      t[i] = max3(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1]),
                  fmaxf(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])));
    m = max3(max3(t[0], t[1], t[2]), max3(t[3], t[4], t[5]), fmaxf(t[6], t[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) m = ck0 + i < lim ? fmaxf(m, __uint_as_float(s[i])) : m;
  }
  return m;
}

// Store 8 32-bit columns (raw bits) of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(taddr), "r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

// Two 32-column loads of this thread's TMEM lane, then one wait.
__device__ __forceinline__ void tmem_ld32x2_wait(uint32_t taddr, uint32_t (&a)[32], uint32_t (&b)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]), "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]), "=r"(a[24]), "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31])
      : "r"(taddr)
      : "memory");
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15]), "=r"(b[16]), "=r"(b[17]), "=r"(b[18]), "=r"(b[19]), "=r"(b[20]), "=r"(b[21]), "=r"(b[22]), "=r"(b[23]), "=r"(b[24]), "=r"(b[25]), "=r"(b[26]), "=r"(b[27]), "=r"(b[28]), "=r"(b[29]), "=r"(b[30]), "=r"(b[31])
      : "r"(taddr + 32)
      : "memory");
}

}  // namespace pa
