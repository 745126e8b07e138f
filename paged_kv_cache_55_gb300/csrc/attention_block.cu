// Attention over 8-bit caches with a scale per (block, KV head): planning,
// split-KV decode and the log-sum-exp merge. Chunked-prefill requests go to
// the tensor-core tiles of attention_block_prefill.cu.
//
// The mathematics. With x_j = scale q.Kc_j ks_j log2 e + log2 vs_j (ks_j, vs_j
// the scales of key j's block) and any reference m,
//   P'_j = 2^(x_j - m),  O = sum_j P'_j Vc_j,  l = sum_j P'_j / vs_j,  out = O / l,
// since P'_j / vs_j = 2^(scale q.K_j log2 e - m) is the plain softmax weight.
// Folding vs into the exponent keeps P' within the fp16 operand's range
// whatever the scales are, with one maximum and one exponent per score.
//
// The decode kernel is bound by HBM: a key costs 2 D bytes per KV head. Its
// work units are (request, KV head, run of 32-key tiles); a unit's 8 columns
// are the (query row, head of the GQA group) pairs, so each byte is read once.
// Every warp is an independent pipeline (own TMA ring, no CTA barrier), takes
// units from a queue, and computes S^T[16 keys x 8 columns] = K Q^T and
// O^T += V^T P^T with m16n8k16 fp16 products, codes widened exactly in
// registers, one fp16 P' per key (11 bits: a weight moves by at most 2^-11 of
// itself). What it does per tile was cut to what the 32 keys need:
//   * the reference m is only moved when a score exceeds it by 2^8 (a warp
//     vote; P' then stays below 2^8 <= fp16's range), so most tiles reduce no
//     maximum and rescale nothing;
//   * masks only in a unit's last tiles;
//   * K's four codes of a word are used in the order the widening leaves them
//     (q is loaded to match); the transposing 8-bit ldmatrix leaves four keys
//     of one d in a word of V; the rows of S and the keys of P V are permuted
//     (s_key, v_key below) so that P needs no further shuffle, eight rows of a
//     shared-memory phase never meet in a bank, and all keys of a lane in a
//     half tile share one 8-key scale group;
//   * block-table entries are loaded one tile ahead, the boxes of a tile are
//     issued by as many lanes, and its scales travel with it by cp.async on
//     the same mbarrier.
// Measured (256 requests, 32 / 8 heads of 128, 958 MB): a step of 173 to 178
// us; the decode kernel 163 to 167 us under a counter, 5.8 TB/s, and with the
// products taken out 153 us, so what is left is the loads' own rate (2 KB boxes
// of 128-byte rows: 6.3 TB/s) and the end of the step, where warps finish
// unevenly. Tried and not kept: K as E4M3 products of a q split into E4M3 terms (no widening; 5 %
// slower at 256 requests, the same at 8 x 32768), 16-byte cp.async in place of
// TMA (2-4 % slower), units that shrink towards the end of the queue (17 %
// slower: a unit's start and its partial cost more than the tail), 8, 10 and
// 14 warps per SM (2-7 % slower), loading the next unit's record and table
// entries several tiles ahead (no difference).
// The planner sizes units from the step's actual lengths, so that a single
// short request still spreads over the GPU and long ones end together.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <float.h>

#include <mutex>
#include <type_traits>

#include "attention_internal.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kCols = 8;    // (query row, head) columns per unit
constexpr int kTile = 32;   // keys per ring tile
constexpr int kRingBytes = 192 * 1024;
constexpr uint64_t kWaitNs = 2000000000;  // 2 s: a TMA never takes this long
constexpr float kGrowLog2 = 8.f;          // P' <= 2^8 between moves of the reference

// Decode warps per SM: a slot (K and V of one tile) is 2 x 32 rows of 64, 128
// or 256 codes; at head_dim 256 six warps of two slots fill the ring.
constexpr int block_warps(int head_dim) { return head_dim == 256 ? 6 : 12; }
// Warps of the whole GPU that units are sized for. A fixed figure (152 SMs),
// so that the sizing calls need no device query.
constexpr int64_t unit_warps(int head_dim) { return 152 * block_warps(head_dim); }

// Unit size in tiles for `total` tiles (over all KV heads) of `pairs` (request,
// KV head) pairs. A pair has at most one unit that is not full, so units of
// total / (warps - pairs) tiles number at most `warps`: one wave, as long as
// the longest unit. While pairs are few (at most an eighth of the warps) that
// is within 15 % of an even share, and the fewest partials. With many pairs
// the shorter requests leave uneven units anyway: then up to kUnitsPerWarp
// units per warp, of at least kMinUnit tiles, which the queue evens out.
constexpr int kUnitsPerWarp = 6, kMinUnit = 8;
__host__ __device__ inline int64_t unit_tiles(int64_t total, int64_t pairs, int64_t warps) {
  int64_t u;
  if (pairs * 8 <= warps) {
    u = (total + warps - pairs - 1) / (warps - pairs);
  } else {
    const int64_t one = (total + warps - 1) / warps;
    const int64_t low = one < kMinUnit ? one : kMinUnit;
    u = (one + kUnitsPerWarp - 1) / kUnitsPerWarp;
    u = u < low ? low : u;
  }
  return u < 1 ? 1 : u;
}

// Prefill tiles over fewer than 3/4 of the SMs are split over their keys, so
// that no SM idles while others walk a long context: into parts of `ranges`
// 128-key ranges (at least kMinRanges: a unit's start and its partial cost
// about one), few enough for one unit per SM. With t tiles and R ranges in all,
// sum ceil(ranges of a tile / u) <= R / u + t <= SMs / KV heads for u = R /
// (SMs / KV heads - t). Merged like the decode partials.
constexpr int kSplitSms = 152, kMinRanges = 2, kRangeKeys = 128;
constexpr int kNoSplit = 1 << 30;
__host__ __device__ inline int part_items(int num_kv_heads) { return kSplitSms / num_kv_heads; }
__host__ __device__ inline int most_split_tiles(int num_kv_heads) { return part_items(num_kv_heads) * 3 / 4; }
__device__ __forceinline__ int part_ranges(int64_t tiles, int64_t ranges, int num_kv_heads) {
  const int64_t slots = part_items(num_kv_heads);
  const int64_t u = (ranges + slots - tiles - 1) / (slots - tiles);
  return static_cast<int>(u < kMinRanges ? kMinRanges : u);
}

struct PlanParams {
  const int32_t *seq_lens, *query_start_loc;
  int32_t num_seqs, total_q, max_query_len, max_seq_len, max_blocks_per_seq, block_size;
  int32_t num_kv_heads;
  int32_t rows_per_item;  // 8 / G
  int32_t tile_pos;       // query positions per prefill tile
  int32_t max_items, max_tiles, max_part_items;
  int64_t warps;          // unit_warps
  int32_t first_units;    // units the decode warps take without the queue
  int32_t *nparts, *first_full, *rest;  // per request: partitions, item of the first full one, of the partial last (or -1)
  int32_t *counts;                      // items, queue, prefill tiles, their queue
  int4 *items, *tiles;
  unsigned int *status;
};

struct DecodeParams {
  const bf16 *q;
  int64_t q_stride;
  const int32_t *block_tables;
  int32_t max_blocks_per_seq, block_size, block_shift;
  int32_t num_heads, num_kv_heads;
  int64_t num_blocks;
  const float *k_scales, *v_scales;
  float scale_log2;
  bf16 *out;
  const int4 *items;
  int32_t *counts;
  int32_t num_seqs, total_q, max_items;
  float *part_o;    // [max_items][Hkv][8][D]
  float *part_lse;  // [max_items][Hkv][8]
  int32_t tiles_follow;
  unsigned int *status;
};

struct MergeParams {
  const int32_t *query_start_loc, *nparts, *first_full, *rest;
  int32_t num_kv_heads, num_heads, num_seqs, max_items, total_q;
  const float *part_o, *part_lse;
  const int4 *tiles;  // prefill tiles (none launched: tile_items 0)
  const int32_t *tile_count;
  int32_t tile_items;  // that may be parts
  const float *tile_o, *tile_lse;
  bf16 *out;
};

// ---- planning --------------------------------------------------------------

// Exclusive scans of N values over a block of NT threads (at most 1024) with
// one barrier: every warp scans the warps' totals for itself. total: the sums.
// `warp_tot` is this scan's own array.
template <int NT, int N>
__device__ __forceinline__ void block_scan(const unsigned long long (&v)[N], unsigned long long (*warp_tot)[32],
                                           unsigned long long (&before)[N], unsigned long long (&total)[N]) {
  constexpr int NWARP = NT / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long incl[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    incl[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long t = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += t;
    }
    if (lane == 31) warp_tot[k][warp] = incl[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    unsigned long long t = lane < NWARP ? warp_tot[k][lane] : 0;
#pragma unroll
    for (int o = 1; o < NWARP; o <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    total[k] = __shfl_sync(0xffffffffu, t, NWARP - 1);
    const unsigned long long below = __shfl_sync(0xffffffffu, t, warp > 0 ? warp - 1 : 0);
    before[k] = (warp > 0 ? below : 0) + incl[k] - v[k];
  }
}

struct Request {
  int q0, ql, len;
  int key_tiles;  // 32-key tiles of a decode request (0: none)
  int tiles;      // prefill tiles of a longer one
};

__device__ __forceinline__ Request read_request(const PlanParams &p, int b, bool report) {
  Request r;
  r.q0 = ld_cg(p.query_start_loc + b);
  const int q1 = ld_cg(p.query_start_loc + b + 1);
  r.len = ld_cg(p.seq_lens + b);
  r.ql = q1 - r.q0;
  r.key_tiles = r.tiles = 0;
  if (r.q0 < 0 || r.ql < 0 || q1 > p.total_q || (b == 0 && r.q0 != 0)) {
    if (report) flag_error(p.status, PA_FLAG_QUERY_LOC);
    return r;
  }
  if (report && b == p.num_seqs - 1 && q1 != p.total_q) flag_error(p.status, PA_FLAG_QUERY_LOC);
  if (r.len < r.ql || r.len > p.max_seq_len || r.ql > p.max_query_len ||
      r.len > static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size) {
    if (report) flag_error(p.status, PA_FLAG_LENGTHS);
    return r;
  }
  if (r.ql == 0) return r;
  if (r.ql > p.rows_per_item)
    r.tiles = (r.ql + p.tile_pos - 1) / p.tile_pos;
  else
    r.key_tiles = (r.len - 1) / kTile + 1;
  return r;
}

// Index r of the half-open prefix range [pre[r], pre[r + 1]) that holds i (n ranges).
__device__ __forceinline__ int find_range(const int *pre, int n, int i) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    if (pre[lo + half] <= i) {
      lo += half;
      n -= half;
    } else {
      n = half;
    }
  }
  return lo;
}

// One CTA. Sweeps over the requests (one read of the lengths when NT threads
// cover them): the tiles of all decode requests, hence the unit size U, and the
// prefill tiles with their key ranges, hence their parts; the number of full
// units, whose items come first in the queue; then the items, each request's
// key_tiles / U full ones and one of the remainder, written by all threads (a
// thread finds an item's request in the prefix sums).
// Item: {b, first query row, rows, position of the first}, {key begin, key
// end, partition (-1: the whole range), partitions}.
template <int NT>
__global__ void __launch_bounds__(NT) block_plan_kernel(const PlanParams p) {
  constexpr int kCountShift = 40;  // a count above 40 bits of tiles
  constexpr unsigned long long kLow = (1ull << kCountShift) - 1;
  __shared__ unsigned long long sum_tot[3][32], full_tot[1][32], scan_tot[2][32];
  __shared__ int pre_full[NT + 1], pre_tile[NT + 1], s_q0[NT], s_ql[NT], s_len[NT];
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const bool once = p.num_seqs <= NT;
  const bool chunks = p.max_query_len > p.rows_per_item;
  const int most_split = chunks && p.max_part_items > 0 ? most_split_tiles(p.num_kv_heads) : 0;
  auto tile_ranges = [&](int len, int ql, int t) {  // 128-key ranges that tile t of a request walks
    return (len - ql + min((t + 1) * p.tile_pos, ql) - 1) / kRangeKeys + 1;
  };
  Request r{};
  // decode key tiles and, above them, decode requests; prefill tiles; their ranges
  unsigned long long mine[3] = {0, 0, 0}, total[3], unused[3];
  for (int b = tid; b < p.num_seqs; b += NT) {
    r = read_request(p, b, true);
    mine[0] += static_cast<unsigned long long>(r.key_tiles) | (r.key_tiles > 0 ? 1ull << kCountShift : 0);
    mine[1] += r.tiles;
    if (r.tiles <= most_split)
      for (int t = 0; t < r.tiles; ++t) mine[2] += tile_ranges(r.len, r.ql, t);
  }
  block_scan<NT>(mine, sum_tot, unused, total);
  const int64_t U64 = unit_tiles(static_cast<int64_t>(total[0] & kLow) * p.num_kv_heads,
                                 static_cast<int64_t>(total[0] >> kCountShift) * p.num_kv_heads, p.warps);
  const int U = U64 > (1 << 24) ? (1 << 24) : static_cast<int>(U64);
  const int unit_keys = U * kTile;
  int split = kNoSplit;  // ranges per part
  if (total[1] > 0 && total[1] <= static_cast<unsigned long long>(most_split))
    split = part_ranges(static_cast<int64_t>(total[1]), static_cast<int64_t>(total[2]), p.num_kv_heads);
  unsigned long long full_total[1] = {0};
  if (!once) {
    unsigned long long full[1] = {0}, none[1];
    for (int b = tid; b < p.num_seqs; b += NT) full[0] += read_request(p, b, false).key_tiles / U;
    block_scan<NT>(full, full_tot, none, full_total);
  }
  int all_full = static_cast<int>(min(full_total[0], static_cast<unsigned long long>(p.max_items)));
  int carry_full = 0, carry_rest = 0, carry_tile = 0;
  for (int base = 0; base < p.num_seqs; base += NT) {
    const int b = base + tid, n = min(NT, p.num_seqs - base);
    if (!once) {
      r = Request{};
      if (b < p.num_seqs) r = read_request(p, b, false);
    }
    if (b >= p.num_seqs) r = Request{};
    const int full = r.key_tiles / U, rest = r.key_tiles % U ? 1 : 0;
    unsigned long long counts[2], ex2[2], tot2[2];
    counts[0] = static_cast<unsigned long long>(full) | (static_cast<unsigned long long>(rest) << kCountShift);
    counts[1] = r.tiles;
    if (split != kNoSplit) {
      counts[1] = 0;
      for (int t = 0; t < r.tiles; ++t) counts[1] += (tile_ranges(r.len, r.ql, t) + split - 1) / split;
    }
    block_scan<NT>(counts, scan_tot, ex2, tot2);
    const unsigned long long ex = ex2[0], tot = tot2[0], ex_tile = ex2[1], tile_tot = tot2[1];
    if (once) {
      full_total[0] = tot & kLow;
      all_full = static_cast<int>(min(full_total[0], static_cast<unsigned long long>(p.max_items)));
    }
    const int ex_full = static_cast<int>(ex & kLow), n_full = static_cast<int>(tot & kLow);
    const int n_tile = static_cast<int>(tile_tot);
    pre_full[tid] = ex_full;
    pre_tile[tid] = static_cast<int>(ex_tile);
    s_q0[tid] = r.q0;
    s_ql[tid] = r.ql;
    s_len[tid] = r.len;
    if (b < p.num_seqs) {
      const int item = all_full + carry_rest + static_cast<int>(ex >> kCountShift);
      p.nparts[b] = full + rest;
      p.first_full[b] = carry_full + ex_full;
      p.rest[b] = rest ? item : -1;
      if (rest && item < p.max_items) {
        p.items[2 * item] = make_int4(b, r.q0, r.ql, r.len - r.ql);
        p.items[2 * item + 1] = make_int4(full * unit_keys, r.len, full ? full : -1, full + rest);
      }
    }
    __syncthreads();
    for (int i = tid; i < n_full; i += NT) {
      const int item = carry_full + i;
      if (item >= p.max_items) break;
      const int k = find_range(pre_full, n, i), part = i - pre_full[k];
      const int len = s_len[k], np = ((len - 1) / kTile + U) / U;
      p.items[2 * item] = make_int4(base + k, s_q0[k], s_ql[k], len - s_ql[k]);
      p.items[2 * item + 1] =
          make_int4(part * unit_keys, static_cast<int>(min(static_cast<long long>(len), (part + 1LL) * unit_keys)),
                    np > 1 ? part : -1, np);
    }
    for (int i = tid; i < n_tile; i += NT) {
      const int tile = carry_tile + i;
      if (tile >= p.max_tiles) break;
      // a request's last tiles see the most keys: queue them first
      const int k = find_range(pre_tile, n, i);
      const int ql = s_ql[k], len = s_len[k], nt = (ql + p.tile_pos - 1) / p.tile_pos;
      int t = nt - 1, part = i - pre_tile[k], parts = 1;
      if (split == kNoSplit) {
        t -= part;
        part = 0;
      } else {
        for (;; --t) {
          parts = (tile_ranges(len, ql, t) + split - 1) / split;
          if (part < parts || t == 0) break;
          part -= parts;
        }
      }
      const int r0 = t * p.tile_pos, npos = min(p.tile_pos, ql - r0), pos0 = (len - ql) + r0, end = pos0 + npos;
      p.tiles[2 * tile] = make_int4(base + k, s_q0[k] + r0, npos, pos0);
      p.tiles[2 * tile + 1] =
          parts > 1 ? make_int4(part * split * kRangeKeys,
                                static_cast<int>(min(static_cast<long long>(end), (part + 1LL) * split * kRangeKeys)),
                                part, parts)
                    : make_int4(0, end, -1, 1);
    }
    carry_full += n_full;
    carry_rest += static_cast<int>(tot >> kCountShift);
    carry_tile += n_tile;
    __syncthreads();  // the prefix arrays and scan_tot are free for the next sweep
  }
  if (tid == 0) {
    int items = all_full + carry_rest;
    if (static_cast<unsigned long long>(carry_rest) + full_total[0] > static_cast<unsigned long long>(p.max_items)) {
      flag_error(p.status, PA_FLAG_LENGTHS);
      items = p.max_items;
    }
    p.counts[0] = items;
    p.counts[1] = p.first_units;
    p.counts[2] = min(carry_tile, p.max_tiles);
    p.counts[3] = 0;
  }
}

// ---- decode ----------------------------------------------------------------

// A ring tile: 32 rows of D codes, 128-byte swizzle (64-byte at D = 64; rows of
// head_dim 80 and 96 padded to 128, zero-filled by TMA; head_dim 256 two atoms
// of 128 codes, atom after atom): eight consecutive rows read at one 16-byte
// chunk hit eight different bank groups.
template <int D>
struct Geom {
  static constexpr int ROW = D <= 64 ? 64 : 128;
  static constexpr int ATOMS = D > 128 ? D / 128 : 1;
  static constexpr int ATOM_BYTES = kTile * ROW;
  static constexpr int TILE_BYTES = ATOMS * ATOM_BYTES;
  static constexpr int SLOT_BYTES = 2 * TILE_BYTES;  // K then V
  static __device__ __forceinline__ uint32_t off(int r, int c) {
    const uint32_t in_atom = ROW == 128 ? r * 128 + (((c ^ r) & 7) << 4) : r * 64 + (((c ^ (r >> 1)) & 3) << 4);
    return ATOMS == 1 ? in_atom : (c >> 3) * ATOM_BYTES + in_atom;
  }
};

// 4 bytes through L1; src_bytes 0 => zero fill.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src, int src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// One arrival on `bar` (counted in its initial count) once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_mbar_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float ld_shared(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// Two 16 x 16 byte matrices, transposed: matrix i's row r at the address lane
// 16 i + r gives; lane l receives rows 4 (l % 4) .. + 3 of columns l / 4 (r0)
// and l / 4 + 8 (r1) of matrix 0, and the same of matrix 1 in r2, r3.
__device__ __forceinline__ void ldsm_b8_x2_t(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
// Key of a 16-key half that row r of S holds: 0-3, 12-15, 4-7, 8-11. P of rows
// 2t, 2t + 1 and 2t + 8, 2t + 9 (one lane's after the transposition) multiplies
// the four keys that lane's V words hold, so V's row i is key
// s_key(2 (i / 4) + i % 2 + 8 (i / 2 % 2)).
__device__ __forceinline__ int s_key(int r) { return r < 4 ? r : (r < 8 ? r + 8 : r - 4); }
__device__ __forceinline__ int v_key(int i) { return s_key(2 * (i >> 2) + (i & 1) + 8 * ((i >> 1) & 1)); }
// Four codes -> fp16 pairs (c0, c1) and (c2, c3), exactly.
__device__ __forceinline__ void widen_pairs(uint32_t w, uint32_t &p01, uint32_t &p23) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(p01), "=r"(p23)
      : "r"(w));
}

struct Unit {
  int valid, item, b, row0, nrows, pos0, kv_begin, kv_end, part, kvh, kb0, kb1;
};

template <int D, int G, int NWARPS, typename E>
__global__ void __launch_bounds__(NWARPS * 32, 1)
    block_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const DecodeParams p) {
  using T = Geom<D>;
  using M = ElemFp16;                                      // operand type, whatever q is
  constexpr int S = kRingBytes / (NWARPS * T::SLOT_BYTES);  // ring slots per warp
  static_assert(S >= 2, "ring needs at least two slots");
  constexpr int MT = D / 16;
  constexpr int DK = (D + 31) / 32;  // 32-d steps (head_dim 80: the last 16 d are zero)
  constexpr int MQ = 2 * DK;         // 16-d rows of O
  constexpr unsigned FULL = 0xffffffffu;

  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[NWARPS][S];
  // per slot: K scales of the tile's four 8-key groups, then their V scales
  __shared__ __align__(16) float scales[NWARPS][S][8];
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // a slot's phase: lane 0's expect_tx and the eight scale copies
  if (threadIdx.x < NWARPS * S) mbar_init(smem_u32(&bars[0][0] + threadIdx.x), 1 + 8);
  if (threadIdx.x == 0) {
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  fence_mbar_init();
  __syncthreads();
  griddep_wait();  // the plan (and the cache scatter before it) must be complete
  if (p.tiles_follow) griddep_launch_dependents();

  const int Hkv = p.num_kv_heads;
  const int total_units = min(max(ld_cg(p.counts), 0), p.max_items) * Hkv;
  const uint32_t my_ring = ring + warp * S * T::SLOT_BYTES;
  const int bs = p.block_size, shift = p.block_shift;
  const int box_shift = min(shift, 5), box_rows = 1 << box_shift, nbox = kTile >> box_shift;

  auto read_unit = [&](int u) {
    Unit U;
    U.valid = u < total_units;
    U.kb0 = U.kb1 = 0;
    if (!U.valid) return U;
    U.item = u / Hkv;
    U.kvh = u - U.item * Hkv;
    const int4 r0 = ld_cg(p.items + 2 * U.item);
    const int4 r1 = ld_cg(p.items + 2 * U.item + 1);
    U.b = r0.x;
    U.row0 = r0.y;
    U.nrows = r0.z;
    U.pos0 = r0.w;
    U.kv_begin = r1.x;
    U.kv_end = r1.y;
    U.part = r1.z;
    // a record is trusted only inside the bounds the host passed; else the unit is dropped
    const bool sane = U.b >= 0 && U.b < p.num_seqs && U.nrows >= 1 && U.nrows <= kCols / G && U.row0 >= 0 &&
                      U.row0 + U.nrows <= p.total_q && U.kv_begin >= 0 && U.kv_begin % kTile == 0 &&
                      U.kv_begin < U.kv_end && U.kv_end <= static_cast<int64_t>(p.max_blocks_per_seq) * bs;
    if (!sane) {
      if (lane == 0) flag_error(p.status, PA_FLAG_LENGTHS);
      U.nrows = 0;  // nothing is read or written
      U.kv_begin = U.kv_end = 0;
    }
    U.kb0 = U.kv_begin / kTile;
    U.kb1 = (U.kv_end + kTile - 1) / kTile;
    return U;
  };
  // Tickets of the queue are drawn a unit ahead: the atomic's answer is first
  // looked at when the next unit's tiles are to be issued.
  const bool queue = total_units > static_cast<int>(gridDim.x) * NWARPS;
  int ticket = total_units;
  auto draw = [&]() {
    if (queue && lane == 0) ticket = atomicAdd(p.counts + 1, 1);
  };
  auto next_unit = [&]() { return read_unit(queue ? __shfl_sync(FULL, ticket, 0) : total_units); };
  // block-table entry of box `lane` of tile kb (negative: no box)
  auto table_entry = [&](const Unit &U, int kb) {
    const int key = kb * kTile + lane * box_rows;
    return lane < nbox && key < U.kv_end
               ? __ldg(p.block_tables + static_cast<int64_t>(U.b) * p.max_blocks_per_seq + (key >> shift))
               : -1;
  };

  // Units are taken in order: `cur` is computed, the producer may be one unit
  // ahead in `nxt`. phys: table entries of the tile it issues next.
  Unit cur = read_unit(blockIdx.x + warp * gridDim.x);  // the first without the queue
  if (cur.valid) draw();
  Unit nxt;
  nxt.valid = 0;
  bool have_nxt = false, on_nxt = false;
  int p_kb = cur.kb0;
  int phys = cur.kb0 < cur.kb1 ? table_entry(cur, cur.kb0) : -1;
  uint32_t issued = 0, consumed = 0;

  // Stage tile kb of unit U into slot issued % S. Boxes past the unit's end
  // (or of a block id out of range) are read at a negative row: zero fill.
  auto issue = [&](const Unit &U, int kb) {
    const uint32_t slot = issued % S;
    const uint32_t bar = smem_u32(&bars[warp][slot]);
    const uint32_t dst = my_ring + slot * T::SLOT_BYTES + lane * box_rows * T::ROW;
    const int key = kb * kTile + lane * box_rows;  // first key of box `lane`
    const bool have = lane < nbox && key < U.kv_end;
    const bool ok = have && phys >= 0 && phys < p.num_blocks;
    if (have && !ok) flag_error(p.status, PA_FLAG_BLOCK_RANGE);
    const int z = ok ? (phys << shift) + (key & (bs - 1)) : -box_rows;
    const int page = ok ? phys : -1;
    if (lane == 0) mbar_arrive_expect_tx(bar, T::SLOT_BYTES);
    // scale of group lane % 4: K's in lanes 0-3, V's in 4-7
    const int gpage = __shfl_sync(FULL, page, ((lane & 3) * 8) >> box_shift);
    if (lane < 8) {
      const bool in = gpage >= 0 && kb * kTile + (lane & 3) * 8 < U.kv_end;
      const float *src = (lane < 4 ? p.k_scales : p.v_scales) + (in ? static_cast<int64_t>(gpage) * Hkv + U.kvh : 0);
      cp_async_4(smem_u32(&scales[warp][slot][lane]), src, in ? 4 : 0);
      cp_async_mbar_arrive(bar);
    }
    if (lane < nbox) {
#pragma unroll
      for (int a = 0; a < T::ATOMS; ++a) {
        tma_load_3d(dst + a * T::ATOM_BYTES, &kmap, bar, a * 128, U.kvh, z);
        tma_load_3d(dst + T::TILE_BYTES + a * T::ATOM_BYTES, &vmap, bar, a * 128, U.kvh, z);
      }
    }
    ++issued;
  };
  // Issue tiles (cur's, then nxt's) while fewer than `limit` are issued.
  auto produce = [&](uint32_t limit) {
    while (issued < limit) {
      if (!on_nxt && p_kb >= cur.kb1) {
        nxt = next_unit();
        have_nxt = true;
        on_nxt = true;
        p_kb = nxt.kb0;
        phys = nxt.kb0 < nxt.kb1 ? table_entry(nxt, nxt.kb0) : -1;
      }
      const Unit &U = on_nxt ? nxt : cur;
      if (p_kb >= U.kb1) break;  // at most one unit ahead
      issue(U, p_kb);
      ++p_kb;
      if (p_kb < U.kb1) phys = table_entry(U, p_kb);
    }
  };

  // ldmatrix rows of a half tile: K's (S rows lane % 16), V's (V rows lane % 16)
  const int krow = s_key(lane & 15), vrow = v_key(lane & 15);
  const int grp = lane >> 4;                           // 8-key scale group of the lane's keys within a half
  const int key_a = s_key(lane >> 2), key_b = s_key((lane >> 2) + 8);  // the lane's two keys of a half

  while (cur.valid) {
    // ---- q fragments (B operand of S^T = K Q^T): k step kk pairs d = 16 kk + 4 (lane % 4) + (0, 1) and (2, 3) ----
    uint32_t qf[MQ][2];
    float col_scale[2] = {p.scale_log2, p.scale_log2};
    {
      const int n = lane >> 2, qi = n / G, g = n % G;
      const bool ok = qi < cur.nrows;
      const bf16 *qp = p.q + static_cast<int64_t>(cur.row0 + (ok ? qi : 0)) * p.q_stride +
                       static_cast<int64_t>(cur.kvh * G + g) * D + 4 * (lane & 3);
#pragma unroll
      for (int kk = 0; kk < MQ; ++kk) {
        const bool in = ok && kk < MT;
        qf[kk][0] = in ? __ldg(reinterpret_cast<const uint32_t *>(qp + 16 * kk)) : 0u;
        qf[kk][1] = in ? __ldg(reinterpret_cast<const uint32_t *>(qp + 16 * kk + 2)) : 0u;
      }
      if constexpr (std::is_same<E, ElemBf16>::value) {
        // bf16 -> fp16: a column whose largest |q| reaches 2^15 is first scaled
        // by 2^-e into [2^14, 2^15), its scores back by 2^e; every value of at
        // least 2^-17 times the column's scale then converts exactly.
        float amax = 0.f;
#pragma unroll
        for (int kk = 0; kk < MQ; ++kk)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            amax = fmaxf(amax, fmaxf(fabsf(ElemBf16::lo(qf[kk][h])), fabsf(ElemBf16::hi(qf[kk][h]))));
        amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 2));
        const int ex = static_cast<int>((__float_as_uint(amax) >> 23) & 0xffu) - 127;
        const int e = ex >= 15 ? min(ex - 14, 120) : 0;
        const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int kk = 0; kk < MQ; ++kk)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            qf[kk][h] = ElemFp16::pack(ElemBf16::lo(qf[kk][h]) * f, ElemBf16::hi(qf[kk][h]) * f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // accumulator column 2 (lane % 4) + j
          const int ec = __shfl_sync(FULL, e, 4 * (2 * (lane & 3) + j));
          col_scale[j] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + ec) << 23);
        }
      }
    }
    int lim[2];  // keys j < lim[e] are visible to accumulator column 2 (lane % 4) + e
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int qi = (2 * (lane & 3) + e) / G;
      lim[e] = min(cur.pos0 + qi + 1, cur.kv_end);
    }
    const int all_see = min(cur.pos0 + 1, cur.kv_end);  // keys every column sees
    float o[MQ][4];
#pragma unroll
    for (int mt = 0; mt < MQ; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
    float m[2] = {-FLT_MAX, -FLT_MAX};  // reference exponents
    float l[2] = {0.f, 0.f};

    for (int kb = cur.kb0; kb < cur.kb1; ++kb) {
      produce(consumed + S);
      const uint32_t slot = consumed % S;
      const bool landed = mbar_wait_bounded(smem_u32(&bars[warp][slot]), (consumed / S) & 1u, kWaitNs);
      if (!__all_sync(FULL, landed)) {  // leave together, never with a diverged warp
        if (lane == 0) {
          flag_error(p.status, PA_FLAG_TIMEOUT);
          for (uint32_t g = consumed; g < issued; ++g)  // this warp's loads still in flight
            (void)mbar_wait_bounded(smem_u32(&bars[warp][g % S]), (g / S) & 1u, kWaitNs);
        }
        __syncwarp();
        return;
      }
      const uint32_t kt = my_ring + slot * T::SLOT_BYTES, vt = kt + T::TILE_BYTES;
      const int key0 = kb * kTile;
      if (key0 + kTile > cur.kv_end) {  // rows past the last key may hold anything: zero them in V
        constexpr int CPR = D / 16;
        const int valid = cur.kv_end - key0, n = (kTile - valid) * CPR;
        for (int i = lane; i < n; i += 32)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(vt + T::off(valid + i / CPR, i % CPR)),
                       "r"(0u)
                       : "memory");
        fence_proxy_async_smem();  // before the slot's next TMA fill
        __syncwarp();
      }
      // scores of half h: keys key_a (columns 0, 1) and key_b (2, 3)
      float s[2][4];
      {
        float sb[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[h][i] = sb[h][i] = 0.f;
#pragma unroll
        for (int j = 0; j < DK; ++j) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r0, r1, r2, r3, a0, a1, a2, a3;
            ldsm_x4(kt + h * 16 * T::ROW + T::off(krow, 2 * j + (lane >> 4)), r0, r1, r2, r3);
            widen_pairs(r0, a0, a2);
            widen_pairs(r1, a1, a3);
            M::mma(s[h], a0, a1, a2, a3, qf[2 * j][0], qf[2 * j][1]);
            widen_pairs(r2, a0, a2);
            widen_pairs(r3, a1, a3);
            M::mma(sb[h], a0, a1, a2, a3, qf[2 * j + 1][0], qf[2 * j + 1][1]);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[h][i] += sb[h][i];
      }
      const uint32_t sc = smem_u32(&scales[warp][slot][grp]);
      const float gk[2] = {ld_shared(sc), ld_shared(sc + 8)}, gv[2] = {ld_shared(sc + 16), ld_shared(sc + 24)};
      if (key0 + kTile > all_see) {  // a unit's last tiles: keys some column does not see
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + 16 * h + (i < 2 ? key_a : key_b) >= lim[i & 1]) s[h][i] = -INFINITY;
      }
      // exponents against the references; a group past the last key has scales
      // 0 and its (masked) scores stay -inf
      float e[2][4], factor[2][2], glv[2];
      float top = -INFINITY;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        glv[h] = __log2f(gv[h]);
#pragma unroll
        for (int c = 0; c < 2; ++c) factor[h][c] = gk[h] > 0.f ? col_scale[c] * gk[h] : 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[h][i] = fmaf(s[h][i], factor[h][i & 1], glv[h] - m[i & 1]);
          top = fmaxf(top, e[h][i]);
        }
      }
      if (__any_sync(FULL, top > kGrowLog2)) {
        // move the references to the columns' maxima (lanes of one column agree)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = -INFINITY;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = c; i < 4; i += 2) {
              e[h][i] = __fadd_rn(__fmul_rn(s[h][i], factor[h][c]), glv[h]);
              mx = fmaxf(mx, e[h][i]);
            }
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, off));
          const float mn = fmaxf(m[c], mx);
          const float al = ex2_approx(m[c] - mn);
          m[c] = mn;
          l[c] *= al;
#pragma unroll
          for (int mt = 0; mt < MQ; ++mt) {
            o[mt][c] *= al;
            o[mt][2 + c] *= al;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = c; i < 4; i += 2) e[h][i] = __fsub_rn(e[h][i], mn);
        }
      }
      uint32_t pk[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float inv = gv[h] > 0.f ? __fdividef(1.f, gv[h]) : 0.f;
        const float p0 = ex2_approx(e[h][0]), p1 = ex2_approx(e[h][1]);
        const float p2 = ex2_approx(e[h][2]), p3 = ex2_approx(e[h][3]);
        l[0] = fmaf(p0 + p2, inv, l[0]);
        l[1] = fmaf(p1 + p3, inv, l[1]);
        pk[h][0] = movmatrix_t(M::pack(p0, p1));
        pk[h][1] = movmatrix_t(M::pack(p2, p3));
      }
      // O^T += V^T P^T: rows lane / 4 and lane / 4 + 8 of m tile mt are d = 16 mt + those
#pragma unroll
      for (int j = 0; j < DK; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r0, r1, r2, r3, a0, a1, a2, a3;
          ldsm_b8_x2_t(vt + h * 16 * T::ROW + T::off(vrow, 2 * j + (lane >> 4)), r0, r1, r2, r3);
          widen_pairs(r0, a0, a2);
          widen_pairs(r1, a1, a3);
          M::mma(o[2 * j], a0, a1, a2, a3, pk[h][0], pk[h][1]);
          widen_pairs(r2, a0, a2);
          widen_pairs(r3, a1, a3);
          M::mma(o[2 * j + 1], a0, a1, a2, a3, pk[h][0], pk[h][1]);
        }
      }
      __syncwarp();  // every lane is done with the slot before it is refilled
      ++consumed;
    }

    // ---- epilogue: normalise, write the output or the partial ----
    if (cur.nrows > 0) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l[0] += __shfl_xor_sync(FULL, l[0], off);
        l[1] += __shfl_xor_sync(FULL, l[1], off);
      }
      // (a NaN sum is no empty one: it reaches the output)
      const float inv0 = l[0] != 0.f ? 1.f / l[0] : 0.f;
      const float inv1 = l[1] != 0.f ? 1.f / l[1] : 0.f;
      if (cur.part < 0) {
        const int col = lane >> 2, qi = col / G, g = col % G;
        bf16 *dst = p.out + static_cast<int64_t>(cur.row0 + (qi < cur.nrows ? qi : 0)) * p.num_heads * D +
                    static_cast<int64_t>(cur.kvh * G + g) * D;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          // transposed: lo8 holds d = 16 mt + 2 (lane % 4) + (0, 1) of one column, hi8 those + 8
          const uint32_t lo8 = movmatrix_t(E::pack(o[mt][0] * inv0, o[mt][1] * inv1));
          const uint32_t hi8 = movmatrix_t(E::pack(o[mt][2] * inv0, o[mt][3] * inv1));
          if (qi < cur.nrows) {
            *reinterpret_cast<uint32_t *>(dst + 16 * mt + 2 * (lane & 3)) = lo8;
            *reinterpret_cast<uint32_t *>(dst + 16 * mt + 2 * (lane & 3) + 8) = hi8;
          }
        }
      } else {
        const int64_t base = (static_cast<int64_t>(cur.item) * Hkv + cur.kvh) * kCols;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = 2 * (lane & 3) + c;
          if (col / G < cur.nrows) {
            const float inv = c ? inv1 : inv0;
            float *dst = p.part_o + (base + col) * D + (lane >> 2);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              dst[16 * mt] = o[mt][c] * inv;
              dst[16 * mt + 8] = o[mt][2 + c] * inv;
            }
            if (lane < 4) p.part_lse[base + col] = l[c] != 0.f ? m[c] + __log2f(l[c]) : -INFINITY;
          }
        }
      }
    }

    // ---- the next unit (the producer may already be streaming it) ----
    if (!have_nxt) nxt = next_unit();
    if (!on_nxt) {
      p_kb = nxt.kb0;
      phys = nxt.kb0 < nxt.kb1 ? table_entry(nxt, nxt.kb0) : -1;
    }
    cur = nxt;
    have_nxt = on_nxt = false;
    if (cur.valid) draw();
  }
}

// ---- merge -----------------------------------------------------------------

// One CTA of NW warps per (request, KV head): the used columns (query rows x
// G, at most 8) rounded up to a power of two NC take a warp each, NW / NC warps
// of a column share its partitions in contiguous runs, joined through shared
// memory in order (the same bits every time), or (NC > NW) a warp takes several
// columns. A warp reads eight partitions at a time with a running maximum of
// their log-sum-exps. Sixteen warps when the pairs are few (their partitions
// are then many), four when there are several CTAs per SM anyway.
// A warp's lanes hold EPL outputs each (head_dim 80, 96: the last lanes' unused).
template <int D>
struct Merged {
  static constexpr int EPL = (D + 31) / 32;
  static constexpr bool VEC4 = D % 128 == 0, VEC2 = D == 64;
  float M = -INFINITY, wsum = 0.f, acc[EPL];
  __device__ __forceinline__ Merged() {
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  }
  // partitions [begin, end), J at a time: row at(k) of o and lse; a partition without keys
  // (lse -inf) is left out, whatever its outputs hold
  template <int J, typename At>
  __device__ __forceinline__ void add(int begin, int end, int lane, const float *lse, const float *o, At at) {
    for (int k0 = begin; k0 < end; k0 += J) {
      float lv[J], ov[J][EPL];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int64_t row = at(min(k0 + j, end - 1));
        lv[j] = ld_cg(lse + row);
        const float *src = o + row * D + lane * EPL;
        if constexpr (VEC2) {
          const float2 v = ld_cg(reinterpret_cast<const float2 *>(src));
          ov[j][0] = v.x, ov[j][1] = v.y;
        } else if constexpr (VEC4) {
#pragma unroll
          for (int e = 0; e < EPL; e += 4) {
            const float4 v = ld_cg(reinterpret_cast<const float4 *>(src + e));
            ov[j][e] = v.x, ov[j][e + 1] = v.y, ov[j][e + 2] = v.z, ov[j][e + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < EPL; ++e) ov[j][e] = lane * EPL + e < D ? ld_cg(src + e) : 0.f;
        }
      }
      float Mn = M;
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (k0 + j < end) Mn = fmaxf(Mn, lv[j]);
      const float Ms = Mn == -INFINITY ? 0.f : Mn;
      const float r = ex2_approx(M - Ms);
      wsum *= r;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] *= r;
      M = Mn;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (k0 + j < end && lv[j] != -INFINITY) {
          const float w = ex2_approx(lv[j] - Ms);
          wsum += w;
#pragma unroll
          for (int e = 0; e < EPL; ++e) acc[e] += w * ov[j][e];
        }
      }
    }
  }
  template <typename E>
  __device__ __forceinline__ void store(bf16 *row, int lane) const {
    const float inv = wsum > 0.f ? 1.f / wsum : (wsum == 0.f ? 0.f : wsum);  // NaN stays NaN
    bf16 *dst = row + lane * EPL;
    if constexpr (VEC2) {
      *reinterpret_cast<uint32_t *>(dst) = E::pack(acc[0] * inv, acc[1] * inv);
    } else if constexpr (VEC4) {
#pragma unroll
      for (int e = 0; e < EPL; e += 4)
        *reinterpret_cast<uint2 *>(dst + e) =
            make_uint2(E::pack(acc[e] * inv, acc[e + 1] * inv), E::pack(acc[e + 2] * inv, acc[e + 3] * inv));
    } else {
#pragma unroll
      for (int e = 0; e < EPL; ++e)
        if (lane * EPL + e < D)
          *reinterpret_cast<unsigned short *>(dst + e) =
              static_cast<unsigned short>(E::pack(acc[e] * inv, 0.f) & 0xffffu);
    }
  }
};

// CTAs of NW warps that merge a part's share (half at most) of a split prefill
// tile's rows, up to four rows a warp, so that the parts of 152 SMs fit about
// one wave (7 chunks of 131 over 1500 keys: the step 34.7 us, with two rows a
// warp 35.2, with one 37.5)
template <int D, int NW>
constexpr int kTileMergeCtas = prefill_tile_rows(D) / 8 / NW;

template <int D, int G, typename E, int NW>
__global__ void __launch_bounds__(NW * 32) block_merge_kernel(const MergeParams p) {
  constexpr int EPL = Merged<D>::EPL, CTAS = kTileMergeCtas<D, NW>;
  __shared__ float s_m[NW], s_w[NW], s_acc[NW][32 * EPL];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = p.num_seqs * p.num_kv_heads;
  if (static_cast<int>(blockIdx.x) >= pairs) {
    // a split prefill tile: a warp per row
    const int i = blockIdx.x - pairs, item = i / (p.num_kv_heads * CTAS);
    const int kvh = (i / CTAS) % p.num_kv_heads, rb = i % CTAS;
    if (item >= min(ld_cg(p.tile_count), p.tile_items)) return;
    const int4 r0 = ld_cg(p.tiles + 2 * item), r1 = ld_cg(p.tiles + 2 * item + 1);
    const int row0 = r0.y, npos = r0.z, parts = r1.w;
    constexpr int ROWS = prefill_tile_rows(D);
    // the CTAs of a part take its share of the tile's rows
    const int part = r1.z, first = item - part;
    if (parts <= 1 || part < 0 || part >= parts || first < 0 || first + parts > p.tile_items) return;
    if (row0 < 0 || npos < 1 || npos * G > ROWS || row0 + npos > p.total_q) return;
    const int row_end = npos * G * (part + 1) / parts;
    for (int row = npos * G * part / parts + rb * NW + warp; row < row_end; row += CTAS * NW) {
      Merged<D> m;
      auto at = [&](int k) { return (static_cast<int64_t>(first + k) * p.num_kv_heads + kvh) * ROWS + row; };
      if (parts <= 2)
        m.template add<2>(0, parts, lane, p.tile_lse, p.tile_o, at);
      else
        m.template add<8>(0, parts, lane, p.tile_lse, p.tile_o, at);
      m.template store<E>(p.out + static_cast<int64_t>(row0 + row / G) * p.num_heads * D +
                              static_cast<int64_t>(kvh * G + row % G) * D,
                          lane);
    }
    return;
  }
  const int b = blockIdx.x / p.num_kv_heads, kvh = blockIdx.x - b * p.num_kv_heads;
  const int np = ld_cg(p.nparts + b), full0 = ld_cg(p.first_full + b), rest = ld_cg(p.rest + b);
  const int q0 = ld_cg(p.query_start_loc + b), ql = ld_cg(p.query_start_loc + b + 1) - q0;
  if (np <= 1 || ql < 1 || ql * G > kCols) return;
  const int cols = ql * G;
  const int nc = cols <= 1 ? 1 : (cols <= 2 ? 2 : (cols <= 4 ? 4 : 8));
  const int wc = nc < NW ? nc : NW;  // columns in parallel
  const int sub = warp / wc, subs = NW / wc;
  for (int col0 = 0; col0 < cols; col0 += wc) {
    const int col = col0 + warp % wc;
    Merged<D> m;
    if (col < cols)
      m.template add<8>(np * sub / subs, np * (sub + 1) / subs, lane, p.part_lse, p.part_o, [&](int k) {
        const int item = min(max(k == np - 1 && rest >= 0 ? rest : full0 + k, 0), p.max_items - 1);
        return (static_cast<int64_t>(item) * p.num_kv_heads + kvh) * kCols + col;
      });
    if (subs > 1) {  // then there is one round of columns
      if (lane == 0) {
        s_m[warp] = m.M;
        s_w[warp] = m.wsum;
      }
#pragma unroll
      for (int e = 0; e < EPL; ++e) s_acc[warp][e * 32 + lane] = m.acc[e];
      __syncthreads();
      if (sub > 0) return;
      for (int k = 1; k < subs; ++k) {
        const int w = k * wc + warp;
        const float Mo = s_m[w], Mn = fmaxf(m.M, Mo), Ms = Mn == -INFINITY ? 0.f : Mn;
        const float ra = ex2_approx(m.M - Ms), rb = ex2_approx(Mo - Ms);
        m.wsum = m.wsum * ra + s_w[w] * rb;
#pragma unroll
        for (int e = 0; e < EPL; ++e) m.acc[e] = m.acc[e] * ra + s_acc[w][e * 32 + lane] * rb;
        m.M = Mn;
      }
    }
    if (col < cols)
      m.template store<E>(p.out + static_cast<int64_t>(q0 + col / G) * p.num_heads * D +
                              static_cast<int64_t>(kvh * G + col % G) * D,
                          lane);
  }
}

// ---- host ------------------------------------------------------------------

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, []() {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// 3-D view of one cache of codes, [num_blocks * block_size rows][Hkv][D], with
// a box of min(block_size, 32) rows x 1 head x 64 or 128 codes.
bool encode_map(CUtensorMap *map, const void *cache, int64_t num_blocks, int32_t num_kv_heads, int32_t head_dim,
                int32_t block_size) {
  auto encode = map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(num_kv_heads),
                              static_cast<cuuint64_t>(num_blocks) * block_size};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim),
                                 static_cast<cuuint64_t>(num_kv_heads) * head_dim};
  const cuuint32_t box[3] = {head_dim <= 64 ? 64u : 128u, 1,
                             static_cast<cuuint32_t>(block_size < kTile ? block_size : kTile)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(cache), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE,
                head_dim <= 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int G, typename E>
cudaError_t launch_typed(const AttnLaunch &a, const BlockWorkspace &w, cudaStream_t stream, int *launched) {
  char *ws = static_cast<char *>(a.workspace);
  constexpr int NW = block_warps(D);
  CUtensorMap kmap, vmap;
  if (!encode_map(&kmap, a.key_cache, a.num_blocks, a.num_kv_heads, D, a.block_size) ||
      !encode_map(&vmap, a.value_cache, a.num_blocks, a.num_kv_heads, D, a.block_size))
    return cudaErrorInvalidValue;
  const int64_t units_upper = static_cast<int64_t>(w.max_items) * a.num_kv_heads;
  const int64_t grid = units_upper < a.sm_count ? units_upper : a.sm_count;  // one CTA per SM

  PlanParams pp;
  pp.seq_lens = a.seq_lens;
  pp.query_start_loc = a.query_start_loc;
  pp.num_seqs = a.num_seqs;
  pp.total_q = a.total_q;
  pp.max_query_len = a.max_query_len;
  pp.max_seq_len = a.max_seq_len;
  pp.max_blocks_per_seq = a.max_blocks_per_seq;
  pp.block_size = a.block_size;
  pp.num_kv_heads = a.num_kv_heads;
  pp.rows_per_item = kCols / G;
  pp.tile_pos = prefill_tile_rows(D) / G;
  pp.max_items = w.max_items;
  pp.max_tiles = w.max_tiles;
  pp.max_part_items = w.part_items;
  pp.warps = unit_warps(D);
  pp.first_units = static_cast<int32_t>(grid * NW);
  pp.nparts = reinterpret_cast<int32_t *>(ws + w.nparts);
  pp.first_full = reinterpret_cast<int32_t *>(ws + w.first_full);
  pp.rest = reinterpret_cast<int32_t *>(ws + w.rest);
  pp.counts = reinterpret_cast<int32_t *>(ws + w.counts);
  pp.items = reinterpret_cast<int4 *>(ws + w.items);
  pp.tiles = reinterpret_cast<int4 *>(ws + w.tiles);
  pp.status = a.status;
  cudaError_t err = a.num_seqs <= 256 ? launch_pdl(block_plan_kernel<256>, dim3(1), dim3(256), 0, stream, pp)
                                      : launch_pdl(block_plan_kernel<1024>, dim3(1), dim3(1024), 0, stream, pp);
  if (err != cudaSuccess) return err;
  ++*launched;

  const bool tiles_follow = a.max_query_len > pp.rows_per_item;
  DecodeParams dp;
  dp.q = static_cast<const bf16 *>(a.q);
  dp.q_stride = a.q_stride;
  dp.block_tables = a.block_tables;
  dp.max_blocks_per_seq = a.max_blocks_per_seq;
  dp.block_size = a.block_size;
  dp.block_shift = a.block_size == 8 ? 3 : (a.block_size == 16 ? 4 : 5);
  dp.num_heads = a.num_heads;
  dp.num_kv_heads = a.num_kv_heads;
  dp.num_blocks = a.num_blocks;
  dp.k_scales = a.k_scales;
  dp.v_scales = a.v_scales;
  dp.scale_log2 = a.scale * 1.4426950408889634f;
  dp.out = static_cast<bf16 *>(a.out);
  dp.items = pp.items;
  dp.counts = pp.counts;
  dp.num_seqs = a.num_seqs;
  dp.total_q = a.total_q;
  dp.max_items = w.max_items;
  dp.part_o = reinterpret_cast<float *>(ws + w.part_o);
  dp.part_lse = reinterpret_cast<float *>(ws + w.part_lse);
  dp.tiles_follow = tiles_follow ? 1 : 0;
  dp.status = a.status;
  constexpr int smem = kRingBytes + 1024;  // ring + alignment slack
  auto kern = block_decode_kernel<D, G, NW, E>;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (err != cudaSuccess) return err;
  if (a.ev_start) cudaEventRecord(a.ev_start, stream);
  err = launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(NW * 32), smem, stream, kmap, vmap, dp);
  if (err != cudaSuccess) return err;
  ++*launched;
  if (a.ev_stop) cudaEventRecord(a.ev_stop, stream);

  if (tiles_follow) {  // some request may be a prefill chunk
    BlockTileParams tp;
    tp.q = dp.q;
    tp.q_stride = a.q_stride;
    tp.block_tables = a.block_tables;
    tp.max_blocks_per_seq = a.max_blocks_per_seq;
    tp.block_size = a.block_size;
    tp.block_shift = dp.block_shift;
    tp.num_heads = a.num_heads;
    tp.num_kv_heads = a.num_kv_heads;
    tp.num_blocks = a.num_blocks;
    tp.scale_log2 = dp.scale_log2;
    tp.out_scale = 1.0f;
    tp.out = dp.out;
    tp.tiles = pp.tiles;
    tp.tile_count = pp.counts + 2;
    tp.tile_counter = pp.counts + 3;
    tp.num_seqs = a.num_seqs;
    tp.total_q = a.total_q;
    tp.max_tiles = w.max_tiles;
    tp.k_scales = a.k_scales;
    tp.v_scales = a.v_scales;
    tp.max_part_items = w.part_items;
    tp.part_o = reinterpret_cast<float *>(ws + w.tile_o);
    tp.part_lse = reinterpret_cast<float *>(ws + w.tile_lse);
    tp.status = a.status;
    if (a.tile_start) cudaEventRecord(a.tile_start, stream);
    err = launch_block_tiles<D, G, E>(kmap, vmap, tp, a.sm_count, stream);
    if (err != cudaSuccess) return err;
    if (a.tile_stop) cudaEventRecord(a.tile_stop, stream);
    ++*launched;
  }

  if (a.max_seq_len > kTile) {  // some request may be split
    MergeParams mp;
    mp.query_start_loc = a.query_start_loc;
    mp.nparts = pp.nparts;
    mp.first_full = pp.first_full;
    mp.rest = pp.rest;
    mp.num_kv_heads = a.num_kv_heads;
    mp.num_heads = a.num_heads;
    mp.num_seqs = a.num_seqs;
    mp.max_items = w.max_items;
    mp.total_q = a.total_q;
    mp.tiles = pp.tiles;
    mp.tile_count = pp.counts + 2;
    mp.tile_items = tiles_follow ? w.part_items : 0;
    mp.tile_o = reinterpret_cast<float *>(ws + w.tile_o);
    mp.tile_lse = reinterpret_cast<float *>(ws + w.tile_lse);
    mp.part_o = dp.part_o;
    mp.part_lse = dp.part_lse;
    mp.out = dp.out;
    const unsigned pairs = static_cast<unsigned>(a.num_seqs * a.num_kv_heads);
    const unsigned part_pairs = static_cast<unsigned>(mp.tile_items * a.num_kv_heads);
    if (pairs <= 2u * static_cast<unsigned>(a.sm_count))
      err = launch_pdl(block_merge_kernel<D, G, E, 16>, dim3(pairs + part_pairs * kTileMergeCtas<D, 16>), dim3(16 * 32),
                       0, stream, mp);
    else
      err = launch_pdl(block_merge_kernel<D, G, E, 4>, dim3(pairs + part_pairs * kTileMergeCtas<D, 4>), dim3(4 * 32), 0,
                       stream, mp);
    if (err != cudaSuccess) return err;
    ++*launched;
  }
  return cudaSuccess;
}

}  // namespace

bool block_workspace_layout(int32_t num_seqs, int32_t total_q, int32_t max_query_len, int32_t max_seq_len,
                            int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, BlockWorkspace &w) {
  if (num_seqs < 0 || total_q < 0 || max_seq_len < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      num_heads % num_kv_heads != 0 || num_heads / num_kv_heads > kCols)
    return false;
  const int G = num_heads / num_kv_heads;
  // The most items that unit_tiles leaves (per KV head): one wave of units when
  // pairs are few; else one item more per request than full units, which are
  // those of one wave (units below kMinUnit), or else of kMinUnit tiles at least
  // and kUnitsPerWarp waves at most. Never more than there are tiles.
  const int64_t key_tiles = (static_cast<int64_t>(max_seq_len) + kTile - 1) / kTile;
  const int64_t all_tiles = static_cast<int64_t>(num_seqs) * key_tiles;
  const int64_t warps = unit_warps(head_dim), wave = (warps + num_kv_heads - 1) / num_kv_heads;
  int64_t items = wave;
  if (static_cast<int64_t>(num_seqs) * num_kv_heads * 8 > warps) {
    int64_t full = (kUnitsPerWarp * warps + num_kv_heads - 1) / num_kv_heads;
    if (full > all_tiles / kMinUnit) full = all_tiles / kMinUnit;
    items = num_seqs + (full > wave ? full : wave);
  }
  if (items > all_tiles) items = all_tiles;
  const int rows = prefill_tile_rows(head_dim);
  const int64_t tiles = (static_cast<int64_t>(total_q) * G + rows - 1) / rows + num_seqs;
  if (items * num_kv_heads > (1LL << 30) || tiles * num_kv_heads > (1LL << 30) ||
      static_cast<int64_t>(num_seqs) * num_kv_heads > (1LL << 30))
    return false;
  w.max_items = static_cast<int32_t>(items > 0 ? items : 1);
  // parts of split prefill tiles: at least kMinRanges ranges each; none where the
  // rows that no decode request can hold already make more tiles than are split
  int64_t split_items = 0;
  const int64_t chunk_rows = total_q - static_cast<int64_t>(num_seqs) * (kCols / G);
  if (max_query_len > kCols / G && chunk_rows * G <= static_cast<int64_t>(most_split_tiles(num_kv_heads)) * rows) {
    const int64_t most = (static_cast<int64_t>(max_seq_len) + kMinRanges * kRangeKeys - 1) / (kMinRanges * kRangeKeys);
    split_items = part_items(num_kv_heads);
    if (most <= 1) split_items = 0;
    if (most * tiles < split_items) split_items = most * tiles;
  }
  w.part_items = static_cast<int32_t>(split_items);
  const int64_t tile_items = tiles > split_items ? tiles : split_items;
  w.max_tiles = static_cast<int32_t>(tile_items > 0 ? tile_items : 1);
  const size_t per_seq = align256(sizeof(int32_t) * (static_cast<size_t>(num_seqs) + 1));
  const size_t parts = static_cast<size_t>(w.max_items) * num_kv_heads * kCols;
  size_t off = 0;
  w.counts = off;     off += 256;
  w.nparts = off;     off += per_seq;
  w.first_full = off; off += per_seq;
  w.rest = off;       off += per_seq;
  w.items = off;      off += align256(sizeof(int4) * 2 * static_cast<size_t>(w.max_items));
  w.tiles = off;      off += align256(sizeof(int4) * 2 * static_cast<size_t>(w.max_tiles));
  w.part_lse = off;   off += align256(sizeof(float) * parts);
  w.part_o = off;     off += align256(sizeof(float) * parts * head_dim);
  const size_t tile_rows = static_cast<size_t>(split_items) * num_kv_heads * rows;
  w.tile_lse = off;   off += align256(sizeof(float) * tile_rows);
  w.tile_o = off;     off += align256(sizeof(float) * tile_rows * head_dim);
  w.total = off;
  return true;
}

cudaError_t launch_block_attention(const AttnLaunch &a, cudaStream_t stream, int *launched) {
  BlockWorkspace w;
  if (!block_workspace_layout(a.num_seqs, a.total_q, a.max_query_len, a.max_seq_len, a.num_heads, a.num_kv_heads,
                              a.head_dim, w))
    return cudaErrorInvalidValue;
  const int G = a.num_heads / a.num_kv_heads;
#define PA_DISPATCH(DD, GG)                                                               \
  if (a.head_dim == DD && G == GG)                                                        \
    return a.dtype == PA_FP16 ? launch_typed<DD, GG, ElemFp16>(a, w, stream, launched)    \
                              : launch_typed<DD, GG, ElemBf16>(a, w, stream, launched);
  PA_DISPATCH(128, 1) PA_DISPATCH(128, 2) PA_DISPATCH(128, 4) PA_DISPATCH(128, 8)
  PA_DISPATCH(64, 1) PA_DISPATCH(64, 2) PA_DISPATCH(64, 4) PA_DISPATCH(64, 8)
  PA_DISPATCH(96, 1) PA_DISPATCH(96, 2) PA_DISPATCH(96, 4) PA_DISPATCH(96, 8)
  PA_DISPATCH(80, 1) PA_DISPATCH(80, 2) PA_DISPATCH(80, 4) PA_DISPATCH(80, 8)
  PA_DISPATCH(256, 1) PA_DISPATCH(256, 2) PA_DISPATCH(256, 4) PA_DISPATCH(256, 8)
#undef PA_DISPATCH
  return cudaErrorInvalidValue;
}

}  // namespace pa
