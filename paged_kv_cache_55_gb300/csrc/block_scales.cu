// 8-bit caches with one scale per (block, KV head): the quantising scatter and
// the copy of scales that goes with a copy-on-write block copy.
//
// A block of one KV head holds E4M3 codes whose values are code * scale, the
// scale a power of two: 2^e with the smallest e >= -64 for which the largest
// finite magnitude written does not exceed 448 * 2^e. Rows are appended to a
// block over several steps, so a block that already holds rows of its request
// keeps the larger of its scale and the one the new rows need; when it grows,
// the codes already there are rewritten under the new scale (code * old / new,
// a shift of the exponent, exact until it reaches the format's subnormals). A
// block whose first row is written takes the scale its new rows need, whatever
// the array held.
//
// A (block, KV head) is owned by one warp for the whole call, so its largest
// magnitude, its old codes and its scale are read and written without
// synchronisation. Ownership follows the block table: request b appends rows
// [ctx, seq_len) and touches blocks ctx / bs .. (seq_len - 1) / bs of its row.
// The kernel reads 2 bytes and writes 1 byte per element: HBM-bound for
// chunks, launch and load latency (lengths -> table -> scale) for decode steps.
#include "cache_write.cuh"
#include "pa_common.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

// Warps per CTA, at most: a lane holds its NV chunks of a block in registers
constexpr int scatter_chunks(int head_dim, int block_size) { return (block_size * head_dim / 8 + 31) / 32; }
constexpr int scatter_warps(int head_dim, int block_size) { return scatter_chunks(head_dim, block_size) > 8 ? 8 : 16; }
constexpr int kMinScaleExp = -64;

// Largest finite magnitude of a 16-bit pair, bit pattern per half (magnitudes
// order like their bits); infinities and NaN count as zero.
template <typename E>
__device__ __forceinline__ uint32_t finite_magnitudes(uint32_t w) {
  constexpr uint32_t kInf2 = E::kUmmaFormat ? 0x7F807F80u : 0x7C007C00u;  // bf16, fp16
  const uint32_t a = w & 0x7FFF7FFFu;
  return a & ~__vcmpgeu2(a, kInf2);
}

// The scale for a largest magnitude `amax` (>= 0, finite): amax = m * 2^x with
// m in [1, 2) needs e = x - 8, one more when m > 1.75 (448 = 1.75 * 2^8).
__device__ __forceinline__ float needed_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, kMinScaleExp);  // amax 0 (and fp32 subnormals) land here
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Four codes under another scale: E4M3(code * ratio); NaN stays NaN.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t h0, h1;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(h0), "=r"(h1)
      : "r"(w));
  const uint32_t p0 = e4m3x2_from_f32(ElemFp16::lo(h0) * ratio, ElemFp16::hi(h0) * ratio);
  const uint32_t p1 = e4m3x2_from_f32(ElemFp16::lo(h1) * ratio, ElemFp16::hi(h1) * ratio);
  return p0 | (p1 << 16);
}

// Eight elements times a factor, as E4M3 codes.
template <typename E>
__device__ __forceinline__ uint2 quantize8_times(uint4 a, float factor) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w};
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) c[k] = e4m3x2_from_f32(E::lo(x[k]) * factor, E::hi(x[k]) * factor);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// A unit: one touched block of a request. Units are numbered so that a unit's
// request can be found: request b's are [start(b), start(b + 1)) with start(b) =
// query_start_loc[b] / bs + 2 b, as n > 0 rows touch at most n / bs + 2 blocks
// (the ones past its last touched block are empty). In steps of one-token
// requests unit u is request u.
struct ScatterUnit {
  int phys, row0, rows, token0;  // block, its first new row, new rows (0: nothing to do), their first token
};

constexpr int kUnitBatch = 16;  // units looked up at a time, one per warp where there are as many

// The unit's request and block, found by a warp together (the same result in
// every lane); errors that only the device sees are flagged.
template <int BS>
__device__ __forceinline__ ScatterUnit find_unit(const BlockScatterLaunch &p, bool single, int u, int lane) {
  constexpr int SHIFT = BS == 8 ? 3 : (BS == 16 ? 4 : 5);
  ScatterUnit r{0, 0, 0, 0};
  int b = u;
  if (!single) {  // the largest b with start(b) <= u: every lane probes one of 32 equal steps
    b = 0;
    for (int n = p.num_seqs; n > 1;) {
      const int step = (n + 31) >> 5, at = lane * step;
      const bool below = at < n && (ld_cg(p.query_start_loc + b + at) >> SHIFT) + 2 * (b + at) <= u;
      const int last = (31 - __clz(__ballot_sync(0xffffffffu, below) | 1)) * step;
      b += last;
      n = min(step, n - last);
    }
  }
  const int q0 = ld_cg(p.query_start_loc + b), q1 = ld_cg(p.query_start_loc + b + 1), len = ld_cg(p.seq_lens + b);
  const int ql = q1 - q0;
  if (q0 < 0 || ql < 0 || q1 > p.total_q || (b == 0 && q0 != 0) || (b == p.num_seqs - 1 && q1 != p.total_q)) {
    flag_error(p.status, PA_FLAG_QUERY_LOC);
    return r;
  }
  if (ql == 0) return r;
  if (len < ql || ql > p.max_query_len || len > static_cast<int64_t>(p.max_blocks_per_seq) * BS) {
    flag_error(p.status, PA_FLAG_LENGTHS);
    return r;
  }
  const int i = single ? 0 : u - ((q0 >> SHIFT) + 2 * b);  // touched block of the request
  const int ctx = len - ql;
  const int64_t first = (static_cast<int64_t>(ctx >> SHIFT) + i) << SHIFT;  // first position of the block
  if (i < 0 || first >= len) return r;
  r.phys = ld_cg(p.block_tables + static_cast<int64_t>(b) * p.max_blocks_per_seq + (first >> SHIFT));
  if (r.phys < 0 || r.phys >= p.num_blocks) {
    flag_error(p.status, PA_FLAG_BLOCK_RANGE);
    return r;
  }
  r.row0 = max(ctx - static_cast<int>(first), 0);
  r.rows = static_cast<int>(min(static_cast<long long>(len) - first, static_cast<long long>(BS))) - r.row0;
  r.token0 = static_cast<int>(q0 + (first + r.row0 - ctx));
  return r;
}

// Items are (unit, K or V, KV head); the resident CTAs take equal runs of them.
// A CTA's warps look its units up together, one unit per warp (lengths, block
// table), then each warp takes items: it loads the block's new rows of its head
// into registers, reduces their largest magnitude, and stores their codes.
// Bound by the latency of the loads of two or three items a warp one after the
// other. Measured (8432 rows of 8 heads of 128 in blocks of 16, 52 MB): 17.6 us;
// with one CTA per unit, which looks its unit up by itself, 21.6 us.
template <int D, int BS, typename E>
__global__ void __launch_bounds__(scatter_warps(D, BS) * 32, 2)
    block_scatter_kernel(const BlockScatterLaunch p, int units, uint64_t per_cta, uint32_t extra) {
  constexpr int CPR = D / 8;                   // 8-element chunks per row
  constexpr int NV = scatter_chunks(D, BS);    // chunks per lane, at most
  __shared__ ScatterUnit s_unit[kUnitBatch];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const bool single = p.max_query_len <= 1;
  const int64_t row8 = static_cast<int64_t>(p.num_kv_heads) * CPR;  // 8-code vectors per cache row
  const uint32_t pairs = 2 * p.num_kv_heads;
  // this CTA's items: `per_cta`, one more in the first `extra` CTAs
  const uint64_t i_begin = per_cta * blockIdx.x + min(blockIdx.x, extra);
  const uint64_t i_end = i_begin + per_cta + (blockIdx.x < extra ? 1 : 0);

  for (uint64_t i0 = i_begin; i0 < i_end;) {
    const int u0 = i0 >> 32 ? static_cast<int>(i0 / pairs) : static_cast<int>(static_cast<uint32_t>(i0) / pairs);
    const int r0 = static_cast<int>(i0 - static_cast<uint64_t>(u0) * pairs);
    const int n_units = min(units - u0, kUnitBatch);
    const int n_items = static_cast<int>(min(i_end - i0, static_cast<uint64_t>(n_units) * pairs - r0));
    if (i0 > i_begin) __syncthreads();  // the last batch's units have been read
    for (int i = warp; i * pairs < n_items + r0; i += warps) {
      const ScatterUnit unit = find_unit<BS>(p, single, u0 + i, lane);
      if (lane == 0) s_unit[i] = unit;
    }
    __syncthreads();
    i0 += n_items;
    for (int item = r0 + warp; item < r0 + n_items; item += warps) {
      const int at_unit = static_cast<uint32_t>(item) / pairs, r = item - at_unit * pairs;
      const ScatterUnit unit = s_unit[at_unit];
      if (unit.rows <= 0) continue;
      const int phys = unit.phys, row0 = unit.row0, n = unit.rows * CPR;
      const int64_t token0 = unit.token0;
      const bool is_v = r >= p.num_kv_heads;
      const int kvh = is_v ? r - p.num_kv_heads : r;
      const int64_t stride8 = (is_v ? p.value_stride : p.key_stride) / 8;
      const uint4 *src = static_cast<const uint4 *>(is_v ? p.value : p.key) + token0 * stride8 +
                         static_cast<int64_t>(kvh) * CPR;
      float *scale_at = (is_v ? p.v_scales : p.k_scales) + static_cast<int64_t>(phys) * p.num_kv_heads + kvh;
      float before = row0 > 0 ? ld_cg(scale_at) : 0.f;
      uint4 x[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int k = lane + 32 * j, row = k / CPR, c = k % CPR;
        x[j] = make_uint4(0u, 0u, 0u, 0u);
        if (k < n) x[j] = ld_cg(src + row * stride8 + c);
      }
      uint32_t m2 = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (32 * j >= n) break;
        m2 = __vimax3_u16x2(m2, x[j].x & 0x7FFF7FFFu, x[j].y & 0x7FFF7FFFu);
        m2 = __vimax3_u16x2(m2, x[j].z & 0x7FFF7FFFu, x[j].w & 0x7FFF7FFFu);
      }
      uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
      if (m >= (E::kUmmaFormat ? 0x7F80u : 0x7C00u)) {  // an infinity or NaN among them: the finite ones alone
        m2 = 0;
#pragma unroll 1
        for (int j = 0; j < NV; ++j) {
          const int k = lane + 32 * j;
          if (k < n) {
            const uint4 v = ld_cg(src + k / CPR * stride8 + k % CPR);
            m2 = __vmaxu2(m2, __vmaxu2(finite_magnitudes<E>(v.x), finite_magnitudes<E>(v.y)));
            m2 = __vmaxu2(m2, __vmaxu2(finite_magnitudes<E>(v.z), finite_magnitudes<E>(v.w)));
          }
        }
        m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
      }
      // a scale that is no positive finite number (never written) counts as 0
      if (!(before > 0.f && before <= 3.4028234e38f)) before = 0.f;
      const float after = fmaxf(before, needed_scale(E::lo(m)));
      uint2 *dst = static_cast<uint2 *>(is_v ? p.value_cache : p.key_cache) + static_cast<int64_t>(phys) * BS * row8 +
                   static_cast<int64_t>(kvh) * CPR;
      if ((__float_as_uint(after) & 0x7FFFFFu) == 0) {
        // a power of two divides by its inverse, exactly
        const float inverse = 1.f / after;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (32 * j >= n) break;
          const int k = lane + 32 * j, row = k / CPR, c = k % CPR;
          if (k < n) dst[(row0 + row) * row8 + c] = quantize8_times<E>(x[j], inverse);
        }
      } else {  // a scale the cache came with
#pragma unroll 1
        for (int k = lane; k < n; k += 32)
          dst[(row0 + k / CPR) * row8 + k % CPR] = quantize8<E>(ld_cg(src + k / CPR * stride8 + k % CPR), after);
      }
      if (row0 > 0 && after != before) {  // the rows already there, under the larger scale
        const float ratio = before / after;
        for (int k = lane; k < row0 * CPR; k += 32) {
          uint2 *at = dst + (k / CPR) * row8 + k % CPR;
          const uint2 v = *at;
          *at = make_uint2(rescale4(v.x, ratio), rescale4(v.y, ratio));
        }
      }
      if (lane == 0) *scale_at = after;
    }
  }
}

template <int D, int BS, typename E>
cudaError_t launch_scatter(const BlockScatterLaunch &p, int sm_count, cudaStream_t stream) {
  const int64_t units =
      p.max_query_len <= 1 ? p.num_seqs : p.total_q / BS + 2 * static_cast<int64_t>(p.num_seqs);
  constexpr int most = scatter_warps(D, BS);
  const int warps = 2 * p.num_kv_heads < most ? 2 * p.num_kv_heads : most;
  // CTAs that are resident together (at most 64 registers a thread for 16
  // warps, 128 for 8); with fewer units one each
  const int64_t slots = static_cast<int64_t>(sm_count) * (32 / warps < 16 ? 32 / warps : 16);
  const uint64_t ctas = units < slots ? units : slots, items = static_cast<uint64_t>(units) * 2 * p.num_kv_heads;
  return launch_pdl(block_scatter_kernel<D, BS, E>, dim3(static_cast<unsigned>(ctas)), dim3(warps * 32), 0, stream, p,
                    static_cast<int>(units), items / ctas, static_cast<uint32_t>(items % ctas));
}

template <int D, typename E>
cudaError_t launch_scatter_bs(const BlockScatterLaunch &p, int sm_count, cudaStream_t stream) {
  switch (p.block_size) {
    case 8: return launch_scatter<D, 8, E>(p, sm_count, stream);
    case 16: return launch_scatter<D, 16, E>(p, sm_count, stream);
    default: return launch_scatter<D, 32, E>(p, sm_count, stream);
  }
}

template <typename E>
cudaError_t launch_scatter_dim(const BlockScatterLaunch &p, int sm_count, cudaStream_t stream) {
  switch (p.head_dim) {
    case 64: return launch_scatter_bs<64, E>(p, sm_count, stream);
    case 80: return launch_scatter_bs<80, E>(p, sm_count, stream);
    case 96: return launch_scatter_bs<96, E>(p, sm_count, stream);
    case 128: return launch_scatter_bs<128, E>(p, sm_count, stream);
    default: return launch_scatter_bs<256, E>(p, sm_count, stream);
  }
}

// One thread per (pair, KV head): the scales of a copied block.
__global__ void __launch_bounds__(256) copy_block_scales_kernel(float *k_scales, float *v_scales,
                                                                const int64_t *__restrict__ mapping,
                                                                int32_t num_pairs, int32_t num_kv_heads,
                                                                int64_t num_blocks, unsigned int *status) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t total = static_cast<int64_t>(num_pairs) * num_kv_heads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t pair = i / num_kv_heads, h = i - pair * num_kv_heads;
    const int64_t src = ld_cg(reinterpret_cast<const long long *>(mapping) + 2 * pair);
    const int64_t dst = ld_cg(reinterpret_cast<const long long *>(mapping) + 2 * pair + 1);
    if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
      if (h == 0) flag_error(status, PA_FLAG_BLOCK_RANGE);
      continue;
    }
    k_scales[dst * num_kv_heads + h] = ld_cg(k_scales + src * num_kv_heads + h);
    v_scales[dst * num_kv_heads + h] = ld_cg(v_scales + src * num_kv_heads + h);
  }
}

}  // namespace

cudaError_t launch_block_scatter(const BlockScatterLaunch &p, int sm_count, cudaStream_t stream) {
  return p.dtype == PA_FP16 ? launch_scatter_dim<ElemFp16>(p, sm_count, stream)
                              : launch_scatter_dim<ElemBf16>(p, sm_count, stream);
}

cudaError_t launch_copy_block_scales(float *k_scales, float *v_scales, const int64_t *mapping, int32_t num_pairs,
                                     int32_t num_kv_heads, int64_t num_blocks, unsigned int *status, int sm_count,
                                     cudaStream_t stream) {
  int64_t ctas = (static_cast<int64_t>(num_pairs) * num_kv_heads + 255) / 256;
  if (ctas > 4 * static_cast<int64_t>(sm_count)) ctas = 4 * static_cast<int64_t>(sm_count);
  return launch_pdl(copy_block_scales_kernel, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, stream, k_scales,
                    v_scales, mapping, num_pairs, num_kv_heads, num_blocks, status);
}

}  // namespace pa
