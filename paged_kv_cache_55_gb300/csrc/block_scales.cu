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

// E4M3 codes of x / scale. A power-of-two scale divides by multiplying with
// its inverse (exact, the same rounding); any other is divided by.
template <typename E>
__device__ __forceinline__ uint2 quantize8_by(uint4 a, float scale, float inverse, bool power_of_two) {
  if (!power_of_two) return quantize8<E>(a, scale);
  const uint32_t x[4] = {a.x, a.y, a.z, a.w};
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) c[k] = e4m3x2_from_f32(E::lo(x[k]) * inverse, E::hi(x[k]) * inverse);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The request that owns unit u: the largest b with start(b) <= u, where
// start(b) = query_start_loc[b] / bs + 2 b. A request of n > 0 rows touches at
// most n / bs + 2 blocks, so the units [start(b), start(b + 1)) cover them.
// Every thread probes one request per round (one round up to 256 requests).
// The last round's probes load the request's lengths as well, and the last
// thread that lies at or below u publishes them: {b, q0, q1, length}.
__device__ __forceinline__ void find_request(const BlockScatterLaunch &p, int shift, int u, int4 *found) {
  __shared__ int s_lo;
  int lo = 0, n = p.num_seqs;  // the answer is in [lo, lo + n)
  for (;;) {
    const int step = (n + blockDim.x - 1) / blockDim.x;
    const int at = static_cast<int>(threadIdx.x) * step;
    int q0 = 0, q1 = 0, len = 0;
    bool below = false, last = false;
    if (at < n) {
      const int b = lo + at;
      q0 = ld_cg(p.query_start_loc + b);
      if (step == 1) {
        q1 = ld_cg(p.query_start_loc + b + 1);
        len = ld_cg(p.seq_lens + b);
      }
      const int next = min(at + step, n);  // the next probe's request
      const int qn = next < n ? (step == 1 ? q1 : ld_cg(p.query_start_loc + lo + next)) : 0;
      below = (q0 >> shift) + 2 * b <= u || at == 0;
      last = below && (next >= n || (qn >> shift) + 2 * (lo + next) > u);
    }
    // (a query_start_loc that is not sorted may elect several threads or none: any one of them is in range)
    if (threadIdx.x == 0) {
      s_lo = lo;
      if (step == 1) *found = make_int4(lo, q0, q1, len);
    }
    __syncthreads();
    if (last) {
      s_lo = lo + at;
      if (step == 1) *found = make_int4(lo + at, q0, q1, len);
    }
    __syncthreads();
    if (step == 1) return;
    const int picked = s_lo;
    n = min(step, n - (picked - lo));
    lo = picked;
    __syncthreads();  // s_lo has been read
  }
}

// One CTA per unit (touched block of a request), a warp per (K or V, KV head):
// a warp loads the block's new rows of its head into registers, reduces their
// largest magnitude, and stores their codes.
template <int D, int BS, typename E>
__global__ void __launch_bounds__(scatter_warps(D, BS) * 32) block_scatter_kernel(const BlockScatterLaunch p) {
  constexpr int CPR = D / 8;                   // 8-element chunks per row
  constexpr int NV = scatter_chunks(D, BS);    // chunks per lane, at most
  constexpr int SHIFT = BS == 8 ? 3 : (BS == 16 ? 4 : 5);
  __shared__ int4 s_found;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int u = blockIdx.x;
  // steps of one-token requests: unit u is request u
  const bool single = p.max_query_len <= 1;
  int b, q0, q1, len;
  if (single) {
    b = u;
    q0 = ld_cg(p.query_start_loc + b);
    q1 = ld_cg(p.query_start_loc + b + 1);
    len = ld_cg(p.seq_lens + b);
  } else {
    find_request(p, SHIFT, u, &s_found);
    const int4 f = s_found;
    b = f.x, q0 = f.y, q1 = f.z, len = f.w;
  }
  const int ql = q1 - q0;
  const bool report = threadIdx.x == 0;
  if (q0 < 0 || ql < 0 || q1 > p.total_q || (b == 0 && q0 != 0) || (b == p.num_seqs - 1 && q1 != p.total_q)) {
    if (report) flag_error(p.status, PA_FLAG_QUERY_LOC);
    return;
  }
  if (ql == 0) return;
  if (len < ql || ql > p.max_query_len || len > static_cast<int64_t>(p.max_blocks_per_seq) * BS) {
    if (report) flag_error(p.status, PA_FLAG_LENGTHS);
    return;
  }
  const int i = single ? 0 : u - ((q0 >> SHIFT) + 2 * b);  // touched block of the request
  const int ctx = len - ql;
  const int64_t first = (static_cast<int64_t>(ctx >> SHIFT) + i) << SHIFT;  // first position of the block
  if (i < 0 || first >= len) return;
  const int phys = ld_cg(p.block_tables + static_cast<int64_t>(b) * p.max_blocks_per_seq + (first >> SHIFT));
  if (phys < 0 || phys >= p.num_blocks) {
    if (report) flag_error(p.status, PA_FLAG_BLOCK_RANGE);
    return;
  }
  const int row0 = max(ctx - static_cast<int>(first), 0);  // rows [row0, row1) of the block are new
  const int row1 = static_cast<int>(min(static_cast<long long>(len) - first, static_cast<long long>(BS)));
  const int64_t token0 = q0 + (first + row0 - ctx);
  const int n = (row1 - row0) * CPR;
  const int64_t row8 = static_cast<int64_t>(p.num_kv_heads) * CPR;  // 8-code vectors per cache row

  for (int r = warp; r < 2 * p.num_kv_heads; r += warps) {
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
      m2 = __vmaxu2(m2, __vmaxu2(x[j].x & 0x7FFF7FFFu, x[j].y & 0x7FFF7FFFu));
      m2 = __vmaxu2(m2, __vmaxu2(x[j].z & 0x7FFF7FFFu, x[j].w & 0x7FFF7FFFu));
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
    const bool power_of_two = (__float_as_uint(after) & 0x7FFFFFu) == 0;
    const float inverse = __frcp_rn(after);

    uint2 *dst = static_cast<uint2 *>(is_v ? p.value_cache : p.key_cache) + static_cast<int64_t>(phys) * BS * row8 +
                 static_cast<int64_t>(kvh) * CPR;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = lane + 32 * j, row = k / CPR, c = k % CPR;
      if (k < n) dst[(row0 + row) * row8 + c] = quantize8_by<E>(x[j], after, inverse, power_of_two);
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

template <int D, int BS, typename E>
cudaError_t launch_scatter(const BlockScatterLaunch &p, cudaStream_t stream) {
  const int64_t units =
      p.max_query_len <= 1 ? p.num_seqs : p.total_q / BS + 2 * static_cast<int64_t>(p.num_seqs);
  constexpr int most = scatter_warps(D, BS);
  const int warps = 2 * p.num_kv_heads < most ? 2 * p.num_kv_heads : most;
  return launch_pdl(block_scatter_kernel<D, BS, E>, dim3(static_cast<unsigned>(units)), dim3(warps * 32), 0, stream,
                    p);
}

template <int D, typename E>
cudaError_t launch_scatter_bs(const BlockScatterLaunch &p, cudaStream_t stream) {
  switch (p.block_size) {
    case 8: return launch_scatter<D, 8, E>(p, stream);
    case 16: return launch_scatter<D, 16, E>(p, stream);
    default: return launch_scatter<D, 32, E>(p, stream);
  }
}

template <typename E>
cudaError_t launch_scatter_dim(const BlockScatterLaunch &p, cudaStream_t stream) {
  switch (p.head_dim) {
    case 64: return launch_scatter_bs<64, E>(p, stream);
    case 80: return launch_scatter_bs<80, E>(p, stream);
    case 96: return launch_scatter_bs<96, E>(p, stream);
    case 128: return launch_scatter_bs<128, E>(p, stream);
    default: return launch_scatter_bs<256, E>(p, stream);
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

cudaError_t launch_block_scatter(const BlockScatterLaunch &p, int /*sm_count*/, cudaStream_t stream) {
  return p.dtype == PA_FP16 ? launch_scatter_dim<ElemFp16>(p, stream) : launch_scatter_dim<ElemBf16>(p, stream);
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
