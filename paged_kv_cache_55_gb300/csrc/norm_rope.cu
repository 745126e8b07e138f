// RMS norm of every query and key head, the position rotation, and the write
// of K and V into the paged cache (or of K into rows), in one pass.
//
// A head row x of D elements becomes y = x * w / sqrt(mean(x^2) + eps), w the
// query or key weights of D elements (a null weight pointer skips the norm);
// rotated pairs (y1, y2) become (y1 cos - y2 sin, y2 cos + y1 sin) with row
// positions[t] of cos_sin_cache, pairs and passed-through elements as in the
// rotary scatter of cache_ops.cu. The sum of squares, the norm and the
// rotation are fp32, and a row is rounded to the element type once, after
// both. V rows are copied. 8-bit caches take codes of the rounded row.
//
// Every element is read and written once: the bytes are the bound for steps
// of many tokens, launch and load latency for a decode step.
//
// Split: a head row belongs to a group of LG lanes (LG the power of two that
// gives a lane at most two 16-byte chunks: 8 lanes at D = 128), so a warp
// holds 32 / LG rows at once and a row's sum of squares is log2(LG) shuffles.
// A lane's two chunks are a rotation's partners (the chunk pair c and
// c + rot / 16 of NEOX pairing, two neighbours otherwise), so rotating needs
// no exchange, and a lane keeps the same place in every row it visits: the 8
// cosines, 8 sines and the weights of its chunks stay in registers across all
// the heads of a token. A lane stores only chunks it loaded, after every load
// of its rows, so q_out may be q and key_out may be key.
#include "cache_write.cuh"
#include "pa_common.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

enum NormRopeDst { kRows = 0, kCache16 = 1, kCache8 = 2 };

constexpr int kNormRopeWarps = 8;  // warps per CTA
constexpr int kNormRopeCtas = 3;   // CTAs per SM (registers: at most 85 a thread)
constexpr int kRowBatch = 2;       // row groups whose loads a warp issues before it stores any

// Eight elements of the type, widened (exact).
template <typename E>
__device__ __forceinline__ void widen8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = E::lo(w[k]);
    f[2 * k + 1] = E::hi(w[k]);
  }
}
template <typename E>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  return make_uint4(E::pack(f[0], f[1]), E::pack(f[2], f[3]), E::pack(f[4], f[5]), E::pack(f[6], f[7]));
}

template <typename E, int LG, bool NEOX, int DST>
__global__ void __launch_bounds__(kNormRopeWarps * 32, kNormRopeCtas) norm_rope_kernel(const NormRopeLaunch p) {
  constexpr int RPW = 32 / LG;  // rows per warp and group
  constexpr unsigned FULL = 0xffffffffu;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot_in_row = lane % LG, row_in_group = lane / LG;
  const int d8 = p.head_dim / 8, half16 = p.rotary_dim / 16;
  // this lane's chunks ca and cb of every row
  const bool rotates = slot_in_row < half16;
  int ca, cb;
  if (NEOX && rotates) {
    ca = slot_in_row;
    cb = slot_in_row + half16;
  } else if (NEOX) {  // chunks past the rotated ones, two by two
    ca = 2 * half16 + 2 * (slot_in_row - half16);
    cb = ca + 1;
  } else {
    ca = 2 * slot_in_row;
    cb = ca + 1;
  }
  const bool has_a = ca < d8, has_b = cb < d8;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint32_t one2 = E::pack(1.f, 1.f);
  const uint4 ones = make_uint4(one2, one2, one2, one2);
  const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
  const uint4 *qw = static_cast<const uint4 *>(p.q_weight), *kw = static_cast<const uint4 *>(p.k_weight);
  const uint4 qwa = norm_q && has_a ? ld_cg(qw + ca) : ones, qwb = norm_q && has_b ? ld_cg(qw + cb) : ones;
  const uint4 kwa = norm_k && has_a ? ld_cg(kw + ca) : ones, kwb = norm_k && has_b ? ld_cg(kw + cb) : ones;
  const float inv_d = 1.0f / static_cast<float>(p.head_dim);

  const int rows = p.num_heads + p.num_kv_heads * (DST == kRows ? 1 : 2);  // q, K and (into a cache) V heads
  const int groups = (rows + RPW - 1) / RPW;
  const int64_t units = static_cast<int64_t>(p.num_tokens) * p.slices;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kNormRopeWarps + warp; u < units;
       u += static_cast<int64_t>(gridDim.x) * kNormRopeWarps) {
    const int32_t t = static_cast<int32_t>(u / p.slices), sl = static_cast<int32_t>(u - static_cast<int64_t>(t) * p.slices);
    const int g_begin = static_cast<int>(static_cast<int64_t>(groups) * sl / p.slices);
    const int g_end = static_cast<int>(static_cast<int64_t>(groups) * (sl + 1) / p.slices);
    const int64_t pos = ld_cg(reinterpret_cast<const long long *>(p.positions) + t);
    int64_t slot = -1;
    if (DST != kRows) slot = ld_cg(reinterpret_cast<const long long *>(p.slot_mapping) + t);
    if (!(pos >= 0 && pos < p.max_position)) {  // the token is skipped
      if (lane == 0 && sl == 0) flag_error(p.status, PA_FLAG_POSITION_RANGE);
      continue;
    }
    if (DST != kRows && slot >= p.num_slots && lane == 0 && sl == 0) flag_error(p.status, PA_FLAG_SLOT_RANGE);
    const bool cached = DST != kRows && slot >= 0 && slot < p.num_slots;  // slot < 0: padding token
    float cs[8], sn[8];
    if (rotates) {
      const float *trow = p.cos_sin + pos * p.rotary_dim + 8 * slot_in_row;
      const float4 c0 = ld_ca4(trow), c1 = ld_ca4(trow + 4);
      const float4 s0 = ld_ca4(trow + p.rotary_dim / 2), s1 = ld_ca4(trow + p.rotary_dim / 2 + 4);
      cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w, cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
      sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w, sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
    } else {  // the identity
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
    }
    for (int g0 = g_begin; g0 < g_end; g0 += kRowBatch) {
      uint4 xa[kRowBatch], xb[kRowBatch];
#pragma unroll
      for (int k = 0; k < kRowBatch; ++k) {
        xa[k] = xb[k] = zero;
        const int row = (g0 + k) * RPW + row_in_group;
        if (g0 + k >= g_end || row >= rows) continue;
        const uint4 *src;
        if (row < p.num_heads) {
          src = static_cast<const uint4 *>(p.q) + t * (p.q_stride / 8) + static_cast<int64_t>(row) * d8;
        } else {
          const int h = row - p.num_heads;
          if (DST != kRows && !cached) continue;
          src = h < p.num_kv_heads
                    ? static_cast<const uint4 *>(p.key) + t * (p.key_stride / 8) + static_cast<int64_t>(h) * d8
                    : static_cast<const uint4 *>(p.value) + t * (p.value_stride / 8) +
                          static_cast<int64_t>(h - p.num_kv_heads) * d8;
        }
        if (has_a) xa[k] = ld_cg(src + ca);
        if (has_b) xb[k] = ld_cg(src + cb);
      }
#pragma unroll
      for (int k = 0; k < kRowBatch; ++k) {
        const int row = (g0 + k) * RPW + row_in_group;
        const bool is_q = row < p.num_heads, is_v = row >= p.num_heads + p.num_kv_heads;
        uint4 oa = xa[k], ob = xb[k];
        if (DST == kRows || !__all_sync(FULL, is_v)) {  // V rows are copied as they are
        float a[8], b[8];
        widen8<E>(xa[k], a);
        widen8<E>(xb[k], b);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
        for (int o = 1; o < LG; o <<= 1) ss += __shfl_xor_sync(FULL, ss, o);
        float r = __frsqrt_rn(fmaf(ss, inv_d, p.eps));
        if (__any_sync(FULL, !(ss <= 3.0e38f))) {
          // the squares of elements beyond 2^63 overflow: sum them again
          // scaled by 2^-140 (eps is far below such a mean)
          float s2 = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float ya = a[i] * 0x1p-70f, yb = b[i] * 0x1p-70f;
            s2 = fmaf(ya, ya, fmaf(yb, yb, s2));
          }
#pragma unroll
          for (int o = 1; o < LG; o <<= 1) s2 += __shfl_xor_sync(FULL, s2, o);
          if (!(ss <= 3.0e38f)) r = __frsqrt_rn(s2 * inv_d) * 0x1p-70f;
        }
        if (!(is_q ? norm_q : norm_k)) r = 1.f;
        float wa[8], wb[8];
        widen8<E>(is_q ? qwa : kwa, wa);
        widen8<E>(is_q ? qwb : kwb, wb);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = a[i] * r * wa[i];
          b[i] = b[i] * r * wb[i];
        }
        if (rotates) {
          if (NEOX) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float y1 = a[i], y2 = b[i];
              a[i] = fmaf(y1, cs[i], -(y2 * sn[i]));
              b[i] = fmaf(y2, cs[i], y1 * sn[i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float y1 = a[2 * i], y2 = a[2 * i + 1], z1 = b[2 * i], z2 = b[2 * i + 1];
              a[2 * i] = fmaf(y1, cs[i], -(y2 * sn[i]));
              a[2 * i + 1] = fmaf(y2, cs[i], y1 * sn[i]);
              b[2 * i] = fmaf(z1, cs[4 + i], -(z2 * sn[4 + i]));
              b[2 * i + 1] = fmaf(z2, cs[4 + i], z1 * sn[4 + i]);
            }
          }
        }
        if (!is_v) {
          oa = narrow8<E>(a);
          ob = narrow8<E>(b);
        }
        }
        if (g0 + k >= g_end || row >= rows) continue;
        if (is_q) {
          uint4 *dst = static_cast<uint4 *>(p.q_out) + t * (p.q_out_stride / 8) + static_cast<int64_t>(row) * d8;
          if (has_a) dst[ca] = oa;
          if (has_b) dst[cb] = ob;
        } else if (DST == kRows) {
          uint4 *dst = static_cast<uint4 *>(p.key_dst) + t * (p.key_out_stride / 8) +
                       static_cast<int64_t>(row - p.num_heads) * d8;
          if (has_a) dst[ca] = oa;
          if (has_b) dst[cb] = ob;
        } else if (cached) {
          const int h = is_v ? row - p.num_heads - p.num_kv_heads : row - p.num_heads;
          const int64_t ofs = (slot * p.num_kv_heads + h) * d8;
          if (DST == kCache16) {
            uint4 *dst = static_cast<uint4 *>(is_v ? p.value_dst : p.key_dst) + ofs;
            if (has_a) dst[ca] = oa;
            if (has_b) dst[cb] = ob;
          } else {
            uint2 *dst = static_cast<uint2 *>(is_v ? p.value_dst : p.key_dst) + ofs;
            const float scale = is_v ? p.v_scale : p.k_scale;
            if (has_a) dst[ca] = quantize8<E>(oa, scale);
            if (has_b) dst[cb] = quantize8<E>(ob, scale);
          }
        }
      }
    }
  }
}

template <typename E, int LG, bool NEOX>
cudaError_t launch_dst(const NormRopeLaunch &p, dim3 grid, cudaStream_t stream) {
  const dim3 block(kNormRopeWarps * 32);
  if (p.dst == kRows) return launch_pdl(norm_rope_kernel<E, LG, NEOX, kRows>, grid, block, 0, stream, p);
  if (p.dst == kCache16) return launch_pdl(norm_rope_kernel<E, LG, NEOX, kCache16>, grid, block, 0, stream, p);
  return launch_pdl(norm_rope_kernel<E, LG, NEOX, kCache8>, grid, block, 0, stream, p);
}

template <typename E, int LG>
cudaError_t launch_lanes(NormRopeLaunch p, int sm_count, cudaStream_t stream) {
  // a token's row groups are split over `slices` warps when the tokens alone
  // would not give every SM its warps
  const int rows = p.num_heads + p.num_kv_heads * (p.dst == kRows ? 1 : 2);
  const int groups = (rows + 32 / LG - 1) / (32 / LG);
  const int64_t want = static_cast<int64_t>(sm_count) * kNormRopeCtas * kNormRopeWarps;
  int64_t slices = (want + p.num_tokens - 1) / p.num_tokens;
  slices = slices > groups ? groups : slices;
  p.slices = static_cast<int32_t>(slices < 1 ? 1 : slices);
  int64_t ctas = (static_cast<int64_t>(p.num_tokens) * p.slices + kNormRopeWarps - 1) / kNormRopeWarps;
  const int64_t cap = static_cast<int64_t>(sm_count) * kNormRopeCtas;
  if (ctas > cap) ctas = cap;
  const dim3 grid(static_cast<unsigned>(ctas));
  return p.is_neox ? launch_dst<E, LG, true>(p, grid, stream) : launch_dst<E, LG, false>(p, grid, stream);
}

template <typename E>
cudaError_t launch_elem(const NormRopeLaunch &p, int sm_count, cudaStream_t stream) {
  const int slots = (p.head_dim / 8 + 1) / 2;  // pairs of chunks in a row
  if (slots <= 4) return launch_lanes<E, 4>(p, sm_count, stream);
  if (slots <= 8) return launch_lanes<E, 8>(p, sm_count, stream);
  if (slots <= 16) return launch_lanes<E, 16>(p, sm_count, stream);
  return launch_lanes<E, 32>(p, sm_count, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeLaunch &p, int sm_count, cudaStream_t stream) {
  return p.dtype == PA_FP16 ? launch_elem<ElemFp16>(p, sm_count, stream) : launch_elem<ElemBf16>(p, sm_count, stream);
}

}  // namespace pa
