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
// no exchange, and a lane keeps the same place in every row it visits: its 8
// cosines and 8 sines serve all the heads of a token. A lane stores only chunks
// it loaded, after every load of its rows, so q_out may be q and key_out may be
// key. A unit of work is BATCH such row groups of one token, all their loads
// issued first; the weights wait in shared memory as floats.
//
// Bound by HBM when there are many tokens, by launch and load latency in a
// decode step. Measured (32 / 8 heads of 128, bf16): 8432 tokens 39.8 us, 5.3
// TB/s, against 49.5 with one row group at a time and weights converted per
// row; what is left is issue (0.48 per cycle at 24 % of the warps: the 123
// registers that hold four groups). 256 tokens 3.6 us, one token 2.4.
#include "cache_write.cuh"
#include "pa_common.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

enum NormRopeDst { kRows = 0, kCache16 = 1, kCache8 = 2 };

constexpr int kNormRopeWarps = 8;    // warps per CTA
constexpr int kNormRopeMaxDim = 512;  // a head row is at most one warp's

// Row groups per unit: four (16 loads of 16 bytes in flight per lane pair) when
// there are tokens enough to fill the GPU, one when a decode step has not even
// a row group per warp (a unit is then as short as it can be).
constexpr int kManyGroups = 4, kFewGroups = 1;
constexpr int norm_rope_ctas(int batch) { return batch == kManyGroups ? 2 : 3; }  // CTAs per SM

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n"
      " mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, w, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 w, {%6, %7};\n"
      " fma.rn.f32x2 z, x, y, w;\n mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Eight elements of the type, widened (exact), in pairs.
template <typename E>
__device__ __forceinline__ void widen8(uint4 v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = make_float2(E::lo(w[k]), E::hi(w[k]));
}
template <typename E>
__device__ __forceinline__ uint4 narrow8(const float2 (&f)[4]) {
  return make_uint4(E::pack(f[0].x, f[0].y), E::pack(f[1].x, f[1].y), E::pack(f[2].x, f[2].y),
                    E::pack(f[3].x, f[3].y));
}

template <typename E, int LG, bool NEOX, int DST, int BATCH>
__global__ void __launch_bounds__(kNormRopeWarps * 32, norm_rope_ctas(BATCH)) norm_rope_kernel(const NormRopeLaunch p) {
  constexpr int RPW = 32 / LG;  // rows per warp and group
  constexpr unsigned FULL = 0xffffffffu;
  __shared__ __align__(16) float s_weight[2][kNormRopeMaxDim];  // q's, K's; 1 where there is no norm
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
  const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
  const float inv_d = 1.0f / static_cast<float>(p.head_dim);

  const int rows = p.num_heads + p.num_kv_heads * (DST == kRows ? 1 : 2);  // q, K and (into a cache) V heads
  const int groups = (rows + RPW - 1) / RPW;
  const int per_token = (groups + BATCH - 1) / BATCH;  // units per token
  const int64_t units = static_cast<int64_t>(p.num_tokens) * per_token;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kNormRopeWarps;
  int64_t u = static_cast<int64_t>(blockIdx.x) * kNormRopeWarps + warp;
  // position and slot of a unit's token are loaded a unit ahead
  int64_t pos = -1, slot = -1;
  auto load_token = [&](int64_t v) {
    if (v < units) {
      const int64_t t = v / per_token;
      pos = ld_cg(reinterpret_cast<const long long *>(p.positions) + t);
      if (DST != kRows) slot = ld_cg(reinterpret_cast<const long long *>(p.slot_mapping) + t);
    }
  };
  load_token(u);
  for (int i = threadIdx.x; i < 2 * p.head_dim; i += blockDim.x) {
    const bool k = i >= p.head_dim;
    const int e = k ? i - p.head_dim : i;
    const unsigned short *w = static_cast<const unsigned short *>(k ? p.k_weight : p.q_weight);
    unsigned short bits = 0;
    if (w) asm volatile("ld.global.cg.u16 %0, [%1];\n" : "=h"(bits) : "l"(w + e) : "memory");
    s_weight[k][e] = w ? E::lo(bits) : 1.f;
  }
  __syncthreads();

  for (; u < units; u += stride) {
    const int32_t t = static_cast<int32_t>(u / per_token), part = static_cast<int32_t>(u - static_cast<int64_t>(t) * per_token);
    const int64_t my_pos = pos, my_slot = slot;
    uint4 xa[BATCH], xb[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      xa[k] = xb[k] = make_uint4(0u, 0u, 0u, 0u);
      const int row = (part * BATCH + k) * RPW + row_in_group;
      if (row >= rows) continue;
      const int h = row - p.num_heads;
      const uint4 *src =
          h < 0 ? static_cast<const uint4 *>(p.q) + t * (p.q_stride / 8) + static_cast<int64_t>(row) * d8
          : h < p.num_kv_heads
              ? static_cast<const uint4 *>(p.key) + t * (p.key_stride / 8) + static_cast<int64_t>(h) * d8
              : static_cast<const uint4 *>(p.value) + t * (p.value_stride / 8) +
                    static_cast<int64_t>(h - p.num_kv_heads) * d8;
      if (has_a) xa[k] = ld_cg(src + ca);
      if (has_b) xb[k] = ld_cg(src + cb);
    }
    load_token(u + stride);
    if (!(my_pos >= 0 && my_pos < p.max_position)) {  // the token is skipped
      if (lane == 0 && part == 0) flag_error(p.status, PA_FLAG_POSITION_RANGE);
      continue;
    }
    if (DST != kRows && my_slot >= p.num_slots && lane == 0 && part == 0) flag_error(p.status, PA_FLAG_SLOT_RANGE);
    const bool cached = DST != kRows && my_slot >= 0 && my_slot < p.num_slots;  // slot < 0: padding token
    float2 cs[4], sn[4];
    if (rotates) {
      const float *trow = p.cos_sin + my_pos * p.rotary_dim + 8 * slot_in_row;
      const float4 c0 = ld_ca4(trow), c1 = ld_ca4(trow + 4);
      const float4 s0 = ld_ca4(trow + p.rotary_dim / 2), s1 = ld_ca4(trow + p.rotary_dim / 2 + 4);
      cs[0] = make_float2(c0.x, c0.y), cs[1] = make_float2(c0.z, c0.w);
      cs[2] = make_float2(c1.x, c1.y), cs[3] = make_float2(c1.z, c1.w);
      sn[0] = make_float2(s0.x, s0.y), sn[1] = make_float2(s0.z, s0.w);
      sn[2] = make_float2(s1.x, s1.y), sn[3] = make_float2(s1.z, s1.w);
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int row = (part * BATCH + k) * RPW + row_in_group;
      if ((part * BATCH + k) * RPW >= rows) break;  // the whole warp's
      const bool is_q = row < p.num_heads, is_v = row >= p.num_heads + p.num_kv_heads;
      uint4 oa = xa[k], ob = xb[k];
      if (DST == kRows || !__all_sync(FULL, is_v)) {  // V rows are copied as they are
        float2 a[4], b[4];
        widen8<E>(xa[k], a);
        widen8<E>(xb[k], b);
        float2 s2 = both(0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = fma2(a[i], a[i], fma2(b[i], b[i], s2));
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = 1; o < LG; o <<= 1) ss += __shfl_xor_sync(FULL, ss, o);
        float r = rsqrtf(fmaf(ss, inv_d, p.eps));
        if (__any_sync(FULL, !(ss <= 3.0e38f))) {
          // the squares of elements beyond 2^63 overflow: sum them again
          // scaled by 2^-140 (eps is far below such a mean)
          const float2 down = both(0x1p-70f);
          s2 = both(0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 ya = mul2(a[i], down), yb = mul2(b[i], down);
            s2 = fma2(ya, ya, fma2(yb, yb, s2));
          }
          float sd = s2.x + s2.y;
#pragma unroll
          for (int o = 1; o < LG; o <<= 1) sd += __shfl_xor_sync(FULL, sd, o);
          if (!(ss <= 3.0e38f)) r = rsqrtf(sd * inv_d) * 0x1p-70f;
        }
        if (!(is_q ? norm_q : norm_k)) r = 1.f;
        const float *w = s_weight[is_q ? 0 : 1];
        const float2 rr = both(r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = mul2(mul2(a[i], rr), *reinterpret_cast<const float2 *>(w + 8 * (has_a ? ca : 0) + 2 * i));
          b[i] = mul2(mul2(b[i], rr), *reinterpret_cast<const float2 *>(w + 8 * (has_b ? cb : 0) + 2 * i));
        }
        if (rotates) {
          if (NEOX) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 y1 = a[i], y2 = b[i];
              a[i] = fma2(y1, cs[i], neg2(mul2(y2, sn[i])));
              b[i] = fma2(y2, cs[i], mul2(y1, sn[i]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {  // pairs 2 i + j of chunk a, and of chunk b
                float2 &y = a[2 * i + j], &z = b[2 * i + j];
                const float c1 = j ? cs[i].y : cs[i].x, n1 = j ? sn[i].y : sn[i].x;
                const float c2 = j ? cs[2 + i].y : cs[2 + i].x, n2 = j ? sn[2 + i].y : sn[2 + i].x;
                y = make_float2(fmaf(y.x, c1, -(y.y * n1)), fmaf(y.y, c1, y.x * n1));
                z = make_float2(fmaf(z.x, c2, -(z.y * n2)), fmaf(z.y, c2, z.x * n2));
              }
            }
          }
        }
        if (!is_v) {
          oa = narrow8<E>(a);
          ob = narrow8<E>(b);
        }
      }
      if (row >= rows) continue;
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
        const int64_t ofs = (my_slot * p.num_kv_heads + h) * d8;
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

template <typename E, int LG, bool NEOX, int BATCH>
cudaError_t launch_dst(const NormRopeLaunch &p, int64_t units, int sm_count, cudaStream_t stream) {
  int64_t ctas = (units + kNormRopeWarps - 1) / kNormRopeWarps;
  const int64_t cap = static_cast<int64_t>(sm_count) * norm_rope_ctas(BATCH);
  if (ctas > cap) ctas = cap;
  const dim3 grid(static_cast<unsigned>(ctas)), block(kNormRopeWarps * 32);
  if (p.dst == kRows) return launch_pdl(norm_rope_kernel<E, LG, NEOX, kRows, BATCH>, grid, block, 0, stream, p);
  if (p.dst == kCache16) return launch_pdl(norm_rope_kernel<E, LG, NEOX, kCache16, BATCH>, grid, block, 0, stream, p);
  return launch_pdl(norm_rope_kernel<E, LG, NEOX, kCache8, BATCH>, grid, block, 0, stream, p);
}

template <typename E, int LG, bool NEOX>
cudaError_t launch_batch(const NormRopeLaunch &p, int sm_count, cudaStream_t stream) {
  const int rows = p.num_heads + p.num_kv_heads * (p.dst == kRows ? 1 : 2);
  const int64_t groups = (rows + 32 / LG - 1) / (32 / LG);
  if (p.num_tokens * groups <= static_cast<int64_t>(sm_count) * norm_rope_ctas(kFewGroups) * kNormRopeWarps)
    return launch_dst<E, LG, NEOX, kFewGroups>(p, p.num_tokens * groups, sm_count, stream);
  return launch_dst<E, LG, NEOX, kManyGroups>(p, p.num_tokens * ((groups + kManyGroups - 1) / kManyGroups), sm_count,
                                              stream);
}

template <typename E, int LG>
cudaError_t launch_lanes(const NormRopeLaunch &p, int sm_count, cudaStream_t stream) {
  return p.is_neox ? launch_batch<E, LG, true>(p, sm_count, stream) : launch_batch<E, LG, false>(p, sm_count, stream);
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
