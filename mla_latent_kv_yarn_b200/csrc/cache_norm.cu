// Cache rows from a raw key projection: norm, rotation and append in one pass,
// to the bf16 or the 8-bit pool; and 8-bit rows read back.
//
//   row = [ c_kv / sqrt(mean(c_kv^2) + eps) * w_kv | rope(k) ],
//   k   = k_pe, or k_pe / sqrt(mean(k_pe^2) + eps) * w_pe
//
// rounded once: to bf16, or to the 8-bit row's codes (blocks of 32, one
// power-of-two scale each).
//
// [P5] "mHC+MLA+MTP 是什么？拆开给 Agent 用的百亿 MoE", section "MLA：256K 上下文的
//      '内存革命'": the cache row is the 512-dim latent and the 64-dim rope key.
// [P1] "256K 长上下文真能本地用：Xing4.0 原生长上下文的工程代价拆解", section 三, 方案 A:
//      the q8_0 cache.
#include <cuda_bf16.h>

#include <cstdint>

#include "norm.cuh"

namespace xmla {

namespace {

constexpr int kAnWarps = 8;
constexpr int kReadThreads = 256;
constexpr int kCodeUnits = kDRow / 16;  // 36 units of 16 codes per row

struct RowPlace {
  const int32_t* block_table;
  const int32_t* seq_ids;
  const int64_t* positions;
  int32_t* status;
  int64_t num_blocks;
  int64_t T;
  int32_t max_blocks;
  int32_t batch;
};

// The pool row of token t at position pos, or -1 (recorded) where its sequence,
// position or block is out of range.
__device__ __forceinline__ int64_t pool_row(const RowPlace& w, int64_t t, int64_t pos) {
  const int32_t s = w.seq_ids[t];
  if (s >= 0 && s < w.batch && pos >= 0 && pos < (int64_t)w.max_blocks * kPage) {
    const int32_t blk = w.block_table[(int64_t)s * w.max_blocks + pos / kPage];
    if (blk >= 0 && (int64_t)blk < w.num_blocks) return (int64_t)blk * kPage + pos % kPage;
  }
  record_status(w.status, XMLA_ERR_DEVICE_OOB);
  return -1;
}

struct AppendNormArgs {
  uint8_t* pool;
  const __nv_bfloat16* c_kv;
  const __nv_bfloat16* k_pe;
  const __nv_bfloat16* w_kv;
  const __nv_bfloat16* w_pe;  // nullable: the rope key is not normed
  int64_t c_stride, k_stride;
  float eps;
  int rotate;
};

// The exponent of a block of the 8-bit row: the smallest e with 127 * 2^e >=
// amax, in [-14, 8].
__device__ __forceinline__ int block_exponent(float amax) {
  if (!(amax > 0.f)) return kQ8EMin;
  int k;
  const float m = frexpf(amax, &k);
  return min(max(m > 127.f / 128.f ? k - 6 : k - 7, kQ8EMin), kQ8EMax);
}
__device__ __forceinline__ uint32_t block_code(float x, int e) {
  return (uint32_t)min(127, max(-127, __float2int_rn(x * __int_as_float((127 - e) << 23)))) & 0xffu;
}

// rms_factor to about half its error: one Newton step, with the rounding errors of the
// mean plus eps and of r * r, takes out those of the root and the quotient.  A code is
// a rounding: the fewer values the float32 error takes past the middle of two codes the
// better (67 million latent values: 112 so, 140 with rms_factor and the weight multiplied
// to the factor first; with sums and products in pairs of floats, for 19% more time, only
// those of blocks whose exponent turned on it).
__device__ __forceinline__ float rms_factor_refined(float sq, int n, float eps) {
  const float mean = sq / (float)n, v = mean + eps, b = v - mean;
  const float rest = (mean - (v - b)) + (eps - b);  // v + rest = mean + eps
  const float r = 1.f / sqrtf(v), p = r * r, q = fmaf(r, r, -p);
  const float res = fmaf(-rest, p, fmaf(-v, q, fmaf(-v, p, 1.f)));
  const float f = fmaf(0.5f * r, res, r);
  return isfinite(f) ? f : r;  // v infinite, 0 or no number
}

// Sixteen lanes per token: lane l of them holds the 16-byte pieces l, l + 16, l +
// 32 and l + 48 of the latent and the rotation pairs l and l + 16 (values l, l + 16
// and those 32 on).  A whole warp per token has half as many values per lane for
// the same lookups, norm factors and addresses: 1.6 us more for 15,001 tokens and 3 us
// more for 16,384 to the 8-bit pool and read back, which take 11.2 us (35 MB) and 22.3
// us.  Bound by latency: about two waves of blocks, each a lookup, its loads and its
// stores one after the other.
constexpr int kAnTokens = 2 * kAnWarps;  // per block

template <bool kQ8>
__global__ void __launch_bounds__(32 * kAnWarps, 4)
    append_norm_kernel(const AppendNormArgs a, const RowPlace place, const RopeTable tab) {
  const int lane = threadIdx.x & 31, l = lane & 15;
  const int64_t t = (int64_t)blockIdx.x * kAnTokens + (threadIdx.x >> 4);
  pdl_wait();
  pdl_launch_dependents();
  // Everything that is fetched is under way before anything is computed, and the
  // rotation's angles, which need the position alone, come first: looking a row's
  // place up takes two loads one after the other, its values take one.
  const int64_t tc = min(t, place.T - 1);
  const int64_t pos = place.positions[tc];
  uint4 xv[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    xv[k] = *reinterpret_cast<const uint4*>(a.c_kv + tc * a.c_stride + 8 * (l + 16 * k));
  const __nv_bfloat16* kp = a.k_pe + tc * a.k_stride;
  float y[4];  // values l, l + 16, l + 32, l + 48
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] = __bfloat162float(kp[l + 16 * k]);
  const int64_t dst_row = t < place.T ? pool_row(place, t, pos) : -1;
  float c[2] = {1.f, 1.f}, s[2] = {0.f, 0.f};
  if (a.rotate) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      rope_cos_sin(pos, tab.inv_freq[l + 16 * k], (float)tab.magnitude, &c[k], &s[k]);
  }
  // (the values stay packed between the passes over them: unpacked, they would
  // take the registers of a block per SM)
  float sq, sq_pe;
  auto squares = [&](float scale) {
    sq = sq_pe = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x[8];
      unpack8(xv[k], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(x[e] * scale, x[e] * scale, sq);
      sq_pe = fmaf(y[k], y[k], sq_pe);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      sq += __shfl_xor_sync(0xffffffffu, sq, o);
      sq_pe += __shfl_xor_sync(0xffffffffu, sq_pe, o);
    }
  };
  squares(1.f);
  float eps = a.eps, eps_pe = a.eps;
  const float scale = rms_scale(sq, kDLatent, eps);
  const float scale_pe = a.w_pe != nullptr ? rms_scale(sq_pe, kDRope, eps) : 1.f;
  if (__any_sync(0xffffffffu, scale != 1.f || scale_pe != 1.f)) {
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] *= scale_pe;
    squares(scale);
    eps = eps * scale * scale;
    eps_pe = eps_pe * scale_pe * scale_pe;
  }
  float f = rms_factor_refined(sq, kDLatent, eps);
  // the values by the factor's power of two first (exact): their products with the
  // weight then stay as small as the results
  float first = scale;
  if (scale == 1.f && f > 0x1p-126f && f < INFINITY) {
    first = __uint_as_float(__float_as_uint(f) & 0x7f800000u);
    f = __uint_as_float((__float_as_uint(f) & 0x007fffffu) | 0x3f800000u);
  }
  // piece k of the normed latent; the weights come from L1
  auto latent = [&](int k, float (&x)[8]) {
    float w[8];
    unpack8(xv[k], x);
    unpack8(*reinterpret_cast<const uint4*>(a.w_kv + 8 * (l + 16 * k)), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * first * w[e] * f;  // (exact up to the last)
  };
  if (a.w_pe != nullptr) {
    const float g = rms_factor(sq_pe, kDRope, eps_pe);
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] *= g * __bfloat162float(a.w_pe[l + 16 * k]);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float u = y[k], v = y[k + 2];
    y[k] = fmaf(u, c[k], -v * s[k]);
    y[k + 2] = fmaf(v, c[k], u * s[k]);
  }
  if constexpr (!kQ8) {
    if (dst_row < 0) return;
    __nv_bfloat16* row = reinterpret_cast<__nv_bfloat16*>(a.pool) + dst_row * kDRow;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x[8];
      latent(k, x);
      *reinterpret_cast<uint4*>(row + 8 * (l + 16 * k)) = pack8(x);
      row[kDLatent + l + 16 * k] = __float2bfloat16_rn(y[k]);
    }
  } else {
    // (lanes of a row that is skipped take part in the exchanges)
    uint8_t* row = a.pool + max(dst_row, (int64_t)0) * kQ8Row;
    const bool stored = dst_row >= 0;
    // The row's last 32 bytes: 18 exponents, 14 zeros.  The four lanes 4 q .. 4 q + 3
    // share block 4 k + q; lane l writes bytes l and 16 + l.
    int tail = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x[8];
      latent(k, x);
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int ex = block_exponent(amax);
      uint32_t code[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) code[e >> 2] |= block_code(x[e], ex) << (8 * (e & 3));
      if (stored)
        *reinterpret_cast<uint2*>(row + 8 * (l + 16 * k)) = make_uint2(code[0], code[1]);
      const int v = __shfl_sync(0xffffffffu, ex, 4 * (l & 3), 16);
      if ((l >> 2) == k) tail = v;
    }
    float a1 = fmaxf(fabsf(y[0]), fabsf(y[1])), a2 = fmaxf(fabsf(y[2]), fabsf(y[3]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, o));
      a2 = fmaxf(a2, __shfl_xor_sync(0xffffffffu, a2, o));
    }
    const int e1 = block_exponent(a1), e2 = block_exponent(a2);
    if (stored) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        row[kDLatent + l + 16 * k] = (uint8_t)block_code(y[k], k < 2 ? e1 : e2);
      row[kDRow + l] = (uint8_t)(int8_t)tail;
      row[kDRow + 16 + l] = (uint8_t)(int8_t)(l == 0 ? e1 : l == 1 ? e2 : 0);
    }
  }
}

// A thread per 16 codes (half a block), kReadUnits of them at once: code * 2^e is
// exact in bf16.
constexpr int kReadUnits = 2;
__global__ void __launch_bounds__(kReadThreads)
    read_q8_kernel(const uint8_t* pool, const RowPlace place, __nv_bfloat16* out,
                   int64_t out_stride) {
  pdl_wait();
  pdl_launch_dependents();
  int64_t t[kReadUnits], src_row[kReadUnits];
  int u[kReadUnits], e[kReadUnits];
  uint4 v[kReadUnits];
#pragma unroll
  for (int n = 0; n < kReadUnits; ++n) {
    const int64_t idx = ((int64_t)blockIdx.x * kReadUnits + n) * kReadThreads + threadIdx.x;
    t[n] = idx / kCodeUnits;
    u[n] = (int)(idx % kCodeUnits);
    src_row[n] = t[n] < place.T ? pool_row(place, t[n], place.positions[t[n]]) : -1;
  }
#pragma unroll
  for (int n = 0; n < kReadUnits; ++n) {
    if (src_row[n] < 0) continue;
    const uint8_t* row = pool + src_row[n] * kQ8Row;
    v[n] = *reinterpret_cast<const uint4*>(row + 16 * u[n]);
    e[n] = (int8_t)row[kDRow + u[n] / 2];
  }
#pragma unroll
  for (int n = 0; n < kReadUnits; ++n) {
    if (src_row[n] < 0) continue;
    const uint32_t word[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
    const float scale = __int_as_float((127 + e[n]) << 23);
    uint4* dst = reinterpret_cast<uint4*>(out + t[n] * out_stride + 16 * u[n]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = (float)(int8_t)(word[2 * k + (i >> 2)] >> (8 * (i & 3))) * scale;
      dst[k] = pack8(x);
    }
  }
}

xmla_status append_norm(void* pool, int64_t num_blocks, const int32_t* block_table,
                        int32_t max_blocks, int32_t batch, const int32_t* seq_ids,
                        const int64_t* positions, const void* c_kv, int64_t c_stride,
                        const void* k_pe, int64_t k_stride, const void* w_kv, const void* w_pe,
                        float eps, const xmla_yarn_cfg* cfg, int64_t T, int32_t* status_dev,
                        void* stream, bool q8) {
  if (T < 0 || num_blocks < 1 || max_blocks < 1 || batch < 1 ||
      (T + kAnWarps - 1) / kAnWarps > 0x7fffffffLL)
    return XMLA_ERR_SHAPE;
  if (cfg != nullptr) {
    if (!yarn_cfg_ok(cfg)) return XMLA_ERR_INVALID_ARG;
    if (cfg->rotary_dim != kDRope) return XMLA_ERR_SHAPE;
  }
  if (!(eps >= 0.f) || !(eps < INFINITY)) return XMLA_ERR_INVALID_ARG;
  if (T == 0) return XMLA_OK;
  if (pool == nullptr || block_table == nullptr || seq_ids == nullptr || positions == nullptr ||
      c_kv == nullptr || k_pe == nullptr || w_kv == nullptr)
    return XMLA_ERR_INVALID_ARG;
  if (((((uintptr_t)pool) | ((uintptr_t)c_kv) | ((uintptr_t)w_kv)) & 15u) || (c_stride & 7) ||
      ((((uintptr_t)k_pe) | ((uintptr_t)w_pe)) & 1u) || c_stride < kDLatent || k_stride < kDRope)
    return XMLA_ERR_INVALID_ARG;
  AppendNormArgs a;
  a.pool = (uint8_t*)pool;
  a.c_kv = (const __nv_bfloat16*)c_kv;
  a.k_pe = (const __nv_bfloat16*)k_pe;
  a.w_kv = (const __nv_bfloat16*)w_kv;
  a.w_pe = (const __nv_bfloat16*)w_pe;
  a.c_stride = c_stride;
  a.k_stride = k_stride;
  a.eps = eps;
  a.rotate = cfg != nullptr ? 1 : 0;
  const RowPlace place{block_table, seq_ids, positions, status_dev, num_blocks, T, max_blocks, batch};
  const RopeTable tab = cfg != nullptr ? make_rope_table(cfg) : RopeTable{};
  const dim3 grid((unsigned)((T + kAnTokens - 1) / kAnTokens));
  const cudaError_t e = launch_pdl(q8 ? append_norm_kernel<true> : append_norm_kernel<false>, grid,
                                   dim3(32 * kAnWarps), 0, (cudaStream_t)stream, a, place, tab);
  return e == cudaSuccess ? XMLA_OK : XMLA_ERR_CUDA;
}

}  // namespace

}  // namespace xmla

using namespace xmla;

extern "C" xmla_status xmla_cache_append_norm(
    void* pool, int64_t num_blocks, const int32_t* block_table, int32_t max_blocks, int32_t batch,
    const int32_t* seq_ids, const int64_t* positions, const void* c_kv, int64_t c_stride,
    const void* k_pe, int64_t k_stride, const void* kv_weight, const void* pe_weight, float eps,
    const xmla_yarn_cfg* rope_cfg, int64_t T, int32_t* status_dev, void* stream) {
  return append_norm(pool, num_blocks, block_table, max_blocks, batch, seq_ids, positions, c_kv,
                     c_stride, k_pe, k_stride, kv_weight, pe_weight, eps, rope_cfg, T, status_dev,
                     stream, false);
}

extern "C" xmla_status xmla_cache_append_norm_q8(
    void* pool_q8, int64_t num_blocks, const int32_t* block_table, int32_t max_blocks,
    int32_t batch, const int32_t* seq_ids, const int64_t* positions, const void* c_kv,
    int64_t c_stride, const void* k_pe, int64_t k_stride, const void* kv_weight,
    const void* pe_weight, float eps, const xmla_yarn_cfg* rope_cfg, int64_t T,
    int32_t* status_dev, void* stream) {
  return append_norm(pool_q8, num_blocks, block_table, max_blocks, batch, seq_ids, positions, c_kv,
                     c_stride, k_pe, k_stride, kv_weight, pe_weight, eps, rope_cfg, T, status_dev,
                     stream, true);
}

extern "C" xmla_status xmla_cache_read_q8(const void* pool_q8, int64_t num_blocks,
                                          const int32_t* block_table, int32_t max_blocks,
                                          int32_t batch, const int32_t* seq_ids,
                                          const int64_t* positions, int64_t T, void* out,
                                          int64_t out_stride, int32_t* status_dev, void* stream) {
  if (T < 0 || num_blocks < 1 || max_blocks < 1 || batch < 1) return XMLA_ERR_SHAPE;
  if (T == 0) return XMLA_OK;
  if (pool_q8 == nullptr || block_table == nullptr || seq_ids == nullptr || positions == nullptr ||
      out == nullptr)
    return XMLA_ERR_INVALID_ARG;
  if ((((uintptr_t)pool_q8) | ((uintptr_t)out)) & 15u || (out_stride & 7) || out_stride < kDRow)
    return XMLA_ERR_INVALID_ARG;
  if (T > (int64_t)0x7fffffff * kReadThreads / kCodeUnits) return XMLA_ERR_SHAPE;
  const RowPlace place{block_table, seq_ids, positions, status_dev, num_blocks, T, max_blocks, batch};
  const int64_t blocks =
      (T * kCodeUnits + kReadUnits * kReadThreads - 1) / (kReadUnits * kReadThreads);
  const cudaError_t e = launch_pdl(read_q8_kernel, dim3((unsigned)blocks), dim3(kReadThreads), 0,
                                   (cudaStream_t)stream, (const uint8_t*)pool_q8, place,
                                   (__nv_bfloat16*)out, out_stride);
  return e == cudaSuccess ? XMLA_OK : XMLA_ERR_CUDA;
}
