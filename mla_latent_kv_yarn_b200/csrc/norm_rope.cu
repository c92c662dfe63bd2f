// Norm of every head of a query or key tensor, with the position rotation in
// the same pass.
//
// y = x / sqrt(mean(x^2) + eps) * w over a head's head_dim values, then YaRN
// RoPE of 64 of them at the row's position; one rounding to bf16.
//
// [P1] "256K 长上下文真能本地用：Xing4.0 原生长上下文的工程代价拆解", section 一: YaRN
//      RoPE of the 64-dim rope part.
#include <cuda_bf16.h>

#include <cstdint>

#include "norm.cuh"

namespace xmla {

namespace {

constexpr int kNormWarps = 8;
constexpr int kNormMaxDim = 1024;
constexpr int kPairs = kDRope / 2;

struct NormRopeArgs {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  const __nv_bfloat16* weight;  // nullable
  const int64_t* positions;     // nullable: no rotation
  int64_t x_row, x_head, o_row, o_head, w_head;
  int32_t n_heads, head_dim, rope_offset;
  int32_t heads_per_block;
  float eps;
};

// Block (row, group of heads); a warp per head.  The rotation's 32 cosines and
// sines depend on the row alone: one warp forms them for the whole block while
// the others fetch their heads.  kVec: 16-byte accesses (lane holds elements
// 8 (lane + 32 k) .. + 7), else single elements lane + 32 k.  kChunks: accesses
// per lane.  Takes what the kernel below does not: heads of more than 256 values, a
// rotated part at an offset not in multiples of 64, and odd sizes or alignments.
// Measured on 4096 rows of 32 heads, rotated (a warp has one head in flight, and all
// wait for the angles): 160 values with offset 96 50 us (1.7 TB/s), 512 96 us (2.8), 1024 172 us
// (3.1), 161 one by one 82 us (1.0).
template <bool kVec, int kChunks>
__global__ void __launch_bounds__(32 * kNormWarps) norm_rope_kernel(const NormRopeArgs a,
                                                                    const RopeTable tab) {
  constexpr int kE = kVec ? 8 : 1;
  __shared__ float cs[2][kPairs];
  __shared__ float part[kNormWarps][kDRope];  // a head's normed rope values
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  const bool rope = a.positions != nullptr;
  const int h_end = min(a.n_heads, (int)(blockIdx.y + 1) * a.heads_per_block);
  bool ready = !rope;
  for (int h = blockIdx.y * a.heads_per_block + warp; h < h_end || !ready; h += kNormWarps) {
    const bool mine = h < h_end;
    float x[kChunks][kE], w[kChunks][kE];
    float sq = 0.f;
    if (mine) {
      const __nv_bfloat16* src = a.x + row * a.x_row + h * a.x_head;
      const __nv_bfloat16* wt = a.weight != nullptr ? a.weight + h * a.w_head : nullptr;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int e0 = kE * (lane + 32 * k);
        const bool in = e0 < a.head_dim;
        if constexpr (kVec) {
          unpack8(in ? *reinterpret_cast<const uint4*>(src + e0) : make_uint4(0u, 0u, 0u, 0u), x[k]);
          const uint4 one = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
          unpack8(in && wt != nullptr ? *reinterpret_cast<const uint4*>(wt + e0) : one, w[k]);
        } else {
          x[k][0] = in ? __bfloat162float(src[e0]) : 0.f;
          w[k][0] = in && wt != nullptr ? __bfloat162float(wt[e0]) : 1.f;
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) sq = fmaf(x[k][e], x[k][e], sq);
      }
    }
    if (!ready) {
      if (warp == kNormWarps - 1)
        rope_cos_sin(a.positions[row], tab.inv_freq[lane], (float)tab.magnitude, &cs[0][lane],
                     &cs[1][lane]);
      __syncthreads();
      ready = true;
      if (!mine) break;
    }
    sq = warp_sum(sq);
    float eps = a.eps;
    const float scale = rms_scale(sq, a.head_dim, eps);
    if (scale != 1.f) {  // the whole warp's
      sq = 0.f;
#pragma unroll
      for (int k = 0; k < kChunks; ++k)
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          x[k][e] *= scale;
          sq = fmaf(x[k][e], x[k][e], sq);
        }
      sq = warp_sum(sq);
      eps = eps * scale * scale;
    }
    const float f = rms_factor(sq, a.head_dim, eps);
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        x[k][e] *= f * w[k][e];
        const int i = kE * (lane + 32 * k) + e - a.rope_offset;
        if (rope && i >= 0 && i < kDRope) part[warp][i] = x[k][e];
      }
    __syncwarp();
    __nv_bfloat16* dst = a.out + row * a.o_row + h * a.o_head;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int e0 = kE * (lane + 32 * k);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int i = e0 + e - a.rope_offset;
        if (rope && i >= 0 && i < kDRope) {
          const float c = cs[0][i & (kPairs - 1)], s = cs[1][i & (kPairs - 1)];
          const float other = part[warp][i ^ kPairs];
          x[k][e] = fmaf(x[k][e], c, i < kPairs ? -other * s : other * s);
        }
      }
      if (e0 < a.head_dim) {
        if constexpr (kVec) *reinterpret_cast<uint4*>(dst + e0) = pack8(x[k]);
        else dst[e0] = __float2bfloat16_rn(x[k][0]);
      }
    }
    __syncwarp();
  }
}

// One head by one warp where its squares leave the range of float32 (rms_scale): a
// rare path of its own, so that the usual one keeps its registers (4096 rows of 32
// heads of 192: 19.1 us with no check of the range, 19.8 us with this, 20.8 us with the
// values scaled in the usual path).  Lane l takes elements l, l + 32, ...: a rotation
// partner is 32 further, so every element is read and written by one lane and out may
// be x.  c, s: the row's cosines and sines.
__device__ __forceinline__ void norm_rope_scaled_head(const NormRopeArgs& a, int64_t row, int h,
                                                      int lane, const float* c, const float* s) {
  const __nv_bfloat16* x = a.x + row * a.x_row + h * a.x_head;
  const __nv_bfloat16* wt = a.weight != nullptr ? a.weight + h * a.w_head : nullptr;
  __nv_bfloat16* y = a.out + row * a.o_row + h * a.o_head;
  float scale = 1.f, sq;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {  // plain, then scaled
    sq = 0.f;
#pragma unroll 1
    for (int e = lane; e < a.head_dim; e += 32) {
      const float v = __bfloat162float(x[e]) * scale;
      sq = fmaf(v, v, sq);
    }
    sq = warp_sum(sq);
    if (pass == 0) scale = rms_scale(sq, a.head_dim, a.eps);
  }
  const float f = rms_factor(sq, a.head_dim, a.eps * scale * scale);
  auto normed = [&](int e) {
    return __bfloat162float(x[e]) * scale * (f * (wt != nullptr ? __bfloat162float(wt[e]) : 1.f));
  };
#pragma unroll 1
  for (int e = lane; e < a.head_dim; e += 32) {
    const int i = a.positions != nullptr ? e - a.rope_offset : -1;
    if (i >= kPairs && i < kDRope) continue;  // with its partner
    const float u = normed(e);
    if (i >= 0 && i < kPairs) {
      const float v = normed(e + kPairs);
      y[e] = __float2bfloat16_rn(fmaf(u, c[i], -v * s[i]));
      y[e + kPairs] = __float2bfloat16_rn(fmaf(v, c[i], u * s[i]));
    } else {
      y[e] = __float2bfloat16_rn(u);
    }
  }
}

// Heads of at most 256 values in 16-byte pieces, the rotated part (if any) at a
// multiple of 64: eight lanes per head, lane l with pieces l, l + 8, ..., so that
// a warp fetches four heads together, every lane takes part for any head_dim in
// multiples of 64, and piece l's rotation partner (32 values on) is piece l ^ 4 of
// the lane four further.  Every warp forms the row's 32 cosines and sines itself,
// one pair per lane, while its heads are on the way: no block-wide wait.
// Measured on 4096 rows of 32 heads of 192 (101 MB, replayed graph): 59 us with a
// warp per head and the angles of a block formed by one warp, 19.8 us (5.1 TB/s) with
// this; bound by memory.  Five blocks per SM instead of four, where the registers
// allow, are worth 1.4 us of it.
template <int kPieces>
__global__ void __launch_bounds__(32 * kNormWarps, kPieces == 4 ? 4 : 5)
    norm_rope_group_kernel(const __grid_constant__ NormRopeArgs a, const RopeTable tab) {
  __shared__ __align__(16) float cs[kNormWarps][2][kPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & 7;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  const int h = (blockIdx.y * kNormWarps + warp) * 4 + (lane >> 3);
  if ((blockIdx.y * kNormWarps + warp) * 4 >= a.n_heads) return;
  const bool mine = h < a.n_heads;
  const int pieces = a.head_dim / 8;
  const __nv_bfloat16* src = a.x + row * a.x_row + (mine ? h : 0) * a.x_head;
  const __nv_bfloat16* wt = a.weight + (mine ? h : 0) * a.w_head;
  uint4 xv[kPieces], wv[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const bool in = l + 8 * k < pieces;
    xv[k] = in ? *reinterpret_cast<const uint4*>(src + 8 * (l + 8 * k)) : make_uint4(0u, 0u, 0u, 0u);
    wv[k] = in && a.weight != nullptr
                ? *reinterpret_cast<const uint4*>(wt + 8 * (l + 8 * k))
                : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  }
  const bool rope = a.positions != nullptr;
  if (rope) {
    rope_cos_sin(a.positions[row], tab.inv_freq[lane], (float)tab.magnitude, &cs[warp][0][lane],
                 &cs[warp][1][lane]);
    __syncwarp();
  }
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    float x[8];
    unpack8(xv[k], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  // heads out of float32's range (marked by -1) are left to the end, when nothing else
  // is kept
  const float f = rms_scale(sq, a.head_dim, a.eps) != 1.f ? -1.f : rms_factor(sq, a.head_dim, a.eps);
  __nv_bfloat16* dst = a.out + row * a.o_row + h * a.o_head;
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    float x[8], w[8];
    unpack8(xv[k], x);
    unpack8(wv[k], w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= f * w[e];
    if (rope && 64 * k == a.rope_offset) {  // uniform
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = __shfl_xor_sync(0xffffffffu, x[e], 4);
        const int i = 8 * (l & 3) + e;
        const float s = cs[warp][1][i];
        x[e] = fmaf(x[e], cs[warp][0][i], l < 4 ? -other * s : other * s);
      }
    }
    if (mine && f >= 0.f && l + 8 * k < pieces) *reinterpret_cast<uint4*>(dst + 8 * (l + 8 * k)) = pack8(x);
  }
  const uint32_t left = __ballot_sync(0xffffffffu, mine && f < 0.f);
  if (left != 0u) {
#pragma unroll 1
    for (int g = 0; g < 4; ++g)
      if ((left >> (8 * g)) & 1u)
        norm_rope_scaled_head(a, row, (blockIdx.y * kNormWarps + warp) * 4 + g, lane, cs[warp][0],
                              cs[warp][1]);
  }
}

template <bool kVec>
static auto norm_kernel(int head_dim) {
  constexpr int kSpan = kVec ? 256 : 32;
  const int chunks = (head_dim + kSpan - 1) / kSpan;
  if constexpr (kVec)
    return chunks <= 1 ? norm_rope_kernel<true, 1>
                       : chunks <= 2 ? norm_rope_kernel<true, 2> : norm_rope_kernel<true, 4>;
  else
    return chunks <= 8 ? norm_rope_kernel<false, 8> : norm_rope_kernel<false, 32>;
}

}  // namespace

}  // namespace xmla

using namespace xmla;

extern "C" xmla_status xmla_norm_rope(const xmla_yarn_cfg* cfg, const void* x,
                                      int64_t x_row_stride, int64_t x_head_stride, void* out,
                                      int64_t out_row_stride, int64_t out_head_stride, int64_t rows,
                                      int32_t n_heads, int32_t head_dim, const void* weight,
                                      int64_t weight_head_stride, float eps, int32_t rope_offset,
                                      const int64_t* positions, void* stream) {
  if (cfg != nullptr) {
    if (!yarn_cfg_ok(cfg)) return XMLA_ERR_INVALID_ARG;
    if (cfg->rotary_dim != kDRope) return XMLA_ERR_SHAPE;
    if (rope_offset < 0 || rope_offset > head_dim - kDRope) return XMLA_ERR_SHAPE;
  }
  if (rows < 0 || rows > 0x7fffffffLL || n_heads < 1 || n_heads > 65535 || head_dim < 1 ||
      head_dim > kNormMaxDim)
    return XMLA_ERR_SHAPE;
  if (!(eps >= 0.f) || !(eps < INFINITY)) return XMLA_ERR_INVALID_ARG;
  if (rows == 0) return XMLA_OK;
  if (x == nullptr || out == nullptr || (cfg != nullptr && positions == nullptr) ||
      x_row_stride < 0 || x_head_stride < 0 || out_row_stride < 0 || out_head_stride < 0 ||
      weight_head_stride < 0)
    return XMLA_ERR_INVALID_ARG;
  if ((((uintptr_t)x) | ((uintptr_t)out) | ((uintptr_t)weight)) & 1u) return XMLA_ERR_INVALID_ARG;
  NormRopeArgs a;
  a.x = (const __nv_bfloat16*)x;
  a.out = (__nv_bfloat16*)out;
  a.weight = (const __nv_bfloat16*)weight;
  a.positions = cfg != nullptr ? positions : nullptr;
  a.x_row = x_row_stride;
  a.x_head = x_head_stride;
  a.o_row = out_row_stride;
  a.o_head = out_head_stride;
  a.w_head = weight_head_stride;
  a.n_heads = n_heads;
  a.head_dim = head_dim;
  a.rope_offset = rope_offset;
  a.eps = eps;
  // few rows: eight heads per block, so that the heads of a row run side by
  // side; many rows: a whole row, so that its angles are formed once
  a.heads_per_block = rows >= 256 ? n_heads : kNormWarps;
  const RopeTable tab = cfg != nullptr ? make_rope_table(cfg) : RopeTable{};
  const bool vec = ((((uintptr_t)x) | ((uintptr_t)out) | ((uintptr_t)weight)) & 15u) == 0 &&
                   ((x_row_stride | x_head_stride | out_row_stride | out_head_stride |
                     weight_head_stride | head_dim) & 7) == 0;
  if (vec && head_dim <= 256 && (cfg == nullptr || rope_offset % 64 == 0)) {
    const dim3 grid((unsigned)rows, (unsigned)((n_heads + 4 * kNormWarps - 1) / (4 * kNormWarps)));
    const int warps = n_heads >= 4 * kNormWarps ? kNormWarps : (n_heads + 3) / 4;
    const cudaError_t e = launch_pdl(head_dim <= 64    ? norm_rope_group_kernel<1>
                                     : head_dim <= 192 ? norm_rope_group_kernel<3>
                                                       : norm_rope_group_kernel<4>,
                                     grid, dim3(32 * warps), 0, (cudaStream_t)stream, a, tab);
    return e == cudaSuccess ? XMLA_OK : XMLA_ERR_CUDA;
  }
  const dim3 grid((unsigned)rows, (unsigned)((n_heads + a.heads_per_block - 1) / a.heads_per_block));
  const cudaError_t e = launch_pdl(vec ? norm_kernel<true>(head_dim) : norm_kernel<false>(head_dim),
                                   grid, dim3(32 * kNormWarps), 0, (cudaStream_t)stream, a, tab);
  return e == cudaSuccess ? XMLA_OK : XMLA_ERR_CUDA;
}
