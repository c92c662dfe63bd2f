// Decode attention of a batch that shares a long prefix: the prefix part,
// computed once for all sequences.
//
// The softmax of a query splits over any partition of the tokens it sees, so
// the prefix that every sequence begins with is one dense problem: R = batch *
// q_len * 32 query rows against n prefix tokens,
//   S = Q K^T           [R, n],   576 products each
//   O = 2^(S - m) C     [R, 512], n products each   (C: the latent columns of K)
// merged afterwards with each sequence's own tokens by their log-sum-exp.  The
// cache rows are read once per row tile instead of once per sequence, and the
// matrix instructions run on 128 rows instead of 32.
//
// [P5] "mHC+MLA+MTP 是什么？拆开给 Agent 用的百亿 MoE", section "MLA：256K 上下文的
//      '内存革命'": the cached latent and rope key serve all heads (and so all
//      rows of one prefix).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>

#include "norm.cuh"
#include "shared_plan.h"
#include "shared_prefix.h"
#include "xmla_device.cuh"

namespace xmla {

namespace {

// ---------------------------------------------------------------- CTA pairs

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// One thread of a converged warp.  Unlike `lane == 0`, the compiler then knows the
// code to be uniform and keeps descriptors and addresses in uniform registers:
// issuing four products, a wait and a commit took 307 cycles instead of 501.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of CTA 0's copy of a shared-memory word of this CTA.
__device__ __forceinline__ uint32_t leader_addr(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
// Arrival that orders no memory accesses (tensor-memory reads are ordered by
// tcgen05.fence).
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait whose acquire covers the other CTA's writes before its arrivals (P
// in its shared memory, its reads of tensor memory).  Phases that complete by
// copies or by tensor-core commits alone are waited for with the plain form,
// which is cheaper: an acquire of cluster scope on every ring slot cost the
// issuing thread more than the products themselves.
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                          int32_t* status, uint64_t limit_ns) {
  return mbar_wait(bar, parity, abort, status, limit_ns) && mbar_try_wait_cluster(bar, parity);
}
// 3-D tile into this CTA's shared memory, counted on its own barrier.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                            int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Rows from `row` on of the column groups from `group` on, into this CTA's shared
// memory; the bytes are counted on CTA 0's barrier.
__device__ __forceinline__ void tma_load_groups_pair(uint32_t dst, const void* tmap, int32_t row,
                                                     int32_t group, uint32_t leader_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(row), "r"(group), "r"(leader_bar)
      : "memory");
}
// D (+)= A B^T over the pair: A's 128 rows and B's rows are half in each CTA.
__device__ __forceinline__ void tc_mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` of both CTAs once everything issued so far has completed.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t v) {
  return pack_f16x2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

constexpr int kRowUnits = kDRow * 2 / 16;  // 72 16-byte units per row

// 16-byte unit u of row `row` in an fp16 operand of n rows, which is stored by
// column groups of 64, [9][n][64]: every tile of the attention is then one copy
// of rows that lie next to each other.
__device__ __forceinline__ int64_t group_unit(int64_t n, int64_t row, int u) {
  return ((int64_t)(u >> 3) * n + row) * 8 + (u & 7);
}

}  // namespace

// ---------------------------------------------------------------- absorbed queries

// q_lat[r, h, :] = q_nope[r, h, :] . W_UK[h] on the tensor cores, one CTA per
// (128 query rows, head, 64 latent columns), K = 128; written as the fp16 row
// of the prefix part and the hi and lo bf16 rows of the own part.  (The CUDA
// cores took 23 us for 32 rows and 40 us for 128, re-reading W_UK for every
// eight rows; here every CTA reads its 16 KB of it once.  Products of 128 columns
// leave half as many CTAs with twice the row pieces to write each; us per call in a
// replayed graph, 128 and 64 columns: 4 sequences over 4,096 tokens 23.1 and 22.7, 32 over 32K 100.7 and 100.0,
// 128 over 16K 188 and 177; 8 with four queries over 192 tokens 28.5 and 29.3.)
// Blocks past the products rotate the rope parts, kRopeRowsPerBlock rows each, and
// then plan the attention's runs and, where it has the own parts, the split-K
// kernel's work items.
constexpr int kAbThreads = 192;  // warp 0 TMA and MMA, warps 2-5 epilogue
constexpr int kRopeRowsPerBlock = 6;
constexpr uint32_t kAbBox = 16384;  // 128 rows x 64 columns
constexpr int kAbCols = 64;         // latent columns of a product
constexpr int kAbParts = kDLatent / kAbCols;
constexpr uint32_t kAbOffBars = 3 * kAbBox;  // after A, two boxes, and B
constexpr uint32_t kAbSmem = kAbOffBars + 32 + 1024;

// hi and lo bf16 parts and the fp16 value of two neighbouring columns
struct QParts {
  uint32_t hi, lo, f16;
};
__device__ __forceinline__ QParts q_parts(float a, float b) {
  const __nv_bfloat162 hv = __floats2bfloat162_rn(a, b);
  const __nv_bfloat162 lv = __floats2bfloat162_rn(a - __low2float(hv), b - __high2float(hv));
  return {*reinterpret_cast<const uint32_t*>(&hv), *reinterpret_cast<const uint32_t*>(&lv),
          pack_f16x2(a, b)};
}

// Eight neighbouring values (16-byte unit u of a 576-wide row) of query row r, head h.
__device__ __forceinline__ void store_query8(const SharedParams& p, int64_t r, int h, int u,
                                         const float (&v)[8]) {
  QParts w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = q_parts(v[2 * k], v[2 * k + 1]);
  if (p.q_ext != nullptr) {
    uint4* ext = reinterpret_cast<uint4*>(p.q_ext);
    ext[(2 * r * kHeads + h) * kRowUnits + u] = make_uint4(w[0].hi, w[1].hi, w[2].hi, w[3].hi);
    ext[((2 * r + 1) * kHeads + h) * kRowUnits + u] =
        make_uint4(w[0].lo, w[1].lo, w[2].lo, w[3].lo);
  }
  reinterpret_cast<uint4*>(p.q16)[group_unit(p.rows, r * kHeads + h, u)] =
      make_uint4(w[0].f16, w[1].f16, w[2].f16, w[3].f16);
}

// The split-K kernel's plan by one warp: unit u = b * q_len + j has w_u pages
// behind the prefix; T is the smallest page count per work item for which
// sum_u max(1, ceil(w_u / T)) fits in the items there are (at least two pages,
// unless all units have fewer); unit u gets ceil(w_u / T) items, consecutive.
constexpr int kPlanPerLane = 8;  // units <= 256
__device__ __forceinline__ void plan_split(const SharedParams& p, int lane) {
  const int per = (p.units + 31) / 32;
  int w[kPlanPerLane];
  int tot = 0, wmax = 0;
#pragma unroll
  for (int k = 0; k < kPlanPerLane; ++k) {
    const int u = lane * per + k;
    w[k] = 0;
    if (k < per && u < p.units) {
      const int64_t n = p.seqlens[u / p.q_len];
      if (n >= 0 && n <= p.max_seqlen)
        w[k] = max(0, (int)((n + kPage - 1) / kPage) - p.prefix_pages);
    }
    tot += w[k];
    wmax = max(wmax, w[k]);
  }
  for (int o = 16; o > 0; o >>= 1) {
    tot += __shfl_xor_sync(0xffffffffu, tot, o);
    wmax = max(wmax, __shfl_xor_sync(0xffffffffu, wmax, o));
  }
  auto items = [&](int T) {  // of this lane's units
    int c = 0;
#pragma unroll
    for (int k = 0; k < kPlanPerLane; ++k)
      if (k < per && lane * per + k < p.units) c += max(1, (w[k] + T - 1) / T);
    return c;
  };
  int lo = max(1, min(2, wmax)), hi = max(lo, wmax);
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    int c = items(mid);
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (c <= p.items) hi = mid;
    else lo = mid + 1;
  }
  const int mine = items(lo);
  int first = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, first, o);
    if (lane >= o) first += x;
  }
  const int total = __shfl_sync(0xffffffffu, first, 31);
  first -= mine;
#pragma unroll
  for (int k = 0; k < kPlanPerLane; ++k) {
    const int u = lane * per + k;
    if (k >= per || u >= p.units) break;
    const int ns = max(1, (w[k] + lo - 1) / lo);
    const int pps = (w[k] + ns - 1) / ns;
    p.unit_tab[u] = make_int2(first, ns);
    for (int s = 0; s < ns; ++s)
      p.work_tab[first + s] = make_int4(u, p.prefix_pages + min(w[k], s * pps),
                                        p.prefix_pages + min(w[k], (s + 1) * pps), 0);
    first += ns;
  }
  for (int k = total + lane; k < p.items; k += 32) p.work_tab[k] = make_int4(-1, 0, 0, 0);
}

// The own places before each sequence, where every run begins and which partials
// every tile has, by one block: threads sum consecutive sequences, a scan adds the
// sums up.
constexpr int kSharedOwnSeqs = (int)(kSharedOwnTokens / kSharedBlock);  // 128 sequences at most
static_assert((kSharedOwnSeqs + 1 + 32) * 4 <= kAbSmem, "the sums of all sequences");
__device__ __forceinline__ void plan_runs(const SharedParams& p, int* cum, int* sums) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int own = 0;
  if (p.own16 != nullptr) {
    const int per = (p.batch + kAbThreads - 1) / kAbThreads;
    const int b0 = min(p.batch, t * per), b1 = min(p.batch, b0 + per);
    int sum = 0;
    for (int b = b0; b < b1; ++b) sum += own_places(p, b);
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += x;
    }
    if (lane == 31) sums[warp] = before;
    __syncthreads();
    before -= sum;
    for (int k = 0; k < warp; ++k) before += sums[k];
    for (int b = b0; b < b1; ++b) {
      cum[b] = before;
      before += own_places(p, b);
      if (b == p.batch - 1) cum[p.batch] = before;
    }
    __syncthreads();
    own = cum[p.batch];
  }
  const SharedWork w = shared_work(p, own);
  for (int run = t; run < p.pairs; run += kAbThreads) p.run_tab[run] = shared_run(p, w, run, cum);
  for (int tile = t; tile < p.tiles; tile += kAbThreads)
    p.tile_tab[tile] = shared_tile_partials(p, w, tile, cum);
  if (p.own16 != nullptr)
    for (int tile = t; tile < p.batch * p.own_tiles; tile += kAbThreads)
      p.tile_tab[p.tiles + tile] = shared_tile_partials(p, w, p.tiles + tile, cum);
}

__global__ void __launch_bounds__(kAbThreads)
    shared_absorb_kernel(const __grid_constant__ CUtensorMap q_map,
                         const __grid_constant__ CUtensorMap wuk_map, const SharedParams p,
                         const RopeTable tab) {
  extern __shared__ uint8_t smem_raw[];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int tiles = (p.units + 127) / 128;
  const int products = tiles * kHeads * kAbParts;
  if ((int)blockIdx.x >= products) {
    pdl_wait();
    pdl_launch_dependents();
    const int blk = (int)blockIdx.x - products;
    const int rope_blocks = (p.units + kRopeRowsPerBlock - 1) / kRopeRowsPerBlock;
    if (blk >= rope_blocks) {
      if (blk == rope_blocks)
        plan_runs(p, reinterpret_cast<int*>(smem_raw) + 32, reinterpret_cast<int*>(smem_raw));
      else if (warp == 0)
        plan_split(p, lane);
      return;
    }
    float2* cs = reinterpret_cast<float2*>(smem_raw);  // [row][pair]
    const int r0 = blk * kRopeRowsPerBlock;
    const int nr = min(kRopeRowsPerBlock, p.units - r0);
    if ((int)threadIdx.x < nr * 32) {
      const int r = r0 + warp;
      float c, s;
      rope_cos_sin((int64_t)p.seqlens[r / p.q_len] - p.q_len + r % p.q_len, tab.inv_freq[lane],
                   (float)tab.magnitude * p.qscale, &c, &s);
      cs[threadIdx.x] = make_float2(c, s);
    }
    __syncthreads();
    // a thread takes eight pairs (8 g .. 8 g + 7, and + 32) of a head
    for (int e = threadIdx.x; e < nr * kHeads * 4; e += kAbThreads) {
      const int rr = e / (kHeads * 4), h = (e >> 2) % kHeads, g = e & 3;
      const int64_t r = r0 + rr;
      const uint4* x = reinterpret_cast<const uint4*>(p.q + (r * kHeads + h) * kDQ + kDNope);
      float a[8], b[8], ya[8], yb[8];
      unpack8(x[g], a);
      unpack8(x[g + 4], b);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 t = cs[rr * 32 + 8 * g + k];
        ya[k] = fmaf(a[k], t.x, -b[k] * t.y);
        yb[k] = fmaf(b[k], t.x, a[k] * t.y);
      }
      store_query8(p, r, h, kDLatent / 8 + g, ya);
      store_query8(p, r, h, kDLatent / 8 + 4 + g, yb);
    }
    return;
  }
  uint32_t base = smem_u32(smem_raw);
  base += (1024u - (base & 1023u)) & 1023u;
  const uint32_t bar_full = base + kAbOffBars, bar_done = bar_full + 8, tmem_slot = bar_full + 16;
  const int n0 = ((int)blockIdx.x % kAbParts) * kAbCols;
  const int h = ((int)blockIdx.x / kAbParts) % kHeads;
  const int r0 = ((int)blockIdx.x / kAbParts) / kHeads * 128;
  if (threadIdx.x == 0) {
    mbar_init(bar_full, 1);
    mbar_init(bar_done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kAbCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");
  if (warp == 0) {
    const bool one = elect_one();
    if (one) {
      mbar_arrive_expect_tx(bar_full, 3 * kAbBox);
      tma_prefetch_desc(&q_map);
    }
    // the weights too may come from the kernel launched just before (loading them
    // ahead of the wait gained nothing measurable)
    pdl_wait();
    pdl_launch_dependents();
    if (one) {
      // B: W_UK[h] rows, columns n0..n0+63; A: q_nope columns of head h, rows r0..
      tma_load_2d(base + 2 * kAbBox, &wuk_map, n0, h * kDNope, bar_full);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        tma_load_3d(base + j * kAbBox, &q_map, 64 * j, h, r0, bar_full);
      if (mbar_wait(bar_full, 0, nullptr, p.status, p.wait_limit_ns)) {
        constexpr uint32_t idesc = idesc_bf16_f32(128, kAbCols, false, true);
        const uint64_t a = smem_desc_sw128(base, 16, 1024);
        const uint64_t b = smem_desc_sw128(base + 2 * kAbBox, kAbBox, 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc_mma_bf16(tmem, a + (((k >> 2) * kAbBox + (k & 3) * 32) >> 4), b + ((k * 2048) >> 4),
                      idesc, k != 0 ? 1u : 0u);
      }
      tc_commit(bar_done);
    }
  } else if (warp == 1) {
    pdl_wait();
    pdl_launch_dependents();
  } else {
    pdl_wait();
    pdl_launch_dependents();
    const int quarter = warp & 3;
    const bool ok = mbar_wait(bar_done, 0, nullptr, p.status, p.wait_limit_ns);
    __syncwarp();
    tc_fence_after();
    // Each thread converts 32 columns of its row; the warp passes them through its
    // part of the (now idle) operand tiles, so that a store instruction writes 64
    // contiguous bytes of eight rows instead of 16 bytes of 32 (128 rows: 12.8 us
    // without, 11.6 us with).
    constexpr uint32_t kPitch = 80;  // 64 bytes of a row and 16 between rows
    uint8_t* stage = smem_raw + (base - smem_u32(smem_raw)) + quarter * 3 * 32 * kPitch;
    const int parts = p.q_ext != nullptr ? 3 : 1;  // fp16, hi, lo
    const int srow = lane >> 2, piece = lane & 3;
#pragma unroll 1
    for (int c = 0; c < kAbCols / 32; ++c) {
      if (r0 + 32 * quarter >= p.units) break;  // the warp's rows are all padding
      float v[32];
      tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + 32 * c, v);
      tc_wait_ld();
      if (!__all_sync(0xffffffffu, ok)) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        QParts w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = q_parts(v[8 * k + 2 * e] * p.qscale, v[8 * k + 2 * e + 1] * p.qscale);
        uint4* dst = reinterpret_cast<uint4*>(stage + lane * kPitch + 16 * k);
        dst[0] = make_uint4(w[0].f16, w[1].f16, w[2].f16, w[3].f16);
        dst[32 * kPitch / 16] = make_uint4(w[0].hi, w[1].hi, w[2].hi, w[3].hi);
        dst[2 * 32 * kPitch / 16] = make_uint4(w[0].lo, w[1].lo, w[2].lo, w[3].lo);
      }
      __syncwarp();
      const int u = (n0 + 32 * c) / 8 + piece;  // 16-byte unit of the 576-wide row
      for (int part = 0; part < parts; ++part) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int rr = srow + 8 * n;
          const int64_t r = r0 + 32 * quarter + rr;
          if (r >= p.units) continue;
          const uint4 val =
              *reinterpret_cast<const uint4*>(stage + (part * 32 + rr) * kPitch + 16 * piece);
          if (part == 0)
            reinterpret_cast<uint4*>(p.q16)[group_unit(p.rows, r * kHeads + h, u)] = val;
          else
            reinterpret_cast<uint4*>(
                p.q_ext)[((2 * r + part - 1) * kHeads + h) * kRowUnits + u] = val;
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, kAbCols);
  }
}

cudaError_t launch_shared_absorb(const CUtensorMap& q_map, const CUtensorMap& wuk_map,
                                 const SharedParams& p, const RopeTable& tab, cudaStream_t st) {
  static bool done[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        shared_absorb_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAbSmem);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  const int64_t blocks = (int64_t)((p.units + 127) / 128) * kHeads * kAbParts +
                         (p.units + kRopeRowsPerBlock - 1) / kRopeRowsPerBlock +
                         1 + (p.work_tab != nullptr ? 1 : 0);
  return launch_pdl(shared_absorb_kernel, dim3((unsigned)blocks), dim3(kAbThreads), kAbSmem, st,
                    q_map, wuk_map, p, tab);
}

// ---------------------------------------------------------------- fp16 copies

// The prefix rows and the own rows as fp16: both operands of a matrix product
// share a type, and with 11 significant bits instead of 8 neither the query nor
// the probabilities add to the error of a bf16 result (a single bf16 query alone
// adds 2^-9 of each score).  Bound by memory: 1152 B in and out per token.  Rows
// past a sequence's end are zeros up to the end of their block of 256.
//
// Runs beside the absorb: it starts once every CTA of that kernel (the split-K
// kernel, where that comes between) has started, and those let it start only
// after their own wait, so all work before this call is complete and nothing
// needs waiting for to begin with.  It waits before it ends: its completion then
// means that of the kernels before it.
//
// The cache rows are read once, the copies many times (by every row tile) right
// after: the rows are loaded to be evicted first and the copies stored to be
// evicted last (8 x 4 queries over 128K tokens, 151 MB of copies, in bursts too short
// for the power limit: 313..328 us per call with plain accesses, 293..302 us so).
constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = kPage * kRowUnits / 2;  // half a page per block

__device__ __forceinline__ uint64_t policy_evict_last() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void store_keep(uint4* dst, const uint4& v, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(dst), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w), "l"(policy)
               : "memory");
}

__global__ void __launch_bounds__(kCopyThreads) shared_copy_kernel(const SharedParams p) {
  pdl_launch_dependents();
  int64_t page = blockIdx.x >> 1;  // page of the destination
  const int half = blockIdx.x & 1;
  int32_t blk;
  int valid = kPage;  // rows of the page that hold tokens
  __half* dst16 = p.kv16;
  int64_t n = (int64_t)p.prefix_pages * kPage;
  if (page < p.prefix_pages) {
    blk = p.prefix_table[page];
  } else {
    page -= p.prefix_pages;
    const int pages = p.own_pad / kPage;
    const int b = (int)(page / pages), i = (int)(page % pages);
    const int tokens = own_tokens(p, b);
    if (i >= own_blocks(tokens) * (kSharedBlock / kPage)) {
      pdl_wait();
      return;
    }
    valid = max(0, min(kPage, tokens - i * kPage));
    blk = valid > 0 ? p.block_table[(int64_t)b * p.max_blocks + p.prefix_pages + i] : 0;
    dst16 = p.own16;
    n = (int64_t)p.batch * p.own_pad;
  }
  if (blk < 0 || (int64_t)blk >= p.num_blocks) {
    if (threadIdx.x == 0) record_status(p.status, XMLA_ERR_DEVICE_OOB);
    blk = 0;
    valid = 0;
  }
  const uint4* src = reinterpret_cast<const uint4*>(p.pool) + (int64_t)blk * kPage * kRowUnits;
  uint4* dst = reinterpret_cast<uint4*>(dst16);
  const uint64_t keep = policy_evict_last();
  constexpr int kPer = kCopyUnits / kCopyThreads;  // 9
  const int u0 = half * kCopyUnits + threadIdx.x;
  uint4 v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int u = u0 + k * kCopyThreads;
    v[k] = u < valid * kRowUnits ? __ldcs(src + u) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int u = u0 + k * kCopyThreads;
    store_keep(dst + group_unit(n, page * kPage + u / kRowUnits, u % kRowUnits),
               make_uint4(bf16x2_to_f16x2(v[k].x), bf16x2_to_f16x2(v[k].y),
                          bf16x2_to_f16x2(v[k].z), bf16x2_to_f16x2(v[k].w)),
               keep);
  }
  pdl_wait();
}

cudaError_t launch_shared_copy(const SharedParams& p, cudaStream_t st) {
  const int64_t pages =
      p.prefix_pages + (p.own16 != nullptr ? (int64_t)p.batch * (p.own_pad / kPage) : 0);
  return launch_pdl(shared_copy_kernel, dim3(2 * (unsigned)pages), dim3(kCopyThreads), 0, st, p);
}

// ---------------------------------------------------------------- whole block table

__global__ void __launch_bounds__(256)
    shared_table_kernel(const SharedParams p, int32_t* __restrict__ table, int32_t cols,
                        int32_t* __restrict__ lens) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e < p.batch) {
    const int n = own_tokens(p, (int)e);
    lens[e] = n > 0 ? p.prefix_pages * kPage + n : 0;
  }
  if (e >= (int64_t)p.batch * cols) return;
  const int b = (int)(e / cols), i = (int)(e % cols);
  table[e] = i < p.prefix_pages ? p.prefix_table[i] : p.block_table[(int64_t)b * p.max_blocks + i];
}

cudaError_t launch_shared_table(const SharedParams& p, int32_t* table, int32_t cols, int32_t* lens,
                                cudaStream_t st) {
  const int64_t blocks = ((int64_t)p.batch * cols + 255) / 256;
  return launch_pdl(shared_table_kernel, dim3((unsigned)blocks), dim3(256), 0, st, p, table, cols,
                    lens);
}

// ---------------------------------------------------------------- attention

// A pair of CTAs takes 128 query rows, 64 per CTA, and blocks of 256 tokens:
//   QK  S[128, 256] = Q K^T: cta_group::2, M = 128, N = 256 (128 tokens from
//       each CTA), K = 576 in 9 chunks of 64;
//   PV  O[128, 512] += P C: two N = 256 products (128 latent columns from each
//       CTA), K = 256 tokens.
// With M = 128 over the pair each CTA holds its 64 rows' accumulators on all
// 128 lanes (lanes 64..127: the second half of the columns), so O takes 256 of
// the 512 tensor-memory columns and two S buffers the other 256; a single CTA
// with 128 rows would need all of them for O.  N = 256 keeps the tensor pipe
// at its full rate (measured: 4096 products per cycle and SM; N = 128: 2222).
// Operands stream through one ring of 16 KB slots in the order in which the
// products are issued, QK(i + 1) ahead of PV(i):
//   K chunk: 128 tokens of this CTA x 64 columns;
//   V chunk: 64 tokens x the 128 latent columns of this CTA (MN-major).
constexpr int kSharedSoftmaxWarps = 8;
constexpr int kSharedWarps = 3 + kSharedSoftmaxWarps;  // TMA, MMA, softmax, TMA
constexpr int kSharedThreads = 32 * kSharedWarps;
constexpr int kSharedSoftmaxThreads = 32 * kSharedSoftmaxWarps;
constexpr int kRing = 7;
constexpr uint32_t kSlotBytes = 16384;
constexpr uint32_t kShOffQ = 0;                                  // 9 chunks of 64 rows x 128 B
constexpr uint32_t kShQBytes = 9 * 8192;
constexpr uint32_t kShOffP = kShOffQ + kShQBytes;                // 4 atoms of 64 rows x 128 B
constexpr uint32_t kShOffRing = kShOffP + 4 * 8192;
constexpr uint32_t kShOffBars = kShOffRing + kRing * kSlotBytes;
enum : int {
  kShFull = 0,                 // CTA 0: bytes of both CTAs
  kShEmpty = kShFull + kRing,  // both
  kShQFull = kShEmpty + kRing, // CTA 0
  kShQEmpty,                   // both
  kShSFull,                    // both, 2
  kShSFree = kShSFull + 2,     // CTA 0, 2
  kShPFull = kShSFree + 2,     // CTA 0: its own warps, and one for all of CTA 1's
  kShPPeer,                    // CTA 1: its warps
  kShPvDone,                   // both
  kShOFree,                    // CTA 0
  kShDrain,                    // CTA 0
  kShBars
};
constexpr uint32_t kShOffRed = (kShOffBars + kShBars * 8 + 15) & ~15u;  // [4][64] floats
constexpr uint32_t kShOffTmem = kShOffRed + 4 * 64 * 4;
constexpr uint32_t kShOffAbort = kShOffTmem + 4;
constexpr uint32_t kShSmem = kShOffAbort + 12 + 1024;
static_assert(kShSmem <= 232448, "shared memory per CTA");
constexpr uint32_t kShColO = 0, kShColS = 256;
// A row's reference maximum is raised only when a score exceeds it by kShLazy
// (log2 units).  Probabilities are 2^(s - m + kShUp): up to 2^15, inside fp16,
// with 2^-31 of the reference still representable for the many small ones.
constexpr float kShLazy = 8.f, kShUp = 7.f;

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kSharedThreads, 1)
    shared_attn_kernel(const __grid_constant__ CUtensorMap q_map,
                       const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map,
                       const __grid_constant__ CUtensorMap ko_map,
                       const __grid_constant__ CUtensorMap vo_map, const SharedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint32_t base = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (base & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  base += pad;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kShOffAbort);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  auto bar = [&](int i) -> uint32_t { return base + kShOffBars + 8u * (uint32_t)i; };
  auto wait = [&](int i, uint32_t parity) {
    return mbar_wait(bar(i), parity, abort_flag, p.status, p.wait_limit_ns);
  };
  auto wait_pair = [&](int i, uint32_t parity) {
    return pair_wait(bar(i), parity, abort_flag, p.status, p.wait_limit_ns);
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kShBars; ++i) {
      const bool by_warps = i == kShSFree || i == kShSFree + 1 || i == kShOFree;
      mbar_init(bar(i), by_warps         ? 2 * kSharedSoftmaxWarps
                        : i == kShPFull ? kSharedSoftmaxWarps + 1
                        : i == kShPPeer ? kSharedSoftmaxWarps
                                        : 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&q_map);
    tma_prefetch_desc(&k_map);
    tma_prefetch_desc(&v_map);
    tma_prefetch_desc(&ko_map);
    tma_prefetch_desc(&vo_map);
  }
  if (warp == 1) tmem_alloc_pair(base + kShOffTmem, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kShOffTmem);
  pdl_wait();
  pdl_launch_dependents();

  const int run = blockIdx.x / 2;  // this pair's
  Segments sg;
  sg.at = p.run_tab[run];

  if (warp == 0 || warp == kSharedWarps - 1) {
    // ================================================================ TMA producers (each CTA)
    // Two warps take the chunks in turn: one alone needs longer to wait for a
    // slot, arm it and issue the copy than the products on it take.
    const uint32_t mine = warp == 0 ? 0u : 1u;
    if (elect_one()) {
      const uint32_t full0 = leader_addr(bar(kShFull)), q_full = leader_addr(bar(kShQFull));
      int slot = 0;
      uint32_t phase = 0, turn = 0;
      bool ok = true;
      // Chunks in the order of the products: K of a block, then V of the block
      // before it, across segments too.
      auto chunk = [&](const CUtensorMap* map, int32_t row, int32_t group) {
        if (turn == mine) {
          if (!(ok = wait(kShEmpty + slot, phase ^ 1u))) return;
          if (rank == 0) mbar_arrive_expect_tx(bar(kShFull + slot), 2 * kSlotBytes);
          tma_load_groups_pair(base + kShOffRing + slot * kSlotBytes, map, row, group,
                               full0 + 8u * (uint32_t)slot);
        }
        turn ^= 1u;
        slot = slot == kRing - 1 ? 0 : slot + 1;
        phase ^= slot == 0 ? 1u : 0u;
      };
      const CUtensorMap* v_prev = nullptr;  // V of the last block whose K was loaded
      int32_t y_prev = 0;
      auto load_v = [&]() {
        for (int c = 0; c < 8 && ok; ++c)
          chunk(v_prev, y_prev + 64 * (c >> 1), 4 * (c & 1) + 2 * (int32_t)rank);
      };
      for (int seg = 0; ok && sg.next(p); ++seg) {
        const CUtensorMap* km = sg.is_own ? &ko_map : &k_map;
        const int32_t y0 =
            (int32_t)((sg.is_own ? (int64_t)sg.seq * p.own_pad : 0) + (int64_t)sg.b0 * kSharedBlock);
        if (mine == 0) {
          if (seg > 0 && !(ok = wait(kShQEmpty, (uint32_t)((seg - 1) & 1)))) break;
          if (rank == 0) mbar_arrive_expect_tx(bar(kShQFull), 2 * kShQBytes);
          tma_load_groups_pair(base + kShOffQ, &q_map, (int32_t)(sg.row0(p) + rank * 64), 0, q_full);
        }
        for (int i = 0; i < sg.n && ok; ++i) {
          const int32_t y = y0 + i * kSharedBlock;
          for (int c = 0; c < 9 && ok; ++c) chunk(km, y + (int32_t)rank * 128, c);
          if (v_prev != nullptr && ok) load_v();
          v_prev = sg.is_own ? &vo_map : &v_map;
          y_prev = y;
        }
      }
      if (v_prev != nullptr && ok) load_v();
      if (!ok) {
        // copies still in flight land within microseconds: give them 2 ms
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ================================================================ matrix products (CTA 0)
    if (rank != 0) {
      // CTA 1: pass on that its P is written.  One thread with nothing outstanding
      // makes the cluster-wide release, instead of eight warps right behind their
      // stores (128 sequences over 16K tokens: 127 -> 117 us).
      if (elect_one()) {
        uint32_t t = 0;
        bool ok = true;
        while (ok && sg.next(p))
          for (int i = 0; i < sg.n && (ok = wait(kShPPeer, t & 1u)); ++i, ++t)
            mbar_arrive_cluster(leader_addr(bar(kShPFull)));
      }
    } else if (elect_one()) {
      constexpr uint32_t idesc_qk = idesc_f16_f32(128, 256, false, false);
      constexpr uint32_t idesc_pv = idesc_f16_f32(128, 256, false, true);
      const uint64_t d_q = smem_desc_sw128(base + kShOffQ, 16, 1024);
      const uint64_t d_p = smem_desc_sw128(base + kShOffP, 16, 1024);
      const uint64_t d_k = smem_desc_sw128(base + kShOffRing, 16, 1024);
      const uint64_t d_v = smem_desc_sw128(base + kShOffRing, 8192, 1024);
      // A chunk's barrier is probed while the products before it are issued, so
      // that a chunk that is there costs no wait: the pipe then runs without gaps
      // (256 cycles per chunk of four products, 307 with a wait each time).
      int slot = 0;
      uint32_t phase = 0;
      uint32_t t = 0, t_pv = 0;  // blocks issued so far, over all segments
      bool ok = true, ready = false;
      // PV of the block before the one whose scores were issued last; o_first: it
      // begins its segment's O, and the segment before it has a number
      bool o_first = false;
      int o_seg = 0;
      auto pv = [&]() {
        // the previous segment's O has been read
        if (o_first && o_seg > 0) ok = wait_pair(kShOFree, (uint32_t)((o_seg - 1) & 1));
        if (!ok || !(ok = wait_pair(kShPFull, t_pv & 1u))) return;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (!ready && !(ok = wait(kShFull + slot, phase))) return;
          const int cur = slot;
          const uint64_t b = d_v + ((uint32_t)slot * (kSlotBytes >> 4));
          slot = slot == kRing - 1 ? 0 : slot + 1;
          phase ^= slot == 0 ? 1u : 0u;
          ready = mbar_test(bar(kShFull + slot), phase);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_pair(tmem + kShColO + 128 * (c & 1), d_p + (((c >> 1) * 8192 + 32 * k) >> 4),
                        b + ((k * 2048) >> 4), idesc_pv, (!o_first || (c >> 1 | k) != 0) ? 1u : 0u);
          tc_commit_pair(bar(kShEmpty + cur));
        }
        tc_commit_pair(bar(kShPvDone));
        ++t_pv;
      };
      for (int seg = 0; ok && sg.next(p); ++seg) {
        ok = wait(kShQFull, (uint32_t)(seg & 1));
        for (int i = 0; i < sg.n && ok; ++i) {
          const uint32_t sb = t & 1u;
          if (t >= 2) ok = wait_pair(kShSFree + sb, ((t - 2) >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + kShColS + 128 * sb;
#pragma unroll
          for (int c = 0; c < 9; ++c) {
            if (!ready && !(ok = wait(kShFull + slot, phase))) break;
            const int cur = slot;
            const uint64_t b = d_k + ((uint32_t)slot * (kSlotBytes >> 4));
            slot = slot == kRing - 1 ? 0 : slot + 1;
            phase ^= slot == 0 ? 1u : 0u;
            ready = mbar_test(bar(kShFull + slot), phase);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_pair(d, d_q + (((uint32_t)c * 8192 + 32 * k) >> 4), b + 2 * k, idesc_qk,
                          (c | k) != 0 ? 1u : 0u);
            tc_commit_pair(bar(kShEmpty + cur));
          }
          if (!ok) break;
          tc_commit_pair(bar(kShSFull + sb));
          if (i == sg.n - 1) tc_commit_pair(bar(kShQEmpty));
          // the block before, of this segment or the last of the one before
          if (t > 0) pv();
          ++t;
          o_first = i == 0;
          o_seg = seg;
        }
      }
      if (t > 0 && ok) pv();
      // everything issued must finish before tensor memory is freed
      tc_commit_pair(bar(kShDrain));
      mbar_wait(bar(kShDrain), 0, nullptr, p.status, p.wait_limit_ns);
    }
  } else {
    // ================================================================ softmax and epilogue
    // Tensor-memory lane L holds row L % 64 of this CTA; its S columns are
    // tokens 128 (L / 64) .. + 127 of the block, its O columns of product n the
    // latent columns 256 n + 128 (L / 64) .. + 127.  Two warps share a lane
    // quarter, 64 S columns (one product's O columns) each.
    const int quarter = warp & 3;
    const int ch = (warp - 2) >> 2;
    const int L = 32 * quarter + lane;
    const int row = L & 63, hb = L >> 6;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
    float* red = reinterpret_cast<float*>(smem + kShOffRed);
    const int atom = 2 * hb + ch;  // this thread's 64 tokens of the block
    uint8_t* p_row = smem + kShOffP + atom * 8192 + row * 128;
    const uint32_t lead_s[2] = {leader_addr(bar(kShSFree)), leader_addr(bar(kShSFree + 1))};
    const uint32_t lead_o = leader_addr(bar(kShOFree));
    int64_t t = 0;     // blocks so far, over all segments
    bool ok = true;    // the same in all softmax threads: they leave together
    bool late = false; // a wait of this thread ran out; told at the next vote
    const int tile_row = (int)rank * 64 + row;
    while (sg.next(p)) {
      const int n = sg.n;
      // tokens this row sees, counted from the segment's first block: all of the
      // prefix; of its own part those up to its query's position
      int64_t sees = (int64_t)p.prefix_pages * kPage;
      if (sg.is_own)
        sees = sg.tokens - p.q_len + 1 +
               min(p.q_len - 1, (sg.tile - sg.seq * p.own_tiles) * kSharedOwnQ + tile_row / kHeads);
      sees -= (int64_t)sg.b0 * kSharedBlock;
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < n && ok; ++i, ++t) {
        const int sb = (int)(t & 1);
        late |= !wait(kShSFull + sb, (uint32_t)((t >> 1) & 1));
        __syncwarp();
        tc_fence_after();
        float s[64];
#pragma unroll
        for (int c = 0; c < 2; ++c)
          tmem_ld32(t_lane + kShColS + 128 * sb + 64 * ch + 32 * c,
                    *reinterpret_cast<float(*)[32]>(s + 32 * c));
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(lead_s[sb]);
        if (sees - i * kSharedBlock < 64 * atom + 64) {
          const int left = (int)max((int64_t)0, sees - i * kSharedBlock - 64 * atom);
#pragma unroll
          for (int k = 0; k < 64; ++k) s[k] = k < left ? s[k] : -INFINITY;
        }
        float mx = s[0];
#pragma unroll
        for (int k = 1; k < 64; ++k) mx = fmaxf(mx, s[k]);
        // one vote per block: has a row's maximum moved, or a wait run out?
        if (named_bar_or(1, kSharedSoftmaxThreads, mx > m + kShLazy || late)) {
          // O and the P buffer are free once the block before is accumulated
          if (t > 0) late |= !wait(kShPvDone, (uint32_t)((t - 1) & 1));
          red[atom * 64 + row] = mx;
          if (named_bar_or(1, kSharedSoftmaxThreads, late)) { ok = false; break; }
          const float mn = fmaxf(fmaxf(fmaxf(red[row], red[64 + row]), fmaxf(red[128 + row], red[192 + row])), m);
          const float alpha = mn == -INFINITY ? 1.f : ex2(m - mn);
          if (i > 0) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              float o[32];
              const uint32_t ta = t_lane + kShColO + 128 * ch + 32 * c;
              tmem_ld32(ta, o);
              tc_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= alpha;
              tmem_st32(ta, o);
            }
            tc_wait_st();
          }
          l *= alpha;
          m = mn;
          named_bar_sync(1, kSharedSoftmaxThreads);  // red is read before it is written again
        }
        const float ref = (m == -INFINITY ? 0.f : m) - kShUp;
        uint32_t w[32];
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float a = ex2(s[2 * k] - ref), b = ex2(s[2 * k + 1] - ref);
          l0 += a;
          l1 += b;
          w[k] = pack_f16x2(a, b);
        }
        l += l0 + l1;
        if (t > 0) late |= !wait(kShPvDone, (uint32_t)((t - 1) & 1));
#pragma unroll
        for (int u = 0; u < 8; ++u)
          *reinterpret_cast<uint4*>(p_row + ((u ^ (row & 7)) << 4)) =
              make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(rank == 0 ? kShPFull : kShPPeer));
      }
      // ---- the segment's partial: unnormalised O, reference maximum and sum
      if (ok) late |= !wait(kShPvDone, (uint32_t)((t - 1) & 1));
      ok = !named_bar_or(1, kSharedSoftmaxThreads, !ok || late);
      // (of an own tile, the rows of its queries only)
      const bool stored = !sg.is_own || (tile_row < p.own_rows &&
                                         sg.row0(p) + tile_row < (int64_t)(sg.seq + 1) * p.q_len * kHeads);
      const int64_t slot = sg.slot(run);
      const int slot_rows = sg.is_own ? p.own_rows : kSharedRows;
      if (ok) {
        // four columns at a time, the 32 rows of the warp side by side: 512 bytes
        // per store (rows of 2 KB each took 10,000 cycles per segment, this 700)
        tc_fence_after();
        float4* dst = reinterpret_cast<float4*>(sg.is_own ? p.own_o : p.part_o) +
                      (slot * (kDLatent / 4) + 64 * ch + 32 * hb) * slot_rows + tile_row;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float o[32];
          tmem_ld32(t_lane + kShColO + 128 * ch + 32 * c, o);
          tc_wait_ld();
          if (stored) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[(8 * c + k) * slot_rows] =
                  make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(lead_o);
      }
      red[atom * 64 + row] = l;
      named_bar_sync(1, kSharedSoftmaxThreads);
      if (hb == 0 && ch == 0 && stored) {
        const float sum = red[row] + red[64 + row] + red[128 + row] + red[192 + row];
        float2* ml = reinterpret_cast<float2*>(sg.is_own ? p.own_ml : p.part_ml);
        ml[slot * slot_rows + tile_row] = ok ? make_float2(m - kShUp, sum) : make_float2(-INFINITY, 0.f);
      }
      named_bar_sync(1, kSharedSoftmaxThreads);
    }
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync_all();  // neither CTA leaves while the other may still reach its shared memory
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem, 512);
  }
}

cudaError_t launch_shared_attn(const CUtensorMap& q_map, const CUtensorMap& k_map,
                               const CUtensorMap& v_map, const CUtensorMap& ko_map,
                               const CUtensorMap& vo_map, const SharedParams& p, cudaStream_t st) {
  static bool done[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        shared_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShSmem);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  return launch_pdl(shared_attn_kernel, dim3(2 * (unsigned)p.pairs), dim3(kSharedThreads),
                    kShSmem, st, q_map, k_map, v_map, ko_map, vo_map, p);
}

// ---------------------------------------------------------------- merge

// A block per (query, 32 latent columns): lane h of each warp has head h's row, a
// warp four columns.  A row's partials -- those of the prefix, then those of its
// own part -- are weighted by 2^(m - M) and divided by the sum; the latent row
// goes out as two bf16 parts, hi = bf16(o) and lo = bf16(o - hi), for the W_UV
// product.  Bound by latency: a thread loads its (m, sum) and values of kDepth
// partials together, whether they turn out to count or not.  A sequence whose
// length leaves its new tokens outside its own pages gets zero rows.
constexpr int kMergeThreads = 256;
constexpr int kMergeCols = 32;
constexpr int kMergeParts = kDLatent / kMergeCols;  // 16

template <int kDepth>
__global__ void __launch_bounds__(kMergeThreads) shared_merge_kernel(const SharedParams p) {
  // the block's 32 x 32 values, hi and lo parts
  __shared__ __align__(16) uint32_t out_s[2][kHeads][kMergeCols / 2 + 4];
  const int unit = blockIdx.x / kMergeParts;  // b * q_len + j
  const int part = blockIdx.x % kMergeParts;
  const int h = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = unit / p.q_len, j = unit - b * p.q_len;
  // Where the partials are depends on the lengths and the plan alone.  Those are
  // complete before this kernel starts: the attention kernel lets it start only
  // after its own wait for the kernels before it.
  const int tokens = own_tokens(p, b);
  const bool own16 = p.own16 != nullptr;
  const int64_t r = (int64_t)unit * kHeads + h;
  const int2 seg = p.tile_tab[(int64_t)unit * kHeads / kSharedRows];  // the same for all heads
  const int2 own = own16 ? p.tile_tab[p.tiles + b * p.own_tiles + j / kSharedOwnQ]
                   : p.work_tab != nullptr ? p.unit_tab[unit]
                                           : make_int2(unit, 1);
  const int segs = seg.y, owns = own.y;
  // rows of a partial, this head's among them, and the step between its column groups
  const int seg_row = (int)(r % kSharedRows), own_row = own16 ? (j % kSharedOwnQ) * kHeads + h : h;
  const int own_rows = own16 ? p.own_rows : kHeads;
  const int64_t seg0 = seg.x, own0 = own.x;
  const int col4 = (kMergeCols / 4) * part + warp;  // this warp's group of four columns
  pdl_wait();
  pdl_launch_dependents();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, sum = 0.f;
  const int n = tokens > 0 ? segs + owns : 0;
  for (int k0 = 0; k0 < n; k0 += kDepth) {
    float2 ml[kDepth];
    float4 v[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      const int k = k0 + i;
      ml[i] = make_float2(-INFINITY, 0.f);
      if (k < segs) {
        const int64_t slot = seg0 + k;
        ml[i] = reinterpret_cast<const float2*>(p.part_ml)[slot * kSharedRows + seg_row];
        v[i] = reinterpret_cast<const float4*>(
            p.part_o)[(slot * (kDLatent / 4) + col4) * kSharedRows + seg_row];
      } else if (k < n) {
        const int64_t slot = own0 + k - segs;
        ml[i] = reinterpret_cast<const float2*>(p.own_ml)[slot * own_rows + own_row];
        v[i] = reinterpret_cast<const float4*>(
            p.own_o)[own16 ? (slot * (kDLatent / 4) + col4) * own_rows + own_row
                           : (slot * own_rows + own_row) * (kDLatent / 4) + col4];
      }
    }
    float Mn = M;
#pragma unroll
    for (int i = 0; i < kDepth; ++i) Mn = fmaxf(Mn, ml[i].y == 0.f ? -INFINITY : ml[i].x);
    const float old = M == -INFINITY ? 0.f : ex2(M - Mn);
    M = Mn;
    sum *= old;
    acc.x *= old;
    acc.y *= old;
    acc.z *= old;
    acc.w *= old;
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      if (ml[i].y == 0.f) continue;  // a partial of no token may hold anything
      const float wk = ex2(ml[i].x - M);
      sum = fmaf(wk, ml[i].y, sum);
      acc.x = fmaf(wk, v[i].x, acc.x);
      acc.y = fmaf(wk, v[i].y, acc.y);
      acc.z = fmaf(wk, v[i].z, acc.z);
      acc.w = fmaf(wk, v[i].w, acc.w);
    }
  }
  if (tokens == 0 && part == 0 && threadIdx.x == 0) record_status(p.status, XMLA_ERR_DEVICE_OOB);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const QParts x = q_parts(acc.x * inv, acc.y * inv);
  const QParts y = q_parts(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(&out_s[0][h][2 * warp]) = make_uint2(x.hi, y.hi);
  *reinterpret_cast<uint2*>(&out_s[1][h][2 * warp]) = make_uint2(x.lo, y.lo);
  __syncthreads();
  // 64 contiguous bytes of a row by four threads; half the block per part
  const int which = threadIdx.x >> 7, row = (threadIdx.x >> 2) & 31, u = threadIdx.x & 3;
  uint4* dst = reinterpret_cast<uint4*>((which == 0 ? p.o_hi : p.o_lo) +
                                        ((int64_t)unit * kHeads + row) * kDLatent + kMergeCols * part);
  dst[u] = *reinterpret_cast<const uint4*>(&out_s[which][row][4 * u]);
}

cudaError_t launch_shared_merge(const SharedParams& p, cudaStream_t st) {
  // partials of a prefix tile, on average, and about two of the own part: up to
  // six fit the shallow variant, whose blocks are three to an SM and not two (128
  // queries over 16K tokens, 5 partials: 22 us with the deep one, 12 with this)
  const bool deep = p.pairs > 4 * p.tiles;
  return launch_pdl(deep ? shared_merge_kernel<16> : shared_merge_kernel<6>,
                    dim3(kMergeParts * (unsigned)p.units), dim3(kMergeThreads), 0, st, p);
}

// ---------------------------------------------------------------- W_UV product

// out[r, h, :] = (o_hi + o_lo)[r, h, :] . W_UV[h]: a cluster of four CTAs per
// (head, 128 query rows), CTA k with latent columns 128 k .. + 127: one 128 x 128
// product per part, K = 128.  Its 32 KB of W_UV are on their way before the wait
// for the merge.  The four partial products meet in shared memory: CTA k adds up
// output columns 32 k .. + 31, in a fixed order, and writes them.  Bound by
// latency; with one CTA per head, as for a prompt chunk, the call waits for all of
// W_UV and O after the merge (2.2 us more per call, at 4 and at 32 queries).
constexpr int kOutThreads = 192;  // warp 0 TMA and MMA, warp 1 tensor memory, 2-5 epilogue
constexpr int kOutSplit = 4;
constexpr uint32_t kOutOffW = 4 * kAbBox;                  // after A: hi and lo, two boxes each
// [4 senders][8 groups of four columns][128 rows][4]: a warp's store to another CTA
// is 512 contiguous bytes
constexpr uint32_t kOutOffIn = kOutOffW + 2 * kAbBox;
constexpr uint32_t kOutInBytes = kOutSplit * 8 * 128 * 16;
constexpr uint32_t kOutOffBars = kOutOffIn + kOutInBytes;
constexpr uint32_t kOutSmem = kOutOffBars + 32 + 1024;
static_assert(kOutSmem <= 232448, "shared memory per CTA");

__global__ void __cluster_dims__(kOutSplit, 1, 1) __launch_bounds__(kOutThreads)
    shared_out_kernel(const __grid_constant__ CUtensorMap hi_map,
                      const __grid_constant__ CUtensorMap lo_map,
                      const __grid_constant__ CUtensorMap wuv_map, const SharedParams p,
                      const uint32_t box_rows, __nv_bfloat16* __restrict__ out) {
  extern __shared__ uint8_t smem_raw[];
  uint32_t base = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (base & 1023u)) & 1023u;
  base += pad;
  const uint32_t bar_full = base + kOutOffBars, bar_done = bar_full + 8, tmem_slot = bar_full + 16;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int k = (int)cta_rank();
  const int h = ((int)blockIdx.x / kOutSplit) % kHeads;
  const int r0 = ((int)blockIdx.x / kOutSplit) / kHeads * 128;
  if (threadIdx.x == 0) {
    mbar_init(bar_full, 1);
    mbar_init(bar_done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");
  if (warp == 0) {
    const bool one = elect_one();
    if (one) {
      tma_prefetch_desc(&hi_map);
      tma_prefetch_desc(&lo_map);
      // W_UV[h] rows 128 k .., v columns in two boxes; A: hi and lo, two boxes each of
      // box_rows rows (the rows there are, rounded up: the others' results are not used)
      mbar_arrive_expect_tx(bar_full, 2 * kAbBox + 4 * box_rows * 128);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        tma_load_2d(base + kOutOffW + j * kAbBox, &wuv_map, 64 * j, h * kDLatent + 128 * k, bar_full);
    }
    pdl_wait();
    pdl_launch_dependents();
    if (one) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        tma_load_3d(base + j * kAbBox, &hi_map, 128 * k + 64 * j, h, r0, bar_full);
        tma_load_3d(base + (2 + j) * kAbBox, &lo_map, 128 * k + 64 * j, h, r0, bar_full);
      }
      if (mbar_wait(bar_full, 0, nullptr, p.status, p.wait_limit_ns)) {
        constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, true);
        const uint64_t b = smem_desc_sw128(base + kOutOffW, kAbBox, 1024);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint64_t a = smem_desc_sw128(base + part * 2 * kAbBox, 16, 1024);
#pragma unroll
          for (int s = 0; s < 8; ++s)
            tc_mma_bf16(tmem, a + (((s >> 2) * kAbBox + (s & 3) * 32) >> 4), b + ((s * 2048) >> 4),
                        idesc, (part | s) != 0 ? 1u : 0u);
        }
      }
      tc_commit(bar_done);
    }
  } else {
    pdl_wait();
    pdl_launch_dependents();
  }
  // every CTA of the cluster runs before any writes into another's shared memory
  __syncwarp();
  cluster_sync_all();
  const int quarter = warp & 3;
  const int row = 32 * quarter + lane;
  const int nr = min(128, p.units - r0);
  if (warp >= 2) {
    mbar_wait(bar_done, 0, nullptr, p.status, p.wait_limit_ns);
    __syncwarp();
    tc_fence_after();
    if (32 * quarter < nr) {
#pragma unroll 1
      for (int q = 0; q < kOutSplit; ++q) {
        float v[32];
        tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + 32 * q, v);
        tc_wait_ld();
        // this CTA's part of output columns 32 q .. + 31, to CTA q
        uint32_t dst;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(dst)
                     : "r"(base + kOutOffIn + (uint32_t)((k * 8 * 128 + row) * 16)), "r"(q));
        if (row < nr) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 2048 * e),
                         "f"(v[4 * e]), "f"(v[4 * e + 1]), "f"(v[4 * e + 2]), "f"(v[4 * e + 3])
                         : "memory");
        }
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();  // all four contributions have landed
  tc_fence_after();
  const float4* in = reinterpret_cast<const float4*>(smem_raw + pad + kOutOffIn);
  for (int e = threadIdx.x; e < nr * 4; e += kOutThreads) {
    const int rr = e >> 2, u = e & 3;  // eight columns
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kOutSplit; ++s) {
      const float4 a = in[(s * 8 + 2 * u) * 128 + rr];
      const float4 b = in[(s * 8 + 2 * u + 1) * 128 + rr];
      x[0] += a.x;
      x[1] += a.y;
      x[2] += a.z;
      x[3] += a.w;
      x[4] += b.x;
      x[5] += b.y;
      x[6] += b.z;
      x[7] += b.w;
    }
    *reinterpret_cast<uint4*>(out + ((int64_t)(r0 + rr) * kHeads + h) * kDV + 32 * k + 8 * u) =
        pack8(x);
  }
  if (warp == 1) {
    __syncwarp();  // its lanes leave the loop after different numbers of rounds
    tmem_dealloc(tmem, 128);
  }
}

cudaError_t launch_shared_out(const CUtensorMap& hi_map, const CUtensorMap& lo_map,
                              const CUtensorMap& wuv_map, const SharedParams& p, uint32_t box_rows,
                              __nv_bfloat16* out, cudaStream_t st) {
  static bool done[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        shared_out_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOutSmem);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  const int64_t blocks = (int64_t)((p.units + 127) / 128) * kHeads * kOutSplit;
  return launch_pdl(shared_out_kernel, dim3((unsigned)blocks), dim3(kOutThreads), kOutSmem, st,
                    hi_map, lo_map, wuv_map, p, box_rows, out);
}

}  // namespace xmla
