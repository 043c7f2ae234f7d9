// The end of a span decode unit (span_decode.cu, span_wide.cu): the results of
// a CTA's groups, of the unit's CTAs and of a shared prefix, joined and written.
#pragma once
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "paged.h"
#include "ptx.cuh"

namespace fia {

constexpr int kMostCtas = 16;        // CTAs of a unit (a cluster; above 8 by leave of the kernel)

// The cluster's barrier in halves: arrive releases this thread's writes, wait
// acquires every CTA's.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_addr(uint32_t smem, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_peer4(uint32_t a, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_peer2(uint32_t a, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}

// The weight of a partial result with maximum m in a sum with maximum top
// (an empty one, m = -inf, has none).
__device__ __forceinline__ float join_weight(float m, float top) { return m == -INFINITY ? 0.f : fast_exp2(m - top); }

// Row of the unit -> head of its group (r < 64): rows are the heads, and within
// a head the tokens.
__device__ __forceinline__ int span_head(const SpanParams& p, int r) { return int((uint32_t(r) * p.q_inv) >> 16); }

// O of a CTA's groups: [group][rows][D] with the float4s of a row XOR-swizzled
// by row, so that the rows of a store instruction do not share banks.
template <int D, int ROWS>
__device__ __forceinline__ int join_at(int g, int r, int c4) {
  return ((g * ROWS + r) * (D / 4) + (c4 ^ ((r & 7) << 1))) * 4;
}

// Results of the cluster's CTAs for this CTA's share of the unit's float4s, and
// their (max, sum) of every row.
template <int D, int ROWS>
struct JoinIn {
  static constexpr int kO = (ROWS * (D / 4) + 8 * kMostCtas) * 16;
  static constexpr int kBytes = kO + kMostCtas * ROWS * 8;
};

// All threads of the CTA.  ob, ml: O (join_at) and (max, sum) [group][rows] of
// this CTA's groups; in: JoinIn.  Every thread has arrived at the cluster's
// barrier (lg != 0) and not yet waited.
template <int D, bool BF16, int ROWS, int GROUPS, int THREADS>
__device__ __forceinline__ void span_join(const SpanParams& p, const float* ob, const float2* ml, void* in, uint32_t lg,
                                          uint32_t rank, int b, int kvh) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int kInML = JoinIn<D, ROWS>::kO;
  const uint32_t in_o = smem_u32(in), in_ml = in_o + kInML;
  const uint32_t cs = 1u << lg;
  const int items = p.rows * (D / 4);   // float4s of the unit
  const int share = ((items + 8 * int(cs) - 1) >> (3 + lg)) << 3;
  // one float4 (not divided by its sum), maximum and sum of this CTA's groups
  auto own = [&](int r, int c4, float4& a, float& l, float& top) {
    top = -INFINITY;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) top = fmaxf(top, ml[g * ROWS + r].x);
    a = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const float2 w2 = ml[g * ROWS + r];
      const float w = join_weight(w2.x, top);
      const float4 x = *reinterpret_cast<const float4*>(ob + join_at<D, ROWS>(g, r, c4));
      l += w * w2.y;
      a.x += w * x.x; a.y += w * x.y; a.z += w * x.z; a.w += w * x.w;
    }
  };
  __syncthreads();
  if (lg != 0) {
    // each float4 goes to the CTA that writes it: the CTAs take eight in turn
    cluster_wait();
    for (int e = threadIdx.x; e < items; e += THREADS) {
      const int r = e / (D / 4), c4 = e % (D / 4);
      float4 a;
      float l, top;
      own(r, c4, a, l, top);
      const int owner = (e >> 3) & int(cs - 1u), slot = ((e >> (3 + lg)) << 3) + (e & 7);
      st_peer4(peer_addr(in_o + (rank * share + slot) * 16, owner), a);
      if (c4 == 0)
        for (uint32_t k = 0; k < cs; ++k) st_peer2(peer_addr(in_ml + (rank * ROWS + r) * 8, k), make_float2(top, l));
    }
    __syncwarp();
    cluster_arrive();
  }
  if (p.n_parts > 0) grid_dep_wait();   // (by every thread: the prefix's results are in)
  if (lg != 0) cluster_wait();          // no CTA reads or writes another's memory from here on
  const float4* xo = static_cast<const float4*>(in);
  const float2* xml = reinterpret_cast<const float2*>(static_cast<const uint8_t*>(in) + kInML);
  for (int i = threadIdx.x; i < share; i += THREADS) {
    const int e = ((((i >> 3) << lg) + int(rank)) << 3) + (i & 7);
    if (e >= items) break;
    const int r = e / (D / 4), c4 = e % (D / 4);
    const int h = span_head(p, r), head = kvh * p.group + h, tokn = r - h * p.q_tokens;
    float4 a;
    float l, top;
    if (lg == 0) {
      own(r, c4, a, l, top);
    } else {
      top = -INFINITY;
      for (uint32_t g = 0; g < cs; ++g) top = fmaxf(top, xml[g * ROWS + r].x);
      a = make_float4(0.f, 0.f, 0.f, 0.f);
      l = 0.f;
      for (uint32_t g = 0; g < cs; ++g) {
        const float2 w2 = xml[g * ROWS + r];
        const float w = join_weight(w2.x, top);
        const float4 x = xo[g * share + i];
        l += w * w2.y;
        a.x += w * x.x; a.y += w * x.y; a.z += w * x.z; a.w += w * x.w;
      }
    }
    // the prefix's parts, kBatch loads in flight, with a running maximum
    constexpr int kBatch = D == 64 ? 16 : 24;
    const int64_t prow = (int64_t(b) * p.N1 + head) * p.q_tokens + tokn;
    for (int g0 = 0; g0 < p.n_parts; g0 += kBatch) {
      float2 w2[kBatch];
      float4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const bool in = g0 + k < p.n_parts;
        const int64_t row = (in ? g0 + k : g0) * p.part_rows + prow;
        w2[k] = p.part_ml[row];
        x[k] = *reinterpret_cast<const float4*>(p.part_o + row * D + c4 * 4);
        if (!in) w2[k].x = -INFINITY;
      }
      float t = top;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) t = fmaxf(t, w2[k].x);
      const float keep = join_weight(top, t);
      l *= keep;
      a.x *= keep; a.y *= keep; a.z *= keep; a.w *= keep;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        // an empty part: its O may be 0 * NaN.  (Tested by its sum, so that the prefix
        // kernel need not mark sums that are NaN: 12.0 -> 13.1 us, 64 sequences 67.7 -> 72.2.)
        if (w2[k].x == -INFINITY) continue;
        const float w = join_weight(w2[k].x, t);
        l += w * w2[k].y;
        a.x += w * x[k].x; a.y += w * x[k].y; a.z += w * x[k].z; a.w += w * x[k].w;
      }
      top = t;
    }
    const bool has = l != 0.f;   // a NaN sum stays a NaN
    const float inv = has ? 1.f / l : 0.f;
    uint2 u;
    u.x = has ? pack2(a.x * inv, a.y * inv, BF16) : 0u;
    u.y = has ? pack2(a.z * inv, a.w * inv, BF16) : 0u;
    T* orow = static_cast<T*>(p.out) + int64_t(b) * p.q_sb + int64_t(head) * p.q_sn + int64_t(tokn) * p.q_ss;
    *reinterpret_cast<uint2*>(orow + c4 * 4) = u;
    if (p.lse != nullptr && c4 == 0)
      p.lse[int64_t(b) * p.lse_sb + int64_t(head) * p.lse_sn + int64_t(tokn) * p.lse_ss] =
          has ? (top + __log2f(l)) * 0.69314718055994531f : INFINITY;
  }
}

// ------------------------------------------------------------------- host
// CTAs of a unit: those whose waves take the least time, a CTA costing its
// groups' tiles and about `start` tiles more (launch, length, page ids, first
// keys, join).  even: units have like lengths; else smaller shares even them out,
// and up to a seventh more by this count is taken for them.  Joining 16 CTAs costs
// about a tile for every 8 rows more than joining 8 (8 units, us with 8 and with
// 16: 4 rows, 4096 keys 11.7, 9.1; 32 rows, 384 keys 6.3, 8.0; 64 rows, 4096 keys
// 14.5, 15.9), and is not done where SMs would share such clusters (16 units of 4
// rows and 32768 keys 69.7, 73.2).
inline int cluster_ctas(int64_t units, int rows, int64_t tiles, int groups, int start, bool even, int per_sm, int n_sm) {
  const int64_t slots = int64_t(per_sm) * n_sm;
  int best = 1;
  int64_t least = 0;
  for (int cs = 1; cs <= (units * kMostCtas <= n_sm ? kMostCtas : kMostCtas / 2); cs *= 2) {
    const int64_t waves = (units * cs + slots - 1) / slots;
    const int64_t cost = waves * ((tiles + cs * groups - 1) / (cs * groups) + start + (cs > 8 ? rows / 8 : 0));
    if (cs == 1 || (even ? cost < least : cost * 7 < least * 8)) best = cs;
    if (cs == 1 || cost < least) least = cost;
  }
  return best;
}

// What the launch adds to the parameters.
inline void set_span_shape(SpanParams& p, int cs) {
  p.lg_cs = 0;
  while (1 << p.lg_cs < cs) ++p.lg_cs;
  p.q_inv = 65536u / unsigned(p.q_tokens) + 1u;   // floor(r q_inv / 2^16) = r / q_tokens for r < 64, q_tokens <= 16
  p.lg_block = -1;
  for (int k = 4; k < 31; ++k)
    if (p.block_size == 1 << k) p.lg_block = k;
}

// Shared memory and clusters of 16, on the first launch on each device.
template <auto Kernel>
cudaError_t prepare_span(int smem) {
  static std::atomic<unsigned long long> done{0};   // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? (1ull << dev) : 0ull;
  if ((done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// One cluster of CTAs per unit, let in while the kernel before it ends.
template <typename P>
cudaError_t launch_span(void (*kernel)(P), const P& args, const SpanParams& p, unsigned threads, size_t smem,
                        cudaStream_t s) {
  const unsigned cs = 1u << p.lg_cs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.B) * cs, unsigned(p.N2));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace fia
