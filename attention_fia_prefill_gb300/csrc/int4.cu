// The 4-bit paged cache: new keys and values quantised on their way to their
// slots, and rows of the sequences read back.  Format: int4.cuh.
#include <algorithm>

#include "int4.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace fia {
namespace {

constexpr int kInt4Threads = 256;
constexpr int kInt4Tokens = 16;                               // tokens of a CTA
constexpr int kInt4Heads = kInt4Threads / (4 * kInt4Tokens);  // heads of a pass: 64 rows, four lanes each

__device__ __forceinline__ uint32_t half_bits(float x) { return uint32_t(__half_as_ushort(__float2half_ru(x))); }
__device__ __forceinline__ uint32_t bf16_bits(float x) { return uint32_t(__bfloat16_as_ushort(__float2bfloat16_ru(x))); }

// a + b of pairs, rounded up.
__device__ __forceinline__ uint64_t f2_add_up(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rp.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float rcp_approx(float x) {   // within 2^-23
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Minimum and maximum of pairs; a NaN stays.
template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Four lanes quantise a row: lane t has columns 32 j + 8 t .. + 7 of every j
// (16-byte loads) and writes the D/8 bytes of units (D/32) 2t .. (one store).
// Steps and codes are the format's to the last bit, in fp32:
//   * step: the least value of the type that is, times 15 (exact in fp32), not below
//     the difference; that is rounded up, which changes no such comparison.  In f16 the
//     value before it, where 15 of it would pass 65504 - low.
//   * code: c = round((x - low) / step (1 - 2^-20)), by one addition and one fused
//     multiply-add into 1.5 * 2^23, whose low bits then hold it.  The factor takes
//     off more than the roundings can add, so c is the code or one less; it is one
//     less exactly where x - low, rounded up, is above step (c + 1/2), which has at
//     most 16 bits.
// Bound: HBM and the instructions (325 a warp for 8 rows of 128) for many tokens: 32771
// of 8 heads x 128, keys and values, 27.0 us behind one another, 5.9 TB/s (alone 30.8,
// with every rounding by CUDA's functions 37.5); a launch and one load's latency for few
// (16 tokens 1.6 us).
template <int D, int NG, bool BF16>
__global__ void __launch_bounds__(kInt4Threads) cache_write_int4_kernel(const __grid_constant__ Int4WriteParams p) {
  constexpr int U = D / 32;                  // columns j, 32 apart
  const bool y = blockIdx.z != 0;
  const int lane4 = threadIdx.x & 3, row = threadIdx.x >> 2;
  const int t = blockIdx.x * kInt4Tokens + row % kInt4Tokens, h = blockIdx.y * kInt4Heads + row / kInt4Tokens;
  grid_dep_launch();
  grid_dep_wait();
  const bool in = t < p.n_tokens && h < p.heads;
  // (the row is loaded with its slot, not behind it: those skipped are few)
  const int slot = in ? p.slots[t] : -1;
  const bool live = slot >= 0 && slot < p.n_slots;
  uint4 x[U];
  if (in) {
    const uint8_t* src = p.src[y] + int64_t(t) * p.src_row[y] + int64_t(h) * (D * 2) + lane4 * 16;
#pragma unroll
    for (int j = 0; j < U; ++j) x[j] = __ldcs(reinterpret_cast<const uint4*>(src + j * 64));
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j) x[j] = make_uint4(0u, 0u, 0u, 0u);
  }
  // ---- low and high of the groups, over the row's four lanes
  uint32_t lo[NG], hi[NG];
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    lo[k] = hi[k] = x[k * (U / NG)].x;
#pragma unroll
    for (int j = k * (U / NG); j < (k + 1) * (U / NG); ++j) {
      lo[k] = min2<BF16>(min2<BF16>(lo[k], x[j].x), min2<BF16>(min2<BF16>(x[j].y, x[j].z), x[j].w));
      hi[k] = max2<BF16>(max2<BF16>(hi[k], x[j].x), max2<BF16>(max2<BF16>(x[j].y, x[j].z), x[j].w));
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      lo[k] = min2<BF16>(lo[k], __shfl_xor_sync(0xffffffffu, lo[k], d));
      hi[k] = max2<BF16>(hi[k], __shfl_xor_sync(0xffffffffu, hi[k], d));
    }
    lo[k] = min2<BF16>(lo[k], __funnelshift_l(lo[k], lo[k], 16));
    hi[k] = max2<BF16>(hi[k], __funnelshift_l(hi[k], hi[k], 16));
  }
  // ---- steps and codes
  uint32_t word[NG], half[U][2];   // (step, low); the lane's units 2 t and 2 t + 1 of every j
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    const float low = int4_pair<BF16>(lo[k]).x, high = int4_pair<BF16>(hi[k]).x;
    const bool fine = low >= -kInt4Most && high <= kInt4Most;   // (not where a value is a NaN or an infinity)
    const float range = fine ? __fsub_ru(high, low) : 0.f;
    // a fifteenth, lowered by 2^-21: its rounding up is the step or the value of the type before it
    const float near = fmaxf(range * ((1.f - 0x1p-21f) / 15.f), kInt4Tiny<BF16>);
    uint32_t bits = BF16 ? bf16_bits(near) : half_bits(near);
    bits += 15.f * int4_pair<BF16>(bits).x < range ? 1u : 0u;
    // (15 steps are a number of fp32, so the comparison with what the rounding down leaves is that with 65504 - low)
    if constexpr (!BF16) bits -= range > 0.f && 15.f * int4_pair<BF16>(bits).x > __fsub_rd(kInt4MostHalf, low) ? 1u : 0u;
    word[k] = bits | ((fine ? lo[k] & 0xffffu : 0x7fffu) << 16);
    const float step = int4_pair<BF16>(bits).x, inv = rcp_approx(step) * (1.f - 0x1p-20f), mid = 0.5f * step;
    constexpr float kMagic = 12582912.f;   // 0x4B400000: its low bits are the rounded sum's
    const uint64_t low2 = f2_pack(-low, -low), inv2 = f2_pack(inv, inv), step2 = f2_pack(step, step), mid2 = f2_pack(mid, mid);
    const uint64_t magic2 = f2_pack(kMagic, kMagic), unmagic2 = f2_pack(-kMagic, -kMagic), minus2 = f2_pack(-1.f, -1.f);
    // two values -> their codes, above 0x4B400000 (the carry is the sign of step (c + 1/2) - (x - low))
    auto code = [&](uint32_t w, uint32_t& c0, uint32_t& c1) {
      const float2 f = int4_pair<BF16>(w);
      const uint64_t d = f2_add_up(f2_pack(f.x, f.y), low2), c = f2_fma(d, inv2, magic2);
      const uint64_t e = f2_fma(d, minus2, f2_fma(step2, f2_add(c, unmagic2), mid2));
      c0 = uint32_t(c) + (uint32_t(e) >> 31);
      c1 = uint32_t(c >> 32) + (uint32_t(e >> 32) >> 31);
    };
#pragma unroll
    for (int j = k * (U / NG); j < (k + 1) * (U / NG); ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t c0, c1, c2, c3;
        code(u ? x[j].z : x[j].x, c0, c1);
        code(u ? x[j].w : x[j].y, c2, c3);
        // (0x4B400000 in four places sums to 0x3F400000 in 32 bits: the low half stays the codes')
        const uint32_t sum = ((c3 * 16u + c2) * 16u + c1) * 16u + c0;
        half[j][u] = fine ? sum & 0xffffu : 0u;
      }
  }
  if (!live) return;
  const int blk = p.lg_block >= 0 ? slot >> p.lg_block : slot / p.block_size, off = slot - blk * p.block_size;
  uint8_t* dst = p.dst[y] + int64_t(blk) * p.dst_blk + int64_t(off) * p.dst_row + int64_t(h) * p.dst_head + lane4 * (D / 8);
  if constexpr (U == 4)
    *reinterpret_cast<uint4*>(dst) = make_uint4(half[0][0] | half[1][0] << 16, half[2][0] | half[3][0] << 16,
                                                half[0][1] | half[1][1] << 16, half[2][1] | half[3][1] << 16);
  else
    *reinterpret_cast<uint2*>(dst) = make_uint2(half[0][0] | half[1][0] << 16, half[0][1] | half[1][1] << 16);
  uint32_t* sc = p.scales[y] + ((int64_t(blk) * p.heads + h) * p.block_size + off) * NG;
#pragma unroll
  for (int k = 0; k < NG; ++k)
    if (lane4 == k) sc[k] = word[k];
}

// Rows of the sequences, packed one after the other.  A CTA has 16 tokens: the
// sequence of the first is the count of running sums up to it (one load per
// thread and one barrier; a binary search is a chain of loads), and each of 16
// threads steps on from there and looks its token's slot up.  Four lanes then
// read a row (its D/8 bytes each) and write 16 bytes of every 32 columns.
// Bound: HBM, of which the outputs are the larger part (8 contexts of up to 14336
// tokens, groups of 32: 49.8 us, 6.2 TB/s, 91% of a copy's rate); for few tokens the
// launch and the chain sums -> page id -> codes (1023 tokens 3.1 us).
template <int D, int NG, bool BF16>
__global__ void __launch_bounds__(kInt4Threads) cache_read_int4_kernel(const __grid_constant__ Int4ReadParams p) {
  constexpr int U = D / 32;
  __shared__ int64_t s_slot[kInt4Tokens];    // row of the pool (token of block 0's first on), -1: zeros, -2: not written
  const int lane4 = threadIdx.x & 3, row = threadIdx.x >> 2;
  const int64_t t0 = int64_t(blockIdx.x) * kInt4Tokens;
  grid_dep_launch();
  grid_dep_wait();
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += kInt4Threads) {
    const int b = b0 + int(threadIdx.x);
    before += __syncthreads_count(b < p.B && p.cu[b] <= t0);
  }
  if (threadIdx.x < kInt4Tokens) {
    const int64_t t = t0 + threadIdx.x;
    int b = before;
    while (b < p.B && p.cu[b] <= t) ++b;
    int64_t slot = -2;
    if (t < p.n_tokens && b < p.B) {
      const int64_t pos = t - (b > 0 ? max(p.cu[b - 1], 0) : 0);
      const int64_t page = p.lg_block >= 0 ? pos >> p.lg_block : pos / p.block_size;
      int id = -1;
      if (pos >= 0 && page < p.table_cols) id = p.block_table[int64_t(b) * p.table_cols + page];
      slot = id >= 0 && id < p.n_blocks ? int64_t(id) * p.block_size + (pos - page * p.block_size) : -1;
    }
    s_slot[threadIdx.x] = slot;
  }
  __syncthreads();
  const int64_t slot = s_slot[row % kInt4Tokens];
  if (slot == -2) return;
  const int64_t t = t0 + row % kInt4Tokens;
  const int blk = slot < 0 ? 0 : int(p.lg_block >= 0 ? slot >> p.lg_block : slot / p.block_size),
            off = slot < 0 ? 0 : int(slot - int64_t(blk) * p.block_size);
  const int units = (p.heads + kInt4Heads - 1) / kInt4Heads;
  for (int i = blockIdx.y; i < units * p.n_tensors; i += gridDim.y) {
    const int y = i >= units, h = (i - y * units) * kInt4Heads + row / kInt4Tokens;
    if (h >= p.heads) continue;
    uint32_t w[U];
    float2 sc[NG];
    if (slot >= 0) {
      const uint8_t* src = p.codes[y] + int64_t(blk) * p.src_blk + int64_t(off) * p.src_row + int64_t(h) * p.src_head + lane4 * (D / 8);
      if constexpr (U == 4) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
      } else {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(src));
        w[0] = v.x; w[1] = v.y;
      }
      const uint32_t* s = p.scales[y] + ((int64_t(blk) * p.heads + h) * p.block_size + off) * NG;
#pragma unroll
      for (int k = 0; k < NG; ++k) sc[k] = int4_pair<BF16>(s[k]);
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) w[j] = 0u;
#pragma unroll
      for (int k = 0; k < NG; ++k) sc[k] = make_float2(0.f, 0.f);
    }
    uint8_t* dst = p.dst[y] + (t * p.heads + h) * (D * 2) + lane4 * 16;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const float2 g = sc[j / (U / NG)];
      uint32_t o[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // unit (2 t + u, j): a half of word u * U / 2 + j / 2
        const uint32_t c = w[u * (U / 2) + j / 2] >> (16 * (j & 1));
#pragma unroll
        for (int e = 0; e < 2; ++e)
          o[2 * u + e] = pack2(fmaf(float(c >> (8 * e) & 15u), g.x, g.y), fmaf(float(c >> (8 * e + 4) & 15u), g.x, g.y), BF16);
      }
      *reinterpret_cast<uint4*>(dst + j * 64) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <bool BF16>
cudaError_t write_type(const Int4WriteParams& p, int D, int NG, dim3 grid, cudaStream_t s) {
  if (D == 128) {
    if (NG == 1) return launch_early(cache_write_int4_kernel<128, 1, BF16>, grid, kInt4Threads, 0, s, p);
    if (NG == 2) return launch_early(cache_write_int4_kernel<128, 2, BF16>, grid, kInt4Threads, 0, s, p);
    return launch_early(cache_write_int4_kernel<128, 4, BF16>, grid, kInt4Threads, 0, s, p);
  }
  if (NG == 1) return launch_early(cache_write_int4_kernel<64, 1, BF16>, grid, kInt4Threads, 0, s, p);
  return launch_early(cache_write_int4_kernel<64, 2, BF16>, grid, kInt4Threads, 0, s, p);
}

template <bool BF16>
cudaError_t read_type(const Int4ReadParams& p, int D, int NG, dim3 grid, cudaStream_t s) {
  if (D == 128) {
    if (NG == 1) return launch_early(cache_read_int4_kernel<128, 1, BF16>, grid, kInt4Threads, 0, s, p);
    if (NG == 2) return launch_early(cache_read_int4_kernel<128, 2, BF16>, grid, kInt4Threads, 0, s, p);
    return launch_early(cache_read_int4_kernel<128, 4, BF16>, grid, kInt4Threads, 0, s, p);
  }
  if (NG == 1) return launch_early(cache_read_int4_kernel<64, 1, BF16>, grid, kInt4Threads, 0, s, p);
  return launch_early(cache_read_int4_kernel<64, 2, BF16>, grid, kInt4Threads, 0, s, p);
}

}  // namespace

cudaError_t launch_cache_write_int4(const Int4WriteParams& p, int head_dim, int groups, bool bf16, cudaStream_t s) {
  const dim3 grid(unsigned((int64_t(p.n_tokens) + kInt4Tokens - 1) / kInt4Tokens),
                  unsigned((p.heads + kInt4Heads - 1) / kInt4Heads), unsigned(p.n_tensors));
  return bf16 ? write_type<true>(p, head_dim, groups, grid, s) : write_type<false>(p, head_dim, groups, grid, s);
}

cudaError_t launch_cache_read_int4(const Int4ReadParams& p, int head_dim, int groups, bool bf16, int n_sm, cudaStream_t s) {
  const int64_t chunks = (int64_t(p.n_tokens) + kInt4Tokens - 1) / kInt4Tokens;
  const int64_t units = int64_t((p.heads + kInt4Heads - 1) / kInt4Heads) * p.n_tensors;
  // a CTA for every pass while there are few chunks, which else take all passes of their tokens
  const int64_t split = std::min(units, std::max<int64_t>(1, 8 * int64_t(n_sm) / chunks));
  const dim3 grid{unsigned(chunks), unsigned(split)};
  return bf16 ? read_type<true>(p, head_dim, groups, grid, s) : read_type<false>(p, head_dim, groups, grid, s);
}

cudaError_t launch_int4_decode(const Int4SpanParams& p, int head_dim, int groups, bool bf16, int n_sm, cudaStream_t s) {
  if (p.s.rows > 32 && groups == 1) return launch_int4_wide(p, head_dim, bf16, n_sm, s);
  if (head_dim == 64) return launch_int4_decode_d64(p, groups, bf16, n_sm, s);
  if (groups == 4) return launch_int4_decode_g32(p, bf16, n_sm, s);
  return groups == 2 ? launch_int4_decode_g64(p, bf16, n_sm, s) : launch_int4_decode_g128(p, bf16, n_sm, s);
}

}  // namespace fia
