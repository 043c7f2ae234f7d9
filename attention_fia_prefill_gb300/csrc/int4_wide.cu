// Decode over a 4-bit paged cache for units of 33..64 rows in one group a row
// (int4_decode.cuh's operator and arithmetic), on the tcgen05 tensor cores: with
// mma.sync every 16 rows unpack the codes again, and 64 of them take four times
// a tile's time on the tensor pipe.
//
//   * A CTA, two to an SM, takes 64 keys a step.  Warps 5..8 load 16 keys each
//     (cp.async, a ring of their own), unpack the codes to fp16 (the nibbles in
//     place, as there) and lay K and V down as the operands that the products
//     read; warp 0 issues the products; warps 1..4 are the softmax.
//   * S = Q K^T and O += P V as in span_wide.cu: Q lies twice in the 128 TMEM
//     lanes, 64 apart, copy g takes columns [32 g, 32 g + 32) of every step for
//     itself and its P is 0 elsewhere.
//   * A 16-byte piece of an operand's row is a word of codes: nibble i of its two
//     units, i = 0..3.  Q is laid down in the same order, 16 times as large where it
//     meets bits 0-3, and O's columns come out in it.
//   * P' is at most 2^15: the maximum is that of S_j + log2(step_j), lowered by 12, and
//     kept until it has grown by 3 (log2 units).  Where every row sees every key and
//     their steps are within 2^8 of each other, the largest S and the largest step bound
//     it.  P' is exact to 11 bits down to 2^-26 (there 2^-18) of a row's largest weight
//     times step, and a key that a row does not see has no part in it.
//   * Even shares or clusters: as there, a step being a chunk.
//   * A wait that runs out leaves NaN in the outputs of its unit and of those that
//     the CTA would have come to.
// In us, here and with mma.sync (and at HBM's rate), 8 heads of 64 rows, caches not in L2: 16
// sequences of 100 to 8192 keys 62, 82 (11); 32 of up to 16384 177, 257 (46); 8 of up to 1024
// 20, 21; one of 500 15, 13.  With 32 rows in four copies 173 where mma.sync takes 154 (32 of up to
// 16384), so units of up to 32 rows are left to that.
// Bound: shared memory's data path.  A step of 64 keys is 1370 cycles, of which the
// products read Q, K and V for 490 and loads, stores and the scales' broadcasts take 925.
// The steps' largest and smallest by redux instead of shuffles: 181 -> 176 us (32 of up to
// 16384); the branch between the two maxima costs f16 at head dim 64 2.5% (153 -> 157).
// K and V unpacked by four warps each were slower (184 -> 217 us), K twice and V once too
// (174 -> 233).
#include <algorithm>
#include <cfloat>
#include <cstring>

#include "host.h"
#include "int4_decode.cuh"

namespace fia {
namespace {

using int4_detail::Piece;
using int4_detail::Share;
using int4_detail::Span;
using int4_detail::kTile;

constexpr int kThreads = 288;
constexpr int kKeys = 64;            // of a step
constexpr int kTiles = kKeys / kTile;
constexpr int R = 64;                // rows of a copy

struct Int4WideParams {
  Int4SpanParams i;
  unsigned long long limit_ns;       // of a wait
};

template <int D>
struct WideCfg {
  static constexpr int kGroups = 128 / R;        // copies of the rows
  static constexpr int kCols = kKeys / kGroups;  // columns of a copy
  static constexpr int kChunks = D / 64;
  static constexpr int kBoxQ = 128 * 128, kBox = kKeys * 128;   // 64 columns of Q, of a step's K or V
  static constexpr int kOperand = kChunks * kBox;
  static constexpr int kStages = 3;              // of a warp's ring
  static constexpr int kCodes = kTile * D / 2;
  static constexpr int kRaw = 2 * (kCodes + kTile * 4);
  static constexpr int kOffK = kChunks * kBoxQ;                // Q before it; V twice
  static constexpr int kOffV = kOffK + kOperand;
  static constexpr int kOffRaw = kOffV + 2 * kOperand;
  static constexpr int kOffScale = kOffRaw + kTiles * kStages * kRaw;
  static constexpr int kScale = 4 * kKeys * 4 + 32;   // of a step, fp32: K's step and low, V's; the tiles' log2(V's largest, smallest step) - 12
  static constexpr int kScales = 4;                   // steps of them
  static constexpr int kOffRow = kOffScale + kScales * kScale; // sum of q and factor of each row
  static constexpr int kEnd = kOffRow + 2 * R * 4;
  // after the loops what the join receives and O of the groups take this place
  static constexpr int kOffIn = 0;
  static constexpr int kOffO = (JoinIn<D, R>::kBytes + 1023) / 1024 * 1024;
  static constexpr int kOffML = kEnd > kOffO + 128 * D * 4 ? kEnd : kOffO + 128 * D * 4;
  static constexpr int kOffBar = kOffML + 128 * 8;
  static constexpr int kSmem = kOffBar + 256 + 1024;
  static_assert(2 * (kSmem + 1024 + int(sizeof(Share))) <= 228 * 1024, "two CTAs per SM");
  // TMEM columns: S twice (its first half becomes P), O
  static constexpr uint32_t kColO = 2 * kKeys, kTmem = 256;
};

struct WideBars {
  uint64_t k_full, v_full[2];      // laid down (4 warps); [step & 1]
  uint64_t c_full[4];              // [step & 3]: the scales are there (4 warps)
  uint64_t s_full[2];              // S is in TMEM, and K's place free
  uint64_t p_full[2];              // P is in TMEM (4 warps)
  uint64_t v_free[2];              // the step's P V is done
  uint64_t drain;                  // after an abort
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(WideBars) <= 256, "barrier area");

// Bounded wait for a phase; one that runs out raises the CTA's abort flag.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (abort != nullptr && *abort != 0) return false;
    if (globaltimer() - t0 > limit_ns) {
      if (abort != nullptr) *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, wait(bar, parity, abort, limit_ns));
}

// log2 of a step of V, lowered by 12 (-42 at least: a page outside the pool has steps of 0).
__device__ __forceinline__ float log2_step(float x) { return int4_detail::log2_approx(fmaf(x, 0x1p-12f, 0x1p-42f)); }

// The 16 bytes of an operand that a word of codes makes.
__device__ __forceinline__ uint4 spread(uint32_t w) {
  const uint32_t w8 = w >> 8;
  return make_uint4(w & 0x000f000fu, w & 0x00f000f0u, w8 & 0x000f000fu, w8 & 0x00f000f0u);
}

template <int D, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 2) int4_wide_kernel(const __grid_constant__ Int4WideParams w) {
  using C = WideCfg<D>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int U = D / 32;
  constexpr int RB = D / 2;
  constexpr int ST = C::kStages;
  constexpr uint32_t kNowhere = 0xffffffffu;
  const Int4SpanParams& ip = w.i;
  const SpanParams& p = ip.s;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Share share;
  uint8_t* smem = align_smem_1024(smem_raw);
  WideBars* bar = reinterpret_cast<WideBars*>(smem + C::kOffBar);
  volatile int* abort_flag = &bar->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t lg = SPLIT ? 0u : uint32_t(p.lg_cs), cs = 1u << lg, rank = SPLIT ? 0u : blockIdx.x & (cs - 1u);
  const int kvh = SPLIT ? blockIdx.x : int(blockIdx.x >> lg);
  int b = SPLIT ? 0 : int(blockIdx.y + blockIdx.z * gridDim.y);
  if (!SPLIT && b >= p.B) return;   // (a whole cluster)
  if (threadIdx.x == 0) {
    mbar_init(&bar->k_full, 4);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->v_full[s], 4);
      mbar_init(&bar->s_full[s], 1);
      mbar_init(&bar->p_full[s], 4);
      mbar_init(&bar->v_free[s], 1);
    }
    for (int s = 0; s < C::kScales; ++s) mbar_init(&bar->c_full[s], 4);
    mbar_init(&bar->drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  grid_dep_wait();
  // (TMEM is held neither while this kernel waits for one before it nor wanted
  // once it has let the next one in: span_wide.cu)
  if (warp == 0) {
    tmem_alloc(&bar->tmem, C::kTmem);
    tmem_relinquish();
  }
  if (SPLIT && warp == 1) share.start(p, ip.heads, kTiles, ip.begin, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  grid_dep_launch();

  const bool gapless = p.pre >= p.kv_max;
  const bool heads_first = p.head_stride != RB;
  bool dead = false;           // a wait of an earlier piece has run out
  int base = 0;                // steps of the earlier pieces: they go on with the barriers' phases
  int turn = 0;
#pragma unroll 1
  do {
  int c0 = 0, c1 = 0;
  if constexpr (SPLIT) {
    const Piece now = share.piece[turn];
    if (now.c1 == 0) break;
    b = now.b;
    c0 = now.c0;
    c1 = now.c1;
  }
  int len;
  if constexpr (SPLIT) len = share.piece[turn].len;
  else asm volatile("ld.global.b32 %0, [%1];" : "=r"(len) : "l"(p.kv_len + b) : "memory");
  const int L = min(max(len, 0), p.kv_max);
  const Span sp(p, L);
  const int first = sp.first;
  // step i is tiles first_tile + i * stride .. + 3 of the list
  const int stride = kTiles << lg, first_tile = SPLIT ? c0 * kTiles : int(rank) * kTiles;
  const int left = sp.n_tiles - first_tile;
  const int n = dead ? 0 : SPLIT ? c1 - c0 : left > 0 ? (left + stride - 1) / stride : 0;
  auto tile_key = [&](int v) -> int {
    if (gapless) return v * kTile;
    return (v < sp.t_sink ? v : sp.t_win + v - sp.t_sink) * kTile;
  };

  // ------------------------------------------------------------------ Q
  // Four lanes a row: lane t has columns 32 j + 8 t .. + 7, units g = 2 t, 2 t + 1
  {
    const int r = int(threadIdx.x) >> 2, t = lane & 3;
    const int h = span_head(p, min(r, R - 1)), tk = r - h * p.q_tokens;
    const bool live = r < p.rows;
    const T* q = static_cast<const T*>(p.q) + int64_t(b) * p.q_sb + int64_t(kvh * p.group + h) * p.q_sn + int64_t(tk) * p.q_ss + 8 * t;
    float c[U][8], top = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (live) v = *reinterpret_cast<const uint4*>(q + 32 * j);
      const float2 f0 = int4_pair<BF16>(v.x), f1 = int4_pair<BF16>(v.y), f2 = int4_pair<BF16>(v.z), f3 = int4_pair<BF16>(v.w);
      c[j][0] = f0.x; c[j][1] = f0.y; c[j][2] = f1.x; c[j][3] = f1.y;
      c[j][4] = f2.x; c[j][5] = f2.y; c[j][6] = f3.x; c[j][7] = f3.y;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(c[j][e]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = int4_detail::q_exponent(top, p.scale_log2);
    const float up = __uint_as_float(uint32_t(127 + e) << 23), down = __uint_as_float(uint32_t(127 - e) << 23);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        c[j][k] *= down;
        sum += c[j][k];
      }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (r < R) {
      if (t == 0) {
        float* row = reinterpret_cast<float*>(smem + C::kOffRow);
        row[r] = sum;
        row[R + r] = fminf(up * p.scale_log2, FLT_MAX);
      }
#pragma unroll
      for (int gh = 0; gh < 2; ++gh)
#pragma unroll
        for (int jp = 0; jp < U / 2; ++jp) {
          const int x = (2 * t + gh) * (U / 2) + jp;    // piece: units (g, 2 jp) and (g, 2 jp + 1)
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float m = i & 1 ? 1.f : 16.f;
            o[i] = int4_detail::half2_bits(c[2 * jp][4 * gh + i] * m, c[2 * jp + 1][4 * gh + i] * m);
          }
#pragma unroll
          for (int g = 0; g < C::kGroups; ++g) {
            const int at = g * R + r;
            *reinterpret_cast<uint4*>(smem + (x >> 3) * C::kBoxQ + at * 128 + (((x & 7) ^ (at & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
    }
  }
  fence_proxy_async_smem();
  __syncthreads();

  if (SPLIT && threadIdx.x == kThreads - 1) share.next(p, kTiles, ip.begin, turn ^ 1);   // (read behind the barriers of this piece's end)
  if (warp == 0) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_f16(128, kKeys, 0, 0, 0);
      constexpr uint32_t idesc_pv = idesc_f16(128, D, 0, 0, 1);
      const uint64_t qd = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t kd = smem_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t vd0 = smem_desc_sw128(smem_u32(smem + C::kOffV), C::kBox, 1024);
      auto qk = [&](int i) -> bool {
        const int it = base + i, s = it & 1;
        if (!wait(&bar->k_full, it & 1, abort_flag, w.limit_ns)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + s * kKeys, qd + uint64_t(((kk >> 2) * C::kBoxQ + (kk & 3) * 32) >> 4),
                 kd + uint64_t(((kk >> 2) * C::kBox + (kk & 3) * 32) >> 4), idesc_qk, kk > 0 ? 1u : 0u);
        mma_commit(&bar->s_full[s]);
        return true;
      };
      bool ok = true;
      if (n > 0) ok = qk(0);
      if (ok && n > 1) ok = qk(1);
      int done = 0;            // P V committed
#pragma unroll 1
      for (int i = 0; ok && i < n; ++i) {
        const int it = base + i, s = it & 1;
        ok = wait(&bar->p_full[s], (it >> 1) & 1, abort_flag, w.limit_ns) &&
             wait(&bar->v_full[s], (it >> 1) & 1, abort_flag, w.limit_ns);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = vd0 + uint64_t(s) * (C::kOperand >> 4);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ts(tmem + C::kColO, tmem + s * kKeys + kk * 8, vd + uint64_t((kk * 2048) >> 4), idesc_pv, (i | kk) != 0 ? 1u : 0u);
        mma_commit(&bar->v_free[s]);
        done = i + 1;
        if (i + 2 < n) ok = qk(i + 2);
      }
      // every product issued has finished before TMEM goes
      if (ok) {
        if (done > 0) wait(&bar->v_free[(base + done - 1) & 1], ((base + done - 1) >> 1) & 1, nullptr, kWaitLimitNs);
      } else {
        mma_commit(&bar->drain);
        wait(&bar->drain, 0, nullptr, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp >= 5) {
    // ---------------------------------------------------- loads and unpacking
    const int dw = warp - 5;                     // this warp's tile of a step
    const int32_t* table = p.block_table + int64_t(b) * p.table_stride;
    uint32_t at_code = kNowhere, at_scale = kNowhere;   // one per lane: row numbers of 32 steps' tiles
    auto batch_rows = [&](int i) {
      const int j = tile_key(first_tile + i * stride + dw);
      const int page = p.lg_block >= 0 ? j >> p.lg_block : j / p.block_size;
      const uint32_t off = uint32_t(j - page * p.block_size);
      at_code = at_scale = kNowhere;
      if (j < L && page < p.table_stride) {
        const int id = table[page];
        if (id >= 0 && id < p.n_blocks) {
          at_scale = (uint32_t(id) * uint32_t(p.N2) + uint32_t(kvh)) * uint32_t(p.block_size) + off;
          at_code = heads_first ? at_scale : (uint32_t(id) * uint32_t(p.block_size) + off) * uint32_t(p.N2) + uint32_t(kvh);
        }
      }
    };
    batch_rows(lane);
    const uint32_t ring = smem_u32(smem + C::kOffRaw) + dw * ST * C::kRaw;
    constexpr int CH = RB / 16, kIts = kTile * CH / 32, kRowsIt = 32 / CH;   // 16-byte pieces of a row; rows at once
    const int row_l = lane / CH, c_l = lane % CH;
    const uint32_t row_stride = uint32_t(p.row_stride);
    const uint8_t* kp = ip.kc + uint32_t(row_l) * row_stride + c_l * 16;
    const uint8_t* vp = ip.vc + uint32_t(row_l) * row_stride + c_l * 16;
    const uint8_t* sc = (lane >= 4 ? ip.vs - 64 : ip.ks) + lane * 16;
    auto issue = [&](int i, uint32_t slot) {
      if (i < n) {
        if (i > 0 && (i & 31) == 0) batch_rows(i + lane);
        const uint32_t code = __shfl_sync(0xffffffffu, at_code, i & 31), scale = __shfl_sync(0xffffffffu, at_scale, i & 31);
        const uint32_t bytes = code != kNowhere ? 16u : 0u;
        const uint64_t at = uint64_t(code != kNowhere ? code : 0u) * RB;
        const uint32_t st = ring + slot;
#pragma unroll
        for (int k = 0; k < kIts; ++k) {
          cp_async_zfill<16>(st + k * 512 + lane * 16, kp + at + k * kRowsIt * row_stride, bytes);
          cp_async_zfill<16>(st + C::kCodes + k * 512 + lane * 16, vp + at + k * kRowsIt * row_stride, bytes);
        }
        if (lane < 8)
          cp_async_zfill<16>(st + 2 * C::kCodes + lane * 16, sc + uint64_t(code != kNowhere ? scale : 0u) * 4, bytes);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) issue(i, i * C::kRaw);
    uint32_t slot = 0, slot_before = (ST - 1) * C::kRaw;
    // codes of one operand: raw pieces of the warp's 16 rows -> rows 16 dw .. of the operand.  (Words 0 and 2, 1 and
    // 3 of a piece in another order for half of the lanes: else two lanes' stores meet in a bank.)
    auto unpack = [&](uint32_t raw, uint8_t* dst) {
#pragma unroll
      for (int k = 0; k < kIts; ++k) {
        uint32_t x[4];
        int4_detail::lds<16>(raw + k * 512 + lane * 16, x);
        const int row = dw * kTile + k * kRowsIt + row_l;
        const bool swap = (c_l & 2) != 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t word = swap ? x[q ^ 2] : x[q];
          const int at = 4 * c_l + (swap ? q ^ 2 : q);
          *reinterpret_cast<uint4*>(dst + (at >> 3) * C::kBox + row * 128 + (((at & 7) ^ (row & 7)) << 4)) = spread(word);
        }
      }
    };
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int it = base + i, s = it & 1;
      int4_detail::wait_group<ST - 2>();
      __syncwarp();            // the tile is in for every lane, and the slot before it has been read
      issue(i + ST - 1, slot_before);
      const uint32_t raw = ring + slot;
      slot_before = slot;
      slot = slot + C::kRaw == ST * C::kRaw ? 0u : slot + C::kRaw;
      if (it >= 1 && !warp_wait(&bar->s_full[s ^ 1], ((it - 1) >> 1) & 1, abort_flag, w.limit_ns)) break;
      unpack(raw, smem + C::kOffK);
      fence_proxy_async_smem();
      warp_arrive(&bar->k_full);
      {   // (the softmax of four steps ago is done: P V of three ago was, before V of the last step came)
        uint32_t k2[1], v2[1];
        int4_detail::lds<4>(raw + 2 * C::kCodes + (lane & 15) * 4, k2);
        int4_detail::lds<4>(raw + 2 * C::kCodes + 64 + (lane & 15) * 4, v2);
        const int j = tile_key(first_tile + i * stride + dw) + (lane & 15);
        const bool any = j < L && (j < p.sink || j >= sp.win);
        const float2 kk = int4_pair<BF16>(k2[0]), vv = int4_pair<BF16>(any ? v2[0] : 0u);
        // (as whole numbers: floats of 0 or more lie in the same order)
        const float most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vv.x)));
        const float least = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(vv.x)));
        float* f = reinterpret_cast<float*>(smem + C::kOffScale + (it & 3) * C::kScale) + dw * kTile + lane;
        if (lane < kTile) {
          f[0] = kk.x * 0x1p20f;   // (products come in units of 2^-20)
          f[kKeys] = kk.y;
          f[2 * kKeys] = vv.x;
          f[3 * kKeys] = vv.y;
        }
        if (lane == 0) {
          f[4 * kKeys - dw * kTile + dw] = log2_step(most);
          f[4 * kKeys - dw * kTile + dw + 4] = log2_step(least);
        }
      }
      warp_arrive(&bar->c_full[it & 3]);
      if (it >= 2 && !warp_wait(&bar->v_free[s], ((it >> 1) - 1) & 1, abort_flag, w.limit_ns)) break;
      unpack(raw + C::kCodes, smem + C::kOffV + s * C::kOperand);
      fence_proxy_async_smem();
      warp_arrive(&bar->v_full[s]);
    }
    cp_async_wait_all();
  } else {
    // ------------------------------------------------------------- softmax
    const int quad = warp & 3, g = quad * 32 / R, r = quad * 32 % R + lane;
    const uint32_t lane_off = uint32_t(quad * 32) << 16;
    const uint32_t col_o = tmem + lane_off + C::kColO;
    const int tok = r - span_head(p, r) * p.q_tokens;      // (rows behind the unit's: whatever)
    const int pos = first + tok, w_lo = int(max(int64_t(pos) - p.pre, int64_t(0)));
    const int win_last = int(max(int64_t(L) - 1 - p.pre, int64_t(0)));
    const int f_sink = min((first + 1) >> 4, win_last == 0 ? sp.t_sink : p.sink >> 4);
    const int f_lo = sp.t_sink + max(0, (win_last + kTile - 1) / kTile - sp.t_win), f_hi = sp.t_sink + ((first + 1) >> 4) - sp.t_win;
    const float* row = reinterpret_cast<const float*>(smem + C::kOffRow);
    const float qs = row[r], cr = row[R + r];
    const uint64_t qs2 = f2_pack(qs, qs), cr2 = f2_pack(cr, cr);
    float m = -INFINITY;
    uint64_t l = 0u, zs = 0u;      // even and odd columns
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int it = base + i, s = it & 1, v0 = first_tile + i * stride;
      if (!warp_wait(&bar->c_full[it & 3], (it >> 2) & 1, abort_flag, w.limit_ns) ||
          !warp_wait(&bar->s_full[s], (it >> 1) & 1, abort_flag, w.limit_ns)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t col_s = tmem + lane_off + s * kKeys;
      const float* sc = reinterpret_cast<const float*>(smem + C::kOffScale + (it & 3) * C::kScale) + g * C::kCols;
      // pairs of columns: S in the products' units, then P
      uint64_t x[C::kCols / 2];
      {
        uint32_t u[C::kCols];
        tmem_ld32(col_s + g * C::kCols, u);
        tmem_wait_ld(u);
#pragma unroll
        for (int e = 0; e < C::kCols / 2; ++e) x[e] = f2_pack(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1]));
      }
      const bool full = v0 + kTiles <= f_sink || (v0 >= f_lo && v0 + kTiles <= f_hi);
#pragma unroll
      for (int c = 0; c < C::kCols / 2; c += 2) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(sc + 2 * c), d = *reinterpret_cast<const ulonglong2*>(sc + kKeys + 2 * c);
        x[c] = f2_fma(x[c], a.x, int4_detail::f2_mul(d.x, qs2));
        x[c + 1] = f2_fma(x[c + 1], a.y, int4_detail::f2_mul(d.y, qs2));
      }
      if (!full) {
#pragma unroll
        for (int c = 0; c < C::kCols / 2; ++c) {
          const int j = tile_key(v0 + (g * C::kCols + 2 * c) / kTile) + 2 * c % kTile;
          float lo, hi;
          f2_unpack(x[c], lo, hi);
          if (j > pos || (j >= p.sink && j < w_lo)) lo = -INFINITY;
          if (j + 1 > pos || (j + 1 >= p.sink && j + 1 < w_lo)) hi = -INFINITY;
          x[c] = f2_pack(lo, hi);
        }
      }
      float top = -INFINITY;
      const float4 a = *reinterpret_cast<const float4*>(sc + 4 * kKeys - g * C::kCols), z = *reinterpret_cast<const float4*>(sc + 4 * kKeys - g * C::kCols + 4);
      const float most = fmax3(fmaxf(a.x, a.y), a.z, a.w);
      if (full && most - fminf(fminf(z.x, z.y), fminf(z.z, z.w)) <= 8.f) {
#pragma unroll
        for (int c = 0; c < C::kCols / 2; ++c) {
          float lo, hi;
          f2_unpack(x[c], lo, hi);
          top = fmax3(top, lo, hi);
        }
        top = fmaf(top, cr, most);
      } else {
#pragma unroll
        for (int c = 0; c < C::kCols / 2; ++c) {
          float lo, hi, st0, st1;
          f2_unpack(x[c], lo, hi);
          f2_unpack(*reinterpret_cast<const uint64_t*>(sc + 2 * kKeys + 2 * c), st0, st1);
          top = fmax3(top, fmaf(lo, cr, log2_step(st0)), fmaf(hi, cr, log2_step(st1)));
        }
      }
      const float m_use = (m == -INFINITY || top > m + 3.f) ? fmaxf(m, top) : m;
      const float alpha = m_use == m ? 1.f : fast_exp2(m - m_use);
      const float mo = m_use == -INFINITY ? 0.f : -m_use;
      const uint64_t alpha2 = f2_pack(alpha, alpha), mo2 = f2_pack(mo, mo);
      l = int4_detail::f2_mul(l, alpha2);
      zs = int4_detail::f2_mul(zs, alpha2);
      m = m_use;
      uint32_t u[C::kCols / 2];
      auto weights = [&](auto whole) {
#pragma unroll
        for (int c = 0; c < C::kCols / 2; c += 2) {
          const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(sc + 2 * kKeys + 2 * c), d = *reinterpret_cast<const ulonglong2*>(sc + 3 * kKeys + 2 * c);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float t0, t1;
            f2_unpack(f2_fma(x[c + k], cr2, mo2), t0, t1);
            const uint64_t y = f2_pack(fast_exp2(t0), fast_exp2(t1));
            l = f2_add(l, y);
            if constexpr (decltype(whole)::value) {
              zs = f2_fma(y, k ? d.y : d.x, zs);
            } else {   // (a low value that a row does not see may be a NaN)
              float s0, s1, y0, y1, z0, z1, d0, d1;
              f2_unpack(x[c + k], s0, s1);
              f2_unpack(y, y0, y1);
              f2_unpack(zs, z0, z1);
              f2_unpack(k ? d.y : d.x, d0, d1);
              zs = f2_pack(s0 != -INFINITY ? fmaf(y0, d0, z0) : z0, s1 != -INFINITY ? fmaf(y1, d1, z1) : z1);
            }
            float p0, p1;
            const uint64_t pk = int4_detail::f2_mul(y, k ? a.y : a.x);
            f2_unpack(pk, p0, p1);
            u[c + k] = int4_detail::half2_bits(p0, p1);
            if constexpr (!BF16) zs = int4_detail::p_rest(pk, u[c + k], zs);
          }
        }
      };
      if (full) weights(std::true_type());
      else weights(std::false_type());
      if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
        // O holds the step before's product once that is done
        if (!warp_wait(&bar->v_free[s ^ 1], ((it - 1) >> 1) & 1, abort_flag, w.limit_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
          uint32_t o[16];
          tmem_ld16(col_o + q * 16, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st16(col_o + q * 16, o);
        }
      }
      // P of all the step's keys, 0 but for the copy's, over S (this lane's alone)
      const uint32_t none[16] = {};
      tmem_st16(col_s + g * 16, u);
      tmem_st16(col_s + (g ^ 1) * 16, none);
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&bar->p_full[s]);
    }
    if (!ok) tmem_wait_st();   // no store to TMEM is pending when it goes
    if (ok && n > 0) ok = warp_wait(&bar->v_free[(base + n - 1) & 1], ((base + n - 1) >> 1) & 1, abort_flag, w.limit_ns);
    tc_fence_after();
    if (ok) {
      // O to its place: every tile has been unpacked and every product is done
      float* ob = reinterpret_cast<float*>(smem + C::kOffO);
      float l0, l1, z0, z1;
      f2_unpack(l, l0, l1);
      f2_unpack(zs, z0, z1);
      const float low = z0 + z1;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t u[32];
        if (n > 0) {
          tmem_ld32(col_o + q * 32, u);
          tmem_wait_ld(u);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) u[e] = 0u;
        }
        // pieces 4 q ..: column 2 i + h of piece x is column i of unit 2 x + h
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int unit = 2 * (4 * q + k) + h, c4 = 8 * (unit % U) + unit / U;
            *reinterpret_cast<float4*>(ob + join_at<D, R>(g, r, c4)) =
                make_float4(fmaf(__uint_as_float(u[8 * k + h]), 0x1p24f, low), fmaf(__uint_as_float(u[8 * k + 2 + h]), 0x1p20f, low),
                            fmaf(__uint_as_float(u[8 * k + 4 + h]), 0x1p24f, low), fmaf(__uint_as_float(u[8 * k + 6 + h]), 0x1p20f, low));
          }
      }
      reinterpret_cast<float2*>(smem + C::kOffML)[g * R + r] = make_float2(m, l0 + l1);
    }
    tc_fence_before();
  }

  // (waited for before the join's first remote store: no CTA's Q and operands are in use)
  __syncwarp();
  if (lg != 0) cluster_arrive();
  __syncthreads();
  tc_fence_after();
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffML);
  float* ob = reinterpret_cast<float*>(smem + C::kOffO);
  if (*abort_flag != 0) {
    const float nan = __uint_as_float(0x7fc00000u);
    for (int e = threadIdx.x; e < 128; e += kThreads) ml[e] = make_float2(nan, nan);
    dead = true;
  }
  base += n;
  if constexpr (SPLIT) {
    const Piece now = share.piece[turn];
    if (now.parts == 1) {
      int4_detail::join_unit<D, BF16, R, C::kGroups, kThreads>(p, ob, ml, smem + C::kOffIn, 0u, 0u, b, kvh);
    } else {
      const int64_t at = 2 * int64_t(int4_detail::share_cta()) + (now.parts > 1 ? 1 : 0);
      int4_detail::write_part<D, R, C::kGroups, kThreads>(p, ob, ml, ip.part_o + at * p.rows * D, ip.part_ml + at * p.rows);
      if (now.parts > 1 && threadIdx.x == 0) ip.heads[int4_detail::share_cta()] = make_int4(b, kvh, now.parts, 0);
    }
    turn ^= 1;
    __syncthreads();           // (Q and the operands take the results' place)
  } else {
    int4_detail::join_unit<D, BF16, R, C::kGroups, kThreads>(p, ob, ml, smem + C::kOffIn, lg, rank, b, kvh);
  }
  } while (SPLIT);
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

template <int D, bool BF16>
cudaError_t launch_one(Int4WideParams w, int n_sm, cudaStream_t s) {
  constexpr int smem = WideCfg<D>::kSmem;
  const Int4SpanParams& ip = w.i;
  if (ip.heads != nullptr) {
    constexpr auto kernel = int4_wide_kernel<D, BF16, true>;
    set_span_shape(w.i.s, 1);
    cudaError_t e = prepare_span<kernel>(smem);
    if (e == cudaSuccess) e = launch_early(kernel, dim3(unsigned(ip.s.N2), unsigned(ip.n_ctas / ip.s.N2)), kThreads, smem, s, w);
    return e == cudaSuccess ? int4_detail::launch_join<D, BF16>(w.i, s) : e;
  }
  constexpr auto kernel = int4_wide_kernel<D, BF16, false>;
  constexpr int kStart = 10;         // start cost of a CTA in steps (2, 5 and 20: each of 98 calls within 5%)
  // (always for units of like lengths: a dearer cluster, to even lengths out, takes 1.01 times as long in the mean of 98 calls
  // of 1 to 64 sequences, and up to 1.30 times: 4 of 64 keys 9.0 -> 11.7 us)
  const int64_t span = std::min<int64_t>(ip.s.kv_max, int64_t(ip.s.sink) + ip.s.pre + ip.s.q_tokens);
  set_span_shape(w.i.s, cluster_ctas(int64_t(ip.s.B) * ip.s.N2, ip.s.rows, span / kKeys + 1, 1, kStart, true, 2, n_sm));
  cudaError_t e = prepare_span<kernel>(smem);
  if (e != cudaSuccess) return e;
  return int4_detail::launch_units(kernel, w, w.i.s, kThreads, smem, s);
}

}  // namespace

cudaError_t launch_int4_wide(const Int4SpanParams& p, int head_dim, bool bf16, int n_sm, cudaStream_t s) {
  if (p.s.rows > 64) return cudaErrorInvalidValue;
  Int4WideParams w;
  memset(&w, 0, sizeof(w));
  w.i = p;
  w.limit_ns = make_status(nullptr).limit_ns;
  if (head_dim == 128) return bf16 ? launch_one<128, true>(w, n_sm, s) : launch_one<128, false>(w, n_sm, s);
  return bf16 ? launch_one<64, true>(w, n_sm, s) : launch_one<64, false>(w, n_sm, s);
}

}  // namespace fia
