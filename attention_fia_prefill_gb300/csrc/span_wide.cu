// Decode over the visible span (span_decode.cu's operator) for units of 17..64
// rows, on the tcgen05 tensor cores.  mma.sync bounds such units: every warp
// reads every tile's fragments from shared memory for 16 rows of its own.
//
//   * A unit (batch, kv head) is run by a cluster of 1..16 CTAs, two to an SM (one
//     chain softmax -> product a CTA); CTA r takes the 64-key tiles r, r + CTAs, ...
//     of the visible span.
//   * S = Q K^T has 128 TMEM lanes, of which a unit fills 17..64.  Q is laid
//     down 2 (4) times, 64 (32) lanes apart, and copy g takes the columns
//     [32 g, 32 g + 32) ([16 g, 16 g + 16)) of every tile: its softmax runs over
//     those keys alone and its P is 0 elsewhere, so the copies are groups with
//     results of their own, joined at the end like the warps' of span_decode.cu,
//     and the four softmax warps share a tile without exchanging anything.  (The
//     products that are 0 cost tensor time that nothing waits for.)
//   * Warp 0 loads by TMA (K and V rings of their own; pages smaller than a tile
//     come as boxes of one page or a part of it, a box a lane), warp 1 issues the
//     products, warps 2..5 are the softmax.  S is double-buffered: the products
//     of tile i + 1 run ahead of the softmax of tile i.
//   * Boxes that no row sees are not read (coordinates outside the tensor: zeros);
//     rows of V that no row sees inside a box are cleared before the product
//     (0 * NaN would reach the sums).
//   * A wait that runs out leaves NaN in the unit's outputs (fia_decode_window has
//     no workspace to report in) and FIA_ERR_TIMEOUT in a status word, if any.
// Bound: HBM with many units (256 of 64 rows and 4096 keys: 84.8 us, 96% of a
// copy's rate; 512 of 32 rows, window 2048: 96 us, 85%); with fewer the chain of a
// tile, 0.6 us for 32 KB (128 units of 64 rows, 2000 to 4096 keys: 42 us, 73%;
// mma.sync 88).  128-key tiles and one CTA an SM: 96, 121 and 51 us.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "host.h"
#include "span_join.cuh"

namespace fia {
namespace {

constexpr int kWideThreads = 192;

struct WideParams {
  SpanParams s;
  CUtensorMap tm_q;               // (D, q_tokens, heads of a group, KV_N, B): a box is a unit's rows
  CUtensorMap tm_k, tm_v;         // (D, block_size, KV_N, blocknum) or (D, S, KV_N, B), boxes of 2^lg_box rows
  int lg_box;
  unsigned long long limit_ns;    // of a wait
};

constexpr int kKeys = 64;            // of a tile
// Start cost of a CTA in tiles.  (1, 2, 4, 8 CTAs of a unit, us, 64 rows, D 128:
// 128 units with 2000..4096 keys 55.0, 42.0, 49.5, 66.9; 64 units of 4096 keys
// 51.9, 37.1, 30.3, 40.4; 256 units 84.9, 97.4, 117, 153.  16 instead of 8: one
// unit of 30000 keys 61.1 -> 35.2.)
constexpr int kWideStart = 10;

template <int D, int R>
struct WideCfg {
  static constexpr int kGroups = 128 / R;        // copies of the rows
  static constexpr int kCols = kKeys / kGroups;  // columns of a copy
  static constexpr int kChunks = D / 64;
  static constexpr int kBoxQ = 128 * 128, kBox = kKeys * 128;   // 64 columns of Q, of a tile
  static constexpr int kTile = kChunks * kBox;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kChunks * kBoxQ;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kEnd = kOffV + kStages * kTile;
  // after the loops what the join receives and O of the groups take this place
  static constexpr int kOffIn = 0;
  static constexpr int kOffO = (JoinIn<D, R>::kBytes + 1023) / 1024 * 1024;
  static constexpr int kOffML = kEnd > kOffO + 128 * D * 4 ? kEnd : kOffO + 128 * D * 4;
  static constexpr int kOffBar = kOffML + 128 * 8;
  static constexpr int kSmem = kOffBar + 256 + 1024;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
  // TMEM columns: S twice (its first half becomes P), O
  static constexpr uint32_t kColO = 2 * kKeys, kTmem = 256;
};

struct WideBars {
  uint64_t q_full;
  uint64_t k_full[4], v_full[4], v_free[4];
  uint64_t s_full[4];      // [step % stages]: S is in TMEM, and the K stage free
  uint64_t p_full[2];      // [step & 1]: P is in TMEM (4 warps)
  uint64_t drain;          // after an abort
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

// N columns of this lane from TMEM column `col` on.
template <int N>
__device__ __forceinline__ void load_columns(uint32_t col, float (&x)[N]) {
  if constexpr (N == 16) {
    uint32_t u[16];
    tmem_ld16(col, u);
    tmem_wait_ld(u);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(u[e]);
  } else {
    uint32_t u[N / 32][32];
#pragma unroll
    for (int q = 0; q < N / 32; ++q) tmem_ld32(col + q * 32, u[q]);
#pragma unroll
    for (int q = 0; q < N / 32; ++q) tmem_wait_ld(u[q]);
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = __uint_as_float(u[e / 32][e % 32]);
  }
}

template <int D, bool BF16, int R>
__global__ void __launch_bounds__(kWideThreads, 2) span_wide_kernel(const __grid_constant__ WideParams w) {
  using C = WideCfg<D, R>;
  constexpr int ST = C::kStages;
  const SpanParams& p = w.s;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  WideBars* bar = reinterpret_cast<WideBars*>(smem + C::kOffBar);
  volatile int* abort_flag = &bar->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t lg = uint32_t(p.lg_cs), cs = 1u << lg, rank = blockIdx.x & (cs - 1u);
  const int b = int(blockIdx.x >> lg), kvh = blockIdx.y;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&w.tm_q);
    tma_prefetch_desc(&w.tm_k);
    tma_prefetch_desc(&w.tm_v);
    mbar_init(&bar->q_full, 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&bar->k_full[s], 1);
      mbar_init(&bar->v_full[s], 1);
      mbar_init(&bar->v_free[s], 1);
      mbar_init(&bar->s_full[s], 1);
    }
    mbar_init(&bar->p_full[0], 4);
    mbar_init(&bar->p_full[1], 4);
    mbar_init(&bar->drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // the copies' rows behind the unit's: zeros
  for (int e = threadIdx.x; e < C::kGroups * (R - p.rows) * (D / 8); e += kWideThreads) {
    const int row = e / (D / 8), c = e % (D / 8), g = row / (R - p.rows), at = g * R + p.rows + row % (R - p.rows);
    *reinterpret_cast<uint4*>(smem + C::kOffQ + (c / 8) * C::kBoxQ + at * 128 + (c % 8) * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  // Behind a prefix kernel, which lets this one go once everything before both
  // is complete, only the join has to wait for it.
  if (p.n_parts == 0) grid_dep_wait();
  int len = p.kv_max;
  if (p.kv_len != nullptr)
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(len) : "l"(p.kv_len + b) : "memory");
  // TMEM is held neither while this kernel waits for one before it, whose CTAs
  // may yet have to get theirs, nor wanted once it has let the next one in, which
  // may hold its own and wait for this one: either could wait forever.
  if (warp == 1) {
    tmem_alloc(&bar->tmem, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  grid_dep_launch();

  const int L = min(max(len, 0), p.kv_max);
  const int first = L - p.q_tokens;               // position of token 0 (may be negative: tokens that see nothing)
  // the tiles that hold a key some row may see: the sinks' and the window's
  const int t_base = p.base / kKeys, t_end = (L + kKeys - 1) / kKeys;
  const int t_sink = min(t_end, max(t_base, (p.sink + kKeys - 1) / kKeys));
  const int win = int(max(int64_t(first) - p.pre, int64_t(0)));   // first key of token 0's window
  const int t_win = max(t_sink, win / kKeys);
  const int n_sink = max(0, t_sink - t_base);
  const int n_tiles = n_sink + max(0, t_end - t_win);
  const int n = n_tiles > int(rank) ? (n_tiles - int(rank) + int(cs) - 1) >> lg : 0;   // this CTA's steps
  auto tile_key = [&](int i) -> int {
    const int v = int(rank) + (i << lg);
    return (v < n_sink ? t_base + v : t_win + v - n_sink) * kKeys;
  };
  auto some_row_sees = [&](int j) -> bool { return j < L && j >= p.base && (j < p.sink || j >= win); };

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    if (lane == 0 && n > 0) {   // (without a tile the results' zeros take this place at once)
      mbar_arrive_expect_tx(&bar->q_full, C::kGroups * C::kChunks * p.rows * 128);
#pragma unroll 1
      for (int g = 0; g < C::kGroups; ++g)
#pragma unroll 1
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_5d(smem + C::kOffQ + c * C::kBoxQ + g * R * 128, &w.tm_q, &bar->q_full, c * 64, 0, 0, kvh, b);
    }
    // a lane loads box `sub` of chunk `chunk` of every tile
    const int lg_per = 6 - w.lg_box, sub = lane & ((1 << lg_per) - 1), chunk = lane >> lg_per;
    const bool mine = chunk < C::kChunks;
    // where this lane's box of tile i starts: row and last coordinate (-1: nowhere)
    auto box_at = [&](int i, int& row, int& id) {
      row = 0;
      id = -1;
      if (i >= n || !mine) return;
      const int k0 = tile_key(i) + (sub << w.lg_box), k1 = k0 + (1 << w.lg_box);
      if (k0 >= L || k1 <= p.base || (k0 >= p.sink && k1 <= win)) return;
      row = k0;
      id = b;
      if (p.block_table != nullptr) {
        const int page = p.lg_block >= 0 ? k0 >> p.lg_block : k0 / p.block_size;
        // (k0 < L: a column of the table)
        id = p.block_table[(k0 < p.shared ? 0 : int64_t(b) * p.table_stride) + page];
        row = k0 - page * p.block_size;
      }
    };
    auto load = [&](int kv, int i, int row, int id) -> bool {
      const int s = i % ST;
      if (i >= ST) {
        uint64_t* freed = kv == 0 ? &bar->s_full[s] : &bar->v_free[s];
        if (!__all_sync(0xffffffffu, wait(freed, ((i / ST) - 1) & 1, abort_flag, w.limit_ns))) return false;
      }
      uint64_t* full = kv == 0 ? &bar->k_full[s] : &bar->v_full[s];
      uint8_t* dst = smem + (kv == 0 ? C::kOffK : C::kOffV) + s * C::kTile;
      if (lane == 0) mbar_arrive_expect_tx(full, C::kTile);
      __syncwarp();
      if (mine)
        tma_load_4d(dst + chunk * C::kBox + ((sub << w.lg_box) * 128), kv == 0 ? &w.tm_k : &w.tm_v, full, chunk * 64, row,
                    kvh, id < p.n_blocks ? id : -1);   // (looked at only here: the load has had a tile's time)
      return true;
    };
    int row, id, row_v = 0, id_v = -1, nk = 0, nv = 0;
    box_at(0, row, id);
#pragma unroll 1
    for (int i = 0; i <= n && n > 0; ++i) {
      // K of tile i, then V of tile i - 1; the next box's page id meanwhile
      if (i < n) {
        if (!load(0, i, row, id)) break;
        nk = i + 1;
      }
      int row_n, id_n;
      box_at(i + 1, row_n, id_n);
      if (i > 0) {
        if (!load(1, i - 1, row_v, id_v)) break;
        nv = i;
      }
      row_v = row;
      id_v = id;
      row = row_n;
      id = id_n;
    }
    __syncwarp();
    if (lane == 0) {
      // Every copy lands before the CTA exits, also where another role gives up
      // after these loads have all been issued (nothing waits for this lane).
      if (n > 0) wait(&bar->q_full, 0, nullptr, kWaitLimitNs);
      for (int s = 0; s < ST; ++s) {
        if (nk > s) wait(&bar->k_full[s], ((nk - 1 - (nk - 1 - s) % ST) / ST) & 1, nullptr, kWaitLimitNs);
        if (nv > s) wait(&bar->v_full[s], ((nv - 1 - (nv - 1 - s) % ST) / ST) & 1, nullptr, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_f16(128, kKeys, BF16 ? 1 : 0, 0, 0);
      constexpr uint32_t idesc_pv = idesc_f16(128, D, BF16 ? 1 : 0, 0, 1);
      const uint64_t qd = smem_desc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
      const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t vd0 = smem_desc_sw128(smem_u32(smem + C::kOffV), C::kBox, 1024);
      auto qk = [&](int i) -> bool {
        const int s = i % ST;
        if (!wait(&bar->k_full[s], (i / ST) & 1, abort_flag, w.limit_ns)) return false;
        tc_fence_after();
        const uint64_t kd = kd0 + uint64_t(s) * (C::kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          mma_ss(tmem + (i & 1) * kKeys, qd + uint64_t(((kk >> 2) * C::kBoxQ + (kk & 3) * 32) >> 4),
                 kd + uint64_t(((kk >> 2) * C::kBox + (kk & 3) * 32) >> 4), idesc_qk, kk > 0 ? 1u : 0u);
        }
        mma_commit(&bar->s_full[s]);
        return true;
      };
      bool ok = n == 0 || wait(&bar->q_full, 0, abort_flag, w.limit_ns);
      if (ok && n > 0) ok = qk(0);
      if (ok && n > 1) ok = qk(1);
      int done = 0;            // P V committed
#pragma unroll 1
      for (int i = 0; ok && i < n; ++i) {
        const int s = i % ST;
        ok = wait(&bar->p_full[i & 1], (i >> 1) & 1, abort_flag, w.limit_ns) &&
             wait(&bar->v_full[s], (i / ST) & 1, abort_flag, w.limit_ns);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = vd0 + uint64_t(s) * (C::kTile >> 4);
        const uint32_t pt = tmem + (i & 1) * kKeys;
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ts(tmem + C::kColO, pt + kk * 8, vd + uint64_t((kk * 2048) >> 4), idesc_pv, (i | kk) != 0 ? 1u : 0u);
        mma_commit(&bar->v_free[s]);
        done = i + 1;
        if (i + 2 < n) ok = qk(i + 2);
      }
      // every product issued has finished before TMEM goes
      if (ok) {
        if (done > 0) wait(&bar->v_free[(done - 1) % ST], ((done - 1) / ST) & 1, nullptr, kWaitLimitNs);
      } else {
        mma_commit(&bar->drain);
        wait(&bar->drain, 0, nullptr, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    const int quad = warp & 3, g = quad * 32 / R, r = quad * 32 % R + lane;
    const uint32_t lane_off = uint32_t(quad * 32) << 16;
    const uint32_t col_o = tmem + lane_off + C::kColO;
    const int tok = r - span_head(p, r) * p.q_tokens;      // (rows behind the unit's: whatever)
    const int pos = first + tok, w_lo = int(max(int64_t(pos) - p.pre, int64_t(0)));
    const int win_last = int(max(int64_t(L) - 1 - p.pre, int64_t(0)));   // the last token's window
    const float sl2 = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int s = i % ST, j0 = tile_key(i);
      if (!__all_sync(0xffffffffu, wait(&bar->s_full[s], (i / ST) & 1, abort_flag, w.limit_ns))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t col_s = tmem + lane_off + (i & 1) * kKeys + g * C::kCols;
      float x[C::kCols];
      load_columns<C::kCols>(col_s, x);
      // every row sees every key of the tile
      const bool full = j0 + kKeys - 1 <= first && j0 >= p.base && (j0 + kKeys <= p.sink || j0 >= win_last);
      if (!full) {
        const int c0 = j0 + g * C::kCols;
#pragma unroll
        for (int c = 0; c < C::kCols; ++c) {
          const int j = c0 + c;
          if (j > pos || j < p.base || (j >= p.sink && j < w_lo)) x[c] = -INFINITY;
        }
      }
      const float m_new = fmaxf(m, tree_max<C::kCols>(x) * sl2);
      // A stale maximum is kept until it grows by more than 8 (log2 units): p <=
      // 2^8 stays exact in fp32 and representable in the cache's type.
      const float m_use = (m == -INFINITY || m_new > m + 8.f) ? m_new : m;
      const float alpha = m_use == m ? 1.f : fast_exp2(m - m_use);
      const float mo = m_use == -INFINITY ? 0.f : m_use;
      l = l * alpha + exp2_and_sum<C::kCols>(x, sl2, mo);
      m = m_use;
      if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
        // O holds the step before's product once its V stage is free
        if (!__all_sync(0xffffffffu, wait(&bar->v_free[(i - 1) % ST], ((i - 1) / ST) & 1, abort_flag, w.limit_ns))) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
          uint32_t u[16];
          tmem_ld16(col_o + q * 16, u);
          tmem_wait_ld(u);
#pragma unroll
          for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha);
          tmem_st16(col_o + q * 16, u);
        }
      }
      // P of all the tile's keys, 0 but for the copy's, over S (this lane's alone)
      uint32_t u[kKeys / 2];
#pragma unroll
      for (int q = 0; q < C::kGroups; ++q)
#pragma unroll
        for (int e = 0; e < C::kCols / 2; ++e)
          u[q * (C::kCols / 2) + e] = q == g ? pack2(x[2 * e], x[2 * e + 1], BF16) : 0u;
      tmem_st32(tmem + lane_off + (i & 1) * kKeys, u);
      const bool whole = j0 + kKeys <= L && j0 >= p.base && (j0 + kKeys <= p.sink || j0 >= win);
      if (!whole) {
        if (!__all_sync(0xffffffffu, wait(&bar->v_full[s], (i / ST) & 1, abort_flag, w.limit_ns))) {
          ok = false;
          break;
        }
        const int row = quad * 32 + lane;
        if (row < kKeys && !some_row_sees(j0 + row)) {
          uint8_t* vs = smem + C::kOffV + s * C::kTile + row * 128;
#pragma unroll
          for (int ch = 0; ch < C::kChunks; ++ch)
#pragma unroll
            for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4*>(vs + ch * C::kBox + q * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&bar->p_full[i & 1]);
    }
    if (!ok) tmem_wait_st();   // no store to TMEM is pending when it goes
    if (ok && n > 0)
      ok = __all_sync(0xffffffffu, wait(&bar->v_free[(n - 1) % ST], ((n - 1) / ST) & 1, abort_flag, w.limit_ns));
    tc_fence_after();
    if (ok) {
      // O to its place: every copy has landed and every product is done.  (Other
      // CTAs' results may land in the queries' place once the cluster's barrier
      // is through, which waits for every thread of this CTA.)
      float* ob = reinterpret_cast<float*>(smem + C::kOffO);
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
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4*>(ob + join_at<D, R>(g, r, q * 8 + e)) = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
      }
      reinterpret_cast<float2*>(smem + C::kOffML)[g * R + r] = make_float2(m, l);
    }
    tc_fence_before();
  }

  // (waited for before the join's first remote store: no CTA's Q and rings are in use)
  __syncwarp();
  if (lg != 0) cluster_arrive();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffML);
  if (*abort_flag != 0) {
    const float nan = __uint_as_float(0x7fc00000u);
    for (int e = threadIdx.x; e < 128; e += kWideThreads) ml[e] = make_float2(nan, nan);
    if (threadIdx.x == 0) {
      // (the word may hold anything until it has this call's epoch: a larger one
      // would hide the raise, and the stamp below would then clear it)
      if (p.n_parts == 0) status_stamp(p.status);
      status_raise(p.status, 10u /* FIA_ERR_TIMEOUT */);
    }
  }
  span_join<D, BF16, R, C::kGroups, kWideThreads>(p, reinterpret_cast<const float*>(smem + C::kOffO), ml,
                                                  smem + C::kOffIn, lg, rank, b, kvh);
  // (a word that this call has raised stays)
  if (p.n_parts == 0 && (threadIdx.x | blockIdx.x | blockIdx.y) == 0) status_stamp(p.status);
}

template <int D, bool BF16, int R>
cudaError_t launch_one(const WideParams& w, cudaStream_t s) {
  constexpr int smem = WideCfg<D, R>::kSmem;
  cudaError_t e = prepare_span<span_wide_kernel<D, BF16, R>>(smem);
  if (e != cudaSuccess) return e;
  return launch_span(span_wide_kernel<D, BF16, R>, w, w.s, kWideThreads, smem, s);
}

template <int D, bool BF16>
cudaError_t launch_wide(const WideParams& w, cudaStream_t s) {
  return w.s.rows <= 32 ? launch_one<D, BF16, 32>(w, s) : launch_one<D, BF16, 64>(w, s);
}

}  // namespace

// Keys of a unit at most.
static int64_t visible_span(const SpanParams& p) {
  return std::min<int64_t>(p.kv_max - p.base, int64_t(p.sink) + p.pre + p.q_tokens);
}

// 17..32 rows with few keys: span_decode.cu starts and ends faster.  (us, here and
// there, D 128, 32 rows, spans of 128, 384, 1024, 2048, 4096 keys: 8 units 7.7 7.6
// 9.2 10.6 13.2 and 6.2 6.4 8.6 10.8 15.2; 64 units 9.5 10.5 14.4 19.2 28.5 and 7.6
// 9.1 13.9 20.6 32.4; 256 units 11.3 16.6 28.4 46.6 82.6 and 10.1 17.0 32.1 55.2
// 100.5.  With 64 rows this kernel is at most 3% behind at 128 keys and ahead from
// 384 on: 256 units 12.9 18.2 30.2 48.7 84.8 and 14.3 23.8 44.7 77.5 208.)
bool span_wide_pays(const SpanParams& p, int n_sm) {
  const int64_t span = visible_span(p);
  return p.rows > 32 || (p.rows > 16 && (span >= 2048 || (span >= 256 && int64_t(p.B) * p.N2 > n_sm)));
}

fia_status launch_span_wide(const SpanParams& p, int head_dim, bool bf16, int n_sm, cudaStream_t s) {
  WideParams w;
  memset(&w, 0, sizeof(w));
  w.s = p;
  set_span_shape(w.s, cluster_ctas(int64_t(p.B) * p.N2, p.rows, visible_span(p) / kKeys + 1, 1, kWideStart, true,
                                   2, n_sm));
  const uint64_t e = 2, D = uint64_t(head_dim), g = uint64_t(p.group), Q = uint64_t(p.q_tokens);
  const uint64_t qd[5] = {D, Q, g, uint64_t(p.N2), uint64_t(p.B)};
  const uint64_t qs[4] = {uint64_t(p.q_ss) * e, uint64_t(p.q_sn) * e, uint64_t(p.q_sn) * g * e, uint64_t(p.q_sb) * e};
  const uint32_t box[5] = {64, uint32_t(Q), uint32_t(g), 1, 1};
  fia_status st = make_map(&w.tm_q, p.q, 5, qd, qs, 0, false, box);
  if (st != FIA_OK) return st;
  const bool paged = p.block_table != nullptr;
  w.lg_box = 6;
  while (paged && p.block_size % (1 << w.lg_box) != 0) --w.lg_box;
  // (without keys every box lies outside, but a map wants an extent)
  const bool none = p.kv_max == 0 || p.n_blocks == 0;
  const uint64_t kd[4] = {D, none ? 1 : uint64_t(paged ? p.block_size : p.kv_max), none ? 1 : uint64_t(p.N2),
                          none ? 1 : uint64_t(p.n_blocks)};
  const uint64_t ks[3] = {none ? D * e : uint64_t(p.row_stride) * e, none ? D * e : uint64_t(p.head_stride) * e,
                          none ? D * e : uint64_t(p.blk_stride) * e};
  st = make_map(&w.tm_k, none ? p.q : p.k, 4, kd, ks, 1u << w.lg_box);
  if (st == FIA_OK) st = make_map(&w.tm_v, none ? p.q : p.v, 4, kd, ks, 1u << w.lg_box);
  if (st != FIA_OK) return st;
  w.limit_ns = make_status(nullptr).limit_ns;
  cudaError_t r;
  if (head_dim == 128)
    r = bf16 ? launch_wide<128, true>(w, s) : launch_wide<128, false>(w, s);
  else
    r = bf16 ? launch_wide<64, true>(w, s) : launch_wide<64, false>(w, s);
  return cuda_check(r, "decode launch");
}

}  // namespace fia
