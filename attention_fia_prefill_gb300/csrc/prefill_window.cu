// Prefill with a sliding window and sink tokens, lengths in device memory:
// row i of a batch, at position p = i + kv_len - q_len, sees key j when j <= p
// and (j >= p - pre or j < sink).  Contiguous or paged K/V, head dims 64 / 128.
//
// The products and the softmax are prefill_pair.cu's: an item is 256 rows of
// one (batch, query head), tiles A and B of 128 rows, and the tensor core
// alternates between them.  A window makes items short (a window of 1024 keys:
// ten steps), so what an item costs beside its steps counts: with one CTA per
// item it was about 10 us (start, lengths, first loads, the pipeline's filling
// and draining, output), as much as eleven tile products.  Here CTAs are
// persistent, one per SM, and walk items blockIdx.x, + gridDim.x, ...:
//   * every ring, barrier and count runs on across items; the next item's Q
//     and first K/V tiles load while the last steps run, its first Q_A K^T and
//     Q_B K^T are issued between the last products of this one, and one tile's
//     warps write their output while the other tile's products run;
//   * warp 0 finds the items (from their index and the lengths on the device; TND
//     by a scan of the running sums), one ahead, and hands them to the other
//     roles through a small ring in shared memory;
//   * a step's tile may need few of its 128 columns: the sinks' tile ceil(sink /
//     16) * 16 of them, tile B's first band tile (before its window, walked
//     because tile A needs it) none, for which 16 are taken.  The products are
//     cut to them;
//   * the code is kept small (rolled loops, short waits, one path for whole tiles
//     and for those on an edge of the window, whose hidden columns come as bit
//     masks): it exceeds an SM's instruction cache, and the misses cost up to a
//     third (cache hit rate 73% at 401 us, 94% at 305);
//   * registers move from the producer's and issuer's warps to the softmax's
//     (setmaxnreg; 384 threads x 168 = 128 x 120 + 256 x 192): a few spilled ones
//     in the softmax's loop cost 5%, 294 -> 275 us with a path of their own for
//     edge tiles; without that path 258.
// Ragged prompts (8 sequences of 256..4096, 32 heads, window 1024): 253 us, one
// CTA per item 350; chunks of 2048 after contexts up to 14336, window 4096: 720
// and 837 us.  Bound: the chain of a tile's step (products 1024 cycles, softmax
// 1300, hand-over 600) with two tiles in flight, and an item's first and last
// steps and output, about 4 us.
// The walk of an item: the tiles of the sinks that the band does not hold, then
// the band's from tile A's first to tile B's last (tile A stops at its own).
#include <algorithm>
#include <type_traits>

#include "paged.h"
#include "ptx.cuh"

namespace fia {
namespace {

constexpr int kPairRows = 2 * kTileM;
constexpr int kInfos = 3;            // items in the ring between warp 0 and the other roles

// One item; n_a, n_b: steps of tiles A and B (n_a <= n_b, or n_b = 0 when tile
// B has no row or no key), steps [0, n_sink) over sinks' tiles, the rest over
// tiles jt0, jt0 + 1, ...  A step takes 128 columns of its tile, but for the
// last sinks' step (cols_sink) and tile B's first band step (cols_b).
struct WinItem {
  int valid, b, h, q0, q_row0, q_len, kv_row0, kv_len, n_a, n_b, n_sink, jt0, cols_sink, cols_b;
};

template <int D>
struct WinCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kBox = 128 * 128;
  static constexpr int kTile = kChunks * kBox;
  static constexpr int kStages = D == 64 ? 3 : 2;       // K ring and V ring
  static constexpr int kOffQ = 0;                       // Q_A, Q_B
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffBar = kOffV + kStages * kTile;
  static constexpr int kSmem = kOffBar + 512 + 1024;
  static constexpr int kThreads = 384;
  static constexpr uint32_t kColO = 256;
};

// Counts run over all items of the CTA: `step` of the K/V rings, `c` of a
// tile's products.  Each barrier's next phase needs its waiter's own next
// action, so a phase parity is never mistaken for the one two before it.
struct WinBars {
  uint64_t q_full[2];          // Q of tile t: phase = items that loaded it
  uint64_t k_full[3], v_full[3];
  uint64_t v_free[3];          // the step's last P V is done (one commit per step)
  uint64_t s_full[2][3];       // [t][c % stages]: S_t is in TMEM; tile B's (A's without B) frees the K stage
  uint64_t p_full[2][2];       // [t][c & 1]: P_t is in TMEM (4 warps)
  uint64_t a_done;             // tile A's last P V of an item is done
  uint64_t b_read;             // tile B's warps have seen their item's last P V (4 warps)
  uint64_t drain;              // after an abort
  uint64_t info_full[kInfos], info_free[kInfos];
  WinItem info[kInfos];
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(WinBars) <= 512, "barrier area");

// Bounded wait for a phase, in few instructions (this kernel's code is larger
// than an SM's instruction cache, and every wait is inlined): a wait that runs
// out only raises the CTA's abort flag, from which thread 0 records
// FIA_ERR_TIMEOUT at the end.
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

// Item x of the call, from sizes and the lengths on the device (taken into
// their tensors' range, whatever they hold).  Items run head by head over one
// pair of tiles (the heads of a group read the same keys), the last pair of a
// batch first.  All lanes of a warp; the result is the same in every lane.
__device__ __forceinline__ WinItem locate_item(const PrefillParams& p, int idx) {
  WinItem it;
  it.valid = 0;
  if (idx >= p.n_items) return it;
  const int lane = threadIdx.x & 31;
  const int x = idx / p.num_heads;
  it.h = idx - x * p.num_heads;
  int q_start = 0, pair = 0;
  if (!p.is_tnd) {
    const int nt = (p.s1 + kPairRows - 1) / kPairRows;
    it.b = x / nt;
    pair = nt - 1 - (x - it.b * nt);
    it.q_len = p.q_lens == nullptr ? p.s1 : min(max(p.q_lens[it.b], 0), p.s1);
  } else {
    int before = 0;
    it.b = -1;
    for (int b0 = 0; b0 < p.n_batch; b0 += 32) {
      const int b = b0 + lane;
      const int s = b < p.n_batch && b > 0 ? min(max(p.q_lens[b - 1], 0), p.s1) : 0;
      const int e = b < p.n_batch ? min(max(p.q_lens[b], s), p.s1) : s;
      int sum = (e - s + kPairRows - 1) / kPairRows;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, x < before + sum);
      if (hit != 0u) {
        const int l = __ffs(hit) - 1;
        it.b = b0 + l;
        pair = __shfl_sync(0xffffffffu, before + sum, l) - 1 - x;
        q_start = __shfl_sync(0xffffffffu, s, l);
        it.q_len = __shfl_sync(0xffffffffu, e - s, l);
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (it.b < 0) return it;
  }
  it.kv_row0 = 0;
  if (p.kv_lens == nullptr) {
    it.kv_len = p.s2;
  } else if (p.is_tnd && p.block_table == nullptr) {
    const int s = it.b > 0 ? min(max(p.kv_lens[it.b - 1], 0), p.s2) : 0;
    it.kv_row0 = s;
    it.kv_len = min(max(p.kv_lens[it.b], s), p.s2) - s;
  } else {
    it.kv_len = min(max(p.kv_lens[it.b], 0), p.s2);
  }
  it.valid = 1;
  it.q0 = pair * kPairRows;
  it.q_row0 = q_start + it.q0;
  // positions of tile A's first row and of both tiles' last rows
  const int64_t d = int64_t(it.kv_len) - it.q_len;
  const int64_t lo = max(int64_t(0), it.q0 + d - p.band_pre);
  const int64_t hi_a = min(it.q0 + kTileM, it.q_len) - 1 + d, hi = min(it.q0 + kPairRows, it.q_len) - 1 + d;
  const bool rows = it.q0 < it.q_len && hi >= 0;   // hi < kv_len, lo <= hi
  it.jt0 = int(lo / kTileN);
  it.n_sink = rows ? min((p.sink + kTileN - 1) / kTileN, it.jt0) : 0;
  it.n_a = rows && hi_a >= 0 ? it.n_sink + int(hi_a / kTileN) - it.jt0 + 1 : 0;
  it.n_b = rows && it.q0 + kTileM < it.q_len ? it.n_sink + int(hi / kTileN) - it.jt0 + 1 : 0;
  auto sinks_of = [&](int tile) -> int { return min((max(p.sink - tile * kTileN, 1) + 15) & ~15, kTileN); };
  it.cols_sink = sinks_of(max(it.n_sink - 1, 0));
  // tile B's window starts past its first band tile, which may hold sinks
  it.cols_b = int64_t(it.jt0 + 1) * kTileN <= it.q0 + kTileM + d - p.band_pre ? sinks_of(it.jt0) : kTileN;
  return it;
}

// K/V tile of step j.
__device__ __forceinline__ int tile_of(const WinItem& it, int j) { return j < it.n_sink ? j : it.jt0 + j - it.n_sink; }

// Columns of the step's tile that tile t takes: a multiple of 16.
__device__ __forceinline__ int columns(int n_sink, int cols_sink, int cols_b, int t, int j) {
  return j == n_sink - 1 ? cols_sink : (t == 1 && j == n_sink) ? cols_b : kTileN;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(WinCfg<D>::kThreads, 1) prefill_window_kernel(const __grid_constant__ PrefillParams p) {
  using C = WinCfg<D>;
  constexpr int ST = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  WinBars* bar = reinterpret_cast<WinBars*>(smem + C::kOffBar);
  volatile int* abort_flag = &bar->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar->q_full[t], 1);
      mbar_init(&bar->p_full[t][0], 4);
      mbar_init(&bar->p_full[t][1], 4);
      for (int s = 0; s < ST; ++s) mbar_init(&bar->s_full[t][s], 1);
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(&bar->k_full[s], 1);
      mbar_init(&bar->v_full[s], 1);
      mbar_init(&bar->v_free[s], 1);
    }
    mbar_init(&bar->a_done, 1);
    mbar_init(&bar->b_read, 4);
    mbar_init(&bar->drain, 1);
    for (int s = 0; s < kInfos; ++s) {
      mbar_init(&bar->info_full[s], 1);
      mbar_init(&bar->info_free[s], 9);   // the MMA issuer and eight softmax warps
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  // The launch overlaps the end of the kernel before; this one lets the next go
  // by ending (let go at the start, its CTAs cost 3%).  TMEM is taken after the
  // wait: no kernel waits with it in hand.
  grid_dep_wait();
  if (threadIdx.x == 0 && blockIdx.x == 0) status_stamp(p.status);
  if (warp == 1) {
    tmem_alloc(&bar->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  const bool is_tnd = p.is_tnd != 0;

  if (warp == 0) {
    // ------------------------------------------------------- items, producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (lane == 0) {
      tma_prefetch_desc(&p.tm_q);
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
    }
    // finds item k and hands it over
    auto leave_item = [&](int k) -> bool {
      bool ok = true;
      if (lane == 0 && k >= kInfos)
        ok = wait(&bar->info_free[k % kInfos], ((k / kInfos) - 1) & 1, abort_flag, p.status.limit_ns);
      ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
      if (!ok) return false;
      const WinItem it = locate_item(p, blockIdx.x + k * gridDim.x);
      if (lane == 0) {
        bar->info[k % kInfos] = it;
        mbar_arrive(&bar->info_full[k % kInfos]);
      }
      __syncwarp();
      return it.valid != 0;
    };
    int step = 0, nk = 0, nv = 0;          // steps loaded; K and V loads issued
    int ca = 0, cb = 0, nqa = 0, nqb = 0;  // the tiles' products so far; Q loads
    // the product that frees each stage's K: 2 count + tile
    int f0 = 0, f1 = 0, f2 = 0;
    bool ok = true, more = true;
#pragma unroll 1
    for (int k = -1; ok && more; ++k) {
      // an item's first steps, then the next item (its lengths take a
      // microsecond to come), then the others; k = -1 has no steps
      WinItem it;
      it.n_a = it.n_b = 0;
      if (k >= 0) it = bar->info[k % kInfos];   // (left by this warp)
      const int n = max(it.n_a, it.n_b);
#pragma unroll 1
      for (int half = 0; half < 2 && ok; ++half) {
        if (half == 1) more = leave_item(k + 1);
        if (lane == 0) {
          const int kvh = it.h / p.group, bc = is_tnd ? 0 : it.b;
          const int rel = it.n_b > 0 ? 2 * cb + 1 : 2 * ca;   // step 0's; + 2 for every step
          const int end = half == 0 ? min(n, ST) : n;
#pragma unroll 1
          for (int j = half == 0 ? 0 : ST; ok && j < end; ++j, ++step) {
            const int s = step % ST;
            const int key = tile_of(it, j) * kTileN;
            int kv_r = it.kv_row0 + key, kv_b = bc;
            if (p.block_table != nullptr) {
              const int page = key / p.block_size;
              kv_b = __ldg(p.block_table + int64_t(it.b) * p.table_stride + page);
              if (kv_b >= p.n_blocks) kv_b = -1;
              kv_r = key - page * p.block_size;
            }
            // K and V of the step; ahead of step 0's, Q of tile A and of tile B
#pragma unroll 1
            for (int kv = 0; kv < 2 && ok; ++kv) {
              const int nq = kv == 0 ? it.n_a : it.n_b;
              if (j == 0 && nq > 0) {
                // once the tile's last product of the item before (count c - 1)
                // is done
                const int c = kv == 0 ? ca : cb;
                ok = c == 0 || wait(&bar->s_full[kv][(c - 1) % ST], ((c - 1) / ST) & 1, abort_flag, p.status.limit_ns);
                if (!ok) break;
                mbar_arrive_expect_tx(&bar->q_full[kv], C::kTile);
#pragma unroll
                for (int ch = 0; ch < C::kChunks; ++ch)
                  tma_load_4d(smem + C::kOffQ + kv * C::kTile + ch * C::kBox, &p.tm_q, &bar->q_full[kv], ch * 64,
                              it.q_row0 + kv * kTileM, it.h, bc);
                if (kv == 0) ++nqa; else ++nqb;
              }
              if (step >= ST) {
                const int f = s == 0 ? f0 : s == 1 ? f1 : f2, c = f >> 1;
                uint64_t* b = kv == 0 ? &bar->s_full[f & 1][c % ST] : &bar->v_free[s];
                ok = wait(b, kv == 0 ? (c / ST) & 1 : ((step / ST) - 1) & 1, abort_flag, p.status.limit_ns);
                if (!ok) break;
              }
              uint64_t* full = kv == 0 ? &bar->k_full[s] : &bar->v_full[s];
              uint8_t* dst = smem + (kv == 0 ? C::kOffK : C::kOffV) + s * C::kTile;
              const CUtensorMap* map = kv == 0 ? &p.tm_k : &p.tm_v;
              mbar_arrive_expect_tx(full, C::kTile);
#pragma unroll
              for (int ch = 0; ch < C::kChunks; ++ch) tma_load_4d(dst + ch * C::kBox, map, full, ch * 64, kv_r, kvh, kv_b);
              if (kv == 0) nk = step + 1; else nv = step + 1;
            }
            const int f = rel + 2 * j;
            f0 = s == 0 ? f : f0;
            f1 = s == 1 ? f : f1;
            f2 = s == 2 ? f : f2;
          }
          if (half == 1) {
            ca += it.n_a;
            cb += it.n_b;
          }
        }
        ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
      }
    }
    if (lane == 0) {
      // Every copy lands before the CTA exits, also where another role gives up
      // after these loads have all been issued (nothing waits for this lane).
      if (nqa > 0) wait(&bar->q_full[0], (nqa - 1) & 1, nullptr, kWaitLimitNs);
      if (nqb > 0) wait(&bar->q_full[1], (nqb - 1) & 1, nullptr, kWaitLimitNs);
      for (int s = 0; s < ST; ++s) {
        if (nk > s) wait(&bar->k_full[s], ((nk - 1 - (nk - 1 - s) % ST) / ST) & 1, nullptr, kWaitLimitNs);
        if (nv > s) wait(&bar->v_full[s], ((nv - 1 - (nv - 1 - s) % ST) / ST) & 1, nullptr, kWaitLimitNs);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_f16(128, 0, BF16 ? 1 : 0, 0, 0);   // N is the step's
      constexpr uint32_t idesc_pv = idesc_f16(128, D, BF16 ? 1 : 0, 0, 1);
      const uint64_t qd0 = smem_desc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
      const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t vd0 = smem_desc_sw128(smem_u32(smem + C::kOffV), C::kBox, 1024);
      constexpr uint64_t kStep = C::kTile >> 4;
      uint64_t* last_bar = nullptr;   // barrier and phase of the latest commit
      uint32_t last_parity = 0;
      int ca = 0, cb = 0, pa = 0, pb = 0;      // Q K^T and P V issued of tiles A and B
      int items_a = 0, items_b = 0;            // items with steps of tile A, of tile B (Q K^T issued)
      // S_t = Q_t K^T of a step; first: of an item (its Q has to be in); wait_k:
      // the first product that reads the step's tile
      auto qk = [&](auto T, int& c, int& items, int step, bool first, bool wait_k, int cols) -> bool {
        constexpr int t = decltype(T)::value;
        const int s = step % ST;
        if (first) {
          if (!wait(&bar->q_full[t], items & 1, abort_flag, p.status.limit_ns)) return false;
          ++items;
        }
        if (wait_k && !wait(&bar->k_full[s], (step / ST) & 1, abort_flag, p.status.limit_ns)) return false;
        tc_fence_after();
        const uint32_t idesc = idesc_qk | (uint32_t(cols) >> 3 << 17);   // (a constant for whole tiles)
        const uint64_t qd = qd0 + t * kStep, kd = kd0 + uint64_t(s) * kStep;
        const uint32_t dst = tmem + t * 128;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = uint64_t(((kk >> 2) * C::kBox + (kk & 3) * 32) >> 4);
          mma_ss(dst, qd + off, kd + off, idesc, kk > 0 ? 1u : 0u);
        }
        last_bar = &bar->s_full[t][c % ST];
        last_parity = (c / ST) & 1;
        mma_commit(last_bar);
        ++c;
        return true;
      };
      // O_t (+)= P_t V of a step; done: the barrier to signal, or none
      auto pv = [&](auto T, int& c, int step, bool first, bool wait_v, int cols, uint64_t* done, uint32_t parity) -> bool {
        constexpr int t = decltype(T)::value;
        const int s = step % ST;
        if (!wait(&bar->p_full[t][c & 1], (c >> 1) & 1, abort_flag, p.status.limit_ns)) return false;
        ++c;
        if (wait_v && !wait(&bar->v_full[s], (step / ST) & 1, abort_flag, p.status.limit_ns)) return false;
        tc_fence_after();
        const uint64_t vd = vd0 + uint64_t(s) * kStep;
        const uint32_t dst = tmem + C::kColO + t * D, pt = tmem + t * 128;
        mma_ts(dst, pt, vd, idesc_pv, first ? 0u : 1u);
        if (cols == kTileN) {
#pragma unroll
          for (int kk = 1; kk < kTileN / 16; ++kk) mma_ts(dst, pt + kk * 8, vd + uint64_t((kk * 2048) >> 4), idesc_pv, 1u);
        } else {
          for (int kk = 1; kk < cols / 16; ++kk) mma_ts(dst, pt + kk * 8, vd + uint64_t((kk * 2048) >> 4), idesc_pv, 1u);
        }
        if (done != nullptr) {
          mma_commit(done);
          last_bar = done;
          last_parity = parity;
        }
        return true;
      };
      constexpr std::integral_constant<int, 0> A{};
      constexpr std::integral_constant<int, 1> B{};
      // what the issuer needs of an item
      struct Steps {
        int valid, n_a, n_b, n_sink, cols_sink, cols_b;
      };
      auto steps_of = [&](int k, Steps& w) -> bool {
        if (!wait(&bar->info_full[k % kInfos], (k / kInfos) & 1, abort_flag, p.status.limit_ns)) return false;
        const WinItem& i = bar->info[k % kInfos];
        w = Steps{i.valid, i.n_a, i.n_b, i.n_sink, i.cols_sink, i.cols_b};
        return true;
      };
      Steps w, nx;
      nx.valid = 0;
      int base = 0, done_a = 0, done_b = 0;    // first step of the item; items of tiles A and B behind it
      bool ok = steps_of(0, w), issued = false;   // issued: the item's first products are
      for (int k = 0; ok && w.valid; ++k) {
        const int n = max(w.n_a, w.n_b);
        auto cols = [&](const Steps& x, int t, int j) { return columns(x.n_sink, x.cols_sink, x.cols_b, t, j); };
        if (n == 0) ok = steps_of(k + 1, nx);
        // tile A alone frees V stages: not before tile B's warps have seen their
        // last item's
        if (n > 0 && w.n_b == 0 && done_b > 0)
          ok = wait(&bar->b_read, (done_b - 1) & 1, abort_flag, p.status.limit_ns);
        // step j = -1 issues the first products, where the item before did not
        for (int j = issued ? 0 : -1; j < n && ok; ++j) {
          const bool last = j == n - 1;
          const int step = base + j;
          if (j > w.n_sink && j + 1 < w.n_a) {
            // both tiles inside the item, whole tiles
            ok = pv(A, pa, step, false, true, kTileN, w.n_b == 0 ? &bar->v_free[step % ST] : nullptr,
                    uint32_t(step / ST) & 1u) &&
                 qk(A, ca, items_a, step + 1, false, true, kTileN);
            if (ok && w.n_b > 0)
              ok = pv(B, pb, step, false, false, kTileN, &bar->v_free[step % ST], uint32_t(step / ST) & 1u) &&
                   qk(B, cb, items_b, step + 1, false, false, kTileN);
            continue;
          }
          if (j >= 0 && j < w.n_a) {
            uint64_t* done = w.n_b == 0 ? &bar->v_free[step % ST] : j == w.n_a - 1 ? &bar->a_done : nullptr;
            ok = pv(A, pa, step, j == 0, true, cols(w, 0, j), done,
                    w.n_b == 0 ? uint32_t(step / ST) & 1u : uint32_t(done_a) & 1u);
          }
          if (ok && last && n > 0) ok = steps_of(k + 1, nx);
          const bool ahead = last && n > 0 && ok && nx.valid != 0;
          if (ok && (j + 1 < w.n_a || (ahead && nx.n_a > 0)))
            ok = qk(A, ca, items_a, step + 1, ahead || j < 0, true, ahead ? cols(nx, 0, 0) : cols(w, 0, j + 1));
          if (ok && j >= 0 && j < w.n_b)
            ok = pv(B, pb, step, j == 0, j >= w.n_a, cols(w, 1, j), &bar->v_free[step % ST], uint32_t(step / ST) & 1u);
          if (ok && (j + 1 < w.n_b || (ahead && nx.n_b > 0)))
            ok = qk(B, cb, items_b, step + 1, ahead || j < 0, ahead ? nx.n_a == 0 : j + 1 >= w.n_a,
                    ahead ? cols(nx, 1, 0) : cols(w, 1, j + 1));
        }
        issued = n > 0 && nx.valid != 0 && max(nx.n_a, nx.n_b) > 0;
        if (ok && n > 0 && w.n_b == 0) {
          // tile A's last P V signalled the V stage: its warps wait on a_done
          const int step = base + n - 1;
          ok = wait(&bar->v_free[step % ST], (step / ST) & 1, abort_flag, p.status.limit_ns);
          if (ok) mbar_arrive(&bar->a_done);
        }
        done_a += w.n_a > 0;
        done_b += w.n_b > 0;
        mbar_arrive(&bar->info_free[k % kInfos]);
        base += n;
        w = nx;
      }
      // every product issued has finished before TMEM goes: the latest commit
      // tracks them all, but for one that an abort left without its own
      if (last_bar != nullptr) wait(last_bar, last_parity, nullptr, kWaitLimitNs);
      if (!ok) {
        mma_commit(&bar->drain);
        wait(&bar->drain, 0, nullptr, kWaitLimitNs);
      }
    }
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int t = (warp - 4) >> 2;              // 0: tile A, 1: tile B
    const int r = 32 * (warp & 3) + lane;
    const uint32_t lane_off = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t col_s = tmem + lane_off + t * 128;
    const uint32_t col_o = tmem + lane_off + C::kColO + t * D;
    const float sl2 = p.scale_log2;
    auto rescale_o = [&](float alpha) {
#pragma unroll 1
      for (int q = 0; q < D / 16; ++q) {
        uint32_t u[16];
        tmem_ld16(col_o + q * 16, u);
        tmem_wait_ld(u);
#pragma unroll
        for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha);
        tmem_st16(col_o + q * 16, u);
      }
    };
    int c = 0, base = 0, items_a = 0;           // products of this tile; first step of the item; items with a tile A
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      ok = __all_sync(0xffffffffu, wait(&bar->info_full[k % kInfos], (k / kInfos) & 1, abort_flag, p.status.limit_ns));
      // (the item stays where it is until this warp frees it: what only the
      // output needs takes no register in the loop)
      const WinItem& it = bar->info[k % kInfos];
      if (!ok || !it.valid) break;
      const int n = t == 0 ? it.n_a : it.n_b, kv_len = it.kv_len, n_sink = it.n_sink;
      const int jt0 = it.jt0 - n_sink;          // of step 0, but for the sinks'
      const int clear_from = t == 0 ? 0 : it.n_a;   // steps whose V tail this tile clears
      const int i = it.q0 + t * kTileM + r;     // this row of the batch
      // the row's position, and the warp's first one (lengths and pre are at
      // most 2^30)
      const int pos = it.kv_len - it.q_len + i, pos_0 = pos - lane;
      // whole tiles for the warp (no key past its first row's last, none before
      // its last row's window) start in [full_lo, full_hi]
      const int full_hi = min(it.kv_len - 1, pos_0) - (kTileN - 1), full_lo = pos_0 + 31 - p.band_pre;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++c) {
        const int kv0 = (j < n_sink ? j : jt0 + j) * kTileN;
        if (!__all_sync(0xffffffffu, wait(&bar->s_full[t][c % ST], (c / ST) & 1, abort_flag, p.status.limit_ns))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool ragged = kv0 + kTileN > kv_len && j >= clear_from;
        const bool edge = kv0 > full_hi || kv0 < full_lo;
        // bit e: column k0 + e is hidden from the row
        auto hidden = [&](int k0) -> uint32_t {
          const int to = min(kv_len - 1, pos) - k0, from = pos - p.band_pre - k0, sinks = min(p.sink - k0, to + 1);
          const uint32_t past = to < 0 ? 0xffffffffu : to >= 31 ? 0u : 0xfffffffeu << to;
          const uint32_t before = from <= 0 ? 0u : from >= 32 ? 0xffffffffu : ~(0xffffffffu << from);
          const uint32_t sink = sinks <= 0 ? 0u : sinks >= 32 ? 0xffffffffu : ~(0xffffffffu << sinks);
          return past | (before & ~sink);
        };
        uint32_t su[4][32];
        tmem_ld32(col_s, su[0]);
        tmem_ld32(col_s + 32, su[1]);
        tmem_ld32(col_s + 64, su[2]);
        tmem_ld32(col_s + 96, su[3]);
        tmem_wait_ld(su[0]);
        tmem_regs_after_wait(su[1]);
        tmem_regs_after_wait(su[2]);
        tmem_regs_after_wait(su[3]);
        if (edge) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t hide = hidden(kv0 + 32 * q);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((hide >> e) & 1u) su[q][e] = __float_as_uint(-INFINITY);
          }
        }
        float* x = reinterpret_cast<float*>(&su[0][0]);
        float a[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) a[q] = fmax3(x[q], x[8 + q], x[16 + q]);
#pragma unroll
        for (int q = 0; q < 8; ++q) a[q] = fmax3(a[q], x[24 + q], x[32 + q]);
#pragma unroll
        for (int q = 0; q < 8; ++q) a[q] = fmax3(a[q], x[40 + q], x[48 + q]);
#pragma unroll
        for (int q = 0; q < 8; ++q) a[q] = fmaxf(a[q], x[56 + q]);
#pragma unroll
        for (int q = 0; q < 8; ++q) a[q] = fmax3(a[q], x[64 + q], x[72 + q]);
#pragma unroll
        for (int q = 0; q < 8; ++q) a[q] = fmax3(a[q], x[80 + q], x[88 + q]);
#pragma unroll
        for (int q = 0; q < 8; ++q) a[q] = fmax3(a[q], x[96 + q], x[104 + q]);
#pragma unroll
        for (int q = 0; q < 8; ++q) a[q] = fmax3(a[q], x[112 + q], x[120 + q]);
        const float m_tile = fmax3(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
        const float m_new = fmaxf(m, m_tile * sl2);
        // Keep a stale max unless it grows by more than 8 (log2 units): p <=
        // 2^8 stays exact in fp32 and representable in bf16 / f16.
        const float m_use = (m == -INFINITY || m_new > m + 8.f) ? m_new : m;
        const float alpha = (m_use == m) ? 1.f : fast_exp2(m - m_use);
        const float mo = (m_use == -INFINITY) ? 0.f : m_use;
        const uint64_t sc2 = f2_pack(sl2, sl2), nmo2 = f2_pack(-mo, -mo);
        uint64_t acc2[2] = {0ull, 0ull};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float y0, y1;
            f2_unpack(f2_fma(f2_pack(x[32 * q + 2 * e], x[32 * q + 2 * e + 1]), sc2, nmo2), y0, y1);
            y0 = fast_exp2(y0);
            y1 = fast_exp2(y1);
            acc2[e & 1] = f2_add(acc2[e & 1], f2_pack(y0, y1));
            u[e] = pack2(y0, y1, BF16);   // the weights' one rounding; their sum is not rounded
          }
          tmem_st16(col_s + q * 16, u);
        }
        float s0, s1;
        f2_unpack(f2_add(acc2[0], acc2[1]), s0, s1);
        l = l * alpha + (s0 + s1);
        // O_t holds the step before's P V: this S was issued after it
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) rescale_o(alpha);
        m = m_use;
        if (ragged) {
          // rows of V past the batch's keys may hold anything, and 0 * NaN is
          // NaN: cleared before the first P V that reads the tile
          const int step = base + j, s = step % ST;
          if (!__all_sync(0xffffffffu, wait(&bar->v_full[s], (step / ST) & 1, abort_flag, p.status.limit_ns))) {
            ok = false;
            break;
          }
          if (r >= kv_len - kv0) {
            uint8_t* vs = smem + C::kOffV + s * C::kTile;
#pragma unroll
            for (int ch = 0; ch < C::kChunks; ++ch)
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint4*>(vs + ch * C::kBox + r * 128 + q * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&bar->p_full[t][c & 1]);
      }
      if (!ok) tmem_wait_st();   // no store to TMEM is pending when it goes
      // ---------------------------------------------------------- output
      const int n_all = max(it.n_a, it.n_b);
      if (ok && n > 0) {
        if (t == 0) {
          ok = __all_sync(0xffffffffu, wait(&bar->a_done, items_a & 1, abort_flag, p.status.limit_ns));
          ++items_a;
        } else {
          const int step = base + n - 1;
          ok = __all_sync(0xffffffffu, wait(&bar->v_free[step % ST], (step / ST) & 1, abort_flag, p.status.limit_ns));
          warp_arrive(&bar->b_read);
        }
        tc_fence_after();
      }
      if (ok) {
        // (the padding rows of a padded layout are written here, as zeros)
        const bool row_valid = i < (is_tnd ? it.q_len : p.s1);
        const bool has = l != 0.f && i < it.q_len;   // a NaN sum stays a NaN
        const float inv_l = has ? 1.f / l : 0.f;
        using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
        const int64_t row = int64_t(it.q_row0) + t * kTileM + r, ob = is_tnd ? 0 : it.b;
        T* orow = reinterpret_cast<T*>(p.out) + ob * p.out_sb + row * p.out_ss + int64_t(it.h) * p.out_sn;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t u[32];
          if (n > 0) {
            tmem_ld32(col_o + q * 32, u);
            tmem_wait_ld(u);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = 0u;
          }
          if (row_valid) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint4 w;
              w.x = pack2(__uint_as_float(u[8 * e + 0]) * inv_l, __uint_as_float(u[8 * e + 1]) * inv_l, BF16);
              w.y = pack2(__uint_as_float(u[8 * e + 2]) * inv_l, __uint_as_float(u[8 * e + 3]) * inv_l, BF16);
              w.z = pack2(__uint_as_float(u[8 * e + 4]) * inv_l, __uint_as_float(u[8 * e + 5]) * inv_l, BF16);
              w.w = pack2(__uint_as_float(u[8 * e + 6]) * inv_l, __uint_as_float(u[8 * e + 7]) * inv_l, BF16);
              if (!has) w = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(orow + q * 32 + e * 8) = w;
            }
          }
        }
        if (row_valid && p.lse != nullptr)
          p.lse[ob * p.lse_sb + row * p.lse_ss + int64_t(it.h) * p.lse_sn] =
              has ? (m + __log2f(l)) * 0.69314718055994531f : INFINITY;
        tc_fence_before();
        warp_arrive(&bar->info_free[k % kInfos]);
      }
      base += n_all;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag != 0) status_raise(p.status, 10u /* FIA_ERR_TIMEOUT */);
}

template <int D, bool BF16>
cudaError_t launch_one(const PrefillParams& p, int n_sm, cudaStream_t s) {
  cudaError_t e = set_smem_once<prefill_window_kernel<D, BF16>>(WinCfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(prefill_window_kernel<D, BF16>, dim3(unsigned(std::min(p.n_items, n_sm))), WinCfg<D>::kThreads,
                      WinCfg<D>::kSmem, s, p);
}

}  // namespace

cudaError_t launch_prefill_window(const PrefillParams& p, int head_dim, bool bf16, int n_sm, cudaStream_t s) {
  if (p.n_items == 0) return cudaSuccess;
  if (head_dim == 128) return bf16 ? launch_one<128, true>(p, n_sm, s) : launch_one<128, false>(p, n_sm, s);
  return bf16 ? launch_one<64, true>(p, n_sm, s) : launch_one<64, false>(p, n_sm, s);
}

}  // namespace fia
