// Decode over the visible span of each sequence: a sliding window and sink
// tokens (fia_decode_window), or the keys behind a shared prefix joined with
// the prefix's partial results (fia_decode_shared_prefix).
//
//   token i of a sequence's Q_S new tokens sits at position p = L - Q_S + i and
//   sees key j when j <= p and (p - j <= pre or j < sink); j >= base only;
//   out = softmax(scale q K^T) V over the keys it sees, lse = log sum exp.
//
// Lengths are read on the device, so the grid depends on sizes alone and a
// captured call follows new lengths.  A unit is (batch, kv head), its rows the
// g heads x Q_S tokens: up to 32 here, more (and 17..32 with many keys) in
// span_wide.cu.  Its keys are the 16-key tiles of the sinks and of [first row's
// window, L): a list whose length the device knows.
//   * Work: a cluster of 1..16 CTAs runs a unit, each CTA four warps.  A warp
//     owns 16 rows (mma.sync m16n8k16); units of up to 16 rows give each warp
//     keys of its own (tile v of the list belongs to group v mod groups), those
//     of 17..32 pair the warps of a group over the same tiles, two a step.
//   * Data: a group streams its tiles through a ring of its own with cp.async
//     (16-byte pieces, XOR-swizzled so that ldmatrix has no bank conflicts): no
//     barrier across groups in the loop.  A tile lies in one page (16 divides
//     the page size); page ids come 32 at a time, one per lane, a batch ahead,
//     and become cache offsets there (one division per tile, not per piece).
//     Keys that no row sees are not read: they are zero-filled (a freed page
//     behind the window may hold anything, and 0 * NaN would reach the sums).
//   * Softmax: running maximum and sum per row and group in fp32, scores in
//     log2 units; P is rounded to the cache's type for the tensor cores (half
//     a step, relative, of each weight), its sum is not rounded.
//   * Join: the groups' (O, max, sum) meet in shared memory, the CTAs' over
//     distributed shared memory, with the exact weights 2^(m - max m): one
//     launch, no workspace, no atomics, the same bits on every run.  Each CTA
//     sends its results to the CTA that writes them (one barrier; reading them
//     there took a second one, so that no CTA left while it was read: 1.5 us).
// Bound: HBM where spans are long (64 sequences x 4 tokens, window 4096: 163 us,
// 95% of a copy's rate); where they are short the chain length -> page ids ->
// keys -> join and code fetched for one use (16 sequences, window 1024: 14.5 us,
// 59%; one sequence 6.2 us).
#include <algorithm>
#include <type_traits>

#include "span_join.cuh"

namespace fia {
namespace {

constexpr int kSpanThreads = 128;
constexpr int kSpanTile = 16;        // keys of a tile

template <int D, int MT>
struct SpanCfg {
  static constexpr int kGroups = 4 / MT;
  // CTAs per SM (registers and shared memory allow it)
  static constexpr int kResident = D == 64 ? 4 : 2;
  // A step takes kSub tiles: the warps of a wider group wait for one another
  // once a step, and their products and row maxima need the work to hide in.
  static constexpr int kSub = MT;
  static constexpr int kStages = MT == 1 ? 3 : 2;   // steps in a group's ring
  static constexpr int kTileBytes = kSpanTile * D * 2;    // K or V
  static constexpr int kStageBytes = 2 * kSub * kTileBytes;
  static constexpr int kRing = kGroups * kStages * kStageBytes;
  // after the loop the rings hold O of every group [kGroups][16 MT][D]
  static constexpr int kO = kGroups * 16 * MT * D * 4;
  static_assert(kO <= kRing, "the groups' results take the rings' place");
  // (max, sum) of every group; what the join receives
  static constexpr int kOffML = kRing;
  static constexpr int kOffIn = kOffML + kGroups * 16 * MT * 8;
  static constexpr int kSmem = kOffIn + JoinIn<D, 16 * MT>::kBytes + 128;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// d += A B, one m16n8k16 tile, fp32 accumulators
template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int D, bool BF16, int MT>
__global__ void __launch_bounds__(kSpanThreads, SpanCfg<D, MT>::kResident) span_decode_kernel(const __grid_constant__ SpanParams p) {
  using C = SpanCfg<D, MT>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int CH = D / 8;                       // 16-byte pieces of a row
  constexpr int KK = D / 16;                      // k-steps of Q K^T
  constexpr int NT = D / 8;                       // n-tiles of O
  constexpr int ST = C::kStages, SUB = C::kSub;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rt = warp % MT, kg = warp / MT;
  const int fg = lane >> 2, ft = lane & 3;
  // grid: (batch x CTA of the unit, kv head).  Divisions by run-time numbers are
  // kept out of the kernel's start and end, which run once from a cold
  // instruction cache: a division is twenty instructions, at ten cycles each.
  const uint32_t lg = uint32_t(p.lg_cs), cs = 1u << lg, rank = blockIdx.x & (cs - 1u);
  const int b = int(blockIdx.x >> lg), kvh = blockIdx.y;

  grid_dep_launch();
  if (lg != 0) cluster_arrive();   // (waited for before the join's first remote store: every CTA runs by then)
  // Behind a prefix kernel, which lets this one go once everything before both
  // is complete, only the join has to wait for it.
  if (p.n_parts == 0) grid_dep_wait();
  // Length, page ids and keys wait for one another: the length first, and
  // without a window, when they do not depend on it, the page ids; the queries
  // load meanwhile.
  int len = p.kv_max;
  if (p.kv_len != nullptr)
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(len) : "l"(p.kv_len + b) : "memory");
  const bool gapless = p.pre >= p.kv_max;      // no window: the tiles are t_base, t_base + 1, ...
  const int t_base = p.base / kSpanTile;
  const int groups = C::kGroups << lg;
  const int gi = int(rank) * C::kGroups + kg;
  const int32_t* table = p.block_table + int64_t(b) * p.table_stride;
  // where the tile of keys j.. starts in the caches, in elements; -1: nowhere
  auto tile_start = [&](int j) -> int64_t {
    if (p.block_table == nullptr) return int64_t(b) * p.blk_stride + int64_t(j) * p.row_stride;
    const int page = p.lg_block >= 0 ? j >> p.lg_block : j / p.block_size;
    if (page >= p.table_stride) return -1;
    const int id = (j < p.shared ? p.block_table : table)[page];
    if (id < 0 || id >= p.n_blocks) return -1;
    return int64_t(id) * p.blk_stride + int64_t(j - page * p.block_size) * p.row_stride;
  };
  // (one per lane: those of the group's first 32 tiles)
  int64_t starts = -1;
  if (gapless) starts = tile_start((t_base + (gi + lane / SUB * groups) * SUB + lane % SUB) * kSpanTile);

  // ---------------------------------------------------------------- Q
  // A fragments of the warp's 16 rows: lane (fg, ft) holds rows fg, fg + 8 at
  // columns 2 ft, 2 ft + 1 and 8 + 2 ft, 9 + 2 ft of every 16
  const int r0 = rt * 16 + fg, r1 = r0 + 8;
  const T* qp = static_cast<const T*>(p.q) + int64_t(b) * p.q_sb + 2 * ft;
  const int h0 = span_head(p, r0), h1 = span_head(p, r1), tk0 = r0 - h0 * p.q_tokens, tk1 = r1 - h1 * p.q_tokens;
  const T* q0 = qp + (kvh * p.group + h0) * p.q_sn + tk0 * p.q_ss;
  const T* q1 = qp + (kvh * p.group + h1) * p.q_sn + tk1 * p.q_ss;
  uint32_t qa[KK][4];
#pragma unroll
  for (int kk = 0; kk < KK; ++kk) {
    qa[kk][0] = r0 < p.rows ? *reinterpret_cast<const uint32_t*>(q0 + kk * 16) : 0u;
    qa[kk][1] = r1 < p.rows ? *reinterpret_cast<const uint32_t*>(q1 + kk * 16) : 0u;
    qa[kk][2] = r0 < p.rows ? *reinterpret_cast<const uint32_t*>(q0 + kk * 16 + 8) : 0u;
    qa[kk][3] = r1 < p.rows ? *reinterpret_cast<const uint32_t*>(q1 + kk * 16 + 8) : 0u;
  }
  const int L = min(max(len, 0), p.kv_max);
  const int first = L - p.q_tokens;               // position of token 0 (may be negative: tokens that see nothing)
  // the tiles that hold a key some row may see: the sinks' [base / 16, t_sink)
  // and [t_win, t_end)
  const int t_end = (L + kSpanTile - 1) / kSpanTile;
  const int t_sink = min(t_end, max(t_base, (p.sink + kSpanTile - 1) / kSpanTile));
  const int win = int(max(int64_t(first) - p.pre, int64_t(0)));   // first key of token 0's window
  const int t_win = max(t_sink, win / kSpanTile);
  const int n_sink = max(0, t_sink - t_base);
  const int n_tiles = n_sink + max(0, t_end - t_win);
  const int n_steps = (n_tiles + SUB - 1) / SUB;
  const int n = n_steps > gi ? (n_steps - gi + groups - 1) / groups : 0;   // this group's steps
  // First key of tile u of the group's i-th step; past the list it is L or more.
  auto tile_key = [&](int i, int u) -> int {
    const int v = (gi + i * groups) * SUB + u;
    if (gapless) return (t_base + v) * kSpanTile;
    return (v < n_sink ? t_base + v : t_win + v - n_sink) * kSpanTile;
  };

  // ---------------------------------------------------------------- loads
  // tile_start of the group's q-th tile (step q / SUB): 32 tiles at a time, one
  // per lane, a batch ahead
  auto start_of = [&](int q) -> int64_t { return tile_start(tile_key(q / SUB, q % SUB)); };
  if (!gapless) starts = start_of(lane);
  int64_t starts_next = -1;
  int batch = 0;
  const uint32_t ring = smem_u32(smem) + kg * ST * C::kStageBytes;
  // this lane's first piece of a tile, and the rows between its pieces
  constexpr int kIts = kSpanTile * CH / (32 * MT), kRowStep = 32 * MT / CH;
  const int row_l = (rt * 32 + lane) / CH, c_l = (rt * 32 + lane) % CH;
  const int64_t lane_off = int64_t(kvh) * p.head_stride + int64_t(row_l) * p.row_stride + c_l * 8;
  const T* kp = static_cast<const T*>(p.k) + lane_off;
  const T* vp = static_cast<const T*>(p.v) + lane_off;
  const int64_t it_off = int64_t(kRowStep) * p.row_stride;
  auto issue = [&](int i) {
    if ((i * SUB >> 5) != batch) {
      starts = starts_next;
      ++batch;
    }
    if ((i * SUB & 31) == 0 && i + 32 / SUB < n) starts_next = start_of(((batch + 1) << 5) + lane);
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      const int64_t at = __shfl_sync(0xffffffffu, starts, (i * SUB + u) & 31);
      if (i < n) {
        const int j0 = tile_key(i, u);
        const uint32_t st = ring + (i % ST) * C::kStageBytes + u * C::kTileBytes + row_l * (D * 2);
        // every key of the tile is one that some row sees
        const bool whole = at >= 0 && j0 + kSpanTile <= L && j0 >= p.base && (j0 + kSpanTile <= p.sink || j0 >= win);
        const T* ks = kp + (at >= 0 ? at : 0);
        const T* vs = vp + (at >= 0 ? at : 0);
#pragma unroll
        for (int it = 0; it < kIts; ++it) {
          const uint32_t dst = st + it * kRowStep * (D * 2) + ((c_l ^ ((row_l + it * kRowStep) & 7)) << 4);
          uint32_t bytes = 16u;
          if (!whole) {
            const int j = j0 + row_l + it * kRowStep;
            bytes = at >= 0 && j < L && j >= p.base && (j < p.sink || j >= win) ? 16u : 0u;
          }
          // (a piece of 0 bytes reads nothing; its address still names the cache)
          cp_async_zfill<16>(dst, bytes != 0u ? ks + it * it_off : static_cast<const T*>(p.k), bytes);
          cp_async_zfill<16>(dst + SUB * C::kTileBytes, bytes != 0u ? vs + it * it_off : static_cast<const T*>(p.v), bytes);
        }
      }
    }
    cp_async_commit();
  };
  auto group_sync = [&]() {
    if constexpr (MT == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + kg), "r"(32 * MT) : "memory");
  };
  for (int i = 0; i < ST - 1; ++i) issue(i);

  const int p0 = first + tk0, p1 = first + tk1;   // the rows' positions
  const int w0 = int(max(int64_t(p0) - p.pre, int64_t(0))), w1 = int(max(int64_t(p1) - p.pre, int64_t(0)));
  const int win_last = int(max(int64_t(L) - 1 - p.pre, int64_t(0)));   // the last token's window
  auto sees = [&](int pos, int w, int j) -> bool { return j <= pos && j >= p.base && (j < p.sink || j >= w); };

  // ---------------------------------------------------------------- the loop
  float o[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  const float sl2 = p.scale_log2;
  const int lr = lane & 7, lm = lane >> 3;
  for (int i = 0; i < n; ++i) {
    cp_async_wait_group<ST - 2>();
    group_sync();            // the tile is in for every warp of the group, and the slot before it has been read
    issue(i + ST - 1);
    const uint32_t ks = ring + (i % ST) * C::kStageBytes, vs = ks + SUB * C::kTileBytes;
    float s[2 * SUB][4];
#pragma unroll
    for (int h = 0; h < 2 * SUB; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[h][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        // matrices: keys 0-7 | 0-7 | 8-15 | 8-15, pieces 2 kk | 2 kk + 1 | ...
        uint32_t f[4];
        const int row = (lm >> 1) * 8 + lr, c = 2 * kk + (lm & 1);
        ldsm4(ks + u * C::kTileBytes + row * (D * 2) + ((c ^ lr) << 4), f);
        mma16<BF16>(s[2 * u], qa[kk], f[0], f[1]);
        mma16<BF16>(s[2 * u + 1], qa[kk], f[2], f[3]);
      }
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      const int j0 = tile_key(i, u);
      // every row sees every key of the tile
      const bool full = j0 + kSpanTile - 1 <= first && j0 >= p.base &&
                        (j0 + kSpanTile <= p.sink || j0 >= win_last);
      if (!full) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = j0 + 8 * h + 2 * ft + e;
            if (!sees(p0, w0, j)) s[2 * u + h][e] = -INFINITY;
            if (!sees(p1, w1, j)) s[2 * u + h][2 + e] = -INFINITY;
          }
      }
#pragma unroll
      for (int h = 2 * u; h < 2 * u + 2; ++h) {
        x0 = fmax3(x0, s[h][0], s[h][1]);
        x1 = fmax3(x1, s[h][2], s[h][3]);
      }
    }
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
    const float n0 = fmaxf(m0, x0 * sl2), n1 = fmaxf(m1, x1 * sl2);
    if (__any_sync(0xffffffffu, n0 != m0 || n1 != m1)) {
      const float a0 = m0 == n0 ? 1.f : fast_exp2(m0 - n0), a1 = m1 == n1 ? 1.f : fast_exp2(m1 - n1);
      l0 *= a0;
      l1 *= a1;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        o[t][0] *= a0;
        o[t][1] *= a0;
        o[t][2] *= a1;
        o[t][3] *= a1;
      }
      m0 = n0;
      m1 = n1;
    }
    const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      uint32_t pa[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* x = s[2 * u + h];
        const float y0 = fast_exp2(fmaf(x[0], sl2, -z0)), y1 = fast_exp2(fmaf(x[1], sl2, -z0));
        const float y2 = fast_exp2(fmaf(x[2], sl2, -z1)), y3 = fast_exp2(fmaf(x[3], sl2, -z1));
        l0 += y0 + y1;
        l1 += y2 + y3;
        pa[2 * h] = pack2(y0, y1, BF16);
        pa[2 * h + 1] = pack2(y2, y3, BF16);
      }
#pragma unroll
      for (int t = 0; t < NT; t += 2) {
        // matrices: keys 0-7 | 8-15 of piece t, then of piece t + 1
        uint32_t f[4];
        const int row = (lm & 1) * 8 + lr, c = t + (lm >> 1);
        ldsm4_trans(vs + u * C::kTileBytes + row * (D * 2) + ((c ^ lr) << 4), f);
        mma16<BF16>(o[t], pa, f[0], f[1]);
        mma16<BF16>(o[t + 1], pa, f[2], f[3]);
      }
    }
  }
  cp_async_wait_all();
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);

  // ---------------------------------------------------------------- join
  __syncthreads();           // every ring has been read
  float* ob = reinterpret_cast<float*>(smem);
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffML);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 8 + 2 * ft;
    *reinterpret_cast<float2*>(ob + join_at<D, 16 * MT>(kg, r0, c >> 2) + (c & 3)) = make_float2(o[t][0], o[t][1]);
    *reinterpret_cast<float2*>(ob + join_at<D, 16 * MT>(kg, r1, c >> 2) + (c & 3)) = make_float2(o[t][2], o[t][3]);
  }
  if (ft == 0) {
    ml[kg * 16 * MT + r0] = make_float2(m0, l0);
    ml[kg * 16 * MT + r1] = make_float2(m1, l1);
  }
  // (nothing here gives up; at the kernel's start, or as the compare-and-swap of
  // the kernels that can, this cost every call 0.2 us)
  if (p.n_parts == 0 && p.status.word != nullptr && (threadIdx.x | blockIdx.x | blockIdx.y) == 0)
    *p.status.word = p.status.epoch << 8;
  span_join<D, BF16, 16 * MT, C::kGroups, kSpanThreads>(p, ob, ml, smem + C::kOffIn, lg, rank, b, kvh);
}

template <int D, bool BF16, int MT>
cudaError_t launch_one(const SpanParams& p, cudaStream_t s) {
  using C = SpanCfg<D, MT>;
  cudaError_t e = prepare_span<span_decode_kernel<D, BF16, MT>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_span(span_decode_kernel<D, BF16, MT>, p, p, kSpanThreads, C::kSmem, s);
}

}  // namespace

// Start cost of a CTA in its groups' 16-key tiles.  (Sweep over 1, 2, 4, 8
// CTAs of a unit, us: 16 sequences x 8 heads, window of 65 tiles 24.0, 17.8, 25.6,
// 41.1; 64 x 8, 257 tiles 170, 193, 197, 273; 32 x 8, lengths up to 513 tiles
// 133, 113, 106, 128.  Where the keys' limit is the tables' and not the window's
// the lengths behind it vary.  Clusters of 16 where 8 were the most: one sequence
// x 8 heads of 32768 keys 61.7 -> 37.6, of a window of 4096 11.7 -> 9.1.)
constexpr int kSpanStart = 4;

cudaError_t launch_span_decode(const SpanParams& params, int head_dim, bool bf16, int n_sm, cudaStream_t s) {
  SpanParams p = params;
  if (p.rows > 32) return cudaErrorInvalidValue;
  const int mt = p.rows <= 16 ? 1 : 2;
  const int64_t span = std::min<int64_t>(p.kv_max - p.base, int64_t(p.sink) + p.pre + p.q_tokens);
  set_span_shape(p, cluster_ctas(int64_t(p.B) * p.N2, p.rows, span / kSpanTile + 1, 4 / mt, kSpanStart,
                                 span < p.kv_max - p.base, head_dim == 64 ? 4 : 2, n_sm));
#define FIA_SPAN(DD, BB) return mt == 1 ? launch_one<DD, BB, 1>(p, s) : launch_one<DD, BB, 2>(p, s)
  if (head_dim == 128) {
    if (bf16) FIA_SPAN(128, true);
    FIA_SPAN(128, false);
  }
  if (bf16) FIA_SPAN(64, true);
  FIA_SPAN(64, false);
#undef FIA_SPAN
}

}  // namespace fia
