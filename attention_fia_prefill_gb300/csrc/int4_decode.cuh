// Decode over a 4-bit paged cache (fia_decode_window_int4): the operator of
// span_decode.cu (window, sinks, lengths on the device), on codes.
//
//   S_j = scale sum_G [ step_jG (q_G . code_jG) + low_jG sum(q_G) ]   (K's groups G)
//   out_G = sum_j (w_j step_jG) code_jG + sum_j w_j low_jG            (V's), w = softmax over the keys seen
//
// so the products run on the codes themselves: 0..15 as fp16 numbers, whatever
// the type of queries, steps and outputs.  A nibble masked in place is a
// subnormal fp16: code 2^-24 in bits 0-3, code 2^-20 in bits 4-7 (products of
// subnormals are exact on the tensor cores, into fp32): one AND makes two values,
// with no conversion and nothing rounded.
//   * Q, scaled by a power of two per row to just below 2^11 in magnitude (q_exponent),
//     is fp16 (exact but for values below 2^-25 of the row's largest, off by 2^-36
//     of it); what multiplies bits 0-3 is 16 times that, so that both places
//     weigh the same.
//   * P' = 2^(S - m) step_j is fp16 (11 bits; a bf16 P would have 8): m is the
//     running maximum of S_j + log2(step_j), less 15, so P' is at most 2^15, and
//     exact to 11 bits down to 2^-29 of the largest.  (log2(step_j) counts as -30
//     at least: sums of 2^(S - m), and these times a low value, stay within fp32.)
//     What the rounding took, times 7.5, joins the low terms where the outputs are fp16
//     (p_rest): the error left is that of codes about their middle.
//   * The low terms and the sums are fp32, outside the products.
// The transposed products S^T = K Q^T and O^T = V^T P^T make the 16 wide side
// that of keys (or columns) and the 8 wide one that of the unit's rows: units of
// up to 8 rows (8 heads a kv head) do half the products that 16 rows would, and
// those of up to 4 take two tiles in one pass of the softmax (HALF, below: 64
// sequences of up to 32768 keys 299 -> 230 us, with CTAs of four warps).  K's
// fragments are words of the row as stored, V's come transposed by ldmatrix (one
// group a row) or from two rows' words by a byte permutation, and P reaches its
// fragment through movmatrix.
//   * Work: a unit (batch, kv head) has 16-key tiles, two a step; a warp has 8 NT
//     rows, and MT warps share a step's tiles.  Few keys: a cluster of 1..16 CTAs
//     runs a unit, as in span_decode.cu.  Many: even shares, whatever the lengths
//     (Share, below), and a second kernel that joins what they cut (64 sequences
//     of up to 32768 keys 230 -> 190 us).
//   * Data: a ring of each group's own (cp.async, three steps), row numbers 32
//     tiles at a time, one per lane.  A tile is read whole: codes are finite
//     whatever they hold, and the scales of keys that no row sees are set to 0 on
//     use.
//   * A step that every row sees whole runs without masks; the row maxima are
//     joined across lanes only in steps that raise one.
// 33 rows and more in one group a row: int4_wide.cu.
// Bound: HBM for units of up to 8 rows and long contexts (64 sequences of up to 32768
// keys, 8 heads: 189 us, 6.2 TB/s, 92% of a copy's rate); a warp's chain load -> product
// -> softmax -> product elsewhere: 16 rows a unit 87 us where HBM would take 43 (64 x 4
// tokens, window 4096; 349 instructions a tile at 1.9 a cycle with 8 warps an SM; 12
// warps of fewer registers take as long), 32 rows 153 where it would take 45 (32 sequences of
// up to 16384 keys; 562 instructions a tile at 1.8 a cycle), 16 sequences of up to 4096 keys 16.5 us, one of
// 20001 12.8 us (start 3, first keys 1.2, ten steps of 0.8, join 2).  Tried for the last:
// a ring of 8 steps 19.4 us (clusters of 16 CTAs then wait for 16 free SMs), of 5 steps
// 12.8, 8 warps a CTA 12.9.  Joining a unit's parts in the CTA that writes the last one
// instead of the second kernel: 190 and 190 us, 17.2 and 17.4 (the kernel's start hides
// behind the first).
#pragma once
#include <algorithm>
#include <cfloat>

#include "int4.cuh"
#include "span_join.cuh"

namespace fia {
namespace int4_detail {

constexpr int kTile = 16;

// NT: 8-row columns of a warp, 0: half of one (4 rows); MT: warps that share a
// group's tiles.
template <int D, int NG, int NT, int MT>
struct Cfg {
  static constexpr int kWarps = 4;
  // CTAs that registers allow an SM, and the clusters' plan counts.  With a cluster's part of shared memory three fit at head
  // dim 128 for 5 to 8 rows, and for fewer in groups of 32 and 64.  Of 224 calls (7 to 72 sequences of 8 heads, up to 512 or 2048
  // keys), in the mean and singly: three counted 0.98 (0.66 to 1.47: 16 sequences of up to 512 keys 10.1 -> 7.0 us, 60 10.5 ->
  // 15.5); the part laid in the rings, so that four fit, and no dearer cluster taken where three do 0.93 (0.68 to 1.28: 56
  // sequences of 512 keys, 8 rows, 9.1 -> 11.1, as they no longer spread three an SM).
  static constexpr int kResident = NT <= 1 ? 4 : 2;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kGroups = kWarps / MT;
  static constexpr int kRows = NT == 0 ? 4 : 8 * NT * MT;   // of a CTA
  static_assert(int4_shape(kRows, NG).resident <= kResident && int4_shape(kRows, NG).groups == kGroups, "host and device agree");
  static constexpr int kParts = NT == 0 ? 2 * kGroups : kGroups;   // results of a CTA, to be joined
  static constexpr int kRowBytes = D / 2;
  static constexpr int kCodes = kTile * kRowBytes;        // of a tile, K or V
  static constexpr int kScales = kTile * NG * 4;
  static constexpr int kTileBytes = 2 * (kCodes + kScales);
  static constexpr int kSub = MT < 2 ? 2 : MT;            // tiles of a step
  static constexpr int kStages = 3;
  static constexpr int kGroupRing = kStages * kSub * kTileBytes;
  static constexpr int kRing = kGroups * kGroupRing;
  static constexpr int kO = kParts * kRows * D * 4;      // after the loop, in the rings' place
  static constexpr int kOffML = kRing > kO ? kRing : kO;
  static constexpr int kOffIn = kOffML + kParts * kRows * 8;
  static constexpr int kOffQ = kOffIn + JoinIn<D, kRows>::kBytes;
  static constexpr int kQ = NT > 1 ? kRows * D * 2 : 0;
  static constexpr int kSmem = kOffQ + kQ + 128;
  // even shares: nothing comes from other CTAs
  static constexpr int kOffQShare = kOffIn, kSmemShare = kOffQShare + kQ + 128;
  static_assert(int4_shape(kRows, NG).resident * (kSmemShare + 128 + 1024) <= 228 * 1024, "as many CTAs of shares as an SM is counted for");
};

// Row of a fragment's index -> key of the tile: a lane pair's keys 2t and 2t + 1
// are t and 7 - t, so that neither K's reads (by rows) nor V's (by pairs) of
// shared memory meet in a bank.
__device__ __forceinline__ int key_of(int x) { return (x & 8) | ((x & 1) ? 7 - ((x & 7) >> 1) : (x & 7) >> 1); }

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
               "{%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
               "{%8, %9}, {%10, %10, %10, %10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t trans8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// sum + 7.5 (P' - P' as fp16): P' code = P' (code - 7.5) + 7.5 P', so with the second term
// whole, a rounding of 2^-12 of P' (about) weighs |code - 7.5| and not code: 2.3 to 2.8
// times less.  16 keys of equal weights, normal values, groups of 32: fp16 outputs off by
// 5.0e-4 -> 2.9e-4 in norm, of which their own rounding is 2.1e-4 (32 sequences, head dim
// 64: 21.0 -> 21.7 us).  bf16 outputs, off by 1.7e-3 by theirs, do without.
__device__ __forceinline__ uint64_t p_rest(uint64_t p, uint32_t rounded, uint64_t sum) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&rounded));
  return f2_fma(f2_fma(f2_pack(h.x, h.y), f2_pack(-1.f, -1.f), p), f2_pack(7.5f, 7.5f), sum);
}
// e with 2^10 <= top 2^-e < 2^11 for a query row of magnitude top, and so large that
// 2^e scale is a normal number: times a hidden score, which is -inf, a factor of 0 would be a
// NaN.  (A row that this scales below 2^10, one of zeros for one, loses digits at 2^-25 times
// 2^e, which scores do not see: 2^e scale is 2^-120 then.)
__device__ __forceinline__ int q_exponent(float top, float scale) {
  return max(max(int(__float_as_uint(top) >> 23) - 137, 7 - int(__float_as_uint(scale) >> 23)), -125);
}
__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int N>
__device__ __forceinline__ void wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t* r) {
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else if constexpr (BYTES == 8)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r[0]) : "r"(addr) : "memory");
}

// What the new tokens of a sequence of L keys see: the tiles of the sinks and
// those of [first key of token 0's window, L).
struct Span {
  int first, t_sink, win, t_win, n_tiles;      // first: position of token 0 (may be negative)
  __device__ __forceinline__ Span(const SpanParams& p, int L) {
    first = L - p.q_tokens;
    const int t_end = (L + kTile - 1) / kTile;
    t_sink = min(t_end, (p.sink + kTile - 1) / kTile);
    win = int(max(int64_t(first) - p.pre, int64_t(0)));
    t_win = max(t_sink, win / kTile);
    n_tiles = t_sink + max(0, t_end - t_win);
  }
};

// Work shared evenly among the CTAs, whatever the lengths are.  A unit's tiles
// come in chunks (a step of every group of a CTA); it has one at least, and
// `begin` more for its start.  For every head the sequences lie in order, W chunks in
// all, and share g of G has [g W / G, (g + 1) W / G): the end of one unit, whole
// ones, the start of another.  CTA (head, g), heads first: those of a share read the
// same tokens at one time, which in a (blocks, slots, heads) cache lie side by side
// (64 sequences of up to 16384 keys 188 -> 130 us).
struct Piece {
  int b, c0, c1;               // chunks [c0, c1) of the head's unit; c1 = 0: none
  int parts;                   // shares from this one on that have parts of the unit; 0: it began before
  int len;                     // of the sequence
};
__device__ __forceinline__ int share_cta() { return int(blockIdx.y * gridDim.x + blockIdx.x); }

struct Share {
  Piece piece[2];
  int64_t work, at, end;       // W; position; end of the share
  int b, cost, pos, len;       // the unit there, its chunks and `begin`, position in it
  int shares;                  // G

  static __device__ __forceinline__ int unit_cost(const SpanParams& p, int len, int chunk, int begin) {
    const int L = min(max(len, 0), p.kv_max);
    return max(1, (Span(p, L).n_tiles + chunk - 1) / chunk) + begin;
  }
  // a b / c: all but huge batches fit 32 bits, where a division is a fifth of the instructions
  static __device__ __forceinline__ int64_t mul_div(int64_t a, int b, int64_t c, bool small) {
    return small ? int64_t(uint32_t(a) * uint32_t(b) / uint32_t(c)) : a * b / c;
  }
  // One warp.  Clears the CTA's entry of heads.
  __device__ __forceinline__ void start(const SpanParams& p, int4* heads, int chunk, int begin, int lane) {
    int n = lane < p.B ? p.kv_len[lane] : 0, c = lane < p.B ? unit_cost(p, n, chunk, begin) : 0;
    int64_t w = c;
    for (int k = lane + 32; k < p.B; k += 32) w += unit_cost(p, p.kv_len[k], chunk, begin);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
    const int g = int(min(int64_t(gridDim.y), w));
    const bool small = w < 0xffffffffll / (int(gridDim.y) + 1);
    const int64_t from = mul_div(w, blockIdx.y, g, small);
    if (lane == 0) {
      heads[share_cta()] = make_int4(0, 0, 0, 0);
      piece[0].c1 = 0;
      work = w;
      shares = g;
      at = from;
      end = mul_div(w, blockIdx.y + 1, g, small);
    }
    __syncwarp();              // another lane may go on from these in next(); shuffles and votes do not order memory
    if (int(blockIdx.y) >= g) return;
    int64_t before = 0;        // of the sequences before
    for (int b0 = 0;;) {
      int64_t sum = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + sum > from);
      if (past != 0) {
        if (lane == __ffs(past) - 1) {
          b = b0 + lane;
          len = n;
          cost = c;
          pos = int(from - (before + sum - c));
          next(p, chunk, begin, 0);
        }
        return;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
      b0 += 32;
      if (b0 >= p.B) return;   // (never: from < W)
      n = b0 + lane < p.B ? p.kv_len[b0 + lane] : 0;
      c = b0 + lane < p.B ? unit_cost(p, n, chunk, begin) : 0;
    }
  }
  // The next piece of the share.  One thread.
  __device__ __forceinline__ void next(const SpanParams& p, int chunk, int begin, int turn) {
    Piece x = {0, 0, 0, 0, 0};
    while (x.c1 == 0 && at < end) {
      if (pos == cost) {
        pos = 0;
        len = p.kv_len[++b];
        cost = unit_cost(p, len, chunk, begin);
      }
      const int take = int(min(end - at, int64_t(cost - pos)));
      x = {b, max(0, pos - begin), max(0, pos + take - begin), 0, len};
      if (x.c1 > 0 && x.c0 == 0) {
        // share of position y: the last g with g W / G <= y
        const int64_t y = at - pos + cost - 1;
        x.parts = 1;
        if (y >= end) {
          const int64_t num = (y + 1) * shares - 1;
          x.parts = (num <= 0xffffffffll && work <= 0xffffffffll ? int(uint32_t(num) / uint32_t(work)) : int(num / work)) - int(blockIdx.y) + 1;
        }
      }
      at += take;
      pos += take;
    }
    piece[turn] = x;
  }
};

static_assert(sizeof(Share) <= 128, "counted with a CTA's shared memory");

// A part of a unit's result, not divided by its sums: the results of the CTA's
// groups joined (as in span_join) and written.  All threads.
template <int D, int ROWS, int GROUPS, int THREADS>
__device__ __forceinline__ void write_part(const SpanParams& p, const float* ob, const float2* ml, float* part_o, float2* part_ml) {
  __syncthreads();
  for (int e = threadIdx.x; e < p.rows * (D / 4); e += THREADS) {
    const int r = e / (D / 4), c4 = e % (D / 4);
    float top = -INFINITY, l = 0.f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) top = fmaxf(top, ml[g * ROWS + r].x);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const float2 w2 = ml[g * ROWS + r];
      const float w = join_weight(w2.x, top);
      const float4 x = *reinterpret_cast<const float4*>(ob + join_at<D, ROWS>(g, r, c4));
      l += w * w2.y;
      a.x += w * x.x; a.y += w * x.y; a.z += w * x.z; a.w += w * x.w;
    }
    reinterpret_cast<float4*>(part_o)[e] = a;
    if (c4 == 0) part_ml[r] = make_float2(top, l);
  }
}

// span_join (span_join.cuh) for a unit of its own: without a prefix's parts, and
// with the short calls in mind, of which it is a third: every row's (max, sum) goes to
// the peers by as many lanes, and the reads of their results overlap.
template <int D, bool BF16, int ROWS, int GROUPS, int THREADS>
__device__ __forceinline__ void join_unit(const SpanParams& p, const float* ob, const float2* ml, void* in, uint32_t lg,
                                          uint32_t rank, int b, int kvh) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int kInML = JoinIn<D, ROWS>::kO;
  const uint32_t in_o = smem_u32(in), in_ml = in_o + kInML;
  const uint32_t cs = 1u << lg;
  const int items = p.rows * (D / 4);   // float4s of the unit
  const int share = ((items + 8 * int(cs) - 1) >> (3 + lg)) << 3;
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
  auto write = [&](int r, int c4, float4 a, float l, float top) {
    const int h = span_head(p, r), head = kvh * p.group + h, tokn = r - h * p.q_tokens;
    const bool has = l != 0.f;   // a NaN sum stays a NaN
    const float inv = has ? 1.f / l : 0.f;
    uint2 u;
    u.x = has ? int4_out<BF16>(a.x * inv, a.y * inv) : 0u;
    u.y = has ? int4_out<BF16>(a.z * inv, a.w * inv) : 0u;
    T* orow = static_cast<T*>(p.out) + int64_t(b) * p.q_sb + int64_t(head) * p.q_sn + int64_t(tokn) * p.q_ss;
    *reinterpret_cast<uint2*>(orow + c4 * 4) = u;
    if (p.lse != nullptr && c4 == 0)
      p.lse[int64_t(b) * p.lse_sb + int64_t(head) * p.lse_sn + int64_t(tokn) * p.lse_ss] =
          has ? (top + __log2f(l)) * 0.69314718055994531f : INFINITY;
  };
  __syncthreads();
  if (lg == 0) {
    for (int e = threadIdx.x; e < items; e += THREADS) {
      float4 a;
      float l, top;
      own(e / (D / 4), e % (D / 4), a, l, top);
      write(e / (D / 4), e % (D / 4), a, l, top);
    }
    return;
  }
  // each float4 goes to the CTA that writes it: the CTAs take eight in turn
  cluster_wait();
  for (int e = threadIdx.x; e < items; e += THREADS) {
    const int r = e / (D / 4), c4 = e % (D / 4);
    float4 a;
    float l, top;
    own(r, c4, a, l, top);
    const int owner = (e >> 3) & int(cs - 1u), slot = ((e >> (3 + lg)) << 3) + (e & 7);
    st_peer4(peer_addr(in_o + (rank * share + slot) * 16, owner), a);
    if (c4 < int(cs)) st_peer2(peer_addr(in_ml + (rank * ROWS + r) * 8, c4), make_float2(top, l));
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();              // no CTA reads or writes another's memory from here on
  const float4* xo = static_cast<const float4*>(in);
  const float2* xml = reinterpret_cast<const float2*>(static_cast<const uint8_t*>(in) + kInML);
  for (int i = threadIdx.x; i < share; i += THREADS) {
    const int e = ((((i >> 3) << lg) + int(rank)) << 3) + (i & 7);
    if (e >= items) break;
    const int r = e / (D / 4);
    float top = -INFINITY, l = 0.f;
#pragma unroll 4
    for (uint32_t g = 0; g < cs; ++g) top = fmaxf(top, xml[g * ROWS + r].x);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (uint32_t g = 0; g < cs; ++g) {
      const float2 w2 = xml[g * ROWS + r];
      const float w = join_weight(w2.x, top);
      const float4 x = xo[g * share + i];
      l += w * w2.y;
      a.x += w * x.x; a.y += w * x.y; a.z += w * x.z; a.w += w * x.w;
    }
    write(r, e % (D / 4), a, l, top);
  }
}

template <int D, int NG, int NTT, int MT, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(Cfg<D, NG, NTT, MT>::kThreads, Cfg<D, NG, NTT, MT>::kResident)
int4_decode_kernel(const __grid_constant__ Int4SpanParams ip) {
  using C = Cfg<D, NG, NTT, MT>;
  // HALF: units of up to 4 rows fill half of a product's 8 columns.  The scores of
  // a second tile move to the lanes of the other half, and P of the two tiles lies
  // side by side: one pass of the softmax serves both, and columns 4-7 of O^T are
  // the second tile's part of rows 0-3.
  constexpr bool HALF = NTT == 0;
  constexpr int NT = HALF ? 1 : NTT;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int U = D / 32;        // columns j, 32 apart: two products of depth 16 (K), two of 16 columns (V)
  constexpr int PER = U / NG;      // of a group
  constexpr bool PAIR = PER >= 2;  // columns j and j + 1 are of one group
  constexpr int SUB = C::kSub, ST = C::kStages;
  constexpr int SETS = HALF ? SUB / 2 : SUB;   // passes of the softmax
  constexpr int RB = C::kRowBytes;
  constexpr uint32_t kNowhere = 0xffffffffu;
  const SpanParams& p = ip.s;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rt = warp % MT, kg = warp / MT;
  const int fg = lane >> 2, ft = lane & 3;
  const int fr = HALF ? ft & 1 : ft, half = HALF ? ft >> 1 : 0;   // this lane's rows are 2 fr, 2 fr + 1 of every 8
  const uint32_t lg = SPLIT ? 0u : uint32_t(p.lg_cs), cs = 1u << lg, rank = SPLIT ? 0u : blockIdx.x & (cs - 1u);
  // clusters: (CTA of the unit, head; sequence), so that heads run side by side as in the shares below
  const int kvh = SPLIT ? blockIdx.x : int(blockIdx.x >> lg);
  int b = SPLIT ? 0 : int(blockIdx.y + blockIdx.z * gridDim.y);
  if (!SPLIT && b >= p.B) return;   // (a whole cluster)

  grid_dep_launch();
  if (lg != 0) cluster_arrive();
  grid_dep_wait();
  const bool gapless = p.pre >= p.kv_max;      // no window: the tiles are 0, 1, ...
  constexpr int kChunk = C::kGroups * SUB;
  const int kBegin = ip.begin;
  // SPLIT: the CTA's share, piece by piece, kept in shared memory
  __shared__ Share share;
  if constexpr (SPLIT) {
    if (warp == 0) share.start(p, ip.heads, kChunk, kBegin, lane);
    __syncthreads();
  }
  int turn = 0;
#pragma unroll 1
  do {
  int c0 = 0, c1 = 0;                          // the chunks to do of the unit
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
  // the tiles of this group's step i: SUB from first_tile + i * stride on
  const int stride = (C::kGroups << lg) * SUB;
  const int first_tile = SPLIT ? (c0 * C::kGroups + kg) * SUB : (int(rank) * C::kGroups + kg) * SUB;
  const int32_t* table = p.block_table + int64_t(b) * p.table_stride;
  const bool heads_first = p.head_stride != RB;          // (blocks, heads, slots): rows of codes lie as their scales
  // Row numbers, from the pools' starts, of the first key of the tile of keys j..: codes' and scales'
  auto tile_rows = [&](int j, uint32_t& code, uint32_t& scale) {
    const int page = p.lg_block >= 0 ? j >> p.lg_block : j / p.block_size;
    const uint32_t off = uint32_t(j - page * p.block_size);
    code = scale = kNowhere;
    if (page < p.table_stride) {
      const int id = table[page];
      if (id >= 0 && id < p.n_blocks) {
        scale = (uint32_t(id) * uint32_t(p.N2) + uint32_t(kvh)) * uint32_t(p.block_size) + off;
        code = heads_first ? scale : (uint32_t(id) * uint32_t(p.block_size) + off) * uint32_t(p.N2) + uint32_t(kvh);
      }
    }
  };
  uint32_t at_code = kNowhere, at_scale = kNowhere;   // one per lane: those of the group's first 32 tiles
  if (gapless) tile_rows((first_tile + lane / SUB * stride + lane % SUB) * kTile, at_code, at_scale);

  // ---------------------------------------------------------------- Q
  // B fragments (row fg of every 8).  Lane ft holds columns 32 j + 8 ft .. + 7;
  // fragment (x, i) of them is what meets nibble i of the K words' halves (below):
  // columns 8 ft + 4 x / PERX + i of two j, or i and i + 4 of one.  i = 0, 2 meet bits 0-3.
  // (two columns of rows: in shared memory, for registers' sake)
  constexpr bool QS = NT > 1;
  uint32_t qb[QS ? 1 : NT][U][4];
  const uint32_t q_at = smem_u32(smem + (SPLIT ? C::kOffQShare : C::kOffQ)) + (rt * NT * U * 32 + lane) * 16;
  // of this lane's rows, as pairs: sums over a group's columns, and the factor to log2
  // units.  (The products come in units of 2^-20: f16 has both in these.  A bf16 row's
  // factor may be so large that fp32 does not hold 2^20 of it, so K's steps get them.)
  uint64_t qs[NT][NG], cr[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = rt * 8 * NT + nt * 8 + fg;
    const int h = span_head(p, r), tk = r - h * p.q_tokens;
    const T* q = static_cast<const T*>(p.q) + int64_t(b) * p.q_sb + int64_t(kvh * p.group + h) * p.q_sn + int64_t(tk) * p.q_ss + 8 * ft;
    uint32_t x[U][4];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r < p.rows) v = *reinterpret_cast<const uint4*>(q + 32 * j);
      x[j][0] = v.x; x[j][1] = v.y; x[j][2] = v.z; x[j][3] = v.w;
    }
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = int4_pair<BF16>(x[j][e]);
        top = fmax3(top, fabsf(f.x), fabsf(f.y));
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = q_exponent(top, p.scale_log2);
    const float up = __uint_as_float(uint32_t(127 + e) << 23), down = __uint_as_float(uint32_t(127 - e) << 23);
    float sum[NG], c[U][8];
#pragma unroll
    for (int k = 0; k < NG; ++k) sum[k] = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = int4_pair<BF16>(x[j][i]);
        c[j][2 * i] = f.x * down;
        c[j][2 * i + 1] = f.y * down;
      }
#pragma unroll
    for (int w = 0; w < U; ++w) {
      uint32_t (&x)[4] = qb[QS ? 0 : nt][w];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float m = i & 1 ? 1.f : 16.f;
        const float lo = PAIR ? c[w / 2 * 2][4 * (w & 1) + i] : c[w][i], hi = PAIR ? c[w / 2 * 2 + 1][4 * (w & 1) + i] : c[w][i + 4];
        x[i] = half2_bits(lo * m, hi * m);
        sum[w / PER] += lo + hi;
      }
      if (QS && kg == 0)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(q_at + (nt * U + w) * 512), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
    }
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
      sum[k] = (sum[k] + __shfl_xor_sync(0xffffffffu, sum[k], 2)) * (BF16 ? 1.f : 0x1p-20f);
      const float s0 = __shfl_sync(0xffffffffu, sum[k], 8 * fr), s1 = __shfl_sync(0xffffffffu, sum[k], 8 * fr + 4);
      qs[nt][k] = f2_pack(s0, s1);
    }
    const float f = fminf((BF16 ? up : up * 0x1p20f) * p.scale_log2, FLT_MAX);
    const float f0 = __shfl_sync(0xffffffffu, f, 8 * fr), f1 = __shfl_sync(0xffffffffu, f, 8 * fr + 4);
    cr[nt] = f2_pack(f0, f1);
  }

  const int L = min(max(len, 0), p.kv_max);
  const Span sp_(p, L);
  const int first = sp_.first, t_sink = sp_.t_sink, t_win = sp_.t_win, win = sp_.win;
  const int win_last = int(max(int64_t(L) - 1 - p.pre, int64_t(0)));   // first key of the last token's window
  const int left = sp_.n_tiles - first_tile;
  const int n = SPLIT ? c1 - c0 : left > 0 ? (left + stride - 1) / stride : 0;   // this group's steps
  // First key of tile u of the group's i-th step; past the list it is L or more.
  auto tile_key = [&](int i, int u) -> int {
    const int v = first_tile + i * stride + u;
    if (gapless) return v * kTile;
    return (v < t_sink ? v : t_win + v - t_sink) * kTile;
  };
  // Tiles of the list that every row sees whole: [0, f_sink) and [f_lo, f_hi) (and some of the others)
  const int f_sink = min((first + 1) >> 4, win_last == 0 ? t_sink : p.sink >> 4);
  const int f_lo = t_sink + max(0, (win_last + kTile - 1) / kTile - t_win), f_hi = t_sink + ((first + 1) >> 4) - t_win;

  // ---------------------------------------------------------------- loads
  // (past the list the page may be anything)
  auto batch_rows = [&](int q, bool look) {
    const int j = tile_key(q / SUB, q % SUB);
    if (look) tile_rows(j, at_code, at_scale);
    if (j >= L) at_code = at_scale = kNowhere;
  };
  batch_rows(lane, !gapless);
  const uint32_t ring = smem_u32(smem) + kg * C::kGroupRing;
  constexpr int CH = RB / 16;                     // 16-byte pieces of a row
  constexpr int kIts = kTile * CH / 32;
  const int row_l = lane / CH, c_l = lane % CH;
  // (pieces trade places by row, so that neither eight rows of one piece nor four of two pieces meet in a bank)
  auto piece = [&](int row, int c) -> uint32_t {
    return uint32_t(row * RB + ((D == 128 ? c ^ (row & 2) ^ (row >> 2 & 1) : c ^ (row >> 2 & 1)) << 4));
  };
  const uint32_t row_stride = uint32_t(p.row_stride);   // (at most 65535 heads)
  const uint8_t* kp = ip.kc + uint32_t(row_l) * row_stride + c_l * 16;
  const uint8_t* vp = ip.vc + uint32_t(row_l) * row_stride + c_l * 16;
  // Scales: 8 NG pieces a tile, K's and V's; a lane's is of tile lane / (8 NG) of those loaded at once
  constexpr int kPer = MT == 1 ? (4 / NG < SUB ? 4 / NG : SUB) : 1;
  const int s_u = lane / (8 * NG), s_c = lane % (8 * NG);
  const uint8_t* sp = (s_c >= 4 * NG ? ip.vs - 64 * NG : ip.ks) + s_c * 16;
  const uint32_t to_code = piece(row_l, c_l), to_scale = s_u * C::kTileBytes + 2 * C::kCodes + s_c * 16;
  constexpr uint32_t kStep = SUB * C::kTileBytes, kEnd = ST * kStep;
  auto issue = [&](int i, uint32_t slot) {
    if (i < n) {
      if (i > 0 && (i * SUB & 31) == 0) batch_rows(i * SUB + lane, true);
#pragma unroll
      for (int u0 = 0; u0 < SUB; u0 += MT) {
        const int u = u0 + rt;
        const uint32_t code = __shfl_sync(0xffffffffu, at_code, (i * SUB + u) & 31);
        const uint32_t st = ring + slot + u * C::kTileBytes;
        // (a page outside the pool, or no tile: zeros)
        const uint32_t bytes = code != kNowhere ? 16u : 0u;
        const uint64_t at = uint64_t(code != kNowhere ? code : 0u) * RB;
#pragma unroll
        for (int it = 0; it < kIts; ++it) {
          cp_async_zfill<16>(st + to_code + it * (32 / CH) * RB, kp + at + it * (32 / CH) * row_stride, bytes);
          cp_async_zfill<16>(st + C::kCodes + to_code + it * (32 / CH) * RB, vp + at + it * (32 / CH) * row_stride, bytes);
        }
        if (u0 % (kPer * MT) == 0) {
          const uint32_t scale = __shfl_sync(0xffffffffu, at_scale, (i * SUB + u + s_u) & 31);
          if (s_u < kPer)
            cp_async_zfill<16>(st + to_scale, sp + uint64_t(scale != kNowhere ? scale : 0u) * (NG * 4), scale != kNowhere ? 16u : 0u);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) issue(i, i * kStep);
  if (SPLIT && threadIdx.x == 0) share.next(p, kChunk, kBegin, turn ^ 1);   // (read behind the barriers of this piece's end)
  if (QS) __syncthreads();

  // ---------------------------------------------------------------- the loop
  float o[NT][U][2][4];
  // of the lane's two rows: maxima and (as pairs) these negated (0 for -inf), sums of
  // weights and of weights times low values
  float m[NT][2];
  uint64_t nz[NT], l[NT], zs[NT][NG];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][j][h][e] = 0.f;
    m[nt][0] = m[nt][1] = -INFINITY;
    nz[nt] = l[nt] = 0u;
#pragma unroll
    for (int k = 0; k < NG; ++k) zs[nt][k] = 0u;
  }
  const int k0 = key_of(fg);                                 // this lane's keys of S^T are k0 and 8 + k0
  const uint32_t k_at = D == 128 ? piece(k0, ft) : piece(k0, ft >> 1) + (ft & 1) * 8;
  // V: the row of lane & 15 for ldmatrix, else rows of keys ft and 7 - ft
  const uint32_t v_at = NG == 1 ? piece((lane & 8) + key_of(lane & 7), lane >> 4)
                                : (D == 128 ? piece(ft, fg >> 1) + (fg & 1) * 8 : piece(ft, fg >> 2) + (fg & 3) * 4);
  [[maybe_unused]] const uint32_t v_at2 = D == 128 ? piece(7 - ft, fg >> 1) + (fg & 1) * 8 : piece(7 - ft, fg >> 2) + (fg & 3) * 4;
  const uint32_t s_at = half * C::kTileBytes + 2 * C::kCodes + k0 * (NG * 4);
  // Step i, in the ring from `step` on.  FULL: every row sees every key.
  auto run = [&](auto full, int i, uint32_t step) {
    constexpr bool FULL = decltype(full)::value;
    // ---- K Q^T of the step's tiles, group by group
    float acc[SUB][NT][NG][4];
    uint32_t w0[SUB][U], w1[SUB][U];
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      lds<RB / 4>(step + u * C::kTileBytes + k_at, w0[u]);
      lds<RB / 4>(step + u * C::kTileBytes + k_at + 8 * RB, w1[u]);
    }
#pragma unroll
    for (int w = 0; w < U; ++w) {
      uint32_t qf[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (QS) {
          lds<16>(q_at + (nt * U + w) * 512, qf[nt]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) qf[nt][e] = qb[nt][w][e];
        }
      }
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        // A word is units (g, j) and (g, j + 1), g = 2 ft and 2 ft + 1: taken as it is, or its
        // halves exchanged so that a fragment is of one j
        const uint32_t sel = w & 1 ? 0x7632u : 0x5410u;
        const uint32_t a = PAIR ? w0[u][(w & 1) * (U / 2) + w / 2] : __byte_perm(w0[u][w / 2], w0[u][U / 2 + w / 2], sel);
        const uint32_t c = PAIR ? w1[u][(w & 1) * (U / 2) + w / 2] : __byte_perm(w1[u][w / 2], w1[u][U / 2 + w / 2], sel);
        const uint32_t a8 = a >> 8, c8 = c >> 8;
        const uint32_t f0[4] = {a & 0x000f000fu, c & 0x000f000fu, a & 0x00f000f0u, c & 0x00f000f0u};
        const uint32_t f1[4] = {a8 & 0x000f000fu, c8 & 0x000f000fu, a8 & 0x00f000f0u, c8 & 0x00f000f0u};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float (&x)[4] = acc[u][nt][w / PER];
          if (w % PER == 0) mma_f16_first(x, f0, qf[nt][0], qf[nt][1]);
          else mma_f16(x, f0, qf[nt][0], qf[nt][1]);
          mma_f16(x, f1, qf[nt][2], qf[nt][3]);
        }
      }
    }
    // V's A halves of words: one unit of two keys (2 ft and 2 ft + 1 of the fragment); keys 0-7, 8-15
    uint32_t va[SUB][U][2];
    auto load_v = [&](int u) {
      const uint32_t st = step + u * C::kTileBytes + C::kCodes;
      if constexpr (NG == 1) {
        // eight units of 16 keys to a matrix pair: lane fg has unit 8 c + fg
#pragma unroll
        for (int c = 0; c < U; c += 2) {
          uint32_t f[4];
          // (piece c is piece 0's place with c's bits changed)
          ldsm4_trans(st + (v_at ^ uint32_t(c << 4)), f);
          va[u][c][0] = f[0]; va[u][c][1] = f[1];
          va[u][c + 1][0] = f[2]; va[u][c + 1][1] = f[3];
        }
      } else {
        // units U fg ..: of keys ft, 7 - ft, 8 + ft, 15 - ft
        uint32_t v[4][U / 2];
        lds<RB / 8>(st + v_at, v[0]);
        lds<RB / 8>(st + v_at2, v[1]);
        lds<RB / 8>(st + v_at + 8 * RB, v[2]);
        lds<RB / 8>(st + v_at2 + 8 * RB, v[3]);
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
          va[u][j][0] = __byte_perm(v[0][j / 2], v[1][j / 2], sel);
          va[u][j][1] = __byte_perm(v[2][j / 2], v[3][j / 2], sel);
        }
      }
    };
    // (ahead of the softmax: 64 sequences 189 -> 187 us, 16 rows 88 -> 87; where it does not pay, 20.9 -> 21.8)
    constexpr bool EARLY = NG == 1 || NT > 1;
    if constexpr (EARLY) {
#pragma unroll
      for (int u = 0; u < SUB; ++u) load_v(u);
    }
    // ---- scores of the lane's rows and keys k0, 8 + k0 of its tiles (times cr: in log2 units)
    uint32_t kw[2][NG], vw[SETS][2][NG];   // (step, low) of K and V
    uint64_t s[SETS][NT][2];               // [key]: of the two rows
#pragma unroll
    for (int v = 0; v < SETS; ++v) {
      const uint32_t sc = step + (HALF ? 2 * v : v) * C::kTileBytes + s_at;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        lds<NG * 4>(sc + q * (8 * NG * 4), kw[q]);
        lds<NG * 4>(sc + C::kScales + q * (8 * NG * 4), vw[v][q]);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          const float2 g = int4_pair<BF16>(kw[q][k]);
          // (by the exponent: a step of 0, of a page outside the pool, meets codes of 0)
          const float step = BF16 ? __uint_as_float((kw[q][k] << 16) + (20u << 23)) : g.x;
          const uint64_t step2 = f2_pack(step, step), low2 = f2_pack(g.y, g.y);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if constexpr (HALF) {
                const float other = __shfl_sync(0xffffffffu, acc[2 * v + 1][nt][k][2 * q + e], lane & ~2);
                y[e] = half ? other : acc[2 * v][nt][k][2 * q + e];
              } else {
                y[e] = acc[v][nt][k][2 * q + e];
              }
            }
            s[v][nt][q] = f2_fma(f2_pack(y[0], y[1]), step2, k == 0 ? f2_mul(low2, qs[nt][k]) : f2_fma(low2, qs[nt][k], s[v][nt][q]));
          }
        }
    }
    // ---- masks, the running maximum of S + log2(step) - 15
    if constexpr (!FULL) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        int pos[2], wlo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = rt * 8 * NT + nt * 8 + 2 * fr + e;
          pos[e] = first + r - span_head(p, r) * p.q_tokens;
          wlo[e] = int(max(int64_t(pos[e]) - p.pre, int64_t(0)));
        }
#pragma unroll
        for (int v = 0; v < SETS; ++v)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int j = tile_key(i, HALF ? 2 * v + half : v) + 8 * q + k0;
            float y[2];
            f2_unpack(s[v][nt][q], y[0], y[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!(j <= pos[e] && (j < p.sink || j >= wlo[e]))) y[e] = -INFINITY;
            s[v][nt][q] = f2_pack(y[0], y[1]);
          }
      }
#pragma unroll
      for (int v = 0; v < SETS; ++v)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int j = tile_key(i, HALF ? 2 * v + half : v) + 8 * q + k0;
          const bool any = j < L && (j < p.sink || j >= win);
#pragma unroll
          for (int k = 0; k < NG; ++k) vw[v][q][k] = any ? vw[v][q][k] : 0u;
        }
    }
    float x[NT][2];
#pragma unroll
    for (int v = 0; v < SETS; ++v) {
      float big[2];   // log2(step 2^-15 + 2^-45): a page outside the pool has steps of 0
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float t = int4_pair<BF16>(vw[v][q][0]).x;
#pragma unroll
        for (int k = 1; k < NG; ++k) t = fmaxf(t, int4_pair<BF16>(vw[v][q][k]).x);
        big[q] = log2_approx(fmaf(t, 0x1p-15f, 0x1p-45f));
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
      {
        float y0[2], y1[2];
        f2_unpack(f2_fma(s[v][nt][0], cr[nt], f2_pack(big[0], big[0])), y0[0], y0[1]);
        f2_unpack(f2_fma(s[v][nt][1], cr[nt], f2_pack(big[1], big[1])), y1[0], y1[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) x[nt][e] = v == 0 ? fmaxf(y0[e], y1[e]) : fmax3(x[nt][e], y0[e], y1[e]);
      }
    }
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) moved |= x[nt][0] > m[nt][0] || x[nt][1] > m[nt][1];
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float a[2], z[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = x[nt][e];
          if (HALF) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
          const float nm = fmaxf(m[nt][e], y);
          a[e] = m[nt][e] == nm ? 1.f : fast_exp2(m[nt][e] - nm);
          z[e] = nm == -INFINITY ? 0.f : -nm;
          m[nt][e] = nm;
        }
        const uint64_t a2 = f2_pack(a[0], a[1]);
        nz[nt] = f2_pack(z[0], z[1]);
        l[nt] = f2_mul(l[nt], a2);
#pragma unroll
        for (int k = 0; k < NG; ++k) zs[nt][k] = f2_mul(zs[nt][k], a2);
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][j][h][e] *= a[e & 1];
      }
    }
    // ---- P and O^T
    uint32_t pb[SUB][NT][NG][2];
#pragma unroll
    for (int v = 0; v < SETS; ++v)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint64_t y[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float t[2];
          f2_unpack(f2_fma(s[v][nt][q], cr[nt], nz[nt]), t[0], t[1]);
          y[q] = f2_pack(fast_exp2(t[0]), fast_exp2(t[1]));
        }
        l[nt] = f2_add(l[nt], f2_add(y[0], y[1]));
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          uint32_t t01[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float2 g = int4_pair<BF16>(vw[v][q][k]);
            if constexpr (FULL) {
              zs[nt][k] = f2_fma(y[q], f2_pack(g.y, g.y), zs[nt][k]);
            } else {   // (a low value that a row does not see may be a NaN)
              float s0, s1, y0, y1, z0, z1;
              f2_unpack(s[v][nt][q], s0, s1);
              f2_unpack(y[q], y0, y1);
              f2_unpack(zs[nt][k], z0, z1);
              zs[nt][k] = f2_pack(s0 != -INFINITY ? fmaf(y0, g.y, z0) : z0, s1 != -INFINITY ? fmaf(y1, g.y, z1) : z1);
            }
            float p0, p1;
            const uint64_t pq = f2_mul(y[q], f2_pack(g.x, g.x));
            f2_unpack(pq, p0, p1);
            const uint32_t h = half2_bits(p0, p1);
            if constexpr (!BF16) zs[nt][k] = p_rest(pq, h, zs[nt][k]);
            t01[q] = trans8(h);
          }
          const uint32_t t0 = t01[0], t1 = t01[1];
          if constexpr (HALF) {   // rows 0-3 (of this fragment: lanes fg) are the first tile's
            pb[2 * v][nt][k][0] = fg < 4 ? t0 : 0u;
            pb[2 * v][nt][k][1] = fg < 4 ? t1 : 0u;
            pb[2 * v + 1][nt][k][0] = fg < 4 ? 0u : t0;
            pb[2 * v + 1][nt][k][1] = fg < 4 ? 0u : t1;
          } else {
            pb[v][nt][k][0] = t0;
            pb[v][nt][k][1] = t1;
          }
        }
      }
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      if constexpr (!EARLY) load_v(u);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const uint32_t a = va[u][j][0], c = va[u][j][1];
        const uint32_t a8 = a >> 8, c8 = c >> 8;
        // rows 0-7: columns in bits 0-3; rows 8-15: the next ones, in bits 4-7
        const uint32_t f0[4] = {a & 0x000f000fu, a & 0x00f000f0u, c & 0x000f000fu, c & 0x00f000f0u};
        const uint32_t f1[4] = {a8 & 0x000f000fu, a8 & 0x00f000f0u, c8 & 0x000f000fu, c8 & 0x00f000f0u};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(o[nt][j][0], f0, pb[u][nt][j / PER][0], pb[u][nt][j / PER][1]);
          mma_f16(o[nt][j][1], f1, pb[u][nt][j / PER][0], pb[u][nt][j / PER][1]);
        }
      }
    }
  };
  uint32_t slot = 0, slot_before = kEnd - kStep;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    wait_group<ST - 2>();
    // the step is in for every lane, and the slot before it has been read
    if constexpr (MT == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + kg), "r"(32 * MT) : "memory");
    issue(i + ST - 1, slot_before);
    const int v0 = first_tile + i * stride;
    if (v0 + SUB <= f_sink || (v0 >= f_lo && v0 + SUB <= f_hi)) run(std::true_type(), i, ring + slot);
    else run(std::false_type(), i, ring + slot);
    slot_before = slot;
    slot = slot + kStep == kEnd ? 0u : slot + kStep;
  }
  cp_async_wait_all();

  // ---------------------------------------------------------------- join
#pragma unroll
  for (int d = 4; d < 32; d <<= 1)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt] = f2_add(l[nt], __shfl_xor_sync(0xffffffffu, l[nt], d));
#pragma unroll
      for (int k = 0; k < NG; ++k) zs[nt][k] = f2_add(zs[nt][k], __shfl_xor_sync(0xffffffffu, zs[nt][k], d));
    }
  __syncthreads();           // every ring has been read
  float* ob = reinterpret_cast<float*>(smem);
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffML);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = rt * 8 * NT + nt * 8 + 2 * fr + e, part = HALF ? 2 * kg + half : kg;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float z2[2];
        f2_unpack(zs[nt][j / PER], z2[0], z2[1]);
        const float z = z2[e];
        const float4 v = make_float4(fmaf(o[nt][j][0][e], 0x1p24f, z), fmaf(o[nt][j][0][2 + e], 0x1p20f, z),
                                     fmaf(o[nt][j][1][e], 0x1p24f, z), fmaf(o[nt][j][1][2 + e], 0x1p20f, z));
        // columns 4 c4 ..: of unit (g = fg, j), or of unit 8 j + fg, which is (g, fg % U)
        const int c4 = NG == 1 ? 8 * (fg % U) + 8 / U * j + fg / U : 8 * j + fg;
        *reinterpret_cast<float4*>(ob + join_at<D, C::kRows>(part, r, c4)) = v;
      }
      float l2[2];
      f2_unpack(l[nt], l2[0], l2[1]);
      if (fg == 0) ml[part * C::kRows + r] = make_float2(m[nt][e], l2[e]);
    }
  if constexpr (SPLIT) {
    const Piece now = share.piece[turn];
    if (now.parts == 1) {
      join_unit<D, BF16, C::kRows, C::kParts, C::kThreads>(p, ob, ml, smem + C::kOffIn, 0u, 0u, b, kvh);
    } else {
      const int64_t at = 2 * int64_t(share_cta()) + (now.parts > 1 ? 1 : 0);
      write_part<D, C::kRows, C::kParts, C::kThreads>(p, ob, ml, ip.part_o + at * p.rows * D, ip.part_ml + at * p.rows);
      if (now.parts > 1 && threadIdx.x == 0) ip.heads[share_cta()] = make_int4(b, kvh, now.parts, 0);
    }
    turn ^= 1;
    __syncthreads();           // (the rings take the results' place)
  } else {
    join_unit<D, BF16, C::kRows, C::kParts, C::kThreads>(p, ob, ml, smem + C::kOffIn, lg, rank, b, kvh);
  }
  } while (SPLIT);
}

// Joins the parts of the units that more than one CTA has worked on: CTA g those
// of the unit whose first part is CTA g's (the next ones are of the next shares'
// CTAs of the head).  A thread has a float4 of a row.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) int4_join_kernel(const __grid_constant__ Int4SpanParams ip) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  const SpanParams& p = ip.s;
  grid_dep_launch();
  grid_dep_wait();
  const int4 head = ip.heads[blockIdx.x];
  if (head.z == 0) return;
  constexpr int kBatch = 8;
  for (int e = blockIdx.y * 256 + int(threadIdx.x); e < p.rows * (D / 4); e += int(gridDim.y) * 256) {
    const int r = e / (D / 4), c4 = e % (D / 4);
    float top = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g0 = 0; g0 < head.z; g0 += kBatch) {
      float2 w2[kBatch];
      float4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int g = min(g0 + k, head.z - 1);
        const int64_t slot = 2 * (int64_t(blockIdx.x) + int64_t(g) * p.N2) + (g == 0 ? 1 : 0);
        w2[k] = ip.part_ml[slot * p.rows + r];
        x[k] = *reinterpret_cast<const float4*>(ip.part_o + (slot * p.rows + r) * D + c4 * 4);
        if (g0 + k >= head.z) w2[k] = make_float2(-INFINITY, 0.f);
      }
      float t = top;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) t = fmaxf(t, w2[k].x);
      const float keep = join_weight(top, t);
      l *= keep;
      a.x *= keep; a.y *= keep; a.z *= keep; a.w *= keep;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (g0 + k >= head.z) continue;
        const float w = join_weight(w2[k].x, t);
        l += w * w2[k].y;
        a.x += w * x[k].x; a.y += w * x[k].y; a.z += w * x[k].z; a.w += w * x[k].w;
      }
      top = t;
    }
    const int h = span_head(p, r), n1 = head.y * p.group + h, tok = r - h * p.q_tokens;
    const bool has = l != 0.f;   // a NaN sum stays a NaN
    const float inv = has ? 1.f / l : 0.f;
    uint2 u;
    u.x = has ? int4_out<BF16>(a.x * inv, a.y * inv) : 0u;
    u.y = has ? int4_out<BF16>(a.z * inv, a.w * inv) : 0u;
    T* orow = static_cast<T*>(p.out) + int64_t(head.x) * p.q_sb + int64_t(n1) * p.q_sn + int64_t(tok) * p.q_ss;
    *reinterpret_cast<uint2*>(orow + c4 * 4) = u;
    if (p.lse != nullptr && c4 == 0)
      p.lse[int64_t(head.x) * p.lse_sb + int64_t(n1) * p.lse_sn + int64_t(tok) * p.lse_ss] =
          has ? (top + __log2f(l)) * 0.69314718055994531f : INFINITY;
  }
}

// A cluster of CTAs per unit, heads side by side, let in while the kernel before
// it ends.
template <typename P>
cudaError_t launch_units(void (*kernel)(P), const P& args, const SpanParams& p, unsigned threads, size_t smem, cudaStream_t s) {
  const unsigned cs = 1u << p.lg_cs, y = unsigned(std::min(p.B, 65535));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.N2) * cs, y, (unsigned(p.B) + y - 1) / y);
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

template <int D, bool BF16>
cudaError_t launch_join(const Int4SpanParams& p, cudaStream_t s) {
  return launch_early(int4_join_kernel<D, BF16>, dim3(unsigned(p.n_ctas), unsigned((p.s.rows * (D / 4) + 255) / 256)), 256, 0, s, p);
}

template <int D, int NG, int NT, int MT, bool BF16>
cudaError_t launch_one(Int4SpanParams p, int n_sm, cudaStream_t s) {
  using C = Cfg<D, NG, NT, MT>;
  if (p.s.rows > C::kRows) return cudaErrorInvalidValue;
  if (p.heads != nullptr) {
    constexpr auto kernel = int4_decode_kernel<D, NG, NT, MT, BF16, true>;
    set_span_shape(p.s, 1);
    cudaError_t e = prepare_span<kernel>(C::kSmemShare);
    if (e == cudaSuccess) e = launch_early(kernel, dim3(unsigned(p.s.N2), unsigned(p.n_ctas / p.s.N2)), C::kThreads, C::kSmemShare, s, p);
    return e == cudaSuccess ? launch_join<D, BF16>(p, s) : e;
  }
  // start cost of a CTA in tiles: 0, 2, 8 of them take 1.20, 1.02, 0.99 times as long in the mean of 196 calls (1 to 64
  // sequences of 8 heads, 4 to 32 rows, up to 16000 keys), and 8 up to 1.09 times (20 of up to 4000 keys 22.7 -> 24.7 us)
  constexpr int kStart = 4;
  const int64_t span = std::min<int64_t>(p.s.kv_max, int64_t(p.s.sink) + p.s.pre + p.s.q_tokens);
  int cs = cluster_ctas(int64_t(p.s.B) * p.s.N2, p.s.rows, span / kTile + 1, C::kGroups, kStart, span < p.s.kv_max,
                        C::kResident, n_sm);
  // (a CTA that never has a step of its own only makes the join longer: one sequence of 37 keys 6.5 -> 5.2 us)
  while (cs > 1 && cs / 2 * C::kGroups * C::kSub * kTile >= span) cs /= 2;
  set_span_shape(p.s, cs);
  cudaError_t e = prepare_span<int4_decode_kernel<D, NG, NT, MT, BF16, false>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_units(int4_decode_kernel<D, NG, NT, MT, BF16, false>, p, p.s, C::kThreads, C::kSmem, s);
}

template <int D, int NG, bool BF16>
cudaError_t launch_rows(const Int4SpanParams& p, int n_sm, cudaStream_t s) {
  if (p.s.rows <= 4) return launch_one<D, NG, 0, 1, BF16>(p, n_sm, s);
  if (p.s.rows <= 8) return launch_one<D, NG, 1, 1, BF16>(p, n_sm, s);
  if (p.s.rows <= 16) return launch_one<D, NG, 2, 1, BF16>(p, n_sm, s);
  if (p.s.rows <= 32) return launch_one<D, NG, 2, 2, BF16>(p, n_sm, s);
  if constexpr (NG == 1) return cudaErrorInvalidValue;   // (int4_wide.cu's)
  else return launch_one<D, NG, 2, 4, BF16>(p, n_sm, s);
}

template <int D, int NG>
cudaError_t launch_groups(const Int4SpanParams& p, bool bf16, int n_sm, cudaStream_t s) {
  return bf16 ? launch_rows<D, NG, true>(p, n_sm, s) : launch_rows<D, NG, false>(p, n_sm, s);
}

}  // namespace int4_detail
}  // namespace fia
