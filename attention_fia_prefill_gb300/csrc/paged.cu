// Bookkeeping of a paged key/value cache on the GPU: block tables and slot
// maps from request lengths, and the write of new rows to their slots.
#include <algorithm>

#include "paged.h"

namespace fia {
namespace {

constexpr int kTableThreads = 256;
constexpr int kTablePer = 4;                                   // requests a thread scans
constexpr int kTableChunk = kTableThreads * kTablePer;         // requests scanned at once
constexpr int kTableTokens = 1024;                             // tokens a CTA writes

// Sum over the block of everything before this thread (and the total), two
// 64-bit values at once: lengths are 32-bit, their sums need not be.
__device__ __forceinline__ void block_scan2(int64_t& a, int64_t& b, int64_t& ta, int64_t& tb, int64_t (*sh)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t ia = a, ib = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t xa = __shfl_up_sync(0xffffffffu, ia, d), xb = __shfl_up_sync(0xffffffffu, ib, d);
    if (lane >= d) {
      ia += xa;
      ib += xb;
    }
  }
  if (lane == 31) {
    sh[warp][0] = ia;
    sh[warp][1] = ib;
  }
  __syncthreads();
  int64_t pa = 0, pb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kTableThreads / 32; ++w) {
    if (w < warp) {
      pa += sh[w][0];
      pb += sh[w][1];
    }
    ta += sh[w][0];
    tb += sh[w][1];
  }
  a = pa + ia - a;
  b = pb + ib - b;
}

// One pass over the tokens.  Request b holds have = ceil(context / bs) blocks
// and needs ceil((context + new) / bs); the blocks it lacks are the free
// list's entries from E_b, the blocks asked for by the requests before it.
// Every CTA scans the requests (new tokens and blocks, kTableChunk at a time)
// and writes the slots of its kTableTokens tokens, which it finds by a binary
// search in the running sum of new tokens.  A new block's first position is a
// new token (have * bs >= context), and the thread that has this token writes
// the block's table entry: no second pass, and no entry is both read and
// written (slots in older blocks come from entries below have).
// Bound: a launch and two dependent loads; the scan of 512 requests repeated
// by every CTA costs less than a launch of its own.
__global__ void __launch_bounds__(kTableThreads) block_table_kernel(const TableParams p) {
  __shared__ int64_t sh[kTableThreads / 32][2];
  __shared__ int s_cu[kTableChunk];        // new tokens up to and with the request, within the chunk
  __shared__ int s_ctx[kTableChunk];
  __shared__ int64_t s_blk[kTableChunk];   // blocks asked for before the request
  const int bs = p.block_size;
  const int64_t t0 = int64_t(blockIdx.x) * kTableTokens;
  const int64_t t1 = min(t0 + kTableTokens, int64_t(p.n_tokens));
  const bool lead = blockIdx.x == 0;
  int64_t tok = 0, blk = 0;   // before this chunk
  for (int base = 0; base < p.B && (lead || tok < t1); base += kTableChunk) {
    int ctx[kTablePer], add[kTablePer], nb[kTablePer];
    int64_t st = 0, sb = 0;
#pragma unroll
    for (int i = 0; i < kTablePer; ++i) {
      const int b = base + int(threadIdx.x) * kTablePer + i;
      ctx[i] = b < p.B ? max(p.context_lens[b], 0) : 0;
      add[i] = b < p.B ? max(p.new_lens[b], 0) : 0;
      const int64_t total = int64_t(ctx[i]) + add[i];
      nb[i] = int((total + bs - 1) / bs - (int64_t(ctx[i]) + bs - 1) / bs);
      st += add[i];
      sb += nb[i];
    }
    int64_t ct, cb;
    block_scan2(st, sb, ct, cb, sh);
#pragma unroll
    for (int i = 0; i < kTablePer; ++i) {
      const int b = base + int(threadIdx.x) * kTablePer + i, c = b - base;
      s_ctx[c] = ctx[i];
      s_blk[c] = blk + sb;
      sb += nb[i];
      st += add[i];
      // a CTA's tokens end below 2^31, so larger sums need not be told apart
      s_cu[c] = int(min(st, int64_t(0x7fffffff)));
      if (lead && b < p.B) {
        p.kv_lens[b] = int(min(int64_t(ctx[i]) + add[i], int64_t(0x7fffffff)));
        p.cu_new_lens[b] = int(min(tok + st, int64_t(0x7fffffff)));
      }
    }
    __syncthreads();
    const int64_t lo = max(t0, tok), hi = min(t1, tok + ct);
    const int n = min(kTableChunk, p.B - base);
    for (int64_t t = lo + threadIdx.x; t < hi; t += kTableThreads) {
      const int x = int(t - tok);
      int l = 0, r = n - 1;   // the first request whose running sum is above x
      while (l < r) {
        const int m = (l + r) >> 1;
        if (s_cu[m] > x) r = m; else l = m + 1;
      }
      const int64_t pos = int64_t(s_ctx[l]) + x - (l > 0 ? s_cu[l - 1] : 0);
      const int64_t page = pos / bs;
      const int off = int(pos - page * bs);
      const int64_t have = (int64_t(s_ctx[l]) + bs - 1) / bs;
      int32_t* row = p.block_table + int64_t(base + l) * p.table_cols;
      int id = -1;
      if (page < p.table_cols) {
        if (page < have) {
          id = row[page];
        } else {
          const int64_t f = s_blk[l] + page - have;
          if (f < p.n_free) id = p.free_blocks[f];
          if (off == 0) row[page] = id;
        }
      }
      const int64_t slot = int64_t(id) * bs + off;
      p.slot_mapping[t] = id < 0 || slot > 0x7fffffff ? -1 : int(slot);
    }
    tok += ct;
    blk += cb;
    __syncthreads();
  }
  for (int64_t t = max(t0, tok) + threadIdx.x; t < t1; t += kTableThreads) p.slot_mapping[t] = -1;
  if (lead && threadIdx.x == 0) p.num_blocks[0] = int(min(blk, int64_t(0x7fffffff)));
}

// One warp copies one token's row of one tensor (16-byte vectors, four in
// flight per lane).  Bound by memory: each row is read and written once.
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheWriteParams p) {
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int y = blockIdx.y, lane = threadIdx.x & 31;
  if (t >= p.n_tokens) return;
  const int slot = p.slots[t];
  if (slot < 0 || slot >= p.n_slots) return;
  const int blk = slot / p.block_size, off = slot - blk * p.block_size;
  const uint8_t* src = p.src[y] + int64_t(t) * p.src_row[y];
  uint8_t* dst = p.dst[y] + int64_t(blk) * p.dst_blk[y] + int64_t(off) * p.dst_row[y];
  const int n = p.vecs[y], hv = p.head_vecs[y];
  const int64_t hs = p.dst_head[y];
  for (int v0 = lane; v0 < n; v0 += 128) {
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (v0 + 32 * i < n) x[i] = __ldcs(reinterpret_cast<const uint4*>(src) + v0 + 32 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = v0 + 32 * i;
      if (v < n) {
        const int h = v / hv;
        *reinterpret_cast<uint4*>(dst + h * hs + int64_t(v - h * hv) * 16) = x[i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_block_table(const TableParams& p, cudaStream_t s) {
  const unsigned grid = unsigned(std::max<int64_t>(1, (int64_t(p.n_tokens) + kTableTokens - 1) / kTableTokens));
  block_table_kernel<<<grid, kTableThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache_write(const CacheWriteParams& p, cudaStream_t s) {
  const dim3 grid(unsigned((int64_t(p.n_tokens) + 7) / 8), p.vecs[1] > 0 ? 2u : 1u);
  cache_write_kernel<<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fia
