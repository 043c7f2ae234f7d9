// Bookkeeping of a paged key/value cache on the GPU: block tables and slot
// maps from request lengths, and the write of new rows to their slots.
#include <algorithm>

#include "paged.h"

namespace fia {
namespace {

constexpr int kTableThreads = 256;
constexpr int kTablePer = 4;                                   // requests a thread scans, tokens it writes
constexpr int kTableChunk = kTableThreads * kTablePer;         // requests scanned at once; tokens of a CTA

__device__ __forceinline__ uint32_t ceil_div(uint32_t a, uint32_t b) { return a / b + (a % b != 0u); }

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
// and writes the slots of its kTableChunk tokens, four consecutive ones to a
// thread, which finds the first by a binary search in the running sum of new
// tokens and steps on from there.  A new block's first position is a new token
// (have * bs >= context), and the thread that has this token writes the
// block's table entry: no second pass, and no entry is both read and written
// (slots in older blocks come from entries below have).
// Bound: a launch and three dependent loads (lengths, block, slot); the scan
// repeated by every CTA costs less than a launch of its own.  16 sequences of
// one token 3.4 us, 512 prompts of up to 2047 tokens (524 thousand slots) 7.0.
__global__ void __launch_bounds__(kTableThreads) block_table_kernel(const TableParams p) {
  __shared__ int64_t sh[kTableThreads / 32][2];
  __shared__ int s_cu[kTableChunk];        // new tokens up to and with the request, within the chunk
  __shared__ int s_ctx[kTableChunk];
  __shared__ int64_t s_blk[kTableChunk];   // blocks asked for before the request
  grid_dep_launch();
  grid_dep_wait();   // the kernel before this one is complete: its writes are read, what it reads may be written
  const uint32_t bs = uint32_t(p.block_size);
  const int64_t t0 = int64_t(blockIdx.x) * kTableChunk;
  const int64_t t1 = min(t0 + kTableChunk, int64_t(p.n_tokens));
  const int64_t mine = t0 + int64_t(threadIdx.x) * kTablePer;   // this thread's first token
  const bool lead = blockIdx.x == 0;
  int slot[kTablePer];
#pragma unroll
  for (int k = 0; k < kTablePer; ++k) slot[k] = -1;
  int64_t tok = 0, blk = 0;   // before this chunk of requests
  for (int base = 0; base < p.B && (lead || tok < t1); base += kTableChunk) {
    int ctx[kTablePer], add[kTablePer];
    uint32_t nb[kTablePer];
    int64_t st = 0, sb = 0;
#pragma unroll
    for (int i = 0; i < kTablePer; ++i) {
      const int b = base + int(threadIdx.x) * kTablePer + i;
      ctx[i] = b < p.B ? max(p.context_lens[b], 0) : 0;
      add[i] = b < p.B ? max(p.new_lens[b], 0) : 0;
    }
#pragma unroll
    for (int i = 0; i < kTablePer; ++i) {
      nb[i] = ceil_div(uint32_t(ctx[i]) + uint32_t(add[i]), bs) - ceil_div(uint32_t(ctx[i]), bs);
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
    // this thread's tokens of this chunk's requests: [lo, hi)
    const int64_t lo = max(mine, tok), hi = min(min(mine + kTablePer, t1), tok + ct);
    if (lo < hi) {
      int l = 0, r = min(kTableChunk, p.B - base) - 1;   // the first request whose running sum is above lo
      const int x0 = int(lo - tok);
      while (l < r) {
        const int m = (l + r) >> 1;
        if (s_cu[m] > x0) r = m; else l = m + 1;
      }
#pragma unroll
      for (int k = 0; k < kTablePer; ++k) {
        const int64_t t = mine + k;
        if (t < lo || t >= hi) continue;
        const int x = int(t - tok);
        while (s_cu[l] <= x) ++l;
        const uint32_t pos = uint32_t(s_ctx[l]) + uint32_t(x - (l > 0 ? s_cu[l - 1] : 0));
        const uint32_t page = pos / bs, off = pos - page * bs, have = ceil_div(uint32_t(s_ctx[l]), bs);
        int32_t* row = p.block_table + int64_t(base + l) * p.table_cols;
        int id = -1;
        if (page < uint32_t(p.table_cols)) {
          if (page < have) {
            id = row[page];
          } else {
            const int64_t f = s_blk[l] + (page - have);
            if (f < p.n_free) id = p.free_blocks[f];
            if (off == 0) row[page] = id;
          }
        }
        const int64_t at = int64_t(id) * bs + off;
        slot[k] = id < 0 || at > 0x7fffffff ? -1 : int(at);
      }
    }
    tok += ct;
    blk += cb;
    __syncthreads();
  }
  int32_t* out = p.slot_mapping + mine;
  if (mine + kTablePer <= t1 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0) {
    *reinterpret_cast<int4*>(out) = make_int4(slot[0], slot[1], slot[2], slot[3]);
  } else {
#pragma unroll
    for (int k = 0; k < kTablePer; ++k)
      if (mine + k < t1) out[k] = slot[k];
  }
  if (lead && threadIdx.x == 0) p.num_blocks[0] = int(min(blk, int64_t(0x7fffffff)));
}

// One warp copies one token's row of one tensor (16-byte vectors, four in
// flight per lane).  Bound by memory: each row is read and written once; 32771
// tokens of 8 heads x 128 (252 MB moved) 40.1 us, 94% of a copy's rate; 16
// tokens 1.8 us, a launch.
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheWriteParams p) {
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int y = blockIdx.y, lane = threadIdx.x & 31;
  grid_dep_launch();
  grid_dep_wait();
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
  const unsigned grid = unsigned(std::max<int64_t>(1, (int64_t(p.n_tokens) + kTableChunk - 1) / kTableChunk));
  return launch_early(block_table_kernel, dim3(grid), kTableThreads, 0, s, p);
}

cudaError_t launch_cache_write(const CacheWriteParams& p, cudaStream_t s) {
  const dim3 grid(unsigned((int64_t(p.n_tokens) + 7) / 8), p.vecs[1] > 0 ? 2u : 1u);
  return launch_early(cache_write_kernel, grid, 256, 0, s, p);
}

}  // namespace fia
