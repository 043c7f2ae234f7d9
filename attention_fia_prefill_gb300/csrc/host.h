// Host helpers of the C ABI shared by its translation units (fia_api.cu
// defines the functions): error strings, tensor checks, layouts, tensor maps.
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/fia.h"
#include "internal.h"

namespace fia {

constexpr size_t kHeader = 256;   // workspace bytes [0, 256): device status word + padding

enum Layout { L_BSH, L_BSND, L_BNSD, L_TND, L_BAD };

// Records the message fia_last_error() returns on this thread; returns s.
fia_status fail(fia_status s, const char* fmt, ...);
fia_status cuda_check(cudaError_t e, const char* what);
// A call's device status: the word at the start of its workspace, a fresh
// epoch, and the wait limit.
DevStatus make_status(void* workspace);
int sm_count();

int64_t numel(const fia_tensor* t);
bool present(const fia_tensor* t);   // rank and data
bool given(const fia_tensor* t);     // rank, and data or zero elements
inline bool is_half(int32_t dt) { return dt == FIA_DTYPE_F16 || dt == FIA_DTYPE_BF16; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool same_shape(const fia_tensor* a, const fia_tensor* b);

Layout parse_layout(const char* s);
fia_status resolve_heads(const fia_params* p, int64_t& N1, int64_t& N2, int64_t max_ratio = 64);
// Shapes of q/k/v in a layout -> (B, N, S, D) (TND: B = -1, S = T).
fia_status dense_dims(const fia_tensor* t, Layout L, int64_t N, int64_t& B, int64_t& S, int64_t& D, const char* name);
// Strides (elements) of (b, n, s) for a layout with N heads of D.
void bns_strides(Layout L, int64_t N, int64_t S, int64_t D, int64_t* st);
fia_status check_lse(const fia_tensor* lse, const fia_params* p, Layout L, int64_t B, int64_t N1, int64_t S1, int64_t T1);
fia_status check_ws(void* ws, size_t have, size_t need);

// rank-d tiled map of 16-bit elements (u8: 8-bit), 128-byte swizzle, box
// {128 bytes, box_rows, 1, ...}; box: all box extents, where more than the
// second differ from 1.
fia_status make_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides_bytes,
                    uint32_t box_rows, bool u8 = false, const uint32_t* box = nullptr);
// The (D, S, N, B) map of a dense tensor (TND: (D, T, N, 1)), boxes of 128 rows.
fia_status dense_map(CUtensorMap* m, const fia_tensor* t, Layout L, int64_t B, int64_t N, int64_t S, int64_t D,
                     bool u8 = false);

// Events the caller asked to have recorded around the main kernel of its next
// call on this thread (fia_profile_next_call); takes them.
void take_profile_events(cudaEvent_t* start, cudaEvent_t* stop);

template <typename F>
cudaError_t profiled(cudaStream_t s, F&& launch) {
  cudaEvent_t a, b;
  take_profile_events(&a, &b);
  if (a != nullptr) {
    cudaError_t e = cudaEventRecord(a, s);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = launch();
  if (e != cudaSuccess) return e;
  if (b != nullptr) return cudaEventRecord(b, s);
  return cudaSuccess;
}

}  // namespace fia
