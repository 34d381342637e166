// What the kernels of the paged key/value cache share: its addressing, the
// batch's sequences, and the sticky status word.  Internal to libft.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ft_internal.h"

namespace ft {
namespace kv {

constexpr int kMaxSeqs = 4096;
constexpr int kMaxKvHeads = 1024;
constexpr int kMinScaleExp = -110;  // smallest scale 2^-110: code * scale is then a normal bf16 value (or 0)
constexpr int kNanScale = 255;

// Host-side checks shared by the entry points (FT_OK, or set_error's status).
ft_status check_pages(const ft_kv_pages* p);
ft_status check_batch(const ft_kv_pages* p, const ft_kv_batch* b);
ft_status check_rows(const char* name, const void* ptr, int64_t token_stride, int64_t head_stride);
// Device address of the current device's sticky status word.
ft_status status_word(int32_t** out);

__device__ __forceinline__ void raise(int32_t* status, int what) { atomicCAS(status, 0, what); }

// A sequence's new tokens and length, held within the batch's bounds.
struct Seq {
  int q0, m, n;  // first row, new tokens, tokens in all
};
__device__ __forceinline__ Seq load_seq(const ft_kv_pages& p, const ft_kv_batch& b, int s, int32_t* status) {
  const int q0 = __ldg(&b.q_start[s]), q1 = __ldg(&b.q_start[s + 1]), n = __ldg(&b.kv_len[s]);
  const int most = (int)(b.table_stride * p.page_tokens);
  Seq r{q0, q1 - q0, n};
  if (q0 < 0 || q1 < q0 || q1 > b.num_tokens || q1 - q0 > b.max_q_len || n < 0 || n > most) {
    raise(status, FT_ERR_INVALID_ARG);
    r = Seq{0, 0, 0};
  }
  return r;
}
// Page of a sequence's token block `i` (which lies within its length), or -1.
__device__ __forceinline__ int load_page(const ft_kv_pages& p, const ft_kv_batch& b, int s, int i, int32_t* status) {
  const int g = __ldg(&b.block_table[s * b.table_stride + i]);
  if ((unsigned)g < (unsigned)p.num_pages) return g;
  raise(status, FT_ERR_INVALID_ARG);
  return -1;
}
// The last s in [0, n) with start[s] <= t (start ascending; 0 if none).
__device__ __forceinline__ int find_seq(const int32_t* start, int n, int t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(&start[mid]) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// 2^(e - 127) of an exponent byte (255: NaN).  Stored bytes are 17..247 or 255.
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e == kNanScale ? 0x7fc00000u : e << 23); }

}  // namespace kv
}  // namespace ft
