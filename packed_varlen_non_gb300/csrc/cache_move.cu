// Rows of a paged cache copied to other slots of it (accepted drafts that move
// up, forked pages); include/h3attn.h states what a group of moves is.
//
// HBM-bound: a row is read and written once.  A block takes a group's rows of one
// head, of k or of v: sixteen lanes a row, all of them read into registers (up to
// 16 chunks a thread) before the barrier and written behind it, which is what
// makes a group's moves simultaneous whatever their slots overlap in.  Every row's
// lanes hold the group's list among them: of equal destinations the last pair's
// row is written, which each row finds out with comparisons and a vote while its
// loads are on their way (from a list in shared memory 0.6 us more for 2,048 pages of
// 16 rows; behind the barrier 12 us more for 512 of 64).  512 pages of 64 rows, 8
// heads: 42 us, 6.3 TB/s, 95 % of the measured copy; 2,048 of 16 rows 51 us.
#include "device_common.cuh"

namespace h3 {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 16;  // rows in work at once

// kN: chunks of a thread (groups of up to 16 kN rows).
template <int kN>
__global__ void __launch_bounds__(kThreads, kN <= 4 ? 8 : 2) cache_move_kernel(const __grid_constant__ CacheMoveArgs a) {
  const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int64_t list = (int64_t)blockIdx.x * a.width;
  __nv_bfloat16* const rows = ((blockIdx.z != 0) ? a.v : a.k) + (int64_t)blockIdx.y * a.head_stride + 8 * c;
  const auto at = [&](int32_t slot) {
    const int32_t page = slot / a.page_size;
    return reinterpret_cast<uint4*>(rows + page * a.page_stride + (int64_t)(slot - page * a.page_size) * a.token_stride);
  };
  // every row's sixteen lanes hold the group's pairs, pair c + 16 i in lane c; a row's own one is its lane r0's
  const int own = (threadIdx.x & 16) | r0;
  int32_t src[kN], dst[kN], to[kN];
  uint4 x[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int p = c + i * kRows;
    src[i] = dst[i] = -1;
    if (p < a.width) {
      src[i] = __ldg(a.src + list + p);
      dst[i] = __ldg(a.dst + list + p);
    }
    if ((uint32_t)src[i] >= (uint32_t)a.n_slots || (uint32_t)dst[i] >= (uint32_t)a.n_slots) dst[i] = -1;  // left out
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int32_t from = __shfl_sync(0xffffffffu, src[i], own);
    to[i] = __shfl_sync(0xffffffffu, dst[i], own);
    if (to[i] >= 0) x[i] = *at(from);
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    bool again = c > r0 && dst[i] == to[i];
#pragma unroll
    for (int j = i + 1; j < kN; ++j) again = again || dst[j] == to[i];
    if ((__ballot_sync(0xffffffffu, again) >> (threadIdx.x & 16) & 0xffffu) != 0) to[i] = -1;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i)
    if (to[i] >= 0) *at(to[i]) = x[i];
}

template <int kN>
cudaError_t launch(const CacheMoveArgs& a, int heads, cudaStream_t stream) {
  cache_move_kernel<kN><<<dim3((unsigned)a.n_groups, (unsigned)heads, 2), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_move(const CacheMoveArgs& a, int heads, cudaStream_t stream) {
  if (a.n_groups == 0) return cudaSuccess;
  if (a.width <= kRows) return launch<1>(a, heads, stream);
  if (a.width <= 4 * kRows) return launch<4>(a, heads, stream);
  return launch<16>(a, heads, stream);
}

}  // namespace h3
