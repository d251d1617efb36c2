// Rows of a paged cache copied to other slots of it (accepted drafts that move
// up, forked pages); include/h3attn.h states what a group of moves is.
//
// HBM-bound: a row is read and written once.  A block takes a group's rows of one
// head, of k or of v: sixteen lanes a row, all of them read into registers (up to
// 16 chunks a thread) before the barrier and written behind it, which is what
// makes a group's moves simultaneous whatever their slots overlap in.  512 pages of
// 64 rows, 8 heads: 45 us, 6.0 TB/s, 89 % of the measured copy.
#include "device_common.cuh"

namespace h3 {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 16;  // rows in work at once

// kN: chunks of a thread (groups of up to 16 kN rows).
template <int kN>
__global__ void __launch_bounds__(kThreads) cache_move_kernel(const __grid_constant__ CacheMoveArgs a) {
  const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int64_t list = (int64_t)blockIdx.x * a.width;
  __nv_bfloat16* const rows = ((blockIdx.z != 0) ? a.v : a.k) + (int64_t)blockIdx.y * a.head_stride + 8 * c;
  const auto at = [&](int32_t slot) {
    const int32_t page = slot / a.page_size;
    return reinterpret_cast<uint4*>(rows + page * a.page_stride + (int64_t)(slot - page * a.page_size) * a.token_stride);
  };
  int32_t to[kN];
  uint4 x[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int r = r0 + i * kRows;
    int32_t from = -1;
    to[i] = -1;
    if (r < a.width) {
      from = __ldg(a.src + list + r);
      to[i] = __ldg(a.dst + list + r);
    }
    if ((uint32_t)from >= (uint32_t)a.n_slots || (uint32_t)to[i] >= (uint32_t)a.n_slots)
      to[i] = -1;
    else
      x[i] = *at(from);
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
