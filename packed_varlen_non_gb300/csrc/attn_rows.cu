// The shared-prefix forward of a few short documents (single queries over a long
// prefix): a pass over the prefix for up to 32 rows does 512 flops x rows per 512
// bytes of K and V and is bound by reading them.  The plan takes this kernel where
// it estimates it to be quicker than the tensor-core kernel's segments: for up to
// 64 to 256 rows, by heads and prefix.
//
// The tensor-core kernel of attn_fwd_tc.cu takes 512 query rows at a time and
// key tiles of 128 one after the other; with 32 rows its softmax chain, not
// the memory, set the time (25 us for 54 MB, 32 rows and 21 heads; this one 14
// us, 4 TB/s, from DRAM or from L2: what is left is the latency of six steps, the
// first copies and the exchange of the results).  Here a block takes up to 32 rows
// of one head over its share of the prefix, two blocks an SM: K and V stream
// through a three-stage ring of asynchronous copies (one 32 KB stage in use, two
// on their way; Q passes through the third, so the first copies are two stages
// too), each of the four warps takes 16 of a stage's 64 keys for all rows -- the
// scores, the softmax with a running maximum of its own and PV as m16n8k16
// products on registers (at 32 rows their rate is not the limit, and they need
// none of the set-up of the tcgen05 path) -- and the four partial results are
// joined in shared memory.  The blocks' partial rows go to the join, which also
// attends to each document's own keys (at most kJoinOwnKeys).
//
// Keys behind the prefix's end are filled with zeros by the copies and masked.
#include "device_common.cuh"

namespace h3 {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kStageKeys = 64;
constexpr int kStages = 3;
constexpr uint32_t kTensorBytes = kStageKeys * 256;       // K or V of a stage: rows of 128 bf16
constexpr uint32_t kStageBytes = 2 * kTensorBytes;
constexpr uint32_t kSmem = kStages * kStageBytes;
constexpr float kRescale = 32.0f;                         // log2 units (see attn_fwd_tc.cu)
constexpr int kORow = 136;  // floats between the joined O rows (eight rows' same dims in different banks)
static_assert(kSmem >= kWarps * kRowsTile * kORow * 4, "the joined O rows reuse the ring");
static_assert(kStageBytes >= kRowsTile * 256, "Q passes through a stage");

// Byte offset of 16-byte chunk c of row r of a stage's K or V (chunks swizzled
// by the row, so that eight rows' same chunk lie in different banks).
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return (uint32_t)(r * 256 + ((c ^ (r & 7)) << 4)); }

// n = 0: the 16 bytes are filled with zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n = 16) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// kM: 16-row tiles of query rows (1 or 2).
template <int kM>
__global__ void __launch_bounds__(kThreads, 2) attn_rows_kernel(RowsArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float2 ml_of[kWarps][kRowsTile];
  const uint32_t base = dev::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;  // fragment row and column group
  // the segment, as the plan lists it (computed: a load would delay the first copies)
  const int piece = blockIdx.x, head = blockIdx.y, q0 = blockIdx.z * kRowsTile, rows = min(kRowsTile, a.S - q0);
  const int key0 = (int)((int64_t)a.tiles * piece / a.pieces) * kKeyTile;
  const int key1 = (int)min((int64_t)a.tiles * (piece + 1) / a.pieces * kKeyTile, (int64_t)a.prefix_len);
  const int64_t col = (int64_t)head * kHeadDim;
  const __nv_bfloat16* kp = a.k_prefix + col;
  const __nv_bfloat16* vp = a.v_prefix + col;
  const int steps = (key1 - key0 + kStageKeys - 1) / kStageKeys;
  // This thread copies 16-byte chunk c of rows r0, r0 + 8, ... of a stage (eight
  // rows apart, a chunk keeps its place in the swizzle).
  const int r0 = threadIdx.x >> 4, c = threadIdx.x & 15;
  const uint32_t to = base + chunk_at(r0, c);
  const int64_t from = (int64_t)(key0 + r0) * a.prefix_stride + 8 * c, rows8 = 8 * a.prefix_stride;
  const auto load = [&](int step) {
    const uint32_t dst = to + (step % kStages) * kStageBytes;
    const int64_t at = from + (int64_t)step * (kStageKeys / 8) * rows8;
    const __nv_bfloat16 *ks = kp + at, *vs = vp + at;
    const int n = key1 - (key0 + step * kStageKeys + r0);  // keys from row r0 to the end
    if (n > kStageKeys - 8) {
#pragma unroll
      for (int i = 0; i < kStageKeys / 8; ++i) {
        copy16(dst + i * 2048, ks + i * rows8);
        copy16(dst + kTensorBytes + i * 2048, vs + i * rows8);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < kStageKeys / 8; ++i) {
        const bool in = 8 * i < n;
        copy16(dst + i * 2048, in ? ks + i * rows8 : kp, in ? 16 : 0);
        copy16(dst + kTensorBytes + i * 2048, in ? vs + i * rows8 : vp, in ? 16 : 0);
      }
    }
  };
  // Q through the last stage, which is loaded only once the first step begins
  const uint32_t qs = base + (kStages - 1) * kStageBytes;
  for (int r = r0; r < 16 * kM; r += 8)
    copy16(qs + chunk_at(r, c), a.q + (int64_t)(q0 + min(r, rows - 1)) * a.q_stride + col + 8 * c, r < rows ? 16 : 0);
  asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (s < steps) load(s);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;");  // (the join waits for this grid's end)

  // Q as A fragments, 8 steps of 16 dims: matrices (rows 0-7, 8-15) x (dims 0-7, 8-15)
  const int mat = lane >> 3, in_mat = lane & 7;
  uint32_t q[kM][8][4];
  asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
  __syncthreads();
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      ldsm4(q[m][k], qs + (chunk_at(16 * m + (mat & 1) * 8 + in_mat, mat >> 1) ^ (32 * k)));
  float o[kM][16][4], mx[kM][2], l[kM][2];
#pragma unroll
  for (int m = 0; m < kM; ++m) {
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[m][n][e] = 0.f;
    mx[m][0] = mx[m][1] = -3.402823466e38f;
    l[m][0] = l[m][1] = 0.f;
  }

  // ldmatrix rows of this lane: K: matrices (keys 0-7, 8-15) x (dims 0-7, 8-15);
  // V, transposed: the same with keys innermost
  // (a row's chunk c lies at c ^ (row & 7): the bytes of step k's chunks differ
  // from the first one's by an exclusive or)
  const uint32_t k_at = chunk_at(16 * warp + (mat >> 1) * 8 + in_mat, mat & 1);
  const uint32_t v_at = chunk_at(16 * warp + (mat & 1) * 8 + in_mat, mat >> 1);

#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncthreads();  // the stage has landed for all, and the one before it is read
    if (step + kStages - 1 < steps) load(step + kStages - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const uint32_t ks = base + (step % kStages) * kStageBytes, vs = ks + kTensorBytes;
    float s[kM][2][4];
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[m][n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t b[4];
      ldsm4(b, ks + (k_at ^ (32 * k)));
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        mma(s[m][0], q[m][k], b[0], b[1]);
        mma(s[m][1], q[m][k], b[2], b[3]);
      }
    }
    const int k0 = key0 + step * kStageKeys + 16 * warp + 2 * t;  // key of s[.][0][0]
    const bool last = step + 1 == steps;
    uint32_t p[kM][4];
#pragma unroll
    for (int m = 0; m < kM; ++m) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[m][n][e] *= a.scale_log2;
          if (last && k0 + 8 * n + (e & 1) >= key1) s[m][n][e] = -INFINITY;
        }
      bool grow = false;
      float next[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // rows g, g + 8
        float v = fmaxf(fmaxf(s[m][0][2 * h], s[m][0][2 * h + 1]), fmaxf(s[m][1][2 * h], s[m][1][2 * h + 1]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
        next[h] = v > mx[m][h] + kRescale ? v : mx[m][h];
        grow = grow || next[h] != mx[m][h];
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f = dev::ex2_approx(mx[m][h] - next[h]);
          mx[m][h] = next[h];
          l[m][h] *= f;
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            o[m][n][2 * h] *= f;
            o[m][n][2 * h + 1] *= f;
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = dev::ex2_approx(s[m][n][2 * h] - mx[m][h]), y = dev::ex2_approx(s[m][n][2 * h + 1] - mx[m][h]);
          l[m][h] += x + y;
          p[m][2 * n + h] = dev::pack_bf16x2(x, y);  // (bf16, as the tensor-core kernel's)
        }
    }
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      uint32_t b[4];
      ldsm4_t(b, vs + (v_at ^ (32 * n)));
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        mma(o[m][2 * n], p[m], b[0], b[1]);
        mma(o[m][2 * n + 1], p[m], b[2], b[3]);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // the ring is free

  // the four warps' results: row r's at word (warp, r, dim)
  float* const os = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = l[m][h];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int r = 16 * m + 8 * h + g;
      if (t == 0) ml_of[warp][r] = make_float2(mx[m][h], sum);
#pragma unroll
      for (int n = 0; n < 16; ++n)
        *reinterpret_cast<float2*>(os + (warp * kRowsTile + r) * kORow + 8 * n + 2 * t) =
            make_float2(o[m][n][2 * h], o[m][n][2 * h + 1]);
    }
  __syncthreads();
  for (int r = warp; r < rows; r += kWarps) {
    float M = ml_of[0][r].x;
#pragma unroll
    for (int x = 1; x < kWarps; ++x) M = fmaxf(M, ml_of[x][r].x);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      const float f = dev::ex2_approx(ml_of[x][r].x - M);
      const float4 v = reinterpret_cast<const float4*>(os + (x * kRowsTile + r) * kORow)[lane];
      sum.x = fmaf(f, v.x, sum.x);
      sum.y = fmaf(f, v.y, sum.y);
      sum.z = fmaf(f, v.z, sum.z);
      sum.w = fmaf(f, v.w, sum.w);
      total = fmaf(f, ml_of[x][r].y, total);
    }
    const int64_t at = ((int64_t)q0 * gridDim.y + (int64_t)head * rows) * a.pieces + piece * rows + r;
    reinterpret_cast<float4*>(a.part_o + at * kHeadDim)[lane] = sum;
    if (lane == 0) a.part_ml[at] = make_float2(M, total);
  }
}

template <int kM>
cudaError_t launch(const RowsArgs& a, int heads, cudaStream_t stream) {
  static SmemAttr attr;
  const cudaError_t e = attr.set(attn_rows_kernel<kM>, (int)kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)a.pieces, (unsigned)heads, (unsigned)((a.S + kRowsTile - 1) / kRowsTile));
  attn_rows_kernel<kM><<<grid, kThreads, kSmem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_rows(const RowsArgs& a, int heads, cudaStream_t stream) {
  return a.S <= 16 ? launch<1>(a, heads, stream) : launch<2>(a, heads, stream);
}

}  // namespace h3
