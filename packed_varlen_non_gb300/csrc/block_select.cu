// Block scores and selection for the block-sparse forward: which key tiles of
// its document each query block attends to.
//
//   qm_i = mean of the q-hat rows of query block i, km_j = mean of the k-hat
//   rows of key tile j (each rounded to fp32), score_ij = <qm_i, km_j>;
//   block i keeps the `keep` tiles of its document with the largest scores,
//   ties to the lower tile.
//
// Which tiles are kept is a discrete answer: a rounding that swaps two scores
// changes it.  Sums and scores are therefore carried as unevaluated pairs of
// fp32 numbers (Knuth's two-sum, and the product's rounding error from one
// fma: Dekker's and Ogita, Rump and Oishi's error-free transformations), good
// to about 2^-44 -- not in fp64, whose rate here is a fiftieth of fp32's: the
// pooling alone would take five times as long as reading its inputs.
//
// Two kernels.  pool_kernel is HBM-bound: it reads q-hat and k-hat once, one
// block per (128-row tile, head), every load of the tile in flight at once, and
// leaves 1.5 KB per tile and head.  Query blocks begin on tile boundaries, so
// the same tiles serve both.  score_kernel gives a warp to a query block and a
// lane to a key tile: 32 tiles' means are staged in shared memory, two dims per
// 8-byte word, and read without conflicts by all warps of the block, which
// share document and head.  The selection is a bitwise search for the keep-th
// largest key in 64-bit order-preserving keys (first the high halves, the low
// ones only among equals), then one ordered pass that writes the kept tiles.
#include "device_common.cuh"
#include "qk_norm.cuh"

namespace h3 {

namespace {

constexpr int kPoolThreads = 256;

// s + err = a + b exactly (Knuth).
__device__ __forceinline__ void two_sum(float& s, float& err, float a, float b) {
  s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  err = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}

// (hi, lo) += x
__device__ __forceinline__ void acc(float& hi, float& lo, float x) {
  float s, e;
  two_sum(s, e, hi, x);
  hi = s;
  lo = __fadd_rn(lo, e);
}
// (hi, lo) += (xh, xl)
__device__ __forceinline__ void acc2(float2& a, const float2& x) {
  acc(a.x, a.y, x.x);
  a.y = __fadd_rn(a.y, x.y);
}

// (hi + lo) / n rounded to fp32: a quotient and its remainder's quotient.
__device__ __forceinline__ float mean_of(const float2& s, float n) {
  const float q = __fdiv_rn(s.x, n);
  const float r = __fadd_rn(__fmaf_rn(-q, n, s.x), s.y);
  const float m = __fadd_rn(q, __fdiv_rn(r, n));
  return isfinite(q) ? m : q;  // (an infinite sum has no remainder)
}

// One (tile, head): sums of q-hat's rows as pairs, means of k-hat's.
__global__ void __launch_bounds__(kPoolThreads) pool_kernel(SelectArgs a) {
  __shared__ float2 part[2][8][128];
  const int tile = blockIdx.x, head = blockIdx.y;
  const int lane16 = threadIdx.x & 15, group = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const int4 t = __ldg(a.tiles + tile);
  const int n = t.y - t.x;
  const __nv_bfloat16* src[2] = {static_cast<const __nv_bfloat16*>(a.q_hat), static_cast<const __nv_bfloat16*>(a.k_hat)};
  uint4 raw[2][8];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = group + 16 * i;
      const __nv_bfloat16* p = src[x] + (int64_t)(t.x + r) * a.stride + head * kHeadDim + lane16 * 8;
      raw[x][i] = r < n ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float2 s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      qkn::unpack8(raw[x][i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc(s[e].x, s[e].y, v[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // the warp's two row groups
      const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, s[e].x, 16), __shfl_xor_sync(0xffffffffu, s[e].y, 16));
      acc2(s[e], o);
      if ((threadIdx.x & 16) == 0) part[x][warp][lane16 * 8 + e] = s[e];
    }
  }
  __syncthreads();
  const int x = threadIdx.x >> 7, d = threadIdx.x & 127;
  float2 s = part[x][0][d];
#pragma unroll
  for (int w = 1; w < 8; ++w) acc2(s, part[x][w][d]);
  const int64_t at = ((int64_t)head * a.n_tiles + tile) * kHeadDim + d;
  if (x == 0)
    a.q_sum[at] = s;
  else
    a.k_mean[at] = mean_of(s, (float)n);
}

// Order-preserving bits of a float that is not NaN (-0 as +0).
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Packed pairs: (a0 b0, a1 b1) and (a0 - b0, a1 - b1).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  dev::fma2(d.x, d.y, a.x, a.y, b.x, b.y, c.x, c.y);
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  dev::add2(d.x, d.y, a.x, a.y, b.x, b.y);
  return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.f, -1.f), a); }

constexpr int kChunk = 32;                       // key tiles staged at a time
constexpr int kChunkRow = kChunk + 1;            // 8-byte words per pair of dims (padded)

// Shared memory: km [64][kChunkRow] float2, qm [warps][64] float2, keys
// [warps][max_tiles] uint64.
__global__ void __launch_bounds__(32 * kSelectWarps) score_kernel(SelectArgs a) {
  extern __shared__ float2 smem[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2* km = smem;
  float2* qm = smem + 64 * kChunkRow + warp * 64;
  uint64_t* keys = reinterpret_cast<uint64_t*>(smem + 64 * kChunkRow + warps * 64) + (int64_t)warp * a.max_tiles;
  const int head = blockIdx.y;
  const int4 g0 = __ldg(reinterpret_cast<const int4*>(a.groups + blockIdx.x));
  const int first = __ldg(&a.groups[blockIdx.x].first);
  const int q0 = g0.x, n = g0.y, tile0 = g0.z, tiles = g0.w;
  const bool active = warp < n;
  // this block's own key tiles, relative to the document
  const int own0 = (first + warp) * a.tiles_per_q_block, own1 = min(own0 + a.tiles_per_q_block, tiles);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pooled sums are complete
  if (active) {
    // mean of the query block: four dims per lane, the sums of up to four tiles
    float2 s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = make_float2(0.f, 0.f);
    for (int t = own0; t < own1; ++t) {
      const float4* p = reinterpret_cast<const float4*>(a.q_sum + ((int64_t)head * a.n_tiles + tile0 + t) * kHeadDim + 4 * lane);
      const float4 u = p[0], v = p[1];
      acc2(s[0], make_float2(u.x, u.y));
      acc2(s[1], make_float2(u.z, u.w));
      acc2(s[2], make_float2(v.x, v.y));
      acc2(s[3], make_float2(v.z, v.w));
    }
    const float rows = (float)(__ldg(&a.tiles[tile0 + own1 - 1].y) - __ldg(&a.tiles[tile0 + own0].x));
    qm[2 * lane] = make_float2(-mean_of(s[0], rows), -mean_of(s[1], rows));  // (negated: see the loop)
    qm[2 * lane + 1] = make_float2(-mean_of(s[2], rows), -mean_of(s[3], rows));
  }
  const float* k_mean = a.k_mean + ((int64_t)head * a.n_tiles + tile0) * kHeadDim;
  for (int c0 = 0; c0 < tiles; c0 += kChunk) {
    __syncthreads();  // (also orders qm before its first read)
    for (int i = threadIdx.x; i < kChunk * 64; i += blockDim.x) {
      const int j = i >> 6, p = i & 63;
      if (c0 + j < tiles)
        km[p * kChunkRow + j] = __ldg(reinterpret_cast<const float2*>(k_mean + (int64_t)(c0 + j) * kHeadDim) + p);
    }
    __syncthreads();
    const int j = c0 + lane;
    if (active && j < tiles) {
      // -score, even and odd dims apart: each product -q k is x + e exactly
      float2 h = make_float2(0.f, 0.f), l = make_float2(0.f, 0.f);
#pragma unroll 8
      for (int p = 0; p < 64; ++p) {
        const float2 nq = qm[p], k = km[p * kChunkRow + lane];
        const float2 x = mul2(nq, k);
        const float2 e = fma2(nq, k, mul2(x, make_float2(-1.f, -1.f)));
        const float2 s = add2(h, x), bb = sub2(s, h);
        const float2 err = add2(sub2(h, sub2(s, bb)), sub2(x, bb));
        h = s;
        l = add2(l, add2(err, e));
      }
      float s, e;
      two_sum(s, e, h.x, h.y);
      const float low = __fadd_rn(e, __fadd_rn(l.x, l.y));
      // normalised pair of the score itself; a low part without a value (an
      // infinite or NaN score) counts as zero
      float hi, lo;
      two_sum(hi, lo, -s, -low);
      if (!isfinite(hi)) hi = -s;
      if (!isfinite(lo)) lo = 0.f;
      uint64_t key = ((uint64_t)ordered(hi) << 32) | ordered(lo);
      if (isnan(hi)) key = 0;                                          // below every number
      if (a.keep_own && j >= own0 && j < own1) key = ~0ull;
      keys[j] = key;
    }
  }
  if (!active) return;
  __syncwarp();
  const int cnt = min(a.keep, tiles);
  // the largest T with at least cnt keys >= T: high halves first
  uint32_t th = 0;
  int above = 0;  // keys whose high half is above th
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = th | (1u << bit);
    int m = 0;
    for (int j = lane; j < tiles; j += 32) m += (uint32_t)(keys[j] >> 32) >= cand;
    m = __reduce_add_sync(0xffffffffu, m);
    if (m >= cnt) th = cand;
    else above = m;
  }
  int equal = 0;
  for (int j = lane; j < tiles; j += 32) equal += (uint32_t)(keys[j] >> 32) == th;
  equal = __reduce_add_sync(0xffffffffu, equal);
  uint64_t T = (uint64_t)th << 32;
  int ties = cnt - above;  // of the keys equal to T, the lowest tiles taken
  if (above + equal > cnt) {
    // low halves among the keys whose high half is th
    uint32_t tl = 0;
    int more = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t cand = tl | (1u << bit);
      int m = 0;
      for (int j = lane; j < tiles; j += 32) m += (uint32_t)(keys[j] >> 32) == th && (uint32_t)keys[j] >= cand;
      m = __reduce_add_sync(0xffffffffu, m);
      if (above + m >= cnt) tl = cand;
      else more = m;
    }
    T |= tl;
    ties = cnt - above - more;
  } else {
    ties = 0;  // every key with high half th is kept: keys >= T
    T -= T > 0 ? 1 : 0;
    if (th == 0) ties = tiles;  // T = 0: keys equal to 0 are kept as well
  }
  const int64_t block = (int64_t)head * a.n_q_blocks + q0 + warp;
  int32_t* out = a.block_idx + block * a.max_blocks;
  int at = 0, taken = 0;
  for (int c0 = 0; c0 < tiles; c0 += 32) {
    const int j = c0 + lane;
    const uint64_t key = j < tiles ? keys[j] : 0;
    const unsigned below = (1u << lane) - 1;
    const bool tie = j < tiles && key == T;
    const unsigned tie_mask = __ballot_sync(0xffffffffu, tie);
    const bool in = j < tiles && (key > T || (tie && taken + __popc(tie_mask & below) < ties));
    const unsigned mask = __ballot_sync(0xffffffffu, in);
    if (in) out[at + __popc(mask & below)] = j;
    at += __popc(mask);
    taken += __popc(tie_mask);
  }
  for (int j = cnt + lane; j < a.max_blocks; j += 32) out[j] = -1;
  if (lane == 0) a.block_cnt[block] = cnt;
}

}  // namespace

cudaError_t launch_block_select(const SelectArgs& a, cudaStream_t stream) {
  pool_kernel<<<dim3(a.n_tiles, a.H), kPoolThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int warps = select_warps(a.max_tiles);
  const size_t smem = (64 * kChunkRow + warps * 64) * sizeof(float2) + (size_t)warps * a.max_tiles * sizeof(uint64_t);
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.n_groups, (unsigned)a.H);
  cfg.blockDim = dim3(32u * (unsigned)warps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, score_kernel, a);
}

}  // namespace h3
