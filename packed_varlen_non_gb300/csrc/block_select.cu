// Block scores and selection for the block-sparse forward: which key tiles of
// its document each query block attends to.
//
//   qm_i = mean of the q-hat rows of query block i, km_j = mean of the k-hat
//   rows of key tile j (each rounded to fp32), score_ij = <qm_i, km_j>;
//   block i keeps the `keep` tiles of its document with the largest scores,
//   ties to the lower tile.
//
// Which tiles are kept is a discrete answer: a rounding that swaps two scores
// changes it.  Sums of rows are therefore carried as unevaluated pairs of fp32
// numbers (error-free transformations of Knuth and Dekker), good to about 2^-44
// -- not in fp64, whose rate here is a fiftieth of fp32's: the pooling alone
// would take five times as long as reading its inputs.  The few scores that fp32
// leaves open are taken in fp64, where the product of two means is exact, the sum
// is good to 2^-46 |qm| |km|, and nothing overflows or vanishes.
//
// pool_kernel is HBM-bound: it reads q-hat and k-hat once and leaves 1.5 KB per
// tile and head.  Four blocks per SM take one (128-row tile, head, tensor) after
// another, the next one's 32 KB on its way to shared memory while this one's are
// summed from registers (a block for each, with its loads straight into registers,
// leaves the memory idle while it sums: 43 us against 37 for 220 MB, 65 against 57
// for 352 MB; the copies alone take 34 and 52.  Three blocks with two stages 39 and
// 61, five with one 39 and 58: the sums' chain needs the warps, and the copies need
// the shared memory).  Query blocks begin on tile boundaries, so the same tiles
// serve both.  Each thread sums sixteen rows of eight dims onto an anchor 2^6
// times above their largest magnitude: every addition then rounds at one fixed
// place, and its error is two subtractions away (four operations an element
// where a two-sum of unordered numbers takes seven: 55 against 40 us for 220 MB,
// q-hat and k-hat of 20,423 tokens and 21 heads, before the copies ran ahead).
//
// score_kernel takes eight query blocks of one document and head.  Its warps
// score 32 dims of 32 tiles at a time, a tile to a lane, against all eight: the
// key means, tiles innermost, are read once per block and straight into
// registers, a batch of loads ahead, the query means come from shared memory as
// broadcasts (with a warp per query block and the key means in shared memory,
// that memory's bandwidth bound it).  Then each warp selects for one query block.
// Scores are first plain fp32 sums with an error bound E; the keep-th largest of
// them, T, is found by a bitwise search over order-preserving keys.  A tile
// above T + 2 E is kept and one below T - 2 E is not, whatever the exact scores
// are.  Only where more tiles lie between than places are left (3 of 1,680 query
// blocks with 160 tiles, and ties) are the scores between computed in fp64 and
// ranked.  It is a chain of waits: 10 us after the pooling for 80 query blocks of
// 160 tiles and 21 heads, half of it hidden behind the pooling's tail (its launch
// is a programmatic dependent one).
#include <algorithm>

#include "device_common.cuh"
#include "qk_norm.cuh"

namespace h3 {

namespace {

constexpr int kPoolThreads = 128;
constexpr int kPoolRows = 16 * kKeyTile / kPoolThreads;  // rows per thread (16 lanes a row)
constexpr int kPoolBlocks = 4;                          // per SM
constexpr int kPoolStages = 1;                          // of a tile's 32 KB each
constexpr uint32_t kPoolStage = kKeyTile * kHeadDim * 2;

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

// Packed pairs of fp32 numbers (one instruction each).
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

// Elementwise larger magnitude of two pairs of bf16 numbers (NaN if either is),
// under a sign that means nothing.
__device__ __forceinline__ uint32_t max_mag_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 16 bytes copied to shared memory, the rows' 256 bytes together from DRAM; zeros
// where `in` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::256B [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0), "l"(policy)
               : "memory");
}

// 1.5 * 2^(e + 6) for a number of exponent e (sums of kPoolRows numbers up to it
// stay in the anchor's binade); no further than the largest exponent.
__device__ __forceinline__ float anchor_of(uint32_t bits) {
  const uint32_t e = min(bits & 0x7f800000u, 248u << 23);
  return __uint_as_float((e + (6u << 23)) | 0x00400000u);
}

static_assert(kPoolRows <= 16, "2^(e + 1) * kPoolRows <= 2^(e + 5)");

// Items, one (tile, tensor, head) each: sums of q-hat's rows as pairs, means of
// k-hat's.  A block takes every gridDim.x-th item and copies kPoolStages
// ahead; a thread reads what it copied itself, so the copies need no barrier.
__global__ void __launch_bounds__(kPoolThreads, kPoolBlocks) pool_kernel(SelectArgs a) {
  extern __shared__ float2 smem[];
  __shared__ float2 part_of[2][kPoolThreads / 32][128];
  const int lane16 = threadIdx.x & 15, group = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;");  // (the scoring blocks wait for this grid's end)
  // (q-hat and k-hat were most likely written just before: lines read here that
  // leave L2 first keep the written ones from being written back meanwhile; with
  // the default policy 70 instead of 65 us after the prologue for 32,768 tokens)
  const uint64_t policy = dev::policy_evict_first();
  const uint32_t own = dev::smem_u32(smem) + threadIdx.x * 16;  // this thread's chunks, kPoolThreads apart
  const uint32_t H = a.H, step = gridDim.x, items = 2u * a.n_tiles * H;  // (items below 2^31)
  const auto rows_of = [&](uint32_t item) {  // (the launch has at most `items` blocks)
    return __ldg(reinterpret_cast<const int2*>(a.tiles + ((min(item, items - 1) / H) >> 1)));
  };
  const auto copy = [&](uint32_t item, int stage, const int2& t) {
    if (item < items) {
      const bool k = (item / H) & 1;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(k ? a.k_hat : a.q_hat) +
                                 (int64_t)(t.x + group) * a.stride + item % H * kHeadDim + lane16 * 8;
      const uint32_t dst = own + stage * kPoolStage;
#pragma unroll
      for (int i = 0; i < kPoolRows; ++i) {
        const bool in = group + kPoolThreads / 16 * i < t.y - t.x;
        copy16(dst + i * kPoolThreads * 16, in ? src + i * (kPoolThreads / 16) * a.stride : src, in, policy);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int2 t[kPoolStages + 1];
#pragma unroll
  for (int x = 0; x <= kPoolStages; ++x) t[x] = rows_of(blockIdx.x + x * step);
#pragma unroll
  for (int x = 0; x < kPoolStages; ++x) copy(blockIdx.x + x * step, x, t[x]);
#pragma unroll 1
  for (uint32_t item = blockIdx.x, k = 0; item < items; item += step, ++k) {
    const uint32_t stage = k % kPoolStages;
    const int head = item % H, tile = (item / H) >> 1, n = t[0].y - t[0].x;
    const bool is_k = (item / H) & 1;
    float2(*const part)[128] = part_of[k & 1];
    asm volatile("cp.async.wait_group %0;" ::"n"(kPoolStages - 1) : "memory");
    uint4 raw[kPoolRows];
#pragma unroll
    for (int i = 0; i < kPoolRows; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(raw[i].x), "=r"(raw[i].y), "=r"(raw[i].z), "=r"(raw[i].w)
                   : "r"(own + stage * kPoolStage + i * kPoolThreads * 16)
                   : "memory");
#pragma unroll
    for (int x = 0; x < kPoolStages; ++x) t[x] = t[x + 1];
    t[kPoolStages] = rows_of(item + (kPoolStages + 1) * step);
    copy(item + kPoolStages * step, stage, t[kPoolStages - 1]);
    uint4 m = raw[0];  // largest magnitude of each dim
#pragma unroll
    for (int i = 1; i < kPoolRows; ++i) {
      m.x = max_mag_bf16x2(m.x, raw[i].x);
      m.y = max_mag_bf16x2(m.y, raw[i].y);
      m.z = max_mag_bf16x2(m.z, raw[i].z);
      m.w = max_mag_bf16x2(m.w, raw[i].w);
    }
    const uint32_t mw[4] = {m.x, m.y, m.z, m.w};
    float2 anchor[4], hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      anchor[e] = make_float2(anchor_of(mw[e] << 16), anchor_of(mw[e]));
      hi[e] = anchor[e];
      lo[e] = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kPoolRows; ++i) {
      float v[8];
      qkn::unpack8(raw[i], v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = make_float2(v[2 * e], v[2 * e + 1]);
        const float2 s = add2(hi[e], x);
        lo[e] = add2(lo[e], sub2(x, sub2(s, hi[e])));
        hi[e] = s;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 h = sub2(hi[e], anchor[e]);
      const float2 own[2] = {make_float2(h.x, lo[e].x), make_float2(h.y, lo[e].y)};
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // the warp's two row groups
        float2 s = own[c];
        acc2(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, 16), __shfl_xor_sync(0xffffffffu, s.y, 16)));
        if ((threadIdx.x & 16) == 0) part[warp][lane16 * 8 + 2 * e + c] = s;
      }
    }
    __syncthreads();
    static_assert(kPoolThreads == kHeadDim, "a thread per dim");
    const int d = threadIdx.x;
    float2 s = part[0][d];
#pragma unroll
    for (int w = 1; w < kPoolThreads / 32; ++w) acc2(s, part[w][d]);
    if (is_k)  // tiles innermost, two dims a word: a warp's lanes score consecutive tiles
      reinterpret_cast<float*>(a.k_mean + ((int64_t)head * 64 + (d >> 1)) * a.n_tiles + tile)[d & 1] = mean_of(s, (float)n);
    else
      a.q_sum[((int64_t)head * a.n_tiles + tile) * kHeadDim + d] = s;
  }
}

// Order-preserving bits of a float that is not NaN (-0 as +0).
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Order-preserving key of a score in fp64 (0 for NaN, below every number's).
__device__ __forceinline__ uint64_t score_key(double s) {
  const uint64_t b = (uint64_t)__double_as_longlong(s + 0.0);
  return isnan(s) ? 0 : (b >> 63) ? ~b : (b | (1ull << 63));
}

// The score of one tile by one lane, in fp64: the products are exact, and whatever
// the means' magnitudes are, nothing overflows or vanishes.  (All tiles of every
// block tied, which takes equal tiles or a zero query block: 20,423 tokens and 21
// heads 315 us for the whole call, 51 for inputs without ties; pairs of fp32
// numbers took 70, but lose their low parts for products below 2^-100 and their
// high ones above 2^127.)  q (shared memory, kSelectWarps words apart) and k (`row`
// words apart), 64 words each.
__device__ __noinline__ uint64_t exact_key_lane(const float2* q, const float2* k, int64_t row) {
  double x = 0.0, y = 0.0;
#pragma unroll 8
  for (int p = 0; p < 64; ++p) {
    const float2 qq = q[p * kSelectWarps], kk = __ldg(k + p * row);
    x = fma((double)qq.x, (double)kk.x, x);
    y = fma((double)qq.y, (double)kk.y, y);
  }
  return score_key(x + y);
}

// The same by a whole warp (every lane gets it): four dims per lane.
__device__ __forceinline__ uint64_t exact_key_warp(const float2* q, const float2* k, int64_t row, int lane) {
  const float2 k0 = __ldg(k + 2 * lane * row), k1 = __ldg(k + (2 * lane + 1) * row);
  const float2 q0 = q[2 * lane * kSelectWarps], q1 = q[(2 * lane + 1) * kSelectWarps];
  double s = fma((double)q0.x, (double)k0.x, (double)q0.y * (double)k0.y) +
             fma((double)q1.x, (double)k1.x, (double)q1.y * (double)k1.y);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return score_key(__shfl_sync(0xffffffffu, s, 0));
}

// The cnt-th largest of a warp's keys 0 .. n - 1 (key(j), called for j of this
// lane: lane, lane + 32, ...) and how many are above it.  Bitwise from the
// first bit in which keys differ; it ends as soon as a candidate has exactly
// cnt keys at or above it, after about log2(n) bits.
template <class Key>
__device__ __forceinline__ uint32_t kth_largest(int n, int cnt, int lane, int* above, Key key) {
  uint32_t any = 0, all = ~0u;
  for (int j = lane; j < n; j += 32) {
    any |= key(j);
    all &= key(j);
  }
  any = __reduce_or_sync(0xffffffffu, any);
  all = __reduce_and_sync(0xffffffffu, all);
  uint32_t th = all;  // the common leading bits; below them, bits that every key has do not matter
  *above = 0;
  const uint32_t differ = any ^ all;
  if (differ == 0) return all;
  const int top = 31 - __clz(differ);
  th &= ~((2u << top) - 1);
#pragma unroll 1
  for (int bit = top; bit >= 0; --bit) {
    const uint32_t cand = th | (1u << bit);
    int m = 0;
    for (int j = lane; j < n; j += 32) m += key(j) >= cand;
    m = __reduce_add_sync(0xffffffffu, m);
    if (m >= cnt) th = cand;
    else *above = m;
    if (m == cnt) break;
  }
  // the smallest key at or above th is the cnt-th largest
  uint32_t least = ~0u;
  for (int j = lane; j < n; j += 32)
    if (key(j) >= th) least = min(least, key(j));
  least = __reduce_min_sync(0xffffffffu, least);
  int greater = 0;
  for (int j = lane; j < n; j += 32) greater += key(j) > least;
  *above = __reduce_add_sync(0xffffffffu, greater);
  return least;
}

constexpr uint32_t kOwnKey = 0xffffffffu;        // above every score's key

// Keys [*lo, *hi] of the scores within 2 E of the one whose key is th (all
// scores where E does not bound them; the own tiles where they fill every place).
__device__ __forceinline__ void border(uint32_t th, float E, uint32_t* lo, uint32_t* hi) {
  *lo = 0;
  *hi = kOwnKey - 1;
  if (th == kOwnKey) {
    *lo = *hi = kOwnKey;
  } else if (E < 0x1p100f) {
    const float T = __uint_as_float((th & 0x80000000u) ? th & 0x7fffffffu : ~th);
    *lo = ordered(__fsub_rd(T, 2.f * E));
    *hi = ordered(__fadd_ru(T, 2.f * E));
  }
}

// The selection where the keys fit in R registers a lane and no exact score is
// needed; false where one is, or where E bounds nothing.  *th: the cnt-th
// largest key.
template <int R>
__device__ __forceinline__ bool pick_few(const uint32_t* keys, int tiles, int cnt, int lane, float E, int32_t* out,
                                         uint32_t* kth) {
  uint32_t r[R];
  uint32_t any = 0, all = ~0u;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int j = 32 * i + lane;
    r[i] = j < tiles ? keys[j] : 0;
    any |= r[i];
    all &= j < tiles ? r[i] : ~0u;
  }
  any = __reduce_or_sync(0xffffffffu, any);
  all = __reduce_and_sync(0xffffffffu, all);
  const uint32_t differ = any ^ all;
  uint32_t th = all;
  if (differ != 0) {
    const int top = 31 - __clz(differ);
    th &= ~((2u << top) - 1);
#pragma unroll 1
    for (int bit = top; bit >= 0; --bit) {
      const uint32_t cand = th | (1u << bit);
      int m = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) m += r[i] >= cand;
      m = __reduce_add_sync(0xffffffffu, m);
      if (m >= cnt) th = cand;
      if (m == cnt) break;
    }
    uint32_t least = ~0u;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (r[i] >= th) least = min(least, r[i]);
    th = __reduce_min_sync(0xffffffffu, least);
  }
  *kth = th;
  uint32_t lo, hi;
  border(th, E, &lo, &hi);
  if (lo == 0) return false;  // (0 also stands behind the last tile)
  unsigned mask[R];
  int ge = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    mask[i] = __ballot_sync(0xffffffffu, r[i] >= lo);
    ge += __popc(mask[i]);
  }
  if (ge != cnt) return false;
  int at = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (r[i] >= lo) out[at + __popc(mask[i] & ((1u << lane) - 1))] = 32 * i + lane;
    at += __popc(mask[i]);
  }
  return true;
}

constexpr int kParts = 4;                        // parts of a score, 32 dims each
constexpr int kPartWords = 64 / kParts;

// Loads that keep their order, so that a batch is in flight at once (scheduled
// by the compiler they went out as their values were needed: an item's scores
// took 5,000 cycles instead of the one wait).
__device__ __forceinline__ float2 load_ordered(const float2* p) {
  float2 v;
  asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 load_ordered(const float4* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}

// Bytes of shared memory: qm [64][kSelectWarps] float2, then for each query block
// its scores' parts [kParts][max_tiles] float, which become its keys (uint32, the
// first part's place) and exact keys (uint64, the last two parts').
size_t score_smem(int warps, int32_t max_tiles) {
  return 64 * kSelectWarps * sizeof(float2) + (size_t)warps * max_tiles * (kParts * sizeof(float));
}

__global__ void __launch_bounds__(32 * kSelectWarps) score_kernel(SelectArgs a) {
  extern __shared__ float2 smem[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ uint32_t kn_of[kParts];  // largest squared norms of the key means' parts (bits of floats >= 0)
  float2* qm = smem + warp;  // word p at qm[p * kSelectWarps]
  float* const parts0 = reinterpret_cast<float*>(smem + 64 * kSelectWarps);
  uint32_t* keys = reinterpret_cast<uint32_t*>(parts0 + (int64_t)warp * kParts * a.max_tiles);
  uint64_t* exact = reinterpret_cast<uint64_t*>(keys + 2 * (int64_t)a.max_tiles);
  const int head = blockIdx.y;
  const int4 g0 = __ldg(reinterpret_cast<const int4*>(a.groups + blockIdx.x));
  const int2 g1 = __ldg(reinterpret_cast<const int2*>(a.groups + blockIdx.x) + 2);
  const int q0 = g0.x, n = g0.y, tile0 = g0.z, tiles = g0.w, first = g1.x;
  const bool active = warp < n;
  // this block's own key tiles, relative to the document, and its rows
  const int own0 = (first + warp) * a.tiles_per_q_block, own1 = min(own0 + a.tiles_per_q_block, tiles);
  const float rows = (float)(min(own1 * kKeyTile, g1.y) - own0 * kKeyTile);
  if (threadIdx.x < kParts) kn_of[threadIdx.x] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pooled sums are complete
  float qn = 0.f;  // squared norm of the query block's mean
  if (active) {
    // mean of the query block: four dims per lane, the sums of up to four tiles
    const float4* p = reinterpret_cast<const float4*>(a.q_sum + ((int64_t)head * a.n_tiles + tile0 + own0) * kHeadDim + 4 * lane);
    float4 u[4], v[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {  // (a tile that the block does not have: the first one's, times zero)
      const int x = own0 + t < own1 ? 64 * t : 0;
      u[t] = load_ordered(p + x);
      v[t] = load_ordered(p + x + 1);
    }
#pragma unroll
    for (int t = 1; t < 4; ++t)
      if (own0 + t >= own1) u[t] = v[t] = make_float4(0.f, 0.f, 0.f, 0.f);
    float2 s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = make_float2(0.f, 0.f);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      acc2(s[0], make_float2(u[t].x, u[t].y));
      acc2(s[1], make_float2(u[t].z, u[t].w));
      acc2(s[2], make_float2(v[t].x, v[t].y));
      acc2(s[3], make_float2(v[t].z, v[t].w));
    }
    const float2 x = make_float2(mean_of(s[0], rows), mean_of(s[1], rows));
    const float2 y = make_float2(mean_of(s[2], rows), mean_of(s[3], rows));
    qm[2 * lane * kSelectWarps] = x;
    qm[(2 * lane + 1) * kSelectWarps] = y;
    qn = x.x * x.x + x.y * x.y + (y.x * y.x + y.y * y.y);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) qn += __shfl_xor_sync(0xffffffffu, qn, off);
  }
  // Scores: a warp takes a part (32 dims) of 32 tiles' scores against all the
  // block's query blocks, so that each word of the key means is read once per
  // block, with one wait.
  const int64_t row = a.n_tiles;
  const float2* k_mean = a.k_mean + (int64_t)head * 64 * row + tile0;
  const int items = (tiles + 31) / 32 * kParts;
  const auto fetch = [&](int i, float2 (&k)[kPartWords]) {
    const float2* kp = k_mean + min(i / kParts * 32 + lane, tiles - 1) + i % kParts * kPartWords * row;
#pragma unroll
    for (int p = 0; p < kPartWords; ++p) k[p] = load_ordered(kp + p * row);
  };
  float2 k[kPartWords];
  if (warp < items) fetch(warp, k);
  __syncthreads();  // the query means
#pragma unroll 1
  for (int i = warp; i < items; i += warps) {
    const int j = i / kParts * 32 + lane, part = i % kParts;
    const float4* q = reinterpret_cast<const float4*>(smem + part * kPartWords * kSelectWarps);
    float2 next[kPartWords];  // the next item's words, on their way
    if (i + warps < items) fetch(i + warps, next);
    float2 h[kSelectWarps], m = make_float2(0.f, 0.f);
#pragma unroll
    for (int x = 0; x < kSelectWarps; ++x) h[x] = make_float2(0.f, 0.f);
#pragma unroll
    for (int p = 0; p < kPartWords; ++p) {
      m = fma2(k[p], k[p], m);
#pragma unroll
      for (int x = 0; x < kSelectWarps / 2; ++x) {
        const float4 qq = q[p * (kSelectWarps / 2) + x];
        h[2 * x] = fma2(make_float2(qq.x, qq.y), k[p], h[2 * x]);
        h[2 * x + 1] = fma2(make_float2(qq.z, qq.w), k[p], h[2 * x + 1]);
      }
    }
    const float norm = m.x + m.y;  // (infinite for one that fp32 does not hold)
    const uint32_t kn = __reduce_max_sync(0xffffffffu, __float_as_uint(norm < INFINITY ? norm : INFINITY));
    if (lane == 0) atomicMax(&kn_of[part], kn);
    if (j < tiles) {
#pragma unroll
      for (int x = 0; x < kSelectWarps; ++x)
        if (x < n) parts0[(x * kParts + part) * a.max_tiles + j] = h[x].x + h[x].y;
    }
#pragma unroll
    for (int p = 0; p < kPartWords; ++p) k[p] = next[p];
  }
  __syncthreads();
  if (!active) return;
  const float* parts = reinterpret_cast<const float*>(keys);
  for (int j = lane; j < tiles; j += 32) {
    const float sum = (parts[j] + parts[a.max_tiles + j]) + (parts[2 * a.max_tiles + j] + parts[3 * a.max_tiles + j]);
    keys[j] = a.keep_own && j >= own0 && j < own1 ? kOwnKey : (isnan(sum) ? 0u : ordered(sum));
  }
  __syncwarp();
  float kn = 0.f;  // (at least the largest squared norm of a key mean)
#pragma unroll
  for (int p = 0; p < kParts; ++p) kn += __uint_as_float(kn_of[p]);
  const int cnt = min(a.keep, tiles);
  const int64_t block = (int64_t)head * a.n_q_blocks + q0 + warp;
  int32_t* out = a.block_idx + block * a.max_blocks;
  for (int j = cnt + lane; j < a.max_blocks; j += 32) out[j] = -1;
  if (lane == 0) a.block_cnt[block] = cnt;
  const unsigned below = (1u << lane) - 1;

  // A score is eight sums of 16 fused products and seven additions, off by at
  // most 24 * 2^-24 |q| |k| (Cauchy-Schwarz).  E has 2.6 times that, for the
  // norms' own rounding too, and terms for underflow: 2^-120 for the products',
  // 2^-70 for the squares' (128 of them, each off by at most 2^-149, hide no more
  // than 2^-71 of a norm).
  const float E = 0x1p-18f * (sqrtf(qn) + 0x1p-70f) * (sqrtf(kn) + 0x1p-70f) + 0x1p-120f;
  uint32_t th;
  if (tiles <= 32 ? pick_few<1>(keys, tiles, cnt, lane, E, out, &th)
      : tiles <= 96 ? pick_few<3>(keys, tiles, cnt, lane, E, out, &th)
                    : tiles <= 256 && pick_few<8>(keys, tiles, cnt, lane, E, out, &th))
    return;
  int above;
  if (tiles > 256) th = kth_largest(tiles, cnt, lane, &above, [&](int j) { return keys[j]; });
  const bool own_only = th == kOwnKey;  // the block's own tiles fill every place, the lowest first
  uint32_t key_lo, key_hi;
  border(th, E, &key_lo, &key_hi);
  int ge = 0;
  for (int j = lane; j < tiles; j += 32) ge += keys[j] >= key_lo;
  ge = __reduce_add_sync(0xffffffffu, ge);
  if (ge == cnt) {  // the tiles around T are exactly the places left
    int at = 0;
    for (int c0 = 0; c0 < tiles; c0 += 32) {
      const int j = c0 + lane;
      const bool in = j < tiles && keys[j] >= key_lo;
      const unsigned mask = __ballot_sync(0xffffffffu, in);
      if (in) out[at + __popc(mask & below)] = j;
      at += __popc(mask);
    }
    return;
  }
  int n_in = 0;
  for (int j = lane; j < tiles; j += 32) n_in += keys[j] > key_hi;
  n_in = __reduce_add_sync(0xffffffffu, n_in);
  const int band = ge - n_in, places = cnt - n_in;
  if (band <= 32) {
    // few tiles around T: lane i takes the i-th of them and ranks its exact key
    int at = 0;
    int* list = reinterpret_cast<int*>(exact);
    for (int c0 = 0; c0 < tiles; c0 += 32) {
      const int j = c0 + lane;
      const bool in = j < tiles && keys[j] >= key_lo && keys[j] <= key_hi;
      const unsigned mask = __ballot_sync(0xffffffffu, in);
      if (in) list[at + __popc(mask & below)] = j;
      at += __popc(mask);
    }
    __syncwarp();
    const int mine = lane < band ? list[lane] : 0;
    uint64_t key = 0;
    for (int i = 0; i < band; ++i) {
      if (own_only) break;
      const uint64_t x = exact_key_warp(qm, k_mean + __shfl_sync(0xffffffffu, mine, i), row, lane);
      if (i == lane) key = x;
    }
    int rank = 0;
    for (int i = 0; i < band; ++i) {
      const uint64_t x = __shfl_sync(0xffffffffu, key, i);
      rank += x > key || (x == key && i < lane);
    }
    // a place each: the tile's key moves above or below the band
    if (lane < band) keys[mine] = rank < places ? kOwnKey : 0u;
    __syncwarp();
    at = 0;
    const uint32_t floor = key_hi == kOwnKey ? kOwnKey : key_hi + 1;
    for (int c0 = 0; c0 < tiles; c0 += 32) {
      const int j = c0 + lane;
      const bool in = j < tiles && keys[j] >= floor;
      const unsigned mask = __ballot_sync(0xffffffffu, in);
      if (in) out[at + __popc(mask & below)] = j;
      at += __popc(mask);
    }
    return;
  }
  // Many (ties): the exact keys of all of them, searched again.
  for (int j = lane; j < tiles; j += 32) {
    const uint32_t x = keys[j];
    exact[j] = x > key_hi ? ~0ull : (x >= key_lo ? exact_key_lane(qm, k_mean + j, row) : 0);
  }
  __syncwarp();
  const uint32_t high = kth_largest(tiles, cnt, lane, &above, [&](int j) { return (uint32_t)(exact[j] >> 32); });
  int more;
  const uint32_t low = kth_largest(tiles, cnt - above, lane, &more, [&](int j) {
    return (uint32_t)(exact[j] >> 32) == high ? (uint32_t)exact[j] : 0u;
  });
  // (at least cnt - above keys have this high half: the zeros of the others change nothing)
  const uint64_t T = ((uint64_t)high << 32) | low;
  int ties = cnt;  // places left for keys equal to T, the lowest tiles first
  int greater = 0;
  for (int j = lane; j < tiles; j += 32) greater += exact[j] > T;
  ties -= __reduce_add_sync(0xffffffffu, greater);
  int at = 0, taken = 0;
  for (int c0 = 0; c0 < tiles; c0 += 32) {
    const int j = c0 + lane;
    const uint64_t key = j < tiles ? exact[j] : 0;
    const bool tie = j < tiles && key == T;
    const unsigned tie_mask = __ballot_sync(0xffffffffu, tie);
    const bool in = j < tiles && (key > T || (tie && taken + __popc(tie_mask & below) < ties));
    const unsigned mask = __ballot_sync(0xffffffffu, in);
    if (in) out[at + __popc(mask & below)] = j;
    at += __popc(mask);
    taken += __popc(tie_mask);
  }
}

}  // namespace

cudaError_t launch_block_select(const SelectArgs& a, cudaStream_t stream) {
  // (both limits before the first launch, so that a refusal leaves nothing launched; the second one for every
  // size: dynamic and static bytes count together against the default of 48 KB)
  static SmemAttr pool_attr, score_attr;
  cudaError_t e = pool_attr.set(pool_kernel, (int)(kPoolStages * kPoolStage));
  if (e == cudaSuccess) e = score_attr.set(score_kernel, (int)score_smem(1, kSelectMaxTiles));
  if (e != cudaSuccess) return e;
  const unsigned blocks = std::min(2u * (unsigned)a.n_tiles * (unsigned)a.H, (unsigned)(kPoolBlocks * a.num_sms));
  pool_kernel<<<blocks, kPoolThreads, kPoolStages * kPoolStage, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int warps = select_warps(a.max_tiles);
  const size_t smem = score_smem(warps, a.max_tiles);  // (at most score_smem(1, kSelectMaxTiles), see select_warps)
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
