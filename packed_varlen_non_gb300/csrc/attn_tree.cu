// Attention for trees of drafted tokens (a single token among them) over a paged
// cache, heads grouped: include/h3attn.h, h3attn_forward_tree.
//
// The pages that define this library have no cache of keys and values; the text tower
// that they name (vllm.cpp PR #26 "feat(minimax-h3)", the device-encoder commit) is
// what answers from one.  The mathematics is the online softmax over key tiles: per query row a
// running reference m and sum l, p = 2^(s - m), O += P V, o = O / l.
//
// What bounds it: reading the cache.  A sequence's T drafts and the G query heads of
// a key head are G T rows over the same keys, 512 flops a row for 512 bytes of K and
// V; up to about 256 rows the tensor cores keep up with HBM.  So the rows of a key head
// fill the 128 lanes of a query tile (packed (token, head) as the causal walk does),
// one or two such tiles share a pass over the keys, and the work is cut by keys, not
// by rows:
//   - a step is one 128-key tile of one item (sequence, key head, up to two query
//     tiles).  Where there are no more items than SMs, every item is cut into equal
//     pieces of at most L tiles, one block each, L the smallest for which there are
//     blocks enough; otherwise the steps of all items, in order, are cut into equal ranges,
//     one per SM, which may hold pieces of several items.  (A second piece costs a block
//     4 us: its first loads and its first step wait for the first one's end.)
//     Where there are more items than SMs and each is a single query tile (kTwo), a range
//     goes to each of a block's two streams, whose piece boundaries then fall into the middle of
//     the other one's pieces.
//     Lengths are on the device, so each block adds them up itself and finds its
//     part; no list is built on the host and one captured graph serves growing
//     sequences.
//   - pieces of items that other blocks share leave partial rows (m, l, O), at most two
//     of them a block; attn_tree_join_kernel combines them in the order of the
//     keys, so results do not depend on which block ends first.
// Per block (one an SM), 12 warps:
//   warps 0..3, 4..7  softmax of stream 0 and 1, a thread a row;
//   warp 8            issues the MMAs: S_s = Q K^T (128 x 128 fp32 in TMEM), O_s += P V with
//                     P (bf16) in S's columns;
//   warp 9            Q tiles;
//   warps 10, 11      K tiles and V tiles, through one ring of five 32 KB slots (160 KB on their way
//                     an SM); a lane a page box: gcd(page_size, 128) rows each.  (A warp issues a
//                     copy in about 100 cycles: pages of 16 take 32 of them a step.)
// Two streams hide the chain S -> softmax -> PV: with two query tiles a stream is a
// query tile; with one, the streams take the key tiles in turn, each with a running
// maximum and O of its own, and the block joins the two at the piece's end.
// Rows behind a sequence's last draft: their scores are masked, their V rows are
// zeroed in shared memory before the PV reads them (0 times a stranger's NaN is not 0).
// Every wait is bounded, as in the forward (attn_fwd_tc.cu).
//
// Measured, in a graph on new inputs for each call: 32 single tokens over 5,033 (32 heads, 8 key heads, pages of 16) 104 to 106
// us, 6.2 to 6.3 TB/s, 93 to 95 % of the measured copy; 512 over 300 tokens 112 us; one over 20,000 24 us (22 where its 82 MB of
// cache lie in L2, as when a graph repeats the call), over none 9.3 us; 16 trees of 16 drafts (28 and 4
// heads, 32,768 tokens) 27 us (26); 8 trees of 64 drafts over 20,423 (64 and 8 heads) 262 us, 1,310 TFLOP/s, in short runs, 283 in
// long ones, under the power limit.  (Figures beside the code are of a graph that repeats one call.)  There the step of two
// query tiles takes 3,500 cycles, 2,048 of them products: a stream's chain is 1,750 cycles of softmax (one warp an SM
// sub-partition, bound by its own latencies), 450 until its PV is issued, 1,300 for PV and the next QK.  Two warps a row
// would halve the softmax, but leave 96 registers a thread, which spill into the step (833 us; as it is, the kernel of one
// range a block spills 176 bytes).  Few sequences: 4,500
// cycles until a block knows its part, 2,800 to its first loads' issue, 1,400 to 2,400 for them, and the join (4 us).
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstring>

#include "device_common.cuh"
#include "launch_common.cuh"
#include "tree_ring.h"

namespace h3 {

namespace {

constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kMmaWarp = 8, kQWarp = 9, kKWarp = 10, kVWarp = 11;
constexpr int kRows = 128;                          // of a query tile, and of a key tile
using ring::kSlots;
using ring::v_entry;
constexpr uint32_t kTileBytes = 128 * 256;          // two halves of 64 dims, 128-byte rows
constexpr uint32_t kHalfBytes = kTileBytes / 2;
constexpr uint32_t kSmemQ = 0;
constexpr uint32_t kSmemKV = 2 * kTileBytes;
constexpr uint32_t kSmemBar = kSmemKV + kSlots * kTileBytes;
constexpr int kNumBars = 4 + 2 * kSlots + 6 + 2;
constexpr uint32_t kSmemMl = kSmemBar + kNumBars * 8;   // float2 [2][128]
constexpr uint32_t kSmemMisc = kSmemMl + 2 * 128 * 8;
constexpr uint32_t kSlack = 496;                        // the base is 1 KB aligned (declared so; checked in the kernel)
constexpr size_t kSmemAlloc = kSmemMisc + 96 + kSlack;
static_assert(kSmemAlloc <= 227 * 1024, "shared memory per CTA");
static_assert(kSmemMl % 16 == 0, "alignment");
constexpr uint32_t kTmemCols = 512;                 // S0 S1 O0 O1, 128 columns each
constexpr uint64_t kTimeoutNs = 2000000000ull;      // 2 s
constexpr float kRescale = 32.0f;                   // log2 units (see attn_fwd_tc.cu)
constexpr float kLowest = -3.402823466e38f;

// kind::f16: fp32 accumulator, bf16 A and B, M = 128, N = 128
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescPV = kIdesc | (1u << 16);  // B (V) MN-major
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}

struct Bars {
  uint32_t base;
  __device__ uint32_t q_full(int i) const { return base + 8 * i; }
  __device__ uint32_t q_empty(int i) const { return base + 8 * (2 + i); }
  __device__ uint32_t full(int i) const { return base + 8 * (4 + i); }
  __device__ uint32_t empty(int i) const { return base + 8 * (4 + kSlots + i); }
  __device__ uint32_t s_ready(int s) const { return base + 8 * (4 + 2 * kSlots + s); }
  __device__ uint32_t p_ready(int s) const { return base + 8 * (6 + 2 * kSlots + s); }
  __device__ uint32_t pv_done(int s) const { return base + 8 * (8 + 2 * kSlots + s); }
  __device__ uint32_t drain() const { return base + 8 * (10 + 2 * kSlots); }
  __device__ uint32_t joined() const { return base + 8 * (11 + 2 * kSlots); }  // both streams' softmax warps
};

// S (TMEM) = Q * K^T, 8 MMAs of 16 dims, issued by one elected lane of the warp.
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t q_smem, uint32_t k_smem) {
  const uint32_t qa = desc_lo(q_smem, 16), kb = desc_lo(k_smem, 16);
#define H3_QK(off, pred)                                                                 \
  "add.u32 x, %1, " off ";\n\tadd.u32 y, %2, " off ";\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t" \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, " pred ";\n\t"
  asm volatile(
      "{\n\t.reg .pred p0, p1, e;\n\telect.sync _|e, 0xffffffff;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"
      "setp.ne.u32 p0, %4, %4;\n\tsetp.eq.u32 p1, %4, %4;\n\t"
      H3_QK("0", "p0") H3_QK("2", "p1") H3_QK("4", "p1") H3_QK("6", "p1")
      H3_QK("1024", "p1") H3_QK("1026", "p1") H3_QK("1028", "p1") H3_QK("1030", "p1")
      "}" ::"r"(d_tmem), "r"(qa), "r"(kb), "r"(kDescHi), "r"(0u), "r"(kIdesc)
      : "memory");
#undef H3_QK
}

// O (TMEM) (+)= P (TMEM, bf16 pairs) * V, 8 MMAs of 16 keys (2 KB of each half apart).
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_smem, bool acc) {
  const uint32_t vb = desc_lo(v_smem, kHalfBytes);
#define H3_PV(p, v, pred)                                                      \
  "add.u32 t, %1, " p ";\n\tadd.u32 y, %2, " v ";\n\tmov.b64 b, {y, %3};\n\t" \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %5, " pred ";\n\t"
  asm volatile(
      "{\n\t.reg .pred p0, p1, e;\n\telect.sync _|e, 0xffffffff;\n\t.reg .b64 b;\n\t.reg .b32 t, y;\n\t"
      "setp.ne.u32 p0, %4, 0;\n\tsetp.eq.u32 p1, %4, %4;\n\t"
      H3_PV("0", "0", "p0") H3_PV("8", "128", "p1") H3_PV("16", "256", "p1") H3_PV("24", "384", "p1")
      H3_PV("32", "512", "p1") H3_PV("40", "640", "p1") H3_PV("48", "768", "p1") H3_PV("56", "896", "p1")
      "}" ::"r"(d_tmem), "r"(p_tmem), "r"(vb), "r"(kDescHi), "r"(acc ? 1u : 0u), "r"(kIdescPV)
      : "memory");
#undef H3_PV
}

__device__ __forceinline__ void commit_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// Four lanes' four blocks of eight words, transposed: block k of lane i becomes lane k's block i.
__device__ __forceinline__ void transpose4(uint32_t (&w)[32], uint32_t lane) {
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    const bool upper = (lane & m) != 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & m) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t &x = w[8 * j + e], &y = w[8 * (j | m) + e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? x : y, m);
        if (upper) x = got;
        else y = got;
      }
    }
  }
}

// A sequence: its drafts [row0, row0 + T), context, key tiles, and items (key head, unit of up to two query tiles).
struct Doc {
  int32_t row0, T, ctx, tiles, qtiles, units;
};
__device__ __forceinline__ int32_t context(const TreeArgs& a, int32_t T, int32_t given) {
  const int64_t most = (int64_t)a.table_width * a.page_size - T;  // (not negative, and below 2^31: checked by the caller)
  return max(0, (int32_t)min((int64_t)given, most));
}
// (kOne, here and below: every item is a single query tile, which spares the divisions)
template <bool kOne>
__device__ __forceinline__ Doc make_doc(const TreeArgs& a, int32_t row0, int32_t row1, int32_t given) {
  Doc d;
  d.row0 = row0;
  d.T = row1 - row0;
  d.ctx = context(a, d.T, given);
  d.tiles = (int32_t)(((int64_t)d.ctx + d.T + kRows - 1) / kRows);
  // (T / toks rounded up: 65536 / toks rounded up is exact here, 191 toks < 65536)
  d.qtiles = kOne ? 1 : a.packs * (int32_t)((uint32_t)(d.T + a.toks - 1) * a.recip_toks >> 16);
  d.units = kOne ? 1 : (d.qtiles + 1) / 2;
  return d;
}
template <bool kOne>
__device__ __forceinline__ Doc doc_of(const TreeArgs& a, int b) {
  return make_doc<kOne>(a, __ldg(a.cu + b), __ldg(a.cu + b + 1), __ldg(a.ctx_lens + b));
}

// A block's share of one item: key tiles [lo, hi).
struct Piece {
  int32_t b, item, kvh, lo, hi;
  int32_t qt, n_qt;    // its first query tile, and how many (1 or 2)
  bool whole;
  bool first;          // of the block's pieces
  int32_t at;          // steps of the block before it
};
// Where a block's range begins (found once, for all roles).
struct Start {
  int32_t b, steps, kvh, unit, lo, row0, row1, given;
};
// Walks a block's range piece by piece; every role runs its own.
template <bool kOne>
struct Walk {
  int32_t b, kvh, unit, lo;
  int32_t left, at;
  int32_t item0;        // of all sequences' items, this one's first (set by the one role that wants it)
  bool first;
  Doc d;
  int32_t row2, given;  // of the next sequence: its end and length, on their way while this one runs
  __device__ void ahead(const TreeArgs& a) {
    const int n = min(b + 1, a.n_docs - 1);
    row2 = __ldg(a.cu + n + 1);
    given = __ldg(a.ctx_lens + n);
  }
  template <class S>
  __device__ void begin(const TreeArgs& a, const S& s) {
    b = s.b;
    left = s.steps;
    at = 0;
    first = true;
    kvh = s.kvh;
    unit = s.unit;
    item0 = 0;
    lo = s.lo;
    ahead(a);
    d = make_doc<kOne>(a, s.row0, s.row1, s.given);
  }
  // the next piece; false at the end
  __device__ bool next(const TreeArgs& a, Piece* p) {
    if (left <= 0) return false;
    if (kvh == a.kv_heads) {
      kvh = 0;
      item0 += a.kv_heads * d.units;
      ++b;
      d = make_doc<kOne>(a, d.row0 + d.T, row2, given);
      ahead(a);
    }
    p->b = b;
    p->item = item0 + (kOne ? kvh : kvh * d.units + unit);
    p->kvh = kvh;
    p->qt = kOne ? 0 : 2 * unit;
    p->n_qt = kOne ? 1 : min(2, d.qtiles - p->qt);
    p->lo = lo;
    p->hi = min(d.tiles, lo + left);
    p->whole = lo == 0 && p->hi == d.tiles;
    p->first = first;
    p->at = at;
    first = false;
    at += p->hi - lo;
    left -= p->hi - lo;
    lo = p->hi;
    if (lo == d.tiles) {
      lo = 0;
      if (kOne || ++unit == d.units) {
        unit = 0;
        ++kvh;
      }
    }
    return true;
  }
};

// A query tile's tokens and first head.
struct QTile {
  int32_t tok0, n_tok, head;
};
template <bool kOne>
__device__ __forceinline__ QTile q_tile(const TreeArgs& a, const Doc& d, int32_t kvh, int32_t qt) {
  if constexpr (kOne) return QTile{d.row0, d.T, kvh * a.group};
  const int32_t block = qt / a.packs, first = block * a.toks;
  return QTile{d.row0 + first, min(a.toks, d.T - first), kvh * a.group + (qt - block * a.packs) * a.pack};
}

// x / d for x < 2^24, d > 0, x / d < 2^22: the reciprocal's quotient is off by less than one before it is cut off.  (Ten instructions
// for the compiler's twenty-five: a block's first instructions take about ten cycles each, as they are fetched.)
__device__ __forceinline__ uint32_t div_small(uint32_t x, uint32_t d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"((float)d));
  const uint32_t q = (uint32_t)((float)x * r);
  const int32_t rest = (int32_t)(x - q * d);
  return rest < 0 ? q - 1 : rest >= (int32_t)d ? q + 1 : q;
}
// x / n, in 32 bits where they hold it.
__device__ __forceinline__ int64_t quotient(int64_t x, int32_t n) {
  return x < ((int64_t)1 << 32) ? (int64_t)((uint32_t)x / (uint32_t)n) : x / n;
}
// floor(total c / grid) for c <= grid < 2^16
__device__ __forceinline__ int64_t share_of(int64_t total, int64_t c, int64_t grid) {
  const int64_t q = quotient(total, (int32_t)grid), r = total - q * grid;
  return q * c + (uint32_t)(r * c) / (uint32_t)grid;
}

// kTwo: the two streams have ranges of their own (below, "more items than SMs").
template <bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = dev::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  if (sbase - raw > kSlack) {
    if (threadIdx.x == 0) atomicExch(a.err, kErrTimeout);  // (outputs are invalid)
    return;
  }
  unsigned char* smem = smem_raw + (sbase - raw);
  const Bars bars{sbase + kSmemBar};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmemMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kSmemMisc + 4);
  volatile Start* const starts = reinterpret_cast<volatile Start*>(smem + kSmemMisc + 8);  // of the block, or of each stream
  const uint32_t warp = dev::warp_id_uniform();
  const uint32_t lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;");  // (the join waits for this grid's end)
  if (warp == kKWarp && lane < 3) dev::tma_prefetch_desc(lane == 0 ? &tm_k : lane == 1 ? &tm_v : &tm_q);
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      dev::mbar_init(bars.q_full(i), 1);
      dev::mbar_init(bars.q_empty(i), 1);
      dev::mbar_init(bars.s_ready(i), 1);
      dev::mbar_init(bars.p_ready(i), 4);
      dev::mbar_init(bars.pv_done(i), 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      dev::mbar_init(bars.full(i), 1);
      dev::mbar_init(bars.empty(i), 1);
    }
    dev::mbar_init(bars.drain(), 1);
    dev::mbar_init(bars.joined(), 8);
    dev::fence_barrier_init();
  }

  if (a.pack * a.toks < kRows) {
    // rows of a query tile that no load fills (their scores must not be anything: see attn_fwd_tc.cu)
    for (uint32_t i = threadIdx.x * 16u; i < 2 * kTileBytes; i += kThreads * 16u)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sbase + kSmemQ + i), "r"(0u) : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();  // the barriers are set
  if (warp == kMmaWarp) {
    dev::tmem_alloc(dev::smem_u32(tmem_slot), kTmemCols);
    dev::tmem_relinquish();
  }

  // What this block does.
  constexpr int kParts = kTwo ? 2 : 1;
  int64_t s0[kParts], s1[kParts];  // steps (pieces) of the block, or steps of each stream
  int64_t total = 0;               // of all
  int32_t most = 0;                // tiles of a piece; 0: ranges
  bool work = false;
  Start own = {};                  // of the block (kTwo: starts, of each stream)
  if (!kTwo && a.by_warp) {
    // Few items, each below 2^21 tiles: every warp adds up the sequences and finds the block's piece by itself.
    const int per = (a.n_docs + 31) / 32, b0 = min((int)lane * per, a.n_docs), b1 = min(b0 + per, a.n_docs);
    Doc d0 = {};  // (the lane's sequence, where there is one to a lane)
    uint32_t tiles = 0;
    for (int b = b0; b < b1; ++b) {
      d0 = doc_of<kTwo>(a, b);
      tiles += (uint32_t)(d0.tiles * d0.units * a.kv_heads);
    }
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    // About the even share and three lengths above it, which are quicker than a second piece: up to three tiles more,
    // or, where an item is one query tile, up to a quarter (memory sets the time, and a block can take more than its
    // share of it: 16 sequences of 5,033 tokens, 128 items of 40 tiles, 57.9 against 60.3 us; up to five eighths was
    // slower, 12 of 20,423 tokens 184 for 155).  The pieces of each, 16 bits for each (not much above twice the blocks).
    const uint32_t share = max(1u, (uint32_t)((float)(tiles + gridDim.x - 1) * a.inv_grid));
    const uint32_t more = a.slot_rows == kRows ? share / 8 : 0;
    const auto length = [&](int i) { return share + max((uint32_t)i, min(i, 2) * more); };
    uint32_t pieces[2] = {0, 0};
    for (int b = b0; b < b1; ++b) {
      const Doc d = per == 1 ? d0 : doc_of<kTwo>(a, b);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pieces[i >> 1] += (uint32_t)(d.units * a.kv_heads) * div_small((uint32_t)d.tiles + length(i) - 1, length(i)) << 16 * (i & 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) pieces[i] = __reduce_add_sync(0xffffffffu, pieces[i]);
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const uint32_t n = pieces[i >> 1] >> 16 * (i & 1) & 0xffff;
      if (n <= gridDim.x) {
        most = (int32_t)length(i);
        total = n;
      }
    }
    if (most > 0) {
      uint32_t mine = 0;
      for (int b = b0; b < b1; ++b) {
        const Doc d = per == 1 ? d0 : doc_of<kTwo>(a, b);
        mine += (uint32_t)(d.units * a.kv_heads) * div_small((uint32_t)(d.tiles + most - 1), (uint32_t)most);
      }
      uint32_t from = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, from, o);
        if ((int)lane >= o) from += x;
      }
      from -= mine;
      const uint32_t c = blockIdx.x;
      s0[0] = c;
      s1[0] = c + 1;
      work = c < (uint32_t)total;
      bool here = false;
      for (int b = b0; b < b1; ++b) {
        const Doc d = per == 1 ? d0 : doc_of<kTwo>(a, b);
        const uint32_t cut = div_small((uint32_t)(d.tiles + most - 1), (uint32_t)most);  // pieces of an item
        const uint32_t n = cut * (uint32_t)(d.units * a.kv_heads);
        if (c - from < n) {  // (c >= from, or the difference is large)
          const uint32_t item = div_small(c - from, cut), i = c - from - item * cut;
          const uint32_t size = div_small((uint32_t)d.tiles, cut), rest = (uint32_t)d.tiles - size * cut;  // the first `rest` have one more
          const int32_t kvh = (int32_t)div_small(item, (uint32_t)d.units);
          own = Start{b, (int32_t)(size + (i < rest)), kvh, (int32_t)item - kvh * d.units, (int32_t)(size * i + min(i, rest)),
                      d.row0, d.row0 + d.T, d.ctx};
          here = true;
        }
        from += n;
      }
      const int src = max(0, __ffs((int)__ballot_sync(0xffffffffu, here)) - 1);
      own = Start{__shfl_sync(0xffffffffu, own.b, src),    __shfl_sync(0xffffffffu, own.steps, src),
                  __shfl_sync(0xffffffffu, own.kvh, src),  __shfl_sync(0xffffffffu, own.unit, src),
                  __shfl_sync(0xffffffffu, own.lo, src),   __shfl_sync(0xffffffffu, own.row0, src),
                  __shfl_sync(0xffffffffu, own.row1, src), __shfl_sync(0xffffffffu, own.given, src)};
    } else {  // ranges after all
      int64_t mine = 0;
      for (int b = b0; b < b1; ++b) {
        const Doc d = per == 1 ? d0 : doc_of<kTwo>(a, b);
        mine += (int64_t)d.tiles * d.units * a.kv_heads;
      }
      int64_t from = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, from, o);
        if ((int)lane >= o) from += x;
      }
      from -= mine;
      total = tiles;
      const int64_t c = blockIdx.x, parts = min((int64_t)gridDim.x, total);
      s0[0] = s1[0] = -1;
      if (c < parts) {
        s0[0] = share_of(total, c, parts);
        s1[0] = share_of(total, c + 1, parts);
      }
      work = s0[0] < s1[0];
      bool here = false;
      for (int b = b0; b < b1; ++b) {
        const Doc d = per == 1 ? d0 : doc_of<kTwo>(a, b);
        const int64_t n = (int64_t)d.tiles * d.units * a.kv_heads;
        if (s0[0] >= from && s0[0] < from + n) {
          const int32_t item = (int32_t)((uint32_t)(s0[0] - from) / (uint32_t)d.tiles), kvh = item / d.units;
          own = Start{b, (int32_t)(s1[0] - s0[0]), kvh, item - kvh * d.units, (int32_t)((s0[0] - from) - (int64_t)item * d.tiles),
                      d.row0, d.row0 + d.T, d.ctx};
          here = true;
        }
        from += n;
      }
      const int src = max(0, __ffs((int)__ballot_sync(0xffffffffu, here)) - 1);
      own = Start{__shfl_sync(0xffffffffu, own.b, src),    __shfl_sync(0xffffffffu, own.steps, src),
                  __shfl_sync(0xffffffffu, own.kvh, src),  __shfl_sync(0xffffffffu, own.unit, src),
                  __shfl_sync(0xffffffffu, own.lo, src),   __shfl_sync(0xffffffffu, own.row0, src),
                  __shfl_sync(0xffffffffu, own.row1, src), __shfl_sync(0xffffffffu, own.given, src)};
    }
    if (blockIdx.x == 0 && warp == 0)
      for (int b = b0; b < b1; ++b) {
        const int32_t given = __ldg(a.ctx_lens + b);
        if (context(a, __ldg(a.cu + b + 1) - __ldg(a.cu + b), given) != given) dev::report_bad_page(a.err);
      }
  } else {
    // Every thread adds up a run of sequences; the one that finds the block's first step in its own tells all.
    const int per = (a.n_docs + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, a.n_docs), b1 = min(b0 + per, a.n_docs);
    int64_t* const sums = reinterpret_cast<int64_t*>(smem + kSmemMl);
    Doc d0 = {};  // (the thread's sequence, where there is one to a thread)
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
      d0 = doc_of<kTwo>(a, b);
      mine += (int64_t)d0.tiles * d0.units * a.kv_heads;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if ((int)lane >= o) incl += x;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < (int)warp) before += sums[w];
      total += sums[w];
    }
    const int64_t parts = min((int64_t)gridDim.x * kParts, total);
#pragma unroll
    for (int x = 0; x < kParts; ++x) {
      const int64_t c = (int64_t)blockIdx.x * kParts + x;
      s0[x] = s1[x] = -1;
      if (c < parts) {
        s0[x] = share_of(total, c, parts);
        s1[x] = share_of(total, c + 1, parts);
        if (s1[x] - s0[x] > INT32_MAX / 4) {  // (thousands of lengths near 2^31: more than the ring's counters hold)
          if (threadIdx.x == 0) dev::report_bad_page(a.err);
          s0[x] = s1[x] = -1;
        }
      }
      work = work || s0[x] < s1[x];
      if (threadIdx.x == 0 && s0[x] == s1[x]) starts[x].steps = 0;
    }
    for (int b = b0; b < b1; ++b) {
      const Doc d = per == 1 ? d0 : doc_of<kTwo>(a, b);
      const int64_t n = (int64_t)d.tiles * d.units * a.kv_heads;
#pragma unroll
      for (int x = 0; x < kParts; ++x)
        if (s0[x] >= before && s0[x] < before + n) {
          volatile Start& start = starts[x];
          const int32_t item = (int32_t)quotient(s0[x] - before, d.tiles);
          const int32_t kvh = kTwo ? item : (int32_t)((uint32_t)item / (uint32_t)d.units);
          start.b = b;
          start.kvh = kvh;
          start.unit = kTwo ? 0 : item - kvh * d.units;
          start.lo = (int32_t)((s0[x] - before) - (int64_t)item * d.tiles);
          start.steps = (int32_t)(s1[x] - s0[x]);
          start.row0 = d.row0;
          start.row1 = d.row0 + d.T;
          start.given = d.ctx;
        }
      if (blockIdx.x == 0 && __ldg(a.ctx_lens + b) != d.ctx) dev::report_bad_page(a.err);
      before += n;
    }
    __syncthreads();
    if (!kTwo && work)
      own = Start{starts[0].b,  starts[0].steps, starts[0].kvh,  starts[0].unit,
                  starts[0].lo, starts[0].row0,  starts[0].row1, starts[0].given};
  }
  const int64_t grid = min((int64_t)gridDim.x * kParts, total);  // (blocks, or streams, that have steps)
  uint32_t tmem = 0;
  if (warp <= kMmaWarp) {  // (softmax and issuer: tensor memory is allocated)
    dev::tc_fence_before();
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * (kMmaWarp + 1)) : "memory");
    dev::tc_fence_after();
    tmem = *tmem_slot;
  }
  // tiles of the block, in the order of the ring: of two ranges one tile each in turn, the longer range's first
  const int32_t of0 = !work ? 0 : kTwo ? starts[0].steps : own.steps, of1 = kTwo && work ? starts[1].steps : 0;
  const int32_t steps = of0 + of1;
  const int lead = kTwo && of1 > of0 ? 1 : 0;  // the stream that begins
  Walk<kTwo> walk;
  Piece p;
  if (!kTwo && work) walk.begin(a, own);
  // The end of every role: all of them are here.  True where one gave up (none does any more); what the others have
  // on its way, whether they noticed or not, then has to land, or end, before the block's memory goes: bounded waits.
  // (Each role has the barrier and its waits at its own end: behind one barrier for all, with what is on its way noted in
  // shared memory, 512 sequences of 300 tokens took 117 to 121 us for 113, 16 trees of 16 drafts 26.9 for 27.1.)
  const auto stopped = [&] {
    dev::tc_fence_before();
    asm volatile("barrier.cta.sync 0;" ::: "memory");
    return *abort_flag != 0;
  };
  const auto landed = [&](uint32_t bar, uint32_t parity) { dev::mbar_wait_bounded(bar, parity & 1, nullptr, nullptr, kTimeoutNs); };

  if (!work) {
    stopped();  // (more blocks than steps)
  } else if (warp == kKWarp || warp == kVWarp) {
    // ---------------- K tiles, V tiles; kTwo: K and V of stream 0, of stream 1 ----
    const int me = warp == kVWarp ? 1 : 0;
    if constexpr (kTwo) {
      if (starts[me].steps > 0) walk.begin(a, starts[me]);
      else walk.left = 0;
    }
    // (kept in L2 instead, tiles that a second unit reads too gain nothing and push the partial rows out of it:
    // 282 against 276 us for 64 drafts over 20,423 tokens)
    const uint64_t pol = dev::policy_evict_first();
    const int n_box = a.n_box;                   // boxes of a tile, a lane each
    const int32_t tiles_at_once = a.at_once;
    const uint32_t dst0 = sbase + kSmemKV + lane * (uint32_t)a.box * 128u;
    int32_t issued = 0;                          // copies of this warp
    const auto entry_of = [&](int32_t c) { return ring::copy_entry<kTwo>(c, me, me ^ lead, steps); };
    uint32_t entry = entry_of(0);                // the one that comes next
    bool ok = true, free = entry < kSlots;       // (the first five entries' slots are)
    // one tile's copies into the entry, and a first look at the slot of the next one
    const auto load = [&](const CUtensorMap* tm, bool in, int32_t page, int32_t c1, int32_t c2, uint32_t bytes) {
      const uint32_t slot = entry % kSlots, bar = bars.full(slot);
      if (!__all_sync(0xffffffffu, free)) {
        // (asked again and again before the bounded wait, whose call costs some 400 cycles: 141 against 126 us for
        // 512 sequences of 300 tokens; softmax warps that wait so take the other stream's issue slots, 265 against 271 us
        // for 64 drafts over 20,423 tokens)
        bool good = false;
#pragma unroll 1
        for (int i = 0; i < 64 && !good; ++i) good = __all_sync(0xffffffffu, dev::mbar_test_wait(bars.empty(slot), ((entry / kSlots) & 1) ^ 1));
        if (!good) {
          if (lane == 0) good = dev::mbar_wait(bars.empty(slot), ((entry / kSlots) & 1) ^ 1, abort_flag, a.err, kTimeoutNs);
          ok = __shfl_sync(0xffffffffu, good, 0);
        }
        if (!ok) return;
      }
      if (lane == 0) dev::mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      const uint32_t next = entry_of(++issued);
      entry = next;
      free = dev::mbar_test_wait(bars.empty(next % kSlots), ((next / kSlots) & 1) ^ 1);
      if (in) {
        const uint32_t dst = dst0 + slot * kTileBytes;
        dev::tma_load_4d(dst, tm, bar, 0, c1, c2, page, pol);
        dev::tma_load_4d(dst + kHalfBytes, tm, bar, 64, c1, c2, page, pol);
      }
    };
    while (ok && walk.next(a, &p)) {
      const int32_t total = walk.d.ctx + walk.d.T;
      const int32_t* table = a.page_table + (int64_t)p.b * a.table_width;
      // Page numbers a window of 32 boxes at a time, a lane each, the next window on
      // its way (a lookup a tile, though asked for a tile ahead, paced the loads: 1,000 cycles a tile).
      const auto box_page = [&](uint32_t i) { return (uint32_t)((uint64_t)i * a.page_mul >> a.page_shift); };
      const auto pages_from = [&](int32_t t) {
        const uint32_t i = (uint32_t)t * n_box + lane;  // (below 2^28 + 32)
        return (int64_t)i * a.box < total ? __ldg(table + box_page(i)) : 0;
      };
      int32_t pages = pages_from(p.lo), pages_next = pages_from(p.lo + tiles_at_once), window = p.lo;
      const uint32_t first = (uint32_t)p.lo * n_box + lane;
      int32_t row = (int32_t)((first - box_page(first) * (uint32_t)a.page_boxes) * (uint32_t)a.box);  // in its page
      for (int32_t t = p.lo; t < p.hi; ++t) {
        if (t - window == tiles_at_once) {
          window = t;
          pages = pages_next;
          pages_next = pages_from(t + tiles_at_once);
        }
        const uint32_t key = (uint32_t)t * kRows + lane * (uint32_t)a.box;
        const bool in = (int)lane < n_box && key < (uint32_t)total;
        int32_t page = __shfl_sync(0xffffffffu, pages, (t - window) * n_box + (int)lane & 31);
        if (in && (uint32_t)page >= (uint32_t)a.n_pages) {
          dev::report_bad_page(a.err);
          page = a.n_pages;  // outside the tensor map: zeros
        }
        const int32_t c1 = a.heads_first ? p.kvh : row, c2 = a.heads_first ? row : p.kvh;
        const uint32_t bytes = (uint32_t)min(n_box, (total - t * kRows + a.box - 1) / a.box) * (uint32_t)a.box * 256u;
        if constexpr (kTwo) {
          load(&tm_k, in, page, c1, c2, bytes);
          if (ok) load(&tm_v, in, page, c1, c2, bytes);
        } else {
          load(me == 1 ? &tm_v : &tm_k, in, page, c1, c2, bytes);
        }
        if (!ok) break;
        row += a.row_step;
        if (row >= a.page_size) row -= a.page_size;
      }
    }
    __syncwarp();
    if (stopped() && lane == 0) {
#pragma unroll 1
      for (int32_t c = ring::first_on_its_way(issued); c < issued; ++c) {
        const uint32_t e = entry_of(c);
        landed(bars.full(e % kSlots), e / kSlots);
      }
    }
  } else if (warp == kQWarp) {
    // ----------------------------------------------------------- Q tiles ----
    uint32_t n[2] = {0, 0};  // loads into each slot
    if (lane == 0) {
      const uint64_t pol = dev::policy_evict_first();
      bool ok = true;
      const auto load = [&](const QTile& q, uint32_t slot) {
        const uint32_t dst = sbase + kSmemQ + slot * kTileBytes, bar = bars.q_full(slot);
        dev::mbar_arrive_expect_tx(bar, 256u * (uint32_t)(a.pack * a.toks));
        dev::tma_load_3d(dst, &tm_q, bar, 0, q.head, q.tok0, pol);
        dev::tma_load_3d(dst + kHalfBytes, &tm_q, bar, 64, q.head, q.tok0, pol);
      };
      // an item that begins with piece y of block (stream) c, whose steps begin at `begin`: its first slot and
      // its pieces, for the join
      const auto note = [&](const Piece& y, int32_t tiles, int64_t c, int64_t begin) {
        if (y.lo != 0) return;
        int64_t pieces = 1;
        if (most > 0)
          pieces = ((uint32_t)tiles + most - 1) / (uint32_t)most;
        else if (y.hi < tiles)  // block (stream) c has steps [total c / grid, total (c + 1) / grid)
          pieces = ((begin + y.at + tiles) * grid - 1) / total - c + 1;
        a.joins[y.item] = make_int2((int32_t)(2 * c) + (y.first ? 0 : 1), (int32_t)pieces);
      };
      if constexpr (kTwo) {
        // A slot to each stream.  One thread serves whichever is free: a wait for one stream's slot would
        // hold up the other's, whose next piece may come first.  (Two lanes, a stream each, would wait
        // for one another at the end of every wait.)
        Walk<kTwo> w[2];
        Piece y[2];
        bool live[2];
        uint32_t idle = 0;
        uint64_t since = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          live[x] = starts[x].steps > 0;
          if (live[x]) {
            w[x].begin(a, starts[x]);
            w[x].item0 = __ldg(a.item0 + w[x].b);
            live[x] = w[x].next(a, &y[x]);
          }
        }
        while (ok && (live[0] || live[1])) {
          bool any = false;
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (live[x] && dev::mbar_test_wait(bars.q_empty(x), (n[x] & 1) ^ 1)) {
              note(y[x], w[x].d.tiles, 2 * (int64_t)blockIdx.x + x, s0[kTwo ? x : 0]);
              load(q_tile<kTwo>(a, w[x].d, y[x].kvh, y[x].qt), (uint32_t)x);
              ++n[x];
              live[x] = w[x].next(a, &y[x]);
              any = true;
            }
          if (any) {
            idle = 0;
          } else {
            __nanosleep(20);
            if ((++idle & 15u) == 0) {  // bounded: two seconds of nothing, or another thread's abort
              const uint64_t now = dev::globaltimer_ns();
              if (idle == 16) since = now;
              ok = *abort_flag == 0;
              if (ok && now - since > kTimeoutNs) {
                *abort_flag = 1;
                atomicExch(a.err, kErrTimeout);
                ok = false;
              }
            }
          }
        }
      } else {
        uint32_t all = 0;
        walk.item0 = __ldg(a.item0 + walk.b);
        while (ok && walk.next(a, &p)) {
          note(p, walk.d.tiles, blockIdx.x, s0[0]);
          for (int i = 0; ok && i < p.n_qt; ++i) {
            ok = dev::mbar_wait(bars.q_empty(all & 1), ((all >> 1) & 1) ^ 1, abort_flag, a.err, kTimeoutNs);
            if (!ok) break;
            load(q_tile<kTwo>(a, walk.d, p.kvh, p.qt + i), all & 1);
            ++all;
          }
        }
        n[0] = (all + 1) / 2;
        n[1] = all / 2;
      }
    }
    __syncwarp();
    if (stopped() && lane == 0) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (n[x]) landed(bars.q_full(x), n[x] - 1);
    }
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------- MMA issuer ----
    // (the whole warp; one lane polls, one elected lane issues)
    // The operands of an MMA are uniform registers: ring positions are counted up from constants here, and what
    // a piece says goes through uniform(), so that no value has to be moved there before each instruction.
    const auto uniform = [](uint32_t x) { return __reduce_or_sync(0xffffffffu, x); };
    const uint32_t tm = uniform(tmem);
    uint32_t n_q = 0, p_it[2] = {0, 0};  // query tiles; key tiles of each stream whose P was awaited
    // slot and phase of the next K and V to come: K of tile t is entry 0, 1, 3, 5, .., V 2, 4, 6, .. (the last one
    // of the block comes an entry early)
    uint32_t k_slot = 0, k_ph = 0, v_slot = 2, v_ph = 0;
    bool k_first = true;
    int32_t tile = 0;                    // of the block
    const int32_t all = (int32_t)uniform((uint32_t)steps);
    bool ok = true, issued = false;
    const auto wait = [&](uint32_t bar, uint32_t parity) {
      bool good = false;
#pragma unroll 1
      for (int i = 0; i < 256 && !good; ++i) good = __all_sync(0xffffffffu, dev::mbar_test_wait(bar, parity));
      if (!good) {
        if (lane == 0) good = dev::mbar_wait(bar, parity, abort_flag, a.err, kTimeoutNs);
        ok = __shfl_sync(0xffffffffu, good, 0) && ok;
      }
      dev::tc_fence_after();
    };
    const auto next_k = [&] {
      const uint32_t step = k_first ? 1 : 2;
      k_first = false;
      k_slot += step;
      if (k_slot >= kSlots) {
        k_slot -= kSlots;
        k_ph ^= 1;
      }
    };
    const auto next_v = [&] {
      ++tile;
      v_slot += tile + 1 < all ? 2 : 1;
      if (v_slot >= kSlots) {
        v_slot -= kSlots;
        v_ph ^= 1;
      }
    };
    if (all == 1) v_slot = 1;
    const auto qk = [&](int s, uint32_t q, uint32_t slot) {
      issue_qk(tm + s * 128, sbase + kSmemQ + q * kTileBytes, sbase + kSmemKV + slot * kTileBytes);
      commit_elect(bars.s_ready(s));
    };
    // Asking a barrier takes 200 cycles, a wait that finds it complete too.  So each is asked before the
    // products of the step before it are issued, and waited for only if it was not complete then.
    const auto ask = [&](uint32_t bar, uint32_t parity) { return dev::mbar_test_wait(bar, parity); };
    const auto need = [&](bool asked, uint32_t bar, uint32_t parity) {
      if (!__all_sync(0xffffffffu, asked)) wait(bar, parity);
    };
    bool p_asked = false, v_asked = false, k_asked = false;
    [[maybe_unused]] bool k_ready = false;
    const auto ask_p = [&](int s, uint32_t it) { p_asked = ask(bars.p_ready(s), it & 1); };
    // asks for the V and K behind the next ones (more_v, more_k: whether they are this block's, this piece's)
    const auto ask_tiles = [&](bool more_v, bool more_k) {
      uint32_t slot = v_slot + 2, ph = v_ph;
      if (slot >= kSlots) slot -= kSlots, ph ^= 1;
      v_asked = ask(bars.full(slot), ph) && more_v;
      slot = k_slot + 2, ph = k_ph;
      if (slot >= kSlots) slot -= kSlots, ph ^= 1;
      k_asked = ask(bars.full(slot), ph) && more_k;
    };
    // stream s's key tile: its PV, then the next tile's QK into the same columns, or the piece's end; `then`
    // asks for what comes next
    const auto step = [&](int s, bool acc, bool more, uint32_t q, auto then) {
      need(p_asked, bars.p_ready(s), p_it[s] & 1);
      if (!ok) return;
      dev::tc_fence_after();
      then();
      issue_pv(tm + 256 + s * 128, tm + s * 128, sbase + kSmemKV + v_slot * kTileBytes, acc);
      if (more)
        qk(s, q, k_slot);
      else
        commit_elect(bars.pv_done(s));
      ++p_it[s];
    };
    if constexpr (kTwo) {
      // Stream lead ^ x is x's; its tiles are the block's x, x + 2, ..  At a piece's end "PV done", and the next
      // QK is the next piece's first, of a Q that was loaded while its last tile was in work.
      Walk<kTwo> w[2];
      int32_t left[2] = {0, 0}, done[2] = {0, 0};  // tiles of the piece to go and behind
      uint32_t qs[2] = {0, 0};
      const uint32_t ld = uniform((uint32_t)lead);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x >= all) break;
        const uint32_t st = ld ^ x;
        w[x].begin(a, starts[st]);
        w[x].next(a, &p);
        left[x] = (int32_t)uniform((uint32_t)(p.hi - p.lo));
        wait(bars.q_full(st), 0);
        ++qs[x];
        wait(bars.full(k_slot), k_ph);
        if (!ok) break;
        issued = true;
        qk(st, st, k_slot);
        commit_elect(bars.empty(k_slot));
        next_k();
        if (left[x] == 1) commit_elect(bars.q_empty(st));
      }
#pragma unroll 1
      for (int32_t t0 = 0; ok && t0 < all; t0 += 2)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int32_t t = t0 + x;
          if (!ok || t >= all) break;
          const uint32_t st = ld ^ x;
          need(v_asked, bars.full(v_slot), v_ph);
          need(p_asked, bars.p_ready(st), p_it[x] & 1);
          if (!ok) break;
          dev::tc_fence_after();
          p_asked = ask(bars.p_ready(st ^ 1), p_it[x ^ 1] & 1);
          const bool more = t + 2 < all;
          ask_tiles(tile + 2 < all, t + 3 < all);
          issue_pv(tm + 256 + st * 128, tm + st * 128, sbase + kSmemKV + v_slot * kTileBytes, done[x] > 0);
          ++p_it[x];
          ++done[x];
          if (--left[x] == 0) {
            commit_elect(bars.pv_done(st));
            done[x] = 0;
            if (more) {
              w[x].next(a, &p);
              left[x] = (int32_t)uniform((uint32_t)(p.hi - p.lo));
              wait(bars.q_full(st), qs[x] & 1);
              ++qs[x];
            }
          }
          if (more) {
            // (what was asked of K concerns the tile behind this one)
            if (!(k_ready && t0 > 0)) wait(bars.full(k_slot), k_ph);
            if (!ok) break;
            qk(st, st, k_slot);
            if (left[x] == 1) commit_elect(bars.q_empty(st));
          }
          commit_elect(bars.empty(v_slot));
          next_v();
          if (more) {
            commit_elect(bars.empty(k_slot));
            next_k();
          }
          k_ready = __all_sync(0xffffffffu, k_asked);
        }
    }
    while (!kTwo && ok && walk.next(a, &p)) {
      const int32_t n = (int32_t)uniform((uint32_t)(p.hi - p.lo));
      const bool two = uniform((uint32_t)p.n_qt) == 2;
      p_asked = v_asked = k_asked = false;
      const uint32_t q0 = n_q & 1, q1 = q0 ^ 1;
      wait(bars.q_full(q0), (n_q >> 1) & 1);
      ++n_q;
      if (two) {
        // stream s: query tile s over every key tile
        wait(bars.q_full(q1), (n_q >> 1) & 1);
        ++n_q;
        wait(bars.full(k_slot), k_ph);
        if (!ok) break;
        issued = true;
        qk(0, q0, k_slot);
        qk(1, q1, k_slot);
        commit_elect(bars.empty(k_slot));
        next_k();
        if (n == 1) {
          commit_elect(bars.q_empty(q0));
          commit_elect(bars.q_empty(q1));
        }
#pragma unroll 1
        for (int32_t j = 0; ok && j < n; ++j) {
          const bool more = j + 1 < n;
          need(v_asked, bars.full(v_slot), v_ph);
          if (more) need(k_asked, bars.full(k_slot), k_ph);
          if (!ok) break;
          step(0, j > 0, more, q0, [&] { ask_p(1, p_it[1]); });
          if (ok) step(1, j > 0, more, q1, [&] {
            ask_p(0, p_it[0]);
            ask_tiles(tile + 2 < all, j + 2 < n);
          });
          if (!ok) break;
          commit_elect(bars.empty(v_slot));
          next_v();
          if (more) {
            commit_elect(bars.empty(k_slot));
            next_k();
          }
          if (j + 2 == n) {
            commit_elect(bars.q_empty(q0));
            commit_elect(bars.q_empty(q1));
          }
        }
      } else {
        // stream s: the one query tile over the key tiles s, s + 2, ...
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (s >= n) break;
          wait(bars.full(k_slot), k_ph);
          if (!ok) break;
          issued = true;
          qk(s, q0, k_slot);
          commit_elect(bars.empty(k_slot));
          next_k();
        }
        if (!ok) break;
        if (n <= 2) commit_elect(bars.q_empty(q0));
#pragma unroll 1
        for (int32_t j0 = 0; ok && j0 < n; j0 += 2)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int32_t j = j0 + s;
            if (!ok || j >= n) break;
            const bool more = j + 2 < n;
            need(v_asked, bars.full(v_slot), v_ph);
            if (more) need(k_asked, bars.full(k_slot), k_ph);
            if (!ok) break;
            step(s, j0 > 0, more, q0, [&] {
              ask_p(s ^ 1, p_it[s ^ 1]);
              ask_tiles(tile + 2 < all, j + 3 < n);
            });
            if (!ok) break;
            commit_elect(bars.empty(v_slot));
            next_v();
            if (more) {
              commit_elect(bars.empty(k_slot));
              next_k();
            }
            if (j + 3 == n) commit_elect(bars.q_empty(q0));
          }
      }
    }
    __syncwarp();
    if (stopped() && issued) {  // every MMA issued so far must finish before TMEM is freed
      commit_elect(bars.drain());
      landed(bars.drain(), 0);
    }
  } else {
    // ----------------------------------------------------------- softmax ----
    const int st = warp >> 2;                     // stream
    const uint32_t row = threadIdx.x & 127;       // TMEM lane, row of the query tile
    const uint32_t lane_base = (warp & 3) * 32;
    const uint32_t t_s = tmem + (lane_base << 16) + st * 128;
    const uint32_t t_o = tmem + (lane_base << 16) + 256;  // O_0; O_1 128 columns on
    float2* const ml_of = reinterpret_cast<float2*>(smem + kSmemMl);
    const uint32_t tok_in = row * a.recip >> 16, sub = row - tok_in * (uint32_t)a.pack;
    uint32_t s_it = 0, done[2] = {0, 0}, joined = 0;  // pieces in which each stream had a tile
    bool ok = true;
    // stream s's last PV of the piece
    const auto finished = [&](int s) {
      ok = dev::mbar_wait(bars.pv_done(s), (s == 0 ? done[0] : done[1]) & 1, abort_flag, a.err, kTimeoutNs) && ok;
    };
    // What a piece is to this row; looked up before the epilogue of the one before it, so that the
    // drafts that the row sees are here when its first tile is (of a short context the only one).
    struct Mine {
      QTile q;
      uint64_t mask;
      int32_t ctx, T;
      bool valid, busy;  // the row is one; any of this warp's is
    };
    const auto look = [&](const Piece& y) {
      Mine x;
      x.q = q_tile<kTwo>(a, walk.d, y.kvh, y.qt + (!kTwo && y.n_qt == 2 ? st : 0));
      x.ctx = walk.d.ctx;
      x.T = walk.d.T;
      x.valid = tok_in < (uint32_t)x.q.n_tok;  // (rows past pack * toks have larger tok_in)
      x.busy = (int32_t)(lane_base * a.recip >> 16) < x.q.n_tok;
      x.mask = 0;
      if (x.valid)
        x.mask = a.tree_mask != nullptr
                     ? __ldg(reinterpret_cast<const unsigned long long*>(a.tree_mask) + x.q.tok0 + (int32_t)tok_in)
                     : ~0ull >> (63 - (x.q.tok0 + (int32_t)tok_in - walk.d.row0));
      return x;
    };
    if constexpr (kTwo) {
      if (starts[st].steps > 0) walk.begin(a, starts[st]);
      else walk.left = 0;
    }
    Piece p_next;
    bool go = walk.next(a, &p_next);
    Mine next{};
    if (go) next = look(p_next);
    while (ok && go) {
      p = p_next;
      const Mine me = next;
      const bool two = kTwo || p.n_qt == 2;  // the stream has the rows to itself
      const QTile& q = me.q;
      const bool valid = me.valid, busy = me.busy;
      const int32_t n = p.hi - p.lo;
      float m = kLowest, l = 0.f;
      for (int32_t j = two ? 0 : st; ok && j < n; j += two ? 1 : 2) {
        const int32_t t = p.lo + j;
        ok = dev::mbar_wait(bars.s_ready(st), s_it & 1, abort_flag, a.err, kTimeoutNs);
        ++s_it;
        __syncwarp();  // lanes leave the wait separately; the TMEM loads are warp-collective
        dev::tc_fence_after();
        if (busy) {
          const int32_t base = t * kRows - me.ctx;  // draft of the tile's first key (negative: context)
          const bool edge = base + kRows > 0;
          uint64_t see[2] = {~0ull, 0};            // keys that the row sees
          if (edge) {
            const uint64_t word = me.mask & (~0ull >> (64 - me.T));
            if (base >= 0) {
              see[0] = word >> base;               // (the last tile begins before the last draft: below 64)
            } else if (base > -64) {
              see[0] = (word << -base) | ((1ull << -base) - 1);
              see[1] = word >> (64 + base);
            } else if (base == -64) {
              see[1] = word;
            } else {
              see[1] = (word << (-base - 64)) | ((1ull << (-base - 64)) - 1);
            }
          }
          // Half of the tile's scores, 64 keys, at a time, each a step of the online softmax: its maximum, then its
          // weights over the first half's columns.  A reference that the second half moves scales the first
          // half's weights where they lie, exactly: references are whole numbers, so alpha is a power of two.
          // (All 128 scores at once spilled to local memory, of which little stays close when shared memory
          // takes most of L1: 4.3 us a step for 1.4.  A loop as it is, not unrolled: a block that has a few
          // tiles fetches every instruction once.)
          float alpha = 1.f;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t r[2][32];
            dev::tmem_ld32(t_s + 64 * h, r[0]);
            dev::tmem_ld32(t_s + 64 * h + 32, r[1]);
            dev::tmem_wait_ld();
            float sv[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) sv[c] = __uint_as_float(r[c >> 5][c & 31]);
            if (edge) {
              const uint64_t half = h == 0 ? see[0] : see[1];
              const uint32_t w[2] = {(uint32_t)half, (uint32_t)(half >> 32)};
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (!((w[c >> 5] >> (c & 31)) & 1u)) sv[c] = -INFINITY;
            }
            float mx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[i] = dev::max3(sv[i], sv[8 + i], sv[16 + i]);
#pragma unroll
            for (int c = 24; c < 56; c += 16)
#pragma unroll
              for (int i = 0; i < 8; ++i) mx[i] = dev::max3(mx[i], sv[c + i], sv[c + 8 + i]);
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[i] = fmaxf(mx[i], sv[56 + i]);
            const float m_new =
                dev::max3(dev::max3(mx[0], mx[1], mx[2]), dev::max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * a.scale_log2;
            if (__any_sync(0xffffffffu, m_new > m + kRescale)) {
              float beta = 1.f;
              if (m_new > m + kRescale) {
                const float up = ceilf(m_new);
                beta = dev::ex2_approx(m - up);
                m = up;
              }
              alpha *= beta;
              l *= beta;
              if (h == 1) {
                uint32_t pr[32];
                dev::tmem_wait_st();
                dev::tmem_ld32(t_s, pr);
                dev::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  pr[c] = dev::pack_bf16x2(__uint_as_float(pr[c] << 16) * beta, __uint_as_float(pr[c] & 0xffff0000u) * beta);
                dev::tmem_st32(t_s, pr);
              }
            }
            const float neg = -m;
            float rs8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            uint32_t pr[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              float x0, x1;
              dev::fma2(x0, x1, sv[2 * c], sv[2 * c + 1], a.scale_log2, a.scale_log2, neg, neg);
              const float p0 = dev::ex2_approx(x0), p1 = dev::ex2_approx(x1);
              const int ai = 2 * (c & 3);
              dev::add2(rs8[ai], rs8[ai + 1], rs8[ai], rs8[ai + 1], p0, p1);
              // bf16, as the operand of the tensor cores: half a step of each weight, the sum keeps fp32
              pr[c] = dev::pack_bf16x2(p0, p1);
            }
            dev::tmem_st32(t_s + 32 * h, pr);  // (over the first half's scores, which are read)
            l += ((rs8[0] + rs8[1]) + (rs8[2] + rs8[3])) + ((rs8[4] + rs8[5]) + (rs8[6] + rs8[7]));
          }
          // (every PV of this stream so far completed before the QK whose S was just read)
          if (j >= (two ? 1 : 2) && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t ov[16];
              dev::tmem_ld16(t_o + st * 128 + c * 16, ov);
              dev::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              dev::tmem_st16(t_o + st * 128 + c * 16, ov);
            }
          }
          dev::tmem_wait_st();
        }
        dev::tc_fence_before();
        // the tile ends early: zero the rows of V behind it, a quarter a warp (two query
        // tiles: the first one's warps, whose PV goes first)
        const int32_t rem = me.ctx + me.T - t * kRows;
        if (rem < kRows && (kTwo || !two || st == 0)) {
          const uint32_t ve = v_entry(kTwo ? 2 * (p.at + j) + (st ^ lead) : p.at + j, steps);
          ok = dev::mbar_wait(bars.full(ve % kSlots), (ve / kSlots) & 1, abort_flag, a.err, kTimeoutNs) && ok;
          const uint32_t v = sbase + kSmemKV + (ve % kSlots) * kTileBytes;
          if (ok)
            for (uint32_t x = (uint32_t)rem * 128u + threadIdx.x % 128 * 16u; x < kHalfBytes; x += 2048u)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + h * kHalfBytes + x), "r"(0u) : "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // visible to the tensor cores
        }
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(bars.p_ready(st));
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) break;
      if (two) {
        finished(st);
      } else {
        finished(0);
        if (n > 1) finished(1);
      }
      ++done[0];
      if (two || n > 1) ++done[1];
      go = walk.next(a, &p_next);
      if (go) next = look(p_next);
      float w0 = 1.f, w1 = 0.f;
      const bool both = !two && n > 1;
      if (!two) {
        // exchange with the other stream's row: o = (w0 O_0 + w1 O_1) / l
        ml_of[st * 128 + row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(bars.joined());
        ok = dev::mbar_wait(bars.joined(), joined & 1, abort_flag, a.err, kTimeoutNs) && ok;
        ++joined;
        const float2 x0 = ml_of[row], x1 = ml_of[128 + row];
        m = fmaxf(x0.x, x1.x);
        w0 = dev::ex2_approx(x0.x - m);
        w1 = dev::ex2_approx(x1.x - m);
        l = w0 * x0.y + w1 * x1.y;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      dev::tc_fence_after();
      if (busy) {
        // two query tiles: all dims of the row; one: half of them in each stream's warps
        const int c0 = two ? 0 : 2 * st, c1 = two ? 4 : 2 * st + 2;
        const int32_t tok = q.tok0 + (int32_t)tok_in, head = q.head + (int32_t)sub;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t at = kTwo ? 2 * (int64_t)blockIdx.x + st : blockIdx.x;
        const int64_t part = (2 * at + (p.first ? 0 : 1)) * a.slot_rows + (!kTwo && two ? st * kRows : 0) + row;
        // (two chunks of 32 dims a turn: one chunk after the other waits for tensor memory each time)
        constexpr int kChunks = 2;
#pragma unroll 1
        for (int c = c0; c < c1; c += kChunks) {
          uint32_t ov[kChunks][32];
#pragma unroll
          for (int y = 0; y < kChunks; ++y) dev::tmem_ld32(t_o + (two ? st * 128 : 0) + (c + y) * 32, ov[y]);
          dev::tmem_wait_ld();
          if (!two) {
#pragma unroll
            for (int y = 0; y < kChunks; ++y) {
              uint32_t o1[32];
              if (both) {
                dev::tmem_ld32(t_o + 128 + (c + y) * 32, o1);
                dev::tmem_wait_ld();
              }
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float x = w0 * __uint_as_float(ov[y][e]);
                ov[y][e] = __float_as_uint(both ? fmaf(w1, __uint_as_float(o1[e]), x) : x);
              }
            }
          }
          if (valid && p.whole) {
            __nv_bfloat16* const dst = a.o + (int64_t)tok * a.o_stride + (int64_t)head * kHeadDim + c * 32;
#pragma unroll
            for (int e = 0; e < 4 * kChunks; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int at = 8 * (e & 3) + 2 * x;
                w[x] = dev::pack_bf16x2(__uint_as_float(ov[e >> 2][at]) * inv, __uint_as_float(ov[e >> 2][at + 1]) * inv);
              }
              *reinterpret_cast<uint4*>(dst + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (kTwo && valid) {
            // (few pieces of a range are shared; with the transposition 512 sequences of 300 tokens took 132 us for 119)
            float* const dst = a.part_o + part * kHeadDim + c * 32;
#pragma unroll
            for (int e = 0; e < 4 * kChunks; ++e) {
              const uint32_t(&w)[32] = ov[e >> 2];
              const int at = 8 * (e & 3);
              dev::st_global_v8(dst + 8 * e, w[at], w[at + 1], w[at + 2], w[at + 3], w[at + 4], w[at + 5], w[at + 6], w[at + 7]);
            }
          } else if (!kTwo && !p.whole) {
            // (a line of a row from four lanes: a row a lane, 32 lines an instruction, 64 rows took 6,300 cycles)
            float* const dst = a.part_o + (part - (lane & 3)) * kHeadDim + c * 32 + 8 * (lane & 3);
            const int32_t rows = q.n_tok * a.pack - (int32_t)(row & ~3u);  // of this row's four on
#pragma unroll
            for (int y = 0; y < kChunks; ++y) {
              uint32_t(&w)[32] = ov[y];
              transpose4(w, lane);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (k < rows)
                  dev::st_global_v8(dst + k * kHeadDim + 32 * y, w[8 * k], w[8 * k + 1], w[8 * k + 2], w[8 * k + 3], w[8 * k + 4],
                                    w[8 * k + 5], w[8 * k + 6], w[8 * k + 7]);
            }
          }
        }
        if (valid && (two || st == 0)) {
          if (!p.whole)
            a.part_ml[part] = make_float2(m, l);
          else if (a.lse != nullptr)
            a.lse[(int64_t)head * a.S + tok] = (m + __log2f(l)) * 0.6931471805599453f;
        }
      }
      dev::tc_fence_before();
      // One query tile: neither stream's next PV may overwrite an O that the other's warps still read (nor
      // its next row the other's m and l).  Two, and one in the next piece, where each stream waits for both's
      // last PVs: both have seen their own here, so no phase of "PV done" is passed over.
      if (!kTwo && (!two || (go && p_next.n_qt == 1))) {
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(bars.joined());
        ok = dev::mbar_wait(bars.joined(), joined & 1, abort_flag, a.err, kTimeoutNs);
        ++joined;
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    __syncwarp();
    stopped();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    dev::tc_fence_after();
    dev::tmem_dealloc(tmem, kTmemCols);
  }
}

// Rows whose item several blocks shared: o = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c -
// M) l_c over the pieces in the order of their keys.  A warp a row, four dims a lane;
// the eight warps of a block share out the pieces of rows that have many.
constexpr int kJoinWarps = 8;
constexpr int kAtOnce = 4;     // partial rows that a warp has on their way

struct Acc {
  float m, l;
  float4 o;
};
__device__ __forceinline__ Acc nothing() { return Acc{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)}; }
__device__ __forceinline__ void add(Acc& x, float m, float l, const float4& o) {
  const float top = fmaxf(x.m, m), ref = top == -INFINITY ? 0.f : top;
  const float wx = dev::ex2_approx(x.m - ref), w = dev::ex2_approx(m - ref);
  x.o = make_float4(fmaf(w, o.x, wx * x.o.x), fmaf(w, o.y, wx * x.o.y), fmaf(w, o.z, wx * x.o.z), fmaf(w, o.w, wx * x.o.w));
  x.l = fmaf(w, l, wx * x.l);
  x.m = top;
}

// Pieces of an item that the join is to combine: none of one that a single block wrote, none where the entry names slots
// that do not exist (a forward that stopped early leaves entries as they were).
__device__ __forceinline__ int32_t pieces_of(const int2& x, int32_t slots) {
  const bool there = x.y > 1 && x.y <= slots && (uint32_t)x.x < (uint32_t)slots && (x.x | 1) + 2 * x.y - 3 < slots;
  return there ? x.y : 0;
}

// kRowsOf rows a warp, whose loads go out together: many rows have few pieces each
// (32,768 of two: 23 us with a row a warp, 11 with two rows).  0: one row a block, whose warps
// share out its pieces (32 rows of 18: 30 us less than a row after the other).  A row a warp: five blocks an
// SM, 48 registers a thread (52 bytes spilled), so that its rows are one wave; the others have four, 64 registers.
template <int kRowsOf>
__global__ void __launch_bounds__(32 * kJoinWarps, kRowsOf == 1 ? 5 : 4) attn_tree_join_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int kN = kRowsOf > 1 ? kRowsOf : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t n_rows = (uint32_t)a.S * (uint32_t)a.H;  // (below 2^31)
  const uint32_t id = kRowsOf == 0 ? blockIdx.x : (blockIdx.x * kJoinWarps + warp) * kN;
  uint32_t tok[kN], head[kN];
  int32_t item[kN], row[kN], n[kN], slot[kN];  // row of the item's partial slots; pieces (0: nothing to join), first slot
#pragma unroll
  for (int e = 0; e < kN; ++e) {
    tok[e] = min(id + e, n_rows - 1) / (uint32_t)a.H;
    head[e] = min(id + e, n_rows - 1) - tok[e] * (uint32_t)a.H;
    const TreeRow r = a.rows[tok[e]];
    const uint32_t kvh = head[e] / (uint32_t)a.group, in = head[e] - kvh * a.group, pk = in / (uint32_t)a.pack, qt = r.qtile + pk;
    item[e] = r.item0 + (int32_t)(kvh * r.units + qt / 2);
    row[e] = (int32_t)((qt & 1) * kRows + r.in_tile * a.pack + (in - pk * a.pack));
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the forward is complete and its writes visible
#pragma unroll
  for (int e = 0; e < kN; ++e) {
    const int2 x = a.joins[item[e]];
    slot[e] = x.x;
    n[e] = id + e >= n_rows ? 0 : pieces_of(x, a.slots);
  }
  // piece i of a row: its block's first slot, but for the first one
  const auto load = [&](int32_t first, int32_t in_slot, int32_t i, float2* ml, float4* o) {
    const int64_t at = (int64_t)(i == 0 ? first : (first | 1) - 1 + 2 * i) * a.slot_rows + in_slot;
    *ml = a.part_ml[at];
    *o = reinterpret_cast<const float4*>(a.part_o + at * kHeadDim)[lane];
  };
  const auto finish = [&](const Acc& acc, uint32_t t, uint32_t h) {
    const float inv = acc.l == 0.f ? 0.f : 1.f / acc.l;
    __nv_bfloat16* const dst = a.o + (int64_t)t * a.o_stride + (int64_t)h * kHeadDim + 4 * lane;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(dev::pack_bf16x2(acc.o.x * inv, acc.o.y * inv), dev::pack_bf16x2(acc.o.z * inv, acc.o.w * inv));
    if (lane == 0 && a.lse != nullptr) a.lse[(int64_t)h * a.S + t] = (acc.m + __log2f(acc.l)) * 0.6931471805599453f;
  };
  if constexpr (kN > 1) {
    Acc acc[kN];
    int32_t most = 0;
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      acc[e] = nothing();
      most = max(most, n[e]);
    }
#pragma unroll 1
    for (int32_t i = 0; i < most; ++i) {
      float2 ml[kN];
      float4 o[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (i < n[e]) load(slot[e], row[e], i, &ml[e], &o[e]);
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (i < n[e]) add(acc[e], ml[e].x, ml[e].y, o[e]);
    }
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (n[e] > 0) finish(acc[e], tok[e], head[e]);
  } else {
    const auto run = [&](int32_t i0, int32_t i1, Acc& acc) {
#pragma unroll 1
      for (int32_t i = i0; i < i1; i += kAtOnce) {
        float2 ml[kAtOnce];
        float4 o[kAtOnce];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
          if (i + e < i1) load(slot[0], row[0], i + e, &ml[e], &o[e]);
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
          if (i + e < i1) add(acc, ml[e].x, ml[e].y, o[e]);
      }
    };
    if (n[0] == 0) return;  // (the same for the whole block where it has one row)
    Acc acc = nothing();
    if constexpr (kRowsOf == 1) {
      run(0, n[0], acc);
    } else {
      __shared__ Acc shared[kJoinWarps][32];
      run(n[0] * warp / kJoinWarps, n[0] * (warp + 1) / kJoinWarps, acc);
      if (warp > 0) shared[warp][lane] = acc;
      __syncthreads();
      if (warp > 0) return;
#pragma unroll 1
      for (int i = 1; i < kJoinWarps; ++i) add(acc, shared[i][lane].m, shared[i][lane].l, shared[i][lane].o);
    }
    finish(acc, tok[0], head[0]);
  }
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
            std::string* why) {
  auto fn = encode_fn();
  if (fn == nullptr) {
    *why = "cuTensorMapEncodeTiled is unavailable";
    return false;
  }
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    *why = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r);
    return false;
  }
  return true;
}

}  // namespace

// More items than blocks, a query tile each: a block's streams have ranges of their own.
static bool two_ranges(const TreeArgs& a) { return a.slot_rows == kRows && a.items > a.grid; }

cudaError_t launch_attn_tree(const TreeArgs& args, const void* q, int64_t q_stride, const h3attn_cache& c, cudaStream_t stream,
                             std::string* why) {
  static SmemAttr attr, attr_two;
  const bool two = two_ranges(args);
  cudaError_t e = two ? attr_two.set(attn_tree_kernel<true>, (int)kSmemAlloc) : attr.set(attn_tree_kernel<false>, (int)kSmemAlloc);
  if (e != cudaSuccess) {
    *why = "cudaFuncSetAttribute(max dynamic shared memory) failed";
    return e;
  }
  TreeArgs a = args;
  a.recip = (65536u + (uint32_t)a.pack - 1) / (uint32_t)a.pack;
  a.page_size = c.page_size;
  a.n_pages = c.n_pages;
  a.box = c.page_size & -c.page_size;  // gcd(page_size, 128), of a multiple of 8
  if (a.box > kRows) a.box = kRows;
  a.n_box = kRows / a.box;
  a.at_once = 32 / a.n_box;
  a.row_step = kRows % a.page_size;
  a.page_boxes = a.page_size / a.box;
  // i / page_boxes = i mul >> shift for i < 2^29: mul exceeds 2^shift / page_boxes by less than 1, and i by that stays
  // below 2^shift / page_boxes
  int bits = 0;
  while ((1ll << bits) < a.page_boxes) ++bits;
  a.page_shift = 29 + bits;
  a.page_mul = (uint32_t)(((1ull << a.page_shift) + a.page_boxes - 1) / a.page_boxes);
  a.inv_grid = 1.f / (float)a.grid;
  a.by_warp = !two && a.items <= a.grid && (int64_t)a.table_width * a.page_size < ((int64_t)1 << 28);
  a.recip_toks = (65536u + (uint32_t)a.toks - 1) / (uint32_t)a.toks;
  CUtensorMap mq, mk, mv;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)a.H, (cuuint64_t)a.S};
    // (one row has no stride: a map's is below 2^40 bytes)
    const cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)(a.S > 1 ? q_stride : (int64_t)a.H * kHeadDim) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.pack, (cuuint32_t)a.toks};
    if (!encode(&mq, q, 3, dims, strides, box, why)) return cudaErrorInvalidValue;
  }
  // the smaller stride first; a dimension of one may have any
  const int64_t tok = c.page_size > 1 ? c.token_stride : kHeadDim, hd = c.num_kv_heads > 1 ? c.head_stride : kHeadDim;
  a.heads_first = hd < tok;
  const cuuint64_t kv_dims[4] = {(cuuint64_t)kHeadDim, (cuuint64_t)(a.heads_first ? c.num_kv_heads : c.page_size),
                                 (cuuint64_t)(a.heads_first ? c.page_size : c.num_kv_heads), (cuuint64_t)c.n_pages};
  const cuuint64_t kv_strides[3] = {(cuuint64_t)(a.heads_first ? hd : tok) * 2, (cuuint64_t)(a.heads_first ? tok : hd) * 2,
                                    (cuuint64_t)(c.n_pages > 1 ? c.page_stride : kHeadDim) * 2};
  const cuuint32_t kv_box[4] = {64, a.heads_first ? 1u : (cuuint32_t)a.box, a.heads_first ? (cuuint32_t)a.box : 1u, 1};
  if (!encode(&mk, c.k, 4, kv_dims, kv_strides, kv_box, why) || !encode(&mv, c.v, 4, kv_dims, kv_strides, kv_box, why))
    return cudaErrorInvalidValue;
  if (two)
    attn_tree_kernel<true><<<(unsigned)a.grid, kThreads, kSmemAlloc, stream>>>(mq, mk, mv, a);
  else
    attn_tree_kernel<false><<<(unsigned)a.grid, kThreads, kSmemAlloc, stream>>>(mq, mk, mv, a);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_tree_join(a, stream, why);
}

cudaError_t launch_tree_join(const TreeArgs& args, cudaStream_t stream, std::string* why) {
  TreeArgs a = args;
  a.slots = (two_ranges(a) ? 4 : 2) * a.grid;
  cudaError_t e = cudaSuccess;
  // Few items have many pieces each (about the blocks by the items): a block a row (1,024 rows of two
  // or three: 7.6 us, 3.7 with a row a warp).  Else a row a warp while that is one wave, five blocks an SM.
  // (Rows are below 2^31.)
  const int64_t rows = a.S * a.H, one = (rows + kJoinWarps - 1) / kJoinWarps;
  if (8 * (int64_t)a.items <= a.grid)
    e = launch_dependent(attn_tree_join_kernel<0>, (unsigned)rows, 32u * kJoinWarps, stream, a);
  else if (one <= (int64_t)5 * a.grid)
    e = launch_dependent(attn_tree_join_kernel<1>, (unsigned)one, 32u * kJoinWarps, stream, a);
  else
    e = launch_dependent(attn_tree_join_kernel<2>, (unsigned)((one + 1) / 2), 32u * kJoinWarps, stream, a);
  if (e != cudaSuccess) *why = "the join launch failed";
  return e;
}

}  // namespace h3
