// Packed varlen non-causal attention on the 5th-generation tensor cores,
// run by CTA pairs.
//
// Pages: vllm.cpp PR #26 "feat(minimax-h3)", PR description (packed varlen
// NON-CAUSAL attention: each query attends to every key of its own
// cu_seqlens document and to nothing else -- a cu_seqlens varlen
// flash-attention call with causal=false) and the warp-per-query-row commit
// (online-softmax recurrence in f32; Q read once per query row).
//
// Design: a cluster of two CTAs (one per SM of a pair) works on one unit of
// 512 query rows of one (head, document); each CTA owns 256 of them as two
// 128-row query tiles s = 0, 1 (rows q0 + 256 s + 128 rank + i).  The MMAs are
// pair instructions (tcgen05 cta_group::2, M = 256): one thread of the even
// CTA issues them, each CTA's tensor core computes its own 128 rows, and each
// CTA holds only half of every B operand -- keys [64 rank, 64 rank + 64) of a
// K tile and dims [64 rank, 64 rank + 64) of a V tile -- so a CTA reads
// (and loads from L2) half the key/value bytes a single-CTA kernel would.
// Per CTA, 11 warps:
//   warp 9       lane 0: TMA producer, its halves of the document's K and V
//                tiles through a 6-slot ring; V(j) and the next K tile form
//                one group behind one barrier.  (FP8: also its own Q tiles,
//                the next unit's behind the current unit's first K/V group.)
//                lane 1 (bf16): the O-store thread (below).
//   warp 10      Q warp: loads this CTA's Q tiles (bf16) into double-buffered
//                slots as they come free, so the next unit's tiles are ready
//                before it starts; as each lands, applies the fused Q prologue
//                in place when asked (RMSNorm with gain, rot96 rotation) and
//                reports the tile ready to the even CTA.
//   warp 8       even CTA: MMA issuer for the pair, S = Q_s K^T and
//                O_s += P V, fp32 accumulators in TMEM.  Both CTAs' warp 8
//                allocate the pair's TMEM together.
//   warps 0..3   softmax for query tile 0 of this CTA,
//   warps 4..7   softmax for query tile 1: one thread per query row reads its
//                S row from TMEM, keeps the running max and sum in registers,
//                writes P as bf16 back into TMEM over its S columns, rescales
//                its O row when the max has grown by more than 2^8, and at the
//                end of the unit writes O / l and the log-sum-exp.  A bf16
//                warp whose 32 rows all lie in the document stages them, bf16,
//                in the unit's Q slot (free once the unit's MMAs are done);
//                other warps store their rows directly.  Either way the four
//                warps of a query tile then report to the O-store thread,
//                which sends the staged rows out with TMA tile stores, waits
//                until they have read the slot and frees it for the Q warp --
//                so the softmax warps never wait on the TMA unit.
// Each 128-key tile is taken in two halves of 64 keys, h = 0, 1, each with
// its own 64 TMEM columns of S: per query tile the issuer runs PV of half h
// of key tile j and then QK of half h of key tile j + 1 into the same
// columns, so the softmax works on the other half while the tensor cores
// compute the next S half -- a query tile's softmax does not wait for its own
// PV and next QK.  Both query tiles and both halves interleave on the tensor
// pipe (order per key tile: tile 0 half 0, tile 1 half 0, tile 0 half 1,
// tile 1 half 1).  A unit only visits its own document's key tiles; keys past
// the document end in the last tile are masked to -inf, rows past it are
// never stored.  Each pair runs its own range of the work list (placed on the
// host longest-processing-time first), and the next unit's first QKs are
// issued right after the current unit's last PVs, so its softmax finds them
// done when it comes back from the epilogue.
//
// Key halves: a CTA holds keys [64 rank, 64 rank + 64) of a tile; half h is
// rows [32 h, 32 h + 32) of both CTAs' halves (the pair MMA takes B's first
// 32 columns from the even CTA), so S column c of half h is key 32 h + c for
// c < 32 and 64 + 32 h + (c - 32) for c >= 32; the PV of a half reads the
// matching 16-key (bf16) or 32-key (FP8) chunks of V.
//
// TMEM columns (each CTA): S0 [0,128) S1 [128,256) O0 [256,384) O1 [384,512),
// S_s half h at S_s + 64 h; P of a half is bf16 packed two per column in the
// half's first 32 columns.
//
// Shared memory rows are 64 bf16 (128 B, 128-byte TMA swizzle).  Q tiles are
// 128 rows x 128 dims (two 16 KB halves); a K half-tile is 64 keys x 128 dims
// (two 8 KB halves), a V half-tile 128 keys x 64 dims (16 KB).  Q and K are
// K-major operands; V is the MN-major B operand of the PV product.
//
// Barriers: completion of the pair's MMAs is multicast to both CTAs (S half
// ready, PV done; FP8: Q slots free).  The MMA-issuing thread paces the tensor
// cores, so per key-tile half it only waits for P and commits: its "P ready"
// barrier of (query tile, half) counts one arrival per softmax warp of both
// CTAs, and softmax warp 0 of each CTA reports half 0 only once its CTA's next
// K/V group has landed; a softmax thread of the unit's last query tile that
// sees S half 1 of key tile t ready frees the ring slots of the group holding
// K(t) (everything before that QK has completed).  "PV done" of a query tile
// and half completes once per unit, after the PV of that half in the unit's
// last key tile: the epilogue waits for both halves.  A rescale of O first
// waits for the other half's latest PV: through the S-ready of the QK issued
// right after it, or "PV done" in the last key tile.  Q tiles:
// the even CTA's "Q ready" barrier counts one arrival from the Q warp of each
// CTA; a bf16 Q slot is freed by the O-store thread after the four softmax
// warps of its query tile in that CTA have reported their epilogue done.
//
// FP8 variant (template argument kFp8, h3attn_forward_fp8): the same kernel
// on e4m3 Q, K and transposed V (channel rows of keys, every document
// starting on a 16-key boundary) with fp32 scales -- kind::f8f6f4 pair MMAs of
// K = 32, 16 KB Q tiles and 8 KB half-tiles in 128-byte rows, P rounded to
// e4m3 and stored four per TMEM column (first 32 columns of S), the q-row x
// key-tile scale folded into the softmax's score multiplier, the per-channel
// V scale applied to O in the epilogue.  Its MMAs are half as long as bf16's,
// so it keeps whole 128-key tiles (one S-ready and one P-ready phase per key
// tile and query tile, P over S, issued by one thread): split into halves,
// the per-half softmax costs measured slower than the chain they remove.
//
// Other key walks (template argument kWalk, bf16): the same pipeline over key
// tiles that are not "the unit's document, in order".  The list walk
// (h3attn_forward_sparse) takes the tiles listed for a query block, the prefix
// walk (h3attn_forward_prefix) the tiles of a prefix that all documents share
// (tensor maps of its own) and then the rows' own documents.  The producer and
// the softmax warps look each tile up (walk_entry, a tile ahead, and key_tile);
// the MMA issuer only counts tiles.  Three things keep rows apart that share
// MMAs or tiles:
//   - keys a row may not see are masked to -inf after the QK, as above;
//   - the rows of a V tile behind its last valid key are zeroed in shared memory
//     before the PV reads them, so that a NaN or infinity behind a document or
//     prefix (weight 0) does not reach its output;
//   - a segment over several documents (prefix walk) runs each one's own tiles
//     for all its rows, but their PVs leave the lanes of O of the other
//     documents' rows alone (the MMA's lane mask).
// A list without a valid tile runs one fully masked tile: o = 0, lse = -inf.
// The causal walk (h3attn_forward_causal) is the document walk up to a segment's
// last token, with every row's own end of the keys.  The query heads that share a key
// head share segments too: a tile's rows are (token, head of the pack) pairs, token
// by token, which one box of a three-dimensional tensor map fetches in that order.
// So a segment spans fewer tokens (4 x 128 / pack), whose keys end at nearly the same
// place, and K and V pass once for all of them.  Tensor-bound: 20,423 tokens, 28 heads over 4, 1,780 us, 1,680
// TFLOP/s (1,683 us in a short burst; 32 heads over 4, whose packs fill the tiles, 1,855 TFLOP/s; the dense forward with
// the same products 1,569 us); sixteen prompts of 32,768 tokens in all, 21 heads, 344 to 350 us in two streams, whose step of
// 1.50 us sets it (370 to 380 of a hundred calls in a row, under the power limit).
// Bound by the tensor pipe for long walks (1.28 us a tile and CTA pair, 512 rows,
// which is the dense forward's rate: 682 us for 1.12e12 flops in a loop, 1,640
// TFLOP/s; 628 us alone); a segment costs another 4 us for its boundary, where
// the pipeline runs empty (measured for segments of 1 to 16 tiles).  For short
// lists and 256-row query blocks that boundary is hidden by a second stream of
// segments (kPair, below).
//
// Every mbarrier wait is bounded: on expiry the CTA raises an abort flag,
// records a timeout in the device error word, drains its own copies and MMAs
// with bounded waits, and leaves through the cluster barrier, where the pair
// frees its TMEM together.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstring>

#include "device_common.cuh"
#include "launch_common.cuh"
#include "qk_norm.cuh"

namespace h3 {

namespace {

constexpr int kThreads = 352;
constexpr int kMmaWarp = 8;
constexpr int kTmaWarp = 9;
constexpr int kQWarp = 10;
constexpr int kTileRows = 128;
// Shared-memory layout: 2 buffers x 2 query tiles, then the ring.  bf16: a Q
// tile is 128 rows x 128 dims in two 16 KB halves of 64 dims, a slot 16 KB;
// fp8 (e4m3): a Q tile is one 16 KB block of 128-byte rows, a slot 8 KB.
// kPair (two streams of segments side by side): two Q tiles and eight ring slots.
template <bool kFp8, bool kPair = false>
struct Cfg {
  static constexpr int Slots = kPair ? 8 : 6;          // ring slots
  static constexpr int Groups = Slots / 2;             // key/value groups in flight
  static constexpr int QTiles = kPair ? 2 : 4;
  // q_full[4] q_empty[4] q_ready[4] kv_full[G] kv_empty[G] s_ready[2][2] p_ready[2][2] pv_done[2][2] drain o_staged[4]
  static constexpr int NumBars = 12 + 2 * Groups + 4 + 4 + 4 + 1 + 4;
  static constexpr uint32_t QTileBytes = kFp8 ? 128 * 128 : 128 * 128 * 2;
  static constexpr uint32_t SlotBytes = kFp8 ? 64 * 128 : 64 * 128 * 2;
  static constexpr uint32_t SmemQ = 0;
  static constexpr uint32_t SmemKV = QTiles * QTileBytes;
  static constexpr uint32_t SmemBar = SmemKV + Slots * SlotBytes;
  static constexpr uint32_t SmemMisc = SmemBar + NumBars * 8;
  static constexpr uint32_t SmemSteps = SmemMisc + 16;  // kPair: of each stream's last segments [2][4][4] (see steps_of)
  static constexpr size_t SmemAlloc = SmemSteps + (kPair ? 128 : 0) + 1024;  // slack to align the base to 1 KB
  static_assert(SmemAlloc <= 227 * 1024, "shared memory per CTA");
};
constexpr uint32_t kQHalfBytes = 128 * 128;            // bf16 Q tile: one half (64 dims)
constexpr uint32_t kKHalfBytes = 64 * 128;             // bf16 K half-tile: one half (64 dims)
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kTimeoutNs = 2000000000ull;         // 2 s
constexpr float kRescaleThreshold = 8.0f;              // log2 units: rescale when max grows by > 2^8
// The other walks rescale O only when a row's maximum has grown by 2^32: P is
// bf16, whose range is fp32's, so p up to 2^32 rounds no worse than p up to 2^8,
// and the sums stay below 2^127 for 2^31 keys and |v| up to 2^64.  A rescale
// costs a warp two trips of its O rows through registers and a wait for the
// other half's PV; with scores spread over tens of log2 units some row of a
// warp crosses 2^8 in most tiles.
constexpr float kRescaleThresholdWalk = 32.0f;
constexpr uint16_t kPairMask = 0x3;
// kPair: steps of its first segment that stream 0 is ahead, or half of them where
// it has fewer than twice as many (a boundary is over in two or three; half of a
// long first segment ahead left stream 1 alone as long at the end, where a tile
// takes 1.05 us for one stream instead of 0.75: 130 against 124 us for two dozen
// documents of 1 to 700 tokens over 2,430 prefix rows)
constexpr uint32_t kHoldSteps = 2;
static_assert(kUnitRows == 4 * kTileRows, "a unit is two query tiles in each CTA of the pair");

// Instruction descriptors, kind::f16: fp32 accumulator, bf16 A and B, M = 256 (pair).
// QK: N = 64 keys (one half of a key tile), A and B K-major; PV: N = 128 dims,
// B (V) MN-major.
constexpr uint32_t kIdescBf16 = (1u << 4) | (1u << 7) | (1u << 10) | ((256u >> 4) << 24);
constexpr uint32_t kIdescQK = kIdescBf16 | ((64u >> 3) << 17);
constexpr uint32_t kIdescPV = kIdescBf16 | ((128u >> 3) << 17) | (1u << 16);
// kind::f8f6f4: e4m3 A and B (type code 0), fp32 accumulator, M = 256, N = 128,
// both K-major (the FP8 pipeline takes whole 128-key tiles)
constexpr uint32_t kIdescF8 = (1u << 4) | ((128u >> 3) << 17) | ((256u >> 4) << 24);

// Q slot i = 2 * buffer + query tile; the unit with ordinal k (per pair) uses
// buffer k & 1.  (kPair: stream s has Q slot s.)
template <bool kPair>
__device__ __forceinline__ int q_slot_of(int k, int s) {
  return kPair ? s : 2 * (k & 1) + s;
}
template <int kGroups>
struct Bars {
  uint32_t base;
  __device__ uint32_t q_full(int i) const { return base + 8 * i; }
  __device__ uint32_t q_empty(int i) const { return base + 8 * (4 + i); }
  __device__ uint32_t q_ready(int i) const { return base + 8 * (8 + i); }
  __device__ uint32_t kv_full(int i) const { return base + 8 * (12 + i); }
  __device__ uint32_t kv_empty(int i) const { return base + 8 * (12 + kGroups + i); }
  // S of key-tile half h of query tile s is in TMEM / P of it is in TMEM
  __device__ uint32_t s_ready(int s, int h) const { return base + 8 * (12 + 2 * kGroups + 2 * s + h); }
  __device__ uint32_t p_ready(int s, int h) const { return base + 8 * (16 + 2 * kGroups + 2 * s + h); }
  // the PV of half h of query tile s in a unit's last key tile has completed
  // (one phase per unit)
  __device__ uint32_t pv_done(int s, int h) const { return base + 8 * (20 + 2 * kGroups + 2 * s + h); }
  __device__ uint32_t drain() const { return base + 8 * (24 + 2 * kGroups); }
  // bf16: the four softmax warps of Q slot i's query tile have finished that
  // unit's epilogue (their O rows staged in the slot or stored)
  __device__ uint32_t o_staged(int i) const { return base + 8 * (25 + 2 * kGroups + i); }
};

// Key walks: the unit's own document (the dense forward), the tiles listed for
// its query block, the shared prefix's tiles and then the document's, the document's
// up to each row itself.
constexpr int kWalkDoc = 0, kWalkList = 1, kWalkPrefix = 2, kWalkCausal = 3;

// kPair (the other walks, segments of up to 256 rows: 256-row query blocks, and
// where the walks are short): a CTA pair runs two streams of segments, each with
// walks of its own -- different lists, of any documents and heads.  Query tile s of both CTAs (rows
// q0 + 128 rank + i) belongs to stream s.  The streams share nothing but the
// tensor cores: the issuer takes whichever stream's next P is ready, and stream
// 1 begins a few steps after stream 0 (kHoldSteps), so that one stream's segment boundary
// (the pipeline running empty, the epilogue, the next Q and first softmax) falls
// into the middle of the other's segment.  Every step needs a K and a V tile per
// query tile, twice the L2 traffic per MMA of a shared walk, and each stream has
// two groups of the ring: group n of stream s, ring slots 4 s + 2 (n & 1) and the
// one after it, holds V(n - 1) and K(n), n counting the stream's steps.  A Q
// slot is free once its segment's last QK is done, a step before the segment
// ends, so one per stream is enough; O rows are stored directly.  (A step of
// both streams takes 1.50 us, one of 512 rows in one stream 1.28.  What makes the
// difference is not known: it does not depend on where in L2 the tiles lie, and no
// unit is full -- over 20 listed tiles a segment the tensor pipe is active 70 % of
// cycles, with its operands' fetches 83 %, against 77 and 90 % in one stream over 40.)
// Warp 9 loads stream 0 and warp 10 stream 1: lane 0 Q, K and V in the order the
// stream needs them, lane 1 reports each Q tile landed.
// Measured, us for 512 rows of a head (two segments) and 2 / 4 / 8 / 16 tiles: one
// 256-row segment at a time with the other query tile idle 13.5 / 18 / 28 / 49;
// two in lockstep 7.5 / 9.7 / 14.8 / 25.1; two streams 5.4 / 7.7 / 13.0 / 24.1.

// What a walk needs besides the unit.
template <int kWalk>
struct Walk {};
template <>
struct Walk<kWalkList> {
  const int32_t* idx;   // [H, blocks, cap]
  const int32_t* cnt;   // [H, blocks]
  int32_t blocks, cap;
};
template <>
struct Walk<kWalkPrefix> {
  CUtensorMap tm_k, tm_v;   // the prefix's rows
  const OwnTile* own;       // own tiles of segments over several documents
  int32_t len, tiles;
};

template <>
struct Walk<kWalkCausal> {
  int32_t pack, toks;   // heads and tokens of a query tile (pack * toks <= 128 rows)
  uint32_t recip;       // row / pack = row * recip >> 16 for rows below 128
  int32_t group;        // query heads of a key head
};

struct UnitGeom {
  int32_t q0, kv0, kv1, head, lo, hi, part, n_st;  // key tiles [lo, hi) of the walk
  int32_t v_off;                                   // FP8: the document's first key in the transposed V
                                                   // causal walk: the key head
  int32_t q1;                                      // end of the unit's query rows
  const int32_t* list;                             // list walk: the segment's tiles, step j's at list[j] (null: none)
  int32_t n;                                       // list walk: entries of the list; the steps after them are masked
                                                   // prefix walk: own tiles of a segment over several documents
};

// First row (token) of this CTA's query tile s of a unit.
template <int kWalk, bool kPair>
__device__ __forceinline__ int32_t tile_row(const UnitGeom& g, int s, uint32_t rank, const Walk<kWalk>& walk) {
  if constexpr (kWalk == kWalkCausal) return g.q0 + ((kPair ? 0 : 2 * s) + (int32_t)rank) * walk.toks;
  return g.q0 + (kPair ? 0 : s * 2 * kTileRows) + (int32_t)rank * kTileRows;
}

// The head whose keys and values a unit reads.
template <int kWalk>
__device__ __forceinline__ int32_t key_head(const UnitGeom& g) {
  return kWalk == kWalkCausal ? g.v_off : g.head;
}

// Entries [*lo, *hi) of its query block's list that a segment (its record's
// second half) visits: piece i of m takes [n i / m, n (i + 1) / m) of the n.
__device__ __forceinline__ int64_t list_range(const int4& x, const Walk<kWalkList>& walk, int32_t* lo, int32_t* hi) {
  *lo = *hi = 0;
  const int64_t block = (int64_t)x.x * walk.blocks + x.y;
  const uint32_t i = (uint32_t)x.z & 0xffffu, m = (uint32_t)x.z >> 16;
  const uint64_t n = (uint64_t)min(max(__ldg(walk.cnt + block), 0), walk.cap);
  *lo = m == 1 ? 0 : (int32_t)(n * i / m);
  *hi = m == 1 ? (int32_t)n : (int32_t)(n * (i + 1) / m);
  return block * walk.cap;
}

template <int kWalk>
__device__ __forceinline__ UnitGeom unit_geom(const WorkUnit* units, int u, const Walk<kWalk>& walk) {
  const int4 w = __ldg(reinterpret_cast<const int4*>(units) + 2 * u);
  const int4 x = __ldg(reinterpret_cast<const int4*>(units) + 2 * u + 1);
  UnitGeom g;
  g.list = nullptr;
  g.n = 0;
  if constexpr (kWalk == kWalkDoc) {
    g.q0 = w.x;
    g.kv0 = w.y;
    g.kv1 = w.z;
    g.head = w.w;
    g.lo = x.x;
    g.hi = x.y;
    g.part = x.z;
    g.v_off = x.w;
    g.q1 = w.z;
    g.n_st = (w.x + 2 * kTileRows < w.z) ? 2 : 1;  // query tile 1 of the pair holds rows from 256 on
  } else {  // a WalkUnit
    g.q0 = w.x;
    g.q1 = w.y;
    g.kv0 = w.z;
    g.kv1 = w.w;
    g.head = x.x;
    g.part = x.w;
    g.v_off = 0;
    g.n_st = (w.x + 2 * kTileRows < w.y) ? 2 : 1;
    if constexpr (kWalk == kWalkCausal) {
      g.lo = x.y;
      g.hi = x.z;
      g.v_off = x.x / walk.group;
      g.n_st = (w.x + 2 * walk.toks < w.y) ? 2 : 1;
    } else if constexpr (kWalk == kWalkPrefix) {
      g.lo = x.y;
      g.hi = x.z;
      g.n = max(-w.w, 0);  // kv0: the first of them in the table
    } else {
      int32_t lo, hi;
      const int64_t at = list_range(x, walk, &lo, &hi);
      g.n = hi - lo;
      if (g.n > 0) g.list = walk.idx + at + lo;
      g.lo = 0;
      g.hi = max(g.n, 1);  // nothing listed: one fully masked tile
    }
  }
  return g;
}

// What a walk looks up for its step j, a tile ahead of its use: the list's entry
// (x), or an own tile's key row, valid keys and query rows.
template <int kWalk>
__device__ __forceinline__ int4 walk_entry(const UnitGeom& g, int j, const Walk<kWalk>& walk) {
  int4 e = make_int4(-1, 0, 0, 0);
  if constexpr (kWalk == kWalkList) {
    if (j < g.n) e.x = __ldg(g.list + j);
  } else if constexpr (kWalk == kWalkPrefix) {
    if (g.n > 0 && j >= walk.tiles) e = __ldg(reinterpret_cast<const int4*>(walk.own + g.kv0 + (j - walk.tiles)));
  }
  return e;
}

// Step j of a unit's walk: the tile's first key row, its valid keys (0 or less:
// none, 128 or more: all), the unit's rows [lo, hi) that see it, and whether it
// lies in the prefix.
struct KeyTile {
  int32_t row, rem, lo, hi;
  bool prefix, bad;
};
template <int kWalk>
__device__ __forceinline__ KeyTile key_tile(const UnitGeom& g, int j, const int4& entry, const Walk<kWalk>& walk) {
  KeyTile t{g.kv0, 0, 0, kUnitRows, false, false};
  if constexpr (kWalk == kWalkDoc || kWalk == kWalkCausal) {
    t.row = g.kv0 + j * kTileRows;
    t.rem = g.kv1 - t.row;
  } else if constexpr (kWalk == kWalkPrefix) {
    t.prefix = j < walk.tiles;
    t.row = (t.prefix ? j : j - walk.tiles) * kTileRows + (t.prefix ? 0 : g.kv0);
    t.rem = (t.prefix ? walk.len : g.kv1) - t.row;
    if (g.n > 0 && !t.prefix) {
      t.row = entry.x;
      t.rem = entry.y;
      t.lo = entry.z;
      t.hi = entry.w;
    }
  } else {
    // a tile outside the document is skipped (and reported by the producer)
    const bool in = (uint32_t)entry.x <= (uint32_t)(g.kv1 - g.kv0 - 1) / kTileRows;
    if (in) {
      t.row = g.kv0 + entry.x * kTileRows;
      t.rem = g.kv1 - t.row;
    }
    t.bad = !in && j < g.n;
  }
  return t;
}

// A bf16 query tile whose first row is `row`, in two halves of 64 dims.
template <int kWalk>
__device__ __forceinline__ void load_q_tile(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int32_t head, int32_t row,
                                            uint64_t pol, const Walk<kWalk>& walk) {
  if constexpr (kWalk == kWalkCausal) {
    dev::mbar_arrive_expect_tx(bar, 256u * (uint32_t)(walk.pack * walk.toks));
    dev::tma_load_3d(dst, tm, bar, 0, head, row, pol);
    dev::tma_load_3d(dst + kQHalfBytes, tm, bar, 64, head, row, pol);
  } else {
    dev::mbar_arrive_expect_tx(bar, Cfg<false>::QTileBytes);
    dev::tma_load_2d(dst, tm, bar, head * 128, row, pol);
    dev::tma_load_2d(dst + kQHalfBytes, tm, bar, head * 128 + 64, row, pol);
  }
}

// This CTA's half of a K tile: keys [key0 + 64 rank, +64), all 128 dims (bf16:
// two boxes of 64 dims; fp8: one box of 128-byte rows).
template <bool kFp8>
__device__ __forceinline__ void load_k_half(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int head,
                                            int32_t key0, uint32_t rank, uint64_t pol) {
  const int32_t row = key0 + 64 * (int32_t)rank;
  dev::tma_load_2d(dst, tm, bar, head * 128, row, pol);
  if constexpr (!kFp8) dev::tma_load_2d(dst + kKHalfBytes, tm, bar, head * 128 + 64, row, pol);
}

// This CTA's half of a V tile: 128 keys, dims [64 rank, 64 rank + 64) (one box;
// fp8: rows of the transposed V, one per channel, 128 keys each).
// key0: the tile's first key row (bf16) or its first key in the transposed V,
// a multiple of 16 (fp8).
template <bool kFp8>
__device__ __forceinline__ void load_v_half(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int head,
                                            int32_t key0, uint32_t rank, uint64_t pol) {
  if constexpr (kFp8)
    dev::tma_load_2d(dst, tm, bar, key0, head * 128 + 64 * (int32_t)rank, pol);
  else
    dev::tma_load_2d(dst, tm, bar, head * 128 + 64 * (int32_t)rank, key0, pol);
}

// Shared-memory descriptors, split into 32-bit words: the high word (stride
// 1024 B between 8-row groups, descriptor version 1, 128-byte swizzle) is the
// same for every operand here; the low word holds the start address >> 4 and
// the leading-byte offset >> 4, and stepping through an operand only adds to
// the address field (addresses stay below 256 KB, so it never carries).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}

// Key-tile halves.  Each CTA holds keys [64 rank, 64 rank + 64) of a 128-key
// tile; half h of the tile is rows [32 h, 32 h + 32) of both CTAs' halves (the
// pair MMA takes B's first 32 columns from the even CTA, the next 32 from the
// odd one), so S column c of half h is key 32 h + c (c < 32) or
// 64 + 32 h + (c - 32) (c >= 32) of the tile.  The half's 32 rows start
// 32 x 128 B = 4 KB into each CTA's K half-tile (a whole number of 1 KB swizzle
// atoms).
constexpr uint32_t kHalfKeyRowsBytes = 32 * 128;

// Key offset within the 128-key tile of S column c (0..63) of half h.
__device__ __forceinline__ int half_key(int c, int h) { return 32 * h + c + (c >= 32 ? 32 : 0); }

// S half (TMEM, 128 x 64 fp32 in each CTA) = Q (smem, K-major) * K^T (smem,
// K-major, 32 keys per CTA): 8 pair MMAs of K = 16 in one block.  Step kk
// reads Q at +(kk/4) 16 KB + (kk%4) 32 B and K at +(kk/4) 8 KB + (kk%4) 32 B.
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t q_smem, uint32_t k_smem) {
  const uint32_t qa = desc_lo(q_smem, 16), kb = desc_lo(k_smem, 16);
  asm volatile(
      "{\n\t.reg .pred p0, p1, e;\n\telect.sync _|e, 0xffffffff;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"
      "setp.ne.u32 p0, %4, %4;\n\t"
      "setp.eq.u32 p1, %4, %4;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p0;\n\t"
      "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p1;\n\t"
      "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p1;\n\t"
      "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p1;\n\t"
      "add.u32 x, %1, 1024;\n\tadd.u32 y, %2, 512;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p1;\n\t"
      "add.u32 x, %1, 1026;\n\tadd.u32 y, %2, 514;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p1;\n\t"
      "add.u32 x, %1, 1028;\n\tadd.u32 y, %2, 516;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p1;\n\t"
      "add.u32 x, %1, 1030;\n\tadd.u32 y, %2, 518;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p1;\n\t}" ::"r"(d_tmem),
      "r"(qa), "r"(kb), "r"(kDescHi), "r"(0u), "r"(kIdescQK)
      : "memory");
}

// O (TMEM fp32) (+)= P (TMEM, bf16 pairs: 32 columns for the half's 64 keys)
// * V (smem, MN-major, 64 dims per CTA), 4 pair MMAs of K = 16 keys.  MMA i
// reads P columns +8 i, i.e. S columns [16 i, 16 i + 16) of the half, whose
// keys are V's 16-key chunk 2h + {0, 1, 4, 5}[i] (2 KB apart in the slot):
// v_smem is chunk 2h's address; the first MMA accumulates only if acc.
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_smem, bool acc) {
  const uint32_t vb = desc_lo(v_smem, Cfg<false>::SlotBytes);
  asm volatile(
      "{\n\t.reg .pred p0, p1, e;\n\telect.sync _|e, 0xffffffff;\n\t.reg .b64 b;\n\t.reg .b32 t, y;\n\t"
      "setp.ne.u32 p0, %4, 0;\n\t"
      "setp.eq.u32 p1, %4, %4;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %5, p0;\n\t"
      "add.u32 t, %1, 8;\n\tadd.u32 y, %2, 128;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [t], b, %5, p1;\n\t"
      "add.u32 t, %1, 16;\n\tadd.u32 y, %2, 512;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [t], b, %5, p1;\n\t"
      "add.u32 t, %1, 24;\n\tadd.u32 y, %2, 640;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [t], b, %5, p1;\n\t}" ::"r"(d_tmem),
      "r"(p_tmem), "r"(vb), "r"(kDescHi), "r"(acc ? 1u : 0u), "r"(kIdescPV)
      : "memory");
}

// The same, leaving the lanes of O whose bits are set in skip (a, b: 8 words, the
// even CTA's 128 lanes first) as they are: rows of other documents than the
// tile's, whose P is 0 but whose O a NaN in V would reach.
__device__ __forceinline__ void issue_pv_skip(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_smem, bool acc, const uint4& a,
                                              const uint4& b) {
  const uint32_t vb = desc_lo(v_smem, Cfg<false>::SlotBytes);
  asm volatile(
      "{\n\t.reg .pred p0, p1, e;\n\telect.sync _|e, 0xffffffff;\n\t.reg .b64 b;\n\t.reg .b32 t, y;\n\t"
      "setp.ne.u32 p0, %4, 0;\n\t"
      "setp.eq.u32 p1, %4, %4;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %5, {%6, %7, %8, %9, %10, %11, %12, %13}, p0;\n\t"
      "add.u32 t, %1, 8;\n\tadd.u32 y, %2, 128;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [t], b, %5, {%6, %7, %8, %9, %10, %11, %12, %13}, p1;\n\t"
      "add.u32 t, %1, 16;\n\tadd.u32 y, %2, 512;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [t], b, %5, {%6, %7, %8, %9, %10, %11, %12, %13}, p1;\n\t"
      "add.u32 t, %1, 24;\n\tadd.u32 y, %2, 640;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [t], b, %5, {%6, %7, %8, %9, %10, %11, %12, %13}, p1;\n\t}" ::"r"(d_tmem),
      "r"(p_tmem), "r"(vb), "r"(kDescHi), "r"(acc ? 1u : 0u), "r"(kIdescPV), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
      "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
      : "memory");
}

// FP8 (whole 128-key tiles, issued by one thread): S = Q (e4m3, 128-byte rows)
// * K^T (e4m3, 64 keys per CTA), 4 pair MMAs of K = 32 (32 bytes of each row
// per step).
__device__ __forceinline__ void issue_qk_f8(uint32_t d_tmem, uint32_t q_smem, uint32_t k_smem) {
  const uint32_t qa = desc_lo(q_smem, 16), kb = desc_lo(k_smem, 16);
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"
      "setp.ne.u32 p0, %4, %4;\n\t"
      "setp.eq.u32 p1, %4, %4;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, p0;\n\t"
      "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, p1;\n\t"
      "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, p1;\n\t"
      "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, p1;\n\t}" ::"r"(d_tmem),
      "r"(qa), "r"(kb), "r"(kDescHi), "r"(0u), "r"(kIdescF8)
      : "memory");
}

// FP8: O (+)= P (TMEM, e4m3, four per column) * V (e4m3, K-major: 64 channels
// per CTA, 128-byte rows of keys), 4 pair MMAs of K = 32 keys.
__device__ __forceinline__ void issue_pv_f8(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_smem, bool acc) {
  const uint32_t vb = desc_lo(v_smem, 16);
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b64 b;\n\t.reg .b32 t, y;\n\t"
      "setp.ne.u32 p0, %4, 0;\n\t"
      "setp.eq.u32 p1, %4, %4;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], [%1], b, %5, p0;\n\t"
      "add.u32 t, %1, 8;\n\tadd.u32 y, %2, 2;\n\tmov.b64 b, {y, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], [t], b, %5, p1;\n\t"
      "add.u32 t, %1, 16;\n\tadd.u32 y, %2, 4;\n\tmov.b64 b, {y, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], [t], b, %5, p1;\n\t"
      "add.u32 t, %1, 24;\n\tadd.u32 y, %2, 6;\n\tmov.b64 b, {y, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], [t], b, %5, p1;\n\t}" ::"r"(d_tmem),
      "r"(p_tmem), "r"(vb), "r"(kDescHi), "r"(acc ? 1u : 0u), "r"(kIdescF8)
      : "memory");
}

// The MMA warp runs its loop with all 32 lanes (warp-uniform values); each
// tcgen05 instruction is issued by one elected lane.  Commit: arrive on the
// barrier at this offset in both CTAs once the pair MMAs issued so far are done.
__device__ __forceinline__ void commit_pair_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"(kPairMask)
      : "memory");
}
__device__ __forceinline__ void commit_pair_local_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// two e4m3 codes of fp32 values (lo in the low byte), round to nearest even, saturating
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// FP8: one query row's 128 scores from TMEM (4 loads of 32 columns); keys past
// the document end (column >= rem) are set to -inf.
__device__ __forceinline__ void load_scores128(uint32_t t_s, uint32_t (&r)[4][32], int rem) {
#pragma unroll
  for (int c = 0; c < 4; ++c) dev::tmem_ld32(t_s + c * 32, r[c]);
  dev::tmem_wait_ld();
  if (rem < kTileRows) {
#pragma unroll
    for (int c = 0; c < 128; ++c)
      if (c >= rem) r[c >> 5][c & 31] = __float_as_uint(-INFINITY);
  }
}

// fp8: 32 accumulator columns times their V channel scales (fp32).
__device__ __forceinline__ void scale_by_channel(uint32_t (&ov)[32], const float* sv) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(sv) + i);
    ov[4 * i] = __float_as_uint(__uint_as_float(ov[4 * i]) * s4.x);
    ov[4 * i + 1] = __float_as_uint(__uint_as_float(ov[4 * i + 1]) * s4.y);
    ov[4 * i + 2] = __float_as_uint(__uint_as_float(ov[4 * i + 2]) * s4.z);
    ov[4 * i + 3] = __float_as_uint(__uint_as_float(ov[4 * i + 3]) * s4.w);
  }
}

// Fused Q prologue for one query row held in shared memory (128-byte swizzled
// K-major tile, two 16 KB halves): RMSNorm with gain and the rot96 rotation,
// in place, with the arithmetic of qk_norm.cuh (the same bits as the
// separate prologue kernel).  Rare (once per row per unit), so kept out of line.
static __device__ __noinline__ void norm_rope_q_row(uint32_t tile, uint32_t r, const float* gain,
                                                    const float2* rope_row, float eps) {
  auto chunk = [&](int c) {  // shared address of dims [8c, 8c + 8) of row r
    return tile + (uint32_t)(c >> 3) * kQHalfBytes + r * 128u + ((((uint32_t)c & 7u) ^ (r & 7u)) << 4);
  };
  auto ld = [&](int c) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(chunk(c)));
    return v;
  };
  auto st = [&](int c, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(chunk(c)), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
  };
  float p[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    float x[8];
    qkn::unpack8(ld(c), x);
    p[c] = qkn::chunk_ss(x);
  }
  const float rr = qkn::inv_rms(qkn::tree16(p), eps);
#pragma unroll 1
  for (int c = 0; c < 6; ++c) {
    float xa[8], xb[8], ya[8], yb[8], cs[8], sn[8];
    qkn::unpack8(ld(c), xa);
    qkn::unpack8(ld(c + 6), xb);
    const float4* ga = reinterpret_cast<const float4*>(gain + 8 * c);
    const float4* gb = reinterpret_cast<const float4*>(gain + 48 + 8 * c);
    const float4 a0 = __ldg(ga), a1 = __ldg(ga + 1), b0 = __ldg(gb), b1 = __ldg(gb + 1);
    const float gav[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
    const float gbv[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
    const float4* t = reinterpret_cast<const float4*>(rope_row + 8 * c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(t + i);  // (cos, sin) of two consecutive angles
      cs[2 * i] = v.x;
      sn[2 * i] = v.y;
      cs[2 * i + 1] = v.z;
      sn[2 * i + 1] = v.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ya[e] = qkn::scale_gain(xa[e], rr, gav[e]);
      yb[e] = qkn::scale_gain(xb[e], rr, gbv[e]);
    }
    float oa[8], ob[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      oa[e] = qkn::rot_lo(ya[e], yb[e], cs[e], sn[e]);
      ob[e] = qkn::rot_hi(yb[e], ya[e], cs[e], sn[e]);
    }
    st(c, qkn::pack8(oa));
    st(c + 6, qkn::pack8(ob));
  }
#pragma unroll 1
  for (int c = 12; c < 16; ++c) {
    float x[8];
    qkn::unpack8(ld(c), x);
    const float4* g = reinterpret_cast<const float4*>(gain + 8 * c);
    const float4 g0 = __ldg(g), g1 = __ldg(g + 1);
    const float gv[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = qkn::scale_gain(x[e], rr, gv[e]);
    st(c, qkn::pack8(x));
  }
}

// kFp8: the FP8 variant -- e4m3 Q, K, V (V transposed, keys contiguous) with
// scales (per query row, per key tile, per V channel), kind::f8f6f4 MMAs,
// P rounded to e4m3; everything else as the bf16 kernel.
// kWalk: the key tiles a unit visits (bf16 only where not its own document).
template <bool kFp8, int kWalk, bool kPair>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attn_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                       ForwardArgs a, int o_tma, const __grid_constant__ Walk<kWalk> walk) {
  static_assert(!kFp8 || kWalk == kWalkDoc, "the FP8 pipeline walks documents");
  static_assert(!kPair || kWalk != kWalkDoc, "two streams: the other walks");
  using C = Cfg<kFp8, kPair>;
  constexpr int kSlots = C::Slots, kGroups = C::Groups;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = dev::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (sbase - raw);
  const Bars<kGroups> bars{sbase + C::SmemBar};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SmemMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::SmemMisc + 4);

  const uint32_t warp = dev::warp_id_uniform();
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t rank = dev::cluster_ctarank();   // 0: issues the pair's MMAs
  const int pair = (int)(blockIdx.x >> 1);
  // this pair's segments, in order (kPair: stream s's first and last in unit_off[4 pair + 2 s] and after it)
  const int u_begin = kPair ? 0 : __ldg(a.unit_off + pair), u_end = kPair ? 0 : __ldg(a.unit_off + pair + 1);
  const auto stream_begin = [&](int s) { return __ldg(a.unit_off + 4 * pair + 2 * s); };
  const auto stream_end = [&](int s) { return __ldg(a.unit_off + 4 * pair + 2 * s + 1); };
  // kPair: at 4 (4 s + (ordinal & 3)): a segment's steps, the first of its steps
  // over a table's own tile (prefix walk; none: the steps), and that entry
  volatile int* const steps_of = reinterpret_cast<volatile int*>(smem + C::SmemSteps);

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) {
      dev::mbar_init(bars.q_full(i), 1);
      // FP8: freed by the MMA issuer after a unit's last QK; bf16: by the
      // O-store thread, once the TMA unit has read the O rows the epilogue
      // staged in the slot
      dev::mbar_init(bars.q_empty(i), 1);
      dev::mbar_init(bars.o_staged(i), 4);
      dev::mbar_init(bars.q_ready(i), 2);           // the Q warp of each CTA of the pair
    }
    for (int s = 0; s < 2; ++s) {
      for (int h = 0; h < 2; ++h) {
        dev::mbar_init(bars.s_ready(s, h), 1);
        dev::mbar_init(bars.p_ready(s, h), 8);      // one arrival per softmax warp of the pair
        dev::mbar_init(bars.pv_done(s, h), 1);
      }
    }
    for (int i = 0; i < kGroups; ++i) {
      dev::mbar_init(bars.kv_full(i), 1);
      dev::mbar_init(bars.kv_empty(i), 1);
    }
    dev::mbar_init(bars.drain(), 1);
    dev::fence_barrier_init();
  }
  if constexpr (kWalk == kWalkCausal) {
    // Rows of a tile that no load fills, where the pack does not divide 128.  (Left as
    // they were, their scores could be anything, and every new maximum among them made
    // the warp rescale O: 1,836 against 1,683 us for 20,423 tokens, packs of seven.)
    if (walk.pack * walk.toks < kTileRows) {
      for (uint32_t i = threadIdx.x * 16u; i < C::SmemKV; i += kThreads * 16u)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sbase + C::SmemQ + i), "r"(0u) : "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
  }
  if (warp == kTmaWarp && lane == 0) {
    dev::tma_prefetch_desc(&tm_q);
    dev::tma_prefetch_desc(&tm_k);
    dev::tma_prefetch_desc(&tm_v);
    if constexpr (kWalk == kWalkPrefix) {
      dev::tma_prefetch_desc(&walk.tm_k);
      dev::tma_prefetch_desc(&walk.tm_v);
    }
  }
  if (warp == kMmaWarp) {
    dev::tmem_alloc_pair(dev::smem_u32(tmem_slot), kTmemCols);
    dev::tmem_relinquish_pair();
  }
  dev::tc_fence_before();
  __syncthreads();
  __syncwarp();
  dev::cluster_sync();  // both CTAs' barriers are initialised before any cross-CTA arrival
  dev::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // the tensor map of a walk's tile
  const auto k_map = [&](const KeyTile& t) {
    if constexpr (kWalk == kWalkPrefix) return t.prefix ? &walk.tm_k : &tm_k;
    return &tm_k;
  };
  const auto v_map = [&](const KeyTile& t) {
    if constexpr (kWalk == kWalkPrefix) return t.prefix ? &walk.tm_v : &tm_v;
    return &tm_v;
  };

  if (kPair && (warp == kTmaWarp || warp == kQWarp)) {
    // ------------------------------------------- kPair: a stream's loads ----
    if constexpr (kPair) {
      const int st = warp == kQWarp ? 1 : 0;
      const int ub = stream_begin(st), ue = stream_end(st);
      if (lane == 0) {
        const uint64_t pol_q = dev::policy_evict_first(), pol_kv = dev::policy_evict_last();
        bool ok = true;
        uint32_t n = 0;      // groups loaded
        int loaded_q = 0;
        int4 entry = {};     // of the tile whose K was sent last
        for (int u = ub; ok && u < ue; ++u) {
          const UnitGeom g = unit_geom<kWalk>(a.units, u, walk);
          // Q: free since the last QK of the segment before (whose last group,
          // with this segment's first K, is on its way)
          ok = dev::mbar_wait(bars.q_empty(st), ((u - ub) & 1) ^ 1, abort_flag, a.err, kTimeoutNs);
          if (!ok) break;
          volatile int* const info = steps_of + 4 * (4 * st + ((u - ub) & 3));  // (the issuer reads it after Q-ready)
          info[0] = g.hi - g.lo;
          info[1] = g.hi - g.lo;
          if constexpr (kWalk == kWalkPrefix)
            if (g.n > 0) {
              info[1] = walk.tiles - g.lo;
              info[2] = g.kv0;
            }
          const uint32_t dst = sbase + C::SmemQ + st * C::QTileBytes;
          const int32_t row = tile_row<kWalk, kPair>(g, st, rank, walk);
          load_q_tile<kWalk>(dst, &tm_q, bars.q_full(st), g.head, row, pol_q, walk);
          ++loaded_q;
          if (u == ub) {
            ok = dev::mbar_wait(bars.kv_empty(2 * st), 1, abort_flag, a.err, kTimeoutNs);
            if (!ok) break;
            entry = walk_entry<kWalk>(g, g.lo, walk);
            const KeyTile t = key_tile<kWalk>(g, g.lo, entry, walk);
            dev::mbar_arrive_expect_tx(bars.kv_full(2 * st), C::SlotBytes);
            load_k_half<kFp8>(sbase + C::SmemKV + (4 * st + 1) * C::SlotBytes, k_map(t), bars.kv_full(2 * st),
                              key_head<kWalk>(g), t.row, rank, pol_kv);
            n = 1;
          }
          for (int j = g.lo; ok && j < g.hi; ++j) {
            const KeyTile vt = key_tile<kWalk>(g, j, entry, walk);
            KeyTile kt = vt;
            int k_head = key_head<kWalk>(g);
            const bool has_k = j + 1 < g.hi || u + 1 < ue;
            if (j + 1 < g.hi) {
              entry = walk_entry<kWalk>(g, j + 1, walk);
              kt = key_tile<kWalk>(g, j + 1, entry, walk);
            } else if (has_k) {
              const UnitGeom gn = unit_geom<kWalk>(a.units, u + 1, walk);
              entry = walk_entry<kWalk>(gn, gn.lo, walk);
              kt = key_tile<kWalk>(gn, gn.lo, entry, walk);
              k_head = key_head<kWalk>(gn);
            }
            if (vt.bad && rank == 0) dev::report_bad_tile(a.err);
            const uint32_t b = 2 * st + (n & 1);
            ok = dev::mbar_wait(bars.kv_empty(b), ((n >> 1) & 1) ^ 1, abort_flag, a.err, kTimeoutNs);
            if (!ok) break;
            const uint32_t slot = sbase + C::SmemKV + (4 * st + 2 * (n & 1)) * C::SlotBytes;
            dev::mbar_arrive_expect_tx(bars.kv_full(b), has_k ? 2 * C::SlotBytes : C::SlotBytes);
            load_v_half<kFp8>(slot, v_map(vt), bars.kv_full(b), key_head<kWalk>(g), vt.row, rank, pol_kv);
            if (has_k) load_k_half<kFp8>(slot + C::SlotBytes, k_map(kt), bars.kv_full(b), k_head, kt.row, rank, pol_kv);
            ++n;
          }
        }
        if (!ok) {  // drain: wait (bounded) for the copies on their way
          for (uint32_t x = 1; x <= 2 && x <= n; ++x)
            dev::mbar_wait_bounded(bars.kv_full(2 * st + ((n - x) & 1)), ((n - x) >> 1) & 1, nullptr, nullptr, kTimeoutNs);
          if (loaded_q) dev::mbar_wait_bounded(bars.q_full(st), (loaded_q - 1) & 1, nullptr, nullptr, kTimeoutNs);
        }
      } else if (lane == 1) {
        // Q-ready counts one arrival per CTA; before the first one, the stream's
        // first K tile must have landed too
        bool ok = true;
        for (int u = ub; ok && u < ue; ++u) {
          ok = dev::mbar_wait(bars.q_full(st), (u - ub) & 1, abort_flag, a.err, kTimeoutNs);
          if (ok && u == ub) ok = dev::mbar_wait(bars.kv_full(2 * st), 0, abort_flag, a.err, kTimeoutNs);
          if (ok) dev::mbar_arrive_cluster(dev::mapa_shared(bars.q_ready(st), 0));
        }
      }
      __syncwarp();
    }
  } else if (warp == kTmaWarp) {
    // ------------------------------------------------------ TMA producer ----
    if (!kFp8 && lane == 1) {
      // bf16 O stores: as the four softmax warps of a query tile finish a
      // unit's epilogue, send the rows they staged in its Q slot (every warp
      // whose 32 rows lie in the document) with TMA tile stores, wait until
      // they have read the slot, and free it for the Q warp's next load.
      uint32_t use[4] = {0, 0, 0, 0};
      bool ok = true;
      int k = 0;
      for (int u = u_begin; ok && u < u_end; ++u, ++k) {
        const UnitGeom g = unit_geom<kWalk>(a.units, u, walk);
#pragma unroll 1
        for (int s = 0; s < 2 && s < g.n_st; ++s) {
          const int i = q_slot_of<kPair>(k, s);
          ok = dev::mbar_wait(bars.o_staged(i), use[i] & 1, abort_flag, a.err, kTimeoutNs);
          ++use[i];
          if (!ok) break;
          if (o_tma != 0 && g.part < 0) {
            const uint32_t tile = sbase + C::SmemQ + i * C::QTileBytes;
            const int32_t base_row = tile_row<kWalk, kPair>(g, s, rank, walk);
            bool any = false;
            int warp_toks = 32;  // rows (tokens) of a warp
            if constexpr (kWalk == kWalkCausal) warp_toks = walk.toks / 4;
#pragma unroll 1
            for (int w = 0; w < 4; ++w) {
              const int32_t row0 = base_row + warp_toks * w;
              if (row0 + warp_toks - 1 >= g.q1) break;  // (the softmax warps' own test)
              if constexpr (kWalk == kWalkCausal) {
                dev::tma_store_3d(&tm_o, tile + 32u * w * 128u, 0, g.head, row0);
                dev::tma_store_3d(&tm_o, tile + kQHalfBytes + 32u * w * 128u, 64, g.head, row0);
              } else {
                dev::tma_store_2d(&tm_o, tile + 32u * w * 128u, g.head * kHeadDim, row0);
                dev::tma_store_2d(&tm_o, tile + kQHalfBytes + 32u * w * 128u, g.head * kHeadDim + 64, row0);
              }
              any = true;
            }
            if (any) {
              dev::bulk_commit();
              dev::bulk_wait_read_all();
            }
          }
          dev::mbar_arrive(bars.q_empty(i));
        }
      }
      dev::bulk_wait_all();  // the O stores are complete
    }
    if (lane == 0) {
      const uint64_t pol_q = dev::policy_evict_first();
      const uint64_t pol_kv = dev::policy_evict_last();
      uint32_t grp = 0, q_use[4] = {0, 0, 0, 0};
      bool ok = true;
      // FP8: Q tiles of the unit with ordinal k, into buffer k & 1 (the slot
      // is freed by the MMA after the last QK of the unit two before).
      auto load_q = [&](const UnitGeom& g, int k) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok || s >= g.n_st) break;
          const int i = 2 * (k & 1) + s;
          ok = dev::mbar_wait(bars.q_empty(i), (q_use[i] & 1) ^ 1, abort_flag, a.err, kTimeoutNs);
          if (!ok) break;
          const uint32_t dst = sbase + C::SmemQ + i * C::QTileBytes;
          dev::mbar_arrive_expect_tx(bars.q_full(i), C::QTileBytes);
          const int32_t row = g.q0 + s * 2 * kTileRows + (int32_t)rank * kTileRows;
          dev::tma_load_2d(dst, &tm_q, bars.q_full(i), g.head * 128, row, pol_q);
          if constexpr (!kFp8)
            dev::tma_load_2d(dst + kQHalfBytes, &tm_q, bars.q_full(i), g.head * 128 + 64, row, pol_q);
          ++q_use[i];
        }
      };
      int k = 0;
      KeyTile kt;  // the tile whose K was sent last (dense: only its row is used)
      for (int u = u_begin; ok && u < u_end; ++u, ++k) {
        const UnitGeom g = unit_geom<kWalk>(a.units, u, walk);
        const bool has_next = u + 1 < u_end;
        // Key/value groups: group 0 is the first unit's first K tile (ring slot
        // 0); group n >= 1 is V(j) with the next K tile -- K(j+1), or the next
        // unit's first K tile -- in slots (2n-1) % kSlots and 2n % kSlots, one
        // full and one empty barrier (index n % kGroups) for both.
        if (k == 0) {
          if constexpr (kFp8) load_q(g, 0);
          if (!ok) break;
          ok = dev::mbar_wait(bars.kv_empty(0), 1, abort_flag, a.err, kTimeoutNs);
          if (!ok) break;
          dev::mbar_arrive_expect_tx(bars.kv_full(0), C::SlotBytes);
          if constexpr (kWalk == kWalkDoc) {
            load_k_half<kFp8>(sbase + C::SmemKV, &tm_k, bars.kv_full(0), g.head, g.kv0 + g.lo * kTileRows, rank,
                              pol_kv);
          } else {
            kt = key_tile<kWalk>(g, g.lo, walk_entry<kWalk>(g, g.lo, walk), walk);
            load_k_half<kFp8>(sbase + C::SmemKV, k_map(kt), bars.kv_full(0), key_head<kWalk>(g), kt.row, rank, pol_kv);
          }
          grp = 1;
        }
        for (int j = g.lo; ok && j < g.hi; ++j) {
          bool has_k = j + 1 < g.hi;
          int k_head = key_head<kWalk>(g);
          const KeyTile vt = kt;  // this step's tile: its K went out a step ago
          if constexpr (kWalk == kWalkDoc) {
            kt.row = g.kv0 + (j + 1) * kTileRows;
          } else {
            if (has_k) kt = key_tile<kWalk>(g, j + 1, walk_entry<kWalk>(g, j + 1, walk), walk);
            if (vt.bad && rank == 0) dev::report_bad_tile(a.err);
          }
          if (!has_k && has_next) {
            const UnitGeom n = unit_geom<kWalk>(a.units, u + 1, walk);
            has_k = true;
            k_head = key_head<kWalk>(n);
            if constexpr (kWalk == kWalkDoc)
              kt.row = n.kv0 + n.lo * kTileRows;
            else
              kt = key_tile<kWalk>(n, n.lo, walk_entry<kWalk>(n, n.lo, walk), walk);
          }
          const uint32_t b = grp % kGroups;
          ok = dev::mbar_wait(bars.kv_empty(b), ((grp / kGroups) & 1) ^ 1, abort_flag, a.err, kTimeoutNs);
          if (!ok) break;
          dev::mbar_arrive_expect_tx(bars.kv_full(b), has_k ? 2 * C::SlotBytes : C::SlotBytes);
          if constexpr (kWalk == kWalkDoc)
            load_v_half<kFp8>(sbase + C::SmemKV + ((2 * grp - 1) % kSlots) * C::SlotBytes, &tm_v, bars.kv_full(b),
                              g.head, (kFp8 ? g.v_off : g.kv0) + j * kTileRows, rank, pol_kv);
          else
            load_v_half<kFp8>(sbase + C::SmemKV + ((2 * grp - 1) % kSlots) * C::SlotBytes, v_map(vt), bars.kv_full(b),
                              key_head<kWalk>(g), vt.row, rank, pol_kv);
          if (has_k) {
            if constexpr (kWalk == kWalkDoc)
              load_k_half<kFp8>(sbase + C::SmemKV + ((2 * grp) % kSlots) * C::SlotBytes, &tm_k, bars.kv_full(b),
                                k_head, kt.row, rank, pol_kv);
            else
              load_k_half<kFp8>(sbase + C::SmemKV + ((2 * grp) % kSlots) * C::SlotBytes, k_map(kt), bars.kv_full(b),
                                k_head, kt.row, rank, pol_kv);
          }
          ++grp;
          // the next unit's Q tiles, behind this unit's first group
          if constexpr (kFp8)
            if (j == g.lo && has_next) load_q(unit_geom<kWalk>(a.units, u + 1, walk), k + 1);
        }
      }
      if (!ok) {
        // drain: wait (bounded) for every copy this thread issued into the ring and Q
        for (uint32_t r = 1; r <= (uint32_t)kGroups && r <= grp; ++r) {
          const uint32_t n = grp - r;
          dev::mbar_wait_bounded(bars.kv_full(n % kGroups), (n / kGroups) & 1, nullptr, nullptr, kTimeoutNs);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (q_use[i]) dev::mbar_wait_bounded(bars.q_full(i), (q_use[i] - 1) & 1, nullptr, nullptr, kTimeoutNs);
      }
    }
  } else if (warp == kMmaWarp) {
    // ----------------------------------------- MMA issuer (even CTA, pair) ----
    if constexpr (kFp8) {
      // FP8: whole 128-key tiles (S of a query tile is one barrier phase, P
      // overwrites it), issued by one thread.  Its MMAs are half as long as
      // bf16's, and the halved pipeline measured slower here: the per-half
      // softmax costs would dominate.
      if (lane == 0 && rank == 0) {
        uint32_t vslot = 1, kslot = 2, q_use[4] = {0, 0, 0, 0}, p_it[2] = {0, 0};
        bool ok = true;
        bool issued = false;
        int k = 0;
        for (int u = u_begin; ok && u < u_end; ++u, ++k) {
          const UnitGeom g = unit_geom<kWalk>(a.units, u, walk);
          const uint32_t qb = 2 * (k & 1);
          // Q tiles of this unit, prepared in both CTAs (and, for the first
          // unit, the first K group landed in both)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!ok || s >= g.n_st) break;
            ok = dev::mbar_wait(bars.q_ready(qb + s), q_use[qb + s] & 1, abort_flag, a.err, kTimeoutNs);
            ++q_use[qb + s];
          }
          // this unit's first K tile: group 0, or the K half of the previous
          // unit's last group (covered by that unit's last P-ready barrier)
          const uint32_t k0 = k == 0 ? 0u : (kslot >= 2 ? kslot - 2 : kslot + kSlots - 2);
          if (!ok) break;
          dev::tc_fence_after();
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (s >= g.n_st) break;
            issue_qk_f8(tmem + s * 128, sbase + C::SmemQ + (qb + s) * C::QTileBytes, sbase + C::SmemKV + k0 * C::SlotBytes);
            dev::mma_commit_pair_mc(bars.s_ready(s, 0), kPairMask);
            if (g.hi - g.lo == 1) dev::mma_commit_pair_mc(bars.q_empty(qb + s), kPairMask);
          }
          issued = true;
          for (int j = g.lo; j < g.hi; ++j) {
            // group grp = V(j) + the next K tile; its arrival in both CTAs is
            // implied by P-ready of query tile 0
            const bool more = j + 1 < g.hi;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              if (s >= g.n_st) break;
              ok = dev::mbar_wait(bars.p_ready(s, 0), p_it[s] & 1, abort_flag, a.err, kTimeoutNs);
              if (!ok) break;
              ++p_it[s];
              dev::tc_fence_after();
              issue_pv_f8(tmem + 256 + s * 128, tmem + s * 128, sbase + C::SmemKV + vslot * C::SlotBytes, j > g.lo);
              if (more) {
                issue_qk_f8(tmem + s * 128, sbase + C::SmemQ + (qb + s) * C::QTileBytes,
                            sbase + C::SmemKV + kslot * C::SlotBytes);
                dev::mma_commit_pair_mc(bars.s_ready(s, 0), kPairMask);
                if (j + 2 == g.hi) dev::mma_commit_pair_mc(bars.q_empty(qb + s), kPairMask);
              } else {
                dev::mma_commit_pair_mc(bars.pv_done(s, 0), kPairMask);  // the unit's O is complete
              }
            }
            if (!ok) break;
            vslot = vslot + 2 >= (uint32_t)kSlots ? vslot + 2 - kSlots : vslot + 2;
            kslot = kslot + 2 >= (uint32_t)kSlots ? kslot + 2 - kSlots : kslot + 2;
          }
        }
        if (!ok && issued) {
          // drain: every MMA issued so far must finish before TMEM is freed
          dev::mma_commit_pair(bars.drain());
          dev::mbar_wait_bounded(bars.drain(), 0, nullptr, nullptr, kTimeoutNs);
        }
      }
    } else if constexpr (kPair) {
      if (rank == 0) {
        // Two streams: the whole warp runs the loop; lane s polls stream s's next
        // barrier without blocking, and the warp serves the streams that are ready.
        // Per stream, its segments' steps are awaited as in the other issuer, so the
        // order of a stream's MMAs (PV, then the next QK into the same columns) is
        // the same.
        int left[2], hi[2] = {0, 0}, j[2] = {0, 0}, h[2] = {0, 0};  // segments to go; steps, step and half of this one
        uint32_t t[2] = {0, 0}, k[2] = {0, 0};  // steps and segments of the stream so far
        bool first[2] = {true, true};           // the next barrier is Q-ready
        int own_from[2] = {0, 0}, own0[2] = {0, 0};  // prefix walk: first step over an own tile, and its entry
        uint4 skip[2][2];                       // lanes that the own tile's PV leaves alone, loaded a step ahead
        bool ok = true, issued = false;
#pragma unroll
        for (int s = 0; s < 2; ++s) left[s] = stream_end(s) - stream_begin(s);
        bool hold = left[0] > 1;                // stream 1 waits until stream 0 is ahead
        uint64_t since = 0;                     // when nothing has been ready from
        uint32_t idle = 0;
        // serves stream s
        auto serve = [&](const int s) {
          dev::tc_fence_after();
          const uint32_t d = tmem + s * 128, qa = sbase + C::SmemQ + s * C::QTileBytes;
          // K(t) lies in group t, V(t) and K(t + 1) in group t + 1
          const uint32_t ring = sbase + C::SmemKV + 4 * s * C::SlotBytes;
          if (first[s]) {
            const uint32_t kb = ring + (2 * (t[s] & 1) + 1) * C::SlotBytes;
            const volatile int* const info = steps_of + 4 * (4 * s + (k[s] & 3));
            hi[s] = info[0];
            if constexpr (kWalk == kWalkPrefix) {
              own_from[s] = info[1];
              own0[s] = info[2];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              issue_qk(d + 64 * x, qa, kb + x * kHalfKeyRowsBytes);
              commit_pair_elect(bars.s_ready(s, x));
            }
            if (hi[s] == 1) commit_pair_elect(bars.q_empty(s));
            ++k[s];
            first[s] = false;
            issued = true;
            return;
          }
          const uint32_t vb = ring + 2 * ((t[s] + 1) & 1) * C::SlotBytes;
          if (kWalk == kWalkPrefix && j[s] >= own_from[s])
            issue_pv_skip(tmem + 256 + s * 128, d + 64 * h[s], vb + 4096 * h[s], true, skip[s][0], skip[s][1]);
          else
            issue_pv(tmem + 256 + s * 128, d + 64 * h[s], vb + 4096 * h[s], j[s] > 0 || h[s] == 1);
          if (j[s] + 1 < hi[s]) {
            issue_qk(d + 64 * h[s], qa, vb + C::SlotBytes + h[s] * kHalfKeyRowsBytes);
            commit_pair_elect(bars.s_ready(s, 0) + 8 * h[s]);
            if (h[s] == 1 && j[s] + 2 == hi[s]) commit_pair_elect(bars.q_empty(s));
          } else {
            commit_pair_elect(bars.pv_done(s, 0) + 8 * h[s]);
          }
          if (h[s] == 1) {
            ++t[s];
            if (++j[s] == hi[s]) {
              j[s] = 0;
              --left[s];
              first[s] = true;
            } else if constexpr (kWalk == kWalkPrefix) {
              if (j[s] >= own_from[s]) {
                const uint4* p = reinterpret_cast<const uint4*>(walk.own[own0[s] + j[s] - own_from[s]].skip[0]);
                skip[s][0] = __ldg(p);
                skip[s][1] = __ldg(p + 1);
              }
            }
          }
          h[s] ^= 1;
        };
        while (ok && (left[0] > 0 || left[1] > 0)) {
          bool good = false;
          if (lane < 2) {
            const bool one = lane == 1;
            const bool f = one ? first[1] : first[0];
            const uint32_t hh = one ? h[1] : h[0], n = f ? (one ? k[1] : k[0]) : (one ? t[1] : t[0]);
            if ((one ? left[1] : left[0]) > 0 && !(one && hold))
              good = dev::mbar_test_wait(f ? bars.q_ready((int)lane) : bars.p_ready((int)lane, 0) + 8 * hh, n & 1);
          }
          const unsigned ready = __ballot_sync(0xffffffffu, good);
          if (ready & 1u) serve(0);
          if (ready & 2u) serve(1);
          hold = hold && left[0] > 0 && (t[0] == 0 || t[0] < min((uint32_t)hi[0] / 2, kHoldSteps));
          if (ready != 0) {
            idle = 0;
          } else if ((++idle & 63u) == 0) {  // bounded: two seconds of nothing, or another thread's abort
            const uint64_t now = dev::globaltimer_ns();
            if (idle == 64) since = now;
            bool stop = false;
            if (lane == 0) {
              stop = *abort_flag != 0;
              if (!stop && now - since > kTimeoutNs) {
                *abort_flag = 1;
                atomicExch(a.err, kErrTimeout);
                stop = true;
              }
            }
            ok = !__shfl_sync(0xffffffffu, stop, 0);
          }
        }
        if (!ok && issued) {
          // drain: every MMA issued so far must finish before TMEM is freed
          __syncwarp();
          commit_pair_local_elect(bars.drain());
          dev::mbar_wait_bounded(bars.drain(), 0, nullptr, nullptr, kTimeoutNs);
        }
      }
    } else if (rank == 0) {
    // bf16: the whole warp runs the loop (its values stay warp-uniform); every
    // tcgen05 MMA and commit is issued by one elected lane.
      // ring slots of the current group's V and K halves: group n uses slots
      // 2n-1 and 2n (mod kSlots), advanced by two per key tile without a division
      uint32_t vslot = 1, kslot = 2, q_use[4] = {0, 0, 0, 0};
      uint32_t p_it[2][2] = {{0, 0}, {0, 0}};
      bool ok = true;
      bool issued = false;
      int k = 0;
      // QK of half h of the key tile in ring slot ks for query tile s (Q slot qs)
      auto qk_half = [&](int s, uint32_t qs, uint32_t ks, int h) {
        const uint32_t d = tmem + s * 128 + h * 64;
        const uint32_t qa = sbase + C::SmemQ + qs * C::QTileBytes;
        const uint32_t kb = sbase + C::SmemKV + ks * C::SlotBytes + h * kHalfKeyRowsBytes;
        issue_qk(d, qa, kb);
        commit_pair_elect(bars.s_ready(s, h));
      };
      // PV of half h of the key tile whose V is in ring slot vs, query tile s
      auto pv_half = [&](int s, uint32_t vs, int h, bool acc) {
        const uint32_t d = tmem + 256 + s * 128, pt = tmem + s * 128 + h * 64;
        const uint32_t vb = sbase + C::SmemKV + vs * C::SlotBytes;
        issue_pv(d, pt, vb + 4096 * h, acc);
      };
      // Prefix walk: the same for an own tile of a segment over several documents,
      // which leaves the other documents' rows alone: their lanes, for query tile
      // s in skip[2 s] and skip[2 s + 1], loaded a tile ahead.
      uint4 skip[4];
      auto load_skip = [&](const UnitGeom& g, int j) {
        if constexpr (kWalk == kWalkPrefix) {
          const uint4* p = reinterpret_cast<const uint4*>(walk.own[g.kv0 + (j - walk.tiles)].skip);
#pragma unroll
          for (int x = 0; x < 4; ++x) skip[x] = __ldg(p + x);
        }
      };
      auto pv_half_skip = [&](int s, uint32_t vs, int h) {
        const uint32_t d = tmem + 256 + s * 128, pt = tmem + s * 128 + h * 64;
        const uint32_t vb = sbase + C::SmemKV + vs * C::SlotBytes;
        issue_pv_skip(d, pt, vb + 4096 * h, true, s == 0 ? skip[0] : skip[2], s == 0 ? skip[1] : skip[3]);
      };
      // The first QK (half h) of query tile s of a unit: Q slot qs (its readiness
      // in both CTAs is awaited before half 0), K in ring slot ks.
      auto first_qk = [&](uint32_t qs, uint32_t ks, int s, int h) {
        if (h == 0) {
          ok = __all_sync(0xffffffffu,
                          dev::mbar_wait(bars.q_ready(qs), q_use[qs] & 1, abort_flag, a.err, kTimeoutNs));
          ++q_use[qs];
          if (!ok) return;
          dev::tc_fence_after();
        }
        qk_half(s, qs, ks, h);
        issued = true;
      };
      auto advance = [&]() {
        vslot = vslot + 2 >= (uint32_t)kSlots ? vslot + 2 - kSlots : vslot + 2;
        kslot = kslot + 2 >= (uint32_t)kSlots ? kslot + 2 - kSlots : kslot + 2;
      };
      for (int u = u_begin; ok && u < u_end; ++u, ++k) {
        const UnitGeom g = unit_geom<kWalk>(a.units, u, walk);
        const uint32_t q_at[2] = {(uint32_t)q_slot_of<kPair>(k, 0), (uint32_t)q_slot_of<kPair>(k, 1)};
        if (k == 0) {
          // the pair's first unit: its first K tile is group 0 (ring slot 0),
          // and Q-ready also covers that group's arrival in both CTAs
          for (int h = 0; ok && h < 2; ++h)
            for (int s = 0; ok && s < g.n_st; ++s) first_qk(q_at[s], 0, s, h);
          if (!ok) break;
        }
        // Per key tile j and half h, for each query tile s: wait for P(s, j, h),
        // then PV(s, j, h) and QK(s, j + 1, h) -- the next key tile's S half
        // goes where P(s, j, h) was, and the softmax works on the other half
        // meanwhile.  In the last key tile all PVs go first (the epilogue
        // waits for them), then the next unit's first QKs.  The next unit's
        // first key tile is the K half of this unit's last group (ring slot
        // kslot in the last key tile); its group is released when the next
        // unit's last query tile sees S of half 1, so that QK comes after
        // every PV of this unit.
        const bool has_next = u + 1 < u_end;
        const UnitGeom gn = unit_geom<kWalk>(a.units, has_next ? u + 1 : u, walk);
        const bool two = g.n_st == 2;
        // steady state: key tiles with a next key tile in this unit
        // (prefix walk: those before the own tiles of a segment over several
        // documents, which a loop of their own takes: selecting between the two
        // PVs here cost the steady state 10 %)
        int j_own = g.hi;
        if constexpr (kWalk == kWalkPrefix)
          if (g.n > 0) j_own = walk.tiles;
        const int j_end = min(g.hi - 1, j_own);
        for (int j = g.lo; ok && j < j_end; ++j) {
          const bool acc0 = j > g.lo;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              if (s == 1 && !two) break;
              // one lane polls P; the warp follows it
              bool good = true;
              if (lane == 0) good = dev::mbar_wait(bars.p_ready(s, h), p_it[s][h] & 1, abort_flag, a.err, kTimeoutNs);
              ok = __shfl_sync(0xffffffffu, good, 0);
              if (!ok) break;
              ++p_it[s][h];
              dev::tc_fence_after();
              pv_half(s, vslot, h, acc0 || h == 1);
              qk_half(s, q_at[s], kslot, h);
            }
            if (!ok) break;
          }
          advance();
        }
        if constexpr (kWalk == kWalkPrefix) {
          if (g.hi > j_own) load_skip(g, j_own);
#pragma unroll 1
          for (int j = j_own; ok && j + 1 < g.hi; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                if (s == 1 && !two) break;
                ok = __all_sync(0xffffffffu,
                                dev::mbar_wait(bars.p_ready(s, h), p_it[s][h] & 1, abort_flag, a.err, kTimeoutNs));
                if (!ok) break;
                ++p_it[s][h];
                dev::tc_fence_after();
                pv_half_skip(s, vslot, h);
                qk_half(s, q_at[s], kslot, h);
              }
              if (!ok) break;
            }
            load_skip(g, j + 1);
            advance();
          }
        }
        if (!ok) break;
        // the last key tile: each PV is followed by "PV done" of its half (the
        // epilogue waits for both halves); the next unit's first QKs follow
        // the last PV, so that the epilogue does not wait behind them
        {
          const bool acc0 = g.hi - 1 > g.lo;
          for (int h = 0; ok && h < 2; ++h) {
#pragma unroll 1
            for (int s = 0; s < g.n_st; ++s) {
              ok = __all_sync(0xffffffffu,
                              dev::mbar_wait(bars.p_ready(s, h), p_it[s][h] & 1, abort_flag, a.err, kTimeoutNs));
              if (!ok) break;
              ++p_it[s][h];
              dev::tc_fence_after();
              if (kWalk == kWalkPrefix && g.hi > j_own)
                pv_half_skip(s, vslot, h);
              else
                pv_half(s, vslot, h, acc0 || h == 1);
              commit_pair_elect(bars.pv_done(s, h));
            }
          }
          if (has_next) {
            for (int h = 0; ok && h < 2; ++h)
              for (int s = 0; ok && s < gn.n_st; ++s) first_qk(q_slot_of<kPair>(k + 1, s), kslot, s, h);
          }
          advance();
        }
      }
      if (!ok && issued) {
        // drain: every MMA issued so far must finish before TMEM is freed
        __syncwarp();
        commit_pair_local_elect(bars.drain());
        dev::mbar_wait_bounded(bars.drain(), 0, nullptr, nullptr, kTimeoutNs);
      }
    }
  } else if (warp == kQWarp) {
    // ----------------------------------------------------------- Q warp ----
    // As each of this CTA's Q tiles lands: with the fused Q prologue,
    // normalise and rotate its rows in place (lane l takes rows l, l+32, ...);
    // then report the tile ready to the even CTA.  Before the first unit's
    // first tile, the first K group must have landed too.
    uint32_t q_use[4] = {0, 0, 0, 0};
    bool ok = true;
    const bool fuse_q = a.gain_q != nullptr;
    const uint64_t pol_q = dev::policy_evict_first();
    int k = 0;
    for (int u = u_begin; ok && u < u_end; ++u, ++k) {
      const UnitGeom g = unit_geom<kWalk>(a.units, u, walk);
#pragma unroll 1
      for (int s = 0; s < 2 && s < g.n_st; ++s) {
        const int i = q_slot_of<kPair>(k, s);
        bool good = true;
        if constexpr (!kFp8) {
          // bf16: this warp loads the tile once its slot is free (the
          // O-store thread has sent the previous unit's O rows out of it)
          if (lane == 0) {
            good = dev::mbar_wait(bars.q_empty(i), (q_use[i] & 1) ^ 1, abort_flag, a.err, kTimeoutNs);
            if (good) {
              const uint32_t dst = sbase + C::SmemQ + i * C::QTileBytes;
              const int32_t row = tile_row<kWalk, kPair>(g, s, rank, walk);
              load_q_tile<kWalk>(dst, &tm_q, bars.q_full(i), g.head, row, pol_q, walk);
            }
          }
          good = __shfl_sync(0xffffffffu, good, 0);
          if (!good) {
            ok = false;
            break;
          }
        }
        good = dev::mbar_wait(bars.q_full(i), q_use[i] & 1, abort_flag, a.err, kTimeoutNs);
        ++q_use[i];
        if (!kFp8 && kWalk == kWalkDoc && good && fuse_q) {
          const int32_t row0 = g.q0 + s * 2 * kTileRows + (int32_t)rank * kTileRows;
          const float* gain = a.gain_q + (int64_t)g.head * a.gain_head_stride;
#pragma unroll 1
          for (uint32_t r = lane; r < (uint32_t)kTileRows; r += 32) {
            const int32_t row = row0 + (int32_t)r;
            if (row < g.kv1)
              norm_rope_q_row(sbase + C::SmemQ + i * C::QTileBytes, r, gain, a.rope + (int64_t)row * kRopeHalf, a.eps);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // visible to the tensor cores
        }
        __syncwarp();
        if (good && k == 0 && s == 0 && lane == 0)
          good = dev::mbar_wait(bars.kv_full(0), 0, abort_flag, a.err, kTimeoutNs);
        if (lane == 0) dev::mbar_arrive_cluster(dev::mapa_shared(bars.q_ready(i), 0));
        ok = __all_sync(0xffffffffu, good);
        if (!ok) break;
      }
    }
    if constexpr (!kFp8) {
      if (!ok && lane == 0) {
        // drain: wait (bounded) for the Q copies this warp issued
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (q_use[i]) dev::mbar_wait_bounded(bars.q_full(i), (q_use[i] - 1) & 1, nullptr, nullptr, kTimeoutNs);
      }
    }
  } else {
    // ---------------------------------------------------------- softmax ----
    const int st = warp >> 2;            // query tile of this warpgroup
    const uint32_t row_in_tile = threadIdx.x & 127;
    const uint32_t row_in_unit = (kPair ? 0 : st * 2 * kTileRows) + rank * kTileRows + row_in_tile;
    const uint32_t lane_base = (warp & 3) * 32;
    const uint32_t t_s = tmem + (lane_base << 16) + st * 128;        // S_s / P_s
    const uint32_t t_o = tmem + (lane_base << 16) + 256 + st * 128;  // O_s
    const uint32_t p_ready_remote[2] = {dev::mapa_shared(bars.p_ready(st, 0), 0),
                                        dev::mapa_shared(bars.p_ready(st, 1), 0)};
    const bool lead_lane = (warp & 3) == 0 && lane == 0;             // one lane per warpgroup
    uint32_t s_it[2] = {0, 0};
    uint32_t n_done = 0;                 // units this query tile has finished (PV-done phases per half)
    uint32_t t0 = 0;                     // key tiles the pair has started before this unit
    bool ok = true;
    const float sl2 = a.scale_log2;
    __nv_bfloat16* og = static_cast<__nv_bfloat16*>(a.o);
    // 32-byte output stores when every row start is 32-byte aligned
    const bool o_wide = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0 && (a.o_stride & 15) == 0;
    const int us = kPair ? stream_begin(st) : u_begin, ue = kPair ? stream_end(st) : u_end;
    for (int u = us; ok && u < ue; ++u) {
      const UnitGeom g = unit_geom<kWalk>(a.units, u, walk);
      const uint32_t t_unit = t0;
      t0 += g.hi - g.lo;
      if (!kPair && st >= g.n_st) continue;
      const uint32_t q_slot = q_slot_of<kPair>(u - us, st);  // this unit's Q tile of this query tile
      // ring bookkeeping by one lane of one warp per CTA
      // (kPair: each query tile has groups of its own)
      const bool releases = lead_lane && (kPair || st == g.n_st - 1);
      const bool checks_kv = lead_lane && (kPair || st == 0);
      // (other walks: finite, so that the exponents of a row that sees no key are -inf, not NaN)
      float m_used = kWalk == kWalkDoc ? -INFINITY : -3.402823466e38f, l = 0.f;
      // fp8: this row's q scale (1 for rows past the tensor, never stored)
      float sq_row = 1.f;
      if constexpr (kFp8) {
        const int32_t row = g.q0 + st * 2 * kTileRows + (int32_t)rank * kTileRows + (int32_t)row_in_tile;
        if (row < a.S) sq_row = __ldg(a.sq + (int64_t)g.head * a.S + row);
      }
      if constexpr (kFp8) {
        // FP8: whole 128-key tiles, one S phase per key tile.
        for (int j = g.lo; j < g.hi; ++j) {
          const uint32_t t = t_unit + (j - g.lo);  // the pair's running key-tile count
          // score scale in log2 units: softmax_scale log2(e) times the q-row and key-tile scales
          const float rsc = sl2 * sq_row * __ldg(a.sk + (int64_t)g.head * a.S + g.kv0 + j * kTileRows);
          // (every lane runs the same bounded wait on the same barrier, timer and
          // abort flag in step, so the warp leaves it with one value of ok)
          ok = dev::mbar_wait(bars.s_ready(st, 0), s_it[0] & 1, abort_flag, a.err, kTimeoutNs);
          if (!ok) break;
          ++s_it[0];
          // S of the last query tile is ready: every MMA before it is done, so
          // the group holding K(t) (and V(t-1)) is free in this CTA
          if (releases) dev::mbar_arrive(bars.kv_empty(t % kGroups));
          // test, without blocking, whether the next K/V group has landed; the
          // blocking wait below then only runs if it had not
          const uint32_t kv_bar = bars.kv_full((t + 1) % kGroups), kv_par = ((t + 1) / kGroups) & 1;
          const bool kv_landed = checks_kv && dev::mbar_test_wait(kv_bar, kv_par);
          __syncwarp();  // lanes leave the wait separately; the TMEM loads are warp-collective
          dev::tc_fence_after();
          uint32_t r[4][32];
          float* sv = reinterpret_cast<float*>(&r[0][0]);
          const int rem = g.kv1 - (g.kv0 + j * kTileRows);
          load_scores128(t_s, r, rem);
          // Row max: eight independent chains of 3-input maxima.
          float mx[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mx[i] = fmaxf(sv[i], sv[8 + i]);
#pragma unroll
          for (int c = 16; c < 128; c += 16)
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[i] = dev::max3(mx[i], sv[c + i], sv[c + 8 + i]);
          const float m_new =
              dev::max3(dev::max3(mx[0], mx[1], mx[2]), dev::max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * rsc;
          // The reference max only moves when the row max grows by more than
          // 2^8 (then O and l are rescaled; the final O / l is unchanged).  The
          // O row is rescaled after P is written: the next PV waits for p_ready.
          float alpha = 1.f;
          if (m_new > m_used + kRescaleThreshold) {
            alpha = dev::ex2_approx(m_used - m_new);  // 0 on the first tile (m_used = -inf)
            m_used = m_new;
          }
          const float neg = -m_used;
          float rs8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t p[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              // packed pair arithmetic: one f32x2 FMA for the exponents, one f32x2 add for the sums
              float x0, x1;
              dev::fma2(x0, x1, sv[64 * h + 2 * c], sv[64 * h + 2 * c + 1], rsc, rsc, neg, neg);
              const float p0 = dev::ex2_approx(x0), p1 = dev::ex2_approx(x1);
              const int ai = 2 * (c & 3);
              dev::add2(rs8[ai], rs8[ai + 1], rs8[ai], rs8[ai + 1], p0, p1);
              // e4m3, four per column (p <= 2^8 < 448: no scale)
              const uint32_t two = e4m3x2(p0, p1);
              p[c >> 1] = (c & 1) ? (p[c >> 1] | (two << 16)) : two;
            }
            uint32_t p16[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) p16[i] = p[i];
            dev::tmem_st16(t_s + 16 * h, p16);
          }
          const float rs = ((rs8[0] + rs8[1]) + (rs8[2] + rs8[3])) + ((rs8[4] + rs8[5]) + (rs8[6] + rs8[7]));
          l = l * alpha + rs;
          // tcgen05.ld/st are warp-collective (.sync.aligned): the rescale runs
          // for the whole warp when any of its rows needs it (alpha = 1
          // elsewhere); every MMA before the QK just read (PV(t-1) included)
          // has completed.
          if (j > g.lo && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t ov[32];
              dev::tmem_ld32(t_o + c * 32, ov);
              dev::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              dev::tmem_st32(t_o + c * 32, ov);
            }
          }
          dev::tmem_wait_st();
          dev::tc_fence_before();
          __syncwarp();
          // the next PV reads V(t) and the QK after it K(t+1): group t+1 must have
          // landed in this CTA before query tile 0 reports P ready
          if (checks_kv && !kv_landed) ok = dev::mbar_wait(kv_bar, kv_par, abort_flag, a.err, kTimeoutNs);
          if (lane == 0) {  // P (and O) of the warp's 32 rows
            if (rank == 0)
              dev::mbar_arrive(bars.p_ready(st, 0));  // the even CTA's own barrier, arrived on locally
            else
              dev::mbar_arrive_cluster(p_ready_remote[0]);
          }
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
        }
      } else {
        // bf16: 64-key halves (see the kernel header).
        int32_t q_end = 0;  // causal walk: the end of this row's keys
        if constexpr (kWalk == kWalkCausal)
          q_end = tile_row<kWalk, kPair>(g, st, rank, walk) + (int32_t)(row_in_tile * walk.recip >> 16) + 1;
        int4 entry_next = walk_entry<kWalk>(g, g.lo, walk);  // an entry is loaded a tile ahead of its use
        for (int j = g.lo; ok && j < g.hi; ++j) {
          const uint32_t t = t_unit + (j - g.lo);  // the pair's running key-tile count
          const float rsc = sl2;  // score scale in log2 units: softmax_scale log2(e)
          const KeyTile tile = key_tile<kWalk>(g, j, entry_next, walk);
          if (kWalk != kWalkDoc && j + 1 < g.hi && (kWalk == kWalkList || g.n > 0))
            entry_next = walk_entry<kWalk>(g, j + 1, walk);
          const int rem_tile = tile.rem;
          // this row's valid keys: none of another document's tile
          int rem = tile.rem;
          if (kWalk == kWalkPrefix && g.n > 0 && ((int32_t)row_in_unit < tile.lo || (int32_t)row_in_unit >= tile.hi)) rem = 0;
          if constexpr (kWalk == kWalkCausal) rem = min(rem, q_end - tile.row);
          // the group holding V(t) and K(t + 1), and the one holding K(t)
          const uint32_t grp = kPair ? 2 * st + ((t + 1) & 1) : (t + 1) % kGroups;
          const uint32_t grp_k = kPair ? 2 * st + (t & 1) : t % kGroups;
          const uint32_t kv_bar = bars.kv_full(grp), kv_par = ((t + 1) / (kPair ? 2 : kGroups)) & 1;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // (no lane leaves here: a failed wait only clears ok, and the
            // warp-uniform vote at the end of the half ends the loop)
            ok = dev::mbar_wait(bars.s_ready(st, h), s_it[h] & 1, abort_flag, a.err, kTimeoutNs) && ok;
            ++s_it[h];
            // S half 1 of the last query tile is ready: every MMA before its QK is
            // done, so the group holding K(t) (and V(t-1)) is free in this CTA
            if (releases && h == 1) dev::mbar_arrive(bars.kv_empty(grp_k));
            __syncwarp();  // lanes leave the wait separately; the TMEM loads are warp-collective
            dev::tc_fence_after();
            const uint32_t t_sh = t_s + 64 * h;  // this half's S, then its P
            uint32_t r[2][32];
            dev::tmem_ld32(t_sh, r[0]);
            dev::tmem_ld32(t_sh + 32, r[1]);
            dev::tmem_wait_ld();
            float sv[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) sv[c] = __uint_as_float(r[c >> 5][c & 31]);
            if (rem < kTileRows) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (half_key(c, h) >= rem) sv[c] = -INFINITY;
            }
            // Row max of the half: eight independent chains of 3-input maxima.
            float mx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[i] = fmaxf(sv[i], sv[8 + i]);
#pragma unroll
            for (int c = 16; c < 64; c += 16)
#pragma unroll
              for (int i = 0; i < 8; ++i) mx[i] = dev::max3(mx[i], sv[c + i], sv[c + 8 + i]);
            const float m_new =
                dev::max3(dev::max3(mx[0], mx[1], mx[2]), dev::max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * rsc;
            // The reference max only moves when the row max grows by more than
            // 2^8 (then O and l are rescaled; the final O / l is unchanged).
            float alpha = 1.f;
            if (m_new > m_used + (kWalk == kWalkDoc ? kRescaleThreshold : kRescaleThresholdWalk)) {
              alpha = dev::ex2_approx(m_used - m_new);  // 0 on the first half of a unit (m_used = -inf)
              m_used = m_new;
            }
            const float neg = -m_used;
            float rs8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            uint32_t p[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              // packed pair arithmetic: one f32x2 FMA for the exponents, one f32x2 add for the sums
              float x0, x1;
              dev::fma2(x0, x1, sv[2 * c], sv[2 * c + 1], rsc, rsc, neg, neg);
              const float p0 = dev::ex2_approx(x0), p1 = dev::ex2_approx(x1);
              const int ai = 2 * (c & 3);
              dev::add2(rs8[ai], rs8[ai + 1], rs8[ai], rs8[ai + 1], p0, p1);
              p[c] = dev::pack_bf16x2(p0, p1);
            }
            dev::tmem_st32(t_sh, p);
            const float rs = ((rs8[0] + rs8[1]) + (rs8[2] + rs8[3])) + ((rs8[4] + rs8[5]) + (rs8[6] + rs8[7]));
            l = l * alpha + rs;
            // tcgen05.ld/st are warp-collective (.sync.aligned): the rescale runs
            // for the whole warp when any of its rows needs it (alpha = 1
            // elsewhere).  The PV of the previous half (the other half) may
            // still be adding into O (every earlier PV of this tile completed
            // before the QK whose S was just read), so it is awaited first: the
            // QK issued right after it fills the other half's next S, which this
            // thread reads next anyway; in the last key tile no such QK may
            // follow, and "PV done" of half 0 is awaited instead.
            if (!(j == g.lo && h == 0) && __any_sync(0xffffffffu, alpha != 1.f)) {
              if (h == 1 && j + 1 == g.hi)
                ok = dev::mbar_wait(bars.pv_done(st, 0), n_done & 1, abort_flag, a.err, kTimeoutNs) && ok;
              else
                ok = dev::mbar_wait(bars.s_ready(st, 1 - h), s_it[1 - h] & 1, abort_flag, a.err, kTimeoutNs) && ok;
              __syncwarp();
              dev::tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint32_t ov[16];
                dev::tmem_ld16(t_o + c * 16, ov);
                dev::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                dev::tmem_st16(t_o + c * 16, ov);
              }
            }
            dev::tmem_wait_st();
            dev::tc_fence_before();
            __syncwarp();
            // half 0's PV reads V(t) and the QK after it K(t+1): group t+1 must have
            // landed in this CTA before query tile 0 reports that P ready
            // (a blocking wait and the cluster-address arrive measured faster here
            // than FP8's non-blocking test and local arrive)
            if (h == 0 && checks_kv) ok = dev::mbar_wait(kv_bar, kv_par, abort_flag, a.err, kTimeoutNs) && ok;
            if constexpr (kWalk != kWalkDoc) {
              // The tile ends early: the rows of V behind its last valid key (this
              // CTA's 64 dims, 128 bytes a row) are zeroed before the PV reads
              // them, by the warp that reports the group landed.
              if (h == 0 && (kPair ? (warp & 3) == 0 : warp == 0) && rem_tile < kTileRows) {
                ok = dev::mbar_wait(kv_bar, kv_par, abort_flag, a.err, kTimeoutNs) && ok;
                const uint32_t v_slot = sbase + C::SmemKV + (kPair ? 2 * grp : (2 * t + 1) % kSlots) * C::SlotBytes;
                if (ok)
                  for (uint32_t b = (uint32_t)max(rem_tile, 0) * 128u + lane * 16u; b < C::SlotBytes; b += 512u)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v_slot + b), "r"(0u) : "memory");
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // visible to the tensor cores
                __syncwarp();
              }
            }
            if (lane == 0) dev::mbar_arrive_cluster(p_ready_remote[h]);  // P (and O) of the warp's 32 rows
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
          }
        }
      }
      if (!ok) break;
      // the unit's last PVs of this query tile, one per half ("PV done" of a
      // half completes once per unit, after its last key tile's PV; FP8: one,
      // after the unit's last PV)
      ok = dev::mbar_wait(bars.pv_done(st, 0), n_done & 1, abort_flag, a.err, kTimeoutNs) &&
           (kFp8 || dev::mbar_wait(bars.pv_done(st, 1), n_done & 1, abort_flag, a.err, kTimeoutNs));
      ++n_done;
      // every lane of a bf16 warp leaves together (FP8's lanes run the bounded
      // waits in step; its loop is sensitive to code shape)
      if constexpr (kFp8) {
        if (!ok) break;
      } else if (!__all_sync(0xffffffffu, ok)) {
        break;
      }
      __syncwarp();
      dev::tc_fence_after();
      const int32_t local = (kPair ? 0 : st * 2 * kTileRows) + (int32_t)rank * kTileRows + (int32_t)row_in_tile;
      int32_t row = g.q0 + local, head = g.head;
      bool valid = row < g.q1;
      // causal walk: token and head of a row of this tile, and its partial row (a head's tokens together)
      [[maybe_unused]] const int32_t tile0 = tile_row<kWalk, kPair>(g, st, rank, walk);
      [[maybe_unused]] const auto packed = [&](uint32_t r, int32_t* tok, int32_t* sub) {
        if constexpr (kWalk == kWalkCausal) {
          const int32_t t = (int32_t)(r * walk.recip >> 16);
          *tok = tile0 + t;
          *sub = (int32_t)r - t * walk.pack;
          return t < walk.toks && *tok < g.q1;
        }
        return false;
      };
      if constexpr (kWalk == kWalkCausal) {
        int32_t sub;
        valid = packed(row_in_tile, &row, &sub);
        head += sub;
      }
      if (g.part >= 0) {
        // A piece of a unit split along the keys: unnormalised O row, its
        // reference max (log2 units) and sum, for the merge pass.
        // (the partial buffer is a device allocation: its 512-byte rows are 32-byte aligned)
        // (dense: slots of kUnitRows rows; other walks: part is the segment's first partial row)
        size_t slot = (kWalk == kWalkDoc ? (size_t)g.part * kUnitRows : (size_t)g.part) + local;
        if constexpr (kWalk == kWalkCausal) slot = (size_t)g.part + (head - g.head) * (g.q1 - g.q0) + (row - g.q0);
        if constexpr (!kFp8 && !kPair) {
          // bf16: each 32-column chunk of the warp's 32 rows goes through its
          // rows of the unit's Q slot (free: the slot is released only after
          // this warp reports), so that every global store writes whole
          // 128-byte row segments: a store instruction covers 4 rows.
          const uint32_t stage = sbase + C::SmemQ + q_slot * C::QTileBytes + lane_base * 128u;
          const size_t slot0 = slot - lane;
          const int32_t row_first = g.q0 + local - (int32_t)lane;
          // (causal walk: rows that no load fills stay zeros, for the segments behind this piece; written over, one
          // prompt of 15,925 tokens and three heads over one took 167 us for 159, of 18,019 and six 330 for 313)
          bool filled = true;
          if constexpr (kWalk == kWalkCausal) filled = (int32_t)row_in_tile < walk.pack * walk.toks;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t ov[32];
            dev::tmem_ld32(t_o + c * 32, ov);
            dev::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t addr = stage + lane * 128u + ((((uint32_t)e) ^ (lane & 7u)) << 4);
              if (filled)
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(ov[4 * e]), "r"(ov[4 * e + 1]),
                             "r"(ov[4 * e + 2]), "r"(ov[4 * e + 3])
                             : "memory");
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t r = 4 * i + (lane >> 3), q = lane & 7u;  // row of the warp, 16-byte piece
              uint4 v;
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                           : "r"(stage + r * 128u + ((q ^ (r & 7u)) << 4))
                           : "memory");
              if constexpr (kWalk == kWalkCausal) {
                int32_t tok, sub;
                if (packed(lane_base + r, &tok, &sub))
                  *reinterpret_cast<uint4*>(a.part_o + ((size_t)g.part + sub * (g.q1 - g.q0) + (tok - g.q0)) * kHeadDim +
                                            c * 32 + 4 * q) = v;
              } else if (row_first + (int32_t)r < g.q1) {
                *reinterpret_cast<uint4*>(a.part_o + (slot0 + r) * kHeadDim + c * 32 + 4 * q) = v;
              }
            }
            __syncwarp();
          }
        } else {
          float* dst = a.part_o + slot * kHeadDim;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t ov[32];
            dev::tmem_ld32(t_o + c * 32, ov);
            dev::tmem_wait_ld();
            if constexpr (kFp8) scale_by_channel(ov, a.sv + g.head * kHeadDim + c * 32);
            if (valid) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                dev::st_global_v8(dst + c * 32 + e * 8, ov[8 * e], ov[8 * e + 1], ov[8 * e + 2], ov[8 * e + 3],
                                  ov[8 * e + 4], ov[8 * e + 5], ov[8 * e + 6], ov[8 * e + 7]);
            }
          }
        }
        if (valid) a.part_ml[slot] = make_float2(m_used, l);
        if constexpr (!kFp8 && !kPair) {
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(bars.o_staged(q_slot));
        }
        continue;
      }
      // (a row that saw no key: O is 0, lse = -inf)
      const float inv = kWalk != kWalkDoc && l == 0.f ? 0.f : 1.f / l;
      bool staged = false;
      if constexpr (!kFp8 && !kPair) staged = o_tma != 0 && __all_sync(0xffffffffu, valid);
      if (staged) {
        // The warp's 32 rows, bf16, into its rows of the unit's Q slot (free:
        // every MMA of the unit is done) in the tile's 128-byte swizzled
        // layout; the O-store thread sends them with two TMA stores (dims
        // 0..63, 64..127) of 32 rows each.
        const uint32_t tile = sbase + C::SmemQ + q_slot * C::QTileBytes;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t ov[32];
          dev::tmem_ld32(t_o + c * 32, ov);
          dev::tmem_wait_ld();
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = dev::pack_bf16x2(__uint_as_float(ov[2 * e]) * inv, __uint_as_float(ov[2 * e + 1]) * inv);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t cc = 4 * c + e;  // 16-byte chunk of the row
            const uint32_t addr = tile + (cc >> 3) * kQHalfBytes + row_in_tile * 128u + (((cc & 7u) ^ (row_in_tile & 7u)) << 4);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[4 * e]), "r"(w[4 * e + 1]),
                         "r"(w[4 * e + 2]), "r"(w[4 * e + 3])
                         : "memory");
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // visible to the TMA unit
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(bars.o_staged(q_slot));  // the store thread sends them
      } else {
        __nv_bfloat16* dst = og + (int64_t)row * a.o_stride + head * kHeadDim;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t ov[32];
          dev::tmem_ld32(t_o + c * 32, ov);
          dev::tmem_wait_ld();
          if constexpr (kFp8) scale_by_channel(ov, a.sv + g.head * kHeadDim + c * 32);
          if (valid) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              w[e] = dev::pack_bf16x2(__uint_as_float(ov[2 * e]) * inv, __uint_as_float(ov[2 * e + 1]) * inv);
            if (o_wide) {  // rows and chunks 32-byte aligned: two 32-byte stores per chunk
              dev::st_global_v8(dst + c * 32, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
              dev::st_global_v8(dst + c * 32 + 16, w[8], w[9], w[10], w[11], w[12], w[13], w[14], w[15]);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint4*>(dst + c * 32 + e * 8) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            }
          }
        }
        if constexpr (!kFp8 && !kPair) {
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(bars.o_staged(q_slot));
        }
      }
      if (valid && a.lse != nullptr)
        a.lse[(int64_t)head * a.S + row] = (m_used + __log2f(l)) * 0.6931471805599453f;
    }
  }

  // Neither CTA leaves (or frees the pair's TMEM) while the other may still
  // arrive on its barriers or run MMAs on its shared memory and TMEM.
  dev::tc_fence_before();
  __syncthreads();
  __syncwarp();  // the cluster barrier is warp-collective (.aligned)
  dev::cluster_sync();
  if (warp == kMmaWarp) {
    dev::tc_fence_after();
    dev::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// Combines the pieces of units split along the keys: one warp per query row,
// four dims per lane.  With M = max_c m_c (log2 units):
//   o = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c,  lse = (M + log2 l) ln 2.
// At 32 registers a thread, eight blocks fit on an SM, so the rows of a
// typical last round (a few thousand warps) run in one wave.  It is launched
// as a programmatic dependent of the forward: its blocks are scheduled as the
// forward's CTAs leave and wait here for the forward's writes.
__global__ void __launch_bounds__(256, 8) attn_merge_kernel(ForwardArgs a) {
  const int warp_global = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int mu = warp_global / kUnitRows, r = warp_global % kUnitRows;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the forward is complete and its writes visible
  if (mu >= a.n_merges) return;
  const MergeUnit m = a.merges[mu];
  const int32_t row = m.q_row0 + r;
  if (row >= m.kv_end) return;
  float M = -INFINITY;
#pragma unroll 4
  for (int c = 0; c < m.n_parts; ++c) M = fmaxf(M, a.part_ml[(size_t)(m.part0 + c) * kUnitRows + r].x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int c = 0; c < m.n_parts; ++c) {
    const size_t slot = (size_t)(m.part0 + c) * kUnitRows + r;
    const float2 ml = a.part_ml[slot];
    const float w = dev::ex2_approx(ml.x - M);
    const float4 o = reinterpret_cast<const float4*>(a.part_o + slot * kHeadDim)[lane];
    acc.x = fmaf(w, o.x, acc.x);
    acc.y = fmaf(w, o.y, acc.y);
    acc.z = fmaf(w, o.z, acc.z);
    acc.w = fmaf(w, o.w, acc.w);
    l = fmaf(w, ml.y, l);
  }
  const float inv = 1.f / l;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + (int64_t)row * a.o_stride + m.head * kHeadDim + 4 * lane;
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(dev::pack_bf16x2(acc.x * inv, acc.y * inv), dev::pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0 && a.lse != nullptr) a.lse[(int64_t)m.head * a.S + row] = (M + __log2f(l)) * 0.6931471805599453f;
}

// Output rows of the list and prefix walks that no segment finishes alone: one
// to eight warps per query row, four dims per lane.  A row's parts are the partial rows of
// its segment's pieces and, for small documents that share a segment with many
// others, the softmax over the document's own keys (at most kJoinOwnKeys),
// computed here in fp32 from q, k and v: a tile of the segment's walk each would
// cost a key-tile period of a CTA pair for a few keys.  With M the largest part
// maximum (log2 units): o = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c.
struct JoinArgs {
  const JoinRec* recs;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t stride;
  __nv_bfloat16* o;
  int64_t o_stride;
  float* lse;
  int64_t S;
  float scale_log2;
  const float* part_o;
  const float2* part_ml;
};

__device__ __forceinline__ float4 load_bf16x4(const __nv_bfloat16* p) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

constexpr int kAtOnce = kJoinParts;

// The rows of a record are a block's; parts are read kAtOnce at a time with their
// maxima and rows together, in one pass with a running maximum, so that a row
// waits for memory about once (two passes over the maxima and then the rows, and
// a lookup of the record: 52 us for 95,000 rows of 142,000 parts; so 33 us).  A
// row of more parts has several warps, whose sums meet in shared memory, in the
// warps' order (eight single queries over 12,000 rows, two heads: 94 parts a row,
// 19 us with one warp, 7 with eight).
__global__ void __launch_bounds__(32 * kJoinRows, 4) attn_join_kernel(JoinArgs a) {
  __shared__ float4 o_of[kJoinRows][32];
  __shared__ float2 ml_of[kJoinRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const JoinRec j = a.recs[blockIdx.x];
  const int rows = j.row1 - j.row0;
  const int shift = join_warps_log2(rows, j.n);  // a row has 1 << shift warps
  const int w = warp & ((1 << shift) - 1);                           // this one of them
  const int32_t row = j.row0 + (warp >> shift);
  const bool active = row < j.row1;
  // own keys (inputs of the forward: they need not wait for it), four at a time
  // with their values
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const int n_keys = active ? j.key_hi - j.key_lo : 0;
  const int key0 = j.key_lo + (n_keys * w >> shift), n_own = (n_keys * (w + 1) >> shift) - (n_keys * w >> shift);
  if (n_own > 0) {
    const int64_t col = (int64_t)j.head * kHeadDim + 4 * lane;
    const float4 q = load_bf16x4(a.q + (int64_t)row * a.stride + col);
#pragma unroll 1
    for (int x0 = 0; x0 < n_own; x0 += 4) {
      float s[4];
      float4 k[4], v[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int64_t at = (int64_t)(key0 + min(x0 + x, n_own - 1)) * a.stride + col;
        k[x] = load_bf16x4(a.k + at);
        v[x] = load_bf16x4(a.v + at);
      }
      float m_new = M;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float d = fmaf(q.x, k[x].x, fmaf(q.y, k[x].y, fmaf(q.z, k[x].z, q.w * k[x].w)));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        s[x] = x0 + x < n_own ? d * a.scale_log2 : -INFINITY;
        m_new = fmaxf(m_new, s[x]);
      }
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float w = dev::ex2_approx(M - ref);
      acc = make_float4(w * acc.x, w * acc.y, w * acc.z, w * acc.w);
      l *= w;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (x0 + x >= n_own) break;
        const float p = dev::ex2_approx(s[x] - ref);
        acc.x = fmaf(p, v[x].x, acc.x);
        acc.y = fmaf(p, v[x].y, acc.y);
        acc.z = fmaf(p, v[x].z, acc.z);
        acc.w = fmaf(p, v[x].w, acc.w);
        l += p;
      }
      M = m_new;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the forward is complete and its writes visible
  const int64_t r0 = (int64_t)j.part + (row - j.q_row0);
  const int n_parts = active ? j.n : 0;
  const int c0 = (int)((int64_t)n_parts * w >> shift), c1 = (int)((int64_t)n_parts * (w + 1) >> shift);
#pragma unroll 1
  for (int c = c0; c < c1; c += kAtOnce) {
    float2 ml[kAtOnce];
    float4 o[kAtOnce];
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      ml[x] = make_float2(-INFINITY, 0.f);
      o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + x < c1) {
        const int64_t r = r0 + (int64_t)(c + x) * j.rows;
        ml[x] = a.part_ml[r];
        o[x] = reinterpret_cast<const float4*>(a.part_o + r * kHeadDim)[lane];
      }
    }
    float m_new = M;
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) m_new = fmaxf(m_new, ml[x].x);
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    const float w = dev::ex2_approx(M - ref);
    acc = make_float4(w * acc.x, w * acc.y, w * acc.z, w * acc.w);
    l *= w;
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      const float wx = dev::ex2_approx(ml[x].x - ref);
      acc.x = fmaf(wx, o[x].x, acc.x);
      acc.y = fmaf(wx, o[x].y, acc.y);
      acc.z = fmaf(wx, o[x].z, acc.z);
      acc.w = fmaf(wx, o[x].w, acc.w);
      l = fmaf(wx, ml[x].y, l);
    }
    M = m_new;
  }
  if (shift > 0) {
    if (lane == 0) ml_of[warp] = make_float2(M, l);
    o_of[warp][lane] = acc;
    __syncthreads();
    if (w > 0 || !active) return;
    const int n = 1 << shift;
    float m_all = M;
    for (int x = 1; x < n; ++x) m_all = fmaxf(m_all, ml_of[warp + x].x);
    const float ref = m_all == -INFINITY ? 0.f : m_all;
    const float own = dev::ex2_approx(M - ref);
    acc = make_float4(own * acc.x, own * acc.y, own * acc.z, own * acc.w);
    l *= own;
    for (int x = 1; x < n; ++x) {
      const float wx = dev::ex2_approx(ml_of[warp + x].x - ref);
      const float4 o = o_of[warp + x][lane];
      acc.x = fmaf(wx, o.x, acc.x);
      acc.y = fmaf(wx, o.y, acc.y);
      acc.z = fmaf(wx, o.z, acc.z);
      acc.w = fmaf(wx, o.w, acc.w);
      l = fmaf(wx, ml_of[warp + x].y, l);
    }
    M = m_all;
  } else if (!active) {
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* dst = a.o + (int64_t)row * a.o_stride + j.head * kHeadDim + 4 * lane;
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(dev::pack_bf16x2(acc.x * inv, acc.y * inv), dev::pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0 && a.lse != nullptr) a.lse[(int64_t)j.head * a.S + row] = (M + __log2f(l)) * 0.6931471805599453f;
}

// 2D tensor map, 128-byte swizzle: inner extent `inner` elements of `esize`
// bytes (the tile box is 128 bytes wide), `outer` rows `row_bytes` apart.
bool make_map(CUtensorMap* m, const void* base, CUtensorMapDataType type, uint32_t esize, uint64_t inner,
              uint64_t outer, uint64_t row_bytes, uint32_t box_rows, std::string* why) {
  auto fn = encode_fn();
  if (fn == nullptr) {
    if (why) *why = "cuTensorMapEncodeTiled is unavailable";
    return false;
  }
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  cuuint32_t box[2] = {128 / esize, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    if (why) *why = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r);
    return false;
  }
  return true;
}

// 3D tensor map of bf16 rows [outer, heads, 128], 128-byte swizzle: boxes of 64
// dims of box_heads heads of box_rows rows.
bool make_map_heads(CUtensorMap* m, const void* base, uint64_t heads, uint64_t outer, uint64_t row_bytes, uint32_t box_heads,
                    uint32_t box_rows, std::string* why) {
  auto fn = encode_fn();
  if (fn == nullptr) {
    if (why) *why = "cuTensorMapEncodeTiled is unavailable";
    return false;
  }
  cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)heads, (cuuint64_t)outer};
  cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)row_bytes};
  cuuint32_t box[3] = {64, box_heads, box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    if (why) *why = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r);
    return false;
  }
  return true;
}

template <bool kFp8, int kWalk, bool kPair = false>
cudaError_t set_smem_attr() {
  static SmemAttr attr;
  return attr.set(attn_fwd_tc_kernel<kFp8, kWalk, kPair>, (int)Cfg<kFp8, kPair>::SmemAlloc);
}

template <bool kFp8>
cudaError_t launch_pairs(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                         int o_tma, const ForwardArgs& a, int device, int num_sms, cudaStream_t stream,
                         std::string* why) {
  cudaError_t e = set_smem_attr<kFp8, kWalkDoc>();
  if (e != cudaSuccess) {
    if (why) *why = "cudaFuncSetAttribute(max dynamic shared memory) failed";
    return e;
  }
  (void)device;
  (void)num_sms;
  if (a.n_pairs < 1 || a.unit_off == nullptr) {
    if (why) *why = "the work list has no CTA pairs";
    return cudaErrorInvalidValue;
  }
  attn_fwd_tc_kernel<kFp8, kWalkDoc, false>
      <<<2 * a.n_pairs, kThreads, Cfg<kFp8>::SmemAlloc, stream>>>(mq, mk, mv, mo, a, o_tma, Walk<kWalkDoc>{});
  e = cudaGetLastError();
  if (e != cudaSuccess || a.n_merges == 0) return e;
  const int64_t warps = (int64_t)a.n_merges * kUnitRows;
  e = launch_dependent(attn_merge_kernel, (unsigned)((warps + 7) / 8), 256u, stream, a);
  if (e != cudaSuccess && why) *why = "the merge launch failed";
  return e;
}

}  // namespace

int forward_slots(int device, int num_sms) {
  // Concurrent CTA pairs: the occupancy of the pair cluster (one CTA per SM),
  // asked once per device; half the SMs if the query fails.  The FP8 kernel
  // has the same threads and registers and less shared memory.
  static int slots[64];
  static std::once_flag once[64];
  if (device < 0 || device >= 64) return num_sms / 2 > 0 ? num_sms / 2 : 1;
  std::call_once(once[device], [device, num_sms] {
    int n = 0;
    int prev = -1;
    cudaGetDevice(&prev);
    if (prev != device) cudaSetDevice(device);
    if (set_smem_attr<false, kWalkDoc>() == cudaSuccess) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 * (num_sms / 2 > 0 ? num_sms / 2 : 1));
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = Cfg<false>::SmemAlloc;
      if (cudaOccupancyMaxActiveClusters(&n, attn_fwd_tc_kernel<false, kWalkDoc, false>, &cfg) != cudaSuccess) n = 0;
    }
    cudaGetLastError();
    if (prev != device && prev >= 0) cudaSetDevice(prev);
    slots[device] = n > 0 ? n : (num_sms / 2 > 0 ? num_sms / 2 : 1);
  });
  return slots[device];
}

namespace {

// Tensor maps of the bf16 forward's q, k, v and o (o_tma: whether O tiles go
// out by TMA: its rows allow a tensor map, 16-byte aligned base and row stride;
// otherwise the epilogue stores them directly).
struct ForwardMaps {
  CUtensorMap q, k, v, o;
  int o_tma;
};
bool make_forward_maps(const ForwardArgs& a, ForwardMaps* m, std::string* why) {
  const uint64_t inner = (uint64_t)a.H * kHeadDim, row = (uint64_t)a.qkv_stride * 2;
  if (!make_map(&m->q, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, inner, a.S, row, kTileRows, why) ||
      !make_map(&m->k, a.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, inner, a.S, row, kTileRows / 2, why) ||
      !make_map(&m->v, a.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, inner, a.S, row, kTileRows, why))
    return false;
  std::memset(&m->o, 0, sizeof(m->o));
  m->o_tma = (reinterpret_cast<uintptr_t>(a.o) & 15u) == 0 && (a.o_stride & 7) == 0 &&
             make_map(&m->o, a.o, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, inner, a.S, (uint64_t)a.o_stride * 2, 32,
                      nullptr);
  return true;
}

// The join of the rows that a walk left in parts.
cudaError_t launch_join(const ForwardArgs& a, const WalkArgs& w, cudaStream_t stream, std::string* why) {
  if (w.n_joins == 0) return cudaSuccess;
  const JoinArgs j{w.joins,
                   static_cast<const __nv_bfloat16*>(a.q),
                   static_cast<const __nv_bfloat16*>(a.k),
                   static_cast<const __nv_bfloat16*>(a.v),
                   a.qkv_stride,
                   static_cast<__nv_bfloat16*>(a.o),
                   a.o_stride,
                   a.lse,
                   a.S,
                   a.scale_log2,
                   a.part_o,
                   a.part_ml};
  const cudaError_t e = launch_dependent(attn_join_kernel, (unsigned)w.n_joins, 32u * (unsigned)w.join_warps, stream, j);
  if (e != cudaSuccess && why) *why = "the join launch failed";
  return e;
}

// The forward over another walk, then the join.
template <int kWalk, bool kPair>
cudaError_t launch_walk(const ForwardMaps& m, const ForwardArgs& a, const WalkArgs& w, const Walk<kWalk>& walk,
                        cudaStream_t stream, std::string* why) {
  cudaError_t e = set_smem_attr<false, kWalk, kPair>();
  if (e != cudaSuccess) {
    if (why) *why = "cudaFuncSetAttribute(max dynamic shared memory) failed";
    return e;
  }
  attn_fwd_tc_kernel<false, kWalk, kPair>
      <<<2 * a.n_pairs, kThreads, Cfg<false, kPair>::SmemAlloc, stream>>>(m.q, m.k, m.v, m.o, a, m.o_tma, walk);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join(a, w, stream, why);
}

}  // namespace

cudaError_t launch_forward(const ForwardArgs& a, int device, int num_sms, cudaStream_t stream, std::string* why) {
  if (a.n_units == 0) return cudaSuccess;
  ForwardMaps m;
  if (!make_forward_maps(a, &m, why)) return cudaErrorInvalidValue;
  return launch_pairs<false>(m.q, m.k, m.v, m.o, m.o_tma, a, device, num_sms, stream, why);
}

cudaError_t launch_forward_list(const ForwardArgs& a, const WalkArgs& w, cudaStream_t stream, std::string* why) {
  ForwardMaps m;
  if (!make_forward_maps(a, &m, why)) return cudaErrorInvalidValue;
  const Walk<kWalkList> walk{w.block_idx, w.block_cnt, w.n_q_blocks, w.max_blocks};
  return w.pair ? launch_walk<kWalkList, true>(m, a, w, walk, stream, why)
                : launch_walk<kWalkList, false>(m, a, w, walk, stream, why);
}

cudaError_t launch_forward_causal(const ForwardArgs& a, const WalkArgs& w, cudaStream_t stream, std::string* why) {
  Walk<kWalkCausal> walk;
  walk.pack = w.pack;
  walk.toks = kTileRows / w.pack;
  walk.recip = (65536u + (uint32_t)w.pack - 1) / (uint32_t)w.pack;
  walk.group = a.H / w.kv_heads;
  ForwardMaps m;
  // (bytes from row to row; one row has no stride: a map's is below 2^40)
  const auto step = [&](int64_t stride, uint64_t width) { return a.S > 1 ? (uint64_t)stride * 2 : width * 2; };
  const uint64_t S = (uint64_t)a.S, width = (uint64_t)a.H * kHeadDim, kv_width = (uint64_t)w.kv_heads * kHeadDim;
  const uint64_t kv_row = step(w.kv_stride, kv_width);
  if (!make_map_heads(&m.q, a.q, (uint64_t)a.H, S, step(a.qkv_stride, width), (uint32_t)walk.pack, (uint32_t)walk.toks, why) ||
      !make_map(&m.k, a.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, kv_width, S, kv_row, kTileRows / 2, why) ||
      !make_map(&m.v, a.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, kv_width, S, kv_row, kTileRows, why))
    return cudaErrorInvalidValue;
  std::memset(&m.o, 0, sizeof(m.o));
  // (O tiles go out by TMA where a warp's 32 rows are whole tokens)
  m.o_tma = 32 % walk.pack == 0 && make_map_heads(&m.o, a.o, (uint64_t)a.H, S, step(a.o_stride, width), (uint32_t)walk.pack,
                                                  32u / (uint32_t)walk.pack, nullptr);
  return w.pair ? launch_walk<kWalkCausal, true>(m, a, w, walk, stream, why)
                : launch_walk<kWalkCausal, false>(m, a, w, walk, stream, why);
}

cudaError_t launch_forward_prefix(const ForwardArgs& a, const WalkArgs& w, cudaStream_t stream, std::string* why) {
  if (w.pieces > 0) {
    const RowsArgs r{static_cast<const __nv_bfloat16*>(a.q),
                     static_cast<const __nv_bfloat16*>(w.k_prefix),
                     static_cast<const __nv_bfloat16*>(w.v_prefix),
                     a.qkv_stride,
                     w.prefix_stride,
                     w.prefix_len,
                     (int32_t)a.S,
                     (int32_t)(((int64_t)w.prefix_len + kTileRows - 1) / kTileRows),
                     w.pieces,
                     a.scale_log2,
                     a.part_o,
                     a.part_ml};
    const cudaError_t e = launch_attn_rows(r, a.H, stream);
    return e != cudaSuccess ? e : launch_join(a, w, stream, why);
  }
  ForwardMaps m;
  if (!make_forward_maps(a, &m, why)) return cudaErrorInvalidValue;
  Walk<kWalkPrefix> walk;
  walk.own = w.own;
  walk.len = w.prefix_len;
  walk.tiles = (int32_t)(((int64_t)w.prefix_len + kTileRows - 1) / kTileRows);
  const uint64_t inner = (uint64_t)a.H * kHeadDim, row = (uint64_t)w.prefix_stride * 2, n = (uint64_t)w.prefix_len;
  if (!make_map(&walk.tm_k, w.k_prefix, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, inner, n, row, kTileRows / 2, why) ||
      !make_map(&walk.tm_v, w.v_prefix, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, inner, n, row, kTileRows, why))
    return cudaErrorInvalidValue;
  return w.pair ? launch_walk<kWalkPrefix, true>(m, a, w, walk, stream, why)
                : launch_walk<kWalkPrefix, false>(m, a, w, walk, stream, why);
}

cudaError_t launch_forward_fp8(const ForwardArgs& a, int device, int num_sms, cudaStream_t stream,
                               std::string* why) {
  if (a.n_units == 0) return cudaSuccess;
  CUtensorMap mq, mk, mv;
  const uint64_t inner = (uint64_t)a.H * kHeadDim;  // bytes per token row of q8 / k8
  if (!make_map(&mq, a.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, inner, a.S, inner, kTileRows, why) ||
      !make_map(&mk, a.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, inner, a.S, inner, kTileRows / 2, why) ||
      // transposed V: H * 128 channel rows of S keys, v_row_bytes apart
      !make_map(&mv, a.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.v_row_bytes, inner, a.v_row_bytes, kTileRows / 2,
                why))
    return cudaErrorInvalidValue;
  CUtensorMap mo;
  std::memset(&mo, 0, sizeof(mo));
  return launch_pairs<true>(mq, mk, mv, mo, 0, a, device, num_sms, stream, why);
}

}  // namespace h3
