// Internal declarations shared by the host side of the library (plan builder,
// C-ABI layer) and the kernel launchers.  Nothing here is part of the ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <string>
#include <vector>

#include "h3attn.h"

namespace h3 {

constexpr int kHeadDim = 128;
constexpr int kRopeDims = 96;
constexpr int kRopeHalf = 48;       // NeoX pairs (j, j + 48), one angle per pair
constexpr int kAxisFreqs = 16;      // angles per axis: 32 rotated dims per axis / 2
constexpr int kUnitRows = 512;      // query rows per attention work unit (a CTA pair, two 128-row tiles each)

// Device error word values (the word is cleared by h3attn_get_device_error).
constexpr uint32_t kErrNone = 0;
constexpr uint32_t kErrTimeout = 1;
constexpr uint32_t kErrBlockIndex = 2;   // a listed key tile outside its document
constexpr uint32_t kErrPage = 3;         // a page outside the cache, or a length outside its table

constexpr int kKeyTile = 128;      // key rows per tile

// One attention work segment: up to kUnitRows query rows of one head inside
// one document [kv_begin, kv_end), over that document's key tiles
// [tile_lo, tile_hi) (all of them unless the unit was split along the keys to
// balance the last wave).  part < 0: the segment writes the final output;
// part >= 0: it writes unnormalised partial results to partial slot `part`
// and a merge pass combines the slots of its unit.
struct WorkUnit {
  int32_t q_row0;
  int32_t kv_begin;
  int32_t kv_end;
  int32_t head;
  int32_t tile_lo;
  int32_t tile_hi;
  int32_t part;
  int32_t v_off;   // the document's first key in the FP8 transposed V (16-key aligned)
};
static_assert(sizeof(WorkUnit) == 32, "WorkUnit is read as two 16-byte vectors");

// A unit split along the keys: its partial slots [part0, part0 + n_parts).
struct MergeUnit {
  int32_t q_row0;
  int32_t kv_end;
  int32_t head;
  int32_t part0;
  int32_t n_parts;
  int32_t pad[3];
};
static_assert(sizeof(MergeUnit) == 32, "MergeUnit is read as two 16-byte vectors");

// The attention work units of a packed layout, in list order (longest
// document first, then head, then query rows), and each document's first key
// in the FP8 transposed V (plan.cpp).  Returns an empty string or an error.
std::string build_units(const int32_t* cu, int32_t n_docs, int32_t num_heads, std::vector<WorkUnit>& units,
                        std::vector<int32_t>& v_off, int64_t* v_pad);

// Estimated run time of a segment (plan.cpp), the cost its placement balances.
int64_t segment_cost(const WorkUnit& u);

// Places the n segments on `grid` persistent CTA pairs in list order, each on
// the pair with the least estimated load so far (LPT placement; the list is
// ordered longest document first), and writes them to `out` grouped by pair:
// pair p runs out[unit_off[p] .. unit_off[p + 1]) in order.  Scratch: pair_of
// [n], load and heap [grid]; unit_off has grid + 1 entries.  Returns the number
// of pairs with work (they are pairs 0 .. that number - 1).  No allocation.
int32_t place_pairs(const WorkUnit* segs, size_t n, int grid, WorkUnit* out, int32_t* unit_off,
                    int32_t* pair_of, int64_t* load, int32_t* heap);

// Build the segment list for `grid` persistent CTA pairs: whole units for the
// full rounds, then the last partial round's units split along their key
// tiles into about `grid` pieces, all placed by place_pairs (plan.cpp).
// unit_off gets n_pairs + 1 entries.
void build_segments(const std::vector<WorkUnit>& units, int grid, std::vector<WorkUnit>& segs,
                    std::vector<int32_t>& unit_off, int32_t* n_pairs, std::vector<MergeUnit>& merges,
                    int32_t* n_parts);

// ---- other key walks (h3attn_forward_sparse, h3attn_forward_prefix) ----

// A work segment of a walk other than the unit's own document: query rows
// [q_row0, q_end) (at most kUnitRows) of one head, and the document [kv_begin,
// kv_end) they lie in.
//   list walk:   a = the query block, b = piece | pieces << 16: the segment
//                takes entries [n i / m, n (i + 1) / m) of the block's n
//                listed tiles (n is read on the device), i = piece, m = pieces
//   prefix walk: key tiles [a, b) of the walk "the prefix's tiles, then the
//                document's".  A segment whose rows belong to several documents
//                has kv_end = -n < 0: n own tiles, entries [kv_begin, kv_begin +
//                n) of the walk's table, follow the prefix; its a lies in the
//                prefix.
//   causal walk: key tiles [a, b) of the document; the rows are tokens, of `pack`
//                query heads from `head` on
// part < 0: the segment writes the output; part >= 0: it writes unnormalised
// rows from row `part` of the partial buffers on, for the join pass.
struct WalkUnit {
  int32_t q_row0;
  int32_t q_end;
  int32_t kv_begin;
  int32_t kv_end;
  int32_t head;
  int32_t a;
  int32_t b;
  int32_t part;
};
static_assert(sizeof(WalkUnit) == sizeof(WorkUnit), "read as two 16-byte vectors");

// A key tile of one document in a segment over several: its first key row and
// valid keys, the segment's rows [lo, hi) (counted from q_row0) that belong to
// the document, and for each query tile s of the pair the lanes of O that the
// tile's PV must leave alone (bit i of word w: row 256 s + 32 w + i).
struct OwnTile {
  int32_t row, rem, lo, hi;
  uint32_t skip[2][8];
};
static_assert(sizeof(OwnTile) == 80, "OwnTile is read as five 16-byte vectors");

// Rows [row0, row1) of one head (a block of the join: at most kJoinRows, a warp
// each; fewer where a row has so many parts that several warps share them) whose output the join pass combines from n partial rows each, piece c of
// row r at partial row part + c * rows + (r - q_row0), and from the keys [key_lo,
// key_hi) of the rows' document, which the join itself attends to (none when
// key_lo == key_hi).
struct JoinRec {
  int32_t row0, row1, head, q_row0;
  int32_t part, rows, n, key_lo;
  int32_t key_hi, pad[3];
};
static_assert(sizeof(JoinRec) == 48, "JoinRec is read as three 16-byte vectors");
constexpr int kJoinRows = 8;         // warps of a join block, and its most rows
constexpr int kJoinParts = 8;        // parts that a warp of the join reads at once

// log2 of the warps that a row of a join record has: enough to read its n parts
// at once, as far as kJoinRows warps go round its rows.
#ifdef __CUDACC__
__host__ __device__
#endif
inline int join_warps_log2(int32_t rows, int32_t n) {
  int s = 0;
  while ((rows << (s + 1)) <= kJoinRows && (kJoinParts << s) < n) ++s;
  return s;
}
constexpr int kJoinOwnKeys = 32;     // longest document the join may attend to itself

// A few short documents over a prefix (attn_rows.cu): kRowsTile rows and one head
// to a segment, a block each; never more than kRowsMax rows in all.
constexpr int kRowsTile = 32;
constexpr int kRowsMax = 1024;

struct WalkPlan {
  bool set = false;
  int32_t pieces = 0;                  // > 0: prefix walk of a few short documents, so many blocks for each head and
                                       // kRowsTile rows (attn_rows.cu, which computes its segments itself)
  int streams = 1;                     // streams of segments that a CTA pair runs side by side
  std::vector<WalkUnit> units;         // grouped by CTA pair
  std::vector<int32_t> unit_off;       // [n_pairs + 1]; two streams: [n_pairs][2] (first, end)
  int32_t n_pairs = 0;
  std::vector<OwnTile> own;            // prefix walk
  std::vector<JoinRec> joins;
  int32_t join_warps = 0;              // warps of a join block: the most that a record needs
  int64_t part_rows = 0;               // partial rows of all segments

  WalkUnit* d_units = nullptr;         // units, then unit_off
  OwnTile* d_own = nullptr;
  JoinRec* d_joins = nullptr;
  float* d_part_o = nullptr;           // [part_rows, 128] unnormalised O
  float2* d_part_ml = nullptr;         // [part_rows] (reference max in log2 units, sum)
};

// The segment lists of the two walks for `grid` CTA pairs (walk_plan.cpp);
// each returns an empty string or an error.
std::string build_list_walk(const int32_t* cu, int32_t n_docs, int32_t num_heads, int32_t q_block, int32_t max_blocks,
                            int grid, WalkPlan& w);
std::string build_prefix_walk(const int32_t* cu, int32_t n_docs, int32_t num_heads, int32_t prefix_len, int grid,
                              WalkPlan& w);

// Causal walk: query heads that share a segment, for `group` query heads of a key
// head: the largest divisor up to 16, so that a tile's 128 rows hold whole tokens and
// few stay empty (none for powers of two, 2 of 128 for six or seven heads).
inline int32_t causal_pack(int32_t group) {
  for (int32_t p = 16; p > 1; --p)
    if (group % p == 0) return p;
  return 1;
}
std::string build_causal_walk(const int32_t* cu, int32_t n_docs, int32_t num_heads, int32_t num_kv_heads, int grid,
                              WalkPlan& w);

// Up to kSelectWarps query blocks of one document, scored by one thread block.
struct SelectGroup {
  int32_t q0, n;          // query blocks [q0, q0 + n)
  int32_t tile0, tiles;   // the document's key tiles [tile0, tile0 + tiles) of the plan's tile table
  int32_t first;          // index of q0 within its document
  int32_t len;            // the document's tokens
  int32_t pad[2];
};
static_assert(sizeof(SelectGroup) == 32, "SelectGroup is read as vectors");
constexpr int kSelectWarps = 8;
constexpr int32_t kSelectMaxTiles = 12288;  // key tiles of the longest document that can be scored
// Query blocks per scoring block: each keeps 16 bytes per key tile in shared memory.
inline int select_warps(int32_t max_tiles) {
  const int n = 192 * 1024 / (16 * (max_tiles > 0 ? max_tiles : 1));
  return n < 1 ? 1 : (n > kSelectWarps ? kSelectWarps : n);
}

struct SparsePlan {
  WalkPlan walk;
  int32_t q_block = 0;
  int32_t max_blocks = 0;
  int32_t n_q_blocks = 0;              // over all documents
  int32_t max_tiles = 0;               // key tiles of the longest document
  std::vector<SelectGroup> groups;
  SelectGroup* d_groups = nullptr;
  float2* d_q_sum = nullptr;           // [H, tiles, 128] sums of q-hat rows (high, low)
  float2* d_k_mean = nullptr;          // [H, 64, tiles] means of k-hat rows, two dims a word
};

struct PrefixPlan {
  WalkPlan walk;
  int32_t len = 0;
};

// What the tree forward's join has to know of a token: its document's first item,
// the first query tile of its heads, its place in it, the document's units of two tiles.
struct TreeRow {
  int32_t item0, qtile, in_tile, units;
};

// Workspace of the tree forward.
struct TreePlan {
  bool set = false;
  int32_t kv_heads = 0;
  int32_t pack = 1;                    // query heads in a query tile (a divisor of the group), and tokens
  int32_t toks = 1;
  int32_t slot_rows = 0;               // rows of a partial slot: of one query tile, or of two
  int32_t grid = 0;                    // blocks; two partial slots each, or each stream
  int32_t items = 0;                   // (sequence, key head, up to two query tiles)
  int32_t max_len = 0;                 // drafts of the longest document
  TreeRow* d_rows = nullptr;           // [S]
  int32_t* d_item0 = nullptr;          // [n_docs] first item of a document
  int2* d_joins = nullptr;             // [items] first partial slot and pieces (the forward's)
  float* d_part_o = nullptr;           // [4 grid 128 rows, 128]
  float2* d_part_ml = nullptr;         // [4 grid 128 rows]
};
constexpr int32_t kTreeMax = 64;       // drafts of a document
constexpr int32_t kTreeDocs = 4096;

struct CausalPlan {
  WalkPlan walk;
  int32_t kv_heads = 0;
};

// Placement core shared by the lists (plan.cpp): segment i, in list order,
// goes to the pair with the least load so far, ties to the lower pair.
template <class Cost>
void assign_pairs(size_t n, Cost cost, int G, int32_t* pair_of, int64_t* load, int32_t* heap) {
  // min-heap of pair indices ordered by (load, index); all loads start at 0,
  // so the identity order is already a heap
  for (int p = 0; p < G; ++p) {
    load[p] = 0;
    heap[p] = p;
  }
  auto before = [load](int32_t a, int32_t b) { return load[a] != load[b] ? load[a] < load[b] : a < b; };
  for (size_t i = 0; i < n; ++i) {
    const int32_t p = heap[0];
    pair_of[i] = p;
    load[p] += cost(i);
    for (int c = 0;;) {
      const int l = 2 * c + 1, r = l + 1;
      int m = c;
      if (l < G && before(heap[l], heap[m])) m = l;
      if (r < G && before(heap[r], heap[m])) m = r;
      if (m == c) break;
      const int32_t t = heap[c];
      heap[c] = heap[m];
      heap[m] = t;
      c = m;
    }
  }
}

// Pair-major order of placed segments (keeping each pair's list order) into
// out and unit_off [G + 1]; heap is scratch.  Returns the pairs with work: as
// every cost is positive and ties go to the lower index, they are the leading
// ones.
template <class Unit>
int32_t group_by_pair(const Unit* segs, size_t n, int G, Unit* out, int32_t* unit_off, const int32_t* pair_of,
                      int32_t* heap) {
  for (int p = 0; p <= G; ++p) unit_off[p] = 0;
  for (size_t i = 0; i < n; ++i) ++unit_off[pair_of[i] + 1];
  for (int p = 0; p < G; ++p) unit_off[p + 1] += unit_off[p];
  for (int p = 0; p < G; ++p) heap[p] = unit_off[p];
  for (size_t i = 0; i < n; ++i) out[heap[pair_of[i]]++] = segs[i];
  int32_t used = 0;
  while (used < G && unit_off[used + 1] > unit_off[used]) ++used;
  return used;
}

struct Plan {
  int device = -1;
  int num_sms = 0;
  int32_t n_docs = 0;
  int32_t num_heads = 0;
  int32_t max_seqlen = 0;
  int64_t S = 0;
  double rope_base = 10000.0;

  std::vector<int32_t> cu_host;      // [n_docs + 1]
  std::vector<double> pos_host;      // [S, 3]
  std::vector<float> rope_host;      // [S, 48, 2] (cos, sin)
  std::vector<WorkUnit> units_host;  // segment list, grouped by CTA pair (see build_segments)
  std::vector<int32_t> unit_off_host;  // [n_pairs + 1]: pair p runs units [unit_off[p], unit_off[p + 1])
  int32_t n_pairs = 0;
  std::vector<MergeUnit> merges_host;
  int32_t n_parts = 0;
  // every document's 128-key tiles: (begin, end, first key in the FP8
  // transposed V, 0); that V gives each document a 16-key aligned start
  std::vector<int4> ktiles_host;
  int64_t v_pad = 0;                 // keys per row of the FP8 transposed V

  int32_t* d_cu = nullptr;
  float2* d_rope = nullptr;          // [S, 48] (cos, sin)
  WorkUnit* d_units = nullptr;       // the segment list, then unit_off (n_pairs + 1 int32)
  int32_t n_units = 0;
  MergeUnit* d_merges = nullptr;
  float* d_part_o = nullptr;         // [n_parts, kUnitRows, 128] unnormalised O
  float2* d_part_ml = nullptr;       // [n_parts, kUnitRows] (running max in log2 units, sum)
  uint32_t* d_err = nullptr;         // device error word
  int4* d_ktiles = nullptr;

  SparsePlan sparse;                 // h3attn_plan_set_sparse
  PrefixPlan prefix;                 // h3attn_plan_set_prefix
  CausalPlan causal;                 // h3attn_plan_set_causal
  TreePlan tree;                     // h3attn_plan_set_tree
};

// Host-side plan construction (plan.cpp); returns an empty string or an error.
// With validate_only, only the document/span checks run (no device needed).
std::string build_plan_host(const h3attn_doc* docs, int32_t n_docs, const h3attn_plan_opts& opts,
                            int grid, Plan& p, bool validate_only = false);

// Error reporting for the C-ABI layer.
h3attn_status fail(h3attn_status s, const char* fmt, ...);
void clear_error();
// Every call that goes to the device begins there with it.  The runtime keeps a
// failed call's error until it is asked for, and launches are checked by asking:
// without it a refused allocation came back as the next call's failed launch.
// (Not in calls that stay on the host: it initialises the driver, after which a
// process may not fork ones that use it.)
void clear_runtime_error();

// The maximum dynamic shared memory of a kernel, set once per kernel and device
// (the attribute belongs to the current device's copy of the kernel).
struct SmemAttr {
  std::once_flag once[64];
  cudaError_t result[64] = {};
  template <class Kernel>
  cudaError_t set(Kernel* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    std::call_once(once[dev], [&] {
      result[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
    return result[dev];
  }
};

// Kernel launchers.
struct PrologueArgs {
  const void* q_in;
  const void* k_in;
  void* q_out;
  void* k_out;
  int64_t in_stride;
  int64_t out_stride;
  const float* gain_q;
  const float* gain_k;
  int64_t gain_head_stride;
  const float2* rope;
  int64_t S;
  int32_t H;
  float eps;
};
cudaError_t launch_qk_prologue(const PrologueArgs& a, int num_sms, cudaStream_t stream);

struct ForwardArgs {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  int64_t qkv_stride;
  int64_t o_stride;
  int64_t S;
  int32_t H;
  float scale_log2;           // softmax_scale * log2(e)
  const WorkUnit* units;
  int32_t n_units;
  const int32_t* unit_off;    // [n_pairs + 1]: pair p runs units [unit_off[p], unit_off[p + 1])
  int32_t n_pairs;            // CTA pairs launched
  uint32_t* err;
  const MergeUnit* merges;    // may be null when n_merges == 0
  int32_t n_merges;
  float* part_o;
  float2* part_ml;
  // Fused Q prologue (gain_q non-null): q holds the raw queries; the forward
  // applies RMSNorm with gain and the rot96 rotation to each Q tile in shared
  // memory, with the separate prologue's arithmetic.
  const float* gain_q;
  int64_t gain_head_stride;
  float eps;
  const float2* rope;          // [S, 48] (cos, sin)
  // FP8 variant (h3attn_forward_fp8): scales of the e4m3 inputs
  const float* sq;             // [H, S]
  const float* sk;             // [H, S]
  const float* sv;             // [H, 128]
  int64_t v_row_bytes;         // row stride of the transposed V (the plan's v_pad)
};
// Work slots of the forward: CTA pairs that run at the same time on `device`
// (the plan's segment list is balanced for this many).
int forward_slots(int device, int num_sms);
cudaError_t launch_forward(const ForwardArgs& a, int device, int num_sms, cudaStream_t stream,
                           std::string* why);
cudaError_t launch_forward_fp8(const ForwardArgs& a, int device, int num_sms, cudaStream_t stream,
                               std::string* why);

// The forward over a list of key tiles per query block, or over a shared prefix
// and the document (a.units, unit_off, n_pairs, part_o and part_ml are those of
// the walk plan; a.merges is unused).
struct WalkArgs {
  const JoinRec* joins;
  int32_t n_joins, join_warps;
  bool pair;                   // two streams of segments on a CTA pair
  int32_t pieces;              // > 0: attn_rows.cu's
  // list walk
  const int32_t* block_idx;    // [H, n_q_blocks, max_blocks]
  const int32_t* block_cnt;    // [H, n_q_blocks]
  int32_t n_q_blocks;
  int32_t max_blocks;
  // prefix walk
  const void* k_prefix;
  const void* v_prefix;
  int64_t prefix_stride;
  int32_t prefix_len;
  const OwnTile* own;
  // causal walk
  int32_t kv_heads, pack;
  int64_t kv_stride;
};
struct RowsArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_prefix;
  const __nv_bfloat16* v_prefix;
  int64_t q_stride, prefix_stride;
  int32_t prefix_len;
  int32_t S, tiles, pieces;    // query rows; the prefix's tiles, cut into pieces for each head and kRowsTile rows
  float scale_log2;
  float* part_o;
  float2* part_ml;
};
cudaError_t launch_attn_rows(const RowsArgs& a, int heads, cudaStream_t stream);

cudaError_t launch_forward_list(const ForwardArgs& a, const WalkArgs& w, cudaStream_t stream, std::string* why);
cudaError_t launch_forward_prefix(const ForwardArgs& a, const WalkArgs& w, cudaStream_t stream, std::string* why);

cudaError_t launch_forward_causal(const ForwardArgs& a, const WalkArgs& w, cudaStream_t stream, std::string* why);

// Trees of drafts over a paged cache (attn_tree.cu).
struct TreeArgs {
  const int32_t* cu;           // [n_docs + 1]
  const TreeRow* rows;         // [S]
  const int32_t* ctx_lens;     // [n_docs]
  const int32_t* page_table;   // [n_docs, table_width]
  const uint64_t* tree_mask;   // [S] or null
  int64_t S;
  int32_t n_docs, H, kv_heads, group, table_width;
  int32_t pack, toks, packs;   // heads and tokens of a query tile, query tiles that a token's group takes
  int32_t slot_rows, grid, items;
  float scale_log2;
  __nv_bfloat16* o;
  int64_t o_stride;
  float* lse;
  const int32_t* item0;        // [n_docs]
  int2* joins;                 // [items]; pieces below two: none to join
  float* part_o;
  float2* part_ml;
  uint32_t* err;
  // (the launcher's)
  uint32_t recip, recip_toks;  // row / pack = row * recip >> 16, and of toks
  float inv_grid;              // 1 / grid
  int32_t slots;               // partial slots: two a block, or a stream
  int32_t by_warp;             // not more items than blocks, each below 2^21 tiles
  int32_t page_size, n_pages;
  int32_t box;                 // rows of the cache that a copy takes: gcd(page_size, 128)
  int32_t n_box, at_once;      // boxes of a 128-key tile, tiles of 32 boxes
  int32_t page_boxes, row_step;  // boxes of a page; 128 mod page_size
  uint32_t page_mul, page_shift;  // box / page_boxes = box * page_mul >> page_shift
  int32_t heads_first;         // the cache's heads lie closer together than its tokens
};
cudaError_t launch_attn_tree(const TreeArgs& a, const void* q, int64_t q_stride, const h3attn_cache& cache, cudaStream_t stream,
                             std::string* why);
cudaError_t launch_tree_join(const TreeArgs& a, cudaStream_t stream, std::string* why);  // (its second launch)

// Block scores and selection (block_select.cu).
struct SelectArgs {
  const void* q_hat;
  const void* k_hat;
  int64_t stride;              // row stride (elements)
  int32_t H;
  const int4* tiles;           // (begin, end, ...) of every document's 128-key tiles
  int32_t n_tiles;
  const SelectGroup* groups;
  int32_t n_groups;
  int32_t max_tiles;           // of one document
  int32_t n_q_blocks;
  int32_t tiles_per_q_block;
  float2* q_sum;
  float2* k_mean;
  int32_t keep;
  int32_t keep_own;
  int32_t max_blocks;
  int32_t* block_idx;          // [H, n_q_blocks, max_blocks]
  int32_t* block_cnt;          // [H, n_q_blocks]
  int32_t num_sms;
};
cudaError_t launch_block_select(const SelectArgs& a, cudaStream_t stream);

// FP8 (e4m3) quantisation of q-hat, k-hat and v (fp8_quant.cu).
struct Fp8QuantArgs {
  const void* q_hat;
  const void* k_hat;
  const void* v;
  int64_t stride;              // row stride of q-hat, k-hat, v (elements)
  int64_t S;
  int32_t H;
  const int4* tiles;           // (begin, end, V key, 0) of every document's 128-key tiles
  int32_t n_tiles;
  void* q8;                    // [S, H, 128] codes
  void* k8;                    // [S, H, 128] codes
  void* v8t;                   // [H, 128, v_pad] codes, keys contiguous, documents 16-key aligned
  int64_t v_pad;
  float* sq;                   // [H, S]
  float* sk;                   // [H, S] (each token carries its tile's scale)
  float* sv;                   // [H, 128]
};
cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, int num_sms, cudaStream_t stream);
// The prologue fused with the q/k quantisation (p: inputs, gains, table; a:
// v and the FP8 outputs), then the v quantisation (fp8_quant.cu).
cudaError_t launch_prologue_fp8(const PrologueArgs& p, const Fp8QuantArgs& a, cudaStream_t stream);

// Rotary positions (rotary.cu): q rows (H of them a token), k rows (Hk) and v rows
// (Hv, copied only); k and v go to rows of their own or, with slots, into a cache.
struct RotaryArgs {
  h3attn_rope rope;
  const int32_t* positions;    // [n_axes, n]
  int64_t n;
  const __nv_bfloat16* q_in;
  __nv_bfloat16* q_out;
  int64_t q_in_stride, q_out_stride;
  const __nv_bfloat16* k_in;
  const __nv_bfloat16* v_in;
  int64_t k_in_stride;         // v's too
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int64_t k_out_stride;        // of a token's rows, or of a token in its page
  int64_t k_out_head_stride;
  const int32_t* slots;        // [n], or null: rows of their own
  int64_t page_stride;
  int32_t page_size, n_slots;
  int32_t H, Hk, Hv;
  int32_t inverse;
  int32_t block_tokens;        // (the launcher's)
};
cudaError_t launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t stream);

// Row moves within a cache (cache_move.cu).
struct CacheMoveArgs {
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  const int32_t* src;          // [n_groups, width]
  const int32_t* dst;
  int64_t n_groups;
  int32_t width, page_size, n_slots;
  int64_t page_stride, token_stride, head_stride;
};
cudaError_t launch_cache_move(const CacheMoveArgs& a, int heads, cudaStream_t stream);

cudaError_t launch_selftest_bounded_wait(uint64_t timeout_ns, uint32_t* d_flag,
                                         cudaStream_t stream);

}  // namespace h3
