// Work lists of the forward's other key walks (host only): attention over a
// list of key tiles per query block, and over a shared prefix and the row's
// own document.
//
// Both lists consist of segments of at most kUnitRows query rows of one head,
// placed on the forward's persistent CTA pairs in list order, each on the pair
// with the least load so far.  Whole segments come first; a tail of them is
// split along its key tiles into pieces small enough to fill the pairs evenly,
// and the join pass combines the pieces' partial rows.  How long the tail is
// and how small its pieces are is chosen by simulating the placement.
#include <algorithm>
#include <cstring>

#include "h3attn_internal.h"

namespace h3 {

namespace {

// A segment before placement.
struct Item {
  WalkUnit u;
  int32_t tiles;      // key tiles (list walk: at most this many)
  int32_t limit;      // every piece begins below this tile
  bool direct;        // writes the output itself unless it is split
  int32_t pieces = 1;
  int32_t part = -1;  // first partial row of piece 0
  int32_t pack = 1;   // causal walk: query heads of its rows
  bool partial() const { return !direct || pieces > 1; }
  int32_t rows() const { return pack * (u.q_end - u.q_row0); }
  // pieces of at most m tiles
  int32_t split(int32_t m) const { return std::max(1, std::min((tiles + m - 1) / m, limit)); }
};

// First tile of piece c of n (c = n: the end): even shares, but every piece
// begins below the item's limit.
int32_t bound(const Item& it, int32_t c, int32_t n) {
  if (c == n) return it.tiles;
  return (int32_t)std::min<int64_t>((int64_t)it.tiles * c / n, it.limit - (n - c));
}

// Rows to combine from the partial rows of an item and from the keys [key_lo,
// key_hi) themselves.
struct Join {
  int32_t row0, row1, head;
  int32_t item;
  int32_t key_lo, key_hi;
  int32_t shift = 0;  // of the head's partial rows in the item's
};

// Times in hundredths of a microsecond, as measured on GB300 for segments of 1 to
// 32 tiles.  A CTA pair runs one segment of up to kUnitRows rows at a time (1.28
// us a tile, and 4 us for its boundary, where the pipeline runs empty), or two
// streams of segments of half as many rows (1.50 us for a tile of each: the same
// products with twice the K and V tiles; but a boundary costs 1.7 us, as the other
// stream goes on).  So streams suit short walks, and rows of many documents, whose own
// tiles then take half as many rows along: 100 documents of 100 tokens over 512
// prefix rows 93 against 119 us, three of 4,096 over 2,430 rows 559 against 512.
// Partial rows cost a segment 1.3 us, and the join kJoinStart and kJoinRow for
// each (142,000 of them measured 33 us).
int64_t piece_cost(int32_t tiles, bool partial, int streams) {
  return (streams == 2 ? (int64_t)150 * tiles + 170 : (int64_t)128 * tiles + 400) + (partial ? 130 : 0);
}
// A pair's time from its streams' loads: a tile of a stream whose other one has
// ended takes 1.05 us.  (Without it tails were split that are better left whole:
// 8,192 tokens, 10 heads, 32 tiles for each 256-row block 124 against 111 us.)
double pair_time(int64_t a, int64_t b) {
  return 0.5 * (double)(a + b) + 0.2 * (double)(a > b ? a - b : b - a);
}
constexpr double kJoinStart = 320.0;
constexpr double kJoinRow = 0.0233;
// Rows of a chunk of the prefix walk whose partial rows cost a tile's time.
constexpr int kRowsPerTile = 87;

// The same for the few-rows kernel's blocks of `tiles` tiles each, two to an SM: a
// step of 64 keys takes a block 0.65 us alone on its SM (0.44 with up to 16 rows)
// and two of them 0.95 us.  Its launch with the join takes 2.5 us less than the
// tensor-core kernel's.
double rows_cost(int32_t tiles, int64_t blocks, int pairs, int32_t S) {
  const double step = blocks > 2 * pairs ? 95.0 : S > 16 ? 65.0 : 44.0;
  return kJoinStart - 250.0 + 2.0 * tiles * step * (double)((blocks + 4 * pairs - 1) / (4 * pairs));
}

// Row numbers are 32-bit, and the walks' go up to a segment past the last row.
bool too_long(const int32_t* cu, int32_t n_docs) { return cu[n_docs] > INT32_MAX - kUnitRows; }
constexpr char kTooLong[] = "too many tokens for the work list of a sparse, prefix or causal forward";

// Splits a tail of the items (in list order) so that the pairs finish together;
// returns the estimated time.
double balance(std::vector<Item>& items, int pairs, int streams) {
  const int G = pairs * streams;
  const size_t U = items.size();
  std::vector<int32_t> pair_of, heap(G);
  std::vector<int64_t> load(G), cost;
  double best = -1.0;
  std::vector<int32_t> best_pieces(U, 1);
  std::vector<int64_t> tail_tiles(U + 1, 0);  // tiles of items [i, U)
  for (size_t i = U; i-- > 0;) tail_tiles[i] = tail_tiles[i + 1] + items[i].tiles;
  const auto consider = [&](size_t whole, int32_t m) {
    cost.clear();
    int64_t rows = 0;
    for (size_t i = 0; i < U; ++i) {
      const int32_t n = i < whole ? 1 : items[i].split(m);
      const bool partial = !items[i].direct || n > 1;
      for (int32_t c = 0; c < n; ++c)
        cost.push_back(piece_cost(bound(items[i], c + 1, n) - bound(items[i], c, n), partial, streams));
      if (partial) rows += (int64_t)n * items[i].rows();
    }
    const double join = rows > 0 ? kJoinStart + (double)rows * kJoinRow : 0.0;
    // (no placement finishes before the mean load or the largest piece)
    int64_t sum = 0, most = 0;
    for (int64_t c : cost) {
      sum += c;
      most = std::max(most, c);
    }
    if (best >= 0.0 && std::max((double)sum / G, streams == 2 ? pair_time(most, 0) : (double)most) + join >= best) return;
    pair_of.resize(cost.size());
    assign_pairs(cost.size(), [&](size_t i) { return cost[i]; }, G, pair_of.data(), load.data(), heap.data());
    double last = 0.0;
    for (int p = 0; p < pairs; ++p) last = std::max(last, pair_time(load[p], streams == 2 ? load[p + pairs] : load[p]));
    const double score = last + join;
    if (best < 0.0 || score < best) {
      best = score;
      for (size_t i = 0; i < U; ++i)
        best_pieces[i] = i < whole ? 1 : items[i].split(m);
    }
  };
  consider(U, 1);
  int32_t longest = 0;
  for (const Item& it : items) longest = std::max(longest, it.tiles);
  const int64_t round = G, full = (int64_t)U / round * round;
  std::vector<std::pair<size_t, int32_t>> tried;
  const auto consider_once = [&](size_t whole, int64_t m) {
    const std::pair<size_t, int32_t> way(whole, (int32_t)std::max<int64_t>(1, m));
    if (way.second >= longest || std::find(tried.begin(), tried.end(), way) != tried.end()) return;
    tried.push_back(way);
    consider(whole, way.second);
  };
  for (int64_t back : {(int64_t)0, round / 4, round / 2, round, 2 * round, full}) {
    if (back > full) continue;
    const size_t whole = (size_t)(full - back);
    if (whole == U) continue;
    // pieces that give every pair 1 .. 4 of them, or cut the longest in 2, 3, 4
    for (int r = 1; r <= 4; ++r) consider_once(whole, (tail_tiles[whole] + round * r - 1) / (round * r));
    for (int n = 2; n <= 4; ++n) consider_once(whole, (longest + n - 1) / n);
  }
  for (size_t i = 0; i < U; ++i) items[i].pieces = best_pieces[i];
  return best;
}

// Pieces, partial rows, placement and join records of the balanced items.
// make(item, piece) gives a piece's segment (part filled in here).
template <class Make>
std::string finish(std::vector<Item>& items, std::vector<Join>& joins, int G, Make make, WalkPlan& w) {
  int64_t rows = 0;
  std::vector<WalkUnit> segs;
  std::vector<int64_t> cost;
  for (Item& it : items) {
    if (it.partial()) {
      it.part = (int32_t)rows;
      rows += (int64_t)it.pieces * it.rows();
      if (rows >= (int64_t(1) << 31)) return "the layout needs 2^31 or more partial rows";
    }
    for (int32_t c = 0; c < it.pieces; ++c) {
      WalkUnit s = make(it, c);
      s.part = it.partial() ? it.part + c * it.rows() : -1;
      segs.push_back(s);
      cost.push_back(piece_cost(bound(it, c + 1, it.pieces) - bound(it, c, it.pieces), it.partial(), w.streams));
    }
  }
  w.part_rows = rows;
  for (size_t i = 0; i < items.size(); ++i)
    if (items[i].direct && items[i].pieces > 1)
      for (int32_t h = 0; h < items[i].pack; ++h) {
        const WalkUnit& u = items[i].u;
        joins.push_back(Join{u.q_row0, u.q_end, u.head + h, (int32_t)i, 0, 0, h * (u.q_end - u.q_row0)});
      }
  w.joins.clear();
  w.join_warps = 0;
  for (const Join& j : joins) {
    JoinRec r;
    std::memset(&r, 0, sizeof(r));
    r.head = j.head;
    r.key_lo = j.key_lo;
    r.key_hi = j.key_hi;
    const Item& it = items[j.item];
    r.part = it.part + j.shift;
    r.rows = it.rows();
    r.n = it.pieces;
    r.q_row0 = it.u.q_row0;
    int32_t most = kJoinRows;  // rows that leave each its warps
    while (most > 1 && kJoinParts * (kJoinRows / most) < r.n) most /= 2;
    for (int32_t x = j.row0; x < j.row1; x += most) {
      r.row0 = x;
      r.row1 = std::min(x + most, j.row1);
      w.join_warps = std::max(w.join_warps, (r.row1 - r.row0) << join_warps_log2(r.row1 - r.row0, r.n));
      w.joins.push_back(r);
    }
  }
  // two streams a pair: twice the bins, the first of every pair before the second
  const int bins = w.streams * G;
  w.units.resize(segs.size());
  std::vector<int32_t> off((size_t)bins + 1), pair_of(segs.size()), heap(bins);
  std::vector<int64_t> load(bins);
  assign_pairs(segs.size(), [&](size_t i) { return cost[i]; }, bins, pair_of.data(), load.data(), heap.data());
  const int32_t used =
      group_by_pair(segs.data(), segs.size(), bins, w.units.data(), off.data(), pair_of.data(), heap.data());
  w.n_pairs = std::min(used, G);
  w.unit_off.clear();
  if (w.streams == 1) {
    w.unit_off.assign(off.begin(), off.begin() + w.n_pairs + 1);
  } else {
    for (int32_t p = 0; p < w.n_pairs; ++p)
      for (int32_t b : {p, p + G}) {
        w.unit_off.push_back(off[b]);
        w.unit_off.push_back(off[b + 1]);
      }
  }
  if (w.joins.size() >= (size_t(1) << 31)) return "the layout needs 2^31 or more join records";
  return "";
}

}  // namespace

std::string build_list_walk(const int32_t* cu, int32_t n_docs, int32_t num_heads, int32_t q_block, int32_t max_blocks,
                            int grid, WalkPlan& w) {
  if (too_long(cu, n_docs)) return kTooLong;
  const int G = grid > 0 ? grid : 1;
  std::vector<int32_t> order(n_docs), block0(n_docs);
  int32_t blocks = 0;
  for (int32_t d = 0; d < n_docs; ++d) {
    order[d] = d;
    block0[d] = blocks;
    blocks += (cu[d + 1] - cu[d] + q_block - 1) / q_block;
  }
  // longest documents first, then head, then query block: the pairs running at
  // one moment read the K and V of one or two heads, which stay in L2
  std::stable_sort(order.begin(), order.end(),
                   [cu](int32_t x, int32_t y) { return cu[x + 1] - cu[x] > cu[y + 1] - cu[y]; });
  // 256-row segments in two streams a pair, or, where the blocks allow it,
  // 512-row ones in one: whichever is estimated to finish first
  std::vector<Item> items;
  double best = -1.0;
  for (int streams = q_block == kUnitRows ? 1 : 2; streams <= 2; ++streams) {
    std::vector<Item> list;
    for (int32_t d : order) {
      const int32_t b = cu[d], e = cu[d + 1];
      const int32_t tiles = std::min(max_blocks, (e - b + kKeyTile - 1) / kKeyTile);
      for (int32_t h = 0; h < num_heads; ++h)
        for (int32_t r = b; r < e;) {
          const int32_t end = (int32_t)std::min<int64_t>((int64_t)r + kUnitRows / streams, e);
          list.push_back(Item{WalkUnit{r, end, b, e, h, block0[d] + (r - b) / q_block, 0, -1}, tiles, tiles, true});
          r = end;
        }
    }
    const double time = balance(list, G, streams);
    if (best < 0.0 || time < best) {
      best = time;
      w.streams = streams;
      items.swap(list);
    }
  }
  for (Item& it : items) it.pieces = std::min(it.pieces, 65535);  // the field's width
  std::vector<Join> joins;
  return finish(items, joins, G, [](const Item& it, int32_t c) {
    WalkUnit s = it.u;
    s.b = (int32_t)((uint32_t)c | ((uint32_t)it.pieces << 16));
    return s;
  }, w);
}

static WalkUnit prefix_piece(const Item& it, int32_t c) {
  WalkUnit s = it.u;
  s.a = bound(it, c, it.pieces);
  s.b = bound(it, c + 1, it.pieces);
  return s;
}

// The prefix walk's segments of up to kUnitRows / streams rows, not yet balanced.
// mix_long: documents longer than a chunk share chunks too, which saves passes
// over the prefix but makes segments that walk several long documents and cannot
// be split there.
static std::string prefix_items(const int32_t* cu, int32_t n_docs, int32_t num_heads, int32_t tp, int streams,
                                bool mix_long, std::vector<OwnTile>& own_tiles, std::vector<Item>& items, std::vector<Join>& joins) {
  const int32_t most = kUnitRows / streams;
  // The rows are cut into chunks of up to `most` rows, which walk the prefix once
  // for all their rows and then their documents' own tiles.  A document joins the
  // open chunk of the documents before it unless that costs it a chunk more.
  struct Piece {
    int32_t doc, row0, row1;
  };
  std::vector<std::vector<Piece>> chunks;
  int32_t filled = 0;  // rows of the last chunk
  const auto tiles_of = [cu](int32_t d) { return (cu[d + 1] - cu[d] + kKeyTile - 1) / kKeyTile; };
  for (int32_t d = 0; d < n_docs; ++d) {
    const int32_t L = cu[d + 1] - cu[d];
    const bool alone = L > most && !mix_long;
    int32_t at = cu[d];
    if (filled > 0 && filled < most && !alone) {
      const int32_t r = std::min(L, most - filled);
      if ((L - r + most - 1) / most < (L - 1) / most + 1) {
        chunks.back().push_back(Piece{d, at, at + r});
        filled += r;
        at += r;
      }
    }
    while (at < cu[d + 1]) {
      const int32_t r = std::min(cu[d + 1] - at, most);
      chunks.push_back({Piece{d, at, at + r}});
      filled = alone ? most : r;
      at += r;
    }
  }
  // What a chunk over several documents walks after the prefix.  Documents of
  // at most kJoinOwnKeys tokens take a whole tile each, for a few keys: where
  // there are more of them than the chunk's partial rows cost (kRowsPerTile),
  // the chunk leaves partial rows and the join attends to them.
  struct Own {
    int32_t first = 0, n = 0;
    bool join = false;
  };
  std::vector<Own> own(chunks.size());
  own_tiles.clear();
  const auto small = [cu](int32_t d) { return cu[d + 1] - cu[d] <= kJoinOwnKeys; };
  for (size_t c = 0; c < chunks.size(); ++c) {
    if (chunks[c].size() == 1) continue;
    const int32_t q0 = chunks[c].front().row0, rows = chunks[c].back().row1 - q0;
    int32_t tiny = 0;
    for (const Piece& p : chunks[c]) tiny += small(p.doc);
    own[c].first = (int32_t)own_tiles.size();
    own[c].join = tiny > 2 + rows / kRowsPerTile;
    for (const Piece& p : chunks[c]) {
      if (own[c].join && small(p.doc)) continue;
      for (int32_t t = cu[p.doc]; t < cu[p.doc + 1]; t += kKeyTile) {
        OwnTile o;
        o.row = t;
        o.rem = cu[p.doc + 1] - t;
        o.lo = p.row0 - q0;
        o.hi = p.row1 - q0;
        for (int32_t r = 0; r < kUnitRows; r += 32) {
          uint32_t skip = 0;
          for (int32_t i = 0; i < 32; ++i) skip |= (uint32_t)(r + i < o.lo || r + i >= o.hi) << i;
          o.skip[r / 256][r % 256 / 32] = skip;
        }
        own_tiles.push_back(o);
      }
    }
    own[c].n = (int32_t)own_tiles.size() - own[c].first;
    if (own_tiles.size() >= (size_t(1) << 31) / sizeof(OwnTile)) return "the layout needs too large a table of own tiles";
  }
  // head by head: the pairs running at one moment share a head's prefix in L2
  for (int32_t h = 0; h < num_heads; ++h) {
    for (size_t x = 0; x < chunks.size(); ++x) {
      const std::vector<Piece>& c = chunks[x];
      const int32_t q0 = c.front().row0, q1 = c.back().row1;
      if (c.size() == 1) {
        const int32_t t = tp + tiles_of(c[0].doc);
        items.push_back(Item{WalkUnit{q0, q1, cu[c[0].doc], cu[c[0].doc + 1], h, 0, t, -1}, t, t, true});
        continue;
      }
      // (n = 0: a chunk of small documents walks the prefix alone)
      const int32_t t = tp + own[x].n;
      if (own[x].join)
        for (const Piece& p : c)
          joins.push_back(Join{p.row0, p.row1, h, (int32_t)items.size(), small(p.doc) ? cu[p.doc] : 0,
                               small(p.doc) ? cu[p.doc + 1] : 0});
      items.push_back(Item{WalkUnit{q0, q1, own[x].first, -own[x].n, h, 0, t, -1}, t, tp, !own[x].join});
    }
  }
  return "";
}

std::string build_prefix_walk(const int32_t* cu, int32_t n_docs, int32_t num_heads, int32_t prefix_len, int grid,
                              WalkPlan& w) {
  if (too_long(cu, n_docs)) return kTooLong;
  const int G = grid > 0 ? grid : 1;
  const int32_t tp = (int32_t)(((int64_t)prefix_len + kKeyTile - 1) / kKeyTile);
  int32_t longest = 0;
  for (int32_t d = 0; d < n_docs; ++d) longest = std::max(longest, cu[d + 1] - cu[d]);
  // Chunks of 512 rows, or of 256 in two streams a pair, long documents sharing
  // chunks or not, whichever is estimated to finish first.
  std::vector<Item> items;
  std::vector<Join> joins;
  double best = -1.0;
  for (int way = 0; way < 4; ++way) {
    const int streams = 1 + way / 2;
    const bool mix_long = way % 2 == 0;
    if (!mix_long && longest <= kUnitRows / streams) continue;
    std::vector<Item> list;
    std::vector<Join> list_joins;
    std::vector<OwnTile> own;
    const std::string why = prefix_items(cu, n_docs, num_heads, tp, streams, mix_long, own, list, list_joins);
    if (!why.empty()) return why;
    const double time = balance(list, G, streams);
    if (best < 0.0 || time < best) {
      best = time;
      w.streams = streams;
      w.own.swap(own);
      items.swap(list);
      joins.swap(list_joins);
    }
  }
  // A few rows of documents that the join can attend to: bound by reading the
  // prefix, a block per SM half (attn_rows.cu), where that is quicker.  Measured in
  // us, this and the tensor-core kernel: single queries, 21 heads over 5,033 rows
  // 64 17.9 / 19.7, 96 24.7 / 20.9; 8 heads 128 15.9 / 17.3, 256 24.9 / 18.5; 21
  // heads over 300 rows 256 13.1 / 14.4.
  const int32_t S = cu[n_docs], row_tiles = (S + kRowsTile - 1) / kRowsTile;
  if (S <= kRowsMax && longest <= kJoinOwnKeys && num_heads <= 65535) {
    const int64_t segs = (int64_t)row_tiles * num_heads;
    // equal pieces that fill the blocks' places once; no more than the join reads at once
    const int32_t most = (int32_t)std::min<int64_t>(std::max<int64_t>(1, 4 * G / segs), kJoinRows * kJoinParts);
    const int32_t each = (tp + most - 1) / most, pieces = (tp + each - 1) / each;
    const double time = rows_cost(each, segs * pieces, G, S) + (double)S * num_heads * pieces * kJoinRow;
    if (time <= best) {
      items.clear();
      joins.clear();
      w.own.clear();
      w.streams = 1;
      w.pieces = pieces;
      for (int32_t q0 = 0; q0 < S; q0 += kRowsTile)
        for (int32_t h = 0; h < num_heads; ++h) {
          const int32_t q1 = std::min(q0 + kRowsTile, S);
          for (int32_t d = 0; d < n_docs; ++d) {
            const int32_t r0 = std::max(cu[d], q0), r1 = std::min(cu[d + 1], q1);
            if (r0 < r1) joins.push_back(Join{r0, r1, h, (int32_t)items.size(), cu[d], cu[d + 1]});
          }
          Item it{WalkUnit{q0, q1, 0, 0, h, 0, tp, -1}, tp, tp, false};
          it.pieces = pieces;
          items.push_back(it);
        }
      return finish(items, joins, (int)std::min<size_t>(items.size() * pieces, size_t(1) << 20), prefix_piece, w);
    }
  }
  return finish(items, joins, G, prefix_piece, w);
}

// Keys and values that the causal walk's segments in work share, in bytes: heads
// are taken in batches of about so much (the L2 holds 129 MB).
constexpr int64_t kCausalBatch = 48 << 20;

std::string build_causal_walk(const int32_t* cu, int32_t n_docs, int32_t num_heads, int32_t num_kv_heads, int grid,
                              WalkPlan& w) {
  if (too_long(cu, n_docs)) return kTooLong;
  const int G = grid > 0 ? grid : 1;
  const int32_t pack = causal_pack(num_heads / num_kv_heads), toks = kKeyTile / pack;
  std::vector<int32_t> order(n_docs);
  for (int32_t d = 0; d < n_docs; ++d) order[d] = d;
  std::stable_sort(order.begin(), order.end(),
                   [cu](int32_t x, int32_t y) { return cu[x + 1] - cu[x] > cu[y + 1] - cu[y]; });
  // Segments of four query tiles, or of two in two streams a pair, whichever is
  // estimated to finish first; longest first within a batch of (document, key head)
  // pairs whose keys and values the L2 holds together.
  std::vector<Item> items;
  double best = -1.0;
  for (int streams = 1; streams <= 2; ++streams) {
    const int32_t most = 4 / streams * toks;
    std::vector<Item> list;
    size_t batch = 0;
    int64_t bytes = 0;
    const auto close = [&] {
      std::stable_sort(list.begin() + batch, list.end(), [](const Item& x, const Item& y) { return x.tiles > y.tiles; });
      batch = list.size();
      bytes = 0;
    };
    for (int32_t d : order) {
      const int32_t b = cu[d], e = cu[d + 1];
      for (int32_t g = 0; g < num_kv_heads; ++g) {
        for (int32_t h = num_heads / num_kv_heads * g; h < num_heads / num_kv_heads * (g + 1); h += pack)
          for (int32_t r = b; r < e;) {
            const int32_t end = (int32_t)std::min<int64_t>((int64_t)r + most, e);
            const int32_t tiles = (end - b + kKeyTile - 1) / kKeyTile;
            list.push_back(Item{WalkUnit{r, end, b, e, h, 0, tiles, -1}, tiles, tiles, true});
            list.back().pack = pack;
            r = end;
            if (list.size() >= (size_t(1) << 30)) return "too many work units";
          }
        bytes += (int64_t)(e - b) * kHeadDim * 4;
        if (bytes >= kCausalBatch) close();
      }
    }
    close();
    const double time = balance(list, G, streams);
    if (best < 0.0 || time < best) {
      best = time;
      w.streams = streams;
      items.swap(list);
    }
  }
  std::vector<Join> joins;
  return finish(items, joins, G, prefix_piece, w);
}

}  // namespace h3
