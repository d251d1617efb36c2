// The ring of K and V tiles of the tree forward (attn_tree.cu): the order of its entries, and which of them a loader
// issues.  Plain arithmetic, so that it can be checked on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define H3_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define H3_HOST_DEVICE inline
#endif

namespace h3 {
namespace ring {

constexpr int kSlots = 5;  // entry e lies in slot e mod 5

// Entries in the order of their loads, which is that of their use: K of the first tile, then K of every
// tile before V of the one before it.
H3_HOST_DEVICE uint32_t k_entry(int32_t t) { return t == 0 ? 0u : 2u * t - 1; }
H3_HOST_DEVICE uint32_t v_entry(int32_t t, int32_t steps) { return t + 1 < steps ? 2u * t + 2 : 2u * t + 1; }

// Copy c of loader `me` (0, 1) of a block with `steps` tiles: one loads K tiles, the other V tiles; or (kTwo) each K and V in
// turn of one stream's tiles, which are the block's `first`, first + 2, ..
template <bool kTwo>
H3_HOST_DEVICE uint32_t copy_entry(int32_t c, int me, int first, int32_t steps) {
  if (!kTwo) return me == 1 ? v_entry(c, steps) : k_entry(c);
  const int32_t t = 2 * (c >> 1) + first;
  return (c & 1) != 0 ? v_entry(t, steps) : k_entry(t);
}

// The first of a loader's `issued` copies that may still be on its way: a copy into a slot goes out when the entry five
// before it has been used, and entries are used in order, so those on their way are among five consecutive entries,
// of which a loader issues three at most.
H3_HOST_DEVICE int32_t first_on_its_way(int32_t issued) { return issued > 3 ? issued - 3 : 0; }

}  // namespace ring
}  // namespace h3
