// What the two bf16 kernels share that read K and V tiles through TMA.
#pragma once

#include "paged_attn.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace {

// Whether tile `t` has tokens that some row of the unit does not see.
template <int BN>
__device__ __forceinline__ bool edge_tile(int t, int pos_first, int pos_last, int window) {
  return t * BN + BN - 1 > pos_first || (window > 0 && t * BN <= pos_last - window);
}
__device__ __forceinline__ bool not_finite(uint32_t two) {
  return (two & 0x7f80u) == 0x7f80u || (two & 0x7f800000u) == 0x7f800000u;
}


// [num_blocks][bs][Hkv][D] bf16, boxes of 64 columns x 1 head x `box` tokens of one page.
bool make_page_map(CUtensorMap* m, const void* base, int num_blocks, int bs, int Hkv, int D, int box_rows) {
  auto enc = get_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)bs, (cuuint64_t)num_blocks};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)Hkv * D * 2, (cuuint64_t)bs * Hkv * D * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Loads of one K or V tile of BN tokens by a whole warp: rows of a page at a time, as boxes
// of `box` tokens x 64 columns.  Pages past the sequence and table entries out of range read
// as zeros, through a coordinate past the last page.
template <int D, int BN>
struct PageLoads {
  const int32_t* table;
  int kl, h, bs, num_blocks, box, per, boxes;
  __device__ PageLoads(const AttnArgs& a, const Item& it, int box_rows)
      : table(a.s.block_tables + (size_t)it.n * a.s.max_blocks), kl(it.r.kl), h(it.h), bs(a.bs),
        num_blocks(a.num_blocks), box(box_rows), per(BN / box_rows), boxes(per * (D / 64)) {}
  // Page of box `e` of tile `t`.
  __device__ __forceinline__ int page(int t, int e) const {
    const int j = t * BN + (e % per) * box;
    const int id = e < boxes && j < kl ? __ldg(table + j / bs) : -1;
    return id >= 0 && id < num_blocks ? id : num_blocks;
  }
  // `first`: page(t, lane), which the caller looked up ahead.
  __device__ __forceinline__ void load(uint8_t* tile, const CUtensorMap* map, uint64_t* bar, int t,
                                       int lane, int first) const {
    for (int e = lane; e < boxes; e += 32) {
      const int panel = e / per, rr = (e - panel * per) * box;
      const int id = e == lane ? first : page(t, e);
      tma_load_4d(tile + panel * (BN * 128) + rr * 128, map, bar, panel * 64, h, (t * BN + rr) % bs, id);
    }
  }
};

}  // namespace
}  // namespace gdn
