// What the attention kernels share: the shared-memory tile of 128 rows of one
// head, its TMA loads and tensor map, and which query sees which key.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace dlo {

// 128 rows of one head: NB blocks of 64 columns (128-byte swizzle), then with
// TAIL 16 more columns (32-byte swizzle).
template <int NB, bool TAIL>
struct AttnTile {
    static constexpr int HDP = NB * 64 + (TAIL ? 16 : 0);   // padded head dim
    static constexpr int BLK = 128 * 128;                   // 128 rows x 128 B (64 cols)
    static constexpr int TBLK = TAIL ? 128 * 32 : 0;        // 128 rows x 32 B (16 cols)
    static constexpr int BYTES = NB * BLK + TBLK;           // one Q, K or V tile
};

template <int NB, bool TAIL>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* main,
                                          const CUtensorMap* tail, int h, int row0, int b,
                                          uint32_t bar) {
    using T = AttnTile<NB, TAIL>;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) tma_load_4d(dst + blk * T::BLK, main, blk * 64, h, row0, b, bar);
    if constexpr (TAIL) tma_load_4d(dst + NB * T::BLK, tail, NB * 64, h, row0, b, bar);
}

// Columns [32 c, 32 c + 32) of row `row` as bf16 (w: 16 pairs) into such a tile,
// in the layout that TMA stores from and loads to.
template <int NB, bool TAIL>
__device__ __forceinline__ void put_row(uint8_t* tile, int row, int c, const uint32_t (&w)[16]) {
    using T = AttnTile<NB, TAIL>;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint4 v = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        if (c < 2 * NB)
            *reinterpret_cast<uint4*>(tile + (c >> 1) * T::BLK + row * 128 + ((((c & 1) * 4 + k) ^ (row & 7)) << 4)) = v;
        else if (TAIL && k < 2)
            *reinterpret_cast<uint4*>(tile + NB * T::BLK + row * 32 + ((k ^ ((row >> 2) & 1)) << 4)) = v;
    }
}

template <int NB, bool TAIL>
__device__ __forceinline__ void store_tile(uint32_t src, const CUtensorMap* main, const CUtensorMap* tail, int h, int row0, int b) {
    using T = AttnTile<NB, TAIL>;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) tma_store_4d(main, src + blk * T::BLK, blk * 64, h, row0, b);
    if constexpr (TAIL) tma_store_4d(tail, src + NB * T::BLK, NB * 64, h, row0, b);
}

// [batch, rows, heads, hd] view of a bf16 matrix whose batch b, row r, head h
// starts at base + (b * rows + r) * ld + h * hd; box of box_cols x box_heads
// heads x 128 / box_heads rows, columns past hd zero-filled.
inline bool make_map4(CUtensorMap* m, const void* base, int batch, int rows, int heads, int hd, int ld,
                      int box_cols, CUtensorMapSwizzle sw, int box_heads = 1) {
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(heads),
                          static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(hd) * 2, static_cast<cuuint64_t>(ld) * 2,
                             static_cast<cuuint64_t>(ld) * 2 * static_cast<cuuint64_t>(rows)};
    cuuint32_t box[4] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_heads),
                         static_cast<cuuint32_t>(128 / box_heads), 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// mbar_wait by a whole warp: the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const volatile int* abort) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort));
}

// Rows [from, 128) of a tile set to zero by `step` threads, this one the lane-th.  Rows behind a sequence's
// end may hold anything; as the contracted index of a product they would turn
// a zero probability times an infinity into NaN.  The caller's mbarrier arrival
// after this orders the writes (async proxy) before the MMA that reads them.
template <int NB, bool TAIL>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int lane, int step) {
    using T = AttnTile<NB, TAIL>;
    const uint4 z = make_uint4(0, 0, 0, 0);
    for (int i = from * 8 + lane; i < 128 * 8; i += step) {
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) reinterpret_cast<uint4*>(tile + blk * T::BLK)[i] = z;
    }
    if constexpr (TAIL)
        for (int i = from * 2 + lane; i < 128 * 2; i += step) reinterpret_cast<uint4*>(tile + NB * T::BLK)[i] = z;
    fence_proxy_async_smem();
}

// Valid rows of sequence b: lens[b] taken into 0 .. n, or n.  Read from L2: a kernel
// may do so before its programmatic-launch wait.
__device__ __forceinline__ int seq_len(const int* lens, int b, int n) {
    return lens ? min(max(__ldcg(lens + b), 0), n) : n;
}

// One past the last key that query i sees (off = nk - nq, cb = causal block,
// 0: none): floor((i + off) / cb) >= floor(j / cb).  cb <= nk.
__device__ __forceinline__ int key_end(int i, int off, int cb, int klen) {
    if (cb == 0) return klen;
    const int t = i + off;
    return t < 0 ? 0 : min(klen, (t / cb + 1) * cb);
}

// The first query that sees key j (may be negative: all do).
__device__ __forceinline__ int query_begin(int j, int off, int cb) { return cb == 0 ? 0 : (j / cb) * cb - off; }

}  // namespace dlo
