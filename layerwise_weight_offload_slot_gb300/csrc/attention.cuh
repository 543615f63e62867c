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

// 32 columns of 32 rows, one row a lane (w: 16 pairs of bf16), to global memory: row(r)
// is where row (lane & ~3) + r of the warp begins (its column 0; NULL: not written), c32
// the first column, hd the columns of a row.  Four lanes first exchange their rows' 16-byte
// pieces, so that an instruction writes 64 bytes of eight rows; 16 bytes of 32 rows take
// four times the cycles (the end of a dK, dV item at head dim 128: 4.4 us).
template <typename Row>
__device__ __forceinline__ void put_rows32(uint32_t (&w)[16], int c32, int hd, int lane, const Row& row) {
#pragma unroll
    for (int x = 1; x <= 2; x <<= 1) {
        const bool up = lane & x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k & x) continue;             // pieces k and k + x change places across lanes that differ by x
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t &a = w[4 * k + u], &b = w[4 * (k + x) + u];
                const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? a : b, x);
                if (up) a = got;
                else b = got;
            }
        }
    }
    const int col = c32 + 8 * (lane & 3);
    if (col >= hd) return;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (__nv_bfloat16* p = row(r)) *reinterpret_cast<uint4*>(p + col) = make_uint4(w[4 * r], w[4 * r + 1], w[4 * r + 2], w[4 * r + 3]);
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
// heads x (128 / box_heads rounded down) rows, columns past hd zero-filled.
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

// Lane 0's value.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Rows [from, to) of a tile set to zero by `step` threads, this one the lane-th.  Rows behind a sequence's
// end may hold anything; as the contracted index of a product they would turn
// a zero probability times an infinity into NaN.  The caller's mbarrier arrival
// after this orders the writes (async proxy) before the MMA that reads them.
template <int NB, bool TAIL>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int lane, int step, int to = 128) {
    using T = AttnTile<NB, TAIL>;
    const uint4 z = make_uint4(0, 0, 0, 0);
    for (int i = from * 8 + lane; i < to * 8; i += step) {
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) reinterpret_cast<uint4*>(tile + blk * T::BLK)[i] = z;
    }
    if constexpr (TAIL)
        for (int i = from * 2 + lane; i < to * 2; i += step) reinterpret_cast<uint4*>(tile + NB * T::BLK)[i] = z;
    fence_proxy_async_smem();
}

// Valid rows of sequence b: lens[b] taken into 0 .. n, or n.  Read from L2: a kernel
// may do so before its programmatic-launch wait.
__device__ __forceinline__ int seq_len(const int* lens, int b, int n) {
    return lens ? min(max(__ldcg(lens + b), 0), n) : n;
}

// Packed sequences: sequence b is rows starts[b] .. starts[b + 1] - 1.  Tiles of t rows
// that do not cross its ends have the slots from starts[b] / t + b on, of which the
// next sequence's lie far enough: floor(s' / t) + 1 - floor(s / t) >= ceil((s' - s) / t).
// So a grid of rows / t + batch slots finds its tiles in the starts alone, without a sum
// over the lengths before it, and a slot too many a sequence finds none.
struct PackedTile {
    int b, tile;                // sequence and which of its tiles; tile < 0: none
    int row0, n;                // the sequence's first row and its length
};

// starts[b] taken into 0 .. rows; L2, as seq_len.
__device__ __forceinline__ int seq_start(const int* starts, int b, int rows) { return min(max(__ldcg(starts + b), 0), rows); }

__host__ __device__ __forceinline__ int packed_slots(int rows, int batch, int t) { return rows / t + batch; }

// The tile of a slot, by a whole warp: 31 sequences a step, with the start of the
// next one beside them (one trip to L2 for up to 31 sequences).
__device__ __forceinline__ PackedTile packed_tile(const int* starts, int batch, int rows, int t, int slot) {
    const int lane = threadIdx.x & 31;
    PackedTile p;
    p.b = 0;
    for (int n = batch;;) {                 // it is one of b .. b + n - 1
        const int step = (n + 30) / 31, i = p.b + min(lane * step, n);
        const int s = seq_start(starts, i, rows);
        const unsigned m = __ballot_sync(0xFFFFFFFFu, lane * step < n && s / t + i <= slot);
        const int k = m ? 31 - __clz(m) : 0;
        if (step == 1) {
            p.b += k;
            p.row0 = __shfl_sync(0xFFFFFFFFu, s, k);
            p.n = max(0, __shfl_sync(0xFFFFFFFFu, s, k + 1) - p.row0);
            break;
        }
        p.b += k * step;
        n = min(step, n - k * step);
    }
    p.tile = slot - (p.row0 / t + p.b);
    if (static_cast<long long>(p.tile) * t >= p.n) p.tile = -1;
    return p;
}

// Rows of sequence b of the other matrix: its first row and length.  `same`: it is packed
// as the one that the tile was found in.
__device__ __forceinline__ void packed_other(const int* starts, int b, int rows, bool same, const PackedTile& p, int& row0, int& n) {
    row0 = same ? p.row0 : seq_start(starts, b, rows);
    n = same ? p.n : max(0, seq_start(starts, b + 1, rows) - row0);
}

// One past the last key that query i sees (off = nk - nq, cb = causal block,
// 0: none): floor((i + off) / cb) >= floor(j / cb).  cb is at most the rows of K, so 2^30:
// nothing here passes 2^31.
__device__ __forceinline__ int key_end(int i, int off, int cb, int klen) {
    if (cb == 0) return klen;
    const int t = i + off;
    return t < 0 ? 0 : min(klen, (t / cb + 1) * cb);
}

// The first query that sees key j (may be negative: all do).
__device__ __forceinline__ int query_begin(int j, int off, int cb) { return cb == 0 ? 0 : (j / cb) * cb - off; }

}  // namespace dlo
