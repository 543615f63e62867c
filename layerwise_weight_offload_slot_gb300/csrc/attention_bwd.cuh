// What the attention backward kernels share: tiles' slots in shared memory, tensor memory
// plans, barriers, the products and the row statistics' operands.
#pragma once
#include "attention.cuh"

namespace dlo {

namespace {

constexpr int kTile = 128;
constexpr int kGroups = 4;                               // warps that share 32 TMEM lanes
constexpr int kCols = kTile / kGroups;                   // columns of each
constexpr int kThreadsB = 128 + 32 * 4 * kGroups;
// Row statistics of one query tile as the operand of one more step of 16 of a
// product: 128 rows x 16 bf16 (32-byte rows, 32-byte swizzle), columns 0..2 the
// three bf16 parts of -L, 3..5 those of -D.
constexpr int kStatBytes = kTile * 32;

// Shared memory of one CTA: two tiles that stay (Q and dO; K and V), slots for the
// two streams of tiles that move (K and V; Q and dO), and per-row values.
//
// A reload takes ~1 us (2000 cycles) from L2, longer than an iteration's
// products.  Tile i of the first stream (K in dq_kernel, Q in dkv_kernel) is
// held from its first product to the last one of its iteration, one of the
// second (V, dO) for a shorter time.  Up to head dim 80 each stream has three
// slots.  Above, the two streams share five (dq) or four (dkv) slots so that
// the earlier freed tile makes room for the tile needed sooner: slot s holds
// first-stream tile s, then second-stream tile s + SLOTS - 2, then first-stream
// tile s + SLOTS, ... (slots 2.. begin with the second stream).  Against separate
// 3 + 2 and 2 + 2 rings this leaves a reload 4/3 (dq) and 1 (dkv) iterations.
struct Slot {
    int s;
    uint32_t ph;              // parity of this use of the slot's barriers
};

template <int SLOTS, bool SHARED, bool SECOND>
__device__ __forceinline__ Slot slot_of(int i) {
    if constexpr (SHARED) {
        const int r = i % SLOTS;
        return SECOND ? Slot{(i + 2) % SLOTS, r >= SLOTS - 2 ? 1u : 0u} : Slot{r, r >= 2 ? 1u : 0u};
    } else {
        constexpr int N = SLOTS / 2;
        return {i % N + (SECOND ? N : 0), static_cast<uint32_t>(i / N) & 1u};
    }
}

template <int NB, bool TAIL, bool DQ>
struct BwdPlan {
    using T = AttnTile<NB, TAIL>;
    static constexpr int TILE = T::BYTES;
    static constexpr bool SHARED = NB == 2;
    static constexpr int SLOTS = SHARED ? (DQ ? 5 : 4) : 6;
    static constexpr int STATS = SHARED ? 2 : 3;            // statistics operands of dkv_kernel, tile i in i % STATS
    static constexpr int A0_OFF = 0, A1_OFF = TILE;
    static constexpr int R_OFF = 2 * TILE;
    // dq: D of each row and four parts of it; dkv: the two selecting operands, then
    // the statistics
    static constexpr int SEL_OFF = R_OFF + SLOTS * TILE;
    static constexpr int STAT_OFF = SEL_OFF + 2 * kStatBytes;
    static constexpr int BAR_OFF = DQ ? SEL_OFF + (1 + kGroups) * kTile * 4 : STAT_OFF + STATS * kStatBytes;
    // a_full, raw0, raw1, s_full, drain2, d_full, e0, e1, done, drain, s_read, d_read, staged; full, empty [SLOTS]
    static constexpr int NBARS = 13 + 2 * SLOTS;
    static constexpr int TMEM_SLOT_OFF = BAR_OFF + NBARS * 8;
    static constexpr int ABORT_OFF = TMEM_SLOT_OFF + 4;
    static constexpr int USED = ABORT_OFF + 4;
    // one CTA per SM (it owns all 512 TMEM columns); 1 KB to align the base
    // where there is room, else the kernel checks that the base is aligned
    static constexpr int WANT = USED + 1024 > 118784 ? USED + 1024 : 118784;
    static constexpr int BYTES = WANT < 227 * 1024 ? WANT : 227 * 1024;
    static_assert(USED <= 227 * 1024, "attention backward shared memory plan exceeds 227 KB");
};

// dkv_kernel's tensor memory: S^T [0, 128), dP^T [128, 256), then dV and dK, then P^T
// and dS^T (64 columns each) where 512 columns hold them.  A P or dS that
// takes the place of its product instead makes the next product wait for it.
template <int HDP>
struct DkvTmem {
    static constexpr uint32_t DV_COL = 256, DK_COL = DV_COL + HDP;
    static constexpr uint32_t FREE = 512 - DK_COL - HDP;
    static constexpr bool P_APART = FREE >= 64, DS_APART = FREE >= 128;
    static constexpr uint32_t P_COL = P_APART ? DK_COL + HDP : 0;
    static constexpr uint32_t DS_COL = DS_APART ? P_COL + 64 : 128;
    // Issuing warps of dkv_kernel.  Two (S and dV; dP and dK) keep the tensor core
    // fed while one waits: at head dim 64 (72) a tile takes 0.90 (1.11) us against
    // 1.09 (1.27).  Where P and dS lie in the places of S and dP, each product
    // has to wait for one of the other kind and the order of issue counts: one
    // (head dim 128: 1.34 against 1.56).
    static constexpr int ISSUERS = P_APART ? 2 : 1;
    static_assert(DK_COL + HDP <= 512, "attention backward tensor memory plan");
};

// 128 x 128 (+)= A B^T over the head dim, both operands K-major in shared memory.
template <int NB, bool TAIL>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t a, uint64_t at, uint64_t b, uint64_t bt) {
    using T = AttnTile<NB, TAIL>;
    constexpr uint32_t id = idesc_bf16_f32(kTile, kTile);
#pragma unroll
    for (int kk = 0; kk < NB * 4; ++kk) {
        const uint32_t off = ((kk >> 2) * T::BLK + (kk & 3) * 32) >> 4;
        tc_mma_f16(d, a + off, b + off, id, kk > 0);
    }
    if constexpr (TAIL) tc_mma_f16(d, at, bt, id, 1u);
}

// 128 x hd += A B: A in TMEM (bf16 pairs: the kCols contracted indices of group
// e at a + GAP e), B a tile of shared memory whose rows are the contracted index.
template <int NB, bool TAIL, int GAP>
__device__ __forceinline__ void mma_accumulate(uint32_t d, uint32_t a, uint64_t b, uint64_t bt, bool first) {
    constexpr uint32_t id = idesc_bf16_f32(kTile, NB * 64, true);
    constexpr uint32_t idt = idesc_bf16_f32(kTile, 16, true);
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk) {
        const uint32_t ak = a + kk / (kCols / 16) * GAP + kk % (kCols / 16) * 8;
        const uint32_t acc = (!first || kk > 0) ? 1u : 0u;
        tc_mma_f16_ts(d, ak, b + ((kk * 2048) >> 4), id, acc);
        if constexpr (TAIL) tc_mma_f16_ts(d + NB * 64, ak, bt + ((kk * 512) >> 4), idt, acc);
    }
}

// x as the sum of three bf16 values (to ~2^-24 of x), two of them in one word.
__device__ __forceinline__ void split3(float x, uint32_t& hi_mid, uint32_t& lo) {
    const float a = __bfloat162float(__float2bfloat16_rn(x));
    const float b = __bfloat162float(__float2bfloat16_rn(x - a));
    hi_mid = pack_bf16x2(a, b);
    lo = __bfloat16_as_ushort(__float2bfloat16_rn(x - a - b));
}

// The end of an issuing warp: on an abort, its MMAs in flight are waited for.
template <typename Fail>
__device__ __forceinline__ void end_issue(bool one, bool ok, uint32_t drain, const volatile int* abort_flag, const Fail& fail) {
    if (one) {
        if (!ok) fail();
        if (*abort_flag) {
            tc_commit(drain);
            mbar_wait(drain, 0, nullptr);
        }
    }
    __syncwarp();
}

// A raw score that no score makes up for: exp of it is 0, and times 0 it is 0.
constexpr float kNothing = -1e30f;

// Row `r` of a statistics operand.
__device__ __forceinline__ void write_stat(uint4* stat, int r, float neg_l, float neg_d) {
    uint32_t l01, l2, d01, d2;
    split3(neg_l, l01, l2);
    split3(neg_d, d01, d2);
    const int x = (r >> 2) & 1;          // 32-byte swizzle: the row's two pieces change places
    stat[2 * r + x] = make_uint4(l01, l2 | (d01 << 16), (d01 >> 16) | (d2 << 16), 0);
    stat[2 * r + 1 - x] = make_uint4(0, 0, 0, 0);
}

}  // namespace

}  // namespace dlo
