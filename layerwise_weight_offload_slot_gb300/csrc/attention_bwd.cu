// Backward pass of softmax attention on the 5th-generation tensor cores.
//
//   P = exp(S - L), S = Q K^T / sqrt(hd);   D = rowsum(dO O)
//   dS = P (dO V^T - D);   dV = P^T dO,  dK = dS^T Q / sqrt(hd),  dQ = dS K / sqrt(hd)
//
// Two launches, each recomputing S and dO V^T for its own direction, so that
// every gradient tile is accumulated by one CTA in tensor memory, in a fixed
// order: seven products instead of the five of a single pass, whose dQ would
// have to be added up in global memory by every key tile's CTA (fp32 traffic
// of nk / 128 times dQ, and sums in the order of arrival).
//
//   dq_kernel   CTA = 128 query rows of one head; walks the key tiles
//               S = Q K^T, dP = dO V^T, dQ += dS K
//   dkv_kernel  CTA = 128 keys of one key/value head; walks the query tiles
//               of every query head that shares it
//               S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//
// In both, dS (and P) is the A operand straight from tensor memory: the
// thread that owns a TMEM lane (a query row, a key) reads 32 columns of the
// fp32 product and writes their bf16 values.  The B operands of the accumulating
// products are the tiles already in shared memory, read MN-major.  20 warps: 0
// TMA, 1 and 2 MMA issue, 4..19 elementwise (four per 32 TMEM lanes, each a
// quarter of the 128 columns).  A product's place is free as soon as it has been
// read, so the next one runs while the elementwise warps work on it.
//
// What bounds it (measured on copies with parts left out, head dim 128): the
// elementwise work is hidden (exponentials left out: same time), loads alone
// take 0.77 us a tile of the dQ kernel, the products 1.2 us where their
// instructions need 0.8 at 1.9 GHz; the tensor core is 56% (dQ) and 70% (dK, dV)
// active over a whole launch, the rest is the start and end of each CTA (~6 us,
// one CTA per SM) and waits between products.  Issue matters: from a branch of a
// single thread an MMA takes ~48 cycles to issue, from a converged warp with
// one elected lane <= 32, and a tile has 24 to 42 of them.
//
// dq_kernel also writes, for dkv_kernel, -L (in units of the raw score) and -D of
// each query as three bf16 parts in an operand tile: dkv_kernel adds them with one
// more K = 16 step of S^T and dP^T (against constant selecting rows), so its
// threads, which own keys, need no per-query values.  (Reading them from shared
// memory took ~1300 wavefronts a tile.)  A row that sees nothing
// has -1e30, which makes P = 0.
//
// D comes from the O that the forward wrote, in bf16, for rows of more than one key
// tile; it is rowsum(P dP), without that rounding, for rows that lie in one.
//
// P and dS are rounded to bf16 as operands of the tensor core (relative 2^-8
// at most each, as P in the forward); every sum is fp32.  Every mbarrier wait is
// bounded; one that runs out sets the error word, all roles leave their
// loops, loads and MMAs in flight are drained and TMEM is freed.
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

struct BwdMaps {
    CUtensorMap q, k, v, d;       // 64-column boxes, 128-byte swizzle (d: dO)
    CUtensorMap qt, kt, vt, dt;   // 16-column tails, 32-byte swizzle
    CUtensorMap gq, gk, gv;       // the gradients, likewise
    CUtensorMap gqt, gkt, gvt;
};

struct BwdArgs {
    const int *q_lens, *k_lens;
    int nq, nk, hd, heads, group, causal_block;
    float scale, scale_log2;      // 1 / sqrt(hd), log2(e) / sqrt(hd)
    const __nv_bfloat16 *O, *dO;
    const float* lse;
    uint4* stats;                 // [batch * heads][query tiles] operands of kStatBytes
    __nv_bfloat16 *dQ, *dK, *dV;
    int ldo, lddo, lddq, lddk, lddv;
    // CTAs that share one gradient tile, each a part of its products' other
    // axis, and the fp32 parts [splits][rows][heads * hd] that they leave
    int splits_q, splits_k;
    float *part_q, *part_k, *part_v;
    int* err;
};

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

struct BwdBars {
    uint32_t a_full, raw0, raw1, s_full, drain2, d_full, e0, e1, done, drain, s_read, d_read, staged, full, empty;
};

template <int SLOTS>
__device__ __forceinline__ BwdBars bwd_bars(uint32_t b) {
    return {b, b + 8, b + 16, b + 24, b + 32, b + 40, b + 48, b + 56, b + 64, b + 72, b + 80, b + 88,
            b + 96, b + 104, b + 104 + 8 * SLOTS};
}

template <int SLOTS>
__device__ __forceinline__ void bwd_init(const BwdBars& m, int done, int readers) {
    mbar_init(m.a_full, 1);
    mbar_init(m.raw0, 1);
    mbar_init(m.raw1, 1);
    mbar_init(m.s_full, 1);
    mbar_init(m.d_full, 1);
    mbar_init(m.e0, 4 * kGroups);
    mbar_init(m.e1, 4 * kGroups);
    mbar_init(m.s_read, 4 * kGroups);
    mbar_init(m.d_read, 4 * kGroups);
    mbar_init(m.staged, 4 * kGroups);
    mbar_init(m.done, done);
    mbar_init(m.drain, 1);
    mbar_init(m.drain2, 1);
    for (int i = 0; i < SLOTS; ++i) {
        mbar_init(m.full + 8 * i, 1);
        mbar_init(m.empty + 8 * i, readers);
    }
    fence_mbar_init();
}

// Loads in flight, for the drain: slots and the parity of each.
struct InFlight {
    uint32_t on = 0, par = 0;
    __device__ void add(Slot s) {
        on |= 1u << s.s;
        par = (par & ~(1u << s.s)) | (s.ph << s.s);
    }
    template <int SLOTS>
    __device__ void drain(uint32_t full) const {
        for (int i = 0; i < SLOTS; ++i)
            if (on & (1u << i)) mbar_wait(full + 8 * i, (par >> i) & 1u, nullptr);
    }
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

// One thread's part of an accumulator row (32-column chunks first, first +
// step, ...) times `scale`: in fp32 to `part` if that is set, else in bf16 to the
// tile in shared memory that TMA then stores (rows and columns past the tensor
// are not written).  `none`: zeros instead, for a row without a visible pair; its
// accumulator is 0, or NaN where the tile's other rows met an infinity.
template <int NB, bool TAIL>
__device__ __forceinline__ void store_row(uint32_t t, uint8_t* tile, int row, float* part, int hd, bool live, bool none, float scale,
                                          int first, int step) {
#pragma unroll 1
    for (int c = first; c < (AttnTile<NB, TAIL>::HDP + 31) / 32; c += step) {
        uint32_t r[32], w[16];
        tmem_ld_32x32b_x32(t + c * 32, r);
        tmem_wait_ld_r(r);
        if (none) {
#pragma unroll
            for (int k = 0; k < 32; ++k) r[k] = 0;
        }
        if (part) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (live && c * 32 + 4 * k < hd)
                    *reinterpret_cast<float4*>(part + c * 32 + 4 * k) =
                        make_float4(__uint_as_float(r[4 * k]) * scale, __uint_as_float(r[4 * k + 1]) * scale,
                                    __uint_as_float(r[4 * k + 2]) * scale, __uint_as_float(r[4 * k + 3]) * scale);
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = pack_bf16x2(__uint_as_float(r[2 * k]) * scale, __uint_as_float(r[2 * k + 1]) * scale);
            put_row<NB, TAIL>(tile, row, c, w);
        }
    }
}

// Zeros to rows [0, n) x hd of a strided bf16 matrix, by the whole CTA.
__device__ __forceinline__ void zero_out(__nv_bfloat16* out, int ld, int n, int hd) {
    const int c8 = hd / 8;
    for (int i = threadIdx.x; i < n * c8; i += kThreadsB)
        reinterpret_cast<uint4*>(out + static_cast<size_t>(i / c8) * ld)[i % c8] = make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ void zero_out(float* out, int ld, int n, int hd) {
    const int c4 = hd / 4;
    for (int i = threadIdx.x; i < n * c4; i += kThreadsB)
        reinterpret_cast<float4*>(out + static_cast<size_t>(i / c4) * ld)[i % c4] = make_float4(0.f, 0.f, 0.f, 0.f);
}

__device__ __forceinline__ float dot8(uint4 a, uint4 b) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]));
        const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&y[i]));
        t += u.x * v.x + u.y * v.y;
    }
    return t;
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

// ------------------------------------------------------------------ dQ
// TMEM: S [0, 128), dP [128, 256), dS [256, 320), dQ [384, 512).  Issue order
// S_0 dP_0 | S_1 dP_1 dQ_0 | S_2 dP_2 dQ_1 | ...: S_{j+1} goes once S_j is read
// and dP_{j+1} once dP_j is, both before the elementwise warps have formed dS_j,
// so that they find their next operands ready.  Two warps issue, S and dP one, dQ
// the other: each waits for its own barriers while the other's products run (a
// tile at head dim 64: 0.74 us, against 0.84 with one).
template <int NB, bool TAIL>
__global__ void __launch_bounds__(kThreadsB, 1)
    dq_kernel(const __grid_constant__ BwdMaps maps, const __grid_constant__ BwdArgs g) {
    using P = BwdPlan<NB, TAIL, true>;
    using T = AttnTile<NB, TAIL>;
    const auto first = [](int i) { return slot_of<P::SLOTS, P::SHARED, false>(i); };
    const auto second = [](int i) { return slot_of<P::SLOTS, P::SHARED, true>(i); };
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(smem);
    const BwdBars m = bwd_bars<P::SLOTS>(sb + P::BAR_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + P::TMEM_SLOT_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P::ABORT_OFF);
    if (smem - smem_raw + P::USED > P::BYTES) {       // the base of dynamic shared memory is 1 KB aligned
        if (threadIdx.x == 0 && g.err) atomicExch(g.err, 1);
        return;
    }
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // with a causal mask the last query tiles see the most keys: first
    const int qtiles = gridDim.x / g.splits_q, split = blockIdx.x % g.splits_q;
    const int qt = qtiles - 1 - blockIdx.x / g.splits_q, h = blockIdx.y, b = blockIdx.z;
    const int row0 = qt * kTile, off = g.nk - g.nq;

    pdl_wait();
    const int qlen = seq_len(g.q_lens, b, g.nq), klen = seq_len(g.k_lens, b, g.nk);
    const int last = min(row0 + kTile, qlen) - 1;
    const int all = last < row0 ? 0 : (key_end(last, off, g.causal_block, klen) + kTile - 1) / kTile;
    // key tiles [j0, j0 + n) are this CTA's
    const int per = (all + g.splits_q - 1) / g.splits_q, j0 = split * per, n = min(all, j0 + per) - j0;
    uint4* stat = split ? nullptr : g.stats + ((static_cast<size_t>(b) * g.heads + h) * qtiles + qt) * (kStatBytes / 16);
    __nv_bfloat16* dq0 = g.dQ + (static_cast<size_t>(b) * g.nq + row0) * g.lddq + h * g.hd;
    const int ldp = g.heads * g.hd;
    float* part0 = g.splits_q == 1 ? nullptr
                                   : g.part_q + ((static_cast<size_t>(split) * gridDim.z + b) * g.nq + row0) * ldp + h * g.hd;
    if (n <= 0) {
        if (stat && threadIdx.x < kTile) write_stat(stat, threadIdx.x, kNothing, 0.f);
        if (part0) zero_out(part0, ldp, min(kTile, g.nq - row0), g.hd);
        else zero_out(dq0, g.lddq, min(kTile, g.nq - row0), g.hd);
        return;
    }

    // D = rowsum(dO O): LP lanes read one row's 16-byte pieces side by side, eight
    // rows a warp, all loads at once: they overlap the set-up.  (One row a lane
    // touches 32 rows a load instruction: set-up took 14000 cycles with 40 x 128
    // columns a row, against 6200.)  Rows that lie in one key tile need neither: their
    // D is rowsum(P dP), formed below without the rounding of O.
    const bool one_tile = all == 1;
    constexpr int LP = NB == 1 && !TAIL ? 8 : 16, RP = 32 / LP;
    float* row_d = reinterpret_cast<float*>(smem + P::SEL_OFF);
    uint4 o[8 / RP], d[8 / RP];
    float l = -INFINITY;
    if (warp >= 4) {
#pragma unroll
        for (int u = 0; u < 8 / RP; ++u) {
            const int row = (warp - 4) * 8 + u * RP + lane / LP, c = lane % LP;
            const bool in = !one_tile && row0 + row < qlen && c < g.hd / 8;
            const size_t r = static_cast<size_t>(b) * g.nq + row0 + row;
            o[u] = in ? reinterpret_cast<const uint4*>(g.O + r * g.ldo + h * g.hd)[c] : make_uint4(0, 0, 0, 0);
            d[u] = in ? reinterpret_cast<const uint4*>(g.dO + r * g.lddo + h * g.hd)[c] : make_uint4(0, 0, 0, 0);
        }
        const int i = row0 + (warp & 3) * 32 + lane;
        if (i < qlen) l = g.lse[(static_cast<size_t>(b) * g.heads + h) * g.nq + i];
    }
    if (threadIdx.x == 0) {
        bwd_init<P::SLOTS>(m, 1, 1);
        *abort_flag = 0;
        // this thread is also the one that loads: the first tiles need not wait
        // for the rest of the set-up
        mbar_arrive_expect_tx(m.a_full, 2 * P::TILE);
        load_tile<NB, TAIL>(sb + P::A0_OFF, &maps.q, &maps.qt, h, row0, b, m.a_full);
        load_tile<NB, TAIL>(sb + P::A1_OFF, &maps.d, &maps.dt, h, row0, b, m.a_full);
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
        tma_prefetch_desc(&maps.d);
    }
    if (warp == 1) {
        tmem_alloc(sb + P::TMEM_SLOT_OFF, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
    // only now: the next kernel's CTAs may allocate TMEM before they wait for
    // this grid, so every CTA of this one must hold its own first
    pdl_launch_dependents();
    auto fail = [&]() {
        *abort_flag = 1;
        if (g.err) atomicExch(g.err, 1);
    };
    // keys behind k_lens end inside the last tile: its K rows there become zero
    // before the MMAs see it (its loads complete on raw0 instead)
    const int fix = klen < g.nk && klen < (j0 + n) * kTile ? klen - (j0 + n - 1) * kTile : kTile;

    if (warp == 0) {
        // ---------------- TMA: K and V
        bool ok = true;
        InFlight in;
        if (lane == 0) {
            const int hk = h / g.group;
            for (int j = 0; j < n; ++j) {
                const Slot k = first(j), v = second(j);
                if (!mbar_wait(m.empty + 8 * k.s, k.ph ^ 1, abort_flag)) { ok = false; break; }
                const bool raw = fix < kTile && j == n - 1;
                const uint32_t full = raw ? m.raw0 : m.full + 8 * k.s;
                mbar_arrive_expect_tx(full, P::TILE);
                load_tile<NB, TAIL>(sb + P::R_OFF + k.s * P::TILE, &maps.k, &maps.kt, hk, (j0 + j) * kTile, b, full);
                if (!raw) in.add(k);
                if (!mbar_wait(m.empty + 8 * v.s, v.ph ^ 1, abort_flag)) {
                    ok = false;
                    if (raw) mbar_wait(m.raw0, 0, nullptr);
                    break;
                }
                mbar_arrive_expect_tx(m.full + 8 * v.s, P::TILE);
                load_tile<NB, TAIL>(sb + P::R_OFF + v.s * P::TILE, &maps.v, &maps.vt, hk, (j0 + j) * kTile, b, m.full + 8 * v.s);
                in.add(v);
            }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (ok && fix < kTile) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(m.raw0, 0, nullptr));
            if (ok) {
                const int st = first(n - 1).s;
                zero_rows<NB, TAIL>(smem + P::R_OFF + st * P::TILE, fix, lane, 32);
                __syncwarp();
                if (lane == 0) mbar_arrive(m.full + 8 * st);
            }
        }
        if (lane == 0) {
            if (!ok) fail();
            if (*abort_flag) {
                mbar_wait(m.a_full, 0, nullptr);
                in.drain<P::SLOTS>(m.full);
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer of S and dP: the warp waits, one lane issues
        const bool one = elect_one();
        const uint64_t q = sw128_kmajor_desc(sb + P::A0_OFF), qtl = sw32_desc(sb + P::A0_OFF + NB * T::BLK);
        const uint64_t d = sw128_kmajor_desc(sb + P::A1_OFF), dtl = sw32_desc(sb + P::A1_OFF + NB * T::BLK);
        const uint64_t k = sw128_kmajor_desc(sb + P::R_OFF);
        const uint64_t ktl = sw32_desc(sb + P::R_OFF + NB * T::BLK);
        const uint64_t v = sw128_kmajor_desc(sb + P::R_OFF), vtl = sw32_desc(sb + P::R_OFF + NB * T::BLK);
        auto issue_s = [&](int j) -> bool {
            const Slot t = first(j);
            if (!warp_wait(m.full + 8 * t.s, t.ph, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (t.s * P::TILE) >> 4;
            if (one) {
                mma_scores<NB, TAIL>(tmem, q, qtl, k + so, ktl + so);
                tc_commit(m.s_full);
            }
            __syncwarp();
            return true;
        };
        auto issue_dp = [&](int j) -> bool {
            const Slot t = second(j);
            if (!warp_wait(m.full + 8 * t.s, t.ph, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (t.s * P::TILE) >> 4;
            if (one) {
                mma_scores<NB, TAIL>(tmem + 128, d, dtl, v + so, vtl + so);
                tc_commit(m.d_full);
                tc_commit(m.empty + 8 * t.s);
            }
            __syncwarp();
            return true;
        };
        bool ok = warp_wait(m.a_full, 0, abort_flag) && issue_s(0) && issue_dp(0);
        for (int j = 1; ok && j < n; ++j)
            ok = warp_wait(m.s_read, (j - 1) & 1, abort_flag) && issue_s(j) && warp_wait(m.d_read, (j - 1) & 1, abort_flag) && issue_dp(j);
        end_issue(one, ok, m.drain, abort_flag, fail);
    } else if (warp == 2) {
        // ---------------- MMA issuer of dQ
        const bool one = elect_one();
        const uint64_t k = sw128_mnmajor_desc(sb + P::R_OFF, T::BLK), ktl = sw32_desc(sb + P::R_OFF + NB * T::BLK);
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const Slot t = first(j);
            if (!warp_wait(m.full + 8 * t.s, t.ph, abort_flag) || !warp_wait(m.e0, j & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t so = (t.s * P::TILE) >> 4;
            if (one) {
                mma_accumulate<NB, TAIL, kCols / 2>(tmem + 384, tmem + 256, k + so, ktl + so, j == 0);
                tc_commit(m.empty + 8 * t.s);
                if (j + 1 == n) tc_commit(m.done);
            }
            __syncwarp();
        }
        end_issue(one, ok, m.drain2, abort_flag, fail);
    } else if (warp >= 4) {
        // ---------------- elementwise: thread = query row, a quarter of the columns
        const int e = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;    // group, TMEM lane
        const int i = row0 + row;
        const int end = i < qlen ? key_end(i, off, g.causal_block, klen) : 0;
#pragma unroll
        for (int u = 0; u < 8 / RP; ++u) {
            float t = dot8(o[u], d[u]);
#pragma unroll
            for (int x = LP / 2; x > 0; x >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, x);
            if (lane % LP == 0) row_d[(warp - 4) * 8 + u * RP + lane / LP] = t;
        }
        // every elementwise warp gets here: no wait comes before
        asm volatile("bar.sync 1, %0;" ::"n"(kThreadsB - 128) : "memory");
        const float l2 = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;   // L in units of log2
        // -L in units of the raw score
        auto write_stats = [&](float delta) {
            if (stat && e == 0) write_stat(stat, row, l2 == INFINITY ? kNothing : -l2 / g.scale_log2, -delta);
        };
        if (!one_tile) write_stats(row_d[row]);
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint64_t scale2 = f32x2(g.scale_log2, g.scale_log2), neg_l2 = f32x2(-l2, -l2);
        uint64_t neg_d = f32x2(-row_d[row], -row_d[row]);
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            if (!warp_wait(m.s_full, j & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            uint32_t r[32];
            tmem_ld_32x32b_x32(tl + kCols * e, r);
            tmem_wait_ld_r(r);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(m.s_read);
            float p[32];
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
                f32x2_split(fma_f32x2(f32x2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), scale2, neg_l2), p[c], p[c + 1]);
                p[c] = ex2_approx(p[c]);
                p[c + 1] = ex2_approx(p[c + 1]);
            }
            if (!warp_wait(m.d_full, j & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            tmem_ld_32x32b_x32(tl + 128 + kCols * e, r);
            tmem_wait_ld_r(r);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(m.d_read);
            const int see = end - (j0 + j) * kTile - kCols * e;     // columns that this row sees
            if (one_tile) {
                // D = rowsum(P dP), the four quarters in their order: with few keys
                // dP - D is small against D, and an O of 8 bits shows in it (relative
                // error of dQ with 3 keys 2.35e-3, with D from O 3.2e-3; causal, 2047
                // tokens, 2.39e-3 and 2.50e-3, for 91.0 us instead of 89.0)
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c < see) sum[c % 4] = fmaf(p[c], __uint_as_float(r[c]), sum[c % 4]);
                float t = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                float* parts = row_d + kTile + row;
                parts[kTile * e] = t;
                __syncwarp();
                if (lane == 0) mbar_arrive(m.e1);
                if (!warp_wait(m.e1, 0, abort_flag)) { ok = false; break; }
                t = (parts[0] + parts[kTile]) + (parts[2 * kTile] + parts[3 * kTile]);
                neg_d = f32x2(-t, -t);
                write_stats(t);
            }
#pragma unroll
            for (int c = 0; c < 32; c += 2)
                f32x2_split(mul_f32x2(f32x2(p[c], p[c + 1]), add_f32x2(f32x2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), neg_d)),
                            p[c], p[c + 1]);
            if (see < kCols) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c >= see) p[c] = 0.f;
            }
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) w[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
            // the last reader of dS's columns, dQ_{j-1}, releases its K slot when done
            if (j > 0) {
                const Slot k = first(j - 1);
                if (!warp_wait(m.empty + 8 * k.s, k.ph, abort_flag)) { ok = false; break; }
                tc_fence_after();       // the store stays behind dQ_{j-1}'s reads
            }
            tmem_st_32x32b_x16(tl + 256 + kCols / 2 * e, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(m.e0);
        }
        if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(m.done, 0, abort_flag));
        if (!ok) {
            if (lane == 0) fail();
        } else {
            tc_fence_after();
            // the slots' tiles have all been read: the first one takes the result
            store_row<NB, TAIL>(tl + 384, smem + P::R_OFF, row, part0 ? part0 + static_cast<size_t>(row) * ldp : nullptr, g.hd, i < g.nq,
                                end <= 0, g.scale, e, kGroups);
            if (!part0) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(m.staged);
                if (warp == 4) {
                    ok = warp_wait(m.staged, 0, abort_flag);
                    if (lane == 0) {
                        if (ok) {
                            store_tile<NB, TAIL>(sb + P::R_OFF, &maps.gq, &maps.gqt, h, row0, b);
                            bulk_commit();
                            bulk_wait_all();
                        } else {
                            fail();
                        }
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ dK, dV
// TMEM: S^T [0, 128), dP^T [128, 256), then dV, dK and, where they fit, P^T and
// dS^T; else these take the places of S^T and dP^T, and then dV_i goes before
// S_{i+1} and dK_i before dP_{i+1} in one order of issue.
template <int NB, bool TAIL>
__global__ void __launch_bounds__(kThreadsB, 1)
    dkv_kernel(const __grid_constant__ BwdMaps maps, const __grid_constant__ BwdArgs g) {
    using P = BwdPlan<NB, TAIL, false>;
    using T = AttnTile<NB, TAIL>;
    using M = DkvTmem<T::HDP>;
    const auto first = [](int i) { return slot_of<P::SLOTS, P::SHARED, false>(i); };
    const auto second = [](int i) { return slot_of<P::SLOTS, P::SHARED, true>(i); };
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(smem);
    const BwdBars m = bwd_bars<P::SLOTS>(sb + P::BAR_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + P::TMEM_SLOT_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P::ABORT_OFF);
    if (smem - smem_raw + P::USED > P::BYTES) {       // the base of dynamic shared memory is 1 KB aligned
        if (threadIdx.x == 0 && g.err) atomicExch(g.err, 1);
        return;
    }
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int kt = blockIdx.x / g.splits_k, split = blockIdx.x % g.splits_k, hk = blockIdx.y, b = blockIdx.z;
    const int key0 = kt * kTile, off = g.nk - g.nq;
    const int qtiles = (g.nq + kTile - 1) / kTile;

    // This grid starts while dq_kernel, whose every CTA has waited for what came
    // before, ends: all inputs are there, and only the row statistics, dq_kernel's
    // own, need the wait.  Every CTA waits before it ends, so that whoever waits
    // for this grid has waited for dq_kernel too.  (In a graph, 256 tokens of 4 heads
    // of 64: 10.1 us for the two launches, 11.3 with the wait here; 2 x 16 heads of
    // 72, 1024 tokens: 48.8, 50.4 with it.)
    const int qlen = seq_len(g.q_lens, b, g.nq), klen = seq_len(g.k_lens, b, g.nk);
    // query tiles [t0, t1) of each of the group's heads, one after the other
    const int t0 = max(0, query_begin(key0, off, g.causal_block)) / kTile;
    const int t1 = key0 < klen ? (qlen + kTile - 1) / kTile : 0;
    const int per = max(0, t1 - t0), all = per * g.group;
    // of these `all` steps, [i0, i0 + n) are this CTA's
    const int share = (all + g.splits_k - 1) / g.splits_k, i0 = split * share, n = min(all, i0 + share) - i0;
    __nv_bfloat16* dk0 = g.dK + (static_cast<size_t>(b) * g.nk + key0) * g.lddk + hk * g.hd;
    __nv_bfloat16* dv0 = g.dV + (static_cast<size_t>(b) * g.nk + key0) * g.lddv + hk * g.hd;
    const int ldp = gridDim.y * g.hd;
    const size_t part_at = ((static_cast<size_t>(split) * gridDim.z + b) * g.nk + key0) * ldp + hk * g.hd;
    const bool parts = g.splits_k > 1;
    if (n <= 0) {
        pdl_wait();
        if (parts) {
            zero_out(g.part_k + part_at, ldp, min(kTile, g.nk - key0), g.hd);
            zero_out(g.part_v + part_at, ldp, min(kTile, g.nk - key0), g.hd);
        } else {
            zero_out(dk0, g.lddk, min(kTile, g.nk - key0), g.hd);
            zero_out(dv0, g.lddv, min(kTile, g.nk - key0), g.hd);
        }
        return;
    }

    if (threadIdx.x == 0) {
        bwd_init<P::SLOTS>(m, M::ISSUERS, M::ISSUERS);
        *abort_flag = 0;
        mbar_arrive_expect_tx(m.a_full, 2 * P::TILE);
        load_tile<NB, TAIL>(sb + P::A0_OFF, &maps.k, &maps.kt, hk, key0, b, m.a_full);
        load_tile<NB, TAIL>(sb + P::A1_OFF, &maps.v, &maps.vt, hk, key0, b, m.a_full);
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
        tma_prefetch_desc(&maps.d);
    }
    for (int i = threadIdx.x; i < 2 * kTile; i += kThreadsB) {
        // ones against -L (first operand) or against -D (second)
        uint4* sel = reinterpret_cast<uint4*>(smem + P::SEL_OFF);
        const int x = (i >> 2) & 1;
        sel[2 * i + x] = i < kTile ? make_uint4(0x3F803F80u, 0x3F80u, 0, 0) : make_uint4(0, 0x3F800000u, 0x3F803F80u, 0);
        sel[2 * i + 1 - x] = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == 1) {
        tmem_alloc(sb + P::TMEM_SLOT_OFF, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
    // only now: the next kernel's CTAs may allocate TMEM before they wait for
    // this grid, so every CTA of this one must hold its own first
    pdl_launch_dependents();
    auto fail = [&]() {
        *abort_flag = 1;
        if (g.err) atomicExch(g.err, 1);
    };
    // queries behind q_lens end inside each head's last tile: its Q and dO rows
    // there become zero before the MMAs see it (loads complete on raw0, raw1)
    const int fix = qlen < g.nq && qlen < t1 * kTile ? qlen - (t1 - 1) * kTile : kTile;

    if (warp == 0) {
        // ---------------- TMA: Q with the row statistics, and dO
        bool ok = true;
        InFlight in;
        uint32_t raws = 0;        // tiles fixed so far
        int qt = t0 + i0 % per, h = hk * g.group + i0 / per;
        for (int i = 0; i < n; ++i) {
            const Slot q = first(i), d = second(i);
            const bool raw = fix < kTile && qt == t1 - 1;
            const uint32_t full0 = raw ? m.raw0 : m.full + 8 * q.s, full1 = raw ? m.raw1 : m.full + 8 * d.s;
            if (lane == 0) {
                ok = mbar_wait(m.empty + 8 * q.s, q.ph ^ 1, abort_flag);
                if (ok) {
                    mbar_arrive_expect_tx(full0, P::TILE + kStatBytes);
                    load_tile<NB, TAIL>(sb + P::R_OFF + q.s * P::TILE, &maps.q, &maps.qt, h, qt * kTile, b, full0);
                    if (i == 0) pdl_wait();
                    bulk_load(sb + P::STAT_OFF + i % P::STATS * kStatBytes,
                              g.stats + ((static_cast<size_t>(b) * g.heads + h) * qtiles + qt) * (kStatBytes / 16), kStatBytes, full0);
                    if (!raw) in.add(q);
                    ok = mbar_wait(m.empty + 8 * d.s, d.ph ^ 1, abort_flag);
                    if (ok) {
                        mbar_arrive_expect_tx(full1, P::TILE);
                        load_tile<NB, TAIL>(sb + P::R_OFF + d.s * P::TILE, &maps.d, &maps.dt, h, qt * kTile, b, full1);
                        if (!raw) in.add(d);
                    } else if (raw) {
                        mbar_wait(m.raw0, raws & 1, nullptr);
                    }
                }
            }
            if (raw) {
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                if (!ok) break;
                const bool a0 = mbar_wait(m.raw0, raws & 1, nullptr), a1 = mbar_wait(m.raw1, raws & 1, nullptr);
                ok = __all_sync(0xFFFFFFFFu, a0 && a1);
                if (!ok) break;
                zero_rows<NB, TAIL>(smem + P::R_OFF + q.s * P::TILE, fix, lane, 32);
                zero_rows<NB, TAIL>(smem + P::R_OFF + d.s * P::TILE, fix, lane, 32);
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(m.full + 8 * q.s);
                    mbar_arrive(m.full + 8 * d.s);
                }
                ++raws;
            }
            if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
            if (++qt == t1) {
                qt = t0;
                ++h;
            }
        }
        if (lane == 0) {
            if (!ok) fail();
            if (*abort_flag) {
                mbar_wait(m.a_full, 0, nullptr);
                in.drain<P::SLOTS>(m.full);
            }
        }
    } else if (warp == 1 || (M::ISSUERS == 2 && warp == 2)) {
        // ---------------- MMA issuers: the warp waits, one lane issues
        const bool one = elect_one();
        const uint64_t k = sw128_kmajor_desc(sb + P::A0_OFF), ktl = sw32_desc(sb + P::A0_OFF + NB * T::BLK);
        const uint64_t v = sw128_kmajor_desc(sb + P::A1_OFF), vtl = sw32_desc(sb + P::A1_OFF + NB * T::BLK);
        const uint64_t r = sw128_kmajor_desc(sb + P::R_OFF), rmn = sw128_mnmajor_desc(sb + P::R_OFF, T::BLK);
        const uint64_t rtl = sw32_desc(sb + P::R_OFF + NB * T::BLK);
        const uint64_t sel = sw32_desc(sb + P::SEL_OFF), stat = sw32_desc(sb + P::STAT_OFF);
        constexpr uint32_t id = idesc_bf16_f32(kTile, kTile);
        const auto full = [&](Slot t) { return warp_wait(m.full + 8 * t.s, t.ph, abort_flag); };
        // a slot is free when both products that read it are done: with one
        // issuer the later one's completion says so, with two each says its own
        const auto issue_s = [&](int i) -> bool {
            const Slot t = first(i);
            if (!full(t)) return false;
            tc_fence_after();
            const uint32_t so = (t.s * P::TILE) >> 4;
            if (one) {
                mma_scores<NB, TAIL>(tmem, k, ktl, r + so, rtl + so);
                tc_mma_f16(tmem, sel, stat + ((i % P::STATS * kStatBytes) >> 4), id, 1u);
                tc_commit(m.s_full);
                if (M::ISSUERS == 2) tc_commit(m.empty + 8 * t.s);
            }
            __syncwarp();
            return true;
        };
        const auto issue_dp = [&](int i) -> bool {
            const Slot t = second(i);
            // the statistics came with Q_i; one issuer has waited for it
            if ((M::ISSUERS == 2 && !full(first(i))) || !full(t)) return false;
            tc_fence_after();
            const uint32_t so = (t.s * P::TILE) >> 4;
            if (one) {
                mma_scores<NB, TAIL>(tmem + 128, v, vtl, r + so, rtl + so);
                tc_mma_f16(tmem + 128, sel + (kStatBytes >> 4), stat + ((i % P::STATS * kStatBytes) >> 4), id, 1u);
                tc_commit(m.d_full);
                if (M::ISSUERS == 2) tc_commit(m.empty + 8 * t.s);
            }
            __syncwarp();
            return true;
        };
        const auto issue_dv = [&](int i) -> bool {
            const Slot t = second(i);
            if (!full(t) || !warp_wait(m.e0, i & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (t.s * P::TILE) >> 4;
            if (one) {
                mma_accumulate<NB, TAIL, M::P_APART ? kCols / 2 : kCols>(tmem + M::DV_COL, tmem + M::P_COL, rmn + so, rtl + so, i == 0);
                tc_commit(m.empty + 8 * t.s);
                if (i + 1 == n) tc_commit(m.done);
            }
            __syncwarp();
            return true;
        };
        const auto issue_dk = [&](int i) -> bool {
            const Slot t = first(i);
            if (!warp_wait(m.e1, i & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (t.s * P::TILE) >> 4;
            if (one) {
                mma_accumulate<NB, TAIL, M::DS_APART ? kCols / 2 : kCols>(tmem + M::DK_COL, tmem + M::DS_COL, rmn + so, rtl + so, i == 0);
                tc_commit(m.empty + 8 * t.s);
                if (i + 1 == n) tc_commit(m.done);
            }
            __syncwarp();
            return true;
        };
        bool ok = warp_wait(m.a_full, 0, abort_flag);
        if constexpr (M::ISSUERS == 1) {
            // written out: through the four calls below a tile takes 6% longer
            ok = ok && issue_s(0) && issue_dp(0);
            for (int i = 0; ok && i < n; ++i) {
                const int st = first(i).s, sd = second(i).s;
                const uint32_t so = (st * P::TILE) >> 4, sdo = (sd * P::TILE) >> 4;
                const bool more = i + 1 < n;
                if (!warp_wait(m.e0, i & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                if (one) {
                    mma_accumulate<NB, TAIL, kCols>(tmem + M::DV_COL, tmem + M::P_COL, rmn + sdo, rtl + sdo, i == 0);
                    tc_commit(m.empty + 8 * sd);
                }
                __syncwarp();
                if (more && !issue_s(i + 1)) { ok = false; break; }
                if (!warp_wait(m.e1, i & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                if (one) {
                    mma_accumulate<NB, TAIL, kCols>(tmem + M::DK_COL, tmem + M::DS_COL, rmn + so, rtl + so, i == 0);
                    tc_commit(m.empty + 8 * st);
                }
                __syncwarp();
                if (more && !issue_dp(i + 1)) { ok = false; break; }
            }
            if (one && ok) tc_commit(m.done);
        } else if (warp == 1) {
            // S_{i+1} takes S_i's place once that is read; where P_i lies there, after dV_i
            ok = ok && issue_s(0);
            for (int i = 0; ok && i < n; ++i) {
                const bool more = i + 1 < n;
                if (M::P_APART && more) ok = warp_wait(m.s_read, i & 1, abort_flag) && issue_s(i + 1);
                ok = ok && issue_dv(i);
                if (!M::P_APART && more) ok = ok && issue_s(i + 1);
            }
        } else {
            // likewise dP_{i+1}, dS_i and dK_i
            ok = ok && issue_dp(0);
            for (int i = 0; ok && i < n; ++i) {
                const bool more = i + 1 < n;
                if (M::DS_APART && more) ok = warp_wait(m.d_read, i & 1, abort_flag) && issue_dp(i + 1);
                ok = ok && issue_dk(i);
                if (!M::DS_APART && more) ok = ok && issue_dp(i + 1);
            }
        }
        end_issue(one, ok, warp == 1 ? m.drain : m.drain2, abort_flag, fail);
    } else if (warp >= 4) {
        // ---------------- elementwise: thread = key, a quarter of the query columns
        const int e = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;    // group, TMEM lane
        const int key = key0 + row;
        const int begin = key < klen ? query_begin(key, off, g.causal_block) : 1 << 30;   // queries that see it: [begin, qlen)
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t ts = tl + kCols * e;
        const uint64_t scale2 = f32x2(g.scale_log2, g.scale_log2);
        bool ok = true;
        int qt = t0 + i0 % per;
        for (int i = 0; i < n; ++i) {
            const int lo = begin - (qt * kTile + kCols * e), hi = qlen - (qt * kTile + kCols * e);
            const bool cut = __any_sync(0xFFFFFFFFu, lo > 0 || hi < kCols);
            if (++qt == t1) qt = t0;
            if (!warp_wait(m.s_full, i & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            uint32_t r[32], w[16];
            float p[32];
            tmem_ld_32x32b_x32(ts, r);
            tmem_wait_ld_r(r);
            if constexpr (M::P_APART) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(m.s_read);
            }
            // the product holds S - L
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
                f32x2_split(mul_f32x2(f32x2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), scale2), p[c], p[c + 1]);
                p[c] = ex2_approx(p[c]);
                p[c + 1] = ex2_approx(p[c + 1]);
            }
            if (cut) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c < lo || c >= hi) p[c] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) w[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
            if constexpr (M::P_APART) {
                // the last reader of its columns, dV_{i-1}, releases its dO slot when done
                const Slot t = second(i - 1);
                if (i > 0 && !warp_wait(m.empty + 8 * t.s, t.ph, abort_flag)) { ok = false; break; }
                tc_fence_after();
                tmem_st_32x32b_x16(tl + M::P_COL + kCols / 2 * e, w);
            } else {
                tmem_st_32x32b_x16(ts, w);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(m.e0);
            if (!warp_wait(m.d_full, i & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            tmem_ld_32x32b_x32(ts + 128, r);
            tmem_wait_ld_r(r);
            if constexpr (M::DS_APART) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(m.d_read);
            }
            // this one dP - D
#pragma unroll
            for (int c = 0; c < 32; c += 2)
                f32x2_split(mul_f32x2(f32x2(p[c], p[c + 1]), f32x2(__uint_as_float(r[c]), __uint_as_float(r[c + 1]))), p[c], p[c + 1]);
            if (cut) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c < lo || c >= hi) p[c] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) w[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
            if constexpr (M::DS_APART) {
                // the last reader of its columns, dK_{i-1}, releases its Q slot when done
                const Slot t = first(i - 1);
                if (i > 0 && !warp_wait(m.empty + 8 * t.s, t.ph, abort_flag)) { ok = false; break; }
                tc_fence_after();
                tmem_st_32x32b_x16(tl + M::DS_COL + kCols / 2 * e, w);
            } else {
                tmem_st_32x32b_x16(ts + 128, w);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(m.e1);
        }
        if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(m.done, 0, abort_flag));
        if (!ok) {
            if (lane == 0) fail();
        } else {
            tc_fence_after();
            // even groups bring dV, odd ones dK, into the first two slots
            const bool k = e & 1;
            float* part = parts ? (k ? g.part_k : g.part_v) + part_at + static_cast<size_t>(row) * ldp : nullptr;
            store_row<NB, TAIL>(tl + (k ? M::DK_COL : M::DV_COL), smem + P::R_OFF + (k ? P::TILE : 0), row, part, g.hd, key < g.nk,
                                begin >= qlen, k ? g.scale : 1.f, e >> 1, kGroups / 2);
            if (!parts) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(m.staged);
                if (warp == 4) {
                    ok = warp_wait(m.staged, 0, abort_flag);
                    if (lane == 0) {
                        if (ok) {
                            store_tile<NB, TAIL>(sb + P::R_OFF, &maps.gv, &maps.gvt, hk, key0, b);
                            store_tile<NB, TAIL>(sb + P::R_OFF + P::TILE, &maps.gk, &maps.gkt, hk, key0, b);
                            bulk_commit();
                            bulk_wait_all();
                        } else {
                            fail();
                        }
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Adds the parts of a split gradient in order and rounds once.  One thread
// eight columns; bound by reading the parts.
struct JoinOne {
    const float* part;
    __nv_bfloat16* out;
    int splits, ld, c8;          // c8: pieces of 8 columns a row
    long long rows;
};
struct JoinArgs {
    JoinOne one[3];
};

__global__ void __launch_bounds__(256) bwd_join_kernel(const __grid_constant__ JoinArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        const JoinOne& j = a.one[t];
        const long long n = j.rows * j.c8;
        if (i >= n) {
            i -= n;
            continue;
        }
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        const float4* p = reinterpret_cast<const float4*>(j.part) + 2 * i;
#pragma unroll 4
        for (int k = 0; k < j.splits; ++k, p += 2 * n) {
            const float4 u = p[0], v = p[1];
            x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
            y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
        }
        const long long row = i / j.c8;
        reinterpret_cast<uint4*>(j.out + row * j.ld)[i - row * j.c8] =
            make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
        return;
    }
}

// Splits and workspace, from the sizes alone.
//   dQ: query tiles that do not fill the SMs share their keys, four key tiles
//     or more to a CTA.
//   dK, dV: likewise over the group's query tiles; with a causal mask also
//     where the longest CTA (all query tiles) has more than an SM's share of
//     the whole (3 sequences of 2047 tokens, 16 heads over 4: 109 us unsplit, 96 in two).
struct BwdSplit {
    int q, k;
    size_t part_q, part_k, part_v, total;      // byte offsets
};

BwdSplit bwd_split(const dlo_attn& a) {
    const long long qt = (a.nq + kTile - 1) / kTile, kt = (a.nk + kTile - 1) / kTile, group = a.heads / a.kv_heads;
    const long long nq = qt * a.heads * a.batch, nk = kt * a.kv_heads * a.batch, steps = qt * group;
    const auto fill = [](long long ctas, long long work) {
        long long s = kGb300Sms / ctas;
        if (s > work / 4) s = work / 4;
        return s < 1 ? 1ll : s > 64 ? 64ll : s;
    };
    BwdSplit b;
    long long sq = fill(nq, kt), sk = fill(nk, steps);
    if (a.causal_block > 0) {
        // about half of all steps are done
        const long long mean = nk * steps / 2 / kGb300Sms + 1;
        long long s = (steps + mean - 1) / mean;
        if (s > steps / 8) s = steps / 8;
        if (s > sk) sk = s > 64 ? 64 : s;
    }
    b.q = static_cast<int>(sq);
    b.k = static_cast<int>(sk);
    const size_t rq = static_cast<size_t>(a.batch) * a.nq * a.heads * a.head_dim * sizeof(float);
    const size_t rk = static_cast<size_t>(a.batch) * a.nk * a.kv_heads * a.head_dim * sizeof(float);
    b.part_q = static_cast<size_t>(a.batch) * a.heads * qt * kStatBytes;
    b.part_k = b.part_q + (b.q > 1 ? b.q * rq : 0);
    b.part_v = b.part_k + (b.k > 1 ? b.k * rk : 0);
    b.total = b.part_v + (b.k > 1 ? b.k * rk : 0);
    return b;
}

template <int NB, bool TAIL>
cudaError_t run_bwd(const BwdMaps& maps, const BwdArgs& g, int batch, int kv_heads, cudaStream_t s,
                    unsigned long long* launches) {
    using PQ = BwdPlan<NB, TAIL, true>;
    using PK = BwdPlan<NB, TAIL, false>;
    static unsigned long long set[2] = {0, 0};
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(&dq_kernel<NB, TAIL>), PQ::BYTES, &set[0]); e != cudaSuccess) return e;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(&dkv_kernel<NB, TAIL>), PK::BYTES, &set[1]); e != cudaSuccess) return e;
    cudaError_t e = launch_k(dq_kernel<NB, TAIL>, dim3((g.nq + kTile - 1) / kTile * g.splits_q, g.heads, batch), kThreadsB, PQ::BYTES, s, maps, g);
    ++*launches;
    if (e != cudaSuccess) return e;
    e = launch_k(dkv_kernel<NB, TAIL>, dim3((g.nk + kTile - 1) / kTile * g.splits_k, kv_heads, batch), kThreadsB, PK::BYTES, s, maps, g);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t attention_bwd_workspace(const dlo_attn& a) {
    return bwd_split(a).total;
}

cudaError_t launch_attention_bwd(const dlo_attn& a, const void* Q, const void* K, const void* V, const void* O,
                                 const float* lse, const void* dO, void* dQ, void* dK, void* dV, void* ws, int* err,
                                 cudaStream_t s, unsigned long long* launches) {
    const int hd = a.head_dim;
    BwdArgs g = {};
    g.q_lens = a.q_lens;
    g.k_lens = a.k_lens;
    g.nq = a.nq;
    g.nk = a.nk;
    g.hd = hd;
    g.heads = a.heads;
    g.group = a.heads / a.kv_heads;
    g.causal_block = a.causal_block < a.nk ? a.causal_block : a.nk;
    g.scale = 1.f / sqrtf(static_cast<float>(hd));
    g.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(hd));
    g.O = static_cast<const __nv_bfloat16*>(O);
    g.dO = static_cast<const __nv_bfloat16*>(dO);
    g.lse = lse;
    g.stats = static_cast<uint4*>(ws);
    const BwdSplit split = bwd_split(a);
    uint8_t* base = static_cast<uint8_t*>(ws);
    g.splits_q = split.q;
    g.splits_k = split.k;
    g.part_q = reinterpret_cast<float*>(base + split.part_q);
    g.part_k = reinterpret_cast<float*>(base + split.part_k);
    g.part_v = reinterpret_cast<float*>(base + split.part_v);
    g.dQ = static_cast<__nv_bfloat16*>(dQ);
    g.dK = static_cast<__nv_bfloat16*>(dK);
    g.dV = static_cast<__nv_bfloat16*>(dV);
    g.ldo = a.ldo;
    g.lddo = a.lddo;
    g.lddq = a.lddq;
    g.lddk = a.lddk;
    g.lddv = a.lddv;
    g.err = err;
    BwdMaps m;
    const CUtensorMapSwizzle w128 = CU_TENSOR_MAP_SWIZZLE_128B, w32 = CU_TENSOR_MAP_SWIZZLE_32B;
    const bool tail = hd > 64 && hd <= 80;
    auto map = [&](CUtensorMap* main, CUtensorMap* tl, const void* p, int rows, int heads, int ld) {
        if (!make_map4(main, p, a.batch, rows, heads, hd, ld, 64, w128)) return false;
        if (tail) return make_map4(tl, p, a.batch, rows, heads, hd, ld, 16, w32);
        *tl = *main;
        return true;
    };
    if (!map(&m.q, &m.qt, Q, a.nq, a.heads, a.ldq) || !map(&m.k, &m.kt, K, a.nk, a.kv_heads, a.ldk) ||
        !map(&m.v, &m.vt, V, a.nk, a.kv_heads, a.ldv) || !map(&m.d, &m.dt, dO, a.nq, a.heads, a.lddo) ||
        !map(&m.gq, &m.gqt, dQ, a.nq, a.heads, a.lddq) || !map(&m.gk, &m.gkt, dK, a.nk, a.kv_heads, a.lddk) ||
        !map(&m.gv, &m.gvt, dV, a.nk, a.kv_heads, a.lddv))
        return cudaErrorInvalidValue;
    cudaError_t e = hd <= 64 ? run_bwd<1, false>(m, g, a.batch, a.kv_heads, s, launches)
                    : tail   ? run_bwd<1, true>(m, g, a.batch, a.kv_heads, s, launches)
                             : run_bwd<2, false>(m, g, a.batch, a.kv_heads, s, launches);
    if (e != cudaSuccess || (split.q == 1 && split.k == 1)) return e;
    const long long rq = static_cast<long long>(a.batch) * a.nq, rk = static_cast<long long>(a.batch) * a.nk;
    const int cq = a.heads * hd / 8, ck = a.kv_heads * hd / 8;
    const JoinArgs j = {{{g.part_q, g.dQ, split.q, a.lddq, cq, split.q > 1 ? rq : 0},
                         {g.part_k, g.dK, split.k, a.lddk, ck, split.k > 1 ? rk : 0},
                         {g.part_v, g.dV, split.k, a.lddv, ck, split.k > 1 ? rk : 0}}};
    const long long n = j.one[0].rows * cq + 2 * j.one[1].rows * ck;
    e = launch_k(bwd_join_kernel, static_cast<unsigned>((n + 255) / 256), 256, 0, s, j);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dlo
