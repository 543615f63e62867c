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
// thread that owns a TMEM lane (a query row, a key) reads 64 columns of the
// fp32 product and writes their bf16 values over the columns it has read.  The
// B operands of the accumulating products are the tiles already in shared
// memory, read MN-major.  12 warps: 0 TMA, 1 MMA issue, 4..11 elementwise (two
// per 32 TMEM lanes, each half of the 128 columns).  The products of tile j + 1
// that do not wait for the elementwise work of tile j are issued before those
// that do, so the tensor core computes while the elementwise warps run.
//
// dq_kernel also writes, for dkv_kernel, L (in units of log2, +inf where a row
// sees nothing, which makes P = 0) and D, 128 of each per query tile.
//
// P and dS are rounded to bf16 as operands of the tensor core (relative 2^-8
// at most, as P in the forward); every sum is fp32.  Every mbarrier wait is
// bounded; one that runs out sets the error word, all roles leave their
// loops, loads and MMAs in flight are drained and TMEM is freed.
#include "attention.cuh"

namespace dlo {

namespace {

constexpr int kTile = 128;
constexpr int kThreadsB = 384;
constexpr int kStatBytes = 2 * kTile * sizeof(float);   // L and D of one query tile

struct BwdMaps {
    CUtensorMap q, k, v, d;       // 64-column boxes, 128-byte swizzle (d: dO)
    CUtensorMap qt, kt, vt, dt;   // 16-column tails, 32-byte swizzle
};

struct BwdArgs {
    const int *q_lens, *k_lens;
    int nq, nk, hd, heads, group, causal_block;
    float scale, scale_log2;      // 1 / sqrt(hd), log2(e) / sqrt(hd)
    const __nv_bfloat16 *O, *dO;
    const float* lse;
    float* stats;                 // [batch * heads][query tiles][L 128 | D 128]
    __nv_bfloat16 *dQ, *dK, *dV;
    int ldo, lddo, lddq, lddk, lddv;
    int* err;
};

template <int NB, bool TAIL>
struct BwdPlan {
    using T = AttnTile<NB, TAIL>;
    static constexpr int TILE = T::BYTES;
    // two tiles stay (Q and dO, or K and V), two rings move
    static constexpr int STAGES = NB == 2 ? 2 : 3;
    static constexpr int A0_OFF = 0, A1_OFF = TILE;
    static constexpr int R0_OFF = 2 * TILE;
    static constexpr int R1_OFF = R0_OFF + STAGES * TILE;
    static constexpr int STAT_OFF = R1_OFF + STAGES * TILE;
    static constexpr int BAR_OFF = STAT_OFF + STAGES * kStatBytes;
    // a_full, raw0, raw1, s_full[2], d_full, e0, e1, done, drain, then full0, full1, empty0, empty1 of each stage
    static constexpr int NBARS = 10 + 4 * STAGES;
    static constexpr int TMEM_SLOT_OFF = BAR_OFF + NBARS * 8;
    static constexpr int ABORT_OFF = TMEM_SLOT_OFF + 4;
    static constexpr int USED = ABORT_OFF + 4 + 1024;
    // one CTA per SM: it owns all 512 TMEM columns
    static constexpr int BYTES = USED > 118784 ? USED : 118784;
    static_assert(BYTES <= 227 * 1024, "attention backward shared memory plan exceeds 227 KB");
};

struct BwdBars {
    uint32_t a_full, raw0, raw1, s_full, d_full, e0, e1, done, drain, full0, full1, empty0, empty1;
};

template <int STAGES>
__device__ __forceinline__ BwdBars bwd_bars(uint32_t b) {
    return {b, b + 8, b + 16, b + 24, b + 40, b + 48, b + 56, b + 64, b + 72,
            b + 80, b + 80 + 8 * STAGES, b + 80 + 16 * STAGES, b + 80 + 24 * STAGES};
}

template <int STAGES>
__device__ __forceinline__ void bwd_init(const BwdBars& m) {
    mbar_init(m.a_full, 1);
    mbar_init(m.raw0, 1);
    mbar_init(m.raw1, 1);
    mbar_init(m.s_full, 1);
    mbar_init(m.s_full + 8, 1);
    mbar_init(m.d_full, 1);
    mbar_init(m.e0, 8);
    mbar_init(m.e1, 8);
    mbar_init(m.done, 1);
    mbar_init(m.drain, 1);
    for (int i = 0; i < STAGES; ++i) {
        mbar_init(m.full0 + 8 * i, 1);
        mbar_init(m.full1 + 8 * i, 1);
        mbar_init(m.empty0 + 8 * i, 1);
        mbar_init(m.empty1 + 8 * i, 1);
    }
    fence_mbar_init();
}

// Loads of a ring in flight, for the drain: stages and the parity of each.
struct InFlight {
    uint32_t on = 0, par = 0;
    __device__ void add(int st, uint32_t ph) {
        on |= 1u << st;
        par = (par & ~(1u << st)) | (ph << st);
    }
    template <int STAGES>
    __device__ void drain(uint32_t full) const {
        for (int i = 0; i < STAGES; ++i)
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

// 128 x hd += A B: A in TMEM (bf16 pairs: contracted indices 0..63 at a, 64..127
// at a + 64), B a tile of shared memory whose rows are the contracted index.
template <int NB, bool TAIL>
__device__ __forceinline__ void mma_accumulate(uint32_t d, uint32_t a, uint64_t b, uint64_t bt, bool first) {
    constexpr uint32_t id = idesc_bf16_f32(kTile, NB * 64, true);
    constexpr uint32_t idt = idesc_bf16_f32(kTile, 16, true);
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk) {
        const uint32_t ak = a + (kk >> 2) * 64 + (kk & 3) * 8;
        const uint32_t acc = (!first || kk > 0) ? 1u : 0u;
        tc_mma_f16_ts(d, ak, b + ((kk * 2048) >> 4), id, acc);
        if constexpr (TAIL) tc_mma_f16_ts(d + NB * 64, ak, bt + ((kk * 512) >> 4), idt, acc);
    }
}

// One thread's part of an accumulator row (32-column chunks c with c % 2 ==
// half, or all of them) times `scale`, as bf16.
template <int HDP>
__device__ __forceinline__ void store_row(uint32_t t, __nv_bfloat16* out, int hd, bool live, float scale, int first,
                                          int step) {
#pragma unroll 1
    for (int c = first; c < (HDP + 31) / 32; c += step) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(t + c * 32, r);
        tmem_wait_ld_r(r);
        if (!live) continue;
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
            if (c * 32 + 8 * k4 < hd) {
                uint32_t w[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    w[u] = pack_bf16x2(__uint_as_float(r[8 * k4 + 2 * u]) * scale, __uint_as_float(r[8 * k4 + 2 * u + 1]) * scale);
                *reinterpret_cast<uint4*>(out + c * 32 + 8 * k4) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// Zeros to rows [0, n) x hd of a strided bf16 matrix, by the whole CTA.
__device__ __forceinline__ void zero_out(__nv_bfloat16* out, int ld, int n, int hd) {
    const int c8 = hd / 8;
    for (int i = threadIdx.x; i < n * c8; i += kThreadsB)
        reinterpret_cast<uint4*>(out + static_cast<size_t>(i / c8) * ld)[i % c8] = make_uint4(0, 0, 0, 0);
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

// ------------------------------------------------------------------ dQ
// TMEM: S in two buffers [0, 128) and [128, 256), dP [256, 384), dQ [384, 512).
// Issue order S_0 dP_0 | S_1 . dP_1 dQ_0 | S_2 . dP_2 dQ_1 | ... where "." waits
// for dS: dP_{j+1} goes before dQ_j because the elementwise warps wait for it.
template <int NB, bool TAIL>
__global__ void __launch_bounds__(kThreadsB, 1)
    dq_kernel(const __grid_constant__ BwdMaps maps, const __grid_constant__ BwdArgs g) {
    using P = BwdPlan<NB, TAIL>;
    using T = AttnTile<NB, TAIL>;
    constexpr int NS = P::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(smem);
    const BwdBars m = bwd_bars<NS>(sb + P::BAR_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + P::TMEM_SLOT_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P::ABORT_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // with a causal mask the last query tiles see the most keys: first
    const int qt = gridDim.x - 1 - blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int row0 = qt * kTile, off = g.nk - g.nq;

    pdl_wait();
    const int qlen = seq_len(g.q_lens, b, g.nq), klen = seq_len(g.k_lens, b, g.nk);
    const int last = min(row0 + kTile, qlen) - 1;
    const int n = last < row0 ? 0 : (key_end(last, off, g.causal_block, klen) + kTile - 1) / kTile;
    float* stat = g.stats + ((static_cast<size_t>(b) * g.heads + h) * gridDim.x + qt) * 2 * kTile;
    __nv_bfloat16* dq0 = g.dQ + (static_cast<size_t>(b) * g.nq + row0) * g.lddq + h * g.hd;
    if (n <= 0) {
        if (threadIdx.x < kTile) {
            stat[threadIdx.x] = INFINITY;
            stat[kTile + threadIdx.x] = 0.f;
        }
        zero_out(dq0, g.lddq, min(kTile, g.nq - row0), g.hd);
        return;
    }

    if (threadIdx.x == 0) {
        bwd_init<NS>(m);
        *abort_flag = 0;
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
    const uint32_t tmem = *tmem_slot;
    // only now: the next kernel's CTAs may allocate TMEM before they wait for
    // this grid, so every CTA of this one must hold its own first
    pdl_launch_dependents();
    auto fail = [&]() {
        *abort_flag = 1;
        if (g.err) atomicExch(g.err, 1);
    };
    // keys behind k_lens end inside the last tile: its K rows there become zero
    // before the MMAs see it (its loads complete on raw0 instead of full0)
    const int fix = klen < g.nk && klen < n * kTile ? klen - (n - 1) * kTile : kTile;

    if (warp == 0) {
        // ---------------- TMA: ring 0 holds K, ring 1 V
        bool ok = true;
        InFlight f0, f1;
        if (lane == 0) {
            const int hk = h / g.group;
            mbar_arrive_expect_tx(m.a_full, 2 * P::TILE);
            load_tile<NB, TAIL>(sb + P::A0_OFF, &maps.q, &maps.qt, h, row0, b, m.a_full);
            load_tile<NB, TAIL>(sb + P::A1_OFF, &maps.d, &maps.dt, h, row0, b, m.a_full);
            for (int j = 0; j < n; ++j) {
                const int st = j % NS;
                const uint32_t ph = (j / NS) & 1;
                if (!mbar_wait(m.empty0 + 8 * st, ph ^ 1, abort_flag)) { ok = false; break; }
                const bool raw = fix < kTile && j == n - 1;
                const uint32_t full = raw ? m.raw0 : m.full0 + 8 * st;
                mbar_arrive_expect_tx(full, P::TILE);
                load_tile<NB, TAIL>(sb + P::R0_OFF + st * P::TILE, &maps.k, &maps.kt, hk, j * kTile, b, full);
                if (!raw) f0.add(st, ph);
                if (!mbar_wait(m.empty1 + 8 * st, ph ^ 1, abort_flag)) {
                    ok = false;
                    if (raw) mbar_wait(m.raw0, 0, nullptr);
                    break;
                }
                mbar_arrive_expect_tx(m.full1 + 8 * st, P::TILE);
                load_tile<NB, TAIL>(sb + P::R1_OFF + st * P::TILE, &maps.v, &maps.vt, hk, j * kTile, b, m.full1 + 8 * st);
                f1.add(st, ph);
            }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (ok && fix < kTile) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(m.raw0, 0, nullptr));
            if (ok) {
                const int st = (n - 1) % NS;
                zero_rows<NB, TAIL>(smem + P::R0_OFF + st * P::TILE, fix, lane, 32);
                __syncwarp();
                if (lane == 0) mbar_arrive(m.full0 + 8 * st);
            }
        }
        if (lane == 0) {
            if (!ok) fail();
            if (*abort_flag) {
                mbar_wait(m.a_full, 0, nullptr);
                f0.drain<NS>(m.full0);
                f1.drain<NS>(m.full1);
            }
        }
    } else if (warp == 1 && lane == 0) {
        // ---------------- MMA issuer
        const uint64_t q = sw128_kmajor_desc(sb + P::A0_OFF), qtl = sw32_desc(sb + P::A0_OFF + NB * T::BLK);
        const uint64_t d = sw128_kmajor_desc(sb + P::A1_OFF), dtl = sw32_desc(sb + P::A1_OFF + NB * T::BLK);
        const uint64_t k = sw128_kmajor_desc(sb + P::R0_OFF), kmn = sw128_mnmajor_desc(sb + P::R0_OFF, T::BLK);
        const uint64_t ktl = sw32_desc(sb + P::R0_OFF + NB * T::BLK);
        const uint64_t v = sw128_kmajor_desc(sb + P::R1_OFF), vtl = sw32_desc(sb + P::R1_OFF + NB * T::BLK);
        auto issue_s = [&](int j) -> bool {
            const int st = j % NS;
            if (!mbar_wait(m.full0 + 8 * st, (j / NS) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (st * P::TILE) >> 4;
            mma_scores<NB, TAIL>(tmem + (j & 1) * 128, q, qtl, k + so, ktl + so);
            tc_commit(m.s_full + 8 * (j & 1));
            return true;
        };
        auto issue_dp = [&](int j) -> bool {
            const int st = j % NS;
            if (!mbar_wait(m.full1 + 8 * st, (j / NS) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (st * P::TILE) >> 4;
            mma_scores<NB, TAIL>(tmem + 256, d, dtl, v + so, vtl + so);
            tc_commit(m.d_full);
            tc_commit(m.empty1 + 8 * st);
            return true;
        };
        bool ok = mbar_wait(m.a_full, 0, abort_flag) && issue_s(0) && issue_dp(0);
        for (int j = 0; ok && j < n; ++j) {
            // S_{j+1} overwrites dS_{j-1}, which dQ_{j-1}, issued before, has read
            if (j + 1 < n && !issue_s(j + 1)) ok = false;
            if (ok && !mbar_wait(m.e0, j & 1, abort_flag)) ok = false;
            if (!ok) break;
            tc_fence_after();
            if (j + 1 < n && !issue_dp(j + 1)) { ok = false; break; }
            const int st = j % NS;
            const uint32_t so = (st * P::TILE) >> 4;
            mma_accumulate<NB, TAIL>(tmem + 384, tmem + (j & 1) * 128, kmn + so, ktl + so, j == 0);
            tc_commit(m.empty0 + 8 * st);
        }
        if (ok) tc_commit(m.done);
        else fail();
        if (*abort_flag) {
            tc_commit(m.drain);
            mbar_wait(m.drain, 0, nullptr);
        }
    } else if (warp >= 4) {
        // ---------------- elementwise: thread = query row, half of the columns
        const int half = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const int i = row0 + row;
        const bool valid = i < qlen;
        const int end = valid ? key_end(i, off, g.causal_block, klen) : 0;
        // D = rowsum(dO O): each half of the threads adds half of the columns
        float* part = reinterpret_cast<float*>(smem + P::STAT_OFF);
        float delta = 0.f;
        if (valid) {
            const uint4* o = reinterpret_cast<const uint4*>(g.O + (static_cast<size_t>(b) * g.nq + i) * g.ldo + h * g.hd);
            const uint4* e = reinterpret_cast<const uint4*>(g.dO + (static_cast<size_t>(b) * g.nq + i) * g.lddo + h * g.hd);
            for (int c = half; c < g.hd / 8; c += 2) delta += dot8(o[c], e[c]);
        }
        part[half * kTile + row] = delta;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        delta = part[row] + part[kTile + row];
        float l2 = INFINITY;
        if (valid) {
            const float l = g.lse[(static_cast<size_t>(b) * g.heads + h) * g.nq + i];
            if (l != -INFINITY) l2 = l * 1.4426950408889634f;
        }
        if (half == 0) {
            stat[row] = l2;
            stat[kTile + row] = delta;
        }
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 64 * half;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const uint32_t ts = tl + (j & 1) * 128;
            bool got = mbar_wait(m.s_full + 8 * (j & 1), (j >> 1) & 1, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got)) { ok = false; break; }
            tc_fence_after();
            uint32_t r[2][32];
            tmem_ld_32x32b_x32(ts, r[0]);
            tmem_ld_32x32b_x32(ts + 32, r[1]);
            tmem_wait_ld_r(r[0]);
            tmem_wait_ld_r(r[1]);
            float p[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) p[c] = ex2_approx(fmaf(__uint_as_float(r[c >> 5][c & 31]), g.scale_log2, -l2));
            got = mbar_wait(m.d_full, j & 1, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got)) { ok = false; break; }
            tc_fence_after();
            tmem_ld_32x32b_x32(tl + 256, r[0]);
            tmem_ld_32x32b_x32(tl + 256 + 32, r[1]);
            tmem_wait_ld_r(r[0]);
            tmem_wait_ld_r(r[1]);
#pragma unroll
            for (int c = 0; c < 64; ++c) p[c] *= __uint_as_float(r[c >> 5][c & 31]) - delta;
            const int see = end - j * kTile - 64 * half;     // columns that this row sees
            if (see < 64) {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (c >= see) p[c] = 0.f;
            }
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) w[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
            tmem_st_32x32b_x32(ts, w);
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
            store_row<T::HDP>(tl - 64 * half + 384, dq0 + static_cast<size_t>(row) * g.lddq, g.hd, i < g.nq, g.scale, half, 2);
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
// TMEM: S^T [0, 128), dP^T [128, 256), dV [256, 384), dK [384, 512); P^T and
// dS^T take the places of S^T and dP^T.  Issue order S_0 dP_0 | . dV_0 S_1 . dK_0
// dP_1 | . dV_1 S_2 . dK_1 dP_2 | ...: dV_i and S_{i+1} run while the elementwise
// warps form dS_i, dK_i and dP_{i+1} while they form P_{i+1}.
template <int NB, bool TAIL>
__global__ void __launch_bounds__(kThreadsB, 1)
    dkv_kernel(const __grid_constant__ BwdMaps maps, const __grid_constant__ BwdArgs g) {
    using P = BwdPlan<NB, TAIL>;
    using T = AttnTile<NB, TAIL>;
    constexpr int NS = P::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(smem);
    const BwdBars m = bwd_bars<NS>(sb + P::BAR_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + P::TMEM_SLOT_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P::ABORT_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kt = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
    const int key0 = kt * kTile, off = g.nk - g.nq;
    const int qtiles = (g.nq + kTile - 1) / kTile;

    pdl_wait();
    const int qlen = seq_len(g.q_lens, b, g.nq), klen = seq_len(g.k_lens, b, g.nk);
    // query tiles [t0, t1) of each of the group's heads, one after the other
    const int t0 = max(0, query_begin(key0, off, g.causal_block)) / kTile;
    const int t1 = key0 < klen ? (qlen + kTile - 1) / kTile : 0;
    const int per = max(0, t1 - t0), n = per * g.group;
    __nv_bfloat16* dk0 = g.dK + (static_cast<size_t>(b) * g.nk + key0) * g.lddk + hk * g.hd;
    __nv_bfloat16* dv0 = g.dV + (static_cast<size_t>(b) * g.nk + key0) * g.lddv + hk * g.hd;
    if (n == 0) {
        zero_out(dk0, g.lddk, min(kTile, g.nk - key0), g.hd);
        zero_out(dv0, g.lddv, min(kTile, g.nk - key0), g.hd);
        return;
    }

    if (threadIdx.x == 0) {
        bwd_init<NS>(m);
        *abort_flag = 0;
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
    const uint32_t tmem = *tmem_slot;
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
        // ---------------- TMA: ring 0 holds Q and the row statistics, ring 1 dO
        bool ok = true;
        InFlight f0, f1;
        uint32_t raws = 0;        // tiles fixed so far
        if (lane == 0) {
            mbar_arrive_expect_tx(m.a_full, 2 * P::TILE);
            load_tile<NB, TAIL>(sb + P::A0_OFF, &maps.k, &maps.kt, hk, key0, b, m.a_full);
            load_tile<NB, TAIL>(sb + P::A1_OFF, &maps.v, &maps.vt, hk, key0, b, m.a_full);
        }
        int qt = t0, h = hk * g.group;
        for (int i = 0; i < n; ++i) {
            const int st = i % NS;
            const uint32_t ph = (i / NS) & 1;
            const bool raw = fix < kTile && qt == t1 - 1;
            const uint32_t full0 = raw ? m.raw0 : m.full0 + 8 * st, full1 = raw ? m.raw1 : m.full1 + 8 * st;
            if (lane == 0) {
                ok = mbar_wait(m.empty0 + 8 * st, ph ^ 1, abort_flag);
                if (ok) {
                    mbar_arrive_expect_tx(full0, P::TILE + kStatBytes);
                    load_tile<NB, TAIL>(sb + P::R0_OFF + st * P::TILE, &maps.q, &maps.qt, h, qt * kTile, b, full0);
                    bulk_load(sb + P::STAT_OFF + st * kStatBytes,
                              g.stats + ((static_cast<size_t>(b) * g.heads + h) * qtiles + qt) * 2 * kTile, kStatBytes, full0);
                    if (!raw) f0.add(st, ph);
                    ok = mbar_wait(m.empty1 + 8 * st, ph ^ 1, abort_flag);
                    if (ok) {
                        mbar_arrive_expect_tx(full1, P::TILE);
                        load_tile<NB, TAIL>(sb + P::R1_OFF + st * P::TILE, &maps.d, &maps.dt, h, qt * kTile, b, full1);
                        if (!raw) f1.add(st, ph);
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
                zero_rows<NB, TAIL>(smem + P::R0_OFF + st * P::TILE, fix, lane, 32);
                zero_rows<NB, TAIL>(smem + P::R1_OFF + st * P::TILE, fix, lane, 32);
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(m.full0 + 8 * st);
                    mbar_arrive(m.full1 + 8 * st);
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
                f0.drain<NS>(m.full0);
                f1.drain<NS>(m.full1);
            }
        }
    } else if (warp == 1 && lane == 0) {
        // ---------------- MMA issuer
        const uint64_t k = sw128_kmajor_desc(sb + P::A0_OFF), ktl = sw32_desc(sb + P::A0_OFF + NB * T::BLK);
        const uint64_t v = sw128_kmajor_desc(sb + P::A1_OFF), vtl = sw32_desc(sb + P::A1_OFF + NB * T::BLK);
        const uint64_t q = sw128_kmajor_desc(sb + P::R0_OFF), qmn = sw128_mnmajor_desc(sb + P::R0_OFF, T::BLK);
        const uint64_t qtl = sw32_desc(sb + P::R0_OFF + NB * T::BLK);
        const uint64_t d = sw128_kmajor_desc(sb + P::R1_OFF), dmn = sw128_mnmajor_desc(sb + P::R1_OFF, T::BLK);
        const uint64_t dtl = sw32_desc(sb + P::R1_OFF + NB * T::BLK);
        auto issue_s = [&](int i) -> bool {
            const int st = i % NS;
            if (!mbar_wait(m.full0 + 8 * st, (i / NS) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (st * P::TILE) >> 4;
            mma_scores<NB, TAIL>(tmem, k, ktl, q + so, qtl + so);
            tc_commit(m.s_full);
            return true;
        };
        auto issue_dp = [&](int i) -> bool {
            const int st = i % NS;
            if (!mbar_wait(m.full1 + 8 * st, (i / NS) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (st * P::TILE) >> 4;
            mma_scores<NB, TAIL>(tmem + 128, v, vtl, d + so, dtl + so);
            tc_commit(m.d_full);
            return true;
        };
        bool ok = mbar_wait(m.a_full, 0, abort_flag) && issue_s(0) && issue_dp(0);
        for (int i = 0; ok && i < n; ++i) {
            const int st = i % NS;
            const uint32_t so = (st * P::TILE) >> 4;
            if (!mbar_wait(m.e0, i & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            mma_accumulate<NB, TAIL>(tmem + 256, tmem, dmn + so, dtl + so, i == 0);
            tc_commit(m.empty1 + 8 * st);
            if (i + 1 < n && !issue_s(i + 1)) { ok = false; break; }
            if (!mbar_wait(m.e1, i & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            mma_accumulate<NB, TAIL>(tmem + 384, tmem + 128, qmn + so, qtl + so, i == 0);
            tc_commit(m.empty0 + 8 * st);
            if (i + 1 < n && !issue_dp(i + 1)) { ok = false; break; }
        }
        if (ok) tc_commit(m.done);
        else fail();
        if (*abort_flag) {
            tc_commit(m.drain);
            mbar_wait(m.drain, 0, nullptr);
        }
    } else if (warp >= 4) {
        // ---------------- elementwise: thread = key, half of the query columns
        const int half = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const int key = key0 + row;
        const int begin = key < klen ? query_begin(key, off, g.causal_block) : 1 << 30;   // queries that see it: [begin, qlen)
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 64 * half;
        bool ok = true;
        int qt = t0;
        for (int i = 0; i < n; ++i) {
            const int st = i % NS;
            const float* stat = reinterpret_cast<const float*>(smem + P::STAT_OFF + st * kStatBytes) + 64 * half;
            const int lo = begin - (qt * kTile + 64 * half), hi = qlen - (qt * kTile + 64 * half);
            const bool cut = __any_sync(0xFFFFFFFFu, lo > 0 || hi < 64);
            if (++qt == t1) qt = t0;
            bool got = mbar_wait(m.full0 + 8 * st, (i / NS) & 1, abort_flag) && mbar_wait(m.s_full, i & 1, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got)) { ok = false; break; }
            tc_fence_after();
            uint32_t r[2][32], w[32];
            float p[64];
            tmem_ld_32x32b_x32(tl, r[0]);
            tmem_ld_32x32b_x32(tl + 32, r[1]);
            tmem_wait_ld_r(r[0]);
            tmem_wait_ld_r(r[1]);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 l = *reinterpret_cast<const float4*>(stat + c);
                p[c + 0] = ex2_approx(fmaf(__uint_as_float(r[c >> 5][(c + 0) & 31]), g.scale_log2, -l.x));
                p[c + 1] = ex2_approx(fmaf(__uint_as_float(r[c >> 5][(c + 1) & 31]), g.scale_log2, -l.y));
                p[c + 2] = ex2_approx(fmaf(__uint_as_float(r[c >> 5][(c + 2) & 31]), g.scale_log2, -l.z));
                p[c + 3] = ex2_approx(fmaf(__uint_as_float(r[c >> 5][(c + 3) & 31]), g.scale_log2, -l.w));
            }
            if (cut) {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (c < lo || c >= hi) p[c] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) w[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
            tmem_st_32x32b_x32(tl, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(m.e0);
            got = mbar_wait(m.d_full, i & 1, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got)) { ok = false; break; }
            tc_fence_after();
            tmem_ld_32x32b_x32(tl + 128, r[0]);
            tmem_ld_32x32b_x32(tl + 128 + 32, r[1]);
            tmem_wait_ld_r(r[0]);
            tmem_wait_ld_r(r[1]);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 e = *reinterpret_cast<const float4*>(stat + kTile + c);
                p[c + 0] *= __uint_as_float(r[c >> 5][(c + 0) & 31]) - e.x;
                p[c + 1] *= __uint_as_float(r[c >> 5][(c + 1) & 31]) - e.y;
                p[c + 2] *= __uint_as_float(r[c >> 5][(c + 2) & 31]) - e.z;
                p[c + 3] *= __uint_as_float(r[c >> 5][(c + 3) & 31]) - e.w;
            }
            if (cut) {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (c < lo || c >= hi) p[c] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) w[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
            tmem_st_32x32b_x32(tl + 128, w);
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
            const uint32_t acc = tl - 64 * half + 256 + 128 * half;
            __nv_bfloat16* out = half ? dk0 + static_cast<size_t>(row) * g.lddk : dv0 + static_cast<size_t>(row) * g.lddv;
            store_row<T::HDP>(acc, out, g.hd, key < g.nk, half ? g.scale : 1.f, 0, 1);
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

template <int NB, bool TAIL>
cudaError_t run_bwd(const BwdMaps& maps, const BwdArgs& g, int batch, int kv_heads, cudaStream_t s,
                    unsigned long long* launches) {
    using P = BwdPlan<NB, TAIL>;
    static unsigned long long set[2] = {0, 0};
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(&dq_kernel<NB, TAIL>), P::BYTES, &set[0]); e != cudaSuccess) return e;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(&dkv_kernel<NB, TAIL>), P::BYTES, &set[1]); e != cudaSuccess) return e;
    cudaError_t e = launch_k(dq_kernel<NB, TAIL>, dim3((g.nq + kTile - 1) / kTile, g.heads, batch), kThreadsB, P::BYTES, s, maps, g);
    ++*launches;
    if (e != cudaSuccess) return e;
    e = launch_k(dkv_kernel<NB, TAIL>, dim3((g.nk + kTile - 1) / kTile, kv_heads, batch), kThreadsB, P::BYTES, s, maps, g);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t attention_bwd_workspace(const dlo_attn& a) {
    return static_cast<size_t>(a.batch) * a.heads * ((a.nq + kTile - 1) / kTile) * kStatBytes;
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
    g.stats = static_cast<float*>(ws);
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
        !map(&m.v, &m.vt, V, a.nk, a.kv_heads, a.ldv) || !map(&m.d, &m.dt, dO, a.nq, a.heads, a.lddo))
        return cudaErrorInvalidValue;
    if (hd <= 64) return run_bwd<1, false>(m, g, a.batch, a.kv_heads, s, launches);
    if (tail) return run_bwd<1, true>(m, g, a.batch, a.kv_heads, s, launches);
    return run_bwd<2, false>(m, g, a.batch, a.kv_heads, s, launches);
}

}  // namespace dlo
