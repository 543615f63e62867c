// Non-causal multi-head attention on the 5th-generation tensor cores.
// O = softmax(Q K^T / sqrt(hd)) V for every head dim that is a multiple of 8
// up to 128.  Q, K and V tiles are whole 64-column blocks (one for hd <= 64,
// two for hd > 80); a head dim of 64 + t (t <= 16, e.g. 72) instead adds a
// 16-column tail block loaded with the 32-byte swizzle.  TMA fills the box
// columns past hd with zeros (a 4-D tensor map [batch, rows, heads, hd] ends
// each head at hd), so the padded columns add nothing to Q K^T and are
// dropped from O.
//
// One CTA per (128 query rows, head, batch); 6 warps:
//   warp 0      TMA: the Q tile once, then K_j and V_j tiles of 128 keys into
//               one ring stage, both completing one barrier (the MMA issuer
//               waits once per tile); rows past a batch's end are zero-filled
//   warp 1      MMA issuer (one elected lane): S_j = Q K_j^T into one of two TMEM S
//               buffers (128 fp32 columns each), and O += P_j V_j into the TMEM
//               O accumulator; issue order S_0, S_1, PV_0, S_2, PV_1, ... so the
//               tensor core computes S_{j+1} while the softmax warps work on S_j
//   warps 2..5  softmax, one thread per query row (its TMEM lane): load S_j,
//               mask keys past nk, running max in the log2 domain, p = 2^(s -
//               m), row sum, P_j as bf16 pairs over the first 64 columns of
//               its own S buffer in TMEM (P V reads A from tensor memory).
//               The reference max only moves
//               when a row's max grows by more than 8 (a factor 256), and only
//               then is that row's O rescaled in TMEM (ld, scale, st) -- the
//               p values stay below 2^8, which bf16 and fp32 hold exactly in
//               range.  At the end O / l is written as bf16.
// V is the B operand of P V in its natural [key][dim] layout, i.e. MN-major
// (dims contiguous): 64-dim blocks of 128-byte rows, one row per key.
//
// DUO (head dims up to 80): two CTAs share an SM.  Each holds one S buffer
// and O in 256 TMEM columns and two K/V stages in ~100 KB of shared memory;
// its MMAs run S_j, PV_j, S_{j+1}, ... and the other CTA's softmax fills the
// tensor core while this one's runs.  A grid of 1.7 waves of single CTAs then
// fits in one wave.  Two CTAs leave a thread 168 registers; 16 bytes spill in the
// inference form, 64 in the training form (2 x 16 heads of 72, 1024 tokens: 18.7 and
// 19.4 us).
//
// Every mbarrier wait is bounded; a wait that runs out sets the error word
// and the abort flag, every role leaves its loop, in-flight TMA loads and
// MMAs are drained (bounded) and TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdlib>

#include "attention.cuh"

namespace dlo {

namespace {

constexpr int TQ = 128;          // query rows per CTA (MMA M, TMEM lanes)
constexpr int TK = 128;          // keys per tile
constexpr int kThreadsA = 192;

template <int NB, bool TAIL, bool DUO = false>
struct AttnPlan {
    static constexpr int HDP = AttnTile<NB, TAIL>::HDP;     // padded head dim
    static constexpr int BLK = AttnTile<NB, TAIL>::BLK;     // 64 columns of a tile
    static constexpr int TILE = AttnTile<NB, TAIL>::BYTES;  // one Q, K or V tile
    // K/V ring depth: three stages when they fit next to Q in shared memory
    // (DUO: two, so two CTAs fit on one SM)
    static constexpr int STAGES = DUO ? 2 : (TILE * 7 + 2048 <= 227 * 1024) ? 3 : 2;
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = Q_OFF + TILE;              // STAGES stages
    static constexpr int V_OFF = K_OFF + STAGES * TILE;     // STAGES stages
    static constexpr int BAR_OFF = V_OFF + STAGES * TILE;
    // q_full, kv_full[3], k_empty[3], 3 spare, v_empty[3], s_full[2], p_full,
    // pv_done, drain
    static constexpr int NBARS = 1 + 12 + 2 + 3;
    static constexpr int TMEM_SLOT_OFF = BAR_OFF + NBARS * 8;
    static constexpr int ABORT_OFF = TMEM_SLOT_OFF + 4;
    static constexpr int USED = ABORT_OFF + 4 + 1024;
    // single CTAs: at least 116 KB, so one CTA per SM owns all 512 TMEM
    // columns; DUO: two CTAs of 256 columns each
    static constexpr int BYTES = DUO ? USED : (USED > 118784 ? USED : 118784);
    static constexpr uint32_t TMEM_COLS = DUO ? 256 : 512;
    static constexpr int SBUF = DUO ? 1 : 2;           // S buffers (128 columns each, from 0)
    static constexpr uint32_t O_COL = SBUF * 128;
    static_assert(!DUO || (NB == 1 && 2 * (USED + 1024) <= 228 * 1024), "DUO: two CTAs per SM");
};

// The training form (TR): masks, shared key/value heads, row statistics, and a
// grid that may split the keys (partial results, joined by a second launch).
struct AttnTrain {
    float* lse;                 // [batch, heads, nq]
    const int *q_lens, *k_lens;
    int causal_block, group, splits;
    int lg;                     // 2^lg query heads of a group share a tile: row r is head r % 2^lg of query r >> lg
    float *po, *pl;             // splits > 1: [splits][batch][heads][nq][hd] and [..][nq]
};

struct AttnMaps {
    CUtensorMap q, k, v;        // 64-column boxes, 128-byte swizzle
    CUtensorMap qt, kt, vt;     // 16-column tail boxes, 32-byte swizzle
    CUtensorMap o, ot;          // TR: the output, stored by TMA
};

template <int NB, bool TAIL, bool DUO, bool TR>
__global__ void __launch_bounds__(kThreadsA, DUO ? 2 : 1)
    attn_tc_kernel(const __grid_constant__ AttnMaps maps, __nv_bfloat16* __restrict__ O, int hd,
                   int nq, int nk, int ldo, float scale_log2, int* err, const AttnTrain tr) {
    using P = AttnPlan<NB, TAIL, DUO>;
    constexpr int HDP = P::HDP;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar = sb + P::BAR_OFF;
    const uint32_t q_full = bar;
    const uint32_t kv_full = bar + 8, k_empty = bar + 32;
    const uint32_t raw = bar + 56, staged = bar + 64, v_empty = bar + 80;
    const uint32_t s_full = bar + 104;
    const uint32_t p_full = bar + 120, pv_done = bar + 128, drain = bar + 136;
    constexpr int NS = P::STAGES;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + P::TMEM_SLOT_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P::ABORT_OFF);

    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int b = blockIdx.z;
    int h = blockIdx.y, qt = blockIdx.x, ntiles = (nk + TK - 1) / TK;
    int t0 = 0, hk = h, qlen = nq, klen = nk, split = 0;   // TR: first key tile, key/value head, valid rows
    int nh = gridDim.y, tq = TQ;                           // TR: query heads, queries per tile
    if constexpr (TR) {
        pdl_wait();             // the lengths may come from the predecessor
        const int off = nk - nq;
        split = qt % tr.splits;
        // with a causal mask the last query tiles have the most keys: first
        qt = gridDim.x / tr.splits - 1 - qt / tr.splits;
        h <<= tr.lg;            // the first of the tile's heads
        nh <<= tr.lg;
        tq >>= tr.lg;
        hk = h / tr.group;
        qlen = seq_len(tr.q_lens, b, nq);
        klen = seq_len(tr.k_lens, b, nk);
        const int last = min(qt * tq + tq, qlen) - 1;
        ntiles = last < qt * tq ? 0 : (key_end(last, off, tr.causal_block, klen) + TK - 1) / TK;
        if (tr.splits > 1) {
            const int per = (ntiles + tr.splits - 1) / tr.splits;
            t0 = split * per;
            ntiles = min(ntiles, t0 + per) - t0;
        }
        if (ntiles <= 0) {      // no key for any of the rows
            pdl_launch_dependents();
            float* lse = tr.splits > 1 ? tr.pl + static_cast<size_t>(split) * gridDim.z * nh * nq : tr.lse;
            const int rows = min(nq - qt * tq, tq) << tr.lg;
            for (int r = threadIdx.x; r < rows; r += kThreadsA)
                lse[(static_cast<size_t>(b) * nh + h + (r & ((1 << tr.lg) - 1))) * nq + qt * tq + (r >> tr.lg)] = -INFINITY;
            if (tr.splits == 1) {
                const int c8 = hd / 8;
                for (int i = threadIdx.x; i < rows * c8; i += kThreadsA) {
                    const int r = i / c8;
                    reinterpret_cast<uint4*>(O + (static_cast<size_t>(b) * nq + qt * tq + (r >> tr.lg)) * ldo +
                                             (h + (r & ((1 << tr.lg) - 1))) * hd)[i % c8] = make_uint4(0, 0, 0, 0);
                }
            }
            return;
        }
    }

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(kv_full + 8 * i, 1);
            mbar_init(k_empty + 8 * i, 1);
            mbar_init(v_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(s_full + 8 * i, 1);
        mbar_init(p_full, 4);
        mbar_init(pv_done, 1);
        mbar_init(drain, 1);
        if constexpr (TR) {
            mbar_init(raw, 1);
            mbar_init(staged, 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
        if constexpr (TR) {     // this thread is the one that loads, and has waited for the predecessor
            mbar_arrive_expect_tx(q_full, P::TILE);
            load_tile<NB, TAIL>(sb + P::Q_OFF, &maps.q, &maps.qt, h, qt * tq, b, q_full);
        }
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    if (warp == 1) {
        tmem_alloc(sb + P::TMEM_SLOT_OFF, P::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
    pdl_wait();                 // predecessor's outputs complete and visible
    pdl_launch_dependents();

    auto fail = [&]() {
        *abort_flag = 1;
        if (err) atomicExch(err, 1);
    };

    // TR: keys behind k_lens end inside the last tile; their V rows become zero
    // before the MMAs see that tile (its loads complete on `raw` instead)
    const int fix = TR && klen < nk && klen < (t0 + ntiles) * TK ? klen - (t0 + ntiles - 1) * TK : TK;
    if (warp == 0) {
        // ---------------- TMA producer
        bool ok = true;
        uint32_t issued = 0;      // stages with a load in flight
        uint32_t par = 0;         // parity of that load's phase
        if (lane == 0) {
            if constexpr (!TR) {
                mbar_arrive_expect_tx(q_full, P::TILE);
                load_tile<NB, TAIL>(sb + P::Q_OFF, &maps.q, &maps.qt, h, qt * tq, b, q_full);
            }
            for (int j = 0; ok && j < ntiles; ++j) {
                const int st = j % NS;
                const uint32_t ph = (j / NS) & 1;
                // the stage's K is free after S_{j-NS}, its V after PV_{j-NS}
                if (!mbar_wait(k_empty + 8 * st, ph ^ 1, abort_flag) ||
                    !mbar_wait(v_empty + 8 * st, ph ^ 1, abort_flag)) {
                    fail();
                    ok = false;
                    break;
                }
                const bool raw_tile = TR && fix < TK && j == ntiles - 1;
                const uint32_t full = raw_tile ? raw : kv_full + 8 * st;
                mbar_arrive_expect_tx(full, 2 * P::TILE);
                load_tile<NB, TAIL>(sb + P::K_OFF + st * P::TILE, &maps.k, &maps.kt, hk, (t0 + j) * TK, b, full);
                load_tile<NB, TAIL>(sb + P::V_OFF + st * P::TILE, &maps.v, &maps.vt, hk, (t0 + j) * TK, b, full);
                if (raw_tile) break;
                issued |= 1u << st;
                par = (par & ~(1u << st)) | (ph << st);
            }
        }
        if constexpr (TR) {
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (ok && fix < TK) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(raw, 0, nullptr));
                if (ok) {
                    const int st = (ntiles - 1) % NS;
                    zero_rows<NB, TAIL>(smem + P::V_OFF + st * P::TILE, fix, lane, 32);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(kv_full + 8 * st);
                } else if (lane == 0) {
                    fail();
                }
            }
        }
        if (lane == 0 && (!ok || *abort_flag)) {
            mbar_wait(q_full, 0, nullptr);
            for (int i = 0; i < NS; ++i)
                if (issued & (1u << i)) mbar_wait(kv_full + 8 * i, (par >> i) & 1u, nullptr);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer: the warp waits, one lane issues
        const bool one = elect_one();
        constexpr uint32_t idesc_s = idesc_bf16_f32(TQ, TK);
        constexpr uint32_t idesc_o = idesc_bf16_f32(TQ, NB * 64, true);
        constexpr uint32_t idesc_ot = idesc_bf16_f32(TQ, 16, true);
        // Descriptors formed once; a descriptor's start-address field holds
        // (address >> 4) and shared addresses stay below 256 KB, so an offset
        // within shared memory adds (offset >> 4).  Every instruction this
        // thread spends between MMAs costs tensor throughput (N=128 MMAs are
        // shorter than the issue path).
        const uint64_t q_desc = sw128_kmajor_desc(sb + P::Q_OFF);
        const uint64_t k_desc0 = sw128_kmajor_desc(sb + P::K_OFF);
        const uint64_t v_desc0 = sw128_mnmajor_desc(sb + P::V_OFF, P::BLK);
        const uint64_t qt_desc = sw32_desc(sb + P::Q_OFF + NB * P::BLK);
        const uint64_t kt_desc0 = sw32_desc(sb + P::K_OFF + NB * P::BLK);
        const uint64_t vt_desc0 = sw32_desc(sb + P::V_OFF + NB * P::BLK);
        bool ok = warp_wait(q_full, 0, abort_flag);
        auto issue_s = [&](int j) -> bool {
            const int st = j % NS;                 // K stage
            const uint32_t ph = (j / NS) & 1;
            const int sbuf = j % P::SBUF;          // S buffer
            // S_j overwrites the columns of S_{j-2} / P_{j-2}: the softmax
            // finished with them before p_full(j-2), and PV_{j-2}, issued
            // earlier by this thread, reads P_{j-2} before this MMA writes
            // (MMAs of one thread execute in issue order)
            if (!warp_wait(kv_full + 8 * st, ph, abort_flag)) return false;
            tc_fence_after();
            const uint32_t d = tmem + sbuf * TK;
            const uint32_t so = (st * P::TILE) >> 4;
            if (one) {
#pragma unroll
                for (int kk = 0; kk < NB * 4; ++kk) {
                    const uint32_t off = ((kk >> 2) * P::BLK + (kk & 3) * 32) >> 4;
                    tc_mma_f16(d, q_desc + off, k_desc0 + so + off, idesc_s, kk > 0);
                }
                if constexpr (TAIL) tc_mma_f16(d, qt_desc, kt_desc0 + so, idesc_s, 1u);
                tc_commit(s_full + 8 * sbuf);
                tc_commit(k_empty + 8 * st);
            }
            __syncwarp();
            return true;
        };
        auto issue_pv = [&](int j) -> bool {
            const int st = j % NS;                 // V stage: landed with K_j (waited in issue_s)
            const int sbuf = j % P::SBUF;          // P lives in S buffer sbuf
            if (!warp_wait(p_full, j & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (st * P::TILE) >> 4;
            if (one) {
#pragma unroll
                for (int kk = 0; kk < TK / 16; ++kk) {
                    const uint32_t a = tmem + sbuf * TK + kk * 8;    // P_j: 16 keys = 8 columns
                    const uint32_t acc = (j > 0 || kk > 0) ? 1u : 0u;
                    tc_mma_f16_ts(tmem + P::O_COL, a, v_desc0 + so + ((kk * 2048) >> 4), idesc_o, acc);
                    if constexpr (TAIL)
                        tc_mma_f16_ts(tmem + P::O_COL + NB * 64, a, vt_desc0 + so + ((kk * 512) >> 4), idesc_ot,
                                      acc);
                }
                tc_commit(pv_done);
                tc_commit(v_empty + 8 * st);
            }
            __syncwarp();
            return true;
        };
        if (ok) ok = issue_s(0);
        // two S buffers: S_{j+1} runs while the softmax works on S_j; one
        // (DUO): S_{j+1} follows PV_j, which reads P_j from the same columns
        // (MMAs of one thread execute in issue order)
        for (int j = 1; ok && j < ntiles; ++j) ok = DUO ? (issue_pv(j - 1) && issue_s(j)) : (issue_s(j) && issue_pv(j - 1));
        if (ok) ok = issue_pv(ntiles - 1);
        if (one) {
            if (!ok) fail();
            if (*abort_flag) {
                tc_commit(drain);
                mbar_wait(drain, 0, nullptr);
            }
        }
        __syncwarp();
    } else if (warp >= 2) {
        // ---------------- softmax: thread = query row
        const int q = warp & 3;
        const int row = q * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
        float m_ref = -INFINITY, l = 0.f;
        const uint64_t scale2 = f32x2(scale_log2, scale_log2);
        bool ok = true;
        int row_end = nk;         // one past the last key of this row
        if constexpr (TR) {
            const int i = qt * tq + (row >> tr.lg);
            row_end = i < qlen ? key_end(i, nk - nq, tr.causal_block, klen) : 0;
        }
        for (int j = 0; j < ntiles; ++j) {
            const int st = j % P::SBUF;
            const uint32_t ph = (j / P::SBUF) & 1;
            bool got = mbar_wait(s_full + 8 * st, ph, abort_flag);
            got = __all_sync(0xFFFFFFFFu, got);
            if (!got) { ok = false; break; }
            tc_fence_after();
            // all of S_j's loads in flight before one wait (the first wait
            // covers every load; the others tie each array to it)
            uint32_t r[TK / 32][32];
#pragma unroll
            for (int c = 0; c < TK / 32; ++c) tmem_ld_32x32b_x32(tl + st * TK + c * 32, r[c]);
#pragma unroll
            for (int c = 0; c < TK / 32; ++c) tmem_wait_ld_r(r[c]);
            float v[TK];
#pragma unroll
            for (int c = 0; c < TK / 32; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) v[c * 32 + i] = __uint_as_float(r[c][i]);
            // raw scores: the row max is taken before scaling (scale > 0), and
            // keys past nk exist only in the last tile
            const int kvalid = row_end - (t0 + j) * TK;
            if (kvalid < TK) {
#pragma unroll
                for (int i = 0; i < TK; ++i)
                    if (i >= kvalid) v[i] = -INFINITY;
            }
            // 8 independent max / sum chains (ILP instead of one 128-long chain)
            float mp[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) mp[u] = v[u];
#pragma unroll
            for (int i = 8; i < TK; ++i) mp[i & 7] = fmaxf(mp[i & 7], v[i]);
            float mt = fmaxf(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])),
                             fmaxf(fmaxf(mp[4], mp[5]), fmaxf(mp[6], mp[7])));
            mt *= scale_log2;
            const bool resc = mt > m_ref + 8.f;
            const float m_new = resc ? mt : m_ref;
            const float corr = resc ? ex2_approx(m_ref - m_new) : 1.f;
            // TR: a row that has seen no key yet keeps m = -inf and p = 0
            const float neg = TR && m_new == -INFINITY ? 0.f : -m_new;
            float sp[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < TK; i += 2) {
                f32x2_split(fma_f32x2(f32x2(v[i], v[i + 1]), scale2, f32x2(neg, neg)), v[i], v[i + 1]);
                v[i] = ex2_approx(v[i]);
                v[i + 1] = ex2_approx(v[i + 1]);
                f32x2_split(add_f32x2(f32x2(sp[i & 7], sp[(i & 7) + 1]), f32x2(v[i], v[i + 1])), sp[i & 7], sp[(i & 7) + 1]);
            }
            const float rs = ((sp[0] + sp[1]) + (sp[2] + sp[3])) + ((sp[4] + sp[5]) + (sp[6] + sp[7]));
            l = l * corr + rs;
            m_ref = m_new;
            // P_j (bf16 pairs) over the first 64 columns of its own S buffer
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = pack_bf16x2(v[64 * c + 2 * i], v[64 * c + 2 * i + 1]);
                tmem_st_32x32b_x32(tl + st * TK + c * 32, w);
            }
            tmem_wait_st();
            // PV_{j-1} must be done before O is rescaled; every phase is waited
            // so the parity stays in step with the barrier
            if (j > 0) {
                got = mbar_wait(pv_done, (j - 1) & 1, abort_flag);
                got = __all_sync(0xFFFFFFFFu, got);
                if (!got) { ok = false; break; }
                tc_fence_after();
            }
            if (j > 0 && __any_sync(0xFFFFFFFFu, resc)) {
#pragma unroll 1
                for (int c = 0; c < (HDP + 31) / 32; ++c) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tl + P::O_COL + c * 32, r);
                    tmem_wait_ld_r(r);
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * corr);
                    tmem_st_32x32b_x32(tl + P::O_COL + c * 32, r);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
        }
        if (ok) {
            bool got = mbar_wait(pv_done, (ntiles - 1) & 1, abort_flag);
            got = __all_sync(0xFFFFFFFFu, got);
            ok = got;
        }
        if (!ok) {
            if (lane == 0) fail();
        } else {
            tc_fence_after();
            // TR: l = 0 where the row sees no key; its accumulator is 0 too, or NaN
            // where the other rows' keys hold an infinite V
            const bool none = TR && l == 0.f;
            const float inv = none ? 0.f : 1.f / l;
            const int grow = qt * tq + (TR ? row >> tr.lg : row);
            const int h0 = h;
            if constexpr (TR) h += row & ((1 << tr.lg) - 1);
            float* prow = nullptr;
            if constexpr (TR) {
                // natural logarithm of the sum of exp(scores)
                const float lse = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * 0.6931471805599453f;
                const size_t r = (static_cast<size_t>(b) * nh + h) * nq + grow;
                if (tr.splits > 1) {
                    const size_t p = static_cast<size_t>(split) * gridDim.z * nh * nq + r;
                    prow = tr.po + p * hd;
                    if (grow < nq) tr.pl[p] = lse;
                } else if (grow < nq) {
                    tr.lse[r] = lse;
                }
            }
            __nv_bfloat16* orow = O + (static_cast<size_t>(b) * nq + grow) * ldo + h * hd;
#pragma unroll 1
            for (int c = 0; c < (HDP + 31) / 32; ++c) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(tl + P::O_COL + c * 32, r);
                tmem_wait_ld_r(r);
                if constexpr (TR) {
                    if (!prow) {        // into Q's place, which every product has read
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = none ? 0 : pack_bf16x2(__uint_as_float(r[2 * i]) * inv, __uint_as_float(r[2 * i + 1]) * inv);
                        put_row<NB, TAIL>(smem + P::Q_OFF, row, c, w);
                        continue;
                    }
                }
                if (grow < nq) {
#pragma unroll
                    for (int k4 = 0; k4 < 4; ++k4) {
                        if (TR && c * 32 + 8 * k4 < hd) {
                            float4* pw = reinterpret_cast<float4*>(prow + c * 32 + 8 * k4);
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                pw[u] = make_float4(__uint_as_float(r[8 * k4 + 4 * u]) * inv, __uint_as_float(r[8 * k4 + 4 * u + 1]) * inv,
                                                    __uint_as_float(r[8 * k4 + 4 * u + 2]) * inv, __uint_as_float(r[8 * k4 + 4 * u + 3]) * inv);
                        } else if (c * 32 + 8 * k4 < hd) {
                            uint4 w;
                            w.x = pack_bf16x2(__uint_as_float(r[8 * k4 + 0]) * inv, __uint_as_float(r[8 * k4 + 1]) * inv);
                            w.y = pack_bf16x2(__uint_as_float(r[8 * k4 + 2]) * inv, __uint_as_float(r[8 * k4 + 3]) * inv);
                            w.z = pack_bf16x2(__uint_as_float(r[8 * k4 + 4]) * inv, __uint_as_float(r[8 * k4 + 5]) * inv);
                            w.w = pack_bf16x2(__uint_as_float(r[8 * k4 + 6]) * inv, __uint_as_float(r[8 * k4 + 7]) * inv);
                            *reinterpret_cast<uint4*>(orow + c * 32 + 8 * k4) = w;
                        }
                    }
                }
            }
            if constexpr (TR) {
                if (!prow) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(staged);
                    if (warp == 2 && warp_wait(staged, 0, abort_flag)) {
                        if (lane == 0) {
                            store_tile<NB, TAIL>(sb + P::Q_OFF, &maps.o, &maps.ot, h0, qt * tq, b);
                            bulk_commit();
                            bulk_wait_all();
                        }
                    } else if (warp == 2 && lane == 0) {
                        fail();
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
        tmem_dealloc(tmem, P::TMEM_COLS);
    }
}

template <int NB, bool TAIL, bool DUO, bool TR = false>
cudaError_t run_tc(const void* Q, const void* K, const void* V, void* O, int batch, int heads,
                   int hd, int nq, int nk, int ldq, int ldk, int ldv, int ldo, int* err,
                   cudaStream_t s, unsigned long long* launches, const AttnTrain& tr = AttnTrain{nullptr, nullptr, nullptr, 0, 1, 1, 0, nullptr, nullptr}) {
    using P = AttnPlan<NB, TAIL, DUO>;
    static_assert(P::BYTES <= 227 * 1024, "attention shared memory plan exceeds 227 KB");
    const void* kernel = reinterpret_cast<const void*>(&attn_tc_kernel<NB, TAIL, DUO, TR>);
    static unsigned long long attr = 0;
    if (cudaError_t e = allow_smem(kernel, P::BYTES, &attr); e != cudaSuccess) return e;
    AttnMaps maps;
    const CUtensorMapSwizzle w128 = CU_TENSOR_MAP_SWIZZLE_128B, w32 = CU_TENSOR_MAP_SWIZZLE_32B;
    const int qh = 1 << tr.lg;
    if (!make_map4(&maps.q, Q, batch, nq, heads, hd, ldq, 64, w128, qh) ||
        !make_map4(&maps.k, K, batch, nk, heads / tr.group, hd, ldk, 64, w128) ||
        !make_map4(&maps.v, V, batch, nk, heads / tr.group, hd, ldv, 64, w128))
        return cudaErrorInvalidValue;
    if (TAIL) {
        if (!make_map4(&maps.qt, Q, batch, nq, heads, hd, ldq, 16, w32, qh) ||
            !make_map4(&maps.kt, K, batch, nk, heads / tr.group, hd, ldk, 16, w32) ||
            !make_map4(&maps.vt, V, batch, nk, heads / tr.group, hd, ldv, 16, w32))
            return cudaErrorInvalidValue;
    } else {
        maps.qt = maps.q;
        maps.kt = maps.k;
        maps.vt = maps.v;
    }
    maps.o = maps.q;
    maps.ot = maps.qt;
    if (TR) {
        if (!make_map4(&maps.o, O, batch, nq, heads, hd, ldo, 64, w128, qh) ||
            (TAIL && !make_map4(&maps.ot, O, batch, nq, heads, hd, ldo, 16, w32, qh)))
            return cudaErrorInvalidValue;
    }
    const float scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(hd));
    const int tq = TQ >> tr.lg;
    dim3 grid((nq + tq - 1) / tq * tr.splits, heads >> tr.lg, batch);
    cudaError_t le_ = launch_k(attn_tc_kernel<NB, TAIL, DUO, TR>, grid, kThreadsA, P::BYTES, s, maps, static_cast<__nv_bfloat16*>(O), hd, nq, nk, ldo, scale_log2, err, tr);
    ++*launches;
    return le_ != cudaSuccess ? le_ : cudaGetLastError();
}

// DLO_ATTN_DUO=0 keeps head dims up to 80 on one CTA per SM (tuning).
bool attn_duo_enabled() {
    static int v = -1;
    if (v < 0) {
        const char* e = std::getenv("DLO_ATTN_DUO");
        v = (e && e[0] == '0') ? 0 : 1;
    }
    return v != 0;
}

}  // namespace

bool attention_tc_supported(int hd) { return hd >= 8 && hd <= 128 && hd % 8 == 0; }

cudaError_t launch_attention_tc(const void* Q, const void* K, const void* V, void* O, int batch,
                                int heads, int hd, int nq, int nk, int ldq, int ldk, int ldv,
                                int ldo, int* err, cudaStream_t s, unsigned long long* launches) {
    // DUO when one CTA per SM would take more than one wave: with fewer CTAs
    // than SMs nothing shares an SM and the serial S / softmax / PV order of
    // a DUO CTA only costs time
    const long long ctas = static_cast<long long>((nq + TQ - 1) / TQ) * heads * batch;
    const bool duo = attn_duo_enabled() && ctas > gemm_num_sms();
    if (!attention_tc_supported(hd)) return cudaErrorInvalidValue;
    if (hd <= 64)
        return duo ? run_tc<1, false, true>(Q, K, V, O, batch, heads, hd, nq, nk, ldq, ldk, ldv, ldo, err, s, launches)
                   : run_tc<1, false, false>(Q, K, V, O, batch, heads, hd, nq, nk, ldq, ldk, ldv, ldo, err, s, launches);
    if (hd <= 80)
        return duo ? run_tc<1, true, true>(Q, K, V, O, batch, heads, hd, nq, nk, ldq, ldk, ldv, ldo, err, s, launches)
                   : run_tc<1, true, false>(Q, K, V, O, batch, heads, hd, nq, nk, ldq, ldk, ldv, ldo, err, s, launches);
    return run_tc<2, false, false>(Q, K, V, O, batch, heads, hd, nq, nk, ldq, ldk, ldv, ldo, err, s, launches);
}

namespace {

// Joins the partial results of a split: lse = log sum_p exp(lse_p), O = sum_p
// exp(lse_p - lse) O_p.  One warp a row; bound by reading the partial rows.
__global__ void __launch_bounds__(256) attn_join_kernel(const float* __restrict__ po, const float* __restrict__ pl,
                                                        int splits, size_t rows, int nq, int heads, int hd,
                                                        __nv_bfloat16* __restrict__ O, int ldo,
                                                        float* __restrict__ lse) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const size_t r = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;     // (b, h, i)
    if (r >= rows) return;
    // lane p holds the weights of parts p and p + 32 (splits <= 64)
    const float l0 = lane < splits ? pl[lane * rows + r] : -INFINITY;
    const float l1 = lane + 32 < splits ? pl[(lane + 32) * rows + r] : -INFINITY;
    float top = fmaxf(l0, l1);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    const float m = top == -INFINITY ? 0.f : top;
    const float w0 = exp2f((l0 - m) * 1.4426950408889634f), w1 = exp2f((l1 - m) * 1.4426950408889634f);
    float total = w0 + w1;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);      // columns 4 lane .. 4 lane + 3
#pragma unroll 4
    for (int p = 0; p < splits; ++p) {
        const float w = __shfl_sync(0xFFFFFFFFu, p < 32 ? w0 : w1, p & 31);
        // weight 0: nothing visible there, its O_p was not written
        if (4 * lane < hd && w != 0.f) {
            const float4 v = reinterpret_cast<const float4*>(po + (p * rows + r) * hd)[lane];
            acc = make_float4(acc.x + w * v.x, acc.y + w * v.y, acc.z + w * v.z, acc.w + w * v.w);
        }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const size_t bh = r / nq, i = r - bh * nq, b = bh / heads, h = bh - b * heads;
    if (4 * lane < hd)
        reinterpret_cast<uint2*>(O + (b * nq + i) * ldo + h * hd)[lane] =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0) lse[r] = total == 0.f ? -INFINITY : m + logf(total);
}

// The grid of a training forward, from the sizes alone.
//  lg: query heads of a group that share a tile (a power of two that divides
//    the group), where that makes fewer tiles: short sequences leave most of a
//    tile of one head empty and read K and V once a head (2 x 16 heads over
//    4, 37 queries, 8192 keys: 19 us against 26).
//  splits: CTAs that share the keys of one tile, as many as fill the SMs when
//    the tiles alone do not, each with at least four key tiles.
struct FwdPlan {
    int lg, splits;
    long long ctas;
};

FwdPlan attn_fwd_plan(const dlo_attn& a) {
    const auto tiles = [&](int lg) {
        const long long tq = TQ >> lg;
        return (a.nq + tq - 1) / tq * (a.heads >> lg) * a.batch;
    };
    FwdPlan p = {0, 1, 0};
    for (int lg = 1; lg <= 7 && (a.heads / a.kv_heads) % (1 << lg) == 0; ++lg)
        if (tiles(lg) < tiles(p.lg)) p.lg = lg;
    const long long ctas = tiles(p.lg), fill = kGb300Sms / ctas, keys = (a.nk + TK - 1) / TK / 4;
    const long long n = fill < keys ? fill : keys;
    p.splits = static_cast<int>(n < 1 ? 1 : n > 64 ? 64 : n);
    p.ctas = ctas * p.splits;
    return p;
}

}  // namespace

size_t attention_fwd_workspace(const dlo_attn& a) {
    const size_t rows = static_cast<size_t>(a.batch) * a.heads * a.nq;
    const int n = attn_fwd_plan(a).splits;
    return 256 + (n > 1 ? n * rows * (a.head_dim + 1) * sizeof(float) : 0);
}

cudaError_t launch_attention_fwd(const dlo_attn& a, const void* Q, const void* K, const void* V, void* O, float* lse,
                                 void* ws, int* err, cudaStream_t s, unsigned long long* launches) {
    const size_t rows = static_cast<size_t>(a.batch) * a.heads * a.nq;
    const FwdPlan plan = attn_fwd_plan(a);
    AttnTrain tr = {lse, a.q_lens, a.k_lens, a.causal_block < a.nk ? a.causal_block : a.nk, a.heads / a.kv_heads,
                    plan.splits, plan.lg, static_cast<float*>(ws), nullptr};
    tr.pl = tr.po + tr.splits * rows * a.head_dim;
    const int hd = a.head_dim;
    const bool duo = attn_duo_enabled() && plan.ctas > kGb300Sms;      // as for launch_attention_tc
    cudaError_t e;
#define DLO_AF(NB, TAIL, DUO)                                                                                    \
    e = run_tc<NB, TAIL, DUO, true>(Q, K, V, O, a.batch, a.heads, hd, a.nq, a.nk, a.ldq, a.ldk, a.ldv, a.ldo, err, \
                                    s, launches, tr)
    if (hd <= 64) {
        if (duo) DLO_AF(1, false, true);
        else DLO_AF(1, false, false);
    } else if (hd <= 80) {
        if (duo) DLO_AF(1, true, true);
        else DLO_AF(1, true, false);
    } else {
        DLO_AF(2, false, false);
    }
#undef DLO_AF
    if (e != cudaSuccess || tr.splits == 1) return e;
    e = launch_k(attn_join_kernel, static_cast<unsigned>((rows + 7) / 8), 256, 0, s, tr.po, tr.pl, tr.splits, rows, a.nq,
                 a.heads, hd, static_cast<__nv_bfloat16*>(O), a.ldo, lse);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_attention(const void* Q, const void* K, const void* V, void* O, int batch,
                             int heads, int hd, int nq, int nk, int ldq, int ldk, int ldv, int ldo,
                             int* err, cudaStream_t s, unsigned long long* launches) {
    if (nq <= 0 || batch <= 0 || heads <= 0) return cudaSuccess;
    if (nk <= 0) return cudaErrorInvalidValue;
    return launch_attention_tc(Q, K, V, O, batch, heads, hd, nq, nk, ldq, ldk, ldv, ldo, err, s, launches);
}

}  // namespace dlo
