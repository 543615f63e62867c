// Attention over packed sequences, backward pass: the two launches and the products
// of attention_bwd.cu (its head says why: dQ by query tiles, then dK and dV by key
// tiles, each accumulated by one CTA in tensor memory), with CTAs that stay and take
// over the work of CTAs not yet launched, as in attention_packed.cu.  A tile of one
// sequence has few steps (three for 300 tokens), each ~1.2 us; a CTA's start and end
// were ~6 us around them.  Now the next item's tiles are loaded and its first products
// run while the last gradient tile leaves tensor memory, from the threads that own
// its rows straight to global memory.
//
// Warps: 0 producer (items and TMA), 1 and 2 MMA issue, 3 rows behind a sequence's end,
// 4..19 elementwise.  Steps of an item are counted on from the items before, and so are
// the uses of every barrier and slot.
//
// Rows behind a sequence's end are the next one's.  Where they are the contracted index
// of a product (K in dQ, Q in dK, dO in dV) warp 3 makes them zero: such a tile's load
// completes `raw` of its slot, and warp 3 then completes `full`.  Elsewhere they stay
// in their own rows, which are not written.
//
// What bounds it: for long sequences the tensor core and, in dQ, the elementwise warps'
// chain of waits, loads and stores (1.13 us a step at head dim 128; attention_bwd.cu's
// kernels, whose loops know where their slots begin, are 5% faster there: 8192 tokens, 40
// heads, 2600 us, these 2735); for short ones the change of items, ~3 us each: the last
// product, the gradient's way out (~0.9), K and V (Q, dO and O) from L2 (1.2) and the first
// products.  16 x 512 tokens of 40 heads of 128: 261 us (dQ 132, tensor pipe 46% active; dK, dV
// 140, 55%), 393 with a CTA an item.
//
// D = rowsum(dO O) is the diagonal of one more product, dO O^T, an item's step before
// the first: O comes by TMA into a slot of the ring, and no thread loads and adds up
// rows.  Rows that lie in one key tile form it from P dP instead, as there.
#include "attention_bwd.cuh"

namespace dlo {

namespace {

struct PackedBwdMaps {
    CUtensorMap q, k, v, d, o;       // 64-column boxes, 128-byte swizzle (d: dO)
    CUtensorMap qt, kt, vt, dt, ot;  // 16-column tails, 32-byte swizzle
};

struct PackedBwdArgs {
    const int *q_starts, *k_starts;
    int batch, rows_q, rows_k, hd, heads, kv_heads, group, causal_block;
    float scale, scale_log2;         // 1 / sqrt(hd), log2(e) / sqrt(hd)
    const float* lse;
    uint4* stats;                    // [heads][query slots] operands of kStatBytes
    __nv_bfloat16 *dQ, *dK, *dV;
    int lddq, lddk, lddv;
    // items that share one gradient tile, each a part of its products' other axis,
    // and the fp32 parts [splits][rows][heads * hd] that they leave
    int splits_q, splits_k;
    float *part_q, *part_k, *part_v;
    int* err;
};

constexpr int kItems = 2;            // items in shared memory

struct BwdItem {
    int n;                           // steps; 0: no visible pair; < 0: no more items
    int i0;                          // the first of them
    int q0, nq, k0, nk;              // the sequence's rows
    int tile, head, split;           // its gradient tile; query head (dQ) or key/value head
    int slot;                        // dQ: the tile's slot; dK, dV: that of the sequence's first query tile
    int all;                         // dQ: key tiles that its rows see; dK, dV: query tiles of a head
    int first;                       // dK, dV: the first of those
};

template <int NB, bool TAIL, bool DQ>
struct PackedBwdPlan {
    using B = BwdPlan<NB, TAIL, DQ>;
    static constexpr int TILE = B::TILE, SLOTS = B::SLOTS, STATS = B::STATS;
    static constexpr bool SHARED = B::SHARED;
    static constexpr int A0_OFF = B::A0_OFF, A1_OFF = B::A1_OFF, R_OFF = B::R_OFF, SEL_OFF = B::SEL_OFF, STAT_OFF = B::STAT_OFF;
    // dQ: four parts of each row's D; dK, dV: the selecting operands and the statistics
    static constexpr int ITEM_OFF = DQ ? SEL_OFF + kGroups * kTile * 4 : STAT_OFF + STATS * kStatBytes;
    static constexpr int ANSWER_OFF = ITEM_OFF + kItems * static_cast<int>(sizeof(BwdItem));
    static constexpr int BAR_OFF = ANSWER_OFF + 16;
    static constexpr int NBARS = 17 + 3 * SLOTS;
    static constexpr int TMEM_SLOT_OFF = BAR_OFF + NBARS * 8;
    static constexpr int ABORT_OFF = TMEM_SLOT_OFF + 4;
    static constexpr int USED = ABORT_OFF + 4;
    // as in BwdPlan
    static constexpr int WANT = USED + 1024 > 118784 ? USED + 1024 : 118784;
    static constexpr int BYTES = WANT < 227 * 1024 ? WANT : 227 * 1024;
    static_assert(USED <= 227 * 1024, "packed attention backward shared memory plan exceeds 227 KB");
    static_assert(ITEM_OFF % 16 == 0 && sizeof(BwdItem) % 16 == 0, "16-byte answers");
};

struct PackedBwdBars {
    uint32_t a_full, a_empty, s_full, d_full, s_read, d_read, e1, done, drain, drain2, answered;
    uint32_t e0, item_full, item_empty;      // [2] each (dK, dV: one e0)
    uint32_t full, empty, raw;       // [SLOTS]
};

template <int SLOTS>
__device__ __forceinline__ PackedBwdBars packed_bars(uint32_t b) {
    return {b,      b + 8,  b + 16,  b + 24,  b + 32,  b + 40,  b + 48,           b + 56,           b + 64,
            b + 72, b + 80, b + 88, b + 104, b + 120, b + 136, b + 136 + 8 * SLOTS, b + 136 + 16 * SLOTS};
}

// done: issuing warps that end a gradient tile; readers: those that read a slot; takers:
// warps that read an item.
template <int SLOTS>
__device__ __forceinline__ void packed_bars_init(const PackedBwdBars& m, int done, int readers, int takers) {
    for (uint32_t b : {m.a_full, m.a_empty, m.s_full, m.d_full, m.drain, m.drain2, m.answered}) mbar_init(b, 1);
    for (uint32_t b : {m.s_read, m.d_read, m.e0, m.e0 + 8, m.e1}) mbar_init(b, 4 * kGroups);
    mbar_init(m.done, done);
    for (int i = 0; i < kItems; ++i) {
        mbar_init(m.item_full + 8 * i, 1);
        mbar_init(m.item_empty + 8 * i, takers);
    }
    for (int i = 0; i < SLOTS; ++i) {
        mbar_init(m.full + 8 * i, 1);
        mbar_init(m.empty + 8 * i, readers);
        mbar_init(m.raw + 8 * i, 1);
    }
    fence_mbar_init();
}

// Loads in flight, for the drain: slots, the parity of each and the barrier that it
// completes (raw or full).  raw_par: the next raw use's parity of each slot.
struct PackedFlight {
    uint32_t on = 0, par = 0, raw = 0, raw_par = 0;
    __device__ uint32_t begin(const PackedBwdBars& m, Slot s, bool is_raw) {
        const uint32_t bit = 1u << s.s;
        on |= bit;
        raw = is_raw ? raw | bit : raw & ~bit;
        const uint32_t ph = is_raw ? (raw_par >> s.s) & 1u : s.ph;
        if (is_raw) raw_par ^= bit;
        par = (par & ~bit) | (ph << s.s);
        return (is_raw ? m.raw : m.full) + 8 * s.s;
    }
    template <int SLOTS>
    __device__ void drain(const PackedBwdBars& m) const {
        for (int i = 0; i < SLOTS; ++i)
            if (on & (1u << i)) mbar_wait(((raw >> i) & 1u ? m.raw : m.full) + 8 * i, (par >> i) & 1u, nullptr);
    }
};

// The producer's side of the items: `take` finds a CTA's item (false: none) and `load`
// brings its tiles (false: a wait ran out).  By warp 0; returns whether all went well.
template <typename Take, typename Load>
__device__ __forceinline__ bool produce(const PackedBwdBars& m, BwdItem* items, uint32_t answer, int lane, const volatile int* abort_flag,
                                        const Take& take, const Load& load) {
    int x = blockIdx.x, y = blockIdx.y, ni = 0;
    const auto put = [&](const BwdItem& it) -> bool {
        const bool room = warp_wait(m.item_empty + 8 * (ni % kItems), ((ni / kItems) & 1) ^ 1, abort_flag);
        if (room && lane == 0) {
            items[ni % kItems] = it;
            mbar_arrive(m.item_full + 8 * (ni % kItems));
        }
        ++ni;
        return room;
    };
    for (int k = 0;; ++k) {
        BwdItem it;
        if (take(x, y, it) && !(put(it) && (it.n == 0 || load(it)))) return false;
        // asked for only now (attention_packed.cu); the answer has to land before this CTA may end
        if (lane == 0) {
            mbar_arrive_expect_tx(m.answered, 16);
            cta_request(answer, m.answered);
        }
        if (!warp_wait(m.answered, k & 1, nullptr)) return false;
        int more = 0;
        if (lane == 0) {
            more = cta_answer(answer, x, y);
            fence_proxy_async_smem();       // read before the next answer is written
        }
        if (!__shfl_sync(0xFFFFFFFFu, more, 0)) break;
        x = __shfl_sync(0xFFFFFFFFu, x, 0);
        y = __shfl_sync(0xFFFFFFFFu, y, 0);
    }
    BwdItem end = {};
    end.n = -1;
    return put(end);
}

// warp_wait over `steps` steps of other warps, as warp 3 waits for an item's last tile: a
// wait's limit for every 65536 of them (a step takes one or two us).  Those warps' own waits are
// of one step each, so one that hangs ends this wait too.
__device__ __forceinline__ bool long_wait(uint32_t bar, uint32_t parity, const volatile int* abort_flag, int steps) {
    for (int k = steps >> 16;; --k) {
        if (warp_wait(bar, parity, abort_flag)) return true;
        if (k == 0 || __any_sync(0xFFFFFFFFu, *abort_flag)) return false;
    }
}

// The i-th item, by a warp that keeps it in registers and gives its place back.  It comes
// when all tiles of the one before are on their way: `steps` steps from now at most.
__device__ __forceinline__ bool take_item(const PackedBwdBars& m, const BwdItem* items, int i, int lane, const volatile int* abort_flag,
                                          BwdItem& it, int steps = 0) {
    if (!long_wait(m.item_full + 8 * (i % kItems), (i / kItems) & 1, abort_flag, steps)) return false;
    it = items[i % kItems];
    __syncwarp();
    if (lane == 0) mbar_arrive(m.item_empty + 8 * (i % kItems));
    return true;
}

// Columns [32 c, 32 c + 32) of the warp's accumulator rows times `scale` to their rows of the
// gradient (out: that of the warp's row 0; rows: how many of its 32 are the sequence's), or
// (part, this lane's row) in fp32 to their part.  `none`: zeros, for a row without a
// visible pair.  The whole warp reads.
__device__ __forceinline__ void put_chunk(uint32_t t, int c, __nv_bfloat16* out, int ld, int rows, float* part, int hd, int lane,
                                          bool none, float scale) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(t + c * 32, r);
    tmem_wait_ld_r(r);
    if (none) {
#pragma unroll
        for (int u = 0; u < 32; ++u) r[u] = 0;
    }
    if (part) {
#pragma unroll
        for (int u = 0; u < 32; u += 4)
            if (lane < rows && c * 32 + u < hd)
                *reinterpret_cast<float4*>(part + c * 32 + u) =
                    make_float4(__uint_as_float(r[u]) * scale, __uint_as_float(r[u + 1]) * scale, __uint_as_float(r[u + 2]) * scale,
                                __uint_as_float(r[u + 3]) * scale);
    } else {
        uint32_t w[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) w[u] = pack_bf16x2(__uint_as_float(r[2 * u]) * scale, __uint_as_float(r[2 * u + 1]) * scale);
        put_rows32(w, c * 32, hd, lane, [&](int k) -> __nv_bfloat16* {
            const int i = (lane & ~3) + k;
            return i < rows ? out + static_cast<size_t>(i) * ld : nullptr;
        });
    }
}

// ------------------------------------------------------------------ dQ
// TMEM: S [0, 128), dP [128, 256), two dS [256, 320) and [320, 384), dQ [384, 512); dO O^T
// of an item takes dP's place before its first dP.  Order of issue as dq_kernel's, but S_j
// goes after dQ_{j-2}: whoever has S_j may then write its dS, where a wait for the dQ before
// cost the elementwise warps 0.13 us a step (8192 tokens of 32 heads of 64: dQ 722 us, 738).
// So a warp may be done with dS_{j+1} before another is with dS_j, and the two arrive on
// barriers of their own: dS number u of a CTA on e0[u % 2].  Number u + 2 waits for dQ
// number u, so it never arrives beside u.
template <int NB, bool TAIL>
__global__ void __launch_bounds__(kThreadsB, 1)
    packed_dq_kernel(const __grid_constant__ PackedBwdMaps maps, const __grid_constant__ PackedBwdArgs g) {
    using P = PackedBwdPlan<NB, TAIL, true>;
    using T = AttnTile<NB, TAIL>;
    const auto first = [](int i) { return slot_of<P::SLOTS, P::SHARED, false>(i); };
    const auto second = [](int i) { return slot_of<P::SLOTS, P::SHARED, true>(i); };
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(smem);
    const PackedBwdBars m = packed_bars<P::SLOTS>(sb + P::BAR_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + P::TMEM_SLOT_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P::ABORT_OFF);
    BwdItem* items = reinterpret_cast<BwdItem*>(smem + P::ITEM_OFF);
    if (smem - smem_raw + P::USED > P::BYTES) {       // the base of dynamic shared memory is 1 KB aligned
        if (threadIdx.x == 0 && g.err) atomicExch(g.err, 1);
        return;
    }
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        packed_bars_init<P::SLOTS>(m, 1, 1, 3 + 4 * kGroups);
        *abort_flag = 0;
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
        tma_prefetch_desc(&maps.d);
        tma_prefetch_desc(&maps.o);
    }
    if (warp == 1) {
        tmem_alloc(sb + P::TMEM_SLOT_OFF, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
    pdl_wait();
    // only now: the next kernel's CTAs may allocate TMEM before they wait for
    // this grid, so every CTA of this one must hold its own first
    pdl_launch_dependents();
    auto fail = [&]() {
        *abort_flag = 1;
        if (g.err) atomicExch(g.err, 1);
    };
    const int slots = packed_slots(g.rows_q, g.batch, kTile);

    if (warp == 0) {
        // ---------------- producer: Q and dO, O, then K and V
        PackedFlight in;
        int t = 0, na = 0;            // steps and items with steps so far
        const auto take = [&](int x, int y, BwdItem& it) -> bool {
            // with a causal mask the last query tiles see the most keys: first
            it.slot = slots - 1 - x / g.splits_q;
            it.split = x % g.splits_q;
            it.head = y;
            const PackedTile p = packed_tile(g.q_starts, g.batch, g.rows_q, kTile, it.slot);
            if (p.tile < 0) return false;
            it.tile = p.tile;
            it.q0 = p.row0;
            it.nq = p.n;
            packed_other(g.k_starts, p.b, g.rows_k, g.q_starts == g.k_starts && g.rows_q == g.rows_k, p, it.k0, it.nk);
            it.all = (key_end(min((it.tile + 1) * kTile, it.nq) - 1, it.nk - it.nq, g.causal_block, it.nk) + kTile - 1) / kTile;
            const int share = (it.all + g.splits_q - 1) / g.splits_q;
            it.i0 = it.split * share;
            it.n = max(0, min(it.all, it.i0 + share) - it.i0);
            it.first = 0;
            return true;
        };
        const auto load = [&](const BwdItem& it) -> bool {
            bool ok = true;
            const int lead = it.all > 1;              // a step for D
            if (lane == 0) {
                const int row = it.q0 + it.tile * kTile, hk = it.head / g.group;
                // Q and dO are free after the last dP of the item before
                ok = na == 0 || mbar_wait(m.a_empty, (na - 1) & 1, abort_flag);
                if (ok) {
                    mbar_arrive_expect_tx(m.a_full, 2 * P::TILE);
                    load_tile<NB, TAIL>(sb + P::A0_OFF, &maps.q, &maps.qt, it.head, row, 0, m.a_full);
                    load_tile<NB, TAIL>(sb + P::A1_OFF, &maps.d, &maps.dt, it.head, row, 0, m.a_full);
                    ++na;
                }
                if (ok && lead) {
                    const Slot o = first(t), v = second(t);
                    ok = mbar_wait(m.empty + 8 * o.s, o.ph ^ 1, abort_flag);
                    if (ok) {
                        const uint32_t full = in.begin(m, o, false);
                        mbar_arrive_expect_tx(full, P::TILE);
                        load_tile<NB, TAIL>(sb + P::R_OFF + o.s * P::TILE, &maps.o, &maps.ot, it.head, row, 0, full);
                        ok = mbar_wait(m.empty + 8 * v.s, v.ph ^ 1, abort_flag);
                        if (ok) mbar_arrive(in.begin(m, v, false));       // nothing comes with it
                    }
                }
                for (int j = 0; ok && j < it.n; ++j) {
                    const Slot k = first(t + lead + j), v = second(t + lead + j);
                    const int key = (it.i0 + j) * kTile;
                    ok = mbar_wait(m.empty + 8 * k.s, k.ph ^ 1, abort_flag);
                    if (!ok) break;
                    const uint32_t fk = in.begin(m, k, it.nk - key < kTile);
                    mbar_arrive_expect_tx(fk, P::TILE);
                    load_tile<NB, TAIL>(sb + P::R_OFF + k.s * P::TILE, &maps.k, &maps.kt, hk, it.k0 + key, 0, fk);
                    ok = mbar_wait(m.empty + 8 * v.s, v.ph ^ 1, abort_flag);
                    if (!ok) break;
                    const uint32_t fv = in.begin(m, v, false);
                    mbar_arrive_expect_tx(fv, P::TILE);
                    load_tile<NB, TAIL>(sb + P::R_OFF + v.s * P::TILE, &maps.v, &maps.vt, hk, it.k0 + key, 0, fv);
                }
            }
            t += lead + it.n;
            return __shfl_sync(0xFFFFFFFFu, ok, 0);
        };
        const bool ok = produce(m, items, sb + P::ANSWER_OFF, lane, abort_flag, take, load);
        if (lane == 0) {
            if (!ok) fail();
            if (*abort_flag) {
                if (na > 0) mbar_wait(m.a_full, (na - 1) & 1, nullptr);
                in.drain<P::SLOTS>(m);
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer of D, S and dP: the warp waits, one lane issues
        const bool one = elect_one();
        const uint64_t q = sw128_kmajor_desc(sb + P::A0_OFF), qtl = sw32_desc(sb + P::A0_OFF + NB * T::BLK);
        const uint64_t d = sw128_kmajor_desc(sb + P::A1_OFF), dtl = sw32_desc(sb + P::A1_OFF + NB * T::BLK);
        const uint64_t r = sw128_kmajor_desc(sb + P::R_OFF), rtl = sw32_desc(sb + P::R_OFF + NB * T::BLK);
        int t = 0, ns = 0, nd = 0, na = 0;      // steps; S and dP issued; items with steps
        // S and dP take the places of the last ones once those are read
        const auto issue_s = [&](int i, bool behind) -> bool {
            const Slot k = first(i), before = first(i - 2);
            if ((ns > 0 && !warp_wait(m.s_read, (ns - 1) & 1, abort_flag)) || !warp_wait(m.full + 8 * k.s, k.ph, abort_flag) ||
                (behind && !warp_wait(m.empty + 8 * before.s, before.ph, abort_flag)))
                return false;
            ++ns;
            tc_fence_after();
            const uint32_t so = (k.s * P::TILE) >> 4;
            if (one) {
                mma_scores<NB, TAIL>(tmem, q, qtl, r + so, rtl + so);
                tc_commit(m.s_full);
            }
            __syncwarp();
            return true;
        };
        const auto issue_dp = [&](int i, bool last) -> bool {
            const Slot v = second(i);
            if ((nd > 0 && !warp_wait(m.d_read, (nd - 1) & 1, abort_flag)) || !warp_wait(m.full + 8 * v.s, v.ph, abort_flag)) return false;
            ++nd;
            tc_fence_after();
            const uint32_t so = (v.s * P::TILE) >> 4;
            if (one) {
                mma_scores<NB, TAIL>(tmem + 128, d, dtl, r + so, rtl + so);
                tc_commit(m.d_full);
                tc_commit(m.empty + 8 * v.s);
                if (last) tc_commit(m.a_empty);
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        BwdItem it;
        for (int i = 0;; ++i) {
            ok = take_item(m, items, i, lane, abort_flag, it);
            const int n = uniform(it.n), lead = uniform(it.all > 1);
            if (!ok || n < 0) break;
            if (n == 0) continue;
            ok = warp_wait(m.a_full, na & 1, abort_flag);
            ++na;
            if (ok && lead) {
                const Slot o = first(t), v = second(t);
                // V's slot too, into which nothing comes: given back before the producer has had
                // it, its `empty` could pass two phases between two looks of the producer
                ok = (nd == 0 || warp_wait(m.d_read, (nd - 1) & 1, abort_flag)) && warp_wait(m.full + 8 * o.s, o.ph, abort_flag) &&
                     warp_wait(m.full + 8 * v.s, v.ph, abort_flag);
                if (ok) {
                    ++nd;
                    tc_fence_after();
                    const uint32_t so = (o.s * P::TILE) >> 4;
                    if (one) {
                        mma_scores<NB, TAIL>(tmem + 128, d, dtl, r + so, rtl + so);
                        tc_commit(m.d_full);
                        tc_commit(m.empty + 8 * o.s);
                        tc_commit(m.empty + 8 * v.s);
                    }
                    __syncwarp();
                }
            }
            t += lead;
            for (int j = 0; ok && j < n; ++j) ok = issue_s(t + j, j >= 2) && issue_dp(t + j, j + 1 == n);
            t += n;
            if (!ok) break;
        }
        end_issue(one, ok, m.drain, abort_flag, fail);
    } else if (warp == 2) {
        // ---------------- MMA issuer of dQ
        const bool one = elect_one();
        const uint64_t k = sw128_mnmajor_desc(sb + P::R_OFF, T::BLK), ktl = sw32_desc(sb + P::R_OFF + NB * T::BLK);
        bool ok = true;
        int t = 0, ne = 0;            // steps; dS so far
        BwdItem it;
        for (int i = 0;; ++i) {
            ok = take_item(m, items, i, lane, abort_flag, it);
            const int n = uniform(it.n);
            if (!ok || n < 0) break;
            if (n == 0) continue;
            t += uniform(it.all > 1);
            for (int j = 0; j < n; ++j, ++ne) {
                const Slot s = first(t + j);
                if (!warp_wait(m.full + 8 * s.s, s.ph, abort_flag) || !warp_wait(m.e0 + 8 * (ne & 1), (ne >> 1) & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const uint32_t so = (s.s * P::TILE) >> 4;
                if (one) {
                    mma_accumulate<NB, TAIL, kCols / 2>(tmem + 384, tmem + 256 + 64 * (ne & 1), k + so, ktl + so, j == 0);
                    tc_commit(m.empty + 8 * s.s);
                    if (j + 1 == n) tc_commit(m.done);
                }
                __syncwarp();
            }
            if (!ok) break;
            t += n;
        }
        end_issue(one, ok, m.drain2, abort_flag, fail);
    } else if (warp == 3) {
        // ---------------- K rows behind the sequence's end
        uint32_t par = 0;
        int t = 0;
        bool ok = true;
        BwdItem it;
        it.n = 0;
        for (int i = 0;; ++i) {
            ok = take_item(m, items, i, lane, abort_flag, it, it.n);
            if (!ok || it.n < 0) break;
            if (it.n == 0) continue;
            t += (it.all > 1) + it.n;
            const int valid = it.nk - (it.i0 + it.n - 1) * kTile, s = first(t - 1).s;
            if (valid >= kTile) continue;
            ok = long_wait(m.raw + 8 * s, (par >> s) & 1u, abort_flag, it.n);
            if (!ok) break;
            par ^= 1u << s;
            zero_rows<NB, TAIL>(smem + P::R_OFF + s * P::TILE, valid, lane, 32);
            __syncwarp();
            if (lane == 0) mbar_arrive(m.full + 8 * s);
        }
        if (!ok && lane == 0) fail();
    } else {
        // ---------------- elementwise: thread = query row, a quarter of the columns
        const int e = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;    // group, TMEM lane
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint64_t scale2 = f32x2(g.scale_log2, g.scale_log2);
        float* parts = reinterpret_cast<float*>(smem + P::SEL_OFF) + row;
        bool ok = true;
        int ne = 0;                   // dS so far
        uint32_t par = 0;             // next parities: bit 0 s_full, 1 d_full, 2 e1, 3 done
        const auto row_lse = [&](const BwdItem& it) {
            const int i = it.tile * kTile + row;
            return i < it.nq ? g.lse[static_cast<size_t>(it.head) * g.rows_q + it.q0 + i] : -INFINITY;
        };
        float l = 0.f;                // of the coming item's row, where `early`
        bool early = false;
        for (int item = 0;; ++item) {
            const BwdItem& it = items[item % kItems];
            ok = warp_wait(m.item_full + 8 * (item % kItems), (item / kItems) & 1, abort_flag);
            const int n = it.n;
            if (!ok || n < 0) break;
            const bool one_tile = it.all <= 1;
            float l2 = INFINITY;          // L in units of log2
            // columns that the row sees, from the item's first key on.  A row behind the
            // queries is not masked (attention_packed.cu): it keeps what it holds to itself
            int end = 1 << 30;
            {
                const int i = it.tile * kTile + row;
                if (i < it.nq) end = key_end(i, it.nk - it.nq, g.causal_block, it.nk) - it.i0 * kTile;
                if (!early) l = row_lse(it);
                if (l != -INFINITY) l2 = l * 1.4426950408889634f;
            }
            const uint64_t neg_l2 = f32x2(-l2, -l2);
            uint64_t neg_d = 0;
            // -L in units of the raw score; a row that sees nothing has none, nor a D
            const auto write_stats = [&](float delta) {
                if (it.split == 0 && e == 0)
                    write_stat(g.stats + (static_cast<size_t>(it.head) * slots + it.slot) * (kStatBytes / 16), row,
                               l2 == INFINITY ? kNothing : -l2 / g.scale_log2, l2 == INFINITY ? 0.f : -delta);
            };
            if (n == 0) write_stats(0.f);
            if (n > 0 && !one_tile) {
                if (!warp_wait(m.d_full, par >> 1 & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                par ^= 2;
                uint32_t r[32];
                tmem_ld_32x32b_x32(tl + 128 + (warp & 3) * 32, r);
                tmem_wait_ld_r(r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(m.d_read);
                float delta = 0.f;        // the diagonal: column `row` of the row
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c == lane) delta = __uint_as_float(r[c]);
                neg_d = f32x2(-delta, -delta);
                write_stats(delta);
            }
            for (int j = 0; j < n; ++j, ++ne) {
                if (!warp_wait(m.s_full, par & 1, abort_flag)) { ok = false; break; }
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
                if (!warp_wait(m.d_full, par >> 1 & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                tmem_ld_32x32b_x32(tl + 128 + kCols * e, r);
                tmem_wait_ld_r(r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(m.d_read);
                par ^= 3;
                const int see = end - j * kTile - kCols * e;     // columns that this row sees
                if (one_tile) {
                    // D = rowsum(P dP), the four quarters in their order (attention_bwd.cu)
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c < see) sum[c % 4] = fmaf(p[c], __uint_as_float(r[c]), sum[c % 4]);
                    float d = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    parts[kTile * e] = d;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(m.e1);
                    if (!warp_wait(m.e1, par >> 2 & 1, abort_flag)) { ok = false; break; }
                    par ^= 4;
                    tc_fence_after();
                    d = (parts[0] + parts[kTile]) + (parts[2 * kTile] + parts[3 * kTile]);
                    neg_d = f32x2(-d, -d);
                    write_stats(d);
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
                // the last reader of dS's columns, the dQ two steps before, was done before S was
                // issued (one of an item before: before that item's end)
                tmem_st_32x32b_x16(tl + 256 + 64 * (ne & 1) + kCols / 2 * e, w);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(m.e0 + 8 * (ne & 1));
            }
            if (!ok) break;
            // the next item's row statistic is on its way while this one's gradient is written
            // (its load would hold up that item's first step by a microsecond)
            const BwdItem& next = items[(item + 1) % kItems];
            early = __all_sync(0xFFFFFFFFu, mbar_try_wait(m.item_full + 8 * ((item + 1) % kItems), ((item + 1) / kItems) & 1));
            if (early && next.n >= 0) l = row_lse(next);
            if (n > 0) {
                ok = warp_wait(m.done, par >> 3 & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                par ^= 8;
            }
            const int i0 = it.tile * kTile + (warp & 3) * 32;         // the warp's first row
            const size_t at = static_cast<size_t>(it.q0) + i0;
            float* part = g.splits_q == 1
                              ? nullptr
                              : g.part_q + ((static_cast<size_t>(it.split) * g.rows_q + at + lane) * g.heads + it.head) * g.hd;
            for (int c = e; c < (T::HDP + 31) / 32; c += kGroups)
                put_chunk(tl + 384, c, g.dQ + at * g.lddq + it.head * g.hd, g.lddq, it.nq - i0, part, g.hd, lane, n == 0 || end <= 0,
                          g.scale);
            // dQ's columns are read before the e0 that lets the next item's first product write them
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(m.item_empty + 8 * (item % kItems));
        }
        if (!ok && lane == 0) fail();
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
// TMEM and orders of issue as dkv_kernel's (DkvTmem).
template <int NB, bool TAIL>
__global__ void __launch_bounds__(kThreadsB, 1)
    packed_dkv_kernel(const __grid_constant__ PackedBwdMaps maps, const __grid_constant__ PackedBwdArgs g) {
    using P = PackedBwdPlan<NB, TAIL, false>;
    using T = AttnTile<NB, TAIL>;
    using M = DkvTmem<T::HDP>;
    const auto first = [](int i) { return slot_of<P::SLOTS, P::SHARED, false>(i); };
    const auto second = [](int i) { return slot_of<P::SLOTS, P::SHARED, true>(i); };
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(smem);
    const PackedBwdBars m = packed_bars<P::SLOTS>(sb + P::BAR_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + P::TMEM_SLOT_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P::ABORT_OFF);
    BwdItem* items = reinterpret_cast<BwdItem*>(smem + P::ITEM_OFF);
    if (smem - smem_raw + P::USED > P::BYTES) {       // the base of dynamic shared memory is 1 KB aligned
        pdl_wait();
        if (threadIdx.x == 0 && g.err) atomicExch(g.err, 1);
        return;
    }
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        packed_bars_init<P::SLOTS>(m, M::ISSUERS, M::ISSUERS, M::ISSUERS + 1 + 4 * kGroups);
        *abort_flag = 0;
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
    const int slots = packed_slots(g.rows_q, g.batch, kTile);      // of a head's row statistics

    // This grid starts while packed_dq_kernel, whose every CTA has waited for what came
    // before, ends: all inputs are there, and only the row statistics need the wait (the
    // producer's, before the first of them) and what is written (the elementwise warps').
    // The end of that grid is one of its items, however long: the warps that wait for
    // the first statistics, or for room behind items without any, wait for it first, as
    // their own waits are for a step.
    if (warp == 0) {
        // ---------------- producer: K and V, then Q with the row statistics, and dO
        PackedFlight in;
        int t = 0, na = 0;
        const auto take = [&](int x, int y, BwdItem& it) -> bool {
            it.split = x % g.splits_k;
            it.head = y;
            const PackedTile p = packed_tile(g.k_starts, g.batch, g.rows_k, kTile, x / g.splits_k);
            if (p.tile < 0) return false;
            it.tile = p.tile;
            it.k0 = p.row0;
            it.nk = p.n;
            packed_other(g.q_starts, p.b, g.rows_q, g.q_starts == g.k_starts && g.rows_q == g.rows_k, p, it.q0, it.nq);
            it.slot = it.q0 / kTile + p.b;
            // query tiles [first, first + all) of each of the group's heads, one after the other
            it.first = max(0, query_begin(it.tile * kTile, it.nk - it.nq, g.causal_block)) / kTile;
            it.all = max(0, (it.nq + kTile - 1) / kTile - it.first);
            const int steps = it.all * g.group, share = (steps + g.splits_k - 1) / g.splits_k;
            it.i0 = it.split * share;
            it.n = max(0, min(steps, it.i0 + share) - it.i0);
            if (it.n == 0) pdl_wait();
            return true;
        };
        const auto load = [&](const BwdItem& it) -> bool {
            bool ok = true;
            if (lane == 0) {
                const int row = it.k0 + it.tile * kTile;
                // K and V are free after the last dP of the item before
                ok = na == 0 || mbar_wait(m.a_empty, (na - 1) & 1, abort_flag);
                if (ok) {
                    mbar_arrive_expect_tx(m.a_full, 2 * P::TILE);
                    load_tile<NB, TAIL>(sb + P::A0_OFF, &maps.k, &maps.kt, it.head, row, 0, m.a_full);
                    load_tile<NB, TAIL>(sb + P::A1_OFF, &maps.v, &maps.vt, it.head, row, 0, m.a_full);
                    ++na;
                }
                int h = it.head * g.group + it.i0 / it.all, qt = it.first + it.i0 % it.all;
                for (int j = 0; ok && j < it.n; ++j) {
                    const Slot q = first(t + j), d = second(t + j);
                    const bool raw = it.nq - qt * kTile < kTile;
                    ok = mbar_wait(m.empty + 8 * q.s, q.ph ^ 1, abort_flag);
                    if (!ok) break;
                    const uint32_t fq = in.begin(m, q, raw);
                    mbar_arrive_expect_tx(fq, P::TILE + kStatBytes);
                    load_tile<NB, TAIL>(sb + P::R_OFF + q.s * P::TILE, &maps.q, &maps.qt, h, it.q0 + qt * kTile, 0, fq);
                    if (t + j == 0) pdl_wait();
                    bulk_load(sb + P::STAT_OFF + (t + j) % P::STATS * kStatBytes,
                              g.stats + (static_cast<size_t>(h) * slots + it.slot + qt) * (kStatBytes / 16), kStatBytes, fq);
                    ok = mbar_wait(m.empty + 8 * d.s, d.ph ^ 1, abort_flag);
                    if (!ok) break;
                    const uint32_t fd = in.begin(m, d, raw);
                    mbar_arrive_expect_tx(fd, P::TILE);
                    load_tile<NB, TAIL>(sb + P::R_OFF + d.s * P::TILE, &maps.d, &maps.dt, h, it.q0 + qt * kTile, 0, fd);
                    if (++qt == it.first + it.all) {
                        qt = it.first;
                        ++h;
                    }
                }
            }
            t += it.n;
            return __shfl_sync(0xFFFFFFFFu, ok, 0);
        };
        const bool ok = produce(m, items, sb + P::ANSWER_OFF, lane, abort_flag, take, load);
        if (lane == 0) {
            if (!ok) fail();
            if (*abort_flag) {
                if (na > 0) mbar_wait(m.a_full, (na - 1) & 1, nullptr);
                in.drain<P::SLOTS>(m);
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
        pdl_wait();
        const auto full = [&](Slot s) { return warp_wait(m.full + 8 * s.s, s.ph, abort_flag); };
        // a slot is free when both products that read it are done: with one
        // issuer the later one's completion says so, with two each says its own
        const auto issue_s = [&](int i) -> bool {
            const Slot s = first(i);
            if (!full(s)) return false;
            tc_fence_after();
            const uint32_t so = (s.s * P::TILE) >> 4;
            if (one) {
                mma_scores<NB, TAIL>(tmem, k, ktl, r + so, rtl + so);
                tc_mma_f16(tmem, sel, stat + ((i % P::STATS * kStatBytes) >> 4), id, 1u);
                tc_commit(m.s_full);
                if (M::ISSUERS == 2) tc_commit(m.empty + 8 * s.s);
            }
            __syncwarp();
            return true;
        };
        const auto issue_dp = [&](int i, bool last) -> bool {
            const Slot s = second(i);
            // the statistics came with Q_i; one issuer has waited for it
            if ((M::ISSUERS == 2 && !full(first(i))) || !full(s)) return false;
            tc_fence_after();
            const uint32_t so = (s.s * P::TILE) >> 4;
            if (one) {
                mma_scores<NB, TAIL>(tmem + 128, v, vtl, r + so, rtl + so);
                tc_mma_f16(tmem + 128, sel + (kStatBytes >> 4), stat + ((i % P::STATS * kStatBytes) >> 4), id, 1u);
                tc_commit(m.d_full);
                if (M::ISSUERS == 2) tc_commit(m.empty + 8 * s.s);
                if (M::ISSUERS == 1 && last) tc_commit(m.a_empty);
            }
            __syncwarp();
            return true;
        };
        const auto issue_dv = [&](int i, bool start, bool end) -> bool {
            const Slot s = second(i);
            if (!full(s) || !warp_wait(m.e0, i & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (s.s * P::TILE) >> 4;
            if (one) {
                mma_accumulate<NB, TAIL, M::P_APART ? kCols / 2 : kCols>(tmem + M::DV_COL, tmem + M::P_COL, rmn + so, rtl + so, start);
                tc_commit(m.empty + 8 * s.s);
                if (end) tc_commit(m.done);
            }
            __syncwarp();
            return true;
        };
        const auto issue_dk = [&](int i, bool start, bool end) -> bool {
            const Slot s = first(i);
            if (!warp_wait(m.e1, i & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (s.s * P::TILE) >> 4;
            if (one) {
                mma_accumulate<NB, TAIL, M::DS_APART ? kCols / 2 : kCols>(tmem + M::DK_COL, tmem + M::DS_COL, rmn + so, rtl + so, start);
                tc_commit(m.empty + 8 * s.s);
                if (end) tc_commit(m.done);
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        int t = 0, na = 0;
        BwdItem it;
        for (int item = 0;; ++item) {
            ok = take_item(m, items, item, lane, abort_flag, it);
            const int n = uniform(it.n);
            if (!ok || n < 0) break;
            if (n == 0) continue;
            ok = warp_wait(m.a_full, na & 1, abort_flag);
            ++na;
            if constexpr (M::ISSUERS == 1) {
                // written out: through the calls above a step takes 6% longer
                ok = ok && issue_s(t) && issue_dp(t, n == 1);
                for (int i = t; ok && i < t + n; ++i) {
                    const int st = first(i).s, sd = second(i).s;
                    const uint32_t so = (st * P::TILE) >> 4, sdo = (sd * P::TILE) >> 4;
                    const bool more = i + 1 < t + n;
                    if (!warp_wait(m.e0, i & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    if (one) {
                        mma_accumulate<NB, TAIL, kCols>(tmem + M::DV_COL, tmem + M::P_COL, rmn + sdo, rtl + sdo, i == t);
                        tc_commit(m.empty + 8 * sd);
                    }
                    __syncwarp();
                    if (more && !issue_s(i + 1)) { ok = false; break; }
                    if (!warp_wait(m.e1, i & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    if (one) {
                        mma_accumulate<NB, TAIL, kCols>(tmem + M::DK_COL, tmem + M::DS_COL, rmn + so, rtl + so, i == t);
                        tc_commit(m.empty + 8 * st);
                    }
                    __syncwarp();
                    if (more && !issue_dp(i + 1, i + 2 == t + n)) { ok = false; break; }
                }
                if (one && ok) tc_commit(m.done);
                __syncwarp();
            } else if (warp == 1) {
                // S_{i+1} takes S_i's place once that is read; where P_i lies there, after dV_i
                // (of the item before: its last S is read before its last dV is issued)
                ok = ok && issue_s(t);
                for (int i = t; ok && i < t + n; ++i) {
                    const bool more = i + 1 < t + n;
                    if (M::P_APART && more) ok = warp_wait(m.s_read, i & 1, abort_flag) && issue_s(i + 1);
                    ok = ok && issue_dv(i, i == t, !more);
                    if (!M::P_APART && more) ok = ok && issue_s(i + 1);
                }
                // K and V have been read by S (complete before dV's operand was) and dP
                if (M::P_APART) ok = ok && warp_wait(m.s_read, (t + n - 1) & 1, abort_flag);
            } else {
                // likewise dP_{i+1}, dS_i and dK_i
                ok = ok && issue_dp(t, false);
                for (int i = t; ok && i < t + n; ++i) {
                    const bool more = i + 1 < t + n;
                    if (M::DS_APART && more) ok = warp_wait(m.d_read, i & 1, abort_flag) && issue_dp(i + 1, false);
                    ok = ok && issue_dk(i, i == t, !more);
                    if (!M::DS_APART && more) ok = ok && issue_dp(i + 1, false);
                }
                if (M::DS_APART) ok = ok && warp_wait(m.d_read, (t + n - 1) & 1, abort_flag);
                // the e1 before the last dK says that S and dP of the item are complete
                if (one && ok) mbar_arrive(m.a_empty);
                __syncwarp();
            }
            if (!ok) break;
            t += n;
        }
        end_issue(one, ok, warp == 1 ? m.drain : m.drain2, abort_flag, fail);
    } else if (warp == 3) {
        // ---------------- Q and dO rows behind the sequence's end
        uint32_t par = 0;
        int t = 0;
        bool ok = true;
        BwdItem it;
        it.n = 0;
        pdl_wait();
        for (int item = 0; ok; ++item) {
            ok = take_item(m, items, item, lane, abort_flag, it, it.n);
            if (!ok || it.n < 0) break;
            const int valid = it.nq - (it.first + it.all - 1) * kTile;
            if (it.n > 0 && valid < kTile) {
                // the steps that end a head's query tiles
                for (int i = it.all - 1 - it.i0 % it.all; ok && i < it.n; i += it.all) {
                    const Slot q = first(t + i), d = second(t + i);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int s = u ? d.s : q.s;
                        ok = ok && long_wait(m.raw + 8 * s, (par >> s) & 1u, abort_flag, it.all);
                        if (!ok) break;
                        par ^= 1u << s;
                        zero_rows<NB, TAIL>(smem + P::R_OFF + s * P::TILE, valid, lane, 32);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(m.full + 8 * s);
                    }
                }
            }
            t += it.n;
        }
        if (!ok && lane == 0) fail();
    } else if (warp >= 4) {
        // ---------------- elementwise: thread = key, a quarter of the query columns
        const int e = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;    // group, TMEM lane
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t ts = tl + kCols * e;
        const uint64_t scale2 = f32x2(g.scale_log2, g.scale_log2);
        bool ok = true;
        int t = 0, na = 0;
        pdl_wait();
        for (int item = 0;; ++item) {
            const BwdItem& it = items[item % kItems];
            ok = warp_wait(m.item_full + 8 * (item % kItems), (item / kItems) & 1, abort_flag);
            const int n = it.n;
            if (!ok || n < 0) break;
            // queries that see the row's key: [begin, nq), counted from the group of columns on.
            // A row behind the keys is not masked: it keeps what it holds to itself
            const int off = it.nk - it.nq;
            const int key = it.tile * kTile + row;
            const int begin = key < it.nk ? query_begin(key, off, g.causal_block) : 0;
            const int nq = it.nq, q_end = it.first + it.all;
            int qt = n > 0 ? it.first + it.i0 % it.all : 0;
            for (int i = t; i < t + n; ++i) {
                const int lo = begin - (qt * kTile + kCols * e), hi = nq - (qt * kTile + kCols * e);
                const bool cut = __any_sync(0xFFFFFFFFu, lo > 0 || hi < kCols);
                if (++qt == q_end) qt = it.first;
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
                    // the last reader of its columns, the dV before, releases its dO slot when done
                    const Slot s = second(i - 1);
                    if (i > t && !warp_wait(m.empty + 8 * s.s, s.ph, abort_flag)) { ok = false; break; }
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
                    // the last reader of its columns, the dK before, releases its Q slot when done
                    const Slot s = first(i - 1);
                    if (i > t && !warp_wait(m.empty + 8 * s.s, s.ph, abort_flag)) { ok = false; break; }
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
            if (!ok) break;
            t += n;
            if (n > 0) {
                ok = warp_wait(m.done, na & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                ++na;
            }
            // even groups bring dV, odd ones dK
            const bool k = e & 1;
            const int i0 = it.tile * kTile + (warp & 3) * 32;         // the warp's first row
            const size_t at = static_cast<size_t>(it.k0) + i0;
            float* part = g.splits_k == 1 ? nullptr
                                          : (k ? g.part_k : g.part_v) +
                                                ((static_cast<size_t>(it.split) * g.rows_k + at + lane) * g.kv_heads + it.head) * g.hd;
            __nv_bfloat16* out = (k ? g.dK + at * g.lddk : g.dV + at * g.lddv) + it.head * g.hd;
            for (int c = e >> 1; c < (T::HDP + 31) / 32; c += kGroups / 2)
                put_chunk(tl + (k ? M::DK_COL : M::DV_COL), c, out, k ? g.lddk : g.lddv, it.nk - i0, part, g.hd, lane,
                          n == 0 || begin >= it.nq, k ? g.scale : 1.f);
            // read before the e0 and e1 that let the next item's first products write there
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(m.item_empty + 8 * (item % kItems));
        }
        if (!ok && lane == 0) fail();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Adds the parts of a split gradient in order and rounds once; rows of no sequence stay
// as they are.  One thread eight columns; bound by reading the parts.
struct PackedJoinOne {
    const float* part;
    __nv_bfloat16* out;
    int splits, ld, c8;              // c8: pieces of 8 columns a row
    int rows;
    const int* starts;
};
struct PackedJoinArgs {
    PackedJoinOne one[3];
    int batch;
};

__global__ void __launch_bounds__(256) packed_bwd_join_kernel(const __grid_constant__ PackedJoinArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        const PackedJoinOne& j = a.one[t];
        const long long n = static_cast<long long>(j.rows) * j.c8;
        if (i >= n) {
            i -= n;
            continue;
        }
        const long long row = i / j.c8;
        if (row < seq_start(j.starts, 0, j.rows) || row >= seq_start(j.starts, a.batch, j.rows)) return;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        const float4* p = reinterpret_cast<const float4*>(j.part) + 2 * i;
#pragma unroll 4
        for (int k = 0; k < j.splits; ++k, p += 2 * n) {
            const float4 u = p[0], v = p[1];
            x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
            y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
        }
        reinterpret_cast<uint4*>(j.out + row * j.ld)[i - row * j.c8] =
            make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
        return;
    }
}

// Splits and workspace, from the sizes alone.
//   dQ: query tiles that do not fill the SMs share their keys, four key tiles of a mean
//     sequence or more to an item.
//   dK, dV: likewise over the group's query tiles.
struct PackedBwdSplit {
    int q, k;
    size_t part_q, part_k, part_v, total;      // byte offsets
};

PackedBwdSplit packed_bwd_split(const dlo_attn_packed& a) {
    const long long tq = packed_slots(a.rows_q, a.batch, kTile), tk = packed_slots(a.rows_k, a.batch, kTile);
    const long long qt = a.rows_q / a.batch / kTile + 1, kt = a.rows_k / a.batch / kTile + 1;       // of a mean sequence
    const auto fill = [](long long items, long long work) {
        long long s = kGb300Sms / items;
        if (s > work / 4) s = work / 4;
        return static_cast<int>(s < 1 ? 1 : s > 64 ? 64 : s);
    };
    PackedBwdSplit b;
    b.q = fill(tq * a.heads, kt);
    b.k = fill(tk * a.kv_heads, qt * (a.heads / a.kv_heads));
    const size_t rq = static_cast<size_t>(a.rows_q) * a.heads * a.head_dim * sizeof(float);
    const size_t rk = static_cast<size_t>(a.rows_k) * a.kv_heads * a.head_dim * sizeof(float);
    b.part_q = static_cast<size_t>(tq) * a.heads * kStatBytes;
    b.part_k = b.part_q + (b.q > 1 ? b.q * rq : 0);
    b.part_v = b.part_k + (b.k > 1 ? b.k * rk : 0);
    b.total = b.part_v + (b.k > 1 ? b.k * rk : 0);
    return b;
}

template <int NB, bool TAIL>
cudaError_t run_packed_bwd(const PackedBwdMaps& maps, const PackedBwdArgs& g, cudaStream_t s, unsigned long long* launches) {
    using PQ = PackedBwdPlan<NB, TAIL, true>;
    using PK = PackedBwdPlan<NB, TAIL, false>;
    constexpr auto dq = packed_dq_kernel<NB, TAIL>;
    constexpr auto dkv = packed_dkv_kernel<NB, TAIL>;
    static unsigned long long set[2] = {0, 0};
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(dq), PQ::BYTES, &set[0]); e != cudaSuccess) return e;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(dkv), PK::BYTES, &set[1]); e != cudaSuccess) return e;
    cudaError_t e = launch_k(dq, dim3(packed_slots(g.rows_q, g.batch, kTile) * g.splits_q, g.heads), kThreadsB, PQ::BYTES, s, maps, g);
    ++*launches;
    if (e != cudaSuccess) return e;
    e = launch_k(dkv, dim3(packed_slots(g.rows_k, g.batch, kTile) * g.splits_k, g.kv_heads), kThreadsB, PK::BYTES, s, maps, g);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t attention_packed_bwd_workspace(const dlo_attn_packed& a) { return packed_bwd_split(a).total; }

cudaError_t launch_attention_packed_bwd(const dlo_attn_packed& a, const void* Q, const void* K, const void* V, const void* O,
                                        const float* lse, const void* dO, void* dQ, void* dK, void* dV, void* ws, int* err,
                                        cudaStream_t s, unsigned long long* launches) {
    const int hd = a.head_dim;
    PackedBwdArgs g = {};
    g.q_starts = a.q_starts;
    g.k_starts = a.k_starts;
    g.batch = a.batch;
    g.rows_q = a.rows_q;
    g.rows_k = a.rows_k;
    g.hd = hd;
    g.heads = a.heads;
    g.kv_heads = a.kv_heads;
    g.group = a.heads / a.kv_heads;
    g.causal_block = a.causal_block < a.rows_k ? a.causal_block : a.rows_k;
    g.scale = 1.f / sqrtf(static_cast<float>(hd));
    g.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(hd));
    g.lse = lse;
    g.stats = static_cast<uint4*>(ws);
    const PackedBwdSplit split = packed_bwd_split(a);
    uint8_t* base = static_cast<uint8_t*>(ws);
    g.splits_q = split.q;
    g.splits_k = split.k;
    g.part_q = reinterpret_cast<float*>(base + split.part_q);
    g.part_k = reinterpret_cast<float*>(base + split.part_k);
    g.part_v = reinterpret_cast<float*>(base + split.part_v);
    g.dQ = static_cast<__nv_bfloat16*>(dQ);
    g.dK = static_cast<__nv_bfloat16*>(dK);
    g.dV = static_cast<__nv_bfloat16*>(dV);
    g.lddq = a.lddq;
    g.lddk = a.lddk;
    g.lddv = a.lddv;
    g.err = err;
    PackedBwdMaps m;
    const CUtensorMapSwizzle w128 = CU_TENSOR_MAP_SWIZZLE_128B, w32 = CU_TENSOR_MAP_SWIZZLE_32B;
    const bool tail = hd > 64 && hd <= 80;
    auto map = [&](CUtensorMap* main, CUtensorMap* tl, const void* p, int rows, int heads, int ld) {
        if (!make_map4(main, p, 1, rows, heads, hd, ld, 64, w128)) return false;
        if (tail) return make_map4(tl, p, 1, rows, heads, hd, ld, 16, w32);
        *tl = *main;
        return true;
    };
    if (!map(&m.q, &m.qt, Q, a.rows_q, a.heads, a.ldq) || !map(&m.k, &m.kt, K, a.rows_k, a.kv_heads, a.ldk) ||
        !map(&m.v, &m.vt, V, a.rows_k, a.kv_heads, a.ldv) || !map(&m.d, &m.dt, dO, a.rows_q, a.heads, a.lddo) ||
        !map(&m.o, &m.ot, O, a.rows_q, a.heads, a.ldo))
        return cudaErrorInvalidValue;
    cudaError_t e = hd <= 64 ? run_packed_bwd<1, false>(m, g, s, launches)
                    : tail   ? run_packed_bwd<1, true>(m, g, s, launches)
                             : run_packed_bwd<2, false>(m, g, s, launches);
    if (e != cudaSuccess || (split.q == 1 && split.k == 1)) return e;
    const int cq = a.heads * hd / 8, ck = a.kv_heads * hd / 8;
    const PackedJoinArgs j = {{{g.part_q, g.dQ, split.q, a.lddq, cq, split.q > 1 ? a.rows_q : 0, a.q_starts},
                               {g.part_k, g.dK, split.k, a.lddk, ck, split.k > 1 ? a.rows_k : 0, a.k_starts},
                               {g.part_v, g.dV, split.k, a.lddv, ck, split.k > 1 ? a.rows_k : 0, a.k_starts}},
                              a.batch};
    const long long n = static_cast<long long>(j.one[0].rows) * cq + 2ll * j.one[1].rows * ck;
    e = launch_k(packed_bwd_join_kernel, static_cast<unsigned>((n + 255) / 256), 256, 0, s, j);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dlo
