// Attention over packed sequences, forward: O = softmax(Q K^T / sqrt(hd)) V within
// each sequence, with row statistics.
//
// The products and the softmax are those of attention_tc.cu: S = Q K^T into tensor
// memory, one thread a query row for the softmax, P (bf16) back over S's columns as
// the A operand of O += P V.  What differs is that tiles are many and short here (a
// tile ends with its sequence, and a sequence of 300 tokens has three tiles of three
// key tiles each), so a CTA's start and end (~4 us: launch, tensor memory, the first
// loads; the last product, O's way out) would cost as much as its products.  So a CTA
// stays: while it works on one tile, its producer warp takes over the index of a CTA
// that has not been launched (cta_request), finds that one's sequence and tile
// (packed_tile), and loads its Q, K and V as the ring gets room; S of the next tile
// runs while the softmax warps write the last one's O.
//
// One item of work: a tile of 128 rows (128 / gh queries of gh heads that share their
// keys), or a part of its keys.  A CTA of the grid is a tile of queries; where that leaves
// SMs idle or sequences unequal (single queries over long caches), it is a run of `per`
// key tiles of a sequence, with an item for every tile of that sequence's queries: then
// the long sequences have the many CTAs, and a second launch joins their parts.  Six warps:
//   warp 0      producer: finds items, writes them to a ring of two in shared memory, TMA
//   warp 1      MMA issuer (one elected lane).  The last V tile of a sequence also
//               holds the next one's rows; those that the last step of 16 keys reads
//               become zero first (0 x infinity)
//   warps 2..5  softmax, one thread a row, and O from tensor memory to its row
// Barriers and buffers run on through the items: tile j of an item that began with c
// tiles behind it is tile c + j.
//
// DUO (head dims up to 80): two CTAs on an SM, one S buffer each, as there (24 images of
// 16 x 72: 51.5 us, 54.4 with one CTA an SM).
//
// What bounds it.  Long sequences: the products and the softmax, 0.85 us a tile at head
// dim 128, as in attention_tc.cu (8192 tokens, 40 heads: 896 us, 1534 TFLOP/s).  Short ones:
// an item of 4 tiles takes 5.9 us, 2.5 of them its end, where the softmax warps wait for the
// last product (0.3), write O (1.6) and begin the next (16 x 512 tokens, 40 heads of 128:
// 100 us, tensor pipe 34% active; a CTA an item took 150).  Single queries: memory (64 x
// 4096 keys, 8 key/value heads of 128: 168 us, 6.4 TB/s, 0.94 of the measured copy); with
// unequal lengths the last items (24 sequences of 422 to 7173 keys: 72 us, 5.6 TB/s).
// Measured and not kept: O in two buffers and four warps more that write it (12 warps leave
// 168 registers a thread: 109 us where 100; with setmaxnreg the compiler spills 1232 bytes),
// two chunks of O at once (104).
//
// Every wait is bounded; one that runs out sets the error word and every role leaves
// its loops, with loads, requests and MMAs in flight waited for.
#include "attention.cuh"

namespace dlo {

namespace {

constexpr int TQ = 128;          // rows of an item (MMA M, TMEM lanes)
constexpr int TK = 128;          // keys per tile
constexpr int kThreadsP = 192;
constexpr int kItems = 2;        // items in shared memory

struct PackedArgs {
    __nv_bfloat16* O;
    float* lse;                  // [heads, rows_q]
    float *po, *pl;              // parts > 1: [parts][heads][rows_q][hd] and [..][rows_q]
    int* count;                  // parts > 1: [heads][rows_q] parts of each row
    const int *q_starts, *k_starts;
    int batch, rows_q, rows_k, hd, heads, group, gh, causal_block, ldo;
    int per, parts;              // key tiles of a part; parts of a row at most (1: CTAs are query tiles)
    float scale_log2;
    int* err;
};

struct PackedMaps {
    CUtensorMap q, k, v;         // 64-column boxes, 128-byte swizzle
    CUtensorMap qt, kt, vt;      // 16-column tail boxes, 32-byte swizzle
};

// One item, as the producer leaves it for the others.
struct Item {
    int n;                       // key tiles; 0: none of its rows sees a key; < 0: no more items
    int t0;                      // the first of them
    int q0, nq, qi;              // the sequence's first row and queries; the item's first query in it
    int k0, nk;
    int head;
    int part, parts;             // which part of its rows' keys, of how many
    int pad[2];
};

template <int NB, bool TAIL, bool DUO>
struct PackedPlan {
    static constexpr int HDP = AttnTile<NB, TAIL>::HDP;
    static constexpr int BLK = AttnTile<NB, TAIL>::BLK;
    static constexpr int TILE = AttnTile<NB, TAIL>::BYTES;
    static constexpr int STAGES = DUO ? 2 : (TILE * 7 + 2048 <= 227 * 1024) ? 3 : 2;
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = Q_OFF + TILE;
    static constexpr int V_OFF = K_OFF + STAGES * TILE;
    static constexpr int ITEM_OFF = V_OFF + STAGES * TILE;
    static constexpr int ANSWER_OFF = ITEM_OFF + kItems * static_cast<int>(sizeof(Item));
    static constexpr int BAR_OFF = ANSWER_OFF + 16;
    // q_full, q_empty, p_full, pv_done, drain, answered, s_full[2], item_full[2], item_empty[2], kv_full, k_empty, v_empty
    static constexpr int NBARS = 12 + 3 * STAGES;
    static constexpr int TMEM_SLOT_OFF = BAR_OFF + NBARS * 8;
    static constexpr int ABORT_OFF = TMEM_SLOT_OFF + 4;
    static constexpr int USED = ABORT_OFF + 4 + 1024;
    // as in attention_tc.cu: one CTA per SM owns all 512 TMEM columns, or two 256 each
    static constexpr int BYTES = DUO ? USED : (USED > 118784 ? USED : 118784);
    static constexpr uint32_t TMEM_COLS = DUO ? 256 : 512;
    static constexpr int SBUF = DUO ? 1 : 2;
    static constexpr uint32_t O_COL = SBUF * 128;
    static_assert(BYTES <= 227 * 1024, "packed attention shared memory plan exceeds 227 KB");
    static_assert(!DUO || (NB == 1 && 2 * (USED + 1024) <= 228 * 1024), "DUO: two CTAs per SM");
    static_assert(ITEM_OFF % 16 == 0 && sizeof(Item) % 16 == 0, "16-byte answers");
};

// The items of CTA (x, y) of the grid: query tiles [tile, end) of a sequence, part
// it.part of each one's keys.  By a whole warp.
struct Work {
    Item it;
    int tile, end;
};

__device__ __forceinline__ void find_work(const PackedArgs& g, int x, int y, Work& w) {
    const int tq = TQ / g.gh;
    const bool same = g.q_starts == g.k_starts && g.rows_q == g.rows_k;
    Item& it = w.it;
    it.head = y * g.gh;
    it.part = 0;
    w.tile = w.end = 0;
    if (g.parts == 1) {
        // with a causal mask the last query tiles have the most keys: first
        const PackedTile p = packed_tile(g.q_starts, g.batch, g.rows_q, tq, packed_slots(g.rows_q, g.batch, tq) - 1 - x);
        if (p.tile < 0) return;
        it.q0 = p.row0;
        it.nq = p.n;
        packed_other(g.k_starts, p.b, g.rows_k, same, p, it.k0, it.nk);
        w.tile = p.tile;
        w.end = p.tile + 1;
    } else {
        // heads side by side: CTAs that run at once read the same rows of K and V
        const int groups = g.heads / g.gh;
        it.head = x % groups * g.gh;
        x /= groups;
        // a sequence without keys has one slot too, for the zeros of its rows
        const PackedTile p = packed_tile(g.k_starts, g.batch, g.rows_k, TK * g.per, x);
        if (p.tile < 0 && (p.n > 0 || x != p.row0 / (TK * g.per) + p.b)) return;
        it.k0 = p.row0;
        it.nk = p.n;
        it.part = max(p.tile, 0);
        packed_other(g.q_starts, p.b, g.rows_q, same, p, it.q0, it.nq);
        w.end = (it.nq + tq - 1) / tq;
    }
}

// The item of query tile `tile`; false: its rows have fewer parts.
__device__ __forceinline__ bool make_item(const PackedArgs& g, int tile, Item& it) {
    const int tq = TQ / g.gh;
    it.qi = tile * tq;
    const int n = (key_end(min(it.qi + tq, it.nq) - 1, it.nk - it.nq, g.causal_block, it.nk) + TK - 1) / TK;
    it.parts = g.parts == 1 ? 1 : max(1, (n + g.per - 1) / g.per);
    const int share = (n + it.parts - 1) / it.parts;
    it.t0 = it.part * share;
    it.n = max(0, min(n, it.t0 + share) - it.t0);
    return it.part < it.parts;
}

// The end of an item for one row of the softmax: O / l (or its part) and the row
// statistic.  o: O's first tensor memory column, read whether there were keys or not (an
// array that one path leaves unset stays in registers all through the loop before).
template <int HDP>
__device__ __forceinline__ void put_rows(const PackedArgs& g, const Item& it, uint32_t o, int row, float m, float l) {
    // l = 0 where the row sees no key: zeros, whatever its accumulator holds
    const bool none = l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    const int head = it.head + row % g.gh, i = it.qi + row / g.gh;
    const bool live = row < TQ / g.gh * g.gh && i < it.nq;   // else a row without a query
    const size_t plane = static_cast<size_t>(g.heads) * g.rows_q;
    const size_t at = static_cast<size_t>(head) * g.rows_q + it.q0 + i, part = it.part * plane + at;
    const bool whole = it.parts == 1;
    // natural logarithm of the sum of exp(scores)
    const float lse = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    if (live) {
        (whole ? g.lse : g.pl)[whole ? at : part] = lse;
        if (g.parts > 1 && it.part == 0) g.count[at] = it.parts;
    }
    // where rows (lane & ~3) + 0..3 of the warp begin
    __nv_bfloat16* to[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = (row & ~3) + k, q = it.qi + r / g.gh;
        to[k] = r < TQ / g.gh * g.gh && q < it.nq ? g.O + (static_cast<size_t>(it.q0) + q) * g.ldo + (it.head + r % g.gh) * g.hd : nullptr;
    }
#pragma unroll 1
    for (int k = 0; k < (HDP + 31) / 32; ++k) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(o + k * 32, r);
        tmem_wait_ld_r(r);
        if (none) {
#pragma unroll
            for (int u = 0; u < 32; ++u) r[u] = 0;
        }
        if (whole) {
            uint32_t w[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) w[u] = pack_bf16x2(__uint_as_float(r[2 * u]) * inv, __uint_as_float(r[2 * u + 1]) * inv);
            put_rows32(w, k * 32, g.hd, row & 31, [&](int i) { return to[i]; });
        } else if (live && !none) {      // the join does not read a part without a key
#pragma unroll
            for (int u = 0; u < 32; u += 4)
                if (k * 32 + u < g.hd)
                    *reinterpret_cast<float4*>(g.po + part * g.hd + k * 32 + u) =
                        make_float4(__uint_as_float(r[u]) * inv, __uint_as_float(r[u + 1]) * inv, __uint_as_float(r[u + 2]) * inv,
                                    __uint_as_float(r[u + 3]) * inv);
        }
    }
}

template <int NB, bool TAIL, bool DUO>
__global__ void __launch_bounds__(kThreadsP, DUO ? 2 : 1)
    packed_fwd_kernel(const __grid_constant__ PackedMaps maps, const __grid_constant__ PackedArgs g) {
    using P = PackedPlan<NB, TAIL, DUO>;
    constexpr int HDP = P::HDP, NS = P::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar = sb + P::BAR_OFF;
    const uint32_t q_full = bar, q_empty = bar + 8, p_full = bar + 16, pv_done = bar + 24, drain = bar + 32, answered = bar + 40;
    const uint32_t s_full = bar + 48, item_full = bar + 64, item_empty = bar + 80;
    const uint32_t kv_full = bar + 96, k_empty = kv_full + 8 * NS, v_empty = k_empty + 8 * NS;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + P::TMEM_SLOT_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P::ABORT_OFF);
    Item* items = reinterpret_cast<Item*>(smem + P::ITEM_OFF);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int tq = TQ / g.gh;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(p_full, 4);
        mbar_init(pv_done, 1);
        mbar_init(drain, 1);
        mbar_init(answered, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(item_full + 8 * i, 1);
            mbar_init(item_empty + 8 * i, 5);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(kv_full + 8 * i, 1);
            mbar_init(k_empty + 8 * i, 1);
            mbar_init(v_empty + 8 * i, 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
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
        if (g.err) atomicExch(g.err, 1);
    };
    // the i-th item, by a warp that then gives its place back
    const auto next_item = [&](int i, Item& it) -> bool {
        if (!warp_wait(item_full + 8 * (i % kItems), (i / kItems) & 1, abort_flag)) return false;
        it = items[i % kItems];
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty + 8 * (i % kItems));
        return true;
    };

    if (warp == 0) {
        // ---------------- producer
        bool ok = true;
        uint32_t on = 0, par = 0;     // K/V loads in flight, and the parity of each one's phase
        int c = 0, nq = 0, ni = 0;    // key tiles, items with keys, items so far
        const auto put = [&](const Item& it) -> bool {
            const bool room = warp_wait(item_empty + 8 * (ni % kItems), ((ni / kItems) & 1) ^ 1, abort_flag);
            if (room && lane == 0) {
                items[ni % kItems] = it;
                mbar_arrive(item_full + 8 * (ni % kItems));
            }
            ++ni;
            return room;
        };
        int x = blockIdx.x, y = blockIdx.y;
        for (int k = 0;; ++k) {
            Work w;
            find_work(g, x, y, w);
            Item& it = w.it;
            for (; ok && w.tile < w.end; ++w.tile) {
                if (!make_item(g, w.tile, it)) continue;
                ok = put(it);
                if (ok && it.n > 0 && lane == 0) {
                    // Q's place is free after the last S of the item before
                    ok = nq == 0 || mbar_wait(q_empty, (nq - 1) & 1, abort_flag);
                    if (ok) {
                        // with 128 % gh != 0 the last rows stay empty
                        mbar_arrive_expect_tx(q_full, P::TILE / TQ * (tq * g.gh));
                        load_tile<NB, TAIL>(sb + P::Q_OFF, &maps.q, &maps.qt, it.head, it.q0 + it.qi, 0, q_full);
                        ++nq;
                    }
                    for (int j = 0; ok && j < it.n; ++j) {
                        const int st = (c + j) % NS, row = it.k0 + (it.t0 + j) * TK, hk = it.head / g.group;
                        const uint32_t ph = ((c + j) / NS) & 1;
                        // the stage's K is free after S_{c+j-NS}, its V after PV_{c+j-NS}
                        ok = mbar_wait(k_empty + 8 * st, ph ^ 1, abort_flag) && mbar_wait(v_empty + 8 * st, ph ^ 1, abort_flag);
                        if (!ok) break;
                        mbar_arrive_expect_tx(kv_full + 8 * st, 2 * P::TILE);
                        load_tile<NB, TAIL>(sb + P::K_OFF + st * P::TILE, &maps.k, &maps.kt, hk, row, 0, kv_full + 8 * st);
                        load_tile<NB, TAIL>(sb + P::V_OFF + st * P::TILE, &maps.v, &maps.vt, hk, row, 0, kv_full + 8 * st);
                        on |= 1u << st;
                        par = (par & ~(1u << st)) | (ph << st);
                    }
                }
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                c += it.n;
            }
            // the next one, asked for only now: a CTA that asks early keeps the item from others
            // that are done sooner (24 single queries over 98304 keys: 94 us, 128 when it asked at the
            // item's start; steps ahead of the last load measured the same as behind it).  The
            // answer has to land before this CTA may end
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(answered, 16);
                cta_request(sb + P::ANSWER_OFF, answered);
            }
            if (!warp_wait(answered, k & 1, nullptr)) {
                ok = false;
                break;
            }
            int more = 0;
            if (lane == 0) {
                more = cta_answer(sb + P::ANSWER_OFF, x, y);
                fence_proxy_async_smem();       // read before the next answer is written
            }
            more = __shfl_sync(0xFFFFFFFFu, more, 0);
            if (!more) break;
            x = __shfl_sync(0xFFFFFFFFu, x, 0);
            y = __shfl_sync(0xFFFFFFFFu, y, 0);
        }
        if (ok) {
            Item end = {};
            end.n = -1;
            ok = put(end);
        }
        if (lane == 0) {
            if (!ok) fail();
            if (*abort_flag) {
                if (nq > 0) mbar_wait(q_full, (nq - 1) & 1, nullptr);
                for (int i = 0; i < NS; ++i)
                    if (on & (1u << i)) mbar_wait(kv_full + 8 * i, (par >> i) & 1u, nullptr);
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer: the warp waits, one lane issues
        const bool one = elect_one();
        constexpr uint32_t idesc_s = idesc_bf16_f32(TQ, TK);
        constexpr uint32_t idesc_o = idesc_bf16_f32(TQ, NB * 64, true);
        constexpr uint32_t idesc_ot = idesc_bf16_f32(TQ, 16, true);
        const uint64_t q_desc = sw128_kmajor_desc(sb + P::Q_OFF);
        const uint64_t k_desc0 = sw128_kmajor_desc(sb + P::K_OFF);
        const uint64_t v_desc0 = sw128_mnmajor_desc(sb + P::V_OFF, P::BLK);
        const uint64_t qt_desc = sw32_desc(sb + P::Q_OFF + NB * P::BLK);
        const uint64_t kt_desc0 = sw32_desc(sb + P::K_OFF + NB * P::BLK);
        const uint64_t vt_desc0 = sw32_desc(sb + P::V_OFF + NB * P::BLK);
        int c = 0, nq = 0;
        const auto issue_s = [&](int t, bool last) -> bool {      // t = c + j
            const int st = t % NS, sbuf = t % P::SBUF;
            // S_t overwrites the columns of S_{t-2} / P_{t-2}: the softmax finished with
            // them before p_full(t-2), and PV_{t-2}, issued earlier by this warp, reads
            // P_{t-2} before this MMA writes (MMAs of one thread execute in issue order)
            if (!warp_wait(kv_full + 8 * st, (t / NS) & 1, abort_flag)) return false;
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
                if (last) tc_commit(q_empty);
            }
            __syncwarp();
            return true;
        };
        const auto issue_pv = [&](int t, bool first, int steps) -> bool {
            const int st = t % NS, sbuf = t % P::SBUF;       // V landed with K (waited in issue_s)
            if (!warp_wait(p_full, t & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t so = (st * P::TILE) >> 4;
            const auto step = [&](int kk) {
                const uint32_t a = tmem + sbuf * TK + kk * 8;    // P: 16 keys = 8 columns
                const uint32_t acc = (!first || kk > 0) ? 1u : 0u;
                tc_mma_f16_ts(tmem + P::O_COL, a, v_desc0 + so + ((kk * 2048) >> 4), idesc_o, acc);
                if constexpr (TAIL)
                    tc_mma_f16_ts(tmem + P::O_COL + NB * 64, a, vt_desc0 + so + ((kk * 512) >> 4), idesc_ot, acc);
            };
            if (one) {
                if (steps == TK / 16) {
#pragma unroll
                    for (int kk = 0; kk < TK / 16; ++kk) step(kk);
                } else {
#pragma unroll 1
                    for (int kk = 0; kk < steps; ++kk) step(kk);
                }
                tc_commit(pv_done);
                tc_commit(v_empty + 8 * st);
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        Item it;
        for (int i = 0;; ++i) {
            ok = next_item(i, it);
            // (by shuffles, so that the compiler knows what is alike in all lanes: the loop's
            // indices, and with them the operands of the MMAs, stay in uniform registers)
            const int n = uniform(it.n);
            if (!ok || n < 0) break;
            if (n == 0) continue;
            // keys of the last tile that some row sees, in steps of 16, and those that exist
            const int end = key_end(min(it.qi + tq, it.nq) - 1, it.nk - it.nq, g.causal_block, it.nk) - (it.t0 + n - 1) * TK;
            const int steps = uniform(min(TK, end + 15) / 16), valid = uniform(it.nk - (it.t0 + n - 1) * TK);
            ok = warp_wait(q_full, nq & 1, abort_flag) && issue_s(c, n == 1);
            ++nq;
            // two S buffers: S_{t+1} runs while the softmax works on S_t; one (DUO): S_{t+1}
            // follows PV_t, which reads P_t from the same columns
            for (int j = 1; ok && j < n; ++j)
                ok = DUO ? (issue_pv(c + j - 1, j == 1, TK / 16) && issue_s(c + j, j + 1 == n))
                         : (issue_s(c + j, j + 1 == n) && issue_pv(c + j - 1, j == 1, TK / 16));
            if (ok && valid < steps * 16)       // V of the last tile has landed with K
                zero_rows<NB, TAIL>(smem + P::V_OFF + (c + n - 1) % NS * P::TILE, valid, lane, 32, steps * 16);
            __syncwarp();
            ok = ok && issue_pv(c + n - 1, n == 1, steps);
            if (!ok) break;
            c += n;
        }
        if (one) {
            if (!ok) fail();
            if (*abort_flag) {
                tc_commit(drain);
                mbar_wait(drain, 0, nullptr);
            }
        }
        __syncwarp();
    } else {
        // ---------------- softmax: thread = row
        const int q = warp & 3;
        const int row = q * 32 + lane;
        const int i_of = row / g.gh;                          // query of the row within an item
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const uint64_t scale2 = f32x2(g.scale_log2, g.scale_log2);
        bool ok = true;
        int c = 0;
        for (int item = 0;; ++item) {
            // read in place (registers are short in the loop), given back at the end
            const Item& it = items[item % kItems];
            ok = warp_wait(item_full + 8 * (item % kItems), (item / kItems) & 1, abort_flag);
            const int n = it.n;
            if (!ok || n < 0) break;
            // one past the row's last key, from the item's first on.  A row without a query is
            // not masked: what it holds stays its own, and one masked row costs its warp 128
            // selects a tile (heads of groups of five fill 125 rows: 8192 tokens of 40 heads
            // over 8, 1170 us, 900 without)
            int row_end = 1 << 30, live_end = 0;
            if (row < tq * g.gh && it.qi + i_of < it.nq)
                live_end = row_end = key_end(it.qi + i_of, it.nk - it.nq, g.causal_block, it.nk) - it.t0 * TK;
            const int warp_end = __reduce_max_sync(0xFFFFFFFFu, live_end);
            float m_ref = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j) {
                const int st = (c + j) % P::SBUF;
                bool got = mbar_wait(s_full + 8 * st, ((c + j) / P::SBUF) & 1, abort_flag);
                got = __all_sync(0xFFFFFFFFu, got);
                if (!got) { ok = false; break; }
                if (warp_end <= 0) {
                    // none of the warp's rows sees a key (single queries leave three warps of four
                    // so): what S and P hold there stays in those rows of O, which are not written
                    if (j > 0 && !warp_wait(pv_done, (c + j - 1) & 1, abort_flag)) { ok = false; break; }
                    if (lane == 0) mbar_arrive(p_full);
                    continue;
                }
                tc_fence_after();
                // all of S's loads in flight before one wait (the first wait covers
                // every load; the others tie each array to it)
                uint32_t r[TK / 32][32];
#pragma unroll
                for (int k = 0; k < TK / 32; ++k) tmem_ld_32x32b_x32(tl + st * TK + k * 32, r[k]);
#pragma unroll
                for (int k = 0; k < TK / 32; ++k) tmem_wait_ld_r(r[k]);
                float v[TK];
#pragma unroll
                for (int k = 0; k < TK / 32; ++k)
#pragma unroll
                    for (int u = 0; u < 32; ++u) v[k * 32 + u] = __uint_as_float(r[k][u]);
                // raw scores: the row max is taken before scaling (scale > 0)
                const int kvalid = row_end - j * TK;
                if (kvalid < TK) {
#pragma unroll
                    for (int u = 0; u < TK; ++u)
                        if (u >= kvalid) v[u] = -INFINITY;
                }
                float mp[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) mp[u] = v[u];
#pragma unroll
                for (int u = 8; u < TK; ++u) mp[u & 7] = fmaxf(mp[u & 7], v[u]);
                float mt = fmaxf(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])),
                                 fmaxf(fmaxf(mp[4], mp[5]), fmaxf(mp[6], mp[7])));
                mt *= g.scale_log2;
                // the reference maximum moves only when a row's grows by more than 8 (a
                // factor 256); only then is that row's O rescaled
                const bool resc = mt > m_ref + 8.f;
                const float m_new = resc ? mt : m_ref;
                const float corr = resc ? ex2_approx(m_ref - m_new) : 1.f;
                // a row that has seen no key yet keeps m = -inf and p = 0
                const float neg = m_new == -INFINITY ? 0.f : -m_new;
                float sp[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < TK / 32; ++k) {
                    uint32_t w[16];
                    // no row of the warp sees these keys: p = 0, as the exponentials would
                    // give.  Worth its branch where two CTAs share the SM (24 images of 16 x
                    // 72: 57 us against 60 at the time), not where one has it (3% slower)
                    if (DUO && k * 32 >= warp_end - j * TK) {
#pragma unroll
                        for (int u = 0; u < 16; ++u) w[u] = 0;
                    } else {
#pragma unroll
                        for (int u = 32 * k; u < 32 * k + 32; u += 2) {
                            f32x2_split(fma_f32x2(f32x2(v[u], v[u + 1]), scale2, f32x2(neg, neg)), v[u], v[u + 1]);
                            v[u] = ex2_approx(v[u]);
                            v[u + 1] = ex2_approx(v[u + 1]);
                            f32x2_split(add_f32x2(f32x2(sp[u & 7], sp[(u & 7) + 1]), f32x2(v[u], v[u + 1])), sp[u & 7], sp[(u & 7) + 1]);
                            w[(u & 31) / 2] = pack_bf16x2(v[u], v[u + 1]);
                        }
                    }
                    // P (bf16 pairs) over the first 64 columns of its own S buffer
                    tmem_st_32x32b_x16(tl + st * TK + k * 16, w);
                }
                const float rs = ((sp[0] + sp[1]) + (sp[2] + sp[3])) + ((sp[4] + sp[5]) + (sp[6] + sp[7]));
                l = l * corr + rs;
                m_ref = m_new;
                tmem_wait_st();
                // the PV before must be done before O is rescaled; every phase is waited
                // (an item's last one below) so the parity stays in step
                if (j > 0) {
                    got = mbar_wait(pv_done, (c + j - 1) & 1, abort_flag);
                    got = __all_sync(0xFFFFFFFFu, got);
                    if (!got) { ok = false; break; }
                    tc_fence_after();
                }
                if (j > 0 && __any_sync(0xFFFFFFFFu, resc)) {
#pragma unroll 1
                    for (int k = 0; k < (HDP + 31) / 32; ++k) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(tl + P::O_COL + k * 32, o);
                        tmem_wait_ld_r(o);
#pragma unroll
                        for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * corr);
                        tmem_st_32x32b_x32(tl + P::O_COL + k * 32, o);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            if (!ok) break;
            c += n;
            if (n > 0) {
                ok = warp_wait(pv_done, (c - 1) & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
            }
            put_rows<HDP>(g, it, tl + P::O_COL, row, m_ref, l);
            // O's columns are read before the p_full that lets the next item's first PV write them
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(item_empty + 8 * (item % kItems));
        }
        if (!ok && lane == 0) fail();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, P::TMEM_COLS);
    }
}

// Joins the parts of the rows that have several: lse = log sum_p exp(lse_p), O = sum_p
// exp(lse_p - lse) O_p.  Four warps a row, each a quarter of its parts (one after the
// other they are a chain of loads: 4 x 16384 keys, 8 key/value heads, in 16 parts a row, 54.7
// us with the launch before it, 58.3 with one warp),
// added up in their order; rows of no sequence stay as they are.
constexpr int kJoinWarps = 4;

__global__ void __launch_bounds__(256) packed_join_kernel(const __grid_constant__ PackedArgs g) {
    __shared__ float4 sums[8][32];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kJoinWarps;
    const size_t rows = static_cast<size_t>(g.heads) * g.rows_q;
    const size_t r = static_cast<size_t>(blockIdx.x) * (8 / kJoinWarps) + warp / kJoinWarps;
    const int h = static_cast<int>(r / g.rows_q), i = static_cast<int>(r - static_cast<size_t>(h) * g.rows_q);
    int parts = 0;                                     // 0 or 1: no row, or written by its one item
    if (r < rows && i >= seq_start(g.q_starts, 0, g.rows_q) && i < seq_start(g.q_starts, g.batch, g.rows_q))
        parts = min(g.count[r], g.parts);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);      // columns 4 lane .. 4 lane + 3
    float m = 0.f, total = 0.f;
    if (parts > 1) {
        // lane p holds the weights of parts p and p + 32 (kParts = 64)
        const float l0 = lane < parts ? g.pl[lane * rows + r] : -INFINITY;
        const float l1 = lane + 32 < parts ? g.pl[(lane + 32) * rows + r] : -INFINITY;
        float top = fmaxf(l0, l1);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
        m = top == -INFINITY ? 0.f : top;
        const float w0 = exp2f((l0 - m) * 1.4426950408889634f), w1 = exp2f((l1 - m) * 1.4426950408889634f);
        total = w0 + w1;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, x);
#pragma unroll 4
        for (int p = sub; p < parts; p += kJoinWarps) {
            const float w = __shfl_sync(0xFFFFFFFFu, p < 32 ? w0 : w1, p & 31);
            // weight 0: nothing visible there, its O_p was not written
            if (4 * lane < g.hd && w != 0.f) {
                const float4 v = reinterpret_cast<const float4*>(g.po + (p * rows + r) * g.hd)[lane];
                acc = make_float4(acc.x + w * v.x, acc.y + w * v.y, acc.z + w * v.z, acc.w + w * v.w);
            }
        }
    }
    sums[warp][lane] = acc;
    __syncthreads();
    if (sub != 0 || parts <= 1) return;
#pragma unroll
    for (int k = 1; k < kJoinWarps; ++k) {
        const float4 v = sums[warp + k][lane];
        acc = make_float4(acc.x + v.x, acc.y + v.y, acc.z + v.z, acc.w + v.w);
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    if (4 * lane < g.hd)
        reinterpret_cast<uint2*>(g.O + static_cast<size_t>(i) * g.ldo + h * g.hd)[lane] =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0) g.lse[r] = total == 0.f ? -INFINITY : m + logf(total);
}

// The grid, from the sizes alone (the lengths are on the device).
//  gh: the divisor of the group that makes the fewest tiles.  A sequence costs a part
//    of a tile a head, or a part of a tile for all heads that share it.
//  per: key tiles of a CTA where CTAs are runs of keys: so many that four items come to
//    an SM (the long ones last as long as the others then), kMinPer at least (each has a
//    start, an end and its part of the join) and no more than kParts parts or kPartBytes
//    for a row that has all keys.  Taken where that gives twice the CTAs that query tiles
//    would.
constexpr int kParts = 64;
constexpr int kMinPer = 4;
constexpr size_t kPartBytes = 512ull << 20;

struct PackedGrid {
    int gh, per, parts;          // parts = 1: CTAs are query tiles
    long long ctas;
};

PackedGrid packed_grid(const dlo_attn_packed& a) {
    const int group = a.heads / a.kv_heads;
    const auto tiles = [&](int gh) { return static_cast<long long>(packed_slots(a.rows_q, a.batch, TQ / gh)) * (a.heads / gh); };
    PackedGrid p = {1, 1, 1, 0};
    for (int gh = 2; gh <= TQ && gh <= group; ++gh)
        if (group % gh == 0 && tiles(gh) < tiles(p.gh)) p.gh = gh;
    p.ctas = tiles(p.gh);
    const int tq = TQ / p.gh;
    const long long keys = (a.rows_k + TK - 1) / TK, query_tiles = (a.rows_q / a.batch + tq - 1) / tq;
    const long long row_bytes = static_cast<long long>(a.heads) * a.rows_q * (a.head_dim + 1) * sizeof(float);
    long long parts = static_cast<long long>(kPartBytes) / row_bytes;
    if (parts > kParts) parts = kParts;
    if (parts < 2) return p;
    long long per = keys * (a.heads / p.gh) * (query_tiles > 0 ? query_tiles : 1) / (4 * kGb300Sms);
    if (per < kMinPer) per = kMinPer;
    if (per < (keys + parts - 1) / parts) per = (keys + parts - 1) / parts;
    if (per >= keys) return p;                        // one part; from here on TK * per <= 2^30
    const long long ctas = static_cast<long long>(packed_slots(a.rows_k, a.batch, TK * static_cast<int>(per))) * (a.heads / p.gh);
    parts = (keys + per - 1) / per;
    if (ctas < 2 * p.ctas || ctas > 0x7FFFFFFF) return p;
    p.per = static_cast<int>(per);
    p.parts = static_cast<int>(parts);
    p.ctas = ctas;
    return p;
}

template <int NB, bool TAIL, bool DUO>
cudaError_t run_packed(const PackedMaps& maps, const PackedArgs& g, cudaStream_t s, unsigned long long* launches) {
    using P = PackedPlan<NB, TAIL, DUO>;
    constexpr auto kernel = packed_fwd_kernel<NB, TAIL, DUO>;
    static unsigned long long attr = 0;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), P::BYTES, &attr); e != cudaSuccess) return e;
    const int groups = g.heads / g.gh;
    const dim3 grid = g.parts > 1 ? dim3(packed_slots(g.rows_k, g.batch, TK * g.per) * groups)
                                  : dim3(packed_slots(g.rows_q, g.batch, TQ / g.gh), groups);
    cudaError_t e = launch_k(kernel, grid, kThreadsP, P::BYTES, s, maps, g);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t attention_packed_fwd_workspace(const dlo_attn_packed& a) {
    const size_t n = packed_grid(a).parts, rows = static_cast<size_t>(a.heads) * a.rows_q;
    return 256 + (n > 1 ? n * rows * (a.head_dim + 1) * sizeof(float) + rows * sizeof(int) : 0);
}

cudaError_t launch_attention_packed_fwd(const dlo_attn_packed& a, const void* Q, const void* K, const void* V, void* O,
                                        float* lse, void* ws, int* err, cudaStream_t s, unsigned long long* launches) {
    const size_t rows = static_cast<size_t>(a.heads) * a.rows_q;
    const PackedGrid plan = packed_grid(a);
    const int hd = a.head_dim;
    PackedArgs g = {};
    g.O = static_cast<__nv_bfloat16*>(O);
    g.lse = lse;
    g.po = static_cast<float*>(ws);
    g.pl = g.po + plan.parts * rows * hd;
    g.count = reinterpret_cast<int*>(g.pl + plan.parts * rows);
    g.q_starts = a.q_starts;
    g.k_starts = a.k_starts;
    g.batch = a.batch;
    g.rows_q = a.rows_q;
    g.rows_k = a.rows_k;
    g.hd = hd;
    g.heads = a.heads;
    g.group = a.heads / a.kv_heads;
    g.gh = plan.gh;
    g.causal_block = a.causal_block < a.rows_k ? a.causal_block : a.rows_k;
    g.ldo = a.ldo;
    g.per = plan.per;
    g.parts = plan.parts;
    g.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(hd));
    g.err = err;
    PackedMaps m;
    const CUtensorMapSwizzle w128 = CU_TENSOR_MAP_SWIZZLE_128B, w32 = CU_TENSOR_MAP_SWIZZLE_32B;
    const bool tail = hd > 64 && hd <= 80;
    auto map = [&](CUtensorMap* main, CUtensorMap* tl, const void* p, int r, int heads, int ld, int box_heads) {
        if (!make_map4(main, p, 1, r, heads, hd, ld, 64, w128, box_heads)) return false;
        if (tail) return make_map4(tl, p, 1, r, heads, hd, ld, 16, w32, box_heads);
        *tl = *main;
        return true;
    };
    if (!map(&m.q, &m.qt, Q, a.rows_q, a.heads, a.ldq, plan.gh) || !map(&m.k, &m.kt, K, a.rows_k, a.kv_heads, a.ldk, 1) ||
        !map(&m.v, &m.vt, V, a.rows_k, a.kv_heads, a.ldv, 1))
        return cudaErrorInvalidValue;
    const bool duo = attn_duo_enabled() && plan.ctas > kGb300Sms;       // fewer: nothing would share an SM
    cudaError_t e;
    if (hd <= 64) e = duo ? run_packed<1, false, true>(m, g, s, launches) : run_packed<1, false, false>(m, g, s, launches);
    else if (tail) e = duo ? run_packed<1, true, true>(m, g, s, launches) : run_packed<1, true, false>(m, g, s, launches);
    else e = run_packed<2, false, false>(m, g, s, launches);
    if (e != cudaSuccess || g.parts == 1) return e;
    e = launch_k(packed_join_kernel, static_cast<unsigned>((rows + 8 / kJoinWarps - 1) / (8 / kJoinWarps)), 256, 0, s, g);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dlo
