// Packed batches: the plan of a batch (row starts and positions) and rotary
// positions.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace dlo {

namespace {

// ------------------------------------------------------------------ plan
// starts[b] = min(rows, len_0 + ... + len_{b-1}), len = the product of a
// sequence's extents; row starts[b] + i has the i-th place of its grid, last axis
// fastest.
//
// A few hundred sequences and tens of thousands of rows: bound by the launch and
// one chain of loads.  So one launch and no pass over the starts before it: every
// CTA adds up the lengths for itself, 256 sequences a step, as far as its own rows
// reach (CTA 0 to the end: it writes the starts), and finds each row's sequence by
// bisection in the step's starts in shared memory.
constexpr int kPlanThreads = 256;
constexpr int kPlanRows = 512;               // rows of one CTA

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const int* grids, const int* offsets, int batch, int axes, int rows,
                                                            int* starts, int* positions) {
    __shared__ int begin[kPlanThreads + 1];
    __shared__ long long sums[kPlanThreads / 32];
    const int t = threadIdx.x, lane = t & 31;
    const int r0 = blockIdx.x * kPlanRows, r1 = positions ? min(rows, r0 + kPlanRows) : 0;
    pdl_wait();
    pdl_launch_dependents();
    long long before = 0;                    // rows of the sequences of earlier steps
    for (int b0 = 0; b0 < batch; b0 += kPlanThreads) {
        const int b = b0 + t;
        long long len = 0;
        if (b < batch) {
            len = 1;
            // more than 2^31 rows are as good as 2^31
            for (int a = 0; a < axes; ++a) len = min(len * max(grids[b * axes + a], 0), 1ll << 31);
        }
        long long sum = len;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const long long u = __shfl_up_sync(0xFFFFFFFFu, sum, x);
            if (lane >= x) sum += u;
        }
        if (lane == 31) sums[t / 32] = sum;
        __syncthreads();
        long long total = 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < t / 32) sum += sums[w];
            total += sums[w];
        }
        const auto row = [&](long long n) { return static_cast<int>(min(before + n, static_cast<long long>(rows))); };
        begin[t] = row(sum - len);
        if (t == 0) begin[kPlanThreads] = row(total);
        if (blockIdx.x == 0) {
            if (b < batch) starts[b] = row(sum - len);
            if (b == batch - 1) starts[batch] = row(sum);
        }
        __syncthreads();
        const int last = min(r1, begin[kPlanThreads]);
        for (int r = max(r0, begin[0]) + t; r < last; r += kPlanThreads) {
            int lo = 0, hi = kPlanThreads;   // begin[lo] <= r < begin[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (begin[mid] <= r) lo = mid;
                else hi = mid;
            }
            unsigned i = r - begin[lo];
            const size_t s = static_cast<size_t>(b0 + lo) * axes;
            for (int a = axes - 1; a >= 0; --a) {
                const unsigned n = grids[s + a], q = i / n;      // not 0: the sequence has rows
                const unsigned at = i - q * n;
                positions[static_cast<size_t>(r) * axes + a] = static_cast<int>(at + (offsets ? offsets[s + a] : 0));
                i = q;
            }
        }
        before += total;
        if (blockIdx.x != 0 && before >= r1) return;
        __syncthreads();
    }
}

// ------------------------------------------------------------------ rotary positions
// Pair p of a row at position n turns by n f_p: (u, v) -> amp (u c - v s, u s + v c).
//
// The angle is kept in turns as a 64-bit fraction: step = f_p / 2 pi * 2^64, and
// n step mod 2^64 loses nothing for any 32-bit n, negative ones too, where a 32-bit
// float product is off by 2^-24 of the whole angle (0.06 rad at position 10^6).  What is
// left is the table's error, n times (up to 2^-24 of a turn at n = 2^31, measured; its bound
// is at dlo_rope_steps), and that the upper 32 bits go to sincospi as a float: off by
// 2^-25 of a half turn.
//
// Bound by memory: x is read and y written once, 16 bytes a thread where the pairs
// allow it.  A row's sines and cosines are formed once, in shared memory, while the
// first loads of x are in flight.  A thread keeps its columns of the head and walks
// heads of one row (wide rows: its sines and cosines stay in registers) or rows (ROWS:
// narrow ones, where a row gives it less than three heads), a few ahead.
constexpr int kRopeThreads = 256;

// Pieces of a thread with loads in flight, and CTAs an SM: a piece of the half layout
// is two loads, its registers are two and a half times the others' (8192 rows of 80
// heads of 128: 51.6 us, 55 with four pieces and three CTAs, 58.8 with two and five;
// interleaved 50.5, 53.6 where the compiler takes what it likes).
template <int V, bool HALF>
constexpr int kAhead = V == 8 && HALF ? 3 : 4;
template <int V, bool HALF>
constexpr int kCtas = V == 8 && HALF ? 4 : 6;

struct RopeArgs {
    const __nv_bfloat16* x;
    __nv_bfloat16* y;
    const int* positions;
    const uint64_t* steps;
    int rows, heads, hd, pairs, axes, ldx, ldy;
    int end[DLO_ROPE_AXES];                  // one past the last pair of each axis
    int turned, items;                       // pieces of a head: turned ones first, then copied ones
    int ny, nr;                              // heads and rows side by side in a CTA
    float amp, amp_sin;                      // amp_sin = -amp in the backward pass
};

template <int V>
struct RopeVec {                             // V bf16 columns
    uint32_t w[V > 1 ? V / 2 : 1];
    __device__ void load(const __nv_bfloat16* p) {
        if constexpr (V == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else if constexpr (V == 2) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (V == 1) {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        } else {
            load_half(p, true);
        }
    }
    __device__ void store(__nv_bfloat16* p) const {
        if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = w[0];
        else if constexpr (V == 1) *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
        else store_half(p, true);
    }
    // by 8 bytes; of eight columns the second four only where `whole`
    __device__ void load_half(const __nv_bfloat16* p, bool whole) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x, w[1] = u.y;
        if constexpr (V == 8) {
            const uint2 v = whole ? *reinterpret_cast<const uint2*>(p + 4) : make_uint2(0, 0);
            w[2] = v.x, w[3] = v.y;
        }
    }
    __device__ void store_half(__nv_bfloat16* p, bool whole) const {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        if constexpr (V == 8)
            if (whole) *reinterpret_cast<uint2*>(p + 4) = make_uint2(w[2], w[3]);
    }
    __device__ float get(int i) const {
        return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    __device__ void put(int i, float a, float b) {      // columns i and i + 1 (i even; V == 1: a alone)
        w[i / 2] = pack_bf16x2(a, b);
    }
};

// HALF: a piece is V columns of the first half of the turned part and their partners
// in the second; else V columns, V / 2 pairs side by side.  ODD (HALF, V = 8, pairs = 4
// mod 8, as a head of 72 has): the partners lie on 8-byte boundaries and the last
// piece has four columns (16381 rows of 48 heads of 96, 72 columns turned: 58.5 us, 60.5
// in pieces of four columns).
template <int V, bool HALF, bool ROWS, bool ODD>
__global__ void __launch_bounds__(kRopeThreads, kCtas<V, HALF>) rope_kernel(const __grid_constant__ RopeArgs g) {
    extern __shared__ float2 turn[];         // [rows of the CTA][pairs]: amp cos, amp sin
    constexpr int P = HALF ? V : V / 2;      // pairs of a piece
    constexpr int A = kAhead<V, HALF>;
    constexpr int R = ROWS ? A : 1; // rows of a thread
    const int c = threadIdx.x % g.items, q = threadIdx.x / g.items, h0 = q % g.ny, rr = q / g.ny;
    const long long first = static_cast<long long>(blockIdx.x) * g.nr * R;
    const int rows = static_cast<int>(min(static_cast<long long>(g.nr) * R, g.rows - first));
    const int heads = rr < g.nr && rr < rows ? g.heads : 0;
    const bool turned = c < g.turned, whole = !ODD || !turned || (c + 1) * V <= g.pairs;
    const int half = HALF ? g.pairs : 0;     // columns between partners
    const int col = turned ? c * V : 2 * g.pairs + (c - g.turned) * V;
    const __nv_bfloat16* x = g.x + (first + rr) * g.ldx + col;
    __nv_bfloat16* y = g.y + (first + rr) * g.ldy + col;
    // piece k of a batch: head h + k ny of the row, or row rr + k nr of the head
    const long long step_x = ROWS ? static_cast<long long>(g.nr) * g.ldx : static_cast<long long>(g.ny) * g.hd;
    const long long step_y = ROWS ? static_cast<long long>(g.nr) * g.ldy : step_x;
    const auto there = [&](int h, int k) { return ROWS ? rr + k * g.nr < rows : h + k * g.ny < heads; };
    RopeVec<V> a[A], b[HALF ? A : 1];
    pdl_wait();
    pdl_launch_dependents();
    const auto load = [&](int h) {
        const __nv_bfloat16* p = x + h * g.hd;
#pragma unroll
        for (int k = 0; k < A; ++k, p += step_x) {
            if (!there(h, k)) break;
            if (ODD && !whole) a[k].load_half(p, false);
            else a[k].load(p);
            if constexpr (HALF) {
                if (turned) {
                    if constexpr (ODD) b[k].load_half(p + half, whole);
                    else b[k].load(p + half);
                }
            }
        }
    };
    if (h0 < heads) load(h0);
    for (int i = threadIdx.x; i < rows * g.pairs; i += kRopeThreads) {
        const int r = i / g.pairs, p = i - r * g.pairs;
        int axis = 0;
        while (p >= g.end[axis]) ++axis;     // end[axes - 1] = pairs
        const long long at = g.positions[(first + r) * g.axes + axis];
        const uint64_t phase = static_cast<uint64_t>(at) * g.steps[p];
        float s, co;
        sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &s, &co);   // 2^-31
        turn[i] = make_float2(g.amp * co, g.amp_sin * s);
    }
    __syncthreads();
    float2 t[P > 0 ? P : 1];
    const auto turns = [&](int r) {
#pragma unroll
        for (int p = 0; p < P; ++p) t[p] = whole || p < P / 2 ? turn[r * g.pairs + c * P + p] : make_float2(0.f, 0.f);
    };
    if (!ROWS && turned && heads) turns(rr);
    for (int h = h0; h < heads; h += ROWS ? g.ny : A * g.ny) {
        if (h != h0) load(h);
        __nv_bfloat16* to = y + h * g.hd;
#pragma unroll
        for (int k = 0; k < A; ++k, to += step_y) {
            if (!there(h, k)) break;
            if (!turned) {
                a[k].store(to);
                continue;
            }
            if (ROWS) turns(rr + k * g.nr);
            if constexpr (HALF) {
                RopeVec<V> u, w;
#pragma unroll
                for (int p = 0; p < V; p += 2) {
                    const int p1 = V > 1 ? p + 1 : p;
                    const float u0 = a[k].get(p), u1 = a[k].get(p1), v0 = b[k].get(p), v1 = b[k].get(p1);
                    u.put(p, u0 * t[p].x - v0 * t[p].y, u1 * t[p1].x - v1 * t[p1].y);
                    w.put(p, u0 * t[p].y + v0 * t[p].x, u1 * t[p1].y + v1 * t[p1].x);
                }
                if (ODD && !whole) u.store_half(to, false);
                else u.store(to);
                if constexpr (ODD) w.store_half(to + half, whole);
                else w.store(to + half);
            } else {
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const float u = a[k].get(2 * p), v = a[k].get(2 * p + 1);
                    a[k].put(2 * p, u * t[p].x - v * t[p].y, u * t[p].y + v * t[p].x);
                }
                a[k].store(to);
            }
        }
    }
}

template <int V, bool HALF, bool ODD = false>
cudaError_t run_rope(RopeArgs g, cudaStream_t s) {
    const int copied = g.x == g.y ? 0 : (g.hd - 2 * g.pairs) / V;
    g.turned = HALF ? (g.pairs + V - 1) / V : 2 * g.pairs / V;
    g.items = g.turned + copied;
    // as many heads side by side as fit, evenly over the passes that the row takes
    const int fit = kRopeThreads / g.items, passes = (g.heads + fit - 1) / fit;
    g.ny = (g.heads + passes - 1) / passes;
    g.nr = kRopeThreads / (g.items * g.ny);
    constexpr int A = kAhead<V, HALF>;
    // rows ahead, unless that leaves SMs without a CTA
    const bool ahead = passes < 3 && static_cast<long long>(g.rows) >= static_cast<long long>(kGb300Sms) * g.nr * A;
    const int rows = g.nr * (ahead ? A : 1);
    const unsigned ctas = static_cast<unsigned>((static_cast<long long>(g.rows) + rows - 1) / rows);
    const size_t smem = static_cast<size_t>(rows) * g.pairs * sizeof(float2);
    return ahead ? launch_big<rope_kernel<V, HALF, true, ODD>>(ctas, kRopeThreads, smem, s, g)
                 : launch_big<rope_kernel<V, HALF, false, ODD>>(ctas, kRopeThreads, smem, s, g);
}

}  // namespace

cudaError_t launch_packed_plan(const int* grids, const int* offsets, int batch, int axes, int rows, int* starts,
                               int* positions, cudaStream_t s, unsigned long long* launches) {
    const int ctas = positions ? (rows + kPlanRows - 1) / kPlanRows : 1;
    cudaError_t e = launch_k(plan_kernel, ctas, kPlanThreads, 0, s, grids, offsets, batch, axes, rows, starts, positions);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_rope(const dlo_rope& r, bool back, const void* x, int ldx, const int* positions, const uint64_t* steps,
                        int rows, void* y, int ldy, cudaStream_t s, unsigned long long* launches) {
    RopeArgs g = {};
    g.x = static_cast<const __nv_bfloat16*>(x);
    g.y = static_cast<__nv_bfloat16*>(y);
    g.positions = positions;
    g.steps = steps;
    g.rows = rows;
    g.heads = r.heads;
    g.hd = r.head_dim;
    g.axes = r.axes;
    g.ldx = ldx;
    g.ldy = ldy;
    for (int a = 0; a < r.axes; ++a) g.end[a] = g.pairs += r.axis[a].dim / 2;
    g.amp = r.amp;
    g.amp_sin = back ? -r.amp : r.amp;
    // the widest piece that whole pairs fill: 16 bytes where the pairs are a multiple of 4,
    // down to a column of 2
    cudaError_t e;
    if (r.layout == DLO_ROPE_HALF) {
        e = g.pairs % 8 == 0   ? run_rope<8, true>(g, s)
            : g.pairs % 8 == 4 ? run_rope<8, true, true>(g, s)
            : g.pairs % 2 == 0 ? run_rope<2, true>(g, s)
                               : run_rope<1, true>(g, s);
    } else {
        e = g.pairs % 4 == 0 ? run_rope<8, false>(g, s) : g.pairs % 2 == 0 ? run_rope<4, false>(g, s) : run_rope<2, false>(g, s);
    }
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dlo
