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
// n step mod 2^64 is the exact fraction of a turn for any 32-bit n, negative ones
// too, where a 32-bit float product is off by 2^-24 of the whole angle (0.06 rad at
// position 10^6).  Its upper 32 bits go to sincospi: off by 2^-25 of a half turn.
//
// Bound by memory: x is read and y written once, 16 bytes a thread where the pairs
// allow it.  A row's sines and cosines are formed once, in shared memory, while the
// first loads of x are in flight; then a thread keeps the columns of its place in
// the head for every head that it walks, so its sines and cosines stay in registers.
constexpr int kRopeThreads = 256;
constexpr int kRopeAhead = 4;                // heads of a thread with loads in flight

struct RopeArgs {
    const __nv_bfloat16* x;
    __nv_bfloat16* y;
    const int* positions;
    const uint64_t* steps;
    int rows, heads, hd, pairs, axes, ldx, ldy;
    int end[DLO_ROPE_AXES];                  // one past the last pair of each axis
    int turned, items;                       // pieces of a head: turned ones first, then copied ones
    int ny, nr;                              // heads side by side and rows of a CTA
    float amp, amp_sin;                      // amp_sin = -amp in the backward pass
};

template <int V>
struct RopeVec {                             // V bf16 columns
    uint32_t w[V > 1 ? V / 2 : 1];
    __device__ void load(const __nv_bfloat16* p) {
        if constexpr (V == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else if constexpr (V == 4) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[0] = u.x, w[1] = u.y;
        } else if constexpr (V == 2) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ void store(__nv_bfloat16* p) const {
        if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = w[0];
        else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
    }
    __device__ float get(int i) const {
        return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    __device__ void put(int i, float a, float b) {      // columns i and i + 1 (i even; V == 1: a alone)
        w[i / 2] = pack_bf16x2(a, b);
    }
};

// HALF: a piece is V columns of the first half of the turned part and their partners
// in the second; else V columns, V / 2 pairs side by side.
template <int V, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs g) {
    extern __shared__ float2 turn[];         // [nr][pairs]: amp cos, amp sin
    constexpr int P = HALF ? V : V / 2;      // pairs of a piece
    const int c = threadIdx.x % g.items, q = threadIdx.x / g.items, h0 = q % g.ny, rr = q / g.ny;
    const long long first = static_cast<long long>(blockIdx.x) * g.nr, row = first + rr;
    const bool in = rr < g.nr && row < g.rows, turned = c < g.turned;
    const int half = HALF ? g.pairs : 0;     // columns between partners
    const int col = turned ? c * V : 2 * g.pairs + (c - g.turned) * V;
    const __nv_bfloat16* x = g.x + row * g.ldx + col;
    __nv_bfloat16* y = g.y + row * g.ldy + col;
    RopeVec<V> a[kRopeAhead], b[HALF ? kRopeAhead : 1];
    pdl_wait();
    pdl_launch_dependents();
    const auto load = [&](int h) {
#pragma unroll
        for (int k = 0; k < kRopeAhead; ++k) {
            const int at = h + k * g.ny;
            if (in && at < g.heads) {
                a[k].load(x + at * g.hd);
                if (HALF && turned) b[k].load(x + at * g.hd + half);
            }
        }
    };
    load(h0);
    const int rows = static_cast<int>(min(static_cast<long long>(g.nr), g.rows - first));
    for (int i = threadIdx.x; i < rows * g.pairs; i += kRopeThreads) {
        const int r = i / g.pairs, p = i - r * g.pairs;
        int axis = 0;
        while (p >= g.end[axis]) ++axis;     // end[axes - 1] = pairs
        const long long n = g.positions[(first + r) * g.axes + axis];
        const uint64_t phase = static_cast<uint64_t>(n) * g.steps[p];
        float s, co;
        sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &s, &co);   // 2^-31
        turn[i] = make_float2(g.amp * co, g.amp_sin * s);
    }
    __syncthreads();
    float2 t[P > 0 ? P : 1];
    if (in && turned) {
#pragma unroll
        for (int p = 0; p < P; ++p) t[p] = turn[rr * g.pairs + c * P + p];
    }
    for (int h = h0; h < g.heads; h += kRopeAhead * g.ny) {
        if (h != h0) load(h);
#pragma unroll
        for (int k = 0; k < kRopeAhead; ++k) {
            const int at = h + k * g.ny;
            if (!in || at >= g.heads) continue;
            if (turned) {
                if constexpr (HALF) {
                    RopeVec<V> u, w;
#pragma unroll
                    for (int p = 0; p < V; p += 2) {
                        const int p1 = V > 1 ? p + 1 : p;
                        const float u0 = a[k].get(p), u1 = a[k].get(p1), v0 = b[k].get(p), v1 = b[k].get(p1);
                        u.put(p, u0 * t[p].x - v0 * t[p].y, u1 * t[p1].x - v1 * t[p1].y);
                        w.put(p, u0 * t[p].y + v0 * t[p].x, u1 * t[p1].y + v1 * t[p1].x);
                    }
                    u.store(y + at * g.hd);
                    w.store(y + at * g.hd + half);
                } else {
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const float u = a[k].get(2 * p), v = a[k].get(2 * p + 1);
                        a[k].put(2 * p, u * t[p].x - v * t[p].y, u * t[p].y + v * t[p].x);
                    }
                    a[k].store(y + at * g.hd);
                }
            } else {
                a[k].store(y + at * g.hd);
            }
        }
    }
}

template <int V, bool HALF>
cudaError_t run_rope(RopeArgs g, cudaStream_t s) {
    const int copied = g.x == g.y ? 0 : (g.hd - 2 * g.pairs) / V;
    g.turned = HALF ? g.pairs / V : 2 * g.pairs / V;
    g.items = g.turned + copied;
    g.ny = kRopeThreads / g.items < g.heads ? kRopeThreads / g.items : g.heads;
    g.nr = kRopeThreads / (g.items * g.ny);
    return launch_k(rope_kernel<V, HALF>, static_cast<unsigned>((g.rows + g.nr - 1) / g.nr), kRopeThreads,
                    static_cast<size_t>(g.nr) * g.pairs * sizeof(float2), s, g);
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
    // the widest piece that whole pairs fill: 16 bytes where the pairs are a multiple of 4
    // (interleaved) or 8 (half layout: heads of 64 and 128; 8 bytes for 72), down to a column
    cudaError_t e;
    if (r.layout == DLO_ROPE_HALF) {
        e = g.pairs % 8 == 0   ? run_rope<8, true>(g, s)
            : g.pairs % 4 == 0 ? run_rope<4, true>(g, s)
            : g.pairs % 2 == 0 ? run_rope<2, true>(g, s)
                               : run_rope<1, true>(g, s);
    } else {
        e = g.pairs % 4 == 0 ? run_rope<8, false>(g, s) : g.pairs % 2 == 0 ? run_rope<4, false>(g, s) : run_rope<2, false>(g, s);
    }
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dlo
