// Normalisation for training: RMSNorm that keeps its row statistic, and the
// backward passes of LayerNorm and RMSNorm with the column sums that are the
// gradients of the modulation or of the weight.
//
// With xh the normalised row and g = dy * gain (gain = 1 + scale, w or 1):
//   LayerNorm  dx = rstd (g - mean(g) - xh mean(g xh)) + dres
//   RMSNorm    dx = r (g - xh mean(g xh)),  xh = x r
//   column sums over the rows of a batch (modulation) or over all rows
//   (weight): sum dy and sum dy xh.
// Everything is bound by HBM: each element of x, dy (and dres) is read once and
// dx written once.  A row lives in the registers of W warps, which also hold
// the gain of their columns (a CTA stays within one batch) and the two
// running column sums of every row they have seen (above 10240 columns, LayerNorm,
// or 12288, RMSNorm, 32 warps share a row with 64 registers a thread, and 664 or 350
// bytes a thread spill: 2048 x 16384, whose column sums take a second launch, runs at
// 1.9 and 1.5 TB/s); the sums of a CTA leave it
// once, as one partial row, and a second launch adds the partial rows in a
// fixed order, so results do not depend on the schedule.  Few rows take one
// launch instead: more CTAs of it read dy and x again for the column sums (their
// order is another one, and RMSNorm in place cannot take it, so the last bits of
// its dw differ between in place and not).
// Sums and statistics are fp32.  (32760 x 5120 LayerNorm backward: 384 us, 6.1
// TB/s; 8192 x 5120 RMSNorm forward 27.9 us, 6.0 TB/s, backward 48 us.)
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace dlo {

namespace {

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ float2 bf2(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

__device__ __forceinline__ float4 bf4(uint2 v) {
    const float2 a = bf2(v.x), b = bf2(v.y);
    return make_float4(a.x, a.y, b.x, b.y);
}

// Sums of v0 and v1 over the W warps that share a row.  red: [2][2][warps],
// two buffers used in turn, so one barrier per row suffices (a buffer is
// written again only after the barrier of the row between).
template <int W, int WARPS>
__device__ __forceinline__ void row_totals(float& v0, float& v1, float (*red)[2][WARPS], int turn, int warp, int lane) {
    v0 = warp_total(v0);
    v1 = warp_total(v1);
    if constexpr (W > 1) {
        if (lane == 0) {
            red[turn][0][warp] = v0;
            red[turn][1][warp] = v1;
        }
        __syncthreads();
        const int w0 = warp - warp % W;
        v0 = 0.f;
        v1 = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            v0 += red[turn][0][w0 + k];
            v1 += red[turn][1][w0 + k];
        }
    }
}

// 16 bytes from global to this thread's own place in shared memory, zeros
// where `in` is false; no barrier is needed between a thread's copies and its
// reads of them, only its own wait.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What multiplies dy before the row sums: nothing, w (bf16) or 1 + scale (fp32)
enum { kGainOne = 0, kGainW = 1, kGainScale = 2 };

// Few rows: the column sums of 32 columns of one batch by one CTA, which reads
// those columns of dy and x again (from L2), in the launch that forms dx.  32 row
// groups of 8 lanes; each adds every 32nd row, then the groups are added in order.
struct ColumnWork {
    int first;                 // CTAs from this one on do columns
    int slabs;                 // of 32 columns
    float *out1, *out2;        // sum dy, sum dy xh
    int ld;
};

__device__ __forceinline__ void column_slab(const ColumnWork& cw, const __nv_bfloat16* dy, const float* x, const float* mean,
                                            const float* rstd, int rows, int D, int rpb, float4 (*sh)[8]) {
    const int id = blockIdx.x - cw.first, b = id / cw.slabs, slab = id - b * cw.slabs;
    const int rg = threadIdx.x >> 3, i = slab * 8 + (threadIdx.x & 7);      // row group, float4 of the row
    const int row0 = b * rpb, n = min(rpb, rows - row0), n4 = D >> 2;
    float4 s1 = make_float4(0.f, 0.f, 0.f, 0.f), s2 = s1;
    if (i < n4) {
#pragma unroll 8
        for (int r = rg; r < n; r += 32) {
            const size_t row = static_cast<size_t>(row0) + r;
            const float4 v = reinterpret_cast<const float4*>(x + row * D)[i], d = bf4(reinterpret_cast<const uint2*>(dy + row * D)[i]);
            const float mu = mean[row], rs = rstd[row];
            s1 = make_float4(s1.x + d.x, s1.y + d.y, s1.z + d.z, s1.w + d.w);
            s2 = make_float4(s2.x + d.x * ((v.x - mu) * rs), s2.y + d.y * ((v.y - mu) * rs), s2.z + d.z * ((v.z - mu) * rs),
                             s2.w + d.w * ((v.w - mu) * rs));
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        sh[rg][threadIdx.x & 7] = which ? s2 : s1;
        __syncthreads();
        if (threadIdx.x < 8 && i < n4) {
            float4 t = sh[0][threadIdx.x];
#pragma unroll
            for (int k = 1; k < 32; ++k) {
                const float4 u = sh[k][threadIdx.x];
                t = make_float4(t.x + u.x, t.y + u.y, t.z + u.z, t.w + u.w);
            }
            reinterpret_cast<float4*>((which ? cw.out2 : cw.out1) + static_cast<size_t>(b) * cw.ld)[i] = t;
        }
        __syncthreads();
    }
}

// One CTA: rows first, first + step, ... of one batch.  Column c of the row
// belongs to the thread whose index within the row's warps is (c / 4) % (32 W).
template <int V4, int W, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS >= 32 ? 1 : 16 / WARPS)
    layernorm_bwd_kernel(const __nv_bfloat16* dy, const float* x, const float* __restrict__ mean,
                         const float* __restrict__ rstd, int rows, int D, int rpb, int parts, int gain_kind,
                         const void* __restrict__ gain, int gain_ld, const float* dres, float* dx,
                         float* __restrict__ sum_dy, float* __restrict__ sum_dyxh, size_t sum_ld, const ColumnWork cw) {
    constexpr int R = WARPS / W;
    extern __shared__ float4 sh[];                  // [R][2][n4] when R > 1
    __shared__ float red[2][2][WARPS];
    pdl_wait();
    pdl_launch_dependents();
    if constexpr (WARPS == 8) {
        if (static_cast<int>(blockIdx.x) >= cw.first) {
            __shared__ float4 cols[32][8];
            column_slab(cw, dy, x, mean, rstd, rows, D, rpb, cols);
            return;
        }
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / parts, part = blockIdx.x - b * parts;
    const int rg = warp / W, t0 = (warp % W) * 32 + lane;
    const int n4 = D >> 2;
    const int row0 = b * rpb;
    const int nrows = min(rpb, rows - row0);
    const float inv_d = 1.f / static_cast<float>(D);
    float4 gn[V4], s1[V4], s2[V4];
#pragma unroll
    for (int j = 0; j < V4; ++j) {
        const int i = t0 + 32 * W * j;
        s1[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        s2[j] = s1[j];
        gn[j] = make_float4(1.f, 1.f, 1.f, 1.f);
        if (gain_kind != kGainOne && i < n4) {
            if (gain_kind == kGainScale) {
                const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(gain) +
                                                                  static_cast<size_t>(b) * gain_ld + 4 * i);
                gn[j] = make_float4(1.f + v.x, 1.f + v.y, 1.f + v.z, 1.f + v.w);
            } else {
                gn[j] = bf4(reinterpret_cast<const uint2*>(gain)[i]);
            }
        }
    }
    int turn = 0;
    for (int r = part * R; r < nrows; r += parts * R, turn ^= 1) {
        const bool live = r + rg < nrows;
        const size_t row = static_cast<size_t>(row0) + (live ? r + rg : r);
        const float4* xr = reinterpret_cast<const float4*>(x + row * D);
        const uint2* dyr = reinterpret_cast<const uint2*>(dy + row * D);
        float4 xv[V4], g[V4], rv[V4];
        uint2 dv[V4];
#pragma unroll
        for (int j = 0; j < V4; ++j) {
            const int i = t0 + 32 * W * j;
            const bool in = live && i < n4;
            xv[j] = in ? xr[i] : make_float4(0.f, 0.f, 0.f, 0.f);
            dv[j] = in ? dyr[i] : make_uint2(0, 0);
        }
        if (dres) {
            const float4* rr = reinterpret_cast<const float4*>(dres + row * D);
#pragma unroll
            for (int j = 0; j < V4; ++j) {
                const int i = t0 + 32 * W * j;
                rv[j] = live && i < n4 ? rr[i] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        } else {
#pragma unroll
            for (int j = 0; j < V4; ++j) rv[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float mu = mean[row], rs = rstd[row];
        float a = 0.f, c = 0.f;
#pragma unroll
        for (int j = 0; j < V4; ++j) {
            // columns past D and rows past the batch have dy = 0: they add nothing
            const float4 d = bf4(dv[j]);
            float4& v = xv[j];
            v = make_float4((v.x - mu) * rs, (v.y - mu) * rs, (v.z - mu) * rs, (v.w - mu) * rs);
            g[j] = make_float4(d.x * gn[j].x, d.y * gn[j].y, d.z * gn[j].z, d.w * gn[j].w);
            a += (g[j].x + g[j].y) + (g[j].z + g[j].w);
            c += (g[j].x * v.x + g[j].y * v.y) + (g[j].z * v.z + g[j].w * v.w);
            s1[j] = make_float4(s1[j].x + d.x, s1[j].y + d.y, s1[j].z + d.z, s1[j].w + d.w);
            s2[j] = make_float4(s2[j].x + d.x * v.x, s2[j].y + d.y * v.y, s2[j].z + d.z * v.z, s2[j].w + d.w * v.w);
        }
        row_totals<W, WARPS>(a, c, red, turn, warp, lane);
        a *= inv_d;
        c *= inv_d;
        if (live) {
            float4* out = reinterpret_cast<float4*>(dx + row * D);
#pragma unroll
            for (int j = 0; j < V4; ++j) {
                const int i = t0 + 32 * W * j;
                if (i < n4)
                    out[i] = make_float4(rs * (g[j].x - a - xv[j].x * c) + rv[j].x, rs * (g[j].y - a - xv[j].y * c) + rv[j].y,
                                         rs * (g[j].z - a - xv[j].z * c) + rv[j].z, rs * (g[j].w - a - xv[j].w * c) + rv[j].w);
            }
        }
    }
    if (!sum_dy) return;
    float* o1 = sum_dy + blockIdx.x * sum_ld;
    float* o2 = sum_dyxh + blockIdx.x * sum_ld;
    if constexpr (R == 1) {
#pragma unroll
        for (int j = 0; j < V4; ++j) {
            const int i = t0 + 32 * W * j;
            if (i < n4) {
                reinterpret_cast<float4*>(o1)[i] = s1[j];
                reinterpret_cast<float4*>(o2)[i] = s2[j];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < V4; ++j) {
            const int i = t0 + 32 * W * j;
            if (i < n4) {
                sh[(rg * 2 + 0) * n4 + i] = s1[j];
                sh[(rg * 2 + 1) * n4 + i] = s2[j];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * n4; i += 32 * WARPS) {
            float4 t = sh[i];
#pragma unroll
            for (int k = 1; k < R; ++k) {
                const float4 u = sh[k * 2 * n4 + i];
                t = make_float4(t.x + u.x, t.y + u.y, t.z + u.z, t.w + u.w);
            }
            reinterpret_cast<float4*>(i < n4 ? o1 : o2)[i < n4 ? i : i - n4] = t;
        }
    }
}

// Places of the ring: one row in use, whose place is filled again only in the
// next step, when every value read from it has been used, the others in flight.
__host__ __device__ constexpr int ring_rows(int warps) { return warps == 32 ? 2 : 4; }

// As column_slab, 64 columns of dw: the sum of dy xh.
__device__ __forceinline__ void column_slab_rms(const ColumnWork& cw, const __nv_bfloat16* dy, int lddy, const __nv_bfloat16* x, int ldx,
                                                const float* rstd, int rows, int D, float4 (*sh)[16]) {
    const int slab = blockIdx.x - cw.first, rg = threadIdx.x >> 3, i = slab * 8 + (threadIdx.x & 7), n8 = D >> 3;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (i < n8) {
#pragma unroll 8
        for (int r = rg; r < rows; r += 32) {
            const uint4 xv = reinterpret_cast<const uint4*>(x + static_cast<size_t>(r) * ldx)[i];
            const uint4 dv = reinterpret_cast<const uint4*>(dy + static_cast<size_t>(r) * lddy)[i];
            const float rs = rstd[r];
            const uint32_t xa[4] = {xv.x, xv.y, xv.z, xv.w}, da[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 xx = bf2(xa[k]), dd = bf2(da[k]);
                s[2 * k] += dd.x * (xx.x * rs);
                s[2 * k + 1] += dd.y * (xx.y * rs);
            }
        }
    }
    sh[rg][2 * (threadIdx.x & 7)] = make_float4(s[0], s[1], s[2], s[3]);
    sh[rg][2 * (threadIdx.x & 7) + 1] = make_float4(s[4], s[5], s[6], s[7]);
    __syncthreads();
    const int c = slab * 16 + threadIdx.x;          // float4 of dw
    if (threadIdx.x < 16 && c < 2 * n8) {
        float4 t = sh[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < 32; ++k) {
            const float4 u = sh[k][threadIdx.x];
            t = make_float4(t.x + u.x, t.y + u.y, t.z + u.z, t.w + u.w);
        }
        reinterpret_cast<float4*>(cw.out1)[c] = t;
    }
}

// RMSNorm backward on bf16 rows of strides ldy, ldx, lddx: dx may be dy or x
// (each element is read by the thread that writes it, before it writes).
template <int V8, int W, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS >= 32 ? 1 : 16 / WARPS)
    rmsnorm_bwd_kernel(const __nv_bfloat16* dy, int lddy, const __nv_bfloat16* x, int ldx,
                       const __nv_bfloat16* __restrict__ w, const float* __restrict__ rstd, int rows, int D, int parts,
                       __nv_bfloat16* dx, int lddx, float* __restrict__ sums, const ColumnWork cw) {
    constexpr int R = WARPS / W;
    extern __shared__ float4 sh[];                  // the ring; at the end [R][D / 4] when R > 1
    __shared__ float red[2][2][WARPS];
    pdl_wait();
    pdl_launch_dependents();
    if constexpr (WARPS == 8) {
        if (static_cast<int>(blockIdx.x) >= cw.first) {
            __shared__ float4 cols[32][16];
            column_slab_rms(cw, dy, lddy, x, ldx, rstd, rows, D, cols);
            return;
        }
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rg = warp / W, t0 = (warp % W) * 32 + lane;
    const int n8 = D >> 3;
    const float inv_d = 1.f / static_cast<float>(D);
    uint4 wv[V8];
    float s[V8][8];
#pragma unroll
    for (int j = 0; j < V8; ++j) {
        const int i = t0 + 32 * W * j;
        wv[j] = i < n8 ? reinterpret_cast<const uint4*>(w)[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[j][k] = 0.f;
    }
    constexpr int T = 32 * WARPS, N = ring_rows(WARPS);
    uint4* ring = reinterpret_cast<uint4*>(sh) + threadIdx.x;          // [N][2 V8][T]
    const auto load = [&](int r, int stage) {
        const bool live = r + rg < rows;
        const size_t row = live ? r + rg : 0;
        const uint4* xr = reinterpret_cast<const uint4*>(x + row * ldx);
        const uint4* dyr = reinterpret_cast<const uint4*>(dy + row * lddy);
#pragma unroll
        for (int j = 0; j < V8; ++j) {
            const int i = t0 + 32 * W * j;
            const bool in = live && i < n8;
            copy16(ring + (stage * 2 * V8 + j) * T, xr + (in ? i : 0), in);
            copy16(ring + (stage * 2 * V8 + V8 + j) * T, dyr + (in ? i : 0), in);
        }
        copies_commit();
    };
    const int step = parts * R;
#pragma unroll
    for (int k = 0; k < N - 1; ++k) load(blockIdx.x * R + k * step, k);
    int turn = 0, stage = 0;
    for (int r = blockIdx.x * R; r < rows; r += step, turn ^= 1) {
        const bool live = r + rg < rows;
        const size_t row = live ? r + rg : r;
        copies_wait<N - 2>();
        uint4 xv[V8], dv[V8];
#pragma unroll
        for (int j = 0; j < V8; ++j) {
            xv[j] = ring[(stage * 2 * V8 + j) * T];
            dv[j] = ring[(stage * 2 * V8 + V8 + j) * T];
        }
        load(r + (N - 1) * step, (stage + N - 1) % N);
        stage = (stage + 1) % N;
        const float rs = rstd[row];
        float c = 0.f, unused = 0.f;
#pragma unroll
        for (int j = 0; j < V8; ++j) {
            const uint32_t xa[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
            const uint32_t da[4] = {dv[j].x, dv[j].y, dv[j].z, dv[j].w};
            const uint32_t wa[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 xx = bf2(xa[k]), dd = bf2(da[k]), ww = bf2(wa[k]);
                const float e0 = dd.x * (xx.x * rs), e1 = dd.y * (xx.y * rs);
                s[j][2 * k] += e0;
                s[j][2 * k + 1] += e1;
                c += e0 * ww.x + e1 * ww.y;
            }
        }
        row_totals<W, WARPS>(c, unused, red, turn, warp, lane);
        c *= inv_d;
        if (live) {
            uint4* out = reinterpret_cast<uint4*>(dx + row * lddx);
#pragma unroll
            for (int j = 0; j < V8; ++j) {
                const int i = t0 + 32 * W * j;
                if (i >= n8) continue;
                const uint32_t xa[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
                const uint32_t da[4] = {dv[j].x, dv[j].y, dv[j].z, dv[j].w};
                const uint32_t wa[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w};
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 xx = bf2(xa[k]), dd = bf2(da[k]), ww = bf2(wa[k]);
                    o[k] = pack_bf16x2(rs * (dd.x * ww.x - xx.x * rs * c), rs * (dd.y * ww.y - xx.y * rs * c));
                }
                out[i] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
    if (!sums) return;
    float4* o = reinterpret_cast<float4*>(sums + static_cast<size_t>(blockIdx.x) * D);
    if constexpr (R > 1) {
        copies_wait<0>();           // the ring's place is used again
        __syncthreads();
    }
    float4* mine = R == 1 ? o : sh + rg * 2 * n8;
#pragma unroll
    for (int j = 0; j < V8; ++j) {
        const int i = t0 + 32 * W * j;
        if (i < n8) {
            mine[2 * i] = make_float4(s[j][0], s[j][1], s[j][2], s[j][3]);
            mine[2 * i + 1] = make_float4(s[j][4], s[j][5], s[j][6], s[j][7]);
        }
    }
    if constexpr (R > 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * n8; i += 32 * WARPS) {
            float4 t = sh[i];
#pragma unroll
            for (int k = 1; k < R; ++k) {
                const float4 u = sh[k * 2 * n8 + i];
                t = make_float4(t.x + u.x, t.y + u.y, t.z + u.z, t.w + u.w);
            }
            o[i] = t;
        }
    }
}

// Adds `parts` partial rows per batch: out[b * out_ld + c] = sum over p of
// part[((b * parts + p) * 2 + which) * D + c] (LayerNorm, both sums) or of one
// row (RMSNorm, nsum = 1).  A CTA owns 32 float4 columns; its 32 warps add
// every 32nd partial row (at most 10, all loads in flight at once), then the
// 32 sums are added in order, eight by eight.  Few columns make few CTAs, so
// latency bounds it: 8 warps, 38 rows each, took 14.5 us for 304 x 5120.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* __restrict__ part, int parts, int n4, int nsum,
                                                           float* out1, float* out2, size_t out_ld) {
    __shared__ float4 sh[32][32];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = (n4 + 31) / 32;
    const int tile = blockIdx.x % tiles, rest = blockIdx.x / tiles;
    const int which = rest % nsum, b = rest / nsum;
    const int i = tile * 32 + lane;
    const auto add = [](float4 a, float4 u) { return make_float4(a.x + u.x, a.y + u.y, a.z + u.z, a.w + u.w); };
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n4) {
        const float4* p = reinterpret_cast<const float4*>(part) + (static_cast<size_t>(b) * parts * nsum + which) * n4 + i;
#pragma unroll 10
        for (int k = warp; k < parts; k += 32) t = add(t, p[static_cast<size_t>(k) * nsum * n4]);
    }
    sh[warp][lane] = t;
    __syncthreads();
    if (warp < 4) {
        t = sh[8 * warp][lane];
#pragma unroll
        for (int k = 1; k < 8; ++k) t = add(t, sh[8 * warp + k][lane]);
    }
    __syncthreads();
    if (warp < 4) sh[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && i < n4) {
#pragma unroll
        for (int k = 1; k < 4; ++k) t = add(t, sh[k][lane]);
        reinterpret_cast<float4*>((which ? out2 : out1) + b * out_ld)[i] = t;
    }
}

// y = x r w with r = 1 / sqrt(mean(x^2) + eps); the row stays in registers.
template <int V8, int W>
__global__ void __launch_bounds__(256)
    rmsnorm_fwd_kernel(const __nv_bfloat16* __restrict__ x, int ldx, int rows, int D,
                       const __nv_bfloat16* __restrict__ w, float eps, __nv_bfloat16* __restrict__ y, int ldy,
                       float* __restrict__ rstd) {
    constexpr int R = 8 / W;
    __shared__ float red[2][2][8];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x * R + warp / W, t0 = (warp % W) * 32 + lane;
    const bool live = row < rows;
    const int n8 = D >> 3;
    const uint4* xr = reinterpret_cast<const uint4*>(x + static_cast<size_t>(live ? row : 0) * ldx);
    uint4 v[V8];
    float q = 0.f, unused = 0.f;
#pragma unroll
    for (int j = 0; j < V8; ++j) {
        const int i = t0 + 32 * W * j;
        v[j] = live && i < n8 ? xr[i] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < V8; ++j) {
        const uint32_t a[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = bf2(a[k]);
            q += f.x * f.x + f.y * f.y;
        }
    }
    row_totals<W, 8>(q, unused, red, 0, warp, lane);
    if (!live) return;
    const float r = rsqrtf(q / static_cast<float>(D) + eps);
    if (t0 == 0) rstd[row] = r;
    uint4* yr = reinterpret_cast<uint4*>(y + static_cast<size_t>(row) * ldy);
#pragma unroll
    for (int j = 0; j < V8; ++j) {
        const int i = t0 + 32 * W * j;
        if (i >= n8) continue;
        const uint4 g = reinterpret_cast<const uint4*>(w)[i];
        const uint32_t a[4] = {v[j].x, v[j].y, v[j].z, v[j].w}, ga[4] = {g.x, g.y, g.z, g.w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = bf2(a[k]), h = bf2(ga[k]);
            o[k] = pack_bf16x2(f.x * r * h.x, f.y * r * h.y);
        }
        yr[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// How the rows of one batch are spread: warps per row (w) and per CTA, CTAs
// per batch (parts).  A row has `vecs` pieces, at most `each` a thread.
struct NormPlan {
    int w, warps, parts;
    long long batches;
};

NormPlan norm_plan(int vecs, int each, int rows, int rpb) {
    NormPlan p;
    p.w = 1;
    while (p.w < 32 && vecs > each * 32 * p.w) p.w *= 2;
    p.warps = p.w <= 8 ? 8 : p.w;
    p.batches = (static_cast<long long>(rows) + rpb - 1) / rpb;
    const int per_sm = p.warps >= 32 ? 1 : 16 / p.warps;
    const int r = p.warps / p.w;
    const long long need = (static_cast<long long>(rpb) + r - 1) / r;        // CTA steps of one batch
    long long parts = (static_cast<long long>(kGb300Sms) * per_sm) / p.batches;
    if (parts > need) parts = need;
    p.parts = static_cast<int>(parts < 1 ? 1 : parts);
    return p;
}

unsigned sum_blocks(long long batches, int nsum, int n4) {
    return static_cast<unsigned>(batches * nsum * ((n4 + 31) / 32));
}

}  // namespace

size_t layernorm_bwd_workspace(int rows, int D, int rpb) {
    if (rows < 1 || D < 4 || rpb < 1) return 0;
    // of the two forms: column sums per batch, or over all rows
    size_t most = 256;
    for (int form = 0; form < 2; ++form) {
        const NormPlan p = norm_plan(D / 4, 5, rows, form ? rows : (rpb < rows ? rpb : rows));
        if (p.parts == 1) continue;
        const size_t n = static_cast<size_t>(p.batches) * p.parts * 2 * D * sizeof(float);
        if (n > most) most = n;
    }
    return most;
}

size_t rmsnorm_bwd_workspace(int rows, int D) {
    if (rows < 1 || D < 8) return 0;
    const NormPlan p = norm_plan(D / 8, 3, rows, rows);
    return 256 + static_cast<size_t>(p.parts) * D * sizeof(float);
}

cudaError_t launch_layernorm_bwd(const void* dy, const float* x, const float* mean, const float* rstd, int rows, int D,
                                 int rpb, const float* scale, int mod_ld, const void* w, const float* dres, float* dx,
                                 float* dshift, float* dscale, int dmod_ld, float* ws, cudaStream_t s,
                                 unsigned long long* launches) {
    // without modulation all rows are one batch
    if (!scale || rpb > rows) rpb = rows;
    const NormPlan p = norm_plan(D / 4, 5, rows, rpb);
    const int kind = scale ? kGainScale : w ? kGainW : kGainOne;
    const void* gain = scale ? static_cast<const void*>(scale) : w;
    // one CTA a batch writes its sums in place, several write partial rows
    const bool direct = p.parts == 1;
    // The sums in the same launch where that is short: at most 2048 rows a slab
    // (64 rows in a row a thread), at most 128 slabs.  In a graph, against the
    // partial rows and their own launch: 1 x 256 x 256 2.2 us (3.9), 2 x 1024 x
    // 1152 7.7 (9.6), 1 x 2048 x 4096 (128 slabs) 30.3 (31.5), but 4 x 1024 x 1152
    // (144) 16.3 (13.6).
    const int slabs = (D + 31) / 32;
    const bool fused = dshift && !direct && p.warps == 8 && rpb <= 2048 && p.batches * slabs <= 128;
    int parts = p.parts;
    if (fused) {
        const long long room = (2 * kGb300Sms - p.batches * slabs) / p.batches;
        if (parts > room) parts = static_cast<int>(room < 1 ? 1 : room);
    }
    float* sums = !dshift || fused ? nullptr : direct ? dshift : ws;
    float* sums2 = !dshift ? nullptr : direct ? dscale : ws + D;
    const size_t sum_ld = direct ? static_cast<size_t>(dmod_ld) : 2 * static_cast<size_t>(D);
    const int r = p.warps / p.w;
    const size_t smem = sums && r > 1 ? static_cast<size_t>(r) * 2 * D * sizeof(float) : 0;
    const int row_ctas = static_cast<int>(p.batches * parts);
    const ColumnWork cw = {row_ctas, slabs, dshift, dscale, dmod_ld};
    const unsigned g = static_cast<unsigned>(row_ctas + (fused ? p.batches * slabs : 0));
    const __nv_bfloat16* d = static_cast<const __nv_bfloat16*>(dy);
    cudaError_t e = cudaErrorInvalidValue;
    const int v4 = (D / 4 + 32 * p.w - 1) / (32 * p.w);
#define DLO_LNB(V, W, N)                                                                                          \
    e = launch_k(layernorm_bwd_kernel<V, W, N>, g, 32 * N, smem, s, d, x, mean, rstd, rows, D, rpb, parts, kind, \
                 gain, mod_ld, dres, dx, sums, sums2, sum_ld, cw)
    if (p.w == 1) {
        if (v4 <= 1) DLO_LNB(1, 1, 8);
        else if (v4 <= 3) DLO_LNB(3, 1, 8);
        else DLO_LNB(5, 1, 8);
    } else if (p.w == 2) {
        if (v4 <= 3) DLO_LNB(3, 2, 8);
        else DLO_LNB(5, 2, 8);
    } else if (p.w == 4) {
        if (v4 <= 3) DLO_LNB(3, 4, 8);
        else DLO_LNB(5, 4, 8);
    } else if (p.w == 8) {
        if (v4 <= 3) DLO_LNB(3, 8, 8);
        else DLO_LNB(5, 8, 8);
    } else if (p.w == 16) {
        DLO_LNB(5, 16, 16);
    } else {
        DLO_LNB(5, 32, 32);
    }
#undef DLO_LNB
    ++*launches;
    if (e != cudaSuccess || !sums || direct) return e != cudaSuccess ? e : cudaGetLastError();
    e = launch_k(column_sums_kernel, sum_blocks(p.batches, 2, D / 4), 1024, 0, s, ws, p.parts, D / 4, 2, dshift, dscale,
                 static_cast<size_t>(dmod_ld));
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_rmsnorm_bwd(const void* dy, int lddy, const void* x, int ldx, const void* w, const float* rstd,
                               int rows, int D, void* dx, int lddx, float* dw, float* ws, cudaStream_t s,
                               unsigned long long* launches) {
    const NormPlan p = norm_plan(D / 8, 3, rows, rows);
    // the sum in the same launch, as in launch_layernorm_bwd (2048 x 4096 rows 14.1
    // us, against 16.1); not in place, where dx takes the place of what the slabs read
    const int slabs = (D + 63) / 64;
    const bool fused = dw && p.parts > 1 && p.warps == 8 && rows <= 2048 && slabs <= 128 && dx != dy && dx != x;
    const int parts = fused && p.parts > 2 * kGb300Sms - slabs ? 2 * kGb300Sms - slabs : p.parts;
    float* sums = !dw || fused ? nullptr : p.parts == 1 ? dw : ws;
    const int r = p.warps / p.w;
    const int v8 = (D / 8 + 32 * p.w - 1) / (32 * p.w), pieces = v8 <= 1 && p.w == 1 ? 1 : 3;
    const size_t ring = static_cast<size_t>(ring_rows(p.warps)) * 2 * pieces * 32 * p.warps * sizeof(uint4);
    const size_t end = sums && r > 1 ? static_cast<size_t>(r) * D * sizeof(float) : 0;
    const size_t smem = ring > end ? ring : end;
    const ColumnWork cw = {parts, slabs, dw, nullptr, 0};
    const unsigned g = static_cast<unsigned>(parts + (fused ? slabs : 0));
    const __nv_bfloat16 *d = static_cast<const __nv_bfloat16*>(dy), *xb = static_cast<const __nv_bfloat16*>(x),
                        *wb = static_cast<const __nv_bfloat16*>(w);
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(dx);
    cudaError_t e = cudaErrorInvalidValue;
#define DLO_RMB(V, W, N) \
    e = launch_big<rmsnorm_bwd_kernel<V, W, N>>(g, 32 * N, smem, s, d, lddy, xb, ldx, wb, rstd, rows, D, parts, o, lddx, sums, cw)
    // three 8-column pieces a thread: with the next row's in registers too, five
    // would spill (8192 x 5120 rows: 89 us, 54 us with three)
    if (p.w == 1) {
        if (v8 <= 1) DLO_RMB(1, 1, 8);
        else DLO_RMB(3, 1, 8);
    } else if (p.w == 2) {
        DLO_RMB(3, 2, 8);
    } else if (p.w == 4) {
        DLO_RMB(3, 4, 8);
    } else if (p.w == 8) {
        DLO_RMB(3, 8, 8);
    } else if (p.w == 16) {
        DLO_RMB(3, 16, 16);
    } else {
        DLO_RMB(3, 32, 32);
    }
#undef DLO_RMB
    ++*launches;
    if (e != cudaSuccess || !sums || sums == dw) return e != cudaSuccess ? e : cudaGetLastError();
    e = launch_k(column_sums_kernel, sum_blocks(1, 1, D / 4), 1024, 0, s, ws, p.parts, D / 4, 1, dw, dw, static_cast<size_t>(0));
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_rmsnorm_fwd(const void* x, int ldx, int rows, int D, const void* w, float eps, void* y, int ldy,
                               float* rstd, cudaStream_t s, unsigned long long* launches) {
    const int n8 = D / 8;
    int wpr = 1;
    while (wpr < 8 && n8 > 5 * 32 * wpr) wpr *= 2;
    const int v8 = (n8 + 32 * wpr - 1) / (32 * wpr);
    const unsigned g = static_cast<unsigned>((static_cast<long long>(rows) + 8 / wpr - 1) / (8 / wpr));
    const __nv_bfloat16 *xb = static_cast<const __nv_bfloat16*>(x), *wb = static_cast<const __nv_bfloat16*>(w);
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(y);
    cudaError_t e = cudaErrorInvalidValue;
#define DLO_RMF(V, W) e = launch_k(rmsnorm_fwd_kernel<V, W>, g, 256, 0, s, xb, ldx, rows, D, wb, eps, o, ldy, rstd)
    if (wpr == 1) {
        if (v8 <= 1) DLO_RMF(1, 1);
        else if (v8 <= 3) DLO_RMF(3, 1);
        else DLO_RMF(5, 1);
    } else if (wpr == 2) {
        if (v8 <= 3) DLO_RMF(3, 2);
        else DLO_RMF(5, 2);
    } else if (wpr == 4) {
        if (v8 <= 3) DLO_RMF(3, 4);
        else DLO_RMF(5, 4);
    } else {
        if (v8 <= 5) DLO_RMF(5, 8);
        else DLO_RMF(10, 8);
    }
#undef DLO_RMF
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dlo
