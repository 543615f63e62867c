// C entries of the operators for packed batches: argument checks, then one
// launcher each; the table of rotary steps.
#include <cmath>

#include "internal.h"

using namespace dlo;

namespace {

constexpr int kMaxRows = 1 << 30;
constexpr int kMaxSeqs = 65535;

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

dlo_status inval(const char* m) { return op_fail(DLO_EINVAL, m); }

const char* attn_problem(const dlo_attn_packed* a) {
    if (!a) return "NULL description";
    if (a->batch < 1 || a->heads < 1 || a->kv_heads < 1 || a->rows_q < 1 || a->rows_k < 1) return "sizes must be >= 1";
    if (a->batch > kMaxSeqs || a->heads > 65535) return "batch and heads must be <= 65535";
    if (a->heads % a->kv_heads) return "heads % kv_heads != 0";
    if (a->head_dim < 8 || a->head_dim % 8 || a->head_dim > 128) return "head_dim % 8 != 0 or > 128";
    if (a->rows_q > kMaxRows || a->rows_k > kMaxRows) return "more than 2^30 rows";
    if (a->causal_block < 0) return "causal_block must be >= 0";
    return nullptr;
}

// What a kernel reads as int32 where it starts.
const char* attn_words(const dlo_attn_packed* a, const int* err) {
    if (!a->q_starts || !a->k_starts) return "NULL starts";
    return aligned_to(a->q_starts, 4) && aligned_to(a->k_starts, 4) && aligned_to(err, 4) ? nullptr : "alignment";
}

bool bad_ld(int ld, int heads, int head_dim) { return ld % 8 || ld < heads * head_dim; }

const char* rope_problem(const dlo_rope* r) {
    if (!r) return "NULL description";
    if (r->heads < 1 || r->heads > 65535) return "heads must be 1 .. 65535";
    if (r->head_dim < 8 || r->head_dim % 8 || r->head_dim > 256) return "head_dim % 8 != 0 or > 256";
    if (r->layout != DLO_ROPE_HALF && r->layout != DLO_ROPE_INTERLEAVED) return "layout";
    if (r->axes < 1 || r->axes > DLO_ROPE_AXES) return "axes must be 1 .. 4";
    if (!std::isfinite(r->amp)) return "amp must be finite";
    int columns = 0;
    for (int i = 0; i < r->axes; ++i) {
        const dlo_rope_axis& a = r->axis[i];
        if (a.dim < 2 || a.dim % 2 || a.dim > r->head_dim) return "dim must be even, 2 .. head_dim";
        columns += a.dim;
        if (!(a.theta > 1.0) || !std::isfinite(a.theta)) return "theta must be finite and > 1";
        if (a.scaling < DLO_ROPE_PLAIN || a.scaling > DLO_ROPE_BY_INDEX) return "scaling";
        if (a.scaling == DLO_ROPE_PLAIN) continue;
        if (!(a.factor >= 1.0) || !std::isfinite(a.factor)) return "factor must be finite and >= 1";
        if (a.scaling == DLO_ROPE_LINEAR || a.scaling == DLO_ROPE_BASE) continue;
        if (!(a.length > 0.0) || !std::isfinite(a.length)) return "length must be finite and > 0";
        if (!(a.slow > 0.0) || !(a.fast > a.slow) || !std::isfinite(a.fast)) return "need 0 < slow < fast";
    }
    if (columns > r->head_dim) return "the axes have more columns than a head";
    return nullptr;
}

// The layout that the two ops need beside the angles.
const char* rope_rows(const dlo_rope* r) {
    if (bad_ld(r->ldx, r->heads, r->head_dim) || bad_ld(r->ldy, r->heads, r->head_dim))
        return "ld % 8 != 0 or smaller than its row";
    return nullptr;
}

dlo_status rope(const dlo_rope* r, bool back, const void* in, int ld_in, const int* positions, const uint64_t* steps,
                int rows, void* out, int ld_out, void* stream) {
    if (!in || !positions || !steps || !out) return inval("NULL operand");
    if (rows < 1 || rows > kMaxRows) return inval("need 1 <= rows <= 2^30");
    if (in == out && ld_in != ld_out) return inval("in place needs the same stride");
    if (!aligned_to(in, 16) || !aligned_to(out, 16) || !aligned_to(positions, 4) || !aligned_to(steps, 8)) return inval("alignment");
    return op_result(launch_rope(*r, back, in, ld_in, positions, steps, rows, out, ld_out, static_cast<cudaStream_t>(stream),
                                 Uncounted()));
}

double clamp01(double v) { return v < 0.0 ? 0.0 : v > 1.0 ? 1.0 : v; }

}  // namespace

extern "C" dlo_status dlo_op_packed_plan(const int* grids, const int* offsets, int batch, int axes, int rows, int* starts,
                                         int* positions, void* stream) {
    if (!grids || !starts) return inval("NULL operand");
    if (batch < 1 || batch > kMaxSeqs) return inval("batch must be 1 .. 65535");
    if (axes < 1 || axes > DLO_ROPE_AXES) return inval("axes must be 1 .. 4");
    if (rows < 1 || rows > kMaxRows) return inval("need 1 <= rows <= 2^30");
    if (!aligned_to(grids, 4) || !aligned_to(offsets, 4) || !aligned_to(starts, 4) || !aligned_to(positions, 4))
        return inval("alignment");
    return op_result(launch_packed_plan(grids, offsets, batch, axes, rows, starts, positions,
                                        static_cast<cudaStream_t>(stream), Uncounted()));
}

// A step's error in turns, u = 2^-53: the exponent, pow (2 u), the divisions and 2 pi leave
// f u (|ln f| + 4), a factor or base up to 3 u f more, over 2 pi: less than 2 u, as f <= 1.  Blended,
// k of f length / 2 pi <= fast turns adds 2 u (|ln f| + 7) f with fast >= 2 slow: less than 4 u in all.
extern "C" dlo_status dlo_rope_steps(const dlo_rope* r, uint64_t* steps, int n) {
    if (const char* m = rope_problem(r)) return inval(m);
    if (!steps) return inval("NULL steps");
    int pairs = 0;
    for (int i = 0; i < r->axes; ++i) pairs += r->axis[i].dim / 2;
    if (n != pairs) return inval("n must be the pairs of a head");
    const double two_pi = 6.283185307179586476925;
    for (int i = 0; i < r->axes; ++i) {
        const dlo_rope_axis& a = r->axis[i];
        double theta = a.theta;
        if (a.scaling == DLO_ROPE_BASE && a.dim > 2) theta *= std::pow(a.factor, a.dim / (a.dim - 2.0));
        double low = 0.0, high = 0.0;          // DLO_ROPE_BY_INDEX: kept below, divided above
        if (a.scaling == DLO_ROPE_BY_INDEX) {
            const auto index = [&](double turns) { return a.dim * std::log(a.length / (two_pi * turns)) / (2.0 * std::log(theta)); };
            low = std::fmax(std::floor(index(a.fast)), 0.0);
            high = std::fmin(std::ceil(index(a.slow)), a.dim - 1.0);
        }
        for (int p = 0; p < a.dim / 2; ++p) {
            double f = std::pow(theta, -2.0 * p / a.dim);
            double keep = 1.0;
            if (a.scaling == DLO_ROPE_LINEAR) keep = 0.0;
            if (a.scaling == DLO_ROPE_BY_TURNS) keep = clamp01((a.length * f / two_pi - a.slow) / (a.fast - a.slow));
            if (a.scaling == DLO_ROPE_BY_INDEX) keep = 1.0 - clamp01((p - low) / std::fmax(high - low, 0.001));
            if (keep < 1.0) f *= keep + (1.0 - keep) / a.factor;
            // f <= 1, so at most 2^64 / 2 pi
            *steps++ = static_cast<uint64_t>(std::nearbyint(f / two_pi * 18446744073709551616.0));
        }
    }
    return DLO_OK;
}

extern "C" dlo_status dlo_op_rope_fwd(const dlo_rope* r, const void* x, const int* positions, const uint64_t* steps, int rows,
                                      void* y, void* stream) {
    if (const char* m = rope_problem(r)) return inval(m);
    if (const char* m = rope_rows(r)) return inval(m);
    return rope(r, false, x, r->ldx, positions, steps, rows, y, r->ldy, stream);
}

extern "C" dlo_status dlo_op_rope_bwd(const dlo_rope* r, const void* dy, const int* positions, const uint64_t* steps, int rows,
                                      void* dx, void* stream) {
    if (const char* m = rope_problem(r)) return inval(m);
    if (const char* m = rope_rows(r)) return inval(m);
    return rope(r, true, dy, r->ldy, positions, steps, rows, dx, r->ldx, stream);
}

extern "C" size_t dlo_attention_packed_fwd_workspace_bytes(const dlo_attn_packed* a) {
    if (const char* m = attn_problem(a)) return inval(m), 0;
    return attention_packed_fwd_workspace(*a);
}

extern "C" size_t dlo_attention_packed_bwd_workspace_bytes(const dlo_attn_packed* a) {
    if (const char* m = attn_problem(a)) return inval(m), 0;
    return attention_packed_bwd_workspace(*a);
}

extern "C" dlo_status dlo_op_attention_packed_fwd(const dlo_attn_packed* a, const void* Q, const void* K, const void* V, void* O,
                                                  float* lse, void* ws, size_t ws_bytes, int* err, void* stream) {
    if (const char* m = attn_problem(a)) return inval(m);
    if (!Q || !K || !V || !O || !lse) return inval("NULL operand");
    if (const char* m = attn_words(a, err)) return inval(m);
    if (bad_ld(a->ldq, a->heads, a->head_dim) || bad_ld(a->ldk, a->kv_heads, a->head_dim) ||
        bad_ld(a->ldv, a->kv_heads, a->head_dim) || bad_ld(a->ldo, a->heads, a->head_dim))
        return inval("ld % 8 != 0 or smaller than its row");
    if (!aligned_to(Q, 16) || !aligned_to(K, 16) || !aligned_to(V, 16) || !aligned_to(O, 16) || !aligned_to(lse, 4))
        return inval("alignment");
    if (ws_bytes < attention_packed_fwd_workspace(*a)) return op_fail(DLO_ENOMEM, "workspace too small");
    if (!ws || !aligned_to(ws, 256)) return inval("workspace must be 256-byte aligned");
    return op_result(launch_attention_packed_fwd(*a, Q, K, V, O, lse, ws, err, static_cast<cudaStream_t>(stream), Uncounted()));
}

extern "C" dlo_status dlo_op_attention_packed_bwd(const dlo_attn_packed* a, const void* Q, const void* K, const void* V,
                                                  const void* O, const float* lse, const void* dO, void* dQ, void* dK, void* dV,
                                                  void* ws, size_t ws_bytes, int* err, void* stream) {
    if (const char* m = attn_problem(a)) return inval(m);
    if (!Q || !K || !V || !O || !lse || !dO || !dQ || !dK || !dV) return inval("NULL operand");
    if (const char* m = attn_words(a, err)) return inval(m);
    if (bad_ld(a->ldq, a->heads, a->head_dim) || bad_ld(a->ldk, a->kv_heads, a->head_dim) ||
        bad_ld(a->ldv, a->kv_heads, a->head_dim) || bad_ld(a->ldo, a->heads, a->head_dim) ||
        bad_ld(a->lddq, a->heads, a->head_dim) || bad_ld(a->lddk, a->kv_heads, a->head_dim) ||
        bad_ld(a->lddv, a->kv_heads, a->head_dim) || bad_ld(a->lddo, a->heads, a->head_dim))
        return inval("ld % 8 != 0 or smaller than its row");
    for (const void* p : {Q, K, V, O, dO, static_cast<const void*>(dQ), static_cast<const void*>(dK),
                          static_cast<const void*>(dV)})
        if (!aligned_to(p, 16)) return inval("alignment");
    if (!aligned_to(lse, 4)) return inval("alignment");
    if (ws_bytes < attention_packed_bwd_workspace(*a)) return op_fail(DLO_ENOMEM, "workspace too small");
    if (!ws || !aligned_to(ws, 256)) return inval("workspace must be 256-byte aligned");
    return op_result(launch_attention_packed_bwd(*a, Q, K, V, O, lse, dO, dQ, dK, dV, ws, err, static_cast<cudaStream_t>(stream),
                                                 Uncounted()));
}
