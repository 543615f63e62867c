// C entries of the training ops: argument checks, then one launcher each.
#include "internal.h"

using namespace dlo;

namespace {

constexpr int kMaxRows = 1 << 30;
constexpr int kMaxNormDim = 20480;

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

dlo_status inval(const char* m) { return op_fail(DLO_EINVAL, m); }

const char* attn_problem(const dlo_attn* a) {
    if (!a) return "NULL description";
    if (a->batch < 1 || a->heads < 1 || a->kv_heads < 1 || a->nq < 1 || a->nk < 1) return "sizes must be >= 1";
    if (a->batch > 65535 || a->heads > 65535) return "batch and heads must be <= 65535";
    if (a->heads % a->kv_heads) return "heads % kv_heads != 0";
    if (a->head_dim < 8 || a->head_dim % 8 || a->head_dim > 128) return "head_dim % 8 != 0 or > 128";
    if (static_cast<long long>(a->batch) * a->nq > kMaxRows || static_cast<long long>(a->batch) * a->nk > kMaxRows)
        return "more than 2^30 rows";
    if (a->causal_block < 0) return "causal_block must be >= 0";
    return nullptr;
}

// The int32 operands, read where a kernel starts.
bool bad_words(const dlo_attn* a, const int* err) {
    return !aligned_to(a->q_lens, 4) || !aligned_to(a->k_lens, 4) || !aligned_to(err, 4);
}

bool bad_ld(int ld, int heads, int head_dim) { return ld % 8 || ld < heads * head_dim; }

}  // namespace

extern "C" size_t dlo_attention_fwd_workspace_bytes(const dlo_attn* a) {
    if (const char* m = attn_problem(a)) return inval(m), 0;
    return attention_fwd_workspace(*a);
}

extern "C" size_t dlo_attention_bwd_workspace_bytes(const dlo_attn* a) {
    if (const char* m = attn_problem(a)) return inval(m), 0;
    return attention_bwd_workspace(*a);
}

extern "C" dlo_status dlo_op_attention_fwd(const dlo_attn* a, const void* Q, const void* K, const void* V, void* O,
                                           float* lse, void* ws, size_t ws_bytes, int* err, void* stream) {
    if (const char* m = attn_problem(a)) return inval(m);
    if (!Q || !K || !V || !O || !lse) return inval("NULL operand");
    if (bad_ld(a->ldq, a->heads, a->head_dim) || bad_ld(a->ldk, a->kv_heads, a->head_dim) ||
        bad_ld(a->ldv, a->kv_heads, a->head_dim) || bad_ld(a->ldo, a->heads, a->head_dim))
        return inval("ld % 8 != 0 or smaller than its row");
    if (!aligned_to(Q, 16) || !aligned_to(K, 16) || !aligned_to(V, 16) || !aligned_to(O, 16) || !aligned_to(lse, 4) ||
        bad_words(a, err))
        return inval("alignment");
    const size_t need = attention_fwd_workspace(*a);
    if (ws_bytes < need) return op_fail(DLO_ENOMEM, "workspace too small");
    if (need && (!ws || !aligned_to(ws, 256))) return inval("workspace must be 256-byte aligned");
    return op_result(launch_attention_fwd(*a, Q, K, V, O, lse, ws, err, static_cast<cudaStream_t>(stream),
                                          Uncounted()));
}

extern "C" dlo_status dlo_op_attention_bwd(const dlo_attn* a, const void* Q, const void* K, const void* V,
                                           const void* O, const float* lse, const void* dO, void* dQ, void* dK,
                                           void* dV, void* ws, size_t ws_bytes, int* err, void* stream) {
    if (const char* m = attn_problem(a)) return inval(m);
    if (!Q || !K || !V || !O || !lse || !dO || !dQ || !dK || !dV) return inval("NULL operand");
    if (bad_ld(a->ldq, a->heads, a->head_dim) || bad_ld(a->ldk, a->kv_heads, a->head_dim) ||
        bad_ld(a->ldv, a->kv_heads, a->head_dim) || bad_ld(a->ldo, a->heads, a->head_dim) ||
        bad_ld(a->lddq, a->heads, a->head_dim) || bad_ld(a->lddk, a->kv_heads, a->head_dim) ||
        bad_ld(a->lddv, a->kv_heads, a->head_dim) || bad_ld(a->lddo, a->heads, a->head_dim))
        return inval("ld % 8 != 0 or smaller than its row");
    for (const void* p : {Q, K, V, O, dO, static_cast<const void*>(dQ), static_cast<const void*>(dK),
                          static_cast<const void*>(dV)})
        if (!aligned_to(p, 16)) return inval("alignment");
    if (!aligned_to(lse, 4) || bad_words(a, err)) return inval("alignment");
    if (ws_bytes < attention_bwd_workspace(*a)) return op_fail(DLO_ENOMEM, "workspace too small");
    if (!ws || !aligned_to(ws, 256)) return inval("workspace must be 256-byte aligned");
    return op_result(launch_attention_bwd(*a, Q, K, V, O, lse, dO, dQ, dK, dV, ws, err,
                                          static_cast<cudaStream_t>(stream), Uncounted()));
}

extern "C" dlo_status dlo_op_layernorm_fwd(const float* x, int rows, int D, int rows_per_batch, const float* shift,
                                           const float* scale, int mod_ld, const void* w, const void* b, float eps,
                                           void* out, float* mean, float* rstd, void* stream) {
    if (!x || !out || !mean || !rstd) return inval("NULL operand");
    if (rows < 1 || rows > kMaxRows || D < 4 || D % 4 || D > kMaxNormDim || rows_per_batch < 1)
        return inval("need 1 <= rows <= 2^30, D % 4 == 0, 4 <= D <= 20480, rows_per_batch >= 1");
    if ((shift == nullptr) != (scale == nullptr) || (w == nullptr) != (b == nullptr) || (scale && w)) return inval("pairs");
    if (!(eps > 0.f)) return inval("eps must be > 0");
    if (scale && (mod_ld % 4 || mod_ld < D || !aligned_to(scale, 16) || !aligned_to(shift, 16))) return inval("mod layout");
    if (!aligned_to(x, 16) || !aligned_to(out, 8) || !aligned_to(w, 8) || !aligned_to(b, 8) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4))
        return inval("alignment");
    return op_result(launch_layernorm(x, rows, D, rows_per_batch, shift, scale, mod_ld, w, b, eps, out,
                                      static_cast<cudaStream_t>(stream), Uncounted(), mean, rstd));
}

extern "C" size_t dlo_layernorm_bwd_workspace_bytes(int rows, int D, int rows_per_batch) {
    if (rows < 1 || rows > kMaxRows || D < 4 || D % 4 || D > kMaxNormDim || rows_per_batch < 1)
        return inval("layernorm sizes"), 0;
    return layernorm_bwd_workspace(rows, D, rows_per_batch);
}

extern "C" dlo_status dlo_op_layernorm_bwd(const void* dy, const float* x, const float* mean, const float* rstd,
                                           int rows, int D, int rows_per_batch, const float* scale, int mod_ld,
                                           const void* w, const float* dres, float* dx, float* dshift, float* dscale,
                                           int dmod_ld, void* ws, size_t ws_bytes, void* stream) {
    if (!dy || !x || !mean || !rstd || !dx) return inval("NULL operand");
    if (rows < 1 || rows > kMaxRows || D < 4 || D % 4 || D > kMaxNormDim || rows_per_batch < 1)
        return inval("need 1 <= rows <= 2^30, D % 4 == 0, 4 <= D <= 20480, rows_per_batch >= 1");
    if (scale && w) return inval("scale and w");
    if ((dshift == nullptr) != (dscale == nullptr) || (dshift && !scale && !w)) return inval("pairs");
    if (scale && (mod_ld % 4 || mod_ld < D || !aligned_to(scale, 16))) return inval("mod layout");
    if (dshift && scale && (dmod_ld % 4 || dmod_ld < D)) return inval("mod layout");
    if (!aligned_to(x, 16) || !aligned_to(dres, 16) || !aligned_to(dx, 16) || !aligned_to(dshift, 16) ||
        !aligned_to(dscale, 16) || !aligned_to(dy, 8) || !aligned_to(w, 8) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return inval("alignment");
    if (dshift) {
        if (ws_bytes < layernorm_bwd_workspace(rows, D, rows_per_batch)) return op_fail(DLO_ENOMEM, "workspace too small");
        if (!ws || !aligned_to(ws, 16)) return inval("workspace must be 16-byte aligned");
    }
    return op_result(launch_layernorm_bwd(dy, x, mean, rstd, rows, D, rows_per_batch, scale, mod_ld, w, dres, dx, dshift,
                                          dscale, scale ? dmod_ld : D, static_cast<float*>(ws),
                                          static_cast<cudaStream_t>(stream), Uncounted()));
}

extern "C" dlo_status dlo_op_rmsnorm_fwd(const void* x, int ldx, int rows, int D, const void* w, float eps, void* y,
                                         int ldy, float* rstd, void* stream) {
    if (!x || !w || !y || !rstd) return inval("NULL operand");
    if (rows < 1 || rows > kMaxRows || D < 8 || D % 8 || D > kMaxNormDim)
        return inval("need 1 <= rows <= 2^30, D % 8 == 0, 8 <= D <= 20480");
    if (ldx % 8 || ldx < D || ldy % 8 || ldy < D) return inval("ld % 8 != 0 or smaller than D");
    if (!(eps > 0.f)) return inval("eps must be > 0");
    if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(y, 16) || !aligned_to(rstd, 4)) return inval("alignment");
    return op_result(launch_rmsnorm_fwd(x, ldx, rows, D, w, eps, y, ldy, rstd, static_cast<cudaStream_t>(stream),
                                        Uncounted()));
}

extern "C" size_t dlo_rmsnorm_bwd_workspace_bytes(int rows, int D) {
    if (rows < 1 || rows > kMaxRows || D < 8 || D % 8 || D > kMaxNormDim) return inval("rmsnorm sizes"), 0;
    return rmsnorm_bwd_workspace(rows, D);
}

extern "C" dlo_status dlo_op_rmsnorm_bwd(const void* dy, int lddy, const void* x, int ldx, const void* w,
                                         const float* rstd, int rows, int D, void* dx, int lddx, float* dw, void* ws,
                                         size_t ws_bytes, void* stream) {
    if (!dy || !x || !w || !rstd || !dx) return inval("NULL operand");
    if (rows < 1 || rows > kMaxRows || D < 8 || D % 8 || D > kMaxNormDim)
        return inval("need 1 <= rows <= 2^30, D % 8 == 0, 8 <= D <= 20480");
    if (lddy % 8 || lddy < D || ldx % 8 || ldx < D || lddx % 8 || lddx < D) return inval("ld % 8 != 0 or smaller than D");
    if ((dx == dy && lddx != lddy) || (dx == x && lddx != ldx)) return inval("in place needs the same stride");
    if (!aligned_to(dy, 16) || !aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(dx, 16) || !aligned_to(dw, 16) ||
        !aligned_to(rstd, 4))
        return inval("alignment");
    if (dw) {
        if (ws_bytes < rmsnorm_bwd_workspace(rows, D)) return op_fail(DLO_ENOMEM, "workspace too small");
        if (!ws || !aligned_to(ws, 16)) return inval("workspace must be 16-byte aligned");
    }
    return op_result(launch_rmsnorm_bwd(dy, lddy, x, ldx, w, rstd, rows, D, dx, lddx, dw, static_cast<float*>(ws),
                                        static_cast<cudaStream_t>(stream), Uncounted()));
}
