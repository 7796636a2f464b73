// abi_block.cu -- C entry points of the training block's operators (norm with
// residual and gate, rotary positions, packed causal attention, gradient
// clipping): argument checks, then the launches.
#include <cmath>

#include "internal.h"
#include "nvtx_range.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool given16(const void* p) { return p && aligned16(p); }

int device_ok() {
    int dev = 0, sms = 0;
    return moe::current_device(&dev, &sms);
}

// A sum over no terms: n floats at p (NULL: not wanted) become 0.
int zero_sum(void* p, int64_t n, void* stream) {
    if (!p) return MOE_OK;
    if (const int rc = device_ok()) return rc;
    return cudaMemsetAsync(p, 0, n * 4, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK : MOE_ECUDA;
}

// Strides of a [T, heads, D] tensor: 16-byte steps wide enough that two rows
// of heads never share an element (an extent of one has no stride).
bool strides_ok(int64_t T, int64_t heads, int64_t D, int64_t st_t, int64_t st_h) {
    if ((T > 1 && (st_t % 8 || st_t < D || st_t >= (1ll << 38))) ||
        (heads > 1 && (st_h % 8 || st_h < D || st_h >= (1ll << 38))))
        return false;
    if (T > 1 && heads > 1)   // (T - 1) st_t may pass 64 bits
        return st_t >= st_h ? st_t >= (heads - 1) * st_h + D : (st_h - D) / st_t >= T - 1;
    return true;
}

int norm_ok(const moe_norm_t* c) {
    if (!c || c->T < 0 || c->d < 8 || c->d > 8192 || c->d % 8 || (c->res_f32 & ~1) ||
        (c->gate_per_token & ~1) || !std::isfinite(c->alpha) || !std::isfinite(c->beta) ||
        !(c->eps >= 0) || !std::isfinite(c->eps))
        return MOE_EINVAL;
    return MOE_OK;
}

int attention_ok(const moe_attention_t* c) {
    if (!c || c->T < 0 || c->T >= (1ll << 31) - 256 || c->n_seqs < 0 || c->n_seqs > (1 << 24) ||
        c->n_heads <= 0 || c->n_kv_heads <= 0 || c->n_heads % c->n_kv_heads ||
        c->n_heads > 65536 || c->head_dim < 8 || c->head_dim > 128 || c->head_dim % 8 ||
        !(c->scale > 0) || !std::isfinite(c->scale) || c->reserved)
        return MOE_EINVAL;
    return MOE_OK;
}

bool qkvo_strides_ok(const moe_attention_t* c) {
    return strides_ok(c->T, c->n_heads, c->head_dim, c->q_t, c->q_h) &&
           strides_ok(c->T, c->n_kv_heads, c->head_dim, c->k_t, c->k_h) &&
           strides_ok(c->T, c->n_kv_heads, c->head_dim, c->v_t, c->v_h) &&
           strides_ok(c->T, c->n_heads, c->head_dim, c->o_t, c->o_h);
}

}  // namespace

extern "C" {

int moe_norm_residual(const moe_norm_t* cfg, const uint16_t* b, const void* r,
                      const uint16_t* gate, const uint16_t* w_post, const uint16_t* w_pre,
                      void* y, uint16_t* n, float* rstd_post, float* rstd_pre, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = norm_ok(cfg)) return rc;
    if (cfg->T == 0) return MOE_OK;
    // a branch comes with its weight, a next norm with its own; one of them
    if (!given16(r) || !b != !w_post || !n != !w_pre || (!b && !n) || (gate && !b) ||
        !aligned16(b) || !aligned16(gate) || !aligned16(w_post) || !aligned16(w_pre) ||
        !aligned16(y) || !aligned16(n) || (!y && !n) || (rstd_post && !b) || (rstd_pre && !n))
        return MOE_EINVAL;
    if (const int rc = device_ok()) return rc;
    return moe::launch_norm_residual(*cfg, b, r, gate, w_post, w_pre, y, n, rstd_post, rstd_pre,
                                     static_cast<cudaStream_t>(stream));
}

int moe_norm_residual_workspace(int64_t T, int32_t d, int64_t* bytes) {
    if (!bytes || T < 0 || d < 8 || d > 8192 || d % 8) return MOE_EINVAL;
    *bytes = moe::norm_backward_ws(T, d);
    return MOE_OK;
}

int moe_norm_residual_backward(const moe_norm_t* cfg, const uint16_t* dn, const void* dy,
                               const uint16_t* b, const void* r, const uint16_t* gate,
                               const uint16_t* w_post, const uint16_t* w_pre,
                               const float* rstd_post, const float* rstd_pre, uint16_t* db,
                               void* dr, void* dgate, float* dw_post, float* dw_pre, void* ws,
                               int64_t ws_bytes, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = norm_ok(cfg)) return rc;
    if (cfg->T == 0) {
        if (const int rc = zero_sum(dw_post, cfg->d, stream)) return rc;
        if (const int rc = zero_sum(dw_pre, cfg->d, stream)) return rc;
        return zero_sum(cfg->gate_per_token ? nullptr : dgate, cfg->d, stream);
    }
    const bool has_b = b != nullptr, has_n = dn != nullptr;
    if (!has_b && !has_n) return MOE_EINVAL;
    if (!dn && !dy) return MOE_EINVAL;
    if (has_b != (w_post != nullptr) || has_b != (db != nullptr) || has_b != (dw_post != nullptr) ||
        has_b != (rstd_post != nullptr))
        return MOE_EINVAL;
    if (has_n != (w_pre != nullptr) || has_n != (dw_pre != nullptr) ||
        has_n != (rstd_pre != nullptr) || (has_n && !r))
        return MOE_EINVAL;
    if ((gate && !has_b) || (gate != nullptr) != (dgate != nullptr) || !given16(dr) ||
        !given16(ws) || !aligned16(dn) || !aligned16(dy) || !aligned16(b) || !aligned16(r) ||
        !aligned16(gate) || !aligned16(w_post) || !aligned16(w_pre) || !aligned16(db) ||
        !aligned16(dgate))
        return MOE_EINVAL;
    if (ws_bytes < moe::norm_backward_ws(cfg->T, cfg->d)) return MOE_ENOSPC;
    if (const int rc = device_ok()) return rc;
    return moe::launch_norm_residual_backward(*cfg, dn, dy, b, r, gate, w_post, w_pre, rstd_post,
                                              rstd_pre, db, dr, dgate, dw_post, dw_pre, ws,
                                              static_cast<cudaStream_t>(stream));
}

int moe_rotary_make_table(const moe_rotary_table_t* cfg, float* table, void* stream) {
    MOE_NVTX_RANGE();
    if (!cfg || cfg->rows < 0 || cfg->rot_dim < 2 || cfg->rot_dim % 2 || cfg->rot_dim > 1024 ||
        cfg->scaling < 0 || cfg->scaling > 3 || !(cfg->base > 1) || !std::isfinite(cfg->base) ||
        !(cfg->factor >= 1) || !std::isfinite(cfg->factor) || !(cfg->magnitude > 0) ||
        !std::isfinite(cfg->magnitude))
        return MOE_EINVAL;
    if (cfg->scaling == 0 && cfg->factor != 1) return MOE_EINVAL;
    if (cfg->scaling == 2 && cfg->rot_dim <= 2) return MOE_EINVAL;
    if (cfg->scaling == 3 && (!(cfg->orig_len > 0) || !std::isfinite(cfg->orig_len) ||
                              !(cfg->beta_slow >= 0) || !(cfg->beta_fast > cfg->beta_slow) ||
                              !std::isfinite(cfg->beta_fast)))
        return MOE_EINVAL;
    if (cfg->rows == 0) return MOE_OK;
    if (!given16(table)) return MOE_EINVAL;
    if (const int rc = device_ok()) return rc;
    return moe::launch_rotary_table(*cfg, table, static_cast<cudaStream_t>(stream));
}

int moe_rotary(const moe_rotary_t* cfg, const uint16_t* q, const uint16_t* k, const float* table,
               const int32_t* pos, uint16_t* q_out, uint16_t* k_out, int32_t* status,
               void* stream) {
    MOE_NVTX_RANGE();
    if (!cfg || cfg->T < 0 || cfg->hq <= 0 || cfg->hk < 0 || cfg->hq > 65536 ||
        cfg->hk > 65536 || cfg->D < 16 || cfg->D > 1024 || cfg->D % 8 || cfg->rot_dim < 16 ||
        cfg->rot_dim % 16 || cfg->rot_dim > cfg->D || (cfg->interleaved & ~1) ||
        (cfg->inverse & ~1) || cfg->table_rows <= 0)
        return MOE_EINVAL;
    if (!strides_ok(cfg->T, cfg->hq, cfg->D, cfg->q_t, cfg->q_h) ||
        !strides_ok(cfg->T, cfg->hq, cfg->D, cfg->qo_t, cfg->qo_h) ||
        (cfg->hk && (!strides_ok(cfg->T, cfg->hk, cfg->D, cfg->k_t, cfg->k_h) ||
                     !strides_ok(cfg->T, cfg->hk, cfg->D, cfg->ko_t, cfg->ko_h))))
        return MOE_EINVAL;
    if (cfg->T == 0) return MOE_OK;
    if (!given16(q) || !given16(q_out) || !given16(table) || !status ||
        (cfg->hk > 0) != (k != nullptr) || (cfg->hk > 0) != (k_out != nullptr) || !aligned16(k) ||
        !aligned16(k_out))
        return MOE_EINVAL;
    // in place means the same strides
    if ((q == q_out && cfg->T > 1 && cfg->q_t != cfg->qo_t) ||
        (q == q_out && cfg->hq > 1 && cfg->q_h != cfg->qo_h) ||
        (k && k == k_out && cfg->T > 1 && cfg->k_t != cfg->ko_t) ||
        (k && k == k_out && cfg->hk > 1 && cfg->k_h != cfg->ko_h))
        return MOE_EINVAL;
    if (const int rc = device_ok()) return rc;
    return moe::launch_rotary(*cfg, q, k, table, pos, q_out, k_out, status,
                              static_cast<cudaStream_t>(stream));
}

int moe_attention_workspace(const moe_attention_t* cfg, int64_t* plan_bytes,
                            int64_t* backward_bytes) {
    if (const int rc = attention_ok(cfg)) return rc;
    if (!plan_bytes || !backward_bytes) return MOE_EINVAL;
    *plan_bytes = moe::attention_plan_bytes(cfg->T, cfg->n_seqs);
    *backward_bytes = moe::attention_backward_ws(cfg->T, cfg->n_heads);
    return MOE_OK;
}

int moe_attention_plan(const moe_attention_t* cfg, const int32_t* cu, void* plan,
                       int64_t plan_bytes, int32_t* status, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = attention_ok(cfg)) return rc;
    if (cfg->T == 0) return MOE_OK;
    if (!cu || !given16(plan) || !status) return MOE_EINVAL;
    if (plan_bytes < moe::attention_plan_bytes(cfg->T, cfg->n_seqs)) return MOE_ENOSPC;
    if (const int rc = device_ok()) return rc;
    return moe::launch_attention_plan(cfg->T, cfg->n_seqs, cu, plan, status,
                                      static_cast<cudaStream_t>(stream));
}

int moe_attention_forward(const moe_attention_t* cfg, const void* plan, const uint16_t* q,
                          const uint16_t* k, const uint16_t* v, uint16_t* out, uint16_t* rest,
                          float* lse, int32_t* status, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = attention_ok(cfg)) return rc;
    if (cfg->T == 0) return MOE_OK;
    if (!qkvo_strides_ok(cfg)) return MOE_EINVAL;
    if (!given16(plan) || !given16(q) || !given16(k) || !given16(v) || !given16(out) ||
        !aligned16(rest) || !lse || !status)
        return MOE_EINVAL;
    if (const int rc = device_ok()) return rc;
    return moe::launch_attention_fwd(*cfg, plan, q, k, v, out, rest, lse, status,
                                     static_cast<cudaStream_t>(stream));
}

int moe_attention_backward(const moe_attention_t* cfg, const void* plan, const uint16_t* q,
                           const uint16_t* k, const uint16_t* v, const uint16_t* out,
                           const uint16_t* rest, const float* lse, const uint16_t* dout,
                           uint16_t* dq, uint16_t* dk, uint16_t* dv, void* ws, int64_t ws_bytes,
                           int32_t* status, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = attention_ok(cfg)) return rc;
    if (cfg->T == 0) return MOE_OK;
    if (!qkvo_strides_ok(cfg) ||
        !strides_ok(cfg->T, cfg->n_heads, cfg->head_dim, cfg->do_t, cfg->do_h) ||
        !strides_ok(cfg->T, cfg->n_heads, cfg->head_dim, cfg->dq_t, cfg->dq_h) ||
        !strides_ok(cfg->T, cfg->n_kv_heads, cfg->head_dim, cfg->dk_t, cfg->dk_h) ||
        !strides_ok(cfg->T, cfg->n_kv_heads, cfg->head_dim, cfg->dv_t, cfg->dv_h))
        return MOE_EINVAL;
    if (!given16(plan) || !given16(q) || !given16(k) || !given16(v) || !given16(out) ||
        !given16(rest) || !lse || !given16(dout) || !given16(dq) || !given16(dk) ||
        !given16(dv) || !given16(ws) || !status)
        return MOE_EINVAL;
    if (ws_bytes < moe::attention_backward_ws(cfg->T, cfg->n_heads)) return MOE_ENOSPC;
    if (const int rc = device_ok()) return rc;
    return moe::launch_attention_bwd(*cfg, plan, q, k, v, out, rest, lse, dout, dq, dk, dv, ws,
                                     status, static_cast<cudaStream_t>(stream));
}

int moe_grad_clip_workspace(int64_t n_tensors, int64_t* bytes) {
    if (!bytes || n_tensors < 0 || n_tensors > (1 << 20)) return MOE_EINVAL;
    *bytes = moe::grad_clip_ws(n_tensors);
    return MOE_OK;
}

int moe_grad_clip(const moe_grad_tensor_t* tensors, int64_t n_tensors, float max_norm,
                  float* norm, void* ws, int64_t ws_bytes, void* stream) {
    MOE_NVTX_RANGE();
    if (n_tensors < 0 || n_tensors > (1 << 20) || !(max_norm > 0)) return MOE_EINVAL;
    if (n_tensors == 0) return zero_sum(norm, 1, stream);
    if (!tensors || !norm || (reinterpret_cast<uintptr_t>(norm) & 3) || !given16(ws))
        return MOE_EINVAL;
    for (int64_t i = 0; i < n_tensors; ++i) {
        const moe_grad_tensor_t& t = tensors[i];
        const uintptr_t both = reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out);
        if (t.numel < 0 || (t.is_bf16 & ~1) || t.reserved || (both & (t.is_bf16 ? 1 : 3)))
            return MOE_EINVAL;
        if (t.numel && (!t.in || !t.out)) return MOE_EINVAL;
    }
    if (ws_bytes < moe::grad_clip_ws(n_tensors)) return MOE_ENOSPC;
    if (const int rc = device_ok()) return rc;
    return moe::launch_grad_clip(tensors, n_tensors, max_norm, norm, ws,
                                 static_cast<cudaStream_t>(stream));
}

}  // extern "C"
