// abi_block.cu -- C entry points of the training block's operators (norm with
// residual and gate, rotary positions, with and without head norms, packed causal
// attention, gradient clipping) and of what stands before and behind the blocks (choice
// of experts, embedding, distillation loss): argument checks, then the launches.
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

// In place means the same strides (an extent of one has none).
bool in_place_ok(const void* in, const void* out, int64_t T, int64_t heads, int64_t in_t,
                 int64_t out_t, int64_t in_h, int64_t out_h) {
    return in != out || ((T <= 1 || in_t == out_t) && (heads <= 1 || in_h == out_h));
}

int head_norm_ok(const moe_head_norm_t* c) {
    if (!c || c->T < 0 || c->hq <= 0 || c->hk < 0 || c->hq > 65536 || c->hk > 65536 ||
        c->D < 16 || c->D > 512 || c->D % 8 || c->rot_dim < 0 || c->rot_dim % 16 ||
        c->rot_dim > c->D || (c->interleaved & ~1) || !(c->eps >= 0) || !std::isfinite(c->eps) ||
        (c->rot_dim > 0 && c->table_rows <= 0))
        return MOE_EINVAL;
    if (!strides_ok(c->T, c->hq, c->D, c->q_t, c->q_h) ||
        !strides_ok(c->T, c->hq, c->D, c->qo_t, c->qo_h) ||
        (c->hk && (!strides_ok(c->T, c->hk, c->D, c->k_t, c->k_h) ||
                   !strides_ok(c->T, c->hk, c->D, c->ko_t, c->ko_h))))
        return MOE_EINVAL;
    return MOE_OK;
}

int routing_ok(const moe_routing_t* c) {
    if (!c || c->T < 0 || c->n_experts <= 0 || c->n_experts > 1024 || c->top_k <= 0 ||
        c->top_k > 32 || (c->score & ~1) || c->n_groups <= 0 || c->n_groups > 32 ||
        c->n_experts % c->n_groups || c->groups_kept <= 0 || c->groups_kept > c->n_groups ||
        c->group_top < 1 || c->group_top > 2 || (c->renorm & ~1) || !std::isfinite(c->scale) ||
        (c->grad_f32 & ~1) || c->reserved)
        return MOE_EINVAL;
    const int per = c->n_experts / c->n_groups;
    if (c->group_top > per || c->top_k > per * c->groups_kept ||
        (c->groups_kept < c->n_groups && per > 32 * moe::router_select_lanes(c->n_groups)))
        return MOE_EINVAL;
    return MOE_OK;
}

bool embedding_sizes_ok(int64_t T, int64_t V, int32_t d) {
    return T >= 0 && T < (1ll << 31) - 256 && V > 0 && V < (1ll << 31) - 256 && d >= 8 &&
           d <= 65536 && d % 8 == 0;
}

int embedding_ok(const moe_embedding_t* c) {
    if (!c || !embedding_sizes_ok(c->T, c->V, c->d) || (c->table_f32 & ~1) || (c->out_f32 & ~1) ||
        (c->accumulate & ~1) || !std::isfinite(c->scale) || c->reserved)
        return MOE_EINVAL;
    return MOE_OK;
}

int distill_ok(const moe_distill_t* c) {
    if (!c || c->T < 0 || c->V <= 0 || c->V >= (1ll << 31) || c->K <= 0 ||
        c->K > MOE_DISTILL_MAX_ENTRIES || (c->z_f32 & ~1) || (c->teacher_f32 & ~1) ||
        !(c->temperature > 0) || !std::isfinite(c->temperature) || !std::isfinite(c->scale) ||
        c->reserved)
        return MOE_EINVAL;
    if (c->T > 1 && (c->z_ld < c->V || c->z_ld >= (1ll << 38))) return MOE_EINVAL;
    return MOE_OK;
}

bool distill_grad_ok(const moe_distill_t* c, const void* z, const void* dz) {
    if (c->T > 1 && (c->dz_ld < c->V || c->dz_ld >= (1ll << 38))) return false;
    return reinterpret_cast<uintptr_t>(dz) % (c->z_f32 ? 4 : 2) == 0 &&
           (z != dz || c->T <= 1 || c->z_ld == c->dz_ld);
}

bool qkvo_strides_ok(const moe_attention_t* c) {
    return strides_ok(c->T, c->n_heads, c->head_dim, c->q_t, c->q_h) &&
           strides_ok(c->T, c->n_kv_heads, c->head_dim, c->k_t, c->k_h) &&
           strides_ok(c->T, c->n_kv_heads, c->head_dim, c->v_t, c->v_h) &&
           strides_ok(c->T, c->n_heads, c->head_dim, c->o_t, c->o_h);
}

}  // namespace

int moe::routing_check(const moe_routing_t* c) { return routing_ok(c); }

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

int moe_head_norm_rotary(const moe_head_norm_t* cfg, const uint16_t* q, const uint16_t* k,
                         const uint16_t* w_q, const uint16_t* w_k, const float* table,
                         const int32_t* pos, uint16_t* q_out, uint16_t* k_out, int32_t* status,
                         void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = head_norm_ok(cfg)) return rc;
    if (cfg->T == 0) return MOE_OK;
    const bool has_k = cfg->hk > 0;
    if (!given16(q) || !given16(w_q) || !given16(q_out) || !status || !aligned16(table) ||
        (cfg->rot_dim > 0) != (table != nullptr) || has_k != (k != nullptr) ||
        has_k != (w_k != nullptr) || has_k != (k_out != nullptr) || !aligned16(k) ||
        !aligned16(w_k) || !aligned16(k_out) ||
        !in_place_ok(q, q_out, cfg->T, cfg->hq, cfg->q_t, cfg->qo_t, cfg->q_h, cfg->qo_h) ||
        (has_k &&
         !in_place_ok(k, k_out, cfg->T, cfg->hk, cfg->k_t, cfg->ko_t, cfg->k_h, cfg->ko_h)))
        return MOE_EINVAL;
    if (const int rc = device_ok()) return rc;
    return moe::launch_head_norm(*cfg, q, k, w_q, w_k, table, pos, q_out, k_out, status,
                                 static_cast<cudaStream_t>(stream));
}

int moe_head_norm_rotary_workspace(int64_t T, int32_t hq, int32_t hk, int32_t D, int64_t* bytes) {
    if (!bytes || T < 0 || hq <= 0 || hk < 0 || D < 16 || D > 512 || D % 8) return MOE_EINVAL;
    *bytes = moe::head_norm_backward_ws(D);
    return MOE_OK;
}

int moe_head_norm_rotary_backward(const moe_head_norm_t* cfg, const uint16_t* dq,
                                  const uint16_t* dk, const uint16_t* q, const uint16_t* k,
                                  const uint16_t* w_q, const uint16_t* w_k, const float* table,
                                  const int32_t* pos, uint16_t* dq_out, uint16_t* dk_out,
                                  float* dw_q, float* dw_k, void* ws, int64_t ws_bytes,
                                  int32_t* status, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = head_norm_ok(cfg)) return rc;
    if (!strides_ok(cfg->T, cfg->hq, cfg->D, cfg->dq_t, cfg->dq_h) ||
        (cfg->hk && !strides_ok(cfg->T, cfg->hk, cfg->D, cfg->dk_t, cfg->dk_h)))
        return MOE_EINVAL;
    if (cfg->T == 0) {
        if (const int rc = zero_sum(dw_q, cfg->D, stream)) return rc;
        return zero_sum(dw_k, cfg->D, stream);
    }
    const bool has_k = cfg->hk > 0;
    if (!given16(dq) || !given16(q) || !given16(w_q) || !given16(dq_out) || !dw_q ||
        !given16(ws) || !status || !aligned16(table) ||
        (cfg->rot_dim > 0) != (table != nullptr) || has_k != (dk != nullptr) ||
        has_k != (k != nullptr) || has_k != (w_k != nullptr) || has_k != (dk_out != nullptr) ||
        has_k != (dw_k != nullptr) || !aligned16(dk) || !aligned16(k) || !aligned16(w_k) ||
        !aligned16(dk_out))
        return MOE_EINVAL;
    if (!in_place_ok(q, dq_out, cfg->T, cfg->hq, cfg->q_t, cfg->qo_t, cfg->q_h, cfg->qo_h) ||
        !in_place_ok(dq, dq_out, cfg->T, cfg->hq, cfg->dq_t, cfg->qo_t, cfg->dq_h, cfg->qo_h) ||
        (has_k &&
         (!in_place_ok(k, dk_out, cfg->T, cfg->hk, cfg->k_t, cfg->ko_t, cfg->k_h, cfg->ko_h) ||
          !in_place_ok(dk, dk_out, cfg->T, cfg->hk, cfg->dk_t, cfg->ko_t, cfg->dk_h, cfg->ko_h))))
        return MOE_EINVAL;
    if (ws_bytes < moe::head_norm_backward_ws(cfg->D)) return MOE_ENOSPC;
    if (const int rc = device_ok()) return rc;
    return moe::launch_head_norm_backward(*cfg, dq, dk, q, k, w_q, w_k, table, pos, dq_out, dk_out,
                                          dw_q, dw_k, ws, status,
                                          static_cast<cudaStream_t>(stream));
}

int moe_router_select(const moe_routing_t* cfg, const float* logits, const float* bias,
                      int32_t* idx, float* w, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = routing_ok(cfg)) return rc;
    if (cfg->T == 0) return MOE_OK;
    if (!given16(logits) || !given16(idx) || !given16(w) || !aligned16(bias)) return MOE_EINVAL;
    if (const int rc = device_ok()) return rc;
    return moe::launch_router_select(*cfg, logits, bias, idx, w,
                                     static_cast<cudaStream_t>(stream));
}

int moe_router_select_backward(const moe_routing_t* cfg, const float* logits, const int32_t* idx,
                               const float* dw, void* dlogits, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = routing_ok(cfg)) return rc;
    if (cfg->T == 0) return MOE_OK;
    if (!given16(logits) || !given16(idx) || !given16(dw) || !given16(dlogits)) return MOE_EINVAL;
    if (const int rc = device_ok()) return rc;
    return moe::launch_router_select_backward(*cfg, logits, idx, dw, dlogits,
                                              static_cast<cudaStream_t>(stream));
}

int moe_embedding(const moe_embedding_t* cfg, const void* table, const int32_t* ids, void* out,
                  int32_t* status, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = embedding_ok(cfg)) return rc;
    if (cfg->T == 0) return MOE_OK;
    if (!given16(table) || !ids || !given16(out) || !status) return MOE_EINVAL;
    if (const int rc = device_ok()) return rc;
    return moe::launch_embedding(*cfg, table, ids, out, status, static_cast<cudaStream_t>(stream));
}

int moe_embedding_workspace(int64_t T, int64_t V, int32_t d, int64_t* plan_bytes) {
    if (!plan_bytes || !embedding_sizes_ok(T, V, d)) return MOE_EINVAL;
    *plan_bytes = moe::embedding_plan_bytes(T, V, d);
    return MOE_OK;
}

int moe_embedding_plan(int64_t T, int64_t V, int32_t d, const int32_t* ids, void* plan,
                       int64_t plan_bytes, int32_t* status, void* stream) {
    MOE_NVTX_RANGE();
    if (!embedding_sizes_ok(T, V, d)) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!ids || !given16(plan) || !status) return MOE_EINVAL;
    if (plan_bytes < moe::embedding_plan_bytes(T, V, d)) return MOE_ENOSPC;
    if (const int rc = device_ok()) return rc;
    return moe::launch_embedding_plan(T, V, d, ids, plan, status,
                                      static_cast<cudaStream_t>(stream));
}

int moe_embedding_backward(const moe_embedding_t* cfg, const void* plan, int64_t plan_bytes,
                           const void* dout, void* dtable, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = embedding_ok(cfg)) return rc;
    if (cfg->T == 0) {
        if (cfg->accumulate) return MOE_OK;
        return zero_sum(dtable, cfg->V * cfg->d / (cfg->table_f32 ? 1 : 2), stream);
    }
    if (!given16(plan) || !given16(dout) || !given16(dtable)) return MOE_EINVAL;
    if (plan_bytes < moe::embedding_plan_bytes(cfg->T, cfg->V, cfg->d)) return MOE_ENOSPC;
    if (const int rc = device_ok()) return rc;
    return moe::launch_embedding_backward(*cfg, plan, dout, dtable,
                                          static_cast<cudaStream_t>(stream));
}

int moe_distill_loss(const moe_distill_t* cfg, const void* z, const int32_t* ids,
                     const void* teacher, const float* weight, float* loss, float* lse,
                     float* total, void* dlogits, int32_t* status, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = distill_ok(cfg)) return rc;
    if (cfg->T == 0) return zero_sum(total, 1, stream);
    if (!z || !ids || !teacher || !loss || !lse || !status ||
        reinterpret_cast<uintptr_t>(z) % (cfg->z_f32 ? 4 : 2) ||
        (dlogits && !distill_grad_ok(cfg, z, dlogits)))
        return MOE_EINVAL;
    if (const int rc = device_ok()) return rc;
    return moe::launch_distill(*cfg, z, ids, teacher, weight, loss, lse, total, dlogits, status,
                               static_cast<cudaStream_t>(stream));
}

int moe_distill_loss_backward(const moe_distill_t* cfg, const void* z, const int32_t* ids,
                              const void* teacher, const float* weight, const float* lse,
                              void* dlogits, int32_t* status, void* stream) {
    MOE_NVTX_RANGE();
    if (const int rc = distill_ok(cfg)) return rc;
    if (cfg->T == 0) return MOE_OK;
    if (!z || !ids || !teacher || !lse || !dlogits || !status ||
        reinterpret_cast<uintptr_t>(z) % (cfg->z_f32 ? 4 : 2) ||
        !distill_grad_ok(cfg, z, dlogits))
        return MOE_EINVAL;
    if (const int rc = device_ok()) return rc;
    return moe::launch_distill_backward(*cfg, z, ids, teacher, weight, lse, dlogits, status,
                                        static_cast<cudaStream_t>(stream));
}

}  // extern "C"
