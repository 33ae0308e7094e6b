// C entry points of the gated delta rule and of the queries' and keys' norms:
// argument checks, then the kernels' launches. Nothing here reads device memory
// or throws.
#include "checks.hpp"
#include "delta_rule.hpp"
#include "qk_norm.hpp"

using namespace fftmv;

namespace {

// A field of `heads` heads of n elements, that a call with rows has to have.
bool heads_ok(const fftmv_heads_t &f, size_t es, int64_t batch, int64_t steps, int64_t heads, int64_t n) {
  if (!field(f.data, es) || f.head < 0) return false;
  int64_t a = 0, b = 0;
  if (__builtin_mul_overflow(heads, f.head, &a) || __builtin_add_overflow(a, n, &b)) return false;
  return strides_ok(batch, f.batch, steps, f.step, b);
}

bool delta_types_ok(int dtype, int decay, int rate) {
  return dtype >= FFTMV_F32 && dtype <= FFTMV_F16 && (decay == FFTMV_DECAY_SIGMOID || decay == FFTMV_DECAY_EXP) &&
         (rate == FFTMV_RATE_SIGMOID || rate == FFTMV_RATE_VALUE);
}

int delta_sizes_ok(int64_t batch, int64_t steps, int64_t key_heads, int64_t heads, int64_t keys, int64_t values) {
  if (batch < 1 || steps < 0 || key_heads < 1 || heads < 1 || heads % key_heads || keys < 1 || values < 1)
    return FFTMV_ERR_INVALID_ARG;
  if (!sizes_fit(batch, steps, heads) || keys > FFTMV_DELTA_KEYS || values > FFTMV_DELTA_VALUES)
    return FFTMV_ERR_UNSUPPORTED_SIZE;
  // one workgroup for each run and head: what a grid takes, and far from where a product of sizes leaves 63 bits
  if (!grid_fits(batch, kWave) || !grid_fits(batch * heads, kWave) || !grid_fits(delta_runs(batch, steps, false), kWave) ||
      !grid_fits(delta_runs(batch, steps, false) * heads, kBlock))
    return FFTMV_ERR_UNSUPPORTED_SIZE;
  return FFTMV_SUCCESS;
}

int check_delta(const fftmv_delta_rule_t *r, bool back) {
  if (!r || !delta_types_ok(r->dtype, r->decay, r->rate) || (r->lengths && r->offsets)) return FFTMV_ERR_INVALID_ARG;
  if (!aligned(r->lengths, 4) || !aligned(r->offsets, 4)) return FFTMV_ERR_INVALID_ARG;
  int64_t runs = 0;
  size_t need = 0;
  const int st = fftmv_delta_rule_sizes(r->batch, r->steps, r->key_heads, r->heads, r->keys, r->values, r->dtype,
                                        r->offsets != nullptr, back, &runs, &need);
  if (st != FFTMV_SUCCESS) return st;
  const size_t es = elem_bytes(r->dtype);
  const int64_t B = r->offsets ? 1 : r->batch, T = r->steps;
  if (T > 0) {
    const fftmv_heads_t *keyed[] = {&r->q, &r->k, back ? &r->dq : nullptr, back ? &r->dk : nullptr};
    const fftmv_heads_t *valued[] = {&r->v, back ? &r->dy : &r->y, back ? &r->dv : nullptr};
    const fftmv_heads_t *gates[] = {&r->gate, &r->beta, back ? &r->dgate : nullptr, back ? &r->dbeta : nullptr};
    for (const auto *f : keyed)
      if (f && !heads_ok(*f, es, B, T, r->key_heads, r->keys)) return FFTMV_ERR_INVALID_ARG;
    for (const auto *f : valued)
      if (f && !heads_ok(*f, es, B, T, r->heads, r->values)) return FFTMV_ERR_INVALID_ARG;
    for (const auto *f : gates)
      if (f && !heads_ok(*f, es, B, T, r->heads, 1)) return FFTMV_ERR_INVALID_ARG;
    if (back && !r->carries) return FFTMV_ERR_INVALID_ARG;
  }
  if (!floats(r->h0) || !floats(r->carries) || !floats(r->h_last) || !floats(r->dh_last) || !floats(r->dh0))
    return FFTMV_ERR_INVALID_ARG;
  if (need && (!r->workspace || !aligned(r->workspace, 16) || r->workspace_bytes < need)) return FFTMV_ERR_INVALID_ARG;
  return FFTMV_SUCCESS;
}

int check_norm(const fftmv_qk_norm_t *n, bool back) {
  if (!n || n->batch < 1 || n->steps < 0 || n->query_heads < 1 || n->key_heads < 0 || n->dim < 1 ||
      n->frequencies < 0 || n->frequencies > n->dim / 2)
    return FFTMV_ERR_INVALID_ARG;
  if (n->dtype < FFTMV_F32 || n->dtype > FFTMV_F16 || (n->norm != FFTMV_NORM_RMS && n->norm != FFTMV_NORM_L2) ||
      (n->pairs != FFTMV_PAIRS_HALVES && n->pairs != FFTMV_PAIRS_NEIGHBOURS) || !(n->eps >= 0.0f))
    return FFTMV_ERR_INVALID_ARG;
  size_t need = 0;
  const int st = fftmv_qk_norm_workspace(n->batch, n->steps, n->query_heads, n->key_heads, n->dim, &need);
  if (st != FFTMV_SUCCESS) return st;
  const size_t es = elem_bytes(n->dtype);
  const int64_t B = n->batch, T = n->steps, H = n->query_heads, K = n->key_heads;
  if (T > 0) {
    if (!heads_ok(n->q, es, B, T, H, n->dim) || !heads_ok(back ? n->dq : n->qy, es, B, T, H, n->dim))
      return FFTMV_ERR_INVALID_ARG;
    if (back && !heads_ok(n->dqy, es, B, T, H, n->dim)) return FFTMV_ERR_INVALID_ARG;
    if (K > 0) {
      if (!heads_ok(n->k, es, B, T, K, n->dim) || !heads_ok(back ? n->dk : n->ky, es, B, T, K, n->dim))
        return FFTMV_ERR_INVALID_ARG;
      if (back && !heads_ok(n->dky, es, B, T, K, n->dim)) return FFTMV_ERR_INVALID_ARG;
    }
    if (n->frequencies && (!n->frequency || !aligned(n->frequency, 8))) return FFTMV_ERR_INVALID_ARG;
    if (n->positions && (!aligned(n->positions, 4) || !strides_ok(B, n->position_batch, T, 1, 1)))
      return FFTMV_ERR_INVALID_ARG;
    if (back && (n->dq_weight || n->dk_weight) &&
        (!n->workspace || !aligned(n->workspace, 16) || n->workspace_bytes < need))
      return FFTMV_ERR_INVALID_ARG;
  }
  if (!aligned(n->lengths, 4) || !floats(n->q_weight) || !floats(n->k_weight) || !floats(n->dq_weight) ||
      !floats(n->dk_weight))
    return FFTMV_ERR_INVALID_ARG;
  return FFTMV_SUCCESS;
}

}  // namespace

extern "C" {

int fftmv_delta_rule_sizes(int64_t batch, int64_t steps, int64_t key_heads, int64_t heads, int64_t keys,
                           int64_t values, int dtype, int packed, int backward, int64_t *runs,
                           size_t *workspace_bytes) {
  if (dtype < FFTMV_F32 || dtype > FFTMV_F16) return FFTMV_ERR_INVALID_ARG;
  const int st = packed ? delta_sizes_ok(batch, 0, key_heads, heads, keys, values)
                        : delta_sizes_ok(batch, steps, key_heads, heads, keys, values);
  if (st != FFTMV_SUCCESS) return st;
  if (packed) {
    if (steps < 0) return FFTMV_ERR_INVALID_ARG;
    if (!sizes_fit(1, steps, 1) || !grid_fits(delta_runs(batch, steps, true) * heads, kBlock))
      return FFTMV_ERR_UNSUPPORTED_SIZE;
  }
  const int64_t n = delta_runs(batch, steps, packed != 0);
  if (runs) *runs = n;
  if (workspace_bytes) *workspace_bytes = delta_workspace(batch, steps, heads, keys, values, packed != 0, backward != 0);
  return FFTMV_SUCCESS;
}

int fftmv_delta_rule_forward(const fftmv_delta_rule_t *r, hipStream_t stream) {
  const int st = check_delta(r, false);
  if (st != FFTMV_SUCCESS) return st;
  return status_of(r->dtype == FFTMV_F32    ? launch_delta_forward_f32(*r, stream)
                   : r->dtype == FFTMV_BF16 ? launch_delta_forward_bf16(*r, stream)
                                            : launch_delta_forward_f16(*r, stream));
}

int fftmv_delta_rule_backward(const fftmv_delta_rule_t *r, hipStream_t stream) {
  const int st = check_delta(r, true);
  if (st != FFTMV_SUCCESS) return st;
  return status_of(r->dtype == FFTMV_F32    ? launch_delta_backward_f32(*r, stream)
                   : r->dtype == FFTMV_BF16 ? launch_delta_backward_bf16(*r, stream)
                                            : launch_delta_backward_f16(*r, stream));
}

int fftmv_delta_rule_step(const fftmv_delta_rule_step_t *r, hipStream_t stream) {
  if (!r || r->places < 1 || (!r->slots && r->batch > r->places) || !delta_types_ok(r->dtype, r->decay, r->rate))
    return FFTMV_ERR_INVALID_ARG;
  const int st = delta_sizes_ok(r->batch, 1, r->key_heads, r->heads, r->keys, r->values);
  if (st != FFTMV_SUCCESS) return st;
  if (!sizes_fit(r->places, 1, 1)) return FFTMV_ERR_UNSUPPORTED_SIZE;
  const size_t es = elem_bytes(r->dtype);
  const int64_t B = r->batch;
  if (!heads_ok(r->q, es, 0, B, r->key_heads, r->keys) || !heads_ok(r->k, es, 0, B, r->key_heads, r->keys) ||
      !heads_ok(r->v, es, 0, B, r->heads, r->values) || !heads_ok(r->y, es, 0, B, r->heads, r->values) ||
      !heads_ok(r->gate, es, 0, B, r->heads, 1) || !heads_ok(r->beta, es, 0, B, r->heads, 1))
    return FFTMV_ERR_INVALID_ARG;
  const int64_t place = r->heads * r->keys * r->values;  // heads is bounded by the grid: this stays inside 63 bits
  if (!r->state || !floats(r->state) || r->state_place < place || !aligned(r->slots, 4) ||
      !strides_ok(r->places, r->state_place, 0, 0, 0))
    return FFTMV_ERR_INVALID_ARG;
  return status_of(launch_delta_step(*r, stream));
}

int fftmv_qk_norm_workspace(int64_t batch, int64_t steps, int64_t query_heads, int64_t key_heads, int64_t dim,
                            size_t *bytes) {
  if (!bytes || batch < 1 || steps < 0 || query_heads < 1 || key_heads < 0 || dim < 1) return FFTMV_ERR_INVALID_ARG;
  // rows and a row's heads are counted in 32 bits
  if (dim > FFTMV_QK_NORM_DIM || !sizes_fit(batch, steps, query_heads) || !sizes_fit(key_heads, 1, 1) ||
      !sizes_fit(batch * steps, 1, kNormRows * (query_heads + key_heads)))
    return FFTMV_ERR_UNSUPPORTED_SIZE;
  *bytes = qk_norm_workspace(batch * steps, query_heads, key_heads, dim);
  return FFTMV_SUCCESS;
}

int fftmv_qk_norm_forward(const fftmv_qk_norm_t *n, hipStream_t stream) {
  const int st = check_norm(n, false);
  return st != FFTMV_SUCCESS ? st : status_of(launch_qk_norm_forward(*n, stream));
}

int fftmv_qk_norm_backward(const fftmv_qk_norm_t *n, hipStream_t stream) {
  const int st = check_norm(n, true);
  return st != FFTMV_SUCCESS ? st : status_of(launch_qk_norm_backward(*n, stream));
}

}  // extern "C"
