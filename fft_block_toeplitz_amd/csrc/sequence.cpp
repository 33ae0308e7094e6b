// C entry points of the sequence operators: argument checks, then the
// kernels' launches. Nothing here reads device memory or throws.
#include "sequence.hpp"

#include "checks.hpp"
#include "group_norm.hpp"
#include "internal.hpp"
#include "recurrence.hpp"

using namespace fftmv;

namespace {

bool types_ok(int dtype, int decay, int drive, int reserved) {
  return dtype >= FFTMV_F32 && dtype <= FFTMV_F16 && decay >= FFTMV_DECAY_SIGMOID && decay <= FFTMV_DECAY_VALUE &&
         (drive == FFTMV_DRIVE_COMPLEMENT || drive == FFTMV_DRIVE_PLAIN) && reserved == 0;
}

int check_recurrence(const fftmv_recurrence_t *r, bool backward) {
  if (!r || r->batch < 1 || r->steps < 0 || r->channels < 1) return FFTMV_ERR_INVALID_ARG;
  if (!types_ok(r->dtype, r->decay, r->drive, 0)) return FFTMV_ERR_INVALID_ARG;
  if (r->lengths && r->offsets) return FFTMV_ERR_INVALID_ARG;
  if (!aligned(r->lengths, 4) || !aligned(r->offsets, 4)) return FFTMV_ERR_INVALID_ARG;
  if (!sizes_fit(r->batch, r->steps, r->channels)) return FFTMV_ERR_UNSUPPORTED_SIZE;
  const size_t es = elem_bytes(r->dtype);
  const int64_t B = r->offsets ? 1 : r->batch, T = r->steps, C = r->channels;
  if (r->steps > 0) {
    if (!field(r->x, es) || !field(r->gate, es)) return FFTMV_ERR_INVALID_ARG;
    if (!strides_ok(B, r->x_batch, T, r->x_step, C) || !strides_ok(B, r->gate_batch, T, r->gate_step, C))
      return FFTMV_ERR_INVALID_ARG;
    if (!backward) {
      if (!field(r->h, es) || !strides_ok(B, r->h_batch, T, r->h_step, C)) return FFTMV_ERR_INVALID_ARG;
    } else {
      if (!field(r->dh, es) || !field(r->dx, es) || !field(r->dgate, es)) return FFTMV_ERR_INVALID_ARG;
      if (!strides_ok(B, r->dh_batch, T, r->dh_step, C) || !strides_ok(B, r->dx_batch, T, r->dx_step, C) ||
          !strides_ok(B, r->dgate_batch, T, r->dgate_step, C))
        return FFTMV_ERR_INVALID_ARG;
    }
  }
  if (!floats(r->h0) || !floats(r->h_last) || !floats(r->carries) || !floats(r->dh_last) || !floats(r->dh0))
    return FFTMV_ERR_INVALID_ARG;
  int64_t carries = 0;
  size_t counters = 0, words = 0;
  const int st = fftmv_recurrence_sizes(r->batch, T, C, r->offsets != nullptr, &carries, &counters, &words);
  if (st != FFTMV_SUCCESS) return st;
  if (backward && carries && !r->carries) return FFTMV_ERR_INVALID_ARG;
  if (words && (!r->workspace || !r->counters || !aligned(r->workspace, 8) || !aligned(r->counters, 8) ||
                r->workspace_bytes < words || r->counter_bytes < counters || r->call == 0))
    return FFTMV_ERR_INVALID_ARG;
  return FFTMV_SUCCESS;
}

int check_group_norm(const fftmv_group_norm_t *g, bool backward) {
  if (!g || g->samples < 1 || g->rows < 0 || g->channels < 1 || g->groups < 1 || g->channels % g->groups)
    return FFTMV_ERR_INVALID_ARG;
  if (g->dtype < FFTMV_F32 || g->dtype > FFTMV_F16 || g->activation < FFTMV_ACT_NONE ||
      g->activation > FFTMV_ACT_GELU || g->reserved != 0 || !(g->eps >= 0.0f))
    return FFTMV_ERR_INVALID_ARG;
  if (!sizes_fit(g->samples, g->rows, g->channels)) return FFTMV_ERR_UNSUPPORTED_SIZE;
  const size_t es = elem_bytes(g->dtype);
  const int64_t N = g->samples, S = g->rows, C = g->channels;
  if (S > 0) {
    if (!field(g->x, es) || !strides_ok(N, g->x_sample, S, g->x_row, C)) return FFTMV_ERR_INVALID_ARG;
    if (!backward) {
      if (!field(g->y, es) || !strides_ok(N, g->y_sample, S, g->y_row, C)) return FFTMV_ERR_INVALID_ARG;
    } else {
      if (!field(g->dy, es) || !field(g->dx, es) || !g->stats) return FFTMV_ERR_INVALID_ARG;
      if (!strides_ok(N, g->dy_sample, S, g->dy_row, C) || !strides_ok(N, g->dx_sample, S, g->dx_row, C))
        return FFTMV_ERR_INVALID_ARG;
    }
  }
  if (!aligned(g->lengths, 4) || !floats(g->weight) || !floats(g->bias) || !floats(g->stats) ||
      !floats(g->dweight) || !floats(g->dbias))
    return FFTMV_ERR_INVALID_ARG;
  size_t need = 0;
  const int st = fftmv_group_norm_workspace(N, S, C, g->groups, g->dtype, backward, &need);
  if (st != FFTMV_SUCCESS) return st;
  if (need && (!g->workspace || !aligned(g->workspace, 16) || g->workspace_bytes < need)) return FFTMV_ERR_INVALID_ARG;
  return FFTMV_SUCCESS;
}

}  // namespace

extern "C" {

int fftmv_recurrence_sizes(int64_t batch, int64_t steps, int64_t channels, int packed, int64_t *carries,
                           size_t *counter_bytes, size_t *workspace_bytes) {
  if (batch < 1 || steps < 0 || channels < 1) return FFTMV_ERR_INVALID_ARG;
  if (!sizes_fit(batch, steps, channels)) return FFTMV_ERR_UNSUPPORTED_SIZE;
  const ScanWorkspace w = scan_workspace_bytes(batch, steps, packed != 0, channels);
  if (carries) *carries = scan_carries(batch, steps, packed != 0);
  if (counter_bytes) *counter_bytes = w.counters;
  if (workspace_bytes) *workspace_bytes = w.words;
  return FFTMV_SUCCESS;
}

int fftmv_recurrence_forward(const fftmv_recurrence_t *r, hipStream_t stream) {
  const int st = check_recurrence(r, false);
  if (st != FFTMV_SUCCESS) return st;
  return status_of(r->dtype == FFTMV_F32    ? launch_recurrence_forward_f32(*r, stream)
                   : r->dtype == FFTMV_BF16 ? launch_recurrence_forward_bf16(*r, stream)
                                            : launch_recurrence_forward_f16(*r, stream));
}

int fftmv_recurrence_backward(const fftmv_recurrence_t *r, hipStream_t stream) {
  const int st = check_recurrence(r, true);
  if (st != FFTMV_SUCCESS) return st;
  return status_of(r->dtype == FFTMV_F32    ? launch_recurrence_backward_f32(*r, stream)
                   : r->dtype == FFTMV_BF16 ? launch_recurrence_backward_bf16(*r, stream)
                                            : launch_recurrence_backward_f16(*r, stream));
}

int fftmv_recurrence_step(const fftmv_recurrence_step_t *r, hipStream_t stream) {
  if (!r || r->batch < 1 || r->channels < 1 || r->places < 1 || (!r->slots && r->batch > r->places))
    return FFTMV_ERR_INVALID_ARG;
  if (!types_ok(r->dtype, r->decay, r->drive, r->reserved)) return FFTMV_ERR_INVALID_ARG;
  if (!sizes_fit(r->batch, r->places, r->channels)) return FFTMV_ERR_UNSUPPORTED_SIZE;
  const size_t es = elem_bytes(r->dtype);
  if (!field(r->x, es) || !field(r->gate, es) || !field(r->h, es) || !r->state || !floats(r->state) ||
      !aligned(r->slots, 4))
    return FFTMV_ERR_INVALID_ARG;
  if (!strides_ok(0, 0, r->batch, r->x_step, r->channels) || !strides_ok(0, 0, r->batch, r->gate_step, r->channels) ||
      !strides_ok(0, 0, r->batch, r->h_step, r->channels) ||
      !strides_ok(0, 0, r->places, r->state_step, r->channels) || r->state_step < r->channels)
    return FFTMV_ERR_INVALID_ARG;
  return status_of(launch_recurrence_step(*r, stream));
}

int fftmv_group_norm_workspace(int64_t samples, int64_t rows, int64_t channels, int64_t groups, int dtype,
                               int backward, size_t *bytes) {
  if (!bytes || samples < 1 || rows < 0 || channels < 1 || groups < 1 || channels % groups || dtype < FFTMV_F32 ||
      dtype > FFTMV_F16)
    return FFTMV_ERR_INVALID_ARG;
  if (!sizes_fit(samples, rows, channels)) return FFTMV_ERR_UNSUPPORTED_SIZE;
  *bytes = norm_plan(samples, rows, channels, groups, dtype, backward != 0).workspace;
  return FFTMV_SUCCESS;
}

int fftmv_group_norm_forward(const fftmv_group_norm_t *g, hipStream_t stream) {
  const int st = check_group_norm(g, false);
  if (st != FFTMV_SUCCESS) return st;
  return status_of(g->dtype == FFTMV_F32    ? launch_group_norm_forward_f32(*g, stream)
                   : g->dtype == FFTMV_BF16 ? launch_group_norm_forward_bf16(*g, stream)
                                            : launch_group_norm_forward_f16(*g, stream));
}

int fftmv_group_norm_backward(const fftmv_group_norm_t *g, hipStream_t stream) {
  const int st = check_group_norm(g, true);
  if (st != FFTMV_SUCCESS) return st;
  return status_of(g->dtype == FFTMV_F32    ? launch_group_norm_backward_f32(*g, stream)
                   : g->dtype == FFTMV_BF16 ? launch_group_norm_backward_bf16(*g, stream)
                                            : launch_group_norm_backward_f16(*g, stream));
}

}  // extern "C"
