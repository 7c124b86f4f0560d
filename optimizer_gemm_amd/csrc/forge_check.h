// Internal: argument checks shared by the C entry points (host code only): shapes, types,
// alignment, extents, overlaps, hyper-parameters and moment slots. Every error is found
// here, before anything is enqueued.
#pragma once

#include <math.h>
#include <stdint.h>

#include "forge_internal.h"

namespace forge {
namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;

int elem_size(int dt) { return dt == FORGE_F32 ? 4 : dt == FORGE_BF16 ? 2 : 1; }

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Byte range a row-major tensor may touch.
struct Range {
  uintptr_t lo, hi;
};
Range range_of(const forge_tensor* t) {
  const uintptr_t lo = (uintptr_t)t->data;
  const int64_t n = t->rows == 0 ? 0 : ((t->rows - 1) * t->ld + t->cols) * elem_size(t->dtype);
  return Range{lo, lo + (uintptr_t)n};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

int check_shape(const forge_tensor* t) {
  if (t->rows < 0 || t->cols < 0 || t->rows >= kMaxDim || t->cols >= kMaxDim) return FORGE_ERR_SHAPE;
  if (t->ld < t->cols) return FORGE_ERR_SHAPE;
  return FORGE_OK;
}

// Dense io tensor (X, dY, W, dX): fp32 or bf16, 16-byte vectors along rows.
int check_io(const forge_tensor* t, int dtype) {
  if (!t) return FORGE_ERR_NULL;
  if (!t->data && t->rows != 0 && t->cols != 0) return FORGE_ERR_NULL;  // empty tensors may be NULL
  if (t->dtype != dtype) return FORGE_ERR_DTYPE;
  int r = check_shape(t);
  if (r) return r;
  const int ve = dtype == FORGE_BF16 ? 8 : 4;
  if (!aligned16(t->data) || t->cols % ve || t->ld % ve) return FORGE_ERR_ALIGN;
  return FORGE_OK;
}

bool is_fp8(int dt) { return dt == FORGE_E4M3 || dt == FORGE_E5M2; }

// FP8 input tensor (X, dY): one byte per element, 16-byte chunks along rows, and a
// device pointer to its float32 dequantisation scale.
int check_fp8(const forge_tensor* t, bool allow_e5m2) {
  if (!t) return FORGE_ERR_NULL;
  if (!t->data && t->rows != 0 && t->cols != 0) return FORGE_ERR_NULL;
  if (!(t->dtype == FORGE_E4M3 || (allow_e5m2 && t->dtype == FORGE_E5M2))) return FORGE_ERR_DTYPE;
  if (!t->scale) return FORGE_ERR_NULL;
  int r = check_shape(t);
  if (r) return r;
  if (!aligned16(t->data) || ((uintptr_t)t->scale & 3u) || t->cols % 16 || t->ld % 16) return FORGE_ERR_ALIGN;
  return FORGE_OK;
}

bool finite(double x) { return isfinite(x) != 0; }

// The kernels address each tensor through 32-bit byte offsets below 2^31.
bool fits_31(const forge_tensor* t) {
  return !t || !t->data || t->rows * t->ld * (int64_t)elem_size(t->dtype) < ((int64_t)1 << 31);
}

int check_hyper(int opt, const forge_hyper* h, int64_t step) {
  if (!h) return FORGE_ERR_NULL;
  if (opt < FORGE_ADAMW || opt > FORGE_RADAM) return FORGE_ERR_HYPER;
  if (step < 1 || step >= ((int64_t)1 << 31)) return FORGE_ERR_HYPER;
  const double f[] = {h->lr, h->beta1, h->beta2, h->eps, h->weight_decay, h->momentum, h->dampening, h->alpha,
                      h->lr_decay, h->momentum_decay};
  for (double x : f)
    if (!finite(x)) return FORGE_ERR_HYPER;
  if (h->lr < 0.0 || h->eps < 0.0 || h->lr_decay < 0.0) return FORGE_ERR_HYPER;
  switch (opt) {
    case FORGE_ADAMW:
    case FORGE_NADAM:
    case FORGE_RADAM:
    case FORGE_LION:
      if (h->beta1 < 0.0 || h->beta1 >= 1.0 || h->beta2 < 0.0 || h->beta2 >= 1.0) return FORGE_ERR_HYPER;
      if (opt == FORGE_NADAM && h->momentum_decay < 0.0) return FORGE_ERR_HYPER;
      break;
    case FORGE_SGD_MOMENTUM:
      if (h->momentum < 0.0 || h->momentum >= 1.0 || h->dampening < 0.0 || h->dampening > 1.0) return FORGE_ERR_HYPER;
      break;
    case FORGE_RMSPROP:
      if (h->alpha < 0.0 || h->alpha >= 1.0) return FORGE_ERR_HYPER;
      break;
    default:
      break;
  }
  if (opt == FORGE_RADAM && h->beta2 <= 0.0) return FORGE_ERR_HYPER;
  return FORGE_OK;
}

// Moment slots: returns the state format (ST_F32 / ST_Q8 / ST_Q8D / ST_BF16) or a negative status.
int check_states(int opt, int io_dtype, const forge_tensor* W, const forge_tensor* m, const forge_tensor* v) {
  const int sl = opt_slots(opt);
  const forge_tensor* slot[2] = {m, v};
  int fmt = -1;
  for (int k = 0; k < 2; ++k) {
    if (!(sl & (1 << k))) continue;
    const forge_tensor* t = slot[k];
    if (!t || (!t->data && t->rows != 0 && t->cols != 0)) return FORGE_ERR_NULL;  // empty states may be NULL
    int r = check_shape(t);
    if (r) return r;
    if (t->rows != W->rows || t->cols != W->cols) return FORGE_ERR_SHAPE;
    int f;
    if (t->dtype == FORGE_F32) {
      f = ST_F32;
      if (!aligned16(t->data) || t->ld % 4) return FORGE_ERR_ALIGN;
    } else if (t->dtype == FORGE_BF16) {
      f = ST_BF16;
      if (io_dtype != FORGE_BF16) return FORGE_ERR_DTYPE;
      if (!aligned16(t->data) || t->ld % 8) return FORGE_ERR_ALIGN;
    } else if ((k == 0 && (t->dtype == FORGE_I8 || t->dtype == FORGE_I8_DYN)) ||
               (k == 1 && (t->dtype == FORGE_U8 || t->dtype == FORGE_U8_DYN))) {
      f = (t->dtype == FORGE_I8 || t->dtype == FORGE_U8) ? ST_Q8 : ST_Q8D;
      if (io_dtype != FORGE_BF16) return FORGE_ERR_DTYPE;
      if (!t->scale) return FORGE_ERR_NULL;
      if (!aligned16(t->data) || t->ld % 16 || ((uintptr_t)t->scale & 3u)) return FORGE_ERR_ALIGN;
      if (t->cols % 64) return FORGE_ERR_UNSUPPORTED;
    } else {
      return FORGE_ERR_DTYPE;
    }
    if (fmt >= 0 && f != fmt) return FORGE_ERR_DTYPE;
    fmt = f;
  }
  return fmt < 0 ? ST_F32 : fmt;
}

// Byte range of a tensor's scale: the [rows, cols / 64] float32 block scales of an INT8
// state, the one float32 dequantisation scale of an FP8 input; empty otherwise.
Range scale_range_of(const forge_tensor* t) {
  const uintptr_t lo = (uintptr_t)t->scale;
  if (!t->scale) return Range{0, 0};
  if (is_fp8(t->dtype)) return Range{lo, lo + 4};
  if (t->dtype == FORGE_I8 || t->dtype == FORGE_U8 || t->dtype == FORGE_I8_DYN || t->dtype == FORGE_U8_DYN)
    return Range{lo, lo + (uintptr_t)(t->rows * (t->cols / 64) * 4)};
  return Range{0, 0};
}

// Everything an output writes (its data and block scales) must overlap nothing else the
// call reads or writes: other outputs' data and scales, inputs' data and scales.
int check_alias(const forge_tensor* const* outs, int n_out, const forge_tensor* const* ins, int n_in) {
  for (int a = 0; a < n_out; ++a) {
    if (!outs[a]) continue;
    const Range wa[2] = {range_of(outs[a]), scale_range_of(outs[a])};
    for (const Range& ra : wa) {
      for (int b = 0; b < n_out; ++b) {
        if (!outs[b]) continue;
        if (b != a && overlap(ra, range_of(outs[b]))) return FORGE_ERR_ALIAS;
        if (overlap(ra, scale_range_of(outs[b])) && !(b == a && &ra == &wa[1])) return FORGE_ERR_ALIAS;
      }
      for (int b = 0; b < n_in; ++b)
        if (ins[b] && (overlap(ra, range_of(ins[b])) || overlap(ra, scale_range_of(ins[b])))) return FORGE_ERR_ALIAS;
    }
  }
  return FORGE_OK;
}

OptArgs make_args(forge_tensor* W, forge_tensor* m, forge_tensor* v, int opt, const forge_scalars& s,
                  uint64_t seed, int64_t step) {
  const int sl = opt_slots(opt);
  OptArgs a{};
  a.W = W->data;
  a.ldw = W->ld;
  if (sl & 1) {
    a.m = m->data;
    a.ldm = m->ld;
    a.m_scale = m->scale;
  }
  if (sl & 2) {
    a.v = v->data;
    a.ldv = v->ld;
    a.v_scale = v->scale;
  }
  a.out = (int32_t)W->rows;
  a.in = (int32_t)W->cols;
  a.rng_base = rng_base(seed, (uint64_t)step);
  a.s = s;
  return a;
}

}  // namespace
}  // namespace forge
