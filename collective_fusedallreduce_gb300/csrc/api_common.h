// Argument checks shared by the entry points (api.cu, api_llm.cu): everything is
// validated on the host before an entry's first CUDA call.
#pragma once

#include <vector>

#include "coco.h"
#include "internal.h"

#define COCO_EXPORT extern "C" __attribute__((visibility("default")))

namespace coco {

// COCO_OK, or COCO_ERR_CUDA with the error kept for coco_last_cuda_error().
coco_status cuda_status(cudaError_t e);

// ------------------------------------------------------------ validation

struct TInfo {
  int dtype = 0, layout = 0, ndim = 0, slice_dim = -1, nranks = 0, ngroups = 0;
  int64_t shape[COCO_MAX_DIMS] = {0, 0, 0};  // as given
  int64_t local[COCO_MAX_DIMS] = {0, 0, 0};  // per-rank
  int64_t numel = 0;                         // per rank
  int64_t bytes = 0;                         // per rank
  const coco_tensor* t = nullptr;
  void* ptr(int g, int r) const { return t->ptr[g * nranks + r]; }
};

// `fp8`: whether the operand may hold e4m3 values (the entry points that take 8-bit operands say so).
inline coco_status check_tensor(const coco_tensor* t, TInfo* o, bool fp8 = false) {
  if (!t) return COCO_ERR_NULL;
  if (t->dtype < COCO_F32 || t->dtype > (fp8 ? COCO_F8E4M3 : COCO_BF16)) return COCO_ERR_DTYPE;
  if (t->layout < COCO_LOCAL || t->layout > COCO_REPLICATED) return COCO_ERR_LAYOUT;
  if (t->ndim < 1 || t->ndim > COCO_MAX_DIMS) return COCO_ERR_SHAPE;
  if (t->nranks < 1 || t->ngroups < 1 || static_cast<int64_t>(t->nranks) * t->ngroups > COCO_MAX_PTRS)
    return COCO_ERR_SHAPE;
  o->t = t;
  o->dtype = t->dtype;
  o->layout = t->layout;
  o->ndim = t->ndim;
  o->nranks = t->nranks;
  o->ngroups = t->ngroups;
  o->numel = 1;
  for (int d = 0; d < t->ndim; ++d) {
    if (t->shape[d] < 0 || t->shape[d] > (int64_t(1) << 40)) return COCO_ERR_SHAPE;
    o->shape[d] = o->local[d] = t->shape[d];
  }
  if (t->layout == COCO_SLICED) {
    if (t->slice_dim < 0 || t->slice_dim >= t->ndim) return COCO_ERR_SHAPE;
    if (t->shape[t->slice_dim] % t->nranks) return COCO_ERR_SHAPE;  // "equally distributed"
    o->slice_dim = t->slice_dim;
    o->local[t->slice_dim] /= t->nranks;
  }
  // at most 2^40 elements per rank (far beyond any device's memory), so no size below overflows
  for (int d = 0; d < t->ndim; ++d) {
    if (o->local[d] != 0 && o->numel > (int64_t(1) << 40) / o->local[d]) return COCO_ERR_SHAPE;
    o->numel *= o->local[d];
  }
  o->bytes = o->numel * dtype_size(t->dtype);
  if (o->numel == 0) return COCO_OK;
  for (int i = 0; i < t->nranks * t->ngroups; ++i) {
    if (!t->ptr[i]) return COCO_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(t->ptr[i]) & 15) return COCO_ERR_ALIGN;
  }
  if (o->local[t->ndim - 1] % (t->dtype == COCO_F8E4M3 ? 16 : 8)) return COCO_ERR_ALIGN;
  return COCO_OK;
}

inline bool same_ranks(const TInfo& a, const TInfo& b) { return a.nranks == b.nranks && a.ngroups == b.ngroups; }

inline bool same_local_shape(const TInfo& a, const TInfo& b) {
  if (a.ndim != b.ndim) return false;
  for (int d = 0; d < a.ndim; ++d)
    if (a.local[d] != b.local[d]) return false;
  return true;
}

struct Range {
  uintptr_t lo, hi;
};
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
inline Range range_of(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + static_cast<uintptr_t>(bytes)};
}

// Outputs must not partially overlap each other or any input. `exact_ok`:
// an output may coincide exactly with an input (element-wise kernels read
// every input element before writing the outputs at the same index).
inline coco_status check_alias(const std::vector<Range>& outs, const std::vector<Range>& ins, bool exact_ok) {
  for (size_t i = 0; i < outs.size(); ++i) {
    for (size_t j = i + 1; j < outs.size(); ++j) {
      if (outs[i].lo == outs[j].lo && outs[i].hi == outs[j].hi) continue;  // the same buffer: written once
      if (overlap(outs[i], outs[j])) return COCO_ERR_ALIAS;
    }
    for (const Range& r : ins) {
      if (!overlap(outs[i], r)) continue;
      if (exact_ok && outs[i].lo == r.lo && outs[i].hi == r.hi) continue;
      return COCO_ERR_ALIAS;
    }
  }
  return COCO_OK;
}

// Distinct output pointers of every group, compacted into tables.out.
inline void fill_outputs(const TInfo& out, ReduceTables* t) {
  for (int g = 0; g < out.ngroups; ++g) {
    int n = 0;
    for (int r = 0; r < out.nranks; ++r) {
      void* p = out.ptr(g, r);
      bool seen = false;
      for (int q = 0; q < n; ++q) seen |= (t->out[g * out.nranks + q] == p);
      if (!seen) t->out[g * out.nranks + n++] = p;
    }
    t->nout[g] = n;
  }
}

inline void tensor_ranges(const TInfo& a, std::vector<Range>* v, bool first_only = false) {
  if (a.bytes == 0) return;
  for (int g = 0; g < a.ngroups; ++g)
    for (int r = 0; r < (first_only ? 1 : a.nranks); ++r) v->push_back(range_of(a.ptr(g, r), a.bytes));
}

}  // namespace coco
