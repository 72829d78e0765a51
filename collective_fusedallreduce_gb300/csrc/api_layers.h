// Checks shared by the entry points of the operators of a language model's layers
// (api_llm.cu, api_layers.cu).
#pragma once

#include "api_common.h"

namespace coco {

inline int64_t blocks128(int64_t n) { return (n + 127) / 128; }

// The pointers of a scale array that goes with `t` (one per rank of every group, `bytes` each; `first_only`:
// one per group is read). Appends their ranges.
inline coco_status check_scales(const float* const* scales, const TInfo& t, int64_t bytes, bool first_only,
                         std::vector<Range>* ranges) {
  if (!scales) return COCO_ERR_NULL;
  for (int g = 0; g < t.ngroups; ++g)
    for (int r = 0; r < (first_only ? 1 : t.nranks); ++r) {
      const float* p = scales[g * t.nranks + r];
      if (!p) return COCO_ERR_NULL;
      if (reinterpret_cast<uintptr_t>(p) & 3) return COCO_ERR_ALIGN;
      ranges->push_back(range_of(p, bytes));
    }
  return COCO_OK;
}

// Outputs of different roles may not share memory at all (check_alias lets one buffer stand for several
// replicas of one output).
inline bool any_overlap(const std::vector<Range>& a, const std::vector<Range>& b) {
  for (const Range& x : a)
    for (const Range& y : b)
      if (overlap(x, y)) return true;
  return false;
}

// Memory of one group's rows. Groups run at the same time, and what orders a write after a read (an output in an
// input's place) or makes equal writes harmless (one buffer for several replicas) holds within a group only.
struct GroupRange {
  Range r;
  int group;
  bool same_place(const GroupRange& o) const { return group == o.group && r.lo == o.r.lo && r.hi == o.r.hi; }
};

inline void group_ranges(const TInfo& a, std::vector<GroupRange>* v, bool first_only = false) {
  if (a.bytes == 0) return;
  for (int g = 0; g < a.ngroups; ++g)
    for (int r = 0; r < (first_only ? 1 : a.nranks); ++r) v->push_back({range_of(a.ptr(g, r), a.bytes), g});
}

// check_alias for outputs that belong to groups.
inline coco_status check_group_alias(const std::vector<GroupRange>& outs, const std::vector<GroupRange>& ins, bool exact_ok) {
  for (size_t i = 0; i < outs.size(); ++i) {
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (overlap(outs[i].r, outs[j].r) && !outs[i].same_place(outs[j])) return COCO_ERR_ALIAS;
    for (const GroupRange& in : ins)
      if (overlap(outs[i].r, in.r) && !(exact_ok && outs[i].same_place(in))) return COCO_ERR_ALIAS;
  }
  return COCO_OK;
}

inline std::vector<Range> plain(const std::vector<GroupRange>& v) {
  std::vector<Range> out;
  for (const GroupRange& x : v) out.push_back(x.r);
  return out;
}

// No C++ exception leaves an entry point: running out of host memory is reported as the CUDA error of that name.
template <typename F>
coco_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return cuda_status(cudaErrorMemoryAllocation);
  }
}

// Rows and columns of a per-rank tensor (all leading dimensions are rows).
inline void rows_cols(const TInfo& t, int64_t* rows, int64_t* cols) {
  *cols = t.local[t.ndim - 1];
  *rows = 1;
  for (int d = 0; d + 1 < t.ndim; ++d) *rows *= t.local[d];
}

// A plain device pointer argument: present, and aligned to `align` bytes (16 where it is read in vectors).
inline coco_status check_ptr(const void* p, uintptr_t align) {
  if (!p) return COCO_ERR_NULL;
  return (reinterpret_cast<uintptr_t>(p) & (align - 1)) ? COCO_ERR_ALIGN : COCO_OK;
}

}  // namespace coco
