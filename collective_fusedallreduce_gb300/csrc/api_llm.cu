// C-ABI entries of the 8-bit and expert-grouped operators: argument validation
// and dispatch. As everywhere in the library, an invalid argument is refused
// before the first CUDA call, no call allocates device memory or synchronises,
// and nothing is kept from one call for the next.

#include <cmath>
#include <cstring>

#include "api_common.h"

using namespace coco;

namespace {

int64_t blocks128(int64_t n) { return (n + 127) / 128; }

// The pointers of a scale array that goes with `t` (one per rank of every group, `bytes` each; `first_only`:
// one per group is read). Appends their ranges.
coco_status check_scales(const float* const* scales, const TInfo& t, int64_t bytes, bool first_only,
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
bool any_overlap(const std::vector<Range>& a, const std::vector<Range>& b) {
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

void group_ranges(const TInfo& a, std::vector<GroupRange>* v, bool first_only = false) {
  if (a.bytes == 0) return;
  for (int g = 0; g < a.ngroups; ++g)
    for (int r = 0; r < (first_only ? 1 : a.nranks); ++r) v->push_back({range_of(a.ptr(g, r), a.bytes), g});
}

// check_alias for outputs that belong to groups.
coco_status check_group_alias(const std::vector<GroupRange>& outs, const std::vector<GroupRange>& ins, bool exact_ok) {
  for (size_t i = 0; i < outs.size(); ++i) {
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (overlap(outs[i].r, outs[j].r) && !outs[i].same_place(outs[j])) return COCO_ERR_ALIAS;
    for (const GroupRange& in : ins)
      if (overlap(outs[i].r, in.r) && !(exact_ok && outs[i].same_place(in))) return COCO_ERR_ALIAS;
  }
  return COCO_OK;
}

std::vector<Range> plain(const std::vector<GroupRange>& v) {
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
void rows_cols(const TInfo& t, int64_t* rows, int64_t* cols) {
  *cols = t.local[t.ndim - 1];
  *rows = 1;
  for (int d = 0; d + 1 < t.ndim; ++d) *rows *= t.local[d];
}

// A plain device pointer argument: present, and aligned to `align` bytes (16 where it is read in vectors).
coco_status check_ptr(const void* p, uintptr_t align) {
  if (!p) return COCO_ERR_NULL;
  return (reinterpret_cast<uintptr_t>(p) & (align - 1)) ? COCO_ERR_ALIGN : COCO_OK;
}

}  // namespace

// -------------------------------------------------------------------- norm

static coco_status allreduce_rmsnorm_impl(const coco_tensor* partials, const coco_tensor* residual,
                                          const void* weight, float eps, const coco_tensor* hidden,
                                          const coco_tensor* normed, float* const* scales, float* rstd,
                                          void* stream) {
  TInfo in, res, hid, nrm;
  coco_status st;
  if ((st = check_tensor(partials, &in)) != COCO_OK) return st;
  if ((st = check_tensor(normed, &nrm, true)) != COCO_OK) return st;
  if (in.layout != COCO_LOCAL || nrm.layout != COCO_REPLICATED) return COCO_ERR_LAYOUT;
  const bool fp8 = nrm.dtype == COCO_F8E4M3;
  if (!fp8 && nrm.dtype != in.dtype) return COCO_ERR_DTYPE;
  if (!same_ranks(in, nrm) || !same_local_shape(in, nrm)) return COCO_ERR_SHAPE;
  if (residual) {
    if ((st = check_tensor(residual, &res)) != COCO_OK) return st;
    if (res.layout != COCO_REPLICATED) return COCO_ERR_LAYOUT;
    if (res.dtype != in.dtype) return COCO_ERR_DTYPE;
    if (!same_ranks(in, res) || !same_local_shape(in, res)) return COCO_ERR_SHAPE;
  }
  if (hidden) {
    if ((st = check_tensor(hidden, &hid)) != COCO_OK) return st;
    if (hid.layout != COCO_REPLICATED) return COCO_ERR_LAYOUT;
    if (hid.dtype != in.dtype) return COCO_ERR_DTYPE;
    if (!same_ranks(in, hid) || !same_local_shape(in, hid)) return COCO_ERR_SHAPE;
  }
  if (!(eps >= 0.0f) || std::isinf(eps)) return COCO_ERR_VALUE;  // also rejects NaN
  if (!fp8 && scales) return COCO_ERR_DTYPE;
  if (in.numel == 0) return COCO_OK;
  int64_t rows, cols;
  rows_cols(in, &rows, &cols);
  if (cols > kNormMaxCols) return COCO_ERR_UNSUPPORTED;
  if ((st = check_ptr(weight, 16)) != COCO_OK) return st;
  if (rstd && (st = check_ptr(rstd, 4)) != COCO_OK) return st;

  std::vector<GroupRange> ins_g, hid_g, nrm_g, aux_g;
  group_ranges(in, &ins_g);
  if (residual) group_ranges(res, &ins_g, true);
  if (hidden) group_ranges(hid, &hid_g);
  group_ranges(nrm, &nrm_g);
  std::vector<Range> aux_r;
  if (fp8 && (st = check_scales(scales, nrm, rows * blocks128(cols) * 4, false, &aux_r)) != COCO_OK) return st;
  for (size_t i = 0; i < aux_r.size(); ++i) aux_g.push_back({aux_r[i], static_cast<int>(i) / nrm.nranks});
  if ((st = check_group_alias(aux_g, ins_g, false)) != COCO_OK) return st;
  std::vector<Range> rstd_r;
  if (rstd) rstd_r.push_back(range_of(rstd, rows * in.ngroups * 4));
  // an element-wise output may take an input's place exactly; e4m3 values are smaller than what they come from
  if ((st = check_group_alias(hid_g, ins_g, true)) != COCO_OK) return st;
  if ((st = check_group_alias(nrm_g, ins_g, !fp8)) != COCO_OK) return st;
  const std::vector<Range> ins = plain(ins_g), hid_r = plain(hid_g), nrm_r = plain(nrm_g);
  const std::vector<Range> w{range_of(weight, cols * dtype_size(in.dtype))};
  if (any_overlap(hid_r, nrm_r) || any_overlap(hid_r, aux_r) || any_overlap(nrm_r, aux_r) ||
      any_overlap(rstd_r, hid_r) || any_overlap(rstd_r, nrm_r) || any_overlap(rstd_r, aux_r) ||
      any_overlap(rstd_r, ins) || any_overlap(w, hid_r) || any_overlap(w, nrm_r) || any_overlap(w, aux_r) ||
      any_overlap(w, rstd_r))
    return COCO_ERR_ALIAS;

  NormLaunch L;
  std::memset(&L, 0, sizeof(L));
  for (int i = 0; i < in.nranks * in.ngroups; ++i) L.t.in[i] = partials->ptr[i];
  for (int g = 0; g < in.ngroups; ++g) {
    const int s0 = g * in.nranks;
    L.t.residual[g] = residual ? res.ptr(g, 0) : nullptr;
    int nh = 0, nn = 0;
    for (int r = 0; r < in.nranks; ++r) {
      if (hidden) {
        bool seen = false;
        for (int q = 0; q < nh; ++q) seen |= L.t.hidden[s0 + q] == hid.ptr(g, r);
        if (!seen) L.t.hidden[s0 + nh++] = hid.ptr(g, r);
      }
      float* sc = fp8 ? scales[s0 + r] : nullptr;
      bool seen = false;
      for (int q = 0; q < nn; ++q) seen |= L.t.normed[s0 + q] == nrm.ptr(g, r) && L.t.scales[s0 + q] == sc;
      if (!seen) {
        L.t.normed[s0 + nn] = nrm.ptr(g, r);
        L.t.scales[s0 + nn++] = sc;
      }
    }
    L.t.nhidden[g] = nh;
    L.t.nnormed[g] = nn;
  }
  L.dtype = in.dtype;
  L.fp8 = fp8;
  L.nranks = in.nranks;
  L.ngroups = in.ngroups;
  L.rows = rows;
  L.cols = static_cast<int32_t>(cols);
  L.eps = eps;
  L.weight = weight;
  L.rstd = rstd;
  return cuda_status(launch_allreduce_rmsnorm(L, static_cast<cudaStream_t>(stream)));
}

COCO_EXPORT coco_status coco_allreduce_rmsnorm(const coco_tensor* partials, const coco_tensor* residual,
                                               const void* weight, float eps, const coco_tensor* hidden,
                                               const coco_tensor* normed, float* const* scales, float* rstd,
                                               void* stream) {
  return guarded([&] {
    return allreduce_rmsnorm_impl(partials, residual, weight, eps, hidden, normed, scales, rstd, stream);
  });
}

COCO_EXPORT size_t coco_allreduce_rmsnorm_backward_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > (int64_t(1) << 40) || cols > kNormMaxCols) return 0;
  return static_cast<size_t>(norm_backward_parts(rows)) * static_cast<size_t>(cols) * 4;
}

static coco_status allreduce_rmsnorm_backward_impl(const coco_tensor* dnormed, const coco_tensor* dhidden,
                                                   const coco_tensor* hidden, const void* weight,
                                                   const float* rstd, const coco_tensor* dx, float* dweight,
                                                   void* workspace, size_t workspace_bytes, void* stream) {
  TInfo in, dh, hid, o;
  coco_status st;
  if ((st = check_tensor(dnormed, &in)) != COCO_OK) return st;
  if ((st = check_tensor(hidden, &hid)) != COCO_OK) return st;
  if ((st = check_tensor(dx, &o)) != COCO_OK) return st;
  if (in.layout != COCO_LOCAL || hid.layout != COCO_REPLICATED || o.layout != COCO_REPLICATED)
    return COCO_ERR_LAYOUT;
  if (hid.dtype != in.dtype || o.dtype != in.dtype) return COCO_ERR_DTYPE;
  if (!same_ranks(in, hid) || !same_ranks(in, o) || !same_local_shape(in, hid) || !same_local_shape(in, o))
    return COCO_ERR_SHAPE;
  if (dhidden) {
    if ((st = check_tensor(dhidden, &dh)) != COCO_OK) return st;
    if (dh.layout != COCO_REPLICATED) return COCO_ERR_LAYOUT;
    if (dh.dtype != in.dtype) return COCO_ERR_DTYPE;
    if (!same_ranks(in, dh) || !same_local_shape(in, dh)) return COCO_ERR_SHAPE;
  }
  int64_t rows, cols;
  rows_cols(in, &rows, &cols);
  if (cols > kNormMaxCols) return COCO_ERR_UNSUPPORTED;
  if (cols == 0) return COCO_OK;
  if ((st = check_ptr(dweight, 4)) != COCO_OK) return st;
  NormBwdLaunch L;
  std::memset(&L, 0, sizeof(L));
  L.dtype = in.dtype;
  L.nranks = in.nranks;
  L.ngroups = in.ngroups;
  L.rows = rows;
  L.cols = static_cast<int32_t>(cols);
  L.dweight = dweight;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) return cuda_status(launch_rmsnorm_backward(L, s));  // no rows: the weight's gradient is zero
  if ((st = check_ptr(weight, 16)) != COCO_OK || (st = check_ptr(rstd, 4)) != COCO_OK ||
      (st = check_ptr(workspace, 16)) != COCO_OK)
    return st;
  const size_t need = coco_allreduce_rmsnorm_backward_bytes(rows * in.ngroups, cols);
  if (workspace_bytes < need) return COCO_ERR_SHAPE;

  std::vector<GroupRange> ins_g, outs_g;
  group_ranges(in, &ins_g);
  group_ranges(hid, &ins_g, true);
  if (dhidden) group_ranges(dh, &ins_g, true);
  group_ranges(o, &outs_g);
  if ((st = check_group_alias(outs_g, ins_g, true)) != COCO_OK) return st;
  const std::vector<Range> ins = plain(ins_g), outs = plain(outs_g);
  const std::vector<Range> small_in{range_of(weight, cols * dtype_size(in.dtype)),
                                    range_of(rstd, rows * in.ngroups * 4)};
  const std::vector<Range> dw{range_of(dweight, cols * 4)};
  const std::vector<Range> ws{range_of(workspace, static_cast<int64_t>(need))};
  if (any_overlap(small_in, outs) || any_overlap(dw, outs) || any_overlap(dw, ins) || any_overlap(dw, small_in) ||
      any_overlap(ws, outs) || any_overlap(ws, ins) || any_overlap(ws, small_in) || any_overlap(ws, dw))
    return COCO_ERR_ALIAS;

  for (int i = 0; i < in.nranks * in.ngroups; ++i) L.in[i] = dnormed->ptr[i];
  for (int g = 0; g < in.ngroups; ++g) {
    L.dhidden[g] = dhidden ? dh.ptr(g, 0) : nullptr;
    L.hidden[g] = hid.ptr(g, 0);
    int n = 0;
    for (int r = 0; r < in.nranks; ++r) {
      bool seen = false;
      for (int q = 0; q < n; ++q) seen |= L.dx[g * in.nranks + q] == o.ptr(g, r);
      if (!seen) L.dx[g * in.nranks + n++] = o.ptr(g, r);
    }
    L.ndx[g] = n;
  }
  L.weight = weight;
  L.rstd = rstd;
  L.partial = static_cast<float*>(workspace);
  return cuda_status(launch_rmsnorm_backward(L, s));
}

COCO_EXPORT coco_status coco_allreduce_rmsnorm_backward(const coco_tensor* dnormed, const coco_tensor* dhidden,
                                                        const coco_tensor* hidden, const void* weight,
                                                        const float* rstd, const coco_tensor* dx, float* dweight,
                                                        void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&] {
    return allreduce_rmsnorm_backward_impl(dnormed, dhidden, hidden, weight, rstd, dx, dweight, workspace,
                                           workspace_bytes, stream);
  });
}

// --------------------------------------------------------------- quantiser

static coco_status quantize_fp8_impl(const coco_tensor* x, int32_t block_rows, const coco_tensor* q,
                                     float* const* scales, void* stream) {
  TInfo in, o;
  coco_status st;
  if ((st = check_tensor(x, &in)) != COCO_OK) return st;
  if ((st = check_tensor(q, &o, true)) != COCO_OK) return st;
  if (in.layout != COCO_LOCAL || o.layout != COCO_LOCAL) return COCO_ERR_LAYOUT;
  if (o.dtype != COCO_F8E4M3) return COCO_ERR_DTYPE;
  if (!same_ranks(in, o) || !same_local_shape(in, o)) return COCO_ERR_SHAPE;
  if (block_rows != 1 && block_rows != 128) return COCO_ERR_VALUE;
  if (in.numel == 0) return COCO_OK;
  // rows: all leading dimensions for one scale per row; matrix by matrix for tiles of 128 rows
  int64_t rows, cols;
  rows_cols(in, &rows, &cols);
  if (cols >= (int64_t(1) << 31)) return COCO_ERR_UNSUPPORTED;
  int64_t matrices = 1;
  if (block_rows == 128 && in.ndim == 3) {
    matrices = in.local[0];
    rows = in.local[1];
  }
  const int64_t per = (block_rows == 1 ? rows : blocks128(rows)) * blocks128(cols);
  std::vector<Range> ins, outs, sc;
  tensor_ranges(in, &ins);
  tensor_ranges(o, &outs);
  if ((st = check_scales(scales, o, matrices * per * 4, false, &sc)) != COCO_OK) return st;
  std::vector<Range> all = outs;
  all.insert(all.end(), sc.begin(), sc.end());
  for (size_t i = 0; i < all.size(); ++i) {  // every rank's values differ: no two outputs may share memory
    for (size_t j = i + 1; j < all.size(); ++j)
      if (overlap(all[i], all[j])) return COCO_ERR_ALIAS;
    for (const Range& r : ins)
      if (overlap(all[i], r)) return COCO_ERR_ALIAS;
  }
  QuantLaunch L;
  std::memset(&L, 0, sizeof(L));
  L.dtype = in.dtype;
  L.block_rows = block_rows;
  L.rows = rows;
  L.cols = static_cast<int32_t>(cols);
  // (matrices of a 3-D tensor are tensors of their own, as many to a launch as its table holds)
  const int64_t count = matrices * in.nranks * in.ngroups;
  for (int64_t first = 0; first < count; first += COCO_MAX_PTRS) {
    L.ntensors = static_cast<int>(count - first < COCO_MAX_PTRS ? count - first : COCO_MAX_PTRS);
    for (int i = 0; i < L.ntensors; ++i) {
      const int64_t p = (first + i) / matrices, m = (first + i) % matrices;
      L.x[i] = static_cast<const char*>(x->ptr[p]) + m * rows * cols * dtype_size(in.dtype);
      L.q[i] = static_cast<char*>(q->ptr[p]) + m * rows * cols;
      L.scales[i] = scales[p] + m * per;
    }
    if ((st = cuda_status(launch_quantize_fp8(L, static_cast<cudaStream_t>(stream)))) != COCO_OK) return st;
  }
  return COCO_OK;
}

COCO_EXPORT coco_status coco_quantize_fp8(const coco_tensor* x, int32_t block_rows, const coco_tensor* q,
                                          float* const* scales, void* stream) {
  return guarded([&] { return quantize_fp8_impl(x, block_rows, q, scales, stream); });
}

// ---------------------------------------------------------------- products

namespace {

bool same_spec(const char* spec, const char* want) {
  for (;; ++spec) {
    if (*spec == ' ') continue;
    if (*spec != *want) return false;
    if (!*want) return true;
    ++want;
  }
}

bool fits_i32(int64_t v) { return v >= 0 && v < (int64_t(1) << 31); }

// The checks that both product entries share, after each has read its shapes into L.
coco_status run_grouped(const TInfo& lhs, const TInfo& rhs, const TInfo& out, const float* const* lhs_scales,
                        const float* const* rhs_scales, int64_t offsets_bytes, GroupedLaunch* L, void* stream) {
  const bool fp8 = lhs.dtype == COCO_F8E4M3;
  coco_status st;
  std::vector<Range> ins, outs;
  tensor_ranges(lhs, &ins, lhs.layout == COCO_REPLICATED);
  tensor_ranges(rhs, &ins, rhs.layout == COCO_REPLICATED);
  if (fp8) {
    const int64_t kb = blocks128(L->k), nb = blocks128(L->n);
    if (lhs.numel > 0 &&
        (st = check_scales(lhs_scales, lhs, L->rows * kb * 4, lhs.layout == COCO_REPLICATED, &ins)) != COCO_OK)
      return st;
    if (rhs.numel > 0 && (st = check_scales(rhs_scales, rhs, static_cast<int64_t>(L->experts) * kb * nb * 4,
                                            rhs.layout == COCO_REPLICATED, &ins)) != COCO_OK)
      return st;
  }
  if (L->offsets) ins.push_back(range_of(L->offsets, offsets_bytes));
  tensor_ranges(out, &outs);
  for (size_t i = 0; i < outs.size(); ++i)  // every rank's product differs
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (overlap(outs[i], outs[j])) return COCO_ERR_ALIAS;
  if ((st = check_alias(outs, ins, false)) != COCO_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  L->nprob = out.nranks * out.ngroups;
  if (lhs.numel == 0 || rhs.numel == 0) {  // an empty contraction (or no rows, or no experts): zeros
    for (int p = 0; p < L->nprob; ++p) {
      cudaError_t e = cudaMemsetAsync(out.t->ptr[p], 0, out.bytes, s);
      if (e != cudaSuccess) return cuda_status(e);
    }
    return COCO_OK;
  }
  for (int g = 0; g < out.ngroups; ++g)
    for (int r = 0; r < out.nranks; ++r) {
      const int p = g * out.nranks + r;
      const int lp = lhs.layout == COCO_REPLICATED ? g * out.nranks : p;
      const int rp = rhs.layout == COCO_REPLICATED ? g * out.nranks : p;
      L->lhs[p] = lhs.t->ptr[lp];
      L->rhs[p] = rhs.t->ptr[rp];
      L->out[p] = out.t->ptr[p];
      L->lhs_scales[p] = fp8 ? lhs_scales[lp] : nullptr;
      L->rhs_scales[p] = fp8 ? rhs_scales[rp] : nullptr;
    }
  L->in_dtype = lhs.dtype;
  L->out_dtype = out.dtype;
  unsigned int* err = gemm_error_word();
  if (!err) return cuda_status(cudaErrorSymbolNotFound);
  const cudaError_t e = launch_grouped(*L, s, err);
  return e == cudaErrorNotSupported ? COCO_ERR_UNSUPPORTED : cuda_status(e);
}

}  // namespace

static coco_status einsum_fp8_impl(const char* spec, const coco_tensor* lhs, const float* const* lhs_scales,
                                   const coco_tensor* rhs, const float* const* rhs_scales,
                                   const coco_tensor* out, void* stream) {
  const bool kn = spec && same_spec(spec, "mk,kn->mn"), nk = spec && same_spec(spec, "mk,nk->mn");
  if (!kn && !nk) return COCO_ERR_UNSUPPORTED;
  TInfo a, b, o;
  coco_status st;
  if ((st = check_tensor(lhs, &a, true)) != COCO_OK) return st;
  if ((st = check_tensor(rhs, &b, true)) != COCO_OK) return st;
  if ((st = check_tensor(out, &o)) != COCO_OK) return st;
  if (a.ndim != 2 || b.ndim != 2 || o.ndim != 2) return COCO_ERR_SHAPE;
  if (a.dtype != COCO_F8E4M3 || b.dtype != COCO_F8E4M3) return COCO_ERR_DTYPE;
  if (!same_ranks(a, b) || !same_ranks(a, o)) return COCO_ERR_SHAPE;
  // a slice is on the contracting dimension (each rank's product is a partial), as for the MatMul of 16-bit types
  const int bk = kn ? 0 : 1;
  if (o.layout != COCO_LOCAL || (a.layout == COCO_SLICED && a.slice_dim != 1) ||
      (b.layout == COCO_SLICED && b.slice_dim != bk))
    return COCO_ERR_LAYOUT;
  if (b.local[bk] != a.local[1] || o.local[0] != a.local[0] || o.local[1] != b.local[1 - bk]) return COCO_ERR_SHAPE;
  for (int d = 0; d < 2; ++d)
    if (!fits_i32(a.local[d]) || !fits_i32(b.local[d])) return COCO_ERR_UNSUPPORTED;
  if (o.numel == 0) return COCO_OK;
  GroupedLaunch L;
  std::memset(&L, 0, sizeof(L));
  L.experts = 1;
  L.form = kn ? GRP_KN : GRP_NK;
  L.rows = static_cast<int32_t>(a.local[0]);
  L.k = static_cast<int32_t>(a.local[1]);
  L.n = static_cast<int32_t>(o.local[1]);
  return run_grouped(a, b, o, lhs_scales, rhs_scales, 0, &L, stream);
}

COCO_EXPORT coco_status coco_einsum_fp8(const char* spec, const coco_tensor* lhs, const float* const* lhs_scales,
                                        const coco_tensor* rhs, const float* const* rhs_scales,
                                        const coco_tensor* out, void* stream) {
  return guarded([&] { return einsum_fp8_impl(spec, lhs, lhs_scales, rhs, rhs_scales, out, stream); });
}

static coco_status grouped_einsum_impl(const char* spec, const coco_tensor* lhs, const float* const* lhs_scales,
                                       const coco_tensor* rhs, const float* const* rhs_scales,
                                       const int32_t* offsets, const coco_tensor* out, void* stream) {
  int form;
  if (spec && same_spec(spec, "tk,ekn->tn")) form = GRP_KN;
  else if (spec && same_spec(spec, "tk,enk->tn")) form = GRP_NK;
  else if (spec && same_spec(spec, "tk,tn->ekn")) form = GRP_GRAD;
  else return COCO_ERR_UNSUPPORTED;
  TInfo a, b, o;
  coco_status st;
  if ((st = check_tensor(lhs, &a, true)) != COCO_OK) return st;
  if ((st = check_tensor(rhs, &b, true)) != COCO_OK) return st;
  if ((st = check_tensor(out, &o)) != COCO_OK) return st;
  const bool grad = form == GRP_GRAD;
  if (a.ndim != 2 || b.ndim != (grad ? 2 : 3) || o.ndim != (grad ? 3 : 2)) return COCO_ERR_SHAPE;
  if (a.dtype != b.dtype) return COCO_ERR_DTYPE;
  if (a.dtype == COCO_F32 || (grad && a.dtype == COCO_F8E4M3)) return COCO_ERR_UNSUPPORTED;
  if (a.dtype != COCO_F8E4M3 && (lhs_scales || rhs_scales)) return COCO_ERR_DTYPE;
  if (!same_ranks(a, b) || !same_ranks(a, o)) return COCO_ERR_SHAPE;
  if (a.layout == COCO_SLICED || b.layout == COCO_SLICED || o.layout != COCO_LOCAL) return COCO_ERR_LAYOUT;
  GroupedLaunch L;
  std::memset(&L, 0, sizeof(L));
  int64_t experts, k, n;
  const int64_t rows = a.local[0];
  if (grad) {
    experts = o.local[0], k = o.local[1], n = o.local[2];
    if (a.local[1] != k || b.local[0] != rows || b.local[1] != n) return COCO_ERR_SHAPE;
  } else {
    experts = b.local[0];
    k = b.local[form == GRP_KN ? 1 : 2];
    n = b.local[form == GRP_KN ? 2 : 1];
    if (a.local[1] != k || o.local[0] != rows || o.local[1] != n) return COCO_ERR_SHAPE;
  }
  if (!fits_i32(rows) || !fits_i32(k) || !fits_i32(n) || experts > kGroupedMaxExperts) return COCO_ERR_UNSUPPORTED;
  if (o.numel == 0) return COCO_OK;
  if (a.numel > 0 && b.numel > 0 && (st = check_ptr(offsets, 4)) != COCO_OK) return st;
  L.experts = static_cast<int32_t>(experts);
  L.form = form;
  L.rows = static_cast<int32_t>(rows);
  L.k = static_cast<int32_t>(k);
  L.n = static_cast<int32_t>(n);
  L.offsets = offsets;
  return run_grouped(a, b, o, lhs_scales, rhs_scales,
                     static_cast<int64_t>(a.nranks) * a.ngroups * (experts + 1) * 4, &L, stream);
}

COCO_EXPORT coco_status coco_grouped_einsum(const char* spec, const coco_tensor* lhs, const float* const* lhs_scales,
                                            const coco_tensor* rhs, const float* const* rhs_scales,
                                            const int32_t* offsets, const coco_tensor* out, void* stream) {
  return guarded([&] { return grouped_einsum_impl(spec, lhs, lhs_scales, rhs, rhs_scales, offsets, out, stream); });
}
