// C-ABI entries of the operators that move tokens to their experts and back, of the
// layer norm after an AllReduce, and of clipping scattered gradients: argument
// validation and dispatch. As everywhere in the library, an invalid argument is
// refused before the first CUDA call, no call allocates device memory or
// synchronises, and nothing is kept from one call for the next.

#include <cmath>
#include <cstring>

#include "api_layers.h"

using namespace coco;

namespace {

using Groups = std::vector<GroupRange>;

// Outputs that every group has its own of: distinct from each other and from every input, replicas of a group aside.
coco_status apart(const Groups& outs, const Groups& ins) { return check_group_alias(outs, ins, false); }

// Plain arrays: no two outputs share memory, nor an output with an input.
coco_status apart(const std::vector<Range>& outs, const std::vector<Range>& ins) {
  for (size_t i = 0; i < outs.size(); ++i) {
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (overlap(outs[i], outs[j])) return COCO_ERR_ALIAS;
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return COCO_ERR_ALIAS;
  }
  return COCO_OK;
}

void append_scales(const std::vector<Range>& r, int per_group, Groups* v) {
  for (size_t i = 0; i < r.size(); ++i) v->push_back({r[i], static_cast<int>(i) / per_group});
}

// Group g's distinct (tensor, scales) outputs.
void fill_rows_out(const TInfo& out, float* const* scales, ExpertTables* t) {
  for (int g = 0; g < out.ngroups; ++g) {
    const int s0 = g * out.nranks;
    int n = 0;
    for (int r = 0; r < out.nranks; ++r) {
      void* p = out.ptr(g, r);
      float* sc = scales ? scales[s0 + r] : nullptr;
      bool seen = false;
      for (int q = 0; q < n; ++q) seen |= t->out[s0 + q] == p && t->out_scales[s0 + q] == sc;
      if (!seen) {
        t->out[s0 + n] = p;
        t->out_scales[s0 + n++] = sc;
      }
    }
    t->nout[g] = n;
  }
}

// The shapes that a routing's operands share: `tok` is [tokens, cols] and `rows` [tokens * choices, cols].
coco_status routed_shapes(const TInfo& tok, const TInfo& rows, ExpertRowsLaunch* L) {
  if (tok.ndim != 2 || rows.ndim != 2 || !same_ranks(tok, rows)) return COCO_ERR_SHAPE;
  if (tok.local[1] != rows.local[1]) return COCO_ERR_SHAPE;
  const int64_t tokens = tok.local[0], n = rows.local[0];
  if (tokens == 0 ? n != 0 : n % tokens != 0) return COCO_ERR_SHAPE;
  if (n >= (int64_t(1) << 31) || tokens >= (int64_t(1) << 31) || tok.local[1] >= (int64_t(1) << 30))
    return COCO_ERR_UNSUPPORTED;
  L->tokens = tokens;
  L->rows = n;
  L->choices = tokens ? static_cast<int32_t>(n / tokens) : 0;
  L->cols = static_cast<int32_t>(tok.local[1]);
  L->nranks = tok.nranks;
  L->ngroups = tok.ngroups;
  return COCO_OK;
}

}  // namespace

// ----------------------------------------------------------------- experts

static coco_status expert_sort_impl(const void* expert_of, int32_t index_bytes, int64_t tokens, int32_t choices,
                                    int32_t experts, int32_t ngroups, int32_t nranks, int32_t* row_of_choice,
                                    int32_t* choice_of_row, int32_t* offsets, void* stream) {
  if (index_bytes != 4 && index_bytes != 8) return COCO_ERR_DTYPE;
  if (tokens < 0 || choices < 0 || experts < 0) return COCO_ERR_SHAPE;
  if (nranks < 1 || ngroups < 1 || static_cast<int64_t>(nranks) * ngroups > COCO_MAX_PTRS) return COCO_ERR_SHAPE;
  const int64_t limit = int64_t(1) << 31;
  if (tokens >= limit || tokens * choices >= limit || experts > kGroupedMaxExperts) return COCO_ERR_UNSUPPORTED;
  const int64_t n = tokens * choices;
  coco_status st;
  if ((st = check_ptr(offsets, 4)) != COCO_OK) return st;
  std::vector<Range> ins, outs{range_of(offsets, static_cast<int64_t>(nranks) * ngroups * (int64_t(experts) + 1) * 4)};
  if (n > 0) {
    if ((st = check_ptr(expert_of, index_bytes)) != COCO_OK || (st = check_ptr(row_of_choice, 4)) != COCO_OK) return st;
    if (choice_of_row && (st = check_ptr(choice_of_row, 4)) != COCO_OK) return st;
    ins.push_back(range_of(expert_of, ngroups * n * index_bytes));
    outs.push_back(range_of(row_of_choice, ngroups * n * 4));
    if (choice_of_row) outs.push_back(range_of(choice_of_row, ngroups * n * 4));
  }
  if ((st = apart(outs, ins)) != COCO_OK) return st;
  ExpertSortLaunch L;
  L.expert_of = expert_of;
  L.index64 = index_bytes == 8;
  L.n = n;
  L.experts = experts;
  L.nranks = nranks;
  L.ngroups = ngroups;
  L.row_of = row_of_choice;
  L.choice_of = n > 0 ? choice_of_row : nullptr;
  L.offsets = offsets;
  return cuda_status(launch_expert_sort(L, static_cast<cudaStream_t>(stream)));
}

COCO_EXPORT coco_status coco_expert_sort(const void* expert_of, int32_t index_bytes, int64_t tokens, int32_t choices,
                                         int32_t experts, int32_t ngroups, int32_t nranks, int32_t* row_of_choice,
                                         int32_t* choice_of_row, int32_t* offsets, void* stream) {
  return guarded([&] {
    return expert_sort_impl(expert_of, index_bytes, tokens, choices, experts, ngroups, nranks, row_of_choice,
                            choice_of_row, offsets, stream);
  });
}

static coco_status expert_dispatch_impl(const coco_tensor* x, const float* const* x_scales,
                                        const int32_t* row_of_choice, const coco_tensor* rows,
                                        float* const* row_scales, void* stream) {
  TInfo in, o;
  coco_status st;
  if ((st = check_tensor(x, &in, true)) != COCO_OK) return st;
  if ((st = check_tensor(rows, &o, true)) != COCO_OK) return st;
  if (in.layout != COCO_REPLICATED || o.layout != COCO_REPLICATED) return COCO_ERR_LAYOUT;
  if (in.dtype != o.dtype) return COCO_ERR_DTYPE;
  const bool fp8 = in.dtype == COCO_F8E4M3;
  if (!fp8 && (x_scales || row_scales)) return COCO_ERR_DTYPE;
  ExpertRowsLaunch L;
  std::memset(&L, 0, sizeof(L));
  if ((st = routed_shapes(in, o, &L)) != COCO_OK) return st;
  if (o.numel == 0) return COCO_OK;
  if ((st = check_ptr(row_of_choice, 4)) != COCO_OK) return st;
  Groups ins, outs, sc_g;
  group_ranges(in, &ins, true);
  group_ranges(o, &outs);
  const int64_t nb = blocks128(L.cols);
  if (fp8) {
    std::vector<Range> sin, sout;
    if ((st = check_scales(x_scales, in, L.tokens * nb * 4, true, &sin)) != COCO_OK) return st;
    if ((st = check_scales(row_scales, o, L.rows * nb * 4, false, &sout)) != COCO_OK) return st;
    append_scales(sin, 1, &ins);
    append_scales(sout, o.nranks, &sc_g);
  }
  if ((st = apart(outs, ins)) != COCO_OK || (st = apart(sc_g, ins)) != COCO_OK) return st;
  const std::vector<Range> at{range_of(row_of_choice, o.ngroups * L.rows * 4)};
  if (any_overlap(plain(outs), plain(sc_g)) || any_overlap(at, plain(outs)) || any_overlap(at, plain(sc_g)))
    return COCO_ERR_ALIAS;
  for (int g = 0; g < in.ngroups; ++g) {
    L.t.in[g] = in.ptr(g, 0);
    L.t.in_scales[g] = fp8 ? x_scales[g * in.nranks] : nullptr;
  }
  fill_rows_out(o, fp8 ? row_scales : nullptr, &L.t);
  L.dtype = in.dtype;
  L.row_of = row_of_choice;
  return cuda_status(launch_expert_dispatch(L, static_cast<cudaStream_t>(stream)));
}

COCO_EXPORT coco_status coco_expert_dispatch(const coco_tensor* x, const float* const* x_scales,
                                             const int32_t* row_of_choice, const coco_tensor* rows,
                                             float* const* row_scales, void* stream) {
  return guarded([&] { return expert_dispatch_impl(x, x_scales, row_of_choice, rows, row_scales, stream); });
}

static coco_status expert_combine_impl(const coco_tensor* rows, const int32_t* row_of_choice, const float* gates,
                                       const coco_tensor* residual, const coco_tensor* out, void* stream) {
  TInfo in, res, o;
  coco_status st;
  if ((st = check_tensor(rows, &in)) != COCO_OK) return st;
  if ((st = check_tensor(out, &o)) != COCO_OK) return st;
  if (in.layout != COCO_LOCAL || o.layout == COCO_SLICED) return COCO_ERR_LAYOUT;
  if (in.dtype != o.dtype) return COCO_ERR_DTYPE;
  const bool summed = o.layout == COCO_REPLICATED;
  ExpertRowsLaunch L;
  std::memset(&L, 0, sizeof(L));
  if ((st = routed_shapes(o, in, &L)) != COCO_OK) return st;
  if (residual) {
    if ((st = check_tensor(residual, &res)) != COCO_OK) return st;
    if (!summed || res.layout != COCO_REPLICATED) return COCO_ERR_LAYOUT;
    if (res.dtype != o.dtype) return COCO_ERR_DTYPE;
    if (!same_ranks(res, o) || !same_local_shape(res, o)) return COCO_ERR_SHAPE;
  }
  if (o.numel == 0) return COCO_OK;
  std::vector<Range> at;
  if (L.rows > 0) {
    if ((st = check_ptr(row_of_choice, 4)) != COCO_OK) return st;
    if (gates && (st = check_ptr(gates, 4)) != COCO_OK) return st;
    at.push_back(range_of(row_of_choice, o.ngroups * L.rows * 4));
    if (gates) at.push_back(range_of(gates, o.ngroups * L.rows * 4));
  }
  Groups ins, res_g, outs;
  group_ranges(in, &ins);
  if (residual) group_ranges(res, &res_g, true);
  group_ranges(o, &outs);
  if ((st = apart(outs, ins)) != COCO_OK) return st;
  if ((st = check_group_alias(outs, res_g, true)) != COCO_OK) return st;  // the sum may take the residual's place
  if (any_overlap(at, plain(outs))) return COCO_ERR_ALIAS;
  if (!summed)  // every rank's sum differs
    for (size_t i = 0; i < outs.size(); ++i)
      for (size_t j = i + 1; j < outs.size(); ++j)
        if (overlap(outs[i].r, outs[j].r)) return COCO_ERR_ALIAS;
  for (int i = 0; i < in.nranks * in.ngroups; ++i) L.t.in[i] = rows->ptr[i];
  for (int g = 0; g < o.ngroups; ++g) L.t.residual[g] = residual ? res.ptr(g, 0) : nullptr;
  if (summed) fill_rows_out(o, nullptr, &L.t);
  else
    for (int i = 0; i < o.nranks * o.ngroups; ++i) L.t.out[i] = out->ptr[i];
  L.dtype = in.dtype;
  L.summed = summed;
  L.row_of = row_of_choice;
  L.gates = gates;
  return cuda_status(launch_expert_combine(L, static_cast<cudaStream_t>(stream)));
}

COCO_EXPORT coco_status coco_expert_combine(const coco_tensor* rows, const int32_t* row_of_choice, const float* gates,
                                            const coco_tensor* residual, const coco_tensor* out, void* stream) {
  return guarded([&] { return expert_combine_impl(rows, row_of_choice, gates, residual, out, stream); });
}

static coco_status expert_combine_backward_impl(const coco_tensor* dout, const coco_tensor* rows,
                                                const int32_t* row_of_choice, const float* gates,
                                                const coco_tensor* drows, float* dgates, void* stream) {
  TInfo d, in, o;
  coco_status st;
  if ((st = check_tensor(dout, &d)) != COCO_OK) return st;
  if ((st = check_tensor(drows, &o)) != COCO_OK) return st;
  if (d.layout != COCO_REPLICATED || o.layout != COCO_REPLICATED) return COCO_ERR_LAYOUT;
  if (d.dtype != o.dtype) return COCO_ERR_DTYPE;
  ExpertRowsLaunch L;
  std::memset(&L, 0, sizeof(L));
  if ((st = routed_shapes(d, o, &L)) != COCO_OK) return st;
  if (L.rows > 0 && (rows == nullptr) != (dgates == nullptr)) return COCO_ERR_NULL;
  if (rows) {
    if ((st = check_tensor(rows, &in)) != COCO_OK) return st;
    if (in.layout != COCO_LOCAL) return COCO_ERR_LAYOUT;
    if (in.dtype != d.dtype) return COCO_ERR_DTYPE;
    if (!same_ranks(in, o) || !same_local_shape(in, o)) return COCO_ERR_SHAPE;
  }
  if (L.cols > kNormMaxCols) return COCO_ERR_UNSUPPORTED;
  if (L.rows == 0) return COCO_OK;
  const int64_t n = o.ngroups * L.rows;
  if (dgates && (st = check_ptr(dgates, 4)) != COCO_OK) return st;
  if (L.cols == 0)  // rows without columns: their products are zero
    return dgates ? cuda_status(cudaMemsetAsync(dgates, 0, n * 4, static_cast<cudaStream_t>(stream))) : COCO_OK;
  if ((st = check_ptr(row_of_choice, 4)) != COCO_OK) return st;
  if (gates && (st = check_ptr(gates, 4)) != COCO_OK) return st;
  Groups ins, outs;
  group_ranges(d, &ins, true);
  if (rows) group_ranges(in, &ins);
  group_ranges(o, &outs);
  if ((st = apart(outs, ins)) != COCO_OK) return st;
  std::vector<Range> at{range_of(row_of_choice, n * 4)}, dg;
  if (gates) at.push_back(range_of(gates, n * 4));
  if (dgates) dg.push_back(range_of(dgates, n * 4));
  if (any_overlap(at, plain(outs)) || any_overlap(dg, plain(outs)) || any_overlap(dg, plain(ins)) ||
      any_overlap(dg, at))
    return COCO_ERR_ALIAS;
  for (int g = 0; g < o.ngroups; ++g) L.t.residual[g] = d.ptr(g, 0);
  if (rows)
    for (int i = 0; i < in.nranks * in.ngroups; ++i) L.t.in[i] = rows->ptr[i];
  fill_rows_out(o, nullptr, &L.t);
  L.dtype = d.dtype;
  L.row_of = row_of_choice;
  L.gates = gates;
  L.dgates = dgates;
  return cuda_status(launch_expert_combine_backward(L, static_cast<cudaStream_t>(stream)));
}

COCO_EXPORT coco_status coco_expert_combine_backward(const coco_tensor* dout, const coco_tensor* rows,
                                                     const int32_t* row_of_choice, const float* gates,
                                                     const coco_tensor* drows, float* dgates, void* stream) {
  return guarded([&] { return expert_combine_backward_impl(dout, rows, row_of_choice, gates, drows, dgates, stream); });
}

// -------------------------------------------------------------- layer norm

static coco_status allreduce_layernorm_impl(const coco_tensor* partials, const coco_tensor* residual,
                                            const void* weight, const void* bias, float eps,
                                            const coco_tensor* hidden, const coco_tensor* normed,
                                            float* const* scales, float* mean, float* rstd, void* stream) {
  TInfo in, res, hid, nrm;
  coco_status st;
  if ((st = check_tensor(partials, &in)) != COCO_OK) return st;
  if ((st = check_tensor(normed, &nrm, true)) != COCO_OK) return st;
  if (in.layout != COCO_LOCAL || nrm.layout != COCO_REPLICATED) return COCO_ERR_LAYOUT;
  const bool fp8 = nrm.dtype == COCO_F8E4M3;
  if (!fp8 && nrm.dtype != in.dtype) return COCO_ERR_DTYPE;
  if (!same_ranks(in, nrm) || !same_local_shape(in, nrm)) return COCO_ERR_SHAPE;
  struct Optional {
    const coco_tensor* t;
    TInfo* i;
  };
  for (const Optional& x : {Optional{residual, &res}, Optional{hidden, &hid}}) {
    if (!x.t) continue;
    if ((st = check_tensor(x.t, x.i)) != COCO_OK) return st;
    if (x.i->layout != COCO_REPLICATED) return COCO_ERR_LAYOUT;
    if (x.i->dtype != in.dtype) return COCO_ERR_DTYPE;
    if (!same_ranks(in, *x.i) || !same_local_shape(in, *x.i)) return COCO_ERR_SHAPE;
  }
  if (!(eps >= 0.0f) || std::isinf(eps)) return COCO_ERR_VALUE;  // also rejects NaN
  if (!fp8 && scales) return COCO_ERR_DTYPE;
  if (in.numel == 0) return COCO_OK;
  int64_t rows, cols;
  rows_cols(in, &rows, &cols);
  if (cols > kNormMaxCols) return COCO_ERR_UNSUPPORTED;
  if ((st = check_ptr(weight, 16)) != COCO_OK) return st;
  if (bias && (st = check_ptr(bias, 16)) != COCO_OK) return st;
  std::vector<Range> stats, params{range_of(weight, cols * dtype_size(in.dtype))};
  if (bias) params.push_back(range_of(bias, cols * dtype_size(in.dtype)));
  for (float* p : {mean, rstd}) {
    if (!p) continue;
    if ((st = check_ptr(p, 4)) != COCO_OK) return st;
    stats.push_back(range_of(p, rows * in.ngroups * 4));
  }
  if (stats.size() == 2 && overlap(stats[0], stats[1])) return COCO_ERR_ALIAS;

  Groups ins_g, hid_g, nrm_g, aux_g;
  group_ranges(in, &ins_g);
  if (residual) group_ranges(res, &ins_g, true);
  if (hidden) group_ranges(hid, &hid_g);
  group_ranges(nrm, &nrm_g);
  std::vector<Range> aux_r;
  if (fp8 && (st = check_scales(scales, nrm, rows * blocks128(cols) * 4, false, &aux_r)) != COCO_OK) return st;
  append_scales(aux_r, nrm.nranks, &aux_g);
  if ((st = apart(aux_g, ins_g)) != COCO_OK) return st;
  // an element-wise output may take an input's place exactly; e4m3 values are smaller than what they come from
  if ((st = check_group_alias(hid_g, ins_g, true)) != COCO_OK) return st;
  if ((st = check_group_alias(nrm_g, ins_g, !fp8)) != COCO_OK) return st;
  const std::vector<Range> ins = plain(ins_g), hid_r = plain(hid_g), nrm_r = plain(nrm_g);
  if (any_overlap(hid_r, nrm_r) || any_overlap(hid_r, aux_r) || any_overlap(nrm_r, aux_r) ||
      any_overlap(stats, hid_r) || any_overlap(stats, nrm_r) || any_overlap(stats, aux_r) || any_overlap(stats, ins) ||
      any_overlap(params, hid_r) || any_overlap(params, nrm_r) || any_overlap(params, aux_r) ||
      any_overlap(params, stats))
    return COCO_ERR_ALIAS;

  LayerNormLaunch L;
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
  L.bias = bias;
  L.mean = mean;
  L.rstd = rstd;
  return cuda_status(launch_allreduce_layernorm(L, static_cast<cudaStream_t>(stream)));
}

COCO_EXPORT coco_status coco_allreduce_layernorm(const coco_tensor* partials, const coco_tensor* residual,
                                                 const void* weight, const void* bias, float eps,
                                                 const coco_tensor* hidden, const coco_tensor* normed,
                                                 float* const* scales, float* mean, float* rstd, void* stream) {
  return guarded([&] {
    return allreduce_layernorm_impl(partials, residual, weight, bias, eps, hidden, normed, scales, mean, rstd, stream);
  });
}

COCO_EXPORT size_t coco_allreduce_layernorm_backward_bytes(int64_t rows, int64_t cols) {
  return 2 * coco_allreduce_rmsnorm_backward_bytes(rows, cols);  // the sums of two gradients
}

static coco_status allreduce_layernorm_backward_impl(const coco_tensor* dnormed, const coco_tensor* dhidden,
                                                     const coco_tensor* hidden, const void* weight, const float* mean,
                                                     const float* rstd, const coco_tensor* dx, float* dweight,
                                                     float* dbias, void* workspace, size_t workspace_bytes,
                                                     void* stream) {
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
  if (dbias && (st = check_ptr(dbias, 4)) != COCO_OK) return st;
  std::vector<Range> dw{range_of(dweight, cols * 4)};
  if (dbias) dw.push_back(range_of(dbias, cols * 4));
  if (dbias && overlap(dw[0], dw[1])) return COCO_ERR_ALIAS;
  LayerNormBwdLaunch L;
  std::memset(&L, 0, sizeof(L));
  L.n.dtype = in.dtype;
  L.n.nranks = in.nranks;
  L.n.ngroups = in.ngroups;
  L.n.rows = rows;
  L.n.cols = static_cast<int32_t>(cols);
  L.n.dweight = dweight;
  L.dbias = dbias;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) return cuda_status(launch_layernorm_backward(L, s));  // no rows: the parameters' gradients are zero
  if ((st = check_ptr(weight, 16)) != COCO_OK || (st = check_ptr(mean, 4)) != COCO_OK ||
      (st = check_ptr(rstd, 4)) != COCO_OK || (st = check_ptr(workspace, 16)) != COCO_OK)
    return st;
  const size_t need = coco_allreduce_layernorm_backward_bytes(rows * in.ngroups, cols);
  if (workspace_bytes < need) return COCO_ERR_SHAPE;

  Groups ins_g, outs_g;
  group_ranges(in, &ins_g);
  group_ranges(hid, &ins_g, true);
  if (dhidden) group_ranges(dh, &ins_g, true);
  group_ranges(o, &outs_g);
  if ((st = check_group_alias(outs_g, ins_g, true)) != COCO_OK) return st;
  const std::vector<Range> ins = plain(ins_g), outs = plain(outs_g);
  const std::vector<Range> small_in{range_of(weight, cols * dtype_size(in.dtype)),
                                    range_of(mean, rows * in.ngroups * 4), range_of(rstd, rows * in.ngroups * 4)};
  const std::vector<Range> ws{range_of(workspace, static_cast<int64_t>(need))};
  if (any_overlap(small_in, outs) || any_overlap(dw, outs) || any_overlap(dw, ins) || any_overlap(dw, small_in) ||
      any_overlap(ws, outs) || any_overlap(ws, ins) || any_overlap(ws, small_in) || any_overlap(ws, dw))
    return COCO_ERR_ALIAS;

  for (int i = 0; i < in.nranks * in.ngroups; ++i) L.n.in[i] = dnormed->ptr[i];
  for (int g = 0; g < in.ngroups; ++g) {
    L.n.dhidden[g] = dhidden ? dh.ptr(g, 0) : nullptr;
    L.n.hidden[g] = hid.ptr(g, 0);
    int n = 0;
    for (int r = 0; r < in.nranks; ++r) {
      bool seen = false;
      for (int q = 0; q < n; ++q) seen |= L.n.dx[g * in.nranks + q] == o.ptr(g, r);
      if (!seen) L.n.dx[g * in.nranks + n++] = o.ptr(g, r);
    }
    L.n.ndx[g] = n;
  }
  L.n.weight = weight;
  L.mean = mean;
  L.n.rstd = rstd;
  L.n.partial = static_cast<float*>(workspace);
  return cuda_status(launch_layernorm_backward(L, s));
}

COCO_EXPORT coco_status coco_allreduce_layernorm_backward(const coco_tensor* dnormed, const coco_tensor* dhidden,
                                                          const coco_tensor* hidden, const void* weight,
                                                          const float* mean, const float* rstd, const coco_tensor* dx,
                                                          float* dweight, float* dbias, void* workspace,
                                                          size_t workspace_bytes, void* stream) {
  return guarded([&] {
    return allreduce_layernorm_backward_impl(dnormed, dhidden, hidden, weight, mean, rstd, dx, dweight, dbias,
                                             workspace, workspace_bytes, stream);
  });
}

// ---------------------------------------------------------------- clipping

static coco_status check_plan(const coco_scattered_plan* p) {
  if (!p) return COCO_ERR_NULL;
  if (p->nbuckets < 0 || p->nbuckets > (int64_t(1) << 40) || p->nranks < 1 || p->nranks > COCO_MAX_PTRS)
    return COCO_ERR_SHAPE;
  if (p->dtype < COCO_F32 || p->dtype > COCO_BF16) return COCO_ERR_DTYPE;
  if (p->nbuckets == 0) return COCO_OK;
  if (!p->table) return COCO_ERR_NULL;
  return (reinterpret_cast<uintptr_t>(p->table) & 15) ? COCO_ERR_ALIGN : COCO_OK;
}

COCO_EXPORT size_t coco_scattered_clip_bytes(void) { return kClipMaxParts * sizeof(double); }

static coco_status clip_impl(const coco_scattered_plan* plan, int mode, float alpha, float max_norm,
                             const coco_scattered_plan* out, float* norm, void* workspace, size_t workspace_bytes,
                             void* stream) {
  coco_status st;
  if ((st = check_plan(plan)) != COCO_OK) return st;
  if (out && (st = check_plan(out)) != COCO_OK) return st;
  if (out && out->nbuckets != plan->nbuckets) return COCO_ERR_SHAPE;
  if (out && mode == CLIP_LOCAL && out->nranks != plan->nranks) return COCO_ERR_SHAPE;
  // one table for both: in place, as without `out`, and no other type or number of ranks than its own
  if (out && plan->nbuckets > 0 && out->table == plan->table &&
      (out->dtype != plan->dtype || out->nranks != plan->nranks))
    return COCO_ERR_SHAPE;
  if (!(max_norm >= 0.0f) || !(alpha == alpha)) return COCO_ERR_VALUE;  // (the first also rejects NaN)
  if ((st = check_ptr(norm, 4)) != COCO_OK || (st = check_ptr(workspace, 16)) != COCO_OK) return st;
  if (workspace_bytes < coco_scattered_clip_bytes()) return COCO_ERR_SHAPE;
  const std::vector<Range> n{range_of(norm, 4)}, ws{range_of(workspace, coco_scattered_clip_bytes())};
  std::vector<Range> tables;
  for (const coco_scattered_plan* p : {plan, out})
    if (p && p->nbuckets > 0) tables.push_back(range_of(p->table, 64 + 12 * p->nbuckets * p->nranks));
  if (any_overlap(n, ws) || any_overlap(n, tables) || any_overlap(ws, tables)) return COCO_ERR_ALIAS;
  if (!out) out = plan;
  ClipLaunch L;
  L.table = plan->table;
  L.out_table = out->table;
  L.nbuckets = plan->nbuckets;
  L.mode = mode;
  L.nranks = plan->nranks;
  L.out_nranks = out->nranks;
  L.dtype = plan->dtype;
  L.out_dtype = out->dtype;
  L.alpha = alpha;
  L.max_norm = max_norm;
  L.norm = norm;
  L.parts = static_cast<double*>(workspace);
  return cuda_status(launch_scattered_clip(L, static_cast<cudaStream_t>(stream)));
}

COCO_EXPORT coco_status coco_scattered_clip(const coco_scattered_plan* plan, int32_t layout, float max_norm,
                                            const coco_scattered_plan* out, float* norm, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  if (layout != COCO_LOCAL && layout != COCO_REPLICATED) return COCO_ERR_LAYOUT;
  return guarded([&] {
    return clip_impl(plan, layout == COCO_LOCAL ? CLIP_LOCAL : CLIP_REPLICATED, 1.0f, max_norm, out, norm, workspace,
                     workspace_bytes, stream);
  });
}

COCO_EXPORT coco_status coco_scattered_allreduce_clip(const coco_scattered_plan* plan, float alpha, float max_norm,
                                                      const coco_scattered_plan* out, float* norm, void* workspace,
                                                      size_t workspace_bytes, void* stream) {
  return guarded([&] {
    return clip_impl(plan, CLIP_SUM, alpha, max_norm, out, norm, workspace, workspace_bytes, stream);
  });
}
