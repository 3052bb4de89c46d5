// experts.cpp -- the entry points of experts and adapters beside the product
// (include/gemm_tune.h): argument checks, workspaces and launches of the
// experts' choice, the layer of gated experts and the requests' adapters.
#include <math.h>

#include <algorithm>

#include "operators.h"

namespace gt {
namespace {

constexpr int64_t kRouteMaxE = 1024, kMostSlots = 64, kMostExperts = 4096, kMostRank = 256;

gt_status route(const gt_route_desc* d) {
  if (!d) return invalid("desc is NULL");
  RouteArgs a;
  if (d->M < 0 || d->E < 0 || d->topk < 0) return invalid("negative dimension");
  GT_CHECK(float_type(d->dtype, -1, "logits", &a.dtype));
  if (d->score < GT_SCORE_SOFTMAX || d->score > GT_SCORE_SIGMOID) return invalid("unknown gt_score");
  if (d->normalise != 0 && d->normalise != 1) return invalid("normalise is 0 or 1");
  if (!isfinite(d->scale)) return invalid("scale must be finite");
  if (d->E > kRouteMaxE) return refuse(GT_ERR_UNSUPPORTED, "gt_route takes at most 1024 experts");
  if (d->topk > kMostSlots) return refuse(GT_ERR_UNSUPPORTED, "gt_route chooses at most 64 experts");
  if (d->topk < 1 || d->topk > d->E) return invalid("topk must be from 1 to the number of experts");
  GT_CHECK(leading(d->ldl, d->E, "logits", &a.ldl));
  GT_CHECK(leading(d->ldi, d->topk, "index", &a.ldi));
  GT_CHECK(leading(d->ldw, d->topk, "weight", &a.ldw));
  if (d->M == 0) return GT_OK;
  GT_CHECK(operand(d->logits, true, d->M, a.ldl, elem_bytes(a.dtype), "logits"));
  GT_CHECK(operand(d->index, true, d->M, a.ldi, 4, "index"));
  GT_CHECK(operand(d->weight, true, d->M, a.ldw, 4, "weight"));
  a.logits = d->logits;
  a.index = d->index;
  a.weight = d->weight;
  a.M = d->M;
  a.E = (int)d->E;
  a.topk = (int)d->topk;
  a.sigmoid = d->score == GT_SCORE_SIGMOID;
  a.normalise = d->normalise != 0;
  a.scale = d->scale;
  a.stream = stream_of(d->stream);
  DeviceState* dev = nullptr;
  GT_CHECK(current_device(&dev));
  if (dev->fake) return GT_OK;
  return launched(launch_route(a), "gt_route");
}

// E matrices of N rows, each of `row` elements (bytes for 4-bit codes), `unit`
// bytes an element.  Their strides; the pointers are looked at by `there`.
gt_status matrices(const void* p, int64_t E, int64_t N, int64_t row, int unit, int64_t ld, int64_t stride, const char* what,
                   ExpertWeights* w) {
  GT_CHECK(leading(ld, row, what, &ld));
  if (ld > INT64_MAX / 16 / std::max<int64_t>(N, 1)) return invalid(std::string(what) + " spans more than 64-bit offsets");
  // matrices may lie inside each other's rows (experts as the middle dimension), rows of one may not overlap
  if (stride <= 0) stride = std::max<int64_t>(N, 1) * ld;
  if (stride < row) return invalid(std::string(what) + ": matrices overlap");
  if (E > 0 && N > 0 && row > 0) {
    GT_CHECK(spans(N, ld, what));
    GT_CHECK(spans(E, stride, what));
  }
  w->p = static_cast<const char*>(p);
  w->scales = nullptr;
  w->ld = ld * unit;
  w->stride = stride * unit;
  w->s_lde = w->s_ldn = w->s_ldg = 0;
  return GT_OK;
}

gt_status matrix_scales(const void* p, int64_t E, int64_t N, int64_t groups, int64_t lde, int64_t ldn, int64_t ldg,
                        const char* what, ExpertWeights* w) {
  w->scales = p;
  w->s_ldn = ldn > 0 ? ldn : std::max<int64_t>(groups, 1);
  w->s_ldg = ldg > 0 ? ldg : 1;
  if (w->s_ldn > INT64_MAX / 16 / std::max<int64_t>(N, 1) || w->s_ldg > INT64_MAX / 16 / std::max<int64_t>(groups, 1))
    return invalid(std::string(what) + " spans more than 64-bit offsets");
  // one matrix after another, whether its rows or its groups lie further apart
  w->s_lde = lde > 0 ? lde : std::max(N * w->s_ldn, groups * w->s_ldg);
  if (E == 0 || N == 0 || groups == 0) return GT_OK;
  GT_CHECK(spans(N, w->s_ldn, what));
  GT_CHECK(spans(groups, w->s_ldg, what));
  return spans(E, w->s_lde, what);
}
// A pointer to weights or scales that there are (`any`), `unit` bytes an element.
gt_status there(const void* p, bool any, int unit, const char* what) { return any ? operand(p, true, 0, 0, unit, what) : GT_OK; }

// A workspace of the caller's or of the stream's, and what is launched on it.
template <class A, class L>
gt_status on_workspace(DeviceState& dev, A& a, size_t need, void* own, int64_t own_bytes, L launch) {
  if (own || own_bytes > 0) {
    if (!own) return invalid("workspace_bytes without a workspace");
    if ((uintptr_t)own % 16) return invalid("workspace is not aligned to 16 bytes");
    if (own_bytes < 0 || (uint64_t)own_bytes < need) return invalid("the workspace is too small");
    if (dev.fake) return GT_OK;
    a.ws = static_cast<char*>(own);
    return launch(a);
  }
  if (dev.fake) return GT_OK;
  void* ws = nullptr;
  std::mutex* mu = nullptr;
  GT_CHECK(operator_workspace(dev, a.stream, kCounterRegion + need, &ws, &mu));
  a.ws = static_cast<char*>(ws) + kCounterRegion;
  std::lock_guard<std::mutex> g(*mu);
  return launch(a);
}

// Workspace of the largest of a call's ranges: few rows may take more than
// many (their sums are cut into more slices), so the last one counts too.
template <class A, class B>
size_t most_bytes(const A& a, int64_t most, B bytes) {
  const size_t whole = bytes(a, std::min(a.M, most));
  return a.M > most && a.M % most ? std::max(whole, bytes(a, a.M % most)) : whole;
}

// The descriptor's sizes, types and the weights' strides.
gt_status moe_shape(const gt_moe_desc* d, MoeArgs* a) {
  if (d->M < 0 || d->K < 0 || d->H < 0 || d->E < 0 || d->topk < 0) return invalid("negative dimension");
  if (d->x_dtype < 0 || d->x_dtype > DT_E4M3) return invalid("unknown type of x");
  if (d->x_dtype != DT_F16 && d->x_dtype != DT_BF16) return refuse(GT_ERR_UNSUPPORTED, "rows of gt_moe are f16 or bf16");
  a->x_dtype = d->x_dtype;
  GT_CHECK(float_type(d->out_dtype, a->x_dtype, "y", &a->out_dtype));
  if (d->format != GT_WEIGHTS_16BIT && d->format != GT_W4_INT4 && d->format != GT_W4_E2M1)
    return invalid("unknown format of the weights");
  a->format = d->format;
  a->scale_dtype = DT_F32;
  a->group_lg = 5;
  if (d->format != GT_WEIGHTS_16BIT) {
    if (d->group != 32 && d->group != 64 && d->group != 128) return invalid("group must be 32, 64 or 128");
    a->group_lg = d->group == 32 ? 5 : (d->group == 64 ? 6 : 7);
    GT_CHECK(float_type(d->scale_dtype, -1, "scales", &a->scale_dtype));
  }
  if (d->activation != GT_ACT_SILU && d->activation != GT_ACT_GELU) return invalid("unknown gt_activation");
  a->activation = d->activation;
  if (d->E > kMostExperts) return refuse(GT_ERR_UNSUPPORTED, "gt_moe takes at most 4096 experts");
  if (d->topk > kMostSlots) return refuse(GT_ERR_UNSUPPORTED, "gt_moe takes at most 64 experts a token");
  if (d->H > (INT64_C(1) << 24) || d->K > (INT64_C(1) << 24)) return refuse(GT_ERR_UNSUPPORTED, "gt_moe takes K and H up to 2^24");
  a->M = d->M;
  a->K = d->K;
  a->H = d->H;
  a->E = (int)d->E;
  a->topk = (int)d->topk;
  a->wide = false;
  const bool k4 = a->format != GT_WEIGHTS_16BIT;
  auto row = [&](int64_t n) { return k4 ? n / 2 + n % 2 : n; };
  GT_CHECK(matrices(d->gate_up, a->E, 2 * a->H, row(a->K), k4 ? 1 : 2, d->gate_up_ld, d->gate_up_stride, "gate_up", &a->gate_up));
  GT_CHECK(matrices(d->down, a->E, a->K, row(a->H), k4 ? 1 : 2, d->down_ld, d->down_stride, "down", &a->down));
  if (k4) {
    const int64_t g = INT64_C(1) << a->group_lg;
    GT_CHECK(matrix_scales(d->gate_up_scales, a->E, 2 * a->H, (a->K + g - 1) / g, d->gate_up_scale_lde, d->gate_up_scale_ldn,
                           d->gate_up_scale_ldg, "gate_up_scales", &a->gate_up));
    GT_CHECK(matrix_scales(d->down_scales, a->E, a->K, (a->H + g - 1) / g, d->down_scale_lde, d->down_scale_ldn, d->down_scale_ldg,
                           "down_scales", &a->down));
  }
  return GT_OK;
}
bool moe_empty(const MoeArgs& a) { return a.H == 0 || a.E == 0 || a.topk == 0; }

gt_status moe(const gt_moe_desc* d) {
  if (!d) return invalid("desc is NULL");
  MoeArgs a;
  GT_CHECK(moe_shape(d, &a));
  GT_CHECK(leading(d->ldx, a.K, "x", &a.ldx));
  GT_CHECK(leading(d->ldi, a.topk, "index", &a.ldi));
  GT_CHECK(leading(d->ldw, a.topk, "weight", &a.ldw));
  GT_CHECK(leading(d->ldb, a.K, "base", &a.ldb));
  GT_CHECK(leading(d->ldy, a.K, "y", &a.ldy));
  const bool any = a.E > 0 && a.H > 0 && a.K > 0, k4 = a.format != GT_WEIGHTS_16BIT;
  GT_CHECK(there(d->gate_up, any, k4 ? 1 : 2, "gate_up"));
  GT_CHECK(there(d->down, any, k4 ? 1 : 2, "down"));
  GT_CHECK(there(d->gate_up_scales, any && k4, elem_bytes(a.scale_dtype), "gate_up_scales"));
  GT_CHECK(there(d->down_scales, any && k4, elem_bytes(a.scale_dtype), "down_scales"));
  if (a.M == 0 || a.K == 0) return GT_OK;
  const bool empty = moe_empty(a);
  GT_CHECK(operand(d->x, !empty, a.M, a.ldx, 2, "x"));
  GT_CHECK(operand(d->index, !empty, a.M, a.ldi, 4, "index"));
  GT_CHECK(operand(d->weight, !empty, a.M, a.ldw, 4, "weight"));
  GT_CHECK(operand(d->base, false, a.M, a.ldb, elem_bytes(a.out_dtype), "base"));
  GT_CHECK(operand(d->y, true, a.M, a.ldy, elem_bytes(a.out_dtype), "y"));
  if (d->base == d->y && a.ldb != a.ldy) return invalid("base is y with another leading dimension");
  // a range of tokens reads its rows of x before it writes its rows of y, which then have to be the same ones
  if (!empty && d->x == d->y && (a.ldx != a.ldy || a.x_dtype != a.out_dtype)) return invalid("x is y with another type or leading dimension");
  a.x = d->x;
  a.index = d->index;
  a.weight = d->weight;
  a.base = d->base;
  a.y = d->y;
  a.ws = nullptr;
  a.stream = stream_of(d->stream);
  DeviceState* dev = nullptr;
  GT_CHECK(current_device(&dev));
  a.cus = dev->cus;
  if (empty) {
    if (dev->fake) return GT_OK;
    return launched(launch_copy_rows(a.base, a.y, a.M, a.K, a.ldb, a.ldy, a.out_dtype, a.stream), "gt_moe");
  }
  a.wide = moe_wide(a);
  const int64_t most = moe_range(a);
  return on_workspace(*dev, a, most_bytes(a, most, moe_workspace_bytes), d->workspace, d->workspace_bytes, [&](MoeArgs& all) {
    for (int64_t m = 0; m < all.M; m += most) {
      MoeArgs r = all;
      r.M = std::min(most, all.M - m);
      r.x = static_cast<const char*>(all.x) + m * all.ldx * 2;
      r.index = all.index + m * all.ldi;
      r.weight = all.weight + m * all.ldw;
      if (all.base) r.base = static_cast<const char*>(all.base) + m * all.ldb * elem_bytes(all.out_dtype);
      r.y = static_cast<char*>(all.y) + m * all.ldy * elem_bytes(all.out_dtype);
      GT_CHECK(launched(launch_moe(r), "gt_moe"));
    }
    return GT_OK;
  });
}

gt_status moe_workspace(const gt_moe_desc* d, int64_t* bytes) {
  if (!d || !bytes) return invalid("desc or bytes is NULL");
  MoeArgs a;
  GT_CHECK(moe_shape(d, &a));
  *bytes = 0;
  if (a.M == 0 || a.K == 0 || moe_empty(a)) return GT_OK;
  DeviceState* dev = nullptr;
  GT_CHECK(current_device(&dev));
  a.cus = dev->cus;
  a.wide = moe_wide(a);
  *bytes = (int64_t)most_bytes(a, moe_range(a), moe_workspace_bytes);
  return GT_OK;
}

gt_status lora_shape(const gt_lora_desc* d, LoraArgs* a) {
  if (d->M < 0 || d->K < 0 || d->N < 0 || d->adapters < 0 || d->rank < 0) return invalid("negative dimension");
  if (d->x_dtype < 0 || d->x_dtype > DT_E4M3) return invalid("unknown type of x");
  if (d->x_dtype != DT_F16 && d->x_dtype != DT_BF16) return refuse(GT_ERR_UNSUPPORTED, "rows of gt_lora are f16 or bf16");
  a->x_dtype = d->x_dtype;
  GT_CHECK(float_type(d->out_dtype, a->x_dtype, "y", &a->out_dtype));
  if (d->adapters > kMostExperts) return refuse(GT_ERR_UNSUPPORTED, "gt_lora takes at most 4096 adapters");
  if (d->rank > kMostRank) return refuse(GT_ERR_UNSUPPORTED, "gt_lora takes ranks up to 256");
  if (d->K > (INT64_C(1) << 24) || d->N > (INT64_C(1) << 24)) return refuse(GT_ERR_UNSUPPORTED, "gt_lora takes K and N up to 2^24");
  a->M = d->M;
  a->K = d->K;
  a->N = d->N;
  a->adapters = (int)d->adapters;
  a->rank = (int)d->rank;
  return GT_OK;
}
bool lora_empty(const LoraArgs& a) { return a.K == 0 || a.adapters == 0 || a.rank == 0; }

gt_status lora(const gt_lora_desc* d) {
  if (!d) return invalid("desc is NULL");
  LoraArgs a;
  GT_CHECK(lora_shape(d, &a));
  GT_CHECK(leading(d->ldx, a.K, "x", &a.ldx));
  GT_CHECK(leading(d->ldb, a.N, "base", &a.ldb));
  GT_CHECK(leading(d->ldy, a.N, "y", &a.ldy));
  GT_CHECK(matrices(d->a, a.adapters, a.rank, a.K, 2, d->a_ld, d->a_stride, "a", &a.a));
  GT_CHECK(matrices(d->b, a.adapters, a.N, a.rank, 2, d->b_ld, d->b_stride, "b", &a.b));
  GT_CHECK(there(d->a, a.adapters > 0 && a.rank > 0 && a.K > 0, 2, "a"));
  GT_CHECK(there(d->b, a.adapters > 0 && a.rank > 0 && a.N > 0, 2, "b"));
  if (a.M == 0 || a.N == 0) return GT_OK;
  const bool empty = lora_empty(a);
  GT_CHECK(operand(d->x, !empty, a.M, a.ldx, 2, "x"));
  GT_CHECK(operand(d->index, !empty, a.M, 1, 4, "index"));
  GT_CHECK(operand(d->scale, false, a.adapters, 1, 4, "scale"));
  GT_CHECK(operand(d->base, false, a.M, a.ldb, elem_bytes(a.out_dtype), "base"));
  GT_CHECK(operand(d->y, true, a.M, a.ldy, elem_bytes(a.out_dtype), "y"));
  if (d->base == d->y && a.ldb != a.ldy) return invalid("base is y with another leading dimension");
  if (!empty && d->x == d->y) return invalid("y is x");
  a.x = d->x;
  a.index = d->index;
  a.scale = d->scale;
  a.base = d->base;
  a.y = d->y;
  a.ws = nullptr;
  a.stream = stream_of(d->stream);
  DeviceState* dev = nullptr;
  GT_CHECK(current_device(&dev));
  a.cus = dev->cus;
  if (empty) {
    if (dev->fake) return GT_OK;
    return launched(launch_copy_rows(a.base, a.y, a.M, a.N, a.ldb, a.ldy, a.out_dtype, a.stream), "gt_lora");
  }
  const int64_t most = lora_range(a);
  return on_workspace(*dev, a, most_bytes(a, most, lora_workspace_bytes), d->workspace, d->workspace_bytes, [&](LoraArgs& all) {
    for (int64_t m = 0; m < all.M; m += most) {
      LoraArgs r = all;
      r.M = std::min(most, all.M - m);
      r.x = static_cast<const char*>(all.x) + m * all.ldx * 2;
      r.index = all.index + m;
      if (all.base) r.base = static_cast<const char*>(all.base) + m * all.ldb * elem_bytes(all.out_dtype);
      r.y = static_cast<char*>(all.y) + m * all.ldy * elem_bytes(all.out_dtype);
      GT_CHECK(launched(launch_lora(r), "gt_lora"));
    }
    return GT_OK;
  });
}

gt_status lora_workspace(const gt_lora_desc* d, int64_t* bytes) {
  if (!d || !bytes) return invalid("desc or bytes is NULL");
  LoraArgs a;
  GT_CHECK(lora_shape(d, &a));
  *bytes = 0;
  if (a.M == 0 || a.N == 0 || lora_empty(a)) return GT_OK;
  DeviceState* dev = nullptr;
  GT_CHECK(current_device(&dev));
  a.cus = dev->cus;
  *bytes = (int64_t)most_bytes(a, lora_range(a), lora_workspace_bytes);
  return GT_OK;
}

}  // namespace
}  // namespace gt

using namespace gt;

extern "C" {

gt_status gt_route(const gt_route_desc* d) { return guarded(route, d); }
gt_status gt_moe(const gt_moe_desc* d) { return guarded(moe, d); }
gt_status gt_lora(const gt_lora_desc* d) { return guarded(lora, d); }
gt_status gt_moe_workspace(const gt_moe_desc* d, int64_t* bytes) {
  return guarded([&](const gt_moe_desc* p) { return moe_workspace(p, bytes); }, d);
}
gt_status gt_lora_workspace(const gt_lora_desc* d, int64_t* bytes) {
  return guarded([&](const gt_lora_desc* p) { return lora_workspace(p, bytes); }, d);
}

}  // extern "C"
