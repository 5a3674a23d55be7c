// Host side of sla_attend and sla_attend_backward: argument checks, the split of the work over
// the SMs, workspace layout, TMA descriptors and kernel launches.
#include <climits>
#include <cmath>

#include "attend.cuh"
#include "attend_backward.cuh"
#include "host.cuh"

namespace {

using namespace sla_host;
using sla::AttendArgs;
using sla::AttendBwdArgs;
using sla::AttendFwdArgs;
using sla::AttendRowsArgs;
using sla::AttendSumArgs;
using sla::kTile;
using sla::RowOut;

// SMs that a launch should fill: the split of the work, and so the workspace's size, must not
// depend on which device is current.
constexpr int kSms = 148;

struct AttendPlan {
  sla_attend_problem p;
  int pad;                                      // Nq rounded up to whole tiles
  long long q_rows, k_rows;                     // B H Nq, B Hk Nk
  int fwd_units, dkv_units, dq_units;           // with their splits
  int fwd_splits, dkv_splits, dq_splits;
};

struct AttendSpace {
  uint32_t* err;
  float *part, *part_lse2;              // forward
  float *nlse, *ndelta, *dq, *dkv;      // backward
  size_t bytes;
};

// Work items of a launch of `units` independent units with `tiles` steps each: fewer units
// than SMs are split over the steps, at least two of them to a part.
int splits_for(long long units, long long tiles) {
  if (units >= kSms) return 1;
  const long long by_sms = kSms / units, by_work = (tiles + 1) / 2;
  return static_cast<int>(by_sms < by_work ? by_sms : by_work < 1 ? 1 : by_work);
}

sla_status make_plan(const sla_attend_problem* p, AttendPlan* w) {
  if (!p) return fail(SLA_ERR_INVALID_ARG, "problem is NULL");
  if (p->B < 1 || p->H < 1 || p->Hk < 1 || p->Nq < 1 || p->Nk < 1)
    return fail(SLA_ERR_INVALID_ARG, "B, H, Hk, Nq and Nk must be >= 1");
  if (p->H % p->Hk) return fail(SLA_ERR_INVALID_ARG, "H=%d is not a multiple of Hk=%d", p->H, p->Hk);
  if (p->D != 64 && p->D != 128) return fail(SLA_ERR_UNSUPPORTED, "D=%d not supported (64 or 128)", p->D);
  if (p->causal != 0 && p->causal != 1) return fail(SLA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!std::isfinite(p->scale) || !(p->scale > 0.f)) return fail(SLA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (p->Nq > (1 << 24) || p->Nk > (1 << 24)) return fail(SLA_ERR_UNSUPPORTED, "Nq, Nk must be at most 2^24");
  const long long BH = static_cast<long long>(p->B) * p->H, BHk = static_cast<long long>(p->B) * p->Hk;
  const long long qt = (p->Nq + kTile - 1) / kTile, kt = (p->Nk + kTile - 1) / kTile, pairs = (qt + 1) / 2;
  if (BH * qt >= (1ll << 28) || BHk * kt >= (1ll << 28)) return fail(SLA_ERR_UNSUPPORTED, "B*H*N too large");
  const long long group = p->H / p->Hk;
  if (group * qt >= (1ll << 30)) return fail(SLA_ERR_UNSUPPORTED, "H / Hk * Nq too large");
  w->p = *p;
  w->pad = static_cast<int>(qt * kTile);
  w->q_rows = BH * p->Nq;
  w->k_rows = BHk * p->Nk;
  w->fwd_splits = splits_for(BH * pairs, kt);
  w->dkv_splits = splits_for(BHk * kt, group * qt);
  w->dq_splits = splits_for(BH * qt, kt);
  w->fwd_units = static_cast<int>(BH * pairs) * w->fwd_splits;
  w->dkv_units = static_cast<int>(BHk * kt) * w->dkv_splits;
  w->dq_units = static_cast<int>(BH * qt) * w->dq_splits;
  return SLA_OK;
}

AttendSpace layout(const AttendPlan& w, uint8_t* base, bool bwd) {
  AttendSpace s{};
  size_t off = 0;
  auto take = [&](size_t floats) {
    float* p = base ? reinterpret_cast<float*>(base + off) : nullptr;
    off += align256(floats * sizeof(float));
    return p;
  };
  s.err = reinterpret_cast<uint32_t*>(take(64));
  const size_t D = w.p.D;
  if (!bwd) {
    if (w.fwd_splits > 1) {
      s.part = take(w.fwd_splits * static_cast<size_t>(w.q_rows) * D);
      s.part_lse2 = take(w.fwd_splits * static_cast<size_t>(w.q_rows));
    }
  } else {
    const size_t stats = static_cast<size_t>(w.p.B) * w.p.H * w.pad;
    s.nlse = take(stats);
    s.ndelta = take(stats);
    if (w.dq_splits > 1) s.dq = take(w.dq_splits * static_cast<size_t>(w.q_rows) * D);
    if (w.dkv_splits > 1) s.dkv = take(2 * w.dkv_splits * static_cast<size_t>(w.k_rows) * D);
  }
  s.bytes = off;
  return s;
}

sla_status check_space(const AttendPlan& w, void* ws, size_t ws_bytes, bool bwd, AttendSpace* s) {
  if (!ws) return fail(SLA_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(SLA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  *s = layout(w, static_cast<uint8_t*>(ws), bwd);
  if (ws_bytes < s->bytes)
    return fail(SLA_ERR_WORKSPACE, "workspace too small: %zu bytes given, %zu needed", ws_bytes, s->bytes);
  return SLA_OK;
}

// A [B, heads, N, D] bf16 operand: rows of 16 bytes, ascending strides where the extent is
// above 1 (a tensor map has no stride of zero).
sla_status check_operand(const char* name, const sla_tensor* t, int B, int heads, int N) {
  if (!t || !aligned16(t->ptr)) return fail(SLA_ERR_INVALID_ARG, "%s must be non-NULL and 16-byte aligned", name);
  const struct {
    int extent;
    int64_t stride;
  } dims[3] = {{B, t->stride_b}, {heads, t->stride_h}, {N, t->stride_n}};
  for (const auto& d : dims) {
    if (d.extent <= 1) continue;
    if (d.stride < 1 || d.stride % 8)
      return fail(SLA_ERR_INVALID_ARG, "%s's strides must be positive multiples of 16 bytes", name);
    if (d.stride >= (1ll << 38)) return fail(SLA_ERR_UNSUPPORTED, "%s's strides must be below 2^38 elements", name);
  }
  return SLA_OK;
}

// Tiles of 128 rows x 64 channels of a checked operand.
sla_status operand_map(CUtensorMap* m, const sla_tensor* t, int B, int heads, int N, int D) {
  const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(N), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(B)};
  const uint64_t strides[3] = {static_cast<uint64_t>(N > 1 ? t->stride_n : D),
                               static_cast<uint64_t>(heads > 1 ? t->stride_h : D),
                               static_cast<uint64_t>(B > 1 ? t->stride_b : D)};
  const uint32_t box[4] = {64, kTile, 1, 1};
  return make_map(m, t->ptr, 4, dims, strides, box);
}

RowOut row_out(const sla_tensor* t, int B, int heads, int N) {
  RowOut o{static_cast<__nv_bfloat16*>(t->ptr), B > 1 ? t->stride_b : 0, heads > 1 ? t->stride_h : 0,
           N > 1 ? t->stride_n : 0, 0};
  o.wide = reinterpret_cast<uintptr_t>(t->ptr) % 32 == 0 && o.sb % 16 == 0 && o.sh % 16 == 0 && o.sn % 16 == 0;
  return o;
}

AttendArgs common_args(const AttendPlan& w, const int32_t* lens, uint32_t* err, int splits, int units) {
  AttendArgs a{};
  a.B = w.p.B;
  a.H = w.p.H;
  a.Hk = w.p.Hk;
  a.G = w.p.H / w.p.Hk;
  a.Nq = w.p.Nq;
  a.Nk = w.p.Nk;
  a.causal = w.p.causal;
  a.splits = splits;
  a.units = units;
  a.scale = w.p.scale;
  a.scale_log2 = w.p.scale * 1.4426950408889634f;
  a.lens = lens;
  a.err = err;
  return a;
}

int persistent_grid(int units) {
  const int n = sm_count();
  return units < n ? units : n;
}

struct Maps {
  CUtensorMap q, k, v, g;
};

sla_status input_maps(Maps* m, const AttendPlan& w, const sla_tensor* q, const sla_tensor* k, const sla_tensor* v,
                      const sla_tensor* g) {
  SLA_TRY(operand_map(&m->q, q, w.p.B, w.p.H, w.p.Nq, w.p.D));
  SLA_TRY(operand_map(&m->k, k, w.p.B, w.p.Hk, w.p.Nk, w.p.D));
  SLA_TRY(operand_map(&m->v, v, w.p.B, w.p.Hk, w.p.Nk, w.p.D));
  if (g) SLA_TRY(operand_map(&m->g, g, w.p.B, w.p.H, w.p.Nq, w.p.D));
  return SLA_OK;
}

template <int D>
sla_status launch_forward(const AttendPlan& w, const Maps& m, const AttendFwdArgs& f, cudaStream_t st) {
  constexpr int smem = sla::AttendSmem<D>::total();
  SLA_TRY(allow_smem(sla::attend_kernel<D>, smem));
  SLA_TRY(launch_dependent(sla::attend_kernel<D>, dim3(persistent_grid(w.fwd_units)), dim3(320), smem, st,
                           "attend_kernel", m.q, m.k, m.v, f));
  if (w.fwd_splits > 1)
    SLA_TRY(launch_dependent(sla::attend_join_kernel<D>, dim3(static_cast<unsigned>((w.q_rows + 7) / 8)), dim3(256), 0,
                             st, "attend_join_kernel", f));
  return SLA_OK;
}

template <int D>
sla_status launch_sum(const float* part, int splits, int H, int N, long long rows, const RowOut& out, cudaStream_t st) {
  const AttendSumArgs a{part, splits, H, N, rows, out};
  constexpr int per = 256 / (D / 8);
  return launch_dependent(sla::attend_sum_kernel<D>, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(256), 0,
                          st, "attend_sum_kernel", a);
}

template <int D>
sla_status launch_backward(const AttendPlan& w, const Maps& m, const AttendRowsArgs& r, AttendBwdArgs f,
                           const AttendSpace& s, const int32_t* lens, cudaStream_t st) {
  constexpr int per = 256 / (D / 8);
  SLA_TRY(launch_dependent(sla::attend_rows_kernel<D>, dim3(static_cast<unsigned>((r.rows + per - 1) / per)), dim3(256),
                           0, st, "attend_rows_kernel", r));
  f.p = common_args(w, lens, s.err, w.dkv_splits, w.dkv_units);
  f.part = s.dkv;
  constexpr int smem_kv = sla::AttendDkvSmem<D>::total();
  SLA_TRY(allow_smem(sla::attend_dkv_kernel<D>, smem_kv));
  SLA_TRY(launch_dependent(sla::attend_dkv_kernel<D>, dim3(persistent_grid(w.dkv_units)), dim3(320), smem_kv, st,
                           "attend_dkv_kernel", m.q, m.k, m.v, m.g, f));
  f.p = common_args(w, lens, s.err, w.dq_splits, w.dq_units);
  f.part = s.dq;
  constexpr int smem_q = sla::AttendDqSmem<D>::total();
  SLA_TRY(allow_smem(sla::attend_dq_kernel<D>, smem_q));
  SLA_TRY(launch_dependent(sla::attend_dq_kernel<D>, dim3(persistent_grid(w.dq_units)), dim3(320), smem_q, st,
                           "attend_dq_kernel", m.q, m.k, m.v, m.g, f));
  if (w.dkv_splits > 1) {
    SLA_TRY(launch_sum<D>(s.dkv, w.dkv_splits, w.p.Hk, w.p.Nk, w.k_rows, f.dk, st));
    SLA_TRY(launch_sum<D>(s.dkv + w.dkv_splits * w.k_rows * D, w.dkv_splits, w.p.Hk, w.p.Nk, w.k_rows, f.dv, st));
  }
  if (w.dq_splits > 1) SLA_TRY(launch_sum<D>(s.dq, w.dq_splits, w.p.H, w.p.Nq, w.q_rows, f.dq, st));
  return SLA_OK;
}

sla_status check_lens(const int32_t* lens) {
  if (reinterpret_cast<uintptr_t>(lens) % 4) return fail(SLA_ERR_INVALID_ARG, "kv_lens must be 4-byte aligned");
  return SLA_OK;
}

}  // namespace

extern "C" {

size_t sla_workspace_size_attend(const sla_attend_problem* p) {
  AttendPlan w;
  if (make_plan(p, &w) != SLA_OK) return 0;
  return layout(w, nullptr, false).bytes;
}

size_t sla_workspace_size_attend_backward(const sla_attend_problem* p) {
  AttendPlan w;
  if (make_plan(p, &w) != SLA_OK) return 0;
  return layout(w, nullptr, true).bytes;
}

sla_status sla_attend(const sla_attend_problem* p, const sla_tensor* q, const sla_tensor* k, const sla_tensor* v,
                      const int32_t* kv_lens, const sla_tensor* out, float* lse, void* ws, size_t ws_bytes,
                      void* stream) {
  AttendPlan w;
  SLA_TRY(make_plan(p, &w));
  SLA_TRY(check_operand("q", q, p->B, p->H, p->Nq));
  SLA_TRY(check_operand("k", k, p->B, p->Hk, p->Nk));
  SLA_TRY(check_operand("v", v, p->B, p->Hk, p->Nk));
  SLA_TRY(check_operand("out", out, p->B, p->H, p->Nq));
  SLA_TRY(check_lens(kv_lens));
  if (!lse || reinterpret_cast<uintptr_t>(lse) % 4) return fail(SLA_ERR_INVALID_ARG, "lse must be non-NULL and 4-byte aligned");
  AttendSpace s;
  SLA_TRY(check_space(w, ws, ws_bytes, false, &s));
  Maps m;
  SLA_TRY(input_maps(&m, w, q, k, v, nullptr));
  AttendFwdArgs f{};
  f.p = common_args(w, kv_lens, s.err, w.fwd_splits, w.fwd_units);
  f.out = row_out(out, p->B, p->H, p->Nq);
  f.lse = lse;
  f.part = s.part;
  f.part_lse2 = s.part_lse2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return p->D == 128 ? launch_forward<128>(w, m, f, st) : launch_forward<64>(w, m, f, st);
}

sla_status sla_attend_backward(const sla_attend_problem* p, const sla_tensor* q, const sla_tensor* k,
                               const sla_tensor* v, const sla_tensor* out, const float* lse, const sla_tensor* dO,
                               const int32_t* kv_lens, const sla_tensor* dq, const sla_tensor* dk,
                               const sla_tensor* dv, void* ws, size_t ws_bytes, void* stream) {
  AttendPlan w;
  SLA_TRY(make_plan(p, &w));
  SLA_TRY(check_operand("q", q, p->B, p->H, p->Nq));
  SLA_TRY(check_operand("k", k, p->B, p->Hk, p->Nk));
  SLA_TRY(check_operand("v", v, p->B, p->Hk, p->Nk));
  SLA_TRY(check_operand("out", out, p->B, p->H, p->Nq));
  SLA_TRY(check_operand("dO", dO, p->B, p->H, p->Nq));
  SLA_TRY(check_operand("dq", dq, p->B, p->H, p->Nq));
  SLA_TRY(check_operand("dk", dk, p->B, p->Hk, p->Nk));
  SLA_TRY(check_operand("dv", dv, p->B, p->Hk, p->Nk));
  SLA_TRY(check_lens(kv_lens));
  if (!lse || reinterpret_cast<uintptr_t>(lse) % 4) return fail(SLA_ERR_INVALID_ARG, "lse must be non-NULL and 4-byte aligned");
  AttendSpace s;
  SLA_TRY(check_space(w, ws, ws_bytes, true, &s));
  Maps m;
  SLA_TRY(input_maps(&m, w, q, k, v, dO));
  const RowOut o = row_out(out, p->B, p->H, p->Nq), g = row_out(dO, p->B, p->H, p->Nq);
  const AttendRowsArgs r{p->H, p->Nq, w.pad, static_cast<long long>(p->B) * p->H * w.pad,
                         o.p,  g.p,   o.sb,  o.sh, o.sn, g.sb, g.sh, g.sn, lse, s.nlse, s.ndelta};
  AttendBwdArgs f{};
  f.nlse = s.nlse;
  f.ndelta = s.ndelta;
  f.pad = w.pad;
  f.dq = row_out(dq, p->B, p->H, p->Nq);
  f.dk = row_out(dk, p->B, p->Hk, p->Nk);
  f.dv = row_out(dv, p->B, p->Hk, p->Nk);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return p->D == 128 ? launch_backward<128>(w, m, r, f, s, kv_lens, st)
                     : launch_backward<64>(w, m, r, f, s, kv_lens, st);
}

}  // extern "C"
