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

// CTAs that a launch has at most: the workspace's size must not depend on which device is
// current, so a B200's 148 SMs are taken as given.
constexpr int kSms = 148;

// How one kernel's units are shared out over its CTAs (see AttendWork).
struct Share {
  int units, ctas, waves, uniform, spans;
  bool cut;  // units may be cut into parts
};

// `units` units of at most `steps` steps each. Whole units leave CTAs idle where there are fewer
// units than CTAs, where the last wave is not full, or where units are of unlike length; then the
// steps behind the whole waves are cut into equal ranges, at least two steps to a range.
// Units of like length: all waves but the last two go out whole, and nothing is cut where that
// saves less than kJoinCost steps, what joining the parts takes (17 us, against 8 us that cutting
// the last of 11 waves of 4 steps saves). Many units of unlike length: over 64 to a CTA their
// differences even out, and the scan over them would cost more than it saves.
constexpr double kJoinCost = 8;

Share share_out(long long units, long long steps, bool uniform) {
  Share s{static_cast<int>(units), 0, 0, uniform ? 1 : 0, 0, false};
  const long long waves = (units + kSms - 1) / kSms, unit = steps + sla::kUnitCost;
  const double saved = static_cast<double>(unit) * (waves - static_cast<double>(units) / kSms);
  const bool short_tail = waves >= 4 && unit < kJoinCost;  // of unlike length: at most about one unit is lost
  if ((uniform && saved < kJoinCost) || short_tail || units > 64ll * kSms || units * unit >= (1ll << 31)) {
    s.ctas = static_cast<int>(units < kSms ? units : kSms);
    s.waves = static_cast<int>(waves);
    return s;
  }
  s.waves = uniform && waves > 2 ? static_cast<int>(waves) - 2 : 0;
  const long long ranges = (units * steps + 1) / 2;
  s.ctas = static_cast<int>(ranges < kSms ? (ranges < 1 ? 1 : ranges) : kSms);
  s.cut = true;
  return s;
}

// Causal without lengths: the units' steps are known here, steps(0) those of each head's longest unit, steps(1) of
// the next. Units are taken whole, longest first, every other wave backwards, where the longest CTA's work passes the
// mean by less than kJoinCost (14 instead of 8: forwards of 12 heads 3 to 5% faster or slower, gradients up to 5%
// slower).
// (Parts joined and whole, us: forward of 2 x 2040 tokens of 16 heads 61.0 and 42.7, with D = 64 50.2 and 38.2;
// 4096 tokens of 40 heads 198.0 and 182.2, their gradients 714 and 661.)
template <class Steps>
void take_whole(Share* s, int spans, bool first_is_longest, const Steps& steps) {
  if (!s->cut || s->units < kSms) return;
  const int heads = s->units / spans;
  int load[kSms] = {}, at = 0, step = 1, longest = 0;
  long long total = 0;
  for (int x = 0; x < spans; ++x) {
    const int n = steps(x) + sla::kUnitCost;
    total += static_cast<long long>(n) * heads;
    for (int h = 0; h < heads; ++h) {
      load[at] += n;
      longest = load[at] > longest ? load[at] : longest;
      at += step;
      if (at < 0 || at == kSms) {  // the next wave runs the other way
        at -= step;
        step = -step;
      }
    }
  }
  if (longest > static_cast<double>(total) / kSms + kJoinCost) return;
  s->ctas = kSms;
  s->waves = (s->units + kSms - 1) / kSms;
  s->spans = first_is_longest ? -spans : spans;
  s->cut = false;
}

struct AttendPlan {
  sla_attend_problem p;
  int pad;             // Nq rounded up to whole tiles
  int narrow, heads, tokens;  // forward: see AttendFwdArgs
  Share fwd, dkv, dq;
};

struct AttendSpace {
  uint32_t* err;
  int4 *meta, *meta_q;              // forward or dK / dV, dQ
  float *part, *part_lse2;          // forward, or dK / dV
  float *nlse, *ndelta, *part_q;    // backward
  size_t bytes;
};

sla_status make_plan(const sla_attend_problem* p, bool has_lens, bool bwd, AttendPlan* w) {
  if (!p) return fail(SLA_ERR_INVALID_ARG, "problem is NULL");
  if (p->B < 1 || p->H < 1 || p->Hk < 1 || p->Nq < 1 || p->Nk < 1)
    return fail(SLA_ERR_INVALID_ARG, "B, H, Hk, Nq and Nk must be >= 1");
  if (p->H % p->Hk) return fail(SLA_ERR_INVALID_ARG, "H=%d is not a multiple of Hk=%d", p->H, p->Hk);
  if (p->D != 64 && p->D != 128) return fail(SLA_ERR_UNSUPPORTED, "D=%d not supported (64 or 128)", p->D);
  if (p->causal != 0 && p->causal != 1) return fail(SLA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!std::isfinite(p->scale * 1.4426950408889634f) || !(p->scale > 0.f))  // as the kernels take it, in base 2
    return fail(SLA_ERR_INVALID_ARG, "scale must be finite, in base 2 too, and > 0");
  if (p->Nq > (1 << 24) || p->Nk > (1 << 24)) return fail(SLA_ERR_UNSUPPORTED, "Nq, Nk must be at most 2^24");
  const long long BH = static_cast<long long>(p->B) * p->H, BHk = static_cast<long long>(p->B) * p->Hk;
  const long long qt = (p->Nq + kTile - 1) / kTile, kt = (p->Nk + kTile - 1) / kTile;
  if (BH * qt >= (1ll << 28) || BHk * kt >= (1ll << 28)) return fail(SLA_ERR_UNSUPPORTED, "B*H*N too large");
  const long long group = p->H / p->Hk;
  if (group * qt >= (1ll << 30)) return fail(SLA_ERR_UNSUPPORTED, "H / Hk * Nq too large");
  w->p = *p;
  w->pad = static_cast<int>(qt * kTile);
  const bool uniform = !p->causal && !has_lens;
  w->narrow = p->Nq <= kTile;
  w->heads = 1;
  w->tokens = w->narrow ? p->Nq : kTile;
  // Tiles of more heads and fewer queries: as few tiles as can be (130 queries of a group of 3: 4 tiles instead of
  // 6), and of equally many the one of fewest queries where the mask is causal, whose diagonal is then
  // cut more finely.
  long long tiles = group * ((p->Nq + w->tokens - 1) / w->tokens);
  for (int h = 2; h <= group && h <= kTile; ++h) {
    const int t = p->Nq < kTile / h ? p->Nq : kTile / h;
    const long long n = (group + h - 1) / h * ((p->Nq + t - 1) / t);
    if (n < tiles || (n == tiles && p->causal && !w->narrow)) {
      if (w->narrow && t < p->Nq) continue;  // one tile of a group holds all queries
      tiles = n;
      w->heads = h;
      w->tokens = t;
    }
  }
  const long long span = (w->narrow ? 1 : 2) * w->tokens, spans = (p->Nq + span - 1) / span;
  const long long fwd_units = BHk * ((group + w->heads - 1) / w->heads) * spans;
  // one tile sees the same keys whatever the mask
  w->fwd = share_out(fwd_units, w->narrow ? (kt + 1) / 2 : kt, w->narrow ? !has_lens : uniform);
  w->dkv = share_out(BHk * kt, group * qt, uniform);
  w->dq = share_out(BH * qt, kt, uniform);
  if (p->causal && !has_lens) {
    // Key tiles that queries up to `last` see.
    const auto key_tiles = [p](long long last) {
      const long long end = p->Nk - p->Nq + (last < p->Nq ? last : p->Nq);
      return end < 1 ? 1 : static_cast<int>((end + kTile - 1) / kTile);
    };
    if (!bwd && !w->narrow)
      take_whole(&w->fwd, static_cast<int>(spans), false, [&](int x) { return key_tiles((spans - x) * span); });
    if (bwd) {
      take_whole(&w->dq, static_cast<int>(qt), false, [&](int x) { return key_tiles((qt - x) * kTile); });
      take_whole(&w->dkv, static_cast<int>(kt), true, [&](int x) {
        const long long first = x * kTile - (p->Nk - p->Nq);  // first query that sees a key of the tile
        return first >= p->Nq ? 1 : static_cast<int>(group * (qt - (first > 0 ? first / kTile : 0)));
      });
    }
  }
  return SLA_OK;
}

AttendSpace layout(const AttendPlan& w, uint8_t* base, bool bwd) {
  AttendSpace s{};
  size_t off = 0;
  auto take = [&](size_t words) {
    float* p = base ? reinterpret_cast<float*>(base + off) : nullptr;
    off += align256(words * sizeof(float));
    return p;
  };
  auto meta = [&](const Share& h) { return h.cut ? reinterpret_cast<int4*>(take(4 * static_cast<size_t>(h.ctas))) : nullptr; };
  s.err = reinterpret_cast<uint32_t*>(take(64));
  const size_t row = w.p.D;
  if (!bwd) {
    s.meta = meta(w.fwd);
    const size_t rows = 2 * static_cast<size_t>(w.fwd.ctas) * (w.narrow ? 1 : 2) * kTile;
    if (w.fwd.cut) {
      s.part = take(rows * row);
      s.part_lse2 = take(rows);
    }
  } else {
    const size_t stats = static_cast<size_t>(w.p.B) * w.p.H * w.pad;
    s.nlse = take(stats);
    s.ndelta = take(stats);
    s.meta = meta(w.dkv);
    s.meta_q = meta(w.dq);
    if (w.dkv.cut) s.part = take(2 * static_cast<size_t>(w.dkv.ctas) * 2 * kTile * row);
    if (w.dq.cut) s.part_q = take(2 * static_cast<size_t>(w.dq.ctas) * kTile * row);
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

// The workspace holds a call with key lengths as well as one without.
size_t space_bytes(const sla_attend_problem* p, bool bwd) {
  AttendPlan a, b;
  if (make_plan(p, false, bwd, &a) != SLA_OK || make_plan(p, true, bwd, &b) != SLA_OK) return 0;
  const size_t x = layout(a, nullptr, bwd).bytes, y = layout(b, nullptr, bwd).bytes;
  return x > y ? x : y;
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
    if (d.stride >= (1ll << 38) / heads) return fail(SLA_ERR_UNSUPPORTED, "%s's strides are too large", name);
  }
  return SLA_OK;
}

// The same for an output.
sla_status check_output(const char* name, const sla_tensor* t, int B, int heads, int N, int D) {
  SLA_TRY(check_operand(name, t, B, heads, N));
  if (!rows_apart(t, B, heads, N, D)) return fail(SLA_ERR_INVALID_ARG, "%s has rows that overlap each other", name);
  return SLA_OK;
}

// The queries as (channel, token, head of the group, key head, sequence): boxes of `tokens` rows of
// `heads` heads.
sla_status query_map(CUtensorMap* m, const sla_tensor* t, const sla_attend_problem& p, int tokens, int heads) {
  const int G = p.H / p.Hk;
  const uint64_t dims[5] = {static_cast<uint64_t>(p.D), static_cast<uint64_t>(p.Nq), static_cast<uint64_t>(G),
                            static_cast<uint64_t>(p.Hk), static_cast<uint64_t>(p.B)};
  const uint64_t strides[4] = {static_cast<uint64_t>(p.Nq > 1 ? t->stride_n : p.D),
                               static_cast<uint64_t>(G > 1 ? t->stride_h : p.D),
                               static_cast<uint64_t>(p.Hk > 1 ? G * t->stride_h : p.D),
                               static_cast<uint64_t>(p.B > 1 ? t->stride_b : p.D)};
  const uint32_t box[5] = {64, static_cast<uint32_t>(tokens), static_cast<uint32_t>(heads), 1, 1};
  return make_map(m, t->ptr, 5, dims, strides, box);
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

AttendArgs common_args(const AttendPlan& w, const int32_t* lens, uint32_t* err, const Share& h, int4* meta) {
  AttendArgs a{};
  a.B = w.p.B;
  a.H = w.p.H;
  a.Hk = w.p.Hk;
  a.G = w.p.H / w.p.Hk;
  a.Nq = w.p.Nq;
  a.Nk = w.p.Nk;
  a.causal = w.p.causal;
  a.units = h.units;
  a.waves = h.waves;
  a.uniform = h.uniform;
  a.spans = h.spans;
  a.meta = meta;
  a.scale = w.p.scale;
  a.scale_log2 = w.p.scale * 1.4426950408889634f;
  a.lens = lens;
  a.err = err;
  return a;
}

struct Maps {
  CUtensorMap q, k, v, g;
};

template <int D>
sla_status launch_forward(const AttendPlan& w, const Maps& m, const AttendFwdArgs& f, cudaStream_t st) {
  constexpr int smem = sla::AttendSmem<D>::total();
  SLA_TRY(allow_smem(sla::attend_kernel<D>, smem));
  SLA_TRY(launch_dependent(sla::attend_kernel<D>, dim3(w.fwd.ctas), dim3(sla::kThreads), smem, st, "attend_kernel", m.q, m.k,
                           m.v, f));
  if (w.fwd.cut)
    SLA_TRY(launch_dependent(sla::attend_join_kernel<D>, dim3(w.fwd.ctas, (w.narrow ? 1 : 2) * kTile / (256 / (D / 8))), dim3(256), 0,
                             st, "attend_join_kernel", f));
  return SLA_OK;
}

template <int D>
sla_status launch_backward(const AttendPlan& w, const Maps& m, const AttendRowsArgs& r, const AttendBwdArgs& kv,
                           const AttendBwdArgs& q, cudaStream_t st) {
  constexpr int per = 256 / (D / 8);
  const unsigned blocks = static_cast<unsigned>(w.p.B) * w.p.H * (w.pad / (per * sla::kRowsUnroll));
  SLA_TRY(launch_dependent(sla::attend_rows_kernel<D>, dim3(blocks), dim3(256), 0, st, "attend_rows_kernel", r));
  constexpr int smem_kv = sla::AttendDkvSmem<D>::total(), smem_q = sla::AttendDqSmem<D>::total();
  SLA_TRY(allow_smem(sla::attend_dkv_kernel<D>, smem_kv));
  SLA_TRY(allow_smem(sla::attend_dq_kernel<D>, smem_q));
  auto run_dkv = [&] {
    return launch_dependent(sla::attend_dkv_kernel<D>, dim3(w.dkv.ctas), dim3(sla::kBwdThreads), smem_kv, st,
                            "attend_dkv_kernel", m.q, m.k, m.v, m.g, kv);
  };
  auto run_dq = [&] {
    return launch_dependent(sla::attend_dq_kernel<D>, dim3(w.dq.ctas), dim3(sla::kBwdThreads), smem_q, st,
                            "attend_dq_kernel", m.q, m.k, m.v, m.g, q);
  };
  SLA_TRY(q.dq_first ? run_dq() : run_dkv());
  SLA_TRY(q.dq_first ? run_dkv() : run_dq());
  if (w.dkv.cut || w.dq.cut) {
    const AttendSumArgs s{kv, q, w.dkv.ctas, w.dq.ctas};
    const int ctas = w.dkv.ctas > w.dq.ctas ? w.dkv.ctas : w.dq.ctas;
    SLA_TRY(launch_dependent(sla::attend_sum_kernel<D>, dim3(ctas, kTile / per, 3), dim3(256), 0, st,
                             "attend_sum_kernel", s));
  }
  return SLA_OK;
}

sla_status check_lens(const int32_t* lens) {
  if (reinterpret_cast<uintptr_t>(lens) % 4) return fail(SLA_ERR_INVALID_ARG, "kv_lens must be 4-byte aligned");
  return SLA_OK;
}

}  // namespace

extern "C" {

size_t sla_workspace_size_attend(const sla_attend_problem* p) {
  return space_bytes(p, false);
}

size_t sla_workspace_size_attend_backward(const sla_attend_problem* p) {
  return space_bytes(p, true);
}

sla_status sla_attend(const sla_attend_problem* p, const sla_tensor* q, const sla_tensor* k, const sla_tensor* v,
                      const int32_t* kv_lens, const sla_tensor* out, float* lse, void* ws, size_t ws_bytes,
                      void* stream) {
  AttendPlan w;
  SLA_TRY(make_plan(p, kv_lens != nullptr, false, &w));
  SLA_TRY(check_operand("q", q, p->B, p->H, p->Nq));
  SLA_TRY(check_operand("k", k, p->B, p->Hk, p->Nk));
  SLA_TRY(check_operand("v", v, p->B, p->Hk, p->Nk));
  SLA_TRY(check_output("out", out, p->B, p->H, p->Nq, p->D));
  SLA_TRY(check_lens(kv_lens));
  if (!lse || reinterpret_cast<uintptr_t>(lse) % 4) return fail(SLA_ERR_INVALID_ARG, "lse must be non-NULL and 4-byte aligned");
  AttendSpace s;
  SLA_TRY(check_space(w, ws, ws_bytes, false, &s));
  Maps m;
  SLA_TRY(query_map(&m.q, q, *p, w.tokens, w.heads));
  SLA_TRY(operand_map(&m.k, k, p->B, p->Hk, p->Nk, p->D));
  SLA_TRY(operand_map(&m.v, v, p->B, p->Hk, p->Nk, p->D));
  AttendFwdArgs f{};
  f.p = common_args(w, kv_lens, s.err, w.fwd, s.meta);
  f.narrow = w.narrow;
  f.heads = w.heads;
  f.tokens = w.tokens;
  f.q_bytes = w.tokens * w.heads * p->D * 2;
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
  SLA_TRY(make_plan(p, kv_lens != nullptr, true, &w));
  SLA_TRY(check_operand("q", q, p->B, p->H, p->Nq));
  SLA_TRY(check_operand("k", k, p->B, p->Hk, p->Nk));
  SLA_TRY(check_operand("v", v, p->B, p->Hk, p->Nk));
  SLA_TRY(check_operand("out", out, p->B, p->H, p->Nq));
  SLA_TRY(check_operand("dO", dO, p->B, p->H, p->Nq));
  SLA_TRY(check_output("dq", dq, p->B, p->H, p->Nq, p->D));
  SLA_TRY(check_output("dk", dk, p->B, p->Hk, p->Nk, p->D));
  SLA_TRY(check_output("dv", dv, p->B, p->Hk, p->Nk, p->D));
  SLA_TRY(check_lens(kv_lens));
  if (!lse || reinterpret_cast<uintptr_t>(lse) % 4) return fail(SLA_ERR_INVALID_ARG, "lse must be non-NULL and 4-byte aligned");
  AttendSpace s;
  SLA_TRY(check_space(w, ws, ws_bytes, true, &s));
  Maps m;
  SLA_TRY(operand_map(&m.q, q, p->B, p->H, p->Nq, p->D));
  SLA_TRY(operand_map(&m.k, k, p->B, p->Hk, p->Nk, p->D));
  SLA_TRY(operand_map(&m.v, v, p->B, p->Hk, p->Nk, p->D));
  SLA_TRY(operand_map(&m.g, dO, p->B, p->H, p->Nq, p->D));
  const RowOut o = row_out(out, p->B, p->H, p->Nq), g = row_out(dO, p->B, p->H, p->Nq);
  const AttendRowsArgs r{p->H, p->Nq, w.pad,
                         o.p,  g.p,   o.sb,  o.sh, o.sn, g.sb, g.sh, g.sn, lse, s.nlse, s.ndelta};
  AttendBwdArgs f{};
  f.p = common_args(w, kv_lens, s.err, w.dkv, s.meta);
  f.part = s.part;
  f.nlse = s.nlse;
  f.ndelta = s.ndelta;
  f.pad = w.pad;
  // Sequences of one key tile: surely none where all have Nk keys and those are more.
  f.dq_first = kv_lens != nullptr || p->Nk <= kTile;
  f.dq = row_out(dq, p->B, p->H, p->Nq);
  f.dk = row_out(dk, p->B, p->Hk, p->Nk);
  f.dv = row_out(dv, p->B, p->Hk, p->Nk);
  AttendBwdArgs fq = f;
  fq.p = common_args(w, kv_lens, s.err, w.dq, s.meta_q);
  fq.part = s.part_q;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return p->D == 128 ? launch_backward<128>(w, m, r, f, fq, st) : launch_backward<64>(w, m, r, f, fq, st);
}

}  // extern "C"
