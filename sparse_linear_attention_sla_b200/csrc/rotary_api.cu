// Host side of sla_rotary and sla_rotary_backward: argument checks and the launch.
#include <cmath>

#include "host.cuh"
#include "rotary.cuh"

namespace {

using namespace sla_host;
using sla::RotaryArgs;

struct RotaryCall {
  int B, N, D;
  int heads[2];
  const sla_tensor* in[2];
  const sla_tensor* out[2];
};

// 16-byte rows: pointer and strides (a stride is not used where its extent is 1).
sla_status check_tensor(const char* name, const sla_tensor* t, int type, int B, int H, int N) {
  const int per16 = type == SLA_F32 ? 4 : 8;
  if (!t || !aligned16(t->ptr)) return fail(SLA_ERR_INVALID_ARG, "%s must be non-NULL and 16-byte aligned", name);
  if ((B > 1 && t->stride_b % per16) || (H > 1 && t->stride_h % per16) || (N > 1 && t->stride_n % per16))
    return fail(SLA_ERR_INVALID_ARG, "%s's strides must be multiples of 16 bytes", name);
  return SLA_OK;
}

template <int D, bool HALVES, typename Tin, typename Tout>
sla_status launch(RotaryArgs& a, int B, cudaStream_t st) {
  constexpr int tokens = sla::kRotaryThreads / (D / 8);
  const long long nx = (a.N + tokens - 1) / tokens;
  const int total = a.heads[0] + a.heads[1];
  // A block forms its tokens' angles once for all heads that it takes, which costs about as much as six heads do: it
  // takes as many as leave one and a half blocks for every SM, in steps of the unrolled loop where there are
  // enough. (One head to a block, four, this rule: 2 x 4093 tokens of 16 + 4 heads of 64 channels 47.6, 17.1,
  // 12.2 us; 2040 tokens of 24 heads of 128: 21.1, 8.9, 6.6, and 8.1 with all 24; 1500 tokens of 48 heads of 64:
  // 13.4, 5.6, 5.1, and 7.4 with 24.)
  long long per = total * nx * B * 2 / (3ll * sm_count());
  per = per < 1 ? 1 : per > total ? total : per;
  if (per > sla::kRotaryUnroll) per = per / sla::kRotaryUnroll * sla::kRotaryUnroll;
  a.heads_per_block = static_cast<int>(per);
  const dim3 grid(static_cast<unsigned>(nx), static_cast<unsigned>((total + per - 1) / per), B);
  if (grid.y > 65535) return fail(SLA_ERR_UNSUPPORTED, "Hq + Hk=%d too large", total);
  sla::rotary_kernel<D, HALVES, Tin, Tout><<<grid, sla::kRotaryThreads, 0, st>>>(a);
  return launched("rotary_kernel");
}

template <int D, bool HALVES>
sla_status launch_types(RotaryArgs& a, int B, int in_type, int out_type, cudaStream_t st) {
  if (in_type == SLA_BF16) return launch<D, HALVES, __nv_bfloat16, __nv_bfloat16>(a, B, st);
  if (out_type == SLA_BF16) return launch<D, HALVES, float, __nv_bfloat16>(a, B, st);
  return launch<D, HALVES, float, float>(a, B, st);
}

sla_status rotate(const sla_rotary_spec* spec, const RotaryCall& c, int in_type, int out_type, float sign,
                  void* stream) {
  if (!spec) return fail(SLA_ERR_INVALID_ARG, "spec is NULL");
  if (c.B < 1 || c.N < 1 || c.heads[0] < 0 || c.heads[1] < 0 || c.heads[0] + static_cast<long long>(c.heads[1]) < 1)
    return fail(SLA_ERR_INVALID_ARG, "B, N and Hq + Hk must be >= 1");
  if (c.D != 64 && c.D != 128) return fail(SLA_ERR_UNSUPPORTED, "D=%d not supported (64 or 128)", c.D);
  if (c.N > (1 << 30)) return fail(SLA_ERR_UNSUPPORTED, "N=%d exceeds 2^30", c.N);  // token indices stay in 32 bits
  if (c.B > 65535) return fail(SLA_ERR_UNSUPPORTED, "B=%d exceeds 65535", c.B);
  if (static_cast<long long>(c.heads[0]) + c.heads[1] > INT_MAX / 2)
    return fail(SLA_ERR_UNSUPPORTED, "Hq + Hk too large");
  const bool types = (in_type == SLA_BF16 && out_type == SLA_BF16) || (in_type == SLA_F32 && out_type == SLA_F32) ||
                     (in_type == SLA_F32 && out_type == SLA_BF16);
  if (!types) return fail(SLA_ERR_UNSUPPORTED, "types %d to %d not supported", in_type, out_type);
  if (spec->n_axes < 1 || spec->n_axes > sla::kMaxAxes)
    return fail(SLA_ERR_INVALID_ARG, "n_axes=%d (1 to %d)", spec->n_axes, sla::kMaxAxes);
  if (spec->pairing != 0 && spec->pairing != 1) return fail(SLA_ERR_INVALID_ARG, "pairing=%d (0 or 1)", spec->pairing);
  if (!std::isfinite(spec->base) || !(spec->base > 0)) return fail(SLA_ERR_INVALID_ARG, "base must be finite and > 0");
  RotaryArgs a{};
  a.N = c.N;
  a.n_axes = spec->n_axes;
  a.log2_base = std::log2(spec->base);
  a.sign = sign;
  long long cells = 1;
  for (int x = 0; x < spec->n_axes; ++x) {
    const int d = spec->channels[x];
    if (d < 2 || d % 2 || d > c.D - a.first[x])
      return fail(SLA_ERR_INVALID_ARG, "axis %d: %d channels (even, at least 2, all axes together at most D)", x, d);
    a.first[x + 1] = a.first[x] + d;
    if (!spec->positions) {
      if (spec->grid[x] < 1) return fail(SLA_ERR_INVALID_ARG, "grid[%d]=%d must be >= 1", x, spec->grid[x]);
      const long long last = static_cast<long long>(spec->start[x]) + spec->grid[x] - 1;
      if (last > INT_MAX) return fail(SLA_ERR_INVALID_ARG, "start[%d] + grid[%d] passes 32 bits", x, x);
      a.grid[x] = spec->grid[x];
      a.start[x] = spec->start[x];
      cells = cells > INT_MAX ? cells : cells * spec->grid[x];
    }
  }
  a.n_turned = cells > INT_MAX ? INT_MAX : static_cast<int>(cells);
  if (spec->positions) {
    if (reinterpret_cast<uintptr_t>(spec->positions) % 4) return fail(SLA_ERR_INVALID_ARG, "positions must be 4-byte aligned");
    if (spec->positions_stride_b < 0) return fail(SLA_ERR_INVALID_ARG, "positions_stride_b must be >= 0");
    a.pos = spec->positions;
    a.pos_b = spec->positions_stride_b;
  }
  static const char* const names[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
  for (int w = 0; w < 2; ++w) {
    a.heads[w] = c.heads[w];
    if (c.heads[w] == 0) continue;
    SLA_TRY(check_tensor(names[w][0], c.in[w], in_type, c.B, c.heads[w], c.N));
    SLA_TRY(check_tensor(names[w][1], c.out[w], out_type, c.B, c.heads[w], c.N));
    if (!rows_apart(c.out[w], c.B, c.heads[w], c.N, c.D))
      return fail(SLA_ERR_INVALID_ARG, "%s has rows that overlap each other", names[w][1]);
    a.t[w] = {c.in[w]->ptr,      c.out[w]->ptr,      c.in[w]->stride_b,  c.in[w]->stride_h, c.in[w]->stride_n,
              c.out[w]->stride_b, c.out[w]->stride_h, c.out[w]->stride_n};
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (c.D == 128)
    return spec->pairing ? launch_types<128, true>(a, c.B, in_type, out_type, st)
                         : launch_types<128, false>(a, c.B, in_type, out_type, st);
  return spec->pairing ? launch_types<64, true>(a, c.B, in_type, out_type, st)
                       : launch_types<64, false>(a, c.B, in_type, out_type, st);
}

}  // namespace

extern "C" {

sla_status sla_rotary(const sla_rotary_spec* spec, int B, int Hq, int Hk, int N, int D, int type, const sla_tensor* q,
                      const sla_tensor* q_out, const sla_tensor* k, const sla_tensor* k_out, void* stream) {
  const RotaryCall c{B, N, D, {Hq, Hk}, {q, k}, {q_out, k_out}};
  return rotate(spec, c, type, type, 1.f, stream);
}

sla_status sla_rotary_backward(const sla_rotary_spec* spec, int B, int Hq, int Hk, int N, int D, int in_type,
                               int out_type, const sla_tensor* dq, const sla_tensor* dq_out, const sla_tensor* dk,
                               const sla_tensor* dk_out, void* stream) {
  const RotaryCall c{B, N, D, {Hq, Hk}, {dq, dk}, {dq_out, dk_out}};
  return rotate(spec, c, in_type, out_type, -1.f, stream);
}

}  // extern "C"
