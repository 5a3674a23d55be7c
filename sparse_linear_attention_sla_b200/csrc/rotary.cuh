// Rotary positions on one to four axes (time, height, width, ...), forward and transposed.
//
// A head's first channels are cut into one run of d_a channels per axis a (the channels behind
// the last run are copied). Pair i of axis a at a token with position p_a turns by
//     phi = p_a * base^(-2 i / d_a):   y1 = x1 cos phi - x2 sin phi,  y2 = x2 cos phi + x1 sin phi,
// (x1, x2) being neighbouring channels or the two halves of the axis' run. The gradient's way
// back is the same turn by -phi.
//
// A stage of the attention's inputs: "SLA: Beyond Sparsity in Diffusion Transformers via
// Fine-Tunable Sparse-Linear Attention" (Abstract) attends over video tokens, whose positions
// have three axes; the rotation itself is the standard one.
//
// Bound by HBM: every element is read once and written once. A thread keeps one 8-channel
// chunk of one token through all heads of q and k that its block takes, so the angles are formed
// once per token and not once per head. They are 64-bit fractions of a turn (see rotary_kernel): an
// fp32 angle at position 1e6 would be off by 0.06, and sines of fp64 angles cost more.
// Measured: 32760 tokens, 12 + 12 heads of 128 channels, bf16: 73 us, 5.5 TB/s of 6.5 measured for a
// plain copy (fp64 angles 83); fp32 gradients to bf16 98 us, 6.1 TB/s.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace sla {

constexpr int kMaxAxes = 4;

struct RotaryTensor {
  const void* x;
  void* y;
  long long xb, xh, xn, yb, yh, yn;  // strides in elements (batch, head, token)
};

struct RotaryArgs {
  RotaryTensor t[2];  // q, k
  int heads[2];
  int N;
  int n_axes;
  int first[kMaxAxes + 1];  // first channel of each axis; the last entry: channels that turn
  int grid[kMaxAxes], start[kMaxAxes];
  int n_turned;             // tokens from here on are copied (the grid's size)
  const int32_t* pos;       // [B or 1, N, n_axes] or null (grid)
  long long pos_b;
  double log2_base;
  float sign;               // +1 forward, -1 transposed
  int heads_per_block;
};

template <typename T>
struct RotaryChunk;  // 8 channels as one thread moves them

template <>
struct RotaryChunk<__nv_bfloat16> {
  uint4 w;
  __device__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  __device__ void set(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<uint32_t*>(&v);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
};

template <>
struct RotaryChunk<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  __device__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

__device__ __forceinline__ float rotary_value(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float rotary_value(const float* p) { return *p; }

// Threads of a block, and heads whose loads are in flight together.
constexpr int kRotaryThreads = 256;
constexpr int kRotaryUnroll = 4;

// HALVES: pairs are (i, i + d_a / 2) of an axis' run, else neighbouring channels. Halves of odd
// widths put a pair's channels at any distance in the row, so a row's chunks meet in shared
// memory (a row's 8 or 16 chunks belong to one warp).
template <int D, bool HALVES, typename Tin, typename Tout>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryArgs a) {
  constexpr int T = D / 8;  // threads of a row
  constexpr int TOKENS = kRotaryThreads / T;
  constexpr int U = kRotaryUnroll;
  __shared__ __align__(16) Tin rows[HALVES ? U : 1][HALVES ? kRotaryThreads * 8 : 1];
  const int c0 = (threadIdx.x % T) * 8;
  const int n = blockIdx.x * TOKENS + threadIdx.x / T;
  const int b = blockIdx.z;
  const int h0 = blockIdx.y * a.heads_per_block;
  const int h1 = min(h0 + a.heads_per_block, a.heads[0] + a.heads[1]);
  const bool in = n < a.N;

  const long long xq = b * a.t[0].xb + n * a.t[0].xn + c0, xk = b * a.t[1].xb + n * a.t[1].xn + c0;
  const long long yq = b * a.t[0].yb + n * a.t[0].yn + c0, yk = b * a.t[1].yb + n * a.t[1].yn + c0;
  RotaryChunk<Tin> x[U];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (in && h + u < h1) {
        const int hk = h + u - a.heads[0];
        x[u].load(hk < 0 ? static_cast<const Tin*>(a.t[0].x) + xq + (h + u) * a.t[0].xh
                         : static_cast<const Tin*>(a.t[1].x) + xk + hk * a.t[1].xh);
      }
    }
  };
  load(h0);  // the first heads are under way while the angles are formed

  // The block's frequencies, one for each pair of channels, then this thread's angles. Pairs of
  // neighbours lie in one thread; halves share theirs through the table of all tokens' pairs.
  // A frequency is held as its fraction of a turn in 64 bits (whole turns per step drop out, positions
  // being whole), so an angle is one integer product, reduced by its overflow. It is off by 2^-32 of a turn at most
  // for the product's dropped bits, by 2^-26 for the fp32 argument of sincospif and by |p| times the fp64 rounding
  // of the frequency.
  __shared__ uint2 freq[D / 2];
  __shared__ float2 table[HALVES ? TOKENS * (D / 2) : 1];
  const int turned_channels = a.first[a.n_axes];
  auto axis_of = [&](int c) {
    int ax = 0;
    while (c >= a.first[ax + 1]) ++ax;
    return ax;
  };
  if (threadIdx.x < D / 2 && 2 * threadIdx.x < turned_channels) {
    const int ax = axis_of(2 * threadIdx.x), d = a.first[ax + 1] - a.first[ax];
    const double f = exp2(-static_cast<double>(2 * threadIdx.x - a.first[ax]) / d * a.log2_base) * 0.15915494309189535;
    const unsigned long long u = static_cast<unsigned long long>((f - floor(f)) * 18446744073709551616.0);
    freq[threadIdx.x] = make_uint2(static_cast<uint32_t>(u), static_cast<uint32_t>(u >> 32));
  }
  const bool turns = in && (a.pos || n < a.n_turned);
  int at[kMaxAxes] = {};  // the token's position on each axis
  if (turns) {
    int q = n;
#pragma unroll
    for (int x = kMaxAxes - 1; x >= 0; --x) {
      if (x >= a.n_axes) continue;
      if (a.pos) {
        at[x] = a.pos[b * a.pos_b + static_cast<long long>(n) * a.n_axes + x];
      } else {
        at[x] = q % a.grid[x] + a.start[x];
        q /= a.grid[x];
      }
    }
  }
  __syncthreads();
  // cos and sin of pair p (counted over all axes) on axis ax.
  auto angle = [&](int p, int ax, float& co, float& s) {
    const uint32_t v = ax == 0 ? at[0] : ax == 1 ? at[1] : ax == 2 ? at[2] : at[3];
    const uint2 f = freq[p];
    // Bits 32..63 of v f modulo 2^64: a negative v, taken as v + 2^32, adds f.x there.
    const uint32_t turn = v * f.y + __umulhi(v, f.x) - (static_cast<int>(v) < 0 ? f.x : 0u);
    sincospif(static_cast<float>(static_cast<int>(turn)) * 0x1p-31f, &s, &co);
    s *= a.sign;
  };

  float cs[8], sn[8];   // y = x cs + partner sn
  int partner[8];       // HALVES: the partner's channel
  uint32_t turned = 0;  // channels that turn
#pragma unroll
  for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f, partner[e] = c0 + e;
  if constexpr (HALVES) {
    if (turns) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = c0 / 2 + e;
        if (2 * p >= turned_channels) continue;
        float co, s;
        angle(p, axis_of(2 * p), co, s);
        table[(threadIdx.x / T) * (D / 2) + p] = make_float2(co, s);
      }
    }
    __syncwarp();  // a row's threads are of one warp
    if (turns) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = c0 + e;
        if (c >= turned_channels) continue;
        const int ax = axis_of(c), half = (a.first[ax + 1] - a.first[ax]) >> 1, l = c - a.first[ax];
        const bool lower = l < half;
        const float2 t = table[(threadIdx.x / T) * (D / 2) + (a.first[ax] >> 1) + (lower ? l : l - half)];
        cs[e] = t.x;
        sn[e] = lower ? -t.y : t.y;
        partner[e] = lower ? c + half : c - half;
        turned |= 1u << e;
      }
    }
  } else if (turns) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int p = (c0 + e) / 2;
      if (2 * p >= turned_channels) continue;
      float co, s;
      angle(p, axis_of(2 * p), co, s);
      cs[e] = cs[e + 1] = co;
      sn[e] = -s;
      sn[e + 1] = s;
      turned |= 3u << e;
    }
  }

  for (int h = h0; h < h1; h += U) {
    if (h > h0) load(h);
    if (HALVES) {
      __syncwarp();  // the previous heads' partners have been read
#pragma unroll
      for (int u = 0; u < U; ++u) x[u].store(&rows[u][threadIdx.x * 8]);
      __syncwarp();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (in && h + u < h1) {
        float f[8], g[8];
        x[u].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other = HALVES ? rotary_value(&rows[u][(threadIdx.x / T) * D + partner[e]]) : f[e ^ 1];
          // a channel that does not turn is copied whatever its neighbour holds
          g[e] = (turned >> e) & 1u ? fmaf(f[e], cs[e], other * sn[e]) : f[e];
        }
        const int hk = h + u - a.heads[0];
        RotaryChunk<Tout> y;
        y.set(g);
        y.store(hk < 0 ? static_cast<Tout*>(a.t[0].y) + yq + (h + u) * a.t[0].yh
                       : static_cast<Tout*>(a.t[1].y) + yk + hk * a.t[1].yh);
      }
    }
  }
}

}  // namespace sla
