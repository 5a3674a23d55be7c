// What the dense attention kernels (forward, dQ, dK / dV) share: the problem, the visible key
// ranges, tensor-core products over 128-row tiles, and row stores.
//
// All of them work on tiles of 128 rows x D channels in shared memory: D / 64 boxes of 128
// rows x 128 bytes in TMA's 128-byte swizzle. Two kinds of product cover forward and backward:
//   ss: D[128 x 128] = A B^T over D channels, both tiles read as rows x channels (K-major)
//   ts: D[128 x D] (+)= P B over 128 rows, P (bf16) in TMEM, B read row by row (MN-major)
#pragma once

#include "sm100.cuh"

namespace sla {

struct AttendArgs {
  int B, H, Hk, G, Nq, Nk;  // G = H / Hk query heads share a key head
  int causal;
  int splits;
  int units;                // work items of the launch
  float scale, scale_log2;  // scale, scale * log2(e)
  const int32_t* lens;      // [B] keys of each sequence, or null (Nk)
  uint32_t* err;
};

constexpr int kTile = 128;                 // rows of every tile
constexpr uint32_t kBox = kTile * 128;     // bytes of one 64-channel box

// Keys of sequence b. A length outside [0, Nk] is taken as the nearer end, so that no access
// leaves the tensors, and recorded.
__device__ __forceinline__ int attend_len(const AttendArgs& a, int b, bool record) {
  if (!a.lens) return a.Nk;
  const int n = a.lens[b];
  const int m = min(max(n, 0), a.Nk);
  if (record && m != n) record_error(a.err, SLA_DEVERR_BAD_LEN);
  return m;
}

// Keys that query rows up to `last` of a sequence with `len` keys see: query i sees the keys
// j < len and, causal, j <= i + len - Nq (the last query sees the last key).
__device__ __forceinline__ int attend_key_end(const AttendArgs& a, int len, int last) {
  return a.causal ? max(0, min(len, last + len - a.Nq + 1)) : len;
}

__device__ __forceinline__ int tiles_of(int n) { return (n + kTile - 1) / kTile; }

// The part [lo, hi) of n tiles that split s of a.splits takes.
__device__ __forceinline__ void split_range(int n, int splits, int s, int& lo, int& hi) {
  const int per = (n + splits - 1) / splits;
  lo = min(n, s * per);
  hi = min(n, lo + per);
}

// One lane of the MMA warp issues. D[128 x 128] = A B^T over D channels.
template <int D>
__device__ __forceinline__ void issue_ss(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem) {
  constexpr uint32_t id = idesc_bf16_f32(128, 128, 0, 0);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t ad = smem_desc_sw128(a_smem + (kk >> 2) * kBox + (kk & 3) * 32, 16, 1024);
    const uint64_t bd = smem_desc_sw128(b_smem + (kk >> 2) * kBox + (kk & 3) * 32, 16, 1024);
    umma_bf16_ss(d_tmem, ad, bd, id, kk > 0 ? 1u : 0u);
  }
}

// D[128 x D] (+)= P B over the tile's 128 rows. P's 16-row steps are 8 TMEM columns each;
// HALF: the columns of rows 64.. start HALF columns behind those of rows 0.. (32: no gap).
template <int D, int HALF>
__device__ __forceinline__ void issue_ts(uint32_t d_tmem, uint32_t p_tmem, uint32_t b_smem, bool accumulate) {
  constexpr uint32_t id = idesc_bf16_f32(128, D, 0, 1);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint64_t bd = smem_desc_sw128(b_smem + kk * 2048, kBox, 1024);
    umma_bf16_ts(d_tmem, p_tmem + (kk >> 2) * HALF + (kk & 3) * 8, bd, id, (accumulate || kk > 0) ? 1u : 0u);
  }
}

// Rows [lo, hi) of a tile to zero, by a whole warp, before an MMA reads them: rows that no
// query or key may see can hold anything, and 0 * NaN is not 0.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int lo, int hi) {
  const int lane = threadIdx.x & 31;
  for (int b = 0; b < D / 64; ++b)
    for (int c = lo * 8 + lane; c < hi * 8; c += 32)
      *reinterpret_cast<uint4*>(tile + b * kBox + c * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// 32 bytes in one store (a full sector) where the address allows, else two of 16.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint4* q = static_cast<uint4*>(p);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// 32 accumulator columns of this thread's row, times f, to global memory as bf16 or fp32.
__device__ __forceinline__ void store_row32(__nv_bfloat16* p, const uint32_t (&x)[32], float f, bool wide) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = pack_bf16x2(__uint_as_float(x[16 * g + 2 * i]) * f, __uint_as_float(x[16 * g + 2 * i + 1]) * f);
    store32(p + 16 * g, w, wide);
  }
}
__device__ __forceinline__ void store_row32(float* p, const uint32_t (&x)[32], float f, bool wide) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(__uint_as_float(x[8 * g + i]) * f);
    store32(p + 8 * g, w, wide);
  }
}

// Where a kernel writes rows: bf16 with strides, or fp32 partial rows [split][row] of D.
struct RowOut {
  __nv_bfloat16* p;
  long long sb, sh, sn;  // elements
  int wide;              // rows start on 32-byte boundaries
};

}  // namespace sla
