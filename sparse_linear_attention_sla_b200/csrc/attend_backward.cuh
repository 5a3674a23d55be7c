// Backward pass of the dense attention: dq, dk, dv of sum(dO * out), the probabilities
// recomputed from the saved log-sum-exp.
//
//   P = 2^(s scale log2(e) - lse2), delta = rowsum(dO * out), dP = dO V^T, T = P * (dP - delta)
//   dV = P^T dO,  dQ = scale T K,  dK = scale T^T Q
// with lse2 = lse log2(e); dK and dV of a shared key head sum over its query heads.
//
// Two tensor-core kernels, one per summation direction, so that every sum runs in a fixed order
// without atomics: attend_dkv_kernel sums over queries (S, dP recomputed, dV, dK: four
// products per tile pair), attend_dq_kernel over keys (S, dP recomputed, dQ: three). The two
// recomputed products cost 2/5 more tensor work than one kernel that would add its dQ tiles
// into global memory in an order that changes from run to run.
//
// P and T are rounded to bf16 for the tensor cores (by at most 2^-8 of each value); S, dP,
// delta, lse and every sum are fp32. Rows without keys have lse = -inf: their P is 0, and
// delta is taken as 0.
#pragma once

#include "attend_common.cuh"

namespace sla {

struct AttendBwdArgs {
  AttendArgs p;
  const float* nlse;    // [B * H, pad] -lse2 (padding rows and rows without keys: -inf)
  const float* ndelta;  // [B * H, pad] -delta
  int pad;              // Nq rounded up to whole tiles
  RowOut dq, dk, dv;
  float* part;          // splits > 1: dQ [splits][B * H * Nq][D], or dK then dV [splits][B * Hk * Nk][D]
};

// -lse2 and -delta of every row, 8 channels a lane. Reads out and dO once (bound by HBM).
struct AttendRowsArgs {
  int H, Nq, pad;
  long long rows;  // B * H * pad
  const __nv_bfloat16 *out, *dO;
  long long ob, oh, on, gb, gh, gn;
  const float* lse;
  float *nlse, *ndelta;
};

template <int D>
__global__ void __launch_bounds__(256) attend_rows_kernel(AttendRowsArgs a) {
  constexpr int T = D / 8;  // lanes of a row, 8 channels each
  const long long i = static_cast<long long>(blockIdx.x) * (256 / T) + threadIdx.x / T;
  const int c = (threadIdx.x % T) * 8;
  grid_dep_wait();
  const int row = static_cast<int>(i % a.pad);
  const long long bh = i / a.pad;
  float nl = -INFINITY, sum = 0.f;
  if (i < a.rows && row < a.Nq) {
    nl = -a.lse[bh * a.Nq + row] * 1.4426950408889634f;
    const long long b = bh / a.H, h = bh % a.H;
    if (nl == INFINITY) {  // a row without keys
      nl = -INFINITY;
    } else {
      const uint4 x = *reinterpret_cast<const uint4*>(a.out + b * a.ob + h * a.oh + row * a.on + c);
      const uint4 y = *reinterpret_cast<const uint4*>(a.dO + b * a.gb + h * a.gh + row * a.gn + c);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 u = unpack_bf16x2(xs[k]), v = unpack_bf16x2(ys[k]);
        sum = fmaf(u.x, v.x, fmaf(u.y, v.y, sum));
      }
    }
  }
#pragma unroll
  for (int o = T / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (c == 0 && i < a.rows) {
    a.nlse[i] = nl;
    a.ndelta[i] = -sum;
  }
}

// Two neighbouring columns as a pair for the paired arithmetic.
__device__ __forceinline__ uint64_t pair_of(const uint32_t* x) {
  return static_cast<uint64_t>(x[0]) | (static_cast<uint64_t>(x[1]) << 32);
}

// ---------------------------------------------------------------------------- dK, dV

// One persistent CTA per SM, 320 threads, on units of 128 keys of one key head x a range of
// the (query head of the group, query tile) pairs that see them:
//   warp 0       TMA: K_j and V_j once, then Q_i, dO_i and the rows' statistics through a ring
//                of two stages
//   warp 1       tcgen05 issuer: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += T^T Q. The
//                queue alternates: while the warps form P of tile i the tensor cores run
//                dK of tile i - 1 and dP of tile i; while they form T, dV of tile i and S of
//                tile i + 1.
//   warps 2..9   thread = key row = TMEM lane; warps 2..5 take the tile's queries 0..63, warps
//                6..9 queries 64..127
// TMEM columns: S^T [0,128) and dP^T [128,256), each overwritten by its bf16 result (queries
// 0..63 at +0, 64..127 at +64, so that each half of the warps overwrites only what it has
// read); dV [256,256+D), dK [384,384+D).
template <int D>
struct AttendDkvSmem {
  static constexpr uint32_t TILE = kTile * D * 2;
  static constexpr uint32_t STATS = 2 * kTile * 4;
  static constexpr uint32_t STAGE = 2 * TILE;
  static constexpr int STAGES = 2;
  static constexpr uint32_t total() { return 2 * TILE + STAGES * (STAGE + STATS) + 1024; }
};

struct DkvUnit {
  int b, hk, key0, split;
  int len, first;  // keys of the sequence; first query tile that sees a key of the tile
  int tiles;       // query tiles per head from there on
  int lo, hi;      // this unit's range of group x tiles
  int dead;        // queries before this row see no key (causal, more queries than keys)
};

__device__ __forceinline__ DkvUnit dkv_unit(const AttendArgs& a, int u, bool record) {
  DkvUnit w;
  const int kt = tiles_of(a.Nk);
  w.split = u % a.splits;
  const int t = u / a.splits;
  w.key0 = t % kt * kTile;
  w.b = t / kt / a.Hk;
  w.hk = t / kt % a.Hk;
  w.len = attend_len(a, w.b, record);
  w.dead = a.causal ? max(0, a.Nq - w.len) : 0;
  const int first_row = a.causal ? max(0, w.key0 - (w.len - a.Nq)) : 0;  // sees key0, causal
  w.first = first_row / kTile;
  w.tiles = w.key0 < w.len && first_row < a.Nq ? tiles_of(a.Nq) - w.first : 0;
  split_range(w.tiles * a.G, a.splits, w.split, w.lo, w.hi);
  return w;
}

template <int D>
__global__ void __launch_bounds__(320, 1)
    attend_dkv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_g,
                      const __grid_constant__ AttendBwdArgs f) {
  using L = AttendDkvSmem<D>;
  constexpr int DB = D / 64, ST = L::STAGES;
  constexpr uint32_t TP = 128, TV = 256, TK = 384;  // TMEM columns of dP^T, dV, dK
  const AttendArgs& a = f.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = base;
  uint8_t* sV = sK + L::TILE;
  uint8_t* ring = sV + L::TILE;                                           // Q then dO
  float* stats = reinterpret_cast<float*>(ring + ST * L::STAGE);          // nlse[128] then ndelta[128]

  __shared__ uint64_t kv_full, kv_free, s_full, dp_full, p_full, t_full, acc_full, acc_free, drain;
  __shared__ uint64_t q_full[ST], g_full[ST], q_free[ST], g_free[ST];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&kv_full, 1);
    mbar_init(&kv_free, 1);
    mbar_init(&s_full, 1);
    mbar_init(&dp_full, 1);
    mbar_init(&p_full, 256);
    mbar_init(&t_full, 256);
    mbar_init(&acc_full, 1);
    mbar_init(&acc_free, 256);
    mbar_init(&drain, 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&g_full[s], 1);
      mbar_init(&q_free[s], 1);
      mbar_init(&g_free[s], 1);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  grid_dep_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tmap(&map_q);
      prefetch_tmap(&map_k);
      prefetch_tmap(&map_v);
      prefetch_tmap(&map_g);
      uint32_t nr = 0, nu = 0, ng = 0;  // Q tiles, units and dO tiles loaded
      bool ok = true;
      for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
        const DkvUnit w = dkv_unit(a, u, true);
        if (w.lo >= w.hi) continue;
        if (nu > 0 && !(ok = mbar_wait(&kv_free, (nu - 1) & 1, a.err, &abort_flag))) break;
        mbar_arrive_expect_tx(&kv_full, 2 * L::TILE);
        for (int b = 0; b < DB; ++b) tma_load_4d(sK + b * kBox, &map_k, &kv_full, b * 64, w.key0, w.hk, w.b);
        for (int b = 0; b < DB; ++b) tma_load_4d(sV + b * kBox, &map_v, &kv_full, b * 64, w.key0, w.hk, w.b);
        ++nu;
        for (int i = w.lo; i < w.hi; ++i) {
          const int h = w.hk * a.G + i / w.tiles, row = (w.first + i % w.tiles) * kTile;
          const uint32_t s = nr % ST, r = nr / ST;
          if (r > 0 && !(ok = mbar_wait(&q_free[s], (r - 1) & 1, a.err, &abort_flag))) break;
          const size_t at = (static_cast<size_t>(w.b) * a.H + h) * f.pad + row;
          uint8_t* stage = ring + s * L::STAGE;
          float* st = stats + s * 2 * kTile;
          mbar_arrive_expect_tx(&q_full[s], L::TILE + L::STATS);
          for (int b = 0; b < DB; ++b) tma_load_4d(stage + b * kBox, &map_q, &q_full[s], b * 64, row, h, w.b);
          bulk_load(st, f.nlse + at, &q_full[s], kTile * 4);
          bulk_load(st + kTile, f.ndelta + at, &q_full[s], kTile * 4);
          ++nr;
          if (r > 0 && !(ok = mbar_wait(&g_free[s], (r - 1) & 1, a.err, &abort_flag))) break;
          mbar_arrive_expect_tx(&g_full[s], L::TILE);
          for (int b = 0; b < DB; ++b)
            tma_load_4d(stage + L::TILE + b * kBox, &map_g, &g_full[s], b * 64, row, h, w.b);
          ++ng;
        }
      }
      if (abort_flag) {  // let every load still in flight land before the CTA retires
        if (nu > 0) mbar_wait(&kv_full, (nu - 1) & 1, nullptr, nullptr);
        for (uint32_t i = nr > ST ? nr - ST : 0; i < nr; ++i) mbar_wait(&q_full[i % ST], (i / ST) & 1, nullptr, nullptr);
        for (uint32_t i = ng > ST ? ng - ST : 0; i < ng; ++i) mbar_wait(&g_full[i % ST], (i / ST) & 1, nullptr, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t k0 = smem_u32(sK), v0 = smem_u32(sV), r0 = smem_u32(ring);
    uint32_t it = 0, nu = 0;  // query tiles and units so far
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.err, &abort_flag));
    };
    for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
      const DkvUnit w = dkv_unit(a, u, false);
      const int n = w.hi - w.lo;
      if (n <= 0) continue;
      // Rows of the unit's query tile i that see no key may hold anything: zero them where the
      // products sum over rows.
      auto clean = [&](uint8_t* tile, int i) {
        const int row = (w.first + (w.lo + i) % w.tiles) * kTile;
        if (row < w.dead) zero_rows<D>(tile, 0, min(kTile, w.dead - row));
      };
      auto issue_s = [&](int i) -> bool {
        const uint32_t t = it + i, s = t % ST;
        if (!wait_all(&q_full[s], (t / ST) & 1)) return false;
        clean(ring + s * L::STAGE, i);
        tc_fence_after();
        if (elect_one()) {
          issue_ss<D>(tmem, k0, r0 + s * L::STAGE);
          umma_commit(&s_full);
        }
        __syncwarp();
        return true;
      };
      auto issue_dp = [&](int i) -> bool {
        const uint32_t t = it + i, s = t % ST;
        if (!wait_all(&g_full[s], (t / ST) & 1)) return false;
        clean(ring + s * L::STAGE + L::TILE, i);
        tc_fence_after();
        if (elect_one()) {
          issue_ss<D>(tmem + TP, v0, r0 + s * L::STAGE + L::TILE);
          umma_commit(&dp_full);
          if (i + 1 == n) umma_commit(&kv_free);  // the unit's last reader of K_j and V_j
        }
        __syncwarp();
        return true;
      };
      if (!(ok = wait_all(&kv_full, nu & 1))) break;
      if (!(ok = issue_s(0) && issue_dp(0))) break;
      if (nu > 0 && !(ok = wait_all(&acc_free, (nu - 1) & 1))) break;
      for (int i = 0; i < n; ++i) {
        const uint32_t t = it + i, s = t % ST;
        const uint32_t q = r0 + s * L::STAGE, g = q + L::TILE;
        if (!(ok = wait_all(&p_full, t & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          issue_ts<D, 64>(tmem + TV, tmem, g, i > 0);
          umma_commit(&g_free[s]);
        }
        __syncwarp();
        if (i + 1 < n && !(ok = issue_s(i + 1))) break;
        if (!(ok = wait_all(&t_full, t & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          issue_ts<D, 64>(tmem + TK, tmem + TP, q, i > 0);
          umma_commit(&q_free[s]);
          if (i + 1 == n) umma_commit(&acc_full);
        }
        __syncwarp();
        if (i + 1 < n && !(ok = issue_dp(i + 1))) break;
      }
      it += n;
      ++nu;
    }
    if (elect_one()) umma_commit(&drain);
    __syncwarp();
    mbar_wait(&drain, 0, nullptr, nullptr);
  } else {
    // ------------------------------------------------------------ P and T, then the epilogue
    const int half = warp >= 6;
    const int r = (warp & 3) * 32 + lane;  // key row of the tile = TMEM lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + half * 64, p_addr = lane_addr + TP + half * 64;
    const float sc = a.scale_log2;
    const uint64_t sc2 = f2_make(sc, sc);
    uint32_t it = 0, nu = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.err, &abort_flag));
    };
    for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
      const DkvUnit w = dkv_unit(a, u, false);
      const int n = w.hi - w.lo;
      const int key = w.key0 + r;
      for (int i = 0; i < n; ++i, ++it) {
        const int row = (w.first + (w.lo + i) % w.tiles) * kTile + half * 64;  // first query of this half
        const float* st = stats + (it % ST) * 2 * kTile + half * 64;
        // First column of this half whose query sees the key, 64: none. Queries from it on all do.
        const int from = key >= w.len ? 64 : a.causal ? max(0, key - (w.len - a.Nq) - row) : 0;
        const bool masked = __any_sync(0xffffffffu, from > 0);
        if (!(ok = wait(&s_full, it & 1))) break;
        if (!(ok = wait(&q_full[it % ST], (it / ST) & 1))) break;  // the rows' statistics
        tc_fence_after();
        uint32_t p[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(s_addr + 32 * c, p[c]);
        tmem_wait_ld();
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(st + 32 * c + e);
            const uint64_t x0 = f2_fma(pair_of(&p[c][e]), sc2, nl.x), x1 = f2_fma(pair_of(&p[c][e + 2]), sc2, nl.y);
            float v[4] = {fast_exp2(f2_lo(x0)), fast_exp2(f2_hi(x0)), fast_exp2(f2_lo(x1)), fast_exp2(f2_hi(x1))};
            if (masked) {
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = 32 * c + e + q >= from ? v[q] : 0.f;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) p[c][e + q] = __float_as_uint(v[q]);
            pk[16 * c + e / 2] = pack_bf16x2(v[0], v[1]);
            pk[16 * c + e / 2 + 1] = pack_bf16x2(v[2], v[3]);
          }
        }
        tmem_st32(s_addr, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full);
        if (!(ok = wait(&dp_full, it & 1))) break;
        tc_fence_after();
        uint32_t d[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(p_addr + 32 * c, d[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const ulonglong2 nd = *reinterpret_cast<const ulonglong2*>(st + kTile + 32 * c + e);
            uint64_t y0 = f2_mul(f2_add(pair_of(&d[c][e]), nd.x), pair_of(&p[c][e]));
            uint64_t y1 = f2_mul(f2_add(pair_of(&d[c][e + 2]), nd.y), pair_of(&p[c][e + 2]));
            float v[4] = {f2_lo(y0), f2_hi(y0), f2_lo(y1), f2_hi(y1)};
            if (masked) {  // dP of a key that is not there may be NaN
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = 32 * c + e + q >= from ? v[q] : 0.f;
            }
            pk[16 * c + e / 2] = pack_bf16x2(v[0], v[1]);
            pk[16 * c + e / 2 + 1] = pack_bf16x2(v[2], v[3]);
          }
        }
        tmem_st32(p_addr, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&t_full);
      }
      if (!ok) break;
      // Warps 2..5 write dV, warps 6..9 dK (times scale); zeros where no query saw the keys.
      if (n > 0) {
        if (!(ok = wait(&acc_full, nu & 1))) break;
        tc_fence_after();
      }
      const RowOut& o = half ? f.dk : f.dv;
      const float mul = half ? a.scale : 1.f;
      const size_t rows = static_cast<size_t>(a.B) * a.Hk * a.Nk;
      const size_t at = (static_cast<size_t>(w.b) * a.Hk + w.hk) * a.Nk + key;
      float* part = f.part + ((half ? 0 : static_cast<size_t>(a.splits)) + w.split) * rows * D + at * D;
      __nv_bfloat16* out = o.p + w.b * o.sb + w.hk * o.sh + key * o.sn;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t x[32];
        if (n > 0) {
          tmem_ld32(lane_addr + (half ? TK : TV) + c0, x);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = 0u;
        }
        if (key < a.Nk) {
          if (a.splits == 1)
            store_row32(out + c0, x, mul, o.wide);
          else
            store_row32(part + c0, x, mul, true);
        }
        __syncwarp();
      }
      if (n > 0) {
        tc_fence_before();
        mbar_arrive(&acc_free);
        ++nu;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------- dQ

// One persistent CTA per SM, 320 threads, on units of 128 query rows of one head x a range of
// key tiles:
//   warp 0       TMA: Q_i and dO_i once, then K_j and V_j through a ring of two stages
//   warp 1       tcgen05 issuer: S = Q K^T (two TMEM buffers), dP = dO V^T, dQ += T K. S of
//                tile j + 1 and dP of tile j + 1 run while the warps form T of tile j.
//   warps 2..9   thread = query row = TMEM lane; warps 2..5 take the tile's keys 0..63, warps
//                6..9 keys 64..127
// TMEM columns: S ping-pong [0,128) [128,256) (T, bf16, over it: keys 0..63 at +0, 64..127 at
// +64), dP [256,384), dQ [384,384+D).
template <int D>
struct AttendDqSmem {
  static constexpr uint32_t TILE = kTile * D * 2;
  static constexpr int STAGES = 2;
  static constexpr uint32_t total() { return (2 + 2 * STAGES) * TILE + 1024; }
};

struct DqUnit {
  int b, h, row0, split;
  int len, lo, n;  // keys of the sequence; first key tile and key tiles of this unit
};

__device__ __forceinline__ DqUnit dq_unit(const AttendArgs& a, int u, bool record) {
  DqUnit w;
  const int qt = tiles_of(a.Nq);
  w.split = u % a.splits;
  const int t = u / a.splits;
  const int i = t % qt;
  w.row0 = (a.causal ? qt - 1 - i : i) * kTile;  // causal: the longest rows first
  w.b = t / qt / a.H;
  w.h = t / qt % a.H;
  w.len = attend_len(a, w.b, record);
  int hi;
  split_range(tiles_of(attend_key_end(a, w.len, min(w.row0 + kTile, a.Nq) - 1)), a.splits, w.split, w.lo, hi);
  w.n = hi - w.lo;
  return w;
}

template <int D>
__global__ void __launch_bounds__(320, 1)
    attend_dq_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_g,
                     const __grid_constant__ AttendBwdArgs f) {
  using L = AttendDqSmem<D>;
  constexpr int DB = D / 64, ST = L::STAGES;
  constexpr uint32_t TP = 256, TQ = 384;  // TMEM columns of dP and dQ
  const AttendArgs& a = f.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sG = sQ + L::TILE;
  uint8_t* ringK = sG + L::TILE;
  uint8_t* ringV = ringK + ST * L::TILE;

  __shared__ uint64_t q_full, q_free, s_full[2], dp_full, dp_free, t_full[2], acc_full, acc_free, drain;
  __shared__ uint64_t k_full[ST], v_full[ST], k_free[ST], v_free[ST];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_free, 1);
    mbar_init(&dp_full, 1);
    mbar_init(&dp_free, 256);
    mbar_init(&acc_full, 1);
    mbar_init(&acc_free, 256);
    mbar_init(&drain, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&t_full[s], 256);
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&k_free[s], 1);
      mbar_init(&v_free[s], 1);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  grid_dep_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tmap(&map_q);
      prefetch_tmap(&map_k);
      prefetch_tmap(&map_v);
      prefetch_tmap(&map_g);
      uint32_t nk = 0, nv = 0, nu = 0;  // K tiles, V tiles and units loaded
      bool ok = true;
      for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
        const DqUnit w = dq_unit(a, u, true);
        if (w.n <= 0) continue;
        if (nu > 0 && !(ok = mbar_wait(&q_free, (nu - 1) & 1, a.err, &abort_flag))) break;
        mbar_arrive_expect_tx(&q_full, 2 * L::TILE);
        for (int b = 0; b < DB; ++b) tma_load_4d(sQ + b * kBox, &map_q, &q_full, b * 64, w.row0, w.h, w.b);
        for (int b = 0; b < DB; ++b) tma_load_4d(sG + b * kBox, &map_g, &q_full, b * 64, w.row0, w.h, w.b);
        ++nu;
        for (int j = 0; j < w.n; ++j) {
          const int key = (w.lo + j) * kTile;
          const uint32_t s = nk % ST, r = nk / ST;
          if (r > 0 && !(ok = mbar_wait(&k_free[s], (r - 1) & 1, a.err, &abort_flag))) break;
          mbar_arrive_expect_tx(&k_full[s], L::TILE);
          for (int b = 0; b < DB; ++b)
            tma_load_4d(ringK + s * L::TILE + b * kBox, &map_k, &k_full[s], b * 64, key, w.h / a.G, w.b);
          ++nk;
          if (r > 0 && !(ok = mbar_wait(&v_free[s], (r - 1) & 1, a.err, &abort_flag))) break;
          mbar_arrive_expect_tx(&v_full[s], L::TILE);
          for (int b = 0; b < DB; ++b)
            tma_load_4d(ringV + s * L::TILE + b * kBox, &map_v, &v_full[s], b * 64, key, w.h / a.G, w.b);
          ++nv;
        }
      }
      if (abort_flag) {  // let every load still in flight land before the CTA retires
        if (nu > 0) mbar_wait(&q_full, (nu - 1) & 1, nullptr, nullptr);
        for (uint32_t i = nk > ST ? nk - ST : 0; i < nk; ++i) mbar_wait(&k_full[i % ST], (i / ST) & 1, nullptr, nullptr);
        for (uint32_t i = nv > ST ? nv - ST : 0; i < nv; ++i) mbar_wait(&v_full[i % ST], (i / ST) & 1, nullptr, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t q0 = smem_u32(sQ), g0 = smem_u32(sG), rk = smem_u32(ringK), rv = smem_u32(ringV);
    uint32_t it = 0, nu = 0;  // key tiles and units so far
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.err, &abort_flag));
    };
    for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
      const DqUnit w = dq_unit(a, u, false);
      const int n = w.n;
      if (n <= 0) continue;
      auto issue_s = [&](int j) -> bool {
        const uint32_t t = it + j, s = t % ST;
        if (!wait_all(&k_full[s], (t / ST) & 1)) return false;
        const int keys = w.len - (w.lo + j) * kTile;  // real keys of the tile
        if (keys < kTile) zero_rows<D>(ringK + s * L::TILE, keys, kTile);
        tc_fence_after();
        if (elect_one()) {
          issue_ss<D>(tmem + (t & 1) * 128, q0, rk + s * L::TILE);
          umma_commit(&s_full[t & 1]);
        }
        __syncwarp();
        return true;
      };
      auto issue_dp = [&](int j) -> bool {
        const uint32_t t = it + j, s = t % ST;
        if (!wait_all(&v_full[s], (t / ST) & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          issue_ss<D>(tmem + TP, g0, rv + s * L::TILE);
          umma_commit(&dp_full);
          umma_commit(&v_free[s]);
          if (j + 1 == n) umma_commit(&q_free);  // the unit's last reader of Q_i and dO_i
        }
        __syncwarp();
        return true;
      };
      if (!(ok = wait_all(&q_full, nu & 1))) break;
      if (!(ok = issue_s(0))) break;
      // dP's columns: the previous unit's last dP has been read
      if (it > 0 && !(ok = wait_all(&dp_free, (it - 1) & 1))) break;
      if (!(ok = issue_dp(0))) break;
      for (int j = 0; j < n; ++j) {
        const uint32_t t = it + j, s = t % ST;
        if (j + 1 < n) {
          if (!(ok = issue_s(j + 1))) break;
          if (!(ok = wait_all(&dp_free, t & 1))) break;
          tc_fence_after();
          if (!(ok = issue_dp(j + 1))) break;
        }
        if (j == 0 && nu > 0 && !(ok = wait_all(&acc_free, (nu - 1) & 1))) break;
        if (!(ok = wait_all(&t_full[t & 1], (t >> 1) & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          issue_ts<D, 64>(tmem + TQ, tmem + (t & 1) * 128, rk + s * L::TILE, j > 0);
          umma_commit(&k_free[s]);
          if (j + 1 == n) umma_commit(&acc_full);
        }
        __syncwarp();
      }
      it += n;
      ++nu;
    }
    if (elect_one()) umma_commit(&drain);
    __syncwarp();
    mbar_wait(&drain, 0, nullptr, nullptr);
  } else {
    // ------------------------------------------------------------ T, then the epilogue
    const int half = warp >= 6;
    const int r = (warp & 3) * 32 + lane;  // query row of the tile = TMEM lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float sc = a.scale_log2;
    const uint64_t sc2 = f2_make(sc, sc);
    uint32_t it = 0, nu = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.err, &abort_flag));
    };
    for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
      const DqUnit w = dq_unit(a, u, false);
      const int n = w.n;
      const int row = w.row0 + r;
      const int end = attend_key_end(a, w.len, row);
      const size_t at = (static_cast<size_t>(w.b) * a.H + w.h) * f.pad + row;
      const float nl = f.nlse[at], nd = f.ndelta[at];
      const uint64_t nl2 = f2_make(nl, nl), nd2 = f2_make(nd, nd);
      for (int j = 0; j < n; ++j, ++it) {
        const int key0 = (w.lo + j) * kTile + half * 64;
        const int upto = end - key0;  // columns of this half that the row sees
        const bool masked = __any_sync(0xffffffffu, upto < 64);
        const uint32_t s_addr = lane_addr + (it & 1) * 128 + half * 64;
        if (!(ok = wait(&s_full[it & 1], (it >> 1) & 1))) break;
        tc_fence_after();
        uint32_t p[2][32], d[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(s_addr + 32 * c, p[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t x = f2_fma(pair_of(&p[c][e]), sc2, nl2);
            p[c][e] = __float_as_uint(fast_exp2(f2_lo(x)));
            p[c][e + 1] = __float_as_uint(fast_exp2(f2_hi(x)));
          }
        }
        if (!(ok = wait(&dp_full, it & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(lane_addr + TP + half * 64 + 32 * c, d[c]);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(&dp_free);
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t y = f2_mul(f2_add(pair_of(&d[c][e]), nd2), pair_of(&p[c][e]));
            float v[2] = {f2_lo(y), f2_hi(y)};
            if (masked) {
#pragma unroll
              for (int q = 0; q < 2; ++q) v[q] = 32 * c + e + q < upto ? v[q] : 0.f;
            }
            pk[16 * c + e / 2] = pack_bf16x2(v[0], v[1]);
          }
        }
        tmem_st32(s_addr, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&t_full[it & 1]);
      }
      if (!ok) break;
      if (n > 0) {
        if (!(ok = wait(&acc_full, nu & 1))) break;
        tc_fence_after();
      }
      // scale times the accumulator: warps 2..5 its first D / 2 channels, warps 6..9 the rest
      const size_t rows = static_cast<size_t>(a.B) * a.H * a.Nq;
      const size_t o = (static_cast<size_t>(w.b) * a.H + w.h) * a.Nq + row;
#pragma unroll 1
      for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
        uint32_t x[32];
        if (n > 0) {
          tmem_ld32(lane_addr + TQ + c0, x);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = 0u;
        }
        if (row < a.Nq) {
          if (a.splits == 1)
            store_row32(f.dq.p + w.b * f.dq.sb + w.h * f.dq.sh + row * f.dq.sn + c0, x, a.scale, f.dq.wide);
          else
            store_row32(f.part + (w.split * rows + o) * D + c0, x, a.scale, true);
        }
        __syncwarp();
      }
      if (n > 0) {
        tc_fence_before();
        mbar_arrive(&acc_free);
        ++nu;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Sum of the splits' fp32 rows in ascending order, rounded once: out [B, H, N, D].
struct AttendSumArgs {
  const float* part;  // [splits][rows][D]
  int splits, H, N;
  long long rows;     // B * H * N
  RowOut out;
};

template <int D>
__global__ void __launch_bounds__(256) attend_sum_kernel(AttendSumArgs a) {
  constexpr int T = D / 8;
  const long long i = static_cast<long long>(blockIdx.x) * (256 / T) + threadIdx.x / T;
  const int c = (threadIdx.x % T) * 8;
  grid_dep_wait();
  if (i >= a.rows) return;
  float s[8] = {};
  for (int k = 0; k < a.splits; ++k) {
    const float4* p = reinterpret_cast<const float4*>(a.part + (k * a.rows + i) * D + c);
    const float4 x = p[0], y = p[1];
    s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w, s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
  }
  const long long bh = i / a.N;
  *reinterpret_cast<uint4*>(a.out.p + (bh / a.H) * a.out.sb + (bh % a.H) * a.out.sh + (i % a.N) * a.out.sn + c) =
      make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7]));
}

}  // namespace sla
