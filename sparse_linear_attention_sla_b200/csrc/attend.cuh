// Dense attention forward: out = softmax(scale q k^T) v over the keys a query may see, and the
// log-sum-exp of every row.
//
// The exact softmax attention of the sparse branch ("SLA: Beyond Sparsity in Diffusion
// Transformers via Fine-Tunable Sparse-Linear Attention", Abstract: exact attention for the
// critical weights) over all keys: with its own number of keys, lengths per sequence, shared
// key heads and a causal mask, as cross attention and token models need it.
//
// Math: one pass over the keys with a running reference m and sum l of each row:
//   p = 2^(s scale log2(e) - m), l += sum p, acc += p v;  out = acc / l, lse = (m + log2 l) ln 2.
// m is the row maximum of the first tile with a visible key and moves (acc and l rescaled)
// only when a tile's sum passes 2^20, as in the sparse kernels. P is rounded to bf16 for the
// tensor cores (each p by at most 2^-8 of itself, independently; l sums the unrounded p);
// S, acc, m and l are fp32. A row without keys gives out = 0 and lse = -inf.
//
// One persistent CTA per SM, 320 threads, on units of 256 query rows of one head (two tiles A
// and B of 128 rows) x a range of 128-key tiles:
//   warp 0       TMA: Q tiles, then K_j and V_j through a ring of five tiles
//   warp 1       TMEM owner and tcgen05 issuer: S_x = Q_x K_j^T, acc_x += P_x V_j. While
//                tile A's warps turn S into P, the tensor cores run tile B's products.
//   warps 2..5   softmax of tile A; warps 6..9 of tile B: thread = query row = TMEM lane
// TMEM columns: S_A [0,128) S_B [128,256) (P, bf16, over the first 64 of its S), acc_A
// [256,256+D), acc_B [384,384+D). MMAs of one thread run in issue order, so S_{j+1} never
// overwrites P_j before the product that reads it.
// With few units the key tiles of a unit are split over several CTAs, which write fp32 rows
// and log2-sums that attend_join_kernel joins in a fixed order.
#pragma once

#include "attend_common.cuh"
#include "softmax_block.cuh"

namespace sla {

template <int D>
struct AttendSmem {
  static constexpr uint32_t TILE = kTile * D * 2;
  static constexpr int STAGES = D == 128 ? 5 : 8;
  static constexpr uint32_t total() { return (2 + STAGES) * TILE + 1024; }
};

struct AttendFwdArgs {
  AttendArgs p;
  RowOut out;
  float* lse;        // [B * H, Nq]
  float* part;       // splits > 1: [splits][B * H * Nq][D] rows, each already divided by its l
  float* part_lse2;  // [splits][B * H * Nq] log2 of the part's sum, m included
};

struct AttendUnit {
  int b, h, row0, split;
  int len;
  int lo, n[2];  // first key tile, key tiles of tile A and of tile B in this unit
};

__device__ __forceinline__ AttendUnit attend_unit(const AttendArgs& a, int u, bool record) {
  AttendUnit w;
  const int pairs = (a.Nq + 2 * kTile - 1) / (2 * kTile);
  w.split = u % a.splits;
  const int t = u / a.splits;
  const int pr = t % pairs, bh = t / pairs;
  w.b = bh / a.H;
  w.h = bh % a.H;
  w.row0 = (a.causal ? pairs - 1 - pr : pr) * 2 * kTile;  // causal: the longest rows first
  w.len = attend_len(a, w.b, record);
  int all[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = w.row0 + x * kTile;
    all[x] = r < a.Nq ? tiles_of(attend_key_end(a, w.len, min(r + kTile, a.Nq) - 1)) : 0;
  }
  int hi;
  split_range(max(all[0], all[1]), a.splits, w.split, w.lo, hi);
#pragma unroll
  for (int x = 0; x < 2; ++x) w.n[x] = max(0, min(hi, all[x]) - w.lo);
  return w;
}

// Keys of 32 columns from key0 on that a row does not see (its keys end at `end`) take -inf.
__device__ __forceinline__ void mask_cols32(uint32_t (&x)[32], int key0, int end) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (key0 + c >= end) x[c] = __float_as_uint(-INFINITY);
}

template <int D>
__global__ void __launch_bounds__(320, 1)
    attend_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ AttendFwdArgs f) {
  using L = AttendSmem<D>;
  constexpr int DB = D / 64, ST = L::STAGES;
  constexpr uint32_t ACC = 256;
  const AttendArgs& a = f.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* ring = sQ + 2 * L::TILE;

  __shared__ uint64_t q_full[2], q_free[2], s_full[2], p_full[2], pv_done[2], acc_free[2];
  __shared__ uint64_t full[ST], empty[ST];
  __shared__ uint64_t drain;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_free[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 128);
      mbar_init(&pv_done[x], 1);
      mbar_init(&acc_free[x], 128);
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&drain, 1);
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
      uint32_t nr = 0, nq[2] = {0, 0};  // ring tiles and Q tiles loaded
      bool ok = true;
      auto load_q = [&](const AttendUnit& w, int x) {
        if (w.n[x] == 0) return;
        if (nq[x] > 0 && !(ok = mbar_wait(&q_free[x], (nq[x] - 1) & 1, a.err, &abort_flag))) return;
        mbar_arrive_expect_tx(&q_full[x], L::TILE);
        for (int b = 0; b < DB; ++b)
          tma_load_4d(sQ + x * L::TILE + b * kBox, &map_q, &q_full[x], b * 64, w.row0 + x * kTile, w.h, w.b);
        ++nq[x];
      };
      auto load = [&](const CUtensorMap* m, const AttendUnit& w, int j) {
        const uint32_t s = nr % ST, r = nr / ST;
        if (r > 0 && !(ok = mbar_wait(&empty[s], (r - 1) & 1, a.err, &abort_flag))) return;
        mbar_arrive_expect_tx(&full[s], L::TILE);
        for (int b = 0; b < DB; ++b)
          tma_load_4d(ring + s * L::TILE + b * kBox, m, &full[s], b * 64, j * kTile, w.h / a.G, w.b);
        ++nr;
      };
      for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
        const AttendUnit w = attend_unit(a, u, true);
        const int n = max(w.n[0], w.n[1]);
        if (n == 0) continue;
        load_q(w, 0);
        if (ok) load(&map_k, w, w.lo);
        if (ok) load_q(w, 1);
        for (int j = 0; ok && j < n; ++j) {
          load(&map_v, w, w.lo + j);
          if (ok && j + 1 < n) load(&map_k, w, w.lo + j + 1);
        }
      }
      if (abort_flag) {  // let every load still in flight land before the CTA retires
        for (int x = 0; x < 2; ++x)
          if (nq[x] > 0) mbar_wait(&q_full[x], (nq[x] - 1) & 1, nullptr, nullptr);
        for (uint32_t i = nr > ST ? nr - ST : 0; i < nr; ++i)
          mbar_wait(&full[i % ST], (i / ST) & 1, nullptr, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t q0 = smem_u32(sQ), r0 = smem_u32(ring);
    uint32_t nr = 0, nu[2] = {0, 0}, np[2] = {0, 0};  // ring tiles, units and P tiles consumed
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.err, &abort_flag));
    };
    for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
      const AttendUnit w = attend_unit(a, u, false);
      const int n = max(w.n[0], w.n[1]);
      if (n == 0) continue;
      // S of key tile j (0-based in the unit) from ring stage sk, for query tile x.
      auto issue_s = [&](int x, int j, uint32_t sk) {
        if (elect_one()) {
          issue_ss<D>(tmem + x * 128, q0 + x * L::TILE, r0 + sk * L::TILE);
          umma_commit(&s_full[x]);
          if (j + 1 == w.n[x]) umma_commit(&q_free[x]);
        }
        __syncwarp();
      };
      uint32_t sk = nr % ST;
      if (!(ok = wait_all(&full[sk], (nr / ST) & 1))) break;
      ++nr;
      for (int x = 0; x < 2 && ok; ++x) {
        if (w.n[x] == 0) continue;
        if (!(ok = wait_all(&q_full[x], nu[x] & 1))) break;
        tc_fence_after();
        issue_s(x, 0, sk);
      }
      if (!ok) break;
      if (elect_one()) umma_commit(&empty[sk]);
      __syncwarp();
      for (int j = 0; ok && j < n; ++j) {
        const uint32_t sv = nr % ST;
        if (!(ok = wait_all(&full[sv], (nr / ST) & 1))) break;
        ++nr;
        const int keys = w.len - (w.lo + j) * kTile;  // real keys of the tile
        if (keys < kTile) zero_rows<D>(ring + sv * L::TILE, keys, kTile);
        const bool more = j + 1 < n;
        if (more) {
          sk = nr % ST;
          if (!(ok = wait_all(&full[sk], (nr / ST) & 1))) break;
          ++nr;
        }
        for (int x = 0; x < 2; ++x) {
          if (j >= w.n[x]) continue;
          if (j == 0 && nu[x] > 0 && !(ok = wait_all(&acc_free[x], (nu[x] - 1) & 1))) break;
          if (!(ok = wait_all(&p_full[x], np[x] & 1))) break;
          ++np[x];
          tc_fence_after();
          if (elect_one()) {
            issue_ts<D, 32>(tmem + ACC + x * 128, tmem + x * 128, r0 + sv * L::TILE, j > 0);
            umma_commit(&pv_done[x]);
          }
          __syncwarp();
          if (j + 1 < w.n[x]) issue_s(x, j + 1, sk);
        }
        if (!ok) break;
        if (elect_one()) {
          umma_commit(&empty[sv]);
          if (more) umma_commit(&empty[sk]);
        }
        __syncwarp();
      }
      for (int x = 0; x < 2; ++x) nu[x] += w.n[x] > 0;
    }
    if (elect_one()) umma_commit(&drain);  // every MMA issued above has finished once this arrives
    __syncwarp();
    mbar_wait(&drain, 0, nullptr, nullptr);
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    const int x = warp >= 6;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + x * 128, o_addr = lane_addr + ACC + x * 128;
    const float sc = a.scale_log2;
    const uint64_t sc2 = f2_make(sc, sc);
    uint32_t ns = 0;  // S tiles so far
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.err, &abort_flag));
    };
    for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
      const AttendUnit w = attend_unit(a, u, false);
      const int row = w.row0 + x * kTile + r;
      const int n = w.n[x];
      const int end = attend_key_end(a, w.len, row);                          // this row's keys
      const int end_min = attend_key_end(a, w.len, w.row0 + x * kTile);       // of the tile's first row
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++ns) {
        if (!(ok = wait(&s_full[x], ns & 1))) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + 32 * c, s[c]);
        tmem_wait_ld();
        const int key0 = (w.lo + j) * kTile;
        if (key0 + kTile > end_min) {
#pragma unroll
          for (int c = 0; c < 4; ++c) mask_cols32(s[c], key0 + 32 * c, end);
        }
        if (__any_sync(0xffffffffu, m == -INFINITY)) {
          const float t = fmaxf(row_max64(s[0], s[1]), row_max64(s[2], s[3])) * sc;
          if (m == -INFINITY) m = t;
        }
        float sum;
        auto exponentials = [&]() {
          const float ref = m == -INFINITY ? 0.f : m;  // no key seen yet: every s is -inf
          const uint64_t nm2 = f2_make(-ref, -ref);
          uint64_t part = 0ull;
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            uint32_t pk[32];
            part = f2_add(part, exp2_block(s[c], s[c + 1], pk, sc2, nm2));
            tmem_st32(s_addr + 16 * c, pk);
          }
          sum = f2_lo(part) + f2_hi(part);
        };
        exponentials();
        if (__any_sync(0xffffffffu, sum > kRefMoveSum)) {
          const float t = fmaxf(m, fmaxf(row_max64(s[0], s[1]), row_max64(s[2], s[3])) * sc);
          const float g = m == -INFINITY ? 1.f : fast_exp2(m - t);
          if (j > 0) {
            if (!(ok = wait(&pv_done[x], (ns - 1) & 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t o[16];
              tmem_ld16(o_addr + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * g);
              tmem_st16(o_addr + c0, o);
            }
          }
          tmem_wait_st();
          l *= g;
          m = t;
          exponentials();
        }
        l += sum;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      // acc / l as bf16, or as a part's fp32 row with its log2-sum
      if (n > 0) {
        if (!(ok = wait(&pv_done[x], (ns - 1) & 1))) break;
        tc_fence_after();
      }
      const bool real = row < a.Nq;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const float lse2 = l > 0.f ? m + __log2f(l) : -INFINITY;
      const size_t at = (static_cast<size_t>(w.b) * a.H + w.h) * a.Nq + row;
      const size_t rows = static_cast<size_t>(a.B) * a.H * a.Nq;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(o_addr + c0, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0u;
        }
        if (l == 0.f) {  // nothing was seen: acc holds no number to keep
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0u;
        }
        if (real) {
          if (a.splits == 1)
            store_row32(f.out.p + w.b * f.out.sb + w.h * f.out.sh + row * f.out.sn + c0, o, inv, f.out.wide);
          else
            store_row32(f.part + (w.split * rows + at) * D + c0, o, inv, true);
        }
        __syncwarp();
      }
      if (real) {
        if (a.splits == 1)
          f.lse[at] = lse2 * 0.69314718055994531f;
        else
          f.part_lse2[w.split * rows + at] = lse2;
      }
      if (n > 0) {
        tc_fence_before();
        mbar_arrive(&acc_free[x]);
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

// out = sum_s 2^(lse2_s - lse2) part_s in ascending s, one warp per row.
template <int D>
__global__ void __launch_bounds__(256) attend_join_kernel(AttendFwdArgs f) {
  const AttendArgs& a = f.p;
  const size_t rows = static_cast<size_t>(a.B) * a.H * a.Nq;
  const size_t at = static_cast<size_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  constexpr int E = D / 32;
  grid_dep_wait();
  if (at >= rows) return;
  float m = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) m = fmaxf(m, f.part_lse2[s * rows + at]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  float sum = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float w = exp2f(f.part_lse2[s * rows + at] - ref);
    sum += w;
    const float* p = f.part + (s * rows + at) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, p[e], acc[e]);
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int row = static_cast<int>(at % a.Nq);
  const size_t bh = at / a.Nq;
  __nv_bfloat16* out = f.out.p + (bh / a.H) * f.out.sb + (bh % a.H) * f.out.sh + row * f.out.sn + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(out + e) = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) f.lse[at] = sum > 0.f ? (m + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace sla
