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
// delta is taken from out as it was given, in bf16 and with P rounded. Over many keys that is no matter; of two keys'
// gradients it would be half of the error (0.0054 instead of 0.0024 of their norm, in bf16). Where a
// sequence's keys fit one tile, the dQ kernel has a row's P and dP at hand and forms delta = sum_j P dP
// itself, for the dK / dV kernel too, which then runs after it. The first queries of longer causal sequences, which
// see no more keys than one tile's, have it so for dQ alone: the dK / dV kernel would have to wait.
//
// P and T are rounded to bf16 for the tensor cores (by at most 2^-8 of each value); S, dP,
// delta, lse and every sum are fp32. Rows without keys have lse = -inf: their P is 0, and
// delta is taken as 0.
#pragma once

#include "attend_common.cuh"

namespace sla {

// A warpgroup for the TMA and MMA warps and four that compute, a quarter of the tile's columns each: the
// exponentials are bound by latency where a scheduler has only two warps to hide it with. Gradients of self
// attention over 8192 tokens, 12 heads: forward and backward 1786 us with four, 1806 with two (causal, 4096
// tokens: 169 and 174), timed in turn.
constexpr int kBwdWarps = 16, kBwdThreads = 128 + 32 * kBwdWarps;

struct AttendBwdArgs {
  AttendArgs p;
  const float* nlse;    // [B * H, pad] -lse2 (padding rows and rows without keys: -inf)
  float* ndelta;        // [B * H, pad] -delta (written by the dQ kernel for sequences of one key tile)
  int dq_first;         // the dQ kernel runs before the dK / dV kernel, and forms such deltas
  int pad;              // Nq rounded up to whole tiles
  RowOut dq, dk, dv;
  float* part;          // parts of units (see AttendWork): dQ [2 * CTAs][128][D], or [2 * CTAs][dK, dV][128][D]
};

// -lse2 and -delta of every row, 8 channels a lane, kRowsUnroll rows a thread so that their loads
// are in flight together. Reads out and dO once (bound by HBM).
struct AttendRowsArgs {
  int H, Nq, pad;
  const __nv_bfloat16 *out, *dO;
  long long ob, oh, on, gb, gh, gn;
  const float* lse;
  float *nlse, *ndelta;
};

constexpr int kRowsUnroll = 4;

template <int D>
__global__ void __launch_bounds__(256) attend_rows_kernel(AttendRowsArgs a) {
  constexpr int T = D / 8, U = kRowsUnroll;  // lanes of a row
  // A block's rows are of one head (pad is a multiple of 128).
  const int per_head = a.pad / (256 / T * U), bh = blockIdx.x / per_head;
  const int row0 = blockIdx.x % per_head * (256 / T * U) + threadIdx.x / T;
  const int c = (threadIdx.x % T) * 8;
  grid_dep_wait();
  grid_dep_launch();
  const int b = bh / a.H, h = bh % a.H;
  const __nv_bfloat16* const out = a.out + b * a.ob + h * a.oh + c;
  const __nv_bfloat16* const dO = a.dO + b * a.gb + h * a.gh + c;
  uint4 x[U], y[U];
  float nl[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = row0 + u * (256 / T);
    x[u] = y[u] = make_uint4(0, 0, 0, 0);
    nl[u] = -INFINITY;
    if (row < a.Nq) {
      nl[u] = -a.lse[static_cast<size_t>(bh) * a.Nq + row] * 1.4426950408889634f;
      x[u] = *reinterpret_cast<const uint4*>(out + row * a.on);
      y[u] = *reinterpret_cast<const uint4*>(dO + row * a.gn);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float sum = 0.f;
    if (nl[u] == INFINITY) {  // a row without keys: its dO may hold anything
      nl[u] = -INFINITY;
    } else {
      const uint32_t xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, ys[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 p = unpack_bf16x2(xs[k]), q = unpack_bf16x2(ys[k]);
        sum = fmaf(p.x, q.x, fmaf(p.y, q.y, sum));
      }
    }
#pragma unroll
    for (int o = T / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (c == 0) {
      const size_t i = static_cast<size_t>(bh) * a.pad + row0 + u * (256 / T);
      a.nlse[i] = nl[u];
      a.ndelta[i] = -sum;
    }
  }
}

// Two neighbouring columns as a pair for the paired arithmetic.
__device__ __forceinline__ uint64_t pair_of(const uint32_t* x) {
  return static_cast<uint64_t>(x[0]) | (static_cast<uint64_t>(x[1]) << 32);
}

// Two pairs from shared memory, as a shared load (a generic one waits in the queue of global accesses).
__device__ __forceinline__ ulonglong2 load_shared16(uint32_t addr) {
  ulonglong2 v;
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(addr));
  return v;
}

// Of 32 columns those before `from` (or, keep_upto, from `upto` on) take `value`.
__device__ __forceinline__ void keep_from(uint32_t (&x)[32], int from, float value) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (c < from) x[c] = __float_as_uint(value);
}
__device__ __forceinline__ void keep_upto(uint32_t (&x)[32], int upto, float value) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (c >= upto) x[c] = __float_as_uint(value);
}

// ---------------------------------------------------------------------------- dK, dV

// One persistent CTA per SM, 640 threads, on units of 128 keys of one key head, a step being a
// (query head of the group, query tile) that sees them:
//   warp 0       TMA: K_j and V_j once, then Q_i, dO_i and the rows' statistics through a ring
//                of two stages
//   warps 1, 3   tcgen05 issuers: S^T = K Q^T and dV += P^T dO; dP^T = V dO^T and dK += T^T Q. While the
//                warps form P of tile i the tensor cores run dK of tile i - 1 and dP of tile i;
//                while they form T, dV of tile i and S of tile i + 1.
//   warp 2       scheduler: the CTA's units
//   warps 4..19  thread = key row = TMEM lane; each warpgroup takes 32 of the tile's queries
// TMEM columns: S^T [0,128) and dP^T [128,256), each overwritten by its bf16 result (32
// queries' S by 16 columns, so that each warpgroup overwrites only what it has read); dV [256,256+D), dK [384,384+D).
template <int D>
struct AttendDkvSmem {
  static constexpr uint32_t TILE = kTile * D * 2;
  static constexpr uint32_t STATS = 2 * kTile * 4;
  static constexpr uint32_t STAGE = 2 * TILE;
  static constexpr int STAGES = 2;
  static constexpr uint32_t total() { return 2 * TILE + STAGES * (STAGE + STATS) + 1024; }
};

struct DkvUnit {
  int b, hk, key0;
  int len, first;  // keys of the sequence; first query tile that sees a key of the tile
  int tiles;       // query tiles per head from there on
  int dead;        // queries before this row see no key (causal, more queries than keys)
};

__device__ __forceinline__ DkvUnit dkv_unit(const AttendArgs& a, int u, bool record) {
  DkvUnit w;
  const int kt = tiles_of(a.Nk);
  w.key0 = u % kt * kTile;
  w.b = u / kt / a.Hk;
  w.hk = u / kt % a.Hk;
  w.len = attend_len(a, w.b, record);
  w.dead = a.causal ? max(0, a.Nq - w.len) : 0;
  const int first_row = a.causal ? max(0, w.key0 - (w.len - a.Nq)) : 0;  // sees key0, causal
  w.first = first_row / kTile;
  w.tiles = w.key0 < w.len && first_row < a.Nq ? tiles_of(a.Nq) - w.first : 0;
  return w;
}

// What the warps need of the current unit: n steps from lo on.
struct DkvItem {
  int b, hk, key0, len, first, tiles, dead, lo, n, slot;
  __device__ __forceinline__ explicit DkvItem(const AttendItem& i)
      : b(i.v[0]), hk(i.v[1]), key0(i.v[2]), len(i.v[3]), first(i.v[4]), tiles(i.v[5]), dead(i.v[6]), lo(i.v[7]),
        n(tiles > 0 ? i.v[8] - lo : 0), slot(i.v[9]) {}
  __device__ __forceinline__ bool stop() const { return b < 0; }
};

template <int ST>
struct DkvBarriers {
  uint64_t kv_full, kv_free, s_full, dp_full, p_full, t_full, acc_full[2], acc_free[2], drain;  // [dV, dK]
  uint64_t q_full[ST], g_full[ST], q_free[ST], g_free[ST];
  int abort_flag;
};

// One of the two MMA warps. Y = 0: S^T(i) = K Q_i^T, then dV += P(i)^T dO_i. Y = 1: dP^T(i) = V dO_i^T, then
// dK += T(i)^T Q_i. Each chain's own order keeps S^T(i + 1) from overwriting P(i), and dP^T(i + 1) T(i).
// What a product needs besides P or T is looked up before P or T is waited for.
template <int D, int Y>
__device__ __forceinline__ void attend_dkv_issue(DkvBarriers<AttendDkvSmem<D>::STAGES>& sh, ItemRing<kBwdWarps>& items,
                                                 const AttendBwdArgs& f, uint8_t* kv, uint8_t* ring) {
  using L = AttendDkvSmem<D>;
  constexpr int ST = L::STAGES;
  constexpr uint32_t col = Y ? 128 : 0, acc = Y ? 384 : 256;          // TMEM columns of the products
  constexpr uint32_t one = Y ? L::TILE : 0, two = Y ? 0 : L::TILE;    // their tiles in a stage
  uint64_t *const full1 = Y ? sh.g_full : sh.q_full, *const free1 = Y ? sh.g_free : sh.q_free;
  uint64_t *const full2 = Y ? sh.q_full : sh.g_full, *const free2 = Y ? sh.q_free : sh.g_free;
  uint64_t *const made = Y ? &sh.dp_full : &sh.s_full, *const formed = Y ? &sh.t_full : &sh.p_full;
  const uint32_t a0 = smem_u32(kv), r0 = smem_u32(ring);
  uint32_t nu = 0, ni = 0, done = 0;  // units with work, items, parity of the next P or T
  RingPos pos;                        // of the first product's tile
  bool ok = true;
  AttendItem item;
  const uint32_t lead = elect_one();
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return warp_wait(bar, parity, f.p.err, &sh.abort_flag); };
  auto issue_first = [&](bool last) {
    issue_ss<D, 128>(lead, col, a0, r0 + pos.s * L::STAGE + one);
    mma_commit(lead, made);
    mma_commit(lead, &free1[pos.s]);
    if (last) mma_commit(lead, &sh.kv_free);  // the unit's last reader of K_j or V_j
    pos.next(ST);
  };
  while (ok) {
    if (!(ok = items.get(ni++, item, f.p.err, &sh.abort_flag))) break;
    const DkvItem w(item);
    if (w.stop()) break;
    const int n = w.n;
    if (n == 0) continue;
    if (!(ok = wait(&sh.kv_full, nu & 1))) break;
    RingPos cur = pos;  // of the second product's tile
    if (!(ok = wait(&full1[pos.s], pos.parity))) break;
    tc_fence_after();
    issue_first(n == 1);
    if (nu > 0 && !(ok = wait(&sh.acc_free[Y], (nu - 1) & 1))) break;
    int i_tile = w.lo % w.tiles;
    for (int i = 0; i < n; ++i) {
      uint8_t* tile = ring + cur.s * L::STAGE + two;
      if (!(ok = wait(&full2[cur.s], cur.parity))) break;
      // Rows that see no key may hold anything: zero them where the product sums over rows.
      const int row = (w.first + i_tile) * kTile;
      if (row < w.dead) zero_rows<D>(tile, 0, min(kTile, w.dead - row));
      if (++i_tile == w.tiles) i_tile = 0;
      if (i + 1 < n && !(ok = wait(&full1[pos.s], pos.parity))) break;
      if (!(ok = wait(formed, done))) break;
      done ^= 1;
      tc_fence_after();
      issue_ts<D, 0, 8, 2, 32>(lead, acc, col, smem_u32(tile), i > 0);
      mma_commit(lead, &free2[cur.s]);
      if (i + 1 == n) mma_commit(lead, &sh.acc_full[Y]);
      cur.next(ST);
      if (i + 1 < n) issue_first(i + 2 == n);
    }
    ++nu;
  }
  mma_commit(lead, &sh.drain);
  mbar_wait(&sh.drain, 0, nullptr, nullptr);
}

template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attend_dkv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_g,
                      const __grid_constant__ AttendBwdArgs f) {
  using L = AttendDkvSmem<D>;
  constexpr int DB = D / 64, ST = L::STAGES;
  constexpr uint32_t TP = 128, TV = 256, TK = 384;  // TMEM columns of dP^T, dV, dK
  const AttendArgs& a = f.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sK = base;
  uint8_t* sV = sK + L::TILE;
  uint8_t* ring = sV + L::TILE;                                           // Q then dO
  float* stats = reinterpret_cast<float*>(ring + ST * L::STAGE);          // nlse[128] then ndelta[128]

  __shared__ DkvBarriers<ST> sh;
  __shared__ uint32_t tmem_base_sh;
  __shared__ ItemRing<kBwdWarps> items;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&sh.kv_full, 1);
    mbar_init(&sh.kv_free, 2);
    mbar_init(&sh.s_full, 1);
    mbar_init(&sh.dp_full, 1);
    mbar_init(&sh.p_full, kBwdWarps);
    mbar_init(&sh.t_full, kBwdWarps);
    mbar_init(&sh.acc_full[0], 1);
    mbar_init(&sh.acc_full[1], 1);
    mbar_init(&sh.acc_free[0], 256);
    mbar_init(&sh.acc_free[1], 256);
    mbar_init(&sh.drain, 2);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&sh.q_full[s], 1);
      mbar_init(&sh.g_full[s], 1);
      mbar_init(&sh.q_free[s], 2);
      mbar_init(&sh.g_free[s], 2);
    }
    items.init();
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  // Behind attend_dq_kernel this one needs its deltas, but only of sequences of one key tile; without such it runs
  // beside that kernel where SMs are free (see there), and waits last.
  bool late = false;
  if (f.dq_first && a.lens) {
    int one_tile = 0;
    for (int b = tid; b < a.B; b += kBwdThreads) one_tile |= attend_len(a, b, false) <= kTile;
    late = !__syncthreads_or(one_tile);
  }
  if (!late) grid_dep_wait();
  grid_dep_launch();
  const auto steps = [&](int u) { return dkv_unit(a, u, false).tiles * a.G; };
  AttendWork work = attend_work(a, steps, kBwdThreads);
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all columns are allocated
  AttendItem item;

  if (warp == kScheduleWarp) {
    if (lane == 0) {
      uint32_t ni = 0;
      int u, lo, hi, n, to, longest = 0;  // steps of the longest item
      bool ok = true;
      DkvUnit w;  // the unit that `next` looked at last, which is the one it gives
      const auto look = [&](int v) {
        w = dkv_unit(a, v, true);
        return w.tiles * a.G;
      };
      while (ok && work.next(a, look, u, lo, hi, n, to)) {
        note_part(a, work, u, lo, hi, n, to);
        item = {w.b, w.hk, w.key0, w.len, w.first, w.tiles, w.dead, lo, hi, part_slot(lo, hi, n)};
        longest = max(longest, hi - lo);
        ok = items.put(ni++, item, longest, a.err, &sh.abort_flag);
      }
      item.v[0] = -1;
      if (ok) items.put(ni, item, longest, a.err, &sh.abort_flag);
    }
    __syncwarp();
  } else if (warp == kProducerWarp) {
    // ------------------------------------------------------------ TMA producer
    uint32_t ni = 0;
    if (lane == 0) {
      prefetch_tmap(&map_q);
      prefetch_tmap(&map_k);
      prefetch_tmap(&map_v);
      prefetch_tmap(&map_g);
      uint32_t nr = 0, nu = 0, ng = 0;  // Q tiles, units and dO tiles loaded
      bool ok = true;
      while (ok) {
        if (!(ok = items.get_one(ni++, item, a.err, &sh.abort_flag))) break;
        const DkvItem w(item);
        if (w.stop()) break;
        if (w.n == 0) continue;
        if (nu > 0 && !(ok = mbar_wait(&sh.kv_free, (nu - 1) & 1, a.err, &sh.abort_flag))) break;
        mbar_arrive_expect_tx(&sh.kv_full, 2 * L::TILE);
        for (int b = 0; b < DB; ++b) tma_load_4d(sK + b * kBox, &map_k, &sh.kv_full, b * 64, w.key0, w.hk, w.b);
        for (int b = 0; b < DB; ++b) tma_load_4d(sV + b * kBox, &map_v, &sh.kv_full, b * 64, w.key0, w.hk, w.b);
        ++nu;
        for (int i = w.lo; i < w.lo + w.n; ++i) {
          const int h = w.hk * a.G + i / w.tiles, row = (w.first + i % w.tiles) * kTile;
          const uint32_t s = nr % ST, r = nr / ST;
          if (r > 0 && !(ok = mbar_wait(&sh.q_free[s], (r - 1) & 1, a.err, &sh.abort_flag))) break;
          const size_t at = (static_cast<size_t>(w.b) * a.H + h) * f.pad + row;
          uint8_t* stage = ring + s * L::STAGE;
          float* st = stats + s * 2 * kTile;
          mbar_arrive_expect_tx(&sh.q_full[s], L::TILE + L::STATS);
          for (int b = 0; b < DB; ++b) tma_load_4d(stage + b * kBox, &map_q, &sh.q_full[s], b * 64, row, h, w.b);
          bulk_load(st, f.nlse + at, &sh.q_full[s], kTile * 4);
          bulk_load(st + kTile, f.ndelta + at, &sh.q_full[s], kTile * 4);
          ++nr;
          if (r > 0 && !(ok = mbar_wait(&sh.g_free[s], (r - 1) & 1, a.err, &sh.abort_flag))) break;
          mbar_arrive_expect_tx(&sh.g_full[s], L::TILE);
          for (int b = 0; b < DB; ++b)
            tma_load_4d(stage + L::TILE + b * kBox, &map_g, &sh.g_full[s], b * 64, row, h, w.b);
          ++ng;
        }
      }
      if (sh.abort_flag) {  // let every load still in flight land before the CTA retires
        if (nu > 0) mbar_wait(&sh.kv_full, (nu - 1) & 1, nullptr, nullptr);
        for (uint32_t i = nr > ST ? nr - ST : 0; i < nr; ++i) mbar_wait(&sh.q_full[i % ST], (i / ST) & 1, nullptr, nullptr);
        for (uint32_t i = ng > ST ? ng - ST : 0; i < ng; ++i) mbar_wait(&sh.g_full[i % ST], (i / ST) & 1, nullptr, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kMmaWarp2) {
    // ------------------------------------------------------------ MMA issuers
    if (warp == kMmaWarp)
      attend_dkv_issue<D, 0>(sh, items, f, sK, ring);
    else
      attend_dkv_issue<D, 1>(sh, items, f, sV, ring);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ P and T, then the epilogue
    const int quarter = (warp >> 2) - 1;  // of the tile's queries; two of them write dV, two dK
    const int half = quarter >> 1;
    const int r = (warp & 3) * 32 + lane;  // key row of the tile = TMEM lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + quarter * 32, p_addr = lane_addr + TP + quarter * 32;
    const float sc = a.scale_log2;
    const uint64_t sc2 = f2_make(sc, sc);
    uint32_t it = 0, nu = 0, ni = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return warp_wait(bar, parity, a.err, &sh.abort_flag);
    };
    while (ok) {
      if (!(ok = items.get(ni++, item, a.err, &sh.abort_flag))) break;
      const DkvItem w(item);
      if (w.stop()) break;
      const int n = w.n;
      const int key = w.key0 + r;
      for (int i = 0; i < n; ++i, ++it) {
        const int row = (w.first + (w.lo + i) % w.tiles) * kTile + quarter * 32;  // first query of this quarter
        const uint32_t st = smem_u32(stats) + ((it % ST) * 2 * kTile + quarter * 32) * 4;
        // First column of this quarter whose query sees the key, 32: none. Queries from it on all do.
        const int from = key >= w.len ? 32 : a.causal ? max(0, key - (w.len - a.Nq) - row) : 0;
        const bool masked = __any_sync(0xffffffffu, from > 0);
        if (!(ok = wait(&sh.s_full, it & 1))) break;
        if (!(ok = wait(&sh.q_full[it % ST], (it / ST) & 1))) break;  // the rows' statistics
        tc_fence_after();
        uint32_t p[32], pk[16];
        tmem_ld32(s_addr, p);
        tmem_wait_ld();
        if (masked) keep_from(p, from, -INFINITY);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const ulonglong2 nl = load_shared16(st + e * 4);
          const uint64_t x0 = f2_fma(pair_of(&p[e]), sc2, nl.x), x1 = f2_fma(pair_of(&p[e + 2]), sc2, nl.y);
          const float v[4] = {fast_exp2(f2_lo(x0)), fast_exp2(f2_hi(x0)), fast_exp2(f2_lo(x1)), fast_exp2(f2_hi(x1))};
#pragma unroll
          for (int q = 0; q < 4; ++q) p[e + q] = __float_as_uint(v[q]);
          pk[e / 2] = pack_bf16x2(v[0], v[1]);
          pk[e / 2 + 1] = pack_bf16x2(v[2], v[3]);
        }
        tmem_st16(s_addr, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full);
        if (!(ok = wait(&sh.dp_full, it & 1))) break;
        tc_fence_after();
        uint32_t d[32];
        tmem_ld32(p_addr, d);
        tmem_wait_ld();
        if (masked) keep_from(d, from, 0.f);  // dP of a key that is not there may be NaN
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const ulonglong2 nd = load_shared16(st + (kTile + e) * 4);
          const uint64_t y0 = f2_mul(f2_add(pair_of(&d[e]), nd.x), pair_of(&p[e]));
          const uint64_t y1 = f2_mul(f2_add(pair_of(&d[e + 2]), nd.y), pair_of(&p[e + 2]));
          pk[e / 2] = pack_bf16x2(f2_lo(y0), f2_hi(y0));
          pk[e / 2 + 1] = pack_bf16x2(f2_lo(y1), f2_hi(y1));
        }
        tmem_st16(p_addr, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.t_full);
      }
      if (!ok) break;
      // Two warpgroups write dV, two dK (times scale), half of the channels each; zeros where no query saw
      // the key (0 times a NaN of dO or q is none).
      if (n > 0) {
        if (!(ok = wait(&sh.acc_full[half], nu & 1))) break;
        tc_fence_after();
      }
      const RowOut& o = half ? f.dk : f.dv;
      const float mul = half ? a.scale : 1.f;
      const uint32_t seen = key < w.len ? 0xffffffffu : 0u;
      const int slot = w.slot;
      float* part = f.part + ((static_cast<size_t>(slot) * 2 + (half ? 0 : 1)) * kTile + r) * D;
      __nv_bfloat16* out = o.p + w.b * o.sb + w.hk * o.sh + key * o.sn;
#pragma unroll 1
      for (int c0 = (quarter & 1) * (D / 2); c0 < ((quarter & 1) + 1) * (D / 2); c0 += 32) {
        uint32_t x[32];
        if (n > 0) {
          tmem_ld32(lane_addr + (half ? TK : TV) + c0, x);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] &= seen;
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = 0u;
        }
        if (key < a.Nk) {
          if (slot < 0)
            store_row32(out + c0, x, mul, o.wide);
          else
            store_row32(part + c0, x, mul, true);
        }
        __syncwarp();
      }
      if (n > 0) {
        tc_fence_before();
        mbar_arrive(&sh.acc_free[half]);
        ++nu;
      }
    }
  }
  if (late) grid_dep_wait();  // this kernel is not done before attend_dq_kernel is
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem_base_sh, 512);
  }
}

// ---------------------------------------------------------------------------- dQ

// One persistent CTA per SM, 640 threads, on units of 128 query rows of one head, a step being a
// key tile:
//   warp 0       TMA: Q_i and dO_i once, then K_j and V_j through a ring of two stages
//   warps 1, 3   tcgen05 issuers: S = Q K^T (two TMEM buffers) and dQ += T K; dP = dO V^T. S and dP of
//                tile j + 1 run while the warps form T of tile j.
//   warp 2       scheduler: the CTA's units
//   warps 4..19  thread = query row = TMEM lane; each warpgroup takes 32 of the tile's keys
// TMEM columns: S ping-pong [0,128) [128,256) (T, bf16, over it: 16 columns over
// each 32), dP [256,384), dQ [384,384+D).
template <int D>
struct AttendDqSmem {
  static constexpr uint32_t TILE = kTile * D * 2;
  static constexpr int STAGES = 2;
  static constexpr uint32_t total() { return (2 + 2 * STAGES) * TILE + 1024; }
};

struct DqUnit {
  int b, h, row0;
  int len, tiles;  // keys of the sequence; key tiles that the unit's rows see
};

__device__ __forceinline__ DqUnit dq_unit(const AttendArgs& a, int u, bool record) {
  DqUnit w;
  const int qt = tiles_of(a.Nq);
  w.row0 = u % qt * kTile;
  w.b = u / qt / a.H;
  w.h = u / qt % a.H;
  w.len = attend_len(a, w.b, record);
  w.tiles = tiles_of(attend_key_end(a, w.len, min(w.row0 + kTile, a.Nq) - 1));
  return w;
}

struct DqItem {
  int b, h, row0, len, lo, n, slot, exact;  // exact: one key tile, delta is formed here (2: and written)
  __device__ __forceinline__ explicit DqItem(const AttendItem& i)
      : b(i.v[0]), h(i.v[1]), row0(i.v[2]), len(i.v[3]), lo(i.v[4]), n(i.v[5]), slot(i.v[6]),
        exact(i.v[7]) {}
  __device__ __forceinline__ bool stop() const { return b < 0; }
};

template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attend_dq_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_g,
                     const __grid_constant__ AttendBwdArgs f) {
  using L = AttendDqSmem<D>;
  constexpr int DB = D / 64, ST = L::STAGES;
  constexpr uint32_t TP = 256, TQ = 384;  // TMEM columns of dP and dQ
  const AttendArgs& a = f.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = base;
  uint8_t* sG = sQ + L::TILE;
  uint8_t* ringK = sG + L::TILE;
  uint8_t* ringV = ringK + ST * L::TILE;

  __shared__ uint64_t q_full, q_free, s_full[2], dp_full, dp_free, t_full[2], acc_full, acc_free, drain;
  __shared__ uint64_t k_full[ST], v_full[ST], k_free[ST], v_free[ST];
  __shared__ uint64_t sum_full;
  __shared__ float sums[2][4][kTile];  // a quarter's part of delta of each row; two buffers
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ ItemRing<kBwdWarps> items;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_free, 2);
    mbar_init(&dp_full, 1);
    mbar_init(&sum_full, kBwdWarps);
    mbar_init(&dp_free, kBwdWarps);
    mbar_init(&acc_full, 1);
    mbar_init(&acc_free, 32 * kBwdWarps);
    mbar_init(&drain, 2);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&t_full[s], kBwdWarps);
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&k_free[s], 1);
      mbar_init(&v_free[s], 1);
    }
    items.init();
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  // Behind attend_dkv_kernel this one runs beside it where SMs are free: that kernel's CTAs let this one in after
  // their own wait for attend_rows_kernel, whose results are all that this one needs of earlier kernels.
  // The wait then comes last.
  if (f.dq_first) grid_dep_wait();
  grid_dep_launch();
  const auto steps = [&](int u) { return dq_unit(a, u, false).tiles; };
  AttendWork work = attend_work(a, steps, kBwdThreads);
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all columns are allocated
  AttendItem item;

  if (warp == kScheduleWarp) {
    if (lane == 0) {
      uint32_t ni = 0;
      int u, lo, hi, n, to, longest = 0;  // steps of the longest item
      bool ok = true;
      DqUnit w;  // the unit that `next` looked at last, which is the one it gives
      const auto look = [&](int v) {
        w = dq_unit(a, v, true);
        return w.tiles;
      };
      while (ok && work.next(a, look, u, lo, hi, n, to)) {
        note_part(a, work, u, lo, hi, n, to);
        item = {w.b, w.h, w.row0, w.len, lo, w.tiles > 0 ? hi - lo : 0, part_slot(lo, hi, n),
                w.tiles != 1 ? 0 : f.dq_first && w.len <= kTile ? 2 : 1};
        longest = max(longest, hi - lo);
        ok = items.put(ni++, item, longest, a.err, &abort_flag);
      }
      item.v[0] = -1;
      if (ok) items.put(ni, item, longest, a.err, &abort_flag);
    }
    __syncwarp();
  } else if (warp == kProducerWarp) {
    // ------------------------------------------------------------ TMA producer
    uint32_t ni = 0;
    if (lane == 0) {
      prefetch_tmap(&map_q);
      prefetch_tmap(&map_k);
      prefetch_tmap(&map_v);
      prefetch_tmap(&map_g);
      uint32_t nk = 0, nv = 0, nu = 0;  // K tiles, V tiles and units loaded
      bool ok = true;
      while (ok) {
        if (!(ok = items.get_one(ni++, item, a.err, &abort_flag))) break;
        const DqItem w(item);
        if (w.stop()) break;
        if (w.n == 0) continue;
        if (nu > 0 && !(ok = mbar_wait(&q_free, (nu - 1) & 1, a.err, &abort_flag))) break;
        mbar_arrive_expect_tx(&q_full, 2 * L::TILE);
        for (int b = 0; b < DB; ++b) tma_load_4d(sQ + b * kBox, &map_q, &q_full, b * 64, w.row0, w.h, w.b);
        for (int b = 0; b < DB; ++b) tma_load_4d(sG + b * kBox, &map_g, &q_full, b * 64, w.row0, w.h, w.b);
        ++nu;
        for (int j = w.lo; j < w.lo + w.n; ++j) {
          const int key = j * kTile;
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
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer of S and dQ
    const uint32_t q0 = smem_u32(sQ), rk = smem_u32(ringK);
    uint32_t it = 0, nu = 0, ni = 0;  // key tiles, units with work and items so far
    RingPos pos;                      // of the next S's K tile
    bool ok = true;
    const uint32_t lead = elect_one();
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return warp_wait(bar, parity, a.err, &abort_flag); };
    while (ok) {
      if (!(ok = items.get(ni++, item, a.err, &abort_flag))) break;
      const DqItem w(item);
      if (w.stop()) break;
      const int n = w.n;
      if (n == 0) continue;
      auto issue_s = [&](int j) -> bool {
        const uint32_t s = pos.s, t = it + j;
        if (!wait(&k_full[s], pos.parity)) return false;
        const int keys = w.len - (w.lo + j) * kTile;  // real keys of the tile
        if (keys < kTile) zero_rows<D>(ringK + s * L::TILE, keys, kTile);
        tc_fence_after();
        issue_ss<D, 128>(lead, (t & 1) * 128, q0, rk + s * L::TILE);
        mma_commit(lead, &s_full[t & 1]);
        if (j + 1 == n) mma_commit(lead, &q_free);  // the unit's last reader of Q_i
        pos.next(ST);
        return true;
      };
      if (!(ok = wait(&q_full, nu & 1))) break;
      RingPos cur = pos;  // of dQ's K tile
      if (!(ok = issue_s(0))) break;
      if (nu > 0 && !(ok = wait(&acc_free, (nu - 1) & 1))) break;
      for (int j = 0; j < n; ++j) {
        const uint32_t t = it + j;
        if (j + 1 < n && !(ok = issue_s(j + 1))) break;
        if (!(ok = wait(&t_full[t & 1], (t >> 1) & 1))) break;
        tc_fence_after();
        issue_ts<D, 0, 8, 2, 32>(lead, TQ, (t & 1) * 128, rk + cur.s * L::TILE, j > 0);
        mma_commit(lead, &k_free[cur.s]);
        if (j + 1 == n) mma_commit(lead, &acc_full);
        cur.next(ST);
      }
      it += n;
      ++nu;
    }
    mma_commit(lead, &drain);
    mbar_wait(&drain, 0, nullptr, nullptr);
  } else if (warp == kMmaWarp2) {
    // ------------------------------------------------------------ MMA issuer of dP
    const uint32_t g0 = smem_u32(sG), rv = smem_u32(ringV);
    uint32_t it = 0, nu = 0, ni = 0;
    RingPos pos;
    bool ok = true;
    const uint32_t lead = elect_one();
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return warp_wait(bar, parity, a.err, &abort_flag); };
    while (ok) {
      if (!(ok = items.get(ni++, item, a.err, &abort_flag))) break;
      const DqItem w(item);
      if (w.stop()) break;
      if (w.n == 0) continue;
      if (!(ok = wait(&q_full, nu & 1))) break;
      for (int j = 0; j < w.n; ++j, ++it) {
        const uint32_t s = pos.s;
        if (!(ok = wait(&v_full[s], pos.parity))) break;
        if (it > 0 && !(ok = wait(&dp_free, (it - 1) & 1))) break;  // the previous dP has been read
        tc_fence_after();
        issue_ss<D, 128>(lead, TP, g0, rv + s * L::TILE);
        mma_commit(lead, &dp_full);
        mma_commit(lead, &v_free[s]);
        if (j + 1 == w.n) mma_commit(lead, &q_free);  // the unit's last reader of dO_i
        pos.next(ST);
      }
      ++nu;
    }
    mma_commit(lead, &drain);
    mbar_wait(&drain, 0, nullptr, nullptr);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ T, then the epilogue
    const int quarter = (warp >> 2) - 1;  // of the tile's keys, then of the channels
    const int r = (warp & 3) * 32 + lane;  // query row of the tile = TMEM lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float sc = a.scale_log2;
    const uint64_t sc2 = f2_make(sc, sc);
    uint32_t it = 0, nu = 0, ni = 0, ne = 0;  // key tiles, units with work, items, exact units
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return warp_wait(bar, parity, a.err, &abort_flag);
    };
    // The next unit, and its rows' statistics, which are on their way while the last unit's rows are written (cross
    // attention over 512 keys, forward and backward, in turn on one GPU: 582.6 us without, 575.1; 575 to 608 on others).
    float nl_next = 0.f, nd_next = 0.f;
    auto look = [&]() -> bool {
      if (!items.get(ni++, item, a.err, &abort_flag)) return false;
      const DqItem w(item);
      if (!w.stop()) {
        const size_t at = (static_cast<size_t>(w.b) * a.H + w.h) * f.pad + w.row0 + r;
        nl_next = f.nlse[at];
        nd_next = f.ndelta[at];
      }
      return true;
    };
    ok = look();
    while (ok) {
      const DqItem w(item);
      if (w.stop()) break;
      const int n = w.n;
      const int row = w.row0 + r;
      const int end = attend_key_end(a, w.len, row);
      const float nl = nl_next, nd = nd_next;
      const uint64_t nl2 = f2_make(nl, nl);
      uint64_t nd2 = f2_make(nd, nd);
      for (int j = 0; j < n; ++j, ++it) {
        const int key0 = (w.lo + j) * kTile + quarter * 32;
        const int upto = end - key0;  // columns of this quarter that the row sees
        const bool masked = __any_sync(0xffffffffu, upto < 32);
        const uint32_t s_addr = lane_addr + (it & 1) * 128 + quarter * 32;
        if (!(ok = wait(&s_full[it & 1], (it >> 1) & 1))) break;
        tc_fence_after();
        uint32_t p[32], d[32], pk[16];
        tmem_ld32(s_addr, p);
        tmem_wait_ld();
        if (masked) keep_upto(p, upto, -INFINITY);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t x = f2_fma(pair_of(&p[e]), sc2, nl2);
          p[e] = __float_as_uint(fast_exp2(f2_lo(x)));
          p[e + 1] = __float_as_uint(fast_exp2(f2_hi(x)));
        }
        if (!(ok = wait(&dp_full, it & 1))) break;
        tc_fence_after();
        tmem_ld32(lane_addr + TP + quarter * 32, d);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&dp_free);
        if (masked) keep_upto(d, upto, 0.f);  // dP of a key that is not there may be NaN
        if (w.exact) {
          uint64_t part = 0ull;
#pragma unroll
          for (int e = 0; e < 32; e += 2) part = f2_fma(pair_of(&p[e]), pair_of(&d[e]), part);
          float(&buffer)[4][kTile] = sums[ne & 1];
          buffer[quarter][r] = f2_lo(part) + f2_hi(part);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sum_full);
          if (!(ok = wait(&sum_full, ne & 1))) break;
          ++ne;
          const float delta = (buffer[0][r] + buffer[1][r]) + (buffer[2][r] + buffer[3][r]);
          nd2 = f2_make(-delta, -delta);
          if (w.exact == 2 && quarter == 0) f.ndelta[(static_cast<size_t>(w.b) * a.H + w.h) * f.pad + row] = -delta;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t y = f2_mul(f2_add(pair_of(&d[e]), nd2), pair_of(&p[e]));
          pk[e / 2] = pack_bf16x2(f2_lo(y), f2_hi(y));
        }
        tmem_st16(s_addr, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&t_full[it & 1]);
      }
      if (!ok || !(ok = look())) break;
      if (n > 0) {
        if (!(ok = wait(&acc_full, nu & 1))) break;
        tc_fence_after();
      }
      // scale times the accumulator, 32 channels to a warpgroup; zeros where the row sees no key
      const int slot = w.slot;
      const int c0 = quarter * 32;
      if (c0 < D) {
        uint32_t x[32];
        if (n > 0) {
          tmem_ld32(lane_addr + TQ + c0, x);
          tmem_wait_ld();
          const uint32_t sees = end > 0 ? 0xffffffffu : 0u;
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] &= sees;
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = 0u;
        }
        if (row < a.Nq) {
          if (slot < 0)
            store_row32(f.dq.p + w.b * f.dq.sb + w.h * f.dq.sh + row * f.dq.sn + c0, x, a.scale, f.dq.wide);
          else
            store_row32(f.part + (static_cast<size_t>(slot) * kTile + r) * D + c0, x, a.scale, true);
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
  if (!f.dq_first) grid_dep_wait();  // this kernel is not done before attend_dkv_kernel is
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem_base_sh, 512);
  }
}

// Joins the parts that attend_dkv_kernel (blockIdx.z 0: dK, 1: dV) and attend_dq_kernel (2) left: for the unit
// that CTA blockIdx.x began and others went on with, the sum of the parts' rows in ascending CTA
// order, rounded once. 8 channels a thread.
struct AttendSumArgs {
  AttendBwdArgs kv, q;
  int kv_ctas, q_ctas;
};

template <int D>
__global__ void __launch_bounds__(256) attend_sum_kernel(const __grid_constant__ AttendSumArgs s) {
  constexpr int T = D / 8;
  grid_dep_wait();
  grid_dep_launch();
  const bool is_q = blockIdx.z == 2;
  const AttendBwdArgs& f = is_q ? s.q : s.kv;
  const AttendArgs& a = f.p;
  const int C = is_q ? s.q_ctas : s.kv_ctas, c0 = blockIdx.x;
  if (c0 >= C || !a.meta) return;
  const int4 meta = a.meta[c0];
  if (meta.x < 0) return;
  const int r = blockIdx.y * (256 / T) + threadIdx.x / T, c = (threadIdx.x % T) * 8;
  const RowOut& o = is_q ? f.dq : blockIdx.z == 0 ? f.dk : f.dv;
  __nv_bfloat16* out;
  if (is_q) {
    const DqUnit w = dq_unit(a, meta.x, false);
    if (w.row0 + r >= a.Nq) return;
    out = o.p + w.b * o.sb + w.h * o.sh + (w.row0 + r) * o.sn + c;
  } else {
    const DkvUnit w = dkv_unit(a, meta.x, false);
    if (w.key0 + r >= a.Nk) return;
    out = o.p + w.b * o.sb + w.hk * o.sh + (w.key0 + r) * o.sn + c;
  }
  float x[8] = {};
  for (int k0 = c0; k0 <= meta.y; k0 += 4) {
    float4 u[4], v[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int k = k0 + p;
      u[p] = v[p] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k > meta.y || part_is_empty(meta.z, C, k)) continue;
      size_t at = static_cast<size_t>(k == c0 ? 2 * k + 1 : 2 * k);
      if (!is_q) at = at * 2 + blockIdx.z;
      const float4* w = reinterpret_cast<const float4*>(f.part + (at * kTile + r) * D + c);
      u[p] = w[0];
      v[p] = w[1];
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      x[0] += u[p].x, x[1] += u[p].y, x[2] += u[p].z, x[3] += u[p].w;
      x[4] += v[p].x, x[5] += v[p].y, x[6] += v[p].z, x[7] += v[p].w;
    }
  }
  *reinterpret_cast<uint4*>(out) =
      make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

}  // namespace sla
