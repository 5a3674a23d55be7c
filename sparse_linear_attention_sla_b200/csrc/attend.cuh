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
// S, acc, m and l are fp32. A row without keys gives out = 0 and lse = -inf; a NaN among a row's scores makes
// both NaN, whole or in parts.
//
// One persistent CTA per SM, 384 threads. A tile is at most 128 rows, `heads` query heads that share a
// key head x `tokens` queries. A unit is, with more than 128 queries, two neighbouring tiles A and B
// that meet the same key tiles; with fewer ("narrow"), one tile whose key tiles go to A and B in
// turn, so that a single token of a group reads its keys once and both halves work:
//   warp 0       TMA: Q, then K_j and V_j tiles through a ring
//   warps 1, 3   tcgen05 issuers of A and of B, on blocks t of 64 keys (half a tile):
//                S_x = Q_x K_t^T, acc_x += P_x V_t
//   warp 2       scheduler: the CTA's units
//   warps 4..7   softmax of A; warps 8..11 of B: thread = query row = TMEM lane
// TMEM columns: S_A [0,128) and S_B [128,256), two buffers of 64 columns each (P_t, bf16, over the
// first 32 of its S_t), acc_A [256,256+D), acc_B [384,384+D). MMAs of one thread run in issue
// order, so S_{t+2} never overwrites P_t before the product that reads it; S_{t+1} is there when
// the warps have formed P_t. (One buffer of 128 keys needs fewer tensor cycles, 2048 instead of
// 2540 for a tile of A and of B, but then the exponentials and the products of a tile take
// turns: 4600 cycles.)
// A row's epilogue takes about 4000 cycles of a unit (a block of 64 keys 1950): rows lie apart, and the code, run once
// a unit, is not at hand. It runs in rounds of 32 channels, and the next unit is looked up while its last product runs
// (cross attention over 512 and 77 keys, in turn on one GPU: 193.7 us with rounds of 64 and the lookup after, 189.9
// with 32, 184.0 so).
// Measured, a call on several GPUs of the kind: 16380 tokens of 12 heads 1436 to 1612 us (1.04 PFLOP/s at 1.65 GHz),
// 2 x 32760 over 512 and 77 keys 184 to 206, one token over 4 x 8 heads of up to 32760 keys 55 to 64 with the join.
// Parts of units (see AttendWork) are fp32 rows divided by their own sum, with the sum's log2;
// attend_join_kernel joins them.
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
  int narrow;        // Nq <= 128: units are one tile
  int heads, tokens; // of a tile: `heads` query heads of a group x `tokens` queries, at most 128 rows
  int q_bytes;       // of one loaded Q tile
  RowOut out;
  float* lse;        // [B * H, Nq]
  float* part;       // [2 * CTAs][rows of a unit][D]
  float* part_lse2;  // [2 * CTAs][rows of a unit]: log2 of the part's sum, its reference included
};

struct AttendUnit {
  int b, h, hk;  // h: the (first) query head
  int row0;      // first query of the unit
  int len;
  int tiles[2];  // key tiles that tile A and tile B see (narrow: both, together)

  __device__ __forceinline__ int steps(int narrow) const {
    return narrow ? (tiles[0] + 1) / 2 : max(tiles[0], tiles[1]);
  }
  // Key tiles of x in the steps [lo, hi), and the j-th of them.
  __device__ __forceinline__ int count(int narrow, int x, int lo, int hi) const {
    return narrow ? max(0, min(hi, (tiles[0] - x + 1) / 2) - lo) : max(0, min(hi, tiles[x]) - lo);
  }
};

// What the warps need of the current unit.
struct AttendItemView {
  int b, h, hk, row0, len;
  int lo, na, nb; // first step; key tiles of A and B
  int slot;       // of its parts, -1: the unit is whole
  int narrow;

  __device__ __forceinline__ AttendItemView(const AttendItem& i, int nar)
      : b(i.v[0]), h(i.v[1]), hk(i.v[2]), row0(i.v[3]), len(i.v[4]), lo(i.v[5]), na(i.v[6]), nb(i.v[7]),
        slot(i.v[8]), narrow(nar) {}
  __device__ __forceinline__ bool stop() const { return b < 0; }
  __device__ __forceinline__ int n(int x) const { return x ? nb : na; }
  __device__ __forceinline__ int tile(int x, int j) const { return narrow ? 2 * (lo + j) + x : lo + j; }
  // Blocks of 64 keys of x: its last tile may hold no second one.
  __device__ __forceinline__ int blocks(int x) const {
    return n(x) == 0 ? 0 : 2 * n(x) - (len - tile(x, n(x) - 1) * kTile <= 64 ? 1 : 0);
  }
};

__device__ __forceinline__ AttendUnit attend_unit(const AttendFwdArgs& f, int u, bool record) {
  const AttendArgs& a = f.p;
  AttendUnit w;
  const int span = (f.narrow ? 1 : 2) * f.tokens;  // queries of a unit
  const int spans = (a.Nq + span - 1) / span, groups = (a.G + f.heads - 1) / f.heads;
  const int g = u / spans;
  w.row0 = u % spans * span;
  w.b = g / groups / a.Hk;
  w.hk = g / groups % a.Hk;
  w.h = w.hk * a.G + g % groups * f.heads;
  w.len = attend_len(a, w.b, record);
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = w.row0 + (f.narrow ? 0 : x * f.tokens);
    w.tiles[x] = r < a.Nq ? tiles_of(attend_key_end(a, w.len, min(r + f.tokens, a.Nq) - 1)) : 0;
  }
  return w;
}

// The head and query of row r of the unit's tile x; false where the row is none.
template <class Unit>
__device__ __forceinline__ bool attend_row(const AttendFwdArgs& f, const Unit& w, int x, int r, int& h, int& i) {
  const int k = f.heads == 1 ? 0 : r / f.tokens, t = r - k * f.tokens;
  h = w.h + k;
  i = w.row0 + (f.narrow ? 0 : x * f.tokens) + t;
  return k < f.heads && t < f.tokens && h < (w.hk + 1) * f.p.G && i < f.p.Nq;
}

// Keys of 32 columns from key0 on that a row does not see (its keys end at `end`) take -inf.
__device__ __forceinline__ void mask_cols32(uint32_t (&x)[32], int key0, int end) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (key0 + c >= end) x[c] = __float_as_uint(-INFINITY);
}

// A row's reference from its largest score `top` so far: m = top sc, and p = 2^(s mul - ref) of a score s, in one
// FMA, with mul = sc and ref = m. The FMA keeps what m lost in its own rounding, a factor of the whole row until
// half a step of m passes the exponent's range (128 at |m| = 2^32). From 2^30 on mul is the power of two below
// sc, so that ref = top mul is exact and the largest p is 1; scores that differ lie 64 apart there by their own
// rounding, so that the others' p, 2^-64 at most, is below 2^-32 either way.
constexpr float kExactRef = 0x1p30f;

__device__ __forceinline__ void attend_refer(float top, float sc, float& m, float& mul, float& ref) {
  m = top * sc;
  const bool exact = fabsf(m) >= kExactRef && fabsf(m) < INFINITY;
  mul = exact ? __uint_as_float(__float_as_uint(sc) & 0x7F800000u) : sc;
  ref = top * mul;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ AttendFwdArgs f) {
  using L = AttendSmem<D>;
  constexpr int DB = D / 64;
  constexpr uint32_t ACC = 256;
  // Narrow: the second Q tile's room is a stage more, and A and B have half of them each.
  const uint32_t ST = f.narrow ? (L::STAGES + 1) / 2 : L::STAGES;
  const AttendArgs& a = f.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = base;
  uint8_t* ring = sQ + (2 - f.narrow) * L::TILE;

  __shared__ uint64_t q_full, q_free, s_full[2][2], p_full[2][2], pv_done[2][2], acc_free[2], b_sums;  // [x][buffer]
  __shared__ uint64_t full[L::STAGES + 1], empty[L::STAGES + 1];
  __shared__ uint64_t drain;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ float sums[2][kTile];  // narrow: m and l of B's rows
  __shared__ ItemRing<8> items;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int narrow = f.narrow;
  if (tid == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_free, 2);
    mbar_init(&b_sums, 128);
    for (int x = 0; x < 2; ++x) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[x][b], 1);
        mbar_init(&p_full[x][b], 128);
        mbar_init(&pv_done[x][b], 1);
      }
      mbar_init(&acc_free[x], 128);
    }
    for (int s = 0; s <= L::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], narrow ? 1 : 2);  // narrow: A and B have stages of their own
    }
    mbar_init(&drain, 2);
    items.init();
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_base_sh, 512);  // all columns, so column addresses count from 0
    tmem_relinquish();
  }
  grid_dep_wait();  // lengths and inputs may come from earlier kernels
  grid_dep_launch();
  const auto steps = [&](int u) { return attend_unit(f, u, false).steps(narrow); };
  AttendWork work = attend_work(a, steps, kThreads);
  __syncthreads();
  tc_fence_after();
  AttendItem item;

  if (warp < 4) regs_down<kIssueRegs>();
  if (warp == kScheduleWarp) {
    if (lane == 0) {
      uint32_t ni = 0;
      int u, lo, hi, n, to, longest = 0;  // steps of the longest item
      bool ok = true;
      AttendUnit w;  // the unit that `next` looked at last, which is the one it gives
      const auto look = [&](int v) {
        w = attend_unit(f, v, true);
        return w.steps(narrow);
      };
      while (ok && work.next(a, look, u, lo, hi, n, to)) {
        note_part(a, work, u, lo, hi, n, to);
        item = {w.b, w.h, w.hk, w.row0, w.len, lo, w.count(narrow, 0, lo, hi), w.count(narrow, 1, lo, hi),
                part_slot(lo, hi, n)};
        longest = max(longest, hi - lo);
        ok = items.put(ni++, item, longest, a.err, &abort_flag);
      }
      item.v[0] = -1;
      if (ok) items.put(ni, item, longest, a.err, &abort_flag);
    }
    __syncwarp();
  } else if (warp == kProducerWarp) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tmap(&map_q);
      prefetch_tmap(&map_k);
      prefetch_tmap(&map_v);
      RingPos pos[2];  // wide: only the first
      uint32_t nr[2] = {0, 0}, nq = 0, ni = 0;  // ring tiles, Q loads and items so far
      bool ok = true;
      while (ok) {
        if (!(ok = items.get_one(ni++, item, a.err, &abort_flag))) break;
        const AttendItemView w(item, narrow);
        if (w.stop()) break;
        if (w.n(0) + w.n(1) == 0) continue;
        auto load = [&](const CUtensorMap* m, int x, int j) {
          const uint32_t s = x * ST + pos[x].s;
          if (nr[x] >= ST && !(ok = mbar_wait(&empty[s], pos[x].parity ^ 1, a.err, &abort_flag))) return;
          mbar_arrive_expect_tx(&full[s], L::TILE);
          for (int b = 0; b < DB; ++b)
            tma_load_4d(ring + s * L::TILE + b * kBox, m, &full[s], b * 64, w.tile(x, j) * kTile, w.hk, w.b);
          ++nr[x];
          pos[x].next(ST);
        };
        if (nq > 0) ok = mbar_wait(&q_free, (nq - 1) & 1, a.err, &abort_flag);
        if (ok) {
          const int q_tiles = narrow || w.n(1) == 0 ? 1 : 2;
          mbar_arrive_expect_tx(&q_full, q_tiles * f.q_bytes);
          for (int x = 0; x < q_tiles; ++x)
            for (int b = 0; b < DB; ++b)
              tma_load_5d(sQ + x * L::TILE + b * kBox, &map_q, &q_full, b * 64, w.row0 + x * f.tokens, w.h % a.G, w.hk,
                          w.b);
          ++nq;
        }
        if (narrow) {
          for (int x = 0; ok && x < 2; ++x)
            if (w.n(x) > 0) load(&map_k, x, 0);
          for (int j = 0; ok && j < w.n(0); ++j) {
            for (int x = 0; ok && x < 2; ++x) {
              if (j >= w.n(x)) continue;
              load(&map_v, x, j);
              if (ok && j + 1 < w.n(x)) load(&map_k, x, j + 1);
            }
          }
        } else {
          const int nt = max(w.n(0), w.n(1));
          if (ok) load(&map_k, 0, 0);
          for (int j = 0; ok && j < nt; ++j) {
            load(&map_v, 0, j);
            if (ok && j + 1 < nt) load(&map_k, 0, j + 1);
          }
        }
      }
      if (abort_flag) {  // let every load still in flight land before the CTA retires
        if (nq > 0) mbar_wait(&q_full, (nq - 1) & 1, nullptr, nullptr);
        for (int x = 0; x < 2; ++x)
          for (uint32_t i = nr[x] > ST ? nr[x] - ST : 0; i < nr[x]; ++i)
            mbar_wait(&full[x * ST + i % ST], (i / ST) & 1, nullptr, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kMmaWarp2) {
    // ------------------------------------------------------------ MMA issuer of tile x
    const int x = warp == kMmaWarp2;
    const uint32_t q0 = smem_u32(sQ) + (narrow ? 0 : x * L::TILE), r0 = smem_u32(ring);
    const uint32_t first = narrow ? x * ST : 0;  // this warp's first stage
    RingPos pos;
    uint32_t nq = 0, ni = 0, nu = 0, g = 0;  // units with work, items, units with tiles of x, blocks before the unit
    bool ok = true;
    const uint32_t lead = elect_one();
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return warp_wait(bar, parity, a.err, &abort_flag); };
    auto commit = [&](uint64_t* bar) { mma_commit(lead, bar); };
    auto arrive = [&](uint64_t* bar) {
      if (lane == 0) mbar_arrive(bar);
      __syncwarp();
    };
    // The next ring tile, once it has landed.
    auto take = [&](uint32_t& s) -> bool {
      s = first + pos.s;
      const bool r = wait(&full[s], pos.parity);
      pos.next(ST);
      return r;
    };
    // S of block t of the unit, from its half of the K tile in stage sk.
    auto issue_s = [&](int t, uint32_t sk) {
      const uint32_t b = (g + t) & 1;
      issue_ss<D, 64>(lead, x * 128 + b * 64, q0, r0 + sk * L::TILE + (t & 1) * 8192);
      commit(&s_full[x][b]);
    };
    while (ok) {
      if (!(ok = items.get(ni++, item, a.err, &abort_flag))) break;
      const AttendItemView w(item, narrow);
      if (w.stop()) break;
      const int n = w.n(x), loaded = narrow ? n : max(w.na, w.nb);  // tiles of x; tiles that the ring brings
      const int nb = w.blocks(x);
      if (max(w.na, w.nb) == 0) continue;
      uint32_t sk = 0, sv = 0;  // stages of the current K and V tile
      if (!(ok = wait(&q_full, nq & 1))) break;
      ++nq;
      if (n > 0) {
        if (!(ok = take(sk))) break;
        tc_fence_after();
        issue_s(0, sk);
        if (nb > 1) issue_s(1, sk);
        commit(&empty[sk]);
      }
      if (n == 1) commit(&q_free);
      if (n == 0) arrive(&q_free);
      for (int j = 0; ok && j < n; ++j) {
        if (!(ok = take(sv))) break;
        const int keys = w.len - w.tile(x, j) * kTile;  // rows behind the sequence's keys
        if (keys < kTile) zero_rows<D>(ring + sv * L::TILE, keys, kTile);
        if (j == 0 && nu > 0 && !(ok = wait(&acc_free[x], (nu - 1) & 1))) break;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 2 * j + e;
          if (t >= nb) break;
          const uint32_t b = (g + t) & 1;
          if (!(ok = wait(&p_full[x][b], ((g + t) >> 1) & 1))) break;
          tc_fence_after();
          issue_ts<D, 0, 4, 4, 32>(lead, ACC + x * 128, x * 128 + b * 64, r0 + sv * L::TILE + e * 8192, t > 0);
          commit(&pv_done[x][b]);
          if (e == 1 || t + 1 == nb) commit(&empty[sv]);
          if (j + 1 < n) {
            if (e == 0 && !(ok = take(sk))) break;
            tc_fence_after();
            if (t + 2 < nb) issue_s(t + 2, sk);
            if (e == 1) commit(&empty[sk]);
          }
        }
        if (j + 2 == n) commit(&q_free);  // no S of this unit is left to issue
      }
      // Wide: tiles that only the other query tile needs.
      for (int j = 2 * n; ok && j < 2 * loaded; ++j) {
        if (!(ok = take(sk))) break;
        arrive(&empty[sk]);
      }
      nu += n > 0;
      g += nb;
    }
    commit(&drain);  // every MMA issued above has finished once this arrives
    mbar_wait(&drain, 0, nullptr, nullptr);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax warpgroups
    regs_up<kComputeRegs>();
    const int x = warp >= 8;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = lane_addr + x * 128, o_addr = lane_addr + ACC + x * 128;
    const float sc = a.scale_log2;
    uint32_t ni = 0, ns = 0, nu = 0, nbb = 0;  // items; blocks of x; narrow: units with tiles of B, and their blocks
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return warp_wait(bar, parity, a.err, &abort_flag); };
    struct Row {
      int h, i, n, other, end, end_min;  // blocks of x and of the other tile; this row's keys, the fewest of a row
      bool real;
    } row;
    auto look = [&](const AttendItemView& w) {
      row.real = attend_row(f, w, x, r, row.h, row.i);
      row.n = w.blocks(x);
      row.other = w.blocks(x ^ 1);
      row.end = attend_key_end(a, w.len, row.i);
      row.end_min = attend_key_end(a, w.len, w.row0 + (narrow ? 0 : x * f.tokens));
    };
    if ((ok = items.get(ni++, item, a.err, &abort_flag))) look(AttendItemView(item, narrow));
    while (ok) {
      const AttendItemView w(item, narrow);
      if (w.stop()) break;
      const int h = row.h, i = row.i, n = row.n, other = row.other, end = row.end, end_min = row.end_min;
      const bool real = row.real;
      float m = -INFINITY, l = 0.f;
      float mul = sc, ref = -INFINITY;  // p = 2^(s mul - ref): see attend_refer
      for (int t = 0; t < n; ++t, ++ns) {
        const uint32_t b = ns & 1, sb = s_addr + b * 64;
        if (!(ok = wait(&s_full[x][b], (ns >> 1) & 1))) break;
        tc_fence_after();
        uint32_t s[2][32];
        tmem_ld32(sb, s[0]);
        tmem_ld32(sb + 32, s[1]);
        tmem_wait_ld();
        const int key0 = w.tile(x, t >> 1) * kTile + (t & 1) * 64;
        if (key0 + 64 > end_min) {
          mask_cols32(s[0], key0, end);
          mask_cols32(s[1], key0 + 32, end);
        }
        if (__any_sync(0xffffffffu, m == -INFINITY)) {
          const float top = row_max64(s[0], s[1]);
          if (m == -INFINITY) attend_refer(top, sc, m, mul, ref);
        }
        uint32_t pk[32];
        auto exponentials = [&]() -> float {
          const float r = ref == -INFINITY ? 0.f : ref;  // no key seen yet: every s is -inf
          const uint64_t part = exp2_block(s[0], s[1], pk, f2_make(mul, mul), f2_make(-r, -r));
          return f2_lo(part) + f2_hi(part);
        };
        float sum = exponentials();
        if (__any_sync(0xffffffffu, sum > kRefMoveSum)) {
          // Only the rows that passed move: a row's bits depend on nothing but its own scores (rows of
          // the tile that are no query hold whatever shared memory held).
          const float top = row_max64(s[0], s[1]), m_old = m, mul_old = mul, ref_old = ref;
          if (sum > kRefMoveSum && top * sc >= m) attend_refer(top, sc, m, mul, ref);
          const float g = m == -INFINITY ? 1.f : fast_exp2(mul == mul_old ? ref_old - ref : m_old - m);
          if (t > 0) {  // S_t was seen, so of the products only the last can be open
            if (!(ok = wait(&pv_done[x][b ^ 1], ((ns - 1) >> 1) & 1))) break;
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
          l *= g;
          sum = exponentials();
        }
        l += sum;
        tmem_st32(sb, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[x][b]);
      }
      if (!ok) break;
      // The next unit, while the last product runs.
      if (!(ok = items.get(ni++, item, a.err, &abort_flag))) break;
      look(AttendItemView(item, narrow));
      // acc / l as bf16, or as a part's fp32 row with its log2-sum. Narrow: A's warps write
      // both, w_x = 2^(m_x - m) being the weight of x's accumulator.
      float weight[2] = {1.f, 0.f};
      if (narrow && x == 1) {
        if (n > 0) {
          if (nu > 0 && !(ok = wait(&acc_free[1], (nu - 1) & 1))) break;  // the last sums have been read
          sums[0][r] = m;
          sums[1][r] = l;
          mbar_arrive(&b_sums);
          ++nu;
        }
        continue;
      }
      const bool both = narrow && other > 0;
      if (both) {
        if (!(ok = wait(&b_sums, nu & 1) && wait(&pv_done[1][(nbb + other - 1) & 1], ((nbb + other - 1) >> 1) & 1))) break;
        const float mb = sums[0][r], lb = sums[1][r];
        const float top = fmaxf(m, mb);
        weight[0] = m == -INFINITY ? 0.f : fast_exp2(m - top);
        weight[1] = mb == -INFINITY ? 0.f : fast_exp2(mb - top);
        l = l * weight[0] + lb * weight[1];
        m = top;
        nbb += other;
        ++nu;
      }
      if (n > 0 && !(ok = wait(&pv_done[x][(ns - 1) & 1], ((ns - 1) >> 1) & 1))) break;
      tc_fence_after();
      // A row that saw no key has l = 0; a NaN in l is none of those, it goes on into out and lse.
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lse2 = l == 0.f ? -INFINITY : m + __log2f(l);
      const size_t part_row = narrow ? static_cast<size_t>(w.slot) * kTile + r
                                     : static_cast<size_t>(w.slot) * 2 * kTile + x * kTile + r;
      __nv_bfloat16* const out = f.out.p + w.b * f.out.sb + h * f.out.sh + i * f.out.sn;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(o_addr + c0, o);
          tmem_wait_ld();
        }
        if (both) {
          uint32_t ob[32];
          tmem_ld32(o_addr + 128 + c0, ob);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c)
            o[c] = __float_as_uint(weight[0] * __uint_as_float(o[c]) + weight[1] * __uint_as_float(ob[c]));
        }
        if (l == 0.f) {  // nothing was seen: the accumulators hold no number to keep
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0u;
        }
        if (real) {
          if (w.slot < 0)
            store_row32(out + c0, o, inv, f.out.wide);
          else
            store_row32(f.part + part_row * D + c0, o, inv, true);
        }
        __syncwarp();
      }
      if (real) {
        if (w.slot < 0)
          f.lse[(static_cast<size_t>(w.b) * a.H + h) * a.Nq + i] = lse2 * 0.69314718055994531f;
        else
          f.part_lse2[part_row] = lse2;
      }
      tc_fence_before();
      if (n > 0) mbar_arrive(&acc_free[x]);
      if (both) mbar_arrive(&acc_free[1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem_base_sh, 512);
  }
}

// Joins the parts of the unit that CTA blockIdx.x of attend_kernel began and others went on
// with: out = sum_p 2^(lse2_p - lse2) part_p in ascending CTA order. 8 channels a thread.
template <int D>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendFwdArgs f) {
  constexpr int T = D / 8;
  const AttendArgs& a = f.p;
  grid_dep_wait();
  grid_dep_launch();
  const int C = gridDim.x, c0 = blockIdx.x;
  const int4 meta = a.meta[c0];
  if (meta.x < 0) return;
  const int rows = f.narrow ? kTile : 2 * kTile;
  const int row = blockIdx.y * (256 / T) + threadIdx.x / T, c = (threadIdx.x % T) * 8;
  const AttendUnit w = attend_unit(f, meta.x, false);
  int h, i;
  if (!attend_row(f, w, row / kTile, row % kTile, h, i)) return;
  // Slots: 2 c0 + 1, then 2 k of every later CTA k up to meta.y; four parts' loads in flight.
  float m = -INFINITY, sum = 0.f, acc[8] = {};
  for (int k0 = c0; k0 <= meta.y; k0 += 4) {
    float lse2[4];
    float4 x[4], y[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int k = k0 + p;
      lse2[p] = -INFINITY;
      x[p] = y[p] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k > meta.y || part_is_empty(meta.z, C, k)) continue;
      const size_t at = static_cast<size_t>(k == c0 ? 2 * k + 1 : 2 * k) * rows + row;
      const float4* v = reinterpret_cast<const float4*>(f.part + at * D + c);
      lse2[p] = f.part_lse2[at];
      x[p] = v[0];
      y[p] = v[1];
    }
    const float top = fmaxf(fmaxf(fmaxf(lse2[0], lse2[1]), fmaxf(lse2[2], lse2[3])), m);
    // No part has seen a key yet: every weight is 0. (The maximum passes a part's NaN over; its weight does not.)
    const float ref = top == -INFINITY ? 0.f : top;
    const float g = exp2f(m - ref);
    sum *= g;
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] *= g;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float e = exp2f(lse2[p] - ref);
      const float v[8] = {x[p].x, x[p].y, x[p].z, x[p].w, y[p].x, y[p].y, y[p].z, y[p].w};
      sum += e;
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = fmaf(e, v[q], acc[q]);
    }
    m = top;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(acc[2 * q] * inv, acc[2 * q + 1] * inv);
  *reinterpret_cast<uint4*>(f.out.p + w.b * f.out.sb + h * f.out.sh + i * f.out.sn + c) =
      make_uint4(o[0], o[1], o[2], o[3]);
  if (c == 0)
    f.lse[(static_cast<size_t>(w.b) * a.H + h) * a.Nq + i] =
        sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace sla
