// What the dense attention kernels (forward, dQ, dK / dV) share: the problem, the visible key
// ranges, tensor-core products over 128-row tiles, and row stores.
//
// All of them work on tiles of 128 rows x D channels in shared memory: D / 64 boxes of 128
// rows x 128 bytes in TMA's 128-byte swizzle. Two kinds of product cover forward and backward:
//   ss: D[128 x 128 or 64] = A B^T over D channels, both tiles read as rows x channels (K-major)
//   ts: D[128 x D] (+)= P B over 64 or 128 rows, P (bf16) in TMEM, B read row by row (MN-major)
#pragma once

#include "sm100.cuh"

namespace sla {

struct AttendArgs {
  int B, H, Hk, G, Nq, Nk;  // G = H / Hk query heads share a key head
  int causal;
  float scale, scale_log2;  // scale, scale * log2(e)
  const int32_t* lens;      // [B] keys of each sequence, or null (Nk)
  uint32_t* err;
  // the launch's work items (see AttendWork)
  int units;
  int waves;    // units c, c + gridDim.x, ... that CTA c takes whole, this many of them
  int uniform;  // every unit has the same number of steps
  int spans;    // not 0: units are taken whole and longest first, |spans| of them to a head, of which the last
                // (below 0: the first) is the longest
  int4* meta;   // [gridDim.x] what attend_join_kernel / attend_sum_kernel join (null: nothing is cut)
};

// Blocks of three warpgroups: the first holds the TMA and the MMA warp, the other two the warps
// that compute. 384 threads are launched with 168 registers each (64512); the first warpgroup
// keeps 72 and the others take 216: 128 * (72 + 2 * 216) = 64512.
constexpr int kThreads = 384;
constexpr int kIssueRegs = 72, kComputeRegs = 216;
static_assert(128 * (kIssueRegs + 2 * kComputeRegs) <= kThreads * 168, "more registers than the block has");

// The first warpgroup's warps. Two issue MMAs, each its own chain of products: what one warp needs to
// wait for a barrier, issue eight MMAs and commit them is over 1000 cycles, about what the tensor
// cores need for them.
constexpr int kProducerWarp = 0, kMmaWarp = 1, kScheduleWarp = 2, kMmaWarp2 = 3;

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

// How a launch's units are shared out. CTA c first takes `waves` whole units c, c + C, ...
// (neighbouring CTAs work on neighbouring units, so a head's tiles stay in L2). The steps of all
// units behind those are laid end to end, each unit followed by kUnitCost steps that stand for
// its loads and its epilogue, and cut into C equal ranges, one per CTA: every CTA gets the same
// work whatever the lengths are, and at most its first and last unit is a part of one. A part
// (steps [lo, hi) of n) is written as fp32 rows into slot 2c (it continues a unit) or 2c + 1 (it
// begins one) and joined afterwards in ascending CTA order. A unit without steps counts as one.
constexpr int kUnitCost = 2;

struct AttendWork {
  int k, u, off, left;
  long long end, total;  // of the range, and all steps

  // The next unit u_ and the steps [lo, hi) of its n that this CTA takes; `to` is where its range
  // ends, in steps from the unit's first.
  template <class Steps>
  __device__ __forceinline__ bool next(const AttendArgs& a, const Steps& steps, int& u_, int& lo, int& hi, int& n,
                                       int& to) {
    if (k < a.waves) {
      // Longest first: every other wave runs backwards, so that long units meet short ones.
      u_ = k * gridDim.x + (a.spans && (k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      ++k;
      if (u_ >= a.units) return false;
      if (a.spans) {
        const int n_spans = abs(a.spans), heads = a.units / n_spans, rank = u_ / heads;
        u_ = u_ % heads * n_spans + (a.spans > 0 ? n_spans - 1 - rank : rank);
      }
      lo = 0;
      hi = n = to = max(1, steps(u_));
      return true;
    }
    while (left > 0) {
      u_ = u++;
      n = max(1, steps(u_));
      lo = off;
      to = min(n + kUnitCost, off + left);
      left -= to - off;
      off = 0;
      hi = min(n, to);
      if (lo < hi) return true;
    }
    return false;
  }
};

// Run by all `threads` (a multiple of 32, at most 1024) threads of the block before its roles
// part: this CTA's range. Thread 0 clears the CTA's entry of meta.
template <class Steps>
__device__ __forceinline__ AttendWork attend_work(const AttendArgs& a, const Steps& steps, int threads) {
  __shared__ int warp_sum[32];
  __shared__ int found[2];
  const int C = gridDim.x, c = blockIdx.x, tid = threadIdx.x;
  const int base = min(a.units, a.waves * C), R = a.units - base;
  AttendWork w{0, 0, 0, 0, 0, 0};
  if (tid == 0 && a.meta) a.meta[c] = make_int4(-1, 0, 0, 0);
  if (R == 0) return w;
  long long total, start, end;
  if (a.uniform) {
    const int n = max(1, steps(base)) + kUnitCost;
    total = static_cast<long long>(R) * n;
    start = total * c / C;
    end = total * (c + 1) / C;
    w.u = base + static_cast<int>(start / n);
    w.off = static_cast<int>(start % n);
  } else {
    // Each thread sums a run of units; a scan over the block gives the runs' places.
    const int run = (R + threads - 1) / threads;
    const int lo = base + min(R, tid * run), hi = base + min(R, (tid + 1) * run);
    int sum = 0;
    for (int u = lo; u < hi; ++u) sum += max(1, steps(u)) + kUnitCost;
    int scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, o);
      if ((tid & 31) >= o) scan += v;
    }
    if ((tid & 31) == 31) warp_sum[tid >> 5] = scan;
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < threads / 32; ++i) {
      if (i < (tid >> 5)) before += warp_sum[i];
      all += warp_sum[i];
    }
    total = all;
    start = total * c / C;
    end = total * (c + 1) / C;
    int at = before + scan - sum;  // this run's place
    if (start >= at && start < at + sum) {
      for (int u = lo; u < hi; ++u) {
        const int n = max(1, steps(u)) + kUnitCost;
        if (start < at + n) {
          found[0] = u;
          found[1] = static_cast<int>(start) - at;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
    w.u = found[0];
    w.off = found[1];
  }
  w.left = static_cast<int>(end - start);
  w.end = end;
  w.total = total;
  return w;
}

// A whole warp waits; all lanes get the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, abort_flag));
}

// How long the scheduler waits for the longest unit so far, of `steps` steps, to end: a key tile's unit has up to 2^30
// (query heads of a group x query tiles), and at 2.1 us a step (D = 128, 1.65 GHz) 960 thousand pass the limit of
// every other wait, which is for one step. Four times that pace is waited for.
constexpr uint64_t kStepWaitNs = 8400;
__host__ __device__ constexpr uint64_t item_wait_ns(int steps) {
  return SLA_WAIT_LIMIT_NS + kStepWaitNs * static_cast<uint64_t>(steps);
}

// The unit that a CTA works on, as its scheduler warp passes it to the other warps.
struct __align__(16) AttendItem {
  int v[12];
};

// A ring of items in shared memory: one warp fills it while the others are still busy with
// earlier units, so that finding a unit (divisions, lengths in global memory) costs them nothing.
template <int COMPUTE_WARPS>
struct ItemRing {
  static constexpr int SLOTS = 4;
  static constexpr int READERS = 3 + COMPUTE_WARPS;  // the producer, the MMA warps and the computing warps
  AttendItem item[SLOTS];
  uint64_t full[SLOTS], empty[SLOTS];

  __device__ __forceinline__ void init() {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], READERS);
    }
  }
  // By one thread. A slot comes free when the readers take the unit in it, which is when they end the one before:
  // no unit so far has had more than `steps` steps.
  __device__ __forceinline__ bool put(uint32_t i, const AttendItem& x, int steps, uint32_t* err,
                                      volatile int* abort_flag) {
    const uint32_t s = i % SLOTS, r = i / SLOTS;
    if (r > 0 && !mbar_wait_for(&empty[s], (r - 1) & 1, err, abort_flag, item_wait_ns(steps))) return false;
    item[s] = x;
    mbar_arrive(&full[s]);
    return true;
  }
  // By one thread, as one of READERS.
  __device__ __forceinline__ bool get_one(uint32_t i, AttendItem& x, uint32_t* err, volatile int* abort_flag) {
    const uint32_t s = i % SLOTS, r = i / SLOTS;
    if (!mbar_wait(&full[s], r & 1, err, abort_flag)) return false;
    x = item[s];
    mbar_arrive(&empty[s]);
    return true;
  }
  // By a whole warp (one of READERS); false: the wait ran out.
  __device__ __forceinline__ bool get(uint32_t i, AttendItem& x, uint32_t* err, volatile int* abort_flag) {
    const uint32_t s = i % SLOTS, r = i / SLOTS;
    if (!warp_wait(&full[s], r & 1, err, abort_flag)) return false;
    x = item[s];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[s]);
    return true;
  }
};

// Where a CTA begins a unit that others go on with: that unit, the last CTA with a part of it and
// all steps, for the join.
__device__ __forceinline__ void note_part(const AttendArgs& a, const AttendWork& w, int u, int lo, int hi, int n,
                                          int to) {
  if (lo != 0 || hi == n) return;
  const int last = static_cast<int>(((w.end - to + n) * gridDim.x - 1) / w.total);  // holds the unit's last step
  a.meta[blockIdx.x] = make_int4(u, last, static_cast<int>(w.total), 0);
}

// The slot of CTA c's part [lo, hi) of n, or -1 where it holds the whole unit.
__device__ __forceinline__ int part_slot(int lo, int hi, int n) {
  if (lo == 0 && hi == n) return -1;
  return 2 * static_cast<int>(blockIdx.x) + (lo == 0 ? 1 : 0);
}

// With fewer steps than CTAs some ranges are empty, and their CTAs hold no part.
__device__ __forceinline__ bool part_is_empty(int total, int C, int c) {
  return static_cast<long long>(total) * c / C == static_cast<long long>(total) * (c + 1) / C;
}


// The MMA warp runs converged and every tcgen05 operation is predicated on its one issuing lane
// (`lead`): operands stay in uniform registers, and issuing an MMA costs no branch. An MMA of 128
// rows takes the tensor cores about 64 cycles, so that the issue, not the product, is the limit
// where the operands are built anew for each.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  if (accumulate)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.eq.u32 p, 0, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, 0, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  if (accumulate)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.eq.u32 p, 0, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, 0, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(lead)
        : "memory");
}
// Arrive on the mbarrier when every MMA issued so far is done.
__device__ __forceinline__ void mma_commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// A 128-byte-swizzle descriptor in two words: the low one holds the start address (in units of 16
// bytes, so the steps of a product add constants) and the leading offset, the high one is a constant.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 1024 bytes between 8-row groups
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
// The same value in all lanes, as the compiler should know.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// D[128 x N] = A B^T over D channels, N = 128 rows of B or 64.
template <int D, int N>
__device__ __forceinline__ void issue_ss(uint32_t lead, uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem) {
  constexpr uint32_t id = idesc_bf16_f32(128, N, 0, 0);
  const uint32_t ad = uniform(desc_lo(a_smem, 16)), bd = uniform(desc_lo(b_smem, 16));
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t step = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
    mma_ss(lead, d_tmem, desc_of(ad + step), desc_of(bd + step), id, kk > 0);
  }
}

// D[128 x D] (+)= P B over the rows [16 K0, 16 K1) of the tile at b_smem. P's 16-row steps are 8 TMEM
// columns each; after every GROUP steps P's columns go on GAP columns behind the group's first.
template <int D, int K0, int K1, int GROUP, int GAP>
__device__ __forceinline__ void issue_ts(uint32_t lead, uint32_t d_tmem, uint32_t p_tmem, uint32_t b_smem,
                                         bool accumulate) {
  constexpr uint32_t id = idesc_bf16_f32(128, D, 0, 1);
  const uint32_t bd = uniform(desc_lo(b_smem, kBox));
  if (accumulate)
    mma_ts(lead, d_tmem, p_tmem + K0 / GROUP * GAP + K0 % GROUP * 8, desc_of(bd + (K0 * 2048 >> 4)), id, true);
  else
    mma_ts(lead, d_tmem, p_tmem + K0 / GROUP * GAP + K0 % GROUP * 8, desc_of(bd + (K0 * 2048 >> 4)), id, false);
#pragma unroll
  for (int kk = K0 + 1; kk < K1; ++kk)
    mma_ts(lead, d_tmem, p_tmem + kk / GROUP * GAP + kk % GROUP * 8, desc_of(bd + (kk * 2048 >> 4)), id, true);
}

// A place in a ring of n stages: its index, and the parity of its current round.
struct RingPos {
  uint32_t s = 0, parity = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++s == n) {
      s = 0;
      parity ^= 1;
    }
  }
};

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

// Where a kernel writes whole rows.
struct RowOut {
  __nv_bfloat16* p;
  long long sb, sh, sn;  // elements
  int wide;              // rows start on 32-byte boundaries
};

}  // namespace sla
