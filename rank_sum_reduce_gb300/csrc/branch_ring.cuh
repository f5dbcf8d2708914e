// branch_ring.cuh -- what the two pipelines of a block's branch share
// (branch_tma.cuh, branch_backward_tma.cuh): tiles of rows streamed through a ring
// of shared-memory stages by TMA bulk copies.
//
// A tile is `teams` consecutive rows (the last one fewer).  One bulk copy brings the
// same slice (a rank, the residual ...) of all rows of a tile; each team of consumer
// warps owns one of them.  A CTA takes every so-many-th tile; in the backward of a
// gate whose rows fewer than all rows share, one contiguous span of rows, whose tiles
// end where a gate row's rows do, so that a gate row is cut by few CTAs.  A row that
// is split over a cluster is the tile of its CTAs, each with one team and its part of
// every slice.
//
// Slices travel in stages of up to `group`, with one full and one empty barrier
// each: the ranks' in order, then those that a row needs to its end, which share
// one stage, so a row waits for and frees few of them.  With few ranks a whole
// tile is one stage (backward, W = 1: one wait and one release per row instead of
// four; the instructions of a row are what bounds it there).
#pragma once

#include "branch.cuh"
#include "ring.cuh"

namespace car {
namespace {

// The pipelines have an instance for each kind of gate, with dropout and without: what
// a row does not do costs it registers and instructions all the same when it is found
// out at run time (backward, W = 1, M = 16389, N = 4096 bf16 without a norm 145 us
// against 103).
enum GateKind : int { kGateNone = 0, kGateShared = 1, kGateOwn = 2 };
// Where a row's gate comes from in the forward: a row in shared memory (also: no
// gate), the ring, L2.
enum GateFrom : int { kFromFactor = 0, kFromRing = 1, kFromRows = 2 };
inline int gate_kind(const BranchArgs& br) { return !br.gate ? kGateNone : br.gate_span == 0 ? kGateOwn : kGateShared; }

// A CTA is four warpgroups of consumers (of which the teams may leave a few warps
// idle) and one whose first warps issue copies.  It is launched with 96 registers a
// thread, the most that five warps on each of the SM's schedulers can have, and the
// consumers take what the producers do without: 512 * 112 + 128 * 24 registers of
// 640 * 96.  In 96 the backward spills 40 to 90 bytes, which costs more than
// anything else in a row (W = 1, M = 13332, N = 1160 fp16, one gate: 66 us against
// 43; N = 11072, W = 4, M = 2000 with norms 105 against 97).
constexpr int kRingConsumers = 512, kRingThreads = 640;
template <bool CONSUMER>
__device__ __forceinline__ void take_registers() {  // every thread of a warpgroup
  if constexpr (CONSUMER) asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 24;");
}

// The columns of this CTA: all, or with SPLIT its part of every row.
template <bool SPLIT>
struct Part {
  int crank, group, groups;  // place in the cluster; the cluster's, of how many
  int col0, V;               // first vector of a row, and how many
  __device__ __forceinline__ explicit Part(const RingPlan& p) {
    crank = SPLIT ? (int)cluster_rank() : 0;
    group = SPLIT ? (int)blockIdx.x / p.cluster : (int)blockIdx.x;
    groups = SPLIT ? (int)gridDim.x / p.cluster : (int)gridDim.x;
    col0 = SPLIT ? crank * p.chunk : 0;
    V = SPLIT ? min(p.chunk, p.vec_per_row - col0) : p.vec_per_row;
  }
};

// The tiles of this CTA in order: every so-many-th, or with CUTS, for a gate that rows
// share, those of one contiguous span.
template <bool CUTS>
struct Tiles {
  int row, end, cut, step;
  template <bool SPLIT>
  __device__ __forceinline__ Tiles(const RingPlan& p, const Part<SPLIT>& part) {
    if (CUTS && p.gate_span) {
      row = (int)span_start(p.rows, part.groups, part.group);
      end = (int)span_start(p.rows, part.groups, part.group + 1);
      cut = (int)(((uint32_t)row / p.gate_span + 1) * p.gate_span);
      step = 0;
    } else {
      row = part.group * p.teams;
      end = cut = p.rows;
      step = part.groups * p.teams;
    }
  }
  __device__ __forceinline__ bool more(const RingPlan& p) const { return row < (CUTS ? end : p.rows); }
  __device__ __forceinline__ int count(const RingPlan& p) const {
    return min((CUTS ? min(end, cut) : p.rows) - row, p.teams);
  }
  __device__ __forceinline__ void next(const RingPlan& p) {
    if (!CUTS || step) {
      row += step;
    } else {
      row += count(p);
      if (row == cut) cut += p.gate_span;
    }
  }
};

// Bytes of a slice's place in a stage.
__host__ __device__ inline uint32_t slice_stride(const RingPlan& p) { return (uint32_t)p.teams * (uint32_t)p.chunk * 16u; }

// Barriers and small arrays (static shared memory).  Row statistics are sums times a
// rounded 1 / N here, where the row kernels divide: a rounding more.
struct RingShared {
  uint64_t full[kMaxRingStages], empty[kMaxRingStages];
  RowSums cluster;          // its exchange, where CTAs share a row
  uint4 drop;               // the generator's state, where registers are short,
  uint32_t first_vec;       // and the launch's first vector of the [M, N] problem
  float4 warp[48];          // [teams][2][3][warps of a team, in fours]: a team has 512 / teams threads at most
  int abort;
};

__device__ __forceinline__ void ring_init(const RingPlan& p, RingShared& s) {  // all threads, before a barrier
  if (threadIdx.x < 48) s.warp[threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; i++) {
      mbar_init(&s.full[i], p.producers);
      mbar_init(&s.empty[i], (uint32_t)(p.teams * p.team_threads) >> 5);
    }
    s.abort = 0;
    row_sums_init(s.cluster, p.cluster);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
}

// As wait_bounded (ring.cuh), but a thread that has to wait is suspended for up to a
// few microseconds at a time: polling warps take issue slots from the others.
__device__ __forceinline__ bool wait_suspended(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  const unsigned long long t0 = globaltimer();
  for (uint32_t i = 0; i < (1u << 30); i++) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(4000u)
        : "memory");
    if (ok) return true;
    if (*abort || globaltimer() - t0 > kWaitLimitNs) return false;
  }
  return false;
}

// Producer `who` of p.producers: issues every p.producers-th slice of each stage,
// then waits for the stages that were filled.  source(q): slice q of row 0.
template <bool CUTS, bool SPLIT, class Source>
__device__ __forceinline__ void ring_produce(const RingPlan& p, const Part<SPLIT>& part, uint8_t* ring, RingShared& s, int who,
                                             unsigned int* err, Source source) {
  const int S = p.stages, slices = p.ranks + p.held;
  const uint32_t stride = slice_stride(p);
  int place = 0;
  uint32_t phase = 0, issued = 0;
  bool ok = true;
  for (Tiles<CUTS> t(p, part); t.more(p) && ok; t.next(p)) {
    const int64_t off = t.row * (int64_t)p.row_bytes + part.col0 * 16;
    const uint32_t bytes = (uint32_t)t.count(p) * (uint32_t)part.V * 16u;
    for (int q = 0; q < slices;) {
      // a stage ends with the ranks unless all of the tile is one
      const int n = p.tile_stages == 1 ? slices : q < p.ranks ? min(p.group, p.ranks - q) : slices - q;
      if (issued >= (uint32_t)S && !mbar_try_wait(&s.empty[place], phase ^ 1u) && !wait_suspended(&s.empty[place], phase ^ 1u, &s.abort)) {
        ok = false;
        break;
      }
      const int mine = (n - who + p.producers - 1) / p.producers;
      mbar_arrive_expect_tx(&s.full[place], bytes * (uint32_t)mine);
      uint8_t* to = ring + (size_t)place * p.group * stride;
      for (int i = who; i < n; i += p.producers) bulk_load(to + (size_t)i * stride, source(q + i) + off, bytes, &s.full[place]);
      q += n;
      issued++;
      if (++place == S) {
        place = 0;
        phase ^= 1u;
      }
    }
  }
  if (!ok) {
    atomicOr(err, 1u);
    *static_cast<volatile int*>(&s.abort) = 1;
  }
  // No copy may still be on its way into a CTA that has exited.  A stage that the
  // other producer gave up on does not complete: that wait runs out.
  const int used = issued < (uint32_t)S ? (int)issued : S;
  for (int k = 0; k < used; k++) {
    const uint32_t c = issued - 1u - (uint32_t)k;
    if (!wait_bounded_drain(&s.full[c % (uint32_t)S], (c / (uint32_t)S) & 1u)) atomicOr(err, 1u);
  }
}

// A consumer thread's place in the ring.  Where a wait runs out the thread carries
// on with whatever the stage holds and stores nothing more: it reaches every one of
// its team's barriers, which have no limit of their own, and later waits return at
// once.
struct RingReader {
  const RingPlan& p;
  RingShared& s;
  unsigned int* err;
  int place = 0;
  uint32_t phase = 0;
  bool failed = false;
  __device__ __forceinline__ RingReader(const RingPlan& plan, RingShared& shared, unsigned int* e) : p(plan), s(shared), err(e) {}
  __device__ __forceinline__ void wait() {
    if (mbar_try_wait(&s.full[place], phase) || failed || wait_suspended(&s.full[place], phase, &s.abort)) return;
    failed = true;
    atomicOr(err, 1u);
    *static_cast<volatile int*>(&s.abort) = 1;
  }
  __device__ __forceinline__ void release() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&s.empty[place]);
    if (++place == p.stages) {
      place = 0;
      phase ^= 1u;
    }
  }
  // A tile in which this team has no row.
  __device__ __forceinline__ void skip() {
    for (int k = 0; k < p.tile_stages; k++) {
      wait();
      release();
    }
  }
};

// The rank sum of this thread's vectors of a row, from the stages that hold the
// ranks; `mine` is the row in stage 0, at[k] this thread's vectors in it.  Leaves
// the reader at the stage that holds the row's other slices, waited for, and
// returns where they begin.
//
// Without BRANCHES a thread whose vectors lie past the row's end works on its last
// one (at[]) and leaves its sums and stores out, here and in what follows: with no
// branches around them the vectors' loads and arithmetic overlap.  Where many
// values are alive that would spill.
template <int DT, int VPT, bool BRANCHES>
__device__ __forceinline__ const uint8_t* ring_rank_sum(const RingPlan& p, RingReader& in, const uint8_t* mine,
                                                        const bool (&ok)[VPT], const int (&at)[VPT], float2 (&acc)[VPT][Pack<DT>::kN / 2]) {
  constexpr int E = Pack<DT>::kN;
  const uint32_t stride = slice_stride(p);
  const bool whole = p.tile_stages == 1;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
#pragma unroll
    for (int e = 0; e < E / 2; e++) acc[k][e] = both(-0.f);  // -0 + x is x, whatever x is
  }
  int q = 0;
  while (true) {
    in.wait();
    const uint8_t* slice = mine + (uint32_t)in.place * (uint32_t)p.group * stride;
    if (q == p.ranks) return slice;
    const int n = min(p.group, p.ranks - q);
    for (int i = 0; i < n; i++, slice += stride) {
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (BRANCHES && !ok[k]) continue;
        float2 f[E / 2];
        widen2<DT>(lds16(slice + at[k]), f);
#pragma unroll
        for (int e = 0; e < E / 2; e++) acc[k][e] = add2(acc[k][e], f[e]);
      }
    }
    if (whole) return slice;
    q += n;
    in.release();
  }
}

// Barriers of the consumers: one for each team of several warps (there are at most
// eight), one for all.
__device__ __forceinline__ void team_barrier(const RingPlan& p, int team) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(p.team_threads) : "memory");
}
__device__ __forceinline__ void consumers_barrier(const RingPlan& p) {
  __syncwarp();
  asm volatile("bar.sync 15, %0;" ::"r"(p.teams * p.team_threads) : "memory");
}

// Sums over a row: the warps of a team.  Every thread adds the warps' partials
// itself, in the same order; they are double-buffered by the parity of the team's
// exchange number x (what exchange x wrote is overwritten by x + 2, after the
// barrier of x + 1, which a warp reaches only once it has read x's).  The row waits
// for each exchange twice, so it is kept short: a barrier in hardware and broadcast
// loads in place of mbarriers and a second round of shuffles.
//
// Within a warp several sums share their shuffles: after the first step the lower
// half of the lanes carries one, the upper half another, after the second a quarter
// each.  Three sums: 6 shuffles, where one after the other would take 15.
template <bool SPLIT, int NS>
__device__ __forceinline__ void team_sums(const RingPlan& p, RingShared& s, int team, uint32_t x, float (&v)[NS],
                                          const ClusterWait& peers) {
  constexpr uint32_t ALL = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, nwarps = p.team_threads >> 5, warp = (threadIdx.x - team * p.team_threads) >> 5;
  float t;        // of sum `which`, in the first of every eight lanes
  int which = 0;
  if constexpr (NS == 1) {
    t = v[0];
    t += __shfl_xor_sync(ALL, t, 16);
    t += __shfl_xor_sync(ALL, t, 8);
  } else {
    const bool upper = lane & 16;
    t = (upper ? v[1] : v[0]) + __shfl_xor_sync(ALL, upper ? v[0] : v[1], 16);
    which = upper ? 1 : 0;
    if constexpr (NS == 2) {
      t += __shfl_xor_sync(ALL, t, 8);
    } else {
      const float c = v[NS - 1] + __shfl_xor_sync(ALL, v[NS - 1], 16);
      const bool third = lane & 8;
      t = (third ? c : t) + __shfl_xor_sync(ALL, third ? t : c, 8);
      if (third) which = 2;
    }
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(ALL, t, o);
  if (nwarps == 1) {
    v[0] = __shfl_sync(ALL, t, 0);
    if constexpr (NS >= 2) v[1] = __shfl_sync(ALL, t, 16);
    if constexpr (NS == 3) v[2] = __shfl_sync(ALL, t, 8);
    if constexpr (SPLIT) cluster_sums(s.cluster, v, x, p.cluster, peers);
    return;
  }
  const int fours = (nwarps + 3) >> 2;
  float4* w = s.warp + (team * 2 + (x & 1u)) * 3 * fours;
  // lanes 0, 16 and 8 write the sums 0, 1 and 2
  if (NS == 1 ? lane == 0 : NS == 2 ? (lane & 15) == 0 : (lane & 7) == 0 && lane < 24)
    reinterpret_cast<float*>(w)[which * 4 * fours + warp] = t;
  team_barrier(p, team);
#pragma unroll
  for (int i = 0; i < NS; i++) {
    const float4 f = w[i * fours];
    float2 a = add2(make_float2(f.x, f.y), make_float2(f.z, f.w));
    if (fours > 1) {
      const float4 g = w[i * fours + 1];
      a = add2(a, add2(make_float2(g.x, g.y), make_float2(g.z, g.w)));
    }
    if (fours > 2) {
#pragma unroll
      for (int j = 2; j < 4; j++) {
        if (j < fours) {
          const float4 g = w[i * fours + j];
          a = add2(a, add2(make_float2(g.x, g.y), make_float2(g.z, g.w)));
        }
      }
    }
    v[i] = __fadd_rn(a.x, a.y);
  }
  if constexpr (SPLIT) cluster_sums(s.cluster, v, x, p.cluster, peers);
}

// Rows of factors in shared memory, in fp32: every vector of them is used once or
// twice per row, and widening one takes eight instructions.  A vector of a 16-bit
// type fills two float4, which lie in two planes so that a warp that takes
// consecutive vectors reads either without bank conflicts.
template <int DT>
__device__ __forceinline__ void row_to_shared(const uint4* __restrict__ a, const uint4* __restrict__ b, int vecs, int threads,
                                              uint8_t* to) {
  constexpr int E = Pack<DT>::kN;
  for (int v = threadIdx.x; v < vecs; v += threads) {
    float2 f[E / 2], g[E / 2];
    widen2<DT>(__ldg((a ? a : b) + v), f);
    if (a && b) {
      widen2<DT>(__ldg(b + v), g);
#pragma unroll
      for (int e = 0; e < E / 2; e++) f[e] = mul2(f[e], g[e]);
    }
#pragma unroll
    for (int e = 0; e < E / 2; e += 2)
      reinterpret_cast<float4*>(to)[(e / 2) * vecs + v] = make_float4(f[e].x, f[e].y, f[e + 1].x, f[e + 1].y);
  }
}
template <int DT>
__device__ __forceinline__ void row_from_shared(const uint8_t* from, int vecs, int v, float2 (&f)[Pack<DT>::kN / 2]) {
#pragma unroll
  for (int e = 0; e < Pack<DT>::kN / 2; e += 2) {
    const float4 x = reinterpret_cast<const float4*>(from)[(e / 2) * vecs + v];
    f[e] = make_float2(x.x, x.y);
    f[e + 1] = make_float2(x.z, x.w);
  }
}

}  // namespace
}  // namespace car
