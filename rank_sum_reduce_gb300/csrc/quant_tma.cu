// quant_tma.cu -- rank sum + residual add + RMSNorm with an 8-bit output and
// its scales for many rows, with the rows streamed into shared memory by TMA
// bulk copies: the operation of fused_quant.cu, organised as the backward's
// pipeline kernel (norm_backward_tma.cu).  A persistent CTA per SM takes tiles
// of `teams` consecutive rows; one bulk copy brings the same slice -- x_0 ..
// x_{W-1}, residual -- of all rows of a tile, and each team of consumer warps
// owns one row.  max |t| is found before the row statistic's barrier and
// crosses it with the sum of squares (quant.cuh).  Every mbarrier wait is
// bounded.
//
// VPT: vectors per consumer thread.  Four (the weight row in shared memory) or
// two (in registers): more of them divide the fixed work of a row (sums over
// the warp, a division, addresses) and make room for more teams, fewer keep a
// row's chain short.  Up to three ranks the CTA is bound by that work, and four
// are faster (W = 1, M = 16389, N = 4096 bf16: 84 -> 70 us; W = 2, M = 2000, N
// = 8192: 26.5 -> 23.9); with more the row waits for its slices and two are (W
// = 8, M = 512, N = 8192: 15.9 against 16.9; W = 4, M = 2000, N = 4096 17.8
// with six slots against 19.0 with four), unless they leave threads without a
// row, which three do not (W = 4, M = 8191, N = 6144: 112 against 95; W = 8, M =
// 1500, N = 5000 31.7 against 25.7, four 27.5).  Rows of more than 2048 vectors
// take five to eight, as few as 512 threads need (W = 1, M = 2000, N = 20000
// bf16: five 52 us, six 65, eight 78), the weight read from L2 once per row (64
// KB of it beside the ring would leave two slots).  The instances for six, seven
// and eight 16-bit vectors spill 24 to 116 bytes (96 registers).  A
// thread's squares are then up to 32 fmas in a row, with 10 levels of additions
// behind them (the halves', a warp's, 16 warps').
#include "car_launch.h"
#include "quant.cuh"
#include "ring.cuh"

namespace car {
namespace {

struct QuantTmaParams {
  RankPtrs in;
  const uint8_t* residual;
  const uint4* weight;
  uint4* residual_out;
  uint4* norm_out;  // may be null
  uint4* ar_out;    // may be null
  QuantOut out;
  unsigned int* err;
  float eps;
  float cols;
  int64_t rows;
  int row_bytes;
  int vec_per_row;
  int slots;
  int teams;         // rows of a tile
  uint32_t producers;   // 1 or 2
  int team_threads;  // multiple of 32
  int nranks;
};

__device__ __forceinline__ const uint8_t* slice_source(const QuantTmaParams& p, int q) {
  return q < p.nranks ? static_cast<const uint8_t*>(p.in.p[q]) : p.residual;
}
__device__ __forceinline__ uint32_t tile_bytes(const QuantTmaParams& p, int64_t row) {
  const int64_t left = p.rows - row;
  return (uint32_t)(left < p.teams ? left : p.teams) * (uint32_t)p.row_bytes;
}

// Producer `who`: every p.producers-th copy of the CTA's sequence; then it waits
// for the copies that it issued (see norm_backward_tma.cu).
__device__ __forceinline__ void produce(const QuantTmaParams& p, uint8_t* ring, uint64_t* full, uint64_t* empty,
                                        volatile int* s_abort, uint32_t who) {
  const int S = p.slots;
  const size_t stride = (size_t)p.teams * p.row_bytes;
  int slot = 0;
  uint32_t phase = 0;
  uint64_t issued = 0;
  bool ok = true;
  for (int64_t row = (int64_t)blockIdx.x * p.teams; row < p.rows && ok; row += (int64_t)gridDim.x * p.teams) {
    const int64_t off = row * (int64_t)p.row_bytes;
    const uint32_t bytes = tile_bytes(p, row);
    for (int q = 0; q <= p.nranks; q++) {
      if (((uint32_t)issued & (p.producers - 1u)) == who) {
        if (issued >= (uint64_t)S && !wait_bounded(&empty[slot], phase ^ 1u, s_abort)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[slot], bytes);
        bulk_load(ring + slot * stride, slice_source(p, q) + off, bytes, &full[slot]);
      }
      issued++;
      if (++slot == S) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
  if (!ok) {
    atomicOr(p.err, 1u);
    *s_abort = 1;
  }
  const int used = issued < (uint64_t)S ? (int)issued : S;
  for (int k = 0; k < used; k++) {  // copy number c is use c / S of slot c % S
    const uint64_t c = issued - 1 - (uint64_t)k;
    if (((uint32_t)c & (p.producers - 1u)) != who) continue;
    if (!wait_bounded_drain(&full[c % (uint64_t)S], (uint32_t)((c / (uint64_t)S) & 1u))) atomicOr(p.err, 1u);
  }
}

// With three or four vectors per thread the weight row lies in shared memory,
// widened: a load more per vector for eight instructions less (W = 1, M = 5851,
// N = 1968: 13.3 against 13.6 us; M = 6124, N = 2592 19.1 against 19.5).  The
// vectors' halves lie in two planes, so that a warp reads either without bank
// conflicts.
template <int DT, int VPT>
constexpr bool kWideWeight = DT != kFP32 && (VPT == 3 || VPT == 4);

template <int DT, int VPT>
__device__ __forceinline__ void consume(const QuantTmaParams& p, const uint8_t* ring, const uint8_t* s_weight, uint64_t* full,
                                        uint64_t* empty, uint64_t* rowbar, float2* s_warp, volatile int* s_abort) {
  constexpr int E = Pack<DT>::kN;
  const int S = p.slots, T = p.team_threads, n = p.nranks;
  const int team = threadIdx.x / T, tid = threadIdx.x - team * T;
  const int warp = tid >> 5, lane = threadIdx.x & 31, nwarps = T >> 5;
  const size_t stride = (size_t)p.teams * p.row_bytes;
  const uint8_t* mine = ring + (size_t)team * p.row_bytes + 16 * tid;  // this thread's first vector in slot 0
  rowbar += team;
  s_warp += team * 2 * nwarps;
  uint4 wv[VPT];
  bool ok[VPT];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    ok[k] = tid + k * T < p.vec_per_row;
    if (VPT == 2) wv[k] = ok[k] ? __ldg(p.weight + tid + k * T) : make_uint4(0u, 0u, 0u, 0u);
  }
  auto widen2 = [](uint4 v, float2 (&f)[E / 2]) {
    float t[E];
    Pack<DT>::widen(v, t);
#pragma unroll
    for (int e = 0; e < E / 2; e++) f[e] = make_float2(t[2 * e], t[2 * e + 1]);
  };
  auto weight = [&](int k, float2 (&f)[E / 2]) {
    if constexpr (kWideWeight<DT, VPT>) lds_wide(s_weight, p.vec_per_row, tid + k * T, f);
    else if constexpr (VPT == 2) widen2(wv[k], f);
    else if constexpr (VPT <= 4) widen2(lds16(s_weight + 16 * (tid + k * T)), f);
    else widen2(__ldg(p.weight + tid + k * T), f);
  };
  int slot = 0;
  uint32_t phase = 0, it = 0;
  bool failed = false;
  auto release = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
  };
  for (int64_t tile = (int64_t)blockIdx.x * p.teams; tile < p.rows; tile += (int64_t)gridDim.x * p.teams) {
    const int64_t row = tile + team;
    if (row >= p.rows) {  // a team without a row in the last tile only lets the slots go
      for (int q = 0; q <= n && !failed; q++) {
        failed = !wait_bounded(&full[slot], phase, s_abort);
        if (!failed) release();
      }
      break;
    }
    const int64_t rbase = row * (int64_t)p.vec_per_row + tid;
    float2 h[VPT][E / 2];
    for (int q = 0; q < n; q++) {
      if (!wait_bounded(&full[slot], phase, s_abort)) {
        failed = true;
        break;
      }
      const uint8_t* sl = mine + slot * stride;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (ok[k]) {
          float2 t[E / 2];
          widen2(lds16(sl + 16 * k * T), t);
#pragma unroll
          for (int e = 0; e < E / 2; e++) h[k][e] = q == 0 ? t[e] : add2(h[k][e], t[e]);
        }
      }
      release();
    }
    if (failed || !wait_bounded(&full[slot], phase, s_abort)) {
      failed = true;
      break;
    }
    // residual, first outputs, sum of squares; then h becomes t = h * w
    float2 ss = make_float2(0.f, 0.f);
    uint32_t gmax[VPT] = {};
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
        float2 rf[E / 2], wf[E / 2];
        float o[E];
        widen2(lds16(mine + slot * stride + 16 * k * T), rf);
        if (p.ar_out) {
#pragma unroll
          for (int e = 0; e < E / 2; e++) o[2 * e] = h[k][e].x, o[2 * e + 1] = h[k][e].y;
          st16(p.ar_out + rbase + k * T, Pack<DT>::narrow(o));
        }
        weight(k, wf);
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < E / 2; e++) {
          const float2 x = add2(h[k][e], rf[e]);
          o[2 * e] = x.x;
          o[2 * e + 1] = x.y;
          ss = fma2(x, x, ss);
          h[k][e] = mul2(x, wf[e]);
          m = max_abs(m, h[k][e].x, h[k][e].y);
        }
        gmax[k] = abs_bits(m);
        st16(p.residual_out + rbase + k * T, Pack<DT>::narrow(o));
      }
    }
    release();
    uint32_t tmax = spread_max<E>(p.out.kind, gmax);
    // row statistics: every warp adds the team's warp partials itself, in the
    // same order; they are double-buffered by row parity
    float sum = warp_sum(ss.x + ss.y);
    if (nwarps > 1) {
      float2* sw = s_warp + nwarps * (it & 1u);
      if (lane == 0) {
        sw[warp] = make_float2(sum, __uint_as_float(tmax));
        mbar_arrive(rowbar);
      }
      if (!wait_bounded(rowbar, it & 1u, s_abort)) {
        failed = true;
        break;
      }
      const float2 part = lane < nwarps ? sw[lane] : make_float2(0.f, 0.f);
      sum = warp_sum(part.x);
      if (p.out.kind == kScaleRow) tmax = warp_max(__float_as_uint(part.y));
    }
    it++;
    const float rms = rsqrtf(__fdiv_rn(sum, p.cols) + p.eps);
    const float inv_row = row_inverse(p.out, row, rms, tmax, tid == 0);
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const int v = tid + k * T;
      const bool grouped = p.out.kind == kScaleGroup128 || p.out.kind == kScaleMx32;
      const float inv = grouped ? group_inverse<E>(p.out, row, v, rms, gmax[k], ok[k]) : inv_row;
      if (ok[k]) {
        float t[E];
#pragma unroll
        for (int e = 0; e < E / 2; e++) t[2 * e] = h[k][e].x, t[2 * e + 1] = h[k][e].y;
        store_e4m3<E>(p.out.q + row * (int64_t)p.vec_per_row * E, v, t, rms, inv);
        if (p.norm_out) {
#pragma unroll
          for (int e = 0; e < E; e++) t[e] = __fmul_rn(t[e], rms);
          st16(p.norm_out + rbase + k * T, Pack<DT>::narrow(t));
        }
      }
    }
  }
  if (failed) {
    atomicOr(p.err, 1u);
    *s_abort = 1;
  }
}

template <int DT, int VPT>
__global__ void __launch_bounds__(512 + 32 * kProducers, 1) reduce_residual_rmsnorm_quant_tma_kernel(const QuantTmaParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int S = p.slots;
  uint8_t* s_weight = smem + (size_t)S * p.teams * p.row_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_weight + (VPT == 3 || VPT == 4 ? 2 * p.row_bytes : 0));
  uint64_t* empty = full + S;
  uint64_t* rowbar = empty + S;                            // [16], by team
  float2* s_warp = reinterpret_cast<float2*>(rowbar + 16);  // [teams][2][warps of a team]: 32 at most
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_warp + 32);
  const int nwarps = p.teams * p.team_threads >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; s++) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], (uint32_t)nwarps);
    }
    for (int t = 0; t < p.teams; t++) mbar_init(&rowbar[t], (uint32_t)(p.team_threads >> 5));
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the first tile into L2 while the previous grid of the stream finishes
  const int64_t first = (int64_t)blockIdx.x * p.teams;
  if (warp == nwarps && lane <= p.nranks)
    prefetch_l2(slice_source(p, lane) + first * (int64_t)p.row_bytes, tile_bytes(p, first));
  __syncthreads();
  pdl_wait_and_release();
  if (warp >= nwarps) {
    if (lane == 0) produce(p, smem, full, empty, s_abort, warp - nwarps);
  } else {
    if constexpr (VPT == 3 || VPT == 4) {
      const int consumers = p.teams * p.team_threads;
      weight_to_shared<DT, kWideWeight<DT, VPT>>(p.weight, p.vec_per_row, consumers, s_weight);
      asm volatile("bar.sync 1, %0;" ::"r"(consumers) : "memory");
    }
    consume<DT, VPT>(p, smem, s_weight, full, empty, rowbar, s_warp, s_abort);
  }
}

using QuantTmaFn = void (*)(const QuantTmaParams);

template <int DT>
QuantTmaFn pick_vpt(int vpt) {
  switch (vpt) {
    case 2: return reduce_residual_rmsnorm_quant_tma_kernel<DT, 2>;
    case 3: return reduce_residual_rmsnorm_quant_tma_kernel<DT, 3>;
    case 4: return reduce_residual_rmsnorm_quant_tma_kernel<DT, 4>;
    case 5: return reduce_residual_rmsnorm_quant_tma_kernel<DT, 5>;
    case 6: return reduce_residual_rmsnorm_quant_tma_kernel<DT, 6>;
    case 7: return reduce_residual_rmsnorm_quant_tma_kernel<DT, 7>;
    default: return reduce_residual_rmsnorm_quant_tma_kernel<DT, 8>;
  }
}
QuantTmaFn pick(int dtype, int vpt) {
  switch (dtype) {
    case kBF16: return pick_vpt<kBF16>(vpt);
    case kFP16: return pick_vpt<kFP16>(vpt);
    default: return pick_vpt<kFP32>(vpt);
  }
}

constexpr int kRingBudget = 216 * 1024;  // ring and weight row

}  // namespace

bool quant_tma_shape(int64_t rows, int vec_per_row, int num_sms, int W, TeamShape* out) {
  const int row_bytes = vec_per_row * 16;
  const int vpt = vec_per_row > 2048 ? (vec_per_row + 511) / 512 : team_vectors(vec_per_row, W <= 3 ? 4 : 2, W <= 3 || vec_per_row > 1536 ? 4 : 3);
  out->vpt = vpt;
  out->use = team_use(vec_per_row, vpt);
  out->team_threads = team_threads(vec_per_row, vpt);
  if (out->team_threads > 512) return false;
  out->teams = 512 / out->team_threads;
  // About one tile's slices in flight, as in the other pipelines: more bulk
  // copies at a time are slower (W = 1, M = 4096, N = 4096: 4 slots 19.3 us, 6
  // 20.5; W = 4, M = 8191, N = 8192 with two vectors: 6 124, 4 146).  An even
  // number: two producers.
  const int slice = out->teams * row_bytes;
  const int weights = vpt == 3 || vpt == 4 ? 2 * row_bytes : 0;  // (fp32 uses half)
  int slots = W < 4 ? 4 : (W + 2) / 2 * 2;
  if (slots > (kRingBudget - weights) / slice) slots = (kRingBudget - weights) / slice;
  if (slots > 4) slots -= slots % kProducers;
  out->producers = slots % kProducers == 0 ? kProducers : 1;
  out->slots = slots;
  const int64_t tiles = (rows + out->teams - 1) / out->teams;
  out->grid = (int)(tiles < num_sms ? tiles : num_sms);
  out->smem = slots * slice + weights + (2 * slots + 16) * 8 + 32 * 8 + 16;
  return slots >= 2;
}

cudaError_t quant_tma_prepare(int dtype, const TeamShape& sh) {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(pick(dtype, sh.vpt)), cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kMaxDynamicSmem);
}

cudaError_t launch_quant_tma(int dtype, int W, const RankPtrs& in, const void* residual, const void* weight, float eps,
                             void* residual_out, const QuantOut& out, void* norm_out, void* ar_out, unsigned int* err,
                             int64_t rows, int64_t cols, int vec_per_row, const TeamShape& sh, cudaStream_t s) {
  QuantTmaParams p;
  p.in = in;
  p.residual = static_cast<const uint8_t*>(residual);
  p.weight = static_cast<const uint4*>(weight);
  p.residual_out = static_cast<uint4*>(residual_out);
  p.norm_out = static_cast<uint4*>(norm_out);
  p.ar_out = static_cast<uint4*>(ar_out);
  p.out = out;
  p.err = err;
  p.eps = eps;
  p.cols = (float)cols;
  p.rows = rows;
  p.row_bytes = vec_per_row * 16;
  p.vec_per_row = vec_per_row;
  p.slots = sh.slots;
  p.teams = sh.teams;
  p.producers = (uint32_t)sh.producers;
  p.team_threads = sh.team_threads;
  p.nranks = W;
  const unsigned threads = (unsigned)(sh.teams * sh.team_threads + 32 * sh.producers);
  return launch_pdl(pick(dtype, sh.vpt), (unsigned)sh.grid, threads, (size_t)sh.smem, s, 1, p);
}

}  // namespace car
