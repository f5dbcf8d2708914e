// norm_backward.cu -- backward of rank sum + residual add + RMSNorm.
//
// Forward (fused_rows.cuh): h = sum_r x_r + residual, rms = rsqrt(mean(h^2) +
// eps), out = h * rms * w.  Given the W rank contributions dy_r of the
// gradient of `out` (a column-parallel product behind the norm leaves one per
// rank), the stored h and the gradient `dres` of residual_out that arrives on
// the skip path:
//   g  = sum_r dy_r                     (fp32, rank order, as the forward's sum)
//   u  = h * rms                        (the normalised row)
//   m  = mean_j(g_j w_j u_j)
//   dx = rms * (g w - u m) + dres       the gradient of residual and of every x_r
//   dw = sum over rows of g * u
// rms and m need two sums over the row, h^2 and g w h, which share one
// exchange; g, h and dres stay in registers across it, so every input is read
// once.  dw is summed over a CTA's rows in fp32 registers; the CTAs' partials
// go to the caller's workspace and a second kernel adds them in a fixed order
// (no float atomics: the same call gives the same bits).
//
// A row is split over a cluster of CTAs as in the forward's row kernel, takes
// one CTA, or shares one with other rows: rows of at most 256 vectors go to
// `teams` of threads of one 512-thread CTA, each at its own pace behind its
// own named barrier.  The teams' weight gradients are added in shared memory
// at the end, so short rows do not multiply the partials (one per CTA).
// Roofline: HBM, (W + 3) * 16 bytes per vector with a skip gradient, and
// 4 * N * groups bytes of partials written and read again (L2).
#include <algorithm>

#include "car_device.cuh"
#include "car_launch.h"

namespace car {
namespace {

struct BackwardParams {
  RankPtrs dy;
  const uint4* h;
  const uint4* dres;   // may be null
  const uint4* weight;
  uint4* dx;
  float* partial;      // [groups, N], or dweight itself with one group; null: no weight gradient
  unsigned int* err;   // as in the forward's row kernel
  float eps;
  float cols;
  int64_t rows;
  int vec_per_row;
  int chunk;           // 16-byte vectors of a row handled by one CTA
  int cluster;
  int teams;           // rows a CTA works on at a time (1 with a cluster)
  int nranks;
  unsigned long long wait_ns;   // as in the forward's row kernel (car_test_delay_partial)
  unsigned long long delay_ns;
  int64_t delay_row;
  int delay_cta;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// This team's piece of `row` -- the n rank slices, h, dres, and the weight with
// `weight` -- into L2, one bulk prefetch per slice by the team's thread t.
__device__ __forceinline__ void prefetch_row(const BackwardParams& p, int n, int64_t row, int col0, int t, bool weight) {
  const int nvec = min(p.chunk, p.vec_per_row - col0);
  if (row >= p.rows || nvec <= 0 || t > n + 2) return;
  const int64_t off = row * (int64_t)p.vec_per_row + col0;
  const uint4* src;
  if (t < n) {
    src = static_cast<const uint4*>(p.dy.p[t]) + off;
  } else if (t == n) {
    src = p.h + off;
  } else if (t == n + 1) {
    if (!p.dres) return;
    src = p.dres + off;
  } else {
    if (!weight) return;
    src = p.weight + col0;
  }
  prefetch_l2(src, (uint32_t)nvec * 16u);
}

__device__ __forceinline__ void team_barrier(int team, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

// CTAs per SM that an instance is compiled for.  The ones held to two spill up
// to 32 bytes, and with eight ranks and two vectors per thread, where 16 loaded
// vectors, g and the weight gradient share 128 registers, 32 (fp32) to 156.
template <int W, int VPT>
constexpr int kBackwardMinCtas = VPT == 1 && (W == 1 || W == 2) ? 2 : 1;

template <int DT, int W, int VPT>
__global__ void __launch_bounds__(kBackwardThreads, kBackwardMinCtas<W, VPT>) reduce_rmsnorm_backward_kernel(const BackwardParams p) {
  constexpr int E = Pack<DT>::kN;
  constexpr int R = W > 0 ? W : kMaxRanks;
  const int n = W > 0 ? W : p.nranks;
  __shared__ float2 s_warp[2][kBackwardThreads / 32];  // warp partials (h^2, g w h), by row parity
  __shared__ __align__(8) float2 s_part[2][8];         // the cluster's CTA partials, by row parity
  __shared__ __align__(8) uint64_t s_xbar[2];
  __shared__ __align__(16) float s_dw[VPT == 1 ? kBackwardThreads * E : 4];  // the teams' weight gradients

  const int C = p.cluster;
  const int crank = C > 1 ? (int)cluster_rank() : 0;
  const int threads = blockDim.x / p.teams;  // of a team, a multiple of 32
  const int team = threadIdx.x / threads, tid = threadIdx.x - team * threads;
  const int64_t group = blockIdx.x / C;
  const int64_t first = group * p.teams + team, step = (int64_t)(gridDim.x / C) * p.teams;
  const int lane = threadIdx.x & 31, warp = tid >> 5, nwarps = threads >> 5, warp0 = team * nwarps;
  const int col0 = crank * p.chunk;
  uint32_t it = 0;
  bool peers_ready = C == 1;
  if (C > 1) {
    if (threadIdx.x == 0) {
      mbar_init(&s_xbar[0], 1);
      mbar_init(&s_xbar[1], 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    cluster_arrive();
  }
  prefetch_row(p, n, first, col0, tid, true);
  pdl_wait_and_release();

  bool ok[VPT];
  uint4 wv[VPT];
  float dw[VPT][E];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const int v = tid + k * threads;
    ok[k] = v < p.chunk && col0 + v < p.vec_per_row;
    wv[k] = ok[k] ? __ldg(p.weight + col0 + v) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int e = 0; e < E; e++) dw[k][e] = 0.f;
  }

  // With one or two ranks and two vectors per thread (one CTA per SM) a row's
  // loads fit in registers beside the previous row's and are issued before
  // that row's statistic: W = 2, M = 2048, N = 8192 bf16 38.0 -> 31.4 us.
  constexpr bool AHEAD = VPT == 2 && (W == 1 || W == 2);
  uint4 raw[VPT][R], hv[VPT], dv[VPT];
  auto load_row = [&](int64_t row, uint4 (&x)[VPT][R], uint4 (&h)[VPT], uint4 (&d)[VPT]) {
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
        const int64_t off = row * (int64_t)p.vec_per_row + col0 + tid + k * threads;
#pragma unroll
        for (int r = 0; r < R; r++)
          if (r < n) x[k][r] = ld_stream(static_cast<const uint4*>(p.dy.p[r]) + off);
        h[k] = ld_stream(p.h + off);
        d[k] = p.dres ? ld_stream(p.dres + off) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  if (AHEAD && first < p.rows) load_row(first, raw, hv, dv);

  for (int64_t row = first; row < p.rows; row += step, it++) {
    prefetch_row(p, n, row + (AHEAD ? 2 : 1) * step, col0, tid, false);
    float g[VPT][E];
    float ss = 0.f, c = 0.f;
    if (!AHEAD) load_row(row, raw, hv, dv);
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
        rank_sum<DT, R>(raw[k], n, g[k]);
        float hf[E], wf[E];
        Pack<DT>::widen(hv[k], hf);
        Pack<DT>::widen(wv[k], wf);
#pragma unroll
        for (int e = 0; e < E; e++) {
          ss = fmaf(hf[e], hf[e], ss);
          c = fmaf(__fmul_rn(g[k][e], wf[e]), hf[e], c);
        }
      }
    }
    uint4 hn[VPT], dn[VPT];
    if (AHEAD && row + step < p.rows) load_row(row + step, raw, hn, dn);
    // Row statistics: warp, team, cluster.  Every warp adds the warp partials
    // itself, in the same order, so one barrier per row is enough: s_warp[b]
    // is next written for row it + 2, after the barrier of row it + 1.
    ss = warp_sum(ss);
    c = warp_sum(c);
    const uint32_t b = it & 1u;
    if (!peers_ready) {
      cluster_wait();
      peers_ready = true;
    }
    if (nwarps > 1) {
      if (lane == 0) s_warp[b][warp0 + warp] = make_float2(ss, c);
      team_barrier(team, threads);
      const float2 mine = lane < nwarps ? s_warp[b][warp0 + lane] : make_float2(0.f, 0.f);
      ss = warp_sum(mine.x);
      c = warp_sum(mine.y);
    }
    if (C > 1) {
      const uint32_t par = (it >> 1) & 1u;
      // test hook: this whole CTA reaches the exchange late
      if (crank == p.delay_cta && row == p.delay_row) spin_ns(p.delay_ns);
      if (warp == 0) {
        if (lane == 0) mbar_arrive_expect_tx(&s_xbar[b], 8u * (uint32_t)C);
        if (lane < C)
          st_async_v2_b32(map_rank(&s_part[b][crank], (uint32_t)lane), __float_as_uint(ss), __float_as_uint(c),
                          map_rank(&s_xbar[b], (uint32_t)lane));
      }
      if (wait_cluster_phase(&s_xbar[b], par, p.wait_ns)) {
        ss = s_part[b][0].x;
        c = s_part[b][0].y;
        for (int r = 1; r < C; r++) {
          ss += s_part[b][r].x;
          c += s_part[b][r].y;
        }
      } else {
        atomicOr(p.err, 1u);
        ss = __int_as_float(0x7fc00000);  // NaN: this row's gradients are not usable
        // the late partials are still waited for, so that none reaches a CTA
        // that has exited and the phases stay in step
        if (!wait_cluster_phase(&s_xbar[b], par)) atomicOr(p.err, 2u);
      }
    }
    const float rms = rsqrtf(__fdiv_rn(ss, p.cols) + p.eps);
    const float m = __fdiv_rn(__fmul_rn(c, rms), p.cols);
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
        float hf[E], wf[E], df[E], o[E];
        Pack<DT>::widen(hv[k], hf);
        Pack<DT>::widen(wv[k], wf);
        Pack<DT>::widen(dv[k], df);
#pragma unroll
        for (int e = 0; e < E; e++) {
          const float u = __fmul_rn(hf[e], rms);
          dw[k][e] = fmaf(g[k][e], u, dw[k][e]);
          o[e] = fmaf(rms, fmaf(-u, m, __fmul_rn(g[k][e], wf[e])), df[e]);
        }
        st16(p.dx + row * (int64_t)p.vec_per_row + col0 + tid + k * threads, Pack<DT>::narrow(o));
      }
      if (AHEAD) {
        hv[k] = hn[k];
        dv[k] = dn[k];
      }
    }
  }
  if (p.partial) {
    if constexpr (VPT == 1) {
      if (p.teams > 1) {  // the first team adds the others' in their order
#pragma unroll
        for (int e = 0; e < E; e += 4)
          *reinterpret_cast<float4*>(s_dw + threadIdx.x * E + e) = make_float4(dw[0][e], dw[0][e + 1], dw[0][e + 2], dw[0][e + 3]);
        __syncthreads();
        if (team == 0) {
          for (int t = 1; t < p.teams; t++) {
#pragma unroll
            for (int e = 0; e < E; e++) dw[0][e] += s_dw[(t * threads + tid) * E + e];
          }
        }
      }
    }
    float* to = p.partial + group * (int64_t)p.vec_per_row * E;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k] && team == 0) {
        const int col = (col0 + tid + k * threads) * E;
#pragma unroll
        for (int e = 0; e < E; e += 4)
          *reinterpret_cast<float4*>(to + col + e) = make_float4(dw[k][e], dw[k][e + 1], dw[k][e + 2], dw[k][e + 3]);
      }
    }
  }
  if (!peers_ready) cluster_wait();
}

// dweight[j] = sum over groups of partial[g][j], in a fixed order: the block's
// threads take VECS vectors of columns and every so-many-th group, all their
// loads in flight together, and those sums are added in order.  The partials
// are a few MB and were just written, so they come from L2: the kernel is
// bound by one L2 latency and its launch.
// The loads of BATCH groups are issued before the first is added: W = 8, M =
// 512, N = 8192 19.8 -> 19.3 us, W = 1, M = 640, N = 1024 5.7 -> 5.1.  Blocks of
// 8 warps and 32 columns while those are few: one fits beside a CTA of the
// pipeline, so that the next call's CTAs need not wait for its end (with the
// batches W = 2, M = 718, N = 4240 11.6 -> 10.2 us; W = 4, M = 2048, N = 4096
// fp32 38.3 -> 36.8).  Otherwise 32 warps and 128 columns (W = 8, M = 200, N =
// 16384 20.5 against 22.0).
constexpr int kFewSumBlocks = 152;  // one per SM
template <int WARPS, int VECS>
__global__ void __launch_bounds__(32 * WARPS)
    sum_partials_kernel(const float4* __restrict__ partial, float4* __restrict__ out, const int groups, const int vecs) {
  constexpr int PARTS = WARPS * 32 / VECS;  // 32 in both forms
  constexpr int BATCH = 5;                  // one partial per SM at a time
  __shared__ float4 s[PARTS][VECS];
  // Released before the wait: the next kernel's prologue and prefetch run in
  // the tail of the one before this.  It waits for this grid in turn, and it
  // is only launched once every CTA here is resident.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int col = threadIdx.x % VECS, part = threadIdx.x / VECS;
  const int v = blockIdx.x * VECS + col;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (v < vecs) {
    for (int g0 = part; g0 < groups; g0 += BATCH * PARTS) {
      float4 x[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; b++) {
        const int g = g0 + b * PARTS;
        x[b] = g < groups ? __ldcg(partial + (int64_t)g * vecs + v) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int b = 0; b < BATCH; b++) {
        a.x += x[b].x;
        a.y += x[b].y;
        a.z += x[b].z;
        a.w += x[b].w;
      }
    }
  }
  s[part][col] = a;
  __syncthreads();
  // one thread per value adds the parts in order
  if (threadIdx.x < 4 * VECS) {
    const float* c = reinterpret_cast<const float*>(&s[0][0]) + threadIdx.x;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < PARTS; w++) sum += c[w * 4 * VECS];
    if (blockIdx.x * VECS + (threadIdx.x >> 2) < vecs) reinterpret_cast<float*>(out)[blockIdx.x * 4 * VECS + threadIdx.x] = sum;
  }
}

using BackwardFn = void (*)(const BackwardParams);

template <int DT>
BackwardFn pick_dt(int W, int vpt) {
  if (vpt == 2) {
    switch (W) {
      case 1: return reduce_rmsnorm_backward_kernel<DT, 1, 2>;
      case 2: return reduce_rmsnorm_backward_kernel<DT, 2, 2>;
      case 4: return reduce_rmsnorm_backward_kernel<DT, 4, 2>;
      case 8: return reduce_rmsnorm_backward_kernel<DT, 8, 2>;
      default: return nullptr;
    }
  }
  if (vpt != 1) return nullptr;
  switch (W) {
    case 1: return reduce_rmsnorm_backward_kernel<DT, 1, 1>;
    case 2: return reduce_rmsnorm_backward_kernel<DT, 2, 1>;
    case 4: return reduce_rmsnorm_backward_kernel<DT, 4, 1>;
    case 8: return reduce_rmsnorm_backward_kernel<DT, 8, 1>;
    case 16: return reduce_rmsnorm_backward_kernel<DT, 16, 1>;
    default: return reduce_rmsnorm_backward_kernel<DT, 0, 1>;
  }
}

BackwardFn pick_backward(int dtype, int W, int vpt) {
  switch (dtype) {
    case kBF16: return pick_dt<kBF16>(W, vpt);
    case kFP16: return pick_dt<kFP16>(W, vpt);
    default: return pick_dt<kFP32>(W, vpt);
  }
}

}  // namespace

bool backward_has_variant(int W, int vpt) {
  return vpt == 1 || (vpt == 2 && (W == 1 || W == 2 || W == 4 || W == 8));
}
int backward_max_threads(int, int) { return kBackwardThreads; }

// Threads are few for a row: as many teams of that many as make 512 threads.
int backward_teams(const FusedShape& sh) {
  return sh.cluster == 1 && sh.vpt == 1 ? std::max(1, kBackwardThreads / sh.threads) : 1;
}

cudaError_t backward_resident_groups(int dtype, int W, const FusedShape& sh, int num_sms, int* groups) {
  *groups = 0;
  BackwardFn fn = pick_backward(dtype, W, sh.vpt);
  if (!fn) return cudaErrorInvalidValue;
  const void* f = reinterpret_cast<const void*>(fn);
  if (sh.cluster == 1) {
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, f, sh.threads * backward_teams(sh), 0);
    *groups = per_sm * num_sms;
    return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)sh.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sh.cluster, 1, 1);
  cfg.blockDim = dim3((unsigned)sh.threads, 1, 1);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(groups, f, &cfg);
}

cudaError_t launch_backward(int dtype, int W, const RankPtrs& dy, const void* h, const void* weight, float eps,
                            const void* dres, void* dx, float* dweight, float* workspace, unsigned int* err,
                            int64_t rows, int64_t cols, int vec_per_row, const FusedShape& sh, const WaitHook& hook,
                            cudaStream_t s) {
  BackwardFn fn = pick_backward(dtype, W, sh.vpt);
  if (!fn) return cudaErrorInvalidValue;
  BackwardParams p;
  p.dy = dy;
  p.h = static_cast<const uint4*>(h);
  p.dres = static_cast<const uint4*>(dres);
  p.weight = static_cast<const uint4*>(weight);
  p.dx = static_cast<uint4*>(dx);
  p.partial = dweight ? (sh.groups > 1 ? workspace : dweight) : nullptr;
  p.err = err;
  p.eps = eps;
  p.cols = (float)cols;
  p.rows = rows;
  p.vec_per_row = vec_per_row;
  p.chunk = (vec_per_row + sh.cluster - 1) / sh.cluster;
  p.cluster = sh.cluster;
  p.teams = backward_teams(sh);
  p.nranks = W;
  p.wait_ns = hook.wait_ns;
  p.delay_ns = hook.delay_ns;
  p.delay_row = hook.delay_row;
  p.delay_cta = hook.delay_cta;
  cudaError_t e = launch_pdl(fn, (unsigned)(sh.groups * sh.cluster), (unsigned)(sh.threads * p.teams), 0, s, (unsigned)sh.cluster, p);
  if (e != cudaSuccess || !dweight || sh.groups == 1) return e;
  return launch_sum_partials(workspace, dweight, sh.groups, cols, s);
}

cudaError_t launch_sum_partials(const float* partial, float* out, int groups, int64_t cols, cudaStream_t s) {
  const int vecs = (int)(cols / 4);
  const bool few = vecs <= 8 * kFewSumBlocks;
  return launch_pdl(few ? sum_partials_kernel<8, 8> : sum_partials_kernel<32, 32>, (unsigned)(few ? (vecs + 7) / 8 : (vecs + 31) / 32),
                    few ? 8u * 32u : 32u * 32u, 0, s, 1, reinterpret_cast<const float4*>(partial),
                    reinterpret_cast<float4*>(out), groups, vecs);
}

}  // namespace car
