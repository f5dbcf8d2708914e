// branch_rows.cu -- a block's branch in one pass over HBM, for few rows: rank
// sum, norm behind the block, gate, dropout, residual add with its scale, and
// the next block's norm.
//
// Per row, with acc the fp32 rank sum:
//   y = acc * rsqrt(mean(acc^2) + norm_eps) * norm_weight     (NORM; else acc)
//   h = residual_scale * residual + drop(y * gate)
//   residual_out = h;  norm_out = h * rsqrt(mean(h^2) + eps) * weight
// The mean of h^2 could be had from sums over acc and the residual in the first
// exchange (h is linear in both), but where the branch cancels the residual
// that difference of large sums loses h: the row has two exchanges instead, one
// after the other, and everything else stays in registers between them.
//
// A row is split over a cluster of CTAs as in fused_rows.cuh, one vector per
// thread: with few rows the two exchanges' latency is the time, and rows that
// are spread over more SMs have the shorter ones.  The mask's bits are computed
// before the first exchange, off its critical path.
// Roofline: HBM, (W + 3) * 16 bytes per vector, 1 more for a stored sum and for
// a gate of each row's own.
#include <algorithm>

#include "branch.cuh"

namespace car {
namespace {

struct BranchParams {
  RankPtrs in;
  const uint4* residual;
  const uint4* weight;
  const uint4* norm_weight;
  const uint4* gate;      // may be null
  uint4* residual_out;
  uint4* norm_out;
  uint4* ar_out;          // may be null
  unsigned int* err;
  DropParams drop;
  float residual_scale;
  float eps, norm_eps;
  float cols;
  int64_t rows;
  uint32_t gate_span;     // rows that share a gate row (1: each has its own)
  int vec_per_row;
  int chunk;              // vectors of a row handled by one CTA
  int cluster;
  int nranks;
  unsigned long long wait_ns;  // as in the fused op's row kernel
  unsigned long long delay_ns;
  int64_t delay_row;
  int delay_cta;
};

// This CTA's piece of `row` into L2, one bulk prefetch per slice.
__device__ __forceinline__ void prefetch_row(const BranchParams& p, int n, int64_t row, int col0, bool weights) {
  const int nvec = min(p.chunk, p.vec_per_row - col0);
  const int t = threadIdx.x;
  if (row >= p.rows || nvec <= 0 || t > n + 3) return;
  const int64_t off = row * (int64_t)p.vec_per_row + col0;
  const uint4* src;
  if (t < n) src = static_cast<const uint4*>(p.in.p[t]) + off;
  else if (t == n) src = p.residual + off;
  else if (t == n + 1) src = p.gate ? p.gate + (int64_t)((uint32_t)row / p.gate_span) * p.vec_per_row + col0 : nullptr;
  else if (t == n + 2) src = weights ? p.weight + col0 : nullptr;
  else src = weights && p.norm_weight ? p.norm_weight + col0 : nullptr;
  if (src) prefetch_l2(src, (uint32_t)nvec * 16u);
}

template <int DT, int W, bool NORM>
__global__ void __launch_bounds__(kBranchThreads) reduce_branch_residual_rmsnorm_kernel(const BranchParams p) {
  constexpr int E = Pack<DT>::kN;
  constexpr int R = W > 0 ? W : kMaxRanks;
  const int n = W > 0 ? W : p.nranks;
  __shared__ __align__(16) RowSums s_sums;
  const int C = p.cluster;
  const int crank = C > 1 ? (int)cluster_rank() : 0;
  const int64_t ngroups = gridDim.x / C;
  const int col0 = crank * p.chunk;
  const ClusterWait peers{crank, p.wait_ns, p.err};
  uint32_t x = 0;  // exchanges done
  bool peers_ready = C == 1;
  if (C > 1) {
    if (threadIdx.x == 0) row_sums_init(s_sums, C);
    __syncthreads();
    cluster_arrive();  // its wait, before the first partial is sent, covers the loads
  }
  prefetch_row(p, n, blockIdx.x / C, col0, true);
  pdl_wait_and_release();
  const DropState state = drop_state(p.drop);
  const int v = threadIdx.x;
  const bool ok = v < p.chunk && col0 + v < p.vec_per_row;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4 wv = ok ? __ldg(p.weight + col0 + v) : zero;
  const uint4 pv = NORM && ok ? __ldg(p.norm_weight + col0 + v) : zero;

  for (int64_t row = blockIdx.x / C; row < p.rows; row += ngroups) {
    const int64_t at = row * (int64_t)p.vec_per_row + col0 + v;
    prefetch_row(p, n, row + ngroups, col0, false);
    uint4 raw[R], rv = zero, gv = zero;
    if (ok) {
#pragma unroll
      for (int r = 0; r < R; r++)
        if (r < n) raw[r] = ld_stream(static_cast<const uint4*>(p.in.p[r]) + at);
      rv = ld_stream(p.residual + at);
      if (p.gate) gv = __ldg(p.gate + (int64_t)((uint32_t)row / p.gate_span) * p.vec_per_row + col0 + v);
    }
    uint32_t bits[E / 2];
    if (p.drop.active) drop_bits<E>(state, at, bits);
    float2 z[E / 2];
    float ss = 0.f;
    if (ok) {
      float acc[E];
      rank_sum<DT, R>(raw, n, acc);
      if (p.ar_out) st16(p.ar_out + at, Pack<DT>::narrow(acc));
#pragma unroll
      for (int e = 0; e < E; e++) ss = fmaf(acc[e], acc[e], ss);
#pragma unroll
      for (int e = 0; e < E / 2; e++) z[e] = make_float2(acc[2 * e], acc[2 * e + 1]);
    }
    if (!peers_ready) {
      cluster_wait();  // every peer's mbarriers are initialised
      peers_ready = true;
    }
    // test hook: this whole CTA reaches the row's first exchange late
    if (C > 1 && crank == p.delay_cta && row == p.delay_row) spin_ns(p.delay_ns);
    if constexpr (NORM) {
      float s[1] = {ss};
      row_sums(s_sums, s, x++, C, peers);
      const float2 q = both(rsqrtf(__fdiv_rn(s[0], p.cols) + p.norm_eps));
      float2 w[E / 2];
      widen2<DT>(pv, w);
#pragma unroll
      for (int e = 0; e < E / 2; e++) z[e] = mul2(mul2(z[e], q), w[e]);
    }
    ss = 0.f;
    if (ok) {
      float2 f[E / 2];
      if (p.gate) {
        widen2<DT>(gv, f);
#pragma unroll
        for (int e = 0; e < E / 2; e++) z[e] = mul2(z[e], f[e]);
      }
      if (p.drop.active) {
#pragma unroll
        for (int e = 0; e < E / 2; e++) z[e] = drop2(p.drop, bits[e], z[e]);
      }
      widen2<DT>(rv, f);
#pragma unroll
      for (int e = 0; e < E / 2; e++) {
        z[e] = fma2(both(p.residual_scale), f[e], z[e]);
        ss = fmaf(z[e].x, z[e].x, ss);
        ss = fmaf(z[e].y, z[e].y, ss);
      }
      st16(p.residual_out + at, narrow2<DT>(z));
    }
    float s[1] = {ss};
    row_sums(s_sums, s, x++, C, peers);
    if (ok) {
      const float2 r = both(rsqrtf(__fdiv_rn(s[0], p.cols) + p.eps));
      float2 w[E / 2];
      widen2<DT>(wv, w);
#pragma unroll
      for (int e = 0; e < E / 2; e++) w[e] = mul2(mul2(z[e], r), w[e]);
      st16(p.norm_out + at, narrow2<DT>(w));
    }
  }
  // nothing reaches this CTA's shared memory after its last exchange; a cluster
  // with no row still pairs its first arrive
  if (!peers_ready) cluster_wait();
}

using BranchFn = void (*)(const BranchParams);

template <int DT, bool NORM>
BranchFn pick_ranks(int W) {
  switch (W) {
    case 1: return reduce_branch_residual_rmsnorm_kernel<DT, 1, NORM>;
    case 2: return reduce_branch_residual_rmsnorm_kernel<DT, 2, NORM>;
    case 4: return reduce_branch_residual_rmsnorm_kernel<DT, 4, NORM>;
    case 8: return reduce_branch_residual_rmsnorm_kernel<DT, 8, NORM>;
    case 16: return reduce_branch_residual_rmsnorm_kernel<DT, 16, NORM>;
    default: return reduce_branch_residual_rmsnorm_kernel<DT, 0, NORM>;
  }
}
BranchFn pick(int dtype, int W, bool norm) {
  switch (dtype) {
    case kBF16: return norm ? pick_ranks<kBF16, true>(W) : pick_ranks<kBF16, false>(W);
    case kFP16: return norm ? pick_ranks<kFP16, true>(W) : pick_ranks<kFP16, false>(W);
    default: return norm ? pick_ranks<kFP32, true>(W) : pick_ranks<kFP32, false>(W);
  }
}

}  // namespace

// How many row groups of this shape can be resident at once, with a norm or
// without.
cudaError_t branch_resident_groups(int dtype, int W, const FusedShape& sh, int num_sms, int* groups) {
  int least = 0;
  for (int norm = 0; norm < 2; norm++) {
    const void* f = reinterpret_cast<const void*>(pick(dtype, W, norm != 0));
    int got = 0;
    cudaError_t e;
    if (sh.cluster == 1) {
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&got, f, sh.threads, 0);
      got *= num_sms;
    } else {
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
      e = cudaOccupancyMaxActiveClusters(&got, f, &cfg);
    }
    if (e != cudaSuccess) return e;
    least = norm ? std::min(least, got) : got;
  }
  *groups = least;
  return cudaSuccess;
}

cudaError_t launch_branch(int dtype, int W, const RankPtrs& in, const BranchArgs& br, const void* residual,
                          const void* weight, float eps, void* residual_out, void* norm_out, void* ar_out,
                          unsigned int* err, int64_t rows, int64_t cols, int vec_per_row, const FusedShape& sh,
                          const WaitHook& hook, cudaStream_t s) {
  BranchParams p;
  p.in = in;
  p.residual = static_cast<const uint4*>(residual);
  p.weight = static_cast<const uint4*>(weight);
  p.norm_weight = static_cast<const uint4*>(br.norm_weight);
  p.gate = static_cast<const uint4*>(br.gate);
  p.residual_out = static_cast<uint4*>(residual_out);
  p.norm_out = static_cast<uint4*>(norm_out);
  p.ar_out = static_cast<uint4*>(ar_out);
  p.err = err;
  p.drop = br.drop;
  p.residual_scale = br.residual_scale;
  p.eps = eps;
  p.norm_eps = br.norm_eps;
  p.cols = (float)cols;
  p.rows = rows;
  p.gate_span = (uint32_t)std::max<int64_t>(br.gate_span, 1);
  p.vec_per_row = vec_per_row;
  p.chunk = (vec_per_row + sh.cluster - 1) / sh.cluster;
  p.cluster = sh.cluster;
  p.nranks = W;
  p.wait_ns = hook.wait_ns;
  p.delay_ns = hook.delay_ns;
  p.delay_row = hook.delay_row;
  p.delay_cta = hook.delay_cta;
  return launch_pdl(pick(dtype, W, br.norm_weight != nullptr), (unsigned)(sh.groups * sh.cluster), (unsigned)sh.threads, 0, s,
                    (unsigned)sh.cluster, p);
}

}  // namespace car
