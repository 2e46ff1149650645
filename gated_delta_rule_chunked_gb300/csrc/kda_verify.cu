// kda_verify.cu -- draft verification: how many drafted tokens of a sequence stand, and the token
// that follows them, from given random numbers.
//
//   accepted while u_j q_j(x_j) < p_j(x_j);  a = their number
//   next = argmax_v r_v / e_v, lowest index on ties;  r = max(p_a - q_a, 0) after a rejection, else p_a
// With e_v ~ Exp(1) the race r_v / e_v is won by v with probability r_v / sum r: no running sum over
// the vocabulary, so the answer does not hang on an order of summation.
// One cluster per sequence: every CTA finds a from the few values at the drafted tokens (redundantly,
// so nothing is exchanged before the stream), streams its share of the rows of the stopping position
// once, and the cluster's winners meet in every CTA through distributed shared memory. The correctly
// rounded division, which decides ties, is made only for entries that an approximate quotient puts
// within 2^-20 of the warp's leader or above it.
// Bound by the bytes of those rows: the target's, the noise, and after a rejection the drafter's. 256 sequences x 131072 fp32, of which
// about half have a draft rejected, 333 MB, in 59.8 us, 5.6 TB/s (82% of a copy): 2048 CTAs in under three waves, each of which starts
// with dependent loads at the drafted tokens. At one sequence by latency, for which the cluster is wide (6 us, and as much again to launch).
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

// 8 CTAs of 256 threads per sequence, five or more on an SM. Compared at 256 sequences x 131072 fp32 where no draft fails (two rows,
// 268 MB): 50 us; with 512 threads 55 to 74; with 4 CTAs 48 to 58, but 11 instead of 8 us for one sequence.
constexpr int VF_T = 256;
constexpr unsigned VF_CL = 8;
constexpr int VF_MAXL = 8;

struct Best {   // the leader of a race; idx = -1: no positive score yet
  float s;
  int i;
};
__device__ __forceinline__ void take(Best &b, float s, int i) {   // i ascending per thread
  if (s > b.s) b = {s, i};
}
__device__ __forceinline__ Best better(Best a, Best b) {
  if (b.i < 0) return a;
  if (a.i < 0 || b.s > a.s || (b.s == a.s && b.i < a.i)) return b;
  return a;
}
__device__ __forceinline__ Best warp_best(Best b) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Best c;
    c.s = __shfl_xor_sync(0xffffffffu, b.s, o);
    c.i = __shfl_xor_sync(0xffffffffu, b.i, o);
    b = better(b, c);
  }
  return b;
}
__device__ __forceinline__ float race(float r, float e) { return r > 0.f ? __fdiv_rn(r, e) : 0.f; }
// An approximate r / e, good to about 2^-22 where it is a normal number; where it is not, inf or 0.
__device__ __forceinline__ float near(float r, float e) {
  float q;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(q) : "f"(e));
  return r * q;
}
// What an approximate score has to reach for the exact one to count: all do against a leader so small
// that the approximation may have been flushed.
__device__ __forceinline__ float bar_for(float best) { return best > 1e-30f ? best * (1.f - 0x1p-20f) : 0.f; }

__device__ __forceinline__ uint32_t peer_u32(const void *p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(a) : "memory");
  return v;
}

template <typename IO>
__device__ __forceinline__ float at(const void *p, size_t i) {
  return to_f(static_cast<const IO *>(p)[i]);
}
// 8 consecutive values from a 16-byte aligned address.
__device__ __forceinline__ void load8(const bf16 *p, float (&x)[8]) {
  const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// The race over this CTA's share [v0, v1) of the vocabulary: r = p - q (q may be null), or p - 1 at entry
// `certain`. VEC: 8 entries per access (rows and shares start on 16 bytes);
// otherwise single entries, eight in flight.
template <typename IO, bool VEC>
__device__ __forceinline__ Best run_race(const IO *p, const IO *q, const float *noise, int certain, int v0, int v1) {
  constexpr int W = VEC ? 8 : 1, U = VEC ? 1 : 8;
  Best b = {0.f, -1};
  float bar = 0.f;
  for (int base = v0; base < v1; base += VF_T * W * U) {   // the same trips for every thread
    float pv[U][W], qv[U][W], e[U][W];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int v = base + (j * VF_T + (int)threadIdx.x) * W;
#pragma unroll
      for (int i = 0; i < W; ++i) pv[j][i] = qv[j][i] = 0.f, e[j][i] = 1.f;
      if (v < v1) {
        if constexpr (VEC) {
          load8(p + v, pv[j]);
          load8(noise + v, e[j]);
          if (q) load8(q + v, qv[j]);
        } else {
          pv[j][0] = to_f(p[v]);
          e[j][0] = noise[v];
          if (q) qv[j][0] = to_f(q[v]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int v = base + (j * VF_T + (int)threadIdx.x) * W;
      bool any = false;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        pv[j][i] = v + i == certain ? pv[j][i] - 1.f : pv[j][i] - qv[j][i];
        any |= near(pv[j][i], e[j][i]) >= bar;
      }
      if (any && v < v1) {
#pragma unroll
        for (int i = 0; i < W; ++i) take(b, race(pv[j][i], e[j][i]), v + i);
        bar = fmaxf(bar, bar_for(b.s));
      }
    }
    bar = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(bar)));   // never negative: its bits order as integers
  }
  return b;
}

// VEC: vocab is a multiple of 8, so every row starts on 16 bytes.
template <typename IO, bool VEC>
__global__ void __launch_bounds__(VF_T, VEC ? 5 : 4) draft_verify_kernel(VerifyParams p) {
  __shared__ int s_acc, s_drafted, s_tok[VF_MAXL];
  __shared__ Best wb[VF_T / 32], cb[2];
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(ranks));
  const int n = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = p.L, V = p.V;
  const int share = ((V + 7) / 8 + (int)ranks - 1) / (int)ranks * 8, v0 = min((int)rank * share, V), v1 = min(v0 + share, V);
  const float *noise = p.noise + (size_t)n * V;
  if (VEC && tid == 32 && v0 < v1) prefetch_l2(noise + v0, (uint32_t)(v1 - v0) * 4u);   // needed whatever is accepted
  if (warp == 0) {   // lane j: draft j
    int tok = -1;
    bool ok = false, drafted = false;
    if (lane < L) {
      tok = p.draft[(size_t)n * L + lane];
      drafted = tok >= 0 && tok < V && (!p.draft_len || lane < p.draft_len[n]);
      if (drafted) {
        const float px = at<IO>(p.p, ((size_t)n * (L + 1) + lane) * V + tok);
        const float qx = p.q ? at<IO>(p.q, ((size_t)n * L + lane) * V + tok) : 1.f;
        ok = __fmul_rn(p.u[(size_t)n * L + lane], qx) < px;
      }
      s_tok[lane] = tok;
    }
    const uint32_t md = __ballot_sync(0xffffffffu, drafted), mo = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) {
      s_drafted = __ffs(~md) - 1;   // leading ones
      s_acc = __ffs(~(md & mo)) - 1;
    }
  }
  __syncthreads();
  const int a = s_acc;
  const bool rejected = a < s_drafted;
  const IO *prow = static_cast<const IO *>(p.p) + ((size_t)n * (L + 1) + a) * V;
  const IO *qrow = rejected && p.q ? static_cast<const IO *>(p.q) + ((size_t)n * L + a) * V : nullptr;
  // The winner over the cluster, in every CTA (set: which of the two places for the CTA's own winner).
  auto winner = [&](Best b, int set) {
    b = warp_best(b);
    if (lane == 0) wb[warp] = b;
    __syncthreads();
    if (warp == 0) {
      b = warp_best(lane < VF_T / 32 ? wb[lane] : Best{0.f, -1});
      if (lane == 0) cb[set] = b;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    b = {0.f, -1};
    if (lane < (int)ranks) {
      b.s = __uint_as_float(peer_u32(&cb[set].s, lane));
      b.i = (int)peer_u32(&cb[set].i, lane);
    }
    return warp_best(b).i;
  };
  // certain: the entry that a certain drafter takes out
  int next = winner(run_race<IO, VEC>(prow, qrow, noise, rejected && !p.q ? s_tok[a] : -1, v0, v1), 0);
  if (next < 0 && rejected)   // nothing left of p - q, for the whole cluster: the race over p
    next = winner(run_race<IO, VEC>(prow, nullptr, noise, -1, v0, v1), 1);
  if (rank == 0 && warp == 0) {
    if (lane <= L) p.tokens[(size_t)n * (L + 1) + lane] = lane < a ? s_tok[lane] : (lane == a ? next : -1);
    if (lane == 0) {
      p.accept[n] = a;
      if (p.first) p.first[n] = L - a;
    }
  }
  __syncwarp();
  // a CTA's shared memory stays until its peers have read it
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyParams &p, bool f32, cudaStream_t s) {
  const bool vec = p.V % 8 == 0;
  auto kern = f32 ? (vec ? draft_verify_kernel<float, true> : draft_verify_kernel<float, false>)
                  : (vec ? draft_verify_kernel<bf16, true> : draft_verify_kernel<bf16, false>);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = VF_CL;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)p.n_seqs * VF_CL);
  cfg.blockDim = dim3(VF_T);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace kda
