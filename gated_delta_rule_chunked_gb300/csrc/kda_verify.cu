// kda_verify.cu -- draft verification: how many drafted tokens of a sequence stand, and the token
// that follows them, from given random numbers.
//
//   accepted while u_j q_j(x_j) < p_j(x_j);  a = their number
//   next = argmax_v r_v / e_v, lowest index on ties;  r = max(p_a - q_a, 0) after a rejection, else p_a
// With e_v ~ Exp(1) the race r_v / e_v is won by v with probability r_v / sum r: no running sum over
// the vocabulary, so the answer does not hang on an order of summation.
// One cluster per sequence: every CTA finds a from the few values at the drafted tokens (redundantly,
// so nothing is exchanged before the stream), streams its share of the three rows of the stopping
// position once, and the cluster's winners meet in rank 0 through distributed shared memory.
// Bound by the bytes of those rows; at one sequence by latency, for which the cluster is wide.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int VF_T = 512;
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

// VEC: vocab is a multiple of 8, so every row starts on 16 bytes.
template <typename IO, bool VEC>
__global__ void __launch_bounds__(VF_T) draft_verify_kernel(VerifyParams p) {
  __shared__ int s_acc, s_drafted, s_tok[VF_MAXL];
  __shared__ Best wb[2][VF_T / 32], cb[2];
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(ranks));
  const int n = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = p.L, V = p.V;
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
  const float *noise = p.noise + (size_t)n * V;
  const int certain = rejected && !p.q ? s_tok[a] : -1;   // the entry a certain drafter takes out
  Best br = {0.f, -1}, bp = {0.f, -1};   // over r, and over p_a in case r has nothing
  auto one = [&](float pv, float qv, float e, int v) {
    const float r = v == certain ? pv - 1.f : pv - qv;
    take(br, race(r, e), v);
    if (rejected) take(bp, race(pv, e), v);
  };
  if constexpr (VEC) {
    const int nv = V / 8, stride = (int)ranks * VF_T;
    for (int k = (int)rank * VF_T + tid; k < nv; k += stride) {
      float pv[8], qv[8], e[8];
      load8(prow + (size_t)k * 8, pv);
      load8(noise + (size_t)k * 8, e);
      if (qrow) load8(qrow + (size_t)k * 8, qv);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) qv[i] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) one(pv[i], qv[i], e[i], k * 8 + i);
    }
  } else {
    const int stride = (int)ranks * VF_T;
    for (int v = (int)rank * VF_T + tid; v < V; v += stride)
      one(to_f(prow[v]), qrow ? to_f(qrow[v]) : 0.f, noise[v], v);
  }
  br = warp_best(br);
  bp = warp_best(bp);
  if (lane == 0) {
    wb[0][warp] = br;
    wb[1][warp] = bp;
  }
  __syncthreads();
  if (warp < 2) {
    Best b = lane < VF_T / 32 ? wb[warp][lane] : Best{0.f, -1};
    b = warp_best(b);
    if (lane == 0) cb[warp] = b;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  if (rank == 0 && warp == 0) {
    Best r = {0.f, -1}, q = {0.f, -1};
    if (lane < (int)ranks) {
      r.s = __uint_as_float(peer_u32(&cb[0].s, lane));
      r.i = (int)peer_u32(&cb[0].i, lane);
      q.s = __uint_as_float(peer_u32(&cb[1].s, lane));
      q.i = (int)peer_u32(&cb[1].i, lane);
    }
    r = warp_best(r);
    q = warp_best(q);
    const int next = r.i >= 0 ? r.i : q.i;
    if (lane <= L) p.tokens[(size_t)n * (L + 1) + lane] = lane < a ? s_tok[lane] : (lane == a ? next : -1);
    if (lane == 0) {
      p.accept[n] = a;
      if (p.first) p.first[n] = L - a;
    }
  }
  __syncwarp();
  // the peers' shared memory stays until rank 0 has read it
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyParams &p, bool f32, cudaStream_t s) {
  const bool vec = p.V % 8 == 0;
  auto kern = f32 ? (vec ? draft_verify_kernel<float, true> : draft_verify_kernel<float, false>)
                  : (vec ? draft_verify_kernel<bf16, true> : draft_verify_kernel<bf16, false>);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 8;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)p.n_seqs * 8);
  cfg.blockDim = dim3(VF_T);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace kda
