// kda_block_norm.cu -- the norm after a block with its gate and residual scale, the residual
// sum and the norm before the next block, forward and backward.
//
//   hat = u r_u, r_u = (mean u^2 + eps)^(-1/2) (1 without w_post);  h = hat act(z);  m = w_post h
//   x = residual + scale m;   normed = w_pre x r_x, r_x = (mean x^2 + eps)^(-1/2)
// Backward, D = d_out, E = d_normed:
//   dx = D + r_x (E w_pre) - x r_x^3 mean((E w_pre) x),  dresidual = dx,  dw_pre = sum E x r_x
//   A = sum dx h per column, so dscale = w_post A and dw_post = scale A (one accumulator)
//   t = dx scale w_post,  dz = t hat act'(z),  dhat = t act(z),  du = r_u (dhat - hat mean(dhat hat))
// Memory-bound: every tensor is read and written once, everything in between is fp32 registers.
// A row is owned by LPR lanes of a warp (short rows) or by a whole CTA (LPR = 0), each thread
// holding VPT vectors of 8 elements.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

// 8 elements of a row in their stored form.
template <typename IO> struct Raw;
template <> struct Raw<bf16> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16 *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
};
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = __ldcs(reinterpret_cast<const float4 *>(p));
    b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
__device__ __forceinline__ void store8(bf16 *p, const float (&x)[8]) {
  uint4 u;
  uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t *>(&b);
  }
  __stcs(reinterpret_cast<uint4 *>(p), u);
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}
// 8 fp32 values of a column vector, or ones.
__device__ __forceinline__ void col8(const float *w, int c, float (&x)[8]) {
  if (w) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(w + c)), b = __ldg(reinterpret_cast<const float4 *>(w + c) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 1.f;
  }
}

// Sum over the lanes that share a row. CTA rows: `red` holds two sets of per-warp partials that
// consecutive calls alternate (`set`), so one barrier per call is enough: a set is rewritten only
// after the barrier of the call in between.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float *red, int set) {
  constexpr int W = LPR ? LPR : 32;
#pragma unroll
  for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (LPR == 0) {
    const int nw = blockDim.x >> 5;
    float *r = red + set * 32;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < nw; ++w) v += r[w];
  }
  return v;
}

template <bool SILU>
__device__ __forceinline__ float gate_of(float z) {
  const float s = __fdividef(1.f, 1.f + __expf(-z));
  return SILU ? z * s : s;
}

// One row per (CTA or LPR lanes); the grid covers all rows.
template <typename IO, int LPR, int VPT>
__global__ void __launch_bounds__(LPR ? 256 : 512) block_norm_fwd_kernel(BlockNormParams p) {
  __shared__ float red[64];
  const int lane = LPR ? (threadIdx.x & (LPR - 1)) : threadIdx.x, step = LPR ? LPR : blockDim.x;
  const int nvec = p.dim >> 3;
  const long long row = LPR ? (long long)blockIdx.x * (blockDim.x / (LPR ? LPR : 1)) + threadIdx.x / (LPR ? LPR : 1) : blockIdx.x;
  const bool live = row < p.rows;   // the dead rows of the last CTA still take part in the shuffles
  const long long base = row * p.dim;
  Raw<IO> u[VPT], z[VPT], r[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + step * j;
    if (live && v < nvec) {
      u[j].load(static_cast<const IO *>(p.u) + base + v * 8);
      if (p.gate) z[j].load(static_cast<const IO *>(p.gate) + base + v * 8);
      if (p.residual) r[j].load(static_cast<const IO *>(p.residual) + base + v * 8);
    }
  }
  float ru = 1.f;
  if (p.w_post) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (live && lane + step * j < nvec) {
        float x[8];
        u[j].get(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
      }
    ru = rsqrtf(row_sum<LPR>(s, red, 0) * p.inv_dim + p.eps);
    if (live && lane == 0) p.rstd_post[row] = ru;
  }
  float x[VPT][8], s = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + step * j;
    if (live && v < nvec) {
      float w[8], g[8];
      u[j].get(x[j]);
      col8(p.w_post, v * 8, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] *= ru * w[e];
      if (p.gate) {
        z[j].get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j][e] *= p.silu ? gate_of<true>(g[e]) : gate_of<false>(g[e]);
      }
      if (p.scale) {
        col8(p.scale, v * 8, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j][e] *= w[e];
      }
      if (p.residual) {
        r[j].get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j][e] += g[e];
      }
      store8(static_cast<IO *>(p.out) + base + v * 8, x[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(x[j][e], x[j][e], s);
    }
  }
  if (!p.w_pre) return;
  const float rx = rsqrtf(row_sum<LPR>(s, red, 1) * p.inv_dim + p.eps);
  if (live && lane == 0) p.rstd_pre[row] = rx;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + step * j;
    if (live && v < nvec) {
      float w[8];
      col8(p.w_pre, v * 8, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] *= rx * w[e];
      store8(static_cast<IO *>(p.normed) + base + v * 8, x[j]);
    }
  }
}

// Persistent: CTA b takes row groups b, b + gridDim, ...; a thread keeps its columns, so A and
// dw_pre accumulate in registers. partial[b][2][d] at the end (the CTA's row groups added in a
// fixed order), summed over b by block_norm_dw_kernel.
template <typename IO, int LPR, int VPT>
__global__ void __launch_bounds__(LPR ? 256 : 512) block_norm_bwd_kernel(BlockNormParams p) {
  extern __shared__ float bn_smem[];   // LPR rows: [2][rows per CTA][d] partials
  __shared__ float red[64];
  constexpr int L1 = LPR ? LPR : 1;
  const int lane = LPR ? (threadIdx.x & (L1 - 1)) : threadIdx.x, step = LPR ? LPR : blockDim.x;
  const int rpc = LPR ? blockDim.x / L1 : 1, sub = LPR ? threadIdx.x / L1 : 0;
  const int nvec = p.dim >> 3;
  float A[VPT][8], P[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) A[j][e] = P[j][e] = 0.f;
  for (long long row0 = (long long)blockIdx.x * rpc; row0 < p.rows; row0 += (long long)gridDim.x * rpc) {
    const long long row = row0 + sub, base = row * p.dim;
    const bool live = row < p.rows;
    const float ru = live && p.w_post ? p.rstd_post[row] : 1.f, rx = live && p.w_pre ? p.rstd_pre[row] : 0.f;
    float x[VPT][8], ep[VPT][8], s = 0.f;   // out, E w_pre
    Raw<IO> u[VPT], z[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + step * j;
      if (live && v < nvec) {
        u[j].load(static_cast<const IO *>(p.u) + base + v * 8);
        if (p.gate) z[j].load(static_cast<const IO *>(p.gate) + base + v * 8);
        if (p.w_pre) {
          Raw<IO> r, en;
          float w[8], t[8];
          if (p.residual) r.load(static_cast<const IO *>(p.residual) + base + v * 8);
          if (p.d_normed) en.load(static_cast<const IO *>(p.d_normed) + base + v * 8);
          u[j].get(x[j]);
          col8(p.w_post, v * 8, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[j][e] *= ru * w[e];
          if (p.gate) {
            z[j].get(t);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j][e] *= p.silu ? gate_of<true>(t[e]) : gate_of<false>(t[e]);
          }
          if (p.scale) {
            col8(p.scale, v * 8, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j][e] *= w[e];
          }
          if (p.residual) {
            r.get(t);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j][e] += t[e];
          }
          if (p.d_normed) {
            en.get(ep[j]);
            col8(p.w_pre, v * 8, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              P[j][e] = fmaf(ep[j][e], x[j][e] * rx, P[j][e]);
              ep[j][e] *= w[e];
              s = fmaf(ep[j][e], x[j][e], s);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) ep[j][e] = 0.f;
          }
        }
      }
    }
    float cx = 0.f;
    if (p.w_pre) cx = row_sum<LPR>(s, red, 0) * p.inv_dim * rx * rx * rx;
    s = 0.f;
    float dh[VPT][8], hat[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + step * j;
      if (live && v < nvec) {
        Raw<IO> d;
        float dx[8], w[8], t[8];
        if (p.d_out) {
          d.load(static_cast<const IO *>(p.d_out) + base + v * 8);
          d.get(dx);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) dx[e] = 0.f;
        }
        if (p.w_pre)
#pragma unroll
          for (int e = 0; e < 8; ++e) dx[e] += rx * ep[j][e] - x[j][e] * cx;
        if (p.residual) store8(static_cast<IO *>(p.d_residual) + base + v * 8, dx);
        u[j].get(hat[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) hat[j][e] *= ru;
        float g[8];
        if (p.gate) {
          z[j].get(t);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float sg = gate_of<false>(t[e]);
            g[e] = p.silu ? t[e] * sg : sg;
            t[e] = p.silu ? sg * fmaf(t[e], 1.f - sg, 1.f) : sg * (1.f - sg);   // act'
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) A[j][e] = fmaf(dx[e], hat[j][e] * g[e], A[j][e]);
        if (p.scale) {
          col8(p.scale, v * 8, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) dx[e] *= w[e];
        }
        col8(p.w_post, v * 8, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dx[e] *= w[e];
          dh[j][e] = dx[e] * g[e];
          s = fmaf(dh[j][e], hat[j][e], s);
        }
        if (p.gate) {
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] *= dx[e] * hat[j][e];
          store8(static_cast<IO *>(p.d_gate) + base + v * 8, t);
        }
      }
    }
    float ch = 0.f;
    if (p.w_post) ch = row_sum<LPR>(s, red, 1) * p.inv_dim;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + step * j;
      if (live && v < nvec) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dh[j][e] = ru * (dh[j][e] - hat[j][e] * ch);
        store8(static_cast<IO *>(p.du) + base + v * 8, dh[j]);
      }
    }
    // without both sums a set of `red` could be rewritten while another warp still reads it
    if (LPR == 0 && !(p.w_pre && p.w_post)) __syncthreads();
  }
  if constexpr (LPR == 0) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + step * j;
      if (v < nvec)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p.partial[((size_t)blockIdx.x * 2) * p.dim + v * 8 + e] = A[j][e];
          p.partial[((size_t)blockIdx.x * 2 + 1) * p.dim + v * 8 + e] = P[j][e];
        }
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + step * j;
      if (v < nvec)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          bn_smem[(size_t)sub * p.dim + v * 8 + e] = A[j][e];
          bn_smem[(size_t)(rpc + sub) * p.dim + v * 8 + e] = P[j][e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.dim; i += blockDim.x) {
      const int which = i / p.dim, c = i - which * p.dim;
      float t = 0.f;
      for (int k = 0; k < rpc; ++k) t += bn_smem[(size_t)(which * rpc + k) * p.dim + c];
      p.partial[((size_t)blockIdx.x * 2 + which) * p.dim + c] = t;
    }
  }
}

// Column sums of the partials in a fixed order: 32 columns x 8 row groups per CTA, then the groups.
__global__ void __launch_bounds__(256) block_norm_dw_kernel(BlockNormParams p, int parts) {
  __shared__ float sa[8][33], sp[8][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  float a = 0.f, b = 0.f;
  if (c < p.dim)
    for (int k = g; k < parts; k += 8) {
      a += p.partial[((size_t)k * 2) * p.dim + c];
      b += p.partial[((size_t)k * 2 + 1) * p.dim + c];
    }
  sa[g][threadIdx.x & 31] = a;
  sp[g][threadIdx.x & 31] = b;
  __syncthreads();
  if (g == 0 && c < p.dim) {
    a = b = 0.f;
    for (int k = 0; k < 8; ++k) {
      a += sa[k][threadIdx.x];
      b += sp[k][threadIdx.x];
    }
    if (p.dw_post) p.dw_post[c] = a * (p.scale ? p.scale[c] : 1.f);
    if (p.dscale) p.dscale[c] = a * (p.w_post ? p.w_post[c] : 1.f);
    if (p.dw_pre) p.dw_pre[c] = b;
  }
}

struct Shape {
  int lpr, vpt, threads;
};
// Rows of at most 32 vectors (d <= 256) share a warp, so no barrier stands between their sums;
// longer rows take a CTA with as few vectors per thread as 512 threads allow.
Shape shape(int dim) {
  const int nvec = dim / 8;
  if (nvec <= 32) {
    int l = 1;
    while (l < nvec) l *= 2;
    return {l, 1, 256};
  }
  const int vpt = nvec <= 256 ? 1 : (nvec <= 1024 ? 2 : 4);
  return {0, vpt, ((nvec + vpt - 1) / vpt + 31) / 32 * 32};
}

typedef void (*Kernel)(BlockNormParams);
template <typename IO>
Kernel fwd_fn(Shape s) {
  switch (s.lpr) {
    case 1: return block_norm_fwd_kernel<IO, 1, 1>;
    case 2: return block_norm_fwd_kernel<IO, 2, 1>;
    case 4: return block_norm_fwd_kernel<IO, 4, 1>;
    case 8: return block_norm_fwd_kernel<IO, 8, 1>;
    case 16: return block_norm_fwd_kernel<IO, 16, 1>;
    case 32: return block_norm_fwd_kernel<IO, 32, 1>;
  }
  return s.vpt == 1 ? block_norm_fwd_kernel<IO, 0, 1> : s.vpt == 2 ? block_norm_fwd_kernel<IO, 0, 2> : block_norm_fwd_kernel<IO, 0, 4>;
}
template <typename IO>
Kernel bwd_fn(Shape s) {
  switch (s.lpr) {
    case 1: return block_norm_bwd_kernel<IO, 1, 1>;
    case 2: return block_norm_bwd_kernel<IO, 2, 1>;
    case 4: return block_norm_bwd_kernel<IO, 4, 1>;
    case 8: return block_norm_bwd_kernel<IO, 8, 1>;
    case 16: return block_norm_bwd_kernel<IO, 16, 1>;
    case 32: return block_norm_bwd_kernel<IO, 32, 1>;
  }
  return s.vpt == 1 ? block_norm_bwd_kernel<IO, 0, 1> : s.vpt == 2 ? block_norm_bwd_kernel<IO, 0, 2> : block_norm_bwd_kernel<IO, 0, 4>;
}
size_t bwd_smem(Shape s, int dim) { return s.lpr ? (size_t)2 * (s.threads / s.lpr) * dim * sizeof(float) : 0; }
}  // namespace

// Backward CTAs: as many as the device holds at once, at most one per row group.
int block_norm_bwd_ctas(long long rows, int dim, bool f32) {
  const Shape s = shape(dim);
  const Kernel fn = f32 ? bwd_fn<float>(s) : bwd_fn<bf16>(s);
  int dev = 0, sms = 0, per = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, fn, s.threads, bwd_smem(s, dim)) != cudaSuccess) {
    (void)cudaGetLastError();
    sms = 152, per = 1;
  }
  const long long most = (long long)sms * (per < 1 ? 1 : per);
  const int rpc = s.lpr ? s.threads / s.lpr : 1;
  const long long groups = (rows + rpc - 1) / rpc;
  return (int)(groups < 1 ? 1 : (groups < most ? groups : most));
}

cudaError_t launch_block_norm_fwd(const BlockNormParams &p, bool f32, cudaStream_t st) {
  if (p.rows == 0) return cudaSuccess;
  const Shape s = shape(p.dim);
  const int rpc = s.lpr ? s.threads / s.lpr : 1;
  const Kernel fn = f32 ? fwd_fn<float>(s) : fwd_fn<bf16>(s);
  fn<<<(unsigned)((p.rows + rpc - 1) / rpc), s.threads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_block_norm_bwd(const BlockNormParams &p, bool f32, cudaStream_t st) {
  const Shape s = shape(p.dim);
  const int ctas = block_norm_bwd_ctas(p.rows, p.dim, f32);
  const Kernel fn = f32 ? bwd_fn<float>(s) : bwd_fn<bf16>(s);
  fn<<<ctas, s.threads, bwd_smem(s, p.dim), st>>>(p);   // no rows: the partials become zero
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.dw_post || p.dscale || p.dw_pre) block_norm_dw_kernel<<<(p.dim + 31) / 32, 256, 0, st>>>(p, ctas);
  return cudaGetLastError();
}

}  // namespace kda
