// kda_ssm.cu -- selective state space scan token by token in fp32 on the CUDA cores: prompts with
// fp32 I/O, and the decode / verify step of both I/O types behind its short convolution.
//
//   h_t = softplus(dt_t + bias),  S_t = exp(h_t a) S_{t-1} + h_t B_t x_t^T,  y_t = S_t^T C_t + d x_t
//
// One CTA owns 64 value columns of one (sequence, head): 256 threads hold the 128 x 64 state in
// registers, thread (g, q) rows 8 g .. 8 g + 7 and columns 4 q .. 4 q + 3 (the 16 lanes of a half
// warp cover a row's 64 columns, so states move as whole 256-byte rows). Per token a thread reads
// 8 values of B, 8 of C and 4 of h x from shared memory for 96 multiply-adds; the sums over the
// 16 row groups meet once per 8 tokens.
// Step: bound by reading and writing the 32 KB state. The convolution runs as a kernel of its own
// (its state is shared by every head of a group, so it cannot be advanced in place by the heads'
// CTAs), and the scan starts under it (programmatic dependent launch): it has its state in
// registers by the time the convolution's rows are there.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int TB = 8;   // tokens per batch (the step's most slots)

__device__ __forceinline__ float step_size(float v, bool softplus) {
  return softplus ? log1pf(expf(-fabsf(v))) + fmaxf(v, 0.f) : v;
}

struct RecSmem {
  float x[TB][SSM_COLS], b[TB][SSM_N], c[TB][SSM_N];
  float h[TB], dec[TB];
  float yp[8][TB][SSM_COLS];   // per warp: sums over its rows
};

// `nt` tokens of the batch in `sm` through the state; commit(t) is called after token t.
template <typename F>
__device__ __forceinline__ void advance(RecSmem &sm, float (&S)[8][4], int t0, int nt, F commit) {
  const int g = threadIdx.x >> 4, q = threadIdx.x & 15, warp = threadIdx.x >> 5;
  for (int t = t0; t < nt; ++t) {
    const float h = sm.h[t], dec = sm.dec[t];
    float4 x = *reinterpret_cast<const float4 *>(&sm.x[t][4 * q]);
    const float hx[4] = {h * x.x, h * x.y, h * x.z, h * x.w};
    float b[8], c[8], y[4] = {0.f, 0.f, 0.f, 0.f};
    *reinterpret_cast<float4 *>(b) = *reinterpret_cast<const float4 *>(&sm.b[t][8 * g]);
    *reinterpret_cast<float4 *>(b + 4) = *reinterpret_cast<const float4 *>(&sm.b[t][8 * g + 4]);
    *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(&sm.c[t][8 * g]);
    *reinterpret_cast<float4 *>(c + 4) = *reinterpret_cast<const float4 *>(&sm.c[t][8 * g + 4]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        S[i][k] = fmaf(S[i][k], dec, b[i] * hx[k]);
        y[k] = fmaf(c[i], S[i][k], y[k]);
      }
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] += __shfl_xor_sync(0xffffffffu, y[k], 16);
    if ((threadIdx.x & 16) == 0) *reinterpret_cast<float4 *>(&sm.yp[warp][t][4 * q]) = make_float4(y[0], y[1], y[2], y[3]);
    commit(t);
  }
}

// The batch's outputs: the eight warps' sums in order, plus the skip.
template <typename IO>
__device__ __forceinline__ void put_y(const RecSmem &sm, int t0, int nt, float d, IO *y, long long ldy) {
  for (int i = threadIdx.x; i < (nt - t0) * SSM_COLS; i += blockDim.x) {
    const int t = t0 + i / SSM_COLS, p = i % SSM_COLS;
    float v = d * sm.x[t][p];
#pragma unroll
    for (int w = 0; w < 8; ++w) v += sm.yp[w][t][p];
    y[t * ldy + p] = from_f<IO>(v);
  }
}

__device__ __forceinline__ void load_state(const float *src, int P, float (&S)[8][4]) {
  const int g = threadIdx.x >> 4, q = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 v = src ? __ldcs(reinterpret_cast<const float4 *>(src + (size_t)(8 * g + i) * P + 4 * q)) : make_float4(0.f, 0.f, 0.f, 0.f);
    S[i][0] = v.x; S[i][1] = v.y; S[i][2] = v.z; S[i][3] = v.w;
  }
}
__device__ __forceinline__ void store_state(float *dst, int P, const float (&S)[8][4]) {
  const int g = threadIdx.x >> 4, q = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    __stcs(reinterpret_cast<float4 *>(dst + (size_t)(8 * g + i) * P + 4 * q), make_float4(S[i][0], S[i][1], S[i][2], S[i][3]));
}

// Prompts. Grid: (value slices of all heads, sequences).
__global__ void __launch_bounds__(256) ssm_rec_kernel(SsmParams p) {
  __shared__ __align__(16) RecSmem sm;
  const int slices = p.P / SSM_COLS, head = blockIdx.x / slices, col0 = (blockIdx.x % slices) * SSM_COLS, n = blockIdx.y;
  const int group = head / (p.H / p.G);
  const long long t0 = p.cu ? p.cu[n] : p.T / p.n_seqs * n, t1 = p.cu ? p.cu[n + 1] : p.T / p.n_seqs * (n + 1);
  const float *x = static_cast<const float *>(p.x) + (long long)head * p.P + col0;
  const float *b = static_cast<const float *>(p.b) + (long long)group * SSM_N, *c = static_cast<const float *>(p.c) + (long long)group * SSM_N;
  float *y = static_cast<float *>(p.y) + (long long)head * p.P + col0;
  const size_t soff = ((size_t)n * p.H + head) * SSM_N * p.P + col0;
  const float a = p.a[head], bias = p.dt_bias ? p.dt_bias[head] : 0.f, d = p.d_skip ? p.d_skip[head] : 0.f;
  float S[8][4];
  load_state(p.h0 ? p.h0 + soff : nullptr, p.P, S);
  for (long long t = t0; t < t1; t += TB) {
    const int nt = (int)(t1 - t < TB ? t1 - t : TB);
    __syncthreads();   // the previous batch is consumed
    for (int i = threadIdx.x; i < nt * SSM_COLS; i += 256) sm.x[i / SSM_COLS][i % SSM_COLS] = (x[(t + i / SSM_COLS) * p.ldx + i % SSM_COLS]);
    for (int i = threadIdx.x; i < nt * SSM_N; i += 256) {
      const int k = i / SSM_N, e = i % SSM_N;
      sm.b[k][e] = (b[(t + k) * p.ldb + e]);
      sm.c[k][e] = (c[(t + k) * p.ldc + e]);
    }
    if ((int)threadIdx.x < nt) {
      const float h = step_size(p.dt[(t + threadIdx.x) * p.H + head] + bias, p.softplus);
      sm.h[threadIdx.x] = h;
      sm.dec[threadIdx.x] = expf(h * a);
    }
    __syncthreads();
    advance(sm, S, 0, nt, [](int) {});
    __syncthreads();
    put_y(sm, 0, nt, d, y + t * (long long)p.H * p.P, (long long)p.H * p.P);
  }
  if (p.hT) store_state(p.hT + soff, p.P, S);
}

// The convolution of the step: two channels per thread, all slots of one sequence. Grid:
// (channel blocks, sequences). Writes fp32 rows to p.conv and advances the convolution state.
template <typename IO>
__global__ void __launch_bounds__(256) ssm_conv_step_kernel(SsmParams p, int C) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");   // the scan loads its state meanwhile
  const int n = blockIdx.y, c = 2 * (blockIdx.x * 256 + threadIdx.x);
  if (c >= C) return;
  const int slot = p.idx ? p.idx[n] : n;
  if (slot < 0 || slot >= p.n_slots) {
    if (c == 0) report(p.status, KDA_ERR_INVALID_ARG_CODE);
    return;
  }
  const int L = p.L, K = p.W - 1;   // K earlier inputs
  const int first = p.first ? min(max(p.first[n], 0), L) : 0, acc = p.acc ? min(max(p.acc[n], 0), L) : L;
  float w0[4], w1[4], win[4][2];   // right-aligned: tap 3 is the current token
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = j - (4 - p.W);
    w0[j] = k >= 0 ? p.cw[(size_t)c * p.W + k] : 0.f;
    w1[j] = k >= 0 ? p.cw[(size_t)(c + 1) * p.W + k] : 0.f;
    win[j][0] = win[j][1] = 0.f;
  }
  const float b0 = p.cbias ? p.cbias[c] : 0.f, b1 = p.cbias ? p.cbias[c + 1] : 0.f;
  IO *st = static_cast<IO *>(p.conv_state) + (size_t)slot * K * C + c;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int k = j - (3 - K);
    if (k >= 0) {
      const float2 v = ld2(st + (size_t)k * C);
      win[j][0] = v.x;
      win[j][1] = v.y;
    }
  }
  const IO *x = static_cast<const IO *>(p.xbc) + (size_t)n * L * C + c;
  float *out = p.conv + (size_t)n * L * C + c;
  for (int s = first; s < L; ++s) {
    const float2 v = ld2(x + (size_t)s * C);
    win[3][0] = v.x;
    win[3][1] = v.y;
    float z0 = b0, z1 = b1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      z0 = fmaf(w0[j], win[j][0], z0);
      z1 = fmaf(w1[j], win[j][1], z1);
    }
    if (p.act) {
      z0 = z0 / (1.f + expf(-z0));
      z1 = z1 / (1.f + expf(-z1));
    }
    *reinterpret_cast<float2 *>(out + (size_t)s * C) = make_float2(z0, z1);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      win[j][0] = win[j + 1][0];
      win[j][1] = win[j + 1][1];
    }
    if (s + 1 == acc)
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int k = j - (3 - K);
        if (k >= 0) st2(st + (size_t)k * C, win[j][0], win[j][1]);
      }
  }
}

// The scan of the step. Grid: (value slices of all heads, sequences).
template <typename IO>
__global__ void __launch_bounds__(256) ssm_step_kernel(SsmParams p, int C) {
  __shared__ __align__(16) RecSmem sm;
  const int slices = p.P / SSM_COLS, head = blockIdx.x / slices, col0 = (blockIdx.x % slices) * SSM_COLS, n = blockIdx.y;
  const int slot = p.idx ? p.idx[n] : n;
  if (slot < 0 || slot >= p.n_slots) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");   // this grid ends after the convolution's
    return;
  }
  const int group = head / (p.H / p.G), L = p.L;
  const int first = p.first ? min(max(p.first[n], 0), L) : 0, acc = p.acc ? min(max(p.acc[n], 0), L) : L;
  float *state = p.state + ((size_t)slot * p.H + head) * SSM_N * p.P + col0;
  float S[8][4];
  load_state(state, p.P, S);
  if ((int)threadIdx.x < L) {
    const float h = step_size(p.dt[((size_t)n * L + threadIdx.x) * p.H + head] + (p.dt_bias ? p.dt_bias[head] : 0.f), p.softplus);
    sm.h[threadIdx.x] = h;
    sm.dec[threadIdx.x] = expf(h * p.a[head]);
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");   // the convolution's rows
  const float *rows = p.conv + (size_t)n * L * C;
  const float *x = rows + head * p.P + col0, *b = rows + p.H * p.P + group * SSM_N, *c = b + p.G * SSM_N;
  for (int i = threadIdx.x; i < (L - first) * (SSM_COLS / 4); i += 256) {
    const int t = first + i / (SSM_COLS / 4), e = i % (SSM_COLS / 4) * 4;
    *reinterpret_cast<float4 *>(&sm.x[t][e]) = __ldcg(reinterpret_cast<const float4 *>(x + (size_t)t * C + e));
  }
  for (int i = threadIdx.x; i < (L - first) * (SSM_N / 4); i += 256) {
    const int t = first + i / (SSM_N / 4), e = i % (SSM_N / 4) * 4;
    *reinterpret_cast<float4 *>(&sm.b[t][e]) = __ldcg(reinterpret_cast<const float4 *>(b + (size_t)t * C + e));
    *reinterpret_cast<float4 *>(&sm.c[t][e]) = __ldcg(reinterpret_cast<const float4 *>(c + (size_t)t * C + e));
  }
  __syncthreads();
  advance(sm, S, first, L, [&](int t) {
    if (t + 1 == acc) store_state(state, p.P, S);
  });
  __syncthreads();
  put_y(sm, first, L, p.d_skip ? p.d_skip[head] : 0.f,
        static_cast<IO *>(p.y) + (size_t)n * L * p.H * p.P + (size_t)head * p.P + col0, (long long)p.H * p.P);
}

}  // namespace

cudaError_t launch_ssm_fwd_f32(const SsmParams &p, cudaStream_t s) {
  ssm_rec_kernel<<<dim3(p.H * (p.P / SSM_COLS), p.n_seqs), 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_ssm_step(const SsmParams &p, bool f32, cudaStream_t s) {
  const int C = p.H * p.P + 2 * p.G * SSM_N;
  const dim3 cgrid((C / 2 + 255) / 256, p.n_seqs);
  if (f32) ssm_conv_step_kernel<float><<<cgrid, 256, 0, s>>>(p, C);
  else ssm_conv_step_kernel<bf16><<<cgrid, 256, 0, s>>>(p, C);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.H * (p.P / SSM_COLS), p.n_seqs);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return f32 ? cudaLaunchKernelEx(&cfg, ssm_step_kernel<float>, p, C) : cudaLaunchKernelEx(&cfg, ssm_step_kernel<bf16>, p, C);
}

}  // namespace kda
