// kda_ssm.cu -- selective state space scan token by token in fp32 on the CUDA cores: prompts with
// fp32 I/O, and the decode / verify step of both I/O types behind its short convolution.
//
//   h_t = softplus(dt_t + bias),  S_t = exp(h_t a) S_{t-1} + h_t B_t x_t^T,  y_t = S_t^T C_t + d x_t
//
// One CTA owns 64 (or 16) value columns of one (sequence, head): 256 threads hold the 128 x 64 state in
// registers, each 8 rows x 4 columns (16 lanes cover a row's 64 columns, so states move as whole 256-byte
// rows). Per token a thread reads 8 values of B, 8 of C and 4 of x from shared memory for 96 operations;
// the sums over the row groups meet once per batch of tokens. No product goes through the tensor cores, whose
// operands would not hold 24 bits. Prompts are bound by the issue of those products and sums (52% of the issue
// slots at two warps a scheduler; 2048 tokens x 96 heads of 64 in 410 us).
// Step: bound by reading and writing the 32 KB state (256 sequences x 4 slots x 96 heads of 64: 314 us for 1.67 GB, 5.3
// TB/s, when every sequence commits; 258 us for 1.38 GB at drawn prefixes, of which a third commit nothing and write no state). The convolution runs as a kernel of
// its own (its state is shared by every head of a group, so it cannot be advanced in place by the heads'
// CTAs), and the scan starts under it (programmatic dependent launch): it has its state in
// registers by the time the convolution's rows are there.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int MAX_SLOTS = 8;   // of a step

__device__ __forceinline__ float step_size(float v, bool softplus) {
  return softplus ? log1pf(expf(-fabsf(v))) + fmaxf(v, 0.f) : v;
}

// W: value columns per CTA; TB: tokens per batch. A thread owns 4 columns of R rows: q = tid % (W / 4) says which columns, g = tid / (W / 4) which rows.
template <int W, int TB>
struct Rec {
  static constexpr int Q = W / 4, G = 256 / Q, R = SSM_N / G;
  typedef float State[R][4];
  struct Smem {
    float x[TB][W], b[TB][SSM_N], c[TB][SSM_N];
    float h[TB], dec[TB];
    float yp[8][TB][W];   // per warp: sums over its rows
  };

  // Tokens t0 .. nt - 1 of the batch in `sm` through the state; commit(t) is called after token t. d x goes with the first
  // rows' sums. (Two fp32 lanes per instruction take ten registers more at W = 64, and with them the fourth CTA of an SM.)
  template <typename F>
  static __device__ __forceinline__ void advance(Smem &sm, State &S, int t0, int nt, float d, F commit) {
    const int g = threadIdx.x / Q, q = threadIdx.x % Q, warp = threadIdx.x >> 5;
    const float dg = g == 0 ? d : 0.f;
    for (int t = t0; t < nt; ++t) {
      const float h = sm.h[t], dec = sm.dec[t];
      const float4 x = *reinterpret_cast<const float4 *>(&sm.x[t][4 * q]);
      const float hx[4] = {h * x.x, h * x.y, h * x.z, h * x.w};
      float y[4] = {dg * x.x, dg * x.y, dg * x.z, dg * x.w};
      constexpr int V = R < 4 ? R : 4;   // rows per read of B and C
#pragma unroll
      for (int j = 0; j < R; j += V) {
        float b[V], c[V];
        if constexpr (V == 4) {
          *reinterpret_cast<float4 *>(b) = *reinterpret_cast<const float4 *>(&sm.b[t][R * g + j]);
          *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(&sm.c[t][R * g + j]);
        } else {
          *reinterpret_cast<float2 *>(b) = *reinterpret_cast<const float2 *>(&sm.b[t][R * g + j]);
          *reinterpret_cast<float2 *>(c) = *reinterpret_cast<const float2 *>(&sm.c[t][R * g + j]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float &s = S[j + i][k];
            s = fmaf(s, dec, b[i] * hx[k]);
            y[k] = fmaf(c[i], s, y[k]);
          }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int o = Q; o < 32; o *= 2) y[k] += __shfl_xor_sync(0xffffffffu, y[k], o);
      if ((threadIdx.x & 31) < Q) *reinterpret_cast<float4 *>(&sm.yp[warp][t][4 * q]) = make_float4(y[0], y[1], y[2], y[3]);
      commit(t);
    }
  }

  // The whole batch, four tokens at a time and two columns per instruction: what a group reads from shared memory is on its way
  // together, and its 16 sums over the lanes that share columns are taken side by side, half of the values handed over at each step.
  // Without OUT only the state moves.
  template <bool OUT>
  static __device__ __forceinline__ void advance_batch(Smem &sm, const float *hs, const float *decs, f2 (&S)[R][2], float d) {
    const int g = threadIdx.x / Q, q = threadIdx.x % Q, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool up = lane & 16, up2 = lane & 8, up4 = lane & 4;
    const float dg = g == 0 ? d : 0.f;
    constexpr int V = R < 4 ? R : 4;   // rows per read of B and C
#pragma unroll 1
    for (int t = 0; t < TB; t += 4) {
      f2 x[4][2], y[4][2];
      const float4 h4 = *reinterpret_cast<const float4 *>(hs + t), dec4 = *reinterpret_cast<const float4 *>(decs + t);
      const float h[4] = {h4.x, h4.y, h4.z, h4.w}, dec[4] = {dec4.x, dec4.y, dec4.z, dec4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4 *>(&sm.x[t + i][4 * q]);
        x[i][0] = two(v.x, v.y), x[i][1] = two(v.z, v.w);
#pragma unroll
        for (int k = 0; k < 2; ++k) y[i][k] = mul2(two(dg, dg), x[i][k]), x[i][k] = mul2(two(h[i], h[i]), x[i][k]);
      }
#pragma unroll
      for (int j = 0; j < R; j += V) {
        float b[4][V], c[4][V];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (V == 4) {
            *reinterpret_cast<float4 *>(b[i]) = *reinterpret_cast<const float4 *>(&sm.b[t + i][R * g + j]);
            if (OUT) *reinterpret_cast<float4 *>(c[i]) = *reinterpret_cast<const float4 *>(&sm.c[t + i][R * g + j]);
          } else {
            *reinterpret_cast<float2 *>(b[i]) = *reinterpret_cast<const float2 *>(&sm.b[t + i][R * g + j]);
            if (OUT) *reinterpret_cast<float2 *>(c[i]) = *reinterpret_cast<const float2 *>(&sm.c[t + i][R * g + j]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              f2 &s = S[j + v][k];
              s = fma2(s, two(dec[i], dec[i]), mul2(two(b[i][v], b[i][v]), x[i][k]));
              if (OUT) y[i][k] = fma2(two(c[i][v], c[i][v]), s, y[i][k]);
            }
      }
      if (!OUT) continue;
      float u[4][4], z[2][4];   // tokens t + 2, t + 3 in the upper lanes, t, t + 1 in the lower ones
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = of2(y[i][0]), b = of2(y[i][1]);
        u[i][0] = a.x, u[i][1] = a.y, u[i][2] = b.x, u[i][3] = b.y;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) z[i][k] = (up ? u[2 + i][k] : u[i][k]) + __shfl_xor_sync(0xffffffffu, up ? u[i][k] : u[2 + i][k], 16);
      if constexpr (Q == 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<float4 *>(&sm.yp[warp][t + (up ? 2 : 0) + i][4 * q]) = make_float4(z[i][0], z[i][1], z[i][2], z[i][3]);
      } else {
        static_assert(Q == 4, "2 or 8 lanes to a column");
        float v[4], o[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = (up2 ? z[1][k] : z[0][k]) + __shfl_xor_sync(0xffffffffu, up2 ? z[0][k] : z[1][k], 8);
#pragma unroll
        for (int k = 0; k < 2; ++k) o[k] = (up4 ? v[2 + k] : v[k]) + __shfl_xor_sync(0xffffffffu, up4 ? v[k] : v[2 + k], 4);
        *reinterpret_cast<float2 *>(&sm.yp[warp][t + (up ? 2 : 0) + (up2 ? 1 : 0)][4 * q + (up4 ? 2 : 0)]) = make_float2(o[0], o[1]);
      }
    }
  }

  // The batch's outputs: the eight warps' sums in order.
  template <typename IO>
  static __device__ __forceinline__ void put_y(const Smem &sm, int t0, int nt, IO *y, long long ldy) {
    for (int i = threadIdx.x; i < (nt - t0) * W; i += blockDim.x) {
      const int t = t0 + i / W, p = i % W;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) v += sm.yp[w][t][p];
      y[t * ldy + p] = from_f<IO>(v);
    }
  }

  static __device__ __forceinline__ void load_state(const float *src, int P, State &S) {
    const int g = threadIdx.x / Q, q = threadIdx.x % Q;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float4 v = src ? __ldcs(reinterpret_cast<const float4 *>(src + (size_t)(R * g + i) * P + 4 * q)) : make_float4(0.f, 0.f, 0.f, 0.f);
      S[i][0] = v.x, S[i][1] = v.y, S[i][2] = v.z, S[i][3] = v.w;
    }
  }
  static __device__ __forceinline__ void store_state(float *dst, int P, const State &S) {
    const int g = threadIdx.x / Q, q = threadIdx.x % Q;
#pragma unroll
    for (int i = 0; i < R; ++i)
      __stcs(reinterpret_cast<float4 *>(dst + (size_t)(R * g + i) * P + 4 * q), make_float4(S[i][0], S[i][1], S[i][2], S[i][3]));
  }
};

// Prompts. Grid: (slices of W value columns of all heads, sequences); eight warps of the state, and a ninth for the next batch's step
// sizes. The next batch's values are on their way while this one's are used. Sequences run in nseg segments of whole batches: STATES
// finds what each but the last adds to the state, and its decay; then every segment starts from what those before it make of h0.
template <int W, int TB, bool STATES>
__global__ void __launch_bounds__(288) ssm_rec_kernel(SsmParams p, int nseg, float *seg_state, float *seg_decay) {
  typedef Rec<W, TB> R;
  if (STATES) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  __shared__ __align__(16) typename R::Smem sm;
  __shared__ __align__(16) float steps[2][2][TB];   // by batch: h, exp(h a)
  const int slices = p.P / W, head = blockIdx.x / slices, col0 = (blockIdx.x % slices) * W;
  const int runs = STATES ? nseg - 1 : nseg, n = blockIdx.y / runs, seg = blockIdx.y % runs;
  const int group = head / (p.H / p.G), tid = threadIdx.x, lane = tid & 31;
  const bool scalars = tid >= 256;
  const long long seq0 = max(p.cu ? (long long)p.cu[n] : p.T / p.n_seqs * n, 0LL), seq1 = min(p.cu ? (long long)p.cu[n + 1] : p.T / p.n_seqs * (n + 1), p.T);
  const long long batches = seq1 > seq0 ? (seq1 - seq0 + TB - 1) / TB : 0;
  const long long t0 = seq0 + batches * seg / nseg * TB, t1 = min(seq1, seq0 + batches * (seg + 1) / nseg * TB);
  const size_t soff = ((size_t)n * p.H + head) * SSM_N * p.P + col0;
  const float a = p.a[head], bias = p.dt_bias ? p.dt_bias[head] : 0.f, d = p.d_skip ? p.d_skip[head] : 0.f;
  typename R::State S;
  if (!scalars) R::load_state(!STATES && p.h0 ? p.h0 + soff : nullptr, p.P, S);
  f2 S2[R::R][2];
#pragma unroll
  for (int i = 0; i < R::R; ++i) S2[i][0] = two(S[i][0], S[i][1]), S2[i][1] = two(S[i][2], S[i][3]);
  if (!STATES && nseg > 1) asm volatile("griddepcontrol.wait;\n" ::: "memory");   // the states' pass
  if (!STATES && !scalars)
#pragma unroll 4
    for (int k = 0; k < seg; ++k) {
      const size_t at = ((size_t)n * (nseg - 1) + k) * gridDim.x + blockIdx.x;
      const float dec = seg_decay[at];
      R::load_state(seg_state + at * SSM_N * W, W, S);
#pragma unroll
      for (int i = 0; i < R::R; ++i) {
        S2[i][0] = fma2(S2[i][0], two(dec, dec), two(S[i][0], S[i][1]));
        S2[i][1] = fma2(S2[i][1], two(dec, dec), two(S[i][2], S[i][3]));
      }
    }
  // thread: four values of B and of C of tokens tid / 32, tid / 32 + 8, ..., and (the first threads) four of x
  constexpr int K = TB / 8;
  float4 xv, bv[K], cv[K];
  const int bt = tid >> 5, be = (tid & 31) * 4, xt = tid / (W / 4), xe = tid % (W / 4) * 4;
  const float *x = static_cast<const float *>(p.x) + (t0 + xt) * p.ldx + (long long)head * p.P + col0 + xe;
  const float *b = static_cast<const float *>(p.b) + (t0 + bt) * p.ldb + (long long)group * SSM_N + be;
  const float *c = static_cast<const float *>(p.c) + (t0 + bt) * p.ldc + (long long)group * SSM_N + be;
  const float *dt = p.dt + (t0 + lane) * p.H + head;
  float *y = static_cast<float *>(p.y) + t0 * p.H * p.P + (long long)head * p.P + col0;
  const long long ldy = (long long)p.H * p.P;
  auto fetch = [&](int left) {   // of the batch that the pointers have reached, `left` tokens before the sequence's end; then past it
    xv = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      bv[k] = cv[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (bt + 8 * k < left) {
        bv[k] = *reinterpret_cast<const float4 *>(b + 8 * k * p.ldb);
        if (!STATES) cv[k] = *reinterpret_cast<const float4 *>(c + 8 * k * p.ldc);
      }
    }
    if (xt < TB && xt < left) xv = *reinterpret_cast<const float4 *>(x);
    x += TB * p.ldx, b += TB * p.ldb, c += TB * p.ldc;
  };
  float dv = 0.f, log_dec = 0.f;
  auto fetch_dt = [&](int left) {
    dv = lane < TB && lane < left ? *dt : 0.f;
    dt += (long long)TB * p.H;
  };
  auto put_steps = [&](int which, int left) {   // past the end: tokens that leave the state as it is
    if (lane < TB) {
      const float h = step_size(dv + bias, p.softplus);
      if (lane < left) log_dec += h * a;
      steps[which][0][lane] = lane < left ? h : 0.f;
      steps[which][1][lane] = lane < left ? expf(h * a) : 1.f;
    }
  };
  int left = (int)(t1 > t0 ? t1 - t0 : 0), which = 0;
  if (left > 0) {
    if (scalars) {
      fetch_dt(left);
      put_steps(0, left);
      fetch_dt(left - TB);
    } else {
      fetch(left);
    }
  }
#pragma unroll 1
  for (; left > 0; left -= TB, which ^= 1, y += TB * ldy) {
    if (!scalars) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        *reinterpret_cast<float4 *>(&sm.b[bt + 8 * k][be]) = bv[k];
        if (!STATES) *reinterpret_cast<float4 *>(&sm.c[bt + 8 * k][be]) = cv[k];
      }
      if (xt < TB) *reinterpret_cast<float4 *>(&sm.x[xt][xe]) = xv;
    }
    __syncthreads();   // the batch is there; the previous one's outputs have been read
    if (scalars) {
      put_steps(which ^ 1, left - TB);
      fetch_dt(left - 2 * TB);
    } else {
      fetch(left - TB);
      R::template advance_batch<!STATES>(sm, steps[which][0], steps[which][1], S2, d);
    }
    __syncthreads();   // the batch is consumed, its sums are there
    if (!STATES) R::put_y(sm, 0, left < TB ? left : TB, y, ldy);
  }
  const size_t at = ((size_t)n * (nseg - 1) + seg) * gridDim.x + blockIdx.x;
  if (STATES && scalars) {
#pragma unroll
    for (int o = 16; o; o >>= 1) log_dec += __shfl_xor_sync(0xffffffffu, log_dec, o);
    if (lane == 0) seg_decay[at] = expf(log_dec);
  }
  if (!scalars && (STATES || (p.hT && seg == nseg - 1))) {
#pragma unroll
    for (int i = 0; i < R::R; ++i) {
      const float2 v = of2(S2[i][0]), w = of2(S2[i][1]);
      S[i][0] = v.x, S[i][1] = v.y, S[i][2] = w.x, S[i][3] = w.y;
    }
    if (STATES) R::store_state(seg_state + at * SSM_N * W, W, S);
    else R::store_state(p.hT + soff, p.P, S);
  }
}

// z / (1 + e^-z). With fp32 I/O to 2^-22 of a value (256 sequences x 4 slots x 96 heads of 64: 326 us, 322 with the approximations). With
// bf16 I/O by the hardware's 2^x and quotient: the rounding of z log2(e) makes that up to (9 + 2.4 |z|) 2^-24 of a value (4e-6 measured
// up to |z| = 85), beside inputs and outputs of 2^-9.
template <typename IO>
__device__ __forceinline__ float silu(float z) {
  if constexpr (sizeof(IO) == 4) return __fdiv_rn(z, 1.f + expf(-z));
  else return __fdividef(z, 1.f + __expf(-z));
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
  IO *st = static_cast<IO *>(p.conv_state) + (size_t)slot * K * C + c;
  const IO *x = static_cast<const IO *>(p.xbc) + (size_t)n * L * C + c;
  float2 row[3 + MAX_SLOTS];   // K earlier inputs in rows 3 - K .. 2, then the slots; all on their way at once
#pragma unroll
  for (int j = 0; j < 3 + MAX_SLOTS; ++j) {
    row[j] = make_float2(0.f, 0.f);
    if (j < 3 ? j >= 3 - K : j - 3 >= first && j - 3 < L) row[j] = j < 3 ? ld2(st + (size_t)(j - (3 - K)) * C) : ld2(x + (size_t)(j - 3) * C);
  }
  float w0[4], w1[4], win[4][2];   // right-aligned: tap 3 is the current token
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = j - (4 - p.W);
    w0[j] = k >= 0 ? p.cw[(size_t)c * p.W + k] : 0.f;
    w1[j] = k >= 0 ? p.cw[(size_t)(c + 1) * p.W + k] : 0.f;
    win[j][0] = j < 3 ? row[j < 3 ? j : 0].x : 0.f;
    win[j][1] = j < 3 ? row[j < 3 ? j : 0].y : 0.f;
  }
  const float b0 = p.cbias ? p.cbias[c] : 0.f, b1 = p.cbias ? p.cbias[c + 1] : 0.f;
  float *out = p.conv + (size_t)n * L * C + c;
#pragma unroll
  for (int s = 0; s < MAX_SLOTS; ++s)
    if (s >= first && s < L) {
      win[3][0] = row[3 + s].x;
      win[3][1] = row[3 + s].y;
      float z0 = b0, z1 = b1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z0 = fmaf(w0[j], win[j][0], z0);
        z1 = fmaf(w1[j], win[j][1], z1);
      }
      if (p.act) {
        z0 = silu<IO>(z0);
        z1 = silu<IO>(z1);
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
__global__ void __launch_bounds__(256, 4) ssm_step_kernel(SsmParams p, int C) {
  typedef Rec<SSM_COLS, MAX_SLOTS> R;
  __shared__ __align__(16) R::Smem sm;
  const int slices = p.P / SSM_COLS, head = blockIdx.x / slices, col0 = (blockIdx.x % slices) * SSM_COLS, n = blockIdx.y;
  const int slot = p.idx ? p.idx[n] : n;
  if (slot < 0 || slot >= p.n_slots) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");   // this grid ends after the convolution's
    return;
  }
  const int group = head / (p.H / p.G), L = p.L;
  const int first = p.first ? min(max(p.first[n], 0), L) : 0, acc = p.acc ? min(max(p.acc[n], 0), L) : L;
  float *state = p.state + ((size_t)slot * p.H + head) * SSM_N * p.P + col0;
  R::State S;
  R::load_state(state, p.P, S);
  // the step sizes fall to the warp with the least to copy; everything is on its way before they are computed
  const int tid = threadIdx.x, ht = tid - 224;
  const bool steps = ht >= 0 && ht < L;
  const float bias = p.dt_bias ? p.dt_bias[head] : 0.f, a = p.a[head];
  const float dt = steps ? p.dt[((size_t)n * L + ht) * p.H + head] : 0.f;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");   // the convolution's rows
  const float *rows = p.conv + (size_t)n * L * C;
  const float *x = rows + head * p.P + col0, *b = rows + p.H * p.P + group * SSM_N, *c = b + p.G * SSM_N;
  const int xt = tid >> 4, xe = (tid & 15) * 4, bt = tid >> 5, be = (tid & 31) * 4;   // one float4 each of x, B and C
  float4 xv, bv, cv;
  const bool xin = xt >= first && xt < L, bin = bt >= first && bt < L;
  if (xin) xv = __ldcg(reinterpret_cast<const float4 *>(x + (size_t)xt * C + xe));
  if (bin) {
    bv = __ldcg(reinterpret_cast<const float4 *>(b + (size_t)bt * C + be));
    cv = __ldcg(reinterpret_cast<const float4 *>(c + (size_t)bt * C + be));
  }
  if (steps) {
    const float h = step_size(dt + bias, p.softplus);
    sm.h[ht] = h;
    sm.dec[ht] = expf(h * a);
  }
  if (xin) *reinterpret_cast<float4 *>(&sm.x[xt][xe]) = xv;
  if (bin) {
    *reinterpret_cast<float4 *>(&sm.b[bt][be]) = bv;
    *reinterpret_cast<float4 *>(&sm.c[bt][be]) = cv;
  }
  __syncthreads();
  R::advance(sm, S, first, L, p.d_skip ? p.d_skip[head] : 0.f, [&](int t) {
    if (t + 1 == acc) R::store_state(state, p.P, S);
  });
  __syncthreads();
  R::put_y(sm, first, L,
           static_cast<IO *>(p.y) + (size_t)n * L * p.H * p.P + (size_t)head * p.P + col0, (long long)p.H * p.P);
}

}  // namespace

// 64 columns per CTA do the least work per token (B and C are read by fewer threads): 2048 tokens x 96 heads of 64 take 410 us.
// Where that leaves the device mostly empty, 16 columns take half the time per token, 92 ns, most of it the issue of a token's products
// and sums: 512 tokens x 2 heads of 128 50 us, 104 us with 64. A second CTA on an SM makes the two about 1.75 times as long.
// Segments shorten the walk where CTAs are still few. The pass over the states takes half the time of a full one, and the second launch
// and the folding about as long as 30 tokens and 2 per segment: 4096 tokens x 2 heads of 64 376 us in one piece and 43 in 16 segments,
// 512 x 2 heads of 128 50 and 16 us, 128 x 2 heads of 128 15 and 9 us. At 256 CTAs of 2048 tokens two segments take 402 us and one 328.
SsmRecPlan ssm_rec_plan(int n_seqs, long long T, int H, int P) {
  SsmRecPlan l = {SSM_COLS, 1, 0};
  if (n_seqs < 1) return l;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    (void)cudaGetLastError();
    sms = 152;
  }
  if ((long long)H * (P / 16) * n_seqs <= 2LL * sms) l.cols = 16;
  const long long ctas = (long long)H * (P / l.cols) * n_seqs;
  const double each = (double)T / n_seqs;
  auto walk = [&](long long n) -> double {   // how much longer n CTAs take than one
    const double m = (double)((n + sms - 1) / sms);
    return l.cols == 16 && m > 1 ? 0.87 * m : m;
  };
  double cost = 0.9 * each * walk(ctas);   // less than a tenth to gain is left alone: 2048 tokens x 96 heads of 64 410 us, 433 in 11 segments
  for (int k = 2; k <= 16 && 16 * k <= each && (long long)n_seqs * k <= 65535; ++k) {
    const double t = 1.5 * each / k * walk(ctas * k) + 30.0 + 2.0 * k;
    if (t < cost) cost = t, l.nseg = k;
  }
  const size_t items = (size_t)(l.nseg - 1) * (size_t)ctas;
  l.bytes = items * SSM_N * l.cols * sizeof(float) + (items * sizeof(float) + 255) / 256 * 256;
  return l;
}

template <int W, int TB>
cudaError_t launch_rec(const SsmParams &p, const SsmRecPlan &l, void *workspace, cudaStream_t s) {
  const unsigned slices = (unsigned)(p.H * (p.P / W));
  float *state = static_cast<float *>(workspace), *decay = state + (size_t)(l.nseg - 1) * p.n_seqs * slices * SSM_N * W;
  if (l.nseg > 1) {
    ssm_rec_kernel<W, TB, true><<<dim3(slices, p.n_seqs * (l.nseg - 1)), 288, 0, s>>>(p, l.nseg, state, decay);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_under(ssm_rec_kernel<W, TB, false>, dim3(slices, p.n_seqs * l.nseg), 288, 0, s, p, l.nseg, state, decay);
  }
  ssm_rec_kernel<W, TB, false><<<dim3(slices, p.n_seqs), 288, 0, s>>>(p, 1, state, decay);
  return cudaGetLastError();
}
cudaError_t launch_ssm_fwd_f32(const SsmParams &p, const SsmRecPlan &l, void *workspace, cudaStream_t s) {
  return l.cols == 16 ? launch_rec<16, 16>(p, l, workspace, s) : launch_rec<SSM_COLS, 8>(p, l, workspace, s);
}

cudaError_t launch_ssm_step(const SsmParams &p, bool f32, cudaStream_t s) {
  const int C = p.H * p.P + 2 * p.G * SSM_N;
  const dim3 cgrid((C / 2 + 255) / 256, p.n_seqs);
  if (f32) ssm_conv_step_kernel<float><<<cgrid, 256, 0, s>>>(p, C);
  else ssm_conv_step_kernel<bf16><<<cgrid, 256, 0, s>>>(p, C);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid(p.H * (p.P / SSM_COLS), p.n_seqs);
  return f32 ? launch_under(ssm_step_kernel<float>, grid, 256, 0, s, p, C) : launch_under(ssm_step_kernel<bf16>, grid, 256, 0, s, p, C);
}

}  // namespace kda
