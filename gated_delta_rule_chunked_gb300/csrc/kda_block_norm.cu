// kda_block_norm.cu -- the norm after a block with its gate and residual scale, the residual
// sum and the norm before the next block, forward and backward.
//
//   hat = u r_u, r_u = (mean u^2 + eps)^(-1/2) (1 without w_post);  h = hat act(z);  m = w_post h
//   x = residual + scale m;   normed = w_pre x r_x, r_x = (mean x^2 + eps)^(-1/2)
// Backward, D = d_out, E = d_normed:
//   dx = D + r_x (E w_pre) - x r_x^3 mean((E w_pre) x),  dresidual = dx,  dw_pre = sum E x r_x
//   A = sum dx h per column, so dscale = w_post A and dw_post = scale A (one accumulator)
//   t = dx scale w_post,  dz = t hat act'(z),  dhat = t act(z),  du = r_u (dhat - hat mean(dhat hat))
// (dhat hat = dx m summed over a row, with m = scale w_post h)
// Memory-bound: every tensor is read and written once, everything in between is fp32 registers. In bf16 the forward
// moves 2.35 GB at 32768 x 7168 in 0.356 ms (6.6 TB/s, 97% of a copy) and 0.30 GB at 393216 x 128 in 51 us (5.9 TB/s); the
// backward moves 1.88 GB at 16384 x 7168 in 0.367 ms (5.1 TB/s): it keeps 14 warps on an SM, whose registers the sums over rows
// and the column vectors fill, and issues in 55% of the slots. In fp32 8192 x 7168 take 174 us forward (6.7 TB/s) and 295 us backward (6.4
// TB/s). The backward of short rows moves 0.50 GB at 393216 x 128 in bf16 in 112 us (4.5 TB/s): a thread asks for its next row only when it
// has stored the current one, at 16 warps an SM.
// Forward: a row is owned by LPR lanes of a warp (short rows) or by a whole CTA (LPR = 0), each thread
// holding VPT vectors of 8 elements.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

// 8 elements of a row in their stored form; as pairs of fp32.
template <typename IO> struct Raw;
template <> struct Raw<bf16> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16 *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void loads(const char *p) { v = *reinterpret_cast<const uint4 *>(p); }   // from shared memory
  __device__ __forceinline__ void get(f2 (&x)[4]) const { x[0] = unpack2(v.x), x[1] = unpack2(v.y), x[2] = unpack2(v.z), x[3] = unpack2(v.w); }
};
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = __ldcs(reinterpret_cast<const float4 *>(p));
    b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ void loads(const char *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ void get(f2 (&x)[4]) const { x[0] = two(a.x, a.y), x[1] = two(a.z, a.w), x[2] = two(b.x, b.y), x[3] = two(b.z, b.w); }
};
__device__ __forceinline__ void store8(bf16 *p, const f2 (&x)[4]) {
  __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3])));
}
__device__ __forceinline__ void store8(float *p, const f2 (&x)[4]) {
  const float2 a = of2(x[0]), b = of2(x[1]), c = of2(x[2]), d = of2(x[3]);
  __stcs(reinterpret_cast<float4 *>(p), make_float4(a.x, a.y, b.x, b.y));
  __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(c.x, c.y, d.x, d.y));
}
// 8 fp32 values of a column vector, or ones.
__device__ __forceinline__ void col8(const float *w, int c, f2 (&x)[4]) {
  if (w) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(w + c)), b = __ldg(reinterpret_cast<const float4 *>(w + c) + 1);
    x[0] = two(a.x, a.y), x[1] = two(a.z, a.w), x[2] = two(b.x, b.y), x[3] = two(b.z, b.w);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = two(1.f, 1.f);
  }
}
__device__ __forceinline__ f2 both(float a) { return two(a, a); }
__device__ __forceinline__ float sum(f2 a) {
  const float2 v = of2(a);
  return v.x + v.y;
}

// Sum over the LPR lanes that share a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over a row that is the CTA's. `red` holds two sets of per-warp partials that consecutive calls
// alternate (`set`), so one barrier per call is enough.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float *red, int set) {
  if constexpr (LPR != 0) {
    return row_sum<LPR>(v);
  } else {
    v = row_sum<32>(v);
    const int nw = blockDim.x >> 5;
    float *r = red + set * 32;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < nw; ++w) v += r[w];
    return v;
  }
}

// 1 / d for d >= 1, within half a unit in the last place and 2^-46: one Newton-Raphson step, r + r (1 - d r), on the hardware's reciprocal
// (2^-23). From 2^126 on that is 0, and stays 0.
__device__ __forceinline__ float reciprocal(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(d));
  return fmaf(r, fmaf(-fminf(d, 0x1p127f), r, 1.f), r);
}
// 1 / (1 + e^-z). fp32 rows by expf and the refined reciprocal, to 2^-22 of a value (8192 x 7168 with SiLU:
// forward 176 -> 178 us, backward 341 -> 353; with a correctly rounded reciprocal 223 and 402). bf16 rows by the hardware's 2^x and reciprocal: the
// rounding of z log2(e) makes that up to (9 + 2.4 |z|) 2^-24 of a value, beside results rounded at 2^-9.
template <typename IO>
__device__ __forceinline__ f2 sigmoid(f2 z) {
  if constexpr (sizeof(IO) == 4) {
    const float2 v = of2(z), d = of2(add2(two(expf(-v.x), expf(-v.y)), both(1.f)));
    return two(reciprocal(d.x), reciprocal(d.y));
  } else {
    const float2 t = of2(mul2(z, both(-LOG2E)));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e.y) : "f"(t.y));
    e = of2(add2(two(e.x, e.y), both(1.f)));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r.y) : "f"(e.y));
    return two(r.x, r.y);
  }
}
enum { GATE_NONE = 0, GATE_SIGMOID = 1, GATE_SILU = 2 };
template <typename IO, int GATE>
__device__ __forceinline__ f2 gate_of(f2 z) {
  return GATE == GATE_SILU ? mul2(z, sigmoid<IO>(z)) : sigmoid<IO>(z);
}

// The backward of 8 columns of a row. Both sums of a row's gradient come from one pass, because
// dx = dx0 - x cx with dx0 = D + r_x E w_pre known before the sums and cx = r_x^3 mean(E w_pre x) after:
//   sum dhat hat = sum dx m = sum dx0 m - cx sum x m
// so a row has one reduction, of three values. The column vectors and the sums over rows stay in registers.
template <typename IO>
struct BwdCols {
  f2 ws[4], wp[4], A[4], P[4];   // w_post scale, w_pre, the sums over rows
  __device__ __forceinline__ BwdCols(const BlockNormParams &p, int c) {
    f2 sc[4];
    col8(p.w_post, c, ws);
    col8(p.scale, c, sc);
    col8(p.w_pre, c, wp);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ws[e] = mul2(ws[e], sc[e]);
      A[e] = P[e] = both(0.f);
    }
  }
};
// FULL: the residual and both gradients are there, as in a training block.
template <typename IO, int GATE, bool FULL>
struct BwdRow {   // what the second half of a row needs of the first, beside u and z
  f2 x[4], dx[4];
  float ru, rx;
  // s = {r_x sum (E w_pre) x, sum dx0 m, sum x m} of these columns.
  __device__ __forceinline__ void first(const BlockNormParams &p, BwdCols<IO> &col, const Raw<IO> &u, const Raw<IO> &z, const Raw<IO> &res, const Raw<IO> &dn,
                                        const Raw<IO> &dout, float (&s)[3]) {
    f2 m[4], t[4];
    u.get(m);
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = mul2(m[e], mul2(both(ru), col.ws[e]));
    if (GATE) {
      z.get(t);
#pragma unroll
      for (int e = 0; e < 4; ++e) m[e] = mul2(m[e], gate_of<IO, GATE>(t[e]));
    }
    if (FULL || p.residual) {
      res.get(x);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = add2(x[e], m[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = m[e];
    }
    if (FULL || p.d_out) {
      dout.get(dx);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) dx[e] = both(0.f);
    }
    f2 s0 = both(0.f), s1 = s0, s2 = s0;
    if (FULL || p.d_normed) {
      dn.get(t);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f2 n = mul2(t[e], both(rx)), f = mul2(n, col.wp[e]);
        col.P[e] = fma2(n, x[e], col.P[e]);
        s0 = fma2(f, x[e], s0);
        dx[e] = add2(dx[e], f);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s1 = fma2(dx[e], m[e], s1);
      s2 = fma2(x[e], m[e], s2);
    }
    s[0] = sum(s0), s[1] = sum(s1), s[2] = sum(s2);
  }
  // With the row's sums: the gradients of its columns, and A.
  __device__ __forceinline__ void second(const BlockNormParams &p, BwdCols<IO> &col, const Raw<IO> &u, const Raw<IO> &z, const float (&s)[3],
                                         long long base) {
    const float cx = s[0] * p.inv_dim * rx * rx, ch = p.w_post ? (s[1] - cx * s[2]) * p.inv_dim : 0.f;
    f2 hat[4], t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) dx[e] = fma2(both(-cx), x[e], dx[e]);
    if (FULL || p.residual) store8(static_cast<IO *>(p.d_residual) + base, dx);
    u.get(hat);
#pragma unroll
    for (int e = 0; e < 4; ++e) hat[e] = mul2(hat[e], both(ru));
    if (GATE) {
      z.get(t);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f2 sg = sigmoid<IO>(t[e]), g = GATE == GATE_SILU ? mul2(t[e], sg) : sg, v = mul2(dx[e], hat[e]);
        // act' = sg + g (1 - sg) for SiLU, sg (1 - sg) for the sigmoid
        const f2 slope = GATE == GATE_SILU ? fma2(mul2(g, both(-1.f)), sg, add2(sg, g)) : fma2(mul2(sg, both(-1.f)), sg, sg);
        t[e] = mul2(mul2(v, col.ws[e]), slope);
        col.A[e] = fma2(v, g, col.A[e]);
        dx[e] = mul2(dx[e], mul2(col.ws[e], g));
      }
      store8(static_cast<IO *>(p.d_gate) + base, t);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        col.A[e] = fma2(dx[e], hat[e], col.A[e]);
        dx[e] = mul2(dx[e], col.ws[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) dx[e] = mul2(both(ru), fma2(both(-ch), hat[e], dx[e]));
    store8(static_cast<IO *>(p.du) + base, dx);
  }
};

// CTAs of 512 threads on an SM, which bounds the registers: a row waits twice for its sums, and only other rows fill those times
// (one CTA more: 32768 x 7168 bf16 0.391 -> 0.356 ms, fp32 5.5 -> 6.8 TB/s; 16384 columns bf16 4.9 -> 6.2 TB/s). In fp32 with
// four vectors a thread a second one would spill.
template <typename IO>
constexpr int fwd_ctas(int lpr, int vpt) {
  if (lpr || vpt == 1) return 0;   // no bound: they hold few registers by themselves, and take more where one CTA is asked for
  return sizeof(IO) == 2 ? (vpt == 2 ? 3 : 2) : (vpt == 2 ? 2 : 1);
}
// One row per (CTA or LPR lanes); the grid covers all rows.
template <typename IO, int GATE, int LPR, int VPT>
__global__ void __launch_bounds__(LPR ? 256 : 512, fwd_ctas<IO>(LPR, VPT)) block_norm_fwd_kernel(BlockNormParams p) {
  __shared__ float red[64];
  const int lane = LPR ? (threadIdx.x & (LPR - 1)) : threadIdx.x, step = LPR ? LPR : blockDim.x;
  const int nvec = p.dim >> 3;
  const long long row = LPR ? (long long)blockIdx.x * (blockDim.x / (LPR ? LPR : 1)) + threadIdx.x / (LPR ? LPR : 1) : blockIdx.x;
  const bool live = row < p.rows;   // the dead rows of the last CTA still take part in the shuffles
  const long long base = row * p.dim;
  if (LPR == 0 && threadIdx.x < 3 && row + p.prefetch_dist < p.rows && p.prefetch_dist > 0) {
    // a later row of each input into L2, for the CTA that will take it
    const void *src = threadIdx.x == 0 ? p.u : (threadIdx.x == 1 ? p.gate : p.residual);
    if (src) prefetch_l2(static_cast<const IO *>(src) + (row + p.prefetch_dist) * p.dim, (uint32_t)(p.dim * sizeof(IO)));
  }
  Raw<IO> u[VPT], z[VPT], r[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + step * j;
    if (live && v < nvec) {
      u[j].load(static_cast<const IO *>(p.u) + base + v * 8);
      if (GATE) z[j].load(static_cast<const IO *>(p.gate) + base + v * 8);
      if (p.residual) r[j].load(static_cast<const IO *>(p.residual) + base + v * 8);
    }
  }
  float ru = 1.f;
  if (p.w_post) {
    f2 s = both(0.f);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (live && lane + step * j < nvec) {
        f2 x[4];
        u[j].get(x);
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fma2(x[e], x[e], s);
      }
    ru = rsqrtf(row_sum<LPR>(sum(s), red, 0) * p.inv_dim + p.eps);
    if (live && lane == 0) p.rstd_post[row] = ru;
  }
  f2 x[VPT][4], s = both(0.f);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + step * j;
    if (live && v < nvec) {
      f2 w[4], g[4];
      u[j].get(x[j]);
      col8(p.w_post, v * 8, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[j][e] = mul2(x[j][e], mul2(both(ru), w[e]));
      if (GATE) {
        z[j].get(g);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] = mul2(x[j][e], gate_of<IO, GATE>(g[e]));
      }
      if (p.scale) {
        col8(p.scale, v * 8, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] = mul2(x[j][e], w[e]);
      }
      if (p.residual) {
        r[j].get(g);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] = add2(x[j][e], g[e]);
      }
      store8(static_cast<IO *>(p.out) + base + v * 8, x[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) s = fma2(x[j][e], x[j][e], s);
    }
  }
  if (!p.w_pre) return;
  const float rx = rsqrtf(row_sum<LPR>(sum(s), red, 1) * p.inv_dim + p.eps);
  if (live && lane == 0) p.rstd_pre[row] = rx;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + step * j;
    if (live && v < nvec) {
      f2 w[4];
      col8(p.w_pre, v * 8, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[j][e] = mul2(x[j][e], mul2(both(rx), w[e]));
      store8(static_cast<IO *>(p.normed) + base + v * 8, x[j]);
    }
  }
}

// Short rows. Persistent: CTA b takes row groups b, b + gridDim, ...; a thread keeps its 8 columns, so A
// and dw_pre accumulate in registers. partial[b][2][d] at the end (the CTA's rows added in a fixed
// order), summed over b by block_norm_dw_kernel.
template <typename IO, int GATE, int LPR>
__global__ void __launch_bounds__(256) block_norm_bwd_short_kernel(BlockNormParams p) {
  extern __shared__ float bn_smem[];   // [2][rows per CTA][d] partials
  const int lane = threadIdx.x & (LPR - 1), rpc = blockDim.x / LPR, sub = threadIdx.x / LPR;
  const int c = lane * 8;
  const bool in = c < p.dim;
  BwdCols<IO> col(p, in ? c : 0);
  for (long long row0 = (long long)blockIdx.x * rpc; row0 < p.rows; row0 += (long long)gridDim.x * rpc) {
    const long long r = row0 + sub, base = r * p.dim + c;
    const bool live = in && r < p.rows;
    BwdRow<IO, GATE, false> row;
    Raw<IO> u, z;
    float s[3] = {0.f, 0.f, 0.f};
    if (live) {
      Raw<IO> res, dn, dout;
      u.load(static_cast<const IO *>(p.u) + base);
      if (GATE) z.load(static_cast<const IO *>(p.gate) + base);
      if (p.residual) res.load(static_cast<const IO *>(p.residual) + base);
      if (p.d_normed) dn.load(static_cast<const IO *>(p.d_normed) + base);
      if (p.d_out) dout.load(static_cast<const IO *>(p.d_out) + base);
      row.ru = p.w_post ? p.rstd_post[r] : 1.f;
      row.rx = p.w_pre ? p.rstd_pre[r] : 0.f;
      row.first(p, col, u, z, res, dn, dout, s);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) s[i] = row_sum<LPR>(s[i]);
    if (live) row.second(p, col, u, z, s, base);
  }
  if (in)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      *reinterpret_cast<float2 *>(&bn_smem[(size_t)sub * p.dim + c + 2 * e]) = of2(col.A[e]);
      *reinterpret_cast<float2 *>(&bn_smem[(size_t)(rpc + sub) * p.dim + c + 2 * e]) = of2(col.P[e]);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.dim; i += blockDim.x) {
    const int which = i / p.dim, col = i - which * p.dim;
    float t = 0.f;
    for (int k = 0; k < rpc; ++k) t += bn_smem[(size_t)(which * rpc + k) * p.dim + col];
    p.partial[((size_t)blockIdx.x * 2 + which) * p.dim + col] = t;
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ranks() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(r));
  return r;
}
// A row's three sums over a cluster. Inside a warp they are reduced together: after two halving steps lane
// group g (8 lanes) holds value g, so six shuffles do. Every warp then sends its parts to every CTA of the
// cluster by asynchronous stores that count on the receiver's barrier: no fence, which would wait for the
// row's stores to global memory. red: [4][64] floats of the receiver, value by warp of the cluster.
constexpr int SENT = 64;   // places per value: 8 CTAs x 8 warps
__device__ __forceinline__ void send_sums(const float (&s)[3], float *red, uint64_t *bar, uint32_t rank, uint32_t ranks) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const bool up = lane & 16, up2 = lane & 8;
  float a = up ? s[2] : s[0], b = up ? 0.f : s[1];   // values 2, 3 above lane 16, 0, 1 below
  a += __shfl_xor_sync(0xffffffffu, up ? s[0] : s[2], 16);
  b += __shfl_xor_sync(0xffffffffu, up ? s[1] : 0.f, 16);
  float v = up2 ? b : a;
  v += __shfl_xor_sync(0xffffffffu, up2 ? a : b, 8);
#pragma unroll
  for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((uint32_t)(lane & 7) < ranks) {
    uint32_t d, m;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(d) : "r"(smem_u32(red + (lane >> 3) * SENT + rank * nw + warp)), "r"(lane & 7));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(m) : "r"(smem_u32(bar)), "r"(lane & 7));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];\n" ::"r"(d), "f"(v), "r"(m) : "memory");
  }
}
__device__ __forceinline__ void take_sums(float (&s)[3], const float *red, uint32_t ranks) {
  const int lane = threadIdx.x & 31, n = (int)(blockDim.x >> 5) * (int)ranks;
  float v = 0.f;
  for (int i = lane & 7; i < n; i += 8) v += red[(lane >> 3) * SENT + i];
#pragma unroll
  for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
#pragma unroll
  for (int i = 0; i < 3; ++i) s[i] = __shfl_sync(0xffffffffu, v, 8 * i);
}

// Long rows: a cluster of CTAs per row, each with 8 columns per thread. Persistent: cluster k of K takes
// rows k, k + K, ...; the row's slices of the inputs arrive by bulk copies into a ring of p.stages buffers
// (a row's buffer serves both its halves, and is refilled at the end of the next row's turn). A row's sums travel while the next row's first half is
// computed. The two arrays of sums alternate: a CTA's parts of row i + 2 are sent after it has all parts
// of row i + 1, and a warp sends those after it has read the sums of row i.
template <typename IO, int GATE, bool FULL>
__global__ void __launch_bounds__(256, 2) block_norm_bwd_kernel(BlockNormParams p) {
  extern __shared__ __align__(128) char bn_ring[];
  __shared__ float red[2][4 * SENT];
  __shared__ __align__(8) uint64_t bar[8];   // 0, 1 the sums, 2.. the ring
  constexpr int VB = 8 * (int)sizeof(IO);   // bytes of a thread's columns
  const uint32_t rank = cluster_rank(), ranks = cluster_ranks();
  const int tid = threadIdx.x, nvec = p.dim >> 3, per = (nvec + (int)ranks - 1) / (int)ranks;
  const int vbeg = (int)rank * per, own = min(per, nvec - vbeg);
  const long long K = gridDim.x / ranks, k0 = blockIdx.x / ranks;
  const bool in = tid < own;
  const int c = (vbeg + (in ? tid : 0)) * 8;
  const uint32_t slice = (uint32_t)own * VB, sent = 16u * ranks * (blockDim.x >> 5);
  const int stride = per * VB, buffer = 5 * stride;   // a tensor's slice, a row's
  if (tid == 0) {
    for (int i = 0; i < 8; ++i) mbar_init(&bar[i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  // every CTA's barriers exist before a peer's sums reach them
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  auto issue = [&](long long r, int b) {   // thread 0
    const void *src[5] = {p.u, p.gate, p.residual, p.d_normed, p.d_out};
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) n += src[i] ? slice : 0u;
    mbar_expect_tx(&bar[2 + b], n);
#pragma unroll
    for (int i = 0; i < 5; ++i)
      if (src[i]) bulk_g2s(bn_ring + b * buffer + i * stride, static_cast<const IO *>(src[i]) + r * p.dim + (size_t)vbeg * 8, slice, &bar[2 + b]);
  };
  long long ahead = k0;   // the next row to ask for: at the end of a turn the previous row's buffer is free, the current row's is not
  if (tid == 0)
    for (int i = 0; i < p.stages - 1 && ahead < p.rows; ++i, ahead += K) issue(ahead, i);
  int fill = p.stages - 1;
  BwdCols<IO> col(p, c);
  BwdRow<IO, GATE, FULL> prev;
  bool ok = true;
  int b = 0, it = 0;
  uint32_t phase = 0;
  float ru = 1.f, rx = 0.f;
  auto stats = [&](long long r) {   // loaded a row ahead
    if (r < p.rows) {
      if (p.w_post) ru = p.rstd_post[r];
      if (p.w_pre) rx = p.rstd_pre[r];
    }
  };
  auto finish = [&](long long r, int pb, int i) {   // the second half of row r = number i, in buffer pb
    ok &= mbar_wait_quiet(&bar[i & 1], (i >> 1) & 1);
    float s[3];
    take_sums(s, red[i & 1], ranks);
    if (in) {
      const char *buf = bn_ring + pb * buffer + (size_t)tid * VB;
      Raw<IO> u, z;
      u.loads(buf);
      z.loads(buf + stride);
      prev.second(p, col, u, z, s, r * p.dim + c);
    }
  };
  stats(k0);
#pragma unroll 2
  for (long long r = k0; r < p.rows; r += K, ++it) {   // two rows a turn: what a row leaves to the next stays where it is
    BwdRow<IO, GATE, FULL> row;
    row.ru = ru, row.rx = rx;
    stats(r + K);
    ok &= mbar_wait_quiet(&bar[2 + b], phase);   // on a timeout carry on to the end: the peers wait for the sums
    float s[3] = {0.f, 0.f, 0.f};
    if (in) {
      const char *buf = bn_ring + b * buffer + (size_t)tid * VB;
      Raw<IO> u, z, res, dn, dout;
      u.loads(buf);
      z.loads(buf + stride);
      res.loads(buf + 2 * stride);
      dn.loads(buf + 3 * stride);
      dout.loads(buf + 4 * stride);
      row.first(p, col, u, z, res, dn, dout, s);
    }
    if (it > 0) finish(r - K, b == 0 ? p.stages - 1 : b - 1, it - 1);
    if (tid == 0) mbar_expect_tx(&bar[it & 1], sent);
    send_sums(s, red[it & 1], &bar[it & 1], rank, ranks);
    prev = row;
    __syncthreads();   // the previous row's buffer is free
    if (tid == 0 && ahead < p.rows) {
      fence_proxy_async();
      issue(ahead, fill);
      ahead += K;
    }
    if (++fill == p.stages) fill = 0;
    if (++b == p.stages) b = 0, phase ^= 1;
  }
  if (it > 0) finish(k0 + (long long)(it - 1) * K, b == 0 ? p.stages - 1 : b - 1, it - 1);
  if (!ok) report(p.status, ERR_TIMEOUT);
  // no CTA leaves while sums are on their way to it, not even after a timeout
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
  if (in)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      *reinterpret_cast<float2 *>(&p.partial[(size_t)k0 * 2 * p.dim + c + 2 * e]) = of2(col.A[e]);
      *reinterpret_cast<float2 *>(&p.partial[((size_t)k0 * 2 + 1) * p.dim + c + 2 * e]) = of2(col.P[e]);
    }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// Column sums of the partials in a fixed order: 32 columns x 32 row groups per CTA, then the groups. Launched under the
// backward kernel's end.
__global__ void __launch_bounds__(1024) block_norm_dw_kernel(BlockNormParams p, int parts) {
  __shared__ float2 sums[32][33];
  const int x = threadIdx.x & 31, c = blockIdx.x * 32 + x, g = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  float2 v = make_float2(0.f, 0.f);
  if (c < p.dim)
#pragma unroll 4
    for (int k = g; k < parts; k += 32) {
      v.x += __ldcg(&p.partial[((size_t)k * 2) * p.dim + c]);
      v.y += __ldcg(&p.partial[((size_t)k * 2 + 1) * p.dim + c]);
    }
  sums[g][x] = v;
  __syncthreads();
  // warp g adds the groups of column g
  v = sums[x][g];
  v.x = row_sum<32>(v.x), v.y = row_sum<32>(v.y);
  const int col = blockIdx.x * 32 + g;
  if (x == 0 && col < p.dim) {
    if (p.dw_post) p.dw_post[col] = v.x * (p.scale ? p.scale[col] : 1.f);
    if (p.dscale) p.dscale[col] = v.x * (p.w_post ? p.w_post[col] : 1.f);
    if (p.dw_pre) p.dw_pre[col] = v.y;
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
template <typename IO, int GATE>
Kernel fwd_fn(Shape s) {
  switch (s.lpr) {
    case 1: return block_norm_fwd_kernel<IO, GATE, 1, 1>;
    case 2: return block_norm_fwd_kernel<IO, GATE, 2, 1>;
    case 4: return block_norm_fwd_kernel<IO, GATE, 4, 1>;
    case 8: return block_norm_fwd_kernel<IO, GATE, 8, 1>;
    case 16: return block_norm_fwd_kernel<IO, GATE, 16, 1>;
    case 32:
      if constexpr (sizeof(IO) == 2)
        if (s.vpt > 1) return s.vpt == 4 ? block_norm_fwd_kernel<IO, GATE, 32, 4> : block_norm_fwd_kernel<IO, GATE, 32, 2>;
      return block_norm_fwd_kernel<IO, GATE, 32, 1>;
  }
  return s.vpt == 1 ? block_norm_fwd_kernel<IO, GATE, 0, 1> : s.vpt == 2 ? block_norm_fwd_kernel<IO, GATE, 0, 2> : block_norm_fwd_kernel<IO, GATE, 0, 4>;
}
template <typename IO, int GATE>
Kernel bwd_fn(int lpr, bool full) {
  switch (lpr) {
    case 1: return block_norm_bwd_short_kernel<IO, GATE, 1>;
    case 2: return block_norm_bwd_short_kernel<IO, GATE, 2>;
    case 4: return block_norm_bwd_short_kernel<IO, GATE, 4>;
    case 8: return block_norm_bwd_short_kernel<IO, GATE, 8>;
    case 16: return block_norm_bwd_short_kernel<IO, GATE, 16>;
    case 32: return block_norm_bwd_short_kernel<IO, GATE, 32>;
  }
  return full ? block_norm_bwd_kernel<IO, GATE, true> : block_norm_bwd_kernel<IO, GATE, false>;
}
int gate_kind(const BlockNormParams &p) { return p.gate ? (p.silu ? GATE_SILU : GATE_SIGMOID) : GATE_NONE; }
Kernel fwd_fn(Shape s, int gate, bool f32) {
  if (f32) return gate == GATE_NONE ? fwd_fn<float, GATE_NONE>(s) : gate == GATE_SILU ? fwd_fn<float, GATE_SILU>(s) : fwd_fn<float, GATE_SIGMOID>(s);
  return gate == GATE_NONE ? fwd_fn<bf16, GATE_NONE>(s) : gate == GATE_SILU ? fwd_fn<bf16, GATE_SILU>(s) : fwd_fn<bf16, GATE_SIGMOID>(s);
}
// full: long rows with a residual and both gradients, compiled without the other cases (16384 x 7168: 0.401 -> 0.371 ms, with two rows a turn).
Kernel bwd_fn(int lpr, int gate, bool full, bool f32) {
  if (f32)
    return gate == GATE_NONE ? bwd_fn<float, GATE_NONE>(lpr, full) : gate == GATE_SILU ? bwd_fn<float, GATE_SILU>(lpr, full) : bwd_fn<float, GATE_SIGMOID>(lpr, full);
  return gate == GATE_NONE ? bwd_fn<bf16, GATE_NONE>(lpr, full) : gate == GATE_SILU ? bwd_fn<bf16, GATE_SILU>(lpr, full) : bwd_fn<bf16, GATE_SIGMOID>(lpr, full);
}

// The backward's launch. Long rows: as few CTAs per row (of 1 to 8) as keep nearly the most columns on an SM that any count does
// (bf16: 5120 columns in 4 of 160 threads 5.2 TB/s, in 4 that fill two thirds of an SM 4.1; 6144 in 3 of 256 5.2, in 4 of 192
// 4.9; 7168 in 4 of 224 5.0, in 7 of 128, a seventh more, 4.9). In fp32 a CTA takes up to 128 threads, whose rows leave room for others
// (2048 columns in 3 of 96, which the rule takes, 6.2 TB/s, in 2 of 128 6.3, in one of 256 5.9). Three to six buffers, as many as leave
// room for the SM's CTAs; all but the current row's are full or being filled (with one more left empty fp32 rows of 1544
// columns 5.1 instead of 6.2 TB/s, of 8192 4.6 and 6.5; bf16, with five or six buffers, the same). The
// count of CTAs sizes the workspace, so it goes by the sizes alone: the gate's kernels are taken to hold as many at once as the SiLU's.
constexpr int BWD_RING = 216 * 1024;   // the rings of an SM's CTAs together
struct BwdLaunch {
  int lpr, threads, cluster, stages, ctas;   // ctas: rows of partials
  size_t smem;
};
BwdLaunch bwd_launch(long long rows, int dim, bool f32) {
  // The occupancy queries cost more than a small launch; a host thread keeps its last answers.
  struct Known {
    int dev, dim, at_once;
    bool f32;
  };
  static thread_local Known known[8];
  static thread_local unsigned next = 0;
  const Shape s = shape(dim);
  BwdLaunch l{};
  int dev = 0, sms = 0, at_once = 0;
  cudaError_t e = cudaGetDevice(&dev);
  for (const Known &k : known)
    if (e == cudaSuccess && k.at_once > 0 && k.dev == dev && k.dim == dim && k.f32 == f32) at_once = k.at_once;
  const bool ask = at_once == 0;
  if (ask && e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const Kernel fn = bwd_fn(s.lpr, GATE_SILU, true, f32);
  long long groups;
  if (s.lpr) {
    const int rpc = s.threads / s.lpr;
    l = {s.lpr, s.threads, 1, 0, 0, (size_t)2 * rpc * dim * sizeof(float)};
    if (ask && e == cudaSuccess) {
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&at_once, fn, l.threads, l.smem);
      at_once *= sms;
    }
    groups = (rows + rpc - 1) / rpc;
  } else {
    const int nvec = dim / 8;
    const int most = f32 && nvec <= 1024 ? 128 : 256;
    struct Cut {
      int per, threads, ctas;   // vectors and threads of a CTA, CTAs on an SM by registers (128 a thread) and a ring of three rows
    };
    auto cut = [&](int cl) -> Cut {
      const int per = (nvec + cl - 1) / cl, threads = (per + 31) / 32 * 32, row = 5 * per * 8 * (f32 ? 4 : 2);
      if (per > most || (cl - 1) * per >= nvec || (cl > 1 && per < 64)) return {0, 0, 0};   // one or two warps: 1544 in bf16 3.9 TB/s, in one CTA 4.7
      const int ctas = 512 / threads < BWD_RING / (3 * row) ? 512 / threads : BWD_RING / (3 * row);
      return {per, threads, ctas};
    };
    int best = 0, cl = 1;
    for (int k = 1; k <= 8; ++k) best = cut(k).ctas * cut(k).per > best ? cut(k).ctas * cut(k).per : best;
    while (cut(cl).ctas * cut(cl).per < 0.87 * best) ++cl;
    const Cut c = cut(cl);
    const int row = 5 * c.per * 8 * (f32 ? 4 : 2), fit = BWD_RING / c.ctas / row, stages = fit > 6 ? 6 : fit;
    l = {0, c.threads, cl, stages, 0, (size_t)stages * row};
    for (int k = 0; ask && k < 6 && e == cudaSuccess; ++k)
      e = cudaFuncSetAttribute(bwd_fn(0, k / 2, k % 2, f32), cudaFuncAttributeMaxDynamicSharedMemorySize, BWD_RING);   // not l.smem: other sizes use the same kernels
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cl;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)cl);
    cfg.blockDim = dim3((unsigned)l.threads);
    cfg.dynamicSmemBytes = l.smem;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (ask && e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&at_once, fn, &cfg);
    groups = rows;
  }
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    at_once = 152;
  } else if (ask && at_once > 0) {
    known[next++ % 8] = {dev, dim, at_once, f32};
  }
  if (at_once < 1) at_once = 1;
  l.ctas = (int)(groups < 1 ? 1 : (groups < at_once ? groups : at_once));
  return l;
}
}  // namespace

int block_norm_bwd_ctas(long long rows, int dim, bool f32) { return bwd_launch(rows, dim, f32).ctas; }

cudaError_t launch_block_norm_fwd(const BlockNormParams &p, bool f32, cudaStream_t st) {
  if (p.rows == 0) return cudaSuccess;
  Shape s = shape(p.dim);
  // bf16 rows of up to 128 vectors stay with a warp, without a barrier for their sums: 264 columns 3.2 -> 5.2 TB/s, 512 6.1 -> 6.5, 640 5.3 ->
  // 6.0, 1024 6.5 -> 6.4 and without residual and second norm 5.6 -> 6.2. In fp32 a CTA per row is as fast or faster (320 columns 7.0, 6.6).
  if (!s.lpr && !f32 && p.dim <= 1024) s = {32, p.dim <= 512 ? 2 : 4, 256};
  const int rpc = s.lpr ? s.threads / s.lpr : 1;
  const Kernel fn = fwd_fn(s, gate_kind(p), f32);
  // about a quarter to a third of the CTAs that the device holds at once (twice as far costs up to 2% in bf16, 15% at 16384 columns of
  // fp32, four times as far more; without it 0.434 instead of 0.394 ms at 32768 x 7168 before the third CTA)
  BlockNormParams q = p;
  int dev = 0, sms = 0;
  if (!s.lpr && cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    q.prefetch_dist = sms * (512 / s.threads);
  fn<<<(unsigned)((p.rows + rpc - 1) / rpc), s.threads, 0, st>>>(q);
  return cudaGetLastError();
}

cudaError_t launch_block_norm_bwd(const BlockNormParams &p, bool f32, cudaStream_t st) {
  const BwdLaunch l = bwd_launch(p.rows, p.dim, f32);
  BlockNormParams q = p;
  q.stages = l.stages;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)l.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(l.ctas * l.cluster));
  cfg.blockDim = dim3((unsigned)l.threads);
  cfg.dynamicSmemBytes = l.smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, bwd_fn(l.lpr, gate_kind(p), p.residual && p.d_out && p.d_normed, f32), q);   // no rows: the partials become zero
  if (e != cudaSuccess) return e;
  if (!p.dw_post && !p.dscale && !p.dw_pre) return cudaSuccess;
  return launch_under(block_norm_dw_kernel, dim3((unsigned)((p.dim + 31) / 32)), 1024, 0, st, p, l.ctas);
}

}  // namespace kda
