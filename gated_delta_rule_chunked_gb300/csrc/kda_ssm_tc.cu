// kda_ssm_tc.cu -- selective state space scan of bf16 prompts on the 5th-generation tensor cores.
//
// Chunks of 128 tokens. With c_i = sum_{k <= i} h_k a log2(e) over the chunk, S the state entering it:
//   G  = C B^T                                              [128 x 128]
//   M  = G o 2^(c_i - c_j) h_j  (j <= i, else 0)
//   Y  = M X + diag(2^c_i) C S + d X
//   S' = 2^c_last S + B^T (w o X),   w_j = 2^(sum_{k > j} h_k a log2 e) h_j
// One CTA owns 64 value columns of one (sequence, head) and walks its chunks; the state stays in the
// registers of one warpgroup (thread = state channel), so the chain between chunks is one multiply-add
// per element. Roles (15 warps):
//   warps 0-3   M from G (TMEM) into TMEM as the A operand of M X; Y to memory (thread = token)
//   warps 4-7   w o X as three bf16 terms, exact to 24 bits (thread = token)
//   warps 8-11  the state: S' and its bf16 operand tile (thread = state channel)
//   warp 12     the TMA loads and the chunk's scalars (softplus, the sums of h a from both ends, so
//               that w does not come from a difference of large sums)
//   warp 13     issues G, C S and M X;  warp 14 issues B^T (w o X)
// Rounding: the products take bf16 operands and add in fp32. X, B, C are bf16 already; M and the
// operand copy of S are rounded once, which leaves y about as far off as its own rounding; the
// state's update is exact to fp32, because the state is carried on and returned in fp32.
// TMEM (512 columns): G 128, M 64 (packed bf16), M X 64, C S 64, the three terms' products 192.
// Long sequences with too few (sequence, head) pairs to fill the GPU are cut into segments: a first
// launch finds every segment's own contribution to the state and its decay (the state products only),
// a second runs the segments from their entering states, which each CTA folds up from those.
// Every wait is bounded; on a timeout the kernel reports KDA_ERR_TIMEOUT, drains and returns.
#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_tc05.cuh"

namespace kda {
namespace {

constexpr int Q = 128;   // tokens per chunk

struct SsmSmem {
  static constexpr int C = 0, B = 32768, X = 65536, STAGE = 81920;   // two 64-column boxes each for C, B
  static constexpr int S = 2 * STAGE;        // state operand [128 n][64 p] bf16, MN-major
  static constexpr int WX = S + 16384;       // three terms [128 tok][64 p] bf16, MN-major
  static constexpr int SC = WX + 3 * 16384;  // fp32 c, h, w of the chunk's tokens
  static constexpr int BAR = SC + 3 * Q * 4;
  static constexpr int TSLOT = BAR + 24 * 8;
  static constexpr int BYTES = TSLOT + 16;
};
static_assert(SsmSmem::BYTES <= 232448, "shared memory of one SM");

// TMEM columns
constexpr uint32_t T_G = 0, T_M = 128, T_Y1 = 192, T_Y2 = 256, T_DS = 320;

enum Bar {
  FULL0, FULL1,      // a stage's boxes landed
  EMPTY0, EMPTY1,    // a stage is consumed: both issuers' commits, and the 256 threads that read X rows
  SFULL, SEMPTY,     // the chunk's scalars written / read by all three warpgroups
  GDONE, GFREE,      // G complete / read out
  MREADY,            // M stored
  YDONE, YFREE,      // both Y products complete / read out
  WXREADY,           // w o X stored (and a short chunk's rows past its end cleared)
  DSDONE, DSFREE,    // the state products complete / read out
  SREADY,            // the state operand stored; phase 0: the initial state
  DRAIN0, DRAIN1,
  NBAR
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem] over one K = 16 step: A's row m is lane m, two bf16 per column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}
// Byte offset of 16-byte chunk k of row r in a [rows][64] bf16 tile with the 128-byte swizzle.
__device__ __forceinline__ uint32_t row_chunk(int r, int k) { return (uint32_t)(r * 128 + ((k ^ (r & 7)) << 4)); }

// STATES: the segments' own state contributions and decays only.
template <bool STATES>
__global__ void __launch_bounds__(480, 1) ssm_tc_kernel(const __grid_constant__ SsmTcParams p) {
  using L = SsmSmem;
  extern __shared__ __align__(1024) char smem[];
  if (smem_u32(smem) & 1023u) {   // the operand tiles' swizzle needs it; not seen
    if (threadIdx.x == 0) report(p.s.status, 3 /* KDA_ERR_CUDA */);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = tid & 127, wg = warp >> 2;
  const int U = p.s.H * (p.s.P / SSM_COLS), nseg = p.nseg, runs = STATES ? nseg - 1 : nseg;
  const int u = blockIdx.x % U, ns = blockIdx.x / U, seg = ns % runs, n = ns / runs;
  const int head = u / (p.s.P / SSM_COLS), col0 = (u % (p.s.P / SSM_COLS)) * SSM_COLS, group = head / (p.s.H / p.s.G);
  const long long seq0 = p.s.cu ? p.s.cu[n] : p.s.T / p.s.n_seqs * n, seq1 = p.s.cu ? p.s.cu[n + 1] : p.s.T / p.s.n_seqs * (n + 1);
  const int all = (int)((seq1 - seq0 + Q - 1) / Q);
  const int first = (int)((long long)all * seg / nseg), nch = (int)((long long)all * (seg + 1) / nseg) - first;
  const long long t_begin = seq0 + (long long)first * Q;
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + L::BAR);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + L::TSLOT);
  float *sc_c = reinterpret_cast<float *>(smem + L::SC), *sc_h = sc_c + Q, *sc_w = sc_h + Q;

  if (tid == 0) {
    const int readers = STATES ? 128 : 256;
    for (int i = 0; i < NBAR; ++i) {
      int count = 128;
      if (i == FULL0 || i == FULL1 || i == GDONE || i == YDONE || i == DSDONE || i == DRAIN0 || i == DRAIN1) count = 1;
      if (i == EMPTY0 || i == EMPTY1) count = readers + (STATES ? 1 : 2);
      if (i == SFULL) count = 32;
      if (i == SEMPTY) count = STATES ? 256 : 384;
      mbar_init(&bar[i], count);
    }
    fence_mbar_init();
  }
  if (warp == 13) tc::alloc(tslot, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tslot, tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  auto len_of = [&](int c) -> int {
    const long long left = seq1 - (t_begin + (long long)c * Q);
    return left < Q ? (int)left : Q;
  };
  bool ok = true;
  int c = 0;

  if (wg == 0) {
    if constexpr (!STATES) {
      // ------------------------------------------------------------ M and Y
      {
        const uint32_t z[16] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k) st16u(tl + T_M + 16 * k, z);   // blocks above the diagonal stay zero
        tc::wait_st();
      }
      const float d = p.s.d_skip ? p.s.d_skip[head] : 0.f;
      bf16 *y = static_cast<bf16 *>(p.s.y) + (long long)head * p.s.P + col0;
      const bool wide = (reinterpret_cast<uintptr_t>(p.s.y) & 31) == 0;
      uint4 xr[8];   // the token's X row, held until its Y is there (the stage is released earlier)
      float ei = 0.f;
      auto store_y = [&](int k) {   // chunk k's outputs, products complete
        const bool live = row < len_of(k);
        bf16 *dst = y + (t_begin + (long long)k * Q + row) * (long long)p.s.H * p.s.P;
        const uint32_t *xw = reinterpret_cast<const uint32_t *>(xr);
        uint32_t o[32];
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
          uint32_t a[32], b[32];
          ld32(tl + T_Y1 + 32 * hb, a);
          ld32(tl + T_Y2 + 32 * hb, b);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t xx = xw[16 * hb + i];
            const float v0 = fmaf(d, __uint_as_float(xx << 16), fmaf(ei, __uint_as_float(b[2 * i]), __uint_as_float(a[2 * i])));
            const float v1 = fmaf(d, __uint_as_float(xx & 0xffff0000u), fmaf(ei, __uint_as_float(b[2 * i + 1]), __uint_as_float(a[2 * i + 1])));
            o[16 * hb + i] = pack2(v0, v1);
          }
        }
        tc::fence_before();
        mbar_arrive(&bar[YFREE]);
        if (live) {
          if (wide) {
#pragma unroll
            for (int k8 = 0; k8 < 4; ++k8)
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(dst + 16 * k8), "r"(o[8 * k8]), "r"(o[8 * k8 + 1]),
                           "r"(o[8 * k8 + 2]), "r"(o[8 * k8 + 3]), "r"(o[8 * k8 + 4]), "r"(o[8 * k8 + 5]), "r"(o[8 * k8 + 6]), "r"(o[8 * k8 + 7])
                           : "memory");
          } else {
#pragma unroll
            for (int k4 = 0; k4 < 8; ++k4)
              *reinterpret_cast<uint4 *>(dst + 8 * k4) = make_uint4(o[4 * k4], o[4 * k4 + 1], o[4 * k4 + 2], o[4 * k4 + 3]);
          }
        }
      };
      for (c = 0; c < nch; ++c) {
        const char *st = smem + (c & 1) * L::STAGE;
        ok = mbar_wait(&bar[SFULL], c & 1) && mbar_wait(&bar[GDONE], c & 1);   // G's commit covers the previous Y products
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc::fence_after();
        const float ci = sc_c[row];
        // M: row i, 32 columns at a time, up to the warp's diagonal block
#pragma unroll
        for (int jb = 0; jb < 4; ++jb)
          if (jb <= warp) {
            uint32_t g[32], m[16];
            ld32(tl + T_G + 32 * jb, g);
            tc::wait_ld();
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 cj = *reinterpret_cast<const float4 *>(sc_c + 32 * jb + j), hj = *reinterpret_cast<const float4 *>(sc_h + 32 * jb + j);
              float v[4] = {__uint_as_float(g[j]) * (ex2(ci - cj.x) * hj.x), __uint_as_float(g[j + 1]) * (ex2(ci - cj.y) * hj.y),
                            __uint_as_float(g[j + 2]) * (ex2(ci - cj.z) * hj.z), __uint_as_float(g[j + 3]) * (ex2(ci - cj.w) * hj.w)};
              if (jb == warp)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = j + e <= lane ? v[e] : 0.f;
              m[j / 2] = pack2(v[0], v[1]);
              m[j / 2 + 1] = pack2(v[2], v[3]);
            }
            st16u(tl + T_M + 16 * jb, m);
          }
        tc::wait_st();
        tc::fence_before();
        mbar_arrive(&bar[GFREE]);
        mbar_arrive(&bar[MREADY]);
        if (c > 0) store_y(c - 1);   // its products were complete with G
        ei = exp2f(ci);
        ok = mbar_wait(&bar[FULL0 + (c & 1)], (c >> 1) & 1);   // complete: G read it
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
#pragma unroll
        for (int k = 0; k < 8; ++k) xr[k] = *reinterpret_cast<const uint4 *>(st + L::X + row_chunk(row, k));
        mbar_arrive(&bar[EMPTY0 + (c & 1)]);
        mbar_arrive(&bar[SEMPTY]);
      }
      if (ok && nch > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bar[YDONE], (nch - 1) & 1));
        tc::fence_after();
        if (ok) store_y(nch - 1);
      }
    }
  } else if (wg == 1) {
    // -------------------------------------------------------------- w o X
    for (c = 0; c < nch; ++c) {
      char *st = smem + (c & 1) * L::STAGE;
      ok = ok && mbar_wait(&bar[SFULL], c & 1) && mbar_wait(&bar[FULL0 + (c & 1)], (c >> 1) & 1);
      if (!ok) break;
      const float w = sc_w[row];
      const bool live = row < len_of(c);
      uint4 o[3][8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint4 v = *reinterpret_cast<const uint4 *>(st + L::X + row_chunk(row, k));
        const uint32_t xw[4] = {v.x, v.y, v.z, v.w};
        uint32_t *o0 = reinterpret_cast<uint32_t *>(&o[0][k]), *o1 = reinterpret_cast<uint32_t *>(&o[1][k]), *o2 = reinterpret_cast<uint32_t *>(&o[2][k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // 24 bits in three truncated terms of 8: the remainders are exact
          const float a = w * __uint_as_float(xw[e] << 16), b = w * __uint_as_float(xw[e] & 0xffff0000u);
          const float a0 = __uint_as_float(__float_as_uint(a) & 0xffff0000u), b0 = __uint_as_float(__float_as_uint(b) & 0xffff0000u);
          const float ar = a - a0, br = b - b0;
          const float a1 = __uint_as_float(__float_as_uint(ar) & 0xffff0000u), b1 = __uint_as_float(__float_as_uint(br) & 0xffff0000u);
          const float a2 = ar - a1, b2 = br - b1;
          o0[e] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
          o1[e] = __byte_perm(__float_as_uint(ar), __float_as_uint(br), 0x7632);
          o2[e] = __byte_perm(__float_as_uint(a2), __float_as_uint(b2), 0x7632);
        }
      }
      if (!live) {   // rows past the sequence's end belong to another one, or to nobody: whatever they hold stays out
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          o[0][k] = o[1][k] = o[2][k] = z;
          *reinterpret_cast<uint4 *>(st + L::X + row_chunk(row, k)) = z;
          *reinterpret_cast<uint4 *>(st + L::B + row_chunk(row, k)) = z;
          *reinterpret_cast<uint4 *>(st + L::B + 16384 + row_chunk(row, k)) = z;
        }
      }
      if (c > 0) ok = mbar_wait(&bar[DSDONE], (c - 1) & 1);   // the tile's previous terms are read
      if (!ok) break;
#pragma unroll
      for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4 *>(smem + L::WX + 16384 * t + row_chunk(row, k)) = o[t][k];
      fence_proxy_async();
      mbar_arrive(&bar[WXREADY]);
      mbar_arrive(&bar[EMPTY0 + (c & 1)]);
      mbar_arrive(&bar[SEMPTY]);
    }
  } else if (wg == 2) {
    // -------------------------------------------------------------- the state: row n of [128][64]
    float S[64];
    const size_t plane = (size_t)SSM_N * SSM_COLS;
    const size_t soff = (((size_t)n * p.s.H + head) * SSM_N + row) * p.s.P + col0;
    if (!STATES && p.s.h0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 v = *reinterpret_cast<const float4 *>(p.s.h0 + soff + 4 * i);
        S[4 * i] = v.x, S[4 * i + 1] = v.y, S[4 * i + 2] = v.z, S[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i) S[i] = 0.f;
    }
    if (!STATES)
      for (int k = 0; k < seg; ++k) {   // the segments before this one
        const size_t at = ((size_t)n * (nseg - 1) + k) * U + u;
        const float dec = p.seg_decay[at];
        const float *e = p.seg_state + at * plane + (size_t)row * SSM_COLS;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float4 v = __ldcg(reinterpret_cast<const float4 *>(e + 4 * i));
          S[4 * i] = fmaf(S[4 * i], dec, v.x);
          S[4 * i + 1] = fmaf(S[4 * i + 1], dec, v.y);
          S[4 * i + 2] = fmaf(S[4 * i + 2], dec, v.z);
          S[4 * i + 3] = fmaf(S[4 * i + 3], dec, v.w);
        }
      }
    auto put = [&]() {   // the operand tile
#pragma unroll
      for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4 *>(smem + L::S + row_chunk(row, k)) = tc::pack8(S + 8 * k);
      fence_proxy_async();
      mbar_arrive(&bar[SREADY]);
    };
    if (!STATES) put();
    float log_dec = 0.f;
    for (c = 0; c < nch; ++c) {
      ok = mbar_wait(&bar[SFULL], c & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const float last = sc_c[Q - 1];
      mbar_arrive(&bar[SEMPTY]);
      const float dec = exp2f(last);
      log_dec += last;
      ok = mbar_wait(&bar[DSDONE], c & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc::fence_after();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float d0[16], d1[16], d2[16];
        tc::ld16(tl + T_DS + 16 * k, d0);
        tc::ld16(tl + T_DS + 64 + 16 * k, d1);
        tc::ld16(tl + T_DS + 128 + 16 * k, d2);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) S[16 * k + i] = fmaf(S[16 * k + i], dec, d0[i] + (d1[i] + d2[i]));
      }
      tc::fence_before();
      mbar_arrive(&bar[DSFREE]);
      if (!STATES && c + 1 < nch) {
        ok = mbar_wait(&bar[YDONE], c & 1);   // C S has read the previous operand
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        put();
      }
    }
    if (ok) {
      float *dst = nullptr;
      if (STATES) {
        const size_t at = ((size_t)n * (nseg - 1) + seg) * U + u;
        dst = p.seg_state + at * plane + (size_t)row * SSM_COLS;
        if (row == 0) p.seg_decay[at] = exp2f(log_dec);
      } else if (p.s.hT && seg == nseg - 1) {
        dst = p.s.hT + soff;
      }
      if (dst)
#pragma unroll
        for (int i = 0; i < 16; ++i) *reinterpret_cast<float4 *>(dst + 4 * i) = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
    }
  } else if (warp == 12) {
    // -------------------------------------------------------------- loads and scalars
    auto issue = [&](int k) {   // lane 0
      char *st = smem + (k & 1) * L::STAGE;
      uint64_t *b = &bar[FULL0 + (k & 1)];
      const int t = (int)(t_begin + (long long)k * Q);
      mbar_expect_tx(b, STATES ? 49152 : 81920);
      if (!STATES) {
        tc::tma_load_2d(st + L::C, &p.tm_c, group * SSM_N, t, b);
        tc::tma_load_2d(st + L::C + 16384, &p.tm_c, group * SSM_N + 64, t, b);
      }
      tc::tma_load_2d(st + L::B, &p.tm_b, group * SSM_N, t, b);
      tc::tma_load_2d(st + L::B + 16384, &p.tm_b, group * SSM_N + 64, t, b);
      tc::tma_load_2d(st + L::X, &p.tm_x, head * p.s.P + col0, t, b);
    };
    const float al = p.s.a[head] * LOG2E, bias = p.s.dt_bias ? p.s.dt_bias[head] : 0.f;
    auto fetch = [&](int k, float (&v)[4]) {
      const int len = len_of(k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * lane + i;
        v[i] = t < len ? p.s.dt[(t_begin + (long long)k * Q + t) * p.s.H + head] : 0.f;
      }
    };
    int issued = 0;
    float v[4];
    if (nch > 0) fetch(0, v);
    if (lane == 0)
      while (issued < nch && issued < 2) issue(issued++);
    issued = nch < 2 ? nch : 2;
    for (c = 0; c < nch; ++c) {
      if (c > 0) ok = mbar_wait(&bar[SEMPTY], (c - 1) & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const int len = len_of(c);
      float h[4], la[4], pre[4], suf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float b = v[i] + bias;
        h[i] = p.s.softplus ? log1pf(expf(-fabsf(b))) + fmaxf(b, 0.f) : b;
        if (4 * lane + i >= len) h[i] = 0.f;
        la[i] = h[i] * al;
      }
      if (c + 1 < nch) fetch(c + 1, v);
      pre[0] = la[0];
#pragma unroll
      for (int i = 1; i < 4; ++i) pre[i] = pre[i - 1] + la[i];
      suf[3] = 0.f;
#pragma unroll
      for (int i = 2; i >= 0; --i) suf[i] = suf[i + 1] + la[i + 1];
      float below = pre[3], above = suf[0] + la[0];   // the lane's total, added up from either end
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const float x = __shfl_up_sync(0xffffffffu, below, o), z = __shfl_down_sync(0xffffffffu, above, o);
        if (lane >= o) below += x;
        if (lane + o < 32) above += z;
      }
      const float left = __shfl_up_sync(0xffffffffu, below, 1), right = __shfl_down_sync(0xffffffffu, above, 1);
      const float bl = lane > 0 ? left : 0.f, ab = lane < 31 ? right : 0.f;
      *reinterpret_cast<float4 *>(sc_c + 4 * lane) = make_float4(bl + pre[0], bl + pre[1], bl + pre[2], bl + pre[3]);
      *reinterpret_cast<float4 *>(sc_h + 4 * lane) = make_float4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<float4 *>(sc_w + 4 * lane) =
          make_float4(h[0] * exp2f(suf[0] + ab), h[1] * exp2f(suf[1] + ab), h[2] * exp2f(suf[2] + ab), h[3] * exp2f(suf[3] + ab));
      mbar_arrive(&bar[SFULL]);
      if (c > 0 && c + 1 < nch) {   // the previous chunk's stage is the next chunk's
        if (lane == 0) {
          ok = mbar_wait(&bar[EMPTY0 + ((c + 1) & 1)], ((c - 1) >> 1) & 1);
          if (ok) issue(c + 1);
        }
        if (!(ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0)) break;
        issued = c + 2;
      }
    }
    // every copy has landed before the CTA leaves, also after a timeout
    if (lane == 0)
      for (int k = issued > 2 ? issued - 2 : 0; k < issued; ++k) mbar_wait(&bar[FULL0 + (k & 1)], (k >> 1) & 1);
    __syncwarp();
  } else if (warp == 13) {
    if (lane == 0) {
      if constexpr (!STATES) {
        // ---------------------------------------------------------- G, C S, M X
        const uint64_t d_s = tc::desc_sw128_mn(smem_u32(smem + L::S), 8192);
        for (c = 0; c < nch; ++c) {
          const uint32_t st = smem_u32(smem + (c & 1) * L::STAGE);
          ok = mbar_wait(&bar[FULL0 + (c & 1)], (c >> 1) & 1);
          if (ok && c > 0) ok = mbar_wait(&bar[GFREE], (c - 1) & 1);
          if (ok && len_of(c) < Q) {   // rows past the end must be cleared; the barrier's previous phase first, so that parities tell
            if (c > 0) ok = mbar_wait(&bar[WXREADY], (c - 1) & 1);
            ok = ok && mbar_wait(&bar[WXREADY], c & 1);
          }
          if (!ok) break;
          tc::fence_after();
          const uint64_t d_c = tc::desc_sw128(st + L::C), d_b = tc::desc_sw128(st + L::B), d_x = tc::desc_sw128_mn(st + L::X, 8192);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint32_t o = (ks >> 2) * (16384 >> 4) + (ks & 3) * 2;
            tc::mma_bf16(tmem + T_G, d_c + o, d_b + o, tc::idesc_bf16(128, 128), ks > 0);
          }
          tc::commit(&bar[GDONE]);
          ok = mbar_wait(&bar[SREADY], c & 1);
          if (ok && c > 0) ok = mbar_wait(&bar[YFREE], (c - 1) & 1);
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint32_t o = (ks >> 2) * (16384 >> 4) + (ks & 3) * 2;
            tc::mma_bf16(tmem + T_Y2, d_c + o, d_s + ks * (2048 >> 4), tc::idesc_bf16_mn(128, 64, false, true), ks > 0);
          }
          ok = mbar_wait(&bar[MREADY], c & 1);
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ts(tmem + T_Y1, tmem + T_M + 8 * ks, d_x + ks * (2048 >> 4), tc::idesc_bf16_mn(128, 64, false, true), ks > 0);
          tc::commit(&bar[YDONE]);
          tc::commit(&bar[EMPTY0 + (c & 1)]);
        }
        tc::commit(&bar[DRAIN0]);   // nothing of this thread runs on once the CTA leaves
        ok &= mbar_wait(&bar[DRAIN0], 0);
      }
    }
    __syncwarp();
  } else {
    if (lane == 0) {
      // ------------------------------------------------------------ B^T (w o X)
      const uint64_t d_w = tc::desc_sw128_mn(smem_u32(smem + L::WX), 16384);
      for (c = 0; c < nch; ++c) {
        ok = mbar_wait(&bar[WXREADY], c & 1);
        if (ok && c > 0) ok = mbar_wait(&bar[DSFREE], (c - 1) & 1);
        if (!ok) break;
        tc::fence_after();
        const uint64_t d_b = tc::desc_sw128_mn(smem_u32(smem + (c & 1) * L::STAGE + L::B), 16384);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc::mma_bf16(tmem + T_DS, d_b + ks * (2048 >> 4), d_w + ks * (2048 >> 4), tc::idesc_bf16_mn(128, 192, true, true), ks > 0);
        tc::commit(&bar[DSDONE]);
        tc::commit(&bar[EMPTY0 + (c & 1)]);
      }
      tc::commit(&bar[DRAIN1]);
      ok &= mbar_wait(&bar[DRAIN1], 0);
    }
    __syncwarp();
  }
  if (!ok) report(p.s.status, ERR_TIMEOUT);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 13) tc::dealloc(tmem, 512);
}

bool map_rows(EncodeTiledFn fn, CUtensorMap *m, const void *base, long long rows, long long width, long long ld) {
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)Q}, estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

// Segments per sequence: the count that takes the fewest chunk times. Without segments every wave of
// CTAs walks whole sequences; with k, a wave walks 1/k of them, at 1.45 times the work (the state
// products run twice) and some fixed cost for the second launch and the folding.
int ssm_segments(int n_seqs, long long T, int units) {
  if (n_seqs < 1 || T < 1) return 1;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    (void)cudaGetLastError();
    sms = 152;
  }
  const double chunks = (double)T / n_seqs / Q, pairs = (double)n_seqs * units;
  int best = 1;
  double cost = chunks * (double)(long long)((pairs + sms - 1) / sms);
  for (int k = 2; k <= 16 && k * 2 <= chunks; ++k) {
    const double t = 1.45 * chunks / k * (double)(long long)((pairs * k + sms - 1) / sms) + 6.0 + 0.5 * k;
    if (t < cost) cost = t, best = k;
  }
  return best;
}

size_t ssm_segment_bytes(int n_seqs, int units, int nseg) {
  if (nseg < 2) return 0;
  const size_t items = (size_t)n_seqs * (nseg - 1) * units;
  return items * SSM_N * SSM_COLS * sizeof(float) + (items * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_ssm_fwd_tc(const SsmParams &s, int nseg, void *workspace, cudaStream_t st) {
  SsmTcParams p{};
  p.s = s;
  p.nseg = nseg;
  const int U = s.H * (s.P / SSM_COLS);
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return cudaErrorNotSupported;
  const long long rows = s.T > 0 ? s.T : 1;
  if (s.T > 0 && (!map_rows(fn, &p.tm_x, s.x, rows, (long long)s.H * s.P, s.ldx) || !map_rows(fn, &p.tm_b, s.b, rows, (long long)s.G * SSM_N, s.ldb) ||
                  !map_rows(fn, &p.tm_c, s.c, rows, (long long)s.G * SSM_N, s.ldc)))
    return cudaErrorInvalidValue;
  if ((size_t)s.n_seqs * nseg * U > 0x7fffffffu) return cudaErrorInvalidConfiguration;
  const size_t items = nseg > 1 ? (size_t)s.n_seqs * (nseg - 1) * U : 0;
  p.seg_state = static_cast<float *>(workspace);
  p.seg_decay = p.seg_state + items * SSM_N * SSM_COLS;
  cudaError_t e = cudaFuncSetAttribute(ssm_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, SsmSmem::BYTES);
  if (e != cudaSuccess) return e;
  if (nseg > 1) {
    e = cudaFuncSetAttribute(ssm_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, SsmSmem::BYTES);
    if (e != cudaSuccess) return e;
    ssm_tc_kernel<true><<<(unsigned)items, 480, SsmSmem::BYTES, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  ssm_tc_kernel<false><<<(unsigned)((size_t)s.n_seqs * nseg * U), 480, SsmSmem::BYTES, st>>>(p);
  return cudaGetLastError();
}

}  // namespace kda
