// kda_ssm_tc.cu -- selective state space scan of bf16 prompts on the 5th-generation tensor cores.
//
// Chunks of 128 tokens. With c_i = sum_{k <= i} h_k a log2(e) over the chunk, S the state entering it:
//   G  = C B^T                                              [128 x 128]
//   M  = G o 2^(c_i - c_j) h_j  (j <= i, else 0)
//   Y  = M X + diag(2^c_i) C S + d X
//   S' = 2^c_last S + B^T (w o X),   w_j = 2^(sum_{k > j} h_k a log2 e) h_j
// One CTA owns 64 value columns of one (sequence, head) at a time and walks its chunks; the state stays in the
// registers of one warpgroup (thread = state channel), so the chain between chunks is one multiply-add
// per element. Roles (28 warps; a role's eight warps are two per 32 rows, each with half of the columns,
// because the work per thread is short chains that one warp per scheduler cannot fill):
//   warps 0-7    M from G (TMEM) into TMEM as the A operand of M X; the previous chunk's Y (thread = token)
//   warps 8-15   w o X as three bf16 terms, exact to 24 bits (thread = token)
//   warps 16-23  the state: S' and its bf16 operand tile (thread = state channel)
//   warp 24      the chunk's scalars (softplus, the sums of h a from both ends, so that w does not
//                come from a difference of large sums)
//   warp 25      issues G, C S and M X;  warp 26 issues B^T (w o X);  warp 27 the TMA loads
// Loops stay rolled: the roles share one instruction cache, and with unrolled bodies every chunk
// fetched its code from beyond it (32768 tokens x 96 heads of 64 in 1.16 instead of 0.92 ms, before the other steps).
// Bound by shared memory: a chunk moves 80 KB in and 16 KB out by TMA, w o X, X, Y and S through registers, and
// the products read 1664 lines of 128 bytes of operands; together 90 to 92% of its cycles, 1.9 us a chunk, with the
// tensor cores 45% and the issue slots 52% busy. 32768 tokens x 96 heads of 64 take 0.486 ms, 2.0 TB/s of inputs and
// outputs, on the 96 SMs that have a head.
// Rounding: the products take bf16 operands and add in fp32. X, B, C are bf16 already; M and the
// operand copy of S are rounded once, which leaves y about as far off as its own rounding; the
// state's update is exact to fp32, because the state is carried on and returned in fp32.
// TMEM (512 columns): G 128, M 64 (packed bf16), M X 64, C S 64, the three terms' products 192.
// Long sequences with too few (sequence, head) pairs to fill the GPU are cut into segments: a first
// launch finds every segment's own contribution to the state and its decay (the state products only),
// a second makes the entering states of those, and a third runs the segments from them.
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
  static constexpr int SC = WX + 3 * 16384;  // fp32 c, h, w, e of the chunk's tokens
  static constexpr int BAR = SC + 4 * Q * 4;
  static constexpr int BARS = 40;            // places for the barriers
  static constexpr int TSLOT = BAR + BARS * 8;
  static constexpr int ORDER = TSLOT + 16;   // the sequences by falling length
  static constexpr int BYTES = ORDER + 256 * 2;
};
static_assert(SsmSmem::BYTES <= 232448, "shared memory of one SM");

// TMEM columns
constexpr uint32_t T_G = 0, T_M = 128, T_Y1 = 192, T_Y2 = 256, T_DS = 320;

enum Bar {
  FULL0, FULL1,      // a stage's B and C landed
  XFULL0, XFULL1,    // its X landed
  EMPTY0, EMPTY1,    // its B and C are read: both issuers' commits
  XEMPTY0, XEMPTY1,  // w o X has read its X
  SFULL, SEMPTY,     // the chunk's scalars written / read by all three warpgroups
  GDONE, GFREE,      // G complete / read out
  MREADY0, MREADY3 = MREADY0 + 3,     // M's columns 32 k .. 32 k + 31 stored (by the warps at and below the diagonal)
  YDONE, YFREE,      // both Y products complete / read out
  YSTAGED0, YSTAGED1,   // a stage's Y in the place of its X
  WXREADY0, WXREADY3 = WXREADY0 + 3,  // w o X of tokens 32 k .. stored
  DSPART0, DSPART3 = DSPART0 + 3,     // the state products have read those tokens
  DSDONE, DSFREE,    // the state products complete / read out
  SREADY,            // the state operand stored; phase 0: the initial state
  TAIL,              // a sequence's short last chunk: the rows past its end are cleared (one phase)
  DRAIN0, DRAIN1,
  NBAR
};
static_assert(NBAR <= SsmSmem::BARS, "a place for every barrier");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// One box from shared memory (128-byte swizzle) to the tensor; joins the thread's bulk group.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, int x, int y, const void *src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void st8u(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// The products are issued by whole warps of which one elected lane acts: the operands then stay in
// uniform registers, where a lone lane's would be moved there one by one for every instruction.
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
// D[tmem] (+)= A[smem] * B[smem] over one K = 16 step.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader));
}
// The same with A in tensor memory: A's row m is lane m, two bf16 per column.
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader));
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_u32(bar)),
      "r"(leader)
      : "memory");
}
// The same box brought into L2 only.
__device__ __forceinline__ void prefetch_2d(const CUtensorMap *map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y) : "memory");
}
// Shared-memory descriptors (SWIZZLE_128B, 1024 bytes between 8-row groups) as their low word: the
// high one is the same for all.
__device__ __forceinline__ uint32_t dlo(uint32_t addr, uint32_t lbo) { return (addr & 0x3FFFF) >> 4 | (lbo >> 4) << 16; }
__device__ __forceinline__ uint64_t desc(uint32_t lo) { return (uint64_t)(64u | 1u << 14 | 2u << 29) << 32 | lo; }
// Byte offset of 16-byte chunk k of row r in a [rows][64] bf16 tile with the 128-byte swizzle.
__device__ __forceinline__ uint32_t row_chunk(int r, int k) { return (uint32_t)(r * 128 + ((k ^ (r & 7)) << 4)); }

// The sequences by falling length, at most MOST_SORTED. The scratch is where a bulk copy lands next.
constexpr int MOST_SORTED = 256;
__device__ __forceinline__ void sort_longest(const int *cu, int n_seqs, int *scratch, uint16_t *order) {
  const int t = threadIdx.x;
  if (t < n_seqs) scratch[t] = cu[t + 1] - cu[t];
  __syncthreads();
  if (t < n_seqs) {
    const int len = scratch[t];
    int rank = 0;
    for (int j = 0; j < n_seqs; ++j) rank += scratch[j] > len || (scratch[j] == len && j < t);
    order[rank] = (uint16_t)t;
  }
  fence_proxy_async();   // the lengths, before that copy
  __syncthreads();
}
// One item of the launch: the token a chunk before its first, its chunks, its unit, and sequence | segment << 16 | the last chunk's tokens << 20.
__device__ __forceinline__ int4 item_of(const SsmTcParams *p, const uint16_t *order, int i) {
  const int U = p->s.H * (p->s.P / SSM_COLS), u = i % U, ns = i / U, seg = ns % p->nseg;
  int n = ns / p->nseg;
  if (p->sorted) n = order[n];
  // token indices fit 32 bits (T < 2^31), and offsets that are no sequence's are taken as an empty one
  const int each = (int)(p->s.T / p->s.n_seqs), seq0 = max(p->s.cu ? p->s.cu[n] : each * n, 0);
  const int seq1 = max(min(p->s.cu ? p->s.cu[n + 1] : each * (n + 1), (int)p->s.T), seq0);
  const int all = (int)(((unsigned)(seq1 - seq0) + Q - 1) / Q), first = (int)((long long)all * seg / p->nseg), last = (int)((long long)all * (seg + 1) / p->nseg);
  return make_int4(seq0 + (first - 1) * Q, last - first, u, n | seg << 16 | min(seq1 - seq0 - (last - 1) * Q, Q) << 20);
}
// Kept out of line: its divisions in every role's loop push the roles' code out of the instruction cache.
__device__ __noinline__ int4 item_at(const SsmTcParams *p, const uint16_t *order, int i) { return item_of(p, order, i); }
// A CTA's way through its items (sequence, segment, unit) and their chunks, the same for every role. Items are dealt out from the longest
// sequence on, forwards and backwards in turn, so that the CTAs end about together.
// Without MANY a CTA has one.
template <bool MANY>
struct Walk {
  int round = 0, left = 0;   // chunks of the item after this one
  int t, u = 0, what;            // the chunk's first token; unit; the rest as item_at gives it
  bool fresh;                // the chunk is an item's first
  __device__ __forceinline__ Walk(const SsmTcParams &p, const uint16_t *order) {
    if (MANY) return;
    const int4 v = item_of(&p, order, (int)blockIdx.x);
    t = v.x, left = v.y, u = v.z, what = v.w;
  }
  __device__ __forceinline__ bool item(const SsmTcParams &p, const uint16_t *order) {   // the next one, which may be empty
    if (!MANY) return ++round == 1;
    const int G = (int)gridDim.x, b = (int)blockIdx.x, i = round * G + (round & 1 ? G - 1 - b : b);   // below 2^31: at most one round past the items
    if ((unsigned)i >= p.items) return false;
    ++round;
    const int4 v = item_at(&p, order, i);
    t = v.x, left = v.y, u = v.z, what = v.w;
    return true;
  }
  __device__ __forceinline__ bool chunk(const SsmTcParams &p, const uint16_t *order) {
    if (!MANY) {
      fresh = round == 0, round = 1;
      if (left == 0) return false;
    } else {
      fresh = left == 0;
      while (left == 0)
        if (!item(p, order)) return false;
    }
    --left;
    t += Q;
    return true;
  }
  __device__ __forceinline__ int len() const { return left == 0 ? what >> 20 : Q; }
  __device__ __forceinline__ int seq() const { return what & 0xffff; }
  __device__ __forceinline__ int seg() const { return what >> 16 & 15; }
  __device__ __forceinline__ int head(const SsmTcParams &p) const { return p.s.P == SSM_COLS ? u : u >> 1; }
  __device__ __forceinline__ int col0(const SsmTcParams &p) const { return p.s.P == SSM_COLS ? 0 : (u & 1) * SSM_COLS; }
};

// w times half of a token's X as three bf16 tiles: 24 bits in truncated terms of 8, so the remainders are exact.
__device__ __forceinline__ void weigh(const char *x, char *wx, int row, int half, float w) {
  const f2 w2 = two(w, w), minus = two(-1.f, -1.f);
#pragma unroll 1
  for (int k = 4 * half; k < 4 * half + 4; ++k) {
    const uint32_t at = row_chunk(row, k);
    const uint4 v = *reinterpret_cast<const uint4 *>(x + at);
    const uint32_t xw[4] = {v.x, v.y, v.z, v.w};
    uint32_t o0[4], o1[4], o2[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f2 v0 = mul2(w2, unpack2(xw[e]));
      const float2 a = of2(v0);
      const f2 v1 = fma2(two(__uint_as_float(__float_as_uint(a.x) & 0xffff0000u), __uint_as_float(__float_as_uint(a.y) & 0xffff0000u)), minus, v0);
      const float2 b = of2(v1);
      const float2 r = of2(fma2(two(__uint_as_float(__float_as_uint(b.x) & 0xffff0000u), __uint_as_float(__float_as_uint(b.y) & 0xffff0000u)), minus, v1));
      o0[e] = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x7632);
      o1[e] = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x7632);
      o2[e] = __byte_perm(__float_as_uint(r.x), __float_as_uint(r.y), 0x7632);
    }
    *reinterpret_cast<uint4 *>(wx + at) = make_uint4(o0[0], o0[1], o0[2], o0[3]);
    *reinterpret_cast<uint4 *>(wx + 16384 + at) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
    *reinterpret_cast<uint4 *>(wx + 32768 + at) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
  }
}
// h of a token, and h a log2(e)
__device__ __forceinline__ float step_of(float v, float bias, int softplus) {
  const float b = v + bias;
  return softplus ? log1pf(expf(-fabsf(b))) + fmaxf(b, 0.f) : b;
}
// 2^-200 is zero in fp32 already: a token that forgets more would only cost the differences of the sums after it their digits
__device__ __forceinline__ float forgets(float h, float al) {
  const float l = h * al;
  return l < -200.f ? -200.f : l;
}

template <bool MANY>
__global__ void __launch_bounds__(896, 1) ssm_tc_kernel(const __grid_constant__ SsmTcParams p) {
  using L = SsmSmem;
  extern __shared__ __align__(1024) char smem[];
  if (smem_u32(smem) & 1023u) {   // the operand tiles' swizzle needs it; not seen
    if (threadIdx.x == 0) report(p.s.status, 3 /* KDA_ERR_CUDA */);
    return;
  }
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, row = tid & 127;
  const int role = warp >> 3, half = (warp >> 2) & 1, wq = warp & 3;   // eight warps per role, two per 32 rows
  uint16_t *order = reinterpret_cast<uint16_t *>(smem + L::ORDER);
  if (p.sorted) sort_longest(p.s.cu, p.s.n_seqs, reinterpret_cast<int *>(smem), order);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + L::BAR);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + L::TSLOT);
  float *sc_c = reinterpret_cast<float *>(smem + L::SC), *sc_h = sc_c + Q, *sc_w = sc_h + Q, *sc_e = sc_w + Q;

  if (tid == 0) {
    for (int i = 0; i < NBAR; ++i) {
      int count = 256;   // every thread of a role
      if (i == FULL0 || i == FULL1 || i == XFULL0 || i == XFULL1 || i == GDONE || i == YDONE || i == DSDONE || i == DRAIN0 || i == DRAIN1) count = 1;
      if (i >= DSPART0 && i <= DSPART3) count = 1;
      if (i >= MREADY0 && i <= MREADY3) count = 64 * (MREADY3 + 1 - i);
      if (i >= WXREADY0 && i <= WXREADY3) count = 64;
      if (i == SFULL) count = 32;
      if (i == EMPTY0 || i == EMPTY1) count = 2;
      if (i == SEMPTY) count = 768;
      mbar_init(&bar[i], count);
    }
    fence_mbar_init();
  }
  if (warp == 25) tc::alloc(tslot, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tslot, tl = tmem + ((uint32_t)(32 * wq) << 16);
  bool ok = true;
  Walk<MANY> w(p, order);
  int c = 0;   // chunks so far, of all items: the barriers' phases go by it

  if (role == 0) {
    // -------------------------------------------------------------- M and Y
    {
      const uint32_t z[8] = {};
#pragma unroll 1
      for (int k = half; k < 8; k += 2) st8u(tl + T_M + 8 * k, z);   // blocks above the diagonal stay zero
      tc::wait_st();
    }
    f2 e2 = two(0.f, 0.f), d2 = e2;
    int len = 0, t = 0, u = 0;   // of the previous chunk
    float d = !MANY && p.s.d_skip ? p.s.d_skip[w.head(p)] : 0.f;
    if (!MANY) d2 = two(d, d);
    for (;; ++c) {
      const bool more = w.chunk(p, order);
      if (c > 0) {   // the previous chunk's Y, while this chunk's G runs
        const int k0 = c - 1;
        char *ys = smem + (k0 & 1) * L::STAGE + L::X;   // in the place of the chunk's X, which everything has read by then
        ok = mbar_wait_quiet(&bar[YDONE], k0 & 1) && mbar_wait_quiet(&bar[XEMPTY0 + (k0 & 1)], (k0 >> 1) & 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc::fence_after();
#pragma unroll 1
        for (int k = 2 * half; k < 2 * half + 2; ++k) {
          float v[16], u[16];
          uint32_t o[8];
          tc::ld16(tl + T_Y1 + 16 * k, v);
          tc::ld16(tl + T_Y2 + 16 * k, u);
          tc::wait_ld();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 xv = *reinterpret_cast<const uint4 *>(ys + row_chunk(row, 2 * k + h));
            const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 8 * h + 2 * i;
              o[4 * h + i] = pack2(fma2(d2, unpack2(xw[i]), fma2(e2, two(u[j], u[j + 1]), two(v[j], v[j + 1]))));
            }
          }
          *reinterpret_cast<uint4 *>(ys + row_chunk(row, 2 * k)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4 *>(ys + row_chunk(row, 2 * k + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        tc::fence_before();
        mbar_arrive(&bar[YFREE]);
        if (len < Q && row < len) {   // a sequence's short last chunk: its box would reach into the next sequence
          bf16 *to = static_cast<bf16 *>(p.s.y) + (long long)(t + row) * p.s.H * p.s.P + u * SSM_COLS;
#pragma unroll 1
          for (int k = 4 * half; k < 4 * half + 4; ++k)
            *reinterpret_cast<uint4 *>(to + 8 * k) = *reinterpret_cast<const uint4 *>(ys + row_chunk(row, k));   // the thread's own
        }
        fence_proxy_async();
        mbar_arrive(&bar[YSTAGED0 + (k0 & 1)]);
      }
      if (!more) break;
      len = w.len(), t = w.t, u = w.u;
      if (MANY && w.fresh && p.s.d_skip) d = p.s.d_skip[w.head(p)];
      // M's columns are free: the products of the previous chunk were issued before this G
      ok = mbar_wait_quiet(&bar[SFULL], c & 1) && mbar_wait_quiet(&bar[GDONE], c & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc::fence_after();
      const float ci = sc_c[row];
      // M: row i, 16 columns at a time, every other block of 16 (the other half's warps take the rest). Left of the
      // diagonal's 32 columns 2^(c_i - c_j) h_j = 2^(c_i - c_r) e_j with the last column r of j's 32,
      // e_j = 2^(c_r - c_j) h_j (both exponents <= 0): no exponential per entry
#pragma unroll 1
      for (int jb = 0; jb < wq; ++jb) {
        const int j0 = 32 * jb + 16 * half;
        float g[16];
        uint32_t m[8];
        tc::ld16(tl + T_G + j0, g);
        const float r = ex2(ci - sc_c[32 * jb + 31]);
        const f2 r2 = two(r, r);
        tc::wait_ld();
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 e = *reinterpret_cast<const float4 *>(sc_e + j0 + j);
          m[j / 2] = pack2(mul2(mul2(two(g[j], g[j + 1]), two(e.x, e.y)), r2));
          m[j / 2 + 1] = pack2(mul2(mul2(two(g[j + 2], g[j + 3]), two(e.z, e.w)), r2));
        }
        st8u(tl + T_M + j0 / 2, m);
        tc::wait_st();
        tc::fence_before();
        mbar_arrive(&bar[MREADY0 + jb]);
      }
      {
        const int j0 = 32 * wq + 16 * half;
        float g[16];
        uint32_t m[8];
        tc::ld16(tl + T_G + j0, g);
        tc::wait_ld();
        tc::fence_before();
        mbar_arrive(&bar[GFREE]);
        const uint32_t keep = ((2u << lane) - 1u) >> (16 * half);   // columns j <= i
        const f2 c2 = two(ci, ci), minus = two(-1.f, -1.f);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 cj = *reinterpret_cast<const float2 *>(sc_c + j0 + j), hj = *reinterpret_cast<const float2 *>(sc_h + j0 + j);
          const float2 x = of2(fma2(two(cj.x, cj.y), minus, c2));
          const float2 v = of2(mul2(mul2(two(ex2(x.x), ex2(x.y)), two(hj.x, hj.y)), two(g[j], g[j + 1])));
          m[j / 2] = pack2(keep >> j & 1u ? v.x : 0.f, keep >> (j + 1) & 1u ? v.y : 0.f);
        }
        st8u(tl + T_M + j0 / 2, m);
        tc::wait_st();
        tc::fence_before();
        mbar_arrive(&bar[MREADY0 + wq]);
      }
      mbar_arrive(&bar[SEMPTY]);
      const float ei = exp2f(ci);
      e2 = two(ei, ei);
      if (MANY) d2 = two(d, d);
    }
  } else if (role == 1) {
    // -------------------------------------------------------------- w o X
    for (; w.chunk(p, order); ++c) {
      char *st = smem + (c & 1) * L::STAGE;
      ok = mbar_wait_quiet(&bar[SFULL], c & 1) && mbar_wait_quiet(&bar[XFULL0 + (c & 1)], (c >> 1) & 1);
      if (!ok) break;
      const int len = w.len();
      const bool live = row < len;
      const float weight = live ? sc_w[row] : 0.f;
      if (len < Q) {
        // the only chunk at which this role waits for B, a sequence's last; the one before in this stage has been used up, or X would not be here
        ok = mbar_wait_quiet(&bar[FULL0 + (c & 1)], (c >> 1) & 1);
        if (!ok) break;
        if (!live) {   // rows past the sequence's end belong to another one, or to nobody: whatever they hold stays out
          const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            *reinterpret_cast<uint4 *>(st + L::B + 16384 * half + row_chunk(row, k)) = z;
            if (k >> 2 == half) *reinterpret_cast<uint4 *>(st + L::X + row_chunk(row, k)) = z;
          }
        }
        fence_proxy_async();
        mbar_arrive(&bar[TAIL]);
      }
      if (c > 0) ok = mbar_wait_quiet(&bar[DSPART0 + wq], (c - 1) & 1);   // the previous terms of these tokens are read
      if (!ok) break;
      weigh(st + L::X, smem + L::WX, row, half, weight);
      fence_proxy_async();
      mbar_arrive(&bar[WXREADY0 + wq]);
      mbar_arrive(&bar[XEMPTY0 + (c & 1)]);
      mbar_arrive(&bar[SEMPTY]);
    }
  } else if (role == 2) {
    // -------------------------------------------------------------- the state: row n of [128][64], 32 columns
    f2 S[16];   // pairs of columns
    if (p.nseg > 1) asm volatile("griddepcontrol.wait;\n" ::: "memory");   // the entering states; nothing else here depends on the kernels before
    while (ok && w.item(p, order)) {
      auto place = [&]() { return (((size_t)w.seq() * p.s.H + w.head(p)) * SSM_N + row) * p.s.P + w.col0(p) + 32 * half; };   // of the row in h0 and hT
      const float *from = p.s.h0 ? p.s.h0 + place() : nullptr;
      if (w.seg() > 0)
        from = p.seg_state + ((((size_t)w.seq() * (p.nseg - 1) + w.seg() - 1) * (p.s.H * (p.s.P / SSM_COLS)) + w.u) * SSM_N + row) * SSM_COLS + 32 * half;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 v = from ? *reinterpret_cast<const float4 *>(from + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
        S[2 * i] = two(v.x, v.y), S[2 * i + 1] = two(v.z, v.w);
      }
      for (; w.left > 0; --w.left, ++c) {
        if (c > 0) {
          ok = mbar_wait_quiet(&bar[YDONE], (c - 1) & 1);   // C S has read the previous operand
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)   // the operand tile
          *reinterpret_cast<uint4 *>(smem + L::S + row_chunk(row, 4 * half + k)) =
              make_uint4(pack2(S[4 * k]), pack2(S[4 * k + 1]), pack2(S[4 * k + 2]), pack2(S[4 * k + 3]));
        fence_proxy_async();
        mbar_arrive(&bar[SREADY]);
        ok = mbar_wait_quiet(&bar[SFULL], c & 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const float last = sc_c[Q - 1];
        mbar_arrive(&bar[SEMPTY]);
        const float dec = exp2f(last);
        const f2 dec2 = two(dec, dec);
        ok = mbar_wait_quiet(&bar[DSDONE], c & 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc::fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k) {   // 8 columns at a time: the registers hold no more
          float d0[8], d1[8], d2[8];
          ld8(tl + T_DS + 32 * half + 8 * k, d0);
          ld8(tl + T_DS + 64 + 32 * half + 8 * k, d1);
          ld8(tl + T_DS + 128 + 32 * half + 8 * k, d2);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            S[4 * k + i] = fma2(S[4 * k + i], dec2, add2(two(d0[2 * i], d0[2 * i + 1]), add2(two(d1[2 * i], d1[2 * i + 1]), two(d2[2 * i], d2[2 * i + 1]))));
        }
        tc::fence_before();
        mbar_arrive(&bar[DSFREE]);
      }
      if (ok && p.s.hT && w.seg() == p.nseg - 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 a = of2(S[2 * i]), b = of2(S[2 * i + 1]);
          *reinterpret_cast<float4 *>(p.s.hT + place() + 4 * i) = make_float4(a.x, a.y, b.x, b.y);
        }
    }
  } else if (warp == 24) {
    // -------------------------------------------------------------- scalars: lane l has tokens 4 l .. 4 l + 3
    float v[4], al = 0.f, bias = 0.f;
    if (!MANY) al = p.s.a[w.head(p)] * LOG2E, bias = p.s.dt_bias ? p.s.dt_bias[w.head(p)] : 0.f;
    auto fetch = [&]() {
      const int len = w.len(), head = w.head(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * lane + i;
        v[i] = t < len ? p.s.dt[(long long)(w.t + t) * p.s.H + head] : 0.f;
      }
    };
    bool more = w.chunk(p, order);
    if (more) fetch();
    for (; more; ++c) {
      const int len = w.len();
      if (MANY && w.fresh) al = p.s.a[w.head(p)] * LOG2E, bias = p.s.dt_bias ? p.s.dt_bias[w.head(p)] : 0.f;
      float h[4] = {v[0], v[1], v[2], v[3]};
      more = w.chunk(p, order);
      if (more) fetch();
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {   // one body for the four: the values rotate
        const float x = step_of(h[0], bias, p.s.softplus);
        h[0] = h[1], h[1] = h[2], h[2] = h[3];
        h[3] = 4 * lane + i < len ? x : 0.f;
      }
      float la[4], pre[4], suf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) la[i] = forgets(h[i], al);
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
      const float end = __shfl_sync(0xffffffffu, below, lane | 7);   // c at the last token of the lane's block of 32
      float e[4], w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pre[i] += bl;
        e[i] = h[i] * ex2(end - pre[i]);
        w[i] = h[i] * exp2f(suf[i] + ab);
      }
      // everything above ran beside the previous chunk; only the stores wait for its readers
      if (c > 0) ok = mbar_wait_quiet(&bar[SEMPTY], (c - 1) & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      *reinterpret_cast<float4 *>(sc_c + 4 * lane) = make_float4(pre[0], pre[1], pre[2], pre[3]);
      *reinterpret_cast<float4 *>(sc_h + 4 * lane) = make_float4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<float4 *>(sc_e + 4 * lane) = make_float4(e[0], e[1], e[2], e[3]);
      *reinterpret_cast<float4 *>(sc_w + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
      mbar_arrive(&bar[SFULL]);
    }
  } else if (warp == 27) {
    // -------------------------------------------------------------- loads
    if (lane == 0) {
      int issued = 0, xissued = 0, group = MANY ? 0 : w.head(p) / (p.s.H / p.s.G);
      int y_last = 0, x_last = 0, y_before = 0, x_before = 0;   // boxes of the last two chunks' outputs; -1: not by box
      bool more = true;
#pragma unroll 1
      for (int end = 0; end < 2; ++c) {
        char *st = smem + (c & 1) * L::STAGE;
        more = more && w.chunk(p, order);
        end += !more;
        const int x_col = w.u * SSM_COLS;
        if (MANY && more && w.fresh) group = w.head(p) / (p.s.H / p.s.G);
        if (more) {   // B and C first: they are free before Y has left from X's place
          if (c >= 2) ok = mbar_wait_quiet(&bar[EMPTY0 + (c & 1)], ((c >> 1) - 1) & 1);
          if (!ok) break;
          uint64_t *b = &bar[FULL0 + (c & 1)];
          mbar_expect_tx(b, 65536);
          for (int k = 0; k < 4; ++k)   // B's two halves, C's two
            tc::tma_load_2d(st + (k < 2 ? L::B : L::C) + 16384 * (k & 1), k < 2 ? &p.tm_b : &p.tm_c, group * SSM_N + 64 * (k & 1), w.t, b);
          issued = c + 1;
          if (w.left > 0) {   // the next chunk's boxes into L2
            for (int k = 0; k < 4; ++k) prefetch_2d(k < 2 ? &p.tm_b : &p.tm_c, group * SSM_N + 64 * (k & 1), w.t + Q);
            prefetch_2d(&p.tm_x, x_col, w.t + Q);
          }
        }
        if (c >= 2) {   // the outputs of two chunks ago leave as one box from the place of their X tile
          ok = mbar_wait_quiet(&bar[YSTAGED0 + (c & 1)], ((c >> 1) - 1) & 1);
          if (!ok) break;
          if (y_before >= 0) {
            tma_store_2d(&p.tm_y, x_before, y_before, st + L::X);
            bulk_commit();
            bulk_wait_read();
          }
        }
        x_before = x_last, y_before = y_last;
        if (more) {
          mbar_expect_tx(&bar[XFULL0 + (c & 1)], 16384);
          tc::tma_load_2d(st + L::X, &p.tm_x, x_col, w.t, &bar[XFULL0 + (c & 1)]);
          xissued = c + 1;
          x_last = x_col, y_last = w.len() == Q ? w.t : -1;
        }
      }
      // every copy has landed, in either direction, before the CTA leaves, also after a timeout
#pragma unroll 1
      for (int k = issued > 2 ? issued - 2 : 0; k < issued; ++k) mbar_wait_quiet(&bar[FULL0 + (k & 1)], (k >> 1) & 1);
#pragma unroll 1
      for (int k = xissued > 2 ? xissued - 2 : 0; k < xissued; ++k) mbar_wait_quiet(&bar[XFULL0 + (k & 1)], (k >> 1) & 1);
      bulk_wait_all();
    }
    __syncwarp();
  } else if (warp == 25) {
    // ------------------------------------------------------------ G, C S, M X
    const uint32_t leader = elect();
    const uint32_t d_s = dlo(smem_u32(smem + L::S), 8192);
    auto all = [&](bool w) { return (bool)__all_sync(0xffffffffu, w); };
#pragma unroll 1
    for (int tails = 0; w.chunk(p, order); ++c) {
      const uint32_t st = smem_u32(smem + (c & 1) * L::STAGE);
      const uint32_t d_c = dlo(st + L::C, 16), d_b = dlo(st + L::B, 16), d_x = dlo(st + L::X, 8192);
      ok = mbar_wait_quiet(&bar[FULL0 + (c & 1)], (c >> 1) & 1) && (c == 0 || mbar_wait_quiet(&bar[GFREE], (c - 1) & 1)) && (w.len() == Q || mbar_wait_quiet(&bar[TAIL], tails & 1));
      if (!(ok = all(ok))) break;
      tails += w.len() < Q;
      tc::fence_after();
#pragma unroll
      for (uint32_t ks = 0; ks < 8; ++ks) {
        const uint32_t o = (ks >> 2) * (16384 >> 4) + (ks & 3) * 2;
        mma_ss(leader, tmem + T_G, desc(d_c + o), desc(d_b + o), tc::idesc_bf16(128, 128), ks > 0);
      }
      commit(leader, &bar[GDONE]);
      ok = mbar_wait_quiet(&bar[SREADY], c & 1) && (c == 0 || mbar_wait_quiet(&bar[YFREE], (c - 1) & 1));
      if (!(ok = all(ok))) break;
      tc::fence_after();
#pragma unroll
      for (uint32_t ks = 0; ks < 8; ++ks)
        mma_ss(leader, tmem + T_Y2, desc(d_c + (ks >> 2) * (16384 >> 4) + (ks & 3) * 2), desc(d_s + ks * (2048 >> 4)),
               tc::idesc_bf16_mn(128, 64, false, true), ks > 0);
      commit(leader, &bar[EMPTY0 + (c & 1)]);
      ok = mbar_wait_quiet(&bar[XFULL0 + (c & 1)], (c >> 1) & 1);
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {   // as M's column blocks become ready
        ok = ok && all(mbar_wait_quiet(&bar[MREADY0 + k], c & 1));
        if (ok) {
          tc::fence_after();
          mma_ts(leader, tmem + T_Y1, tmem + T_M + 16 * k, desc(d_x + k * (4096 >> 4)), tc::idesc_bf16_mn(128, 64, false, true), k > 0);
          mma_ts(leader, tmem + T_Y1, tmem + T_M + 16 * k + 8, desc(d_x + k * (4096 >> 4) + (2048 >> 4)), tc::idesc_bf16_mn(128, 64, false, true), 1);
        }
      }
      if (!ok) break;
      commit(leader, &bar[YDONE]);
    }
    commit(leader, &bar[DRAIN0]);   // nothing of this thread runs on once the CTA leaves
    ok &= mbar_wait_quiet(&bar[DRAIN0], 0);
  } else {
    // -------------------------------------------------------------- B^T (w o X)
    const uint32_t leader = elect();
    const uint32_t d_w = dlo(smem_u32(smem + L::WX), 16384);
#pragma unroll 1
    for (; w.chunk(p, order); ++c) {
      const uint32_t d_b = dlo(smem_u32(smem + (c & 1) * L::STAGE + L::B), 16384);
      ok = mbar_wait_quiet(&bar[FULL0 + (c & 1)], (c >> 1) & 1) && (c == 0 || mbar_wait_quiet(&bar[DSFREE], (c - 1) & 1));
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        ok = __all_sync(0xffffffffu, ok && mbar_wait_quiet(&bar[WXREADY0 + k], c & 1));
        if (ok) {
          tc::fence_after();
          mma_ss(leader, tmem + T_DS, desc(d_b + k * (4096 >> 4)), desc(d_w + k * (4096 >> 4)), tc::idesc_bf16_mn(128, 192, true, true), k > 0);
          mma_ss(leader, tmem + T_DS, desc(d_b + k * (4096 >> 4) + (2048 >> 4)), desc(d_w + k * (4096 >> 4) + (2048 >> 4)),
                 tc::idesc_bf16_mn(128, 192, true, true), 1);
          commit(leader, &bar[DSPART0 + k]);
        }
      }
      if (!ok) break;
      commit(leader, &bar[DSDONE]);
      commit(leader, &bar[EMPTY0 + (c & 1)]);
    }
    commit(leader, &bar[DRAIN1]);
    ok &= mbar_wait_quiet(&bar[DRAIN1], 0);
  }
  if (!ok) report(p.s.status, ERR_TIMEOUT);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 25) tc::dealloc(tmem, 512);
}

// What a segment of whole chunks adds to the state, sum_j w_j B_j x_j^T, and its decay. With w counted to the segment's end instead of
// the chunk's, the chunks' products only have to be added up. The chunks go from the last to the first, so that a chunk's weights need
// only the sum of h a over the chunks already taken. Two sets of eight warps take every other chunk: w o X into the set's tiles, and the
// products of its previous chunk out of its half of tensor memory into fp32 registers (left there to add up over a segment they would
// be truncated at every step: the state was off by 1.4e-5 of its largest value after 85 chunks, now by 7e-7). Warp 16 has the scalars,
// warp 17 the products, warp 18 the loads. X has a third stage, so that it is there when a set's tiles have been read; B is not needed
// before w o X is formed. About 0.9 us a chunk where the scan itself takes 1.9.
struct StSmem {
  static constexpr int B = 0, X = 2 * 32768;
  static constexpr int WX = X + 3 * 16384;   // three terms per set
  static constexpr int SC = WX + 2 * 49152;  // fp32 w of the set's tokens
  static constexpr int BAR = SC + 2 * Q * 4;
  static constexpr int TSLOT = BAR + 20 * 8;
  static constexpr int BYTES = TSLOT + 16;
};
// two of each, by set, but three of X's and one for the end
enum StBar { ST_B, ST_WX = 2, ST_READ = 4, ST_S = 6, ST_SFREE = 8, ST_X = 10, ST_XFREE = 13, ST_END = 16, ST_NBAR };
static_assert(ST_NBAR <= 20 && StSmem::BYTES <= 232448, "places");

__global__ void __launch_bounds__(608, 1) ssm_states_kernel(const __grid_constant__ SsmTcParams p) {
  using L = StSmem;
  extern __shared__ __align__(1024) char smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) report(p.s.status, 3 /* KDA_ERR_CUDA */);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");   // the kernels after this one wait for its end where they read
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, row = tid & 127;
  const int U = p.s.H * (p.s.P / SSM_COLS), nseg = p.nseg;
  const int u = blockIdx.x % U, ns = blockIdx.x / U, seg = ns % (nseg - 1), n = ns / (nseg - 1);
  const int head = u / (p.s.P / SSM_COLS), col0 = (u % (p.s.P / SSM_COLS)) * SSM_COLS, group = head / (p.s.H / p.s.G);
  const int each = (int)(p.s.T / p.s.n_seqs), seq0 = max(p.s.cu ? p.s.cu[n] : each * n, 0);
  const int seq1 = max(min(p.s.cu ? p.s.cu[n + 1] : each * (n + 1), (int)p.s.T), seq0);
  const int all = (int)(((unsigned)(seq1 - seq0) + Q - 1) / Q);
  const int first = (int)((long long)all * seg / nseg), nch = (int)((long long)all * (seg + 1) / nseg) - first;
  auto token = [&](int i) { return seq0 + (first + nch - 1 - i) * Q; };   // of the i-th chunk taken: a whole one, the last segment is not run
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + L::BAR);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + L::TSLOT);
  float *sc_w = reinterpret_cast<float *>(smem + L::SC);
  if (tid == 0) {
    for (int i = 0; i < ST_NBAR; ++i) mbar_init(&bar[i], i / 2 == ST_WX / 2 || i / 2 == ST_SFREE / 2 || (i >= ST_XFREE && i < ST_END) ? 256 : i / 2 == ST_S / 2 ? 32 : 1);
    fence_mbar_init();
  }
  if (warp == 17) tc::alloc(tslot, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tslot;
  const size_t at = ((size_t)n * (nseg - 1) + seg) * U + u;
  bool ok = true;
  if (warp < 16) {
    const int set = warp >> 3, half = (warp >> 2) & 1;
    const uint32_t from = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 192 * set + 32 * half;
    f2 S[16];   // 32 columns of a row
#pragma unroll
    for (int i = 0; i < 16; ++i) S[i] = two(0.f, 0.f);
    auto take = [&](int i) {   // chunk i's products
      ok = __all_sync(0xffffffffu, ok && mbar_wait_quiet(&bar[ST_READ + set], (i >> 1) & 1));
      if (!ok) return;
      tc::fence_after();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float d0[8], d1[8], d2[8];
        ld8(from + 8 * k, d0);
        ld8(from + 64 + 8 * k, d1);
        ld8(from + 128 + 8 * k, d2);
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 4; ++e)
          S[4 * k + e] = add2(S[4 * k + e], add2(two(d0[2 * e], d0[2 * e + 1]), add2(two(d1[2 * e], d1[2 * e + 1]), two(d2[2 * e], d2[2 * e + 1]))));
      }
      tc::fence_before();
    };
    int xs = set, xphase = 0, i = set;   // i % 3, i / 3 & 1
    for (; i < nch; i += 2) {
      if (i >= 2) take(i - 2);
      ok = ok && mbar_wait_quiet(&bar[ST_X + xs], xphase) && mbar_wait_quiet(&bar[ST_S + set], (i >> 1) & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const float w = sc_w[set * Q + row];
      mbar_arrive(&bar[ST_SFREE + set]);
      weigh(smem + L::X + 16384 * xs, smem + L::WX + 49152 * set, row, half, w);
      fence_proxy_async();
      mbar_arrive(&bar[ST_WX + set]);
      mbar_arrive(&bar[ST_XFREE + xs]);
      xs += 2;
      if (xs >= 3) xs -= 3, xphase ^= 1;
    }
    if (i >= 2) take(i - 2);
    // the second set's sums join the first's; every product and load is done with this part of shared memory once both have taken theirs
    char *meet = smem + L::WX + row * 256;
    asm volatile("bar.sync 1, 512;\n" ::: "memory");
    if (set == 1)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 a = of2(S[2 * k]), b = of2(S[2 * k + 1]);
        *reinterpret_cast<float4 *>(meet + (((8 * half + k) ^ (row & 15)) << 4)) = make_float4(a.x, a.y, b.x, b.y);
      }
    asm volatile("bar.sync 1, 512;\n" ::: "memory");
    if (set == 0) {
      float *dst = p.seg_state + at * SSM_N * SSM_COLS + (size_t)row * SSM_COLS + 32 * half;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float4 o = *reinterpret_cast<const float4 *>(meet + (((8 * half + k) ^ (row & 15)) << 4));
        const float2 a = of2(S[2 * k]), b = of2(S[2 * k + 1]);
        *reinterpret_cast<float4 *>(dst + 4 * k) = make_float4(a.x + o.x, a.y + o.y, b.x + o.z, b.y + o.w);
      }
    }
  } else if (warp == 16) {   // lane l has tokens 4 l .. 4 l + 3
    const float al = p.s.a[head] * LOG2E, bias = p.s.dt_bias ? p.s.dt_bias[head] : 0.f;
    auto fetch = [&](int i, float (&v)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = p.s.dt[(long long)(token(i) + 4 * lane + k) * p.s.H + head];
    };
    float v[4], later = 0.f;   // sum of h a over the chunks taken
    if (nch > 0) fetch(0, v);
    for (int i = 0; i < nch; ++i) {
      float h[4], w[4], suf[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = step_of(v[k], bias, p.s.softplus);
      if (i + 1 < nch) fetch(i + 1, v);
      suf[3] = 0.f;
#pragma unroll
      for (int k = 2; k >= 0; --k) suf[k] = suf[k + 1] + forgets(h[k + 1], al);
      float above = suf[0] + forgets(h[0], al);
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const float z = __shfl_down_sync(0xffffffffu, above, o);
        if (lane + o < 32) above += z;
      }
      const float right = __shfl_down_sync(0xffffffffu, above, 1), ab = (lane < 31 ? right : 0.f) + later;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = h[k] * exp2f(suf[k] + ab);
      later += __shfl_sync(0xffffffffu, above, 0);
      if (i >= 2) ok = mbar_wait_quiet(&bar[ST_SFREE + (i & 1)], ((i >> 1) - 1) & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      *reinterpret_cast<float4 *>(sc_w + (i & 1) * Q + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
      mbar_arrive(&bar[ST_S + (i & 1)]);
    }
    if (lane == 0) p.seg_decay[at] = exp2f(later);
  } else if (warp == 17) {
    const uint32_t leader = elect();
#pragma unroll 1
    for (int i = 0; i < nch; ++i) {
      const uint32_t d_b = dlo(smem_u32(smem + L::B + (i & 1) * 32768), 16384), d_w = dlo(smem_u32(smem + L::WX + (i & 1) * 49152), 16384);
      ok = mbar_wait_quiet(&bar[ST_B + (i & 1)], (i >> 1) & 1) && mbar_wait_quiet(&bar[ST_WX + (i & 1)], (i >> 1) & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc::fence_after();
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k)
        mma_ss(leader, tmem + 192 * (i & 1), desc(d_b + k * (2048 >> 4)), desc(d_w + k * (2048 >> 4)), tc::idesc_bf16_mn(128, 192, true, true), k > 0);
      commit(leader, &bar[ST_READ + (i & 1)]);
    }
    commit(leader, &bar[ST_END]);
    ok &= mbar_wait_quiet(&bar[ST_END], 0);
  } else if (lane == 0) {
    int issued = 0, xissued = 0, xs = 0, xphase = 0;
    auto load_x = [&]() {   // of the next chunk that has none
      if (xissued >= 3 && !mbar_wait_quiet(&bar[ST_XFREE + xs], xphase ^ 1)) return false;
      mbar_expect_tx(&bar[ST_X + xs], 16384);
      tc::tma_load_2d(smem + L::X + 16384 * xs, &p.tm_x, head * p.s.P + col0, token(xissued), &bar[ST_X + xs]);
      ++xissued;
      if (++xs == 3) xs = 0, xphase ^= 1;
      return true;
    };
    if (nch > 0) ok = load_x();
    for (int i = 0; i < nch && ok; ++i) {
      if (xissued < nch) ok = load_x();
      if (ok && i >= 2) ok = mbar_wait_quiet(&bar[ST_READ + (i & 1)], ((i >> 1) - 1) & 1);
      if (!ok) break;
      mbar_expect_tx(&bar[ST_B + (i & 1)], 32768);
      for (int k = 0; k < 2; ++k) tc::tma_load_2d(smem + L::B + 32768 * (i & 1) + 16384 * k, &p.tm_b, group * SSM_N + 64 * k, token(i), &bar[ST_B + (i & 1)]);
      issued = i + 1;
      if (i + 2 < nch) {
        prefetch_2d(&p.tm_x, head * p.s.P + col0, token(i + 2));
        for (int k = 0; k < 2; ++k) prefetch_2d(&p.tm_b, group * SSM_N + 64 * k, token(i + 2));
      }
    }
    // everything has landed before the CTA leaves, also after a timeout
    for (int i = issued > 2 ? issued - 2 : 0; i < issued; ++i) ok &= mbar_wait_quiet(&bar[ST_B + (i & 1)], (i >> 1) & 1);
    for (int i = xissued > 3 ? xissued - 3 : 0; i < xissued; ++i) ok &= mbar_wait_quiet(&bar[ST_X + i % 3], (i / 3) & 1);
  }
  if (!ok) report(p.s.status, ERR_TIMEOUT);
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 17) tc::dealloc(tmem, 512);
}

// From what the segments add and their decays to the states that the segments after them start from, in place. Grid: (units of all
// sequences, eighths of a state); a thread has four columns of a row, all segments' on their way at once.
constexpr int MOST_SEGS = 16;
__global__ void __launch_bounds__(256) ssm_fold_kernel(SsmTcParams p) {
  const int U = p.s.H * (p.s.P / SSM_COLS), u = blockIdx.x % U, n = blockIdx.x / U, m = p.nseg - 1;
  const int head = u / (p.s.P / SSM_COLS), col0 = (u % (p.s.P / SSM_COLS)) * SSM_COLS, e = blockIdx.y * 256 + threadIdx.x;
  float4 v[MOST_SEGS - 1];
  float dec[MOST_SEGS - 1];
  auto place = [&](int k) { return reinterpret_cast<float4 *>(p.seg_state + (((size_t)n * m + k) * U + u) * SSM_N * SSM_COLS) + e; };
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
#pragma unroll
  for (int k = 0; k < MOST_SEGS - 1; ++k)
    if (k < m) v[k] = *place(k), dec[k] = p.seg_decay[((size_t)n * m + k) * U + u];
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.s.h0) S = *reinterpret_cast<const float4 *>(p.s.h0 + (((size_t)n * p.s.H + head) * SSM_N + e / 16) * p.s.P + col0 + e % 16 * 4);
#pragma unroll
  for (int k = 0; k < MOST_SEGS - 1; ++k)
    if (k < m) {
      S.x = fmaf(S.x, dec[k], v[k].x), S.y = fmaf(S.y, dec[k], v[k].y), S.z = fmaf(S.z, dec[k], v[k].z), S.w = fmaf(S.w, dec[k], v[k].w);
      *place(k) = S;
    }
}

bool map_rows(EncodeTiledFn fn, CUtensorMap *m, const void *base, long long rows, long long width, long long ld) {
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)Q}, estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

// Segments per sequence: the count that takes the fewest chunk times (about 1.9 us each). Every wave of CTAs walks a k-th of a sequence;
// the states' pass takes half of a full chunk's time per chunk, a wave's start about 2.5 chunk times, the two further launches 3 and
// each segment half of one. 32768 tokens x 24 units (heads x head_dim / 64): 477 us in one piece, 138 in 6 segments; x 40 units 480 us,
// 257 in 3, 247 in 11; x 96 units, which keep 96 SMs busy, 483 us and at best 518, in 3. 4096 tokens x 24 units: 67 and 34 us.
int ssm_segments(int n_seqs, long long T, int units) {
  if (n_seqs < 1 || T < 1) return 1;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    (void)cudaGetLastError();
    sms = 152;
  }
  const double chunks = (double)T / n_seqs / Q;
  auto waves = [&](long long k) { return (double)(((long long)n_seqs * units * k + sms - 1) / sms); };
  int best = 1;
  double cost = (chunks + 2.5) * waves(1) + 2.0;
  for (int k = 2; k <= MOST_SEGS && k * 2 <= chunks && (long long)n_seqs * units * k < SSM_TC_ITEMS; ++k) {
    const double full = waves(k), states = waves(k - 1);
    const double t = chunks / k * (full + 0.5 * states) + 2.5 * (full + states) + 5.0 + 0.5 * k;
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
  p.sorted = s.cu && s.n_seqs > 1 && s.n_seqs <= MOST_SORTED;
  const int U = s.H * (s.P / SSM_COLS);
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return cudaErrorNotSupported;
  const long long rows = s.T > 0 ? s.T : 1;
  if (s.T > 0 && (!map_rows(fn, &p.tm_x, s.x, rows, (long long)s.H * s.P, s.ldx) || !map_rows(fn, &p.tm_b, s.b, rows, (long long)s.G * SSM_N, s.ldb) ||
                  !map_rows(fn, &p.tm_c, s.c, rows, (long long)s.G * SSM_N, s.ldc) ||
                  !map_rows(fn, &p.tm_y, s.y, rows, (long long)s.H * s.P, (long long)s.H * s.P)))
    return cudaErrorInvalidValue;
  p.items = (unsigned)((size_t)s.n_seqs * nseg * U);
  const size_t items = nseg > 1 ? (size_t)s.n_seqs * (nseg - 1) * U : 0;
  p.seg_state = static_cast<float *>(workspace);
  p.seg_decay = p.seg_state + items * SSM_N * SSM_COLS;
  // once per host thread and device: the kernels' shared memory
  static thread_local int ready = -1;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && ready != dev) {
    e = cudaFuncSetAttribute(ssm_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, SsmSmem::BYTES);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(ssm_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, SsmSmem::BYTES);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(ssm_states_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, StSmem::BYTES);
    if (e == cudaSuccess) ready = dev;
  }
  if (e != cudaSuccess) return e;
  // Short items: a CTA stays and goes on into the next one, so that its loads, state and first products come under the last one's end.
  // 64 sequences of 128 tokens x 96 heads 389 us with a CTA each, 235 so; 32 of 512 326 and 278; 16 of 1024 257 and 239; 4 of 4096 214
  // and 220 (the dealing out is fixed, where single CTAs go to whichever SM is free: eight from 0 to 5501 tokens 191 and 205).
  const bool many = p.items > (unsigned)sms && s.T < (long long)12 * Q * s.n_seqs * nseg;
  const unsigned ctas = many ? (unsigned)sms : p.items;
  const auto kernel = many ? ssm_tc_kernel<true> : ssm_tc_kernel<false>;
  if (nseg > 1) {
    ssm_states_kernel<<<(unsigned)items, 608, StSmem::BYTES, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_under(ssm_fold_kernel, dim3((unsigned)(s.n_seqs * U), SSM_N * SSM_COLS / 1024), 256, 0, st, p);
    if (e != cudaSuccess) return e;
    return launch_under(kernel, dim3(ctas), 896, SsmSmem::BYTES, st, p);
  }
  kernel<<<ctas, 896, SsmSmem::BYTES, st>>>(p);
  return cudaGetLastError();
}

}  // namespace kda
