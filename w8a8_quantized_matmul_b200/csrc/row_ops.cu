// Row operators that make the INT8 rows of a W8A8 layer.
//
//   RMS norm with the residual's addition   h = x + r,  H = round(h)
//                                           u = h * gamma,  w = u * s_rcp
//                                           rstd = 1 / sqrt(mean(h^2) + eps)
//                                           codes of w, x_scale = max|w| * rstd,
//                                           Xn = fp16(u * rstd)
//   SwiGLU                                  z = g / (1 + exp(-g)) * up,  w = z * s_rcp
//                                           codes of w, z_scale = max|w|, Z = fp16(z)
//
// Codes are the library's absmax codes clamp(rint(fl32(fl32(w*127)/max|w|))).
// rstd is positive and common to a row, so it cancels in the codes of the
// normalised row and only scales the row's absmax: the sum of squares and the
// maximum are reduced together, in one pass over a row that stays in registers.
//
// Both are bound by HBM: a norm with an fp16 residual moves 7 bytes per element
// (x and r read, H and the code written), SwiGLU 5.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "int8mm.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "quant_common.cuh"

namespace i8mm {

namespace {

struct RowArgs {
  const __half* X;        // norm: [M][K]; SwiGLU: [M][2K], gate then up
  const void* residual;   // norm: [M][K] fp16 or fp32, or nullptr
  const __half* gamma;    // norm: [K]
  const float* s_rcp;     // [K] or nullptr
  void* H;                // norm: [M][K] in the residual's type, or nullptr
  __half* Xn;             // [M][K] or nullptr
  int8_t* Xq;             // [M][K] or nullptr
  float* x_scale;         // [M]
  int M, K;
  float eps;
};

enum Stream { kNone, kF16, kF32 };   // the residual's type

// Up to this many rows per SM a CTA takes one row.
constexpr int kRowPerCta = 2;
constexpr float kHuge = 0x1p100f, kTiny = 0x1p-90f;

// A pair of fp32 values as one 64-bit register and back, without the shifts that
// would keep the compiler from placing the halves where they are.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

// Four pairs of fp32 values.
struct Oct {
  uint64_t v[4];
};

__device__ __forceinline__ Oct oct_h(const uint4& u) {
  const __half2* h = reinterpret_cast<const __half2*>(&u);
  Oct o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    o.v[i] = pair2(f.x, f.y);
  }
  return o;
}
__device__ __forceinline__ Oct oct_f(const float4& a, const float4& b) {
  return Oct{{pair2(a.x, a.y), pair2(a.z, a.w), pair2(b.x, b.y), pair2(b.z, b.w)}};
}
__device__ __forceinline__ Oct load_oct_f(const float* p) {
  const float4* q = reinterpret_cast<const float4*>(p);
  return oct_f(__ldg(q), __ldg(q + 1));
}
__device__ __forceinline__ Oct mul(const Oct& a, const Oct& b) {
  Oct o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.v[i] = mul2(a.v[i], b.v[i]);
  return o;
}
__device__ __forceinline__ uint4 pack_h(const Oct& a) {
  uint4 u;
  __half2* h = reinterpret_cast<__half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = split2(a.v[i]);
    h[i] = __floats2half2_rn(f.x, f.y);
  }
  return u;
}
// max(m, |a|, |b|), NaN where one of them is: a row that holds one has to say so in its
// scale (the instruction is the same without .NaN, which would drop it).
__device__ __forceinline__ float max_abs3(float m, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float absmax(const Oct& a, float m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = split2(a.v[i]);
    m = max_abs3(m, f.x, f.y);
  }
  return m;
}

// Eight codes clamp(rint(fl32(fl32(w*127)/a))), |w| <= a, with k = fl(127/a): w*k and
// the quotient are within 3 * 127 * 2^-24 < 2^-15 of each other, so its nearest
// integer is the code unless it lies that close to the middle between two. `far`
// gets the largest distance from the integers; where it is above kSure the
// vector's codes are taken from the quotient itself (codes8_exact).
constexpr float kSure = 0.5f - 0x1p-15f;

__device__ __forceinline__ uint2 pack8b(const uint32_t (&b)[8]) {
  return make_uint2(
      __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
      __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}

__device__ __forceinline__ uint2 codes8_near(const Oct& w, uint64_t k2, float* far) {
  uint32_t b[8];
  float d = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t m = fma2(w.v[i], k2, pair2(kMagic, kMagic));
    const float2 s = split2(m);
    b[2 * i] = __float_as_uint(s.x);
    b[2 * i + 1] = __float_as_uint(s.y);
    // magic - m is minus the integer
    const float2 e = split2(fma2(w.v[i], k2, sub2(pair2(kMagic, kMagic), m)));
    d = max_abs3(d, e.x, e.y);
  }
  *far = d;
  return pack8b(b);
}

// The correctly rounded quotient without a division: n = fl(w*127), ra = fl(1/a),
// q = fl(n*ra) is within 2 steps of n/a, one correction q += (n - q*a)*ra leaves an
// error far below a step before its rounding, so within one step after it, and from
// there Markstein's theorem (see quant_common.cuh) makes the second correction's
// result the rounded quotient. The remainders are exact where a is neither tiny nor
// huge; other rows take codes8_div.
__device__ __forceinline__ uint2 codes8_exact(const Oct& w, float a) {
  const float r = quant_rcp(a);
  const uint64_t na2 = pair2(-a, -a), ra2 = pair2(r, r);
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t n = mul2(w.v[i], pair2(127.0f, 127.0f));
    uint64_t q = mul2(n, ra2);
    q = fma2(fma2(q, na2, n), ra2, q);
    q = fma2(fma2(q, na2, n), ra2, q);
    const float2 s = split2(add2(q, pair2(kMagic, kMagic)));
    b[2 * i] = __float_as_uint(s.x);
    b[2 * i + 1] = __float_as_uint(s.y);
  }
  return pack8b(b);
}

__device__ __forceinline__ uint2 codes8_div(const Oct& w, float a) {
  int q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = split2(w.v[i]);
    q[2 * i] = quant_code(f.x, a);
    q[2 * i + 1] = quant_code(f.y, a);
  }
  return make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
}

// silu(g) for eight fp16 values. With n = -|g| and t = e^n <= 1, silu(g) =
// max(g, 0) + n * t / (1 + t): nothing overflows, and nothing cancels (the second
// term is at most half the first). t = 2^y * (1 + c), y the rounded product of n and
// log2 e; c = n - y * ln 2, with ln 2 in two parts, takes back y's rounding and that of
// the constant, which the size of n multiplies (with ln 2 in one part the result was off by 15
// half steps at g = -60). c is below 2^-17, so that what 1 + c leaves out is nothing.
// With ex2.approx within 2^-22 and rcp.approx within 2^-23 the result is within 10
// half steps of fp32: 4 and 2, and one each for 1 + c, n * t, 1 + t and the last step (a
// Newton step on the reciprocal would take one away and cost 5% of the time). Below
// g = -87.3 t leaves fp32's normal range and counts as 0.
// A gate of +inf, where n * t would be NaN, gives +inf: a positive gate enters n as -128 at
// least, where t is 0 already; -inf gives NaN, as g / (1 + exp(-g)) does, and so does
// NaN, through max(g, 0).
__device__ __forceinline__ Oct silu8(const uint4& u) {
  constexpr float kLog2e = 1.44269504088896340736f;
  constexpr float kLn2 = 0.69314718055994530942f;
  constexpr float kLn2Low = static_cast<float>(0.69314718055994530942 - static_cast<double>(kLn2));
  const __half2* h = reinterpret_cast<const __half2*>(&u);
  Oct o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 nf = __half22float2(__hmin2(h[i], __hmax2(__hneg2(h[i]), __float2half2_rn(-128.0f))));
    const float2 gf = __half22float2(__hmax2_nan(h[i], __float2half2_rn(0.0f)));
    const uint64_t n = pair2(nf.x, nf.y);
    const uint64_t y = mul2(n, pair2(kLog2e, kLog2e));
    const uint64_t c = fma2(y, pair2(-kLn2Low, -kLn2Low), fma2(y, pair2(-kLn2, -kLn2), n));
    const float2 y1 = split2(y);
    float e0, e1, r0, r1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(y1.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(y1.y));
    uint64_t t = pair2(e0, e1);
    t = fma2(t, c, t);
    const float2 d1 = split2(add2(t, pair2(1.0f, 1.0f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d1.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d1.y));
    o.v[i] = fma2(mul2(n, t), pair2(r0, r1), pair2(gf.x, gf.y));
  }
  return o;
}

// Raw operands of one vector of eight values: X, or the gate, and the residual
// (fp16 in r0, fp32 in r0 and r1) or the up projection (r0).
struct Raw {
  uint4 x, r0, r1;
};

// What a row's arrays start with; a thread's values lie at 32-bit offsets from there.
template <bool NORM, int STREAM>
struct Row {
  const __half* x;       // X, or the gate
  const char* r;         // the residual
  char* H;
  __device__ __forceinline__ Row(const RowArgs& a, size_t row) {
    x = a.X + row * (NORM ? a.K : 2 * static_cast<size_t>(a.K));
    const size_t bytes = row * a.K * (STREAM == kF32 ? 4 : 2);
    r = static_cast<const char*>(a.residual) + bytes;
    H = a.H ? static_cast<char*>(a.H) + bytes : nullptr;
  }
  // Operand `part` of the vector at column k.
  __device__ __forceinline__ const void* at(uint32_t k, int part, uint32_t K) const {
    if constexpr (!NORM) return x + (part ? K : 0u) + k;
    if (part == 0) return x + k;
    if constexpr (STREAM == kF32) return r + 4 * k + 16 * (part - 1);
    return r + 2 * k;
  }
};

template <bool NORM, int STREAM>
constexpr int kParts = NORM ? (STREAM == kNone ? 1 : STREAM == kF16 ? 2 : 3) : 2;

// u of the vector at column k of a row; adds the squares of h to sq, writes H (an
// fp32 H into shared memory at `park` where that is not 0).
template <bool NORM, int STREAM>
__device__ __forceinline__ Oct make_u(const RowArgs& a, const Row<NORM, STREAM>& row, uint32_t k,
                                      const Raw& w, const uint4& gamma, uint64_t& sq,
                                      uint32_t park = 0) {
  if constexpr (!NORM) {
    return mul(silu8(w.x), oct_h(w.r0));
  } else {
    const Oct g = oct_h(gamma);
    Oct h = oct_h(w.x);
    if constexpr (STREAM != kNone) {
      const Oct r = STREAM == kF16 ? oct_h(w.r0)
                                   : oct_f(*reinterpret_cast<const float4*>(&w.r0),
                                           *reinterpret_cast<const float4*>(&w.r1));
#pragma unroll
      for (int i = 0; i < 4; ++i) h.v[i] = add2(h.v[i], r.v[i]);
      if (row.H) {
        if constexpr (STREAM == kF16) {
          *reinterpret_cast<uint4*>(row.H + 2 * k) = pack_h(h);
        } else {
          float4* q = reinterpret_cast<float4*>(row.H + 4 * k);
          const float2 h0 = split2(h.v[0]), h1 = split2(h.v[1]), h2 = split2(h.v[2]), h3 = split2(h.v[3]);
          if (park) {
            sts16(park, make_float4(h0.x, h0.y, h1.x, h1.y));
            sts16(park + 16, make_float4(h2.x, h2.y, h3.x, h3.y));
          } else {
            q[0] = make_float4(h0.x, h0.y, h1.x, h1.y);
            q[1] = make_float4(h2.x, h2.y, h3.x, h3.y);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sq = fma2(h.v[i], h.v[i], sq);
    return mul(h, g);
  }
}

template <bool NORM>
__device__ __forceinline__ uint4 load_gamma(const RowArgs& a, uint32_t k) {
  return NORM ? __ldg(reinterpret_cast<const uint4*>(a.gamma + k)) : make_uint4(0, 0, 0, 0);
}
template <bool SMOOTH>
__device__ __forceinline__ void load_s(const RowArgs& a, uint32_t k, float4 (&s)[2]) {
  if constexpr (SMOOTH) {
    s[0] = __ldg(reinterpret_cast<const float4*>(a.s_rcp + k));
    s[1] = __ldg(reinterpret_cast<const float4*>(a.s_rcp + k) + 1);
  }
}

// The maximum of |w|, and w in u's place unless u itself is asked for (Xn): s_rcp is
// then read once.
template <bool SMOOTH>
__device__ __forceinline__ void keep_w(const RowArgs& a, const float4 (&s)[2], Oct& u, float& top) {
  if constexpr (SMOOTH) {
    const Oct w = mul(u, oct_f(s[0], s[1]));
    top = absmax(w, top);
    if (!a.Xn) u = w;
  } else {
    top = absmax(u, top);
  }
}

// Sum and maximum (NaN if a thread has one) over the T threads of a row; every thread gets them. The
// barrier alone does: `red` alternates between two rows' parts.
__device__ __forceinline__ void reduce_row(float& sq, float& top, float (*red)[2][32], uint32_t turn, int T) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  // non-negative floats order like their bit patterns, and the NaN of max_abs3 lies above inf
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
  if (T == 32) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float(*r)[32] = red[turn & 1];
  if (lane == 0) {
    r[0][warp] = sq;
    r[1][warp] = top;
  }
  __syncthreads();
  const bool live = lane < (T >> 5);
  sq = live ? r[0][lane] : 0.0f;
  top = live ? r[1][lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
}

// Scale, Xn and codes of a row whose u are in registers.
template <bool NORM, bool SMOOTH, int V>
__device__ __forceinline__ void finish_row(const RowArgs& a, size_t row, const Oct (&u)[V], float sq, float top) {
  const uint32_t t = threadIdx.x, T = blockDim.x, K = a.K;
  float rstd = 1.0f;
  if constexpr (NORM) rstd = __frcp_rn(__fsqrt_rn(__fdiv_rn(sq, static_cast<float>(a.K)) + a.eps));
  const size_t base = row * K;
  if (a.Xn) {
    __half* xn = a.Xn + base;
    const uint64_t r2 = pair2(rstd, rstd);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t k = 8 * (t + j * T);
      if (k >= K) continue;
      Oct n = u[j];
      if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < 4; ++i) n.v[i] = mul2(n.v[i], r2);
      }
      *reinterpret_cast<uint4*>(xn + k) = pack_h(n);
    }
  }
  if (!a.Xq) return;
  if (t == 0) a.x_scale[row] = top * rstd;
  int8_t* xq = a.Xq + base;
  auto codes = [&](auto make) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t c = 8 * (t + j * T);
      if (c >= K) continue;
      Oct w = u[j];
      if (SMOOTH && a.Xn) w = mul(w, load_oct_f(a.s_rcp + c));
      *reinterpret_cast<uint2*>(xq + c) = make(w);
    }
  };
  if (top >= kTiny && top <= kHuge) {
    const float k = __fdiv_rn(127.0f, top);
    const uint64_t k2 = pair2(k, k);
    codes([&](const Oct& w) {
      float far;
      uint2 q = codes8_near(w, k2, &far);
      if (far > kSure) q = codes8_exact(w, top);
      return q;
    });
  } else {
    codes([&](const Oct& w) { return codes8_div(w, top); });
  }
}

// Few rows, or rows of more than 32768 values: one row per CTA, V vectors of eight
// values per thread.
template <bool NORM, int STREAM, bool SMOOTH, int V>
__global__ void __launch_bounds__(1024) row_kernel(RowArgs a) {
  __shared__ float red[2][2][32];
  const uint32_t t = threadIdx.x, T = blockDim.x, K = a.K;
  griddep_wait();
  griddep_launch_dependents();
  const Row<NORM, STREAM> row(a, blockIdx.x);
  Oct u[V];
  uint64_t sq2 = 0;
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t k = 8 * (t + j * T);
    if (k >= K) continue;
    Raw w;
    float4 s[2];
    const uint4 gamma = load_gamma<NORM>(a, k);
    load_s<SMOOTH>(a, k, s);
    w.x = *static_cast<const uint4*>(row.at(k, 0, K));
    if constexpr (kParts<NORM, STREAM> > 1) w.r0 = *static_cast<const uint4*>(row.at(k, 1, K));
    if constexpr (kParts<NORM, STREAM> > 2) w.r1 = *static_cast<const uint4*>(row.at(k, 2, K));
    u[j] = make_u<NORM, STREAM>(a, row, k, w, gamma, sq2);
    keep_w<SMOOTH>(a, s, u[j], top);
  }
  float sq = split2(sq2).x + split2(sq2).y;
  reduce_row(sq, top, red, 0, T);
  finish_row<NORM, SMOOTH, V>(a, blockIdx.x, u, sq, top);
}

// Many rows: the CTAs stay and take every gridDim.x-th row. What a thread reads
// comes through a ring in shared memory that is its own, two or three vectors ahead
// and on into the next rows, so that loads are in flight while a row is reduced
// and coded; no other thread touches the ring, so it needs no barrier. With the
// loads seen to, the instructions bound both operators, SwiGLU most: hence the
// paired fp32 arithmetic, 32-bit offsets, and codes and gates without divisions.
// Three deep where a vector is 48 bytes: what L1 has left then holds gamma and s_rcp.
template <int P>
constexpr int kDepth = P == 3 ? 3 : 4;

template <bool NORM, int STREAM, bool SMOOTH, int V>
__global__ void __launch_bounds__(V == 4 ? 1024 : V == 2 && SMOOTH ? 512 : 32) row_stream_kernel(RowArgs a) {
  extern __shared__ __align__(16) uint4 ring[];   // [depth][parts][T]
  __shared__ float red[2][2][32];
  constexpr int P = kParts<NORM, STREAM>;
  const uint32_t t = threadIdx.x, T = blockDim.x, K = a.K;
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t M = a.M;
  uint32_t next = blockIdx.x;   // row and vector of the next copy
  uint32_t nk = 8 * t;
  Row<NORM, STREAM> ahead(a, next);
  const uint32_t stage = P * T * 16, mine = smem_addr(ring + t), end = mine + kDepth<P> * stage;
  // An fp32 residual, and H: 32 bytes per thread, side by side. The lanes of a warp
  // move them as 64 pieces of 16 bytes, lane and lane + 32, so that an access of the
  // warp is 512 bytes in a row; each lane's own 32 lie at wide + 16 t.
  const uint32_t lane = t & 31, wide = T * 16;
  const uint32_t piece = 4 * lane;                       // columns from the warp's first
  uint32_t put = mine, got = mine;
  auto fetch = [&]() {
    if constexpr (P == 3) {
      __syncwarp();                                      // the stage's last vectors are out of it
      const uint32_t k0 = nk - 8 * lane;                 // the warp's first column
      const uint32_t to = put + wide + 16 * (t - lane);  // put is at 16 t already
      if (next < M) {
        if (nk < K) cp_async16(put, ahead.at(nk, 0, K), 16);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (k0 + piece + 128 * i < K) cp_async16(to + 512 * i, ahead.r + 4 * (k0 + piece + 128 * i), 16);
      }
    } else if (next < M && nk < K) {
#pragma unroll
      for (int i = 0; i < P; ++i) cp_async16(put + i * wide, ahead.at(nk, i, K), 16);
    }
    cp_async_commit();
    put = put + stage == end ? mine : put + stage;
    nk += 8 * T;
    if (nk >= 8 * T * V) {
      nk = 8 * t;
      next += gridDim.x;
      ahead = Row<NORM, STREAM>(a, next);
    }
  };
#pragma unroll
  for (int i = 0; i < kDepth<P> - 1; ++i) fetch();
  // With s_rcp a thread keeps its columns' gamma and s_rcp in registers: read again
  // for each row they were as much traffic from L1 as the row itself.
  constexpr bool kHold = SMOOTH && V == 2;
  uint4 g_held[V];
  float4 s_held[V][2];
  if constexpr (kHold) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (8 * (t + j * T) < K) {
        g_held[j] = load_gamma<NORM>(a, 8 * (t + j * T));
        load_s<SMOOTH>(a, 8 * (t + j * T), s_held[j]);
      }
  }
  uint32_t turn = 0;
  for (uint32_t r = blockIdx.x; r < M; r += gridDim.x, ++turn) {
    const Row<NORM, STREAM> row(a, r);
    Oct u[V];
    uint64_t sq2 = 0;
    float top = 0.0f;
    // gamma comes from L1 or L2, one vector ahead of its use
    uint4 gamma = make_uint4(0, 0, 0, 0), after = gamma;
    if (!kHold && 8 * t < K) gamma = load_gamma<NORM>(a, 8 * t);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float4 s[2];
      if (!kHold) {
        if (j + 1 < V && 8 * (t + (j + 1) * T) < K) after = load_gamma<NORM>(a, 8 * (t + (j + 1) * T));
        if (8 * (t + j * T) < K) load_s<SMOOTH>(a, 8 * (t + j * T), s);
      }
      fetch();
      cp_async_wait<kDepth<P> - 1>();
      const uint32_t k = 8 * (t + j * T);
      const uint32_t from = got;
      got = got + stage == end ? mine : got + stage;
      const uint32_t own = from + wide + 16 * t;         // P == 3
      if constexpr (P == 3) __syncwarp();                // the other lanes' copies
      if (k < K) {
        Raw w;
        w.x = lds16(from);
        if constexpr (P == 2) w.r0 = lds16(from + wide);
        if constexpr (P == 3) {
          w.r0 = lds16(own);
          w.r1 = lds16(own + 16);
        }
        u[j] = make_u<NORM, STREAM>(a, row, k, w, kHold ? g_held[j] : gamma, sq2, P == 3 ? own : 0);
        keep_w<SMOOTH>(a, kHold ? s_held[j] : s, u[j], top);
      }
      if constexpr (P == 3) {
        if (row.H) {
          __syncwarp();
          const uint32_t k0 = k - 8 * lane;
          const uint32_t at = from + wide + 16 * (t - lane);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (k0 + piece + 128 * i < K)
              *reinterpret_cast<uint4*>(row.H + 4 * (k0 + piece + 128 * i)) = lds16(at + 512 * i);
        }
      }
      gamma = after;
    }
    float sq = split2(sq2).x + split2(sq2).y;
    reduce_row(sq, top, red, turn, T);
    finish_row<NORM, SMOOTH, V>(a, r, u, sq, top);
  }
  cp_async_wait<0>();
}

cudaError_t launch_pdl(const void* kernel, int grid, int block, int smem, const RowArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<RowArgs*>(&a)};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

template <bool NORM, int STREAM, bool SMOOTH, int V>
cudaError_t launch_stream_as(const RowArgs& a, int T, int sms, int dev, cudaStream_t s) {
  const void* kernel = reinterpret_cast<const void*>(row_stream_kernel<NORM, STREAM, SMOOTH, V>);
  const int bytes = kDepth<kParts<NORM, STREAM>> * kParts<NORM, STREAM> * 16;   // of the ring, per thread
  static int resident[64][33] = {};   // CTAs per SM, by device and warps
  int per = dev < 64 ? resident[dev][T / 32] : 0;
  if (per == 0) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         bytes * (V == 4 ? 1024 : V == 2 && SMOOTH ? 512 : 32));
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, T, bytes * T);
    if (e != cudaSuccess) return e;
    if (per < 1) per = 1;
    if (dev < 64) resident[dev][T / 32] = per;
  }
  const int grid = a.M < sms * per ? a.M : sms * per;
  return launch_pdl(kernel, grid, T, bytes * T, a, s);
}

template <bool NORM, int STREAM, bool SMOOTH>
cudaError_t launch_rows_as(const RowArgs& a, cudaStream_t s) {
  const int nv = a.K / 8;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count(dev);
  auto threads = [&](int V) { return ((nv + V - 1) / V + 31) / 32 * 32; };
  if (a.M > kRowPerCta * sms && a.K <= 32768) {
    if (nv <= 32) return launch_stream_as<NORM, STREAM, SMOOTH, 1>(a, threads(1), sms, dev, s);
    if (nv <= (SMOOTH ? 1024 : 64)) return launch_stream_as<NORM, STREAM, SMOOTH, 2>(a, threads(2), sms, dev, s);
    return launch_stream_as<NORM, STREAM, SMOOTH, 4>(a, threads(4), sms, dev, s);
  }
  auto one = [&](auto kernel, int V) {
    return launch_pdl(reinterpret_cast<const void*>(kernel), a.M, threads(V), 0, a, s);
  };
  if (nv <= 1024) return one(row_kernel<NORM, STREAM, SMOOTH, 1>, 1);
  if (nv <= 4096) return one(row_kernel<NORM, STREAM, SMOOTH, 4>, 4);
  return one(row_kernel<NORM, STREAM, SMOOTH, 8>, 8);
}

template <bool NORM, int STREAM>
cudaError_t launch_rows(const RowArgs& a, cudaStream_t s) {
  return a.s_rcp ? launch_rows_as<NORM, STREAM, true>(a, s) : launch_rows_as<NORM, STREAM, false>(a, s);
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

}  // namespace i8mm

using namespace i8mm;

extern "C" {

int int8_rmsnorm_quantize_rows(const void* X, const void* residual, int residual_fp32,
                               const void* gamma, const float* s_rcp, int M, int K, float eps,
                               void* H, void* Xn, int8_t* Xq, float* x_scale,
                               i8mm_stream_t stream) {
  int st = abi_check_sizes(M, 1, K);
  if (st != I8MM_OK) return st;
  if (!(eps > 0.0f) || std::isinf(eps)) return I8MM_ERR_INVALID_ARG;
  if (M == 0) return I8MM_OK;
  if (!X || !gamma || (!Xn && !Xq) || (!Xq) != (!x_scale) || (H && !residual))
    return I8MM_ERR_INVALID_ARG;
  if (!a16(X) || !a16(residual) || !a16(gamma) || !a16(s_rcp) || !a16(H) || !a16(Xn) || !a16(Xq) ||
      !a16(x_scale))
    return I8MM_ERR_ALIGNMENT;
  if ((st = abi_check_device()) != I8MM_OK) return st;
  RowArgs a{};
  a.X = static_cast<const __half*>(X);
  a.residual = residual;
  a.gamma = static_cast<const __half*>(gamma);
  a.s_rcp = s_rcp;
  a.H = H;
  a.Xn = static_cast<__half*>(Xn);
  a.Xq = Xq;
  a.x_scale = x_scale;
  a.M = M;
  a.K = K;
  a.eps = eps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = !residual        ? launch_rows<true, kNone>(a, s)
                        : !residual_fp32 ? launch_rows<true, kF16>(a, s)
                                         : launch_rows<true, kF32>(a, s);
  return abi_cuda_fail("row_kernel (RMS norm) launch", e);
}

int int8_swiglu_quantize_rows(const void* GU, const float* s_rcp, int M, int I, void* Z, int8_t* Zq,
                              float* z_scale, i8mm_stream_t stream) {
  int st = abi_check_sizes(M, 1, I);
  if (st != I8MM_OK) return st;
  if (M == 0) return I8MM_OK;
  if (!GU || (!Z && !Zq) || (!Zq) != (!z_scale)) return I8MM_ERR_INVALID_ARG;
  if (!a16(GU) || !a16(s_rcp) || !a16(Z) || !a16(Zq) || !a16(z_scale)) return I8MM_ERR_ALIGNMENT;
  if ((st = abi_check_device()) != I8MM_OK) return st;
  RowArgs a{};
  a.X = static_cast<const __half*>(GU);
  a.s_rcp = s_rcp;
  a.Xn = static_cast<__half*>(Z);
  a.Xq = Zq;
  a.x_scale = z_scale;
  a.M = M;
  a.K = I;
  return abi_cuda_fail("row_kernel (SwiGLU) launch",
                       launch_rows<false, kNone>(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
