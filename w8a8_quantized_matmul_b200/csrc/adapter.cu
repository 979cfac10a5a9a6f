// Low-rank adapters of many requests beside a shared projection:
//
//   Y[i] = fp16( Y0[i] + scaling[a] * B[a] (A[a] x_i) ),  a = adapter_idx[i]
//
// A token whose index lies outside [0, n_adapters) has no adapter: Y[i] = Y0[i].
// The work is bound by memory (x, Y0 and Y once each, the used adapters once),
// for few tokens by latency, so both halves group the tokens of one adapter and
// read its weights once for the group:
//   shrink   t_i = A[a] x_i, fp32 sums; K is split over CTAs
//   expand   Y[i] = Y0[i] + f_i * B[a] t'_i
// t' = t * 2^-e, e the exponent of the token's largest |t|, and f = scaling * 2^e:
// t' is then within (-1, 1] whatever the inputs' range. It enters the second
// product as two fp16 parts, hi = fp16(t') and lo = fp16(t' - hi), so that what
// is lost of it is below 2^-22 of the token's largest t; one part alone would
// lose 2^-12, as much as the rounding of Y. Sums are fp32 throughout, and none
// depends on the order of the tokens or of the CTAs.
//
// Two forms, by the number of tokens:
//
// Few tokens (small_tokens): groups of up to 16 tokens, mma.sync m16n8k16 with the
//   adapter's rows as its 16-row operand. Fragments are loaded straight from
//   global memory (shrink) or a ring in shared memory (expand), 16 bytes per lane: a
//   lane's eight consecutive halves are used as the k slots of two MMAs, the same for
//   both operands, so the sum over k is only reordered. Every CTA finds its group
//   itself from adapter_idx (a warp walks the indices once), and the expand kernel
//   does so, and asks for its part of B and Y0, while the shrink kernel still runs
//   (programmatic dependent launch). 16 tokens, 4096 x 4096, rank 16: 5.0 us, of
//   which two kernels' latency is nearly all; 201 x 4112 x 10007, rank 8: 19 us.
//
// Larger M: a plan kernel sorts the tokens by adapter into tiles of up to 128;
//   shrink and expand run on tcgen05 (M = 128). 4096 tokens, 8192 x 28672, rank 64:
//   134 us in a CUDA graph (profiled by itself: plan 6, shrink 25, expand 105 to 110);
//   the bytes that have to move take 88 us at the copy rate.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "int8mm.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "quant_common.cuh"

namespace i8mm {

namespace {

constexpr int kMaxRank = 128;
constexpr int kMaxAdapters = 4096;
constexpr int kMaxSmallTokens = 1024;
// Up to this many tokens the form of groups of 16 is the faster one. Its products
// go through mma.sync and its groups read B again for every 16 tokens, so that the
// larger the rank the sooner the tiles of 128 win, and the more adapters there are
// (tiles mostly empty) the later. Measured, us (groups / tiles; K x N, rank, adapters):
//    768 tokens  4096 x 4096, 16, 4    24 / 23      768 tokens  8192 x 28672, 16, 4     51 / 52
//   1024 tokens  4096 x 4096, 16, 4    26 / 24     1024 tokens  8192 x 28672, 16, 4     60 / 53
//   1024 tokens  4096 x 4096, 16, 48   43 / 38     1024 tokens  8192 x 28672, 16, 48    90 / 114
//   1024 tokens  4096 x 4096, 16, 128  50 / 62     1024 tokens  8192 x 28672, 16, 128  110 / 247
//    384 tokens  4096 x 4096, 32, 4    15 / 21      384 tokens  8192 x 28672, 32, 4     40 / 40
//    512 tokens  4096 x 4096, 32, 4    23 / 22      512 tokens  8192 x 28672, 32, 4     49 / 38
//    512 tokens  4096 x 4096, 32, 48   28 / 33      512 tokens  8192 x 28672, 32, 48    74 / 103
//    256 tokens  8192 x 28672, 64, 4   45 / 37      128 tokens  8192 x 28672, 64, 24    53 / 67
//     32 tokens  4096 x 4096, 128, 4   19 / 22       32 tokens  8192 x 28672, 128, 24  101 / 79
constexpr int small_tokens(int R, int n) {
  return R <= 16 ? (n < 32 ? 768 : kMaxSmallTokens) : R <= 32 ? (n < 16 ? 384 : 512) : R <= 64 ? 192 : 16;
}

struct AdapterArgs {
  const __half* X;       // [M][K]
  const __half* A;       // [n][R][K]
  const __half* B;       // [n][N][R]
  const int32_t* idx;    // [M]
  const float* scaling;  // [n]
  const __half* Y0;      // [M][N]
  __half* Y;             // [M][N], may be Y0
  int M, N, K, n, R;
  int32_t* head;         // workspace: [0] tiles of the plan, [1] device status, [2] tiles with an adapter
  // few tokens
  float* part;           // [S][M][R] partial t over the S slices of K
  int S, slice;          // slices of K and their width
  // larger M
  int4* tiles;           // {adapter or -1, first row, rows, 0} in plan order
  int32_t* perm;         // [M] token of each plan row
  float* factor;         // [M] f of each plan row
  __half *hi, *lo;       // [M][R] t' of each plan row
  int cluster;           // CTAs per cluster of the shrink kernel: 1, 2, 4 or 8
};

// The adapter of a token, -1 for none.
__device__ __forceinline__ int adapter_of(const AdapterArgs& p, int i) {
  const int a = __ldcg(p.idx + i);
  return a >= 0 && a < p.n ? a : -1;
}

// 2^-e and 2^e for e with 2^(e-1) <= m < 2^e (1 and 1 for m = 0 or where m is
// not a normal number of moderate size).
__device__ __forceinline__ void power_pair(float m, float* down, float* up) {
  int e = static_cast<int>(__float_as_uint(m) >> 23) - 126;
  if (m == 0.0f || e < -100 || e > 100) e = m == 0.0f ? 0 : max(-100, min(100, e));
  *down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  *up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// ---------------------------------------------------------------- few tokens
constexpr int kChunk = 16;            // tokens of a group
constexpr int kSmallThreads = 128;
constexpr int kMaxSlices = 16;        // of K
constexpr int kNBlock = 256;          // columns of Y per expand CTA, 64 per warp

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The group of a CTA: the g-th of the groups that the tokens form when every
// adapter's tokens (and those without one), in order, are cut into kChunk.
struct Group {
  int adapter;            // -1: tokens without an adapter
  int count;              // 0: there is no g-th group
  int token[kChunk];
};

// All threads of a CTA call find_group. which(groups): the CTA's group of that many (0
// unless COUNT), asked of all warps. One warp's worth of tokens needs no more than the
// warp's votes; more are walked to the CTA's group, with each adapter's tokens so far in
// seen ([n + 1] ints of shared memory).
__device__ __forceinline__ void clear_seen(const AdapterArgs& p, int* seen) {
  for (int i = threadIdx.x; i <= p.n; i += kSmallThreads) seen[i] = 0;
  __syncthreads();
}
__device__ __forceinline__ void fetch_adapters(const AdapterArgs& p, int16_t* adapter) {
#pragma unroll
  for (int i = 0; i < kMaxSmallTokens; i += kSmallThreads)
    if (i + static_cast<int>(threadIdx.x) < p.M)
      adapter[i + threadIdx.x] = static_cast<int16_t>(adapter_of(p, i + threadIdx.x));
}
__device__ __forceinline__ int count_groups(const AdapterArgs& p, const int16_t* adapter, int* seen) {
  clear_seen(p, seen);
  int groups = 0;
  for (int i0 = 0; i0 < p.M; i0 += kSmallThreads) {
    const int i = i0 + threadIdx.x;
    bool head = false;                     // whichever token it is, every kChunk-th opens a group
    if (i < p.M) head = atomicAdd(&seen[adapter[i] < 0 ? p.n : adapter[i]], 1) % kChunk == 0;
    groups += __syncthreads_count(head);
  }
  return groups;
}
template <bool COUNT, class Which>
__device__ __forceinline__ void find_group(const AdapterArgs& p, Which which, int* seen, Group* out) {
  __shared__ int16_t adapter[kMaxSmallTokens];
  if (p.M <= 32) {
    const int lane = threadIdx.x & 31;
    const int a = lane < p.M ? adapter_of(p, lane) : -2;
    const int rank = __popc(__match_any_sync(0xffffffffu, a) & ((1u << lane) - 1u));
    const uint32_t heads = __ballot_sync(0xffffffffu, a != -2 && rank % kChunk == 0);
    const int g = which(__popc(heads));
    if (threadIdx.x < 32) {
      int want = -2, first = 0;
      if (g < __popc(heads)) {
        const uint32_t src = __fns(heads, 0, g + 1);
        want = __shfl_sync(0xffffffffu, a, src);
        first = __shfl_sync(0xffffffffu, rank, src);
      }
      const bool mine = want != -2 && a == want && rank >= first && rank < first + kChunk;
      if (mine) out->token[rank - first] = lane;
      const int count = __popc(__ballot_sync(0xffffffffu, mine));
      if (lane == 0) {
        out->adapter = want;
        out->count = count;
      }
    }
    __syncthreads();
    return;
  }
  fetch_adapters(p, adapter);
  int all = 0;
  if constexpr (COUNT) all = count_groups(p, adapter, seen);
  const int g = which(all);
  clear_seen(p, seen);
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int groups = 0, want = -2, first = 0, count = 0;   // want: the adapter, once found
    for (int i0 = 0; i0 < p.M; i0 += 32) {
      const int i = i0 + lane;
      const bool live = i < p.M;
      const int a = live ? adapter[i] : -2;
      const uint32_t same = __match_any_sync(0xffffffffu, a);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int slot = a < 0 ? p.n : a;
      const int rank = live ? seen[slot] + before : 1;
      __syncwarp();
      if (live && before == 0) seen[slot] = rank + __popc(same);
      __syncwarp();
      if (want == -2) {
        const uint32_t heads = __ballot_sync(0xffffffffu, live && rank % kChunk == 0);
        if (groups + __popc(heads) > g) {
          const uint32_t src = __fns(heads, 0, g - groups + 1);
          want = __shfl_sync(0xffffffffu, a, src);
          first = __shfl_sync(0xffffffffu, rank, src);
        }
        groups += __popc(heads);
      }
      if (want != -2) {
        const bool mine = live && a == want && rank >= first && rank < first + kChunk;
        if (mine) out->token[rank - first] = i;
        count += __popc(__ballot_sync(0xffffffffu, mine));
        if (count == kChunk) break;
      }
    }
    if (lane == 0) {
      out->adapter = want;
      out->count = count;
    }
  }
  __syncthreads();
}

// Grid (S, groups). MT: 16-row tiles of the adapter's R rows.
template <int MT>
__global__ void __launch_bounds__(kSmallThreads) small_shrink_kernel(AdapterArgs p) {
  extern __shared__ __align__(16) uint8_t small_smem[];
  __shared__ Group grp;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.head[1] = 0;
  find_group<false>(p, [](int) { return static_cast<int>(blockIdx.y); }, reinterpret_cast<int*>(small_smem), &grp);
  const int count = grp.count, a = grp.adapter;
  if (count == 0 || a < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int sub = p.slice / 4;                                   // columns of a warp
  const int k0 = blockIdx.x * p.slice + warp * sub;
  const int k1 = min(p.K, min(k0 + sub, static_cast<int>(blockIdx.x + 1) * p.slice));
  const __half* x[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    x[j] = p.X + static_cast<size_t>(grp.token[min(8 * j + g, count - 1)]) * p.K;
  const __half* w = p.A + static_cast<size_t>(a) * p.R * p.K;
  float d[MT][2][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll(MT <= 2 ? 4 : MT == 4 ? 2 : 1)
  for (int k = k0; k < k1; k += 32) {
    const int c = k + 8 * t;
    const bool in = c < k1;
    uint4 xv[2], av[MT][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      xv[j] = in && 8 * j + g < count ? __ldg(reinterpret_cast<const uint4*>(x[j] + c)) : zero;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * i + 8 * h + g;
        av[i][h] = in && r < p.R ? __ldg(reinterpret_cast<const uint4*>(w + static_cast<size_t>(r) * p.K + c)) : zero;
      }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const uint32_t f0[4] = {av[i][0].x, av[i][1].x, av[i][0].y, av[i][1].y};
      const uint32_t f1[4] = {av[i][0].z, av[i][1].z, av[i][0].w, av[i][1].w};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mma16816(d[i][j], f0, xv[j].x, xv[j].y);
        mma16816(d[i][j], f1, xv[j].z, xv[j].w);
      }
    }
  }
  // Sum over the four warps (in their order), [token][row] in shared memory.
  float* red = reinterpret_cast<float*>(small_smem);             // [4][kChunk][16 * MT + 1]
  constexpr int ld = 16 * MT + 1;
  __syncthreads();                                               // `seen` is no longer read
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        red[(warp * kChunk + 8 * j + 2 * t + (e & 1)) * ld + 16 * i + g + 8 * (e >> 1)] = d[i][j][e];
  __syncthreads();
  for (int e = threadIdx.x; e < count * p.R; e += kSmallThreads) {
    const int tok = e / p.R, r = e - tok * p.R;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < 4; ++v) s += red[(v * kChunk + tok) * ld + r];
    p.part[(static_cast<size_t>(blockIdx.x) * p.M + grp.token[tok]) * p.R + r] = s;
  }
}

// Where N is not a multiple of 8 the rows of Y lie at any 2-byte address. A warp then
// moves a row of a CTA's 16 x 256 piece with one 16-byte access per lane between the
// first and the last such address inside it, and the up to seven values on either
// side one by one; B t' comes to these lanes through shared memory, column c of a
// token at (c % 8) * 33 + c / 8, so that lanes 8 columns apart meet different banks
// wherever the row begins. (Y0 and Y through shared memory at their columns, 2 bytes a
// time, took a third longer.)
constexpr int kSpreadLd = 8 * 33;

struct RowPart {
  int vec, edge;          // columns of this lane's vector and of its single value, or -1
};
__device__ __forceinline__ RowPart row_part(size_t at, int n, int lane) {   // Y and Y0 are 16-byte aligned
  const int head = min(n, static_cast<int>((8 - (at & 7)) & 7));
  const int vecs = (n - head) / 8;
  const int tail = head + 8 * vecs;
  RowPart r;
  r.vec = lane < vecs ? head + 8 * lane : -1;
  r.edge = lane < head ? lane : lane >= 8 && lane < 15 && tail + lane - 8 < n ? tail + lane - 8 : -1;
  return r;
}

// Stages of the ring that a warp of the expand kernel has for itself.
template <int RB>
constexpr int kExpandDepth = RB < 1 ? 3 : 2;

// The CTAs are shared out among the groups that there are (the host only has a bound:
// of a stack of 1000 adapters a batch may use four; 512 x 8192 x 28672, rank 16, so: 189 us
// with the CTAs dealt out to the possible groups, 52 so): a group's CTAs take its
// blocks of columns in turn. RB:
// 32-wide blocks of R, 0 for R <= 16 (a lane then holds four consecutive halves of
// a row, the k slots of one MMA); VEC: N a multiple of 8. What a warp reads of B, and
// of Y0 where VEC, comes through a ring in shared memory that is its own, one or two blocks ahead.
template <int RB, bool VEC>
__global__ void __launch_bounds__(kSmallThreads) small_expand_kernel(AdapterArgs p) {
  extern __shared__ __align__(16) uint8_t small_smem[];
  __shared__ Group grp;
  __shared__ float fac[kChunk];
  __shared__ float spread[VEC ? 1 : kChunk * kSpreadLd];
  constexpr int D = kExpandDepth<RB>;
  constexpr bool HALF = RB == 0;
  constexpr int kWide = HALF ? 16 : 32 * RB;                     // R, padded
  griddep_launch_dependents();
  // The shrink kernel lets this one start only after its own wait, so everything
  // before it is complete: only what it writes itself (part) has to be waited for.
  // What is read before that goes past L1. Every CTA waits before it ends, so that
  // this kernel never ends before the shrink kernel.
  const int b_bytes = 128 * p.R;                                 // of a stage, per warp: 64 rows
  const int stage_bytes = 4 * b_bytes + (VEC ? 64 * kSmallThreads : 0);
  float* ts = reinterpret_cast<float*>(small_smem + D * stage_bytes);   // [kChunk][kWide + 4]
  constexpr int ld = kWide + 4;
  // the two parts of t', [kChunk][kWide + 8] halves each
  __half* parts = reinterpret_cast<__half*>(ts + kChunk * ld);
  constexpr int ldp = kWide + 8;
  const int blocks = (p.N + kNBlock - 1) / kNBlock;
  int columns = 1, first = 0;              // CTAs of a group, this one's place among them
  find_group<true>(p, [&](int groups) {
    const int most = max(1, static_cast<int>(gridDim.x) / groups);
    const int share = (blocks - 1) / min(blocks, most) + 1;     // no CTA has more blocks than this
    columns = (blocks - 1) / share + 1;
    const int g = blockIdx.x / columns;
    first = blockIdx.x - g * columns;
    return g;
  }, reinterpret_cast<int*>(ts), &grp);
  // The same in all lanes, and said so: where the compiler cannot tell, a block of rank 64
  // takes 2 us longer (32 tokens, 4096 x 4096: 13.2 us against 11.3).
  columns = __shfl_sync(0xffffffffu, columns, 0);
  first = __shfl_sync(0xffffffffu, first, 0);
  const int count = grp.count, a = grp.adapter;
  if (count == 0 || (a < 0 && p.Y == p.Y0)) {
    griddep_wait();
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  size_t at[4];                                                  // rows of the lane's four tokens
#pragma unroll
  for (int j = 0; j < 4; ++j)
    at[j] = static_cast<size_t>(grp.token[min(8 * (j >> 1) + 2 * t + (j & 1), count - 1)]) * p.N;
  const bool two = count > 8;                                    // a second tile of eight tokens
  const uint32_t ring = smem_addr(small_smem);
  auto y_slot = [&](int stg, int j) {
    return ring + stg * stage_bytes + 4 * b_bytes + (j * kSmallThreads + threadIdx.x) * 16;
  };
  // A warp's 64 rows of B are contiguous. They are copied in 16-byte pieces by the
  // whole warp; piece c goes to c with its low three bits XORed by its row / 8, so that
  // the eight lanes g, which read rows 8 apart, meet different banks.
  const int row_pieces = p.R >> 3;
  auto b_piece = [&](int row, int kc) {                          // byte offset in the warp's part
    return ((row * row_pieces + kc) ^ ((row >> 3) & 7)) * 16;
  };
  // Of a block: the lane's eight consecutive columns n0 .. are rows n0 + 2i + h of B for
  // (tile i, half h); with Y0 of these and the lane's four tokens: 2t, 2t + 1, 8 + 2t,
  // 8 + 2t + 1.
  const int8_t* bsrc = reinterpret_cast<const int8_t*>(p.B + static_cast<size_t>(max(a, 0)) * p.N * p.R);
  auto fetch = [&](int blk, int stg) {
    const int w0 = blk * kNBlock + warp * 64, n0 = w0 + 8 * g;
    __syncwarp();                                                // the stage has been read
    if (blk < blocks && w0 < p.N) {
      if (a >= 0) {
        const int pieces = min(64, p.N - w0) * row_pieces;
        const int8_t* from = bsrc + static_cast<size_t>(w0) * (2 * p.R);
        const uint32_t to = ring + stg * stage_bytes + warp * b_bytes;
        for (int c = lane; c < pieces; c += 32)
          cp_async16(to + ((c ^ ((c / p.R) & 7)) << 4), from + 16 * c, 16u);   // c / R = row / 8
      }
      if constexpr (VEC) {
        if (n0 < p.N) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (8 * (j >> 1) + 2 * t + (j & 1) < count) cp_async16(y_slot(stg, j), p.Y0 + at[j] + n0, 16u);
        }
      }
    }
    cp_async_commit();
  };
  // not VEC: rows warp, warp + 4, .. of Y0, a block ahead in registers
  uint4 yv[VEC ? 1 : kChunk / 4];
  __half ye[VEC ? 1 : kChunk / 4];
  auto rows = [&](int blk, auto act) {
    const int n0 = blk * kNBlock, n = min(kNBlock, p.N - n0);
#pragma unroll
    for (int i = 0; i < kChunk / 4; ++i) {
      const int tok = warp + 4 * i;
      if (tok < count) {
        const size_t from = static_cast<size_t>(grp.token[tok]) * p.N + n0;
        act(i, from, row_part(from, n, lane), tok);
      }
    }
  };
  auto fetch_rows = [&](int blk) {
    if constexpr (!VEC) {
      if (blk < blocks)
        rows(blk, [&](int i, size_t from, RowPart q, int) {
          if (q.vec >= 0) yv[i] = __ldcg(reinterpret_cast<const uint4*>(p.Y0 + from + q.vec));
          if (q.edge >= 0) ye[i] = __ldcg(p.Y0 + from + q.edge);
        });
    }
  };
  fetch_rows(first);
#pragma unroll
  for (int i = 0; i < D - 1; ++i) fetch(first + i * columns, i);
  griddep_wait();
  if (a >= 0) {
    // t of the group: the slices of K in order, then the token's power of two.
    __syncthreads();                                             // `seen` is no longer read
    for (int e = threadIdx.x; e < kChunk * kWide; e += kSmallThreads) {
      const int tok = e / kWide, r = e - tok * kWide;
      float s = 0.0f;
      if (tok < count && r < p.R) {
        const float* q = p.part + static_cast<size_t>(grp.token[tok]) * p.R + r;
        float f[kMaxSlices];
#pragma unroll
        for (int v = 0; v < kMaxSlices; ++v)
          f[v] = v < p.S ? __ldcg(q + static_cast<size_t>(v) * p.M * p.R) : 0.0f;
#pragma unroll
        for (int v = 0; v < kMaxSlices; ++v) s += f[v];
      }
      ts[tok * ld + r] = s;
    }
    __syncthreads();
    // Every eight threads take a token's maximum.
    const int tok = threadIdx.x >> 3;
    float m = 0.0f;
    for (int r = threadIdx.x & 7; r < kWide; r += 8) m = fmaxf(m, fabsf(ts[tok * ld + r]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float down, up;
    power_pair(m, &down, &up);
    for (int r = threadIdx.x & 7; r < kWide; r += 8) {
      const float f = ts[tok * ld + r] * down;
      const __half h = __float2half_rn(f);
      parts[tok * ldp + r] = h;
      parts[(kChunk + tok) * ldp + r] = __float2half_rn(f - __half2float(h));
    }
    if ((threadIdx.x & 7) == 0) fac[tok] = p.scaling[a] * up;
    __syncthreads();
  }
  // Where the lane's rows of B lie in the warp's part (for R > 64 worked out each time).
  constexpr int kOff = RB == 2 ? 2 : 1;
  uint32_t b_off[kOff][8];
#pragma unroll
  for (int rb = 0; rb < kOff; ++rb)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      b_off[rb][i] = HALF ? b_piece(8 * g + i, t >> 1) + 8 * (t & 1) : b_piece(8 * g + i, 4 * rb + t);
  const uint32_t parts_at = smem_addr(parts);
  int stg = 0;
  for (int blk = first; blk < blocks; blk += columns) {
    fetch(blk + (D - 1) * columns, stg == 0 ? D - 1 : stg - 1);
    cp_async_wait<D - 1>();
    __syncwarp();                                                // the other lanes' pieces
    const int n0 = blk * kNBlock + warp * 64 + 8 * g;
    const uint32_t b_at = ring + stg * stage_bytes + warp * b_bytes;
    float d[4][2][4] = {};
    if (a >= 0) {
      constexpr int kPairs = HALF ? 2 : 4;                       // pairs of a lane's halves of t'
#pragma unroll
      for (int rb = 0; rb < (HALF ? 1 : RB); ++rb) {
        uint32_t hi[2][kPairs], lo[2][kPairs];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (j == 1 && !two) continue;
          const uint32_t q = parts_at + ((8 * j + g) * ldp + 32 * rb + 2 * kPairs * t) * 2;
          if constexpr (HALF) {
            const uint2 u = lds8(q), v = lds8(q + kChunk * ldp * 2);
            hi[j][0] = u.x, hi[j][1] = u.y, lo[j][0] = v.x, lo[j][1] = v.y;
          } else {
            const uint4 u = lds16(q), v = lds16(q + kChunk * ldp * 2);
            hi[j][0] = u.x, hi[j][1] = u.y, hi[j][kPairs - 2] = u.z, hi[j][kPairs - 1] = u.w;
            lo[j][0] = v.x, lo[j][1] = v.y, lo[j][kPairs - 2] = v.z, lo[j][kPairs - 1] = v.w;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (HALF) {
            uint2 u = make_uint2(0, 0), v = u;                   // zeros past R
            if (4 * t < p.R) {
              u = lds8(b_at + b_off[0][2 * i]);
              v = lds8(b_at + b_off[0][2 * i + 1]);
            }
            const uint32_t f0[4] = {u.x, v.x, u.y, v.y};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (j == 1 && !two) continue;
              mma16816(d[i][j], f0, hi[j][0], hi[j][1]);
              mma16816(d[i][j], f0, lo[j][0], lo[j][1]);
            }
          } else {
            uint4 u = make_uint4(0, 0, 0, 0), v = u;
            if (32 * rb + 8 * t < p.R) {
              u = lds16(b_at + (RB <= 2 ? b_off[rb % kOff][2 * i] : b_piece(8 * g + 2 * i, 4 * rb + t)));
              v = lds16(b_at + (RB <= 2 ? b_off[rb % kOff][2 * i + 1] : b_piece(8 * g + 2 * i + 1, 4 * rb + t)));
            }
            const uint32_t f0[4] = {u.x, v.x, u.y, v.y};
            const uint32_t f1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (j == 1 && !two) continue;
              mma16816(d[i][j], f0, hi[j][0], hi[j][1]);
              mma16816(d[i][j], f1, hi[j][kPairs - 2], hi[j][kPairs - 1]);
              mma16816(d[i][j], f0, lo[j][0], lo[j][1]);
              mma16816(d[i][j], f1, lo[j][kPairs - 2], lo[j][kPairs - 1]);
            }
          }
        }
      }
    }
    // Tile i holds the columns n0 + 2i (e < 2) and n0 + 2i + 1 of tokens 2t + (e & 1).
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int tok = 8 * (j >> 1) + 2 * t + (j & 1);
        if (tok >= count || n0 >= p.N) continue;
        uint4 y = lds16(y_slot(stg, j));
        if (a >= 0) {
          const float f = fac[tok];
          __half2* h = reinterpret_cast<__half2*>(&y);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(h[i]);
            h[i] = __floats2half2_rn(fmaf(f, d[i][j >> 1][j & 1], v.x),
                                     fmaf(f, d[i][j >> 1][2 + (j & 1)], v.y));
          }
        }
        *reinterpret_cast<uint4*>(p.Y + at[j] + n0) = y;
      }
    } else {
      if (a >= 0) {
        __syncthreads();                                         // the last block's values have been taken
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int tok = 8 * (j >> 1) + 2 * t + (j & 1);
          if (tok >= count) continue;
          float* to = spread + tok * kSpreadLd + 8 * warp + g;
#pragma unroll
          for (int i = 0; i < 8; ++i) to[i * 33] = d[i >> 1][j >> 1][2 * (i & 1) + (j & 1)];
        }
        __syncthreads();
      }
      rows(blk, [&](int i, size_t to, RowPart q, int tok) {
        const float* from = spread + tok * kSpreadLd;
        const float f = a >= 0 ? fac[tok] : 0.0f;
        if (q.vec >= 0) {
          __half* h = reinterpret_cast<__half*>(&yv[i]);
          if (a >= 0)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int c = q.vec + k;
              h[k] = __float2half_rn(fmaf(f, from[(c & 7) * 33 + (c >> 3)], __half2float(h[k])));
            }
          *reinterpret_cast<uint4*>(p.Y + to + q.vec) = yv[i];
        }
        if (q.edge >= 0) {
          const int c = q.edge;
          if (a >= 0) ye[i] = __float2half_rn(fmaf(f, from[(c & 7) * 33 + (c >> 3)], __half2float(ye[i])));
          p.Y[to + c] = ye[i];
        }
      });
      fetch_rows(blk + columns);
    }
    stg = stg + 1 == D ? 0 : stg + 1;
  }
  cp_async_wait<0>();
}

cudaError_t launch_pdl(const void* kernel, dim3 grid, int block, size_t smem, cudaStream_t s,
                       void** args, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

// At most this many groups: one for every kChunk tokens, and one more that is
// not full for every adapter in use and for the tokens without one.
int max_groups(const AdapterArgs& p, int per) {
  const int kinds = p.n + 1 < p.M ? p.n + 1 : p.M;
  return p.M / per + kinds;
}

cudaError_t launch_small(AdapterArgs p, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count(dev);
  const int groups = max_groups(p, kChunk);
  const size_t seen = (static_cast<size_t>(p.n) + 1) * 4;
  const int blocks = (p.N + kNBlock - 1) / kNBlock;
  void* args[] = {&p};
  auto shrink = [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    const size_t red = sizeof(float) * 4 * kChunk * (16 * MT + 1);
    return launch_pdl(reinterpret_cast<const void*>(small_shrink_kernel<MT>), dim3(p.S, groups),
                      kSmallThreads, red > seen ? red : seen, s, args);
  };
  auto expand = [&](auto rb) {
    constexpr int RB = decltype(rb)::value;
    const bool vec = p.N % 8 == 0;
    const size_t wide = RB ? 32 * RB : 16;
    const size_t ts = kChunk * (4 * (wide + 4) + 2 * 2 * (wide + 8));
    const size_t ring = static_cast<size_t>(kExpandDepth<RB>) * (512 * p.R + (vec ? 64 * kSmallThreads : 0));
    const size_t bytes = ring + (ts > seen ? ts : seen);
    const cudaError_t e = vec ? allow_max_smem<small_expand_kernel<RB, true>>()
                              : allow_max_smem<small_expand_kernel<RB, false>>();
    if (e != cudaSuccess) return e;
    // As many CTAs as run at a time (one per possible group at least), each with its
    // share of a group's column blocks: a CTA finds its group and t once.
    const int fit = static_cast<int>(228 * 1024 / (bytes + (vec ? 3 : 20) * 1024));   // by shared memory
    const int at_once = sms * (fit < 1 ? 1 : fit > 5 ? 5 : fit);
    const int64_t most = static_cast<int64_t>(groups) * blocks;
    const int ctas = at_once < groups ? groups : static_cast<int>(at_once < most ? at_once : most);
    return launch_pdl(vec ? reinterpret_cast<const void*>(small_expand_kernel<RB, true>)
                          : reinterpret_cast<const void*>(small_expand_kernel<RB, false>),
                      dim3(ctas), kSmallThreads, bytes, s, args);
  };
  using std::integral_constant;
  e = p.R <= 16   ? shrink(integral_constant<int, 1>{})
      : p.R <= 32 ? shrink(integral_constant<int, 2>{})
      : p.R <= 64 ? shrink(integral_constant<int, 4>{})
                  : shrink(integral_constant<int, 8>{});
  if (e != cudaSuccess) return e;
  return p.R <= 16   ? expand(integral_constant<int, 0>{})
         : p.R <= 32 ? expand(integral_constant<int, 1>{})
         : p.R <= 64 ? expand(integral_constant<int, 2>{})
                     : expand(integral_constant<int, 4>{});
}

// ---------------------------------------------------------------- larger M
constexpr int kTile = 128;             // tokens of a tile
constexpr int kPlanThreads = 1024;

// Sorts the tokens by adapter (those without one last) and cuts each adapter's
// tokens into tiles. One CTA: two passes over the indices around a prefix sum
// over the adapters. The order of an adapter's tokens is left open.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(AdapterArgs p) {
  extern __shared__ __align__(16) uint8_t small_smem[];
  int32_t* count = reinterpret_cast<int32_t*>(small_smem);   // [n + 1], then the next free row
  __shared__ int32_t sums[2][32];
  const int kinds = p.n + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  for (int k = tid; k < kinds; k += kPlanThreads) count[k] = 0;
  __syncthreads();
  // Rows of a warp that share an adapter take their places with one atomic.
  auto fetch = [&](int i) { return i < p.M ? adapter_of(p, i) : -2; };
  auto place = [&](int a) {
    const uint32_t same = __match_any_sync(0xffffffffu, a);
    const int leader = __ffs(same) - 1;
    int at = 0;
    if (lane == leader && a != -2) at = atomicAdd(&count[a < 0 ? p.n : a], __popc(same));
    at = __shfl_sync(0xffffffffu, at, leader);
    return at + __popc(same & ((1u << lane) - 1u));
  };
  const int rounds = (p.M + kPlanThreads - 1) / kPlanThreads;
  constexpr int kHeld = 8;               // indices of a thread that stay in registers
  int held[kHeld];
#pragma unroll
  for (int r = 0; r < kHeld; ++r) held[r] = fetch(r * kPlanThreads + tid);
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r < rounds) place(held[r]);
  for (int r = kHeld; r < rounds; ++r) place(fetch(r * kPlanThreads + tid));
  __syncthreads();
  // Prefix sums over the kinds, in order: tokens and tiles before each.
  const int per = (kinds + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(kinds, tid * per), hi = min(kinds, lo + per);
  int rows = 0, tiles = 0;
  for (int k = lo; k < hi; ++k) {
    rows += count[k];
    tiles += (count[k] + kTile - 1) / kTile;
  }
  int rsum = rows, tsum = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int r = __shfl_up_sync(0xffffffffu, rsum, o), t = __shfl_up_sync(0xffffffffu, tsum, o);
    if (lane >= o) {
      rsum += r;
      tsum += t;
    }
  }
  if (lane == 31) {
    sums[0][warp] = rsum;
    sums[1][warp] = tsum;
  }
  __syncthreads();
  // The warps before this one: each lane one warp's sums.
  int rbefore = lane < warp ? sums[0][lane] : 0, tbefore = lane < warp ? sums[1][lane] : 0;
  const int row_base = __reduce_add_sync(0xffffffffu, rbefore);
  const int tile_base = __reduce_add_sync(0xffffffffu, tbefore);
  int row0 = row_base + rsum - rows, tile0 = tile_base + tsum - tiles;
  for (int k = lo; k < hi; ++k) {
    const int c = count[k];
    if (k == p.n) p.head[2] = tile0;
    for (int j = 0; j < c; j += kTile)
      p.tiles[tile0++] = make_int4(k == p.n ? -1 : k, row0 + j, min(kTile, c - j), 0);
    count[k] = row0;
    row0 += c;
  }
  if (tid == kPlanThreads - 1) {
    p.head[0] = tile0;
    p.head[1] = 0;
  }
  __syncthreads();
  auto put = [&](int r, int a) {
    const int at = place(a);
    if (a != -2) p.perm[at] = r * kPlanThreads + tid;
  };
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r < rounds) put(r, held[r]);
  for (int r = kHeld; r < rounds; ++r) put(r, fetch(r * kPlanThreads + tid));
  griddep_launch_dependents();
}

// Shrink: a team of `split` CTAs of a cluster takes a tile of 128 tokens, each CTA a part of
// K: D[128 tokens][R] = X rows . A[a]^T on tcgen05, 64 columns of K per stage.
// The tokens' rows lie anywhere, so four warps gather them with 16-byte
// asynchronous copies, eight lanes per 128-byte row piece, into the swizzled
// layout that the MMA reads; A comes by TMA. The partial sums are exchanged
// through the cluster's shared memory: each CTA finishes 128 / split tokens. The split is the
// largest whose CTAs are resident at once, by the tiles that there are, not by the host's
// bound on them: one CTA alone on its SM streams 16 KB in 0.73 us (156 CTAs: 3.4 TB/s), 296
// CTAs read 5.7 TB/s between them.
constexpr int kMaxSplit = 8;
constexpr int kShrinkThreads = 160;    // four copying warps (also the epilogue), one for the MMAs
constexpr int kMaxShrinkStages = 6;
constexpr int kXBytes = kTile * 128;

__host__ __device__ constexpr int shrink_tmem(int R) { return R <= 32 ? 32 : R <= 64 ? 64 : 128; }

// CTAs that an SM holds: three stages at least in each.
__host__ __device__ constexpr int shrink_per_sm(int R) { return R <= 64 ? 3 : 2; }

struct ShrinkSmem {
  int stage, stages, part_ld, ring, bars, bytes;
};
__host__ __device__ inline ShrinkSmem shrink_smem(int R) {
  ShrinkSmem L;
  const int rp = (R + 15) / 16 * 16;
  L.stage = kXBytes + rp * 128;
  L.part_ld = rp + 4;                                        // fp32 partials [128][part_ld]
  const int part = kTile * L.part_ld * 4;
  L.stages = (shrink_per_sm(R) == 3 ? 72 : 106) * 1024 / L.stage;
  if (L.stages > kMaxShrinkStages) L.stages = kMaxShrinkStages;
  L.ring = L.stages * L.stage;
  if (L.ring < part) L.ring = part;                          // they take the ring's place
  L.bars = (L.ring + 15) / 16 * 16;
  L.bytes = 1024 + L.bars + (2 * kMaxShrinkStages + 1) * 8 + 32;
  const int least = cluster_tmem_smem(shrink_tmem(R));
  if (L.bytes < least) L.bytes = least;
  return L;
}

// The cluster's CTAs form teams of `split` with a tile each. (With the split a variable
// every call took 1.2 us longer.)
template <int split>
__device__ __forceinline__ void shrink_tiles(const CUtensorMap& tmA, const AdapterArgs& p, const ShrinkSmem& L,
                                             uint8_t* sm, uint32_t tmem, int ntiles) {
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L.bars);
  uint64_t* empty = full + kMaxShrinkStages;
  uint64_t* done = empty + kMaxShrinkStages;
  volatile int32_t* stop = reinterpret_cast<volatile int32_t*>(reinterpret_cast<uint32_t*>(done + 1) + 1);
  float* part = reinterpret_cast<float*>(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t stages = L.stages;
  const int rp = (p.R + 15) / 16 * 16;
  const int nkb = (p.K + 63) / 64;
  const int cluster = blockIdx.x / p.cluster, clusters = gridDim.x / p.cluster;
  const int teams = p.cluster / split;
  const int team = static_cast<int>(cluster_ctarank()) / split;
  const int rank = static_cast<int>(cluster_ctarank()) % split;
  // Blocks rank, rank + split, .. of K: the team's CTAs read neighbouring pieces of
  // a row at about the same time.
  const int blocks = nkb > rank ? (nkb - rank + split - 1) / split : 0;
  uint32_t it = 0;                                           // stages so far
  uint32_t round = 0;                                        // tiles so far with work for this CTA
  // As many turns for every team of a cluster, the last ones without a tile for some.
  for (int t0 = cluster; t0 < ntiles; t0 += clusters * teams) {
    const int t = t0 + team * clusters;
    const bool live = t < ntiles;
    const int nb = live ? blocks : 0;
    const int4 tile = live ? p.tiles[t] : make_int4(0, 0, 0, 0);
    if (live && warp < 4) {
      // ---------------------------------------------------------- gather
      const int c = lane & 7;                                // 16-byte piece of the 128
      const int r0 = warp * 32 + (lane >> 3);                // rows r0, r0 + 4, ..
      const __half* src[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + 4 * i;
        src[i] = p.X + static_cast<size_t>(p.perm[tile.y + min(r, tile.z - 1)]) * p.K + 8 * c;
      }
      for (int j = 0; j < nb; ++j) {
        const uint32_t g = it + j;
        const uint32_t s = g % stages;
        wait_or_give_up(&empty[s], ((g / stages) & 1) ^ 1, stop, p.head + 1);
        const int k = (rank + j * split) * 64;
        const uint32_t bytes = k + 8 * c < p.K ? 16u : 0u;   // zeros past K
        const uint32_t dst = smem_addr(sm + s * L.stage);
        if (tid == 0) {
          if (*stop) {
            mbar_arrive(&full[s]);
          } else {
            mbar_arrive_expect_tx(&full[s], rp * 128);
            tma_load_3d(sm + s * L.stage + kXBytes, &tmA, &full[s], k, 0, tile.x);
          }
        }
        if (!*stop) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = r0 + 4 * i;
            if (r < tile.z)
              cp_async16(dst + r * 128 + ((c ^ (r & 7)) << 4), bytes ? src[i] + k : p.X, bytes);
          }
        }
        cp_async_mbar_arrive(&full[s]);
      }
    } else if (live) {
      // ---------------------------------------------------------- MMAs
      const uint32_t idesc = make_idesc(1 /*f32*/, 0 /*fp16*/, kTile, rp);
      for (int j = 0; j < nb; ++j) {
        const uint32_t g = it + j;
        const uint32_t s = g % stages;
        if (!__all_sync(0xffffffffu, wait_or_give_up(&full[s], (g / stages) & 1, stop, p.head + 1))) break;
        // The gathered rows were written through the generic proxy. The fence
        // stands here, after their barrier: in the gathering threads it would
        // wait for the copies of the stages behind as well.
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t a = sw128_kmajor_desc(smem_addr(sm + s * L.stage));
        const uint64_t b = sw128_kmajor_desc(smem_addr(sm + s * L.stage + kXBytes));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16_elect(tmem, a + 2 * kk, b + 2 * kk, idesc, (j | kk) != 0);
        mma_commit_elect(&empty[s]);
      }
      if (nb > 0) mma_commit_elect(done);
    }
    it += nb;
    // -------------------------------------------------------------- partial sums
    if (live && warp < 4) {
      bool have = nb > 0;
      if (have) have = __all_sync(0xffffffffu, wait_or_give_up(done, round & 1, stop, p.head + 1));
      tc_fence_after();
      float* row = part + (warp * 32 + lane) * L.part_ld;
      // Every stage has been consumed once `done` completes: the ring is free.
      named_bar_sync(1, 128);
      for (int c = 0; c < rp; c += 16) {
        uint32_t acc[16];
        if (have) {
          tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, acc);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<uint4*>(row + c + i) = make_uint4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
      }
      tc_fence_before();
    }
    if (nb > 0) ++round;
    __syncwarp();
    cluster_sync();
    // Eight threads per token finish this CTA's 128 / split tokens: the partials of the
    // team in their order, the largest |t|, and the two parts of t'.
    if (live && warp < 4) {
      for (int r0 = 0; r0 < kTile / split; r0 += 16) {
        const int r = rank * (kTile / split) + r0 + (tid >> 3);
        const int c0 = 4 * (tid & 7);
        float v[kMaxRank / 32][4];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < kMaxRank / 32; ++i) {
          const int c = c0 + 32 * i;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][e] = 0.0f;
          if (c < p.R) {
            float f[split][4];
#pragma unroll
            for (int q = 0; q < split; ++q)
              asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(f[q][0]), "=f"(f[q][1]), "=f"(f[q][2]), "=f"(f[q][3])
                           : "r"(cluster_addr(part + r * L.part_ld + c, team * split + q)));
#pragma unroll
            for (int q = 0; q < split; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e) v[i][e] += f[q][e];
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(v[i][e]));
          }
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (r < tile.z) {
          float down, up;
          power_pair(m, &down, &up);
          const size_t at = static_cast<size_t>(tile.y + r);
          if ((tid & 7) == 0) p.factor[at] = p.scaling[tile.x] * up;
#pragma unroll
          for (int i = 0; i < kMaxRank / 32; ++i) {
            const int c = c0 + 32 * i;
            if (c < p.R) {
              __half2 h[2], l[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float x = v[i][2 * e] * down, y = v[i][2 * e + 1] * down;
                h[e] = __floats2half2_rn(x, y);
                const float2 back = __half22float2(h[e]);
                l[e] = __floats2half2_rn(x - back.x, y - back.y);
              }
              *reinterpret_cast<uint2*>(p.hi + at * p.R + c) = *reinterpret_cast<const uint2*>(h);
              *reinterpret_cast<uint2*>(p.lo + at * p.R + c) = *reinterpret_cast<const uint2*>(l);
            }
          }
        }
      }
    }
    __syncwarp();
    cluster_sync();                                          // the partials are no longer read
    // The next tile's copies go where this one's partials were.
    fence_proxy_async_smem();
  }
}

__global__ void __launch_bounds__(kShrinkThreads) tile_shrink_kernel(const __grid_constant__ CUtensorMap tmA,
                                                                     AdapterArgs p) {
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  uint8_t* sm = dyn_smem + ((1024u - (smem_addr(dyn_smem) & 1023u)) & 1023u);
  const ShrinkSmem L = shrink_smem(p.R);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L.bars);
  uint64_t* empty = full + kMaxShrinkStages;
  uint64_t* done = empty + kMaxShrinkStages;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int32_t* stop = reinterpret_cast<volatile int32_t*>(tslot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t tcols = shrink_tmem(p.R);

  if (tid == 0) {
    for (int s = 0; s < L.stages; ++s) {
      mbar_init(&full[s], 128 + 1);      // the gathering threads, and A's copy
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *stop = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmA);
  }
  if (warp == 4) {
    tmem_alloc(tslot, tcols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  griddep_wait();
  griddep_launch_dependents();

  const int ntiles = p.head[2];                              // those with an adapter come first
  auto fits = [&](int split) {
    return split <= p.cluster && static_cast<int64_t>(ntiles) * split <= gridDim.x;
  };
  if (fits(8))
    shrink_tiles<8>(tmA, p, L, sm, tmem, ntiles);
  else if (fits(4))
    shrink_tiles<4>(tmA, p, L, sm, tmem, ntiles);
  else if (fits(2))
    shrink_tiles<2>(tmA, p, L, sm, tmem, ntiles);
  else
    shrink_tiles<1>(tmA, p, L, sm, tmem, ntiles);
  tc_fence_before();
  __syncthreads();
  if (*stop) let_copies_land();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
}

// Expand: D[128 tokens][128 columns] = (hi | lo) . B[a] rows^T on tcgen05. The blocks
// of 128 columns of all tiles, tile by tile, are dealt out in equal runs, one CTA
// per SM: within a tile t' stays in shared memory, B comes block by block into two
// buffers, two accumulators let the MMAs of a block run under the epilogue of the
// one before, and Y0 comes one or two blocks ahead (a 16-byte copy per lane, half a
// warp per row, the tokens' rows lie anywhere). A thread of the epilogue holds one
// token's row of D, adds it to Y0 in shared memory, and the block leaves as it
// came. Direct reads and writes from a layout with columns across the lanes, 4
// bytes each, needed four times the instructions and ran at 2.9 TB/s.
constexpr int kCols = 128;
// Epilogue warps: the copies of rows at any address are many short steps (4096 x 4096 x
// 10007, rank 64: 149 us with 8, 110 with 16); aligned rows do 1% better with 8.
template <bool VEC>
constexpr int kEpiWarps = VEC ? 8 : 16;
template <bool VEC>
constexpr int kExpandThreads = 32 * kEpiWarps<VEC> + 64;
constexpr int kYLd = kCols + 8;                  // halves between rows of a staged block

// Not VEC: f B t' of a block, column c of a token at (c % 8) * 17 + c / 8, for the
// same reason as in the kernel for few tokens; an odd distance between tokens, so that
// the lanes that write one column of 32 tokens meet different banks too.
constexpr int kSpreadTileLd = 8 * 17 + 1;

struct ExpandSmem {
  int blocks, ystages, b, y, bars, bytes;
};
__host__ __device__ inline ExpandSmem expand_smem(int R) {
  ExpandSmem L;
  L.blocks = (R + 63) / 64;                                 // 64-wide pieces of R
  L.ystages = L.blocks == 1 ? 4 : 2;
  L.b = 2 * L.blocks * kTile * 128;                         // after [hi, lo][blocks][128][128 B]
  L.y = L.b + 2 * L.blocks * kCols * 128;                   // after [2][blocks][128][128 B]
  int y = L.ystages * kTile * kYLd * 2;
  if (y < kTile * kSpreadTileLd * 4) y = kTile * kSpreadTileLd * 4;
  L.bars = (L.y + y + 15) / 16 * 16;
  L.bytes = 1024 + L.bars + 10 * 8 + 32;
  return L;
}

// What half a warp (16 lanes, this one `l`) moves of a row's columns [n0, n0 + w),
// w <= 128, when the row may lie at any 2-byte address: a 16-byte vector per lane
// between the first and the last such address, and one value each on either side.
struct RowPiece {
  int vec, edge;          // column of this lane's vector and of its single value, or -1
};
__device__ __forceinline__ RowPiece row_piece(size_t at, int w, int l) {
  const int head = min(w, static_cast<int>((8 - (at & 7)) & 7));
  const int vecs = (w - head) / 8;
  const int tail = head + 8 * vecs;
  RowPiece r;
  r.vec = l < vecs ? head + 8 * l : -1;
  r.edge = l < head ? l : l >= 8 && tail + l - 8 < w ? tail + l - 8 : -1;
  return r;
}

template <bool VEC>   // N a multiple of 8: every row of Y is 16-byte aligned
__global__ void __launch_bounds__(kExpandThreads<VEC>, 1) tile_expand_kernel(
    const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmHi,
    const __grid_constant__ CUtensorMap tmLo, AdapterArgs p) {
  constexpr int kEpi = kEpiWarps<VEC>;
  constexpr int kRowsEach = kTile / (2 * kEpi);    // rows that half a warp copies
  constexpr int kColsEach = kCols * 4 / kEpi;      // columns of a token that a thread works on
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  uint8_t* sm = dyn_smem + ((1024u - (smem_addr(dyn_smem) & 1023u)) & 1023u);
  const ExpandSmem L = expand_smem(p.R);
  uint64_t* tfull = reinterpret_cast<uint64_t*>(sm + L.bars);
  uint64_t* tempty = tfull + 1;
  uint64_t* bfull = tfull + 2;        // [2]
  uint64_t* bempty = tfull + 4;       // [2]
  uint64_t* afull = tfull + 6;        // [2]
  uint64_t* aempty = tfull + 8;       // [2]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(tfull + 10);
  volatile int32_t* stop = reinterpret_cast<volatile int32_t*>(tslot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(tfull, 1);
    mbar_init(tempty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bfull[i], 1);
      mbar_init(&bempty[i], 1);
      mbar_init(&afull[i], 1);
      mbar_init(&aempty[i], kEpi);
    }
    *stop = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmHi);
    tma_prefetch_desc(&tmLo);
  }
  if (warp == kEpi) {
    tmem_alloc(tslot, 2 * kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  griddep_wait();
  griddep_launch_dependents();

  // In place, the tiles without an adapter (the last ones) need nothing.
  const int ntiles = p.Y == p.Y0 ? p.head[2] : p.head[0];
  const int nblocks = (p.N + kCols - 1) / kCols;
  const int64_t total = static_cast<int64_t>(ntiles) * nblocks;
  const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
  uint32_t nt = 0, nb = 0;            // tiles and blocks so far (those with an adapter)
  for (int64_t at = total * blockIdx.x / gridDim.x; at < end;) {
    const int ti = static_cast<int>(at / nblocks);
    const int4 tile = p.tiles[ti];
    const int b0 = static_cast<int>(at - static_cast<int64_t>(ti) * nblocks);
    const int b1 = static_cast<int>(min(static_cast<int64_t>(nblocks), b0 + (end - at)));
    at += b1 - b0;
    if (warp == kEpi + 1) {
      // ------------------------------------------------------------ copies
      if (tile.x >= 0 && lane == 0) {
        if (wait_or_give_up(tempty, (nt & 1) ^ 1, stop, p.head + 1)) {
          mbar_arrive_expect_tx(tfull, 2 * L.blocks * kTile * 128);
          for (int i = 0; i < L.blocks; ++i) {
            tma_load_2d(sm + i * kTile * 128, &tmHi, tfull, 64 * i, tile.y);
            tma_load_2d(sm + (L.blocks + i) * kTile * 128, &tmLo, tfull, 64 * i, tile.y);
          }
        }
        for (int b = b0; b < b1; ++b) {
          const uint32_t g = nb + (b - b0);
          if (!wait_or_give_up(&bempty[g & 1], ((g >> 1) & 1) ^ 1, stop, p.head + 1)) break;
          uint8_t* dst = sm + L.b + (g & 1) * L.blocks * kCols * 128;
          mbar_arrive_expect_tx(&bfull[g & 1], L.blocks * kCols * 128);
          for (int i = 0; i < L.blocks; ++i)
            tma_load_3d(dst + i * kCols * 128, &tmB, &bfull[g & 1], 64 * i, b * kCols, tile.x);
        }
      }
      __syncwarp();
    } else if (warp == kEpi) {
      // ------------------------------------------------------------ MMAs
      if (tile.x >= 0) {
        constexpr uint32_t idesc = make_idesc(1 /*f32*/, 0 /*fp16*/, kTile, kCols);
        bool ok = __all_sync(0xffffffffu, wait_or_give_up(tfull, nt & 1, stop, p.head + 1));
        for (int b = b0; b < b1 && ok; ++b) {
          const uint32_t g = nb + (b - b0);
          ok = __all_sync(0xffffffffu,
                          wait_or_give_up(&aempty[g & 1], ((g >> 1) & 1) ^ 1, stop, p.head + 1) &&
                              wait_or_give_up(&bfull[g & 1], (g >> 1) & 1, stop, p.head + 1));
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + (g & 1) * kCols;
          uint32_t more = 0;
          for (int part = 0; part < 2; ++part)
            for (int i = 0; i < L.blocks; ++i) {
              const uint64_t t = sw128_kmajor_desc(smem_addr(sm + (part * L.blocks + i) * kTile * 128));
              const uint64_t w = sw128_kmajor_desc(smem_addr(sm + L.b + ((g & 1) * L.blocks + i) * kCols * 128));
              const int steps = (min(64, p.R - 64 * i) + 15) / 16;
              for (int kk = 0; kk < steps; ++kk) {
                mma_f16_elect(d, t + 2 * kk, w + 2 * kk, idesc, more);
                more = 1;
              }
            }
          mma_commit_elect(&bempty[g & 1]);
          mma_commit_elect(&afull[g & 1]);
        }
        if (ok) mma_commit_elect(tempty);
      }
    } else {
      // ------------------------------------------------------------ epilogue
      named_bar_sync(1, 32 * kEpi);    // the last tile's blocks have left shared memory
      // Copies: rows team + 2 kEpi i, team the 16 lanes' number. Arithmetic: token
      // 32 (warp % 4) + lane, kColsEach columns from kColsEach (warp / 4).
      const int team = tid >> 4, l = tid & 15;
      size_t row[kRowsEach];
#pragma unroll
      for (int i = 0; i < kRowsEach; ++i)
        row[i] = static_cast<size_t>(p.perm[tile.y + min(team + 2 * kEpi * i, tile.z - 1)]) * p.N;
      const int q = warp & 3, c0 = (warp >> 2) * kColsEach;
      const int tok = q * 32 + lane;
      const bool live = 32 * q < tile.z;            // the warp has a token
      const float f = tile.x >= 0 && tok < tile.z ? p.factor[tile.y + tok] : 0.0f;
      __half* const ys = reinterpret_cast<__half*>(sm + L.y);
      uint4 v[VEC ? 1 : kRowsEach];            // VEC: copied asynchronously; else on the way in registers
      __half e[VEC ? 1 : kRowsEach];
      float* const spread = reinterpret_cast<float*>(sm + L.y);   // not VEC
      auto fetch_row = [&](int b, int i) {    // not VEC
        if constexpr (!VEC) {
          const int n0 = b * kCols;
          const RowPiece pc = row_piece(row[i] + n0, min(kCols, p.N - n0), l);
          if (team + 2 * kEpi * i < tile.z) {
            if (pc.vec >= 0) v[i] = *reinterpret_cast<const uint4*>(p.Y0 + row[i] + n0 + pc.vec);
            if (pc.edge >= 0) e[i] = p.Y0[row[i] + n0 + pc.edge];
          }
        }
      };
      auto fetch = [&](int b, int stage) {
        const int n0 = b * kCols, w = min(kCols, p.N - n0);
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i) {
          const int r = team + 2 * kEpi * i;
          if constexpr (!VEC)
            fetch_row(b, i);
          else if (r < tile.z && 8 * l < w)
            cp_async16(smem_addr(ys + (stage * kTile + r) * kYLd + 8 * l), p.Y0 + row[i] + n0 + 8 * l, 16);
        }
        if constexpr (VEC) cp_async_commit();
      };
      auto leave = [&](int b, int stage) {
        const int n0 = b * kCols, w = min(kCols, p.N - n0);
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i) {
          const int r = team + 2 * kEpi * i;
          if (r >= tile.z) continue;
          if constexpr (VEC) {
            const __half* src = ys + (stage * kTile + r) * kYLd;
            if (8 * l < w)
              *reinterpret_cast<uint4*>(p.Y + row[i] + n0 + 8 * l) = *reinterpret_cast<const uint4*>(src + 8 * l);
          } else {
            const RowPiece pc = row_piece(row[i] + n0, w, l);
            const float* from = spread + r * kSpreadTileLd;
            auto add = [&](__half y, int c) {
              return tile.x < 0 ? y : __float2half_rn(__half2float(y) + from[(c & 7) * 17 + (c >> 3)]);
            };
            if (pc.vec >= 0) {
              __half* h = reinterpret_cast<__half*>(&v[i]);
#pragma unroll
              for (int k = 0; k < 8; ++k) h[k] = add(h[k], pc.vec + k);
              *reinterpret_cast<uint4*>(p.Y + row[i] + n0 + pc.vec) = v[i];
            }
            if (pc.edge >= 0) p.Y[row[i] + n0 + pc.edge] = add(e[i], pc.edge);
            if (b + 1 < b1) fetch_row(b + 1, i);
          }
        }
      };
      // Blocks on the way beside the one in work: all stages but one (VEC), or one in registers.
      const int ahead = VEC ? L.ystages - 1 : 1;
      for (int j = 0; j < ahead; ++j) {
        if (b0 + j < b1)
          fetch(b0 + j, j);
        else if constexpr (VEC)
          cp_async_commit();
      }
      bool ok = true;
      for (int b = b0; b < b1; ++b) {
        const uint32_t g = nb + (b - b0);
        const int j = b - b0;
        const int stage = VEC ? j % L.ystages : j & 1;
        if constexpr (VEC) {
          if (b + ahead < b1)
            fetch(b + ahead, (j + ahead) % L.ystages);
          else
            cp_async_commit();
          if (ahead == 3)
            cp_async_wait<3>();
          else
            cp_async_wait<1>();
        }
        named_bar_sync(1, 32 * kEpi);
        if (tile.x >= 0) {
          ok = ok && __all_sync(0xffffffffu, wait_or_give_up(&afull[g & 1], (g >> 1) & 1, stop, p.head + 1));
          tc_fence_after();
          const uint32_t d_at = tmem + (static_cast<uint32_t>(q * 32) << 16) + (g & 1) * kCols + c0;
          auto read_out = [&] {                     // the accumulator is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&aempty[g & 1]);
          };
          if constexpr (VEC) {
            // All of the thread's part of D at once: one wait for tensor memory, and the MMAs
            // of the block after the next need not wait for the arithmetic (4096 x 8192 x
            // 28672, rank 64: 138.5 us with 16 columns at a time, 133.8 so).
            uint32_t acc[kColsEach / 16][16];
            if (ok && live) {
#pragma unroll
              for (int c = 0; c < kColsEach / 16; ++c) tmem_ld_32x32b_x16(d_at + 16 * c, acc[c]);
              tmem_ld_wait();
            } else {
#pragma unroll
              for (int i = 0; i < kColsEach; ++i) acc[i / 16][i % 16] = 0u;
            }
            read_out();
            uint4* mine = reinterpret_cast<uint4*>(ys + (stage * kTile + tok) * kYLd + c0);
            if (live) {
#pragma unroll
              for (int h = 0; h < kColsEach / 8; ++h) {
                uint4 y = mine[h];
                __half2* y2 = reinterpret_cast<__half2*>(&y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 u = __half22float2(y2[i]);
                  y2[i] = __floats2half2_rn(fmaf(f, __uint_as_float(acc[h / 2][8 * (h & 1) + 2 * i]), u.x),
                                            fmaf(f, __uint_as_float(acc[h / 2][8 * (h & 1) + 2 * i + 1]), u.y));
                }
                mine[h] = y;
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < kColsEach; c += 16) {
              uint32_t acc[16];
              if (ok) {
                tmem_ld_32x32b_x16(d_at + c, acc);
                tmem_ld_wait();
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = 0u;
              }
              // f times the sum here, Y0 where it is: a lane of `leave` has eight columns
              // of eight other tokens
#pragma unroll
              for (int i = 0; i < 16; ++i)
                spread[tok * kSpreadTileLd + (i & 7) * 17 + (c0 + c + i) / 8] = f * __uint_as_float(acc[i]);
            }
            read_out();
          }
          named_bar_sync(1, 32 * kEpi);
        }
        leave(b, stage);
        // Whoever fills this stage next moves the same pieces of it as here.
      }
      if constexpr (VEC) cp_async_wait<0>();
    }
    if (tile.x >= 0) {
      ++nt;
      nb += b1 - b0;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*stop) let_copies_land();
  if (warp == kEpi) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kCols);
  }
}

cudaError_t launch_large(AdapterArgs p, cudaStream_t s) {
  CUtensorMap tmA, tmB, tmHi, tmLo;
  const int rp = (p.R + 15) / 16 * 16;
  const auto f16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (!make_tmap_3d_sw128(&tmA, p.A, f16, 2, p.K, p.R, p.n, rp) ||
      !make_tmap_3d_sw128(&tmB, p.B, f16, 2, p.R, p.N, p.n, kCols) ||
      !make_tmap_sw128(&tmHi, p.hi, f16, 2, p.R, p.M, kTile) ||
      !make_tmap_sw128(&tmLo, p.lo, f16, 2, p.R, p.M, kTile))
    return cudaErrorInvalidValue;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count(dev);
  const ShrinkSmem LS = shrink_smem(p.R);
  const ExpandSmem LE = expand_smem(p.R);
  const bool vec = p.N % 8 == 0;
  if ((e = allow_max_smem<tile_shrink_kernel>()) != cudaSuccess) return e;
  if ((e = vec ? allow_max_smem<tile_expand_kernel<true>>()
                 : allow_max_smem<tile_expand_kernel<false>>()) != cudaSuccess)
    return e;
  const int tiles = max_groups(p, kTile);

  void* plan_args[] = {&p};
  e = launch_pdl(reinterpret_cast<const void*>(plan_kernel), dim3(1), kPlanThreads,
                 (static_cast<size_t>(p.n) + 1) * 4, s, plan_args);
  if (e != cudaSuccess) return e;
  // The host knows the least and the largest number of tiles; the kernel splits its
  // clusters into teams when there are more than the least.
  const int fit = shrink_per_sm(p.R) * sms;
  p.cluster = kMaxSplit;
  while (p.cluster > 1 && static_cast<int64_t>((p.M + kTile - 1) / kTile) * p.cluster > fit) p.cluster /= 2;
  // A GPC holds whole clusters only: of eight CTAs, three per SM, 47 are resident at once and
  // 49 are not (1500 x 4096 x 4096, rank 16, 64 adapters: 45 us and 58).
  int clusters = p.cluster == 8 ? fit / 8 * 6 / 7 : fit / p.cluster;
  if (clusters > tiles) clusters = tiles;
  void* shrink_args[] = {&tmA, &p};
  e = launch_pdl(reinterpret_cast<const void*>(tile_shrink_kernel), dim3(clusters * p.cluster),
                 kShrinkThreads, LS.bytes, s, shrink_args, p.cluster);
  if (e != cudaSuccess) return e;
  const int64_t blocks = static_cast<int64_t>(tiles) * ((p.N + kCols - 1) / kCols);
  const int ctas = blocks < sms ? static_cast<int>(blocks) : sms;
  void* expand_args[] = {&tmB, &tmHi, &tmLo, &p};
  return launch_pdl(vec ? reinterpret_cast<const void*>(tile_expand_kernel<true>)
                        : reinterpret_cast<const void*>(tile_expand_kernel<false>),
                    dim3(ctas), vec ? kExpandThreads<true> : kExpandThreads<false>, LE.bytes, s, expand_args);
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Each fills in the parts of the workspace that its form uses (offsets from ws) and
// returns their size.
size_t carve_small(AdapterArgs* p, uint8_t* ws) {
  // About 512 columns per CTA (four warps of four 32-column steps each), half as many
  // for the larger ranks, whose steps do not all fit into the registers; at most kMaxSlices.
  const int cols = p->R <= 32 ? 512 : 256;
  const int s = (p->K + cols - 1) / cols;
  p->S = s < kMaxSlices ? s : kMaxSlices;
  p->slice = ((p->K + p->S - 1) / p->S + 127) / 128 * 128;
  p->head = reinterpret_cast<int32_t*>(ws);
  p->part = reinterpret_cast<float*>(ws + 256);
  return 256 + up256(static_cast<size_t>(p->S) * p->M * p->R * 4);
}

size_t carve_large(AdapterArgs* p, uint8_t* ws) {
  size_t off = 256;
  auto take = [&](size_t bytes) {
    uint8_t* at = ws + off;
    off += up256(bytes);
    return at;
  };
  const size_t M = p->M;
  p->head = reinterpret_cast<int32_t*>(ws);
  p->tiles = reinterpret_cast<int4*>(take(static_cast<size_t>(max_groups(*p, kTile)) * sizeof(int4)));
  p->perm = reinterpret_cast<int32_t*>(take(M * 4));
  p->factor = reinterpret_cast<float*>(take(M * 4));
  p->hi = reinterpret_cast<__half*>(take(M * p->R * 2));
  p->lo = reinterpret_cast<__half*>(take(M * p->R * 2));
  return off;
}

int check_adapter(int M, int N, int K, int n_adapters, int R) {
  const int st = abi_check_sizes(M, N, K);
  if (st != I8MM_OK) return st;
  if (n_adapters < 1 || n_adapters > kMaxAdapters || R < 8 || R > kMaxRank || R % 8 != 0)
    return I8MM_ERR_INVALID_ARG;
  return I8MM_OK;
}

}  // namespace

}  // namespace i8mm

using namespace i8mm;

extern "C" {

size_t int8_adapter_add_workspace_size(int M, int N, int K, int n_adapters, int R) {
  if (check_adapter(M, N, K, n_adapters, R) != I8MM_OK) return 0;
  // The most that a call with no larger arguments needs, in either form: the form for few
  // tokens needs more than the other (1 MB at most), and up to fewer tokens the larger the
  // rank, so a call's own need would shrink as its batch or rank grows.
  AdapterArgs p{};
  p.M = M;
  p.K = K;
  p.n = n_adapters;
  p.R = R;
  size_t most = carve_large(&p, nullptr);
  for (const int top : {16, 32, 64, kMaxRank}) {   // the ranks that small_tokens tells apart
    p.R = R < top ? R : top;
    const int tokens = small_tokens(p.R, n_adapters);
    p.M = M < tokens ? M : tokens;
    const size_t need = carve_small(&p, nullptr);
    if (need > most) most = need;
  }
  return most;
}

int int8_adapter_add(const void* X, const void* A, const void* B, const int32_t* adapter_idx,
                     const float* scaling, int M, int N, int K, int n_adapters, int R,
                     const void* Y0, void* Y, void* workspace, size_t workspace_bytes,
                     i8mm_stream_t stream) {
  int st = check_adapter(M, N, K, n_adapters, R);
  if (st != I8MM_OK) return st;
  if (M == 0 || N == 0) return I8MM_OK;
  if (!X || !A || !B || !adapter_idx || !scaling || !Y0 || !Y) return I8MM_ERR_INVALID_ARG;
  auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!a16(X) || !a16(A) || !a16(B) || !a16(adapter_idx) || !a16(scaling) || !a16(Y0) || !a16(Y))
    return I8MM_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < int8_adapter_add_workspace_size(M, N, K, n_adapters, R))
    return I8MM_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return I8MM_ERR_ALIGNMENT;
  // In place, or apart: a Y that starts inside Y0 (or Y0 inside Y) has no answer.
  const uintptr_t y = reinterpret_cast<uintptr_t>(Y), y0 = reinterpret_cast<uintptr_t>(Y0);
  const size_t ybytes = static_cast<size_t>(M) * N * 2;
  if (y != y0 && y < y0 + ybytes && y0 < y + ybytes) return I8MM_ERR_INVALID_ARG;
  if ((st = abi_check_device()) != I8MM_OK) return st;
  AdapterArgs p{};
  p.X = static_cast<const __half*>(X);
  p.A = static_cast<const __half*>(A);
  p.B = static_cast<const __half*>(B);
  p.idx = adapter_idx;
  p.scaling = scaling;
  p.Y0 = static_cast<const __half*>(Y0);
  p.Y = static_cast<__half*>(Y);
  p.M = M;
  p.N = N;
  p.K = K;
  p.n = n_adapters;
  p.R = R;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool small = M <= small_tokens(R, n_adapters);
  if (small)
    carve_small(&p, ws);
  else
    carve_large(&p, ws);
  return abi_cuda_fail("adapter kernel launch", small ? launch_small(p, s) : launch_large(p, s));
}

}  // extern "C"
