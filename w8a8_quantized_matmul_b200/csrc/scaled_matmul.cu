// The product of rows that are quantised already:
//
//   Y[i][n] = fp16( C_i32[i][n] * x_scale[i] * w_scale[n] / 127^2 ),  C_i32 = Xq . Wq^T
//
// Many tokens: the tcgen05 INT8 GEMM of gemm_sm100.cu without an outlier product,
// whose 256 x 256 tiles need enough of them to fill the GPU. Fewer: the kernel of
// this file, for which reading Wq is what bounds it. There the weight's rows are the
// 128-row operand of the MMA and the tokens, padded to 16 .. 256, its columns;
// a cluster of S CTAs splits K of a 128-row tile, so that small weights too are
// read by the whole GPU. INT32 partial sums are exact, so neither the split nor
// its order changes a bit of Y.
//
// Warp roles of a CTA: warp 0 copies (TMA, 128 columns of K per stage: 16 KB of
// Wq and the tokens' codes), warp 1 owns TMEM and issues the MMAs, warps 2 to 5
// take the result: with S = 1 straight from TMEM to Y (a lane holds one column
// of Y; lane pairs swap so that each stores two columns of one token); with S > 1
// through shared memory, where every CTA of the cluster sums the S partials of
// its share of the tokens over distributed shared memory. Asking for the first of
// Wq in L2 while the kernel before still runs was tried: 0.7 us less for a
// feed-forward block of 16 tokens, but 0.3 to 4 us more for products in a row.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "int8mm.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace i8mm {

namespace {

constexpr int kRows = 128;             // weight rows of a tile
constexpr int kKB = 128;               // int8 columns of a stage
constexpr int kWBytes = kRows * kKB;
constexpr int kMaxTok = 256;
constexpr int kMaxSplit = 8;
constexpr int kMaxStages = 10;
constexpr int kThreads = 192;

// Where a product without a status word of its own records a wait that gave up.
static __device__ int32_t g_stream_status;

struct StreamArgs {
  const float* x_scale;   // [M]
  const float* w_scale;   // [N]
  __half* Y;              // [M][N]
  int32_t* status;        // or nullptr: g_stream_status
  int M, N, K;
  int tok;                // tokens of a block, the MMA's N: a multiple of 16, at most kMaxTok
  int split;              // S
  int stages;
};

__host__ __device__ constexpr int tmem_cols(int tok) {
  return tok <= 32 ? 32 : tok <= 64 ? 64 : tok <= 128 ? 128 : 256;
}

// Tokens whose partial sums fit at once where the ring was.
__host__ __device__ inline int reduce_tokens(int tok) { return tok < 128 ? tok : 128; }

struct StreamSmem {
  int stage, ring, xs, bars, bytes;
};
__host__ __device__ inline StreamSmem stream_smem(int tok, int stages, int split) {
  StreamSmem L;
  L.stage = kWBytes + tok * kKB;
  L.ring = stages * L.stage;
  const int red = split > 1 ? reduce_tokens(tok) * kRows * 4 : 0;   // [tokens][128] int32
  if (L.ring < red) L.ring = red;
  L.xs = L.ring;                                    // [tok] x_scale / 127^2
  L.bars = L.xs + tok * 4;
  L.bytes = 1024 + L.bars + (2 * kMaxStages + 1) * 8 + 16;
  const int least = split > 1 ? cluster_tmem_smem(tmem_cols(tok)) : 0;
  if (L.bytes < least) L.bytes = least;
  return L;
}

template <bool EVEN>   // N even: two columns per store
__device__ __forceinline__ void store_pair(__half* y, size_t at, int n, int N, float v0, float v1) {
  if constexpr (EVEN) {
    *reinterpret_cast<__half2*>(y + at + n) = __floats2half2_rn(v0, v1);
  } else {
    y[at + n] = __float2half_rn(v0);
    if (n + 1 < N) y[at + n + 1] = __float2half_rn(v1);
  }
}

template <bool EVEN>
__global__ void __launch_bounds__(kThreads) weight_stream_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                 const __grid_constant__ CUtensorMap tmX,
                                                                 StreamArgs a) {
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  uint8_t* sm = dyn_smem + ((1024u - (smem_addr(dyn_smem) & 1023u)) & 1023u);
  const StreamSmem L = stream_smem(a.tok, a.stages, a.split);
  float* xs = reinterpret_cast<float*>(sm + L.xs);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L.bars);
  uint64_t* empty = full + kMaxStages;
  uint64_t* done = empty + kMaxStages;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int32_t* stop = reinterpret_cast<volatile int32_t*>(tslot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* const status = a.status ? a.status : &g_stream_status;
  const int S = a.split;
  const int rank = static_cast<int>(cluster_ctarank());
  const int n0 = static_cast<int>(blockIdx.x / S) * kRows;
  const int t0 = blockIdx.y * a.tok;
  const int nkb = (a.K + kKB - 1) / kKB;
  const int nb = nkb > rank ? (nkb - rank + S - 1) / S : 0;   // stages: blocks rank, rank + S, ..
  const uint32_t tcols = tmem_cols(a.tok);

  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *stop = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tslot, tcols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  griddep_wait();
  griddep_launch_dependents();

  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      for (int j = 0; j < nb; ++j) {
        const int s = j % a.stages;
        if (!wait_or_give_up(&empty[s], ((j / a.stages) & 1) ^ 1, stop, status)) break;
        uint8_t* w = sm + s * L.stage;
        const int k = (rank + j * S) * kKB;
        mbar_arrive_expect_tx(&full[s], L.stage);
        tma_load_2d(w, &tmW, &full[s], k, n0);
        tma_load_2d(w + kWBytes, &tmX, &full[s], k, t0);
      }
    }
  } else if (warp == 1) {
    const uint32_t idesc = make_idesc(2 /*s32*/, 1 /*signed*/, kRows, a.tok);
    for (int j = 0; j < nb && ok; ++j) {
      const int s = j % a.stages;
      ok = __all_sync(0xffffffffu, wait_or_give_up(&full[s], (j / a.stages) & 1, stop, status));
      if (!ok) break;
      const uint64_t w = sw128_kmajor_desc(smem_addr(sm + s * L.stage));
      const uint64_t x = sw128_kmajor_desc(smem_addr(sm + s * L.stage + kWBytes));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_i8_elect(tmem, w + 2 * kk, x + 2 * kk, idesc, (j | kk) != 0);
      mma_commit_elect(&empty[s]);
    }
    // `done` says that every stage has arrived and been consumed.
    if (ok) mma_commit_elect(done);
  } else {
    const int q = warp & 3;
    const int et = tid - 64;
    const int nl = q * 32 + lane;                  // this lane's row of the tile = column of Y
    const float ws = n0 + nl < a.N ? a.w_scale[n0 + nl] : 0.0f;
    for (int t = et; t < a.tok; t += 128)
      xs[t] = t0 + t < a.M ? a.x_scale[t0 + t] * (1.0f / 16129.0f) : 0.0f;
    named_bar_sync(1, 128);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
    if (S == 1) {
      ok = __all_sync(0xffffffffu, wait_or_give_up(done, 0, stop, status));
      tc_fence_after();
      const int np = n0 + (nl & ~1);
      const float wo = __shfl_xor_sync(0xffffffffu, ws, 1);
      const float w0 = lane & 1 ? wo : ws, w1 = lane & 1 ? ws : wo;
      for (int c = 0; c < min(a.tok, a.M - t0) && ok; c += 16) {
        uint32_t acc[16];
        tmem_ld_32x32b_x16(lane_base + c, acc);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool odd = lane & 1;
          const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? acc[2 * i] : acc[2 * i + 1], 1);
          const int32_t c0 = static_cast<int32_t>(odd ? got : acc[2 * i]);
          const int32_t c1 = static_cast<int32_t>(odd ? acc[2 * i + 1] : got);
          const int t = c + 2 * i + (lane & 1);
          if (t0 + t < a.M && np < a.N)
            store_pair<EVEN>(a.Y, static_cast<size_t>(t0 + t) * a.N, np, a.N,
                             static_cast<float>(c0) * (xs[t] * w0), static_cast<float>(c1) * (xs[t] * w1));
        }
      }
      tc_fence_before();
    }
  }
  if (S > 1) {
    // Partials [token][128] of up to 128 tokens at a time, in the ring's place: `done`
    // completes when its last stage has been consumed.
    int32_t* part = reinterpret_cast<int32_t*>(sm);
    const int step = reduce_tokens(a.tok);
    const int live = min(a.tok, a.M - t0);
    for (int c0 = 0; c0 < live; c0 += step) {
      if (warp >= 2) {
        const int q = warp & 3;
        if (c0 == 0) {
          ok = __all_sync(0xffffffffu, wait_or_give_up(done, 0, stop, status));
          tc_fence_after();
          if (!ok) let_copies_land();               // they go where the partials will
          named_bar_sync(1, 128);
        }
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
        for (int c = 0; c < min(step, live - c0); c += 16) {
          uint32_t acc[16];
          if (nb > 0 && ok) {
            tmem_ld_32x32b_x16(lane_base + c0 + c, acc);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = 0u;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) part[(c + i) * kRows + q * 32 + lane] = static_cast<int32_t>(acc[i]);
        }
        tc_fence_before();
      }
      __syncwarp();
      cluster_sync();
      // Tokens rank, rank + S, .. of these, a warp each, four columns per lane; two
      // tokens' partials are on the way together.
      if (warp >= 2) {
        const int nl = 4 * lane;
        const int n = n0 + nl;
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = n + i < a.N ? a.w_scale[n + i] : 0.0f;
        const int end = min(step, live - c0);
        for (int t = rank + S * (warp - 2); t < end; t += 8 * S) {
          int32_t v[2][kMaxSplit][4];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r)
              if (r < S && t + 4 * S * u < end)
                asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v[u][r][0]), "=r"(v[u][r][1]), "=r"(v[u][r][2]), "=r"(v[u][r][3])
                             : "r"(cluster_addr(part + (t + 4 * S * u) * kRows + nl, r)));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int tt = t + 4 * S * u;
            if (tt >= end) break;
            int32_t c[4] = {0, 0, 0, 0};
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r)
              if (r < S)
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i] += v[u][r][i];
            const float x = xs[c0 + tt];
            const size_t at = static_cast<size_t>(t0 + c0 + tt) * a.N;
#pragma unroll
            for (int i = 0; i < 4; i += 2)
              if (n + i < a.N)
                store_pair<EVEN>(a.Y, at, n + i, a.N, static_cast<float>(c[i]) * (x * w[i]),
                                 static_cast<float>(c[i + 1]) * (x * w[i + 1]));
          }
        }
      }
      __syncwarp();
      cluster_sync();   // read by the peers: may be overwritten, and the CTA may end
    }
  }
  if (!ok) let_copies_land();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
}

template <bool EVEN>
cudaError_t launch_stream(const GemmArgs& g, cudaStream_t s, int tok, int split, int budget) {
  StreamArgs a{};
  a.x_scale = g.x_scale;
  a.w_scale = g.w_scale;
  a.Y = static_cast<__half*>(g.out);
  a.status = g.status;
  a.M = g.M;
  a.N = g.N;
  a.K = g.K;
  a.tok = tok;
  a.split = split;
  const int per = ((g.K + kKB - 1) / kKB + split - 1) / split;
  a.stages = budget / (kWBytes + tok * kKB);
  if (a.stages > per) a.stages = per;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  const StreamSmem L = stream_smem(tok, a.stages, split);
  CUtensorMap tmW, tmX;
  std::memset(&tmW, 0, sizeof(tmW));
  std::memset(&tmX, 0, sizeof(tmX));
  if (!make_tmap_sw128(&tmW, g.Wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.K, g.N, kRows) ||
      !make_tmap_sw128(&tmX, g.Xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.K, g.M, tok))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_max_smem<weight_stream_kernel<EVEN>>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((g.N + kRows - 1) / kRows * split, (g.M + tok - 1) / tok);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L.bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, weight_stream_kernel<EVEN>, tmW, tmX, a);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

// Which kernel, and how K is split. Measured on B200 (us, cold weights):
//   tokens x K x N        this file   gemm_sm100.cu
//   1 x 4096 x 4096          6.1          18.1
//   16 x 8192 x 28672       39.3          44.2
//   100 x 4096 x 10007      13.7          22.2
//   128 x 4096 x 16384      17.4          21.2
//   256 x 4096 x 4096       13.9          15.1
//   512 x 8192 x 1024       15.8          24.4
//   512 x 4096 x 4096       18.6          15.2
//   256 x 4096 x 16384      24.9          18.3
//   1500 x 1024 x 700       14.6           9.7
//   4096 x 4096 x 10007    172           139
// Up to 128 tokens this file's kernel; above, the one whose estimate is lower: the
// GEMM takes a wave of its 256 x 256 tiles, one per CTA pair, in 5.5 us + 2.35 ns
// per column of K; a CTA here brings in 95 KB of codes per us, and its epilogue
// costs 8 ns per token, twice that with partial sums.
cudaError_t launch_scaled(const GemmArgs& g, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count(dev);
  // Equal blocks of at most kMaxTok tokens, in steps of the MMA's 16.
  const int tblocks = (g.M + kMaxTok - 1) / kMaxTok;
  const int tok = ((g.M + tblocks - 1) / tblocks + 15) / 16 * 16;
  const int64_t blocks = static_cast<int64_t>((g.N + kRows - 1) / kRows) * ((g.M + tok - 1) / tok);
  const int nkb = (g.K + kKB - 1) / kKB;
  // The split with the shortest way through K for the SM that has most CTAs, if by
  // 5% at least; two CTAs per SM. With more than 128 tokens the exchange of the
  // partial sums costs more than a split above 4 gains (129 x 8192 x 5000: 26.2 us
  // with 7, 15.7 with 3).
  int split = 1;
  double way = 1e30;
  for (int c = 1; c <= (tok > 128 ? 4 : kMaxSplit) && c <= nkb && (c == 1 || c * blocks <= 2 * sms); ++c) {
    const double w = static_cast<double>((c * blocks + sms - 1) / sms) / c;
    if (w < 0.95 * way) {
      way = w;
      split = c;
    }
  }
  if (g.M > 128) {
    const int64_t tiles = static_cast<int64_t>((g.M + 255) / 256) * ((g.N + 255) / 256);
    const int64_t waves = (tiles + sms / 2 - 1) / (sms / 2);
    const double gemm = 5.5 + 2.35e-3 * g.K * waves;
    const double here = 5.0 + way * nkb * (16.0 + tok / 8.0) / 95.0 + tok * (split > 1 ? 0.016 : 0.008);
    if (gemm <= here) return launch_gemm_mixed(g, s);
  }
  // One CTA per SM takes the SM's shared memory, unless in clusters above 4: those
  // find room in a GPC only two to an SM (512 x 8192 x 1024, split 8: 25.8 us against 19.4).
  const int budget = (split <= 4 && split * blocks <= sms ? 212 : 104) * 1024;
  return g.N % 2 == 0 ? launch_stream<true>(g, s, tok, split, budget)
                      : launch_stream<false>(g, s, tok, split, budget);
}

}  // namespace

cudaError_t weight_stream_status_word(int32_t** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_stream_status);
}

}  // namespace i8mm

using namespace i8mm;

extern "C" int int8_scaled_matmul(const int8_t* Xq, const float* x_scale, const int8_t* Wq,
                                  const float* w_scale, int M, int N, int K, void* Y,
                                  int32_t* status, i8mm_stream_t stream) {
  int st = abi_check_sizes(M, N, K);
  if (st != I8MM_OK) return st;
  if (M == 0 || N == 0) return I8MM_OK;
  if (!Xq || !x_scale || !Wq || !w_scale || !Y) return I8MM_ERR_INVALID_ARG;
  auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!a16(Xq) || !a16(x_scale) || !a16(Wq) || !a16(w_scale) || !a16(Y)) return I8MM_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(status) & 3u) != 0) return I8MM_ERR_ALIGNMENT;
  if ((st = abi_check_device()) != I8MM_OK) return st;
  GemmArgs g{};
  g.Xq = Xq;
  g.Wq = Wq;
  g.x_scale = x_scale;
  g.w_scale = w_scale;
  g.n_outliers = nullptr;
  g.out = Y;
  g.M = M;
  g.N = N;
  g.K = K;
  g.status = status;
  g.ld = 64;
  return abi_cuda_fail("product kernel launch", launch_scaled(g, static_cast<cudaStream_t>(stream)));
}

extern "C" int int8_scaled_matmul_status(i8mm_stream_t stream) {
  int st = abi_check_device();
  if (st != I8MM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t* word[2] = {};
  int32_t h[2] = {};
  cudaError_t e = gemm_status_word(&word[0]);
  if (e == cudaSuccess) e = weight_stream_status_word(&word[1]);
  for (int i = 0; i < 2 && e == cudaSuccess; ++i)
    e = cudaMemcpyAsync(&h[i], word[i], 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  // Only a word that holds something is cleared: nothing is lost that comes in meanwhile.
  for (int i = 0; i < 2 && e == cudaSuccess; ++i)
    if (h[i] != 0) e = cudaMemsetAsync(word[i], 0, 4, s);
  if (e == cudaSuccess && (h[0] != 0 || h[1] != 0)) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();   // do not leave it for the next launch
    return abi_cuda_fail("status read", e);
  }
  return h[0] != 0 ? h[0] : h[1];
}
