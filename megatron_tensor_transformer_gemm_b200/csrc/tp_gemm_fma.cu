// fp32 GEMM on the FMA units over matrices whose rows are spread over the shards:
// D[M, N] = A[M, K] . B[N, K]^T (+ D), every product and sum in fp32. The shards of
// a vocab-sharded weight are blocks of rows of one [Vp, hidden] matrix, so one
// launch covers all of them whichever dimension the vocab is: N (scores), K (the
// input gradient) or M (the weight gradient).
//
// A CTA of 256 threads computes a (16 TM) x 128 tile, a thread TM x 8 of it in
// registers, over K blocks that two shared-memory buffers hold in [K][M] and
// [K][N] order: the next block's global loads are in flight while this one is
// multiplied (for TM = 8 blocks of 8: 16 need registers that are not there, 2079 us for
// 2064 below).
// Two columns share an instruction (fma.f32x2, each lane rounded as the scalar one),
// the row's value doubled by moves, which use another pipe: half the instructions of
// the multiply-adds leave room for the loads, 2330 -> 2079 us; the value doubled in
// shared memory instead lost. It is bound by the FMA units (128 a clock and SM, 72
// TFLOP/s at the clocks seen): a head of 2048 x 16000 x 512 takes 2064 us for its three
// products, 49 TFLOP/s; 500 x 8201 x 512 313 us, whose 260 tiles fill 88 % of the
// places. TM = 8 does the work of a block in 32 paired multiply-adds per four 16-byte
// shared loads; 128 x 256 tiles with one CTA an SM took 2451. TM = 2 is for few rows,
// where the tile's height is what is wasted. Launches with few tiles split K: split s
// writes its own partial of D and an ordered reduce adds them (which also shortens the
// running sums).
#include <algorithm>

#include "tp_device.cuh"
#include "tp_internal.h"

namespace {

using tpi::FmaGemm;
using tpi::RowBlocks;

constexpr int kBN = 128;
// K blocks: 8 for tiles of 128 rows, else 16 (registers are free there, and few rows wait
// for their loads: 16 x 2000 x 128 in 23 us for 26).
template <int TM>
constexpr int kBK = TM == 8 ? 8 : 16;
constexpr int kMaxBK = 16;
constexpr int kPad = 4;  // keeps 16-byte shared loads aligned, store conflicts two-way

__device__ __forceinline__ const float* row_of(const RowBlocks& m, int r) {
  const int b = r < m.rows ? 0 : r / m.rows;
  return m.p[b] + static_cast<int64_t>(r - b * m.rows) * m.ld;
}

// A thread's 16-byte piece i of an operand's [ROWS x BK] tiles: 4 values along the
// operand's contiguous dimension. A K-major piece stays in its row, so its address is
// stepped; an MN-major one finds its row anew in each K block, which costs fewer
// registers than stepping it (where the kernel has none left).
template <int ROWS, bool MN, int BK>
struct Piece {
  const float* p;
  int k;  // its index in K; far past the end for rows the matrix does not have
  __device__ __forceinline__ void start(const RowBlocks& m, int i, int r0, int rows, int k0) {
    const int r = r0 + (MN ? i % (ROWS / 4) * 4 : i / (BK / 4));
    k = k0 + (MN ? i / (ROWS / 4) : i % (BK / 4) * 4);
    if (r >= rows) k = 1 << 30;
    p = nullptr;
    if constexpr (!MN) {
      if (r < rows) p = row_of(m, r) + k;
    }
  }
  __device__ __forceinline__ float4 next(const RowBlocks& m, int i, int r0, int k1) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k < k1) v = *reinterpret_cast<const float4*>(MN ? row_of(m, k) + (r0 + i % (ROWS / 4) * 4) : p);
    k += BK;
    if constexpr (!MN) p += BK;
    return v;
  }
};
template <int ROWS, bool MN, int BK>
__device__ __forceinline__ void store_piece(float (*s)[ROWS + kPad], int i, const float4& v) {
  if constexpr (MN) {
    *reinterpret_cast<float4*>(&s[i / (ROWS / 4)][i % (ROWS / 4) * 4]) = v;
  } else {
    const int r = i / (BK / 4), k = i % (BK / 4) * 4;
    s[k][r] = v.x;
    s[k + 1][r] = v.y;
    s[k + 2][r] = v.z;
    s[k + 3][r] = v.w;
  }
}

template <int TM, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(256, 2) fma_gemm_kernel(const __grid_constant__ FmaGemm g, int tiles_n, int k_split,
                                                          float* part) {
  tpd::pdl_entry();
  constexpr int BM = 16 * TM, BK = kBK<TM>;
  constexpr int APIECES = BM * BK / 4, ALOADS = (APIECES + 255) / 256, BLOADS = kBN * BK / 4 / 256;
  __shared__ __align__(16) float sA[2][BK][BM + kPad];
  __shared__ __align__(16) float sB[2][BK][kBN + kPad];
  const int tid = threadIdx.x, tx = (tid >> 5 & 1) * 8 + (tid & 7), ty = (tid >> 6) * 4 + (tid >> 3 & 3);
  const int mt = static_cast<int>(blockIdx.x) / tiles_n, nt = static_cast<int>(blockIdx.x) - mt * tiles_n;
  const int m0 = mt * BM, n0 = nt * kBN;
  const int k0 = static_cast<int>(blockIdx.y) * k_split, k1 = min(g.K, k0 + k_split);

  uint64_t acc[TM][4];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0;

  float4 ra[ALOADS], rb[BLOADS];
  Piece<BM, A_MN, BK> pa[ALOADS];
  Piece<kBN, B_MN, BK> pb[BLOADS];
#pragma unroll
  for (int l = 0; l < ALOADS; ++l) pa[l].start(g.A, tid + l * 256, m0, g.M, k0);
#pragma unroll
  for (int l = 0; l < BLOADS; ++l) pb[l].start(g.B, tid + l * 256, n0, g.N, k0);
  auto load = [&]() {
#pragma unroll
    for (int l = 0; l < ALOADS; ++l)
      if (APIECES % 256 == 0 || tid + l * 256 < APIECES) ra[l] = pa[l].next(g.A, tid + l * 256, m0, k1);
#pragma unroll
    for (int l = 0; l < BLOADS; ++l) rb[l] = pb[l].next(g.B, tid + l * 256, n0, k1);
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int l = 0; l < ALOADS; ++l)
      if (APIECES % 256 == 0 || tid + l * 256 < APIECES) store_piece<BM, A_MN, BK>(sA[buf], tid + l * 256, ra[l]);
#pragma unroll
    for (int l = 0; l < BLOADS; ++l) store_piece<kBN, B_MN, BK>(sB[buf], tid + l * 256, rb[l]);
  };
  load();
  store(0);
  __syncthreads();
  int buf = 0;
  for (int kb = k0; kb < k1; kb += BK) {
    if (kb + BK < k1) load();
#pragma unroll
    for (int k = 0; k < BK; ++k) {
      float a[TM];
      if constexpr (TM == 8) {
        const float4 u = *reinterpret_cast<const float4*>(&sA[buf][k][ty * 4]);
        const float4 v = *reinterpret_cast<const float4*>(&sA[buf][k][BM / 2 + ty * 4]);
        a[0] = u.x; a[1] = u.y; a[2] = u.z; a[3] = u.w;
        a[4] = v.x; a[5] = v.y; a[6] = v.z; a[7] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < TM; ++i) a[i] = sA[buf][k][ty * TM + i];
      }
      const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(&sB[buf][k][tx * 4]);
      const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&sB[buf][k][kBN / 2 + tx * 4]);
      const uint64_t bb[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
      for (int i = 0; i < TM; ++i) {  // columns in pairs
        const uint64_t aa = tpd::f2_pack(a[i], a[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[i][j]) : "l"(aa), "l"(bb[j]));
      }
    }
    if (kb + BK < k1) store(buf ^ 1);
    __syncthreads();  // the next block is in place, and this one has been read
    buf ^= 1;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = m0 + (TM == 8 ? (i / 4) * (BM / 2) + ty * 4 + i % 4 : ty * TM + i);
    if (m >= g.M) continue;
    float* row = part ? part + (static_cast<int64_t>(blockIdx.y) * g.M + m) * g.N : const_cast<float*>(row_of(g.D, m));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int n = n0 + q * (kBN / 2) + tx * 4;
      if (n >= g.N) continue;
      const float2 lo = tpd::f2_unpack(acc[i][2 * q]), hi = tpd::f2_unpack(acc[i][2 * q + 1]);
      float4 v = make_float4(lo.x, lo.y, hi.x, hi.y);
      if (g.add && !part) {
        const float4 o = *reinterpret_cast<const float4*>(row + n);
        v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
      }
      *reinterpret_cast<float4*>(row + n) = v;
    }
  }
}

int sm_count() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = 148;
  }
  return n;
}

// Rows per tile (32 for at most 64 rows of D, else 128), and the K split that
// brings the launch nearest to two CTAs per SM (at most 16, at least 128 of K each).
struct Shape {
  int tm, tiles_n, tiles, splits, k_split;
};
Shape shape_of(const FmaGemm& g) {
  Shape s{};
  s.tm = g.M <= 64 ? 2 : 8;
  s.tiles_n = (g.N + kBN - 1) / kBN;
  s.tiles = (g.M + 16 * s.tm - 1) / (16 * s.tm) * s.tiles_n;
  const int want = g.add ? 1 : std::max(1, 2 * sm_count() / s.tiles);
  int n = std::max(1, std::min({want, TP_MAX_SHARDS, g.K / 128}));
  s.k_split = ((g.K + n - 1) / n + kMaxBK - 1) / kMaxBK * kMaxBK;
  s.splits = (g.K + s.k_split - 1) / s.k_split;
  return s;
}

}  // namespace

namespace tpi {

size_t fma_gemm_scratch(const FmaGemm& g) {
  const Shape s = shape_of(g);
  return s.splits > 1 ? static_cast<size_t>(s.splits) * g.M * g.N * sizeof(float) : 0;
}

tp_status launch_fma_gemm(const FmaGemm& g, float* part, cudaStream_t st) {
  const Shape s = shape_of(g);
  float* p = s.splits > 1 ? part : nullptr;
  const dim3 grid(static_cast<unsigned>(s.tiles), static_cast<unsigned>(s.splits));
  // Two kernels that follow a fork of streams overlap only when neither is launched
  // programmatically: with the attribute the second began after the first had ended
  // (launched one by one, 2048 x 16000 x 512 took 2583 us in place of 2338).
  const bool early = pdl_enabled() && !g.beside;
#define TP_FMA(TM, AM, BM) (void)launch_as(early, fma_gemm_kernel<TM, AM, BM>, grid, dim3(256), 0, st, g, s.tiles_n, s.k_split, p)
#define TP_FMA_TM(AM, BM)                 \
  do {                                    \
    if (s.tm == 2) TP_FMA(2, AM, BM);     \
    else TP_FMA(8, AM, BM);               \
  } while (0)
  if (!g.a_mn && !g.b_mn) TP_FMA_TM(false, false);
  else if (!g.a_mn) TP_FMA_TM(false, true);
  else if (g.b_mn) TP_FMA_TM(true, true);
  else return fail(TP_ERR_ARG, "fp32 GEMM: operand layouts");
#undef TP_FMA_TM
#undef TP_FMA
  TP_TRY(after_launch("fma_gemm"));
  if (!p) return TP_OK;
  PtrArray P{};
  MutPtrArray out{};
  for (int i = 0; i < s.splits; ++i) P.p[i] = p + static_cast<size_t>(i) * g.M * g.N;
  const int blocks = (g.M + g.D.rows - 1) / g.D.rows;
  for (int i = 0; i < blocks; ++i) out.p[i] = const_cast<float*>(g.D.p[i]);
  return launch_reduce(P, s.splits, nullptr, nullptr, PtrArray{}, false, out, blocks > 1, blocks, g.M, g.N, TP_F32, TP_F32,
                       st);
}

}  // namespace tpi
