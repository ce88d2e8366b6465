// Output head fused with its softmax cross-entropy (TP walkthrough 2kiu.com
// §6.2): loss, log-sum-exp and the gradients of X and of the vocab-sharded
// head weight from X and W, without keeping the scores z = X W^T.
//
//   lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,label
//   d_tv  = exp(z_tv - lse_t) - [v = label],  dX = scale * d W,  dW = scale * d^T X
//
// For a token whose label is all but certain both differences are small against what they
// are taken of: lse or the softmax rounded to fp32 would leave few digits of them. So the
// label stays out of the sum over the others, and with o their share and t the label's,
// both relative to the larger of the two maxima, loss = log1p(o / t) and the label's d is
// -o / (o + t), each good to a few roundings of its own size.
//
// Tokens are taken a chunk at a time. For bf16 plans the scores live only in the
// tensor cores' fp32 accumulators: the GEMM's epilogue leaves, per row and slot of
// 64 columns, their maximum m and sum of 2^(z log2 e - m), and, when
// gradients are wanted, the exponentials themselves in 16 bits (relative to the
// slot's maximum). A row kernel merges the slots (the running maximum and sum of a
// softmax, joined), adds the label's score, and turns the exponentials into d in
// place with one factor 2^(m - M) / (o + t) per slot; then the two products, whose
// epilogues apply the scale (in d's rounding to bf16 the labels' entries, all near
// -scale, would share one error, up to 2^-8 of the gradients). So each score is
// computed once: 6 T V h operations for loss and gradients, against
// 8 for recomputing the scores in the backward, at 6 bytes of traffic per score.
// fp32 plans keep the chunk's scores in fp32.
// Bound by the tensor cores: 4096 x 131072 x 4096 over 8 shards in 10.6-11.4 ms, 1160-1247
// TFLOP/s at the power limit of the GPU at hand (scores 3.4, rows 0.4, dX 3.2, dW 3.5 ms);
// 32768 tokens of it, in 8 chunks, 91 ms, 1159; 2048 x 32000 x 512 in 290 us replayed, 694
// TFLOP/s: its tiles have 8 K blocks, shorter than the epilogue; 61 tokens' losses in
// 55 us, W read once at 4.8 TB/s.
#include <algorithm>

#include "tp_device.cuh"
#include "tp_internal.h"

namespace {

using tpi::GemmBatch;
using tpi::GemmProblem;
using tpi::MutPtrArray;
using tpi::PtrArray;

constexpr unsigned kStatusBadIndex = 2u;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// (max, sum of 2^(x - max)) pairs in the log2 domain; {-inf, 0} is the empty set.
__device__ __forceinline__ float2 merge(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  if (m == -INFINITY) return make_float2(m, a.y + b.y);  // nothing yet (or NaN sums)
  return make_float2(m, a.y * tpd::ex2(a.x - m) + b.y * tpd::ex2(b.x - m));
}

// A row's softmax split into the label's share t and the others' o, both relative to 2^M.
struct Split {
  float M, o, t;
  __device__ __forceinline__ float sum() const { return o + t; }
  __device__ __forceinline__ float lse() const { return (M + log2f(sum())) * kLn2; }
};
// rest: (max, sum) of all columns but the label's, whose score is z (kept: a label that counts).
// t is taken from z itself, so that M's own rounding is in both shares alike.
__device__ __forceinline__ Split split_row(const float2& rest, bool kept, float z) {
  if (!kept) return Split{rest.x, rest.y, 0.f};
  const float M = fmaxf(rest.x, z * kLog2e);
  return Split{M, rest.y * tpd::ex2(rest.x - M), tpd::ex2(fmaf(z, kLog2e, -M))};
}
__device__ __forceinline__ float row_loss(const Split& s, const float2& rest, float z) {
  if (z * kLog2e >= rest.x) return log1pf(s.o / s.t);
  return (fmaf(-z, kLog2e, s.M) + log2f(s.sum())) * kLn2;  // at least log 2: nothing cancels
}

template <int THREADS>
__device__ __forceinline__ float2 block_merge(float2 v, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = merge(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float2 t = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) t = merge(t, red[w]);
  return t;
}

// One CTA per token row of fp32 scores z [rows, ld]: a pass for the running
// (max, sum), then (d != NULL) a pass that writes d, which may be z itself.
constexpr int kRowThreads = 512;
__global__ void __launch_bounds__(kRowThreads) ce_rows_kernel(const float* z, int64_t ld, int vocab, const int32_t* labels,
                                                              float scale, float* loss, float* lse_out, float* d,
                                                              unsigned* status) {
  tpd::pdl_entry();
  __shared__ float2 red[kRowThreads / 32];
  const int64_t t = blockIdx.x;
  const int label = labels[t];
  const bool ignore = label < 0 || label >= vocab;
  const float* row = z + t * ld;
  const float zl = ignore ? 0.f : row[label];  // read before block_merge's barrier: d may be z
  float2 acc = make_float2(-INFINITY, 0.f);
  for (int c = threadIdx.x * 4; c < vocab; c += kRowThreads * 4) {
    const float4 u = *reinterpret_cast<const float4*>(row + c);
    float x[4] = {u.x, u.y, u.z, u.w};
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (c + e >= vocab || c + e == label) x[e] = -INFINITY;
      m = fmaxf(m, x[e]);
    }
    m *= kLog2e;
    const float mo = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += tpd::ex2(fmaf(x[e], kLog2e, -mo));
    acc = merge(acc, make_float2(m, sum));
  }
  const float2 rest = block_merge<kRowThreads>(acc, red);
  const Split s = split_row(rest, !ignore, zl);
  if (threadIdx.x == 0) {
    if (label >= vocab) atomicOr(status, kStatusBadIndex);
    loss[t] = ignore ? 0.f : row_loss(s, rest, zl);
    if (lse_out) lse_out[t] = s.lse();
  }
  if (!d) return;
  float* drow = d + t * ld;
  const float k = scale / s.sum(), at_label = -(s.o / s.sum()) * scale;
  for (int64_t c = threadIdx.x * 4; c < ld; c += kRowThreads * 4) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (!ignore && c < vocab) {
      const float4 u = *reinterpret_cast<const float4*>(row + c);
      x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = c + e == label ? at_label : c + e < vocab ? tpd::ex2(fmaf(x[e], kLog2e, -s.M)) * k : 0.f;
    }
    *reinterpret_cast<float4*>(drow + c) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// Merges a row's slot statistics, adds the label's score and writes loss and
// lse; then (e != NULL) turns the row's exponentials into d in place.
// The label's score is a dot product of its own, in fp32 by the CTA: the tensor
// cores' long accumulation is less exact, and a confident token's loss is the
// difference of lse and this score. gridDim.y CTAs share a row's second part
// (few rows: the merge is short and repeated by each). lo_at != 0: d's rounding error,
// in bf16 too, goes lo_at vectors behind d, and x2 receives X twice.
constexpr int kFinThreads = 256;
__global__ void __launch_bounds__(kFinThreads) ce_finish_kernel(
    const float4* stats, int shard_pairs, const __nv_bfloat16* X,
    const __grid_constant__ PtrArray W, int h, int vocab, int Vs, int p, const int32_t* labels, float* loss,
    float* lse_out, uint4* e, int64_t lo_at, uint4* x2, unsigned* status) {
  tpd::pdl_entry();
  __shared__ float2 red[kFinThreads / 32];
  __shared__ float dot[kFinThreads / 32];
  const int64_t t = blockIdx.x;
  const int label = labels[t];
  const bool ignore = label < 0 || label >= vocab;
  float z = 0.f;
  if (!ignore) {
    const uint4* x = reinterpret_cast<const uint4*>(X + t * h);
    const int sh = label / Vs;
    const uint4* w = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(W.p[sh]) +
                                                    static_cast<int64_t>(label - sh * Vs) * h);
    for (int i = threadIdx.x; i < h / 8; i += kFinThreads) {
      const uint4 a = x[i], b = w[i];
      const uint32_t au[4] = {a.x, a.y, a.z, a.w}, bu[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = tpd::unpack_bf16x2(au[q]), g = tpd::unpack_bf16x2(bu[q]);
        z = fmaf(f.x, g.x, z);
        z = fmaf(f.y, g.y, z);
      }
    }
  }
  const float4* st = stats + t * p * shard_pairs;
  float2 acc = make_float2(-INFINITY, 0.f);
  for (int i = threadIdx.x; i < p * shard_pairs; i += kFinThreads) {
    const float4 v = st[i];
    acc = merge(acc, make_float2(v.x, v.y));
    if ((i % shard_pairs) * 128 + 64 < Vs) acc = merge(acc, make_float2(v.z, v.w));  // the pair's second slot has columns
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  if ((threadIdx.x & 31) == 0) dot[threadIdx.x >> 5] = z;
  const float2 rest = block_merge<kFinThreads>(acc, red);  // its barrier covers dot
  z = 0.f;
#pragma unroll
  for (int w = 0; w < kFinThreads / 32; ++w) z += dot[w];
  const Split sp = split_row(rest, !ignore, z);
  if (threadIdx.x == 0 && blockIdx.y == 0) {
    if (label >= vocab) atomicOr(status, kStatusBadIndex);
    loss[t] = ignore ? 0.f : row_loss(sp, rest, z);
    if (lse_out) lse_out[t] = sp.lse();
  }
  if (!e) return;
  if (x2 && blockIdx.y == 0) {  // X beside itself, for the two parts of d
    const uint4* x = reinterpret_cast<const uint4*>(X + t * h);
    for (int i = threadIdx.x; i < h / 8; i += kFinThreads) x2[t * (h / 8) + i] = x2[(t + gridDim.x) * (h / 8) + i] = x[i];
  }
  const int nv = Vs / 8, total = p * nv;  // 16-byte vectors of the row
  uint4* row = e + t * total;
  const int per = (total + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);
  const int lo = static_cast<int>(blockIdx.y) * per, hi = min(total, lo + per);
  if (ignore) {
    for (int i = lo + threadIdx.x; i < hi; i += kFinThreads) {
      row[i] = make_uint4(0, 0, 0, 0);
      if (lo_at) row[i + lo_at] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const float inv = 1.f / sp.sum(), at_label = -(sp.o / sp.sum());
#pragma unroll 4
  for (int i = lo + threadIdx.x; i < hi; i += kFinThreads) {
    const uint4 u = row[i];
    const int sh = i / nv, c = (i - sh * nv) * 8;
    const float4* at = st + sh * shard_pairs + c / 128;
    const float m = c & 64 ? at->z : at->x;  // -inf: all its exps are 0
    const float f = tpd::ex2(m - sp.M) * inv;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float d[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 v = tpd::unpack_unit16x2(w[q]);
      d[2 * q] = v.x * f;
      d[2 * q + 1] = v.y * f;
    }
    if (i == label / 8) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q == label % 8) d[q] = at_label;
    }
    const uint32_t r[4] = {tpd::pack_bf16x2(d[0], d[1]), tpd::pack_bf16x2(d[2], d[3]), tpd::pack_bf16x2(d[4], d[5]),
                           tpd::pack_bf16x2(d[6], d[7])};
    row[i] = make_uint4(r[0], r[1], r[2], r[3]);
    if (lo_at) {
      uint32_t s[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 v = tpd::unpack_bf16x2(r[q]);
        s[q] = tpd::pack_bf16x2(d[2 * q] - v.x, d[2 * q + 1] - v.y);
      }
      row[i + lo_at] = make_uint4(s[0], s[1], s[2], s[3]);
    }
  }
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Tokens per chunk: the caller's, or one chunk for all tokens unless chunks of
// about 1 GiB of scores make the workspace (scores and fp32 sums of dW) smaller.
int64_t pick_chunk(int64_t T, int64_t Vp, int64_t h, double score_bytes, bool dw_sums, int64_t asked) {
  if (asked > 0) return std::min(asked, T);
  const double all = static_cast<double>(T) * Vp * score_bytes;
  const double part = static_cast<double>(1u << 30);
  if (all <= part + (dw_sums ? 4.0 * Vp * h : 0.0)) return T;
  const int64_t most = std::max<int64_t>(1024, static_cast<int64_t>(part / (Vp * score_bytes)) / 256 * 256);
  const int64_t n = (T + most - 1) / most;
  return std::min(T, ((T + n - 1) / n + 255) / 256 * 256);
}

}  // namespace

namespace tpi {

// fp32 plans: the chunk's scores in fp32, a row kernel, and the FMA GEMM for the
// three products (the shards are blocks of rows of one matrix).
static tp_status linear_ce_f32(tp_plan* plan, int64_t T, const float* X, const PtrArray& W, const int32_t* labels,
                               float scale, float* loss, float* lse, float* dX, const MutPtrArray& dW, int64_t chunk,
                               unsigned* status, cudaStream_t st) {
  const int p = plan->p, h = plan->hidden, V = plan->vocab, Vp = plan->vocab_padded, Vs = Vp / p;
  const bool dw = dW.p[0] != nullptr, grad = dX || dw;
  const int64_t Tc = pick_chunk(T, Vp, h, 4.0, false, chunk), nch = (T + Tc - 1) / Tc;
  auto plain = [](const float* a, int64_t ld) {
    RowBlocks m{};
    m.p[0] = a;
    m.ld = ld;
    m.rows = 0x7fffffff;
    return m;
  };
  auto shards = [&](const void* const* a) {
    RowBlocks m{};
    for (int i = 0; i < p; ++i) m.p[i] = static_cast<const float*>(a[i]);
    m.ld = h;
    m.rows = Vs;
    return m;
  };
  auto scores = [&](float* z, int64_t t0, int64_t n) {
    return FmaGemm{static_cast<int>(n), Vp, h, plain(X + t0 * h, h), shards(W.p), plain(z, Vp), false, false, false, false};
  };
  // The gradients' products beside one another, the one's tiles filling the other's
  // last wave: 2048 x 16000 x 512 2326 -> 2072 us, 256 x 4000 x 256 124 -> 75, 500 x
  // 8201 x 512 326 -> 318, 2 x 1000 x 64 25 either way. Not bf16's, which take turns on whole SMs: 500 x 5003 x 1024
  // 54 -> 61 us.
  const bool both = dX && dw && side_free(plan);
  auto dx_gemm = [&](float* d, int64_t t0, int64_t n) {
    FmaGemm g{static_cast<int>(n), h, Vp, plain(d, Vp), shards(W.p), plain(dX + t0 * h, h), false, true, false, both};
    g.D.rows = g.M;
    return g;
  };
  auto dw_gemm = [&](float* d, int64_t t0, int64_t n) {
    return FmaGemm{Vp, h, static_cast<int>(n), plain(d, Vp), plain(X + t0 * h, h),
                   shards(const_cast<const void* const*>(dW.p)), true, true, t0 > 0, both};
  };
  const size_t z_bytes = round256(static_cast<size_t>(Tc) * Vp * 4);
  size_t part_bytes = 0, w_bytes = 0;  // over the first (longest) and the last chunk
  for (int64_t t0 : {static_cast<int64_t>(0), (nch - 1) * Tc}) {
    const int64_t n = std::min(Tc, T - t0);
    FmaGemm z = scores(nullptr, t0, n);
    z.D.rows = z.M;
    part_bytes = std::max(part_bytes, fma_gemm_scratch(z));
    if (dX) part_bytes = std::max(part_bytes, fma_gemm_scratch(dx_gemm(nullptr, t0, n)));
    if (dw) w_bytes = std::max(w_bytes, fma_gemm_scratch(dw_gemm(nullptr, t0, n)));
  }
  part_bytes = round256(part_bytes);
  const size_t w_at = both ? part_bytes : 0;
  void* ws = nullptr;
  TP_TRY(scratch(plan, z_bytes + std::max(part_bytes, w_at + w_bytes), st, &ws));
  float* z = static_cast<float*>(ws);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + z_bytes);
  float* w_part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + z_bytes + w_at);
  for (int64_t t0 = 0; t0 < T; t0 += Tc) {
    const int64_t n = std::min(Tc, T - t0);
    FmaGemm g = scores(z, t0, n);
    g.D.rows = g.M;
    TP_TRY(launch_fma_gemm(g, part, st));
    (void)launch(ce_rows_kernel, dim3(static_cast<unsigned>(n)), dim3(kRowThreads), 0, st, z, static_cast<int64_t>(Vp), V,
                 labels + t0, scale, loss + t0, lse ? lse + t0 : nullptr, grad ? z : nullptr, status);
    TP_TRY(after_launch("vocab_linear_cross_entropy rows"));
    const SideFork side(st, both);  // joined before the next chunk
    TP_TRY(side.status());
    if (dX) TP_TRY(launch_fma_gemm(dx_gemm(z, t0, n), part, st));
    if (dw) TP_TRY(launch_fma_gemm(dw_gemm(z, t0, n), w_part, side.stream()));
  }
  return TP_OK;
}

tp_status launch_vocab_linear_ce(tp_plan* plan, int64_t T, const void* X, const PtrArray& W, const int32_t* labels,
                                 float scale, float* loss, float* lse, void* dX, const MutPtrArray& dW, int64_t chunk,
                                 cudaStream_t st) {
  unsigned* status = nullptr;
  TP_TRY(device_status_word(&status));
  if (plan->dtype == TP_F32)
    return linear_ce_f32(plan, T, static_cast<const float*>(X), W, labels, scale, loss, lse, static_cast<float*>(dX), dW,
                         chunk, status, st);
  const int p = plan->p, h = plan->hidden, V = plan->vocab, Vp = plan->vocab_padded, Vs = Vp / p;
  constexpr size_t es = 2;
  const bool grad = dX || dW.p[0], dw = dW.p[0] != nullptr;
  // without gradients, 8 bytes are kept per slot of 64 scores
  const int64_t Tc = pick_chunk(T, Vp, h, grad ? 2.0 : 0.125, dw, chunk);
  const int64_t nch = (T + Tc - 1) / Tc;
  // Chunks of at most 64 tokens carry d in two bf16 parts, in 2n rows that still fit one
  // tile row of dX and, up to 32 tokens, one K block of dW: with few tokens a row of the
  // gradients has one or two large terms, whose rounding it would carry whole (relative
  // errors up to 0.004 in place of the result's own 0.0017).
  const bool two = grad && Tc <= 64;
  const int fold = two ? 2 : 1;

  // products with d of a chunk of n tokens starting at token t0
  auto dx_batch = [&](const void* d, int64_t t0, int64_t n) {
    GemmBatch b{};
    b.n = p;
    b.b_mn = true;
    b.epi = EPI_STORE;
    b.kcat = true;
    b.scaled = true;
    b.alpha = scale;
    for (int i = 0; i < p; ++i) {
      GemmProblem& g = b.g[i];
      g.M = static_cast<int>(fold * n);
      g.N = h;
      g.K = Vs;
      g.A = static_cast<const uint8_t*>(d) + static_cast<size_t>(i) * Vs * es;
      g.lda = Vp;
      g.B = W.p[i];
      g.ldb = h;
      g.D = static_cast<uint8_t*>(dX) + static_cast<size_t>(t0) * h * es;
      g.ldd = h;
    }
    return b;
  };
  const void* x2 = nullptr;  // X twice, beside d's two parts
  auto dw_batch = [&](const void* d, int64_t t0, int64_t n) {
    GemmBatch b{};
    b.n = p;
    b.a_mn = b.b_mn = true;
    b.epi = EPI_STORE;
    b.scaled = true;
    b.alpha = scale;
    for (int i = 0; i < p; ++i) {
      GemmProblem& g = b.g[i];
      g.M = Vs;
      g.N = h;
      g.K = static_cast<int>(fold * n);
      g.A = static_cast<const uint8_t*>(d) + static_cast<size_t>(i) * Vs * es;
      g.lda = Vp;
      g.B = two ? x2 : static_cast<const uint8_t*>(X) + static_cast<size_t>(t0) * h * es;
      g.ldb = h;
      g.D = dW.p[i];
      g.ldd = h;
    }
    return b;
  };

  // the scores of a chunk, of which the statistics (and the exponentials) are kept
  auto score_batch = [&](void* out, int64_t t0, int64_t n) {
    GemmBatch b{};
    b.n = p;
    b.epi = EPI_CE;
    for (int i = 0; i < p; ++i) {
      GemmProblem& g = b.g[i];
      g.M = static_cast<int>(n);
      g.N = Vs;
      g.K = h;
      g.A = static_cast<const uint8_t*>(X) + static_cast<size_t>(t0) * h * es;
      g.lda = h;
      g.B = W.p[i];
      g.ldb = h;
      g.D = out ? static_cast<uint8_t*>(out) + static_cast<size_t>(i) * Vs * es : nullptr;
      g.ldd = Vp;
    }
    b.ce_vocab = V;
    b.ce_labels = labels + t0;
    return b;
  };
  const int shard_pairs = (Vs + 127) / 128;  // pairs of slots, see GemmBatch::ce_stats

  // scratch: d (from the exponentials or scores) | statistics | fp32 sums of dW | split-K partials
  const int sx = dX ? gemm_cat_split(dx_batch(nullptr, 0, Tc), TP_MAX_SHARDS / fold) : 1;
  const int sw = dw && nch == 1 ? gemm_split_k(dw_batch(nullptr, 0, Tc)) : 1;
  const size_t d_bytes = grad ? round256(static_cast<size_t>(fold * Tc) * Vp * es) : 0;
  const size_t st_bytes = round256(static_cast<size_t>(Tc) * p * shard_pairs * sizeof(float4));
  const size_t acc_bytes = dw && nch > 1 ? round256(static_cast<size_t>(Vp) * h * 4) : 0;
  const bool x_parts = dX && (sx > 1 || two);
  const size_t part_bytes = round256(std::max(x_parts ? static_cast<size_t>(sx) * fold * Tc * h * 4 : 0,
                                              sw > 1 ? static_cast<size_t>(sw) * Vp * h * 4 : 0));
  const size_t x2_bytes = two && dw ? static_cast<size_t>(2 * Tc) * h * es : 0;
  void* ws = nullptr;
  TP_TRY(scratch(plan, d_bytes + st_bytes + acc_bytes + part_bytes + x2_bytes, st, &ws));
  uint8_t* db = static_cast<uint8_t*>(ws);
  float2* stats = reinterpret_cast<float2*>(db + d_bytes);
  float* acc = reinterpret_cast<float*>(db + d_bytes + st_bytes);
  float* part = reinterpret_cast<float*>(db + d_bytes + st_bytes + acc_bytes);
  uint4* xx = x2_bytes ? reinterpret_cast<uint4*>(db + d_bytes + st_bytes + acc_bytes + part_bytes) : nullptr;
  x2 = xx;

  for (int64_t c = 0; c < nch; ++c) {
    const int64_t t0 = c * Tc, n = std::min(Tc, T - t0);
    GemmBatch b = score_batch(grad ? db : nullptr, t0, n);
    b.ce_stats = stats;
    b.ce_pairs = static_cast<int64_t>(p) * shard_pairs;
    TP_TRY(launch_gemm_bf16(b, st));
    // a few rows: enough CTAs a row to fill the GPU with the second part
    const int64_t parts = grad ? std::max<int64_t>(1, std::min<int64_t>(512 / n, Vp / 8 / kFinThreads)) : 1;
    (void)launch(ce_finish_kernel, dim3(static_cast<unsigned>(n), static_cast<unsigned>(parts)), dim3(kFinThreads), 0, st,
                 reinterpret_cast<const float4*>(stats), shard_pairs, static_cast<const __nv_bfloat16*>(X) + t0 * h, W, h,
                 V, Vs, p, labels + t0, loss + t0, lse ? lse + t0 : nullptr,
                 grad ? reinterpret_cast<uint4*>(db) : nullptr, two ? n * (Vp / 8) : int64_t{0}, xx, status);
    TP_TRY(after_launch("vocab_linear_cross_entropy rows"));
    if (dX) {
      const GemmBatch x = dx_batch(db, t0, n);
      if (x_parts) TP_TRY(launch_gemm_cat_split(x, sx, part, st, fold));
      else TP_TRY(launch_gemm_bf16(x, st));
    }
    if (dw) {
      GemmBatch w = dw_batch(db, t0, n);
      if (sw > 1) {
        TP_TRY(launch_gemm_split(w, sw, part, st));
      } else {
        for (int i = 0; nch > 1 && i < p; ++i) {
          float* a = acc + static_cast<size_t>(i) * Vs * h;
          if (c > 0) {
            w.g[i].acc = a;
            w.g[i].ldacc = h;
          }
          if (c < nch - 1) w.g[i].D = a;
        }
        w.out_f32 = c < nch - 1;
        TP_TRY(launch_gemm_bf16(w, st));
      }
    }
  }
  return TP_OK;
}

}  // namespace tpi
