// The junction of two sublayers, forward and backward: the block's output f is
// normalised, gated and added to the scaled residual stream, and the next
// block's input is normalised from the sum (TP walkthrough 2kiu.com §3.3: the
// statistics span the whole hidden dim of a row).
//
//   n = Norm_post(f)  (or f),  x_out = rs * x + g n,  y = Norm_pre(x_out)
//
// Norm is LayerNorm or RMSNorm with fp32 statistics; y is taken from x_out as it
// is stored. The gate g has gate_rows rows, row r of the tokens using row
// r % gate_rows: 1 is a gate per channel, `batch` a gate per sequence of
// sequence-major tokens.
#include <algorithm>

#include "tp_device.cuh"
#include "tp_internal.h"

namespace {

using tpi::GatedNorm;

constexpr float kEps = 1e-5f;

template <typename T>
struct Vec16 {
  static constexpr int N = 16 / sizeof(T);
  __device__ static void unpack(const uint4 u, float (&f)[N]) {
    if constexpr (sizeof(T) == 2) {
      const float2 a = tpd::unpack_bf16x2(u.x), b = tpd::unpack_bf16x2(u.y), c = tpd::unpack_bf16x2(u.z),
                   d = tpd::unpack_bf16x2(u.w);
      f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y; f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
    } else {
      f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
      f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    }
  }
  __device__ static uint4 pack(const float (&f)[N]) {
    if constexpr (sizeof(T) == 2)
      return make_uint4(tpd::pack_bf16x2(f[0], f[1]), tpd::pack_bf16x2(f[2], f[3]), tpd::pack_bf16x2(f[4], f[5]),
                        tpd::pack_bf16x2(f[6], f[7]));
    else
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// Sum over the CTA, the same in every thread. `red` has two halves used in turn
// (`turn` counts the sums), so one barrier a sum is enough: a half is written
// again only after the barrier of the sum in between.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* red, int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (THREADS == 32) return v;
  float* half = red + (turn++ & 1) * (THREADS / 32);
  if ((threadIdx.x & 31) == 0) half[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) s += half[w];
  return s;
}

// Mean and reciprocal deviation of the row held in v (thread tid owns vectors
// tid + i * THREADS): the mean, then the mean square about it, two exact passes
// over the registers (RMSNorm: the second only, about zero).
template <typename T, int THREADS, int VPT, bool RMS>
__device__ __forceinline__ void row_stats(const uint4 (&v)[VPT], int vpr, float inv_h, float* red, int& turn, float& mean,
                                          float& rstd) {
  constexpr int N = Vec16<T>::N;
  mean = 0.f;
  if (!RMS) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {  // vectors past the row hold zeros
      float x[N];
      Vec16<T>::unpack(v[i], x);
#pragma unroll
      for (int e = 0; e < N; ++e) s += x[e];
    }
    mean = block_sum<THREADS>(s, red, turn) * inv_h;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (threadIdx.x + i * THREADS < vpr) {
      float x[N];
      Vec16<T>::unpack(v[i], x);
#pragma unroll
      for (int e = 0; e < N; ++e) q += (x[e] - mean) * (x[e] - mean);
    }
  }
  rstd = rsqrtf(block_sum<THREADS>(q, red, turn) * inv_h + kEps);
}

// One CTA per row; the row of x and of f stay packed in registers from their
// one load to the stores, so the two norms cost no extra pass over memory.
template <typename T, int THREADS, int VPT, bool RMS>
__global__ void __launch_bounds__(THREADS) gated_norm_fwd_kernel(const __grid_constant__ GatedNorm p) {
  tpd::pdl_entry();
  constexpr int N = Vec16<T>::N;
  __shared__ float red[2 * (THREADS / 32)];
  const int64_t r = blockIdx.x;
  const int vpr = static_cast<int>(p.h / N);
  const float inv_h = 1.f / static_cast<float>(p.h);
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + r * p.h);
  const uint4* f = reinterpret_cast<const uint4*>(static_cast<const T*>(p.f) + r * p.h);
  const uint4* gate =
      p.gate ? reinterpret_cast<const uint4*>(static_cast<const T*>(p.gate) + r % p.gate_rows * p.h) : nullptr;
  int turn = 0;
  uint4 fv[VPT], xv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * THREADS;
    fv[i] = xv[i] = make_uint4(0, 0, 0, 0);
    if (c < vpr) {
      fv[i] = __ldcs(f + c);
      xv[i] = __ldcs(x + c);
    }
  }
  float mean = 0.f, rstd = 1.f;
  if (p.post_g) {
    row_stats<T, THREADS, VPT, RMS>(fv, vpr, inv_h, red, turn, mean, rstd);
    if (p.stats && threadIdx.x == 0) {
      if (!RMS) p.stats[r] = mean;
      p.stats[p.rows + r] = rstd;
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * THREADS;
    if (c >= vpr) continue;
    float a[N], b[N], w[N];
    Vec16<T>::unpack(fv[i], a);
    Vec16<T>::unpack(xv[i], b);
    if (p.post_g) {
      Vec16<T>::unpack(static_cast<const uint4*>(p.post_g)[c], w);
#pragma unroll
      for (int e = 0; e < N; ++e) a[e] = (a[e] - mean) * rstd * w[e];
      if (!RMS) {
        Vec16<T>::unpack(static_cast<const uint4*>(p.post_b)[c], w);
#pragma unroll
        for (int e = 0; e < N; ++e) a[e] += w[e];
      }
    }
    if (gate) {
      Vec16<T>::unpack(gate[c], w);
#pragma unroll
      for (int e = 0; e < N; ++e) a[e] *= w[e];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) a[e] = fmaf(p.rs, b[e], a[e]);
    xv[i] = Vec16<T>::pack(a);  // rounded: what the next norm and the backward read
    reinterpret_cast<uint4*>(static_cast<T*>(p.x_out) + r * p.h)[c] = xv[i];
  }
  if (!p.pre_g) return;
  row_stats<T, THREADS, VPT, RMS>(xv, vpr, inv_h, red, turn, mean, rstd);
  if (p.stats && threadIdx.x == 0) {
    if (!RMS) p.stats[2 * p.rows + r] = mean;
    p.stats[3 * p.rows + r] = rstd;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * THREADS;
    if (c >= vpr) continue;
    float a[N], w[N];
    Vec16<T>::unpack(xv[i], a);
    Vec16<T>::unpack(static_cast<const uint4*>(p.pre_g)[c], w);
#pragma unroll
    for (int e = 0; e < N; ++e) a[e] = (a[e] - mean) * rstd * w[e];
    if (!RMS) {
      Vec16<T>::unpack(static_cast<const uint4*>(p.pre_b)[c], w);
#pragma unroll
      for (int e = 0; e < N; ++e) a[e] += w[e];
    }
    reinterpret_cast<uint4*>(static_cast<T*>(p.y) + r * p.h)[c] = Vec16<T>::pack(a);
  }
}

// ------------------------------------------------------------------ backward
// With xh the normalised rows, D = dx_out + rstd2 (dy g2 - m1 - xh2 m2) is the
// gradient of x_out (m1 = mean(dy g2), m2 = mean(dy g2 xh2); m1 = 0 for RMSNorm),
// dx = rs D, and with a = g D g1 the gradient of f is rstd1 (a - mean(a) - xh1
// mean(a xh1)). Sums over rows: P = sum dy xh2 and Q = sum dy are the pre-norm's
// parameter gradients; A = sum D xh1 and S = sum D, kept per gate row, give the
// gate's (g1 A + b1 S) and the post-norm's (sum over gate rows of g A, g S).
//
// Persistent CTAs: the tokens in gate-row-major order (position q = b * n + j is
// token j * gate_rows + b) are cut into one contiguous range per CTA, so a CTA
// sums A and S over runs of one gate row and writes a run's sums once; the run
// of CTA c and gate row b has slot c + b, since both only grow along the order.
// A row's inputs arrive by bulk copies a few rows ahead; a thread owns the same
// columns of every row and keeps its column sums in registers. No atomics: the
// sums are added in a fixed order by a second kernel.
constexpr int kStages = 3;

__device__ __forceinline__ int64_t range_lo(int64_t rows, int64_t G, int64_t c) { return rows * c / G; }
// The CTA whose range holds position q.
__device__ __forceinline__ int64_t range_of(int64_t rows, int64_t G, int64_t q) { return ((q + 1) * G - 1) / rows; }

// Sum of a pair over the CTA (or the CL CTAs of a cluster that share a row) and
// whether every thread's wait succeeded; one barrier, buffers used in turn.
template <int THREADS, int CL>
__device__ __forceinline__ bool pair_sum(float2& v, bool ok, float4* red, int& turn, uint32_t rank) {
  constexpr int W = THREADS / 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  const bool all = __all_sync(0xffffffffu, ok);
  float4* half = red + (turn++ & 1) * (W * CL);
  if ((threadIdx.x & 31) == 0) {
    const float4 mine = make_float4(v.x, v.y, all ? 0.f : 1.f, 0.f);
    float4* slot = half + rank * W + (threadIdx.x >> 5);
    *slot = mine;
    if (CL == 2) {
      const uint32_t far = tpd::map_shared(tpd::smem_u32(slot), rank ^ 1u);
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(far), "f"(mine.x), "f"(mine.y), "f"(mine.z),
                   "f"(mine.w)
                   : "memory");
    }
  }
  if (CL == 2) tpd::cluster_sync_all();
  else __syncthreads();
  float bad = 0.f;
  v = make_float2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < W * CL; ++w) {
    const float4 t = half[w];
    v.x += t.x;
    v.y += t.y;
    bad += t.z;
  }
  return bad == 0.f;
}

template <typename T, int THREADS, int VPT, int CL, bool RMS>
__global__ void __launch_bounds__(THREADS) gated_norm_bwd_kernel(const __grid_constant__ GatedNorm p, int64_t G, int narr,
                                                                 int vec_cta, unsigned* status) {
  constexpr int N = Vec16<T>::N;
  extern __shared__ __align__(128) uint8_t sbuf[];
  __shared__ uint64_t bar[kStages];
  __shared__ int abort_flag;
  __shared__ float4 red[2 * CL * (THREADS / 32)];
  const uint32_t rank = CL == 2 ? tpd::cluster_ctarank() : 0u;
  const int64_t cta = blockIdx.x / CL;
  const int vpr = static_cast<int>(p.h / N);
  const int v0 = static_cast<int>(rank) * vec_cta;              // this CTA's vectors of a row
  const int nv = min(vec_cta, vpr - v0);
  const uint32_t slice = static_cast<uint32_t>(nv) * 16u;
  const float inv_h = 1.f / static_cast<float>(p.h);
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < kStages; ++s) tpd::mbar_init(&bar[s], 1);
    tpd::fence_barrier_init();
  }
  __syncthreads();
  if (CL == 2) tpd::cluster_sync_all();  // the peer runs before its shared memory is written
  tpd::pdl_entry();

  const bool pre = p.pre_g != nullptr, post = p.post_g != nullptr, use_f = post || p.gate;
  const int64_t lo = range_lo(p.rows, G, cta), hi = range_lo(p.rows, G, cta + 1);
  const int64_t B = p.gate ? p.gate_rows : 1, per = p.rows / B;
  auto token = [&](int64_t q) { const int64_t b = q / per; return (q - b * per) * B + b; };
  // arrays of a stage, in order of presence: dx_out, then x_out and dy, then f
  const int o_dx = 0, o_x = (p.dx_out ? 1 : 0), o_f = o_x + (pre ? 2 : 0);
  const uint32_t arr = static_cast<uint32_t>(vec_cta) * 16u, stage_bytes = arr * narr;
  auto issue = [&](int64_t q) {  // thread 0
    const int s = static_cast<int>((q - lo) % kStages);
    const int64_t off = token(q) * p.h + static_cast<int64_t>(v0) * N;
    uint8_t* dst = sbuf + static_cast<size_t>(s) * stage_bytes;
    tpd::mbar_arrive_expect_tx(&bar[s], slice * narr);
    if (p.dx_out) tpd::bulk_load(dst, static_cast<const T*>(p.dx_out) + off, slice, &bar[s]);
    if (pre) {
      tpd::bulk_load(dst + o_x * arr, static_cast<const T*>(p.x_in) + off, slice, &bar[s]);
      tpd::bulk_load(dst + (o_x + 1) * arr, static_cast<const T*>(p.dy) + off, slice, &bar[s]);
    }
    if (use_f) tpd::bulk_load(dst + o_f * arr, static_cast<const T*>(p.f) + off, slice, &bar[s]);
  };
  int64_t issued = lo;
  if (threadIdx.x == 0)
    for (; issued < hi && issued < lo + kStages; ++issued) issue(issued);

  uint4 g2[VPT], w1[VPT], gw[VPT];  // pre-norm weight, post-norm weight, gate row
  float P[VPT][N], Q[VPT][N], A[VPT][N], S[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * THREADS;
    g2[i] = w1[i] = gw[i] = make_uint4(0, 0, 0, 0);
    if (c < nv && pre) g2[i] = static_cast<const uint4*>(p.pre_g)[v0 + c];
    if (c < nv && post) w1[i] = static_cast<const uint4*>(p.post_g)[v0 + c];
#pragma unroll
    for (int e = 0; e < N; ++e) P[i][e] = Q[i][e] = A[i][e] = S[i][e] = 0.f;
  }
  // A run of one gate row ends: its sums to slot cta + b.
  auto flush = [&](int64_t b) {
    float* out = p.seg + (cta + b) * 2 * p.h;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * THREADS;
      if (c < nv) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          float* at = out + static_cast<int64_t>(v0 + c) * N + e;
          *reinterpret_cast<float4*>(at) = make_float4(A[i][e], A[i][e + 1], A[i][e + 2], A[i][e + 3]);
          if (!RMS) *reinterpret_cast<float4*>(at + p.h) = make_float4(S[i][e], S[i][e + 1], S[i][e + 2], S[i][e + 3]);
        }
      }
#pragma unroll
      for (int e = 0; e < N; ++e) A[i][e] = S[i][e] = 0.f;
    }
  };

  int turn = 0;
  int64_t run = -1;  // gate row of the current run
  float st_m1 = 0.f, st_r1 = 1.f, st_m2 = 0.f, st_r2 = 1.f;
  auto load_stats = [&](int64_t t) {
    if (post) {
      if (!RMS) st_m1 = p.stats[t];
      st_r1 = p.stats[p.rows + t];
    }
    if (pre) {
      if (!RMS) st_m2 = p.stats[2 * p.rows + t];
      st_r2 = p.stats[3 * p.rows + t];
    }
  };
  if (lo < hi) load_stats(token(lo));
  bool good = true;
  for (int64_t q = lo; q < hi; ++q) {
    const int64_t k = q - lo, t = token(q), b = q / per;
    const int s = static_cast<int>(k % kStages);
    if (b != run) {
      if (run >= 0 && use_f) flush(run);
      run = b;
      if (p.gate) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = threadIdx.x + i * THREADS;
          if (c < nv)
            gw[i] = reinterpret_cast<const uint4*>(static_cast<const T*>(p.gate) + b * p.h)[v0 + c];
        }
      }
    }
    const float mean1 = st_m1, rstd1 = st_r1, mean2 = st_m2, rstd2 = st_r2;
    if (q + 1 < hi) load_stats(token(q + 1));  // a row early
    // a wait that gave up computes on an unfinished stage; the sum below then
    // stops every thread of the row before anything is written
    const bool ok = tpd::mbar_wait(&bar[s], static_cast<uint32_t>(k / kStages) & 1u, &abort_flag, status);
    const uint8_t* stage = sbuf + static_cast<size_t>(s) * stage_bytes;
    const uint4* s_dx = reinterpret_cast<const uint4*>(stage + o_dx * arr);
    const uint4* s_x = reinterpret_cast<const uint4*>(stage + o_x * arr);
    const uint4* s_dy = reinterpret_cast<const uint4*>(stage + (o_x + 1) * arr);
    const uint4* s_f = reinterpret_cast<const uint4*>(stage + o_f * arr);
    float2 m = make_float2(0.f, 0.f);
    if (pre) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * THREADS;
        if (c < nv) {
          float x[N], d[N], w[N];
          Vec16<T>::unpack(s_x[c], x);
          Vec16<T>::unpack(s_dy[c], d);
          Vec16<T>::unpack(g2[i], w);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float xh = (x[e] - mean2) * rstd2, gy = d[e] * w[e];
            if (!RMS) m.x += gy;
            m.y = fmaf(gy, xh, m.y);
            P[i][e] = fmaf(d[e], xh, P[i][e]);
            if (!RMS) Q[i][e] += d[e];
          }
        }
      }
    }
    good = pair_sum<THREADS, CL>(m, ok, red, turn, rank);
    if (!good) break;
    // every thread is past the row before this one: its stage takes a new row
    if (threadIdx.x == 0 && k >= 1 && issued < hi) issue(issued++);
    m.x *= inv_h;
    m.y *= inv_h;
    float a[VPT][N];
    float2 u = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * THREADS;
      if (c >= nv) continue;
      float D[N], o[N];
#pragma unroll
      for (int e = 0; e < N; ++e) D[e] = 0.f;
      if (p.dx_out) Vec16<T>::unpack(s_dx[c], D);
      if (pre) {
        float x[N], d[N], w[N];
        Vec16<T>::unpack(s_x[c], x);
        Vec16<T>::unpack(s_dy[c], d);
        Vec16<T>::unpack(g2[i], w);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float xh = (x[e] - mean2) * rstd2;
          D[e] = fmaf(rstd2, d[e] * w[e] - (RMS ? 0.f : m.x) - xh * m.y, D[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = p.rs * D[e];
      reinterpret_cast<uint4*>(static_cast<T*>(p.dx) + t * p.h)[v0 + c] = Vec16<T>::pack(o);
      float x[N], w[N];
      if (use_f) {
        Vec16<T>::unpack(s_f[c], x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          x[e] = (x[e] - mean1) * rstd1;
          A[i][e] = fmaf(D[e], x[e], A[i][e]);
          if (!RMS) S[i][e] += D[e];
        }
      }
      if (p.gate) {
        Vec16<T>::unpack(gw[i], w);
#pragma unroll
        for (int e = 0; e < N; ++e) D[e] *= w[e];
      }
      if (post) {
        Vec16<T>::unpack(w1[i], w);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          D[e] *= w[e];
          if (!RMS) u.x += D[e];
          u.y = fmaf(D[e], x[e], u.y);
        }
      }
#pragma unroll
      for (int e = 0; e < N; ++e) a[i][e] = D[e];
    }
    if (post) {
      good = pair_sum<THREADS, CL>(u, true, red, turn, rank);
      u.x *= inv_h;
      u.y *= inv_h;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * THREADS;
      if (c >= nv) continue;
      if (post) {
        float x[N];
        Vec16<T>::unpack(s_f[c], x);
#pragma unroll
        for (int e = 0; e < N; ++e)
          a[i][e] = rstd1 * (a[i][e] - (RMS ? 0.f : u.x) - (x[e] - mean1) * rstd1 * u.y);
      }
      reinterpret_cast<uint4*>(static_cast<T*>(p.df) + t * p.h)[v0 + c] = Vec16<T>::pack(a[i]);
    }
  }
  if (good) {
    if (run >= 0 && use_f) flush(run);
    if (pre) {
      float* out = p.cta_part + cta * 2 * p.h;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * THREADS;
        if (c < nv) {
#pragma unroll
          for (int e = 0; e < N; e += 4) {
            float* at = out + static_cast<int64_t>(v0 + c) * N + e;
            *reinterpret_cast<float4*>(at) = make_float4(P[i][e], P[i][e + 1], P[i][e + 2], P[i][e + 3]);
            if (!RMS) *reinterpret_cast<float4*>(at + p.h) = make_float4(Q[i][e], Q[i][e + 1], Q[i][e + 2], Q[i][e + 3]);
          }
        }
      }
    }
  } else if (threadIdx.x == 0) {
    // let the loads still in flight land (bounded) before the CTA exits
    for (int s = 0; s < kStages; ++s) {
      int again = 0;
      const int64_t n = issued - lo;  // rows issued; stage s holds the last with index = s mod kStages
      if (n > s) {
        const int64_t last = s + (n - 1 - s) / kStages * kStages;
        tpd::mbar_wait(&bar[s], static_cast<uint32_t>(last / kStages) & 1u, &again, nullptr, 1000000ull);
      }
    }
  }
  if (CL == 2) tpd::cluster_sync_all();  // neither CTA leaves while its peer may still write to it
}

// The column sums of the backward, each in a fixed order: a block owns 32
// columns, warp w takes CTAs w, w + 8, ... and the warps' sums are added in
// order. blockIdx.y = 0: the norms' parameters (and a single gate row);
// blockIdx.y = b + 1: gate row b of several.
constexpr int kSumWarps = 8;
template <typename T>
__global__ void __launch_bounds__(32 * kSumWarps) gated_norm_sums_kernel(const __grid_constant__ GatedNorm p, int64_t G, int rms) {
  tpd::pdl_entry();
  __shared__ float red[6][kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int64_t B = p.gate ? p.gate_rows : 1, per = p.rows / B;
  const bool use_f = p.post_g || p.gate;
  const bool all = blockIdx.y == 0;
  float v[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // P, Q, sum of g A, of g S, A, S
  if (col < p.h) {
    int64_t c0 = 0, c1 = G;
    if (!all) {
      c0 = range_of(p.rows, G, (blockIdx.y - 1) * per);
      c1 = range_of(p.rows, G, blockIdx.y * per - 1) + 1;
    }
#pragma unroll 4
    for (int64_t c = c0 + warp; c < c1; c += kSumWarps) {
      if (all && p.pre_g) {
        v[0] += p.cta_part[(c * 2) * p.h + col];
        if (!rms) v[1] += p.cta_part[(c * 2 + 1) * p.h + col];
      }
      if (use_f) {
        int64_t b0 = range_lo(p.rows, G, c) / per, b1 = (range_lo(p.rows, G, c + 1) - 1) / per;
        if (!all) b0 = b1 = blockIdx.y - 1;
        for (int64_t b = b0; b <= b1; ++b) {
          const float A = p.seg[((c + b) * 2) * p.h + col], S = rms ? 0.f : p.seg[((c + b) * 2 + 1) * p.h + col];
          if (all) {
            const float g = p.gate ? static_cast<float>(static_cast<const T*>(p.gate)[b * p.h + col]) : 1.f;
            v[2] = fmaf(g, A, v[2]);
            v[3] = fmaf(g, S, v[3]);
          }
          v[4] += A;
          v[5] += S;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) red[i][warp][lane] = v[i];
  __syncthreads();
  if (warp != 0 || col >= p.h) return;
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    v[i] = red[i][0][lane];
#pragma unroll
    for (int w = 1; w < kSumWarps; ++w) v[i] += red[i][w][lane];
  }
  if (all) {
    if (p.dpre_g) p.dpre_g[col] = v[0];
    if (p.dpre_b && !rms) p.dpre_b[col] = v[1];
    if (p.dpost_g) p.dpost_g[col] = v[2];
    if (p.dpost_b && !rms) p.dpost_b[col] = v[3];
  }
  if (p.dgate && (all ? B == 1 : true)) {
    const float g1 = p.post_g ? static_cast<float>(static_cast<const T*>(p.post_g)[col]) : 1.f;
    const float b1 = p.post_g && !rms ? static_cast<float>(static_cast<const T*>(p.post_b)[col]) : 0.f;
    p.dgate[(all ? 0 : blockIdx.y - 1) * p.h + col] = g1 * v[4] + b1 * v[5];
  }
}

// ---------------------------------------------------------------- dispatch
// Threads and vectors per thread of the forward, by the row's 16-byte vectors.
template <typename T, bool RMS>
void launch_fwd(const GatedNorm& p, cudaStream_t st) {
  const int64_t v = p.h * static_cast<int64_t>(sizeof(T)) / 16;
  const dim3 grid(static_cast<unsigned>(p.rows));
  if (v <= 32) (void)tpi::launch(gated_norm_fwd_kernel<T, 32, 1, RMS>, grid, dim3(32), 0, st, p);
  else if (v <= 64) (void)tpi::launch(gated_norm_fwd_kernel<T, 64, 1, RMS>, grid, dim3(64), 0, st, p);
  else if (v <= 128) (void)tpi::launch(gated_norm_fwd_kernel<T, 128, 1, RMS>, grid, dim3(128), 0, st, p);
  else if (v <= 256) (void)tpi::launch(gated_norm_fwd_kernel<T, 128, 2, RMS>, grid, dim3(128), 0, st, p);
  else if (v <= 512) (void)tpi::launch(gated_norm_fwd_kernel<T, 128, 4, RMS>, grid, dim3(128), 0, st, p);
  else if (v <= 1024) (void)tpi::launch(gated_norm_fwd_kernel<T, 256, 4, RMS>, grid, dim3(256), 0, st, p);
  else (void)tpi::launch(gated_norm_fwd_kernel<T, 256, 8, RMS>, grid, dim3(256), 0, st, p);
}

template <typename T, int THREADS, int VPT, int CL, bool RMS>
tp_status launch_bwd(tp_plan* plan, GatedNorm p, cudaStream_t st) {
  constexpr int N = Vec16<T>::N;
  auto kernel = gated_norm_bwd_kernel<T, THREADS, VPT, CL, RMS>;
  const int vpr = static_cast<int>(p.h / N), vec_cta = (vpr + CL - 1) / CL;
  const bool pre = p.pre_g != nullptr, use_f = p.post_g || p.gate;
  const int narr = (p.dx_out ? 1 : 0) + (pre ? 2 : 0) + (use_f ? 1 : 0);
  const int smem = kStages * narr * vec_cta * 16;
  unsigned* status = nullptr;
  TP_TRY(tpi::device_status_word(&status));
  int64_t grid = 1;
  TP_TRY(tpi::persistent_grid(reinterpret_cast<const void*>(kernel), THREADS, smem, p.rows * CL, &grid));
  const int64_t G = std::max<int64_t>(1, grid / CL);
  const int64_t B = p.gate ? p.gate_rows : 1;
  const size_t seg = use_f ? static_cast<size_t>(G + B - 1) * 2 * p.h * sizeof(float) : 0;
  const size_t part = pre ? static_cast<size_t>(G) * 2 * p.h * sizeof(float) : 0;
  void* ws = nullptr;
  TP_TRY(tpi::scratch(plan, seg + part + 16, st, &ws));
  p.seg = static_cast<float*>(ws);
  p.cta_part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + seg);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(G * CL));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = tpi::pdl_enabled() ? 2 : 1;
  TP_TRY(tpi::cuda_status(cudaLaunchKernelEx(&cfg, kernel, p, G, narr, vec_cta, status), "gated_residual_norm_bwd"));
  TP_TRY(tpi::after_launch("gated_residual_norm_bwd"));
  if (!(p.dgate || p.dpost_g || p.dpre_g)) return TP_OK;
  const dim3 g2(static_cast<unsigned>((p.h + 31) / 32), p.dgate && B > 1 ? static_cast<unsigned>(B + 1) : 1u);
  (void)tpi::launch(gated_norm_sums_kernel<T>, g2, dim3(32 * kSumWarps), 0, st, p, G, RMS ? 1 : 0);
  return tpi::after_launch("gated_residual_norm_bwd/sums");
}

// By the row's 16-byte vectors: up to two per thread, so the column sums stay in
// registers; rows past 1024 vectors are shared by a cluster of two CTAs.
template <typename T, bool RMS>
tp_status dispatch_bwd(tp_plan* plan, const GatedNorm& p, cudaStream_t st) {
  const int64_t v = p.h * static_cast<int64_t>(sizeof(T)) / 16;
  if (v <= 64) return launch_bwd<T, 64, 1, 1, RMS>(plan, p, st);
  if (v <= 128) return launch_bwd<T, 128, 1, 1, RMS>(plan, p, st);
  if (v <= 256) return launch_bwd<T, 256, 1, 1, RMS>(plan, p, st);
  if (v <= 512) return launch_bwd<T, 256, 2, 1, RMS>(plan, p, st);
  if (v <= 1024) return launch_bwd<T, 512, 2, 1, RMS>(plan, p, st);
  return launch_bwd<T, 512, 2, 2, RMS>(plan, p, st);
}

}  // namespace

namespace tpi {

tp_status launch_gated_norm_fwd(const GatedNorm& p, bool rms, tp_dtype dt, cudaStream_t st) {
  if (dt == TP_BF16) {
    if (rms) launch_fwd<__nv_bfloat16, true>(p, st);
    else launch_fwd<__nv_bfloat16, false>(p, st);
  } else {
    if (rms) launch_fwd<float, true>(p, st);
    else launch_fwd<float, false>(p, st);
  }
  return after_launch("gated_residual_norm_fwd");
}

tp_status launch_gated_norm_bwd(tp_plan* plan, const GatedNorm& p, bool rms, tp_dtype dt, cudaStream_t st) {
  if (dt == TP_BF16)
    return rms ? dispatch_bwd<__nv_bfloat16, true>(plan, p, st) : dispatch_bwd<__nv_bfloat16, false>(plan, p, st);
  return rms ? dispatch_bwd<float, true>(plan, p, st) : dispatch_bwd<float, false>(plan, p, st);
}

}  // namespace tpi
