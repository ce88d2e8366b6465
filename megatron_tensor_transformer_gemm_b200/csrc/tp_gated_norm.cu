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
  // The same as N / 2 pairs of fp32, each in one 64-bit register.
  __device__ static void unpack(const uint4 u, uint64_t (&f)[N / 2]) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i] = tpd::f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
      f[0] = tpd::f2_pack(__uint_as_float(u.x), __uint_as_float(u.y));
      f[1] = tpd::f2_pack(__uint_as_float(u.z), __uint_as_float(u.w));
    }
  }
  __device__ static uint4 pack(const uint64_t (&f)[N / 2]) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 a = tpd::f2_unpack(f[i]);
      v[2 * i] = a.x;
      v[2 * i + 1] = a.y;
    }
    return pack(v);
  }
  __device__ static uint4 pack(const float (&f)[N]) {
    if constexpr (sizeof(T) == 2)
      return make_uint4(tpd::pack_bf16x2(f[0], f[1]), tpd::pack_bf16x2(f[2], f[3]), tpd::pack_bf16x2(f[4], f[5]),
                        tpd::pack_bf16x2(f[6], f[7]));
    else
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// Sum over the THREADS threads of a row (a warp, or the CTA), the same in every one. `red` has two halves used in turn
// (`turn` counts the sums), so one barrier a sum is enough: a half is written
// again only after the barrier of the sum in between.
template <int THREADS>
__device__ __forceinline__ float row_sum(float v, float* red, int& turn) {
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
__device__ __forceinline__ void row_stats(const uint4 (&v)[VPT], int tid, int vpr, float inv_h, float* red, int& turn,
                                          float& mean, float& rstd) {
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
    mean = row_sum<THREADS>(s, red, turn) * inv_h;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (tid + i * THREADS < vpr) {
      float x[N];
      Vec16<T>::unpack(v[i], x);
#pragma unroll
      for (int e = 0; e < N; ++e) q += (x[e] - mean) * (x[e] - mean);
    }
  }
  rstd = rsqrtf(row_sum<THREADS>(q, red, turn) * inv_h + kEps);
}

// A warp per row (four rows a CTA) up to 128 vectors, else a CTA per row; the
// row of x and of f stay packed in registers from their one load to the stores,
// so the two norms cost no extra pass over memory. Bound by HBM: 32768 x 4096 bf16
// LayerNorm, both norms and a gate, in 173 us replayed on the same buffers, 6.2 TB/s
// (a copy: 6.5), and 191-199 us on several sets of buffers in turn. 128 threads of 4
// vectors there: 256 of 2 took 230 us, 64 of 8 203. One row of 4096 takes 4.1 us, the
// launch and two reductions.
constexpr int kWarpRows = 4;
template <typename T, int THREADS, int VPT, bool RMS>
__global__ void __launch_bounds__(THREADS == 32 ? 32 * kWarpRows : THREADS) gated_norm_fwd_kernel(const __grid_constant__ GatedNorm p) {
  tpd::pdl_entry();
  constexpr int N = Vec16<T>::N;
  __shared__ float red[2 * (THREADS / 32)];
  const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t r = THREADS == 32 ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (THREADS == 32 && r >= p.rows) return;
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
    const int c = tid + i * THREADS;
    fv[i] = xv[i] = make_uint4(0, 0, 0, 0);
    if (c < vpr) {
      fv[i] = __ldcs(f + c);
      xv[i] = __ldcs(x + c);
    }
  }
  float mean = 0.f, rstd = 1.f;
  if (p.post_g) {
    row_stats<T, THREADS, VPT, RMS>(fv, tid, vpr, inv_h, red, turn, mean, rstd);
    if (p.stats && tid == 0) {
      if (!RMS) p.stats[r] = mean;
      p.stats[p.rows + r] = rstd;
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * THREADS;
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
  row_stats<T, THREADS, VPT, RMS>(xv, tid, vpr, inv_h, red, turn, mean, rstd);
  if (p.stats && tid == 0) {
    if (!RMS) p.stats[2 * p.rows + r] = mean;
    p.stats[3 * p.rows + r] = rstd;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * THREADS;
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
// Persistent CTAs: the tokens in gate-row-major order (position q = b * per + j is
// token j * gate_rows + b) are cut into one contiguous range per CTA, so a CTA
// sums A and S over runs of one gate row and writes a run's sums once; the run
// of CTA c and gate row b has slot c + b, since both only grow along the order.
// A row's inputs arrive by bulk copies a few rows ahead; a thread owns the same
// columns of every row and keeps its column sums in registers. No atomics: the
// sums are added in a fixed order by a second kernel.
// Bound by HBM for RMSNorm: 8192 x 8192 bf16 with 8 gate rows and every sum 146 us,
// 5.5 TB/s. LayerNorm has two sums more a column, whose registers leave half as many
// rows in flight: 202 us, 4.0 TB/s; 32768 x 4096 363 us, 4.4. In fp32 2049 x 520
// takes 15 us: two launches and 512 CTAs' partial sums beside 26 MB of rows.
constexpr int kStages = 3;

__device__ __forceinline__ int64_t range_lo(int64_t rows, int64_t G, int64_t c) { return rows * c / G; }
// The CTA whose range holds position q.
__device__ __forceinline__ int64_t range_of(int64_t rows, int64_t G, int64_t q) { return ((q + 1) * G - 1) / rows; }

// A walk over positions without divisions: gate row b, index j in its run, token
// t. 32 bits: there are fewer than 2^31 rows.
struct Walk {
  int b, j, t;
  __device__ __forceinline__ void start(int64_t q, int64_t per, int B) {
    b = static_cast<int>(q / per);
    j = static_cast<int>(q - b * per);
    t = static_cast<int>(static_cast<int64_t>(j) * B + b);
  }
  __device__ __forceinline__ void next(int per, int B) {
    t += B;
    if (++j == per) {
      j = 0;
      t = ++b;
    }
  }
};
template <typename T>
__device__ __forceinline__ void unpack_shared(uint32_t addr, uint64_t (&f)[Vec16<T>::N / 2]) {
  Vec16<T>::unpack(tpd::ld_shared_v4(addr), f);
}
// The backward's arithmetic runs on pairs of fp32 (one instruction for two
// columns); each lane rounds as the scalar operation does.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t both(float a) { return tpd::f2_pack(a, a); }
__device__ __forceinline__ float sum2(uint64_t a) {
  const float2 f = tpd::f2_unpack(a);
  return f.x + f.y;
}
// N fp32 values of one vector of a row as one or two 16-byte pieces `apart` bytes apart.
template <int N>
__device__ __forceinline__ void store_f32(uint32_t addr, uint32_t apart, const uint64_t (&v)[N / 2]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(addr + i * apart), "l"(v[2 * i]), "l"(v[2 * i + 1]) : "memory");
}
template <int N>
__device__ __forceinline__ void load_f32(uint32_t addr, uint32_t apart, uint64_t (&v)[N / 2]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[2 * i]), "=l"(v[2 * i + 1]) : "r"(addr + i * apart) : "memory");
}

// Sum of a pair over the CTA (or the CL CTAs of a cluster that share a row) and
// whether every thread's wait succeeded; one barrier, buffers used in turn.
// Slots past the CTA's last warp hold zeros, so the loop needs no count.
template <int MAXT, int CL>
__device__ __forceinline__ bool pair_sum(float2& v, bool ok, float2* red, int& turn, uint32_t rank) {
  constexpr int MAXW = MAXT / 32;
  uint64_t t = tpd::f2_pack(v.x, v.y);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t = tpd::add2(t, __shfl_xor_sync(0xffffffffu, t, o));
  v = tpd::f2_unpack(t);
  float2* half = red + (turn++ & 1) * (MAXW * CL + 2);
  float2* slot = half + rank * MAXW + (threadIdx.x >> 5);
  if (CL == 1) {
    if ((threadIdx.x & 31) == 0) *slot = v;
    if (__syncthreads_or(!ok)) return false;
  } else {
    // the flags of the two CTAs sit behind the pairs: any failed wait of a row
    // marks its CTA's flag in both
    float2* flag = half + CL * MAXW + rank;
    const bool bad = __syncthreads_or(!ok);
    if ((threadIdx.x & 31) == 0) {
      *slot = v;
      const uint32_t far = tpd::map_shared(tpd::smem_u32(slot), rank ^ 1u);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(far), "f"(v.x), "f"(v.y) : "memory");
    }
    if (threadIdx.x == 0) {
      const float f = bad ? 1.f : 0.f;
      *flag = make_float2(f, f);
      const uint32_t far = tpd::map_shared(tpd::smem_u32(flag), rank ^ 1u);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %1};" ::"r"(far), "f"(f) : "memory");
    }
    tpd::cluster_sync_all();
    if (half[CL * MAXW].x + half[CL * MAXW + 1].x != 0.f) return false;
  }
  uint64_t a = 0, b = 0;
#pragma unroll
  for (int w = 0; w < MAXW * CL; w += 2) {  // two slots a load
    const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(half + w);
    a = tpd::add2(a, u.x);
    b = tpd::add2(b, u.y);
  }
  v = tpd::f2_unpack(tpd::add2(a, b));
  return true;
}

// ALL: a pre-norm, a post-norm, a gate and dx_out are all there (the usual
// junction); the other instances test for each.
template <typename T, int MAXT, int VPT, int CL, bool RMS, bool ALL>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 512 / MAXT : 1) gated_norm_bwd_kernel(const __grid_constant__ GatedNorm p, int64_t G, int narr,
                                                              int vec_cta, unsigned* status) {
  constexpr int N = Vec16<T>::N;
  extern __shared__ __align__(128) uint8_t sbuf[];
  __shared__ uint64_t bar[kStages];
  __shared__ int abort_flag;
  __shared__ __align__(16) float2 red[2 * (CL * (MAXT / 32) + 2)];
  const uint32_t rank = CL == 2 ? tpd::cluster_ctarank() : 0u;
  const int64_t cta = blockIdx.x / CL;
  const int nth = blockDim.x;
  const int vpr = static_cast<int>(p.h / N);
  const int v0 = static_cast<int>(rank) * vec_cta;              // this CTA's vectors of a row
  const int nv = min(vec_cta, vpr - v0);
  const uint32_t slice = static_cast<uint32_t>(nv) * 16u;
  const float inv_h = 1.f / static_cast<float>(p.h);
  for (int i = threadIdx.x; i < 2 * (CL * (MAXT / 32) + 2); i += nth) red[i] = make_float2(0.f, 0.f);
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < kStages; ++s) tpd::mbar_init(&bar[s], 1);
    tpd::fence_barrier_init();
  }
  __syncthreads();
  if (CL == 2) tpd::cluster_sync_all();  // the peer runs before its shared memory is written
  tpd::pdl_entry();

  const bool pre = ALL || p.pre_g != nullptr, post = ALL || p.post_g != nullptr, gated = ALL || p.gate != nullptr;
  const bool has_dx = ALL || p.dx_out != nullptr, use_f = post || gated;
  const int64_t lo = range_lo(p.rows, G, cta);
  const int count = static_cast<int>(range_lo(p.rows, G, cta + 1) - lo);  // rows of this CTA
  const int B = gated ? static_cast<int>(p.gate_rows) : 1, per = static_cast<int>(p.rows) / B;
  // arrays of a stage, in order of presence: dx_out, then x_out and dy, then f
  const int o_x = has_dx ? 1 : 0, o_f = o_x + (pre ? 2 : 0);
  const uint32_t arr = static_cast<uint32_t>(vec_cta) * 16u, stage_bytes = arr * narr;
  Walk at;
  at.start(lo, per, B);
  // thread 0's: the next row to load and its stage, rows whose loads are not issued
  __shared__ Walk ahead;
  __shared__ int in_stage, to_issue;
  auto issue = [&]() {  // thread 0, after a barrier behind the stage's last use
    Walk w = ahead;
    tpd::fence_proxy_async_smem();  // the threads' own writes to the stage come before the copies'
    const int64_t off = w.t * p.h + static_cast<int64_t>(v0) * N;
    uint8_t* dst = sbuf + static_cast<uint32_t>(in_stage) * stage_bytes;
    uint64_t* br = &bar[in_stage];
    tpd::mbar_arrive_expect_tx(br, slice * narr);
    if (has_dx) tpd::bulk_load(dst, static_cast<const T*>(p.dx_out) + off, slice, br);
    if (pre) {
      tpd::bulk_load(dst + o_x * arr, static_cast<const T*>(p.x_in) + off, slice, br);
      tpd::bulk_load(dst + (o_x + 1) * arr, static_cast<const T*>(p.dy) + off, slice, br);
    }
    if (use_f) tpd::bulk_load(dst + o_f * arr, static_cast<const T*>(p.f) + off, slice, br);
    w.next(per, B);
    ahead = w;
    --to_issue;
    in_stage = in_stage + 1 == kStages ? 0 : in_stage + 1;
  };
  if (threadIdx.x == 0) {
    ahead = at;
    in_stage = 0;
    to_issue = count;
    for (int s = 0; s < kStages && to_issue > 0; ++s) issue();
    if (rank == 0 && use_f) p.runs[cta] = make_int2(at.b, static_cast<int>((lo + count - 1) / per));
  }

  uint4 g2[VPT];     // pre-norm weight
  // The gate row times the post-norm's weight: in registers for RMSNorm, else
  // behind the stages (LayerNorm's four column sums leave no room), as is a row's
  // a = that times D, which otherwise replaces the stage's x_out and dy. Each
  // thread reads only what it wrote there itself.
  uint64_t w1[RMS ? VPT : 1][N / 2];
  const uint32_t s_w = tpd::smem_u32(sbuf) + kStages * stage_bytes;
  const uint32_t s_a = s_w + (RMS ? 0u : arr * (N / 4));
  uint64_t P[VPT][N / 2], Q[VPT][N / 2], A[VPT][N / 2], S[VPT][N / 2];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * nth;
    g2[i] = make_uint4(0, 0, 0, 0);
    if (c < nv && pre) g2[i] = static_cast<const uint4*>(p.pre_g)[v0 + c];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) P[i][e] = Q[i][e] = A[i][e] = S[i][e] = 0;
  }
  auto write_sums = [&](float* out, uint64_t (&first)[VPT][N / 2], uint64_t (&second)[VPT][N / 2]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * nth;
      if (c < nv) {
        float* to = out + static_cast<int64_t>(v0 + c) * N;
#pragma unroll
        for (int e = 0; e < N / 2; e += 2) {
          *reinterpret_cast<ulonglong2*>(to + 2 * e) = make_ulonglong2(first[i][e], first[i][e + 1]);
          if (!RMS) *reinterpret_cast<ulonglong2*>(to + p.h + 2 * e) = make_ulonglong2(second[i][e], second[i][e + 1]);
        }
      }
#pragma unroll
      for (int e = 0; e < N / 2; ++e) first[i][e] = second[i][e] = 0;
    }
  };

  int turn = 0, s = 0;
  uint32_t phase = 0;
  int run = -1;  // gate row of the current run
  // The row's statistics as xh = (x + c) * r, c = -mean: the difference first. As x * r + c r,
  // an instruction less, xh would be off by 2^-24 of mean * r however small it is itself.
  float r1 = 1.f, c1 = 0.f, r2 = 1.f, c2 = 0.f;
  auto load_stats = [&](int t) {
    if (post) {
      r1 = p.stats[p.rows + t];
      if (!RMS) c1 = -p.stats[t];
    }
    if (pre) {
      r2 = p.stats[3 * p.rows + t];
      if (!RMS) c2 = -p.stats[2 * p.rows + t];
    }
  };
  load_stats(at.t);  // every CTA has a row (G <= rows)
  bool good = true;
  for (int left = count; left > 0; --left) {
    const int64_t row_at = at.t * p.h + static_cast<int64_t>(v0) * N;  // this CTA's part of the row
    if (at.b != run) {
      if (run >= 0 && use_f) write_sums(p.seg + (cta + run) * 2 * p.h, A, S);
      run = at.b;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * nth;
        uint64_t wv[N / 2];
#pragma unroll
        for (int e = 0; e < N / 2; ++e) wv[e] = both(1.f);
        if (c < nv && gated)
          Vec16<T>::unpack(reinterpret_cast<const uint4*>(static_cast<const T*>(p.gate) + run * p.h)[v0 + c], wv);
        if (c < nv && post) {
          uint64_t w[N / 2];
          Vec16<T>::unpack(static_cast<const uint4*>(p.post_g)[v0 + c], w);
#pragma unroll
          for (int e = 0; e < N / 2; ++e) wv[e] = mul2(wv[e], w[e]);
        }
        if constexpr (RMS) {
#pragma unroll
          for (int e = 0; e < N / 2; ++e) w1[i][e] = wv[e];
        } else if (c < nv) {
          store_f32<N>(s_w + c * 16, arr, wv);
        }
      }
    }
    const float R1 = r1, C1 = c1, R2 = r2, C2 = c2;
    at.next(per, B);
    if (left > 1) load_stats(at.t);  // a row early
    // a wait that gave up computes on an unfinished stage; the sum below then
    // stops every thread of the row before anything is written
    const bool ok = tpd::mbar_wait(&bar[s], phase, &abort_flag, status);
    const uint32_t s_dx = tpd::smem_u32(sbuf) + static_cast<uint32_t>(s) * stage_bytes;
    const uint32_t s_x = s_dx + o_x * arr, s_dy = s_x + arr, s_f = s_dx + o_f * arr;
    if (++s == kStages) {
      s = 0;
      phase ^= 1u;
    }
    uint64_t mx = 0, my = 0;
    if (pre) {
      const uint64_t r = both(R2), k = both(C2);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * nth;
        if (c < nv) {
          uint64_t x[N / 2], d[N / 2], w[N / 2];
          unpack_shared<T>(s_x + c * 16, x);
          unpack_shared<T>(s_dy + c * 16, d);
          Vec16<T>::unpack(g2[i], w);
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            const uint64_t xh = mul2(RMS ? x[e] : tpd::add2(x[e], k), r), gy = mul2(d[e], w[e]);
            if (!RMS) mx = tpd::add2(mx, gy);
            my = fma2(gy, xh, my);
            P[i][e] = fma2(d[e], xh, P[i][e]);
            if (!RMS) Q[i][e] = tpd::add2(Q[i][e], d[e]);
          }
        }
      }
    }
    float2 m = make_float2(RMS ? 0.f : sum2(mx), sum2(my));
    good = pair_sum<MAXT, CL>(m, ok, red, turn, rank);
    if (!good) break;
    // every thread is past the row before this one: its stage takes a new row
    if (threadIdx.x == 0 && left < count && to_issue > 0) issue();
    // D = dx_out + R2 (gy - m1 - xh m2), xh = (x + C2) R2
    const float m1 = m.x * inv_h, m2 = m.y * inv_h;
    const uint64_t fx = both(-R2 * m2 * R2), f0 = both(-R2 * m1), fr = both(R2), rs = both(p.rs), c2v = both(C2);
    const uint64_t r1v = both(R1), c1v = both(C1);
    const uint32_t at_a = pre ? s_x : s_a;
    uint64_t ux = 0, uy = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * nth;
      if (c >= nv) continue;
      uint64_t D[N / 2], o[N / 2];
#pragma unroll
      for (int e = 0; e < N / 2; ++e) D[e] = 0;
      if (has_dx) unpack_shared<T>(s_dx + c * 16, D);
      if (pre) {
        uint64_t x[N / 2], d[N / 2], w[N / 2];
        unpack_shared<T>(s_x + c * 16, x);
        unpack_shared<T>(s_dy + c * 16, d);
        Vec16<T>::unpack(g2[i], w);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          const uint64_t v = RMS ? D[e] : tpd::add2(D[e], f0);
          D[e] = fma2(RMS ? x[e] : tpd::add2(x[e], c2v), fx, fma2(mul2(d[e], w[e]), fr, v));
        }
      }
#pragma unroll
      for (int e = 0; e < N / 2; ++e) o[e] = mul2(rs, D[e]);
      reinterpret_cast<uint4*>(static_cast<T*>(p.dx) + row_at)[c] = Vec16<T>::pack(o);
      uint64_t x[N / 2];
      if (use_f) {
        unpack_shared<T>(s_f + c * 16, x);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          x[e] = mul2(RMS ? x[e] : tpd::add2(x[e], c1v), r1v);
          A[i][e] = fma2(D[e], x[e], A[i][e]);
          if (!RMS) S[i][e] = tpd::add2(S[i][e], D[e]);
        }
      }
      if constexpr (RMS) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) D[e] = mul2(D[e], w1[i][e]);
      } else {
        uint64_t w[N / 2];
        load_f32<N>(s_w + c * 16, arr, w);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) D[e] = mul2(D[e], w[e]);
      }
      if (post) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          if (!RMS) ux = tpd::add2(ux, D[e]);
          uy = fma2(D[e], x[e], uy);
        }
      }
      store_f32<N>(at_a + c * 16, arr, D);
    }
    uint64_t fu = 0, fc = 0;
    if (post) {
      float2 u = make_float2(RMS ? 0.f : sum2(ux), sum2(uy));
      good = pair_sum<MAXT, CL>(u, true, red, turn, rank);
      // df = R1 (a - u1 - xh u2), xh = (f + C1) R1
      const float u1 = u.x * inv_h, u2 = u.y * inv_h;
      fu = both(-R1 * u2 * R1);
      fc = both(RMS ? 0.f : -R1 * u1);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * nth;
      if (c >= nv) continue;
      uint64_t o[N / 2];
      load_f32<N>(at_a + c * 16, arr, o);
      if (post) {
        uint64_t x[N / 2];
        unpack_shared<T>(s_f + c * 16, x);
#pragma unroll
        for (int e = 0; e < N / 2; ++e)
          o[e] = fma2(RMS ? x[e] : tpd::add2(x[e], c1v), fu, RMS ? mul2(o[e], r1v) : fma2(o[e], r1v, fc));
      }
      reinterpret_cast<uint4*>(static_cast<T*>(p.df) + row_at)[c] = Vec16<T>::pack(o);
    }
  }
  if (good) {
    if (use_f) write_sums(p.seg + (cta + run) * 2 * p.h, A, S);
    if (pre) write_sums(p.cta_part + cta * 2 * p.h, P, Q);
  } else if (threadIdx.x == 0) {
    // let the loads still in flight land (bounded) before the CTA exits: stage i
    // holds the last issued row whose index is i mod kStages
    const int n = count - to_issue;
    for (int i = 0; i < kStages && i < n; ++i) {
      int again = 0;
      const int last = i + (n - 1 - i) / kStages * kStages;
      tpd::mbar_wait(&bar[i], static_cast<uint32_t>(last / kStages) & 1u, &again, nullptr, 1000000ull);
    }
  }
  if (CL == 2) tpd::cluster_sync_all();  // neither CTA leaves while its peer may still write to it
}

// The column sums of the backward, each in a fixed order. A block owns 32
// columns, eight lanes of four. blockIdx.y = 0: the norms' parameters (and a single
// gate row); its kSumRows groups of eight lanes take CTAs g, g + kSumRows, ... .
// blockIdx.y = y: gate rows 4 (y - 1) ... of several, a quarter of the groups each.
// Four CTAs' loads are in flight in a group and warps add by shuffles: with one load
// at a time and sums through shared memory the 8192 x 8192 case took 158 us in place
// of 146, 2049 x 520 21.8 in place of 15.0.
constexpr int kSumRows = 64;
__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
}
template <typename T>
__device__ __forceinline__ float4 four(const void* v, int64_t at) {
  const T* s = static_cast<const T*>(v) + at;
  return make_float4(static_cast<float>(s[0]), static_cast<float>(s[1]), static_cast<float>(s[2]), static_cast<float>(s[3]));
}
template <typename T, bool RMS>
__global__ void __launch_bounds__(8 * kSumRows) gated_norm_sums_kernel(const __grid_constant__ GatedNorm p, int64_t G) {
  tpd::pdl_entry();
  __shared__ float4 red[6][kSumRows / 4][8];
  const int group = threadIdx.x >> 3, lane = threadIdx.x & 7;  // group and its lane
  const int64_t col = (static_cast<int64_t>(blockIdx.x) * 8 + lane) * 4;
  const int64_t B = p.gate ? p.gate_rows : 1, per = p.rows / B;
  const bool use_f = p.post_g || p.gate, all = blockIdx.y == 0, in = col < p.h;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 v[6];  // P, Q, sum of g A, of g S, A, S
#pragma unroll
  for (int i = 0; i < 6; ++i) v[i] = zero;
  constexpr int kQuarter = kSumRows / 4;
  const int64_t gate_row = all ? 0 : (blockIdx.y - 1) * 4 + group / kQuarter;
  const bool mine = gate_row < B;
  int64_t c0 = 0, c1 = G;
  if (!all && mine) {
    c0 = range_of(p.rows, G, gate_row * per);
    c1 = range_of(p.rows, G, (gate_row + 1) * per - 1) + 1;
  }
  if (in && mine) {
    if (all && p.pre_g) {
#pragma unroll 4
      for (int64_t c = group; c < G; c += kSumRows) {
        const float* s = p.cta_part + c * 2 * p.h + col;
        add4(v[0], *reinterpret_cast<const float4*>(s));
        if (!RMS) add4(v[1], *reinterpret_cast<const float4*>(s + p.h));
      }
    }
    if (use_f && (!all || B == 1)) {
      const int first = all ? group : group % kQuarter, step = all ? kSumRows : kQuarter;
#pragma unroll 4
      for (int64_t c = c0 + first; c < c1; c += step) {
        const float* s = p.seg + (c + gate_row) * 2 * p.h + col;
        add4(v[4], *reinterpret_cast<const float4*>(s));
        if (!RMS) add4(v[5], *reinterpret_cast<const float4*>(s + p.h));
      }
    } else if (use_f && (p.dpost_g || p.dpost_b)) {  // several gate rows, weighted
      auto add = [&](const float4& A, const float4& S, const float4& g) {
        v[2].x = fmaf(g.x, A.x, v[2].x); v[2].y = fmaf(g.y, A.y, v[2].y);
        v[2].z = fmaf(g.z, A.z, v[2].z); v[2].w = fmaf(g.w, A.w, v[2].w);
        if (!RMS) {
          v[3].x = fmaf(g.x, S.x, v[3].x); v[3].y = fmaf(g.y, S.y, v[3].y);
          v[3].z = fmaf(g.z, S.z, v[3].z); v[3].w = fmaf(g.w, S.w, v[3].w);
        }
      };
      auto load = [&](int64_t c, int b, float4& A, float4& S, float4& g) {
        const float* s = p.seg + (c + b) * 2 * p.h + col;
        A = *reinterpret_cast<const float4*>(s);
        if (!RMS) S = *reinterpret_cast<const float4*>(s + p.h);
        g = four<T>(p.gate, static_cast<int64_t>(b) * p.h + col);
      };
      constexpr int U = 4;  // CTAs whose loads are in flight together
      for (int64_t c0 = group; c0 < G; c0 += U * kSumRows) {
        int2 r[U];
        float4 A[U], S[U], g[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          r[u] = c0 + u * kSumRows < G ? p.runs[c0 + u * kSumRows] : make_int2(0, -1);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          A[u] = S[u] = g[u] = zero;
          if (r[u].y >= 0) load(c0 + u * kSumRows, r[u].x, A[u], S[u], g[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          add(A[u], S[u], g[u]);
          for (int b = r[u].x + 1; b <= r[u].y; ++b) {  // a CTA whose rows pass into further gate rows
            load(c0 + u * kSumRows, b, A[u], S[u], g[u]);
            add(A[u], S[u], g[u]);
          }
        }
      }
    }
  }
  // the four groups of a warp, then the warps, in order
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    if (RMS && (i & 1)) continue;
#pragma unroll
    for (int o = 8; o <= 16; o <<= 1)
      add4(v[i], make_float4(__shfl_xor_sync(0xffffffffu, v[i].x, o), __shfl_xor_sync(0xffffffffu, v[i].y, o),
                             __shfl_xor_sync(0xffffffffu, v[i].z, o), __shfl_xor_sync(0xffffffffu, v[i].w, o)));
    if ((threadIdx.x & 31) < 8) red[i][threadIdx.x >> 5][lane] = v[i];
  }
  __syncthreads();
  constexpr int kWarps = kSumRows / 4;
  if (all) {  // group i adds the warps' sums of v[i]
    if (group < 6 && !(RMS && (group & 1))) {
      float4 t = red[group][0][lane];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) add4(t, red[group][w][lane]);
      red[group][0][lane] = t;
    }
    __syncthreads();
    if (group != 0 || !in) return;
#pragma unroll
    for (int i = 0; i < 6; ++i)
      if (!(RMS && (i & 1))) v[i] = red[i][0][lane];
  } else {  // the first group of each quarter, its gate row's two sums
    if (group % kQuarter != 0 || !in || !mine) return;
#pragma unroll
    for (int i = 4; i < 6; ++i) {
      if (RMS && (i & 1)) continue;
      v[i] = red[i][group / 4][lane];
#pragma unroll
      for (int w = 1; w < kWarps / 4; ++w) add4(v[i], red[i][group / 4 + w][lane]);
    }
  }
  if (all && B == 1 && use_f) {  // one gate row: its weight once, after the sum
    const float4 g = p.gate ? four<T>(p.gate, col) : make_float4(1.f, 1.f, 1.f, 1.f);
    v[2] = make_float4(g.x * v[4].x, g.y * v[4].y, g.z * v[4].z, g.w * v[4].w);
    v[3] = make_float4(g.x * v[5].x, g.y * v[5].y, g.z * v[5].z, g.w * v[5].w);
  }
  auto put = [&](float* out, const float4& s) {
    if (out) *reinterpret_cast<float4*>(out + col) = s;
  };
  if (all) {
    put(p.dpre_g, v[0]);
    put(p.dpost_g, v[2]);
    if (!RMS) {
      put(p.dpre_b, v[1]);
      put(p.dpost_b, v[3]);
    }
  }
  if (p.dgate && (all ? B == 1 : true)) {
    const float4 g = p.post_g ? four<T>(p.post_g, col) : make_float4(1.f, 1.f, 1.f, 1.f);
    const float4 b = p.post_g && !RMS ? four<T>(p.post_b, col) : zero;
    put(p.dgate + gate_row * p.h,
        make_float4(g.x * v[4].x + b.x * v[5].x, g.y * v[4].y + b.y * v[5].y, g.z * v[4].z + b.z * v[5].z,
                    g.w * v[4].w + b.w * v[5].w));
  }
}

// ---------------------------------------------------------------- dispatch
// Threads and vectors per thread of the forward, by the row's 16-byte vectors.
template <typename T, int THREADS, int VPT, bool RMS>
void launch_fwd(const GatedNorm& p, cudaStream_t st) {
  const int64_t ctas = THREADS == 32 ? (p.rows + kWarpRows - 1) / kWarpRows : p.rows;
  (void)tpi::launch(gated_norm_fwd_kernel<T, THREADS, VPT, RMS>, dim3(static_cast<unsigned>(ctas)),
                    dim3(THREADS == 32 ? 32 * kWarpRows : THREADS), 0, st, p);
}
template <typename T, bool RMS>
void dispatch_fwd(const GatedNorm& p, cudaStream_t st) {
  const int64_t v = p.h * static_cast<int64_t>(sizeof(T)) / 16;
  if (v <= 32) launch_fwd<T, 32, 1, RMS>(p, st);
  else if (v <= 64) launch_fwd<T, 32, 2, RMS>(p, st);
  else if (v <= 128) launch_fwd<T, 32, 4, RMS>(p, st);
  else if (v <= 256) launch_fwd<T, 64, 4, RMS>(p, st);
  else if (v <= 512) launch_fwd<T, 128, 4, RMS>(p, st);
  else if (v <= 1024) launch_fwd<T, 256, 4, RMS>(p, st);
  else launch_fwd<T, 512, 4, RMS>(p, st);
}

constexpr int kMinRows = 4;
template <typename T, int MAXT, int VPT, int CL, bool RMS, bool ALL>
tp_status launch_bwd(tp_plan* plan, GatedNorm p, cudaStream_t st) {
  constexpr int N = Vec16<T>::N;
  auto kernel = gated_norm_bwd_kernel<T, MAXT, VPT, CL, RMS, ALL>;
  const int vpr = static_cast<int>(p.h / N), vec_cta = (vpr + CL - 1) / CL;
  const int threads = std::min(MAXT, ((vec_cta + VPT - 1) / VPT + 31) / 32 * 32);
  const bool pre = p.pre_g != nullptr, use_f = p.post_g || p.gate;
  const int narr = (p.dx_out ? 1 : 0) + (pre ? 2 : 0) + (use_f ? 1 : 0);
  // the stages; LayerNorm's fp32 weights; without a pre-norm, the row's a
  const int smem = (kStages * narr + (RMS ? 0 : N / 4) + (pre ? 0 : N / 4)) * vec_cta * 16;
  unsigned* status = nullptr;
  TP_TRY(tpi::device_status_word(&status));
  int64_t grid = 1;
  // at least kMinRows rows a CTA: below that the partial sums outweigh the rows
  TP_TRY(tpi::persistent_grid(reinterpret_cast<const void*>(kernel), threads, smem,
                              (p.rows + kMinRows - 1) / kMinRows * CL, &grid));
  const int64_t G = std::max<int64_t>(1, grid / CL);
  const int64_t B = p.gate ? p.gate_rows : 1;
  const size_t seg = use_f ? static_cast<size_t>(G + B - 1) * 2 * p.h * sizeof(float) : 0;
  const size_t part = pre ? static_cast<size_t>(G) * 2 * p.h * sizeof(float) : 0;
  void* ws = nullptr;
  TP_TRY(tpi::scratch(plan, seg + part + G * sizeof(int2), st, &ws));
  p.seg = static_cast<float*>(ws);
  p.cta_part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + seg);
  p.runs = reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + seg + part);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(G * CL));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  const bool pdl = tpi::pdl_enabled();
  cfg.attrs = pdl ? attr : attr + 1;
  cfg.numAttrs = (pdl ? 1 : 0) + (CL > 1 ? 1 : 0);
  TP_TRY(tpi::cuda_status(cudaLaunchKernelEx(&cfg, kernel, p, G, narr, vec_cta, status), "gated_residual_norm_bwd"));
  TP_TRY(tpi::after_launch("gated_residual_norm_bwd"));
  if (!(p.dgate || p.dpost_g || p.dpost_b || p.dpre_g || p.dpre_b)) return TP_OK;
  const dim3 g2(static_cast<unsigned>((p.h + 31) / 32), p.dgate && B > 1 ? static_cast<unsigned>((B + 3) / 4 + 1) : 1u);
  (void)tpi::launch(gated_norm_sums_kernel<T, RMS>, g2, dim3(8 * kSumRows), 0, st, p, G);
  return tpi::after_launch("gated_residual_norm_bwd/sums");
}

// By the row's 16-byte vectors: up to two per thread, so the column sums stay in
// registers; rows past 1024 vectors are shared by a cluster of two CTAs.
template <typename T, bool RMS, bool ALL>
tp_status dispatch_bwd(tp_plan* plan, const GatedNorm& p, cudaStream_t st) {
  const int64_t v = p.h * static_cast<int64_t>(sizeof(T)) / 16;
  if (v <= 128) return launch_bwd<T, 64, 2, 1, RMS, ALL>(plan, p, st);
  if (v <= 256) return launch_bwd<T, 128, 2, 1, RMS, ALL>(plan, p, st);
  if (v <= 512) return launch_bwd<T, 256, 2, 1, RMS, ALL>(plan, p, st);
  if (v <= 1024) return launch_bwd<T, 512, 2, 1, RMS, ALL>(plan, p, st);
  return launch_bwd<T, 512, 2, 2, RMS, ALL>(plan, p, st);
}
template <typename T, bool RMS>
tp_status dispatch_bwd(tp_plan* plan, const GatedNorm& p, cudaStream_t st) {
  return p.dx_out && p.pre_g && p.post_g && p.gate ? dispatch_bwd<T, RMS, true>(plan, p, st)
                                                    : dispatch_bwd<T, RMS, false>(plan, p, st);
}

}  // namespace

namespace tpi {

tp_status launch_gated_norm_fwd(const GatedNorm& p, bool rms, tp_dtype dt, cudaStream_t st) {
  if (dt == TP_BF16) {
    if (rms) dispatch_fwd<__nv_bfloat16, true>(p, st);
    else dispatch_fwd<__nv_bfloat16, false>(p, st);
  } else {
    if (rms) dispatch_fwd<float, true>(p, st);
    else dispatch_fwd<float, false>(p, st);
  }
  return after_launch("gated_residual_norm_fwd");
}

tp_status launch_gated_norm_bwd(tp_plan* plan, const GatedNorm& p, bool rms, tp_dtype dt, cudaStream_t st) {
  if (dt == TP_BF16)
    return rms ? dispatch_bwd<__nv_bfloat16, true>(plan, p, st) : dispatch_bwd<__nv_bfloat16, false>(plan, p, st);
  return rms ? dispatch_bwd<float, true>(plan, p, st) : dispatch_bwd<float, false>(plan, p, st);
}

}  // namespace tpi
