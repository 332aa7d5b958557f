// Root-mean-square norm with the residual's addition, and its gradients.
//
//   r = x + residual,  rstd = 1 / sqrt(mean r^2 + eps),  y = r rstd w
//   dr = rstd (dy w - r rstd^2 mean(dy w r)) + dr_in,  dw = sum over rows of dy r rstd
//
// Bound by HBM (3 or 4 elements of traffic against 7 or 18 operations): a row
// is read once into the registers of TH threads, VPT vectors of 16 bytes each,
// summed across them, and written. 8-bit outputs find their group's maximum
// over the neighbouring lanes that hold the group, so nothing is read again.
// The backward kernel's CTAs walk over rows with their columns' part of dw in
// registers and leave one slab each.
//
// 16384 rows of 2048 bf16 take 41 us forward (268 MB, 6.5 TB/s) and 51 us
// backward: 46 us for the rows (268 MB, 5.8 TB/s), the rest for the sum of 608
// slabs. 16384 rows of 4096 to 8 bits take 80 us (472 MB, 5.9 TB/s): with
// registers for 1536 threads an SM, w loaded only after the row's sum (87 us
// before both; 95 us at 1792 threads, which spill). Two vectors a thread: four
// leave too few warps to cover the barriers, and forward CTAs that stay and load
// rows ahead were slower (170 us against 126 us at the time).
#include <type_traits>

#include <cuda_fp8.h>

#include "seq_common.cuh"

namespace cig {
namespace {

constexpr float kE4M3Max = 448.f;
constexpr int kStages = 4;  // rows of the backward pass's ring

// a, b -> the larger, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The largest of a, |b| and |c| (a >= 0), NaN if any is.
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return max_nan(a, b); }
};

// Combines v over TH threads of a row in a fixed order; every thread gets the
// result. `part` holds one float a warp, two such rows in turn (a warp may
// still read the one while another writes the next); called by all threads of
// the CTA.
template <int TH, class Op>
__device__ __forceinline__ float over_row(float v, float (*parts)[32], int& turn, Op op) {
#pragma unroll
  for (int m = 16; m >= 1; m /= 2) v = op(v, __shfl_xor_sync(0xffffffffu, v, m));
  if constexpr (TH > 32) {
    constexpr int kWarps = TH / 32;
    const int warp = threadIdx.x >> 5;
    float* part = parts[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    if constexpr (kWarps >= 4) {
      float4 all = *reinterpret_cast<const float4*>(part);
#pragma unroll
      for (int j = 4; j < kWarps; j += 4) {
        const float4 q = *reinterpret_cast<const float4*>(part + j);
        all = make_float4(op(all.x, q.x), op(all.y, q.y), op(all.z, q.z), op(all.w, q.w));
      }
      v = op(op(all.x, all.y), op(all.z, all.w));
    } else {
      v = op(part[0], part[1]);
    }
  }
  return v;
}

// A group's scale, top / 448, and q = y inv. A group of NaN, and one whose
// scale rounds to 0, has scale 1. inv = 0: 448 / top or a factor on the way to it
// would leave the normal numbers, and the quotient is taken in two steps.
struct Scale {
  float scale, inv;
};
__device__ __forceinline__ Scale scale_of(float top) {
  Scale s;
  s.scale = top * (1.f / kE4M3Max);
  s.inv = kE4M3Max * rcp_fast(top);
  if (!(top > 1e-30f && top < 1e37f)) {
    const bool plain = !(s.scale > 0.f);
    s.inv = plain ? 1.f : 0.f;
    if (plain) s.scale = 1.f;
  }
  return s;
}
// y / scale for a group whose maximum is far from 1: both sides times a power
// of two. (All of a group that reaches infinity becomes 0 or NaN.)
__device__ __forceinline__ float far_quotient(float y, const Scale& s) {
  const float f = s.scale < 1.f ? 0x1p96f : 0x1p-32f;
  return y * f * rcp_fast(s.scale * f);
}
__device__ __forceinline__ uint8_t to_e4m3(float y, const Scale& s) {
  return __nv_cvt_float_to_fp8(s.inv != 0.f ? y * s.inv : far_quotient(y, s), __NV_SATFINITE, __NV_E4M3);
}
template <int V, int P>
__device__ __forceinline__ Pack<uint8_t, V> to_e4m3(float2 (&y)[P], const Scale& s) {
  Pack<uint8_t, V> o;
  if (s.inv == 0.f) {
#pragma unroll
    for (int p = 0; p < P; ++p) y[p] = make_float2(far_quotient(y[p].x, s), far_quotient(y[p].y, s));
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p) y[p] = __fmul2_rn(y[p], both(s.inv));
  }
  if constexpr (V == 1) {
    o.v[0] = __nv_cvt_float_to_fp8(y[0].x, __NV_SATFINITE, __NV_E4M3);
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p)
      *reinterpret_cast<__nv_fp8x2_storage_t*>(&o.v[2 * p]) = __nv_cvt_float2_to_fp8x2(y[p], __NV_SATFINITE, __NV_E4M3);
  }
  return o;
}

// x + residual, rounded once to the type they are kept in. (16-bit sums take one
// packed instruction for two elements; unpacked to fp32 and packed again they
// took ten, a quarter of the row's.)
__device__ __forceinline__ float sum_of(float a, float b) { return a + b; }
__device__ __forceinline__ __nv_bfloat16 sum_of(__nv_bfloat16 a, __nv_bfloat16 b) { return __hadd_rn(a, b); }
__device__ __forceinline__ __half sum_of(__half a, __half b) { return __hadd_rn(a, b); }
__device__ __forceinline__ __nv_bfloat162 sum_of(__nv_bfloat162 a, __nv_bfloat162 b) { return __hadd2_rn(a, b); }
__device__ __forceinline__ __half2 sum_of(__half2 a, __half2 b) { return __hadd2_rn(a, b); }
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> sum_of(const Pack<T, V>& a, const Pack<T, V>& b) {
  Pack<T, V> r;
  if constexpr (sizeof(T) == 2 && V > 1) {
    using Pair = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
#pragma unroll
    for (int i = 0; i < V; i += 2)
      *reinterpret_cast<Pair*>(&r.v[i]) = sum_of(*reinterpret_cast<const Pair*>(&a.v[i]), *reinterpret_cast<const Pair*>(&b.v[i]));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = sum_of(a.v[i], b.v[i]);
  }
  return r;
}

// The thread's part of w, as pairs.
template <typename T, int V, int TH, int VPT>
__device__ __forceinline__ void load_w(const seq_norm_args& a, int tid, int vecs, float2 (&w)[VPT][kPairs<V>]) {
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = k * TH + tid;
    if (v < vecs && a.w_dtype == CONV_F32) {
      unpack(load_pack<V>(static_cast<const float*>(a.w) + v * V), w[k]);
    } else {
      unpack(v < vecs ? load_pack<V>(static_cast<const T*>(a.w) + v * V) : zero_pack<T, V>(), w[k]);
    }
  }
}
template <typename T, int V, int TH, int VPT>
__device__ __forceinline__ void load_row(const T* p, int tid, int vecs, Pack<T, V> (&v)[VPT]) {
#pragma unroll
  for (int k = 0; k < VPT; ++k)
    v[k] = k * TH + tid < vecs ? load_pack_once<V>(p + (k * TH + tid) * V) : zero_pack<T, V>();
}

template <typename T, int V, int TH, int VPT, bool kOut8>
__global__ void __launch_bounds__(TH == 32 ? 128 : TH, V > 1 && TH >= 128 && TH < 1024 ? 1536 / TH : 1) norm_fwd_kernel(const __grid_constant__ seq_norm_args a) {
  constexpr int kRows = TH == 32 ? 4 : 1;  // rows of a CTA
  constexpr int P = kPairs<V>;
  __shared__ __align__(16) float part[2][32];
  __shared__ unsigned tops[V == 1 && kOut8 ? 512 : 1];  // scalar rows: maxima of up to 8192 / 32 groups
  int turn = 0;
  const int tid = threadIdx.x % TH, c = (int)a.c, vecs = c / V;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TH;
  if (kRows > 1 && row >= a.n) return;  // whole warps
  Pack<T, V> px[VPT];
  load_row<T, V, TH, VPT>(static_cast<const T*>(a.x.data) + row * a.x.stride_n, tid, vecs, px);
  float2 w[VPT][P], y[VPT][P];
  if (a.residual.data) {
    Pack<T, V> pr[VPT];
    load_row<T, V, TH, VPT>(static_cast<const T*>(a.residual.data) + row * a.residual.stride_n, tid, vecs, pr);
#pragma unroll
    for (int k = 0; k < VPT; ++k) px[k] = sum_of(px[k], pr[k]);  // normed as it is kept
  }
  if (a.r.data) {
    T* rout = static_cast<T*>(a.r.data) + row * a.r.stride_n;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (k * TH + tid < vecs) store_pack(rout + (k * TH + tid) * V, px[k]);
  }
  float2 sq = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    unpack(px[k], y[k]);
#pragma unroll
    for (int p = 0; p < P; ++p) sq = __ffma2_rn(y[k][p], y[k][p], sq);
  }
  const float rstd = rsqrtf(over_row<TH>(sq.x + sq.y, part, turn, Add()) * (1.f / (float)c) + a.eps);
  load_w<T, V, TH, VPT>(a, tid, vecs, w);
  if (a.rstd && tid == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int p = 0; p < P; ++p) y[k][p] = __fmul2_rn(__fmul2_rn(y[k][p], both(rstd)), w[k][p]);
  if constexpr (!kOut8) {
    T* out = static_cast<T*>(a.y.data) + row * a.y.stride_n;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (k * TH + tid < vecs) store_pack(out + (k * TH + tid) * V, pack<T, V>(y[k]));
  } else {
    float top[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      top[k] = 0.f;
      if (k * TH + tid < vecs) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          if (V > 1) top[k] = max_abs_nan(top[k], y[k][p].x, y[k][p].y);
          else top[k] = max_nan(top[k], fabsf(y[k][p].x));
        }
      }
    }
    const int shift = a.group ? __ffs(a.group) - 1 : 0;  // group is 32, 64 or 128
    const int groups = a.group ? (c + a.group - 1) >> shift : 1;
    if (a.group == 0) {
      float all = top[0];
#pragma unroll
      for (int k = 1; k < VPT; ++k) all = max_nan(all, top[k]);
      all = over_row<TH>(all, part, turn, Max());
#pragma unroll
      for (int k = 0; k < VPT; ++k) top[k] = all;
    } else if constexpr (V > 1) {
      // The group's vectors are group / V neighbouring lanes.
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        for (int m = 1; m * V < a.group; m *= 2) top[k] = max_nan(top[k], __shfl_xor_sync(0xffffffffu, top[k], m));
    } else {
      // |y| as unsigned bits orders like the value, with NaN on top.
      static_assert(TH >= 128, "one row a CTA");
      for (int k = threadIdx.x; k < groups; k += TH) tops[k] = 0u;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = k * TH + tid;
        if (v < vecs) atomicMax(&tops[v >> shift], __float_as_uint(top[k]));
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = k * TH + tid;
        if (v < vecs) top[k] = __uint_as_float(tops[v >> shift]);
      }
    }
    uint8_t* out = static_cast<uint8_t*>(a.y.data) + row * a.y.stride_n;
    float* scales = a.scale + row * groups;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = k * TH + tid, col = v * V;
      if (v >= vecs) continue;
      const Scale s = scale_of(top[k]);
      if (a.group ? (col & (a.group - 1)) == 0 : v == 0) scales[a.group ? col >> shift : 0] = s.scale;
      store_pack(out + col, to_e4m3<V>(y[k], s));
    }
  }
}

// Rows too long for registers: three passes over the row (the later ones from
// L2), one element a thread and step (2048 rows of 20480 bf16: 111 us, floor 50).
template <typename T>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(const __grid_constant__ seq_norm_args a) {
  __shared__ __align__(16) float part[2][32];
  int turn = 0;
  const int64_t row = blockIdx.x;
  const bool w32 = a.w_dtype == CONV_F32;
  const T* x = static_cast<const T*>(a.x.data) + row * a.x.stride_n;
  const T* res = a.residual.data ? static_cast<const T*>(a.residual.data) + row * a.residual.stride_n : nullptr;
  T* rout = a.r.data ? static_cast<T*>(a.r.data) + row * a.r.stride_n : nullptr;
  auto value = [&](int64_t k) {
    T v = x[k];
    if (res) v = sum_of(v, res[k]);
    return v;
  };
  float sum = 0.f;
  for (int64_t k = threadIdx.x; k < a.c; k += 1024) {
    const float v = to_f32(value(k));
    sum = fmaf(v, v, sum);
  }
  const float rstd = rsqrtf(over_row<1024>(sum, part, turn, Add()) / (float)a.c + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  if (!a.out8) {
    T* out = static_cast<T*>(a.y.data) + row * a.y.stride_n;
    for (int64_t k = threadIdx.x; k < a.c; k += 1024) {
      const T v = value(k);  // before r is written, which may be x or the residual
      if (rout) rout[k] = v;
      store_out(out + k, to_f32(v) * rstd * param<T>(a.w, k, w32));
    }
    return;
  }
  uint8_t* out = static_cast<uint8_t*>(a.y.data) + row * a.y.stride_n;
  const int64_t groups = a.group ? (a.c + a.group - 1) / a.group : 1;
  const int64_t width = a.group ? a.group : a.c;
  if (a.group == 0) {
    float top = 0.f;
    for (int64_t k = threadIdx.x; k < a.c; k += 1024)
      top = max_nan(top, fabsf(to_f32(value(k)) * rstd * param<T>(a.w, k, w32)));
    top = over_row<1024>(top, part, turn, Max());
    const Scale s = scale_of(top);
    if (threadIdx.x == 0) a.scale[row] = s.scale;
    for (int64_t k = threadIdx.x; k < a.c; k += 1024) {
      const T v = value(k);
      if (rout) rout[k] = v;
      out[k] = to_e4m3(to_f32(v) * rstd * param<T>(a.w, k, w32), s);
    }
    return;
  }
  // A warp a group (32 to 128 columns).
  const int lane = threadIdx.x & 31;
  for (int64_t g = threadIdx.x >> 5; g < groups; g += 32) {
    T v[4];
    float y[4], top = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t k = g * width + j * 32 + lane;
      const bool in = j * 32 < width && k < a.c;
      v[j] = in ? value(k) : zero_of<T>();
      y[j] = in ? to_f32(v[j]) * rstd * param<T>(a.w, k, w32) : 0.f;
      top = max_nan(top, fabsf(y[j]));
    }
#pragma unroll
    for (int m = 16; m >= 1; m /= 2) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, m));
    const Scale s = scale_of(top);
    if (lane == 0) a.scale[row * groups + g] = s.scale;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t k = g * width + j * 32 + lane;
      if (j * 32 < width && k < a.c) {
        if (rout) rout[k] = v[j];
        out[k] = to_e4m3(y[j], s);
      }
    }
  }
}

// CTAs walk over rows. Vector rows come through a ring of kStages rows in
// shared memory by asynchronous copies: each thread copies and reads back its
// own vectors, so that the ring needs no barrier.
template <typename T, int V, int TH, int VPT>
__global__ void __launch_bounds__(TH == 32 ? 128 : TH) norm_bwd_kernel(const __grid_constant__ seq_norm_args a) {
  constexpr int kThreads = TH == 32 ? 128 : TH, kRows = kThreads / TH, P = kPairs<V>;
  constexpr bool kRing = V > 1;
  extern __shared__ __align__(16) uint8_t ring[];  // [kStages][3][VPT][kThreads] vectors of 16 bytes
  __shared__ __align__(16) float part[2][32];
  __shared__ float2 dws[kRows > 1 ? kRows * TH * P : 1];
  int turn = 0;
  signal_dependents();
  const int tid = threadIdx.x % TH, row_in = threadIdx.x / TH, c = (int)a.c, vecs = c / V;
  float2 w[VPT][P], dw[VPT][P] = {};
  load_w<T, V, TH, VPT>(a, tid, vecs, w);
  const int64_t step = (int64_t)gridDim.x * kRows;
  const T* dr = static_cast<const T*>(a.dr.data);
  int64_t row = (int64_t)blockIdx.x * kRows + row_in;
  auto at = [&](int stage, int which, int k) {
    return ring + (((stage * 3 + which) * VPT + k) * kThreads + threadIdx.x) * 16;
  };
  auto copy = [&](int64_t i, int stage) {
    if (i < a.n) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int64_t col = (k * TH + tid) * V;
        if (k * TH + tid < vecs) {
          cp_async16(at(stage, 0, k), static_cast<const T*>(a.r.data) + i * a.r.stride_n + col, 16);
          cp_async16(at(stage, 1, k), static_cast<const T*>(a.dy.data) + i * a.dy.stride_n + col, 16);
          if (dr) cp_async16(at(stage, 2, k), dr + i * a.dr.stride_n + col, 16);
        }
      }
    }
    cp_async_commit();
  };
  if constexpr (kRing) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) copy(row + s * step, s);
  }
  int stage = 0;
  for (; row < a.n; row += step) {
    const float rstd = a.rstd[row];
    Pack<T, V> pr[VPT], py[VPT], pd[VPT];
    if constexpr (kRing) {
      copy(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
      cp_async_wait<kStages - 1>();
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const bool in = k * TH + tid < vecs;
        pr[k] = in ? *reinterpret_cast<const Pack<T, V>*>(at(stage, 0, k)) : zero_pack<T, V>();
        py[k] = in ? *reinterpret_cast<const Pack<T, V>*>(at(stage, 1, k)) : zero_pack<T, V>();
        pd[k] = in && dr ? *reinterpret_cast<const Pack<T, V>*>(at(stage, 2, k)) : zero_pack<T, V>();
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    } else {
      load_row<T, V, TH, VPT>(static_cast<const T*>(a.r.data) + row * a.r.stride_n, tid, vecs, pr);
      load_row<T, V, TH, VPT>(static_cast<const T*>(a.dy.data) + row * a.dy.stride_n, tid, vecs, py);
      if (dr) {
        load_row<T, V, TH, VPT>(dr + row * a.dr.stride_n, tid, vecs, pd);
      } else {
#pragma unroll
        for (int k = 0; k < VPT; ++k) pd[k] = zero_pack<T, V>();
      }
    }
    float2 hat[VPT][P], g[VPT][P], sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      unpack(pr[k], hat[k]);
      unpack(py[k], g[k]);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        hat[k][p] = __fmul2_rn(hat[k][p], both(rstd));
        dw[k][p] = __ffma2_rn(g[k][p], hat[k][p], dw[k][p]);
        g[k][p] = __fmul2_rn(g[k][p], w[k][p]);
        sum = __ffma2_rn(g[k][p], hat[k][p], sum);
      }
    }
    const float mean = over_row<TH>(sum.x + sum.y, part, turn, Add()) * (1.f / (float)c);
    T* dx = static_cast<T*>(a.dx.data) + row * a.dx.stride_n;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float2 o[P];
      unpack(pd[k], o);
#pragma unroll
      for (int p = 0; p < P; ++p) o[p] = __ffma2_rn(both(rstd), __ffma2_rn(hat[k][p], both(-mean), g[k][p]), o[p]);
      if (k * TH + tid < vecs) store_pack(dx + (k * TH + tid) * V, pack<T, V>(o));
    }
  }
  float* slab = static_cast<float*>(a.ws) + (int64_t)blockIdx.x * a.c;
  auto put = [&](int64_t col, float2 v) {  // a pair of columns from `col` on
    if (col < c) slab[col] = v.x;
    if (V > 1 && col + 1 < c) slab[col + 1] = v.y;
  };
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    if constexpr (kRows > 1) {
      __syncthreads();
#pragma unroll
      for (int p = 0; p < P; ++p) dws[(row_in * TH + tid) * P + p] = dw[k][p];
      __syncthreads();
      for (int u = threadIdx.x; u < TH * P; u += kThreads) {
        float2 v = dws[u];
#pragma unroll
        for (int r = 1; r < kRows; ++r) v = __fadd2_rn(v, dws[r * TH * P + u]);
        put((int64_t)k * TH * V + (V == 1 ? u : 2 * u), v);
      }
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) put((int64_t)(k * TH + tid) * V + 2 * p, dw[k][p]);
    }
  }
}

// Rows too long for registers: the slab itself holds dw's running sums. One
// element a thread and step, r and dy read twice, far from the floor: 366 us for
// 4096 rows of 12288 bf16 (59 us), 356 us for 8192 of 5120 fp32 (99 us).
template <typename T>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const __grid_constant__ seq_norm_args a) {
  __shared__ __align__(16) float part[2][32];
  int turn = 0;
  signal_dependents();
  const bool w32 = a.w_dtype == CONV_F32;
  float* slab = static_cast<float*>(a.ws) + (int64_t)blockIdx.x * a.c;
  for (int64_t k = threadIdx.x; k < a.c; k += 1024) slab[k] = 0.f;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const T* r = static_cast<const T*>(a.r.data) + row * a.r.stride_n;
    const T* dy = static_cast<const T*>(a.dy.data) + row * a.dy.stride_n;
    const T* dr = a.dr.data ? static_cast<const T*>(a.dr.data) + row * a.dr.stride_n : nullptr;
    T* dx = static_cast<T*>(a.dx.data) + row * a.dx.stride_n;
    const float rstd = a.rstd[row];
    float sum = 0.f;
    for (int64_t k = threadIdx.x; k < a.c; k += 1024) {
      const float hat = to_f32(r[k]) * rstd, g = to_f32(dy[k]);
      slab[k] = fmaf(g, hat, slab[k]);
      sum = fmaf(g * param<T>(a.w, k, w32), hat, sum);
    }
    const float mean = over_row<1024>(sum, part, turn, Add()) / (float)a.c;
    for (int64_t k = threadIdx.x; k < a.c; k += 1024) {
      const float hat = to_f32(r[k]) * rstd;
      const float v = rstd * fmaf(-hat, mean, to_f32(dy[k]) * param<T>(a.w, k, w32));
      store_out(dx + k, v + (dr ? to_f32(dr[k]) : 0.f));
    }
  }
}

// kBwd: there is a backward kernel of this size.
template <typename T, int V, int TH, int VPT, bool kBwd = true>
cudaError_t launch_as(const seq_norm_args& a, bool bwd, cudaStream_t st) {
  constexpr int kThreads = TH == 32 ? 128 : TH, kRows = kThreads / TH;
  if (bwd) {
    if constexpr (kBwd) {
      constexpr int kSmem = V > 1 ? kStages * 3 * VPT * kThreads * 16 : 0;
      constexpr auto kernel = norm_bwd_kernel<T, V, TH, VPT>;
      const cudaError_t err = allow_smem<kernel>(kSmem);
      if (err != cudaSuccess) return err;
      kernel<<<(unsigned)norm_bwd_slabs(a.n, a.c), kThreads, kSmem, st>>>(a);
    }
  } else {
    const unsigned grid = (unsigned)((a.n + kRows - 1) / kRows);
    if (a.out8) norm_fwd_kernel<T, V, TH, VPT, true><<<grid, kThreads, 0, st>>>(a);
    else norm_fwd_kernel<T, V, TH, VPT, false><<<grid, kThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
bool vectors(const seq_norm_args& a) {
  constexpr int V = 16 / sizeof(T);
  auto ok = [&](const seq_tensor& v, int64_t size, int64_t bytes) {
    return !v.data || (reinterpret_cast<uintptr_t>(v.data) % bytes == 0 && v.stride_n * size % bytes == 0);
  };
  const int64_t e = sizeof(T);
  return a.c % V == 0 && ok(a.x, e, 16) && ok(a.residual, e, 16) && ok(a.r, e, 16) && ok(a.dy, e, 16) && ok(a.dr, e, 16) &&
         ok(a.dx, e, 16) && ok(a.y, a.out8 ? 1 : e, a.out8 ? V : 16) &&
         reinterpret_cast<uintptr_t>(a.w) % (a.w_dtype == CONV_F32 ? 4 * V : 16) == 0;
}

template <typename T>
cudaError_t launch_typed(const seq_norm_args& a, bool bwd, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  if (vectors<T>(a)) {
    const int64_t vecs = a.c / V;
    if (vecs <= 32) return launch_as<T, V, 32, 1>(a, bwd, st);
    if (vecs <= 64) return launch_as<T, V, 64, 1>(a, bwd, st);
    if (vecs <= 128) return launch_as<T, V, 64, 2>(a, bwd, st);
    if (vecs <= 256) return launch_as<T, V, 128, 2>(a, bwd, st);
    if (vecs <= 512) return launch_as<T, V, 256, 2>(a, bwd, st);
    if (vecs <= 1024) return launch_as<T, V, 512, 2>(a, bwd, st);
    if (vecs <= 2048 && !bwd) return launch_as<T, V, 1024, 2, false>(a, bwd, st);
  } else {
    if (a.c <= 512) return launch_as<T, 1, 128, 4>(a, bwd, st);
    if (a.c <= 2048) return launch_as<T, 1, 512, 4>(a, bwd, st);
    if (a.c <= 8192) return launch_as<T, 1, 1024, 8>(a, bwd, st);
  }
  if (bwd) norm_bwd_long_kernel<T><<<(unsigned)norm_bwd_slabs(a.n, a.c), 1024, 0, st>>>(a);
  else norm_fwd_long_kernel<T><<<(unsigned)a.n, 1024, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch(const seq_norm_args& a, bool bwd, cudaStream_t st) {
  if (a.dtype == CONV_F32) return launch_typed<float>(a, bwd, st);
  if (a.dtype == CONV_BF16) return launch_typed<__nv_bfloat16>(a, bwd, st);
  return launch_typed<__half>(a, bwd, st);
}

}  // namespace

// CTAs of the backward pass, and with them slabs: a fixed number for each of 152
// SMs by the row's length, at least four rows each. In 16 bits all of them run at
// once, as 512 threads an SM (1024 up to 256 columns; 304 slabs in place of 608 at
// 2048 columns: 55 us against 51, 456: 50). In fp32 from 513 columns on a CTA's
// ring takes 48 to 192 KB, and half of them run at a time. The sizes alone count,
// so that a workspace fits any call.
int64_t norm_bwd_slabs(int64_t n, int64_t c) {
  const int64_t threads = c <= 1024 ? 128 : c <= 2048 ? 256 : c <= 4096 ? 512 : 1024;
  int64_t most = 152 * (1024 / threads);
  if (most > (n + 3) / 4) most = (n + 3) / 4;
  return most < 1 ? 1 : most;
}

cudaError_t launch_seq_norm_fwd(const seq_norm_args& a, cudaStream_t st) { return launch(a, false, st); }
cudaError_t launch_seq_norm_bwd(const seq_norm_args& a, cudaStream_t st) {
  cudaError_t err = launch(a, true, st);
  if (err != cudaSuccess) return err;
  return launch_seq_slab_sum(
      slab_sum(static_cast<const float*>(a.ws), norm_bwd_slabs(a.n, a.c), slab_out(a.dw, a.c)), true, st);
}

}  // namespace cig
