// What the forward and the backward scan share: where a CTA works, and how
// tiles of tokens and rows of states move.
#pragma once

#include "seq_common.cuh"

namespace cig {

struct ScanParams {
  seq_scan_args a;
  ScanPlan p;
  float* carry;   // [n][segments][c][s]
  float* decay;   // [n][segments][c]
  float* dbc;     // [blocks][n][l][2][s]
  float* sums;    // [n * segments][c (s + 2)]: dA, dD, ddt_bias
  int64_t checkpoints;  // kept states of a sequence
  bool vec;       // x, dt, z, dy, y and gradients by packs of E channels
  bool vec_bc;    // B and C by 16-byte units
};

// Where a CTA works.
struct ScanPlace {
  int64_t i, seg, grp, c0;  // sequence, segment, group, first channel
  int channels;             // valid channels
  int64_t block;            // channel block over all groups
  int64_t t0, t1;           // its tokens
  int64_t len;              // used tokens of the sequence
};

template <int CH>
__device__ __forceinline__ ScanPlace scan_place(const ScanParams& p, int64_t seg) {
  ScanPlace w;
  const int64_t id = blockIdx.x;
  w.block = id % p.p.blocks;
  w.i = id / p.p.blocks;
  w.seg = seg;
  w.grp = w.block / p.p.blocks_per_group;
  const int64_t per_group = p.a.c / p.a.g;
  const int64_t in_group = (w.block % p.p.blocks_per_group) * CH;
  w.c0 = w.grp * per_group + in_group;
  w.channels = (int)(per_group - in_group < CH ? per_group - in_group : CH);
  w.t0 = seg * p.p.segment;
  w.t1 = w.t0 + p.p.segment < p.a.l ? w.t0 + p.p.segment : p.a.l;
  w.len = seq_length(p.a.lengths, w.i, p.a.l);
  return w;
}

// Copies a [TT][CH] tile of tokens (from tb, valid below tend) into `dst`;
// elements outside are zero. Packs of E elements are dealt to the threads
// round robin.
template <typename T, int TT, int CH, int E>
__device__ __forceinline__ void stage_tokens(uint8_t* dst, const seq_tensor& v, const ScanPlace& w, int64_t tb,
                                             int64_t tend, bool vec) {
  constexpr int PR = CH / E;
  static_assert(E * sizeof(T) == 16, "a pack is one asynchronous copy");
  const T* base = static_cast<const T*>(v.data) + w.i * v.stride_n + tb * v.stride_l + w.c0;
  const int rows = tend - tb < TT ? (int)(tend - tb) : TT;
#pragma unroll
  for (int k = 0; k < (TT * PR + kScanThreads - 1) / kScanThreads; ++k) {
    const int u = threadIdx.x + k * kScanThreads, row = u / PR, col = (u % PR) * E;
    if (TT * PR % kScanThreads != 0 && u >= TT * PR) break;
    uint8_t* to = dst + (row * CH + col) * (int)sizeof(T);
    const T* from = base + row * v.stride_l + col;
    if (vec) {
      const bool in = row < rows && col < w.channels;
      if (!in) from = static_cast<const T*>(v.data);
      cp_async16(to, from, in ? 16u : 0u);
    } else {
      T* out = reinterpret_cast<T*>(to);
#pragma unroll
      for (int e = 0; e < E; ++e) out[e] = row < rows && col + e < w.channels ? from[e] : zero_of<T>();
    }
  }
}
// E results of one token; `room` valid channels from the first on.
template <typename T, int E>
__device__ __forceinline__ void store_tokens(T* to, const Pack<T, E>& v, int room, bool vec) {
  if (vec) {
    constexpr int H = E * sizeof(T) > 16 ? 16 / (int)sizeof(T) : E;
#pragma unroll
    for (int e = 0; e < E; e += H) store_pack(to + e, *reinterpret_cast<const Pack<T, H>*>(&v.v[e]));
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e < room) to[e] = v.v[e];
  }
}

// Units of a [TT][SP] tile (B or C) are dealt to the threads round robin; the
// thread that copies a unit also converts it. Tokens from tend on are 0.
template <typename T, int TT, int SP>
__device__ __forceinline__ void stage_bc(uint8_t* dst, const seq_tensor& v, const ScanParams& p, const ScanPlace& w,
                                         int64_t tb, int64_t tend) {
  const int s = (int)p.a.s;
  const T* base = static_cast<const T*>(v.data) + w.i * v.stride_n + tb * v.stride_l + w.grp * s;
  const int rows = tend - tb < TT ? (int)(tend - tb) : TT;
  if (p.vec_bc) {
    constexpr int U = 16 / (int)sizeof(T), kUnits = SP >= U ? SP / U : 1;
#pragma unroll
    for (int k = 0; k < (TT * kUnits + kScanThreads - 1) / kScanThreads; ++k) {
      const int u = threadIdx.x + k * kScanThreads, row = u / kUnits, col = (u % kUnits) * U;
      if (u < TT * kUnits && col < s) {
        const bool in = row < rows;
        cp_async16(dst + (row * SP + col) * (int)sizeof(T),
                   in ? base + row * v.stride_l + col : static_cast<const T*>(v.data), in ? 16u : 0u);
      }
    }
  } else {
    T* out = reinterpret_cast<T*>(dst);
    for (int u = threadIdx.x; u < TT * SP; u += kScanThreads) {
      const int row = u / SP, col = u % SP;
      if (col < s) out[u] = row < rows ? base[row * v.stride_l + col] : zero_of<T>();
    }
  }
}
template <typename T, int TT, int SP>
__device__ __forceinline__ void convert_bc(float* dst, const uint8_t* src, const ScanParams& p) {
  const T* raw = reinterpret_cast<const T*>(src);
  const int s = (int)p.a.s;
  if (p.vec_bc) {
    constexpr int U = 16 / (int)sizeof(T), kUnits = SP >= U ? SP / U : 1;
#pragma unroll
    for (int k = 0; k < (TT * kUnits + kScanThreads - 1) / kScanThreads; ++k) {
      const int u = threadIdx.x + k * kScanThreads, row = u / kUnits, col = (u % kUnits) * U;
      if (u < TT * kUnits && col < s) {
        float2 v[U / 2];
        unpack(load_pack<U>(raw + row * SP + col), v);
#pragma unroll
        for (int e = 0; e < U / 2; e += 2)
          *reinterpret_cast<float4*>(dst + row * SP + col + 2 * e) = make_float4(v[e].x, v[e].y, v[e + 1].x, v[e + 1].y);
      }
    }
  } else {
    for (int u = threadIdx.x; u < TT * SP; u += kScanThreads)
      if (u % SP < s) dst[u] = to_f32(raw[u]);
  }
}

// Columns s .. SP of the fp32 B and C tiles are 0 throughout.
template <int TT, int SP>
__device__ __forceinline__ void clear_padding(float* dst, int s) {
  for (int u = threadIdx.x; u < TT * SP; u += kScanThreads)
    if (u % SP >= s) dst[u] = 0.f;
}

// NS consecutive fp32 of shared memory.
template <int NS>
__device__ __forceinline__ void load_states(const float* p, float2 (&v)[NS / 2]) {
  if constexpr (NS % 4 == 0) {
#pragma unroll
    for (int k = 0; k < NS; k += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + k);
      v[k / 2] = make_float2(q.x, q.y);
      v[k / 2 + 1] = make_float2(q.z, q.w);
    }
  } else {
    v[0] = *reinterpret_cast<const float2*>(p);
  }
}

// A lane's states of a dense [..][s] row in global memory (k0 = its first
// state; states at and past s read as 0 and are not written). Aligned rows of
// a multiple of 4 states move by 16 bytes.
template <int NS>
__device__ __forceinline__ void load_row(const float* row, int k0, int s, float2 (&v)[NS / 2]) {
  if (NS % 4 == 0 && (s & 3) == 0 && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
#pragma unroll
    for (int k = 0; k + 3 < NS; k += 4) {
      const float4 q = k0 + k < s ? *reinterpret_cast<const float4*>(row + k0 + k) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[k / 2] = make_float2(q.x, q.y);
      v[k / 2 + 1] = make_float2(q.z, q.w);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NS / 2; ++j) {
    v[j].x = k0 + 2 * j < s ? row[k0 + 2 * j] : 0.f;
    v[j].y = k0 + 2 * j + 1 < s ? row[k0 + 2 * j + 1] : 0.f;
  }
}
template <int NS>
__device__ __forceinline__ void store_row(float* row, int k0, int s, const float2 (&v)[NS / 2]) {
  if (NS % 4 == 0 && (s & 3) == 0 && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
#pragma unroll
    for (int k = 0; k + 3 < NS; k += 4)
      if (k0 + k < s)
        *reinterpret_cast<float4*>(row + k0 + k) = make_float4(v[k / 2].x, v[k / 2].y, v[k / 2 + 1].x, v[k / 2 + 1].y);
    return;
  }
#pragma unroll
  for (int j = 0; j < NS / 2; ++j) {
    if (k0 + 2 * j < s) row[k0 + 2 * j] = v[j].x;
    if (k0 + 2 * j + 1 < s) row[k0 + 2 * j + 1] = v[j].y;
  }
}

// Plan and strides checked by the host: whether packs of E channels (16 bytes)
// are aligned and never straddle the end of a group.
template <typename T>
inline bool scan_vec(const seq_scan_args& a, int e, bool backward) {
  const int64_t size = sizeof(T);
  auto ok = [&](const seq_tensor& t) {
    return !t.data || (reinterpret_cast<uintptr_t>(t.data) % 16 == 0 && t.stride_n * size % 16 == 0 &&
                       t.stride_l * size % 16 == 0);
  };
  const bool v = a.c / a.g % e == 0 && ok(a.x) && ok(a.dt) && ok(a.z);
  return backward ? v && ok(a.dy) && ok(a.dx) && ok(a.ddt) && ok(a.dz) : v && ok(a.y);
}
template <typename T>
inline bool scan_vec_bc(const seq_scan_args& a) {
  auto ok = [&](const seq_tensor& t) {
    return reinterpret_cast<uintptr_t>(t.data) % 16 == 0 && t.stride_n * (int64_t)sizeof(T) % 16 == 0 &&
           t.stride_l * (int64_t)sizeof(T) % 16 == 0;
  };
  return a.s * (int64_t)sizeof(T) % 16 == 0 && ok(a.b) && ok(a.cc);
}

inline ScanParams scan_params(const seq_scan_args& a, const ScanPlan& p, bool backward) {
  ScanParams q;
  q.a = a;
  q.p = p;
  const ScanWorkspace w = scan_workspace(p, a.n, a.l, a.c, a.s, backward);
  char* base = static_cast<char*>(a.ws);
  q.carry = reinterpret_cast<float*>(base + w.carry);
  q.decay = reinterpret_cast<float*>(base + w.decay);
  q.dbc = reinterpret_cast<float*>(base + w.dbc);
  q.sums = reinterpret_cast<float*>(base + w.sums);
  q.checkpoints = (a.l + kScanCheckpoint - 1) / kScanCheckpoint;
  return q;
}

}  // namespace cig
