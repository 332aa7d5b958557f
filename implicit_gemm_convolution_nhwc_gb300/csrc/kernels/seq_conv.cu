// Causal depthwise convolution along time: forward, backward and one token.
//
//   v[t][c] = bias[c] + sum_{j<W} w[c][j] x[t-(W-1)+j][c],  y = v or silu(v)
//
// Forward and backward are bound by HBM (2 and 3 elements of traffic for 2 W
// and 6 W operations and one exp): a thread owns one vector of channels and
// walks along a strip of tokens with the last W-1 inputs in registers, so each
// input is read once but for the W-1 tokens before a strip, and a warp's
// accesses are whole rows of 512 bytes. Loads are a block of tokens ahead, in
// shared memory. Pairs of channels share each instruction, and blocks wholly
// inside run without checks: with scalar arithmetic and a check a token the
// forward took 103 us where it now takes 23 (8 x 2048 tokens of 2048 bf16
// channels: 134 MB, 5.7 TB/s), the backward 163 us, now 40 (201 MB, 5.0 TB/s).
// (The forward's 128 registers spill 12 bytes a thread with SiLU and four taps of
// eight 16-bit channels; the backward's 127 do not spill.) Where 16 bytes do not
// fit, by channels, strides or addresses, a thread has one channel and no loads
// ahead, and issue bounds it: 49 and 115 us at 2046 channels.
#include "seq_common.cuh"

namespace cig {
namespace {

constexpr int kFwdThreads = 128;
// Tokens handled at a time: a block's loads are issued together, and the last
// inputs live in a ring of kBlock registers, token t at t mod kBlock, so that
// the window moves without copies (W <= kBlock).
constexpr int kBlock = 4;

// Vectors on their way from global memory: a thread's own slots of shared
// memory, kStages blocks of kBlock tokens of N tensors, filled by asynchronous
// copies and read back by the same thread, so that no barrier is needed and the
// loads ahead take no registers. Against loads of a block into registers before
// its first token: backward 50 -> 40 us, prompts of unequal length 51 -> 43 us.
// More stages than two gain nothing (backward 40 us with three, 41 with four;
// prompts 48 and 49).
constexpr int kStages = 2;
template <int kThreads, int N, int kBytes>
struct Ahead {
  static constexpr int kSmem = kStages * kBlock * N * kThreads * kBytes;
  uint8_t* base;
  __device__ __forceinline__ explicit Ahead(uint8_t* smem) : base(smem + threadIdx.x * kBytes) {}
  __device__ __forceinline__ uint8_t* slot(int stage, int u, int which) const {
    return base + ((stage * kBlock + u) * N + which) * (kThreads * kBytes);
  }
  template <typename T>
  __device__ __forceinline__ void fetch(int stage, int u, int which, const T* from) const {
    if constexpr (kBytes == 16) {
      cp_async16(slot(stage, u, which), from, 16);
    } else {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem_u32(slot(stage, u, which))), "l"(from) : "memory");
    }
  }
};

struct ConvParams {
  seq_conv_args a;
  int64_t strip, strips, vecs;
};

// N consecutive parameters stored as TW. By 16-byte loads where kVec says that
// w and bias are 16-byte aligned (the host checked) and N TW are multiples of
// 16 bytes; else one by one: four fp32 taps of one channel are 16 bytes too, but
// stand wherever their element's alignment allows.
template <bool kVec, int N, typename TW>
__device__ __forceinline__ void load_params(const TW* p, float (&v)[N]) {
  constexpr int U = kVec && N * sizeof(TW) % 16 == 0 ? 16 / (int)sizeof(TW) : 1;
#pragma unroll
  for (int k = 0; k < N; k += U) {
    const Pack<TW, U> q = load_pack<U>(p + k);
#pragma unroll
    for (int e = 0; e < U; ++e) v[k + e] = to_f32(q.v[e]);
  }
}
// The V channels' filters and biases.
template <typename T, int V, int W>
__device__ __forceinline__ void load_taps(const seq_conv_args& a, int64_t c0, float2 (&w)[W][kPairs<V>],
                                          float2 (&bias)[kPairs<V>]) {
  constexpr bool kVec = V > 1;
  float wv[V * W], bv[V] = {};
  if (a.w_dtype == CONV_F32) {
    load_params<kVec>(static_cast<const float*>(a.w) + c0 * W, wv);
    if (a.bias) load_params<kVec>(static_cast<const float*>(a.bias) + c0, bv);
  } else {
    load_params<kVec>(static_cast<const T*>(a.w) + c0 * W, wv);
    if (a.bias) load_params<kVec>(static_cast<const T*>(a.bias) + c0, bv);
  }
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) {
    bias[i] = make_float2(bv[2 * i], V > 1 ? bv[V > 1 ? 2 * i + 1 : 0] : 0.f);
#pragma unroll
    for (int j = 0; j < W; ++j)
      w[j][i] = make_float2(wv[2 * i * W + j], V > 1 ? wv[V > 1 ? (2 * i + 1) * W + j : 0] : 0.f);
  }
}

// x at time t of sequence i (t < 0: from the state, or 0).
template <typename T, int V, int W>
__device__ __forceinline__ Pack<T, V> history(const seq_conv_args& a, int64_t i, int64_t t, int64_t c0) {
  if (t >= 0) return load_pack<V>(static_cast<const T*>(a.x.data) + i * a.x.stride_n + t * a.x.stride_l + c0);
  if (a.state && t >= -(W - 1))
    return load_pack<V>(static_cast<const T*>(a.state) + (i * (W - 1) + t + (W - 1)) * a.c + c0);
  return zero_pack<T, V>();
}
// The W - 1 tokens before t0 (a multiple of kBlock), into their places of the ring.
template <typename T, int V, int W>
__device__ __forceinline__ void load_window(const seq_conv_args& a, int64_t i, int64_t t0, int64_t len, int64_t c0,
                                            float2 (&ring)[kBlock][kPairs<V>]) {
#pragma unroll
  for (int j = 1; j < W; ++j) {
    const int64_t t = t0 - j;
    unpack(t < len ? history<T, V, W>(a, i, t, c0) : zero_pack<T, V>(), ring[kBlock - j]);
  }
}
// bias + sum_j w[j] x[t - (W-1) + j] for the pair v and the token u of a block.
template <int P, int W>
__device__ __forceinline__ float2 taps(const float2 (&w)[W][P], const float2 (&ring)[kBlock][P], float2 acc, int u, int v) {
#pragma unroll
  for (int j = 0; j < W; ++j) acc = __ffma2_rn(w[j][v], ring[(u - (W - 1) + j) & (kBlock - 1)][v], acc);
  return acc;
}

template <typename T, int V, int W, bool kSilu>
__global__ void __launch_bounds__(kFwdThreads, 4) conv_fwd_kernel(const __grid_constant__ ConvParams p) {
  constexpr int P = kPairs<V>;
  extern __shared__ __align__(16) uint8_t smem[];
  const seq_conv_args& a = p.a;
  const int64_t id = (int64_t)blockIdx.x * kFwdThreads + threadIdx.x;
  const int64_t vec = id % p.vecs, row = id / p.vecs;
  const int64_t i = row / p.strips;
  if (i >= a.n) return;
  const int64_t s = row % p.strips, c0 = vec * V;
  const int64_t len = seq_length(a.lengths, i, a.l);
  const int64_t t0 = s * p.strip;
  // Tokens of the strip, and those of them inside the sequence.
  const int count = (int)(a.l - t0 < p.strip ? a.l - t0 : p.strip);
  const int inside = (int)(len < t0 ? 0 : (len - t0 < count ? len - t0 : count));
  T* y = static_cast<T*>(a.y.data) + i * a.y.stride_n + t0 * a.y.stride_l + c0;
  const int64_t sx = a.x.stride_l, sy = a.y.stride_l;
  int tb = 0;
  if (inside > 0) {
    float2 w[W][P], bias[P], ring[kBlock][P];
    load_taps<T, V, W>(a, c0, w, bias);
    load_window<T, V, W>(a, i, t0, len, c0, ring);
    const T* x = static_cast<const T*>(a.x.data) + i * a.x.stride_n + t0 * a.x.stride_l + c0;
    const Ahead<kFwdThreads, 1, V * (int)sizeof(T)> ahead(smem);
    auto fetch = [&](int from, int stage) {
      if constexpr (V > 1) {
#pragma unroll
        for (int u = 0; u < kBlock; ++u)
          if (from + u < inside) ahead.fetch(stage, u, 0, x + u * sx);
        cp_async_commit();
        x += kBlock * sx;
      }
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(k * kBlock, k);
    int stage = 0;
    for (; tb < inside; tb += kBlock) {
      Pack<T, V> next[kBlock];
      if constexpr (V > 1) {
        fetch(tb + (kStages - 1) * kBlock, stage == 0 ? kStages - 1 : stage - 1);
        cp_async_wait<kStages - 1>();
#pragma unroll
        for (int u = 0; u < kBlock; ++u) next[u] = *reinterpret_cast<const Pack<T, V>*>(ahead.slot(stage, u, 0));
        stage = stage == kStages - 1 ? 0 : stage + 1;
      } else {
#pragma unroll
        for (int u = 0; u < kBlock; ++u) next[u] = tb + u < inside ? load_pack_once<V>(x + u * sx) : zero_pack<T, V>();
        x += kBlock * sx;
      }
      if (tb + kBlock <= inside) {
#pragma unroll
        for (int u = 0; u < kBlock; ++u) {
          unpack(next[u], ring[u]);
          float2 out[P];
#pragma unroll
          for (int v = 0; v < P; ++v) {
            out[v] = taps<P, W>(w, ring, bias[v], u, v);
            if (kSilu) out[v] = __fmul2_rn(out[v], sigmoid_pair(out[v]));
          }
          store_pack(y + u * sy, pack<T, V>(out));
        }
      } else {  // the sequence ends inside the block
#pragma unroll
        for (int u = 0; u < kBlock; ++u) {
          if (tb + u >= count) break;
          unpack(tb + u < inside ? next[u] : zero_pack<T, V>(), ring[u]);
          float2 out[P];
#pragma unroll
          for (int v = 0; v < P; ++v) {
            out[v] = taps<P, W>(w, ring, bias[v], u, v);
            if (kSilu) out[v] = __fmul2_rn(out[v], sigmoid_pair(out[v]));
          }
          store_pack(y + u * sy, tb + u < inside ? pack<T, V>(out) : zero_pack<T, V>());
        }
      }
      y += kBlock * sy;
    }
  }
  // tb: past the last block that holds a used token
  for (; tb < count; ++tb, y += sy) store_pack(y, zero_pack<T, V>());
  // The state after the last token, by the threads that read the state (rows
  // of a state_out that is the state itself are read before they are
  // written: row j comes from row j + len).
  if (s == 0 && a.state_out) {
    T* so = static_cast<T*>(a.state_out) + i * (W - 1) * a.c + c0;
    for (int j = 0; j < W - 1; ++j) store_pack(so + j * a.c, history<T, V, W>(a, i, len - (W - 1) + j, c0));
  }
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kFwdThreads) conv_step_kernel(const __grid_constant__ ConvParams p) {
  const seq_conv_args& a = p.a;
  const int64_t id = (int64_t)blockIdx.x * kFwdThreads + threadIdx.x;
  const int64_t i = id / p.vecs, c0 = (id % p.vecs) * V;
  if (i >= a.n) return;
  T* y = static_cast<T*>(a.y.data) + i * a.y.stride_n + c0;
  const int64_t slot = a.slots ? a.slots[i] : i;
  if (slot < 0 || slot >= a.n_slots) {
    store_pack(y, zero_pack<T, V>());
    return;
  }
  T* st = static_cast<T*>(a.state_out) + slot * (W - 1) * a.c + c0;
  Pack<T, V> in[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) in[j] = load_pack<V>(st + j * a.c);
  in[W - 1] = load_pack<V>(static_cast<const T*>(a.x.data) + i * a.x.stride_n + c0);
  float2 w[W][kPairs<V>], out[kPairs<V>];
  load_taps<T, V, W>(a, c0, w, out);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_pack(st + j * a.c, in[j + 1]);
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float2 v[kPairs<V>];
    unpack(in[j], v);
#pragma unroll
    for (int k = 0; k < kPairs<V>; ++k) out[k] = __ffma2_rn(w[j][k], v[k], out[k]);
  }
#pragma unroll
  for (int k = 0; k < kPairs<V>; ++k)
    if (a.silu) out[k] = __fmul2_rn(out[k], sigmoid_pair(out[k]));
  store_pack(y, pack<T, V>(out));
}

// Backward. A thread walks its strip once: at token t it has dv[t] = dy[t]
// act'(v[t]) from the window of inputs, adds dv[t] x[t-(W-1)+j] to dw[j], and
// dx[t-(W-1)] = sum_j w[j] dv[t-j] is complete; the W-1 tokens after the strip
// are walked for dx alone.
constexpr int kBwdThreads = 32 * kConvBwdRows;

template <typename T, int V, int W, bool kSilu>
__global__ void __launch_bounds__(kBwdThreads, 2) conv_bwd_kernel(const __grid_constant__ ConvParams p) {
  constexpr int P = kPairs<V>;
  const seq_conv_args& a = p.a;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 part[kConvBwdRows][32 * P];
  signal_dependents();
  const int lane = threadIdx.x & 31, row_in = threadIdx.x >> 5;
  const int64_t vec = (int64_t)blockIdx.y * 32 + lane;
  const int64_t row = (int64_t)blockIdx.x * kConvBwdRows + row_in;
  const int64_t i = row / p.strips, s = row % p.strips, c0 = vec * V;
  float2 sums[W + 1][P] = {};  // dw, db
  if (vec < p.vecs && i < a.n) {
    const int64_t len = seq_length(a.lengths, i, a.l);
    const int64_t t0 = s * p.strip;
    const int count = (int)(a.l - t0 < p.strip ? a.l - t0 : p.strip);
    const int walk = count + W - 1;
    const int inside = (int)(len < t0 ? 0 : (len - t0 < walk ? len - t0 : walk));
    float2 w[W][P], bias[P], ring[kBlock][P], dvs[kBlock][P] = {};
    load_taps<T, V, W>(a, c0, w, bias);
    load_window<T, V, W>(a, i, t0, len, c0, ring);
    const T* x = static_cast<const T*>(a.x.data) + i * a.x.stride_n + t0 * a.x.stride_l + c0;
    const T* dy = static_cast<const T*>(a.dy.data) + i * a.dy.stride_n + t0 * a.dy.stride_l + c0;
    T* dx = static_cast<T*>(a.dx.data) + i * a.dx.stride_n + (t0 - (W - 1)) * a.dx.stride_l + c0;
    const int64_t sx = a.x.stride_l, sy = a.dy.stride_l, sd = a.dx.stride_l;
    // dv of token u of a block, from its dy
    auto through_act = [&](int u) {
#pragma unroll
      for (int v = 0; v < P; ++v) {
        const float2 pre = taps<P, W>(w, ring, bias[v], u, v);
        // silu'(v) = sig (1 + v (1 - sig))
        const float2 sig = sigmoid_pair(pre);
        const float2 less = __ffma2_rn(sig, both(-1.f), both(1.f));
        dvs[u][v] = __fmul2_rn(dvs[u][v], __fmul2_rn(sig, __ffma2_rn(pre, less, both(1.f))));
      }
    };
    auto add_sums = [&](int u) {
#pragma unroll
      for (int v = 0; v < P; ++v) {
        sums[W][v] = __fadd2_rn(sums[W][v], dvs[u][v]);
#pragma unroll
        for (int j = 0; j < W; ++j)
          sums[j][v] = __ffma2_rn(dvs[u][v], ring[(u - (W - 1) + j) & (kBlock - 1)][v], sums[j][v]);
      }
    };
    auto gather = [&](int u, float2(&out)[P]) {
#pragma unroll
      for (int v = 0; v < P; ++v)
#pragma unroll
        for (int j = 0; j < W; ++j) out[v] = __ffma2_rn(w[j][v], dvs[(u - j) & (kBlock - 1)][v], out[v]);
    };
    const Ahead<kBwdThreads, 2, V * (int)sizeof(T)> ahead(smem);
    auto fetch = [&](int from, int stage) {
      if constexpr (V > 1) {
#pragma unroll
        for (int u = 0; u < kBlock; ++u) {
          if (from + u < inside) {
            ahead.fetch(stage, u, 0, x + u * sx);
            ahead.fetch(stage, u, 1, dy + u * sy);
          }
        }
        cp_async_commit();
        x += kBlock * sx;
        dy += kBlock * sy;
      }
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(k * kBlock, k);
    int stage = 0;
    for (int tb = 0; tb < walk; tb += kBlock) {
      if constexpr (V > 1) {
        fetch(tb + (kStages - 1) * kBlock, stage == 0 ? kStages - 1 : stage - 1);
        cp_async_wait<kStages - 1>();
      }
      // Token u's x (0) or dy (1).
      auto token = [&](int u, int which) {
        if constexpr (V > 1) return *reinterpret_cast<const Pack<T, V>*>(ahead.slot(stage, u, which));
        else return load_pack<V>(which == 0 ? x + u * sx : dy + u * sy);
      };
      // Blocks wholly inside the strip and the sequence, with no gradient of
      // the final state to add, run without checks.
      if (tb >= W - 1 && tb + kBlock <= count && tb + kBlock <= inside && !a.dstate_out) {
        Pack<T, V> nx[kBlock], ny[kBlock];
#pragma unroll
        for (int u = 0; u < kBlock; ++u) {
          nx[u] = token(u, 0);
          ny[u] = token(u, 1);
        }
#pragma unroll
        for (int u = 0; u < kBlock; ++u) {
          unpack(nx[u], ring[u]);
          unpack(ny[u], dvs[u]);
          if (kSilu) through_act(u);
          add_sums(u);
          float2 out[P] = {};
          gather(u, out);
          store_pack(dx + u * sd, pack<T, V>(out));
        }
      } else {
#pragma unroll
        for (int u = 0; u < kBlock; ++u) {
          const int t = tb + u;
          if (t >= walk) break;
          const bool in = t < inside;
          unpack(in ? token(u, 0) : zero_pack<T, V>(), ring[u]);
          unpack(in ? token(u, 1) : zero_pack<T, V>(), dvs[u]);
          if (kSilu && in) through_act(u);
          if (t < count) add_sums(u);
          float2 out[P] = {};
          const int64_t to = t0 + t - (W - 1);  // the token whose dx is complete
          if (a.dstate_out && (t >= W - 1 || s == 0)) {
            const int64_t j_state = to - len + (W - 1);
            if (j_state >= 0 && j_state < W - 1)
              unpack(load_pack<V>(static_cast<const T*>(a.dstate_out) + (i * (W - 1) + j_state) * a.c + c0), out);
          }
          // Where none of the dv is inside nothing is added: weights that are
          // not finite would make NaN of the zeros.
          if (inside > 0 && t < inside + W - 1) gather(u, out);
          if (t >= W - 1) {
            store_pack(dx + u * sd, pack<T, V>(out));
          } else if (s == 0 && a.dstate) {
            store_pack(static_cast<T*>(a.dstate) + (i * (W - 1) + t) * a.c + c0, pack<T, V>(out));
          }
        }
      }
      if constexpr (V > 1) {
        stage = stage == kStages - 1 ? 0 : stage + 1;
      } else {
        x += kBlock * sx;
        dy += kBlock * sy;
      }
      dx += kBlock * sd;
    }
  }
  // Sums over the CTA's strips in order, one slab row [W + 1][c] a CTA.
  float* slab = static_cast<float*>(a.ws) + (int64_t)blockIdx.x * (W + 1) * a.c;
#pragma unroll
  for (int k = 0; k <= W; ++k) {
#pragma unroll
    for (int v = 0; v < P; ++v) part[row_in][lane * P + v] = sums[k][v];
    __syncthreads();
    for (int e = threadIdx.x; e < 32 * P; e += kBwdThreads) {
      float2 sum = part[0][e];
#pragma unroll
      for (int r = 1; r < kConvBwdRows; ++r) sum = __fadd2_rn(sum, part[r][e]);
      const int64_t c = (int64_t)blockIdx.y * 32 * V + (V == 1 ? e : 2 * e);
      if (c < a.c) slab[(int64_t)k * a.c + c] = sum.x;
      if (V > 1 && c + 1 < a.c) slab[(int64_t)k * a.c + c + 1] = sum.y;
    }
    __syncthreads();
  }
}

// Whether every address of a view is a multiple of `bytes`.
bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
template <typename T>
bool view_aligned(const seq_tensor& t, int64_t bytes) {
  const int64_t e = sizeof(T);
  return !t.data || (aligned(t.data, bytes) && t.stride_n * e % bytes == 0 && t.stride_l * e % bytes == 0);
}
template <typename T>
bool vectors(const seq_conv_args& a, int v) {
  const int64_t bytes = v * sizeof(T);
  return a.c % v == 0 && view_aligned<T>(a.x, bytes) && view_aligned<T>(a.y, bytes) && view_aligned<T>(a.dy, bytes) &&
         view_aligned<T>(a.dx, bytes) && aligned(a.state, bytes) && aligned(a.state_out, bytes) &&
         aligned(a.dstate, bytes) && aligned(a.dstate_out, bytes) && aligned(a.w, 16) && aligned(a.bias, 16);
}

// Tokens of a strip (at least `least`, a multiple of kBlock) such that the CTAs
// fill the GPU's places in whole rounds: the last round is as long as a full one.
// Of the first rounds that keep a strip at 128 tokens or less the cheapest is
// taken, at the strip's tokens and about eight more for its start (taps, window,
// W - 1 tokens read twice). `ctas` of a number of strips; `strips` that a number
// of CTAs hold. With strips of powers of two instead (64 forward, 128 backward)
// 8 x 2048 tokens of 2048 channels left 16 % of the places empty: forward 25.4 us,
// so 23.6 us; backward 55.7 us, so 49.8 us; 4 prompts of up to 4096 tokens by 4096
// channels, 1.7 rounds, 55.3 us, so 51.1 us (all before loads went ahead; at most
// 64 tokens: 46 us for those prompts against 43). The places are those of 152 SMs
// whatever the device, so that a workspace's size follows from the call's alone.
constexpr int64_t kFwdPlaces = 152 * 4, kBwdPlaces = 152 * 2;
template <class Ctas, class Strips>
int64_t balanced_strip(int64_t l, int64_t least, int64_t places, Ctas ctas, Strips strips) {
  constexpr int64_t kMost = 128, kStart = 8;
  const int64_t first = (ctas((l + kMost - 1) / kMost) + places - 1) / places;
  int64_t best = kMost, best_cost = 0;
  for (int64_t rounds = first < 1 ? 1 : first; rounds < first + 3; ++rounds) {
    const int64_t some = strips(rounds * places);
    if (some < 1) continue;
    int64_t strip = ((l + some - 1) / some + kBlock - 1) / kBlock * kBlock;
    if (strip > kMost) strip = kMost;
    if (strip < least) strip = least;
    const int64_t cost = rounds * (strip + kStart);
    if (best_cost == 0 || cost < best_cost) {
      best = strip;
      best_cost = cost;
    }
  }
  return best;
}

enum Which { kFwd, kBwd, kStep };

template <Which kWhich, typename T, int V, int W>
cudaError_t launch_as(const seq_conv_args& a, cudaStream_t st) {
  ConvParams p;
  p.a = a;
  p.vecs = a.c / V;
  if constexpr (kWhich == kStep) {
    const int64_t threads = a.n * p.vecs;
    conv_step_kernel<T, V, W><<<(unsigned)((threads + kFwdThreads - 1) / kFwdThreads), kFwdThreads, 0, st>>>(p);
  } else if constexpr (kWhich == kFwd) {
    const int64_t per_strip = a.n * p.vecs;
    p.strip = balanced_strip(a.l, 8, kFwdPlaces, [&](int64_t strips) { return (strips * per_strip + kFwdThreads - 1) / kFwdThreads; },
                             [&](int64_t ctas) { return ctas * kFwdThreads / per_strip; });
    p.strips = (a.l + p.strip - 1) / p.strip;
    if (p.strips < 1) p.strips = 1;  // an empty prompt still moves its state on
    const int64_t threads = a.n * p.strips * p.vecs;
    const unsigned grid = (unsigned)((threads + kFwdThreads - 1) / kFwdThreads);
    constexpr int kSmem = V > 1 ? Ahead<kFwdThreads, 1, V * (int)sizeof(T)>::kSmem : 0;  // under 48 KB
    if (a.silu) conv_fwd_kernel<T, V, W, true><<<grid, kFwdThreads, kSmem, st>>>(p);
    else conv_fwd_kernel<T, V, W, false><<<grid, kFwdThreads, kSmem, st>>>(p);
  } else {
    const ConvBwdPlan b = conv_bwd_plan(a.n, a.l, a.c);
    p.strip = b.strip;
    p.strips = b.strips;
    const dim3 grid((unsigned)b.slabs, (unsigned)((p.vecs + 31) / 32));
    constexpr int kSmem = V > 1 ? Ahead<kBwdThreads, 2, V * (int)sizeof(T)>::kSmem : 0;
    constexpr auto with_silu = conv_bwd_kernel<T, V, W, true>, without = conv_bwd_kernel<T, V, W, false>;
    cudaError_t err = a.silu ? allow_smem<with_silu>(kSmem) : allow_smem<without>(kSmem);
    if (err != cudaSuccess) return err;
    (a.silu ? with_silu : without)<<<grid, kBwdThreads, kSmem, st>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const SlabOut dw = {a.dw, a.c * W, a.c, 1, W};  // from [W][c]
    return launch_seq_slab_sum(slab_sum(static_cast<const float*>(a.ws), b.slabs, dw, slab_out(a.db, a.c)), true, st);
  }
  return cudaGetLastError();
}

template <Which kWhich, typename T, int V>
cudaError_t launch_width(const seq_conv_args& a, cudaStream_t st) {
  switch (a.width) {
    case 1: return launch_as<kWhich, T, V, 1>(a, st);
    case 2: return launch_as<kWhich, T, V, 2>(a, st);
    case 3: return launch_as<kWhich, T, V, 3>(a, st);
    default: return launch_as<kWhich, T, V, 4>(a, st);
  }
}

// 16 bytes a thread; half of that for 16-bit tensors in the backward pass,
// whose sums take four registers a channel more.
template <Which kWhich, typename T>
cudaError_t launch_typed(const seq_conv_args& a, cudaStream_t st) {
  constexpr int kVec = kWhich == kBwd ? 4 : 16 / (int)sizeof(T);
  return vectors<T>(a, kVec) ? launch_width<kWhich, T, kVec>(a, st) : launch_width<kWhich, T, 1>(a, st);
}

template <Which kWhich>
cudaError_t launch(const seq_conv_args& a, cudaStream_t st) {
  if (a.dtype == CONV_F32) return launch_typed<kWhich, float>(a, st);
  if (a.dtype == CONV_BF16) return launch_typed<kWhich, __nv_bfloat16>(a, st);
  return launch_typed<kWhich, __half>(a, st);
}

}  // namespace

ConvBwdPlan conv_bwd_plan(int64_t n, int64_t l, int64_t c) {
  const int64_t columns = ((c + 3) / 4 + 31) / 32;  // CTAs side by side
  ConvBwdPlan p;
  p.strip = 16;
  if (n > 0)
    p.strip = balanced_strip(l, 16, kBwdPlaces,
                             [&](int64_t strips) { return (n * strips + kConvBwdRows - 1) / kConvBwdRows * columns; },
                             [&](int64_t ctas) { return ctas / columns * kConvBwdRows / n; });
  p.strips = (l + p.strip - 1) / p.strip;
  if (p.strips < 1) p.strips = 1;
  p.slabs = (n * p.strips + kConvBwdRows - 1) / kConvBwdRows;
  return p;
}

cudaError_t launch_seq_conv_fwd(const seq_conv_args& a, cudaStream_t st) { return launch<kFwd>(a, st); }
cudaError_t launch_seq_conv_bwd(const seq_conv_args& a, cudaStream_t st) { return launch<kBwd>(a, st); }
cudaError_t launch_seq_conv_step(const seq_conv_args& a, cudaStream_t st) { return launch<kStep>(a, st); }

}  // namespace cig
