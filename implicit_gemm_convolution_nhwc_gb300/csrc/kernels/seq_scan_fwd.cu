// Selective scan over a prompt.
//
//   h[t] = exp(delta A) h[t-1] + delta x B,  y = (C . h + D x) silu(z)
//
// Per token, channel and state: one exp and four fp32 operations (delta A,
// u B, and two multiply-adds), against 4 elements of HBM traffic per token and
// channel, so with 16 states the arithmetic bounds it: the special-function
// unit alone takes 4.2 cycles a warp and state, packed fp32 another 5.
//
// A lane holds NS states of a channel, as packed pairs, and LN neighbouring
// lanes hold the channel's NS LN >= s states (states past s have A = B = C = 0
// and stay 0). With all 16 states in one lane B and C, which all channels
// share, are read from shared memory by broadcast, and nothing crosses lanes:
// the loop alone takes 7.2 cycles a state with 16 states a lane, 8.7 with 8,
// 15.7 with 4, at four warps a scheduler. The shared loads are not what holds
// it up (7.0 cycles without them): the exponentials take 4.1, the four packed
// operations a pair 4.6, and the two overlap only in part.
//
// A CTA of 128 threads owns 128 / LN channels. Raw tokens arrive by asynchronous
// copies, two tiles ahead; B and C are converted to fp32 one tile ahead, so that
// a tile takes one barrier. delta, delta x and y of G tokens stay in registers:
// each of a channel's lanes converts its share of them, and passes delta and
// delta x on by shuffles where LN > 1. (Converted by the whole CTA through shared
// memory, with three barriers a tile, a prompt of 16384 tokens of 2048 channels
// and 16 states took 288 us; this way 273, with eight tokens a step in place of
// four 267: 18 cycles a state in the two launches together, of which the loops
// would take 12. The second launch's 128 registers spill 8 bytes a thread in 16
// bits with 16 states a lane, 12 in fp32.)
//
// Tokens follow one another, so few sequences times channels leave the GPU
// empty: the time axis is then cut into segments. A first launch computes each
// segment's own end state (from a zero start, C and y left out) and the sum of
// its deltas; in the second each segment starts from
// h <- exp(A sum delta_j) h + own_j over the segments j before it.
#include <type_traits>

#include "seq_scan.cuh"

namespace cig {
namespace {

template <typename T, int NS_, int LN_>
struct FwdTile {
  static constexpr int NS = NS_, LN = LN_, SP = NS * LN, CH = kScanThreads / LN;
  static constexpr int TT = LN == 1 && sizeof(T) == 4 ? 8 : 16;  // four CTAs an SM
  static constexpr int G = 8;                      // tokens a step of the loop
  static constexpr int E = 16 / (int)sizeof(T);   // elements of a staged pack
  static constexpr int kTok = TT * CH * (int)sizeof(T), kBc = TT * SP * (int)sizeof(T);
  static constexpr int kStages = 3, kStage = 3 * kTok + 2 * kBc;
  static constexpr int kB = kStages * kStage, kC = kB + 2 * TT * SP * 4;  // [2][TT][SP] fp32
  static constexpr int kBytes = kC + 2 * TT * SP * 4;
  static_assert(kScanCheckpoint % TT == 0 && TT % G == 0, "checkpoints stand at the start of tiles");
};

// kCarry: the first launch of a segmented scan.
template <typename T, int NS, int LN, bool kCarry>
__global__ void __launch_bounds__(kScanThreads, NS * LN == 64 ? 3 : 4) scan_fwd_kernel(const __grid_constant__ ScanParams p) {
  using Tile = FwdTile<T, NS, LN>;
  constexpr int TT = Tile::TT, CH = Tile::CH, SP = Tile::SP, E = Tile::E, G = Tile::G, P = NS / 2;
  extern __shared__ __align__(128) uint8_t smem[];
  float* sB = reinterpret_cast<float*>(smem + Tile::kB);  // [2][TT][SP]
  float* sC = reinterpret_cast<float*>(smem + Tile::kC);  // [2][TT][SP]

  if (kCarry) signal_dependents();
  const seq_scan_args& a = p.a;
  const ScanPlace w = scan_place<CH>(p, blockIdx.y);
  const int lane_ch = threadIdx.x / LN, q = threadIdx.x % LN, k0 = q * NS;
  const bool live = lane_ch < w.channels;
  const int64_t ch = w.c0 + lane_ch, nseg = p.p.segments;
  const int s = (int)a.s;
  const bool gate = !kCarry && a.z.data != nullptr;
  // Tokens worked on: past the length y is 0 and the state stays.
  const int64_t tend = w.t1 < w.len ? w.t1 : w.len;

  const int64_t tiles = tend > w.t0 ? (tend - w.t0 + TT - 1) / TT : 0;

  auto stage = [&](int64_t tile, int buf) {
    if (tile < tiles) {
      const int64_t tb = w.t0 + tile * TT;
      uint8_t* to = smem + buf * Tile::kStage;
      stage_tokens<T, TT, CH, E>(to, a.x, w, tb, tend, p.vec);
      stage_tokens<T, TT, CH, E>(to + Tile::kTok, a.dt, w, tb, tend, p.vec);
      if (gate) stage_tokens<T, TT, CH, E>(to + 2 * Tile::kTok, a.z, w, tb, tend, p.vec);
      stage_bc<T, TT, SP>(to + 3 * Tile::kTok, a.b, p, w, tb, tend);
      if (!kCarry) stage_bc<T, TT, SP>(to + 3 * Tile::kTok + Tile::kBc, a.cc, p, w, tb, tend);
    }
    cp_async_commit();
  };
  auto convert = [&](int64_t tile, int buf) {
    if (tile >= tiles) return;
    const uint8_t* raw = smem + buf * Tile::kStage + 3 * Tile::kTok;
    const int to = (int)(tile & 1) * TT * SP;
    convert_bc<T, TT, SP>(sB + to, raw, p);
    if (!kCarry) convert_bc<T, TT, SP>(sC + to, raw + Tile::kBc, p);
  };
  stage(0, 0);
  stage(1, 1);

  clear_padding<2 * TT, SP>(sB, s);
  clear_padding<2 * TT, SP>(sC, s);

  // exp(delta A) = 2^(delta A log2 e)
  if (!kCarry && nseg > 1) wait_for_primary();
  float2 A2[P], h[P];
#pragma unroll
  for (int j = 0; j < P; ++j) A2[j] = h[j] = make_float2(0.f, 0.f);
  if (live) {
    load_row<NS>(a.A + ch * s, k0, s, A2);
#pragma unroll
    for (int j = 0; j < P; ++j) A2[j] = __fmul2_rn(A2[j], both(kLog2e));
    // With segments the first launch keeps the start state in the last
    // segment's carry (so that state_out may be the state itself) and starts
    // segment 0 from it.
    if (kCarry || nseg == 1) {
      if (w.seg == 0 && a.state) load_row<NS>(a.state + (w.i * a.c + ch) * s, k0, s, h);
      if (kCarry && w.seg == 0) store_row<NS>(p.carry + ((w.i * nseg + nseg - 1) * a.c + ch) * s, k0, s, h);
    } else {
      load_row<NS>(p.carry + ((w.i * nseg + (w.seg == 0 ? nseg - 1 : 0)) * a.c + ch) * s, k0, s, h);
      // Loads of several segments are in flight at a time.
      constexpr int kAhead = 4;
      for (int64_t j = 1; j < w.seg; j += kAhead) {
        float2 own[kAhead][P];
        float sum[kAhead];
#pragma unroll
        for (int b = 0; b < kAhead; ++b) {
          const int64_t jj = j + b < w.seg ? j + b : w.seg - 1;
          load_row<NS>(p.carry + ((w.i * nseg + jj) * a.c + ch) * s, k0, s, own[b]);
          sum[b] = p.decay[(w.i * nseg + jj) * a.c + ch];
        }
#pragma unroll
        for (int b = 0; b < kAhead; ++b) {
          if (j + b < w.seg) {
#pragma unroll
            for (int m = 0; m < P; ++m) h[m] = __ffma2_rn(exp2_pair(__fmul2_rn(A2[m], both(sum[b]))), h[m], own[b][m]);
          }
        }
      }
    }
  }

  const float bias = live && a.dt_bias ? a.dt_bias[ch] : 0.f, D = live && a.D ? a.D[ch] : 0.f;
  float sum = 0.f;
  T* y = static_cast<T*>(a.y.data) + w.i * a.y.stride_n + ch;
  cp_async_wait<1>();
  convert(0, 0);
  int buf = 0;
  for (int64_t tile = 0; tile < tiles; ++tile, buf = buf == 2 ? 0 : buf + 1) {
    cp_async_wait<0>();
    // The next tile has landed, this one's B and C are converted, and the
    // buffers of the one before are free.
    __syncthreads();
    stage(tile + 2, buf == 0 ? 2 : buf - 1);
    convert(tile + 1, buf == 2 ? 0 : buf + 1);

    const int64_t tb = w.t0 + tile * TT;
    const int used = tend - tb < TT ? (int)(tend - tb) : TT;
    if (!kCarry && a.checkpoints && (TT == kScanCheckpoint || tb % kScanCheckpoint == 0) && live)
      store_row<NS>(a.checkpoints + ((w.i * p.checkpoints + tb / kScanCheckpoint) * a.c + ch) * s, k0, s, h);
    const T* at = reinterpret_cast<const T*>(smem + buf * Tile::kStage) + q * CH + lane_ch;
    const float* bat = sB + (int)(tile & 1) * TT * SP + k0;
    const float* cat = sC + (int)(tile & 1) * TT * SP + k0;
    // G tokens; each of the channel's lanes converts every LN-th.
    auto step = [&](int g, auto whole) {
      constexpr int M = G / LN;
      float x[M], d[M], u[M];
#pragma unroll
      for (int k = 0; k < M; ++k) {
        x[k] = to_f32(at[(g + k * LN) * CH]);
        d[k] = to_f32(at[(TT + g + k * LN) * CH]) + bias;
      }
      if (a.softplus) {
#pragma unroll
        for (int k = 0; k < M; ++k) d[k] = softplus(d[k]);
      }
#pragma unroll
      for (int k = 0; k < M; ++k) {
        if (!decltype(whole)::value && g + k * LN + q >= used) d[k] = 0.f;  // x and B are 0 there
        u[k] = d[k] * x[k];
      }
      float yv[G];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        float delta = d[i / LN], in = u[i / LN];
        if constexpr (LN > 1) {
          delta = __shfl_sync(0xffffffffu, delta, i % LN, LN);
          in = __shfl_sync(0xffffffffu, in, i % LN, LN);
        }
        float2 b[P], c[P];
        load_states<NS>(bat + (g + i) * SP, b);
        if (!kCarry) load_states<NS>(cat + (g + i) * SP, c);
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < P; ++m) {
          const float2 decay = decay_pair(both(delta), A2[m]);
          h[m] = __ffma2_rn(decay, h[m], __fmul2_rn(both(in), b[m]));
          if (!kCarry) acc = m == 0 ? __fmul2_rn(c[m], h[m]) : __ffma2_rn(c[m], h[m], acc);
        }
        if (kCarry) sum += delta;
        yv[i] = acc.x + acc.y;
      }
      if constexpr (!kCarry) {
        float out[M];
#pragma unroll
        for (int k = 0; k < M; ++k) {
          float v[LN];
#pragma unroll
          for (int j = 0; j < LN; ++j) v[j] = yv[k * LN + j];
          out[k] = fmaf(D, x[k], sum_over_lanes<LN>(v, q));
        }
        if (gate) {
#pragma unroll
          for (int k = 0; k < M; ++k) {
            const float z = to_f32(at[(2 * TT + g + k * LN) * CH]);
            out[k] *= z * sigmoid(z);
          }
        }
        T* to = y + (tb + g + q) * a.y.stride_l;
#pragma unroll
        for (int k = 0; k < M; ++k) {
          if (live && (decltype(whole)::value || g + k * LN + q < used)) store_out(to, out[k]);
          to += LN * a.y.stride_l;
        }
      }
    };
    int g = 0;
#pragma unroll 1
    for (; g + G <= used; g += G) step(g, std::true_type());
    if (g < used) step(g, std::false_type());
  }
  if constexpr (!kCarry) {  // tokens past the length
    if (live)
      for (int64_t t = (tend > w.t0 ? tend : w.t0) + q; t < w.t1; t += LN) y[t * a.y.stride_l] = zero_of<T>();
  }
  if (!live) return;
  if (kCarry) {
    store_row<NS>(p.carry + ((w.i * nseg + w.seg) * a.c + ch) * s, k0, s, h);
    if (q == 0) p.decay[(w.i * nseg + w.seg) * a.c + ch] = sum;
  } else if (a.state_out && w.seg == nseg - 1) {
    store_row<NS>(a.state_out + (w.i * a.c + ch) * s, k0, s, h);
  }
}

template <typename T, int NS, int LN>
cudaError_t launch_as(const seq_scan_args& a, const ScanPlan& plan, cudaStream_t st) {
  using Tile = FwdTile<T, NS, LN>;
  ScanParams p = scan_params(a, plan, false);
  p.vec = scan_vec<T>(a, Tile::E, false);
  p.vec_bc = scan_vec_bc<T>(a);
  constexpr auto main_kernel = scan_fwd_kernel<T, NS, LN, false>, carry_kernel = scan_fwd_kernel<T, NS, LN, true>;
  cudaError_t err = allow_smem<main_kernel>(Tile::kBytes);
  if (err != cudaSuccess) return err;
  const unsigned ctas = (unsigned)(a.n * plan.blocks);
  if (plan.segments > 1) {
    err = allow_smem<carry_kernel>(Tile::kBytes);
    if (err != cudaSuccess) return err;
    carry_kernel<<<dim3(ctas, (unsigned)(plan.segments - 1)), kScanThreads, Tile::kBytes, st>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    return launch_dependent(main_kernel, dim3(ctas, (unsigned)plan.segments), kScanThreads, Tile::kBytes, st, p);
  }
  main_kernel<<<ctas, kScanThreads, Tile::kBytes, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const seq_scan_args& a, const ScanPlan& p, cudaStream_t st) {
  if (p.per_lane == 4) return p.lanes == 1 ? launch_as<T, 4, 1>(a, p, st) : launch_as<T, 4, 2>(a, p, st);
  if (p.per_lane == 8) {
    if (p.lanes == 1) return launch_as<T, 8, 1>(a, p, st);
    return p.lanes == 2 ? launch_as<T, 8, 2>(a, p, st) : launch_as<T, 8, 4>(a, p, st);
  }
  if (p.lanes == 1) return launch_as<T, 16, 1>(a, p, st);
  return p.lanes == 2 ? launch_as<T, 16, 2>(a, p, st) : launch_as<T, 16, 4>(a, p, st);
}

}  // namespace

cudaError_t launch_seq_scan_fwd(const seq_scan_args& a, const ScanPlan& p, cudaStream_t st) {
  if (a.dtype == CONV_F32) return launch_typed<float>(a, p, st);
  if (a.dtype == CONV_BF16) return launch_typed<__nv_bfloat16>(a, p, st);
  return launch_typed<__half>(a, p, st);
}

}  // namespace cig
