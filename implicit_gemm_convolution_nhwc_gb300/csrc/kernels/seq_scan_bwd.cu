// Gradients of the selective scan.
//
// With dy' = dy silu(z) and G[t] = C dy' + exp(delta A)[t+1] G[t+1]:
//   dx = delta (G . B) + D dy'            dB = sum over channels of G delta x
//   d delta = G . (A p + x B)             dC = sum over channels of dy' h
//   dA = sum over tokens of G p delta     dD = sum of dy' x
//   dz = dy (C . h + D x) silu'(z)        with p = exp(delta A) h[t-1]
//
// Tokens run from the last to the first with G in registers. The forward pass
// keeps one state in 16 tokens: from it a lane recomputes the states of the 16
// tokens into registers and then walks back over them. Per token, channel and
// state that is two exps and 14 fp32 operations, and sums in both directions:
// over the states (of y, dx and d delta) and over the channels (of dB and dC).
//
// A lane holds NS states of one channel; a warp is LN groups of lanes (the
// states) by 32 / LN channels, a CTA four warps. Sums over states cross the LN
// groups for LN tokens at once, sums over a warp's channels halve the values
// at each exchange. Matrix products with a matrix of ones in the exchanges'
// place (two each, for all 22 bits) took longer (656 us against 491 us at the
// time): each product wants its operands in neighbouring registers.
//
// 4 x 2048 tokens of 2048 channels and 16 states take 410 us, 336 us of them in
// the main launch: 197 cycles a token and warp at four warps a scheduler, for 120
// instructions. No unit is full (issue 61 %, shared memory 59 %, fp32 39 %,
// special functions 19 %); it is bound by the latencies along a token (the
// recurrence, the exchanges), which four warps hide in part: at three CTAs an
// SM it took a fifth longer. The bound of 128 registers that four CTAs need
// spills little: 48 bytes stored and 44 loaded a thread with four states a lane,
// 28 and 44 with two. All segments wait for the first launch. The last one needs
// nothing of it, but starting it early gained just 2 us and was not kept.
//
// The warps' sums meet in shared memory, the channel blocks' in one slab each
// in the workspace. Everything is added in an order fixed by the sizes.
//
// A time axis cut into segments runs as in the forward pass, mirrored: a first
// launch computes each segment's own gradient at its start.
#include <type_traits>

#include "seq_scan.cuh"

namespace cig {
namespace {

// The order of a lane's four states. dB and dC are summed over the CL lanes of a
// group by halving: at each exchange a lane keeps half of its values and sends
// the other half, which takes two selections a value, by the lane's number,
// where all lanes hold their states in the same order. So the upper half of a
// group's lanes holds its two pairs of states the other way round, and in the
// first exchange everyone keeps register pair 0 and sends pair 1. `turn` is 0
// or 2, the first state of pair 0.
template <int NS>
__device__ __forceinline__ void turn_pairs(float2 (&v)[NS / 2], int turn) {
  if constexpr (NS == 4) {
    const float2 a = turn ? v[1] : v[0], b = turn ? v[0] : v[1];
    v[0] = a;
    v[1] = b;
  }
}
__device__ __forceinline__ float2 from_lane(float2 v, int mask) {
  return make_float2(__shfl_xor_sync(0xffffffffu, v.x, mask), __shfl_xor_sync(0xffffffffu, v.y, mask));
}
template <int NS>
__device__ __forceinline__ void load_turned(const float* p, int turn, float2 (&v)[NS / 2]) {
  v[0] = *reinterpret_cast<const float2*>(p + turn);
  if constexpr (NS == 4) v[1] = *reinterpret_cast<const float2*>(p + (turn ^ 2));
}

// Sums v[k], k < W, over the CL lanes of a group (their values are halved at
// each step until one is left). On return v[0 ..] are the sums of the values
// from `base` on; `first` is false on lanes that repeat another lane's.
template <int W, int CL>
__device__ __forceinline__ void sum_over_channels(float (&v)[W], int lane, int& base, bool& first) {
  base = 0;
  first = true;
  int width = W;
#pragma unroll
  for (int mask = CL / 2; mask >= 1; mask /= 2) {
    const bool up = (lane & mask) != 0;
    if (width > 1) {
      width /= 2;
#pragma unroll
      for (int k = 0; k < W / 2; ++k) {
        if (k < width) {
          const float keep = up ? v[k + width] : v[k], send = up ? v[k] : v[k + width];
          v[k] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
        }
      }
      if (up) base += width;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], mask);
      if (up) first = false;
    }
  }
}

// Sums v[k], k < LN, over the LN lane groups: group q ends with the sum of v[q].
template <int LN>
__device__ __forceinline__ float sum_over_groups(float (&v)[LN], int q) {
#pragma unroll
  for (int w = LN / 2; w >= 1; w /= 2) {
    const bool up = (q & w) != 0;
#pragma unroll
    for (int k = 0; k < w; ++k) {
      const float keep = up ? v[k + w] : v[k], send = up ? v[k] : v[k + w];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, send, w * (32 / LN));
    }
  }
  return v[0];
}

template <typename T, int NS_, int LN_>
struct BwdTile {
  static constexpr int NS = NS_, LN = LN_, SP = NS * LN, CL = 32 / LN, CH = kScanThreads / LN;
  static constexpr int TT = 32, CK = kScanCheckpoint;
  static constexpr int E = 16 / (int)sizeof(T);             // elements of a staged pack
  static constexpr int PAIRS = TT * CH / 2 / kScanThreads;  // pairs of channels of a thread
  static constexpr int DP = CH + 4, YP = CH + 8;  // pitches: LN tokens of CL channels on different banks
  static constexpr int kTok = TT * CH * (int)sizeof(T), kBc = TT * SP * (int)sizeof(T);
  static constexpr int kStage = 4 * kTok + 2 * kBc;
  static constexpr int kDd = 2 * kStage;            // float2 [TT][DP]: delta, delta x (then G . B)
  static constexpr int kDy = kDd + TT * DP * 8;     // [TT][DP]: dy silu(z)
  static constexpr int kB = kDy + TT * DP * 4;      // [TT][SP]
  static constexpr int kC = kB + TT * SP * 4;       // [TT][SP]
  static constexpr int kY = kC + TT * SP * 4;       // [TT][YP]: C . h
  static constexpr int kQA = kY + TT * YP * 4;      // [TT][YP]: G p . A2
  static constexpr int kRed = kQA + TT * YP * 4;    // [4][CK][2 SP]: a warp's dB, dC
  static constexpr int kBytes = kRed + 4 * CK * 2 * SP * 4;
  static_assert(CH >= E && PAIRS >= 1 && kScanThreads % (CH / 2) == 0, "a thread keeps its pair of channels");
};

template <typename T, int NS, int LN>
__global__ void __launch_bounds__(kScanThreads, LN <= 4 ? 4 : 2) scan_bwd_kernel(const __grid_constant__ ScanParams p) {
  using Tile = BwdTile<T, NS, LN>;
  constexpr int TT = Tile::TT, CH = Tile::CH, CL = Tile::CL, SP = Tile::SP, E = Tile::E, DP = Tile::DP, YP = Tile::YP,
                CK = Tile::CK, P = NS / 2;
  extern __shared__ __align__(128) uint8_t smem[];
  float2* sdd = reinterpret_cast<float2*>(smem + Tile::kDd);
  float* sdy = reinterpret_cast<float*>(smem + Tile::kDy);
  float* sB = reinterpret_cast<float*>(smem + Tile::kB);
  float* sC = reinterpret_cast<float*>(smem + Tile::kC);
  float* sY = reinterpret_cast<float*>(smem + Tile::kY);
  float* sQA = reinterpret_cast<float*>(smem + Tile::kQA);
  float* sred = reinterpret_cast<float*>(smem + Tile::kRed);

  signal_dependents();
  const seq_scan_args& a = p.a;
  const ScanPlace w = scan_place<CH>(p, blockIdx.y);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane / CL, k0 = q * NS, lane_ch = warp * CL + lane % CL;
  const int turn = NS == 4 && (lane & (CL / 2)) ? 2 : 0;
  const bool live = lane_ch < w.channels;
  const int64_t ch = w.c0 + lane_ch, nseg = p.p.segments;
  const int s = (int)a.s;
  const bool gate = a.z.data != nullptr;
  // Tokens worked on: past the length all gradients are 0, and G passes by.
  const int64_t tend = w.t1 < w.len ? w.t1 : w.len;
  const int64_t tiles = tend > w.t0 ? (tend - w.t0 + TT - 1) / TT : 0;

  auto stage = [&](int64_t tb, int buf) {
    uint8_t* to = smem + buf * Tile::kStage;
    stage_tokens<T, TT, CH, E>(to, a.x, w, tb, tend, p.vec);
    stage_tokens<T, TT, CH, E>(to + Tile::kTok, a.dt, w, tb, tend, p.vec);
    if (gate) stage_tokens<T, TT, CH, E>(to + 2 * Tile::kTok, a.z, w, tb, tend, p.vec);
    stage_tokens<T, TT, CH, E>(to + 3 * Tile::kTok, a.dy, w, tb, tend, p.vec);
    stage_bc<T, TT, SP>(to + 4 * Tile::kTok, a.b, p, w, tb, tend);
    stage_bc<T, TT, SP>(to + 4 * Tile::kTok + Tile::kBc, a.cc, p, w, tb, tend);
    cp_async_commit();
  };
  if (tiles > 0) stage(w.t0 + (tiles - 1) * TT, 0);

  clear_padding<TT, SP>(sB, s);
  clear_padding<TT, SP>(sC, s);

  if (nseg > 1) wait_for_primary();
  float2 A2[P], aG[P], dA[P];  // aG: exp(delta A)[t+1] G[t+1]
#pragma unroll
  for (int j = 0; j < P; ++j) A2[j] = aG[j] = dA[j] = make_float2(0.f, 0.f);
  if (live) {
    load_row<NS>(a.A + ch * s, k0, s, A2);
#pragma unroll
    for (int j = 0; j < P; ++j) A2[j] = __fmul2_rn(A2[j], both(kLog2e));
    if (w.seg == nseg - 1) {
      if (a.dstate_out) load_row<NS>(a.dstate_out + (w.i * a.c + ch) * s, k0, s, aG);
    } else {
      load_row<NS>(p.carry + ((w.i * nseg + nseg - 1) * a.c + ch) * s, k0, s, aG);
      for (int64_t j = nseg - 2; j > w.seg; --j) {
        float2 own[P];
        load_row<NS>(p.carry + ((w.i * nseg + j) * a.c + ch) * s, k0, s, own);
        const float sum = p.decay[(w.i * nseg + j) * a.c + ch];
#pragma unroll
        for (int m = 0; m < P; ++m) aG[m] = __ffma2_rn(exp2_pair(__fmul2_rn(A2[m], both(sum))), aG[m], own[m]);
      }
    }
    turn_pairs<NS>(A2, turn);
    turn_pairs<NS>(aG, turn);
  }
  // A thread's pairs of channels are the same in every row.
  const int pair_row = threadIdx.x / (CH / 2), pair_col = threadIdx.x % (CH / 2) * 2;
  constexpr int kPairRows = kScanThreads / (CH / 2);
  const int room = w.channels - pair_col;
  float2 bias = make_float2(0.f, 0.f), D = bias;
  if (room > 0) {
    if (a.dt_bias) bias.x = a.dt_bias[w.c0 + pair_col];
    if (a.D) D.x = a.D[w.c0 + pair_col];
  }
  if (room > 1) {
    if (a.dt_bias) bias.y = a.dt_bias[w.c0 + pair_col + 1];
    if (a.D) D.y = a.D[w.c0 + pair_col + 1];
  }
  float2 sum_dD = make_float2(0.f, 0.f), sum_bias = sum_dD;
  int buf = 0;
  for (int64_t tile = tiles - 1; tile >= 0; --tile, buf ^= 1) {
    const int64_t tb = w.t0 + tile * TT;
    cp_async_wait<0>();
    __syncthreads();  // the tile has landed
    const uint8_t* raw = smem + buf * Tile::kStage;
    const T* rx = reinterpret_cast<const T*>(raw) + pair_col;
    const int used = tend - tb < TT ? (int)(tend - tb) : TT;
    auto convert = [&](auto softplus_too, auto whole) {
#pragma unroll
      for (int k = 0; k < Tile::PAIRS; ++k) {
        const int row = pair_row + k * kPairRows;
        const T* at = rx + row * CH;
        float2 d = __fadd2_rn(load_pair(at + TT * CH), bias);
        if constexpr (decltype(softplus_too)::value) d = make_float2(softplus(d.x), softplus(d.y));
        if constexpr (!decltype(whole)::value) {
          if (row >= used) d = make_float2(0.f, 0.f);  // x, dy, B and C are 0 there
        }
        float2 dy = load_pair(at + 3 * TT * CH);
        if (gate) {
          const float2 z = load_pair(at + 2 * TT * CH);
          dy = __fmul2_rn(dy, __fmul2_rn(z, sigmoid_pair(z)));
        }
        const float2 u = __fmul2_rn(d, load_pair(at));
        *reinterpret_cast<float4*>(sdd + row * DP + pair_col) = make_float4(d.x, u.x, d.y, u.y);
        *reinterpret_cast<float2*>(sdy + row * DP + pair_col) = dy;
      }
    };
    if (used < TT) {
      if (a.softplus) convert(std::true_type(), std::false_type());
      else convert(std::false_type(), std::false_type());
    } else {
      if (a.softplus) convert(std::true_type(), std::true_type());
      else convert(std::false_type(), std::true_type());
    }
    convert_bc<T, TT, SP>(sB, raw + 4 * Tile::kTok, p);
    convert_bc<T, TT, SP>(sC, raw + 4 * Tile::kTok + Tile::kBc, p);
    __syncthreads();
    if (tile > 0) stage(tb - TT, buf ^ 1);

#pragma unroll 1
    for (int sub = (used - 1) / CK * CK; sub >= 0; sub -= CK) {
      const int64_t ts = tb + sub;
      float2 h[CK + 1][P];  // the states before the block's tokens and after the last
#pragma unroll
      for (int m = 0; m < P; ++m) h[0][m] = make_float2(0.f, 0.f);
      if (live) {
        const float* kept = a.checkpoints + ((w.i * p.checkpoints + ts / CK) * a.c + ch) * s;
        load_row<NS>(kept, k0, s, h[0]);
        // The block before this one comes next: its states are on their way meanwhile.
        if (ts > w.t0 && k0 < s) asm volatile("prefetch.global.L1 [%0];" ::"l"(kept - a.c * s + k0));
      }
      turn_pairs<NS>(h[0], turn);
#pragma unroll
      for (int i = 0; i < CK; ++i) {
        const float2 dd = sdd[(sub + i) * DP + lane_ch];
        float2 b[P];
        load_turned<NS>(sB + (sub + i) * SP + k0, turn, b);
#pragma unroll
        for (int m = 0; m < P; ++m)
          h[i + 1][m] = __ffma2_rn(decay_pair(both(dd.x), A2[m]), h[i][m], __fmul2_rn(both(dd.y), b[m]));
      }
      float2 dAs[P];
#pragma unroll
      for (int m = 0; m < P; ++m) dAs[m] = make_float2(0.f, 0.f);
#pragma unroll
      for (int g = CK - LN; g >= 0; g -= LN) {
        float yv[LN], gb[LN], qa[LN];
#pragma unroll
        for (int i = LN - 2; i >= 0; i -= 2) {  // two tokens: i + 1, then i
          float2 db[2][P], dc[2][P];
#pragma unroll
          for (int o = 1; o >= 0; --o) {
            const int t = sub + g + i + o;
            const float2 dd = sdd[t * DP + lane_ch];
            const float dy = sdy[t * DP + lane_ch];
            float2 b[P], c[P];
            load_turned<NS>(sB + t * SP + k0, turn, b);
            load_turned<NS>(sC + t * SP + k0, turn, c);
            float2 y2 = make_float2(0.f, 0.f), gb2 = y2, qa2 = y2;
#pragma unroll
            for (int m = 0; m < P; ++m) {
              const float2 ht = h[g + i + o + 1][m];
              const float2 G = __ffma2_rn(c[m], both(dy), aG[m]);
              aG[m] = __fmul2_rn(decay_pair(both(dd.x), A2[m]), G);
              const float2 Gp = __fmul2_rn(aG[m], h[g + i + o][m]);
              db[o][m] = __fmul2_rn(G, both(dd.y));
              dc[o][m] = __fmul2_rn(ht, both(dy));
              y2 = m == 0 ? __fmul2_rn(c[m], ht) : __ffma2_rn(c[m], ht, y2);
              gb2 = m == 0 ? __fmul2_rn(G, b[m]) : __ffma2_rn(G, b[m], gb2);
              qa2 = m == 0 ? __fmul2_rn(Gp, A2[m]) : __ffma2_rn(Gp, A2[m], qa2);
              dAs[m] = __ffma2_rn(Gp, both(dd.x), dAs[m]);
            }
            yv[i + o] = y2.x + y2.y;
            gb[i + o] = gb2.x + gb2.y;
            qa[i + o] = qa2.x + qa2.y;
          }
          // Over the warp's channels, a token at a time.
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            constexpr int kLanes = NS == 4 ? CL / 2 : CL;  // after the exchange of pairs
            if constexpr (NS == 4) {
              db[o][0] = __fadd2_rn(db[o][0], from_lane(db[o][1], CL / 2));
              dc[o][0] = __fadd2_rn(dc[o][0], from_lane(dc[o][1], CL / 2));
            }
            float v[4] = {db[o][0].x, db[o][0].y, dc[o][0].x, dc[o][0].y};
            int base;
            bool first;
            sum_over_channels<4, kLanes>(v, lane, base, first);
            constexpr int kLeft = 4 > kLanes ? 4 / kLanes : 1;
            if (first) {
              float* to = sred + (warp * CK + g + i + o) * 2 * SP + k0 + turn;
#pragma unroll
              for (int k = 0; k < kLeft; ++k) to[(base + k) / 2 * SP + (base + k) % 2] = v[k];
            }
          }
        }
        const int t = sub + g + q;
        const float y_sum = sum_over_groups<LN>(yv, q), gb_sum = sum_over_groups<LN>(gb, q),
                    qa_sum = sum_over_groups<LN>(qa, q);
        __syncwarp();  // all groups have read delta x, whose place G . B takes
        sY[t * YP + lane_ch] = y_sum;
        sdd[t * DP + lane_ch].y = gb_sum;
        sQA[t * YP + lane_ch] = qa_sum;
      }
#pragma unroll
      for (int m = 0; m < P; ++m) dA[m] = __fadd2_rn(dA[m], dAs[m]);
      __syncthreads();
      // The CTA's dB and dC of these 16 tokens; 0 past the length, where states
      // or gradients that are not finite have made NaN of their products with 0.
      float* slab = p.dbc + ((w.block * a.n + w.i) * a.l + ts) * 2 * s;
      const int tokens = w.t1 - ts < CK ? (int)(w.t1 - ts) : CK;
      const int valid = used - sub;
      if (s == SP) {
        for (int u = threadIdx.x * 4; u < tokens * 2 * SP; u += kScanThreads * 4) {
          float4 v = *reinterpret_cast<const float4*>(sred + u);
#pragma unroll
          for (int r = 1; r < 4; ++r) {
            const float4 o = *reinterpret_cast<const float4*>(sred + r * CK * 2 * SP + u);
            v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
          }
          if (u / (2 * SP) >= valid) v = make_float4(0.f, 0.f, 0.f, 0.f);
          *reinterpret_cast<float4*>(slab + u) = v;
        }
      } else {
        for (int u = threadIdx.x; u < tokens * 2 * SP; u += kScanThreads) {
          const int i = u / SP, k = u % SP;  // i: token and kind
          if (k < s) {
            float v = sred[u];
#pragma unroll
            for (int r = 1; r < 4; ++r) v += sred[r * CK * 2 * SP + u];
            slab[i * s + k] = i / 2 < valid ? v : 0.f;
          }
        }
      }
      __syncthreads();
    }
    // dx, ddt and dz of the tile.
    const int64_t t = tb + pair_row;
    T* dx = static_cast<T*>(a.dx.data) + w.i * a.dx.stride_n + t * a.dx.stride_l + w.c0 + pair_col;
    T* ddt = static_cast<T*>(a.ddt.data) + w.i * a.ddt.stride_n + t * a.ddt.stride_l + w.c0 + pair_col;
    T* dz = gate ? static_cast<T*>(a.dz.data) + w.i * a.dz.stride_n + t * a.dz.stride_l + w.c0 + pair_col : nullptr;
    const int rows = w.t1 - tb < TT ? (int)(w.t1 - tb) : TT;
    if (room > 0) {
#pragma unroll
      for (int k = 0; k < Tile::PAIRS; ++k) {
        const int row = pair_row + k * kPairRows;
        if (row >= rows) break;
        float2 ox[1], od[1], oz[1];
        ox[0] = od[0] = oz[0] = make_float2(0.f, 0.f);
        if (row < used) {
          const T* at = rx + row * CH;
          const float4 dd = *reinterpret_cast<const float4*>(sdd + row * DP + pair_col);
          const float2 delta = make_float2(dd.x, dd.z), gb = make_float2(dd.y, dd.w), x = load_pair(at);
          const float2 dy = *reinterpret_cast<const float2*>(sdy + row * DP + pair_col);
          const float2 qa = *reinterpret_cast<const float2*>(sQA + row * YP + pair_col);
          ox[0] = __ffma2_rn(delta, gb, __fmul2_rn(D, dy));
          od[0] = __ffma2_rn(x, gb, __fmul2_rn(qa, both(1.f / kLog2e)));  // A2 carries log2 e
          if (a.softplus) {
            const float2 v = __fadd2_rn(load_pair(at + TT * CH), bias);
            od[0] = __fmul2_rn(od[0], make_float2(softplus_grad(v.x), softplus_grad(v.y)));
          }
          sum_dD = __ffma2_rn(dy, x, sum_dD);
          sum_bias = __fadd2_rn(sum_bias, od[0]);
          if (gate) {
            const float2 z = load_pair(at + 2 * TT * CH), sig = sigmoid_pair(z);
            const float2 y = __ffma2_rn(D, x, *reinterpret_cast<const float2*>(sY + row * YP + pair_col));
            const float2 grad =
                __fmul2_rn(sig, __ffma2_rn(z, __ffma2_rn(sig, both(-1.f), both(1.f)), both(1.f)));  // silu'(z)
            oz[0] = __fmul2_rn(__fmul2_rn(load_pair(at + 3 * TT * CH), y), grad);
          }
        }
        store_tokens<T, 2>(dx, pack<T, 2>(ox), room, p.vec);
        store_tokens<T, 2>(ddt, pack<T, 2>(od), room, p.vec);
        if (gate) store_tokens<T, 2>(dz, pack<T, 2>(oz), room, p.vec);
        dx += kPairRows * a.dx.stride_l;
        ddt += kPairRows * a.ddt.stride_l;
        dz += kPairRows * a.dz.stride_l;
      }
    }
  }

  // Tiles past the length, and the dB and dC of blocks past it.
  for (int64_t t = w.t0 + tiles * TT + pair_row; t < w.t1 && room > 0; t += kPairRows) {
    auto clear = [&](const seq_tensor& v) {
      store_tokens<T, 2>(static_cast<T*>(v.data) + w.i * v.stride_n + t * v.stride_l + w.c0 + pair_col,
                         zero_pack<T, 2>(), room, p.vec);
    };
    clear(a.dx);
    clear(a.ddt);
    if (gate) clear(a.dz);
  }
  const int64_t done = tend > w.t0 ? w.t0 + (tend - w.t0 + CK - 1) / CK * CK : w.t0;
  float* slab = p.dbc + ((w.block * a.n + w.i) * a.l + done) * 2 * s;
  for (int64_t u = threadIdx.x; u < (w.t1 - done) * 2 * s; u += kScanThreads) slab[u] = 0.f;
  if (live) {
    turn_pairs<NS>(aG, turn);
    turn_pairs<NS>(dA, turn);
    store_row<NS>(p.sums + (w.i * nseg + w.seg) * a.c * (s + 2) + ch * s, k0, s, dA);
    if (a.dstate && w.seg == 0) store_row<NS>(a.dstate + (w.i * a.c + ch) * s, k0, s, aG);
  }
  // The partial sums of a pair of channels, in order.
  __syncthreads();
  float2* parts = reinterpret_cast<float2*>(sred);  // [kPairRows][2][CH / 2]
  parts[(pair_row * 2 + 0) * (CH / 2) + pair_col / 2] = sum_dD;
  parts[(pair_row * 2 + 1) * (CH / 2) + pair_col / 2] = sum_bias;
  __syncthreads();
  for (int u = threadIdx.x; u < 2 * CH; u += kScanThreads) {
    const int which = u / CH, c = u % CH;
    if (c >= w.channels) continue;
    const float* f = reinterpret_cast<const float*>(sred) + which * CH + c;
    float v = f[0];
#pragma unroll
    for (int r = 1; r < kPairRows; ++r) v += f[r * 2 * CH];
    p.sums[((w.i * nseg + w.seg) * (s + 2) + s + which) * a.c + w.c0 + c] = v;
  }
}

// The first launch of a segmented pass: G from a zero end, over the tokens of
// every segment but the first. Nothing is summed over channels here, so it runs
// as the forward pass does: each lane converts its own channel's tokens in
// registers, one barrier a tile. plan.carry_lanes gives the lanes of a channel.
template <typename T, int NS_, int LN_>
struct CarryTile {
  static constexpr int NS = NS_, LN = LN_, SP = NS * LN, CH = kScanThreads / LN;
  static constexpr int TT = 16, G = LN < 8 ? 8 : LN;
  static constexpr int E = 16 / (int)sizeof(T);
  static constexpr int kTok = TT * CH * (int)sizeof(T), kBc = TT * SP * (int)sizeof(T);
  static constexpr int kStage = 3 * kTok + kBc, kC = 3 * kStage;  // [2][TT][SP] fp32
  static constexpr int kBytes = kC + 2 * TT * SP * 4;
};
template <typename T, int NS, int LN>
__global__ void __launch_bounds__(kScanThreads, 4) scan_bwd_carry_kernel(const __grid_constant__ ScanParams p) {
  using Tile = CarryTile<T, NS, LN>;
  constexpr int TT = Tile::TT, CH = Tile::CH, SP = Tile::SP, E = Tile::E, G = Tile::G, P = NS / 2;
  extern __shared__ __align__(128) uint8_t smem[];
  float* sC = reinterpret_cast<float*>(smem + Tile::kC);

  signal_dependents();
  const seq_scan_args& a = p.a;
  const ScanPlace w = scan_place<CH>(p, blockIdx.y + 1);
  const int lane_ch = threadIdx.x / LN, q = threadIdx.x % LN, k0 = q * NS;
  const bool live = lane_ch < w.channels, gate = a.z.data != nullptr;
  const int64_t ch = w.c0 + lane_ch, nseg = p.p.segments;
  const int s = (int)a.s;
  const int64_t tend = w.t1 < w.len ? w.t1 : w.len;
  const int64_t tiles = tend > w.t0 ? (tend - w.t0 + TT - 1) / TT : 0;

  auto stage = [&](int64_t tile, int buf) {
    if (tile >= 0) {
      const int64_t tb = w.t0 + tile * TT;
      uint8_t* to = smem + buf * Tile::kStage;
      stage_tokens<T, TT, CH, E>(to, a.dt, w, tb, tend, p.vec);
      stage_tokens<T, TT, CH, E>(to + Tile::kTok, a.dy, w, tb, tend, p.vec);
      if (gate) stage_tokens<T, TT, CH, E>(to + 2 * Tile::kTok, a.z, w, tb, tend, p.vec);
      stage_bc<T, TT, SP>(to + 3 * Tile::kTok, a.cc, p, w, tb, tend);
    }
    cp_async_commit();
  };
  auto convert = [&](int64_t tile, int buf) {
    if (tile >= 0) convert_bc<T, TT, SP>(sC + (int)(tile & 1) * TT * SP, smem + buf * Tile::kStage + 3 * Tile::kTok, p);
  };
  stage(tiles - 1, 0);
  stage(tiles - 2, 1);
  clear_padding<2 * TT, SP>(sC, s);

  float2 A2[P], aG[P];  // aG: exp(delta A)[t+1] G[t+1]
#pragma unroll
  for (int j = 0; j < P; ++j) A2[j] = aG[j] = make_float2(0.f, 0.f);
  float bias = 0.f, sum = 0.f;
  if (live) {
    load_row<NS>(a.A + ch * s, k0, s, A2);
#pragma unroll
    for (int j = 0; j < P; ++j) A2[j] = __fmul2_rn(A2[j], both(kLog2e));
    if (w.seg == nseg - 1 && a.dstate_out) load_row<NS>(a.dstate_out + (w.i * a.c + ch) * s, k0, s, aG);
    if (a.dt_bias) bias = a.dt_bias[ch];
  }
  cp_async_wait<1>();
  convert(tiles - 1, 0);
  int buf = 0;
  for (int64_t tile = tiles - 1; tile >= 0; --tile, buf = buf == 2 ? 0 : buf + 1) {
    cp_async_wait<0>();
    __syncthreads();  // as in the forward pass
    stage(tile - 2, buf == 0 ? 2 : buf - 1);
    convert(tile - 1, buf == 2 ? 0 : buf + 1);

    const int64_t tb = w.t0 + tile * TT;
    const int used = tend - tb < TT ? (int)(tend - tb) : TT;
    const T* at = reinterpret_cast<const T*>(smem + buf * Tile::kStage) + q * CH + lane_ch;
    const float* cat = sC + (int)(tile & 1) * TT * SP + k0;
    auto step = [&](int g, auto whole) {
      constexpr int M = G / LN;
      float d[M], dy[M];
#pragma unroll
      for (int k = 0; k < M; ++k) {
        d[k] = to_f32(at[(g + k * LN) * CH]) + bias;
        dy[k] = to_f32(at[(TT + g + k * LN) * CH]);
      }
      if (a.softplus) {
#pragma unroll
        for (int k = 0; k < M; ++k) d[k] = softplus(d[k]);
      }
      if (gate) {
#pragma unroll
        for (int k = 0; k < M; ++k) {
          const float z = to_f32(at[(2 * TT + g + k * LN) * CH]);
          dy[k] *= z * sigmoid(z);
        }
      }
      if constexpr (!decltype(whole)::value) {
#pragma unroll
        for (int k = 0; k < M; ++k)
          if (g + k * LN + q >= used) d[k] = 0.f;  // dy and C are 0 there
      }
#pragma unroll
      for (int i = G - 1; i >= 0; --i) {
        float delta = d[i / LN], in = dy[i / LN];
        if constexpr (LN > 1) {
          delta = __shfl_sync(0xffffffffu, delta, i % LN, LN);
          in = __shfl_sync(0xffffffffu, in, i % LN, LN);
        }
        float2 c[P];
        load_states<NS>(cat + (g + i) * SP, c);
#pragma unroll
        for (int m = 0; m < P; ++m)
          aG[m] = __fmul2_rn(decay_pair(both(delta), A2[m]), __ffma2_rn(c[m], both(in), aG[m]));
        sum += delta;
      }
    };
    int g = used / G * G;
    if (g < used) step(g, std::false_type());
#pragma unroll 1
    for (g -= G; g >= 0; g -= G) step(g, std::true_type());
  }
  if (!live) return;
  store_row<NS>(p.carry + ((w.i * nseg + w.seg) * a.c + ch) * s, k0, s, aG);
  if (q == 0) p.decay[(w.i * nseg + w.seg) * a.c + ch] = sum;
}
template <typename T, int NS, int LN>
cudaError_t launch_carry(ScanParams p, cudaStream_t st) {
  using Tile = CarryTile<T, NS, LN>;
  constexpr auto kernel = scan_bwd_carry_kernel<T, NS, LN>;
  const cudaError_t err = allow_smem<kernel>(Tile::kBytes);
  if (err != cudaSuccess) return err;
  const int64_t segments = p.p.segments;
  p.p.blocks_per_group = (p.a.c / p.a.g + Tile::CH - 1) / Tile::CH;
  p.p.blocks = p.a.g * p.p.blocks_per_group;
  p.vec = scan_vec<T>(p.a, Tile::E, true);
  kernel<<<dim3((unsigned)(p.a.n * p.p.blocks), (unsigned)(segments - 1)), kScanThreads, Tile::kBytes, st>>>(p);
  return cudaGetLastError();
}
// What is left: dB and dC, the channel blocks of a group in order, rounded
// once, and the parameters' sums. A CTA of the first fold_ctas takes 64 units of
// U consecutive elements of one group ([i][t][kind][s]), by kChains chains of
// channel blocks; the other CTAs sum slabs.
constexpr int kChains = 4;
template <typename T, int U>
__global__ void __launch_bounds__(64 * kChains) scan_finish_kernel(const __grid_constant__ ScanParams p,
                                                                   const __grid_constant__ SlabSum q, int64_t fold_ctas) {
  __shared__ __align__(16) float part[kChains * 64 * U > 8 * 33 ? kChains * 64 * U : 8 * 33];
  wait_for_primary();
  if (blockIdx.x >= fold_ctas) {
    sum_slabs<64 * kChains / 32>(q, blockIdx.x - fold_ctas, reinterpret_cast<float(*)[33]>(part));
    return;
  }
  const seq_scan_args& a = p.a;
  const int x = threadIdx.x % 64, y = threadIdx.x / 64;
  const int64_t per_block = a.n * a.l * 2 * a.s, units = per_block / U;  // U divides s
  const int64_t ctas = (units + 63) / 64, grp = blockIdx.x / ctas, e = (blockIdx.x % ctas * 64 + x) * U;
  Pack<float, U> v = zero_pack<float, U>();
  if (e < per_block) {
    const float* from = p.dbc + grp * p.p.blocks_per_group * per_block + e;
    constexpr int kAhead = 8;
    for (int64_t b = y; b < p.p.blocks_per_group; b += kAhead * kChains) {
      Pack<float, U> o[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        o[k] = b + k * kChains < p.p.blocks_per_group ? load_pack_once<U>(from + (b + k * kChains) * per_block)
                                                      : zero_pack<float, U>();
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u) v.v[u] += o[k].v[u];
    }
  }
  store_pack(part + threadIdx.x * U, v);
  __syncthreads();
  if (y != 0 || e >= per_block) return;
#pragma unroll
  for (int r = 1; r < kChains; ++r)
#pragma unroll
    for (int u = 0; u < U; ++u) v.v[u] += part[(r * 64 + x) * U + u];
  const int64_t row = e / a.s, k = e % a.s, t = row / 2 % a.l, i = row / 2 / a.l;
  const seq_tensor& o = row % 2 == 0 ? a.db : a.dc;
  T* to = static_cast<T*>(o.data) + i * o.stride_n + t * o.stride_l + grp * a.s + k;
#pragma unroll
  for (int u = 0; u < U; ++u) store_out(to + u, v.v[u]);
}

template <typename T, int NS, int LN>
cudaError_t launch_as(const seq_scan_args& a, const ScanPlan& plan, cudaStream_t st) {
  using Tile = BwdTile<T, NS, LN>;
  ScanParams p = scan_params(a, plan, true);
  p.vec = scan_vec<T>(a, Tile::E, true);
  p.vec_bc = scan_vec_bc<T>(a);
  constexpr int kSmem = Tile::kBytes;
  constexpr auto main_kernel = scan_bwd_kernel<T, NS, LN>;
  cudaError_t err = allow_smem<main_kernel>(kSmem);
  if (err != cudaSuccess) return err;
  const unsigned ctas = (unsigned)(a.n * plan.blocks);  // > 0: the caller takes n = 0 apart
  if (plan.segments > 1) {
    err = plan.carry_lanes == LN ? launch_carry<T, NS, LN>(p, st) : launch_carry<T, 2 * NS, LN / 2>(p, st);
    if (err != cudaSuccess) return err;
    err = launch_dependent(main_kernel, dim3(ctas, (unsigned)plan.segments), kScanThreads, kSmem, st, p);
  } else {
    main_kernel<<<ctas, kScanThreads, kSmem, st>>>(p);
    err = cudaGetLastError();
  }
  if (err != cudaSuccess) return err;
  const SlabSum q = slab_sum(p.sums, a.n * plan.segments, slab_out(a.dA, a.c * a.s), slab_out(a.dD, a.c),
                             slab_out(a.ddt_bias, a.c));
  const int64_t unit = a.s % 4 == 0 ? 4 : 1, fold_ctas = a.g * ((a.n * a.l * 2 * a.s / unit + 63) / 64);
  const unsigned grid = (unsigned)(fold_ctas + q.blocks());
  if (unit == 4) return launch_dependent(scan_finish_kernel<T, 4>, grid, 64 * kChains, 0, st, p, q, fold_ctas);
  return launch_dependent(scan_finish_kernel<T, 1>, grid, 64 * kChains, 0, st, p, q, fold_ctas);
}

template <typename T>
cudaError_t launch_typed(const seq_scan_args& a, const ScanPlan& p, cudaStream_t st) {
  if (p.per_lane == 2) return launch_as<T, 2, 4>(a, p, st);
  if (p.lanes == 4) return launch_as<T, 4, 4>(a, p, st);
  if (p.lanes == 8) return launch_as<T, 4, 8>(a, p, st);
  return launch_as<T, 4, 16>(a, p, st);
}

}  // namespace

cudaError_t launch_seq_scan_bwd(const seq_scan_args& a, const ScanPlan& p, cudaStream_t st) {
  if (a.dtype == CONV_F32) return launch_typed<float>(a, p, st);
  if (a.dtype == CONV_BF16) return launch_typed<__nv_bfloat16>(a, p, st);
  return launch_typed<__half>(a, p, st);
}

}  // namespace cig
