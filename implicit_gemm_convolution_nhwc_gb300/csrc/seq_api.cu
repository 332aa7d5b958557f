// C ABI of the sequence operators (conv_seq.h): argument checks, plans and
// workspaces. Everything is checked here before the first launch; the
// kernels' launchers take valid arguments.
#include <cmath>

#include "conv_internal.h"
#include "seq_internal.h"

namespace cig {
namespace {

constexpr int64_t kMaxChannels = 1 << 20;
constexpr int64_t kMaxElems = (int64_t)1 << 48;   // of any one tensor: byte offsets stay far inside int64
constexpr int64_t kMaxBlocks = 0x7fffffff;        // CTAs along a grid's x

bool dtype_ok(int32_t d) { return d == CONV_F32 || d == CONV_BF16 || d == CONV_F16; }
int64_t elem_size(int32_t d) { return d == CONV_F32 ? 4 : 2; }

// a * b * c <= limit for non-negative factors, without overflow.
bool product_fits(int64_t a, int64_t b, int64_t c, int64_t limit) {
  if (a == 0 || b == 0 || c == 0) return true;
  return a <= limit && b <= limit / a && c <= limit / a / b;
}

uint64_t round256(uint64_t v) { return (v + 255) / 256 * 256; }

// A view of [n][l][width] tokens. The stride along a single sequence or token is
// not used.
conv_status check_view(seq_tensor t, int64_t n, int64_t l, int64_t width, int64_t size, bool output) {
  if (n == 0 || l == 0) return CONV_OK;
  if (!t.data) return CONV_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(t.data) % size != 0) return CONV_ERR_ALIGNMENT;
  if (n == 1) t.stride_n = 0;
  if (l == 1) t.stride_l = 0;
  if (t.stride_n < 0 || t.stride_l < 0) return CONV_ERR_INVALID_ARG;
  if (t.stride_n > kMaxElems || t.stride_l > kMaxElems) return CONV_ERR_OVERFLOW;
  if (!product_fits(n - 1, t.stride_n, 1, kMaxElems) || !product_fits(l - 1, t.stride_l, 1, kMaxElems))
    return CONV_ERR_OVERFLOW;
  if (output) {
    const int64_t over_l = (l - 1) * t.stride_l + width, over_n = (n - 1) * t.stride_n + width;
    const bool n_outer = (l == 1 || t.stride_l >= width) && (n == 1 || t.stride_n >= over_l);
    const bool l_outer = (n == 1 || t.stride_n >= width) && (l == 1 || t.stride_l >= over_n);
    if (!n_outer && !l_outer) return CONV_ERR_INVALID_ARG;
  }
  return CONV_OK;
}
conv_status check_dense(const void* p, int64_t size, bool required) {
  if (!p) return required ? CONV_ERR_INVALID_ARG : CONV_OK;
  return reinterpret_cast<uintptr_t>(p) % size == 0 ? CONV_OK : CONV_ERR_ALIGNMENT;
}

#define CIG_TRY(expr)                     \
  do {                                    \
    const conv_status st_ = (expr);       \
    if (st_ != CONV_OK) return st_;       \
  } while (0)

conv_status check_workspace(const void* ws, uint64_t given, uint64_t need) {
  if (need == 0) return CONV_OK;
  if (given < need) return CONV_ERR_WORKSPACE_TOO_SMALL;
  if (!ws) return CONV_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(ws) % 16 == 0 ? CONV_OK : CONV_ERR_ALIGNMENT;
}

// ---------------------------------------------------------------- convolution

conv_status check_conv_sizes(int64_t n, int64_t l, int64_t c, int64_t width) {
  if (n < 0 || l < 0 || c < 1 || width < 1) return CONV_ERR_INVALID_ARG;
  if (width > 4 || c > kMaxChannels) return CONV_ERR_UNSUPPORTED;
  if (!product_fits(n, l + 4, c, kMaxElems)) return CONV_ERR_OVERFLOW;
  // The element-by-element kernels run c threads a strip of at least 8 tokens.
  if (!product_fits(n, l / 8 + 1, (c + 127) / 128, kMaxBlocks)) return CONV_ERR_UNSUPPORTED;
  return CONV_OK;
}

uint64_t conv_ws_bytes(int64_t n, int64_t l, int64_t c, int64_t width) {
  return round256((uint64_t)conv_bwd_plan(n, l, c).slabs * (uint64_t)((width + 1) * c) * 4);
}

conv_status check_conv(const seq_conv_args* a) {
  if (!a) return CONV_ERR_INVALID_ARG;
  CIG_TRY(check_conv_sizes(a->n, a->l, a->c, a->width));
  if (!dtype_ok(a->dtype) || (a->w_dtype != a->dtype && a->w_dtype != CONV_F32)) return CONV_ERR_INVALID_ARG;
  if ((a->silu != 0 && a->silu != 1) || a->reserved != 0) return CONV_ERR_INVALID_ARG;
  const int64_t e = elem_size(a->dtype), we = elem_size(a->w_dtype);
  CIG_TRY(check_view(a->x, a->n, a->l, a->c, e, false));
  CIG_TRY(check_dense(a->w, we, true));
  CIG_TRY(check_dense(a->bias, we, false));
  CIG_TRY(check_dense(a->state, e, false));
  CIG_TRY(check_dense(a->state_out, e, false));
  CIG_TRY(check_dense(a->lengths, 4, false));
  return CONV_OK;
}

// ---------------------------------------------------------------- scan

conv_status check_scan_sizes(int64_t n, int64_t l, int64_t c, int64_t s, int64_t g) {
  if (n < 0 || l < 0 || c < 1 || s < 1 || g < 1 || c % g != 0) return CONV_ERR_INVALID_ARG;
  if (s > 64 || c > kMaxChannels) return CONV_ERR_UNSUPPORTED;
  if (!product_fits(n, l + 16, c * s, kMaxElems)) return CONV_ERR_OVERFLOW;
  if (!product_fits(n, c, 1, kMaxBlocks)) return CONV_ERR_UNSUPPORTED;
  return CONV_OK;
}
// The backward pass's last launch: 64 or 256 elements of dB and dC a CTA, and
// 32 of the parameters' gradients.
conv_status check_scan_bwd_sizes(int64_t n, int64_t l, int64_t c, int64_t s, int64_t g) {
  CIG_TRY(check_scan_sizes(n, l, c, s, g));
  return product_fits(n, l, g * s, kMaxBlocks / 2 * 32) ? CONV_OK : CONV_ERR_UNSUPPORTED;
}

conv_status check_scan(const seq_scan_args* a) {
  if (!a) return CONV_ERR_INVALID_ARG;
  CIG_TRY(check_scan_sizes(a->n, a->l, a->c, a->s, a->g));
  if (!dtype_ok(a->dtype) || (a->softplus != 0 && a->softplus != 1)) return CONV_ERR_INVALID_ARG;
  const int64_t e = elem_size(a->dtype);
  CIG_TRY(check_view(a->x, a->n, a->l, a->c, e, false));
  CIG_TRY(check_view(a->dt, a->n, a->l, a->c, e, false));
  if (a->z.data) CIG_TRY(check_view(a->z, a->n, a->l, a->c, e, false));
  CIG_TRY(check_view(a->b, a->n, a->l, a->g * a->s, e, false));
  CIG_TRY(check_view(a->cc, a->n, a->l, a->g * a->s, e, false));
  CIG_TRY(check_dense(a->A, 4, true));
  CIG_TRY(check_dense(a->D, 4, false));
  CIG_TRY(check_dense(a->dt_bias, 4, false));
  CIG_TRY(check_dense(a->lengths, 4, false));
  // Rows of states move by 16 bytes where s is a multiple of 4.
  const int64_t se = a->s % 4 == 0 ? 16 : 4;
  CIG_TRY(check_dense(a->state, se, false));
  CIG_TRY(check_dense(a->state_out, se, false));
  CIG_TRY(check_dense(a->checkpoints, 16, false));
  return CONV_OK;
}

// ---------------------------------------------------------------- norm

conv_status check_rows(const seq_tensor& v, int64_t n, int64_t c, int64_t size, bool required, bool output) {
  const void* p = v.data;
  const int64_t stride = v.stride_n;
  if (!p) return required && n > 0 ? CONV_ERR_INVALID_ARG : CONV_OK;
  if (reinterpret_cast<uintptr_t>(p) % size != 0) return CONV_ERR_ALIGNMENT;
  if (stride < 0 || (output && n > 1 && stride < c)) return CONV_ERR_INVALID_ARG;
  if (n > 1 && !product_fits(n - 1, stride, 1, kMaxElems)) return CONV_ERR_OVERFLOW;
  return CONV_OK;
}

conv_status check_norm(const seq_norm_args* a) {
  if (!a) return CONV_ERR_INVALID_ARG;
  if (a->n < 0 || a->c < 1) return CONV_ERR_INVALID_ARG;
  if (a->c > (int64_t)1 << 30 || a->n > kMaxBlocks) return CONV_ERR_UNSUPPORTED;
  if (!product_fits(a->n, a->c, 1, kMaxElems)) return CONV_ERR_OVERFLOW;
  if (!dtype_ok(a->dtype) || (a->w_dtype != a->dtype && a->w_dtype != CONV_F32)) return CONV_ERR_INVALID_ARG;
  if (!(a->eps >= 0.f) || std::isinf(a->eps) || a->reserved != 0) return CONV_ERR_INVALID_ARG;
  CIG_TRY(check_dense(a->w, elem_size(a->w_dtype), true));
  return CONV_OK;
}

}  // namespace

// ---------------------------------------------------------------- scan plan

// The forward pass holds up to 16 states in a lane; where even the most
// segments leave CTA places empty it spreads a channel's states over twice the
// lanes (a token's latency then counts: 5 prompts of 333 tokens by 1000
// channels 24.6 -> 21.6 us; on a full GPU two lanes are slower, 16384 tokens of
// 2048 channels 267 -> 291 us). The backward pass keeps 16 tokens of the
// states in registers, so it holds four in a lane.
//
// A segmented time axis costs a second reading of all tokens, so it is taken
// only where the unsegmented grid leaves over half of the GPU's CTA places
// empty, and then fills them: once (four CTAs an SM) in the forward pass (twice:
// 267 -> 293 us), twice in the backward pass, whose shorter, later CTAs even out
// the SMs' loads (4 x 2048 tokens of 2048 channels: 461 us with 512 CTAs, 411 us
// with 1024, 408 us with 1536).
//
// The backward pass's first launch takes half the lanes with twice the states
// where that still gives two CTAs an SM (the same case: 429 us without, 411 us
// with it; with a quarter of the lanes, 1.3 CTAs an SM, 20 us slower again).
ScanPlan scan_plan(int64_t n, int64_t l, int64_t c, int64_t s, int64_t g, bool backward, int sms) {
  ScanPlan p;
  const int64_t places = (int64_t)sms * (backward ? 8 : 4);
  auto blocks = [&](int lanes) { return (c / g + kScanThreads / lanes - 1) / (kScanThreads / lanes); };
  if (backward) {
    p.per_lane = s <= 8 ? 2 : 4;
    p.lanes = s <= 16 ? 4 : s <= 32 ? 8 : 16;
    p.tile = 32;
  } else {
    p.per_lane = s <= 4 ? 4 : s <= 8 ? 8 : 16;
    p.lanes = s <= 16 ? 1 : s <= 32 ? 2 : 4;
    p.tile = 16;
    const int64_t most = l / (2 * p.tile) > 1 ? l / (2 * p.tile) : 1;
    if (p.per_lane > 4 && p.lanes < 4 && n * g * blocks(p.lanes) * most < places) {
      p.per_lane /= 2;
      p.lanes *= 2;
    }
  }
  p.channels = kScanThreads / p.lanes;
  p.blocks_per_group = blocks(p.lanes);
  p.blocks = g * p.blocks_per_group;
  const int64_t ctas = n * p.blocks > 0 ? n * p.blocks : 1;
  int64_t segments = 1;
  if (2 * ctas <= places) {
    segments = places / ctas;
    const int64_t most = l / (2 * p.tile);  // at least two tiles a segment
    if (segments > most) segments = most;
    if (segments > 64) segments = 64;
    if (segments < 1) segments = 1;
  }
  p.segment = ((l + segments - 1) / segments + p.tile - 1) / p.tile * p.tile;
  if (p.segment < p.tile) p.segment = p.tile;
  p.segments = (l + p.segment - 1) / p.segment;
  if (p.segments < 1) p.segments = 1;
  p.carry_lanes = p.lanes;
  if (backward && n * g * blocks(p.lanes / 2) * (p.segments - 1) >= 2 * (int64_t)sms) p.carry_lanes /= 2;
  return p;
}

ScanWorkspace scan_workspace(const ScanPlan& p, int64_t n, int64_t l, int64_t c, int64_t s, bool backward) {
  ScanWorkspace w = {};
  uint64_t at = 0;
  auto take = [&](int64_t floats) {
    const uint64_t here = at;
    at += round256((uint64_t)floats * 4);
    return here;
  };
  const bool split = p.segments > 1;
  w.carry = take(split ? n * p.segments * c * s : 0);
  w.decay = take(split ? n * p.segments * c : 0);
  if (backward) {
    w.dbc = take(p.blocks * n * l * 2 * s);
    w.sums = take(n * p.segments * c * (s + 2));
  }
  w.bytes = at;
  return w;
}

}  // namespace cig

using namespace cig;

extern "C" {

// ---------------------------------------------------------------- convolution

conv_status seq_conv_workspace_bytes(int64_t n, int64_t l, int64_t c, int64_t width, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_INVALID_ARG;
  CIG_TRY(check_conv_sizes(n, l, c, width));
  *bytes = conv_ws_bytes(n, l, c, width);
  return CONV_OK;
}

conv_status seq_conv_fwd(const seq_conv_args* a, void* stream) {
  CIG_TRY(check_conv(a));
  CIG_TRY(check_view(a->y, a->n, a->l, a->c, elem_size(a->dtype), true));
  if (a->n == 0) return CONV_OK;
  seq_conv_args b = *a;
  b.dy = b.dx = seq_tensor{nullptr, 0, 0};
  b.dstate = nullptr;
  b.dstate_out = nullptr;
  return launch_seq_conv_fwd(b, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

conv_status seq_conv_bwd(const seq_conv_args* a, void* stream) {
  CIG_TRY(check_conv(a));
  const int64_t e = elem_size(a->dtype);
  CIG_TRY(check_view(a->dy, a->n, a->l, a->c, e, false));
  CIG_TRY(check_view(a->dx, a->n, a->l, a->c, e, true));
  CIG_TRY(check_dense(a->dstate_out, e, false));
  CIG_TRY(check_dense(a->dstate, e, false));
  CIG_TRY(check_dense(a->dw, 4, true));
  CIG_TRY(check_dense(a->db, 4, false));
  CIG_TRY(check_workspace(a->ws, a->ws_bytes, conv_ws_bytes(a->n, a->l, a->c, a->width)));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->n == 0) {
    const SlabSum zero = slab_sum(nullptr, 0, slab_out(a->dw, a->c * a->width), slab_out(a->db, a->c));
    return launch_seq_slab_sum(zero, false, st) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
  }
  seq_conv_args b = *a;
  b.y = seq_tensor{nullptr, 0, 0};
  b.state_out = nullptr;
  return launch_seq_conv_bwd(b, st) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

conv_status seq_conv_step(const seq_conv_args* a, void* stream) {
  CIG_TRY(check_conv(a));
  if (a->l != 1) return CONV_ERR_INVALID_ARG;
  CIG_TRY(check_view(a->y, a->n, 1, a->c, elem_size(a->dtype), true));
  if (a->n_slots < 0 || (!a->slots && a->n_slots < a->n)) return CONV_ERR_INVALID_ARG;
  if (!product_fits(a->n_slots, 4, a->c, kMaxElems)) return CONV_ERR_OVERFLOW;
  if (a->n == 0) return CONV_OK;
  if (!a->state_out && a->width > 1 && a->n_slots > 0) return CONV_ERR_INVALID_ARG;
  CIG_TRY(check_dense(a->slots, 4, false));
  seq_conv_args b = *a;
  b.dy = b.dx = seq_tensor{nullptr, 0, 0};
  b.state = b.dstate_out = nullptr;
  b.dstate = nullptr;
  return launch_seq_conv_step(b, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

// ---------------------------------------------------------------- scan

conv_status seq_scan_workspace_bytes_for(int64_t n, int64_t l, int64_t c, int64_t s, int64_t g, int32_t backward,
                                         int32_t sm_count, uint64_t* bytes) {
  if (!bytes || sm_count < 1) return CONV_ERR_INVALID_ARG;
  CIG_TRY(check_scan_sizes(n, l, c, s, g));
  uint64_t need = scan_workspace(scan_plan(n, l, c, s, g, false, sm_count), n, l, c, s, false).bytes;
  if (backward) {  // one workspace serves both passes
    CIG_TRY(check_scan_bwd_sizes(n, l, c, s, g));
    const uint64_t more = scan_workspace(scan_plan(n, l, c, s, g, true, sm_count), n, l, c, s, true).bytes;
    if (more > need) need = more;
  }
  *bytes = need;
  return CONV_OK;
}

conv_status seq_scan_workspace_bytes(int64_t n, int64_t l, int64_t c, int64_t s, int64_t g, int32_t backward,
                                     uint64_t* bytes) {
  const int sms = current_sm_count();
  if (sms < 1) return CONV_ERR_CUDA;
  return seq_scan_workspace_bytes_for(n, l, c, s, g, backward, sms, bytes);
}

conv_status seq_scan_checkpoint_bytes(int64_t n, int64_t l, int64_t c, int64_t s, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_INVALID_ARG;
  CIG_TRY(check_scan_sizes(n, l, c, s, 1));
  *bytes = (uint64_t)n * (uint64_t)((l + kScanCheckpoint - 1) / kScanCheckpoint) * (uint64_t)(c * s) * 4;
  return CONV_OK;
}

conv_status seq_scan_fwd(const seq_scan_args* a, void* stream) {
  CIG_TRY(check_scan(a));
  CIG_TRY(check_view(a->y, a->n, a->l, a->c, elem_size(a->dtype), true));
  if (a->n == 0) return CONV_OK;
  const int sms = current_sm_count();
  if (sms < 1) return CONV_ERR_CUDA;
  const ScanPlan p = scan_plan(a->n, a->l, a->c, a->s, a->g, false, sms);
  CIG_TRY(check_workspace(a->ws, a->ws_bytes, scan_workspace(p, a->n, a->l, a->c, a->s, false).bytes));
  return launch_seq_scan_fwd(*a, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

conv_status seq_scan_bwd(const seq_scan_args* a, void* stream) {
  CIG_TRY(check_scan(a));
  CIG_TRY(check_scan_bwd_sizes(a->n, a->l, a->c, a->s, a->g));
  const int64_t e = elem_size(a->dtype), se = a->s % 4 == 0 ? 16 : 4;
  CIG_TRY(check_view(a->dy, a->n, a->l, a->c, e, false));
  CIG_TRY(check_view(a->dx, a->n, a->l, a->c, e, true));
  CIG_TRY(check_view(a->ddt, a->n, a->l, a->c, e, true));
  if (a->z.data) CIG_TRY(check_view(a->dz, a->n, a->l, a->c, e, true));
  CIG_TRY(check_view(a->db, a->n, a->l, a->g * a->s, e, true));
  CIG_TRY(check_view(a->dc, a->n, a->l, a->g * a->s, e, true));
  CIG_TRY(check_dense(a->checkpoints, 16, a->n > 0 && a->l > 0));
  CIG_TRY(check_dense(a->dA, 4, true));
  CIG_TRY(check_dense(a->dD, 4, false));
  CIG_TRY(check_dense(a->ddt_bias, 4, false));
  CIG_TRY(check_dense(a->dstate_out, se, false));
  CIG_TRY(check_dense(a->dstate, se, false));
  if ((a->dD && !a->D) || (a->ddt_bias && !a->dt_bias) || (a->dz.data && !a->z.data)) return CONV_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->n == 0) {
    const SlabSum zero = slab_sum(nullptr, 0, slab_out(a->dA, a->c * a->s), slab_out(a->dD, a->c), slab_out(a->ddt_bias, a->c));
    return launch_seq_slab_sum(zero, false, st) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
  }
  const int sms = current_sm_count();
  if (sms < 1) return CONV_ERR_CUDA;
  const ScanPlan p = scan_plan(a->n, a->l, a->c, a->s, a->g, true, sms);
  CIG_TRY(check_workspace(a->ws, a->ws_bytes, scan_workspace(p, a->n, a->l, a->c, a->s, true).bytes));
  return launch_seq_scan_bwd(*a, p, st) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

conv_status seq_scan_step(const seq_scan_args* a, void* stream) {
  CIG_TRY(check_scan(a));
  if (a->l != 1) return CONV_ERR_INVALID_ARG;
  CIG_TRY(check_view(a->y, a->n, 1, a->c, elem_size(a->dtype), true));
  if (a->n_slots < 0 || (!a->slots && a->n_slots < a->n)) return CONV_ERR_INVALID_ARG;
  if (!product_fits(a->n_slots, a->c, a->s, kMaxElems)) return CONV_ERR_OVERFLOW;
  if (!product_fits(a->n, a->c, 16, kMaxBlocks * 64)) return CONV_ERR_UNSUPPORTED;
  if (a->n == 0) return CONV_OK;
  if (!a->state_out && a->n_slots > 0) return CONV_ERR_INVALID_ARG;
  CIG_TRY(check_dense(a->slots, 4, false));
  return launch_seq_scan_step(*a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

// ---------------------------------------------------------------- norm

conv_status seq_norm_workspace_bytes(int64_t n, int64_t c, uint64_t* bytes) {
  if (!bytes || n < 0 || c < 1) return CONV_ERR_INVALID_ARG;
  if (!product_fits(n, c, 1, kMaxElems)) return CONV_ERR_OVERFLOW;
  *bytes = round256((uint64_t)norm_bwd_slabs(n, c) * (uint64_t)c * 4);
  return CONV_OK;
}

conv_status seq_norm_fwd(const seq_norm_args* a, void* stream) {
  CIG_TRY(check_norm(a));
  const int64_t e = elem_size(a->dtype);
  if ((a->out8 != 0 && a->out8 != 1) || (a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128))
    return CONV_ERR_INVALID_ARG;
  if (!a->out8 && a->group != 0) return CONV_ERR_INVALID_ARG;
  CIG_TRY(check_rows(a->x, a->n, a->c, e, true, false));
  CIG_TRY(check_rows(a->residual, a->n, a->c, e, false, false));
  CIG_TRY(check_rows(a->y, a->n, a->c, a->out8 ? 1 : e, true, true));
  CIG_TRY(check_rows(a->r, a->n, a->c, e, false, true));
  CIG_TRY(check_dense(a->scale, 4, a->out8 && a->n > 0));
  CIG_TRY(check_dense(a->rstd, 4, false));
  if (a->n == 0) return CONV_OK;
  seq_norm_args b = *a;
  b.dy = b.dr = b.dx = seq_tensor{nullptr, 0, 0};
  return launch_seq_norm_fwd(b, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

conv_status seq_norm_bwd(const seq_norm_args* a, void* stream) {
  CIG_TRY(check_norm(a));
  const int64_t e = elem_size(a->dtype);
  CIG_TRY(check_rows(a->r, a->n, a->c, e, true, false));
  CIG_TRY(check_rows(a->dy, a->n, a->c, e, true, false));
  CIG_TRY(check_rows(a->dr, a->n, a->c, e, false, false));
  CIG_TRY(check_rows(a->dx, a->n, a->c, e, true, true));
  CIG_TRY(check_dense(a->rstd, 4, a->n > 0));
  CIG_TRY(check_dense(a->dw, 4, true));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->n == 0) {
    return launch_seq_slab_sum(slab_sum(nullptr, 0, slab_out(a->dw, a->c)), false, st) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
  }
  CIG_TRY(check_workspace(a->ws, a->ws_bytes, round256((uint64_t)norm_bwd_slabs(a->n, a->c) * (uint64_t)a->c * 4)));
  seq_norm_args b = *a;
  b.x = b.residual = b.y = seq_tensor{nullptr, 0, 0};
  return launch_seq_norm_bwd(b, st) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

}  // extern "C"
