// Norm and rotary positions of queries, keys and index vectors, and their
// gradients (msa_rope.cuh has a row's arithmetic).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "msa_rope.cuh"

namespace msa {
namespace rope {

constexpr int64_t kMaxStride = int64_t(1) << 40;

// Rows of `heads` heads of `tokens` tokens that do not overlap, in 16-byte steps.
static bool bad_strides(int64_t token, int64_t head, int64_t heads, int64_t tokens) {
  if (token < 128 || head < 128 || token > kMaxStride || head > kMaxStride || token % 8 || head % 8) return true;
  return (heads > 1 && tokens > 1) && token < (heads - 1) * head + 128 && head < (tokens - 1) * token + 128;
}

int check_problem(const msa_rope_problem* p) {
  if (!p) return MSA_ERR_INVALID_ARGUMENT;
  if (p->tokens < 0) return MSA_ERR_INVALID_ARGUMENT;
  if (p->head_dim != kHeadDim || p->tokens > cache::kMaxCount) return MSA_ERR_UNSUPPORTED_SHAPE;
  if (p->rotary_dim < 0 || p->rotary_dim > 128 || p->rotary_dim % 32) return MSA_ERR_UNSUPPORTED_SHAPE;
  if (p->num_axes < 1 || p->num_axes > 4) return MSA_ERR_UNSUPPORTED_SHAPE;
  constexpr float kMost = 1.2676506002282294e30f;  // 2^100
  if (!(p->eps >= 1.f / kMost && p->eps <= kMost) || !isfinite(p->weight_offset)) return MSA_ERR_INVALID_ARGUMENT;
  if (!(p->cos_scale > 0.f && p->cos_scale < kInf)) return MSA_ERR_INVALID_ARGUMENT;
  bool turned = false;
  for (int i = 0; i < MSA_ROPE_TENSORS; ++i) {
    const msa_rope_tensor& t = p->tensor[i];
    if (t.heads < 0 || t.flags > 15) return MSA_ERR_INVALID_ARGUMENT;
    if (t.heads > kGroup * cache::kMaxHeads) return MSA_ERR_UNSUPPORTED_SHAPE;
    if (t.heads == 0) continue;
    if (t.weight && !aligned16(t.weight)) return MSA_ERR_INVALID_ARGUMENT;
    if (bad_strides(t.x_token, t.x_head, t.heads, p->tokens) || bad_strides(t.y_token, t.y_head, t.heads, p->tokens))
      return MSA_ERR_INVALID_ARGUMENT;
    turned |= (t.flags & MSA_ROPE_ROTATE) != 0;
  }
  if (turned && p->rotary_dim == 0) return MSA_ERR_INVALID_ARGUMENT;
  if (p->rotary_dim > 0 && (!p->pairs || !aligned16(p->pairs))) return MSA_ERR_INVALID_ARGUMENT;
  return MSA_OK;
}

template <bool kAdjacent>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(RowsArgs a) {
  __shared__ Table<kTile> s_tab;
  cache::after_previous_kernel();
  if (status_bad(a.status)) return;
  rows_block<kAdjacent>(a, blockIdx.x, s_tab);
}

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------
// With g the gradient turned back, r the inverse rms and u = g w:
//   dx = r (u - x r mean(u x) r),  dw = sum over rows of g x r.
// A warp keeps its four heads and takes a slice of the tokens, so that the
// weights' gradients gather in registers; the CTA adds its warps' up at its end
// and leaves a row per weight (`slot`) and slice in the workspace, which a second
// kernel adds up in a fixed order.
struct GradArgs {
  Tensor t[kTensors];
  const uint16_t* dy[kTensors];
  uint16_t* dx[kTensors];
  int64_t y_token[kTensors], y_head[kTensors];
  int slot[kTensors];   // first row of the tensor's partial sums in a slice's; -1: none
  int first[kTensors];  // group that the tensor's first head is in
  Angles an;
  float eps, offset;
  int T, heads;
  int tile, tiles, slices, groups, units, phases, slots;
  float* partial;  // [slices][slots][128]
  int32_t* status;
};

template <bool kAdjacent>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(GradArgs a) {
  __shared__ Table<kTile> s_tab;
  __shared__ float s_dw[kThreads / 8][128];
  cache::after_previous_kernel();
  if (status_bad(a.status)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, j = lane & 7;
  const int slice = blockIdx.x / a.groups, group = blockIdx.x - slice * a.groups;
  const int phase = warp / a.units, unit = group * a.units + warp - phase * a.units;
  const int hh = unit * 4 + (lane >> 3);
  const bool live = hh < a.heads && phase < a.phases;
  int da, db, head;
  lane_dims(j, a.an.R, da, db);
  const int k = tensor_of(a, live ? hh : 0, head);
  const Tensor& t = a.t[k];
  const bool norm = t.flags & MSA_ROPE_NORM, turn = turns(t, j, a.an.R);
  float w[16], dw[16];
  load_weights(t, head, da, db, a.offset, w);
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i] = 0.f;
  for (int tile = slice; tile < a.tiles; tile += a.slices) {
    const int64_t t0 = (int64_t)tile * a.tile;
    const int n = (int)min((int64_t)a.tile, a.T - t0);
    __syncthreads();  // the tile before has been read
    fill_table<kAdjacent>(s_tab, a.an, t0, n);
    __syncthreads();
    const int64_t x0 = t0 * t.x_token + head * t.x_head, y0 = t0 * a.y_token[k] + head * a.y_head[k];
    for (int i = phase; i < n && phase < a.phases; i += a.phases) {
      const bool here = live && a.an.positions[(t0 + i) * a.an.A] >= 0;
      uint4 xa = make_uint4(0, 0, 0, 0), xb = xa, ga = xa, gb = xa;
      if (here) {
        const uint16_t* x = t.x + x0 + i * t.x_token;
        const uint16_t* dy = a.dy[k] + y0 + i * a.y_token[k];
        xa = *reinterpret_cast<const uint4*>(x + da);
        xb = *reinterpret_cast<const uint4*>(x + db);
        ga = *reinterpret_cast<const uint4*>(dy + da);
        gb = *reinterpret_cast<const uint4*>(dy + db);
      }
      float g[16], v[16];
      unpack8(ga, g);
      unpack8(gb, g + 8);
      unpack8(xa, v);
      unpack8(xb, v + 8);
      if (turn) {
        float4 cs[4];
        load_angles(s_tab.cs[i], j, cs);
        rotate<kAdjacent, true>(g, cs);
      }
      float scale;
      const float sum = row_sum(squares(v));
      const float r = inverse_rms(v, norm ? sum : 0.f, a.eps, scale);
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        v[e] *= r;  // the normed row without its weight
        if (norm) dw[e] = fmaf(g[e], v[e], dw[e]);
        g[e] *= w[e];
        dot = fmaf(g[e], v[e], dot);
      }
      const float mean = row_sum(dot) * (1.f / 128.f);
      if (norm) {
        const float rr = r * scale;
#pragma unroll
        for (int e = 0; e < 16; ++e) g[e] = rr * fmaf(-v[e], mean, g[e]);
      }
      if (here) {
        uint16_t* dx = a.dx[k] + x0 + i * t.x_token;
        *reinterpret_cast<uint4*>(dx + da) = pack8(g);
        *reinterpret_cast<uint4*>(dx + db) = pack8(g + 8);
      }
    }
  }
  // the CTA's sums: heads that share a weight in the order of the warps and rows
  float* mine = s_dw[tid >> 3];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mine[da + i] = live ? dw[i] : 0.f;
    mine[db + i] = live ? dw[8 + i] : 0.f;
  }
  __syncthreads();
  const int d = tid & 127;
  float* out = a.partial + (int64_t)slice * a.slots * 128 + d;
  for (int i = 0, before = 0; i < kTensors; ++i) {
    const int end = a.t[i].end;
    if (a.slot[i] >= 0) {
      // this CTA's heads of the tensor, and its rows (of the warps' first phase)
      const int lo = max(before, group * a.units * 4), hi = min(end, (group + 1) * a.units * 4);
      const int row0 = lo - group * a.units * 4, rows = hi - lo;
      if (a.t[i].flags & MSA_ROPE_PER_HEAD) {
        for (int r = tid >> 7; r < rows; r += 2) {
          float s = 0.f;
          for (int p = 0; p < a.phases; ++p) s += s_dw[p * a.units * 4 + row0 + r][d];
          out[(int64_t)(a.slot[i] + lo - before + r) * 128] = s;
        }
      } else if (rows > 0 && tid < 128) {
        float s = 0.f;
        for (int p = 0; p < a.phases; ++p)
          for (int r = 0; r < rows; ++r) s += s_dw[p * a.units * 4 + row0 + r][d];
        out[(int64_t)(a.slot[i] + group - a.first[i]) * 128] = s;
      }
    }
    before = end;
  }
}

struct SumArgs {
  const float* partial;
  void* dw[kTensors];
  int wide[kTensors];  // fp32
  int slot[kTensors], end[kTensors];  // first slot; rows of weights of this tensor and those before it
  int per[kTensors];   // slots that make one row of weights
  int slices, slots;
  int32_t* status;
};

// A CTA adds up one row of weights: thread (part, dim) every eighth partial row.
constexpr int kSumParts = 8;
__global__ void __launch_bounds__(128 * kSumParts) weight_sum_kernel(SumArgs a) {
  __shared__ float s_part[kSumParts][128];
  cache::after_previous_kernel();
  if (status_bad(a.status)) return;
  int k = 0, before = 0;
  while (k + 1 < kTensors && (int)blockIdx.x >= a.end[k]) before = a.end[k++];
  const int row = blockIdx.x - before, d = threadIdx.x & 127, part = threadIdx.x >> 7;
  const int per = a.per[k];
  const float* src = a.partial + (int64_t)(a.slot[k] + row * per) * 128 + d;
  float s = 0.f;
  for (int i = part; i < a.slices * per; i += kSumParts) {
    const int slice = i / per;
    s += src[((int64_t)slice * a.slots + i - slice * per) * 128];
  }
  s_part[part][d] = s;
  __syncthreads();
  if (part) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kSumParts; ++i) s += s_part[i][d];
  if (a.wide[k]) static_cast<float*>(a.dw[k])[(int64_t)row * 128 + d] = s;
  else static_cast<uint16_t*>(a.dw[k])[(int64_t)row * 128 + d] = (uint16_t)(pack_bf16x2(s, 0.f) & 0xFFFFu);
}

// How the gradients' tokens and partial sums are cut.  It depends on the problem
// alone: the workspace's size and the order of the sums do.
struct GradCut {
  Cut c;
  int heads, tile, tiles, slices, slots;
  int slot[kTensors], first[kTensors], per[kTensors];
};
constexpr int kGradCtas = 2 * 152;
static GradCut cut_grad(const msa_rope_problem* p) {
  GradCut g{};
  for (int i = 0; i < kTensors; ++i) g.heads += p->tensor[i].heads;
  if (g.heads == 0) return g;
  g.c = cut_heads(g.heads);
  g.tile = cut_tokens(p->tokens, g.c.groups, 152, kTile, 1);
  if (g.tile < g.c.phases) g.tile = g.c.phases;
  g.tiles = (p->tokens + g.tile - 1) / g.tile;
  const int want = (kGradCtas + g.c.groups - 1) / g.c.groups;
  g.slices = g.tiles < want ? g.tiles : want;
  int at = 0;
  for (int i = 0; i < kTensors; ++i) {
    const msa_rope_tensor& t = p->tensor[i];
    const int span = g.c.units * 4;  // heads of a group
    g.slot[i] = g.slots;
    g.first[i] = at / span;
    g.per[i] = 1;
    if (t.heads && (t.flags & MSA_ROPE_PER_HEAD)) g.slots += t.heads;
    else if (t.heads) g.slots += g.per[i] = (at + t.heads - 1) / span - at / span + 1;
    at += t.heads;
  }
  return g;
}

}  // namespace rope
}  // namespace msa

using namespace msa;

namespace {

// Device pointers of the tensors that are there.
template <class T>
bool bad_rows(const msa_rope_problem* p, T* const* ptrs) {
  if (!ptrs) return true;
  for (int i = 0; i < rope::kTensors; ++i)
    if (p->tensor[i].heads && (!ptrs[i] || !aligned16(ptrs[i]))) return true;
  return false;
}

template <class Args>
int set_tensors(Args& a, const msa_rope_problem* p, const uint16_t* const* x) {
  int end = 0;
  for (int i = 0; i < rope::kTensors; ++i) {
    const msa_rope_tensor& t = p->tensor[i];
    end += t.heads;
    a.t[i] = rope::Tensor{t.heads ? x[i] : nullptr, t.weight, t.x_token, t.x_head, t.flags, end};
    a.y_token[i] = t.y_token;
    a.y_head[i] = t.y_head;
  }
  return end;
}

}  // namespace

extern "C" {

int msa_rope_pairs(const double* inv_freq, const int32_t* axes, int32_t num_pairs, msa_rope_pair* pairs) {
  if (!inv_freq || !pairs || num_pairs < 0 || num_pairs > kHeadDim / 2) return MSA_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < num_pairs; ++i) {
    if (!isfinite(inv_freq[i])) return MSA_ERR_INVALID_ARGUMENT;
    const double turns = fabs(inv_freq[i]) / 6.283185307179586476925;
    const double part = ldexp(turns - floor(turns), 64);  // < 2^64: a double below 1 is at most 1 - 2^-53
    const uint64_t u = part < 4503599627370496.0 ? (uint64_t)(part + 0.5) : (uint64_t)part;
    pairs[i].turns = inv_freq[i] < 0 ? 0 - u : u;
    pairs[i].axis = axes ? axes[i] : 0;
    pairs[i].reserved = 0;
    if (pairs[i].axis < 0 || pairs[i].axis > 3) return MSA_ERR_INVALID_ARGUMENT;
  }
  return MSA_OK;
}

int msa_norm_rope(const msa_rope_problem* p, const uint16_t* const* x, const int32_t* positions, uint16_t* const* y,
                  int32_t* d_status, void* stream) {
  int rc = rope::check_problem(p);
  if (rc) return rc;
  rope::RowsArgs a{};
  if (!x || !y || !d_status || !aligned16(d_status)) return MSA_ERR_INVALID_ARGUMENT;
  if (p->tokens && (bad_rows(p, x) || bad_rows(p, y) || !positions || !aligned16(positions)))
    return MSA_ERR_INVALID_ARGUMENT;
  if ((rc = check_device_current())) return rc;
  a.heads = set_tensors(a, p, x);
  if (p->tokens == 0 || a.heads == 0) return MSA_OK;
  for (int i = 0; i < rope::kTensors; ++i) a.y[i] = p->tensor[i].heads ? y[i] : nullptr;
  a.an = rope::angles_of(p, positions, d_status);
  a.eps = p->eps;
  a.offset = p->weight_offset;
  a.T = p->tokens;
  const rope::Cut c = rope::cut_heads(a.heads);
  a.groups = c.groups; a.units = c.units; a.phases = c.phases;
  int32_t sms = 0;
  if ((rc = sm_count_current(&sms))) return rc;
  a.tile = rope::cut_tokens(a.T, a.groups, sms, rope::kTile, 1);
  a.status = d_status;
  const int64_t ctas = (int64_t)((a.T + a.tile - 1) / a.tile) * a.groups;
  if (ctas > INT32_MAX) return MSA_ERR_UNSUPPORTED_SHAPE;
  return cache::launch_kernel(p->adjacent ? rope::norm_rope_kernel<true> : rope::norm_rope_kernel<false>,
                              dim3((unsigned)ctas), rope::kThreads, 0, stream, 1, a);
}

size_t msa_norm_rope_bwd_bytes(const msa_rope_problem* p) {
  if (rope::check_problem(p)) return 0;
  const rope::GradCut g = rope::cut_grad(p);
  return round_up((size_t)g.slices * g.slots * 512 + 256, 256);
}

int msa_norm_rope_bwd(const msa_rope_problem* p, const uint16_t* const* dy, const uint16_t* const* x,
                      const int32_t* positions, uint16_t* const* dx, void* const* dw, int32_t* d_status, void* ws,
                      size_t ws_bytes, void* stream) {
  int rc = rope::check_problem(p);
  if (rc) return rc;
  if (!dy || !x || !dx || !dw || !d_status || !aligned16(d_status) || !ws || !aligned16(ws))
    return MSA_ERR_INVALID_ARGUMENT;
  if (p->tokens && (bad_rows(p, dy) || bad_rows(p, x) || bad_rows(p, dx) || !positions || !aligned16(positions)))
    return MSA_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < rope::kTensors; ++i) {
    const msa_rope_tensor& t = p->tensor[i];
    if (t.heads && dw[i] && (!aligned16(dw[i]) || !t.weight || !(t.flags & MSA_ROPE_NORM)))
      return MSA_ERR_INVALID_ARGUMENT;
  }
  if (ws_bytes < msa_norm_rope_bwd_bytes(p)) return MSA_ERR_INVALID_ARGUMENT;
  if ((rc = check_device_current())) return rc;
  const rope::GradCut g = rope::cut_grad(p);
  if (g.heads == 0) return MSA_OK;
  rope::SumArgs s{};
  rope::GradArgs a{};
  set_tensors(a, p, x);
  int rows = 0;
  for (int i = 0; i < rope::kTensors; ++i) {
    const msa_rope_tensor& t = p->tensor[i];
    const bool want = t.heads && dw[i];
    if (want) rows += t.flags & MSA_ROPE_PER_HEAD ? t.heads : 1;
    s.dw[i] = want ? dw[i] : nullptr;
    s.wide[i] = (t.flags & MSA_ROPE_WEIGHT_FP32) != 0;
    s.slot[i] = g.slot[i];
    s.per[i] = g.per[i];
    s.end[i] = rows;
    a.dy[i] = t.heads ? dy[i] : nullptr;
    a.dx[i] = t.heads ? dx[i] : nullptr;
    a.slot[i] = want ? g.slot[i] : -1;
    a.first[i] = g.first[i];
  }
  s.partial = static_cast<const float*>(ws);
  s.slices = g.slices;
  s.slots = g.slots;
  s.status = d_status;
  if (p->tokens) {
    a.an = rope::angles_of(p, positions, d_status);
    a.eps = p->eps;
    a.offset = p->weight_offset;
    a.T = p->tokens;
    a.heads = g.heads;
    a.tile = g.tile; a.tiles = g.tiles; a.slices = g.slices; a.slots = g.slots;
    a.groups = g.c.groups; a.units = g.c.units; a.phases = g.c.phases;
    a.partial = static_cast<float*>(ws);
    a.status = d_status;
    rc = cache::launch_kernel(p->adjacent ? rope::norm_rope_bwd_kernel<true> : rope::norm_rope_bwd_kernel<false>,
                              dim3((unsigned)(g.slices * g.c.groups)), rope::kThreads, 0, stream, 1, a);
    if (rc) return rc;
  }
  if (rows == 0) return MSA_OK;
  return cache::launch_kernel(rope::weight_sum_kernel, dim3((unsigned)rows), 128 * rope::kSumParts, 0, stream, 1, s);
}

}  // extern "C"
