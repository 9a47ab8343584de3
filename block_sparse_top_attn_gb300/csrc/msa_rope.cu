// Norm and rotary positions of queries, keys and index vectors, and their
// gradients (msa_rope.cuh has a row's arithmetic).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "msa_rope.cuh"

namespace msa {
namespace rope {

constexpr int64_t kMaxStride = int64_t(1) << 38;  // times 2^24 tokens: within 64 bits

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
  if (p->zero_padding < 0 || p->zero_padding > 1) return MSA_ERR_INVALID_ARGUMENT;
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

constexpr int kRowCtas = 3;  // of the largest size on an SM
// Most tokens of a CTA: SMs differ in speed, and shares that all start at once end
// when the slowest does (131k tokens x 152 heads 1725 us, in shares of 32 tokens
// 1464; 32k x 68 208 and 175).
constexpr int kRowTokens = 32;
constexpr int kRowThreads = 32 * (kRowWarps + 1);
// Where the next kernel's CTAs come up early: behind so few that they are in nobody's way
// (a captured decode step of one request, norm and append apart, 21.6 us, else 22.5; of
// 16 requests 26.2, else 23.6).
constexpr unsigned kFewCtas = 16;
template <bool kAdjacent>
__global__ void __launch_bounds__(kRowThreads, kRowCtas) norm_rope_kernel(RowsArgs a) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  if (gridDim.x <= kFewCtas) cache::after_previous_kernel();
  else cache::after_previous_kernel<false>();
  rows_block<kAdjacent>(a, blockIdx.x, status_bad(a.status), *reinterpret_cast<RowsShared*>(s_raw));
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
  int T, heads, slots;
  Cut cut;
  float* partial;  // [slices][slots][128]
  int32_t* status;
};

// 1 / sqrt(mean + eps) of a row's sum of squares.  v holds the row times `scale` (1, or
// kDown where its squares leave fp32's range) after it: v * result is the normed row
// either way.  Whole warps call it.
MSA_DEV float inverse_rms(Values& v, float sum, float eps, float& scale) {
  scale = 1.f;
  if (__any_sync(0xffffffffu, !(sum < kInf))) {
    const bool far = !(sum < kInf);
    if (far) {
      scale = kDown;
      eps = 0.f;
    }
    times(v, scale);
    const float again = row_sum(squares(v));
    if (far) sum = again;
  }
  return rsqrtf(fmaf(sum, 1.f / 128.f, eps));
}

constexpr int kGradStages = 3, kGradCtas = 2, kGradWarps = 9, kGradThreads = 32 * (kGradWarps + 1);
struct GradShared {
  Table<kTile> tab[2];
  union {
    Stage ring[kGradWarps][kGradStages][2];  // x and dy
    float dw[kGradWarps * 4][128];
  };
};

// The rows of one warp; false if the status was set (rows_block).
template <bool kAdjacent>
MSA_DEV bool grad_rows(const GradArgs& a, GradShared& s, bool bad, int slice, int group, int n, int apart) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane & 7;
  const int phase = warp / a.cut.units, unit = group * a.cut.units + warp - phase * a.cut.units;
  const int hh = unit * 4 + (lane >> 3);
  const bool live = hh < a.heads;
  int da, db, head;
  lane_dims(j, a.an.R, da, db);
  const int k = tensor_of(a, live ? hh : 0, head);
  const Tensor& t = a.t[k];
  const int sa = granule_slot(da >> 3), sb = granule_slot(db >> 3);
  const int phases = a.cut.phases;
  const int64_t first = slice + (int64_t)phase * apart, step = (int64_t)phases * apart;  // this warp's tokens
  const int64_t x_step = step * t.x_token, y_step = step * a.y_token[k];
  const int64_t x0 = first * t.x_token + head * t.x_head;
  const uint16_t *x = t.x + x0, *dy = a.dy[k] + first * a.y_token[k] + head * a.y_head[k];  // next to copy
  uint16_t* dx = a.dx[k] + x0;
  auto& ring = s.ring[warp];
  int ahead = phase;
  auto copy = [&](int stage) {
    if (live && ahead < n) {
      copy_row(ring[stage][0], x, lane);
      copy_row(ring[stage][1], dy, lane);
    }
    copies_commit();
    ahead += phases;
    x += x_step;
    dy += y_step;
  };
#pragma unroll
  for (int i = 0; i < kGradStages - 1; ++i) copy(i);
  if (!live)  // rows that are not there count as zeros
    for (int i = lane & 7; i < kGradStages * 2 * 16; i += 8)
      ring[i >> 5][i >> 4 & 1].row[lane >> 3][i & 15] = make_uint4(0, 0, 0, 0);
  const bool norm = t.flags & MSA_ROPE_NORM, turn = turns(t, j, a.an.R);
  Values w, dw;
  load_weights<kAdjacent>(t, head, da, db, a.offset, w);
#pragma unroll
  for (int i = 0; i < 4; ++i) dw.a[i] = dw.b[i] = 0;
  if (__syncthreads_or(bad)) {  // the first table is there
    copies_wait<0>();
    return false;
  }
  int stage = 0, next = kGradStages - 1, i = phase;
  for (int at = 0, table = 0; at < n; at += kTile, ++table) {
    const Table<kTile>& tab = s.tab[table & 1];
    for (; i < min(at + kTile, n); i += phases) {
      copies_wait<kGradStages - 2>();
      __syncwarp();  // the lanes' copies have landed; the stage before has been read
      const uint4 *xr = ring[stage][0].row[lane >> 3], *gr = ring[stage][1].row[lane >> 3];
      uint4 xa = xr[sa], xb = xr[sb], ga = gr[sa], gb = gr[sb];
      copy(next);
      next = stage;
      stage = stage + 1 == kGradStages ? 0 : stage + 1;
      if (tab.live[i - at]) {
        Values v, g;
        unpack<kAdjacent>(xa, xb, v);
        unpack<kAdjacent>(ga, gb, g);
        if (turn) rotate<true>(g, tab.cs[i - at], j);
        float scale;
        const float sum = row_sum(squares(v));
        const float r = inverse_rms(v, norm ? sum : 0.f, a.eps, scale);
        if (norm) {
          times(v, r);  // the normed row without its weight
          uint64_t dot = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dw.a[e] = f2_fma(g.a[e], v.a[e], dw.a[e]);
            dw.b[e] = f2_fma(g.b[e], v.b[e], dw.b[e]);
            g.a[e] = f2_mul(g.a[e], w.a[e]);
            g.b[e] = f2_mul(g.b[e], w.b[e]);
            dot = f2_fma(g.a[e], v.a[e], dot);
            dot = f2_fma(g.b[e], v.b[e], dot);
          }
          float lo, hi;
          f2_unpack(dot, lo, hi);
          // the rows' lanes are those of one tensor
          const float mean = row_sum(lo + hi, 0xFFu << (lane & 24)) * (-1.f / 128.f);
          const uint64_t m = f2_pack(mean, mean);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            g.a[e] = f2_fma(v.a[e], m, g.a[e]);
            g.b[e] = f2_fma(v.b[e], m, g.b[e]);
          }
          times(g, r * scale);
        }
        pack<kAdjacent>(g, ga, gb);
        if (live) {
          *reinterpret_cast<uint4*>(dx + da) = ga;
          *reinterpret_cast<uint4*>(dx + db) = gb;
        }
      }
      dx += x_step;
    }
    __syncthreads();  // it has been read, the next one is there
  }
  // the sums, by rows of the CTA (the rings have been read)
  float* row = s.dw[warp * 4 + (lane >> 3)];
  float sums[16];
  in_order<kAdjacent>(dw, sums);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    row[da + e] = live ? sums[e] : 0.f;
    row[db + e] = live ? sums[8 + e] : 0.f;
  }
  return true;
}

template <bool kAdjacent>
__global__ void __launch_bounds__(kGradThreads, kGradCtas) norm_rope_bwd_kernel(GradArgs a) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  GradShared& s = *reinterpret_cast<GradShared*>(s_raw);
  cache::after_previous_kernel();
  const bool bad = status_bad(a.status);
  const int tid = threadIdx.x, slice = blockIdx.x / a.cut.groups, group = blockIdx.x - slice * a.cut.groups;
  const int apart = a.cut.slices, n = (a.T - slice + apart - 1) / apart;
  const int row_threads = 32 * a.cut.units * a.cut.phases;
  if (tid >= row_threads) {
    if (!fill_tables<kAdjacent>(a.an, s.tab, bad, row_threads, slice, n, apart, [](int64_t) {})) return;
  } else if (!grad_rows<kAdjacent>(a, s, bad, slice, group, n, apart)) {
    return;
  }
  // the CTA's sums: heads that share a weight in the order of the warps and rows
  __syncthreads();
  // threads behind the last 128 of the CTA have no part in it
  if (tid >> 7 >= (int)blockDim.x >> 7) return;
  const int d = tid & 127, units = a.cut.units, phases = a.cut.phases;
  float* out = a.partial + (int64_t)slice * a.slots * 128 + d;
  for (int i = 0, before = 0; i < kTensors; ++i) {
    const int end = a.t[i].end;
    if (a.slot[i] >= 0) {
      // this CTA's heads of the tensor, and its rows (of the warps' first phase)
      const int lo = max(before, group * units * 4), hi = min(end, (group + 1) * units * 4);
      const int row0 = lo - group * units * 4, rows = hi - lo;
      if (a.t[i].flags & MSA_ROPE_PER_HEAD) {
        for (int r = tid >> 7; r < rows; r += (int)blockDim.x >> 7) {
          float s1 = 0.f;
          for (int p = 0; p < phases; ++p) s1 += s.dw[p * units * 4 + row0 + r][d];
          out[(int64_t)(a.slot[i] + lo - before + r) * 128] = s1;
        }
      } else if (rows > 0 && tid < 128) {
        float s1 = 0.f;
        for (int p = 0; p < phases; ++p)
          for (int r = 0; r < rows; ++r) s1 += s.dw[p * units * 4 + row0 + r][d];
        out[(int64_t)(a.slot[i] + group - a.first[i]) * 128] = s1;
      }
    }
    before = end;
  }
}

struct SumArgs {
  Tensor t[kTensors];  // of the gradients' rows, for the zeros of padding
  uint16_t* dx[kTensors];
  const int32_t* positions;
  int A, T, heads;
  unsigned sums;  // CTAs that add; those behind them write zeros
  const float* partial;
  void* dw[kTensors];
  int wide[kTensors];  // fp32
  int slot[kTensors], end[kTensors];  // first slot; rows of weights of this tensor and those before it
  int per[kTensors];   // slots that make one row of weights
  int slices, slots;
  int32_t* status;
};

constexpr int kSumParts = 16;
// Zeros to the padding among the CTA's tokens, a warp 32 of them.  Here, where the loads
// of the weights' sums leave time: in norm_rope_bwd_kernel, by the warps of the rows or by
// those of the angles, the registers' different use made 32k tokens x 68 heads 281 us
// of 261.
MSA_DEV void zero_tokens(const SumArgs& a, int cta) {
  const int lane = threadIdx.x & 31, t0 = cta * 32 * kSumParts + (threadIdx.x & ~31);
  const bool padding = t0 + lane < a.T && a.positions[(int64_t)(t0 + lane) * a.A] < 0;
  for (unsigned left = __ballot_sync(0xffffffffu, padding); left; left &= left - 1) {
    const int64_t t = t0 + __ffs(left) - 1;
    zero_heads(0, a.heads, lane, 32, [&](int hh) {
      int head;
      const int k = tensor_of(a, hh, head);
      return a.dx[k] + t * a.t[k].x_token + head * a.t[k].x_head;
    });
  }
}

// A CTA adds up 32 dims of one row of weights: a warp every 16th slice, sixteen loads
// in flight.
__global__ void __launch_bounds__(32 * kSumParts) weight_sum_kernel(SumArgs a) {
  __shared__ float s_part[kSumParts][32];
  cache::after_previous_kernel();
  const bool bad = status_bad(a.status);  // decided on below: the load does not hold up the others
  if (blockIdx.x >= a.sums) {
    if (!__syncthreads_or(bad)) zero_tokens(a, (int)(blockIdx.x - a.sums));
    return;
  }
  const int all = blockIdx.x >> 2;  // row of all tensors' weights
  int row = all, slot = a.slot[0], per = a.per[0], wide = a.wide[0];
  void* dw = a.dw[0];
#pragma unroll
  for (int i = 1; i < kTensors; ++i)
    if (all >= a.end[i - 1]) {
      row = all - a.end[i - 1];
      slot = a.slot[i];
      per = a.per[i];
      wide = a.wide[i];
      dw = a.dw[i];
    }
  const int d = (blockIdx.x & 3) * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  const int64_t step = (int64_t)a.slots * 128;
  float s = 0.f;
  for (int p = 0; p < per; ++p) {
    const float* src = a.partial + (int64_t)(slot + row * per + p) * 128 + d;
    for (int i0 = part; i0 < a.slices; i0 += 16 * kSumParts) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = i0 + i * kSumParts < a.slices ? src[(i0 + i * kSumParts) * step] : 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) s += x[i];
    }
  }
  s_part[part][threadIdx.x & 31] = s;
  if (__syncthreads_or(bad) || part) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kSumParts; ++i) s += s_part[i][threadIdx.x];
  if (wide) static_cast<float*>(dw)[(int64_t)row * 128 + d] = s;
  else static_cast<uint16_t*>(dw)[(int64_t)row * 128 + d] = (uint16_t)(pack_bf16x2(s, 0.f) & 0xFFFFu);
}

// How the gradients' tokens and partial sums are cut.  It depends on the problem
// alone: the workspace's size and the order of the sums do.
struct GradCut {
  Cut c;
  int heads, slots;
  int slot[kTensors], first[kTensors], per[kTensors];
};
static GradCut cut_grad(const msa_rope_problem* p) {
  GradCut g{};
  for (int i = 0; i < kTensors; ++i) g.heads += p->tensor[i].heads;
  if (g.heads == 0) return g;
  g.c = cut_rows(g.heads, p->tokens, 152, kGradCtas * (kGradWarps + 1), kGradWarps);
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

// f / 2 pi modulo a turn, in units of 2^-64, rounded once: the quotient in two parts,
// q + rest, by 2 pi in two parts, so that it is within 2^-104 of itself.
uint64_t turns_per_position(double f) {
  constexpr double kHi = 6.283185307179586, kLo = 2.4492935982947064e-16;  // 2 pi
  const double q = f / kHi;
  double rest = fma(-q, kLo, fma(-q, kHi, f)) / kHi;
  rest -= floor(rest + 0.5);                    // a q beyond 2^52 leaves whole turns
  const double part = ldexp(q - floor(q), 64);  // < 2^64: a double below 1 is at most 1 - 2^-53
  const double whole = floor(part);
  return (uint64_t)whole + (uint64_t)(int64_t)floor(part - whole + ldexp(rest, 64) + 0.5);
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
    const uint64_t u = turns_per_position(fabs(inv_freq[i]));
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
  a.zero = p->zero_padding;
  int32_t sms = 0;
  if ((rc = sm_count_current(&sms))) return rc;
  a.cut = rope::cut_rows(a.heads, a.T, sms, rope::kRowCtas * (rope::kRowWarps + 1),
                         rope::kRowWarps);
  a.cut.at_most(a.T, rope::kRowTokens);
  a.status = d_status;
  return cache::launch_kernel(p->adjacent ? rope::norm_rope_kernel<true> : rope::norm_rope_kernel<false>,
                              dim3((unsigned)(a.cut.slices * a.cut.groups)), a.cut.threads(), sizeof(rope::RowsShared),
                              stream, 1, a);
}

size_t msa_norm_rope_bwd_bytes(const msa_rope_problem* p) {
  if (rope::check_problem(p)) return 0;
  const rope::GradCut g = rope::cut_grad(p);
  return round_up((size_t)g.c.slices * g.slots * 512 + 256, 256);
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
  s.slices = g.c.slices;
  s.slots = g.slots;
  s.status = d_status;
  if (p->tokens) {
    a.an = rope::angles_of(p, positions, d_status);
    a.eps = p->eps;
    a.offset = p->weight_offset;
    a.T = p->tokens;
    a.heads = g.heads;
    a.slots = g.slots;
    a.cut = g.c;
    a.partial = static_cast<float*>(ws);
    a.status = d_status;
    rc = cache::launch_kernel(p->adjacent ? rope::norm_rope_bwd_kernel<true> : rope::norm_rope_bwd_kernel<false>,
                              dim3((unsigned)(g.c.slices * g.c.groups)), g.c.threads(), sizeof(rope::GradShared),
                              stream, 1, a);
    if (rc) return rc;
  }
  s.sums = (unsigned)rows * 4;
  unsigned zeros = 0;
  if (p->zero_padding && p->tokens) {
    for (int i = 0; i < rope::kTensors; ++i) {
      s.t[i] = a.t[i];
      s.dx[i] = a.dx[i];
    }
    s.heads = g.heads;
    s.positions = positions;
    s.A = p->num_axes;
    s.T = p->tokens;
    zeros = ((unsigned)p->tokens + 32 * rope::kSumParts - 1) / (32 * rope::kSumParts);
  }
  if (s.sums + zeros == 0) return MSA_OK;
  return cache::launch_kernel(rope::weight_sum_kernel, dim3(s.sums + zeros), 32 * rope::kSumParts, 0, stream, 1, s);
}

}  // extern "C"
