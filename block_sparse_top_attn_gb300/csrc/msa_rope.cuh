// Norm and rotary positions of heads: arguments, angles and the arithmetic of a
// row, shared by msa_norm_rope, its gradients and the serving append.
//
// Eight lanes hold a row (one head of one token, 128 dims, 256 bytes): lane j two
// granules of 8 dims, a lane's pairs both whole: with R rotated dims, lanes
// j < R / 16 hold dims 8j .. and R / 2 + 8j .. (the two halves of pairs 8j ..), the
// others the dims behind R.  Dims are paired within a lane in either layout, a
// row's sum takes three shuffles, and a warp's four rows are 1 KB, in 16-byte
// accesses of 32 bytes or more side by side.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "msa_cache.cuh"

namespace msa {
namespace rope {

constexpr int kTensors = 4;   // q, k, q_index, k_index
constexpr int kTile = 16;     // most tokens of a tile
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kInf = __builtin_huge_valf();

struct Angles {  // where a call's angles come from
  const msa_rope_pair* pairs;
  const int32_t* positions;
  int R, A;  // rotated dims, position columns
  float scale;
  int32_t* status;
};

struct Tensor {
  const uint16_t* x;
  const void* w;
  int64_t x_token, x_head;
  uint32_t flags;
  int end;  // heads of this tensor and those before it
};

// Whether lane j's dims of a tensor are rotated.
MSA_DEV bool turns(const Tensor& t, int j, int R) { return (t.flags & MSA_ROPE_ROTATE) && j < R >> 4; }

// First dims of lane j's granules.
MSA_DEV void lane_dims(int j, int R, int& a, int& b) {
  const int n = R >> 4;
  if (j < n) {
    a = 8 * j;
    b = (R >> 1) + 8 * j;
  } else {
    a = R + 8 * (j - n);
    b = a + 8 * (8 - n);
  }
}

// Cosine and sine of a fraction of a turn.  The quarter turn is taken off exactly,
// so what the functions get is below 1/8 turn and as exact as its 24 bits.
MSA_DEV void cos_sin(uint64_t turn, float scale, float& c, float& s) {
  const uint64_t shifted = turn + (1ull << 61);
  const int64_t rest = (int64_t)(turn - (shifted & (3ull << 62)));
  float sn, cs;
  sincospif((float)rest * 1.0842021724855044e-19f, &sn, &cs);  // 2^-63: half turns
  sn *= scale;
  cs *= scale;
  const int quarter = (int)(shifted >> 62);
  c = quarter & 1 ? sn : cs;
  s = quarter & 1 ? cs : sn;
  if (quarter == 1 || quarter == 2) c = -c;
  if (quarter >= 2) s = -s;
}

// Pair of entry e of lane j < R / 16.
template <bool kAdjacent>
MSA_DEV int pair_of(int j, int e, int R) {
  if constexpr (kAdjacent) return e < 4 ? 4 * j + e : (R >> 2) + 4 * j + e - 4;
  else return 8 * j + e;
}

// Fraction of a turn of pair p at token t.
MSA_DEV uint64_t turn_of(const Angles& a, int p, int64_t t) {
  const int4 w = reinterpret_cast<const int4*>(a.pairs)[p];
  const uint64_t turns = (uint64_t)(uint32_t)w.y << 32 | (uint32_t)w.x;
  const int axis = (unsigned)w.z < (unsigned)a.A ? w.z : 0;
  if (axis != w.z) set_status(a.status, MSA_ERR_INVALID_ARGUMENT);
  return turns * (uint64_t)(int64_t)a.positions[t * a.A + axis];
}

// Entries 2 * e2 and 2 * e2 + 1 of lane j < R / 16 at a token: (cos, sin, cos, sin).
template <bool kAdjacent>
MSA_DEV float4 entry_pair(const Angles& a, int j, int e2, int64_t t) {
  float4 x;
  cos_sin(turn_of(a, pair_of<kAdjacent>(j, 2 * e2, a.R), t), a.scale, x.x, x.y);
  cos_sin(turn_of(a, pair_of<kAdjacent>(j, 2 * e2 + 1, a.R), t), a.scale, x.z, x.w);
  return x;
}

// A tile's angles in shared memory: a row of [4][8] float4 per token (lane j's
// entries 2 * e2 .. at [e2][j], so that eight lanes read 128 bytes side by side).
// Lanes j >= R / 16 have none.
template <int kRows>
struct Table {
  float4 cs[kRows][32];
};
template <bool kAdjacent, int kRows>
MSA_DEV void fill_table(Table<kRows>& tab, const Angles& a, int64_t t0, int n) {
  for (int i = threadIdx.x; i < n * 32; i += kThreads) {
    const int row = i >> 5, e2 = (i >> 3) & 3, j = i & 7;
    if (j < a.R >> 4) tab.cs[row][i & 31] = entry_pair<kAdjacent>(a, j, e2, t0 + row);
  }
}
MSA_DEV void load_angles(const float4* row, int j, float4 (&cs)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = row[i * 8 + j];
}

MSA_DEV void unpack8(uint4 u, float* v) {
  v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xFFFF0000u);
  v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  v[4] = __uint_as_float(u.z << 16); v[5] = __uint_as_float(u.z & 0xFFFF0000u);
  v[6] = __uint_as_float(u.w << 16); v[7] = __uint_as_float(u.w & 0xFFFF0000u);
}
MSA_DEV uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// A lane's 16 weights of a head, the offset added; 1 where there are none.
MSA_DEV void load_weights(const Tensor& t, int head, int a, int b, float offset, float (&w)[16]) {
  if (!(t.flags & MSA_ROPE_NORM) || !t.w) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 1.f;
    return;
  }
  const int64_t at = t.flags & MSA_ROPE_PER_HEAD ? (int64_t)head * 128 : 0;
  if (t.flags & MSA_ROPE_WEIGHT_FP32) {
    const float* p = static_cast<const float*>(t.w) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 u = *reinterpret_cast<const float4*>(p + (i < 2 ? a : b) + 4 * (i & 1));
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(t.w) + at;
    unpack8(*reinterpret_cast<const uint4*>(p + a), w);
    unpack8(*reinterpret_cast<const uint4*>(p + b), w + 8);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] += offset;
}

// Sum over the eight lanes of a row; all of them get it.
MSA_DEV float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
MSA_DEV float squares(const float (&v)[16]) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s0 = fmaf(v[i], v[i], s0);
    s1 = fmaf(v[8 + i], v[8 + i], s1);
  }
  return s0 + s1;
}

// 1 / sqrt(mean + eps) of a row's sum of squares.  Rows whose squares leave fp32's
// range (elements above 10^18) are scaled by 2^-64 first, where eps does not count.
// Whole warps call this; v holds the row times `scale` after it (v * result is the
// normed row either way).
MSA_DEV float inverse_rms(float (&v)[16], float sum, float eps, float& scale) {
  scale = 1.f;
  if (__any_sync(0xffffffffu, !(sum < kInf))) {
    const bool far = !(sum < kInf);
    if (far) {
      scale = 5.421010862427522e-20f;  // 2^-64
      eps = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= scale;
    const float again = row_sum(squares(v));
    if (far) sum = again;
  }
  return rsqrtf(fmaf(sum, 1.f / 128.f, eps));
}

// The lane's pairs turned; kBack: by the opposite angle.
template <bool kAdjacent, bool kBack>
MSA_DEV void rotate(float (&v)[16], const float4 (&cs)[4]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float c = e & 1 ? cs[e >> 1].z : cs[e >> 1].x;
    const float s0 = e & 1 ? cs[e >> 1].w : cs[e >> 1].y;
    const float s = kBack ? -s0 : s0;
    const int i = kAdjacent ? 2 * e : e, k = kAdjacent ? 2 * e + 1 : e + 8;
    const float a = v[i], b = v[k];
    v[i] = fmaf(a, c, -(b * s));
    v[k] = fmaf(b, c, a * s);
  }
}

// One row: normed if `norm`, then turned by the angles at `row` if `turn` (this
// lane's dims are: a turn by nothing would carry infinities from pair to pair).
template <bool kAdjacent>
MSA_DEV void norm_rotate(float (&v)[16], const float (&w)[16], const float4* row, int j, bool norm, bool turn,
                         float eps) {
  float scale;
  const float sum = row_sum(squares(v));
  const float inv = inverse_rms(v, norm ? sum : 0.f, eps, scale);
  const float r = norm ? inv : 1.f;  // w is 1 without a norm
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = v[i] * r * w[i];
  if (turn) {
    float4 cs[4];
    load_angles(row, j, cs);
    rotate<kAdjacent, false>(v, cs);
  }
}

// Host side.
int check_problem(const msa_rope_problem* p);
inline const Angles angles_of(const msa_rope_problem* p, const int32_t* positions, int32_t* status) {
  return Angles{p->pairs, positions, p->rotary_dim, p->num_axes, p->cos_scale, status};
}

// How the rows of a call's tensors are cut: a unit is four heads (of the tensors'
// heads one after the other) of a token, a warp's share; `units` of them to a
// CTA's warps, `groups` CTAs side by side; with few units, `phases` warps take
// a tile's tokens in turn.
struct Cut {
  int groups, units, phases;
};
inline Cut cut_heads(int64_t heads) {
  const int64_t u = (heads + 3) / 4;
  Cut c;
  c.groups = (int)((u + kWarps - 1) / kWarps);
  c.units = (int)((u + c.groups - 1) / c.groups);
  c.phases = kWarps / c.units;
  return c;
}
// Tokens of a tile: the most whose tiles still give every SM two CTAs.
inline int cut_tokens(int64_t tokens, int64_t groups, int sms, int most, int least) {
  int tile = most;
  while (tile > least && (tokens + tile - 1) / tile * groups < 2 * (int64_t)sms) tile >>= 1;
  return tile;
}

// Rows in and out, by CTAs of (tile of tokens, group of heads).
struct RowsArgs {
  Tensor t[kTensors];
  uint16_t* y[kTensors];
  int64_t y_token[kTensors], y_head[kTensors];
  Angles an;
  float eps, offset;
  int T, heads;  // of all tensors
  int tile, groups, units, phases;
  int32_t* status;
};

// Index of the tensor that flattened head `hh` belongs to, and its head there.
template <class Args>
MSA_DEV int tensor_of(const Args& a, int hh, int& head) {
  int i = 0, before = 0;
#pragma unroll
  for (int k = 0; k + 1 < kTensors; ++k)
    if (hh >= a.t[k].end) {
      i = k + 1;
      before = a.t[k].end;
    }
  head = hh - before;
  return i;
}

template <bool kAdjacent>
MSA_DEV void rows_block(const RowsArgs& a, int64_t block, Table<kTile>& tab) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, j = lane & 7;
  const int64_t tile = block / a.groups;
  const int group = (int)(block - tile * a.groups);
  const int64_t t0 = tile * a.tile;
  const int n = (int)min((int64_t)a.tile, a.T - t0);
  fill_table<kAdjacent>(tab, a.an, t0, n);
  const int phase = warp / a.units, unit = group * a.units + warp - phase * a.units;
  const int hh = unit * 4 + (lane >> 3);
  const bool live = hh < a.heads;
  int da, db, head;
  lane_dims(j, a.an.R, da, db);
  const int k = tensor_of(a, live ? hh : 0, head);
  const Tensor& t = a.t[k];
  const bool norm = t.flags & MSA_ROPE_NORM, turn = turns(t, j, a.an.R);
  float w[16];
  load_weights(t, head, da, db, a.offset, w);
  const uint16_t* x = t.x + t0 * t.x_token + head * t.x_head;
  uint16_t* y = a.y[k] + t0 * a.y_token[k] + head * a.y_head[k];
  __syncthreads();
  if (phase >= a.phases) return;
  for (int i = phase; i < n; i += a.phases) {
    uint4 ua = make_uint4(0, 0, 0, 0), ub = ua;
    if (live) {
      ua = *reinterpret_cast<const uint4*>(x + i * t.x_token + da);
      ub = *reinterpret_cast<const uint4*>(x + i * t.x_token + db);
    }
    float v[16];
    unpack8(ua, v);
    unpack8(ub, v + 8);
    norm_rotate<kAdjacent>(v, w, tab.cs[i], j, norm, turn, a.eps);
    if (live && a.an.positions[(t0 + i) * a.an.A] >= 0) {
      *reinterpret_cast<uint4*>(y + i * a.y_token[k] + da) = pack8(v);
      *reinterpret_cast<uint4*>(y + i * a.y_token[k] + db) = pack8(v + 8);
    }
  }
}

}  // namespace rope
}  // namespace msa
