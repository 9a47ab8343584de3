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
constexpr int kTile = 8;      // tokens of a table of angles
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowWarps = 8;  // warps of a CTA that take rows, beside one for the angles
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

// Cosine and sine of a fraction of a turn.  The quarter turns are taken off exactly,
// and the eighth that is left is as exact as its 24 bits, so that the Taylor
// polynomials of degrees 9 and 10 (off by 2^-28.5 and 2^-32 of the value) serve: within
// 6 u of a relative error, u = 2^-24: 4 u from the argument, 2 u from the sums.
MSA_DEV void cos_sin(uint64_t turn, float scale, float& c, float& s) {
  const uint64_t shifted = turn + (1ull << 61);
  const int64_t rest = (int64_t)(turn - (shifted & (3ull << 62)));
  const uint64_t size = rest < 0 ? 0 - (uint64_t)rest : (uint64_t)rest;
  // in radians: the high word times pi 2^-31, the low one times pi 2^-63
  float x = fmaf((float)(uint32_t)size, 3.4061215800865545e-19f, (float)(uint32_t)(size >> 32) * 1.4629180792671596e-09f);
  x = rest < 0 ? -x : x;
  const float z = x * x;
  float sn = fmaf(z, 1.f / 362880.f, -1.f / 5040.f), cs = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  sn = fmaf(z, sn, 1.f / 120.f);
  cs = fmaf(z, cs, -1.f / 720.f);
  sn = fmaf(z, sn, -1.f / 6.f);
  cs = fmaf(z, cs, 1.f / 24.f);
  sn = fmaf(x * z, sn, x) * scale;
  cs = fmaf(z, fmaf(z, cs, -0.5f), 1.f) * scale;
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

// Turns per position of pair p, and its position column.
struct Pair {
  uint64_t turns;
  int axis;
};
MSA_DEV Pair load_pair(const Angles& a, int p) {
  const int4 w = reinterpret_cast<const int4*>(a.pairs)[p];
  Pair x;
  x.turns = (uint64_t)(uint32_t)w.y << 32 | (uint32_t)w.x;
  x.axis = (unsigned)w.z < (unsigned)a.A ? w.z : 0;
  if (x.axis != w.z) set_status(a.status, MSA_ERR_INVALID_ARGUMENT);
  return x;
}
// Fraction of a turn at a position, and at token t.
MSA_DEV uint64_t turn_at(const Pair& p, int position) { return p.turns * (uint64_t)(int64_t)position; }
MSA_DEV uint64_t turn_of(const Angles& a, const Pair& p, int64_t t) {
  return turn_at(p, a.positions[t * a.A + p.axis]);
}

// A tile's angles in shared memory: a row of [4][8] float4 per token, lane j's
// entries 2 * e2 and 2 * e2 + 1 at [e2][j] as (cos, cos, sin, sin): eight lanes read
// 128 bytes side by side, and two entries are one operand of the packed
// arithmetic.  Lanes j >= R / 16 have none.
template <int kRows>
struct Table {
  float4 cs[kRows][32];
  int live[kRows];  // the token is no padding
};
// Fills tables, by `threads` threads of which this is `thread`: it has the same two
// pairs in every row.
template <bool kAdjacent>
struct Filler {
  Pair p0, p1;
  int thread;
  int at, row0, step;  // place in a row, the thread's first row, rows between two of its rows
  MSA_DEV Filler(const Angles& a, int thread_, int threads) : thread(thread_) {
    const int lanes = a.R >> 4, row = 4 * lanes;
    p0 = p1 = Pair{0, 0};
    at = -1;
    row0 = step = 0;
    if (lanes == 0) return;
    step = threads / row;
    row0 = thread / row;
    if (row0 >= step) return;
    const int i = thread - row0 * row, e2 = i / lanes, j = i - e2 * lanes;
    at = e2 * 8 + j;
    p0 = load_pair(a, pair_of<kAdjacent>(j, 2 * e2, a.R));
    p1 = load_pair(a, pair_of<kAdjacent>(j, 2 * e2 + 1, a.R));
  }
  // Of tokens t0, t0 + apart, .., n of them (no more than there are threads).
  template <int kRows>
  MSA_DEV void fill(Table<kRows>& tab, const Angles& a, int64_t t0, int n, int apart = 1) const {
    if (thread < n) tab.live[thread] = a.positions[(t0 + (int64_t)thread * apart) * a.A] >= 0;
    if (at < 0 || row0 >= n) return;
    // Positions a row ahead.  Not unrolled: in a short call the code's own way to the SM counts (a step of 256 tokens
    // 10.4 us, so 9.9).
    const int32_t* src = a.positions + (t0 + (int64_t)row0 * apart) * a.A;
    const int64_t next = (int64_t)step * apart * a.A;
    int q0 = src[p0.axis], q1 = src[p1.axis];
#pragma unroll 1
    for (int row = row0; row < n; row += step) {
      const uint64_t u0 = turn_at(p0, q0), u1 = turn_at(p1, q1);
      src += next;
      if (row + step < n) {
        q0 = src[p0.axis];
        q1 = src[p1.axis];
      }
      float4 x;
      cos_sin(u0, a.scale, x.x, x.z);
      cos_sin(u1, a.scale, x.y, x.w);
      tab.cs[row][at] = x;
    }
  }
};

// A lane's 16 values as its eight pairs (a, b), two pairs a word: dims (p, p + R / 2)
// come from its two granules, dims (2p, 2p + 1) from the halves of its words.
struct Values {
  uint64_t a[4], b[4];
};
template <bool kAdjacent>
MSA_DEV void unpack(uint4 ua, uint4 ub, Values& v) {
  const uint32_t w[8] = {ua.x, ua.y, ua.z, ua.w, ub.x, ub.y, ub.z, ub.w};
  auto lo = [&](int i) { return __uint_as_float(w[i] << 16); };
  auto hi = [&](int i) { return __uint_as_float(w[i] & 0xFFFF0000u); };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.a[i] = kAdjacent ? f2_pack(lo(2 * i), lo(2 * i + 1)) : f2_pack(lo(i), hi(i));
    v.b[i] = kAdjacent ? f2_pack(hi(2 * i), hi(2 * i + 1)) : f2_pack(lo(4 + i), hi(4 + i));
  }
}
// The values in the order of the granules' dims.
template <bool kAdjacent>
MSA_DEV void in_order(const Values& v, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kAdjacent) {
      f2_unpack(v.a[i], x[4 * i], x[4 * i + 2]);
      f2_unpack(v.b[i], x[4 * i + 1], x[4 * i + 3]);
    } else {
      f2_unpack(v.a[i], x[2 * i], x[2 * i + 1]);
      f2_unpack(v.b[i], x[8 + 2 * i], x[8 + 2 * i + 1]);
    }
  }
}
template <bool kAdjacent>
MSA_DEV void from_order(const float (&x)[16], Values& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.a[i] = kAdjacent ? f2_pack(x[4 * i], x[4 * i + 2]) : f2_pack(x[2 * i], x[2 * i + 1]);
    v.b[i] = kAdjacent ? f2_pack(x[4 * i + 1], x[4 * i + 3]) : f2_pack(x[8 + 2 * i], x[8 + 2 * i + 1]);
  }
}
template <bool kAdjacent>
MSA_DEV void pack(const Values& v, uint4& ua, uint4& ub) {
  float x[16];
  in_order<kAdjacent>(v, x);
  ua = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  ub = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]),
                  pack_bf16x2(x[14], x[15]));
}

// A lane's 16 weights of a head, the offset added; 1 where there are none.
template <bool kAdjacent>
MSA_DEV void load_weights(const Tensor& t, int head, int a, int b, float offset, Values& w) {
  float x[16];
  if (!(t.flags & MSA_ROPE_NORM) || !t.w) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 1.f;
  } else {
    const int64_t at = t.flags & MSA_ROPE_PER_HEAD ? (int64_t)head * 128 : 0;
    if (t.flags & MSA_ROPE_WEIGHT_FP32) {
      const float* p = static_cast<const float*>(t.w) + at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 u = *reinterpret_cast<const float4*>(p + (i < 2 ? a : b) + 4 * (i & 1));
        x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = u.z; x[4 * i + 3] = u.w;
      }
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(t.w) + at;
      Values u;
      unpack<kAdjacent>(*reinterpret_cast<const uint4*>(p + a), *reinterpret_cast<const uint4*>(p + b), u);
      in_order<kAdjacent>(u, x);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] += offset;
  }
  from_order<kAdjacent>(x, w);
}

// Sum over the eight lanes of a row; all of them get it.
MSA_DEV float row_sum(float x, unsigned lanes = 0xffffffffu) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) x += __shfl_xor_sync(lanes, x, o);
  return x;
}
MSA_DEV float squares(const Values& v) {
  uint64_t s = f2_mul(v.a[0], v.a[0]), t = f2_mul(v.b[0], v.b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    s = f2_fma(v.a[i], v.a[i], s);
    t = f2_fma(v.b[i], v.b[i], t);
  }
  float lo, hi;
  f2_unpack(f2_add(s, t), lo, hi);
  return lo + hi;
}
MSA_DEV void times(Values& v, float x) {
  const uint64_t xx = f2_pack(x, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.a[i] = f2_mul(v.a[i], xx);
    v.b[i] = f2_mul(v.b[i], xx);
  }
}
MSA_DEV void times(Values& v, const Values& w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.a[i] = f2_mul(v.a[i], w.a[i]);
    v.b[i] = f2_mul(v.b[i], w.b[i]);
  }
}

// The lane's pairs turned by the angles of a table's row; kBack: the other way.
template <bool kBack>
MSA_DEV void rotate(Values& v, const float4* row, int j) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 x = row[i * 8 + j];
    const uint64_t c = f2_pack(x.x, x.y), s = f2_pack(x.z, x.w);
    const uint64_t a = v.a[i], b = v.b[i];
    if constexpr (kBack) {
      v.a[i] = f2_fma(a, c, f2_mul(b, s));
      v.b[i] = f2_sub(f2_mul(b, c), f2_mul(a, s));
    } else {
      v.a[i] = f2_sub(f2_mul(a, c), f2_mul(b, s));
      v.b[i] = f2_fma(b, c, f2_mul(a, s));
    }
  }
}

// Rows whose squares leave fp32's range (they have an element above 2^60) are scaled by
// this first: of any bf16 values 128 squares then sum to 2^127 at most, and what a small
// value beside a large one loses, 2^-82, is 2^-139 of its normed one.
constexpr float kDown = 3.3881317890172014e-21f;  // 2^-68

// A row's values times its weights, and what is left of the norm, 1 / sqrt(mean(x^2) +
// eps) (1 without a norm), which waits for the other lanes while the values are
// turned.
// turn: what is done to the weighted values meanwhile; again(ua, ub): the row once
// more.  Whole warps call it.
template <bool kAdjacent, class Turn, class Again>
MSA_DEV float weigh(uint4 ua, uint4 ub, const Values& w, bool norm, float eps, Values& v, Turn turn, Again again) {
  unpack<kAdjacent>(ua, ub, v);
  float sum = row_sum(squares(v));
  times(v, w);
  turn(v);
  if (__any_sync(0xffffffffu, norm && !(sum < kInf))) {
    const bool far = norm && !(sum < kInf);
    again(ua, ub);
    unpack<kAdjacent>(ua, ub, v);
    times(v, far ? kDown : 1.f);
    const float scaled = row_sum(squares(v));
    if (far) {
      sum = scaled;
      eps = 0.f;  // no more than 2^-21 of the mean there
    }
    times(v, w);
    turn(v);
  }
  return norm ? rsqrtf(fmaf(sum, 1.f / 128.f, eps)) : 1.f;
}
// One row: normed, and turned by the angles at `row` if `turn` (this lane's dims
// are: a turn by nothing would carry infinities from pair to pair).
template <bool kAdjacent, class Again>
MSA_DEV void norm_rotate(uint4& ua, uint4& ub, const Values& w, const float4* row, int j, bool norm, bool turn,
                         float eps, Again again) {
  Values v;
  const float r = weigh<kAdjacent>(
      ua, ub, w, norm, eps, v,
      [&](Values& x) {
        if (turn) rotate<false>(x, row, j);
      },
      again);
  times(v, r);
  pack<kAdjacent>(v, ua, ub);
}

// Host side.
int check_problem(const msa_rope_problem* p);
inline const Angles angles_of(const msa_rope_problem* p, const int32_t* positions, int32_t* status) {
  return Angles{p->pairs, positions, p->rotary_dim, p->num_axes, p->cos_scale, status};
}

// How the rows of a call's tensors are cut: a unit is four heads (of the tensors'
// heads one after the other) of a token, a warp's share; `units` of them to a
// CTA's warps, `groups` CTAs side by side; with few units, `phases` warps take
// tokens in turn.  A CTA keeps its heads, and so their weights, and takes one of
// `slices` equal shares of the tokens, every slices-th one, as many as `warps` of an
// SM hold.
struct Cut {
  int groups, units, phases, slices;
  void at_most(int64_t tokens, int64_t per_cta) {
    const int64_t least = (tokens + per_cta - 1) / per_cta;
    if (slices < least) slices = (int)least;
  }
  int threads() const { return 32 * (units * phases + 1); }  // and a warp for the angles
};
inline Cut cut_rows(int64_t heads, int64_t tokens, int64_t sms, int warps, int most_units) {
  const int64_t u = (heads + 3) / 4;
  Cut c;
  c.groups = (int)((u + most_units - 1) / most_units);
  c.units = (int)((u + c.groups - 1) / c.groups);
  c.phases = most_units / c.units;
  const int64_t most = sms * (warps / (c.units * c.phases + 1)) / c.groups;
  c.slices = (int)(tokens < most ? tokens : most > 1 ? most : 1);
  return c;
}
// Rows in and out, by CTAs of (slice of the tokens, group of heads).
struct RowsArgs {
  Tensor t[kTensors];
  uint16_t* y[kTensors];
  int64_t y_token[kTensors], y_head[kTensors];
  Angles an;
  float eps, offset;
  int T, heads;  // of all tensors
  int zero;      // rows of padding are zeros
  Cut cut;
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

MSA_DEV void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
MSA_DEV void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
MSA_DEV void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

// Rows on their way to a warp: four rows a stage, in whole lines, whatever dims a
// lane then takes (two lines of 128 bytes a row for any R; the lanes' own granules
// are 64 bytes apart and less for R < 128).  The bytes in flight take no registers.
// The upper granules are stored with their halves exchanged, so that the lanes'
// reads of R = 64 meet no bank twice.
constexpr int kStages = 4;  // a power of two
struct Stage {
  uint4 row[4][16];
};
MSA_DEV int granule_slot(int g) { return g ^ (g >> 1 & 4); }
MSA_DEV void copy_row(Stage& s, const uint16_t* row, int lane) {
  const int r = lane >> 3, j = lane & 7;
  copy16(&s.row[r][granule_slot(j)], row + 8 * j);
  copy16(&s.row[r][granule_slot(j + 8)], row + 64 + 8 * j);
}
// Two tables in turn: the CTA's warps behind those of the rows (one, as a rule) fill
// one while the others use the other.
// (Filled by all warps, each its part, between a barrier and the next: 32k tokens x
// 68 heads 190 us, with registers that spill, against 180.)
// padding(token): what they do about a token that is padding.
template <bool kAdjacent, class Padding>
MSA_DEV bool fill_tables(const Angles& a, Table<kTile> (&tab)[2], bool bad, int before, int64_t first, int n,
                         int apart, Padding padding) {
  const Filler<kAdjacent> filler(a, threadIdx.x - before, blockDim.x - before);
  auto fill = [&](int k) {
    if (k * kTile < n)
      filler.fill(tab[k & 1], a, first + (int64_t)k * kTile * apart, min(n - k * kTile, kTile), apart);
  };
  fill(0);
  if (__syncthreads_or(bad)) return false;
  for (int k = 0; k * kTile < n; ++k) {
    fill(k + 1);
    for (int i = 0; i < min(n - k * kTile, kTile); ++i)
      if (!tab[k & 1].live[i]) padding(first + (int64_t)(k * kTile + i) * apart);
    __syncthreads();
  }
  return true;
}
// Rows of `heads` heads from hh on become zeros, by `threads` threads of which this is
// `thread`; row(hh) is where a head's begins.
template <class Row>
MSA_DEV void zero_heads(int hh, int heads, int thread, int threads, Row row) {
  for (int u = thread; u < heads * 16; u += threads)
    *reinterpret_cast<uint4*>(row(hh + (u >> 4)) + 8 * (u & 15)) = make_uint4(0, 0, 0, 0);
}
struct RowsShared {
  Table<kTile> tab[2];
  Stage ring[kRowWarps][kStages];
};

// bad: the status was set before the call.  The CTA decides on it at its first
// barrier, so that the load does not hold up the others, and as a whole: another
// CTA may set the status between two warps' reads.
template <bool kAdjacent>
MSA_DEV void rows_block(const RowsArgs& a, int block, bool bad, RowsShared& s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, j = lane & 7;
  const int slice = block / a.cut.groups, group = block - slice * a.cut.groups;
  const int apart = a.cut.slices, n = (a.T - slice + apart - 1) / apart;
  if (warp >= a.cut.units * a.cut.phases) {
    const int before = 32 * a.cut.units * a.cut.phases;
    fill_tables<kAdjacent>(a.an, s.tab, bad, before, slice, n, apart, [&](int64_t t) {
      if (!a.zero) return;
      const int hh = group * a.cut.units * 4, heads = min(a.heads - hh, a.cut.units * 4);
      zero_heads(hh, heads, tid - before, blockDim.x - before, [&](int h) {
        int head;
        const int k = tensor_of(a, h, head);
        return a.y[k] + t * a.y_token[k] + head * a.y_head[k];
      });
    });
    return;
  }
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
  const uint16_t* x = t.x + first * t.x_token + head * t.x_head;  // of the next row to copy
  uint16_t* y = a.y[k] + first * a.y_token[k] + head * a.y_head[k];
  Stage* ring = s.ring[warp];
  int ahead = phase;  // its token
  auto copy = [&](int stage) {
    if (live && ahead < n) copy_row(ring[stage], x, lane);
    copies_commit();
    ahead += phases;
    x += x_step;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) copy(i);
  const bool norm = t.flags & MSA_ROPE_NORM, turn = turns(t, j, a.an.R);
  Values w;
  load_weights<kAdjacent>(t, head, da, db, a.offset, w);
  if (__syncthreads_or(bad)) {  // the first table is there
    copies_wait<0>();
    return;
  }
  int stage = 0, i = phase;
  for (int at = 0, table = 0; at < n; at += kTile, ++table) {
    const Table<kTile>& tab = s.tab[table & 1];
    for (; i < min(at + kTile, n); i += phases) {
      copies_wait<kStages - 2>();
      __syncwarp();  // the lanes' copies have landed; the stage before has been read
      const uint4* row = ring[stage].row[lane >> 3];
      uint4 ua = row[sa], ub = row[sb];
      copy((stage + kStages - 1) & (kStages - 1));
      stage = (stage + 1) & (kStages - 1);
      if (tab.live[i - at]) {
        norm_rotate<kAdjacent>(ua, ub, w, tab.cs[i - at], j, norm, turn, a.eps, [&](uint4& xa, uint4& xb) {
          xa = row[sa];  // the stage is not copied to before the next row
          xb = row[sb];
        });
        if (live) {
          *reinterpret_cast<uint4*>(y + da) = ua;
          *reinterpret_cast<uint4*>(y + db) = ub;
        }
      }
      y += y_step;
    }
    __syncthreads();  // it has been read, the next one is there
  }
}

}  // namespace rope
}  // namespace msa
