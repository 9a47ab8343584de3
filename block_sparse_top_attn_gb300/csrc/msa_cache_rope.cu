// Serving: a step's tensors normed, rotated and appended to the 4-bit cache in one
// launch (msa_rope.cuh has a row's arithmetic, msa_cache.cuh the cache's).
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "msa_rope.cuh"

namespace msa {
namespace rope {

constexpr int kKvTile = 32;  // most tokens of a tile of K and V
constexpr int kIndexRows = kThreads / 8;  // rows of a pass
constexpr int kIndexTokens = 64;          // whose angles are made at once
constexpr int kIndexHeads = 2;            // heads of index keys that a CTA takes at once

struct AppendRopeArgs {
  RowsArgs q;    // q and q_index: rows in and out
  Tensor k, ki;  // their `end` is not used
  const uint16_t* v;
  int64_t v_token, v_head;
  const int64_t* slot_map;
  const int32_t *cu_tokens, *chunks;
  uint8_t* cache;
  uint16_t *index_tail, *index_pool;
  int T, H, B, R, NC;
  int positions;         // max_blocks * B: a request's most tokens
  int64_t slots;         // num_pages * B
  float k_mul, v_mul;    // 2^-exp
  int index_blocks, kv_blocks;  // CTAs of index keys, of K and V; the others take q's rows
  uint64_t kv_turns;            // takes_turn
  int index_heads, index_groups, index_chunks;  // heads of a CTA, CTAs of a chunk's heads, chunks of a CTA
  int kv_tile, kv_groups, kv_heads;  // tokens of a tile; groups of heads side by side, heads of a group
  int32_t* status;
};

// ---------------------------------------------------------------------------
// K: codes of the exact value
// ---------------------------------------------------------------------------
// The cache keeps a value by the interval it lies in, so an error of fp32 counts
// only next to a border, and there by a whole code.  With amp = |a cos| + |b sin| and
// u = 2^-24, fp32 forms y to within 21 u amp: 12 u for the weighted a and b and the
// inverse rms (the sum of 128 squares in chains of 4 and 6 more additions, halved by
// the root; rsqrtf 2 ulp; the weight's offset and products), 9 u for the cosine (6), its
// scale, the products and the sum.  The code's quotient adds 4 u, and the eps that is
// left out of rows scaled by kDown up to 4 u: 29 u in all.  A group with a value (or a
// scale) nearer to a border than 32 u amp is done again exactly, from the inputs, behind
// the others: one group in 1,000, which costs a step of 64 tokens 0.7 us of 5.1.
constexpr float kUlps = 32.f;

// Exact enough means pairs of fp32, hi + lo, by the error-free sums and products of
// Knuth and Dekker: an fp64 instruction takes a warp 70 cycles here, a product of
// pairs 16 (a step of 64 tokens was 7.7 us with fp64, and 6.0 with pairs).  Errors stay
// below 2^-38 of amp; what is nearer to a border than that is one value in 10^10.
struct Split {
  float hi, lo;
};
// x as a pair, for constants.
__host__ __device__ constexpr Split parts(double x) { return Split{(float)x, (float)(x - (double)(float)x)}; }
MSA_DEV Split sum_of(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return Split{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
MSA_DEV Split sum_of(Split a, Split b) {
  Split s = sum_of(a.hi, b.hi);
  s.lo += a.lo + b.lo;
  return s;
}
MSA_DEV Split product(Split a, Split b) {
  const float p = __fmul_rn(a.hi, b.hi);
  return Split{p, fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, __fmaf_rn(a.hi, b.hi, -p)))};
}
// k + z * x, |k| above the product.
MSA_DEV Split horner(Split k, Split z, Split x) {
  const Split p = product(z, x);
  const float s = __fadd_rn(k.hi, p.hi);
  return Split{s, __fadd_rn(__fsub_rn(k.hi, s), p.hi) + (p.lo + k.lo)};
}

// Cosine and sine of a fraction of a turn: the quarter turns are taken off exactly, and
// the Taylor polynomials do for the eighth that is left (48 of its bits).
MSA_DEV void cos_sin_split(uint64_t turn, Split& c, Split& s) {
  const uint64_t shifted = turn + (1ull << 61);
  const int64_t rest = (int64_t)(turn - (shifted & (3ull << 62)));
  const uint64_t size = rest < 0 ? 0 - (uint64_t)rest : (uint64_t)rest;  // up to 2^61
  const float a = (float)(uint32_t)(size >> 37), b = (float)((uint32_t)(size >> 13) & 0xFFFFFFu);
  constexpr Split unit = parts(4.681337853654911e-08);  // pi 2^-26
  Split x;
  x.hi = __fmul_rn(a, unit.hi);
  x.lo = fmaf(b, 2.7902947984069054e-15f, fmaf(a, unit.lo, __fmaf_rn(a, unit.hi, -x.hi)));  // pi 2^-50
  if (rest < 0) x = Split{-x.hi, -x.lo};
  const Split z = product(x, x);
  constexpr Split one = parts(1.0), s3 = parts(-1.0 / 6), s5 = parts(1.0 / 120), s7 = parts(-1.0 / 5040);
  constexpr Split c2 = parts(-0.5), c4 = parts(1.0 / 24), c6 = parts(-1.0 / 720);
  Split sn{fmaf(z.hi, fmaf(z.hi, 1.f / 6227020800.f, -1.f / 39916800.f), 1.f / 362880.f), 0.f};
  Split cs{fmaf(z.hi, fmaf(z.hi, 1.f / 479001600.f, -1.f / 3628800.f), 1.f / 40320.f), 0.f};
  sn = product(x, horner(one, z, horner(s3, z, horner(s5, z, horner(s7, z, sn)))));
  cs = horner(one, z, horner(c2, z, horner(c4, z, horner(c6, z, cs))));
  const int quarter = (int)(shifted >> 62);
  c = quarter & 1 ? sn : cs;
  s = quarter & 1 ? cs : sn;
  if (quarter == 1 || quarter == 2) c = Split{-c.hi, -c.lo};
  if (quarter >= 2) s = Split{-s.hi, -s.lo};
}
// factor / sqrt(m), 2^-100 <= m: a step of Newton's method from the fp32 root of m
// times an even power of two.
MSA_DEV Split inverse_root(Split m, float factor) {
  const int e = (int)(__float_as_uint(m.hi) >> 23) - 127 & ~1;
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
  const float h = m.hi * down, l = m.lo * down, r = rsqrtf(h), p = __fmul_rn(r, r);
  // 1 - m r^2
  const float t = fmaf(-l, p, fmaf(-h, __fmaf_rn(r, r, -p), fmaf(-h, p, 1.f)));
  factor *= __uint_as_float((uint32_t)(127 - e / 2) << 23);
  return Split{r * factor, r * 0.5f * t * factor};
}

// Dim `d` of a K row (in shared memory) times `scale` and its weight and rotated; what
// is left of the norm is the row's inverse rms.
template <bool kAdjacent>
MSA_DEV Split turned_dim(const AppendRopeArgs& a, const uint4* row, float scale, int head, int64_t t, int d) {
  auto weighted = [&](int i) {
    const uint32_t x = reinterpret_cast<const uint16_t*>(row + granule_slot(i >> 3))[i & 7];
    const Split v{__uint_as_float(x << 16) * scale, 0.f};
    if (!(a.k.flags & MSA_ROPE_NORM) || !a.k.w) return v;
    const int64_t at = (a.k.flags & MSA_ROPE_PER_HEAD ? head * 128 : 0) + i;
    const float w = a.k.flags & MSA_ROPE_WEIGHT_FP32
                        ? static_cast<const float*>(a.k.w)[at]
                        : __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.k.w)[at] << 16);
    return product(v, sum_of(w, a.q.offset));
  };
  const int R = a.q.an.R;
  const Split own = weighted(d);
  if (!(a.k.flags & MSA_ROPE_ROTATE) || d >= R) return own;
  const bool second = kAdjacent ? d & 1 : d >= R / 2;
  const int p = kAdjacent ? d >> 1 : second ? d - R / 2 : d;
  const int partner = kAdjacent ? d ^ 1 : second ? p : d + R / 2;
  Split s, c;
  cos_sin_split(turn_of(a.q.an, load_pair(a.q.an, p), t), c, s);
  if (!second) s = Split{-s.hi, -s.lo};
  return product(sum_of(product(own, c), product(weighted(partner), s)), Split{a.q.an.scale, 0.f});
}

MSA_DEV float scale_value(uint32_t s8) {
  return __half2float(__ushort_as_half((uint16_t)(cache::e4m3x2_to_half(s8) & 0xFFFFu)));
}

// A pair whose second part is no more than a rounding of the first lies above a border
// that fp32 holds, or on it and `up`.
MSA_DEV bool beyond(const Split& x, float border, bool up) {
  return x.hi > border || (x.hi == border && (x.lo > 0.f || (x.lo == 0.f && up)));
}
// e4m3 scale of a group whose largest magnitude (times 2^-exp) is `amax`.
MSA_DEV uint32_t exact_scale(const Split& amax) {
  auto above = [&](uint32_t lo) {  // of lo and lo + 1, the upper one is nearer (a tie goes to the even one)
    const uint32_t h = cache::e4m3x2_to_half(lo | (lo + 1) << 8);  // six times their middle has 8 bits at most
    return beyond(amax, 3.f * (__half2float(__ushort_as_half((uint16_t)(h & 0xFFFFu))) +
                               __half2float(__ushort_as_half((uint16_t)(h >> 16)))), lo & 1);
  };
  uint16_t s2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.f), "f"(amax.hi * (1.f / 6.f)));
  uint32_t s8 = s2 & 0xFFu;  // the scale or one beside it
  while (s8 < 126 && above(s8)) ++s8;
  while (s8 > 0 && !above(s8 - 1)) --s8;
  return s8;
}
MSA_DEV uint32_t exact_code(const Split& m, bool negative, float s) {
  if (!(s > 0.f)) return 0;
  const uint32_t c = beyond(m, 0.25f * s, false) + beyond(m, 0.75f * s, true) + beyond(m, 1.25f * s, false) +
                     beyond(m, 1.75f * s, true) + beyond(m, 2.5f * s, false) + beyond(m, 3.5f * s, true) +
                     beyond(m, 5.f * s, false);
  return c && negative ? c | 8u : c;
}

MSA_DEV uint8_t* cache_tile(const AppendRopeArgs& a, int64_t slot, int head, int& tok) {
  const int lb = a.B == 128 ? 7 : 6;  // log2 of the block
  const int off = (int)(slot & (a.B - 1));
  tok = off % cache::kTile;
  return a.cache + cache::tile_index(slot >> lb, head, a.H, a.B / cache::kTile, off / cache::kTile) *
                       cache::kTileBytes;
}

// Codes and scale of 16 dims from dim0 on of token t's K row, by half a warp, a lane a
// dim (the other half does the same).
template <bool kAdjacent>
MSA_DEV void exact_group(const AppendRopeArgs& a, const uint4* row, int64_t slot, int64_t t, int head, int dim0) {
  const int lane = threadIdx.x & 15;
  Split r{a.k_mul, 0.f};
  float scale = 1.f;
  if (a.k.flags & MSA_ROPE_NORM) {
    const uint4 u = row[granule_slot(lane)];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    auto sum = [&]() {  // of the squares of the row times scale; a square is exact
      Split s{0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16) * scale;
        s = sum_of(s, Split{__fmul_rn(x, x), 0.f});
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1)
        s = sum_of(s, Split{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
      return s;
    };
    Split s = sum();
    float eps = a.q.eps;
    if (__any_sync(0xffffffffu, !(s.hi < kInf))) {  // all lanes have the same sum
      scale = kDown;
      eps = eps * scale * scale;
      s = sum();
    }
    Split m = sum_of(s.hi * (1.f / 128.f), eps);
    m.lo += s.lo * (1.f / 128.f);
    r = inverse_root(m, a.k_mul);
  }
  const Split turned = product(turned_dim<kAdjacent>(a, row, scale, head, t, dim0 + lane), r);
  Split own = sum_of(turned.hi, turned.lo);
  // What saturates in any case is cut off: fp32 may not have held it, and then its second part is NaN.
  constexpr float kMost = 1.8446744073709552e19f;  // 2^64
  if (!(fabsf(turned.hi) < kMost)) own = Split{copysignf(kMost, turned.hi), 0.f};
  const bool negative = own.hi < 0.f;
  own = Split{fabsf(own.hi), negative ? -own.lo : own.lo};
  Split m = own;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const Split other{__shfl_xor_sync(0xffffffffu, m.hi, o), __shfl_xor_sync(0xffffffffu, m.lo, o)};
    if (other.hi > m.hi || (other.hi == m.hi && other.lo > m.lo)) m = other;
  }
  const uint32_t s8 = exact_scale(m);
  uint32_t codes = exact_code(own, negative, scale_value(s8)) << 4 * (lane & 7);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) codes |= __shfl_xor_sync(0xffffffffu, codes, o);
  int tok;
  uint8_t* out = cache_tile(a, slot, head, tok);
  if ((lane & 7) == 0)
    *reinterpret_cast<uint32_t*>(out + cache::OFF_KC + tok * cache::kRowBytes + (dim0 >> 1) + (lane >> 1)) = codes;
  if (lane == 0) out[cache::OFF_KS + tok * cache::kScales + (dim0 >> 4)] = (uint8_t)s8;
}

// Half of a scale group: a lane's eight values, its neighbour's the rest.
struct Half {
  uint32_t codes, scale;  // codes of the lane's eight, the group's scale
  bool doubt;             // fp32 does not tell
};
MSA_DEV uint32_t codes8(const uint64_t (&q)[4]) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(q[i], x[2 * i], x[2 * i + 1]);
  return cache::e2m1x8(x);
}
// Rounds with the error to either side: where the results differ, there is a border
// between them.  exact: the values are the inputs themselves, and rounded by
// quantize16's rule.
MSA_DEV Half round_half(const float* v, float amp, float mul, bool exact) {
  Half h;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  amp = fmaxf(amp, __shfl_xor_sync(0xffffffffu, amp, 1));  // by every lane, whether it is exact or not
  const float amax = __uint_as_float(m) * mul;
  constexpr float kSixth = 1.f / 6.f, kError = kUlps * 5.9604644775390625e-8f;  // 2^-24
  const float t0 = amax * kSixth;
  const float t = amax < 4096.f ? __fmaf_rn(__fmaf_rn(-6.f, t0, amax), kSixth, t0) : t0;
  // t is two roundings from amax / 6
  const float dt = exact ? 0.f : fmaf(amp * mul, kError * kSixth, t * 2.384185791015625e-7f);  // 2^-22
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(t + dt), "f"(fmaxf(t - dt, 0.f)));
  h.scale = two & 0xFFu;
  h.codes = 0;
  h.doubt = h.scale != (uint32_t)two >> 8;
  if (m >= 0x7F800000u || mul != mul) {  // a NaN scale: the group reads back as NaN
    h.scale = 0x7F;
    h.doubt = false;
  } else if (h.scale) {
    const float inv = __frcp_rn(scale_value(h.scale)) * mul;
    // the quotient's own roundings: 4 u of it, which is no more than amp
    const float dq = exact ? 0.f : fmaf(amp * inv, kError, 9.5367431640625e-7f);
    const uint64_t inv2 = f2_pack(inv, inv), up = f2_pack(dq, dq), down = f2_pack(-dq, -dq);
    const uint64_t snap = f2_pack(768.f, 768.f);
    uint64_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t x = f2_pack(v[2 * i], v[2 * i + 1]);
      const uint64_t q = exact ? f2_sub(f2_fma(x, inv2, snap), snap) : f2_mul(x, inv2);
      lo[i] = f2_add(q, down);
      hi[i] = f2_add(q, up);
    }
    h.codes = codes8(lo);
    h.doubt |= h.codes != codes8(hi);
  }
  return h;
}

// Largest |a cos| + |b sin| of each granule of a weighted row.
template <bool kAdjacent>
MSA_DEV void amplitudes(const Values& v, const float4* row, int j, bool turn, float (&amp)[2]) {
  amp[0] = amp[1] = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 x = turn ? row[i * 8 + j] : make_float4(1.f, 1.f, 0.f, 0.f);
    float a0, a1, b0, b1;
    f2_unpack(v.a[i], a0, a1);
    f2_unpack(v.b[i], b0, b1);
    const float fa = fmaxf(fmaf(fabsf(a0), fabsf(x.x), fabsf(b0 * x.z)), fmaf(fabsf(a1), fabsf(x.y), fabsf(b1 * x.w)));
    const float fb = fmaxf(fmaf(fabsf(b0), fabsf(x.x), fabsf(a0 * x.z)), fmaf(fabsf(b1), fabsf(x.y), fabsf(a1 * x.w)));
    amp[kAdjacent ? i >> 1 : 0] = fmaxf(amp[kAdjacent ? i >> 1 : 0], fa);
    amp[kAdjacent ? i >> 1 : 1] = fmaxf(amp[kAdjacent ? i >> 1 : 1], fb);
  }
}

// K and V of a tile of tokens and a group of heads, four rows of each a pass; the next
// pass's are on their way meanwhile.
struct KvShared {
  Table<kKvTile> tab;
  Stage ring[kWarps][2][2];  // K and V
};
template <bool kAdjacent>
MSA_DEV void kv_block(const AppendRopeArgs& a, int block, bool bad, KvShared& s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, j = lane & 7;
  const int tile = block / a.kv_groups, group = block - tile * a.kv_groups;
  const int64_t t0 = (int64_t)tile * a.kv_tile;
  const int n = (int)min((int64_t)a.kv_tile, a.T - t0);
  const int h0 = group * a.kv_heads, hn = min(a.kv_heads, a.H - h0);
  const bool norm = a.k.flags & MSA_ROPE_NORM, turn = turns(a.k, j, a.q.an.R);
  const bool exact = !norm && !turn;  // the lane's values are its inputs
  int da, db;
  lane_dims(j, a.q.an.R, da, db);
  const int sa = granule_slot(da >> 3), sb = granule_slot(db >> 3);
  const int shift = 31 - __clz(a.kv_tile);
  // four tokens of a head side by side in a warp: their cache rows follow one another
  int64_t slot = -1, next_slot;
  int first = 0, next_first;  // position
  auto load = [&](int base, int stage) {
    const int u = base + (lane >> 3), i = u & (a.kv_tile - 1), hs = u >> shift;
    next_slot = -1;
    next_first = 0;
    if (i < n && hs < hn) {
      const int64_t t = t0 + i, h = h0 + hs;
      next_slot = a.slot_map[t];
      next_first = a.q.an.positions[t * a.q.an.A];
      copy_row(s.ring[warp][stage][0], a.k.x + t * a.k.x_token + h * a.k.x_head, lane);
      copy_row(s.ring[warp][stage][1], a.v + t * a.v_token + h * a.v_head, lane);
    }
    copies_commit();
  };
  load(warp * 4, 0);  // ahead of the angles: one chain of loads for both
  Values w;
  load_weights<kAdjacent>(a.k, h0, da, db, a.q.offset, w);
  Filler<kAdjacent>(a.q.an, tid, kThreads).fill(s.tab, a.q.an, t0, n);
  if (__syncthreads_or(bad)) {
    copies_wait<0>();
    return;
  }
  const Table<kKvTile>& tab = s.tab;
  int stage = 0;
  for (int base = warp * 4; base < hn << shift; base += kThreads / 8, stage ^= 1) {
    const int u = base + (lane >> 3), i = u & (a.kv_tile - 1), hs = u >> shift, h = h0 + hs;
    const int64_t t = t0 + i;
    slot = next_slot;
    first = next_first;
    __syncwarp();  // the next stage has been read
    load(base + kThreads / 8, stage ^ 1);
    if (a.k.flags & MSA_ROPE_PER_HEAD) load_weights<kAdjacent>(a.k, hs < hn ? h : h0, da, db, a.q.offset, w);
    bool live = i < n && hs < hn;
    if (live && (slot < 0 || slot >= a.slots || first < 0)) {
      if (slot != -1) set_status(a.status, MSA_ERR_INVALID_CACHE);
      live = false;
    }
    copies_wait<1>();
    __syncwarp();  // the lanes' copies have landed
    const uint4 *row = s.ring[warp][stage][0].row[lane >> 3], *vrow = s.ring[warp][stage][1].row[lane >> 3];
    auto read = [&](uint4& xa, uint4& xb) {  // padding may hold anything
      xa = live ? row[sa] : make_uint4(0, 0, 0, 0);
      xb = live ? row[sb] : make_uint4(0, 0, 0, 0);
    };
    uint4 ua, ub;
    read(ua, ub);
    Values val;
    float amp[2], v[16];
    const float r = weigh<kAdjacent>(
        ua, ub, w, norm, a.q.eps, val,
        [&](Values& x) {
          amplitudes<kAdjacent>(x, tab.cs[i], j, turn, amp);
          if (turn) rotate<false>(x, tab.cs[i], j);
        },
        read);
    in_order<kAdjacent>(val, v);
    // the inverse rms goes into the factor of the rounding
    const float mul = r * a.k_mul;
    const Half ha = round_half(v, amp[0], mul, exact), hb = round_half(v + 8, amp[1], mul, exact);
    if (live) {
      int tok;
      uint8_t* out = cache_tile(a, slot, h, tok);
      *reinterpret_cast<uint32_t*>(out + cache::OFF_KC + tok * cache::kRowBytes + (da >> 1)) = ha.codes;
      *reinterpret_cast<uint32_t*>(out + cache::OFF_KC + tok * cache::kRowBytes + (db >> 1)) = hb.codes;
      // of the two lanes of a group, one stores the first granules' scale, one the second's
      out[cache::OFF_KS + tok * cache::kScales + ((j & 1 ? db : da) >> 4)] = (uint8_t)(j & 1 ? hb.scale : ha.scale);
      const uint4 v0 = vrow[granule_slot(2 * j)], v1 = vrow[granule_slot(2 * j + 1)];
      const uint32_t vw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
      uint2 vc;
      const uint32_t vs = cache::quantize16(vw, a.v_mul, vc);
      *reinterpret_cast<uint2*>(out + cache::OFF_VC + cache::v_code_offset(tok, j)) = vc;
      out[cache::OFF_VS + j * cache::kTile + tok] = (uint8_t)vs;
    }
    // Groups in doubt, by their first lane.
    auto groups = [&](bool doubt) {  // one of a group's lanes may see it, or both
      const unsigned m = __ballot_sync(0xffffffffu, live && doubt);
      return (uint64_t)((m | m >> 1) & 0x55555555u);
    };
    uint64_t left = groups(ha.doubt) | groups(hb.doubt) << 32;
    if (left) __syncwarp();  // what is there of the groups is overwritten
    for (; left; left &= left - 1) {
      const int group = __ffsll(left) - 1, from = group & 31;
      const int dim0 = __shfl_sync(0xffffffffu, group < 32 ? da : db, from);
      const int64_t at = __shfl_sync(0xffffffffu, slot, from), token = __shfl_sync(0xffffffffu, t, from);
      const int head = __shfl_sync(0xffffffffu, h, from);
      exact_group<kAdjacent>(a, s.ring[warp][stage][0].row[from >> 3], at, token, head, dim0);
    }
  }
}

// ---------------------------------------------------------------------------
// index keys
// ---------------------------------------------------------------------------
// A CTA takes some heads of up to eight chunks, a warp each.  A warp stores its
// chunk's rows to the tail by itself (a decode step's one token, the last tokens of
// a prompt).  A chunk that completes a block is the CTA's work, after that.  All of a
// warp's or CTA's loads are under way together, the angles made behind them.
struct IndexShared {
  union {
    Table<kChunk> own[kWarps];
    Table<kIndexTokens> tab;
  };
  uint4 rows[kIndexTokens][kIndexHeads][16];  // as they come, then normed and rotated; eight tokens a warp, or the CTA's
  int average[kWarps];
};

// Rows wait in shared memory, where a lane copies its own granules and reads them back
// itself, and take no registers while the angles are made.
constexpr int kIndexSteps = 4;  // of a row for each eight lanes
static_assert(kIndexTokens * kIndexHeads <= kIndexSteps * kIndexRows && kChunk * kIndexHeads <= kIndexSteps * 4 &&
                  kChunk * kWarps <= kIndexTokens,
              "a CTA's rows of 64 tokens and a warp's of a chunk");

template <bool kAdjacent>
MSA_DEV void store_tail(const AppendRopeArgs& a, const cache::IndexPlan& x, int h0, int hn, int warp, IndexShared& s) {
  const int lane = threadIdx.x & 31, j = lane & 7, n = x.p1 - x.p0;  // at most a chunk
  const int64_t hs = (int64_t)a.H * 128, t0 = x.cu0 + x.p0 - x.past;
  const bool norm = a.ki.flags & MSA_ROPE_NORM, turn = turns(a.ki, j, a.q.an.R);
  Table<kChunk>& tab = s.own[warp];
  auto* rows = s.rows + warp * kChunk;
  int da, db;
  lane_dims(j, a.q.an.R, da, db);
  for (int h1 = h0; h1 < h0 + hn; h1 += kIndexHeads) {
    // row r is token r / heads and head r % heads: the lane's head is the same in every step
    const int shift = min(kIndexHeads, h0 + hn - h1) - 1, sub = lane >> 3 & shift, h = h1 + sub;
#pragma unroll
    for (int e = 0; e < kIndexSteps; ++e) {
      const int i = (e * 4 + (lane >> 3)) >> shift;
      if (i < n) {
        const uint16_t* src = a.ki.x + (t0 + i) * a.ki.x_token + h * a.ki.x_head;
        copy16(&rows[i][sub][da >> 3], src + da);
        copy16(&rows[i][sub][db >> 3], src + db);
      }
    }
    copies_commit();
    Values w;
    load_weights<kAdjacent>(a.ki, h, da, db, a.q.offset, w);
    if (h1 == h0) {
      Filler<kAdjacent>(a.q.an, lane, 32).fill(tab, a.q.an, t0, n);
      __syncwarp();
    }
    copies_wait<0>();
    uint16_t* tail = a.index_tail + ((int64_t)x.r * 2 + (x.open & 1)) * a.B * hs + h * 128;
#pragma unroll 1
    for (int e = 0; e * 4 < n << shift; ++e) {
      const int i = (e * 4 + (lane >> 3)) >> shift, row = i < n ? i : 0;  // a row of its own, or any
      uint4 ua, ub;
      auto read = [&](uint4& xa, uint4& xb) {
        xa = i < n ? rows[row][sub][da >> 3] : make_uint4(0, 0, 0, 0);
        xb = i < n ? rows[row][sub][db >> 3] : make_uint4(0, 0, 0, 0);
      };
      read(ua, ub);
      norm_rotate<kAdjacent>(ua, ub, w, tab.cs[row], j, norm, turn, a.q.eps, read);
      if (i < n) {
        uint16_t* out = tail + ((x.p0 + i) & (a.B - 1)) * hs;
        *reinterpret_cast<uint4*>(out + da) = ua;
        *reinterpret_cast<uint4*>(out + db) = ub;
      }
    }
  }
}

// A chunk that completes a block, by the CTA: 64 tokens of the block at a time, those
// of earlier calls as they are in the tail, those of this call normed and rotated, go
// to shared memory and are added in the order of the tokens, so that the mean does not
// depend on how a prompt was cut.
template <bool kAdjacent>
MSA_DEV void average_heads(const AppendRopeArgs& a, const cache::IndexPlan& x, int h0, int hn,
                           const Filler<kAdjacent>& filler, bool& filled, IndexShared& s) {
  const int tid = threadIdx.x, g = tid >> 3, j = tid & 7;
  const int64_t hs = (int64_t)a.H * 128;
  const bool norm = a.ki.flags & MSA_ROPE_NORM, turn = turns(a.ki, j, a.q.an.R);
  int da, db;
  lane_dims(j, a.q.an.R, da, db);
  const int shift = hn - 1, sub = g & shift, h = h0 + sub;
  const uint16_t* src = a.ki.x + h * a.ki.x_head;
  uint16_t* tail = a.index_tail + (int64_t)x.r * 2 * a.B * hs + h * 128;
  const int64_t slot = x.last >= 0 ? a.slot_map[x.last] : -1;
  const bool average = slot >= 0 && slot < a.slots;  // else reported by the rows' own CTAs, or left out
  const int olds = max(0, x.cu0 - (x.last - (a.B - 1)));  // tokens of the block from earlier calls
  const int64_t block_t = x.last - (a.B - 1);  // token of the block's first position, were it of this call
  float lo = 0.f, hi = 0.f;
  // The segments of 64 tokens to average, then those to store (the rows of the incomplete block, behind the barriers
  // that follow the tail's last reads).
  const int averages = average ? a.B / kIndexTokens : 0, stores = (x.p1 - x.p0 + kIndexTokens - 1) / kIndexTokens;
#pragma unroll 1
  for (int seg = 0; seg < averages + stores; ++seg) {
    const bool store = seg >= averages;
    const int q = x.p0 + (seg - averages) * kIndexTokens, at = seg * kIndexTokens;
    const int count = store ? min(kIndexTokens, x.p1 - q) : kIndexTokens;
    const int old = store ? 0 : max(0, min(kIndexTokens, olds - at));          // rows from the tail, then fresh ones
    const int64_t t = store ? x.cu0 + q - x.past : block_t + max(at, olds);  // token of the first of these
    const uint16_t* from = tail + ((int64_t)(x.avg_blk & 1) * a.B + at) * hs;
    if (seg) __syncthreads();  // the segment before has been added up
#pragma unroll
    for (int e = 0; e < kIndexSteps; ++e) {
      const int i = (e * kIndexRows + g) >> shift;
      if (i < count) {
        const uint16_t* row = i < old ? from + i * hs : src + (t + i - old) * a.ki.x_token;
        copy16(&s.rows[i][sub][da >> 3], row + da);
        copy16(&s.rows[i][sub][db >> 3], row + db);
      }
    }
    copies_commit();
    if (old < count && !filled) filler.fill(s.tab, a.q.an, t, count - old);
    Values w;
    load_weights<kAdjacent>(a.ki, h, da, db, a.q.offset, w);
    copies_wait<0>();
    __syncthreads();  // the angles are there
#pragma unroll 1
    for (int e = 0; e < kIndexSteps; ++e) {
      const int i = (e * kIndexRows + g) >> shift;
      const bool fresh = i >= old && i < count;
      if (!__any_sync(0xffffffffu, fresh)) continue;
      const int row = fresh ? i : 0;  // a row of its own, or any
      uint4 ua, ub;
      auto read = [&](uint4& xa, uint4& xb) {
        xa = fresh ? s.rows[row][sub][da >> 3] : make_uint4(0, 0, 0, 0);
        xb = fresh ? s.rows[row][sub][db >> 3] : make_uint4(0, 0, 0, 0);
      };
      read(ua, ub);
      norm_rotate<kAdjacent>(ua, ub, w, s.tab.cs[fresh ? i - old : 0], j, norm, turn && fresh, a.q.eps, read);
      if (!fresh) continue;
      if (store) {
        uint16_t* out = tail + ((int64_t)(x.open & 1) * a.B + ((q + i) & (a.B - 1))) * hs;
        *reinterpret_cast<uint4*>(out + da) = ua;
        *reinterpret_cast<uint4*>(out + db) = ub;
      } else {
        s.rows[i][sub][da >> 3] = ua;
        s.rows[i][sub][db >> 3] = ub;
      }
    }
    __syncthreads();  // the rows are there, the angles have been read
    if (store || tid >= hn * 64) continue;
    const uint32_t* row = reinterpret_cast<const uint32_t*>(s.rows[0][tid >> 6]) + (tid & 63);
#pragma unroll 8
    for (int i = 0; i < kIndexTokens; ++i) {
      const uint32_t u = row[i * kIndexHeads * 64];
      lo = __fadd_rn(lo, __uint_as_float(u << 16));
      hi = __fadd_rn(hi, __uint_as_float(u & 0xFFFF0000u));
    }
    if (seg == averages - 1) {
      const float inv = 1.f / (float)a.B;  // a power of two: the product is the quotient
      *reinterpret_cast<uint32_t*>(a.index_pool + (slot >> (a.B == 128 ? 7 : 6)) * hs + h0 * 128 + 2 * tid) =
          pack_bf16x2(lo * inv, hi * inv);
    }
  }
  // the angles serve the next heads where there is one table of them
  filled = averages == 1 && stores == 0;
}
template <bool kAdjacent>
MSA_DEV void average_block(const AppendRopeArgs& a, const cache::IndexPlan& x, int h0, int hn, IndexShared& s) {
  const Filler<kAdjacent> filler(a.q.an, threadIdx.x, kThreads);
  bool filled = false;
  for (int h = h0; h < h0 + hn; h += kIndexHeads) {
    average_heads<kAdjacent>(a, x, h, min(kIndexHeads, h0 + hn - h), filler, filled, s);
    __syncthreads();  // the rows have been added up
  }
}

template <bool kAdjacent>
MSA_DEV void index_block(const AppendRopeArgs& a, int block, bool bad, IndexShared& s) {
  const int row = block / a.index_groups, h0 = (block - row * a.index_groups) * a.index_heads;
  const int hn = min(a.index_heads, a.H - h0);
  const int warp = threadIdx.x >> 5, g0 = row * a.index_chunks;
  cache::IndexPlan x;
  const bool todo = !__any_sync(0xffffffffu, bad) && warp < a.index_chunks && g0 + warp < a.NC &&
                    cache::plan_index(a, g0 + warp, (threadIdx.x & 31) == 0, x);
  const bool average = todo && x.last >= 0;
  if (todo && !average) store_tail<kAdjacent>(a, x, h0, hn, warp, s);
  if ((threadIdx.x & 31) == 0) s.average[warp] = average;
  __syncthreads();
  for (int i = 0; i < a.index_chunks; ++i)
    if (s.average[i]) {
      cache::plan_index(a, g0 + i, false, x);
      average_block<kAdjacent>(a, x, h0, hn, s);
    }
}

constexpr size_t kAppendShared = sizeof(IndexShared);
static_assert(sizeof(RowsShared) <= kAppendShared && sizeof(KvShared) <= kAppendShared, "one size for every CTA");
// The CTAs of index keys come first: a block's mean takes longest.  Where CTAs come in
// many waves, those of K and V and of Q then take turns in proportion to their numbers:
// K's are bound by instructions and Q's by memory, and an SM should hold both (4 x 8192
// tokens 407 us, with K's before Q's 435).  Where all run together K's come before Q's.
// turns: count * 2^32 / of, rounded up, so that `of` turns take count.
MSA_DEV bool takes_turn(int64_t& block, uint64_t turns) {
  const int64_t before = (int64_t)(block * turns >> 32), after = (int64_t)((block + 1) * turns >> 32);
  block = after > before ? before : block - before;
  return after > before;
}
// kCtas: of an SM.  Two leave room for more loads under way at once, which counts where
// all CTAs run together (a step of 256 tokens 8.0 us, with three 10.9; 2,900 tokens of
// prompt pieces 27, 34); where they come in many waves three do more (4 x 8192 tokens
// 423 us, with three 407).
template <bool kAdjacent, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) append_rope_kernel(AppendRopeArgs a) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  // The next kernel's CTAs do not come up early: beside these they take slots and issue (a captured decode step of 16
  // requests 22.6 us, with them 25.0; an append of 256 tokens and its read 11.6, 16.3).
  cache::after_previous_kernel<false>();
  const bool bad = status_bad(a.status);
  int64_t block = blockIdx.x;
  if (block < a.index_blocks) {
    index_block<kAdjacent>(a, (int)block, bad, *reinterpret_cast<IndexShared*>(s_raw));
    return;
  }
  block -= a.index_blocks;
  bool kv = block < a.kv_blocks;
  if constexpr (kCtas == 3) kv = takes_turn(block, a.kv_turns);
  else if (!kv) block -= a.kv_blocks;
  if (kv)
    kv_block<kAdjacent>(a, (int)block, bad, *reinterpret_cast<KvShared*>(s_raw));
  else
    rows_block<kAdjacent>(a.q, (int)block, bad, *reinterpret_cast<RowsShared*>(s_raw));
}

// Tokens of a tile: the most whose tiles still give every SM two CTAs.
inline int cut_tokens(int64_t tokens, int64_t groups, int sms, int most, int least) {
  int tile = most;
  while (tile > least && (tokens + tile - 1) / tile * groups < 2 * (int64_t)sms) tile >>= 1;
  return tile;
}

}  // namespace rope
}  // namespace msa

using namespace msa;

extern "C" int msa_cache_append_rope(const msa_cache_problem* c, const msa_rope_problem* p, const uint16_t* q,
                                     const uint16_t* k, const uint16_t* v, const uint16_t* q_index,
                                     const uint16_t* k_index, const int32_t* positions, const int64_t* slot_map,
                                     const int32_t* cu_tokens, const int32_t* chunks, uint16_t* q_out,
                                     uint16_t* q_index_out, uint8_t* kv_cache, uint16_t* index_tail,
                                     uint16_t* index_pool, int32_t* d_status, void* stream) {
  int rc = cache::check_cache_problem(c);
  if (rc || (rc = rope::check_problem(p))) return rc;
  const msa_rope_tensor* t = p->tensor;
  const int H = c->num_kv_heads;
  if (p->tokens != c->token_cap || t[MSA_ROPE_K].heads != H || t[MSA_ROPE_V].heads != H || t[MSA_ROPE_V].flags ||
      (t[MSA_ROPE_Q].heads && t[MSA_ROPE_Q].heads != c->num_q_heads) ||
      (t[MSA_ROPE_Q_INDEX].heads && t[MSA_ROPE_Q_INDEX].heads != H) ||
      (t[MSA_ROPE_K_INDEX].heads && t[MSA_ROPE_K_INDEX].heads != H))
    return MSA_ERR_INVALID_ARGUMENT;
  auto bad = [](std::initializer_list<const void*> ptrs) {
    for (const void* x : ptrs)
      if (!x || !aligned16(x)) return true;
    return false;
  };
  const bool index = t[MSA_ROPE_K_INDEX].heads > 0;
  if (bad({k, v, positions, slot_map, kv_cache, d_status})) return MSA_ERR_INVALID_ARGUMENT;
  if (t[MSA_ROPE_Q].heads && bad({q, q_out})) return MSA_ERR_INVALID_ARGUMENT;
  if (t[MSA_ROPE_Q_INDEX].heads && bad({q_index, q_index_out})) return MSA_ERR_INVALID_ARGUMENT;
  if (index && bad({k_index, cu_tokens, chunks, index_tail, index_pool})) return MSA_ERR_INVALID_ARGUMENT;
  if ((rc = check_device_current())) return rc;
  int32_t sms = 0;
  if ((rc = sm_count_current(&sms))) return rc;
  rope::AppendRopeArgs a{};
  auto tensor = [&](int i, const uint16_t* x, int end) {
    return rope::Tensor{t[i].heads ? x : nullptr, t[i].weight, t[i].x_token, t[i].x_head, t[i].flags, end};
  };
  a.T = p->tokens; a.H = H; a.B = c->block_size; a.R = c->num_requests; a.NC = c->chunk_cap;
  // q and index q as two of the row kernel's tensors, the others empty
  const int nq = t[MSA_ROPE_Q].heads, ni = t[MSA_ROPE_Q_INDEX].heads;
  a.q.t[0] = tensor(MSA_ROPE_Q, q, nq);
  a.q.t[1] = tensor(MSA_ROPE_Q_INDEX, q_index, nq + ni);
  a.q.t[2] = a.q.t[3] = a.q.t[1];
  const int role[2] = {MSA_ROPE_Q, MSA_ROPE_Q_INDEX};
  for (int i = 0; i < 2; ++i) {
    a.q.y_token[i] = t[role[i]].y_token;
    a.q.y_head[i] = t[role[i]].y_head;
  }
  a.q.y[0] = q_out;
  a.q.y[1] = q_index_out;
  a.q.an = rope::angles_of(p, positions, d_status);
  a.q.eps = p->eps;
  a.q.offset = p->weight_offset;
  a.q.T = a.T;
  a.q.zero = p->zero_padding;
  a.q.heads = nq + ni;
  a.q.status = a.status = d_status;
  a.k = tensor(MSA_ROPE_K, k, 0);
  a.ki = tensor(MSA_ROPE_K_INDEX, k_index, 0);
  a.v = v;
  a.v_token = t[MSA_ROPE_V].x_token;
  a.v_head = t[MSA_ROPE_V].x_head;
  a.slot_map = slot_map; a.cu_tokens = cu_tokens; a.chunks = chunks;
  a.cache = kv_cache; a.index_tail = index_tail; a.index_pool = index_pool;
  a.positions = c->max_blocks * c->block_size;
  a.slots = (int64_t)c->num_pages * c->block_size;
  a.k_mul = cache::exp2i(-c->k_exp);
  a.v_mul = cache::exp2i(-c->v_exp);
  a.kv_groups = (H + 7) / 8;
  a.kv_heads = (H + a.kv_groups - 1) / a.kv_groups;
  // Tokens that give half of a CTA's warps work (a step of 64 tokens 5.1 us, all of them 5.4).
  int rows = 4;
  while (rows < rope::kKvTile && rows * a.kv_heads < rope::kIndexRows / 2) rows *= 2;
  a.kv_tile = rope::cut_tokens(a.T, a.kv_groups, sms, rows < 16 ? 16 : rows, rows);
  const int64_t kv_blocks = (int64_t)((a.T + a.kv_tile - 1) / a.kv_tile) * a.kv_groups;
  // Few heads and chunks to a CTA where the CTAs find room, so that heads, and blocks that end in neighbouring chunks
  // (requests of one length), do not wait for one another; else eight heads, which share their angles (4 x 8192 tokens
  // 406 us, with two 431).  A mean takes longest among chunks of several tokens, by the capacities: one head there
  // (prompt pieces 27.2 us, with two 29.6), two for single tokens (a step of 256 8.1, with one 12.9).
  const bool prompts = c->token_cap / c->chunk_cap >= 3;
  a.index_heads = (int64_t)c->chunk_cap * H > 16 * (int64_t)sms ? 8 : prompts ? 1 : rope::kIndexHeads;
  a.index_groups = (H + a.index_heads - 1) / a.index_heads;
  a.index_chunks = rope::kWarps;
  auto index_ctas = [&](int64_t chunks) { return (c->chunk_cap + chunks - 1) / chunks * a.index_groups; };
  while (a.index_chunks > 1 && index_ctas(a.index_chunks / 2) <= sms) a.index_chunks /= 2;
  const int64_t index_blocks = index ? index_ctas(a.index_chunks) : 0;
  int64_t q_blocks = 0;
  if (a.q.heads) {
    a.q.cut = rope::cut_rows(a.q.heads, a.T, sms, 2 * rope::kWarps, rope::kWarps - 1);
    // In a step all CTAs should run at once: q's tokens go to as many as the others leave room for (a step of 64 tokens
    // 5.4 us, with shares of 12 tokens 6.1).  Where that makes shares of more than 12 tokens,
    // shares of 12 to 64, by the call's size: enough to mix with K's CTAs.
    const int64_t room = (2 * (int64_t)sms - index_blocks - kv_blocks) / a.q.cut.groups;
    const int64_t per = (int64_t)a.T * a.q.cut.groups / (8 * (int64_t)sms);
    const int64_t tokens = room > 0 && a.T <= 12 * room ? (a.T + room - 1) / room : per < 12 ? 12 : per > 64 ? 64 : per;
    a.q.cut.slices = (int)((a.T + tokens - 1) / tokens);
    q_blocks = (int64_t)a.q.cut.slices * a.q.cut.groups;
  }
  if (index_blocks + kv_blocks + q_blocks > INT32_MAX) return MSA_ERR_UNSUPPORTED_SHAPE;
  a.index_blocks = (int)index_blocks;
  a.kv_blocks = (int)kv_blocks;
  const uint64_t turns = (uint64_t)(kv_blocks + q_blocks);
  a.kv_turns = turns ? (((uint64_t)kv_blocks << 32) + turns - 1) / turns : 0;
  const bool many = index_blocks + kv_blocks + q_blocks > 8 * (int64_t)sms;
  auto* kernel = p->adjacent ? (many ? rope::append_rope_kernel<true, 3> : rope::append_rope_kernel<true, 2>)
                             : (many ? rope::append_rope_kernel<false, 3> : rope::append_rope_kernel<false, 2>);
  return cache::launch_kernel(kernel, dim3((unsigned)(index_blocks + kv_blocks + q_blocks)), rope::kThreads,
                              rope::kAppendShared, stream, 1, a);
}
