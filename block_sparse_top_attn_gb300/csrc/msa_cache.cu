// Serving over the 4-bit paged cache: step tables, cache writer and reader,
// block selection.  (The attention over the cache is in msa_cache_fwd.cu.)
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "msa_cache.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace cache {

int check_cache_problem(const msa_cache_problem* p) {
  if (!p) return MSA_ERR_INVALID_ARGUMENT;
  if (p->num_requests < 1 || p->num_pages < 1 || p->max_blocks < 1 || p->num_kv_heads < 1 || p->token_cap < 1 ||
      p->chunk_cap < 1)
    return MSA_ERR_INVALID_ARGUMENT;
  if (p->head_dim != kHeadDim || (p->block_size != 64 && p->block_size != 128) || p->query_chunk != kChunk)
    return MSA_ERR_UNSUPPORTED_SHAPE;
  if (p->num_kv_heads > kMaxHeads || p->num_q_heads != kGroup * p->num_kv_heads) return MSA_ERR_UNSUPPORTED_SHAPE;
  if (p->topk < 1 || p->topk > kMaxTopk) return MSA_ERR_UNSUPPORTED_SHAPE;
  if (p->num_requests > kMaxRequests || p->num_pages > kMaxCount || p->max_blocks > kMaxBlocks ||
      p->token_cap > kMaxCount || p->chunk_cap > kMaxCount)
    return MSA_ERR_UNSUPPORTED_SHAPE;
  if (p->k_exp < -kMaxExp || p->k_exp > kMaxExp || p->v_exp < -kMaxExp || p->v_exp > kMaxExp)
    return MSA_ERR_INVALID_ARGUMENT;
  if (!(p->softmax_scale > 0.f && p->softmax_scale <= 3.4028234663852886e38f)) return MSA_ERR_INVALID_ARGUMENT;
  return MSA_OK;
}

// ---------------------------------------------------------------------------
// step: block table, slots, positions and chunks from the lengths
// ---------------------------------------------------------------------------
struct StepArgs {
  const int32_t *new_lens, *seq_lens, *ring;
  int32_t *free_ring, *block_table, *seq_lens_out, *ring_out, *cu_tokens;
  int64_t* slot_map;
  int32_t *positions, *chunks;
  int R, P, M, B, T, NC;
  int32_t* status;
};

constexpr int kStepThreads = 1024;

// Exclusive prefix sums over the CTA of three 64-bit values per thread.
__device__ void scan3(int64_t (&v)[3], int64_t (&total)[3], int64_t (*s)[33]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    inc[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc[i], o);
      if (lane >= o) inc[i] += y;
    }
    if (lane == 31) s[i][warp] = inc[i];
  }
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int64_t own = s[i][lane];
      int64_t x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      s[i][lane] = x - own;
      if (lane == 31) s[i][32] = x;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    v[i] = s[i][warp] + inc[i] - v[i];
    total[i] = s[i][32];
  }
}

// Largest r in [0, n) with off[r] <= x (off ascending, off[0] <= x).
__device__ __forceinline__ int last_at_or_below(const int32_t* off, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One cluster of 1 to 8 CTAs.  Every CTA scans all lengths (a few KB from L2)
// into shared memory, so no CTA waits for another's tables; the chunks, eight
// tokens each, are then spread over the cluster, one chunk a thread.  The
// lengths and the ring may be updated in place, so they are written after a
// cluster barrier that follows every read of them.  Latency-bound: the bytes
// (12 per token, 16 per chunk) take microseconds only for 100k tokens.
__global__ void __launch_bounds__(kStepThreads) step_kernel(StepArgs a) {
  extern __shared__ int32_t s_off[];  // cu_tokens, cu_chunks, cu_alloc: R + 1 each
  __shared__ int64_t s_scan[3][33];
  __shared__ int s_err;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x;
  int32_t* cu = s_off;
  int32_t* cch = cu + (a.R + 1);
  int32_t* cal = cch + (a.R + 1);
  if (tid == 0) s_err = status_bad(a.status) ? MSA_ERR_INVALID_ARGUMENT : 0;  // any value: skip
  __syncthreads();
  const int head = a.ring[0], count = a.ring[1];
  // thread t owns requests [t * per, t * per + per)
  const int per = (a.R + kStepThreads - 1) / kStepThreads;
  int64_t v[3] = {0, 0, 0};  // tokens, chunks, (blocks taken << 32) + blocks given back
  int err = 0;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r >= a.R) break;
    const int n = a.new_lens[r], past = a.seq_lens[r];
    if (n < -1 || past < 0 || past > a.M * a.B) { err = MSA_ERR_INVALID_CACHE; break; }
    const int held = (past + a.B - 1) / a.B;
    if (n < 0) {
      v[2] += held;
    } else {
      if (n > a.M * a.B - past) { err = MSA_ERR_CAPACITY; break; }
      v[0] += n;
      if (n > 0) v[1] += (past + n - 1) / kChunk - past / kChunk + 1;
      v[2] += (int64_t)((past + n + a.B - 1) / a.B - held) << 32;
    }
  }
  if (err) atomicMax(&s_err, err);
  int64_t total[3];
  scan3(v, total, s_scan);
  const int64_t taken = total[2] >> 32, given = total[2] & 0xffffffff;
  if (tid == 0 && !s_err) {
    if (head < 0 || head >= a.P || count < 0 || count > a.P) s_err = MSA_ERR_INVALID_CACHE;
    else if (total[0] > a.T || total[1] > a.NC || taken > count) s_err = MSA_ERR_CAPACITY;
    else if (count - taken + given > a.P) s_err = MSA_ERR_INVALID_CACHE;
  }
  __syncthreads();
  const bool ok = s_err == 0;
  if (ok) {
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r >= a.R) break;
      const int n = max(a.new_lens[r], 0), past = a.seq_lens[r];
      cu[r] = (int)v[0];
      cch[r] = (int)v[1];
      cal[r] = (int)(v[2] >> 32);
      v[0] += n;
      if (n > 0) v[1] += (past + n - 1) / kChunk - past / kChunk + 1;
      if (n > 0) v[2] += (int64_t)((past + n + a.B - 1) / a.B - (past + a.B - 1) / a.B) << 32;
    }
    __syncthreads();
    const int nchunks = (int)total[1], ntok = (int)total[0];
    for (int g = rank * kStepThreads + tid; g < a.NC; g += ranks * kStepThreads) {
      int4 row = make_int4(-1, -1, -1, -1);
      if (g < nchunks) {
        const int r = last_at_or_below(cch, a.R, g);
        const int past = a.seq_lens[r], n = a.new_lens[r];
        const int c = past / kChunk + g - cch[r];
        const int first = max(past, c * kChunk), last = min(past + n, c * kChunk + kChunk);
        const int held = (past + a.B - 1) / a.B, blk = first / a.B;
        int page;
        if (blk < held) {
          page = a.block_table[(int64_t)r * a.M + blk];
        } else {
          page = a.free_ring[(int)(((int64_t)head + cal[r] + blk - held) % a.P)];
          if (first % a.B == 0) a.block_table[(int64_t)r * a.M + blk] = page;
        }
        row = make_int4(r, cu[r] + first - past, last - first, first);
        const int64_t slot = (int64_t)page * a.B + first % a.B;
        for (int i = 0; i < row.z; ++i) {
          a.slot_map[row.y + i] = slot + i;
          a.positions[row.y + i] = first + i;
        }
      }
      reinterpret_cast<int4*>(a.chunks)[g] = row;
    }
    for (int t = ntok + rank * kStepThreads + tid; t < a.T; t += ranks * kStepThreads) {
      a.slot_map[t] = -1;
      a.positions[t] = -1;
    }
    if (rank == 0) {
      for (int r = tid; r < a.R; r += kStepThreads) a.cu_tokens[r] = cu[r];
      if (tid == 0) a.cu_tokens[a.R] = ntok;
    }
  }
  // every read of the lengths and the ring is done
  cluster.sync();
  if (ok && rank == 0) {
    // pages of finished requests, in (request, block) order behind the ring's
    // last entry: those entries hold no free page, so nothing read above is
    // overwritten.  v[2]'s low half: this thread's first place.
    int at = (int)(v[2] & 0xffffffff);
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r >= a.R) break;
      const int n = a.new_lens[r], past = a.seq_lens[r];
      if (n < 0) {
        const int held = (past + a.B - 1) / a.B;
        for (int b = 0; b < held; ++b)
          a.free_ring[(int)(((int64_t)head + count + at + b) % a.P)] = a.block_table[(int64_t)r * a.M + b];
        at += held;
      }
      a.seq_lens_out[r] = n < 0 ? 0 : past + n;
    }
    if (tid == 0) {
      a.ring_out[0] = (int)((head + taken) % a.P);
      a.ring_out[1] = (int)(count - taken + given);
    }
  }
  if (!ok && rank == 0 && tid == 0) set_status(a.status, s_err);
}

// ---------------------------------------------------------------------------
// append and read: bf16 rows <-> 4-bit tiles
// ---------------------------------------------------------------------------
struct AppendArgs {
  const uint16_t *k, *v, *k_index;
  const int64_t* slot_map;
  const int32_t *cu_tokens, *chunks;
  uint8_t* cache;
  uint16_t *index_tail, *index_pool;
  int T, H, B, R, NC;
  int64_t slots;  // P * B
  float k_mul, v_mul;  // 2^-exp
  int index_blocks;    // leading CTAs that keep the pooled index keys
  int32_t* status;
};

// 16 bf16 values as fp32 (exact), two 16-byte loads.
MSA_DEV void load16(const uint16_t* src, float (&x)[16], uint32_t& amax) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(src)), b = __ldg(reinterpret_cast<const uint4*>(src) + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    amax = max(amax, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
  }
}

// Clears the sign of the codes that are zero, so that equal values have equal
// bytes.
MSA_DEV uint32_t unsigned_zeros(uint32_t w) {
  const uint32_t m = w & 0x77777777u;
  return w & (((m << 1 | m << 2 | m << 3) & 0x88888888u) | 0x77777777u);
}

// One group of 16 values to codes (8 bytes) and an e4m3 scale.  The quotient
// x / s is formed as x * (1 / s): it is either a border between two codes (a
// multiple of 1/4) or at least 2^-11 away from it, because x has 8 significant
// bits and border * s 7.  Rounding it to a multiple of 2^-14 (the addition of
// 1.5 * 2^9) therefore undoes the reciprocal's error, and the conversion's ties
// are those of the exact quotient.
MSA_DEV uint32_t quantize16(const float (&x)[16], uint32_t amax_bits, float mul, uint2& codes) {
  codes = make_uint2(0, 0);
  if (amax_bits >= 0x7F800000u) return 0x7F;  // a NaN scale: the group reads back as NaN
  // amax <= 2^128 and mul <= 2^32: an overflow to infinity saturates below
  const float t = __fdiv_rn(__uint_as_float(amax_bits) * mul, 6.f);
  uint16_t s2;
  asm("{\n\tcvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n\t}" : "=h"(s2) : "f"(0.f), "f"(t));
  const uint32_t s8 = s2 & 0xFFu;
  if (s8 == 0) return 0;
  const uint32_t sh = e4m3x2_to_half(s8);
  const float s = __half2float(__ushort_as_half((uint16_t)(sh & 0xFFFFu)));
  const float inv = __fdiv_rn(1.f, s) * mul;  // a power of two apart, exact
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = fminf(fmaxf(x[8 * h + i] * inv, -8.f), 8.f);
      q[i] = __fadd_rn(__fadd_rn(y, 768.f), -768.f);
    }
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(out[h])
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  }
  codes = make_uint2(unsigned_zeros(out[0]), unsigned_zeros(out[1]));
  return s8;
}

// Index keys of one (chunk, head), by one warp, lane l owning dims 4l..4l+3.
// The chunk that ends a block averages the block's tokens, those of earlier
// calls from the tail.  The first chunk of a request then stores the request's
// incomplete block's rows of this call: one warp does both, so a tail buffer is
// read before it is overwritten (a lane reads and writes its own dims only).
MSA_DEV void index_chunk(const AppendArgs& a, int g, int h, int lane) {
  const int4 c = reinterpret_cast<const int4*>(a.chunks)[g];
  const int r = c.x, row0 = c.y, n = c.z, pos0 = c.w;
  if (r < 0) return;
  int cu0 = 0, cu1 = 0;
  bool good = r < a.R && n >= 1 && n <= kChunk && row0 >= 0 && row0 <= a.T - n && pos0 >= 0;
  if (good) {
    cu0 = a.cu_tokens[r];
    cu1 = a.cu_tokens[r + 1];
    good = cu0 >= 0 && cu0 <= row0 && cu1 >= row0 + n && cu1 <= a.T && pos0 >= row0 - cu0 &&
           pos0 % a.B + n <= a.B;
  }
  if (!good) {
    if (lane == 0) set_status(a.status, MSA_ERR_INVALID_CACHE);
    return;
  }
  const int64_t hs = (int64_t)a.H * 128;  // elements from one token's row to the next
  const int d = h * 128 + lane * 4;
  const int end = pos0 + (cu1 - row0);     // position behind the request's last new token
  const int past = pos0 - (row0 - cu0);
  uint16_t* tail = a.index_tail + (int64_t)r * 2 * a.B * hs + d;
  // averages the block that ends at row `last` (its last token)
  auto average = [&](int last, int blk) {
    const int64_t slot = a.slot_map[last];
    if (slot < 0 || slot >= a.slots) return;  // reported by the rows' own CTAs, or left out
    const uint16_t* old = tail + (int64_t)(blk & 1) * a.B * hs;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int i = 0; i < a.B; ++i) {
      const int row = last - (a.B - 1) + i;
      const uint2 w = *reinterpret_cast<const uint2*>(row >= cu0 ? a.k_index + row * hs + d : old + i * hs);
      acc[0] = __fadd_rn(acc[0], __uint_as_float(w.x << 16));
      acc[1] = __fadd_rn(acc[1], __uint_as_float(w.x & 0xFFFF0000u));
      acc[2] = __fadd_rn(acc[2], __uint_as_float(w.y << 16));
      acc[3] = __fadd_rn(acc[3], __uint_as_float(w.y & 0xFFFF0000u));
    }
    const float inv = 1.f / (float)a.B;  // a power of two: the product is the quotient
    uint2 o;
    o.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    o.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2*>(a.index_pool + (slot / a.B) * hs + d) = o;
  };
  const int blk0 = past / a.B, blk = pos0 / a.B;
  if (blk > blk0 && (pos0 + n) % a.B == 0) average(row0 + n - 1, blk);
  if (row0 == cu0) {
    const int first_end = (blk0 + 1) * a.B;
    if (first_end <= end) average(cu0 + first_end - past - 1, blk0);
    const int open = end / a.B;  // the block that stays incomplete
    uint16_t* dst = tail + (int64_t)(open & 1) * a.B * hs;
    for (int p = max(past, open * a.B); p < end; ++p)
      *reinterpret_cast<uint2*>(dst + (p % a.B) * hs) =
          *reinterpret_cast<const uint2*>(a.k_index + (cu0 + p - past) * hs + d);
  }
}

__global__ void __launch_bounds__(256) append_kernel(AppendArgs a) {
  if (status_bad(a.status)) return;
  if ((int)blockIdx.x < a.index_blocks) {
    const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (w < (int64_t)a.NC * a.H) index_chunk(a, (int)(w / a.H), (int)(w % a.H), threadIdx.x & 31);
    return;
  }
  // a thread takes one group of 16 dims of K and of V: no value crosses threads
  const int64_t i = (int64_t)(blockIdx.x - a.index_blocks) * blockDim.x + threadIdx.x;
  const int64_t row = i >> 3;  // token * H + head
  const int grp = (int)(i & 7);
  if (row >= (int64_t)a.T * a.H) return;
  const int t = (int)(row / a.H), h = (int)(row % a.H);
  const int64_t slot = a.slot_map[t];
  if (slot < 0 || slot >= a.slots) {
    if (slot != -1) set_status(a.status, MSA_ERR_INVALID_CACHE);
    return;
  }
  float x[16];
  uint32_t amax;
  uint2 kc, vc;
  load16(a.k + row * 128 + grp * 16, x, amax);
  const uint32_t ks = quantize16(x, amax, a.k_mul, kc);
  load16(a.v + row * 128 + grp * 16, x, amax);
  const uint32_t vs = quantize16(x, amax, a.v_mul, vc);
  const int off = (int)(slot % a.B), tok = off % kTile;
  uint8_t* tile = a.cache + tile_index(slot / a.B, h, a.H, a.B / kTile, off / kTile) * kTileBytes;
  *reinterpret_cast<uint2*>(tile + OFF_KC + tok * kRowBytes + grp * 8) = kc;
  *reinterpret_cast<uint2*>(tile + OFF_VC + v_code_offset(tok, grp)) = vc;
  tile[OFF_KS + tok * kScales + grp] = (uint8_t)ks;
  tile[OFF_VS + grp * kTile + tok] = (uint8_t)vs;
}

struct ReadArgs {
  const int64_t* slots;
  const uint8_t* cache;
  uint16_t *k, *v;
  int T, H, B;
  int64_t nslots;
  float k_mul, v_mul;  // 2^exp
  int32_t* status;
};

// 16 codes and their scale as bf16.
MSA_DEV void dequantize16(uint2 codes, uint32_t scale, float mul, uint16_t* dst) {
  uint32_t s = e4m3x2_to_half(scale);
  s = __byte_perm(s, s, 0x1010);
  uint32_t out[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p[4];
    e2m1x8_to_half(h ? codes.y : codes.x, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t y = mul_half2(p[i], s);
      out[4 * h + i] = pack_bf16x2(__half2float(__ushort_as_half((uint16_t)(y & 0xFFFFu))) * mul,
                                   __half2float(__ushort_as_half((uint16_t)(y >> 16))) * mul);
    }
  }
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

__global__ void __launch_bounds__(256) read_kernel(ReadArgs a) {
  if (status_bad(a.status)) return;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t row = i >> 3;
  const int grp = (int)(i & 7);
  if (row >= (int64_t)a.T * a.H) return;
  const int t = (int)(row / a.H), h = (int)(row % a.H);
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.nslots) {
    if (slot != -1) set_status(a.status, MSA_ERR_INVALID_CACHE);
    return;
  }
  const int off = (int)(slot % a.B), tok = off % kTile;
  const uint8_t* tile = a.cache + tile_index(slot / a.B, h, a.H, a.B / kTile, off / kTile) * kTileBytes;
  dequantize16(*reinterpret_cast<const uint2*>(tile + OFF_KC + tok * kRowBytes + grp * 8),
               tile[OFF_KS + tok * kScales + grp], a.k_mul, a.k + row * 128 + grp * 16);
  dequantize16(*reinterpret_cast<const uint2*>(tile + OFF_VC + v_code_offset(tok, grp)),
               tile[OFF_VS + grp * kTile + tok], a.v_mul, a.v + row * 128 + grp * 16);
}

// ---------------------------------------------------------------------------
// select: scores of a chunk against its request's pooled index keys, top-k
// ---------------------------------------------------------------------------
struct SelectArgs {
  const uint16_t *q_index, *pool;
  const int32_t *block_table, *chunks;
  int32_t* sel;
  int R, P, M, B, T, NC, H, K;
  int32_t* status;
};
constexpr int kSelThreads = 256;

// A score as an unsigned key of the same order (-0 counts as +0).
MSA_DEV uint32_t score_key(float s) {
  const uint32_t u = __float_as_uint(__fadd_rn(s, 0.f));
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (chunk, head): the scores of all earlier blocks as ordered keys
// in shared memory (one block a thread, so the sum keeps its order), then a
// radix selection of the (K-1)-th largest key, 8 bits a pass.
__global__ void __launch_bounds__(kSelThreads) select_kernel(SelectArgs a) {
  extern __shared__ uint32_t s_key[];  // [M]
  __shared__ float s_q[128];
  __shared__ uint32_t s_hist[256], s_prefix, s_need, s_count;
  __shared__ uint32_t s_topk[kMaxTopk];
  __shared__ int s_topb[kMaxTopk];
  if (status_bad(a.status)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x, h = blockIdx.y;
  const int4 c = reinterpret_cast<const int4*>(a.chunks)[g];
  if (c.x < 0) return;
  const int n = c.w / a.B;  // earlier blocks
  if (c.x >= a.R || c.z < 1 || c.z > kChunk || c.y < 0 || c.y > a.T - c.z || c.w < 0 || n >= a.M) {
    if (tid == 0) set_status(a.status, MSA_ERR_INVALID_CACHE);
    return;
  }
  const int64_t hs = (int64_t)a.H * 128;
  if (tid < 128) {
    const uint16_t* src = a.q_index + (int64_t)c.y * hs + h * 128 + tid;
    float acc = 0.f;
    for (int i = 0; i < c.z; ++i) acc = __fadd_rn(acc, __uint_as_float((uint32_t)src[i * hs] << 16));
    const uint32_t m = pack_bf16x2(__fdiv_rn(acc, (float)c.z), 0.f);
    s_q[tid] = __uint_as_float(m << 16);
  }
  if (tid == 0) { s_prefix = 0; s_count = 0; }
  __syncthreads();
  const int32_t* table = a.block_table + (int64_t)c.x * a.M;
  for (int b = tid; b < n; b += kSelThreads) {
    const int page = table[b];
    float s = 0.f;
    if (page < 0 || page >= a.P) {
      set_status(a.status, MSA_ERR_INVALID_CACHE);
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(a.pool + page * hs + h * 128);
#pragma unroll 8
      for (int i = 0; i < 16; ++i) {
        const uint4 w = __ldg(src + i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s = __fmaf_rn(s_q[8 * i + 2 * e], __uint_as_float(u[e] << 16), s);
          s = __fmaf_rn(s_q[8 * i + 2 * e + 1], __uint_as_float(u[e] & 0xFFFF0000u), s);
        }
      }
    }
    s_key[b] = score_key(s);
  }
  const int keep = min(a.K - 1, n);
  uint32_t thr = 0;   // keys above it are kept, of those equal to it the first s_need
  if (keep > 0 && keep < n) {
    if (tid == 0) s_need = keep;
    for (int shift = 24; shift >= 0; shift -= 8) {
      s_hist[tid] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix, need = s_need;
      const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      for (int b = tid; b < n; b += kSelThreads)
        if ((s_key[b] & mask) == prefix) atomicAdd(&s_hist[(s_key[b] >> shift) & 255], 1u);
      __syncthreads();
      if (warp == 0) {
        // digits from the top: lane l holds digits 255 - 8l .. 248 - 8l
        uint32_t cnt[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) { cnt[i] = s_hist[255 - 8 * lane - i]; sum += cnt[i]; }
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        uint32_t above = inc - sum;
        if (above < need && inc >= need) {
          int i = 0;
          for (; i < 7; ++i) {
            if (above + cnt[i] >= need) break;
            above += cnt[i];
          }
          s_prefix = prefix | ((uint32_t)(255 - 8 * lane - i) << shift);
          s_need = need - above;
        }
      }
      __syncthreads();
    }
    thr = s_prefix;
  } else {
    __syncthreads();
    if (tid == 0) s_need = 0;  // every earlier block is kept: all keys are above 0
    __syncthreads();
  }
  // the kept blocks, in any order
  if (keep > 0) {
    for (int b = tid; b < n; b += kSelThreads)
      if (keep == n || s_key[b] > thr) {
        const uint32_t at = atomicAdd(&s_count, 1u);
        s_topk[at] = s_key[b];
        s_topb[at] = b;
      }
    __syncthreads();
    if (warp == 0 && keep < n) {
      // of the keys equal to the threshold, the lowest blocks
      uint32_t at = s_count, need = s_need;
      for (int b0 = 0; b0 < n && need; b0 += 32) {
        const bool eq = b0 + lane < n && s_key[b0 + lane] == thr;
        const uint32_t m = __ballot_sync(0xffffffffu, eq);
        const uint32_t before = __popc(m & ((1u << lane) - 1u));
        if (eq && before < need) {
          s_topk[at + before] = thr;
          s_topb[at + before] = b0 + lane;
        }
        const uint32_t got = min((uint32_t)__popc(m), need);
        at += got;
        need -= got;
      }
    }
    __syncthreads();
  }
  // rank among the kept: higher key first, then the lower block
  int32_t* out = a.sel + ((int64_t)h * a.NC + g) * a.K;
  if (tid < a.K) {
    if (tid == 0) out[0] = n;
    if (tid < keep) {
      int rank = 0;
      for (int i = 0; i < keep; ++i)
        rank += s_topk[i] > s_topk[tid] || (s_topk[i] == s_topk[tid] && s_topb[i] < s_topb[tid]);
      out[1 + rank] = s_topb[tid];
    }
    if (tid > keep) out[tid] = -1;
  }
}

}  // namespace cache
}  // namespace msa

using namespace msa;

namespace {

bool bad_pointers(const void* const* ptrs, int n) {
  for (int i = 0; i < n; ++i)
    if (!ptrs[i] || !aligned16(ptrs[i])) return true;
  return false;
}

}  // namespace

extern "C" {

size_t msa_cache_bytes(const msa_cache_problem* p) {
  if (cache::check_cache_problem(p) != MSA_OK) return 0;
  return (size_t)p->num_pages * p->num_kv_heads * (p->block_size / cache::kTile) * cache::kTileBytes;
}

int64_t msa_cache_chunk_bound(int64_t tokens, int64_t num_requests) {
  if (tokens < 0 || num_requests < 0) return 0;
  const int64_t x = tokens / kChunk + 2 * num_requests;
  return x < tokens ? x : tokens;
}

int msa_cache_step(const msa_cache_problem* p, const int32_t* new_lens, const int32_t* seq_lens, const int32_t* ring,
                   int32_t* free_ring, int32_t* block_table, int32_t* seq_lens_out, int32_t* ring_out,
                   int32_t* cu_tokens, int64_t* slot_map, int32_t* positions, int32_t* chunks, int32_t* d_status,
                   void* stream) {
  int rc = cache::check_cache_problem(p);
  if (rc) return rc;
  const void* ptrs[] = {new_lens, seq_lens, ring,     free_ring, block_table, seq_lens_out,
                        ring_out, cu_tokens, slot_map, positions, chunks,      d_status};
  if (bad_pointers(ptrs, 12)) return MSA_ERR_INVALID_ARGUMENT;
  if ((rc = check_device_current())) return rc;
  cache::StepArgs a{new_lens,  seq_lens, ring,      free_ring, block_table, seq_lens_out, ring_out,
                    cu_tokens, slot_map, positions, chunks,    p->num_requests, p->num_pages, p->max_blocks,
                    p->block_size, p->token_cap, p->chunk_cap, d_status};
  const size_t smem = (size_t)3 * (p->num_requests + 1) * sizeof(int32_t);
  if ((rc = cuda_status(cudaFuncSetAttribute(cache::step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             3 * (cache::kMaxRequests + 1) * (int)sizeof(int32_t)))))
    return rc;
  // CTAs of the cluster: one per 1024 chunks (or padding rows), at most 8
  const int64_t rows = p->chunk_cap > p->token_cap / 8 ? p->chunk_cap : p->token_cap / 8;
  unsigned ctas = 1;
  while (ctas < 8 && (int64_t)ctas * cache::kStepThreads < rows) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(cache::kStepThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, cache::step_kernel, a));
}

int msa_cache_append(const msa_cache_problem* p, const uint16_t* k, const uint16_t* v, const uint16_t* k_index,
                     const int64_t* slot_map, const int32_t* cu_tokens, const int32_t* chunks, uint8_t* kv_cache,
                     uint16_t* index_tail, uint16_t* index_pool, int32_t* d_status, void* stream) {
  int rc = cache::check_cache_problem(p);
  if (rc) return rc;
  const void* ptrs[] = {k, v, slot_map, kv_cache, d_status, k_index, cu_tokens, chunks, index_tail, index_pool};
  if (bad_pointers(ptrs, k_index ? 10 : 5)) return MSA_ERR_INVALID_ARGUMENT;
  if ((rc = check_device_current())) return rc;
  const int64_t T = p->token_cap, H = p->num_kv_heads, NC = p->chunk_cap;
  const int64_t kv_blocks = (T * H * 8 + 255) / 256, idx_blocks = k_index ? (NC * H * 32 + 255) / 256 : 0;
  if (kv_blocks + idx_blocks > INT32_MAX) return MSA_ERR_UNSUPPORTED_SHAPE;
  cache::AppendArgs a{k, v, k_index, slot_map, cu_tokens, chunks, kv_cache, index_tail, index_pool, (int)T, (int)H,
                      p->block_size, p->num_requests, (int)NC, (int64_t)p->num_pages * p->block_size,
                      cache::exp2i(-p->k_exp), cache::exp2i(-p->v_exp), (int)idx_blocks, d_status};
  cache::append_kernel<<<(unsigned)(kv_blocks + idx_blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

int msa_cache_read(const msa_cache_problem* p, const int64_t* slots, const uint8_t* kv_cache, uint16_t* k, uint16_t* v,
                   int32_t* d_status, void* stream) {
  int rc = cache::check_cache_problem(p);
  if (rc) return rc;
  const void* ptrs[] = {slots, kv_cache, k, v, d_status};
  if (bad_pointers(ptrs, 5)) return MSA_ERR_INVALID_ARGUMENT;
  if ((rc = check_device_current())) return rc;
  const int64_t T = p->token_cap, H = p->num_kv_heads;
  const int64_t blocks = (T * H * 8 + 255) / 256;
  if (blocks > INT32_MAX) return MSA_ERR_UNSUPPORTED_SHAPE;
  cache::ReadArgs a{slots, kv_cache, k, v, (int)T, (int)H, p->block_size, (int64_t)p->num_pages * p->block_size,
                    cache::exp2i(p->k_exp), cache::exp2i(p->v_exp), d_status};
  cache::read_kernel<<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

int msa_cache_select(const msa_cache_problem* p, const uint16_t* q_index, const uint16_t* index_pool,
                     const int32_t* block_table, const int32_t* chunks, int32_t* sel, int32_t* d_status,
                     void* stream) {
  int rc = cache::check_cache_problem(p);
  if (rc) return rc;
  const void* ptrs[] = {q_index, index_pool, block_table, chunks, sel, d_status};
  if (bad_pointers(ptrs, 6)) return MSA_ERR_INVALID_ARGUMENT;
  if ((rc = check_device_current())) return rc;
  cache::SelectArgs a{q_index, index_pool, block_table, chunks, sel, p->num_requests, p->num_pages, p->max_blocks,
                      p->block_size, p->token_cap, p->chunk_cap, p->num_kv_heads, p->topk, d_status};
  if ((rc = cuda_status(cudaFuncSetAttribute(cache::select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             cache::kMaxBlocks * 4))))
    return rc;
  cache::select_kernel<<<dim3((unsigned)p->chunk_cap, (unsigned)p->num_kv_heads), cache::kSelThreads,
                         (size_t)p->max_blocks * 4, static_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
