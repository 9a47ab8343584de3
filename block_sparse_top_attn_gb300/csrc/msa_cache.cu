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

constexpr int kStepThreads = 512;
constexpr uint32_t kSat = 1u << 30;  // sums saturate here: above every capacity

// Sums of non-negative counts that saturate instead of wrapping (associative).
MSA_DEV uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }

// Largest r in [0, n) with off[r] <= x (off ascending, off[0] <= x).
__device__ __forceinline__ int last_at_or_below(const int32_t* off, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

struct StepTables {
  int32_t *cu, *chunks, *taken, *given;  // exclusive sums over the requests, [R + 1] each
  int32_t* past;                         // cached lengths
  __device__ StepTables(int32_t* s, int R)
      : cu(s), chunks(s + (R + 1)), taken(s + 2 * (R + 1)), given(s + 3 * (R + 1)), past(s + 4 * (R + 1)) {}
};
constexpr int kStepArrays = 5;

struct StepSums {
  uint32_t ntok, nchunks, ntaken, ngiven;
  int head, count;
  int err;
};

// Every CTA scans all lengths (a few KB from L2) into its shared memory, so no
// CTA waits for another's tables: see StepTables.  Thread t owns requests [t * per, t * per + per).
__device__ StepSums step_scan(const StepArgs& a, int32_t* s_off) {
  __shared__ uint32_t s_sum[4][kStepThreads / 32];
  __shared__ int s_err;
  const StepTables s(s_off, a.R);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  StepSums z;
  const bool stale = status_bad(a.status);
  z.head = a.ring[0];
  z.count = a.ring[1];
  if (tid == 0) s_err = 0;
  const int per = (a.R + kStepThreads - 1) / kStepThreads;
  uint32_t v[4] = {0, 0, 0, 0};
  int err = stale ? MSA_ERR_INVALID_ARGUMENT : 0;  // any value: skip
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r >= a.R) break;
    const int n = a.new_lens[r], past = a.seq_lens[r];
    if (n < -1 || past < 0 || past > a.M * a.B) { err = MSA_ERR_INVALID_CACHE; break; }
    if (n > a.M * a.B - past) { err = MSA_ERR_CAPACITY; break; }
    const int held = (past + a.B - 1) / a.B, m = max(n, 0);
    s.cu[r] = (int)v[0];  // within the thread's requests; its offset is added below
    s.chunks[r] = (int)v[1];
    s.taken[r] = (int)v[2];
    s.given[r] = (int)v[3];
    s.past[r] = past;
    v[0] = sat_add(v[0], m);
    if (m > 0) v[1] = sat_add(v[1], (past + m - 1) / kChunk - past / kChunk + 1);
    v[2] = sat_add(v[2], (past + m + a.B - 1) / a.B - held);
    if (n < 0) v[3] = sat_add(v[3], held);
  }
  uint32_t inc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) inc[i] = v[i];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc[i], o);
      if (lane >= o) inc[i] = sat_add(inc[i], y);
    }
  }
  if (lane == 31) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s_sum[i][warp] = inc[i];
  }
  __syncthreads();
  if (err) atomicMax(&s_err, err);
  // every warp adds up the warps before it and all of them
  uint32_t before[4], all[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = lane < kStepThreads / 32 ? s_sum[i][lane] : 0;
    before[i] = lane < warp ? x : 0;
    all[i] = x;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      before[i] = sat_add(before[i], __shfl_xor_sync(0xffffffffu, before[i], o));
      all[i] = sat_add(all[i], __shfl_xor_sync(0xffffffffu, all[i], o));
    }
  }
  uint32_t ex[4];  // exclusive: the lanes before this one in the warp, the warps before it
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc[i], 1);
    ex[i] = sat_add(before[i], lane ? y : 0);
  }
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r >= a.R) break;
    s.cu[r] += (int)ex[0];  // not used when a sum has saturated
    s.chunks[r] += (int)ex[1];
    s.taken[r] += (int)ex[2];
    s.given[r] += (int)ex[3];
  }
  if (tid == 0) s.cu[a.R] = (int)all[0];
  __syncthreads();
  z.ntok = all[0]; z.nchunks = all[1]; z.ntaken = all[2]; z.ngiven = all[3];
  z.err = s_err;
  if (!z.err) {
    if (z.head < 0 || z.head >= a.P || z.count < 0 || z.count > a.P) z.err = MSA_ERR_INVALID_CACHE;
    else if (z.ntok > (uint32_t)a.T || z.nchunks > (uint32_t)a.NC || z.ntaken > (uint32_t)z.count)
      z.err = MSA_ERR_CAPACITY;
    else if ((uint32_t)z.count - z.ntaken + z.ngiven > (uint32_t)a.P) z.err = MSA_ERR_INVALID_CACHE;
  }
  return z;
}

// The lengths, the ring and the pages of finished requests, by one CTA once
// nothing reads them any more.  The pages join the ring behind its last entry,
// in (request, block) order: those entries hold no free page, so nothing that
// the step takes from the ring is overwritten.
__device__ void step_finish(const StepArgs& a, const StepSums& z, const StepTables& s) {
  for (uint32_t j = threadIdx.x; j < z.ngiven; j += kStepThreads) {
    const int r = last_at_or_below(s.given, a.R, (int)j);
    a.free_ring[((int64_t)z.head + z.count + j) % a.P] = __ldcg(&a.block_table[(int64_t)r * a.M + j - s.given[r]]);
  }
  for (int r = threadIdx.x; r < a.R; r += kStepThreads)
    a.seq_lens_out[r] = a.new_lens[r] < 0 ? 0 : s.past[r] + s.cu[r + 1] - s.cu[r];
  if (threadIdx.x == 0) {
    a.ring_out[0] = (int)(((int64_t)z.head + z.ntaken) % a.P);
    a.ring_out[1] = (int)((uint32_t)z.count - z.ntaken + z.ngiven);
  }
}

// Latency-bound: a batch's lengths are a few KB and the outputs 12 bytes per
// token and 16 per chunk.  A token a thread (slots and positions leave in whole
// lines), then a chunk a thread.
// kCluster: the grid is one cluster, and its first CTA finishes the step behind
// a cluster barrier that follows every read of the lengths and the ring (which
// may be updated in place).  Otherwise step_finish_kernel does, in a launch of
// its own.
template <bool kCluster>
__global__ void __launch_bounds__(kStepThreads) step_kernel(StepArgs a) {
  extern __shared__ int32_t s_off[];
  const StepTables s(s_off, a.R);
  const int tid = threadIdx.x, stride = gridDim.x * kStepThreads;
  after_previous_kernel();
  const StepSums z = step_scan(a, s_off);
  if (!z.err) {
    const int ntok = (int)z.ntok, nchunks = (int)z.nchunks;
    for (int t = blockIdx.x * kStepThreads + tid; t < a.T; t += stride) {
      int64_t slot = -1;
      int pos = -1;
      if (t < ntok) {
        const int r = last_at_or_below(s.cu, a.R, t), past = s.past[r];
        pos = past + t - s.cu[r];
        const int held = (past + a.B - 1) / a.B, blk = pos / a.B;
        int page;
        if (blk < held) {
          page = a.block_table[(int64_t)r * a.M + blk];
        } else {
          page = a.free_ring[((int64_t)z.head + s.taken[r] + blk - held) % a.P];
          if (pos % a.B == 0) a.block_table[(int64_t)r * a.M + blk] = page;
        }
        slot = (int64_t)page * a.B + pos % a.B;
      }
      a.slot_map[t] = slot;
      a.positions[t] = pos;
    }
    for (int g = blockIdx.x * kStepThreads + tid; g < a.NC; g += stride) {
      int4 row = make_int4(-1, -1, -1, -1);
      if (g < nchunks) {
        const int r = last_at_or_below(s.chunks, a.R, g), past = s.past[r];
        const int c = past / kChunk + g - s.chunks[r];
        const int first = max(past, c * kChunk), last = min(past + s.cu[r + 1] - s.cu[r], c * kChunk + kChunk);
        row = make_int4(r, s.cu[r] + first - past, last - first, first);
      }
      reinterpret_cast<int4*>(a.chunks)[g] = row;
    }
    if (blockIdx.x == 0)
      for (int r = tid; r <= a.R; r += kStepThreads) a.cu_tokens[r] = s.cu[r];
  }
  if constexpr (kCluster) {
    cg::this_cluster().sync();
    if (blockIdx.x == 0 && !z.err) step_finish(a, z, s);
  }
  if (z.err && blockIdx.x == 0 && tid == 0) set_status(a.status, z.err);
}

__global__ void __launch_bounds__(kStepThreads) step_finish_kernel(StepArgs a) {
  extern __shared__ int32_t s_off[];
  after_previous_kernel();
  const StepSums z = step_scan(a, s_off);
  if (!z.err) step_finish(a, z, StepTables(s_off, a.R));
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
  int positions;  // M * B: a request's most tokens
  int64_t slots;  // P * B
  float k_mul, v_mul;  // 2^-exp
  bool wide;           // k and v are aligned to 32 bytes
  int index_blocks;    // leading CTAs that keep the pooled index keys
  int32_t* status;
};

// Token and head of the u-th row: four tokens of one head, then the next head,
// so that a warp (four rows of eight groups) covers whole sectors of a tile's
// code rows and scales when the tokens' slots follow one another.
MSA_DEV void row_of(int64_t u, int heads, int& t, int& h) {
  const int64_t quad = u >> 2;
  // 32-bit where it fits: a 64-bit division is slow
  const int64_t tq = quad < (int64_t(1) << 32) ? (uint32_t)quad / (uint32_t)heads : quad / heads;
  h = (int)(quad - tq * heads);
  t = (int)(tq * 4 + (u & 3));
}
inline int64_t row_blocks(int64_t tokens, int64_t heads, int64_t rows) {  // CTAs of `rows` rows
  return ((tokens + 3) / 4 * 4 * heads + rows - 1) / rows;
}

// Index keys of one chunk, by one CTA: a warp takes half the dims of a head at a
// time, a lane two dims, which it alone reads and writes (so that what is averaged
// before it is overwritten is read before).
MSA_DEV void index_chunk(const AppendArgs& a, int g) {
  IndexPlan x;
  if (!plan_index(a, g, threadIdx.x == 0, x)) return;
  const int64_t hs = (int64_t)a.H * 128;  // elements from one token's row to the next
  for (int unit = threadIdx.x >> 5; unit < 2 * a.H; unit += blockDim.x >> 5) {
    const int d = unit * 64 + (threadIdx.x & 31) * 2;
    uint16_t* tail = a.index_tail + (int64_t)x.r * 2 * a.B * hs + d;
    auto average = [&] {
      const int64_t slot = a.slot_map[x.last];
      if (slot < 0 || slot >= a.slots) return;  // reported by the rows' own CTAs, or left out
      const uint16_t* old = tail + (int64_t)(x.avg_blk & 1) * a.B * hs;
      float lo = 0.f, hi = 0.f;
      const int olds = max(0, x.cu0 - (x.last - (a.B - 1)));  // tokens of earlier calls
      add_rows(old, hs, olds, lo, hi);
      add_rows(a.k_index + (int64_t)(x.last - (a.B - 1) + olds) * hs + d, hs, a.B - olds, lo, hi);
      const float inv = 1.f / (float)a.B;  // a power of two: the product is the quotient
      *reinterpret_cast<uint32_t*>(a.index_pool + (slot / a.B) * hs + d) = pack_bf16x2(lo * inv, hi * inv);
    };
    if (x.last >= 0) average();
    // the rows of the incomplete block
    uint16_t* dst = tail + (int64_t)(x.open & 1) * a.B * hs;
    for (int q = x.p0; q < x.p1; q += kChunk) {
      uint32_t w[kChunk];
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (q + i < x.p1) w[i] = *reinterpret_cast<const uint32_t*>(a.k_index + (x.cu0 + q + i - x.past) * hs + d);
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (q + i < x.p1) *reinterpret_cast<uint32_t*>(dst + ((q + i) % a.B) * hs) = w[i];
    }
  }
}

__global__ void __launch_bounds__(256, 6) append_kernel(AppendArgs a) {
  after_previous_kernel();
  if (status_bad(a.status)) return;
  if ((int)blockIdx.x < a.index_blocks) {
    index_chunk(a, blockIdx.x);
    return;
  }
  // a thread takes one group of 16 dims of K and of V: no value crosses threads
  const int64_t i = (int64_t)(blockIdx.x - a.index_blocks) * blockDim.x + threadIdx.x;
  const int grp = (int)(i & 7);
  int t, h;
  row_of(i >> 3, a.H, t, h);
  if (t >= a.T) return;
  const int64_t row = (int64_t)t * a.H + h;
  const int64_t slot = a.slot_map[t];
  if (slot < 0 || slot >= a.slots) {
    if (slot != -1) set_status(a.status, MSA_ERR_INVALID_CACHE);
    return;
  }
  uint32_t kw[8], vw[8];
  load32(a.k + row * 128 + grp * 16, a.wide, kw);
  load32(a.v + row * 128 + grp * 16, a.wide, vw);
  uint2 kc, vc;
  const uint32_t ks = quantize16(kw, a.k_mul, kc), vs = quantize16(vw, a.v_mul, vc);
  const int lb = a.B == 128 ? 7 : 6;  // log2 of the block
  const int off = (int)(slot & (a.B - 1)), tok = off % kTile;
  uint8_t* tile = a.cache + tile_index(slot >> lb, h, a.H, a.B / kTile, off / kTile) * kTileBytes;
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
  bool wide;           // k and v are aligned to 32 bytes
  int32_t* status;
};

// 16 codes and their scale as bf16.
MSA_DEV void dequantize16(uint2 codes, uint32_t scale, float mul, uint16_t* dst, bool wide) {
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
  store32(dst, wide, out);
}

// A thread takes the same group of two rows, so that two chains of loads (slot,
// then codes and scales) are in flight: the kernel is bound by their latency.
__global__ void __launch_bounds__(256) read_kernel(ReadArgs a) {
  after_previous_kernel();
  if (status_bad(a.status)) return;
  const int grp = threadIdx.x & 7;
  const int lb = a.B == 128 ? 7 : 6;  // log2 of the block
  const uint8_t* tile[2];
  int64_t row[2];
  int tok[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int t, h;
    row_of(((int64_t)blockIdx.x * 2 + i) * (256 / 8) + (threadIdx.x >> 3), a.H, t, h);
    tile[i] = nullptr;
    if (t >= a.T) continue;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.nslots) {
      if (slot != -1) set_status(a.status, MSA_ERR_INVALID_CACHE);
      continue;
    }
    const int off = (int)(slot & (a.B - 1));
    row[i] = ((int64_t)t * a.H + h) * 128 + grp * 16;
    tok[i] = off % kTile;
    tile[i] = a.cache + tile_index(slot >> lb, h, a.H, a.B / kTile, off / kTile) * kTileBytes;
  }
  uint2 kc[2], vc[2];
  uint32_t ks[2], vs[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!tile[i]) continue;
    kc[i] = *reinterpret_cast<const uint2*>(tile[i] + OFF_KC + tok[i] * kRowBytes + grp * 8);
    vc[i] = *reinterpret_cast<const uint2*>(tile[i] + OFF_VC + v_code_offset(tok[i], grp));
    ks[i] = tile[i][OFF_KS + tok[i] * kScales + grp];
    vs[i] = tile[i][OFF_VS + grp * kTile + tok[i]];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!tile[i]) continue;
    dequantize16(kc[i], ks[i], a.k_mul, a.k + row[i], a.wide);
    dequantize16(vc[i], vs[i], a.v_mul, a.v + row[i], a.wide);
  }
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

// A score as an unsigned key of the same order (-0 counts as +0).
MSA_DEV uint32_t score_key(float s) {
  const uint32_t u = __float_as_uint(__fadd_rn(s, 0.f));
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kCand = 128;  // candidates that the final ranking takes

// Scratch of one row's selection.
struct SelectScratch {
  uint32_t hist[256];        // digit d at [(255 - d) % 8][(255 - d) / 8]: a lane's eight lie in eight rows
  uint32_t prefix, need, bin, count;
  uint64_t cand[kCand];      // key, then the complement of the block: a larger number is better
};

// The topk - 1 best of n keys, by NT threads (a warp, or the whole CTA).  A
// radix selection of the keep-th largest key, 8 bits a pass, until the keys of
// the threshold's digits and above are few (two passes but for heavy ties); those
// are then ranked against one another as (key, block), which settles ties.
template <int NT>
__device__ void select_row(const uint32_t* key, int n, int K, SelectScratch& s, int32_t* out) {
  const int tid = threadIdx.x % NT, lane = tid & 31;
  auto sync = [] {
    if constexpr (NT == 32) __syncwarp(); else __syncthreads();
  };
  const int keep = min(K - 1, n);
  if (tid == 0) {
    s.prefix = 0;
    s.need = keep;
    s.bin = n;
    s.count = 0;
  }
  sync();
  int shift = 32;  // digits above this are settled: keys >= prefix in them are candidates
  while (shift > 0 && (uint32_t)keep - s.need + s.bin > (uint32_t)kCand) {
    shift -= 8;
    for (int i = tid; i < 256; i += NT) s.hist[i] = 0;
    const uint32_t prefix = s.prefix, need = s.need;
    sync();
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int b = tid; b < n; b += NT) {
      const uint32_t k = key[b];
      if ((k & mask) == prefix) {
        const uint32_t e = 255 - ((k >> shift) & 255);
        atomicAdd(&s.hist[(e & 7) * 32 + (e >> 3)], 1u);
      }
    }
    sync();
    if (tid < 32) {
      // digits from the top: lane l holds digits 255 - 8l .. 248 - 8l
      uint32_t cnt[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) { cnt[i] = s.hist[i * 32 + lane]; sum += cnt[i]; }
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
        s.prefix = prefix | ((uint32_t)(255 - 8 * lane - i) << shift);
        s.need = need - above;
        s.bin = cnt[i];
      }
    }
    sync();
  }
  const uint32_t prefix = s.prefix;  // keys >= it are candidates, keep - need of them above its digits
  if (keep > 0) {
    if (shift > 0 || (uint32_t)keep - s.need + s.bin <= (uint32_t)kCand) {
      for (int b = tid; b < n; b += NT)
        if (key[b] >= prefix) s.cand[atomicAdd(&s.count, 1u)] = (uint64_t)key[b] << 32 | (uint32_t)~b;
      sync();
    } else {
      // more equal keys than the list holds: those above, then the lowest blocks
      for (int b = tid; b < n; b += NT)
        if (key[b] > prefix) s.cand[atomicAdd(&s.count, 1u)] = (uint64_t)key[b] << 32 | (uint32_t)~b;
      sync();
      if (tid < 32) {
        uint32_t at = s.count, need = s.need;
        for (int b0 = 0; b0 < n && need; b0 += 32) {
          const bool eq = b0 + lane < n && key[b0 + lane] == prefix;
          const uint32_t m = __ballot_sync(0xffffffffu, eq);
          const uint32_t before = __popc(m & ((1u << lane) - 1u));
          if (eq && before < need) s.cand[at + before] = (uint64_t)prefix << 32 | (uint32_t)~(b0 + lane);
          const uint32_t got = min((uint32_t)__popc(m), need);
          at += got;
          need -= got;
        }
        if (lane == 0) s.count = at;
      }
      sync();
    }
    const int count = (int)s.count;
    for (int i = tid; i < count; i += NT) {
      const uint64_t mine = s.cand[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < count; ++j) rank += s.cand[j] > mine;
      if (rank < keep) out[1 + rank] = (int32_t)~(uint32_t)mine;
    }
  }
  if (tid == 0) out[0] = n;
  for (int i = tid; i < K; i += NT)
    if (i > keep) out[i] = -1;
}

// A CTA scores G consecutive chunks of one head (G = 1, or 8: one warp's
// selection each).  The pooled keys of a request are read once for all of its
// chunks in the CTA: a warp copies 32 of them (256 bytes each, from 32 pages)
// into shared memory, two whole rows per asynchronous copy, and a lane then
// takes a key, so that every score keeps its order of additions.  Read by each
// lane from global memory instead, 32 rows per load cost 32 cycles of the L1's
// tags (64 x 8 rows of 1024 keys: 42 us); one bulk copy a row is held to about
// 18 cycles each (34 us).  Rows are 272 bytes apart: eight lanes' 16-byte reads
// cover all banks.
template <int G, int W>
struct SelectShared {
  static constexpr int kWarps = W;
  static constexpr int kPitch = 272;
  alignas(16) uint8_t rows[kWarps][32 * kPitch];
  alignas(16) float q[G][128];
  SelectScratch scratch[G];
  int n[G];
};

template <int G, int W>
__global__ void __launch_bounds__(32 * W, 1) select_kernel(SelectArgs a) {
  using S = SelectShared<G, W>;
  constexpr int kThreads = 32 * S::kWarps;
  extern __shared__ __align__(16) uint8_t s_raw[];
  S& s = *reinterpret_cast<S*>(s_raw);
  uint32_t* s_key = reinterpret_cast<uint32_t*>(s_raw + sizeof(S));  // [G][M]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // heads fastest: CTAs that run together read neighbouring rows of a page
  const int g0 = (int)(blockIdx.x / a.H) * G, h = (int)(blockIdx.x % a.H);
  const int64_t hs = (int64_t)a.H * 128;
  after_previous_kernel();
  // lane r of every warp holds chunk row g0 + r
  int4 mine = make_int4(-1, 0, 0, 0);
  if (lane < G && g0 + lane < a.NC) mine = reinterpret_cast<const int4*>(a.chunks)[g0 + lane];
  // One decision for the CTA: another CTA may set the status between two warps'
  // reads, and a warp that left would leave shared memory behind that the others
  // take rows' lengths and list positions from.
  if (__syncthreads_or(status_bad(a.status))) return;
  for (int lo = 0, hi; lo < G; lo = hi) {
    // a run of chunks of one request
    hi = lo + 1;
    const int request = __shfl_sync(0xffffffffu, mine.x, lo);
    if (request < 0) continue;
    if constexpr (G > 1) {
      const unsigned other = __ballot_sync(0xffffffffu, lane >= G || mine.x != request) >> lo;
      hi = lo + __ffs(other) - 1;  // lane 31 is always another
    }
    int most = lane >= lo && lane < hi ? mine.w : -1;
    if constexpr (G > 1) {
#pragma unroll
      for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    } else {
      most = __shfl_sync(0xffffffffu, most, 0);
    }
    __syncthreads();  // the run before has been read
    const int nmax = request < a.R && most >= 0 ? min(most / a.B, a.M) : 0;
    const int32_t* table = a.block_table + (int64_t)request * a.M;
    // this lane's page of the 32 keys from block b0 on
    auto page_of = [&](int b0) {
      int page = b0 + lane < nmax ? table[b0 + lane] : 0;
      if (page < 0 || page >= a.P) {
        set_status(a.status, MSA_ERR_INVALID_CACHE);
        page = 0;
      }
      return page;
    };
    auto copy = [&](int b0, int pages) {
      const int part = lane & 15;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = 2 * i + (lane >> 4);
        const int64_t page = __shfl_sync(0xffffffffu, pages, row);
        if (b0 + row < nmax)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           smem_u32(&s.rows[warp][row * S::kPitch + part * 16])),
                       "l"(a.pool + page * hs + h * 128 + part * 8)
                       : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int pages = 0;
    if (warp * 32 < nmax) {
      copy(warp * 32, page_of(warp * 32));
      pages = page_of(warp * 32 + kThreads);
    }
    // pooled queries and the rows' numbers of earlier blocks (-1: a bad row)
    for (int i = tid; i < (hi - lo) * 128; i += kThreads) {
      const int row = i >> 7, d = i & 127;
      const int src_lane = lo + row;  // the same for a warp's 32 dims
      const int4 cc = make_int4(__shfl_sync(0xffffffffu, mine.x, src_lane), __shfl_sync(0xffffffffu, mine.y, src_lane),
                                __shfl_sync(0xffffffffu, mine.z, src_lane), __shfl_sync(0xffffffffu, mine.w, src_lane));
      const bool good = cc.x < a.R && cc.z >= 1 && cc.z <= kChunk && cc.y >= 0 && cc.y <= a.T - cc.z && cc.w >= 0 &&
                        cc.w / a.B < a.M;
      float acc = 0.f;
      if (good) {
        const uint16_t* src = a.q_index + (int64_t)cc.y * hs + h * 128 + d;
        uint16_t x[kChunk];
#pragma unroll
        for (int k = 0; k < kChunk; ++k) x[k] = k < cc.z ? src[k * hs] : 0;
#pragma unroll
        for (int k = 0; k < kChunk; ++k)
          if (k < cc.z) acc = __fadd_rn(acc, __uint_as_float((uint32_t)x[k] << 16));
        acc = __uint_as_float(pack_bf16x2(__fdiv_rn(acc, (float)cc.z), 0.f) << 16);
      }
      s.q[row][d] = acc;
      if (d == 0) {
        s.n[row] = good ? cc.w / a.B : -1;
        if (!good) set_status(a.status, MSA_ERR_INVALID_CACHE);
      }
    }
    __syncthreads();
    for (int b0 = warp * 32; b0 < nmax; b0 += kThreads) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
      float x[G];
#pragma unroll
      for (int r = 0; r < G; ++r) x[r] = 0.f;
      const uint8_t* src = &s.rows[warp][lane * S::kPitch];
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const uint4 u = *reinterpret_cast<const uint4*>(src + 16 * i);
#pragma unroll
        for (int r = 0; r < G; ++r) {
          const float4 qa = *reinterpret_cast<const float4*>(&s.q[r][8 * i]);
          const float4 qb = *reinterpret_cast<const float4*>(&s.q[r][8 * i + 4]);
          x[r] = __fmaf_rn(qa.x, __uint_as_float(u.x << 16), x[r]);
          x[r] = __fmaf_rn(qa.y, __uint_as_float(u.x & 0xFFFF0000u), x[r]);
          x[r] = __fmaf_rn(qa.z, __uint_as_float(u.y << 16), x[r]);
          x[r] = __fmaf_rn(qa.w, __uint_as_float(u.y & 0xFFFF0000u), x[r]);
          x[r] = __fmaf_rn(qb.x, __uint_as_float(u.z << 16), x[r]);
          x[r] = __fmaf_rn(qb.y, __uint_as_float(u.z & 0xFFFF0000u), x[r]);
          x[r] = __fmaf_rn(qb.z, __uint_as_float(u.w << 16), x[r]);
          x[r] = __fmaf_rn(qb.w, __uint_as_float(u.w & 0xFFFF0000u), x[r]);
        }
      }
      __syncwarp();  // every lane has read its key: the rows may be overwritten
      if (b0 + kThreads < nmax) {
        copy(b0 + kThreads, pages);
        pages = page_of(b0 + 2 * kThreads);
      }
      if (b0 + lane < nmax) {
#pragma unroll
        for (int r = 0; r < G; ++r)
          if (r < hi - lo) s_key[(int64_t)r * a.M + b0 + lane] = score_key(x[r]);
      }
    }
    __syncthreads();
    if constexpr (G == 1) {
      if (s.n[0] >= 0) select_row<kThreads>(s_key, s.n[0], a.K, s.scratch[0], a.sel + ((int64_t)h * a.NC + g0) * a.K);
    } else {
      static_assert(G <= S::kWarps, "a warp per row");
      if (warp < hi - lo && s.n[warp] >= 0)
        select_row<32>(s_key + (int64_t)warp * a.M, s.n[warp], a.K, s.scratch[warp],
                       a.sel + ((int64_t)h * a.NC + g0 + lo + warp) * a.K);
    }
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
  const size_t row = (size_t)cache::kStepArrays * sizeof(int32_t);
  const size_t smem = row * (p->num_requests + 1), largest = row * (cache::kMaxRequests + 1);
  // CTAs: a token (or chunk) a thread.  Up to 32 x 512 rows form one cluster and one launch;
  // above that a grid over the GPU and a second launch that finishes the step.
  const int64_t rows = p->chunk_cap > p->token_cap ? p->chunk_cap : p->token_cap;
  const int64_t want = (rows + cache::kStepThreads - 1) / cache::kStepThreads;
  if (want <= 32) {
    unsigned ctas = 1;
    while (ctas < 8 && ctas < want) ctas *= 2;
    return cache::launch_kernel(cache::step_kernel<true>, dim3(ctas), cache::kStepThreads, smem, stream, ctas, a,
                                largest);
  }
  int32_t sms = 0;
  if ((rc = sm_count_current(&sms))) return rc;
  rc = cache::launch_kernel(cache::step_kernel<false>, dim3((unsigned)(want < sms ? want : sms)), cache::kStepThreads,
                            smem, stream, 1, a, largest);
  if (rc) return rc;
  return cache::launch_kernel(cache::step_finish_kernel, dim3(1), cache::kStepThreads, smem, stream, 1, a, largest);
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
  const int64_t kv_blocks = cache::row_blocks(T, H, 32), idx_blocks = k_index ? NC : 0;
  if (kv_blocks + idx_blocks > INT32_MAX) return MSA_ERR_UNSUPPORTED_SHAPE;
  cache::AppendArgs a{k, v, k_index, slot_map, cu_tokens, chunks, kv_cache, index_tail, index_pool, (int)T, (int)H,
                      p->block_size, p->num_requests, (int)NC, p->max_blocks * p->block_size,
                      (int64_t)p->num_pages * p->block_size, cache::exp2i(-p->k_exp), cache::exp2i(-p->v_exp),
                      cache::aligned32(k, v), (int)idx_blocks, d_status};
  return cache::launch_kernel(cache::append_kernel, dim3((unsigned)(kv_blocks + idx_blocks)), 256, 0, stream, 1, a);
}

int msa_cache_read(const msa_cache_problem* p, const int64_t* slots, const uint8_t* kv_cache, uint16_t* k, uint16_t* v,
                   int32_t* d_status, void* stream) {
  int rc = cache::check_cache_problem(p);
  if (rc) return rc;
  const void* ptrs[] = {slots, kv_cache, k, v, d_status};
  if (bad_pointers(ptrs, 5)) return MSA_ERR_INVALID_ARGUMENT;
  if ((rc = check_device_current())) return rc;
  const int64_t T = p->token_cap, H = p->num_kv_heads;
  const int64_t blocks = cache::row_blocks(T, H, 64);
  if (blocks > INT32_MAX) return MSA_ERR_UNSUPPORTED_SHAPE;
  cache::ReadArgs a{slots, kv_cache, k, v, (int)T, (int)H, p->block_size, (int64_t)p->num_pages * p->block_size,
                    cache::exp2i(p->k_exp), cache::exp2i(p->v_exp), cache::aligned32(k, v), d_status};
  return cache::launch_kernel(cache::read_kernel, dim3((unsigned)blocks), 256, 0, stream, 1, a);
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
  // Chunks of several tokens (by the capacities: the lengths are on the device)
  // come from prompts, whose chunks share a request's keys: 8 of them to a CTA,
  // while 8 rows of scores fit shared memory.  (One to a CTA: 62 us for the same
  // prompts.)
  const int64_t H = p->num_kv_heads, NC = p->chunk_cap;
  if (NC * H > INT32_MAX) return MSA_ERR_UNSUPPORTED_SHAPE;
  const size_t row = (size_t)p->max_blocks * 4;
  constexpr size_t kSmem = 227 * 1024;
  auto launch = [&](auto kernel, size_t smem, int64_t ctas, int threads) {
    return cache::launch_kernel(kernel, dim3((unsigned)ctas), threads, smem, stream, 1, a, kSmem);
  };
  if (p->token_cap / p->chunk_cap >= 3) {
    // 16 warps share the eight chunks' 500 keys better than 8 do (21 against
    // 24 us for 2 x 2048 tokens over 32k cached ones)
    const size_t s16 = sizeof(cache::SelectShared<8, 16>) + 8 * row, s8 = sizeof(cache::SelectShared<8, 8>) + 8 * row;
    if (s16 <= kSmem) return launch(cache::select_kernel<8, 16>, s16, (NC + 7) / 8 * H, 512);
    if (s8 <= kSmem) return launch(cache::select_kernel<8, 8>, s8, (NC + 7) / 8 * H, 256);
  }
  if (sizeof(cache::SelectShared<1, 4>) + row <= kSmem)
    return launch(cache::select_kernel<1, 4>, sizeof(cache::SelectShared<1, 4>) + row, NC * H, 128);
  // the longest tables: a warp less, so that the scores fit
  static_assert(sizeof(cache::SelectShared<1, 3>) + cache::kMaxBlocks * 4 <= kSmem, "the longest table's scores fit");
  return launch(cache::select_kernel<1, 3>, sizeof(cache::SelectShared<1, 3>) + row, NC * H, 96);
}

}  // extern "C"
