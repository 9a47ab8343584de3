// Attention of a serving step's new tokens over the selected blocks of the
// 4-bit paged cache: per (query token, KV head) the 16 query heads attend the
// keys of the chunk's selected blocks at or before the token,
//   s_j = scale q k_j,  o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
// in one pass with a running maximum.
//
// Three kernels share the rounding, the tile lists and the result's definition:
//  - here, for few items: a cluster of CTAs per (token, KV head), each with a
//    share of the tiles, joined through distributed shared memory;
//  - msa_cache_batch.cuh, for many single tokens: persistent CTAs;
//  - msa_cache_chunk.cuh, for chunks of several tokens: 128 rows on tcgen05.
//
// Single tokens.  A token and KV head read 144 bytes per key and do 8192
// operations on them, 57 per byte, so the cache's bytes set the floor.  The 16
// heads of one KV head are the 16 rows of an m16n8k16 MMA, which leaves no row
// unused; a 128-row tcgen05 tile would hold one token's 16 rows and 112 empty
// ones, and its operands would have to be decoded into shared memory (64 KB
// written and read per 128 keys, more than the time of their DRAM bytes).  Codes
// become fp16 in registers, in the layout of the MMA's B fragment.  A warp takes
// 32 keys, so that four chains of score MMAs overlap (256 tokens x 8 heads x 2048
// keys: 162 us, and 214 for a form with 16 keys a warp).
// What bounds it now: about 600 instructions per 32 keys and warp, of them 128
// conversions and 128 products at two cycles each and 64 MMAs at eight.  Such a mix
// issues at most about 0.6 instructions a cycle, which would be 114 us for that
// case; the kernel takes 149 at 0.46, the rest being the latency of a tile's own
// chain.  8 warps with 200 registers: 149 us, 12 with 128: 154.
//
// In this kernel warp 0 compacts the selection and looks up the pages while warp
// 3 stages the query; whole 9 KB tiles (codes and scales of 64 keys are
// contiguous) come by bulk copies.  Two pairs of warps take alternate tiles, each
// with its own stages; each warp has its own running maximum and output, and
// nothing is shared until the tiles are done.  The parts of the warps, then those
// of the cluster's CTAs, are joined in a fixed order.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "msa_cache.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace cache {

constexpr int kConsumers = 4;
constexpr int kFwdThreads = 32 * kConsumers;
constexpr int kStages = 6, kPairStages = kStages / 2;
constexpr int kMaxTiles = 64;   // 64-key tiles of an item: up to 32 blocks of 128 keys
// Weights are p = 2^(s - m) with m kLift below the running maximum, which moves
// when a score passes it by kTau: 2^kLift <= the largest p < 2^(kLift + kTau),
// inside fp16's range, and a weight loses bits to fp16's subnormals only below
// 2^-(14 + kLift) of the largest.
constexpr float kTau = 8.f, kLift = 7.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct FwdCacheArgs {
  const uint16_t* q;
  const uint8_t* cache;
  const int32_t *block_table, *chunks, *sel;
  uint16_t* o;
  float* lse;
  int R, P, M, B, T, NC, H, K;
  int slots;         // token slots of a chunk in the grid
  float scale_log2;  // softmax scale * 2^k_exp * log2 e
  float v_mul;       // 2^v_exp
  int32_t* status;
};

struct FwdShared {
  alignas(128) uint8_t ring[kStages][kTileBytes];  // reused for the partial outputs
  alignas(8) uint64_t full[kStages], empty[kStages];
  alignas(16) uint4 q[8][32];  // the 16 query rows as A fragments of the 8 k-steps, by lane
  float qs[16];              // powers of two that undo their scaling
  int64_t tile[kMaxTiles];   // tile index in the cache
  int32_t key0[kMaxTiles];   // position of its first key
  int32_t ntiles;            // of this CTA
  int32_t skip;              // the item is refused, or a wait gave up: no CTA of the cluster writes
  float m[kConsumers][16], l[kConsumers][16];
  float cm[16], cl[16];      // joined over the warps
};
static_assert(sizeof(float) * kConsumers * 16 * 128 <= kStages * kTileBytes, "partials fit the ring");

MSA_DEV void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
MSA_DEV uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The factor that turns a row's products into powers of two.  Not below the
// smallest normal number: a masked score is -inf and has to stay it, and 0 * inf
// is not.
MSA_DEV float score_factor(float row_scale, float scale_log2) { return fmaxf(row_scale * scale_log2, 1.17549435e-38f); }

// A row of q as fp16 A-fragment words: the lane's 32 dims (32 t .. 32 t + 31),
// scaled by a power of two that puts the row's largest element at 2^14, so
// that a bf16 element loses bits only below 2^-31 of the largest.  Returns the
// inverse power.
MSA_DEV float load_q_row(const uint16_t* src, uint32_t (&w)[16]) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 x = reinterpret_cast<const uint4*>(src)[i];
    w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max(amax, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int e = max((int)(amax >> 7), 15);  // biased exponent; 15: rows of tiny values keep a normal inverse
  const float mul = __uint_as_float((uint32_t)(268 - e) << 23);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    w[i] = pack_half2(__uint_as_float(w[i] << 16) * mul, __uint_as_float(w[i] & 0xFFFF0000u) * mul);
  return __uint_as_float((uint32_t)(e - 14) << 23);
}

// One warp's 32 keys (from key kw of a tile) for the 16 rows whose A fragments
// are q: scores, running maximum m and sum l, output o.  Keys 0 .. reach of the
// 32 may be attended (reach >= 0).  sc0, sc1: the factors that turn the scores of
// rows gid and gid + 8 into powers of two.
MSA_DEV void attend32(const uint8_t* tile, int kw, int reach, const uint4 (*q)[32], float sc0, float sc1, int lane,
                      float (&o)[16][4], float (&m)[2], float (&l)[2]) {
  const int gid = lane >> 2, t = lane & 3;
  // S = Q K^T: column c of n-tile jj is key 16 (jj >> 1) + 4 (c >> 1) +
  // 2 (jj & 1) + (c & 1), k-step ks contracts dims 32 t + 4 ks .. + 3 of
  // each lane t.  The four n-tiles' chains are interleaved.
  float sv[4][4];
  uint4 kc[4];
  uint32_t ksc[4];
#pragma unroll
  for (int jj = 0; jj < 4; ++jj) {
    const int key = kw + 16 * (jj >> 1) + 4 * (gid >> 1) + 2 * (jj & 1) + (gid & 1);
    kc[jj] = *reinterpret_cast<const uint4*>(tile + OFF_KC + key * kRowBytes + t * 16);
    ksc[jj] = e4m3x2_to_half(*reinterpret_cast<const uint16_t*>(tile + OFF_KS + key * kScales + 2 * t));
    sv[jj][0] = sv[jj][1] = sv[jj][2] = sv[jj][3] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t hk[4][4];
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      e2m1x8_to_half(i == 0 ? kc[jj].x : i == 1 ? kc[jj].y : i == 2 ? kc[jj].z : kc[jj].w, hk[jj]);
      const uint32_t sc = __byte_perm(ksc[jj], ksc[jj], i < 2 ? 0x1010 : 0x3232);
#pragma unroll
      for (int e = 0; e < 4; ++e) hk[jj][e] = mul_half2(hk[jj][e], sc);
    }
    const uint4 qa = q[2 * i][lane], qb = q[2 * i + 1][lane];
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) mma_f16(sv[jj], qa.x, qa.y, qa.z, qa.w, hk[jj][0], hk[jj][1]);
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) mma_f16(sv[jj], qb.x, qb.y, qb.z, qb.w, hk[jj][2], hk[jj][3]);
  }
  // the lane's keys: 16 (jj >> 1) + 4 t + 2 (jj & 1) + e; rows gid and gid + 8
  float bm0 = -CUDART_INF_F, bm1 = -CUDART_INF_F;
  const int left = reach - 4 * t;  // its keys up to this one may be attended
  uint32_t vs[2];
#pragma unroll
  for (int st2 = 0; st2 < 2; ++st2)
    vs[st2] = *reinterpret_cast<const uint32_t*>(tile + OFF_VS + gid * kTile + kw + 16 * st2 + 4 * t);
  if (reach < 31) {
    // keys that may not be attended hold anything: their scores are
    // replaced, and a zero scale makes their values zero (a code alone is
    // always finite)
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool in = 16 * (jj >> 1) + 2 * (jj & 1) + e <= left;
        sv[jj][e] = in ? sv[jj][e] : -CUDART_INF_F;
        sv[jj][2 + e] = in ? sv[jj][2 + e] : -CUDART_INF_F;
      }
#pragma unroll
    for (int st2 = 0; st2 < 2; ++st2) {
      const int lf = left - 16 * st2;
      if (lf < 3) vs[st2] = lf < 0 ? 0u : vs[st2] & (0xFFFFFFFFu >> (8 * (3 - lf)));
    }
  }
#pragma unroll
  for (int jj = 0; jj < 4; ++jj) {
    bm0 = max3(bm0, sv[jj][0], sv[jj][1]);
    bm1 = max3(bm1, sv[jj][2], sv[jj][3]);
  }
  bm0 = fmaxf(bm0, __shfl_xor_sync(0xffffffffu, bm0, 1));
  bm1 = fmaxf(bm1, __shfl_xor_sync(0xffffffffu, bm1, 1));
  bm0 = fmaxf(bm0, __shfl_xor_sync(0xffffffffu, bm0, 2));
  bm1 = fmaxf(bm1, __shfl_xor_sync(0xffffffffu, bm1, 2));
  bm0 *= sc0;  // sc > 0, so the maximum of the scaled scores
  bm1 *= sc1;
  const bool up0 = bm0 > m[0] + (kLift + kTau), up1 = bm1 > m[1] + (kLift + kTau);
  if (__any_sync(0xffffffffu, up0 || up1)) {
    const float al0 = up0 ? ex2_approx(m[0] + kLift - bm0) : 1.f;
    const float al1 = up1 ? ex2_approx(m[1] + kLift - bm1) : 1.f;
    if (up0) m[0] = bm0 - kLift;
    if (up1) m[1] = bm1 - kLift;
    l[0] *= al0;
    l[1] *= al1;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      o[i][0] *= al0;
      o[i][1] *= al0;
      o[i][2] *= al1;
      o[i][3] *= al1;
    }
  }
  const float m0 = m[0] == -CUDART_INF_F ? 0.f : -m[0], m1 = m[1] == -CUDART_INF_F ? 0.f : -m[1];
  uint32_t pa[8];
#pragma unroll
  for (int jj = 0; jj < 4; ++jj) {
    const float p0 = ex2_approx(__fmaf_rn(sv[jj][0], sc0, m0)), p1 = ex2_approx(__fmaf_rn(sv[jj][1], sc0, m0));
    const float p2 = ex2_approx(__fmaf_rn(sv[jj][2], sc1, m1)), p3 = ex2_approx(__fmaf_rn(sv[jj][3], sc1, m1));
    l[0] += p0 + p1;
    l[1] += p2 + p3;
    // fp16 keeps 11 bits of a weight, 3 more than bf16
    pa[2 * jj] = pack_half2(p0, p1);
    pa[2 * jj + 1] = pack_half2(p2, p3);
  }
  // O += P V: column c = gid of n-tile j is dim 16 gid + j, so a lane's
  // V words are one scale group of its four keys of each 16
#pragma unroll
  for (int st2 = 0; st2 < 2; ++st2) {
    const uint32_t* p4 = &pa[4 * st2];
    uint2 vw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      vw[e] = *reinterpret_cast<const uint2*>(tile + OFF_VC + v_code_offset(kw + 16 * st2 + 4 * t + e, gid));
    const uint32_t s01 = e4m3x2_to_half(vs[st2] & 0xFFFFu), s23 = e4m3x2_to_half(vs[st2] >> 16);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      // bytes of two keys' codes at one dim, even and odd dims apart
      constexpr uint32_t LO = 0x0F0F0F0Fu;
      const uint32_t w0 = w ? vw[0].y : vw[0].x, w1 = w ? vw[1].y : vw[1].x;
      const uint32_t w2 = w ? vw[2].y : vw[2].x, w3 = w ? vw[3].y : vw[3].x;
      uint32_t ev01[4], od01[4], ev23[4], od23[4];
      e2m1x8_to_half((w0 & LO) | ((w1 << 4) & ~LO), ev01);
      e2m1x8_to_half((w2 & LO) | ((w3 << 4) & ~LO), ev23);
      e2m1x8_to_half(((w0 >> 4) & LO) | (w1 & ~LO), od01);
      e2m1x8_to_half(((w2 >> 4) & LO) | (w3 & ~LO), od23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mma_f16(o[8 * w + 2 * i], p4[0], p4[1], p4[2], p4[3], mul_half2(ev01[i], s01),
                mul_half2(ev23[i], s23));
        mma_f16(o[8 * w + 2 * i + 1], p4[0], p4[1], p4[2], p4[3], mul_half2(od01[i], s01),
                mul_half2(od23[i], s23));
      }
    }
  }
}


// A chunk's selected tiles, by one warp: lane k's block (-1: none), its page and
// the number of its 64-key tiles that start at or before the chunk's last token.
// False (and *status) if the chunk row, the selection or a page is bad.
// entry: this lane's slot of the selection (-1 beyond topk).
MSA_DEV bool list_tiles(const FwdCacheArgs& a, const int4& c, int entry, int lane, int& b, int& page, int& ntl) {
  b = max(entry, -1);
  page = 0;
  ntl = 0;
  int code = MSA_OK;
  if (c.x >= a.R || c.z < 1 || c.z > kChunk || c.y < 0 || c.y > a.T - c.z || c.w < 0 || c.w % kChunk + c.z > kChunk ||
      c.w / a.B >= a.M) {
    code = MSA_ERR_INVALID_CACHE;
  } else {
    const unsigned same = __match_any_sync(0xffffffffu, b);
    if (__any_sync(0xffffffffu, b > c.w / a.B || (b >= 0 && __popc(same) > 1))) {
      code = MSA_ERR_INVALID_SELECTION;
    } else if (b >= 0) {
      page = a.block_table[(int64_t)c.x * a.M + b];
      ntl = a.B == 128 && b * 128 + 64 <= c.w + c.z - 1 ? 2 : 1;
    }
    if (__any_sync(0xffffffffu, page < 0 || page >= a.P)) code = MSA_ERR_INVALID_CACHE;
  }
  if (code != MSA_OK) {
    if (lane == 0) set_status(a.status, code);
    return false;
  }
  return true;
}

__global__ void __launch_bounds__(kFwdThreads, 3) fwd_cache_kernel(FwdCacheArgs a) {
  extern __shared__ __align__(128) uint8_t s_raw[];
  FwdShared& s = *reinterpret_cast<FwdShared*>(s_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pair = warp >> 1;
  const int item = blockIdx.x / ranks, h = blockIdx.y;
  const int g = item / a.slots, slot = item % a.slots;
  after_previous_kernel<false>();
  // three loads in flight together: a chain of them is a good part of an item
  int entry = -1;
  bool stale = false;
  if (warp == 0) {
    stale = status_bad(a.status);
    if (lane < a.K) entry = a.sel[((int64_t)h * a.NC + g) * a.K + lane];
  }
  // the same for every CTA of the cluster, so all of them leave here or none
  const int4 c = reinterpret_cast<const int4*>(a.chunks)[g];
  if (c.x < 0 || slot >= c.z) return;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 2);
    }
    fence_mbar_init();
  }
  if (warp == 0) {
    // the chunk's tiles; rank takes every ranks-th.  The lanes vote on the status:
    // list_tiles needs all of them or none.
    int b, page, ntl;
    const bool good = !__any_sync(0xffffffffu, stale) && list_tiles(a, c, entry, lane, b, page, ntl);
    if (!good) ntl = 0;
    int x = ntl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int total = __shfl_sync(0xffffffffu, x, 31);
    if (good) {
      for (int i = 0; i < ntl; ++i) {
        const int at = x - ntl + i;
        if (at % ranks == rank) {
          s.tile[at / ranks] = tile_index(page, h, a.H, a.B / kTile, i);
          s.key0[at / ranks] = b * a.B + i * kTile;
        }
      }
    }
    if (lane == 0) {
      s.ntiles = good ? (total - rank + ranks - 1) / ranks : 0;
      s.skip = !good;
    }
  }
  // the 16 query rows of a token, by warp 3 (warp 0 has the list, warps 0 and 2
  // the copies to see to).  A row outside the tensor belongs to a refused chunk.
  auto stage_q = [&](int tok) {
    if (warp != 3) return;
    const int gid = lane >> 2, t = lane & 3;
    const int64_t row0 = (int64_t)min(max(c.y + tok, 0), a.T - 1) * a.H * kGroup + h * kGroup;
    uint32_t q0[16], q1[16];
    const uint16_t* src = a.q + (row0 + gid) * 128 + 32 * t;
    const float x0 = load_q_row(src, q0), x1 = load_q_row(src + 8 * 128, q1);
    if (t == 0) {
      s.qs[gid] = x0;
      s.qs[gid + 8] = x1;
    }
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) s.q[ks][lane] = make_uint4(q0[2 * ks], q1[2 * ks], q0[2 * ks + 1], q1[2 * ks + 1]);
  };
  stage_q(slot);
  __syncthreads();
  const int ntiles = s.ntiles;
  for (int tok = slot; tok < c.z; tok += a.slots) {
    const int qpos = c.w + tok;
    const int64_t row0 = (int64_t)(c.y + tok) * a.H * kGroup + h * kGroup;
    const int pdone = (tok - slot) / a.slots * ((ntiles - pair + 1) / 2);  // the pair's tiles of earlier tokens
    float o[16][4];
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
    bool ok = true;
    // tiles of this warp's pair: pair, pair + 2, ..., in the pair's own stages
    const int mine = (ntiles - pair + 1) / 2, ptotal = pdone + mine;
    int issued = pdone;  // copies so far (the pair's first lane)
    auto issue = [&] {
      const int st = pair * kPairStages + issued % kPairStages;
      mbar_arrive_expect_tx(&s.full[st], kTileBytes);
      bulk_load(s.ring[st], a.cache + s.tile[2 * (issued - pdone) + pair] * kTileBytes, kTileBytes, &s.full[st]);
      ++issued;
    };
    const bool loader = (warp & 1) == 0 && lane == 0;
    if (loader)
      while (issued < ptotal && issued < pdone + kPairStages) issue();
    {
      const int gid = lane >> 2;
      if (tok != slot) {
        stage_q(tok);
        __syncthreads();
      }
      const float sc0 = score_factor(s.qs[gid], a.scale_log2), sc1 = score_factor(s.qs[gid + 8], a.scale_log2);
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      for (int n = pdone; n < ptotal; ++n) {
        const int st = pair * kPairStages + n % kPairStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&s.full[st], (n / kPairStages) & 1, a.status));
        if (!ok) break;
        const uint8_t* tile = s.ring[st];
        const int kw = 32 * (warp & 1);                              // the warp's first key in the tile
        const int k0 = s.key0[2 * (n - pdone) + pair] + kw;          // and its position
        if (k0 <= qpos) {
          attend32(tile, kw, qpos - k0, s.q, sc0, sc1, lane, o, m, l);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[st]);
        // refill the stage of the tile before: its other reader is rarely late
        if (loader && n > pdone && issued < ptotal) {
          const int pn = n - 1;
          if (mbar_wait(&s.empty[pair * kPairStages + pn % kPairStages], (pn / kPairStages) & 1, a.status)) issue();
        }
        __syncwarp();
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      }
    }
    // every tile has landed and been read; after a wait that gave up, copies
    // may be in flight: they land before the CTA's shared memory is let go
    const bool bad = __syncthreads_or(!ok);
    if (bad && loader) {
      for (int n = max(issued - kPairStages, pdone); n < issued; ++n)
        mbar_wait(&s.full[pair * kPairStages + n % kPairStages], (n / kPairStages) & 1, a.status);
      s.skip = 1;
    }
    // join the warps: partial outputs in the ring, [warp][16 rows][128 dims],
    // 16-byte units XORed by row so that neither side conflicts
    float* part = reinterpret_cast<float*>(&s.ring[0][0]);
    if (!bad) {
      const int gid = lane >> 2, t = lane & 3;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = gid + 8 * r;
        if (t == 0) {
          s.m[warp][row] = m[r];
          s.l[warp][row] = l[r];
        }
        // dims 32 t + 16 e + j of the row
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int unit = 8 * t + 4 * e + i;
            *reinterpret_cast<float4*>(part + (warp * 16 + row) * 128 + 4 * (unit ^ (row & 7))) =
                make_float4(o[4 * i][2 * r + e], o[4 * i + 1][2 * r + e], o[4 * i + 2][2 * r + e],
                            o[4 * i + 3][2 * r + e]);
          }
      }
    }
    __syncthreads();
    bool skip = bad;
    if (!bad) {
      // thread: one row, 16 dims (units 4 cg .. 4 cg + 3)
      const int row = tid >> 3, cg8 = tid & 7;
      float mm = s.m[0][row];
#pragma unroll
      for (int w = 1; w < kConsumers; ++w) mm = fmaxf(mm, s.m[w][row]);
      float ll = 0.f, acc[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) {
        const float wm = s.m[w][row];
        const float f = wm == -CUDART_INF_F ? 0.f : ex2_approx(wm - mm);
        ll += f * s.l[w][row];
        if (wm != -CUDART_INF_F || s.l[w][row] != 0.f) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 x =
                *reinterpret_cast<const float4*>(part + (w * 16 + row) * 128 + 4 * ((4 * cg8 + i) ^ (row & 7)));
            acc[4 * i] += f * x.x;
            acc[4 * i + 1] += f * x.y;
            acc[4 * i + 2] += f * x.z;
            acc[4 * i + 3] += f * x.w;
          }
        }
      }
      // this CTA's part of the cluster's result, in place of warp 0's
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(part + row * 128 + 4 * ((4 * cg8 + i) ^ (row & 7))) =
            make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
      if (cg8 == 0) {
        s.cm[row] = mm;
        s.cl[row] = ll;
      }
    }
    cluster.sync();
    for (int r = 0; r < ranks; ++r) skip |= *cluster.map_shared_rank(&s.skip, r) != 0;
    // rank joins rows rank * 16 / ranks ..: a warp takes a row, a lane 4 dims
    const int rows = 16 / ranks;
    for (int i = warp; i < rows && !skip; i += kConsumers) {
      const int row = rank * rows + i, unit = lane;
      float mm = -CUDART_INF_F;
      for (int r = 0; r < ranks; ++r) mm = fmaxf(mm, *cluster.map_shared_rank(&s.cm[row], r));
      float ll = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int r = 0; r < ranks; ++r) {
        const float wm = *cluster.map_shared_rank(&s.cm[row], r), wl = *cluster.map_shared_rank(&s.cl[row], r);
        const float f = wm == -CUDART_INF_F ? 0.f : ex2_approx(wm - mm);
        ll += f * wl;
        const float4 x = *reinterpret_cast<const float4*>(
            cluster.map_shared_rank(part + row * 128 + 4 * (unit ^ (row & 7)), r));
        if (wm != -CUDART_INF_F || wl != 0.f) {
          acc[0] += f * x.x;
          acc[1] += f * x.y;
          acc[2] += f * x.z;
          acc[3] += f * x.w;
        }
      }
      const float inv = ll == 0.f ? 0.f : a.v_mul / ll;
      *reinterpret_cast<uint2*>(a.o + (row0 + row) * 128 + 4 * unit) =
          make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
      if (unit == 0) a.lse[row0 + row] = ll == 0.f ? -CUDART_INF_F : (mm + log2f(ll)) * kLn2;
    }
    cluster.sync();  // the peers' parts have been read
    if (tok + a.slots < c.z && !skip) {
      // the ring was written by the join: order that before the next copies
      fence_async_smem();
      __syncthreads();
    }
    if (skip) return;  // the same in every CTA of the cluster
  }
}

}  // namespace cache
}  // namespace msa

#include "msa_cache_batch.cuh"
#include "msa_cache_chunk.cuh"

using namespace msa;

extern "C" int msa_cache_fwd(const msa_cache_problem* p, const uint16_t* q, const uint8_t* kv_cache,
                             const int32_t* block_table, const int32_t* chunks, const int32_t* sel, uint16_t* o,
                             float* lse, int32_t* d_status, void* stream) {
  int rc = cache::check_cache_problem(p);
  if (rc) return rc;
  const void* ptrs[] = {q, kv_cache, block_table, chunks, sel, o, lse, d_status};
  for (const void* x : ptrs)
    if (!x || !aligned16(x)) return MSA_ERR_INVALID_ARGUMENT;
  if ((rc = check_device_current())) return rc;
  int32_t sms = 0;
  if ((rc = sm_count_current(&sms))) return rc;
  cache::FwdCacheArgs a;
  a.q = q; a.cache = kv_cache; a.block_table = block_table; a.chunks = chunks; a.sel = sel; a.o = o; a.lse = lse;
  a.R = p->num_requests; a.P = p->num_pages; a.M = p->max_blocks; a.B = p->block_size; a.T = p->token_cap;
  a.NC = p->chunk_cap; a.H = p->num_kv_heads; a.K = p->topk;
  a.scale_log2 = p->softmax_scale * cache::exp2i(p->k_exp) * cache::kLog2e;
  a.v_mul = cache::exp2i(p->v_exp);
  a.slots = 1;
  a.status = d_status;
  // This rule and the next ones know the capacities only: the lengths are on the
  // device.  Where chunk_cap is a bound (msa_cache_chunk_bound counts idle requests
  // too) and well above the chunks there are, few long pieces may look like single
  // tokens; the results are the same, the time is not.
  // Token slots of a chunk in the grid: one where tokens and chunk rows are
  // equal in number (decode), else twice the mean, at most 8.  A chunk with more
  // tokens than slots takes them in turn; a slot without a token costs the
  // launch of a CTA that leaves at once.
  a.slots = (int)((p->token_cap + (int64_t)p->chunk_cap - 1) / p->chunk_cap);
  if (a.slots > 1) a.slots *= 2;
  if (a.slots > kChunk) a.slots = kChunk;
  const int64_t items = (int64_t)p->chunk_cap * a.slots;
  // CTAs of a cluster share an item's tiles while that leaves at most two CTAs to
  // an SM.  Beyond that it loses: an item's start and join cost about 6 us
  // whatever its tiles (2048 items in clusters of 2: 291 us against 162).
  const int tiles = p->topk * (p->block_size / cache::kTile);
  int ranks = 1;
  while (ranks < 8 && ranks * 2 <= tiles && items * p->num_kv_heads * ranks * 2 <= 2 * sms) ranks *= 2;
  if (ranks > 1)
    return cache::launch_kernel(cache::fwd_cache_kernel, dim3((unsigned)(items * ranks), (unsigned)p->num_kv_heads),
                                cache::kFwdThreads, sizeof(cache::FwdShared), stream, (unsigned)ranks, a);
  // Chunk rows with 1.25 tokens and more on average (3 new tokens a request and
  // more, where all requests have some): the 128-row kernel, which takes the same
  // time for one token of a chunk as for eight, where the single-token kernel takes
  // them one after another (32 tiles, 8 heads: 3 tokens x 8 requests 30 against 47
  // us, 8 tokens x 16 requests 41 against 149; 2 tokens x 64 requests 85 against 87).
  // In clusters the single-token kernel is faster (32 tokens x 2 heads x 32 tiles 16
  // against 30).
  if (4 * (int64_t)p->token_cap >= 5 * (int64_t)p->chunk_cap) {
    const bool wide = cache::aligned32(q, o) && cache::aligned32(kv_cache, nullptr);
    const auto kernel = wide ? cache::chunk::fwd_chunk_kernel<true> : cache::chunk::fwd_chunk_kernel<false>;
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess) return MSA_ERR_CUDA;
    // the warpgroups' register shares add up to the launch's registers, or
    // setmaxnreg would wait for ever
    if (attr.numRegs * 3 < cache::chunk::kSoftmaxRegs + cache::chunk::kDecodeRegs + cache::chunk::kOtherRegs)
      return MSA_ERR_CUDA;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             (int)cudaSharedmemCarveoutMaxShared) != cudaSuccess)
      return MSA_ERR_CUDA;
    const int64_t chunks = (int64_t)p->chunk_cap * p->num_kv_heads;
    const int grid = (int)(chunks < 2 * sms ? chunks : 2 * sms);
    return cache::launch_kernel(kernel, dim3((unsigned)grid), cache::chunk::kThreads, cache::chunk::SMEM, stream, 1, a);
  }
  // enough items to keep every SM busy: persistent CTAs
  if (cudaFuncSetAttribute(cache::batch::fwd_batch_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                           (int)cudaSharedmemCarveoutMaxShared) != cudaSuccess)
    return MSA_ERR_CUDA;
  const int64_t all = (int64_t)p->chunk_cap * p->num_kv_heads;
  const int64_t slots = (int64_t)cache::batch::kCtasPerSm * sms;
  const int grid = (int)(all < slots ? all : slots);
  return cache::launch_kernel(cache::batch::fwd_batch_kernel, dim3((unsigned)grid), cache::batch::kThreads,
                              sizeof(cache::batch::Shared), stream, 1, a);
}
