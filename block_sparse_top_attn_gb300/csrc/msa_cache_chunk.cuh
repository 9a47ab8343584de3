// Attention over the 4-bit cache for chunks of several tokens: per (query
// chunk, KV head) the 128 rows (8 tokens x 16 q-heads) attend the chunk's
// selected key tiles,
//   S_j = Q K_j^T, P_j = 2^(S_j - m), O += P_j V_j
// with tcgen05 MMAs of M = 128, fp32 accumulators in TMEM and P_j read from
// TMEM, as in the training forward; K_j and V_j are decoded from the cache into
// fp16 shared-memory operands by four warps of their own.
//
// A tile is decoded once for the 128 rows, against once per token in the
// single-token kernel.  Bound by shared memory: per 64-key tile 32 KB are
// stored by the decoders and 64 KB read by the MMAs (Q again for every tile),
// 768 cycles at 128 bytes a cycle, against about 700 of MMA issue.  The codes
// go from global memory to the decoders' registers one tile ahead and never
// through shared memory, which keeps 18 KB per tile off that path.
//
// Warps 0-3: softmax, one row per thread.  Warps 4-7: decoders.  Warp 8: MMA
// issue.  Warp 9: the tile lists, one item ahead.  Nothing synchronises the
// whole CTA between items: the decoders run ahead into the next item as far as
// the two K and V buffers allow.
#pragma once

namespace msa {
namespace cache {
namespace chunk {

constexpr int kThreads = 384;            // three warpgroups; two warps of the last stay idle
constexpr int kDecodeWarp = 4, kIssueWarp = 8, kListWarp = 9;
constexpr uint32_t OFF_Q = 0;            // [2 halves][128 rows][128 B]
constexpr uint32_t OFF_K = 32768;        // 2 buffers x [2 halves][64 keys][128 B]
constexpr uint32_t OFF_V = 65536;        // 2 buffers x [2 halves][64 keys][128 B]
constexpr uint32_t OFF_CTL = 98304;
constexpr uint32_t ALIGN_SLACK = 768;
constexpr uint32_t TMEM_COLS = 256;
constexpr uint32_t COL_S = 0, COL_P = 64, COL_O = 128;  // S 64 columns, P 2 x 32 (fp16 pairs), O 128

struct Control {
  uint64_t q_full;                  // Q written (4 softmax warps), one phase per item with tiles
  uint64_t k_full[2], v_full[2];    // decoded (4 decoder warps)
  uint64_t s_full[2];               // S_n done (MMA commit), by n & 1: K buffer n & 1 is free too
  uint64_t s_read;                  // S_n read (4 softmax warps)
  uint64_t p_full[2];               // P_n written, O rescaled (4 softmax warps)
  uint64_t pv_done[2];              // P_n V_n done (MMA commit), by n & 1: V buffer n & 1 is free too
  uint64_t list_full[2], list_free[2];
  uint32_t tmem;
  struct List {
    int4 row;                       // the chunk-table row
    int32_t head, ntiles;           // ntiles: -1 ends the walk
    int64_t tile[kMaxTiles];
    int32_t key0[kMaxTiles];
  } list[2];
};
constexpr uint32_t SMEM = OFF_CTL + sizeof(Control) + ALIGN_SLACK;
static_assert(2 * (SMEM + 1024) <= 227 * 1024, "two CTAs per SM");

template <int N>
MSA_DEV void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
MSA_DEV void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

MSA_DEV bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}

// One decoder thread's share of a tile: 64 dims (half a row) of one key, of K
// and of V, with their scales.
struct Codes {
  uint4 k[2], v[2];
  uint32_t ks, vs;  // four e4m3 scales each
};
MSA_DEV void load_codes(Codes& c, const uint8_t* tile, int key, int half) {
  const uint4* k = reinterpret_cast<const uint4*>(tile + OFF_KC + key * kRowBytes + half * 32);
  const uint4* v = reinterpret_cast<const uint4*>(tile + OFF_VC + v_code_offset(key, half * 4));
  c.k[0] = __ldg(k);
  c.k[1] = __ldg(k + 1);
  c.v[0] = __ldg(v);
  c.v[1] = __ldg(v + 1);
  c.ks = __ldg(reinterpret_cast<const uint32_t*>(tile + OFF_KS + key * kScales + half * 4));
  const uint8_t* s = tile + OFF_VS + half * 4 * kTile + key;
  c.vs = __ldg(s) | __ldg(s + kTile) << 8 | __ldg(s + 2 * kTile) << 16 | (uint32_t)__ldg(s + 3 * kTile) << 24;
}
// Bytes of w that are the e4m3 NaN (0x7F; scales have no sign), as 0xFF.
MSA_DEV uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w, 0x7F7F7F7Fu); }

// 64 codes to fp16 in the 128-byte swizzled row at dst (row = key).
MSA_DEV void decode_row(uint8_t* dst, const uint4 (&c)[2], uint32_t scales, int key) {
  const uint32_t s01 = e4m3x2_to_half(scales & 0xFFFFu), s23 = e4m3x2_to_half(scales >> 16);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t sp = g < 2 ? s01 : s23;
    const uint32_t sc = __byte_perm(sp, sp, (g & 1) ? 0x3232 : 0x1010);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int w = 2 * g + h;  // word of 8 dims
      const uint4& q = c[w >> 2];
      uint32_t x[4];
      e2m1x8_to_half((w & 3) == 0 ? q.x : (w & 3) == 1 ? q.y : (w & 3) == 2 ? q.z : q.w, x);
      *reinterpret_cast<uint4*>(dst + ((w ^ (key & 7)) << 4)) =
          make_uint4(mul_half2(x[0], sc), mul_half2(x[1], sc), mul_half2(x[2], sc), mul_half2(x[3], sc));
    }
  }
}

__global__ void __launch_bounds__(kThreads, 2) fwd_chunk_kernel(FwdCacheArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uintptr_t raw = reinterpret_cast<uintptr_t>(smem_raw);
  const uintptr_t pad = ((raw + 1023) & ~uintptr_t(1023)) - raw;
  if (pad > ALIGN_SLACK) {  // uniform across the block: nothing has started yet
    after_previous_kernel<false>();
    if (threadIdx.x == 0) set_status(a.status, MSA_ERR_CUDA);
    return;
  }
  uint8_t* sm = smem_raw + pad;
  Control& ct = *reinterpret_cast<Control*>(sm + OFF_CTL);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&ct.q_full, 4);
    mbar_init(&ct.s_read, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ct.k_full[i], 4);
      mbar_init(&ct.v_full[i], 4);
      mbar_init(&ct.s_full[i], 1);
      mbar_init(&ct.p_full[i], 4);
      mbar_init(&ct.pv_done[i], 1);
      mbar_init(&ct.list_full[i], 1);
      mbar_init(&ct.list_free[i], 9);  // softmax and decoder warps, the issuer
    }
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&ct.tmem, TMEM_COLS);
    tmem_relinquish();
  }
  after_previous_kernel<false>();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ct.tmem;
  const uint32_t sbase = smem_u32(sm);
  constexpr uint32_t ID_S = idesc_f16_f32(128, 64, false, false);
  constexpr uint32_t ID_O = idesc_f16_f32(128, 128, false, true);
  const int64_t items = (int64_t)a.H * a.NC;
  // Tiles are numbered through all items of the CTA: tile n uses K, V and P
  // buffer n & 1 and parity (n >> 1) & 1 of their barriers.  Item i uses list
  // buffer i & 1.
  if (warp < kDecodeWarp) {
    // ---------------- softmax, one row per thread ----------------
    regs_inc<136>();
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    uint32_t seq = 0;
    for (uint32_t i = 0;; ++i) {
      if (!warp_wait(&ct.list_full[i & 1], (i >> 1) & 1, a.status)) break;
      const Control::List& li = ct.list[i & 1];
      const int4 c = li.row;
      const int h = li.head, ntiles = li.ntiles;
      if (ntiles < 0) break;
      const int slot = tid >> 4, hh = tid & 15;
      const int qpos = slot < c.z ? c.w + slot : -1;
      const int64_t row = (int64_t)(c.y + min(slot, c.z - 1)) * a.H * kGroup + h * kGroup + hh;
      // the row of Q as fp16, scaled by a power of two that puts its largest
      // element at 2^14 (a bf16 element then loses bits only below 2^-31 of it).
      // An item without tiles has no phase of q_full: nothing would keep these
      // warps from running through several such items ahead of the issuer.
      float sc = 0.f;
      if (ntiles > 0) {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + row * 128);
        uint4 v[16];
        uint32_t amax = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          v[k] = __ldg(src + k);
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = max(amax, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
        }
        const int ex = max((int)(amax >> 7), 15);
        const float mul = __uint_as_float((uint32_t)(268 - ex) << 23);
        sc = score_factor(__uint_as_float((uint32_t)(ex - 14) << 23), a.scale_log2);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = pack_half2(__uint_as_float(w[e] << 16) * mul, __uint_as_float(w[e] & 0xFFFF0000u) * mul);
          *reinterpret_cast<uint4*>(sm + OFF_Q + (k >> 3) * 16384 + tid * 128 + (((k & 7) ^ (tid & 7)) << 4)) =
              make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      if (ntiles > 0) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.q_full);
      }
      float m_run = -CUDART_INF_F, l_run = 0.f;
      bool ok = true;
      for (int j = 0; j < ntiles; ++j) {
        const uint32_t n = seq + j, bf = n & 1;
        const int key0 = li.key0[j];
        if (!(ok = warp_wait(&ct.s_full[bf], (n >> 1) & 1, a.status))) break;
        tc_fence_after();
        float xs[64];
        {
          uint32_t sv0[32], sv1[32];
          tmem_ld32x(tmem + lane_base + COL_S, sv0);
          tmem_ld32x(tmem + lane_base + COL_S + 32, sv1);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            xs[e] = __uint_as_float(sv0[e]);
            xs[32 + e] = __uint_as_float(sv1[e]);
          }
        }
        // S_n is in registers: the next S GEMM may overwrite it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.s_read);
        if (key0 + 63 > c.w) {  // not every key precedes every row
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (key0 + e > qpos) xs[e] = -CUDART_INF_F;
        }
        float m4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int e = 0; e < 64; e += 8) {
#pragma unroll
          for (int r = 0; r < 4; ++r) m4[r] = max3(m4[r], xs[e + 2 * r], xs[e + 2 * r + 1]);
        }
        const float bmax = max3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * sc;  // log2 units (sc > 0)
        const bool upd = bmax > m_run + (kLift + kTau);
        const bool resc = upd && m_run > -CUDART_INF_F;
        const float alpha = upd ? ex2_approx(m_run + kLift - bmax) : 1.f;
        if (upd) {
          l_run *= alpha;
          m_run = bmax - kLift;
        }
        const float nm = m_run == -CUDART_INF_F ? 0.f : -m_run;
        uint32_t pk[32];
        const uint64_t sc2 = f2_pack(sc, sc), nm2 = f2_pack(nm, nm);
        uint64_t ls2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          float y0, y1;
          f2_unpack(f2_fma(f2_pack(xs[e], xs[e + 1]), sc2, nm2), y0, y1);
          const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
          ls2[(e >> 1) & 1] = f2_add(ls2[(e >> 1) & 1], f2_pack(p0, p1));
          pk[e >> 1] = pack_half2(p0, p1);  // fp16: 11 bits of a weight
        }
        {
          float a0, a1, b0, b1;
          f2_unpack(ls2[0], a0, a1);
          f2_unpack(ls2[1], b0, b1);
          l_run += (a0 + a1) + (b0 + b1);
        }
        // P V of the tile before: done before O is rescaled and before its
        // successor's P is signalled, so its phases are taken in order
        if (j > 0 && !(ok = warp_wait(&ct.pv_done[bf ^ 1], ((n - 1) >> 1) & 1, a.status))) break;
        if (__any_sync(0xffffffffu, resc)) {  // warp-collective TMEM access
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < 128; c0 += 32) {
            uint32_t ov[32];
            tmem_ld32x(tmem + lane_base + COL_O + c0, ov);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32x(tmem + lane_base + COL_O + c0, ov);
          }
        }
        tmem_st32x(tmem + lane_base + COL_P + bf * 32, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.p_full[bf]);
      }
      if (!ok) break;
      if (ntiles > 0 && !warp_wait(&ct.pv_done[(seq + ntiles - 1) & 1], ((seq + ntiles - 1) >> 1) & 1, a.status)) break;
      tc_fence_after();
      if (qpos >= 0) a.lse[row] = l_run == 0.f ? -CUDART_INF_F : (m_run + log2f(l_run)) * kLn2;
      const float inv = l_run == 0.f ? 0.f : a.v_mul / l_run;  // a NaN stays one
      // dims (groups of 16) in which a token of the chunk that this row attends
      // has a NaN value (see the decoders): the chunk's own tile, if selected
      uint32_t nan_groups = 0;
      if (c.z > 1) {
        for (int j = 0; j < ntiles; ++j)
          if (li.key0[j] == c.w / kTile * kTile) {
            const int at = c.w % kTile / 8 * 8;  // the chunk's 8 positions in the tile
            const uint8_t* vs = a.cache + li.tile[j] * kTileBytes + OFF_VS + at;
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const uint2 s8 = __ldg(reinterpret_cast<const uint2*>(vs + g * kTile));
              const uint64_t nan = (uint64_t)nan_bytes(s8.y) << 32 | nan_bytes(s8.x);
              // positions c.w + 1 .. qpos
              const int lo = c.w % 8 + 1, hi = qpos < 0 ? 0 : qpos % 8 + 1;
              const uint64_t mine = hi > lo ? (~uint64_t(0) >> (64 - 8 * (hi - lo))) << (8 * lo) : 0;
              if (nan & mine) nan_groups |= 1u << g;
            }
          }
      }
      uint4* dst = reinterpret_cast<uint4*>(a.o + row * 128);
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += 32) {
        uint32_t v[32];
        if (ntiles > 0) {
          tmem_ld32x(tmem + lane_base + COL_O + c0, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0u;
        }
        if (nan_groups) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (nan_groups >> ((c0 + e) / 16) & 1) v[e] = 0x7FC00000u;
        }
        if (qpos >= 0) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
            dst[c0 / 8 + q4] = make_uint4(
                pack_bf16x2(__uint_as_float(v[8 * q4 + 0]) * inv, __uint_as_float(v[8 * q4 + 1]) * inv),
                pack_bf16x2(__uint_as_float(v[8 * q4 + 2]) * inv, __uint_as_float(v[8 * q4 + 3]) * inv),
                pack_bf16x2(__uint_as_float(v[8 * q4 + 4]) * inv, __uint_as_float(v[8 * q4 + 5]) * inv),
                pack_bf16x2(__uint_as_float(v[8 * q4 + 6]) * inv, __uint_as_float(v[8 * q4 + 7]) * inv));
        }
      }
      tc_fence_before();
      seq += ntiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ct.list_free[i & 1]);
    }
  } else if (warp < kIssueWarp) {
    // ---------------- decoders ----------------
    regs_dec<72>();
    const int t = tid - 32 * kDecodeWarp, key = t & 63, half = t >> 6;
    uint32_t n = 0;
    for (uint32_t i = 0;; ++i) {
      if (!warp_wait(&ct.list_full[i & 1], (i >> 1) & 1, a.status)) break;
      const Control::List& li = ct.list[i & 1];
      const int ntiles = li.ntiles, last = li.row.w + li.row.z - 1;  // the chunk's last position
      if (ntiles < 0) break;
      bool ok = true;
      Codes cur, nxt;
      if (ntiles > 0) load_codes(cur, a.cache + li.tile[0] * kTileBytes, key, half);
      for (int j = 0; j < ntiles; ++j, ++n) {
        const uint32_t bf = n & 1, ph = (n >> 1) & 1;
        if (j + 1 < ntiles) load_codes(nxt, a.cache + li.tile[j + 1] * kTileBytes, key, half);
        if (n >= 2 && !(ok = warp_wait(&ct.s_full[bf], ph ^ 1, a.status))) break;  // S_{n-2} has read its K
        decode_row(sm + OFF_K + bf * 16384 + half * 8192 + key * 128, cur.k, cur.ks, key);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.k_full[bf]);
        if (n >= 2 && !(ok = warp_wait(&ct.pv_done[bf], ph ^ 1, a.status))) break;  // P V_{n-2} has read its V
        // Keys behind the chunk hold anything: a zero scale makes them zero (a
        // code alone is always finite; a weight of zero times NaN would not be).
        // A NaN value of one of the chunk's own tokens must not reach the tokens
        // before it: it counts as zero here, and the softmax warps put it into the
        // rows that attend it.
        const int pos = li.key0[j] + key;
        uint32_t vs = cur.vs;
        if (pos > li.row.w) vs = pos <= last ? vs & ~nan_bytes(vs) : 0u;
        decode_row(sm + OFF_V + bf * 16384 + half * 8192 + key * 128, cur.v, vs, key);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.v_full[bf]);
        cur = nxt;
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(&ct.list_free[i & 1]);
    }
  } else {
    regs_dec<32>();
    if (warp == kIssueWarp) {
      // ---------------- MMA issue ----------------
      uint32_t seq = 0, nq = 0;  // nq: items with tiles
      bool ok = true;
      auto issue_s = [&](uint32_t n) {
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t half = kk >> 2, sub = (kk & 3) * 32;
            umma_bf16(tmem + COL_S, sdesc_sw128(sbase + OFF_Q + half * 16384 + sub, 16, 1024),
                      sdesc_sw128(sbase + OFF_K + (n & 1) * 16384 + half * 8192 + sub, 16, 1024), ID_S, kk > 0);
          }
          umma_commit(&ct.s_full[n & 1]);
        }
        __syncwarp();
      };
      for (uint32_t i = 0;; ++i) {
        if (!warp_wait(&ct.list_full[i & 1], (i >> 1) & 1, a.status)) break;
        const int ntiles = ct.list[i & 1].ntiles;
        if (ntiles < 0) break;
        // the list is not looked at again
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.list_free[i & 1]);
        if (ntiles > 0) {
          if (!(ok = warp_wait(&ct.q_full, nq++ & 1, a.status))) break;
          // the S columns: every softmax warp has read the last item's before it wrote Q
          if (seq > 0 && !(ok = warp_wait(&ct.s_read, (seq - 1) & 1, a.status))) break;
          if (!(ok = warp_wait(&ct.k_full[seq & 1], (seq >> 1) & 1, a.status))) break;
          tc_fence_after();
          issue_s(seq);
        }
        for (int j = 0; j < ntiles; ++j) {
          const uint32_t n = seq + j, bf = n & 1;
          if (j + 1 < ntiles) {
            ok = warp_wait(&ct.k_full[bf ^ 1], ((n + 1) >> 1) & 1, a.status) && warp_wait(&ct.s_read, n & 1, a.status);
            if (!ok) break;
            tc_fence_after();
            issue_s(n + 1);
          }
          ok = warp_wait(&ct.p_full[bf], (n >> 1) & 1, a.status) && warp_wait(&ct.v_full[bf], (n >> 1) & 1, a.status);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16_ts(tmem + COL_O, tmem + COL_P + bf * 32 + kk * 8,
                           sdesc_sw128(sbase + OFF_V + bf * 16384 + kk * 2048, 8192, 1024), ID_O,
                           (j > 0 || kk > 0) ? 1u : 0u);
            umma_commit(&ct.pv_done[bf]);
          }
          __syncwarp();
        }
        if (!ok) break;
        seq += ntiles;
      }
    } else if (warp == kListWarp) {
      // ---------------- tile lists ----------------
      const bool stale = status_bad(a.status);
      uint32_t i = 0;
      for (int64_t w = blockIdx.x;; w += gridDim.x) {
        int4 c = make_int4(-1, 0, 0, 0);
        int h = 0;
        bool end = stale || w >= items;
        if (!end) {
          h = (int)(w % a.H);  // heads fastest: neighbouring CTAs read neighbouring tiles
          c = reinterpret_cast<const int4*>(a.chunks)[w / a.H];
          if (c.x < 0) continue;
        }
        int total = -1, x = 0, ntl = 0, page = 0, b = -1;
        if (!end) {
          const int entry = lane < a.K ? a.sel[((int64_t)h * a.NC + w / a.H) * a.K + lane] : -1;
          if (!list_tiles(a, c, entry, lane, b, page, ntl)) continue;
          x = ntl;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          total = __shfl_sync(0xffffffffu, x, 31);
        }
        if (i >= 2 && !warp_wait(&ct.list_free[i & 1], ((i >> 1) & 1) ^ 1, a.status)) break;
        Control::List& li = ct.list[i & 1];
        for (int k = 0; k < ntl; ++k) {
          li.tile[x - ntl + k] = tile_index(page, h, a.H, a.B / kTile, k);
          li.key0[x - ntl + k] = b * a.B + k * kTile;
        }
        if (lane == 0) {
          li.row = c;
          li.head = h;
          li.ntiles = total;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.list_full[i & 1]);
        ++i;
        if (end) break;
      }
    }
  }
  // Every role has left its loop; after a wait that gave up, the others' waits
  // have run out too.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

}  // namespace chunk
}  // namespace cache
}  // namespace msa
