// Attention over the 4-bit cache for chunks of several tokens: per (query
// chunk, KV head) the 128 rows (8 tokens x 16 q-heads) attend the chunk's
// selected key tiles,
//   S_j = Q K_j^T, P_j = 2^(S_j - m), O += P_j V_j
// with tcgen05 MMAs of M = 128, fp32 accumulators in TMEM and P_j read from
// TMEM, as in the training forward; K_j and V_j are decoded from the cache into
// fp16 shared-memory operands by four warps of their own.
//
// A tile is decoded once for the 128 rows, against once per token in the
// single-token kernel.  Per 64-key tile 32 KB are stored to shared memory by the
// decoders and 64 KB read by the MMAs (Q again for every tile): 768 cycles at 128
// bytes a cycle, against about 700 of MMA issue and 1230 measured: instruction
// issue, shared memory and the chain S, softmax, P V are all half used, and
// instruction fetches are the most frequent of the stalls that are not waits.
// The codes go from global memory to the decoders' registers and never through
// shared memory, which keeps 18 KB per tile off that path.  A row's next codes are
// loaded as soon as its registers are free, K after K, V after V: loads before the
// decoding of K hold up its stores, and S waits for K (220 against 217 us).
//
// S has two buffers, so that S_{n+1} runs during the softmax of S_n; P_n takes the
// place of its own S_n, which is what makes room for them in the 256 columns that
// two CTAs per SM leave each (with one S and two P: 248 against 243 us).  S and P V
// are issued by threads of their own, whose waits then do not delay each other's MMAs.
//
// Warps 0-3: softmax, one row per thread.  Warps 4-7: decoders.  Warps 8 and 9: issue of
// the S and the P V MMAs.  Warp 10: the tile lists, one item ahead, and what takes a
// chain of loads: the next item's Q on its way to L2, NaNs among the chunk's own
// values (236 us with these, 241 without).  Nothing synchronises the whole CTA
// between items: the decoders run ahead into the next item as far as the two K
// and V buffers allow.  (A next item's Q or codes loaded before this one's end:
// 239 and 232 us, slower although the waits are shorter.)
//
// Times: 3.4k new tokens x 4 heads x 2048 keys, 195 us (983 TFLOP/s); 4k x 8 heads
// the same 492 us (1102 TFLOP/s).
#pragma once

namespace msa {
namespace cache {
namespace chunk {

constexpr int kThreads = 384;            // three warpgroups; a warp of the last stays idle
// of a thread, by warpgroup: the softmax needs no more, as it reads S in halves, and the issuers keep
// their descriptors (88, 72, 80 gives 210 us, 104, 72, 64 214, none of its own to a warpgroup 221, against 207)
constexpr int kSoftmaxRegs = 104, kDecodeRegs = 64, kOtherRegs = 72;
constexpr int kDecodeWarp = 4, kScoreWarp = 8, kOutWarp = 9, kListWarp = 10;
constexpr uint32_t OFF_Q = 0;            // [2 halves][128 rows][128 B]
constexpr uint32_t OFF_K = 32768;        // 2 buffers x [2 halves][64 keys][128 B]
constexpr uint32_t OFF_V = 65536;        // 2 buffers x [2 halves][64 keys][128 B]
constexpr uint32_t OFF_CTL = 98304;
constexpr uint32_t ALIGN_SLACK = 768;
constexpr uint32_t TMEM_COLS = 256;
constexpr uint32_t COL_S = 0, COL_O = 128;  // S 2 x 64 columns (P, fp16 pairs, over the first 32 of its own), O 128

struct Control {
  uint64_t q_full;                  // Q written (4 softmax warps), one phase per item with tiles
  uint64_t k_full[2], v_full[2];    // decoded (4 decoder warps)
  uint64_t s_full[2];               // S_n done (MMA commit), by n & 1: K buffer n & 1 is free too
  uint64_t p_full[2];               // P_n written, O rescaled (4 softmax warps)
  uint64_t pv_done[2];              // P_n V_n done (MMA commit), by n & 1: V and S buffer n & 1 are free too
  uint64_t list_full[2], list_free[2];
  uint32_t tmem;
  int32_t gave_up;                  // a wait ran out
  struct List {
    int4 row;                       // the chunk-table row
    int32_t head, ntiles;           // ntiles: -1 ends the walk
    // bit p of byte g: the value of the chunk's position p (of 8) is NaN in dims
    // 16 g .. 16 g + 15; bits of positions without a token hold anything
    alignas(8) uint8_t nan[8];
    int64_t tile[kMaxTiles];
    int32_t key0[kMaxTiles];
  } list[2];
};
constexpr uint32_t SMEM = OFF_CTL + sizeof(Control) + ALIGN_SLACK;
static_assert(2 * (SMEM + 1024) <= 227 * 1024, "two CTAs per SM");

MSA_DEV void tmem_st16x(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
template <int N>
MSA_DEV void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
MSA_DEV void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// mbar_wait in few instructions: six roles' loops share the instruction cache (208
// us with mbar_wait, 199 with this).  A wait that gives up leaves a mark, which
// becomes the status at the end.
MSA_DEV bool short_wait(uint64_t* bar, uint32_t parity, int32_t* gave_up) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
#pragma unroll 1
  do {
    if (mbar_try_wait(bar, parity)) return true;
  } while (global_ns() - t0 <= kWaitLimitNs);
  *gave_up = 1;
  return false;
}
MSA_DEV bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* gave_up) {
  return __all_sync(0xffffffffu, short_wait(bar, parity, gave_up));
}

// One decoder thread's share of a tile: 64 dims (half a row) of one key, of K
// and of V, with their scales.
struct Codes {
  uint32_t w[8];
  uint32_t scales;  // four e4m3
};
template <bool kWide>
MSA_DEV void load_k(Codes& c, const uint8_t* tile, int key, int half) {
  load32(tile + OFF_KC + key * kRowBytes + half * 32, kWide, c.w);
  c.scales = *reinterpret_cast<const uint32_t*>(tile + OFF_KS + key * kScales + half * 4);
}
template <bool kWide>
MSA_DEV void load_v(Codes& c, const uint8_t* tile, int key, int half) {
  load32(tile + OFF_VC + v_code_offset(key, half * 4), kWide, c.w);
  const uint8_t* s = tile + OFF_VS + half * 4 * kTile + key;
  c.scales = s[0] | s[kTile] << 8 | s[2 * kTile] << 16 | (uint32_t)s[3 * kTile] << 24;
}
// Bytes of w that are the e4m3 NaN (0x7F; scales have no sign), as 0xFF.
MSA_DEV uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w, 0x7F7F7F7Fu); }

// 64 codes to fp16 in the 128-byte swizzled row at dst (row = key).
MSA_DEV void decode_row(uint8_t* dst, const uint32_t (&c)[8], uint32_t scales, int key) {
  const uint32_t s01 = e4m3x2_to_half(scales & 0xFFFFu), s23 = e4m3x2_to_half(scales >> 16);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t sp = g < 2 ? s01 : s23;
    const uint32_t sc = __byte_perm(sp, sp, (g & 1) ? 0x3232 : 0x1010);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int w = 2 * g + h;  // word of 8 dims
      uint32_t x[4];
      e2m1x8_to_half(c[w], x);
      *reinterpret_cast<uint4*>(dst + ((w ^ (key & 7)) << 4)) =
          make_uint4(mul_half2(x[0], sc), mul_half2(x[1], sc), mul_half2(x[2], sc), mul_half2(x[3], sc));
    }
  }
}

// kWide: q, o and the cache are aligned to 32 bytes (a flag at run time is two
// paths in the decoders' loop: 234 against 231 us)
template <bool kWide>
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
    ct.gave_up = 0;
    mbar_init(&ct.q_full, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ct.k_full[i], 4);
      mbar_init(&ct.v_full[i], 4);
      mbar_init(&ct.s_full[i], 1);
      mbar_init(&ct.p_full[i], 4);
      mbar_init(&ct.pv_done[i], 1);
      mbar_init(&ct.list_full[i], 1);
      mbar_init(&ct.list_free[i], 10);  // softmax and decoder warps, the two issuers
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
  // Tiles are numbered through all items of the CTA: tile n uses K, V and S
  // buffer n & 1 and parity (n >> 1) & 1 of their barriers.  Item i uses list
  // buffer i & 1.
  if (warp < kDecodeWarp) {
    // ---------------- softmax, one row per thread ----------------
    regs_inc<kSoftmaxRegs>();
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    uint32_t seq = 0;
    for (uint32_t i = 0;; ++i) {
      if (!warp_wait(&ct.list_full[i & 1], (i >> 1) & 1, &ct.gave_up)) break;
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
        uint32_t v[8][8];
        uint32_t amax = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          load32(a.q + row * 128 + k * 16, kWide, v[k]);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = max(amax, max(v[k][e] & 0x7FFFu, (v[k][e] >> 16) & 0x7FFFu));
        }
        const int ex = max((int)(amax >> 7), 15);
        const float mul = __uint_as_float((uint32_t)(268 - ex) << 23);
        sc = score_factor(__uint_as_float((uint32_t)(ex - 14) << 23), a.scale_log2);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t w = v[k >> 1][(k & 1) * 4 + e];
            y[e] = pack_half2(__uint_as_float(w << 16) * mul, __uint_as_float(w & 0xFFFF0000u) * mul);
          }
          *reinterpret_cast<uint4*>(sm + OFF_Q + (k >> 3) * 16384 + tid * 128 + (((k & 7) ^ (tid & 7)) << 4)) =
              make_uint4(y[0], y[1], y[2], y[3]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.q_full);
      }
      float m_run = -CUDART_INF_F, l_run = 0.f;
      bool ok = true;
      for (int j = 0; j < ntiles; ++j) {
        const uint32_t n = seq + j, bf = n & 1;
        const int key0 = li.key0[j];
        if (!(ok = warp_wait(&ct.s_full[bf], (n >> 1) & 1, &ct.gave_up))) break;
        tc_fence_after();
        const uint32_t col = tmem + lane_base + COL_S + bf * 64;
        // Two halves of 32 columns, read once for the maximum and once for the weights:
        // half the instructions of one long run, and half the registers.
        float m4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll 1
        for (int hf = 0; hf < 64; hf += 32) {
          uint32_t sv[32];
          tmem_ld32x(col + hf, sv);
          tmem_ld_wait();
          if (key0 + 63 > c.w) {  // not every key precedes every row
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (key0 + hf + e > qpos) sv[e] = 0xFF800000u;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              m4[r] = max3(m4[r], __uint_as_float(sv[e + 2 * r]), __uint_as_float(sv[e + 2 * r + 1]));
          }
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
        const uint64_t sc2 = f2_pack(sc, sc), nm2 = f2_pack(nm, nm);
        uint64_t ls2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll 1
        for (int hf = 0; hf < 64; hf += 32) {
          uint32_t sv[32], pk[16];
          tmem_ld32x(col + hf, sv);
          tmem_ld_wait();
          if (key0 + 63 > c.w) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (key0 + hf + e > qpos) sv[e] = 0xFF800000u;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float y0, y1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), sc2, nm2), y0, y1);
            const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
            ls2[(e >> 1) & 1] = f2_add(ls2[(e >> 1) & 1], f2_pack(p0, p1));
            pk[e >> 1] = pack_half2(p0, p1);  // fp16: 11 bits of a weight
          }
          tmem_st16x(col + hf / 2, pk);  // columns that have been read
        }
        {
          float a0, a1, b0, b1;
          f2_unpack(ls2[0], a0, a1);
          f2_unpack(ls2[1], b0, b1);
          l_run += (a0 + a1) + (b0 + b1);
        }
        if (__any_sync(0xffffffffu, resc)) {  // warp-collective TMEM access
          // P V of the tile before.  (Its phase cannot be taken for the one before it:
          // S_{n-1} was issued after P_{n-3} V_{n-3}.)
          if (!(ok = warp_wait(&ct.pv_done[bf ^ 1], ((n - 1) >> 1) & 1, &ct.gave_up))) break;
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
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.p_full[bf]);
      }
      if (!ok) break;
      const uint32_t nl = seq + ntiles - 1;  // the item's last tile
      if (ntiles > 0 && !warp_wait(&ct.pv_done[nl & 1], (nl >> 1) & 1, &ct.gave_up)) break;
      tc_fence_after();
      if (qpos >= 0) a.lse[row] = l_run == 0.f ? -CUDART_INF_F : (m_run + log2f(l_run)) * kLn2;
      const float inv = l_run == 0.f ? 0.f : a.v_mul / l_run;  // a NaN stays one
      // dims (groups of 16) in which a token of the chunk that this row attends
      // has a NaN value (see the decoders)
      uint32_t nan_groups = 0;
      const uint64_t nan = *reinterpret_cast<const uint64_t*>(li.nan);
      if (nan && qpos >= 0) {
        const uint32_t mine = (2u << (qpos & 7)) - (2u << (c.w & 7));  // positions c.w + 1 .. qpos
#pragma unroll
        for (int g = 0; g < 8; ++g)
          if ((uint32_t)(nan >> (8 * g)) & mine & 0xFFu) nan_groups |= 1u << g;
      }
#pragma unroll 1
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
            if (nan_groups >> (c0 / 16 + e / 16) & 1) v[e] = 0x7FC00000u;
        }
        if (qpos >= 0) {
#pragma unroll
          for (int k = 0; k < 32; k += 16) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              w[e] = pack_bf16x2(__uint_as_float(v[k + 2 * e]) * inv, __uint_as_float(v[k + 2 * e + 1]) * inv);
            store32(a.o + row * 128 + c0 + k, kWide, w);
          }
        }
      }
      tc_fence_before();
      seq += ntiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ct.list_free[i & 1]);
    }
  } else if (warp < kScoreWarp) {
    // ---------------- decoders ----------------
    regs_dec<kDecodeRegs>();
    const int t = tid - 32 * kDecodeWarp, key = t & 63, half = t >> 6;
    uint32_t n = 0;
    for (uint32_t i = 0;; ++i) {
      if (!warp_wait(&ct.list_full[i & 1], (i >> 1) & 1, &ct.gave_up)) break;
      const Control::List& li = ct.list[i & 1];
      const int ntiles = li.ntiles, last = li.row.w + li.row.z - 1;  // the chunk's last position
      if (ntiles < 0) break;
      bool ok = true;
      Codes k, v;
      if (ntiles > 0) {
        const uint8_t* tile = a.cache + li.tile[0] * kTileBytes;
        load_k<kWide>(k, tile, key, half);
        load_v<kWide>(v, tile, key, half);
      }
      for (int j = 0; j < ntiles; ++j, ++n) {
        const uint32_t bf = n & 1, ph = (n >> 1) & 1;
        const uint8_t* next = a.cache + li.tile[min(j + 1, ntiles - 1)] * kTileBytes;
        if (n >= 2 && !(ok = warp_wait(&ct.s_full[bf], ph ^ 1, &ct.gave_up))) break;  // S_{n-2} has read its K
        decode_row(sm + OFF_K + bf * 16384 + half * 8192 + key * 128, k.w, k.scales, key);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.k_full[bf]);
        if (j + 1 < ntiles) load_k<kWide>(k, next, key, half);
        if (n >= 2 && !(ok = warp_wait(&ct.pv_done[bf], ph ^ 1, &ct.gave_up))) break;  // P V_{n-2} has read its V
        // Keys behind the chunk hold anything: a zero scale makes them zero (a
        // code alone is always finite; a weight of zero times NaN would not be).
        // A NaN value of one of the chunk's own tokens must not reach the tokens
        // before it: it counts as zero here, and the softmax warps put it into the
        // rows that attend it.
        const int pos = li.key0[j] + key;
        uint32_t vs = v.scales;
        if (pos > li.row.w) vs = pos <= last ? vs & ~nan_bytes(vs) : 0u;
        decode_row(sm + OFF_V + bf * 16384 + half * 8192 + key * 128, v.w, vs, key);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.v_full[bf]);
        if (j + 1 < ntiles) load_v<kWide>(v, next, key, half);
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(&ct.list_free[i & 1]);
    }
  } else {
    regs_dec<kOtherRegs>();
    if (warp == kScoreWarp) {
      // ---------------- S = Q K^T: one thread ----------------
      if (elect_one()) {
        // a descriptor's low bits are the address / 16: offsets add to it
        const uint64_t qdesc = sdesc_sw128(sbase + OFF_Q, 16, 1024), kdesc0 = sdesc_sw128(sbase + OFF_K, 16, 1024);
        uint32_t n = 0, nq = 0;  // nq: items with tiles
        bool ok = true;
        for (uint32_t i = 0; ok; ++i) {
          if (!short_wait(&ct.list_full[i & 1], (i >> 1) & 1, &ct.gave_up)) break;
          const int ntiles = ct.list[i & 1].ntiles;
          if (ntiles < 0) break;
          mbar_arrive(&ct.list_free[i & 1]);  // the list is not looked at again
          if (ntiles > 0 && !short_wait(&ct.q_full, nq++ & 1, &ct.gave_up)) break;
          for (int j = 0; j < ntiles; ++j, ++n) {
            ok = short_wait(&ct.k_full[n & 1], (n >> 1) & 1, &ct.gave_up);
            // the S columns: P_{n-2} has been read from them
            if (ok && n >= 2) ok = short_wait(&ct.pv_done[n & 1], ((n >> 1) & 1) ^ 1, &ct.gave_up);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kdesc = kdesc0 + (n & 1) * (16384 >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_bf16(tmem + COL_S + (n & 1) * 64, qdesc + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                        kdesc + (((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), ID_S, kk > 0);
            umma_commit(&ct.s_full[n & 1]);
          }
        }
      }
    } else if (warp == kOutWarp) {
      // ---------------- O += P V: one thread ----------------
      if (elect_one()) {
        const uint64_t vdesc = sdesc_sw128(sbase + OFF_V, 8192, 1024);
        uint32_t n = 0;
        bool ok = true;
        for (uint32_t i = 0; ok; ++i) {
          if (!short_wait(&ct.list_full[i & 1], (i >> 1) & 1, &ct.gave_up)) break;
          const int ntiles = ct.list[i & 1].ntiles;
          if (ntiles < 0) break;
          mbar_arrive(&ct.list_free[i & 1]);
          for (int j = 0; j < ntiles; ++j, ++n) {
            const uint32_t bf = n & 1;
            ok = short_wait(&ct.p_full[bf], (n >> 1) & 1, &ct.gave_up) &&
                 short_wait(&ct.v_full[bf], (n >> 1) & 1, &ct.gave_up);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16_ts(tmem + COL_O, tmem + COL_S + bf * 64 + kk * 8,
                           vdesc + ((bf * 16384 + kk * 2048) >> 4), ID_O,
                           (j > 0 || kk > 0) ? 1u : 0u);
            umma_commit(&ct.pv_done[bf]);
          }
        }
      }
    } else if (warp == kListWarp) {
      // ---------------- tile lists ----------------
      const bool stale = __any_sync(0xffffffffu, status_bad(a.status));
      uint32_t i = 0;
      int4 c_next = make_int4(-1, 0, 0, 0);
      int entry_next = -1;
      auto fetch = [&](int64_t w) {  // chunk row and selection, one item ahead
        c_next = make_int4(-1, 0, 0, 0);
        entry_next = -1;
        if (w >= items) return;
        const int64_t g = w / a.H;
        c_next = reinterpret_cast<const int4*>(a.chunks)[g];
        if (lane < a.K) entry_next = a.sel[((w - g * a.H) * a.NC + g) * a.K + lane];
      };
      if (!stale) fetch(blockIdx.x);
      for (int64_t w = blockIdx.x;; w += gridDim.x) {
        const int4 c = c_next;
        const int entry = entry_next;
        const int h = (int)(w % a.H);  // heads fastest: neighbouring CTAs read neighbouring tiles
        const bool end = stale || w >= items;
        if (!end) {
          fetch(w + gridDim.x);
          if (c.x < 0) continue;
        }
        int total = -1, x = 0, ntl = 0, page = 0, b = -1;
        uint32_t nan = 0;
        if (!end) {
          if (!list_tiles(a, c, entry, lane, b, page, ntl)) continue;
          // Q of the item: on its way to L2 while the item before is attended
          for (int tok = 0; tok < c.z; ++tok) {
            const uint16_t* line = a.q + ((int64_t)(c.y + tok) * a.H + h) * kGroup * 128 + lane * 64;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
          }
          x = ntl;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          total = __shfl_sync(0xffffffffu, x, 31);
          // NaN scales of the values of the chunk's own positions, if its block is selected
          const uint32_t own = __ballot_sync(0xffffffffu, c.z > 1 && b == c.w / a.B);
          if (own) {
            const int own_page = __shfl_sync(0xffffffffu, page, __ffs(own) - 1);
            if (lane < 8) {
              const uint8_t* vs = a.cache + tile_index(own_page, h, a.H, a.B / kTile, c.w % a.B / kTile) * kTileBytes +
                                  OFF_VS + lane * kTile + c.w % kTile / 8 * 8;
              const uint2 s8 = *reinterpret_cast<const uint2*>(vs);
              // one bit of each byte, gathered in the top four
              nan = ((nan_bytes(s8.x) & 0x01010101u) * 0x10204080u) >> 28 |
                    ((nan_bytes(s8.y) & 0x01010101u) * 0x10204080u) >> 28 << 4;
            }
          }
        }
        if (i >= 2 && !warp_wait(&ct.list_free[i & 1], ((i >> 1) & 1) ^ 1, &ct.gave_up)) break;
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
        if (lane < 8) li.nan[lane] = (uint8_t)nan;
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
  if (tid == 0 && ct.gave_up) set_status(a.status, MSA_ERR_TIMEOUT);
  if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

}  // namespace chunk
}  // namespace cache
}  // namespace msa
