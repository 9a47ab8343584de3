// Attention over the 4-bit cache for batches of single tokens: the same work per
// (token, KV head) as the cluster kernel, by persistent CTAs whose copies never
// stop between items.
//
// Warp 4 serves: it walks the CTA's items, and for each writes the tile list and
// the query's A fragments (two buffers) and then feeds the tiles through the ring;
// while the last tiles of an item are still being read it has the next item's
// list ready, so the chain of loads that an item starts with (chunk row and
// selection, pages, tiles: 3 us) is hidden.  Warps 0-3 attend: tile n goes to warps
// 2 (n & 1) and 2 (n & 1) + 1, 32 keys each.  At an item's end the odd warps leave
// their part in shared memory for the even ones and go on; warp 2 then leaves its
// own for warp 0, which writes the rows.  Nothing synchronises the whole CTA.
//
// 256 tokens x 8 heads x 2048 keys: 149 us (4.1 TB/s of cache bytes, 227 TFLOP/s) against
// 156 with one CTA an item; x 64 keys 23 against 30.
#pragma once

namespace msa {
namespace cache {
namespace batch {

constexpr int kThreads = 160;
// Even, so that a stage only ever holds tiles of one pair of warps: a pair then
// waits for every phase of the stage's barrier.  (With an odd ring a pair that
// skips the other's phase could take the phase before it, of the same parity,
// for its own.)
constexpr int kRing = 8;
static_assert(kRing % 2 == 0, "a stage belongs to one pair of warps");
constexpr int kCtasPerSm = 2;

struct Shared {
  alignas(128) uint8_t ring[kRing][kTileBytes];
  float4 part[2][16][32];             // a warp's output, [pair][n-tile][lane]
  float2 part_ml[2][2][32];           // its m and l, [pair][row half][lane]
  struct Item {
    uint4 q[8][32];                   // the 16 query rows as A fragments of the 8 k-steps, by lane
    float qs[16];                     // powers of two that undo their scaling
    int64_t row0;                     // first output row
    int32_t qpos, ntiles;             // ntiles: -1 ends the walk
    int32_t key0[kMaxTiles];          // position of each tile's first key
  } item[2];
  int64_t tile[kMaxTiles];            // tile indexes of the item being fed (the service warp's own)
  alignas(8) uint64_t full[kRing], empty[kRing];
  uint64_t item_full[2], item_free[2];
  uint64_t part_full[2], part_free[2];  // the odd warp's part, by pair
  uint64_t pair_full;                   // warp 2's joined part, in part[1]
};
static_assert(kCtasPerSm * (sizeof(Shared) + 1024) <= 227 * 1024, "the CTAs of an SM fit");

MSA_DEV bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}

// o, m, l += a partner's (x at [n-tile][lane], ml at [row half][lane])
MSA_DEV void join(float (&o)[16][4], float (&m)[2], float (&l)[2], const float4 (*x)[32], const float2 (*ml)[32],
                  int lane) {
  float fa[2], fb[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float2 b = ml[r][lane];
    const float mm = fmaxf(m[r], b.x);
    // a part without keys has m = -inf and l = 0; a NaN l stays a NaN
    fa[r] = m[r] == -CUDART_INF_F ? 0.f : ex2_approx(m[r] - mm);
    fb[r] = b.x == -CUDART_INF_F ? 0.f : ex2_approx(b.x - mm);
    m[r] = mm;
    l[r] = fa[r] * l[r] + fb[r] * b.y;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float4 y = x[i][lane];
    o[i][0] = fa[0] * o[i][0] + fb[0] * y.x;
    o[i][1] = fa[0] * o[i][1] + fb[0] * y.y;
    o[i][2] = fa[1] * o[i][2] + fb[1] * y.z;
    o[i][3] = fa[1] * o[i][3] + fb[1] * y.w;
  }
}
MSA_DEV void leave(const float (&o)[16][4], const float (&m)[2], const float (&l)[2], float4 (*x)[32],
                   float2 (*ml)[32], int lane) {
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i][lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
#pragma unroll
  for (int r = 0; r < 2; ++r) ml[r][lane] = make_float2(m[r], l[r]);
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) fwd_batch_kernel(FwdCacheArgs a) {
  extern __shared__ __align__(128) uint8_t s_raw[];
  Shared& s = *reinterpret_cast<Shared*>(s_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.item_full[i], 1);
      mbar_init(&s.item_free[i], 4);
      mbar_init(&s.part_full[i], 1);
      mbar_init(&s.part_free[i], 1);
    }
    mbar_init(&s.pair_full, 1);
    fence_mbar_init();
  }
  after_previous_kernel<false>();
  __syncthreads();
  // Tiles are numbered through all items of the CTA: tile n uses stage n % kRing,
  // lap n / kRing.  Item i uses buffer i & 1, and has one phase of every part
  // barrier whether or not a warp had tiles.
  if (warp == 4) {
    // ---------------- service: items, copies ----------------
    const int64_t items = (int64_t)a.H * a.NC;
    const bool stale = __any_sync(0xffffffffu, status_bad(a.status));  // an earlier error: no items
    bool ok = true;
    uint32_t i = 0, n = 0;
    for (int64_t w = blockIdx.x; !stale && ok && w < items; w += gridDim.x) {
      // heads fastest: CTAs that run together read neighbouring tiles
      const int64_t g = w / a.H;
      const int h = (int)(w - g * a.H);
      const int entry = lane < a.K ? a.sel[((int64_t)h * a.NC + g) * a.K + lane] : -1;
      const int4 c = reinterpret_cast<const int4*>(a.chunks)[g];
      if (c.x < 0) continue;
      int b, page, ntl;
      if (!list_tiles(a, c, entry, lane, b, page, ntl)) continue;
      int x = ntl;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const int total = __shfl_sync(0xffffffffu, x, 31);
      for (int k = 0; k < ntl; ++k) s.tile[x - ntl + k] = tile_index(page, h, a.H, a.B / kTile, k);
      for (int tok = 0; ok && tok < c.z; ++tok, ++i) {
        const int gid = lane >> 2, t = lane & 3;
        const int64_t row0 = (int64_t)(c.y + tok) * a.H * kGroup + h * kGroup;
        uint32_t q0[16], q1[16];
        const uint16_t* src = a.q + (row0 + gid) * 128 + 32 * t;
        const float x0 = load_q_row(src, q0), x1 = load_q_row(src + 8 * 128, q1);
        if (i >= 2 && !(ok = warp_wait(&s.item_free[i & 1], ((i >> 1) & 1) ^ 1, a.status))) break;
        Shared::Item& it = s.item[i & 1];
        if (t == 0) {
          it.qs[gid] = x0;
          it.qs[gid + 8] = x1;
        }
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          it.q[ks][lane] = make_uint4(q0[2 * ks], q1[2 * ks], q0[2 * ks + 1], q1[2 * ks + 1]);
        for (int k = 0; k < ntl; ++k) it.key0[x - ntl + k] = b * a.B + k * kTile;
        if (lane == 0) {
          it.row0 = row0;
          it.qpos = c.w + tok;
          it.ntiles = total;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s.item_full[i & 1]);
          for (int j = 0; j < total; ++j, ++n) {
            const uint32_t st = n % kRing, lap = n / kRing;
            if (lap > 0 && !(ok = mbar_wait(&s.empty[st], (lap - 1) & 1, a.status))) break;
            mbar_arrive_expect_tx(&s.full[st], kTileBytes);
            bulk_load(s.ring[st], a.cache + s.tile[j] * kTileBytes, kTileBytes, &s.full[st]);
          }
        }
        __syncwarp();
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      }
      __syncwarp();  // lane 0 has read the list
    }
    if (ok) {
      if (i >= 2) ok = warp_wait(&s.item_free[i & 1], ((i >> 1) & 1) ^ 1, a.status);
      if (ok && lane == 0) {
        s.item[i & 1].ntiles = -1;
        mbar_arrive(&s.item_full[i & 1]);
      }
    }
    // after a wait that gave up, copies may be in flight: they land before the
    // CTA's shared memory is let go
    if (!ok && lane == 0)
      for (uint32_t k = n > kRing ? n - kRing : 0; k < n; ++k)
        mbar_wait(&s.full[k % kRing], (k / kRing) & 1, a.status);
  } else {
    // ---------------- attention ----------------
    const int pair = warp >> 1, kw = 32 * (warp & 1);
    const int gid = lane >> 2, t = lane & 3;
    uint32_t base = 0;  // tiles of earlier items
    for (uint32_t i = 0;; ++i) {
      const uint32_t ph = (i >> 1) & 1;
      if (!warp_wait(&s.item_full[i & 1], ph, a.status)) break;
      const Shared::Item& it = s.item[i & 1];
      const int ntiles = it.ntiles, qpos = it.qpos;
      if (ntiles < 0) break;
      const float sc0 = score_factor(it.qs[gid], a.scale_log2), sc1 = score_factor(it.qs[gid + 8], a.scale_log2);
      float o[16][4], m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      bool ok = true;
      for (uint32_t n = base + ((base ^ pair) & 1); n < base + ntiles; n += 2) {
        const uint32_t st = n % kRing;
        if (!(ok = warp_wait(&s.full[st], (n / kRing) & 1, a.status))) break;
        const int reach = qpos - (it.key0[n - base] + kw);
        if (reach >= 0) attend32(s.ring[st], kw, reach, it.q, sc0, sc1, lane, o, m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[st]);
      }
      if (!ok) break;
      base += ntiles;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      }
      if (warp & 1) {
        if (i >= 1 && !warp_wait(&s.part_free[pair], (i - 1) & 1, a.status)) break;
        leave(o, m, l, s.part[pair], s.part_ml[pair], lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.part_full[pair]);
      } else {
        if (!warp_wait(&s.part_full[pair], i & 1, a.status)) break;
        join(o, m, l, s.part[pair], s.part_ml[pair], lane);
        if (warp == 2) {
          // into the places that this lane has just read; warp 0 frees them
          leave(o, m, l, s.part[1], s.part_ml[1], lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.pair_full);
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.part_free[0]);
          if (!warp_wait(&s.pair_full, i & 1, a.status)) break;
          join(o, m, l, s.part[1], s.part_ml[1], lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.part_free[1]);
          // lane: dims 32 t .. 32 t + 31 of rows gid and gid + 8
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float inv = l[r] == 0.f ? 0.f : a.v_mul / l[r];  // a NaN stays one
            const int64_t row = it.row0 + gid + 8 * r;
            uint4* dst = reinterpret_cast<uint4*>(a.o + row * 128 + 32 * t);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  w[y] = pack_bf16x2(o[8 * k + 2 * y][2 * r + e] * inv, o[8 * k + 2 * y + 1][2 * r + e] * inv);
                dst[2 * e + k] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            if (t == 0) a.lse[row] = l[r] == 0.f ? -CUDART_INF_F : (m[r] + log2f(l[r])) * kLn2;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.item_free[i & 1]);
    }
  }
  __syncthreads();  // the service warp may still wait for copies
}

}  // namespace batch
}  // namespace cache
}  // namespace msa
