// The 4-bit paged key/value cache: tile layout, decoding and argument checks
// shared by the serving kernels.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "msa_common.cuh"
#include "msa_host.cuh"

namespace msa {
namespace cache {

constexpr int kTile = 64;         // tokens of a cache tile
constexpr int kRowBytes = 64;     // 128 codes of 4 bits
constexpr int kScales = 8;        // e4m3 scales of a row, one per 16 dims
constexpr uint32_t OFF_KC = 0, OFF_KS = 4096, OFF_VC = 4608, OFF_VS = 8704;
constexpr uint32_t kTileBytes = MSA_CACHE_TILE_BYTES;
constexpr int kMaxRequests = 8192;
constexpr int kMaxBlocks = kMaxRows;
constexpr int kMaxCount = 1 << 24;  // pages, token rows, chunk rows
constexpr int kMaxHeads = 1024;
constexpr int kMaxExp = 32;

// Byte of unit `u` (8 bytes: one scale group) of token `t` in the V code
// plane.  The XOR spreads the four token rows that a quad of an MMA B fragment
// reads (t, t + 4, t + 8, t + 12, the same unit) over all 32 banks.
MSA_DEV uint32_t v_code_offset(int t, int u) { return (uint32_t)(t * kRowBytes + u * 8) ^ (uint32_t)((t & 12) << 3); }

// Two e2m1 codes (the low and high half of a byte) as fp16 values, exact.
MSA_DEV void e2m1x8_to_half(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two e4m3 scales as fp16 values, exact (NaN stays NaN).
MSA_DEV uint32_t e4m3x2_to_half(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}" : "=r"(h) : "r"(two));
  return h;
}
// A code has 2 significant bits and a scale 4, so their product (magnitudes
// from 2^-10 to 2688) is exact in fp16.
MSA_DEV uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 2^e for -126 <= e <= 127.
__host__ __device__ __forceinline__ float exp2i(int e) {
  union { uint32_t u; float f; } x;
  x.u = (uint32_t)(e + 127) << 23;
  return x.f;
}

// 32 bytes in one load or store (a whole sector a lane), or in two where the
// tensors are aligned to 16 bytes only.  Plain loads, here and for every tensor of
// these kernels: a kernel may come up while the one before it still writes what
// it reads (after_previous_kernel), and the read-only path is for memory that
// nothing writes as long as the kernel lives.  What is loaded here is read once and
// leaves the L1 to others (3.4k new tokens x 4 heads: 195 us, 201 without the hint).
MSA_DEV void load32(const void* src, bool wide, uint32_t (&u)[8]) {
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
        : "l"(src));
  } else {
    const uint4 a = static_cast<const uint4*>(src)[0], b = static_cast<const uint4*>(src)[1];
    u[0] = a.x; u[1] = a.y; u[2] = a.z; u[3] = a.w;
    u[4] = b.x; u[5] = b.y; u[6] = b.z; u[7] = b.w;
  }
}
MSA_DEV void store32(void* dst, bool wide, const uint32_t (&u)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                 "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}
inline bool aligned32(const void* a, const void* b) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 31u) == 0;
}

// Clears the sign of the codes that are zero, so that equal values have equal
// bytes.
MSA_DEV uint32_t unsigned_zeros(uint32_t w) {
  const uint32_t m = w & 0x77777777u;
  return w & (((m << 1 | m << 2 | m << 3) & 0x88888888u) | 0x77777777u);
}

// Eight e2m1 codes of eight values, zeros without a sign.
MSA_DEV uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t codes;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(codes)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return unsigned_zeros(codes);
}

// One group of 16 bf16 values (8 words) to codes (8 bytes) and an e4m3 scale.
// Quotients are formed so that the conversions' ties are those of the exact
// ones: max / 6 with one correction step (exact where the quotient has 24 bits,
// as every midpoint of two scales does), and x / s as x * (1 / s), which is
// either a border between two codes (a multiple of 1/4) or at least 2^-11 away
// from it, because x has 8 significant bits and border * s 7; rounding it to a
// multiple of 2^-14 (the addition of 1.5 * 2^9) undoes the reciprocal's error.
MSA_DEV uint32_t quantize16(const uint32_t (&w)[8], float mul, uint2& codes) {
  codes = make_uint2(0, 0);
  uint32_t m2 = w[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
  const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  if (m >= 0x7F80u) return 0x7F;  // a NaN scale: the group reads back as NaN
  // max * mul may overflow to infinity: the scale saturates, and so do the codes
  const float amax = __uint_as_float(m << 16) * mul;
  constexpr float kSixth = 1.f / 6.f;
  const float t0 = amax * kSixth;
  const float t = amax < 4096.f ? __fmaf_rn(__fmaf_rn(-6.f, t0, amax), kSixth, t0) : t0;  // far above 6 * 448
  uint16_t s2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.f), "f"(t));
  const uint32_t s8 = s2 & 0xFFu;
  if (s8 == 0) return 0;
  const float s = __half2float(__ushort_as_half((uint16_t)(e4m3x2_to_half(s8) & 0xFFFFu)));
  const float inv = __frcp_rn(s) * mul;
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = w[4 * h + i];
      q[2 * i] = __fadd_rn(__fmaf_rn(__uint_as_float(x << 16), inv, 768.f), -768.f);
      q[2 * i + 1] = __fadd_rn(__fmaf_rn(__uint_as_float(x & 0xFFFF0000u), inv, 768.f), -768.f);
    }
    out[h] = e2m1x8(q);
  }
  codes = make_uint2(out[0], out[1]);
  return s8;
}

// What a chunk does for the pooled index keys.
// The chunk that ends a block averages the block's tokens, those of earlier
// calls from the tail; a chunk of the request's incomplete block stores its rows
// to the tail.  Where the incomplete block uses the buffer that the first
// block's average reads (an even number of blocks apart), the chunk that
// averages stores them too, after it.  The first block's average is made by the
// request's first chunk, others by the chunk that ends the block.  Most chunks of
// a prompt have nothing to do.
struct IndexPlan {
  int r, cu0, past;  // request, its first token row, its cached tokens
  int open;          // its incomplete block
  int last;          // the last token's row of the block to average (-1: none)
  int avg_blk;       // that block
  int p0, p1;        // positions to store
};

// False where the chunk has nothing to do or is not there.  report: this thread
// reports a row that does not fit.
template <class Args>
MSA_DEV bool plan_index(const Args& a, int g, bool report, IndexPlan& x) {
  const int4 c = reinterpret_cast<const int4*>(a.chunks)[g];
  const int r = c.x, row0 = c.y, n = c.z, pos0 = c.w;
  if (r < 0) return false;
  const int lb = 31 - __clz(a.B);  // a block is a power of two
  int cu0 = 0, cu1 = 0;
  bool good = r < a.R && n >= 1 && n <= kChunk && row0 >= 0 && row0 <= a.T - n && pos0 >= 0;
  if (good) {
    cu0 = a.cu_tokens[r];
    cu1 = a.cu_tokens[r + 1];
    good = cu0 >= 0 && cu0 <= row0 && cu1 >= row0 + n && cu1 <= a.T && pos0 >= row0 - cu0 &&
           pos0 <= a.positions - (cu1 - row0) && (pos0 & (a.B - 1)) + n <= a.B;
  }
  if (!good) {
    if (report) set_status(a.status, MSA_ERR_INVALID_CACHE);
    return false;
  }
  const int end = pos0 + (cu1 - row0);     // position behind the request's last new token
  const int past = pos0 - (row0 - cu0);
  const int blk0 = past >> lb, blk = pos0 >> lb, open = end >> lb;
  const bool shared_buffer = open > blk0 && (open & 1) == (blk0 & 1) && (past & (a.B - 1)) != 0;
  x.r = r; x.cu0 = cu0; x.past = past; x.open = open;
  x.last = -1;
  if (row0 == cu0 && open > blk0) x.last = cu0 + (blk0 + 1) * a.B - past - 1;
  else if (row0 != cu0 && blk > blk0 && ((pos0 + n) & (a.B - 1)) == 0) x.last = row0 + n - 1;
  x.avg_blk = row0 == cu0 ? blk0 : blk;
  x.p0 = x.p1 = 0;
  if (shared_buffer) {
    if (row0 == cu0) { x.p0 = open * a.B; x.p1 = end; }
  } else if (blk == open) {
    x.p0 = pos0;
    x.p1 = pos0 + n;
  }
  return x.last >= 0 || x.p0 < x.p1;
}

// Adds rows' two dims (bf16, `stride` elements apart) to lo and hi, in order, 16 in
// flight.
MSA_DEV void add_rows(const uint16_t* src, int64_t stride, int rows, float& lo, float& hi) {
  for (; rows > 0; rows -= 16, src += 16 * stride) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = i < rows ? *reinterpret_cast<const uint32_t*>(src + i * stride) : 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < rows) {
        lo = __fadd_rn(lo, __uint_as_float(w[i] << 16));
        hi = __fadd_rn(hi, __uint_as_float(w[i] & 0xFFFF0000u));
      }
  }
}

MSA_DEV int64_t tile_index(int64_t page, int head, int heads, int tiles_per_page, int tile) {
  return (page * heads + head) * tiles_per_page + tile;
}

int check_cache_problem(const msa_cache_problem* p);

// The kernels of a serving step are a few microseconds each and follow one
// another, so they are launched with programmatic serialisation: a kernel's CTAs
// may come up while the one before it drains, and wait here, before they touch
// memory, until it has completed.  Every thread passes here first.  kEarly lets
// the next kernel's CTAs come up as soon as all of this one's run (a step of 64
// requests 5.2 -> 4.3 us, a selection 5.8 -> 5.2); the attention kernels, which
// fill the SMs, do without (the chunk kernel 248 -> 264 us with it).
template <bool kEarly = true>
MSA_DEV void after_previous_kernel() {
  if constexpr (kEarly) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches kernel(args) that way; cluster > 1: in clusters of that many CTAs
// along x.  largest: the kernel's largest dynamic shared memory, where it varies.
template <class Args>
inline int launch_kernel(void (*kernel)(Args), dim3 grid, int threads, size_t smem, void* stream, unsigned cluster,
                         const Args& args, size_t largest = 0) {
  cudaError_t e = allow_smem(kernel, smem, largest ? largest : smem);
  if (e != cudaSuccess) return MSA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args));
}

}  // namespace cache
}  // namespace msa
