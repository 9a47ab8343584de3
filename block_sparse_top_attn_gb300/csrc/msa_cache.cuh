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
