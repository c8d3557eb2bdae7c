// strided.h -- what the products of experts and of the orthogonalised update share: descriptors, operands that the reduction runs
// across (read from LDS by its transpose read), and a kernel's allowance of LDS.
#pragma once

#include <atomic>

#include "common.h"
#include "lds_ring.h"

namespace moe {
namespace {

constexpr uint32_t kNoOffset = 0x80000000u;   // past every descriptor's bytes: reads zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, int64_t bytes) {
    const uint64_t u = (uint64_t)p;
    const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(u >> 32)) << 32 |
                          (uint32_t)__builtin_amdgcn_readfirstlane((int)u);
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, __builtin_amdgcn_readfirstlane((int)bytes),
                                             0x00020000);
}

// Operands whose rows are the reduction's are staged as they lie in memory, rows of a multiple of 256 bytes, and read by the LDS
// transpose read: the 16 lanes of a group address 4 rows x 32 bytes and receive four rows of one value each.  Slots of 16 bytes
// are permuted so that the eight rows that a read's half wave touches lie in different banks.
__device__ __forceinline__ int strided_slot(int k) { return 2 * ((k & 3) | (((k >> 3) & 1) << 2)); }

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
// ROW: bytes between staged rows.
template <int ROW>
__device__ __forceinline__ bf16x8 read_strided(const char *p) {
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)p);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)(p + 4 * ROW));
    return __builtin_bit_cast(bf16x8, (v8s)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Lets a kernel use `lds` bytes of shared memory, once on each device.
inline hipError_t allow_lds(const void *kernel, int lds, std::atomic<uint64_t> &allowed) {
    int device = 0;
    hipError_t e = hipGetDevice(&device);
    if (e != hipSuccess) return e;
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e == hipSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    return e;
}

}  // namespace
}  // namespace moe
