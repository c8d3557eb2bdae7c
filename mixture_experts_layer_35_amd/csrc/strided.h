// strided.h -- what the products of experts and of the orthogonalised update share: descriptors, operands that the reduction runs
// across (read from LDS by its transpose read), and a kernel's allowance of LDS.
#pragma once

#include <atomic>

#include "common.h"
#include "internal.h"
#include "lds_ring.h"

namespace moe {
namespace {

constexpr uint32_t kNoOffset = 0x80000000u;   // past every descriptor's bytes: reads zeros

// A raw buffer descriptor of `bytes` bytes at p, the same in all lanes.
typedef int i32x4s __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4s words_of(const void *p, int64_t bytes) {
    const uint64_t u = (uint64_t)p;
    return i32x4s{__builtin_amdgcn_readfirstlane((int)u), __builtin_amdgcn_readfirstlane((int)(u >> 32)),
                  __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, int64_t bytes) {
    const i32x4s w = words_of(p, bytes);
    const uint64_t base = (uint64_t)(uint32_t)w[1] << 32 | (uint32_t)w[0];
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, w[2], 0x00020000);
}

// Direct loads of 16 bytes a lane into LDS at `to` (the same in all lanes) + 16 * lane.  As asm they have no registers to wait
// for, and the compiler does not know that they write LDS: with the builtins it waits for every load under way before each
// transpose read of LDS (512 rows an expert, the gradient at x: 1080 us of loads and reads against 385 without the reads).
// Nor does it count them when it waits for loads of its own, which then takes longer than it has to: values that such loads bring
// are settled (arrived) before the next direct load.  Whoever reads what they bring waits for them by itself (wait_vmcnt and a
// barrier).  M0 holds the place; kernels with these loads use nothing else that reads M0.
__device__ __forceinline__ int lds_place(const void *p) {
    return (int)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}
__device__ __forceinline__ void fill16(i32x4s r, uint32_t voff, int soff, int to) {
    // what asm takes in scalar registers is said to be the same in all lanes where it is used
    r = i32x4s{__builtin_amdgcn_readfirstlane(r[0]), __builtin_amdgcn_readfirstlane(r[1]), __builtin_amdgcn_readfirstlane(r[2]),
               0x00020000};
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :
                 : "v"(voff), "s"(r), "s"(__builtin_amdgcn_readfirstlane(soff)), "s"(__builtin_amdgcn_readfirstlane(to))
                 : "memory");
}
__device__ __forceinline__ void fill16(const void *p, int to) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(p), "s"(__builtin_amdgcn_readfirstlane(to))
                 : "memory");
}

// Waits for loaded values here and not at their uses.
template <class T>
__device__ __forceinline__ void arrived(T &v) { asm volatile("" : "+v"(v)); }

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

// Eight values of a fp32 or bf16 array from `at` on, zeros past n of them: 16-byte accesses, which the memory pipeline takes at
// every address.
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
template <int DT>
__device__ __forceinline__ void load8(const void *x, int64_t at, int64_t n, float (&v)[8]) {
    if (n >= 8) {
        if (DT == DT_F32) {
            const f32x4 lo = *(const f32x4_any *)((const float *)x + at), hi = *(const f32x4_any *)((const float *)x + at + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = lo[k];
                v[4 + k] = hi[k];
            }
        } else {
            const u32x4 w = *(const u32x4_any *)((const uint16_t *)x + at);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = __uint_as_float(w[k] << 16);
                v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = k >= n ? 0.0f : DT == DT_F32 ? ((const float *)x)[at + k] : bf16_to_f32(((const uint16_t *)x)[at + k]);
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
