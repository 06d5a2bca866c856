// Loads from global memory straight into LDS, and transposing LDS reads, for the attention
// kernels.
#pragma once
#include "gdn_common.h"

namespace gdn {

typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}

// A running softmax's exponents are taken against a reference that follows the maximum only once
// that is more than LAG above it (powers of two). Weights then reach 2^LAG, which neither fp32
// sums nor bf16 weights mind, and sums and outputs are rescaled a few times in all instead of at
// every step in which one of a wave's rows finds a new maximum.
constexpr float LAG = 8.f;

// LDS by 32-bit byte offset: the compiler otherwise carries some addresses as 64-bit generic
// pointers, two registers each.
typedef __attribute__((address_space(3))) char lds_char;
template <typename V>
__device__ __forceinline__ V lds_get(uint32_t at) {
    return *(const __attribute__((address_space(3))) V*)(lds_char*)(uintptr_t)at;
}
template <typename V>
__device__ __forceinline__ void lds_put(uint32_t at, V v) {
    *(__attribute__((address_space(3))) V*)(lds_char*)(uintptr_t)at = v;
}

// 64 lanes x 16 bytes from `base` + each lane's `offset` to the 1 KiB of LDS at `lds` (wave
// uniform, lane l's piece at 16 l). No register receives data, and the compiler does not count
// the load: lds_loads_done() has to come before the barrier behind which the data is read.
// m0 carries the LDS address; it is a reserved register that the compiler sets right before an
// instruction of its own that reads it, of which these kernels have none (no clobber can be named).
// (The builtin for the same instruction makes the compiler wait for every such load before any
// later LDS read, which would end the overlap of one tile's load with the other's use.)
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t offset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(base)
                 : "memory");
}
// The same with a 64-bit address per lane.
__device__ __forceinline__ void load_to_lds(const void* lane_address, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(lane_address)
                 : "memory");
}
// A loaded value is first looked at here: nothing that depends on it moves up to its load.
__device__ __forceinline__ void arrived(int& x) { asm volatile("" : "+v"(x)); }
// Makes the compiler wait for these registers' loads here. Left to their first use inside a loop,
// the wait would be repeated in every pass and take the tile loads behind them along.
template <int N>
__device__ __forceinline__ void arrived(bf16x8 (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; i++) asm volatile("" : "+v"(x[i]));
}
__device__ __forceinline__ void lds_loads_done() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Transposing read of 16-bit elements. Every 16 lanes read a block of 4 rows x 16 columns: lane
// i passes the address of 4 columns (4 (i & 3) ..) of row i >> 2 and receives column i of the 4
// rows.
__device__ __forceinline__ bf16x4 lds_read_tr(const char* p) {
    typedef __attribute__((address_space(3))) s16x4* lptr;
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr)(p)));
}
__device__ __forceinline__ bf16x4 lds_read_tr(uint32_t at) {
    typedef __attribute__((address_space(3))) s16x4* lptr;
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr)(uintptr_t)at));
}
__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
    bf16x8 r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        r[i] = a[i];
        r[4 + i] = b[i];
    }
    return r;
}

// Maximum over the four lanes that are equal modulo 16, in the vector pipe.
__device__ __forceinline__ float max_groups(float x) {
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    uint32_t b = __float_as_uint(x);
    u32x2 r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    b = __float_as_uint(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
    r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
// Maximum over a lane and its partner 32 lanes on, in the vector pipe: the exchange leaves the
// lower halves in one register and the upper halves in the other.
__device__ __forceinline__ float max_halves(float x) {
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    const uint32_t b = __float_as_uint(x);
    const u32x2 r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

}  // namespace gdn
