// Device-side building blocks shared by the matrix-core attention kernels (gfx950, wave64).
//
// Both products of attention run in transposed form on 32 x 32 x 16 tiles,
//   S^T[key, row] = K Q^T   and   O^T[d, row] = V^T P^T:
// lane l holds column l % 32 (a query row) of each result, elements 8 (e / 4) + 4 (l / 32) + e % 4
// for e = 0 .. 15.  A lane's eight S elements of registers 8 s .. 8 s + 7 are the keys
// 16 s + 4 (l / 32) + {0, 1, 2, 3, 8, 9, 10, 11}; V's fragments are read in that order, so they are
// the second product's operand as they stand.
#pragma once

#include "common.h"

namespace w4a16 {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ f32x16 mfma(const u32x4& a, const u32x4& b, const f32x16& c) {
    if constexpr (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
}

// Transposing LDS read: the 16 lanes of a group read 4 rows of 16 values (lane i: values
// 4 (i % 4) .. + 3 of row i / 4); lane i receives column i, the four rows in order.
__device__ __forceinline__ u32x2 lds_read_tr(const uint16_t* p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4*)p));
}

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

// the values of lanes l % 32 and l % 32 + 32, in both lanes
__device__ __forceinline__ void halves(float x, float& lo, float& hi) {
    const int i = __builtin_bit_cast(int, x);
    const auto r = __builtin_amdgcn_permlane32_swap(i, i, false, false);
    const int a = r[0], b = r[1];        // (a bit cast of r[1] itself reads element 0)
    lo = __builtin_bit_cast(float, a);
    hi = __builtin_bit_cast(float, b);
}
__device__ __forceinline__ float max_halves(float x) {
    float lo, hi;
    halves(x, lo, hi);
    return fmaxf(lo, hi);
}
__device__ __forceinline__ float sum_halves(float x) {
    float lo, hi;
    halves(x, lo, hi);
    return lo + hi;
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (DT == DT_F16) return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
    else return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// Where 16-byte piece c of row r of a [keys, D] tile sits in its row: the pieces are permuted so
// that the 32 rows of a fragment read (K), the 4 rows x 64 bytes of a transposing read (V) and the
// pieces of a store that skips 2 or 4 of them fall in different banks.
template <int D>
__device__ __forceinline__ int swz_k(int r, int c) {
    return D == 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int swz_v(int r, int c) {
    return D == 128 ? c ^ ((r & 3) * 5) : c ^ (((r << 1) & 4) | ((r >> 1) & 3));
}

}  // namespace w4a16
