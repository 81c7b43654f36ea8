// Device-side building blocks of the paged 8-bit KV cache (gfx950, wave64): where a call's tokens
// lie, the codes' two formats, and rotations by a position.
//
// A pool holds N pages of `page` tokens (16, 32, 64 or 128).  Of kv head h, page i holds
//   keys    [page, D] codes from byte ((i Hkv + h) page D), a token's row after the other, and
//   values  [D, page] codes, a dimension's tokens after one another,
// and one fp32 scale each.  Values lie across because the second product of attention sums over
// tokens: its operand wants consecutive tokens of a dimension, which then come from memory as they are.
#pragma once

#include "attn.h"
#include "launch.h"

namespace w4a16 {

enum { FMT_INT8 = 0, FMT_E4M3 = 1 };
template <int FMT>
constexpr float kTop = FMT == FMT_INT8 ? 127.0f : 448.0f;       // largest code

// ---- codes

template <int FMT>
__device__ __forceinline__ float code_value(uint32_t word, int byte) {
    if constexpr (FMT == FMT_INT8) return (float)(int8_t)(word >> (8 * byte));
    switch (byte) {
        case 0: return __builtin_amdgcn_cvt_f32_fp8(word, 0);
        case 1: return __builtin_amdgcn_cvt_f32_fp8(word, 1);
        case 2: return __builtin_amdgcn_cvt_f32_fp8(word, 2);
        default: return __builtin_amdgcn_cvt_f32_fp8(word, 3);
    }
}
// Four quotients x / s as codes: to nearest, ties to even, infinities to the largest code, NaN to 0.
template <int FMT>
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
    const float x[4] = {a, b, c, d};
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v = x[i] == x[i] ? x[i] : 0.0f;
        y[i] = fminf(fmaxf(v, -kTop<FMT>), kTop<FMT>);
    }
    if constexpr (FMT == FMT_INT8) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= ((uint32_t)(int)__builtin_rintf(y[i]) & 255u) << (8 * i);
        return w;
    }
    return __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false), true);
}
// The same for quotients that are numbers of at most the largest code, up to their rounding: the sum with 1.5 * 2^23
// holds the nearest whole number, ties to even, in its last byte.
template <int FMT>
__device__ __forceinline__ uint32_t pack_numbers(float a, float b, float c, float d) {
    if constexpr (FMT == FMT_INT8) {
        const auto bits = [](float x) { return __builtin_bit_cast(uint32_t, x + 12582912.0f); };
        const uint32_t lo = perm(bits(b), bits(a), 0x0C0C0400u), hi = perm(bits(d), bits(c), 0x04000C0Cu);
        return lo | hi;
    }
    return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
}
// x / s in three operations: with r the reciprocal of s rounded to nearest, the remainder of x r is exact and its
// correction gives the quotient rounded to nearest (Markstein), away from the ends of the range.
struct Divisor {
    float s, r;
    bool plain;
    __device__ __forceinline__ explicit Divisor(float scale)
        : s(scale), r(1.0f / scale), plain(scale > 7.9e-31f && scale < 1.2e30f) {}      // 2^-100 .. 2^100
    __device__ __forceinline__ float quotient(float x) const {
        const float q = x * r;
        return fmaf(fmaf(-q, s, x), r, q);
    }
};
// Four codes of a page whose scale has grown, times old / new scale, rounded again.
template <int FMT>
__device__ __forceinline__ uint32_t requantize(uint32_t w, float r) {
    return pack_codes<FMT>(code_value<FMT>(w, 0) * r, code_value<FMT>(w, 1) * r, code_value<FMT>(w, 2) * r,
                           code_value<FMT>(w, 3) * r);
}

// ---- rotations

// cos and sin of 2 pi t / 2^64: the position times the pair's 64-bit fraction of a turn, taken modulo
// 2^64, is the angle exactly, however far the position (fp32 angles are off by 0.06 at position 10^6).
// Reduced to an eighth of a turn, then the Taylor series to x^9 and x^10 (off by 2^-28 and less).
__device__ __forceinline__ void turn_cos_sin(uint64_t t, float& c, float& s) {
    const uint32_t quarter = (uint32_t)((t + (1ull << 61)) >> 62);
    const long long r = (long long)(t - ((uint64_t)quarter << 62));
    const uint64_t a = (uint64_t)(r < 0 ? -r : r);                 // (small angles of either sign keep their bits)
    const float z = fmaf((float)(uint32_t)(a >> 32), 4294967296.0f, (float)(uint32_t)a) * 3.4061215800e-19f;   // 2 pi / 2^64
    const float x = r < 0 ? -z : z, y = x * x;
    const float sn = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
    const float cn =
        fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    c = quarter & 1 ? sn : cn;
    s = quarter & 1 ? cn : sn;
    if ((quarter + 1) & 2) c = -c;
    if (quarter & 2) s = -s;
}

__device__ __forceinline__ void position_cos_sin(int position, long long freq, float m, float& c, float& s) {
    turn_cos_sin((uint64_t)(long long)position * (uint64_t)freq, c, s);
    c *= m;
    s *= m;
}

// One pair turned; in these steps everywhere, so that all ways to a rotation give the same bits (nor is the rounding
// to 16 bits that may follow taken into the last of them).
__device__ __forceinline__ void turn_pair(float& x0, float& x1, float c, float s) {
    const float y = fmaf(x0, c, -(x1 * s));
    x1 = fmaf(x1, c, x0 * s);
    x0 = y;
    asm("" : "+v"(x0), "+v"(x1));
}

// ---- where tokens are

// The last sequence whose first token is at or before `token` of the T packed ones (64-way search, one
// load a level).  Empty sequences share their first token with the next, so it is the token's own.
__device__ __forceinline__ int sequence_of(const int* __restrict__ cu, int B, int T, int token, int lane) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) >> 6, b = lo + lane * step;
        const bool in = b < hi && min(max(cu[b], 0), T) <= token;
        const int n = __builtin_popcountll(__builtin_amdgcn_ballot_w64(in));
        if (n == 0) break;
        lo += (n - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Tokens of one page that a call is about: sequence b's page `index` (negative: before the sequence),
// its slots [off, off + n), which are the packed tokens from `token` on; false for none.
//
// The last tokens of a sequence touch at most tokens / page + 2 pages.  Sequence b owns the slots
// first(b) = cu[b] / page + 2 b and on; first() grows by at least that many a sequence, so the last b with
// first(b) <= slot is the only candidate.
struct PageTokens {
    int b, index, off, n, token;
};
__device__ __forceinline__ bool page_tokens(const int* __restrict__ lens, const int* __restrict__ cu, int B, int T,
                                            int shift, int slot, int lane, PageTokens& p) {
    int b, first, n, len;
    if (cu && B <= 64) {
        // a lane a sequence: everything in one round of loads
        const int c0 = min(max(cu[min(lane, B)], 0), T), c1 = cu[min(lane + 1, B)];
        const int ln = lens[min(lane, B - 1)];
        const unsigned long long m = __builtin_amdgcn_ballot_w64(lane < B && (c0 >> shift) + 2 * lane <= slot);
        b = m ? 63 - __builtin_clzll(m) : 0;
        first = __builtin_amdgcn_readlane(c0, b);
        n = min(max(__builtin_amdgcn_readlane(c1, b), first), T) - first;
        len = __builtin_amdgcn_readlane(ln, b);
        slot -= (first >> shift) + 2 * b;
    } else if (cu) {
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int step = (hi - lo + 63) >> 6, at = lo + lane * step;
            const bool in = at < hi && (min(max(cu[at], 0), T) >> shift) + 2 * at <= slot;
            const int found = __builtin_popcountll(__builtin_amdgcn_ballot_w64(in));
            if (found == 0) break;
            lo += (found - 1) * step;
            hi = min(hi, lo + step);
        }
        b = lo;
        first = __builtin_amdgcn_readfirstlane(min(max(cu[b], 0), T));
        n = __builtin_amdgcn_readfirstlane(min(max(cu[b + 1], first), T)) - first;
        len = __builtin_amdgcn_readfirstlane(lens[b]);
        slot -= (first >> shift) + 2 * b;
    } else {
        b = slot;
        first = slot;
        n = 1;
        len = __builtin_amdgcn_readfirstlane(lens[b]);
        slot = 0;
    }
    // (a longer sequence than any table holds has no pages there: kept where sums stay in 32 bits)
    len = min(max(len, 0), 1 << 25);
    const int before = len - n;
    p.b = b;
    p.index = (before >> shift) + slot;
    const int start = p.index << shift;
    const int lo = max(before, start), hi = min(len, start + (1 << shift));
    p.off = lo - start;
    p.n = hi - lo;
    p.token = first + (lo - before);
    return slot >= 0 && p.n > 0;
}

// The page's number in the pool, or -1: outside the table, or an entry that is no page.
__device__ __forceinline__ int page_id(const int* __restrict__ table, int P, int N, int b, int index) {
    if (index < 0 || index >= P) return -1;
    const int id = __builtin_amdgcn_readfirstlane(table[(long long)b * P + index]);
    return id >= 0 && id < N ? id : -1;
}

}  // namespace w4a16
