// Decode attention over the quantized cache on the matrix cores: one query per sequence and head
// over a prefix that all sequences of the batch share followed by the sequence's own tokens, and
// decode attention that also adds up the attention weight every cached token receives.
//
//   out[b, h] = sum_t p_t v_t,  p = softmax_t(q[b, h] . k_t / sqrt(D)),  k_t = s_t (c_t - z_t)
//
// over the P shared tokens and the lengths[b] own ones (kv head h / (Hq / Hkv)), and
//   sums[b, kv head, t] = weights[b, kv head, t] + sum over the group's heads of p_t.
//
// A block takes query rows that read the same cached rows and one span of their tokens (a split);
// a second launch joins the splits (short sequences: one launch, kv_whole_kernel).  Two ways to take them:
//   Attend, for the many rows of a prefix (all B * G queries of a kv head, 32 a wave): the codes are
//     turned into fp16 once per block, in LDS, and the prefix is read once per 128 rows.
//   Stream, for tiles of 16 rows (a sequence's own cache: the G heads of a kv head; a prefix of few
//     queries, or short beside the own caches): every wave streams tokens of its own, with no barrier
//     between the first and the join.
// Both multiply on the matrix cores, transposed (attn.h): S^T = K Q^T leaves a query row to a lane,
// which turns its scores into weights, and O^T = V^T P^T takes them from the lane's registers.
// A code goes in as the exact fp16 value (c - z) 2^-9, and a token's scales stay out of the 16-bit
// operands: K's multiplies the fp32 score, V's the softmax weight before it is rounded to fp16.
// bf16 queries are scaled by a power of two (query_exponent) and become fp16 exactly (8-bit
// significands; entries below 2^-21 of their row's largest may be off by 2^-29 of that one).
// Rounded to 16 bits are only the weights p s_t (fp16, relative 2^-11, scaled so that the largest
// s_t seen so far becomes 2^7 and small ones keep their bits) and the output.  Scores, maxima,
// sums and outputs are fp32.
#include <algorithm>

#include "attn.h"
#include "launch.h"

namespace w4a16 {

namespace {

constexpr int kThreads = 256;

// The codes of one 32-bit word as exact fp16 values: int8 c 2^-9 (4 codes, in order) or nibbles
// (u - z) 2^-9 (8 codes, order 0 4 1 5 2 6 3 7; exact for |u - z| <= 2048).  Masks or byte permutes
// leave the unsigned code as the subnormal u 2^-24 (two of the four masks: 16 u 2^-24), one packed
// fused multiply-add scales it and takes the zero point out.
__device__ __forceinline__ f16x2 as_h2(uint32_t w) { return __builtin_bit_cast(f16x2, w); }
__device__ __forceinline__ uint32_t as_u(f16x2 h) { return __builtin_bit_cast(uint32_t, h); }
__device__ __forceinline__ f16x2 both(float v) { return f16x2{(_Float16)v, (_Float16)v}; }
constexpr float kCodeUnit = 512.0f;                        // 2^9
__device__ __forceinline__ void codes_int8(uint32_t w, uint32_t out[2]) {
    const uint32_t b = w ^ 0x80808080u;                    // c + 128 per byte
    out[0] = as_u(__builtin_elementwise_fma(as_h2(perm(0u, b, 0x0C010C00u)), both(32768.0f), both(-0.25f)));
    out[1] = as_u(__builtin_elementwise_fma(as_h2(perm(0u, b, 0x0C030C02u)), both(32768.0f), both(-0.25f)));
}
__device__ __forceinline__ void codes_int4(uint32_t w, const u32x4& z9, uint32_t out[4]) {    // z9: -z 2^-9 of each
    unpack_mask_f16(w, out);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = as_u(__builtin_elementwise_fma(as_h2(out[i]), both(i & 1 ? 2048.0f : 32768.0f), as_h2(z9[i])));
}
__device__ __forceinline__ u32x4 same_zero(uint32_t pair) { return u32x4{pair, pair, pair, pair}; }

// the lanes 32 .. 63 of a and the lanes 0 .. 31 of b trade places
__device__ __forceinline__ void swap_halves(float& a, float& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(int, a), __builtin_bit_cast(int, b), false,
                                                    false);
    const int x = r[0], y = r[1];
    a = __builtin_bit_cast(float, x);
    b = __builtin_bit_cast(float, y);
}

// The power of two 2^e that a row of a bf16 query takes on its way to fp16, its largest entry being
// mx, the largest of all rows top (0: nothing finite).  The common factor brings top into [2^14,
// 2^15) and goes out of the scores with K's scales (cl); rows below 2^-10 of top, whose bits it would
// push out of fp16 (2^-21 of 2^4 has its last of 8 bits at fp16's last, 2^-24), take a factor of their own, and
// their scores rowf.  Returns whether there are any.
__device__ __forceinline__ float finite_or_zero(float x) { return x < __builtin_inff() ? x : 0.0f; }
__device__ __forceinline__ bool query_exponent(float mx, float top, int& e, float& cl, float& rowf) {
    const int e0 = top > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
    const bool mixed = __builtin_amdgcn_ballot_w64(mx > 0.0f && mx < top * 9.765625e-4f) != 0;   // 2^-10
    e = mixed && mx > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(mx) : e0;
    cl = ldexpf(cl, -e0);
    rowf = ldexpf(1.0f, e0 - e);
    return mixed;
}

// One set of caches as a block sees it: the rows of one (sequence and) kv head.
struct CacheRows {
    const unsigned char *kc, *vc;
    const uint16_t *ks, *kz, *vs, *vz;
};

template <int BITS, int D, int KT, int NBUF>
struct TileLds {
    uint16_t k[NBUF][KT * D], v[NBUF][KT * D];       // reused for the waves' outputs at the end
    float ks[NBUF][KT], vs[NBUF][KT];
    float vmax[NBUF][KT / 64];                       // largest V scale of 64 tokens
    float m[4][32], l[4][32];
};

// Orders what one wave writes to LDS before what its other lanes read of it (the LDS pipe keeps a
// wave's accesses in order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_lds_fence() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// The largest of the 64 lanes' values, in every lane.
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp_mov<0xB1>(v));
    v = fmaxf(v, dpp_mov<0x4E>(v));
    v = fmaxf(v, dpp_mov<0x141>(v));
    v = fmaxf(v, dpp_mov<0x140>(v));
    float r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 16 * i));
    return fmaxf(fmaxf(r[0], r[1]), fmaxf(r[2], r[3]));
}

// Tokens [t0, t1) of a cache for the 32 WQ rows from row0 on (R in all): row r is query head
// hq0 + (r / G) * Hq + r % G of the batch.  Writes each row's (max, sum) to ml and its unnormalized
// output to po at index head * nsplit + split.
// The waves stand along the rows, or (WQ = 2, WK = 2: up to 64 rows) in pairs along the rows and the
// tokens, each pair's two softmax states joined at the end.  Codes are loaded one tile ahead into
// registers, 16 bytes a lane, and stored as fp16 into LDS whose 16-byte pieces are permuted to spread
// both products' reads over the banks (the counters still show 0.8 conflict cycles an LDS instruction with
// 4-bit codes and 0.6 with 8-bit ones, not traced to an access); with two buffers (WK = 1) a tile costs one
// barrier.
// Bound by instructions rather than by its bytes: per code three or four operations to make it fp16
// (per block, so 128 rows share them), per score a scale, an exponential, a sum, another scale and a
// rounding.  128 sequences behind 32768 KV4 tokens, 32 heads on 8, D = 128 (70 GFLOP; with own caches of up
// to 1024 tokens 117 MB of cache): 105 us for the launch (117 traced), 0.67 PFLOP/s; the vector units are busy 42 %
// of the cycles, the matrix cores 27 %, and waves wait 33 % of theirs.  Tried and slower or equal: tiles
// of 32 tokens (three waves a SIMD instead of two: 165 us against 126 then), the scores of the next
// tile interleaved with the weights of this one as in attention.hip (118 us; with a second set of
// code registers 143), one wave a SIMD with twice the registers (166), blocks of eight waves and 256 rows,
// which halve the work on codes (131 against 115).
template <int BITS, int D, int WQ, int WK>
struct Attend {
    static constexpr int NBUF = WK == 1 ? 2 : 1;
    static constexpr int KT = WK == 1 ? 64 : 128;          // tokens of a tile
    static constexpr int KW = KT / WK;                     // tokens of a wave's share
    static constexpr int KB = KW / 32;
    static constexpr int RB = BITS == 8 ? D : D / 2;       // bytes of a cached row
    static constexpr int PR = RB / 16;                     // 16-byte pieces of it
    static constexpr int PIECES = KT * PR;
    static constexpr int PT = (PIECES + kThreads - 1) / kThreads;
    using Lds = TileLds<BITS, D, KT, NBUF>;

    static __device__ __forceinline__ void run(Lds& lds, const uint16_t* __restrict__ q, bool bf16, int Hq, int G,
                                               long long hq0, int row0, int R, CacheRows c, int t0, int t1, int nsplit,
                                               int split, float2* __restrict__ ml, float* __restrict__ po) {
        const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
        const int n = lane & 31, h = lane >> 5;
        const int wq = wave % WQ, wk = wave / WQ;
        const int row = row0 + 32 * wq + n;
        const int rr = min(row, R - 1);
        const long long head = hq0 + (long long)(rr / G) * Hq + rr % G;

        // the row's query as fp16, in the codes' order, times 2^e
        u32x4 qf[D / 16];
        float cl, rowf = 1.0f;                             // score scale: 2^9 log2(e) / sqrt(D) / 2^e
        bool mixed = false;                                // wave-uniform: the rows' factors differ
        {
            u32x4 raw[D / 16];
            const uint16_t* qp = q + head * D + 8 * h;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) raw[s] = *reinterpret_cast<const u32x4*>(qp + 16 * s);
            cl = 1.4426950408889634f * kCodeUnit / sqrtf((float)D);
            if (bf16) {
                float mx = 0.0f;
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx = fmaxf(mx, fmaxf(fabsf(bf2f(raw[s][i] & 0xFFFFu)), fabsf(bf2f(raw[s][i] >> 16))));
                // one factor for all rows of the block, which goes into K's scales
                mx = finite_or_zero(max_halves(mx));
                const float wave_mx = wave_max(mx);
                if (lane == 0) lds.m[wave][0] = wave_mx;
                __syncthreads();
                const float top = fmaxf(fmaxf(lds.m[0][0], lds.m[1][0]), fmaxf(lds.m[2][0], lds.m[3][0]));
                int e;
                mixed = query_exponent(mx, top, e, cl, rowf);
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        raw[s][i] = pack2<DT_F16>(ldexpf(bf2f(raw[s][i] & 0xFFFFu), e), ldexpf(bf2f(raw[s][i] >> 16), e));
            }
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                if constexpr (BITS == 4) {
                    uint32_t o[4];
                    permute_x8(raw[s].x, raw[s].y, raw[s].z, raw[s].w, o);
                    qf[s] = u32x4{o[0], o[1], o[2], o[3]};
                } else {
                    qf[s] = raw[s];
                }
            }
        }

        f32x16 o[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
        const float NEG = -__builtin_inff();
        // A weight is kept as 2^(s - sub), sub = m - lv with 2^lv = 128 / vcap, vcap the largest V scale so
        // far: that is what the second product takes (times the token's V scale, so at most 2^15),
        // and the common factor goes through l and O alike.  m may lag the maximum by 8.
        float sub = 0.0f, l = 0.0f;                        // base-2 domain
        float vcap = 5.9604644775390625e-8f;               // fp16's smallest
        float lv = 31.0f;                                  // log2(128 / vcap)

        u32x4 kr[PT], vr[PT];
        uint16_t pks = 0, pvs = 0, pkz[PT], pvz[PT];
        auto load = [&](int t) {
            const int base = t0 + t * KT;
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                const int p = tid + kThreads * i;
                // tokens behind the span: its last one, masked out of the scores
                const uint32_t tok = (uint32_t)min(base + p / PR, t1 - 1);
                if (PIECES % kThreads == 0 || p < PIECES) {
                    const size_t off = (size_t)tok * RB + 16 * (p % PR);
                    kr[i] = *reinterpret_cast<const u32x4*>(c.kc + off);
                    vr[i] = *reinterpret_cast<const u32x4*>(c.vc + off);
                    if constexpr (BITS == 4) {
                        pkz[i] = c.kz[tok];
                        pvz[i] = c.vz[tok];
                    }
                }
            }
            if (tid < KT) {
                const uint32_t tok = (uint32_t)min(base + tid, t1 - 1);
                pks = c.ks[tok];
                pvs = c.vs[tok];
            }
        };
        auto store = [&](int buf) {
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                const int p = tid + kThreads * i;
                if (PIECES % kThreads == 0 || p < PIECES) {
                    const int r = p / PR, pc = p % PR;
                    constexpr int OUT = BITS == 8 ? 2 : 4;  // fp16 pieces per 16 bytes of codes
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const u32x4 w = kv ? vr[i] : kr[i];
                        uint16_t* dst = (kv ? lds.v[buf] : lds.k[buf]) + r * D;
#pragma unroll
                        for (int j = 0; j < OUT; ++j) {
                            uint32_t d[4];
                            if constexpr (BITS == 8) {
                                codes_int8(w[2 * j], d);
                                codes_int8(w[2 * j + 1], d + 2);
                            } else {
                                const _Float16 z = __builtin_bit_cast(_Float16, kv ? pvz[i] : pkz[i]);
                                codes_int4(w[j], same_zero(as_u(f16x2{z, z} * both(-0.001953125f))), d);
                            }
                            const int ch = OUT * pc + j;
                            *reinterpret_cast<u32x4*>(dst + 8 * (kv ? swz_v<D>(r, ch) : swz_k<D>(r, ch))) =
                                u32x4{d[0], d[1], d[2], d[3]};
                        }
                    }
                }
            }
            if (tid < KT) {                                // whole waves
                const float s = h2f(pvs);
                lds.ks[buf][tid] = h2f(pks) * cl;
                lds.vs[buf][tid] = s;
                const float mx = wave_max(fabsf(s));
                if (lane == 0) lds.vmax[buf][tid >> 6] = mx;
            }
        };

        const int ntiles = (t1 - t0 + KT - 1) / KT;
        load(0);
        for (int t = 0; t < ntiles; ++t) {
            const int buf = NBUF == 2 ? t & 1 : 0;
            if (NBUF == 1 && t > 0) __syncthreads();       // the previous tile is done with
            store(buf);
            __syncthreads();
            if (t + 1 < ntiles) load(t + 1);

            const uint16_t* K = lds.k[buf] + wk * KW * D;
            const uint16_t* V = lds.v[buf] + wk * KW * D;
            const float* ksp = lds.ks[buf] + wk * KW;
            const float* vsp = lds.vs[buf] + wk * KW;
            const int tok0 = t0 + t * KT + wk * KW;        // first token of the wave's share
            f32x16 S[KB];
#pragma unroll
            for (int b = 0; b < KB; ++b) {
#pragma unroll
                for (int e = 0; e < 16; ++e) S[b][e] = 0.0f;
                const int r = 32 * b + n;                  // (KW is a multiple of 32: same swizzle)
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const u32x4 a = *reinterpret_cast<const u32x4*>(K + r * D + 8 * swz_k<D>(r, 2 * s + h));
                    S[b] = mfma<DT_F16>(a, qf[s], S[b]);
                }
            }
            if (mixed) {
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int e = 0; e < 16; ++e) S[b][e] *= rowf;
            }
            // exponents: the score times K's scale and the row's factor, minus the reference
            float mx = NEG;
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 s4 = *reinterpret_cast<const f32x4*>(ksp + 32 * b + 8 * g + 4 * h);
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[b][4 * g + j] = fmaf(S[b][4 * g + j], s4[j], -sub);
                }
            if (tok0 + KW > t1) {
                const int left = t1 - tok0 - 4 * h;        // (one register to compare constants with)
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (32 * b + 8 * (e >> 2) + (e & 3) >= left) S[b][e] = NEG;
            }
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) mx = fmaxf(mx, S[b][e]);
            mx = max_halves(mx);
            const float vm = __builtin_bit_cast(
                float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, lds.vmax[buf][wk * KW / 64])));
            if (t == 0 || vm > vcap || __builtin_amdgcn_ballot_w64(mx > 8.0f + lv)) {
                vcap = fmaxf(vcap, vm);
                const float ln = 7.0f - __builtin_amdgcn_logf(vcap);
                // the largest exponent becomes lv (the first tile's too, however low); a share of the
                // first tile without any token stays as it is, and all its weights are 0
                const float up = t > 0 ? fmaxf(mx, lv) : mx == NEG ? ln : mx;
                const float d = up - ln, f = exp2_raw(-d);
                lv = ln;
                sub += d;
                if (t > 0) {
                    l *= f;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[i][e] *= f;
                }
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int e = 0; e < 16; ++e) S[b][e] -= d;
            }
            u32x4 P[2 * KB];
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 s4 = *reinterpret_cast<const f32x4*>(vsp + 32 * b + 8 * g + 4 * h);
                    float p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[j] = exp2_raw(S[b][4 * g + j]);
                        l += p[j];
                        p[j] *= s4[j];
                    }
                    P[2 * b + (g >> 1)][2 * (g & 1)] = pack2<DT_F16>(p[0], p[1]);
                    P[2 * b + (g >> 1)][2 * (g & 1) + 1] = pack2<DT_F16>(p[2], p[3]);
                }
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int s = 0; s < 2 * KB; ++s) {
                    const int r = 16 * s + 4 * h + ((lane & 15) >> 2);
                    const int ch = 4 * i + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
                    const u32x2 a0 = lds_read_tr(V + r * D + 8 * swz_v<D>(r, ch) + 4 * (lane & 1));
                    const u32x2 a1 = lds_read_tr(V + (r + 8) * D + 8 * swz_v<D>(r + 8, ch) + 4 * (lane & 1));
                    o[i] = mfma<DT_F16>(u32x4{a0.x, a0.y, a1.x, a1.y}, P[s], o[i]);
                }
        }

        l = sum_halves(l);
        const float m = l == 0.0f ? NEG : sub;             // the reference of l and O (NaN: of no number)
        if constexpr (BITS == 4) {
            // lane halves hold elements 0 4 1 5 and 2 6 3 7 of every eight: to 0 .. 3 and 4 .. 7
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float e0 = o[i][4 * g], e1 = o[i][4 * g + 1], e2 = o[i][4 * g + 2], e3 = o[i][4 * g + 3];
                    swap_halves(e0, e1);
                    swap_halves(e2, e3);
                    o[i][4 * g] = e0;
                    o[i][4 * g + 1] = e2;
                    o[i][4 * g + 2] = e1;
                    o[i][4 * g + 3] = e3;
                }
        }
        const long long at = head * nsplit + split;
        if constexpr (WK == 1) {
            // through LDS, so that a row is stored as whole lines: lanes store 16 bytes 4 rows of a
            // column apart otherwise (32 sequences behind 4096 tokens: 4 us of 23)
            if (h == 0 && row < R) ml[at] = make_float2(m, l);
            static_assert(sizeof(lds.k) + sizeof(lds.v) >= 4 * 32 * D * sizeof(float), "output buffer");
            static_assert(offsetof(Lds, v) == sizeof(lds.k), "output buffer spans k and v");
            constexpr int CQ = D / 4;                      // 16-byte pieces of a row
            f32x4* ow = reinterpret_cast<f32x4*>(lds.k) + wave * 32 * CQ;
            __syncthreads();                               // everyone is done with K and V
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    ow[n * CQ + ((8 * i + 2 * g + h) ^ (n % CQ))] =
                        f32x4{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]} * kCodeUnit;
            wave_lds_fence();
            const int c = lane % CQ;
#pragma unroll 4
            for (int r = lane / CQ; r < 32; r += 64 / CQ) {
                const int gr = row0 + 32 * wq + r;
                if (gr < R) {
                    const long long to = (hq0 + (long long)(gr / G) * Hq + gr % G) * nsplit + split;
                    *reinterpret_cast<f32x4*>(po + to * D + 4 * c) = ow[r * CQ + (c ^ (r % CQ))];
                }
            }
        } else {
            // join the WK waves of each row set: every wave leaves its output, rescaled to the
            // common maximum, in LDS, and adds up its share of the elements over all of them
            __syncthreads();
            if (h == 0) {
                lds.m[wave][n] = m;
                lds.l[wave][n] = l;
            }
            __syncthreads();
            float M = NEG, L = 0.0f;
#pragma unroll
            for (int w = 0; w < WK; ++w) M = fmaxf(M, lds.m[w * WQ + wq][n]);
#pragma unroll
            for (int w = 0; w < WK; ++w)
                L += M == NEG ? 0.0f : lds.l[w * WQ + wq][n] * exp2_raw(lds.m[w * WQ + wq][n] - M);
            const float f = M == NEG ? 0.0f : exp2_raw(m - M) * kCodeUnit;
            float* ow = reinterpret_cast<float*>(lds.k);   // [wave][D / 4][32 rows][4] floats
            static_assert(sizeof(lds.k) + sizeof(lds.v) >= 4 * 32 * D * sizeof(float), "join buffer");
            static_assert(offsetof(Lds, v) == sizeof(lds.k), "join buffer spans k and v");
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<f32x4*>(ow + ((wave * (D / 4) + 8 * i + 2 * g + h) * 32 + n) * 4) =
                        f32x4{o[i][4 * g] * f, o[i][4 * g + 1] * f, o[i][4 * g + 2] * f, o[i][4 * g + 3] * f};
            __syncthreads();
            if (row < R) {
                if (wk == 0 && h == 0) ml[at] = make_float2(M, L);
                constexpr int NQ = D / 4 / WK / 2;         // 16-byte groups per lane half
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    const int dq = (wk * NQ + i) * 2 + h;
                    f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < WK; ++w)
                        a += *reinterpret_cast<const f32x4*>(ow + (((w * WQ + wq) * (D / 4) + dq) * 32 + n) * 4);
                    *reinterpret_cast<f32x4*>(po + at * D + 4 * dq) = a;
                }
            }
        }
    }
};

// 16 rows x 16 keys (S) or 16 elements (O) per tile: lane l holds column l % 16 (a query row), rows
// 4 (l / 16) + i.
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// Transposing LDS reads of the four groups of 16 lanes: 8-bit (8 rows of 16 bytes, lanes 2 r and
// 2 r + 1 at row r) and 4-bit (16 rows of 16 nibbles, lane r at row r); lane i of a group receives
// column i, the rows in order.
typedef int i32x2 __attribute__((ext_vector_type(2)));
template <int BITS>
__device__ __forceinline__ u32x2 lds_read_tr_codes(const unsigned char* p) {
    const auto q = (__attribute__((address_space(3))) i32x2*)p;
    if constexpr (BITS == 8) return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(q));
    else return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr4_b64_v2i32(q));
}

// The same value of the four lanes l % 16 + 16 k: their maximum / sum, in all of them.
template <class Op>
__device__ __forceinline__ float across_quarters(float x, Op op) {
    int i = __builtin_bit_cast(int, x);
    const auto r = __builtin_amdgcn_permlane16_swap(i, i, false, false);
    int a = r[0], b = r[1];
    float lo, hi;
    halves(op(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)), lo, hi);
    return op(lo, hi);
}

// Tokens [t0, t1) of a cache for the rows row0 .. row0 + 15 (R in all; numbered as in
// Attend), 16 x 16 x 32 products.  The cache is read once, so the aim is loads in flight and few
// instructions: each of the block's NW waves streams tiles of its own (wave, wave + NW, ...), with no
// barrier until they are joined at the end, and loads the next tile while it works on one.
// Measured: 16 sequences of up to 4096 KV8 tokens, 32 heads, D = 128 (318 MB with the scores): 62 us,
// 5.1 TB/s; 8 of up to 65536 KV4 tokens, 32 heads on 8 (365 MB): 94 us, 3.9 TB/s, the vector units busy
// 60 % of the cycles (twice the codes a byte).  Three blocks a CU: four spilled (254 us against 97 then).
// The staged form before it, with barriers between tiles, took 112 and 220 us for the same.
//   K's codes go from memory to the matrix cores: lane l loads the quarter l / 16 of every 64 bytes
//     (32 for the shortest rows) of key l % 16's row, so a load covers whole cache lines, and the
//     query's fragment is loaded in the same order.
//   V's codes are stored to LDS as they are and read back transposed (8- or 4-bit).
//   Codes become exact normal fp16 values with their zero point taken out (codes_int8 / codes_int4):
//     subnormals u 2^-24 would do without the multiply-add, but the matrix cores align a product by its
//     operands' exponents, a subnormal's being 2^-14, and drop what falls below: with 4-bit codes that
//     left sums off by 2^-15 of sum(p z), more than the output's rounding.
// Weights p s_t enter the second product times 128 / vcap, vcap the largest V scale so far, and the
// running maximum may lag by 8, so that they stay below 2^15; an fp16 subnormal among them is below
// 2^-14 of that, so its rounding adds at most 2^-32 vcap.
// WHOLE: the tokens [0, n2) of a second cache follow, and the block sees everything its rows do: it
// normalizes and rounds them to out instead of leaving them to a merge.
// SCORES: every score (base 2) is left in `score`, for row r and token t at index r spad + t, r the row's head
// in the batch, or (kInLds) its lane.
constexpr int kNone = 0, kInMemory = 1, kInLds = 2;
// ONCE: the codes are read once and loaded so that the caches do not keep them.
template <bool ONCE, class V>
__device__ __forceinline__ V load_codes(const unsigned char* p) {
    if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
    else return *reinterpret_cast<const V*>(p);
}
template <int BITS, int D, int SCORES, bool WHOLE = false, int NW = 4, bool ONCE = false>
struct Stream {
    static constexpr int KT = BITS == 8 && D == 128 ? 32 : 64;   // tokens of a tile
    static constexpr int NS = KT / 16;                           // S tiles
    static constexpr int RB = BITS == 8 ? D : D / 2;             // bytes of a cached row
    static constexpr int KW = RB / 16;                           // K: dwords per lane and S tile
    static constexpr int KB = RB / 4 < 16 ? RB / 4 : 16;         // K: bytes per load
    static constexpr int KQ = KB * 8 / BITS;                     // codes per load
    static constexpr int VL = KT * RB / 1024 > 0 ? KT * RB / 1024 : 1;   // V: 16-byte loads per lane
    static constexpr int VP = RB / 16;                           // 16-byte pieces of a row
    static constexpr int QS = D / 32;                            // k-steps of the first product
    static constexpr float LAG = 8.0f, VNORM = 128.0f;
    static_assert(KT * RB % 1024 == 0, "whole loads");

    struct alignas(16) WaveLds {
        unsigned char v[KT * RB];
        float ks[KT], vs[KT];
        _Float16 kz[BITS == 4 ? KT : 4], vz[BITS == 4 ? KT : 4];     // -z 2^-9
    };
    union Lds {
        WaveLds w[NW];
        float join[NW][D / 4][16][4];
    };

    // Where 16-byte piece c of token r's V row sits: spread over the banks for the transposing reads,
    // whose 32 lanes of a pass take one piece of the tokens 4 q + {0 .. 3} (+ 16 k), q of two values.
    static __device__ __forceinline__ int vpiece(int r, int c) {
        if constexpr (VP == 8) return c ^ (((r >> 1) & 1) | ((r >> 1) & 2) | ((r >> 2) & 4));
        else if constexpr (VP == 4 && BITS == 8) return c ^ (((r >> 2) & 1) | ((r >> 3) & 2));
        else if constexpr (VP == 4) return c ^ ((r >> 4) & 3);
        else return c ^ ((r >> 5) & 1);
    }

    static __device__ __forceinline__ void run(Lds& lds, float (*sm)[16], float (*sl)[16],
                                               const uint16_t* __restrict__ q, bool bf16, int Hq, int G, long long hq0,
                                               int row0, int R, const CacheRows& c1, int t0, int t1, int nsplit,
                                               int split, float2* __restrict__ ml, float* __restrict__ po,
                                               float* __restrict__ score, int spad, const CacheRows& c2 = {}, int n2 = 0,
                                               uint16_t* __restrict__ out = nullptr) {
        const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
        const int n = lane & 15, qd = lane >> 4;
        const int row = row0 + n;
        const int rr = min(row, R - 1);
        const long long head = hq0 + (long long)(rr / G) * Hq + rr % G;
        WaveLds& L = lds.w[wave];

        u32x4 kr[NS * KW / 4 > 0 ? NS * KW / 4 : 1], vr[VL];
        uint16_t pk = 0, pv = 0, pkz = 0, pvz = 0;
        const int tiles1 = (t1 - t0 + KT - 1) / KT;
        // tile t: its cache, first token and the end of the span that it is in
        auto place = [&](int t, int& tok, int& end) -> const CacheRows& {
            if (WHOLE && t >= tiles1) {
                tok = (t - tiles1) * KT;
                end = n2;
                return c2;
            }
            tok = t0 + t * KT;
            end = t1;
            return c1;
        };
        auto load = [&](int t) {
            int base, end;
            const CacheRows c = place(t, base, end);
            // tokens behind the span: its last one, masked out of the scores
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const uint32_t off = (uint32_t)min(base + 16 * s + n, end - 1) * RB + KB * qd;
                if constexpr (KW == 2) {
                    const u32x2 x = load_codes<ONCE, u32x2>(c.kc + off);
                    kr[s / 2][2 * (s % 2)] = x.x;
                    kr[s / 2][2 * (s % 2) + 1] = x.y;
                } else {
#pragma unroll
                    for (int i = 0; i < KW / 4; ++i)
                        kr[s * (KW / 4) + i] = load_codes<ONCE, u32x4>(c.kc + off + 64 * i);
                }
            }
#pragma unroll
            for (int i = 0; i < VL; ++i) {
                const int p = lane + 64 * i;
                vr[i] = load_codes<ONCE, u32x4>(c.vc + (uint32_t)min(base + p / VP, end - 1) * RB + 16 * (p % VP));
            }
            const uint32_t tok = (uint32_t)min(base + lane % KT, end - 1);
            if constexpr (KT == 64) {
                pk = c.ks[tok];
                pv = c.vs[tok];
            } else {
                pk = (lane < 32 ? c.ks : c.vs)[tok];             // lower half K's, upper half V's scales
            }
            if constexpr (BITS == 4) {
                pkz = c.kz[tok];
                pvz = c.vz[tok];
            }
        };
        const int tiles = tiles1 + (WHOLE ? (n2 + KT - 1) / KT : 0);
        if (wave < tiles) load(wave);
        __builtin_amdgcn_sched_barrier(0);

        // the row's query as fp16 times 2^e, in the order of the codes
        u32x4 qf[QS];
        float cl, rowf = 1.0f;                             // score scale: 2^9 log2(e) / sqrt(D) / 2^e
        {
            const uint16_t* qp = q + head * D + KQ * qd;
#pragma unroll
            for (int s = 0; s < QS; ++s)
                qf[s] = *reinterpret_cast<const u32x4*>(qp + 8 * s % KQ + 4 * KQ * (8 * s / KQ));
            cl = 1.4426950408889634f * kCodeUnit / sqrtf((float)D);
            if (bf16) {
                float mx = 0.0f;
#pragma unroll
                for (int s = 0; s < QS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx = fmaxf(mx, fmaxf(fabsf(bf2f(qf[s][i] & 0xFFFFu)), fabsf(bf2f(qf[s][i] >> 16))));
                // one factor for all rows of the tile, which goes into K's scales
                mx = finite_or_zero(across_quarters(mx, [](float a, float b) { return fmaxf(a, b); }));
                int e;
                query_exponent(mx, wave_max(mx), e, cl, rowf);
#pragma unroll
                for (int s = 0; s < QS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        qf[s][i] = pack2<DT_F16>(ldexpf(bf2f(qf[s][i] & 0xFFFFu), e), ldexpf(bf2f(qf[s][i] >> 16), e));
            }
#pragma unroll
            for (int s = 0; s < QS; ++s) {
                if constexpr (BITS == 4) {
                    uint32_t o[4];
                    permute_x8(qf[s].x, qf[s].y, qf[s].z, qf[s].w, o);
                    qf[s] = u32x4{o[0], o[1], o[2], o[3]};
                }
            }
        }

        constexpr int OT = D / 16;
        f32x4 o[OT];
#pragma unroll
        for (int i = 0; i < OT; ++i) o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const float NEG = -__builtin_inff();
        float m = NEG, l = 0.0f;                           // base-2 domain
        float vcap = 5.9604644775390625e-8f;               // fp16's smallest

        for (int t = wave; t < tiles; t += NW) {
            // this tile's V codes and parameters to LDS
#pragma unroll
            for (int i = 0; i < VL; ++i) {
                const int p = lane + 64 * i;
                *reinterpret_cast<u32x4*>(L.v + (p / VP) * RB + 16 * vpiece(p / VP, p % VP)) = vr[i];
            }
            const float vsc = KT == 64 ? h2f(pv) : lane < 32 ? 0.0f : h2f(pk);
            if (__builtin_amdgcn_ballot_w64(fabsf(vsc) > vcap)) {
                const float vn = wave_max(fmaxf(fabsf(vsc), vcap));
                const float f = vcap / vn;
                vcap = vn;
#pragma unroll
                for (int i = 0; i < OT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][e] *= f;
            }
            const float vinv = VNORM / vcap;
            if constexpr (KT == 64) {
                L.ks[lane] = h2f(pk) * cl;
                L.vs[lane] = vsc * vinv;
            } else {
                (lane < 32 ? L.ks : L.vs)[lane & 31] = lane < 32 ? h2f(pk) * cl : vsc * vinv;
            }
            if constexpr (BITS == 4) {
                L.kz[lane] = __builtin_bit_cast(_Float16, pkz) * (_Float16)-0.001953125f;
                L.vz[lane] = __builtin_bit_cast(_Float16, pvz) * (_Float16)-0.001953125f;
            }
            wave_lds_fence();

            f32x4 S[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                S[s] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                u32x4 z = {0, 0, 0, 0};
                if constexpr (BITS == 4) {
                    const _Float16 zk = L.kz[16 * s + n];
                    z = same_zero(as_u(f16x2{zk, zk}));
                }
#pragma unroll
                for (int k = 0; k < QS; ++k) {
                    uint32_t d[4];
                    if constexpr (BITS == 8) {
                        const int at = s * KW + 2 * k;
                        codes_int8(kr[at / 4][at % 4], d);
                        codes_int8(kr[at / 4][at % 4 + 1], d + 2);
                    } else {
                        const int at = s * KW + k;
                        codes_int4(kr[at / 4][at % 4], z, d);
                    }
                    S[s] = mfma16(u32x4{d[0], d[1], d[2], d[3]}, qf[k], S[s]);
                }
            }
            if (t + NW < tiles) load(t + NW);

            int tok0, end;
            place(t, tok0, end);
            float mt = NEG;
#pragma unroll
            for (int s = 0; s < NS; ++s) S[s] = S[s] * (*reinterpret_cast<const f32x4*>(&L.ks[16 * s + 4 * qd]) * rowf);
            if (tok0 + KT > end) {
                const int left = end - tok0 - 4 * qd;
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (16 * s + i >= left) S[s][i] = NEG;
            }
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) mt = fmaxf(mt, S[s][i]);
            if constexpr (SCORES != kNone) {
                if (row < R) {
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        const int tok = tok0 + 16 * s + 4 * qd;
                        if (tok < end) *reinterpret_cast<f32x4*>(score + (SCORES == kInLds ? n : head) * spad + tok) = S[s];
                    }
                }
            }
            mt = across_quarters(mt, [](float a, float b) { return fmaxf(a, b); });
            if (__builtin_amdgcn_ballot_w64(mt > m + LAG)) {
                const float mn = fmaxf(m, mt);
                const float f = mn == NEG ? 1.0f : exp2_raw(m - mn);
                m = mn;
                l *= f;
#pragma unroll
                for (int i = 0; i < OT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][e] *= f;
            }
            const float ms = m == NEG ? 0.0f : m;          // a row with nothing yet: every weight is 0
            u32x4 P[NS / 2];
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const f32x4 v4 = *reinterpret_cast<const f32x4*>(&L.vs[16 * s + 4 * qd]);
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[i] = exp2_raw(S[s][i] - ms);
                    l += p[i];
                    p[i] *= v4[i];
                }
                P[s / 2][2 * (s % 2)] = pack2<DT_F16>(p[0], p[1]);
                P[s / 2][2 * (s % 2) + 1] = pack2<DT_F16>(p[2], p[3]);
            }
            // O += V^T P^T; 4-bit: the tokens' zero points in the order of the fragment
            u32x4 z[NS / 2];
#pragma unroll
            for (int k = 0; k < NS / 2; ++k)
                if constexpr (BITS == 4) {
                    const u32x2 z0 = *reinterpret_cast<const u32x2*>(&L.vz[32 * k + 4 * qd]);
                    const u32x2 z1 = *reinterpret_cast<const u32x2*>(&L.vz[32 * k + 16 + 4 * qd]);
                    z[k] = u32x4{z0.x, z0.y, z1.x, z1.y};
                }
#pragma unroll
            for (int i = 0; i < OT; ++i) {
                if constexpr (BITS == 8) {
#pragma unroll
                    for (int k = 0; k < NS / 2; ++k) {
                        const int r = n >> 1;                                      // row of the lane pair
                        const int tok = 32 * k + 4 * qd + (r & 3) + 16 * (r >> 2);
                        const u32x2 w = lds_read_tr_codes<8>(L.v + tok * RB + 16 * vpiece(tok, i) + 8 * (n & 1));
                        uint32_t d[4];
                        codes_int8(w.x, d);
                        codes_int8(w.y, d + 2);
                        o[i] = mfma16(u32x4{d[0], d[1], d[2], d[3]}, P[k], o[i]);
                    }
                } else {
                    // row r of the group is the token whose nibble the masks put at its place: nibbles
                    // a and a + 4 of a dword are elements 2 a and 2 a + 1 of the fragment
                    const int j = 2 * (n & 3) + ((n >> 2) & 1);
                    const int tok = 32 * (n >> 3) + 4 * qd + (j & 3) + 16 * (j >> 2);
                    const u32x2 w = lds_read_tr_codes<4>(L.v + tok * RB + 16 * vpiece(tok, i >> 1) + 8 * (i & 1));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t d[4];
                        codes_int4(k ? w.y : w.x, z[k], d);
                        o[i] = mfma16(u32x4{d[0], d[1], d[2], d[3]}, P[k], o[i]);
                    }
                }
            }
            wave_lds_fence();                              // before the next tile overwrites this one
        }

        // join the waves: each leaves its output, rescaled to the common maximum, in LDS and adds up its
        // share of the elements over all of them
        l = across_quarters(l, [](float a, float b) { return a + b; });
        if (qd == 0) {
            sm[wave][n] = m;
            sl[wave][n] = l;
        }
        __syncthreads();
        float M = sm[0][n], Lt = 0.0f;
#pragma unroll
        for (int w = 1; w < NW; ++w) M = fmaxf(M, sm[w][n]);
#pragma unroll
        for (int w = 0; w < NW; ++w) Lt += M == NEG ? sl[w][n] : sl[w][n] * exp2_raw(sm[w][n] - M);   // (0 or NaN)
        const float f = M == NEG ? 0.0f : exp2_raw(m - M) * (vcap / VNORM * kCodeUnit);
#pragma unroll
        for (int i = 0; i < OT; ++i)
            *reinterpret_cast<f32x4*>(lds.join[wave][4 * i + qd][n]) = o[i] * f;
        __syncthreads();
        if (row < R) {
            const long long at = WHOLE ? head : head * nsplit + split;
            if (!WHOLE && wave == 0 && qd == 0) ml[at] = make_float2(M, Lt);
#pragma unroll
            for (int i = 0; i < (D / 16 + NW - 1) / NW; ++i) {
                const int dq = 4 * (wave + NW * i) + qd;
                if (D / 16 < NW && dq >= D / 4) break;
                f32x4 a = *reinterpret_cast<const f32x4*>(lds.join[0][dq][n]);
#pragma unroll
                for (int w = 1; w < NW; ++w) a += *reinterpret_cast<const f32x4*>(lds.join[w][dq][n]);
                if constexpr (WHOLE) {
                    uint16_t r[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float v = tiles > 0 ? a[j] / Lt : 0.0f;        // (no token at all: zeros)
                        r[j] = bf16 ? f2bf_bits(v) : f2h_bits(v);
                    }
                    // out is aligned to its elements only
#pragma unroll
                    for (int j = 0; j < 4; ++j) out[at * D + 4 * dq + j] = r[j];
                } else {
                    *reinterpret_cast<f32x4*>(po + at * D + 4 * dq) = a;
                }
            }
        }
    }
};

template <int BITS, int D>
__device__ __forceinline__ CacheRows cache_rows(const KvCache& c, long long rowbase) {
    constexpr int RB = BITS == 8 ? D : D / 2;
    CacheRows r;
    r.kc = static_cast<const unsigned char*>(c.kc) + rowbase * RB;
    r.vc = static_cast<const unsigned char*>(c.vc) + rowbase * RB;
    r.ks = c.ks + rowbase;
    r.vs = c.vs + rowbase;
    r.kz = BITS == 4 ? c.kz + rowbase : nullptr;
    r.vz = BITS == 4 ? c.vz + rowbase : nullptr;
    return r;
}

// A split with nothing in it: (-inf, 0) per row; the merge does not look at its output.
__device__ __forceinline__ void empty_split(long long hq0, int G, int Hq, int row0, int rows, int nsplit, int split,
                                            float2* ml) {
    for (int i = threadIdx.x; i < rows; i += kThreads) {
        const int r = row0 + i;
        ml[(hq0 + (long long)(r / G) * Hq + r % G) * nsplit + split] = make_float2(-__builtin_inff(), 0.0f);
    }
}

// The shared prefix in the first `pblocks` blocks, the sequences' own caches in the others, so that the
// arithmetic of the one and the loads of the other share the GPU.
//   Prefix, WQ > 0 (many rows): block = (kv head and split, tile of 32 WQ rows).  The row tiles of one
//     span run on one XCD, one after the other, so that the span's codes are read from HBM once.
//   Prefix, WQ == 0 (streamed): block = kv head, split, tile of 16 of its B G rows.
//   Own caches: block = split, sequence, kv head, tile of 16 of its G heads.  Splits vary slowest and
//     each turns the rest by one: consecutive blocks run on the 8 XCDs in turn, and the late splits
//     of short sequences, which are empty, have to fall on all of them (with the splits fastest, 16
//     sequences of 1024 .. 4096 tokens and 4 splits took 12 us longer, two XCDs having no empty
//     split at all).
struct DecodeGrid {
    int pblocks, psplit, pchunk, P, Pmax;    // prefix splits come first among a row's nsplit
    int osplit, ochunk, Tmax, nsplit;
};
template <int BITS, int D, int WQ>
struct PrefixKind {
    using type = Attend<BITS, D, WQ, 4 / WQ>;
};
template <int BITS, int D>
struct PrefixKind<BITS, D, 0> {
    using type = Stream<BITS, D, kNone>;
};
template <int BITS, int D, int WQ, bool SCORES, bool ONCE>
__global__ __launch_bounds__(kThreads, WQ == 0 ? 3 : 2)    // (streaming alone: three blocks a CU)
void kv_decode_kernel(const uint16_t* __restrict__ q, int bf16, int B, int Hq, int Hkv, KvCache prefix, KvCache own,
                      const int* __restrict__ lens, DecodeGrid g, float2* __restrict__ ml, float* __restrict__ po,
                      float* __restrict__ score, int spad) {
    using A = typename PrefixKind<BITS, D, WQ>::type;
    using S = Stream<BITS, D, SCORES ? kInMemory : kNone, false, 4, ONCE>;
    __shared__ union alignas(16) {
        typename A::Lds a;
        typename S::Lds s;
    } lds;
    __shared__ float sm[4][16], sl[4][16];
    const int G = Hq / Hkv;
    int id = blockIdx.x;
    if (id < g.pblocks) {
        const int R = B * G;
        constexpr int RT = WQ > 0 ? 32 * WQ : 16;
        const int rtiles = (R + RT - 1) / RT;
        const int j = id / 8;
        const int span = id % 8 + 8 * (j / rtiles), rt = j % rtiles;
        if (span >= Hkv * g.psplit) return;
        const int kvh = span / g.psplit, split = span % g.psplit;
        const int t0 = split * g.pchunk, t1 = min(g.P, t0 + g.pchunk);
        const CacheRows c = cache_rows<BITS, D>(prefix, (long long)kvh * g.Pmax);
        if constexpr (WQ > 0)
            A::run(lds.a, q, bf16 != 0, Hq, G, (long long)kvh * G, rt * RT, R, c, t0, t1, g.nsplit, split, ml, po);
        else
            A::run(lds.a, sm, sl, q, bf16 != 0, Hq, G, (long long)kvh * G, rt * RT, R, c, t0, t1, g.nsplit, split, ml,
                   po, nullptr, 0);
        return;
    }
    id -= g.pblocks;
    const int htiles = (G + 15) / 16, pairs = B * Hkv * htiles;
    const int os = id / pairs;
    id = (id % pairs + os) % pairs;
    const int row0 = 16 * (id % htiles);
    id /= htiles;
    const int kvh = id % Hkv, b = id / Hkv;
    const long long hq0 = (long long)b * Hq + (long long)kvh * G;
    const int T = min(max(lens[b], 0), g.Tmax);
    const int t0 = os * g.ochunk, t1 = min(T, t0 + g.ochunk), split = g.psplit + os;
    if (t0 >= t1) {
        empty_split(hq0, G, Hq, row0, min(16, G - row0), g.nsplit, split, ml);
        return;
    }
    S::run(lds.s, sm, sl, q, bf16 != 0, Hq, G, hq0, row0, G,
           cache_rows<BITS, D>(own, ((long long)b * Hkv + kvh) * g.Tmax), t0, t1, g.nsplit, split, ml, po, score, spad);
}

// Short sequences in one launch: block = sequence, kv head, tile of 16 of its G heads, over the prefix
// and the sequence's own tokens.  SCORES (G <= 16, no prefix): then the accumulated weights, from the scores
// that the block's waves have just written (up to kLdsTokens tokens to LDS).  Bound by the latency of a
// few dependent tiles a wave: 4 sequences behind 333 KV8 tokens, D = 64: 6.4 us; one of 500, with
// weights: 7.2.
constexpr int kLdsTokens = 512, kLdsStride = kLdsTokens + 4;     // (+ 4: the 16 rows start in different banks)
template <int BITS, int D, int SCORES, int NW>
__global__ __launch_bounds__(64 * NW, 2) void kv_whole_kernel(const uint16_t* __restrict__ q, int bf16, int Hq, int Hkv,
                                                               KvCache prefix, int P, int Pmax, KvCache own,
                                                               const int* __restrict__ lens, int Tmax,
                                                               uint16_t* __restrict__ out, float* score, int spad,
                                                               const float* weights, float* sums) {
    using S = Stream<BITS, D, SCORES, true, NW>;
    __shared__ typename S::Lds lds;
    __shared__ float sm[NW][16], sl[NW][16];
    __shared__ __attribute__((aligned(16))) float near[SCORES == kInLds ? 16 * kLdsStride : 4];
    const int G = Hq / Hkv, htiles = (G + 15) / 16;
    const int row0 = 16 * (blockIdx.x % htiles);
    const int bh = blockIdx.x / htiles, kvh = bh % Hkv, b = bh / Hkv;
    const long long hq0 = (long long)b * Hq + (long long)kvh * G;
    const int T = min(max(lens[b], 0), Tmax);
    const CacheRows mine = cache_rows<BITS, D>(own, (long long)bh * Tmax);
    if constexpr (SCORES != kNone) {
        const int stride = SCORES == kInLds ? kLdsStride : spad;
        float* at0 = SCORES == kInLds ? near : score;
        S::run(lds, sm, sl, q, bf16 != 0, Hq, G, hq0, row0, G, mine, 0, T, 0, 0, nullptr, nullptr, at0, stride, mine, 0,
               out);
        // sm, sl: written before the barrier that the scores were written before
        for (int t = 4 * threadIdx.x; t < T; t += 256 * NW) {
            f32x4 w = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int g = 0; g < G; ++g) {
                float M = sm[0][g], L = 0.0f;
#pragma unroll
                for (int i = 1; i < NW; ++i) M = fmaxf(M, sm[i][g]);
#pragma unroll
                for (int i = 0; i < NW; ++i) L += sl[i][g] * exp2_raw(sm[i][g] - M);
                const f32x4 s =
                    *reinterpret_cast<const f32x4*>(at0 + (SCORES == kInLds ? g : hq0 + g) * stride + t);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = fmaf(exp2_raw(s[j] - M), 1.0f / L, w[j]);
            }
            const long long at = (long long)bh * Tmax + t;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (t + j < T) sums[at + j] = (weights ? weights[at + j] : 0.0f) + w[j];
        }
    } else {
        S::run(lds, sm, sl, q, bf16 != 0, Hq, G, hq0, row0, G, cache_rows<BITS, D>(prefix, (long long)kvh * Pmax), 0, P, 0,
               0, nullptr, nullptr, nullptr, 0, mine, T, out);
    }
}

// (max, sum) over all splits of a row; every lane of the wave gets it.
__device__ __forceinline__ void row_stats(const float2* __restrict__ ml, int nsplit, int lane, float& M, float& L) {
    const float NEG = -__builtin_inff();
    float m = NEG, l = 0.0f;
    for (int j = lane; j < nsplit; j += 64) {
        const float2 v = ml[j];
        const float mn = fmaxf(m, v.x);
        l = mn == NEG ? l + v.y : l * exp2_raw(m - mn) + v.y * exp2_raw(v.x - mn);     // (at -inf: 0 or NaN)
        m = mn;
    }
    M = wave_max(m);
    L = wave_sum(m == NEG ? l : l * exp2_raw(m - M));
}

// out = sum_j O_j 2^(m_j - M) / sum_j l_j 2^(m_j - M) over the splits j.  One block per query head of
// the batch: each group of D / 4 threads adds up splits grp, grp + NG, ... (16 bytes a thread, several
// loads in flight), the groups are added through LDS; a row without any token gets zeros, one of scores
// that are no numbers NaN.  Bound by the
// latency of two dependent loads, then by the partial outputs' bytes: 2.7 us for 32 heads, 4.2 us
// for 1024 of 17 splits, 9.3 us (39 MB) for 4096 of up to 18.
template <int D>
__device__ __forceinline__ void merge_row(float (*part)[D], long long head, const float2* __restrict__ ml,
                                          const float* __restrict__ po, int nsplit, int bf16, bool tokens,
                                          uint16_t* __restrict__ out) {
    constexpr int CQ = D / 4, NG = kThreads / CQ;
    const int tid = threadIdx.x, c = tid % CQ, grp = tid / CQ;
    const float2* mlr = ml + head * nsplit;
    const float* pr = po + head * nsplit * D + 4 * c;
    float M, L;
    row_stats(mlr, nsplit, tid & 63, M, L);
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int j = grp; j < nsplit; j += NG) {
        const float2 v = mlr[j];
        const f32x4 x = *reinterpret_cast<const f32x4*>(pr + (long long)j * D);
        // an empty split's output is not defined
        if (v.y != 0.0f) acc += x * exp2_raw(v.x - M);
    }
    *reinterpret_cast<f32x4*>(&part[grp][4 * c]) = acc;
    __syncthreads();
    if (tid < D) {
        float s = part[0][tid];
#pragma unroll
        for (int i = 1; i < NG; ++i) s += part[i][tid];
        const float v = tokens ? s / L : 0.0f;
        out[head * D + tid] = bf16 ? f2bf_bits(v) : f2h_bits(v);
    }
}

template <int D>
__global__ __launch_bounds__(kThreads) void kv_merge_kernel(const float2* __restrict__ ml, const float* __restrict__ po,
                                                            int nsplit, int bf16, int Hq, int P,
                                                            const int* __restrict__ lens, uint16_t* __restrict__ out) {
    __shared__ __attribute__((aligned(16))) float part[kThreads / (D / 4)][D];
    merge_row<D>(part, blockIdx.x, ml, po, nsplit, bf16, P > 0 || lens[blockIdx.x / Hq] > 0, out);
}

// Output and accumulated weights in one launch: the first `heads` blocks merge a query head each,
// the others turn kSpan scores of a (sequence, kv head) into weights: a token's p of each head is
// 2^(score - M) / L, so the streaming kernel leaves the scores (base 2, fp32) instead of reading the
// cache twice.  Bound by the scores' bytes, G x 4 a token and kv head: 7.8 us (15 MB) for 16 x 32 heads
// of up to 4096 tokens, 15 us (70 MB, G = 4) for 8 x 32 of up to 65536.
constexpr int kSpan = 4 * kThreads;
constexpr int kStatHeads = 64;           // heads whose statistics are at hand at a time
template <int D>
__global__ __launch_bounds__(kThreads) void kv_weights_kernel(const float2* __restrict__ ml,
                                                              const float* __restrict__ po, int nsplit, int bf16,
                                                              uint16_t* __restrict__ out, int heads, int Hq, int Hkv,
                                                              const int* __restrict__ lens, int Tmax, int spans,
                                                              const float* __restrict__ score, int spad,
                                                              const float* weights, float* sums) {   // (may be one)
    __shared__ __attribute__((aligned(16))) float part[kThreads / (D / 4)][D];
    __shared__ float2 stat[kStatHeads];                    // a head's maximum and 1 / sum
    if (blockIdx.x < (unsigned)heads) {
        merge_row<D>(part, blockIdx.x, ml, po, nsplit, bf16, lens[blockIdx.x / Hq] > 0, out);
        return;
    }
    const int i = blockIdx.x - heads;
    const int bh = i / spans, t0 = (i % spans) * kSpan;
    const int b = bh / Hkv, G = Hq / Hkv;
    const int T = min(max(lens[b], 0), Tmax);
    if (t0 >= T) return;
    const long long hq0 = (long long)b * Hq + (long long)(bh % Hkv) * G;
    const int t = t0 + 4 * threadIdx.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const long long at = (long long)bh * Tmax + t;
    float before[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) before[j] = weights && t + j < T ? weights[at + j] : 0.0f;
    f32x4 w = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int g0 = 0; g0 < G; g0 += kStatHeads) {
        const int gn = min(G - g0, kStatHeads);
        if (g0 > 0) __syncthreads();
        for (int g = wave; g < gn; g += kThreads / 64) {
            float M, L;
            row_stats(ml + (hq0 + g0 + g) * nsplit, nsplit, lane, M, L);
            if (lane == 0) stat[g] = make_float2(M, 1.0f / L);
        }
        __syncthreads();
        if (t < T) {
            const float* sp = score + (hq0 + g0) * spad + t;
#pragma unroll 4
            for (int g = 0; g < gn; ++g) {
                const f32x4 s = *reinterpret_cast<const f32x4*>(sp + (long long)g * spad);
                const float2 st = stat[g];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = fmaf(exp2_raw(s[j] - st.x), st.y, w[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (t + j < T) sums[at + j] = before[j] + w[j];
}

// ------------------------------------------------------------------------------- host side

// Blocks to aim for: streaming, 8 a CU against ragged lengths (1024, 4096 and 8192 within 3 % or slower);
// Attend, the 2 a CU that run at once.  A split has at least 256 tokens: a row of its partial output is as
// large as four rows of KV8 cache, and 128 rows write one each (32 sequences behind 4096 tokens: 128 and
// 64 tokens, 28 and 37 us against 23).
constexpr long long kBlocks = 2048;
constexpr long long kPrefixBlocks = 512;
constexpr int kMinChunk = 256;
// Own caches that are read once (one tile of heads) and are most of the work pass the GPU's caches by: with
// weights, caches that are not in the last-level cache (as between the layers of a model) of 17 MB 13.0 -> 12.0 us,
// 134 MB 42.8 -> 40.1, 268 MB 62.3 -> 55.6, 537 MB 119 -> 106; one and the same cache again and again 10.9 -> 10.8,
// 34.0 -> 39.6, 49.3 -> 55.4, 117 -> 106.  Not behind a longer prefix: 128 sequences of up to 1024 behind 32768
// tokens 118.8 -> 120.2, 32 of up to 512 behind 4096 21.8 -> 23.0; nor where two tiles of heads read them: G = 32,
// 34 MB, 33.5 -> 38.1.
constexpr int kOnceHeads = 16;

int divup(long long a, long long b) { return (int)((a + b - 1) / b); }

int chunk_of(long long T, long long tiles, long long blocks, long long least) {
    const long long ns = blocks / tiles > 1 ? blocks / tiles : 1;
    return (int)(divup(divup(T, ns), least) * least);
}
// tokens per split of a sequence's own cache, and of the prefix
int own_chunk(long long B, long long Hq, long long Hkv, long long T) {
    return chunk_of(T, B * Hkv * divup(Hq / Hkv, 16), kBlocks, kMinChunk);
}
// How the R = B G rows of a kv head meet the prefix: streamed (0) where they are one tile of Stream's, or
// where the own caches are most of the work (the kernel then runs three blocks a CU instead of two), else
// Attend with WQ = 2 or 4.  Whole calls, streamed / 2 / 4, KV8, 32 heads on 8, D = 128:
//   16 sequences of up to 4096 own tokens, no prefix / 512 tokens   23.3 / 25.7 / 25.8, 24.7 / 27.3 / 27.3 us
//   64 of up to 2048, 512 / 4096 tokens                 39.4 / 41.1 / 40.8, 54.5 / 52.7 / 48.2
//   8 rows, 4096 / 32768 tokens, 100 own ones           16.8 / 16.9 / 17.2, 25.9 / 26.5 / 32.2
//   20, 64 rows, 32768 tokens                           33.8 / 26.6 / 33.3, 40.0 / 31.2 / 37.2
//   128, 256 rows, 32768 tokens                         61.0 / 40.4 / 41.2, 98.1 / 65.1 / 61.1
// (128 rows of bf16, 4096 tokens and up to 512 own ones: 24.4 / 23.0 / 21.0, so those take 4; of fp16 with
// hardly any own ones 64-row blocks were 19.6 against 22.2: type and own length were not varied apart).
int prefix_wq(long long R, long long P, long long Tmax) { return R <= 16 || 4 * P <= Tmax ? 0 : R <= 64 ? 2 : 4; }
int prefix_chunk(long long B, long long Hq, long long Hkv, long long P, long long Tmax) {
    if (P == 0) return kMinChunk;
    const long long R = B * (Hq / Hkv);
    const int wq = prefix_wq(R, P, Tmax);
    return wq == 0 ? chunk_of(P, Hkv * divup(R, 16), kBlocks, kMinChunk)
                   : chunk_of(P, Hkv * divup(R, 32 * wq), kPrefixBlocks, kMinChunk);
}

// Waves of a block that takes a sequence and kv head whole (kv_whole_kernel), or 0: splits that a second
// launch joins.  Us in a graph, whole / split; a call by itself saves 3 - 4 us of submission besides, so that
// a little more is taken where few blocks leave the GPU empty.  KV8, D = 128:
//   prefix (3 / 4 of the tokens) and own caches, 4 waves: 1 x 8, 16 x 8, 64 x 8 kv heads of 512 tokens 8.0 / 8.5,
//     8.2 / 12.4, 11.6 / 17.1; 64 x 32 33 / 32, 256 x 32 139 / 125 (the prefix is read again for every sequence);
//     64 x 8 of 768, 1024, 1536 14.9 / 18.2, 18.1 / 18.8, 24.2 / 21.5; 16 x 32, one row each, of 768 15.8 / 12.6
//   8 waves: 1 x 8 of 768, 1024 9.5 / 8.3, 10.8 / 8.3; 16 x 8 9.9 / 12.6, 11.2 / 12.7; 32 x 8 10.3 / 16.4,
//     11.4 / 16.5
//   with weights, 4 waves: 1 x 8 of 512 9.3 / 9.7; 64 x 8 of 1024, 2048 27.4 / 34.0, 50.1 / 55.1; of ragged lengths
//     1024 kv heads of 2048, 4096 (4-bit) 52.7 / 53.2, 113.0 / 112.9
//   8 waves: 1 x 8 of 768, 1024 11.1 / 9.7, 12.6 / 9.7 (4-bit 9.3 / 9.1, 11.0 / 9.2); 16 x 8 11.7 / 12.8, 14.0 /
//     14.1, 1536 17.6 / 17.5; of 512 tokens 10.3 against 10.0 with 4 waves
int whole_shared(long long B, long long Hkv, long long G, long long P, long long Tmax) {
    const long long N = P + Tmax, blocks = B * Hkv * divup(G, 16);
    if (N <= 512 && B * Hkv * P <= (1 << 20)) return 4;
    if (N <= 768 && blocks <= 256) return 8;
    return N <= 1024 && B * G > 16 && blocks <= 512 ? (blocks <= 256 ? 8 : 4) : 0;
}
int whole_weights(long long B, long long Hkv, long long G, long long Tmax) {
    const long long blocks = B * Hkv;
    if (G > 16) return 0;
    if (Tmax <= 512) return 4;
    if (blocks <= 256) return Tmax <= 768 || (Tmax <= 1024 && blocks >= 128) ? 8 : 0;
    return Tmax <= 2048 && Tmax * Tmax <= 4096 * blocks ? 4 : 0;
}

long long parts_floats(long long heads, long long ns, long long D) { return heads * ns * (D + 2); }

template <int BITS, int D>
hipError_t shared(const KvSharedArgs& a, float* work, hipStream_t st) {
    const int G = a.Hq / a.Hkv;
    const long long heads = (long long)a.B * a.Hq, R = (long long)a.B * G;
#define W4A16_WHOLE(NW)                                                                                                \
    hipLaunchKernelGGL((kv_whole_kernel<BITS, D, kNone, NW>), dim3((unsigned)(a.B * a.Hkv * divup(G, 16))),            \
                       dim3(64 * NW), 0, st, static_cast<const uint16_t*>(a.q), a.dtype == DT_BF16, a.Hq, a.Hkv,       \
                       a.prefix, a.P, a.Pmax, a.own, a.lens, a.Tmax, static_cast<uint16_t*>(a.out), nullptr, 0,        \
                       nullptr, nullptr)
    if (const int nw = whole_shared(a.B, a.Hkv, G, a.P, a.Tmax)) {
        if (nw == 4) W4A16_WHOLE(4);
        else W4A16_WHOLE(8);
        return hipGetLastError();
    }
#undef W4A16_WHOLE
    const int wq = prefix_wq(R, a.P, a.Tmax);
    DecodeGrid g = {};
    g.P = a.P;
    g.Pmax = a.Pmax;
    g.Tmax = a.Tmax;
    g.pchunk = prefix_chunk(a.B, a.Hq, a.Hkv, a.P, a.Tmax);
    g.psplit = divup(a.P, g.pchunk);
    g.pblocks = (int)(8 * divup((long long)a.Hkv * g.psplit, 8) * (long long)divup(R, wq ? 32 * wq : 16));
    g.ochunk = own_chunk(a.B, a.Hq, a.Hkv, a.Tmax);
    g.osplit = divup(a.Tmax, g.ochunk);
    g.nsplit = g.psplit + g.osplit;
    float* po = work;                                       // 16-byte aligned rows first
    float2* ml = reinterpret_cast<float2*>(work + heads * g.nsplit * D);
    const auto q = static_cast<const uint16_t*>(a.q);
    const int bf16 = a.dtype == DT_BF16;
    const dim3 grid((unsigned)(g.pblocks + (long long)a.B * a.Hkv * divup(G, 16) * g.osplit));
#define W4A16_DECODE(WQ, ONCE)                                                                                         \
    hipLaunchKernelGGL((kv_decode_kernel<BITS, D, WQ, false, ONCE>), grid, dim3(kThreads), 0, st, q, bf16, a.B, a.Hq,  \
                       a.Hkv, a.prefix, a.own, a.lens, g, ml, po, nullptr, 0)
    if (wq == 2) W4A16_DECODE(2, false);
    else if (wq == 4) W4A16_DECODE(4, false);
    else if (G <= kOnceHeads) W4A16_DECODE(0, true);
    else W4A16_DECODE(0, false);
#undef W4A16_DECODE
    hipLaunchKernelGGL((kv_merge_kernel<D>), dim3((unsigned)heads), dim3(kThreads), 0, st, ml, po, g.nsplit, bf16,
                       a.Hq, a.P, a.lens, static_cast<uint16_t*>(a.out));
    return hipGetLastError();
}

int score_pad(long long Tmax) { return (int)((Tmax + 3) / 4 * 4); }

template <int BITS, int D>
hipError_t weights(const KvWeightsArgs& a, float* work, hipStream_t st) {
    const int G = a.Hq / a.Hkv;
    DecodeGrid g = {};
    g.Tmax = a.Tmax;
    g.ochunk = own_chunk(a.B, a.Hq, a.Hkv, a.Tmax);
    g.osplit = g.nsplit = divup(a.Tmax, g.ochunk);
    const int ns = g.nsplit;
    const long long heads = (long long)a.B * a.Hq;
    const int spad = score_pad(a.Tmax);
    float* score = work;
    float* po = work + heads * spad;
    float2* ml = reinterpret_cast<float2*>(po + heads * ns * D);
    const int bf16 = a.dtype == DT_BF16;
#define W4A16_WHOLE(SCORES, NW)                                                                                        \
    hipLaunchKernelGGL((kv_whole_kernel<BITS, D, SCORES, NW>), dim3((unsigned)(a.B * a.Hkv)), dim3(64 * NW), 0, st,    \
                       static_cast<const uint16_t*>(a.q), bf16, a.Hq, a.Hkv, KvCache{}, 0, 0, a.own, a.lens, a.Tmax,   \
                       static_cast<uint16_t*>(a.out), score, spad, a.weights, a.sums)
    if (const int nw = whole_weights(a.B, a.Hkv, G, a.Tmax)) {
        if (a.Tmax <= kLdsTokens) W4A16_WHOLE(kInLds, 4);
        else if (nw == 4) W4A16_WHOLE(kInMemory, 4);
        else W4A16_WHOLE(kInMemory, 8);
        return hipGetLastError();
    }
#undef W4A16_WHOLE
    const unsigned blocks = (unsigned)((long long)a.B * a.Hkv * divup(G, 16) * g.osplit);
#define W4A16_DECODE(ONCE)                                                                                             \
    hipLaunchKernelGGL((kv_decode_kernel<BITS, D, 0, true, ONCE>), dim3(blocks), dim3(kThreads), 0, st,                \
                       static_cast<const uint16_t*>(a.q), bf16, a.B, a.Hq, a.Hkv, KvCache{}, a.own, a.lens, g, ml, po, \
                       score, spad)
    if (G <= kOnceHeads) W4A16_DECODE(true);
    else W4A16_DECODE(false);
#undef W4A16_DECODE
    const int spans = divup(a.Tmax, kSpan);
    hipLaunchKernelGGL((kv_weights_kernel<D>), dim3((unsigned)(heads + (long long)a.B * a.Hkv * spans)),
                       dim3(kThreads), 0, st, ml, po, ns, bf16, static_cast<uint16_t*>(a.out), (int)heads, a.Hq, a.Hkv,
                       a.lens, a.Tmax, spans, score, spad, a.weights, a.sums);
    return hipGetLastError();
}

}  // namespace

long long kv_shared_call_floats(long long B, long long Hq, long long Hkv, long long P, long long Tmax, long long D) {
    if (whole_shared(B, Hkv, Hq / Hkv, P, Tmax)) return 0;
    return parts_floats(B * Hq, divup(P, prefix_chunk(B, Hq, Hkv, P, Tmax)) + divup(Tmax, own_chunk(B, Hq, Hkv, Tmax)), D);
}

long long kv_weights_call_floats(long long B, long long Hq, long long Hkv, long long Tmax, long long D) {
    if (whole_weights(B, Hkv, Hq / Hkv, Tmax)) return Tmax <= kLdsTokens ? 0 : B * Hq * score_pad(Tmax);
    return B * Hq * score_pad(Tmax) + parts_floats(B * Hq, divup(Tmax, own_chunk(B, Hq, Hkv, Tmax)), D);
}

// The sizes that callers are told: what any call of at most B sequences, P and Tmax tokens uses.  (What a
// call uses itself falls here and there as these grow: chunks are rounded up, and the rules above
// change the kernel.)  A row has at most max(1, blocks / tiles) splits and one per kMinChunk tokens, so
// over all b <= B:
//   own caches, b Hkv tiles(G) tiles: Hq b max(1, min(c / b, s)) <= Hq max(B, min(c, B s)), with
//     c = kBlocks / (Hkv tiles(G)) and s the splits of kMinChunk tokens;
//   prefix, Hkv divup(b G, rt) tiles of rt rows for b Hq rows: blocks / tiles splits are at most blocks rt
//     rows' outputs, kBlocks of 16 or kPrefixBlocks of 64 or, for more than 64 rows, of 128.
static long long own_rows(long long B, long long Hq, long long Hkv, long long Tmax) {
    const long long c = kBlocks / (Hkv * divup(Hq / Hkv, 16));
    return Hq * std::max(B, std::min(c, B * divup(Tmax, kMinChunk)));
}
static long long prefix_rows(long long B, long long Hq, long long Hkv, long long P) {
    if (P == 0) return 0;
    const long long most = std::max(16 * kBlocks, (B * (Hq / Hkv) > 64 ? 128 : 64) * kPrefixBlocks);
    return std::max(B * Hq, std::min(most, B * Hq * divup(P, kMinChunk)));
}

long long kv_shared_workspace_floats(long long B, long long Hq, long long Hkv, long long P, long long Tmax,
                                     long long D) {
    // whole_shared, where every smaller call is one of its too (the last rule asks for more than 16 rows)
    const long long G = Hq / Hkv, N = P + Tmax, blocks = B * Hkv * divup(G, 16);
    if (whole_shared(B, Hkv, G, P, Tmax) && (N <= 512 || (N <= 768 && blocks <= 256) || G > 16)) return 0;
    return (prefix_rows(B, Hq, Hkv, P) + own_rows(B, Hq, Hkv, Tmax)) * (D + 2);
}

long long kv_weights_workspace_floats(long long B, long long Hq, long long Hkv, long long Tmax, long long D) {
    const bool few = Hq / Hkv <= 16;
    if (few && Tmax <= kLdsTokens) return 0;
    const long long scores = B * Hq * score_pad(Tmax);
    // whole_weights at every smaller size too
    if (few && Tmax <= 768 && B * Hkv <= 256) return scores;
    return scores + own_rows(B, Hq, Hkv, Tmax) * (D + 2);
}

hipError_t launch_kv_shared(const KvSharedArgs& a, float* work, hipStream_t st) {
    if (a.bits == 8) return a.D == 64 ? shared<8, 64>(a, work, st) : shared<8, 128>(a, work, st);
    return a.D == 64 ? shared<4, 64>(a, work, st) : shared<4, 128>(a, work, st);
}

hipError_t launch_kv_weights(const KvWeightsArgs& a, float* work, hipStream_t st) {
    if (a.bits == 8) return a.D == 64 ? weights<8, 64>(a, work, st) : weights<8, 128>(a, work, st);
    return a.D == 64 ? weights<4, 64>(a, work, st) : weights<4, 128>(a, work, st);
}

}  // namespace w4a16
