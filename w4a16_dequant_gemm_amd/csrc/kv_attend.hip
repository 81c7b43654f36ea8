// Decode attention over the quantized cache on the matrix cores: one query per sequence and head
// over a prefix that all sequences of the batch share followed by the sequence's own tokens, and
// decode attention that also adds up the attention weight every cached token receives.
//
//   out[b, h] = sum_t p_t v_t,  p = softmax_t(q[b, h] . k_t / sqrt(D)),  k_t = s_t (c_t - z_t)
//
// over the P shared tokens and the lengths[b] own ones (kv head h / (Hq / Hkv)), and
//   sums[b, kv head, t] = weights[b, kv head, t] + sum over the group's heads of p_t.
//
// A block takes up to 32 WQ query rows that read the same cached rows and one span of tokens (a
// split).  Rows of the shared prefix are all B * G queries of a kv head (the prefix is read once per
// 128 of them, not once per sequence); rows of a sequence's own cache are the G heads of a kv head.
// The tokens go through in tiles: the codes are loaded coalesced one tile ahead into registers,
// turned into exact fp16 integers (c - z) and stored to LDS, and the four waves of the block
// multiply them on the matrix cores (attn.h), side by side along the rows (WQ = 4, many rows) or
// along the tokens (WK = 4, few rows: each wave then has its own softmax state and the four are
// joined at the end).  A token's scales stay out of the 16-bit operands: K's multiplies the fp32
// score, V's the softmax weight before it is rounded to fp16.  bf16 queries are scaled by a power
// of two per row so that their largest entry is in [2^14, 2^15) and become fp16 exactly (8-bit
// significands; an entry below 2^-28 of the row's largest may lose bits, 2^-39 of that entry).
// Rounded to 16 bits are only the weights p s_t (fp16, relative 2^-11, scaled so that the largest
// s_t seen so far becomes 2^7 and small ones keep their bits) and the output.  Scores, maxima,
// sums and outputs are fp32; splits are joined by a second launch.
#include "attn.h"
#include "launch.h"

namespace w4a16 {

namespace {

constexpr int kThreads = 256;

// The codes of one 32-bit word as exact fp16 integers: int8 c (4 codes, in order) or nibbles
// u - z (8 codes, order 0 4 1 5 2 6 3 7).  The code is OR-ed / permuted into the mantissa of 1024.
__device__ __forceinline__ f16x2 as_h2(uint32_t w) { return __builtin_bit_cast(f16x2, w); }
__device__ __forceinline__ uint32_t as_u(f16x2 h) { return __builtin_bit_cast(uint32_t, h); }
__device__ __forceinline__ void codes_int8(uint32_t w, uint32_t out[2]) {
    const uint32_t b = w ^ 0x80808080u;                    // c + 128 per byte
    const f16x2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
    out[0] = as_u(as_h2(perm(0x64646464u, b, 0x04010400u)) - off);
    out[1] = as_u(as_h2(perm(0x64646464u, b, 0x04030402u)) - off);
}
__device__ __forceinline__ void codes_int4(uint32_t w, f16x2 z, uint32_t out[4]) {
    const f16x2 off = {(_Float16)1024.0f, (_Float16)1024.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = as_u(as_h2(((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u) - off - z);
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

// The largest of the 64 lanes' non-negative values, in every lane.
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

// Tokens [t0, t1) of a cache for the rows row0 .. (R in all): row r is query head
// hq0 + (r / G) * Hq + r % G of the batch.  Writes each row's (max, sum) to ml and its unnormalized
// output (elements in storage order, see codes_int4) to po at index head * nsplit + split.
// SCORES: also the base-2 scores, score[head * spad + token].
template <int BITS, int D, int WQ, int WK, bool SCORES>
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
                                               int split, float2* __restrict__ ml, float* __restrict__ po,
                                               float* __restrict__ score, int spad) {
        const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
        const int n = lane & 31, h = lane >> 5;
        const int wq = wave % WQ, wk = wave / WQ;
        const int row = row0 + 32 * wq + n;
        const int rr = min(row, R - 1);
        const long long head = hq0 + (long long)(rr / G) * Hq + rr % G;

        // the row's query as fp16, in the codes' order, times 2^e
        u32x4 qf[D / 16];
        float cl;                                          // score scale: log2(e) / sqrt(D) / 2^e
        {
            u32x4 raw[D / 16];
            const uint16_t* qp = q + head * D + 8 * h;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) raw[s] = *reinterpret_cast<const u32x4*>(qp + 16 * s);
            cl = 1.4426950408889634f / sqrtf((float)D);
            if (bf16) {
                float mx = 0.0f;
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx = fmaxf(mx, fmaxf(fabsf(bf2f(raw[s][i] & 0xFFFFu)), fabsf(bf2f(raw[s][i] >> 16))));
                mx = max_halves(mx);
                const int e = mx > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(mx) : 0;
                cl = ldexpf(cl, -e);
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
        float m = NEG, l = 0.0f;                           // base-2 domain
        // weights enter the second product times 128 / vcap, vcap the largest V scale so far
        float vcap = 5.9604644775390625e-8f;               // fp16's smallest

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
                                codes_int4(w[j], f16x2{z, z}, d);
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
                lds.ks[buf][tid] = h2f(pks);
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
            // scores in the base-2 domain: times K's scale and the row's factor
            const bool tail = tok0 + KW > t1;
            float mt = NEG;
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 s4 = *reinterpret_cast<const f32x4*>(ksp + 32 * b + 8 * g + 4 * h);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float v = S[b][4 * g + j] * (s4[j] * cl);
                        if (tail && tok0 + 32 * b + 8 * g + 4 * h + j >= t1) v = NEG;
                        S[b][4 * g + j] = v;
                        mt = fmaxf(mt, v);
                    }
                }
            if constexpr (SCORES) {
                if (row < R) {
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const int tok = tok0 + 32 * b + 8 * g + 4 * h;
                            if (tok < t1)
                                *reinterpret_cast<f32x4*>(score + head * spad + tok) =
                                    f32x4{S[b][4 * g], S[b][4 * g + 1], S[b][4 * g + 2], S[b][4 * g + 3]};
                        }
                }
            }
            mt = max_halves(mt);
            const float vm = __builtin_bit_cast(
                float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, lds.vmax[buf][wk * KW / 64])));
            // the maximum may lag by 8 (weights up to 2^8), so O is rarely rescaled
            if (vm > vcap || __builtin_amdgcn_ballot_w64(mt > m + 8.0f)) {
                const float mn = fmaxf(m, mt), vn = fmaxf(vcap, vm);
                const float f = mn == NEG ? 1.0f : exp2_raw(m - mn);
                const float fo = f * (vcap / vn);
                m = mn;
                vcap = vn;
                l *= f;
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[i][e] *= fo;
            }
            const float vinv = 128.0f / vcap;
            const float ms = m == NEG ? 0.0f : m;          // a row with nothing yet: every weight is 0
            u32x4 P[2 * KB];
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 s4 = *reinterpret_cast<const f32x4*>(vsp + 32 * b + 8 * g + 4 * h);
                    float p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[j] = exp2_raw(S[b][4 * g + j] - ms);
                        l += p[j];
                        p[j] *= s4[j] * vinv;
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
        const float vout = vcap * 0.0078125f;              // O in its own units
        const long long at = head * nsplit + split;
        if constexpr (WK == 1) {
            if (row < R) {
                if (h == 0) ml[at] = make_float2(m, l);
                float* op = po + at * D + 4 * h;
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        *reinterpret_cast<f32x4*>(op + 32 * i + 8 * g) =
                            f32x4{o[i][4 * g] * vout, o[i][4 * g + 1] * vout, o[i][4 * g + 2] * vout,
                                  o[i][4 * g + 3] * vout};
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
            const float f = M == NEG ? 0.0f : exp2_raw(m - M) * vout;
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

// The shared prefix: block = (kv head and split, tile of 32 WQ rows).  The row tiles of one span run
// on one XCD, one after the other, so that the span's codes are read from HBM once.
template <int BITS, int D, int WQ>
__global__ __launch_bounds__(kThreads, 2) void kv_prefix_kernel(const uint16_t* __restrict__ q, int bf16, int B, int Hq,
                                                                int Hkv, KvCache c, int P, int Pmax, int chunk,
                                                                int psplit, int nsplit, float2* __restrict__ ml,
                                                                float* __restrict__ po) {
    using A = Attend<BITS, D, WQ, 4 / WQ, false>;
    __shared__ __attribute__((aligned(16))) typename A::Lds lds;
    const int G = Hq / Hkv, R = B * G;
    const int rtiles = (R + 32 * WQ - 1) / (32 * WQ);
    const int j = blockIdx.x / 8;
    const int span = blockIdx.x % 8 + 8 * (j / rtiles), rt = j % rtiles;
    if (span >= Hkv * psplit) return;
    const int kvh = span / psplit, split = span % psplit;
    const int t0 = split * chunk, t1 = min(P, t0 + chunk);
    A::run(lds, q, bf16 != 0, Hq, G, (long long)kvh * G, rt * 32 * WQ, R,
           cache_rows<BITS, D>(c, (long long)kvh * Pmax), t0, t1, nsplit, split, ml, po, nullptr, 0);
}

// The sequences' own caches: block = (split, kv head and tile of 32 of its heads, sequence).
template <int BITS, int D, bool SCORES>
__global__ __launch_bounds__(kThreads, 2) void kv_own_kernel(const uint16_t* __restrict__ q, int bf16, int Hq, int Hkv,
                                                             KvCache c, const int* __restrict__ lens, int Tmax,
                                                             int chunk, int first, int nsplit, float2* __restrict__ ml,
                                                             float* __restrict__ po, float* __restrict__ score,
                                                             int spad) {
    using A = Attend<BITS, D, 1, 4, SCORES>;
    __shared__ __attribute__((aligned(16))) typename A::Lds lds;
    const int G = Hq / Hkv, htiles = (G + 31) / 32;
    const int kvh = blockIdx.y / htiles, row0 = 32 * (blockIdx.y % htiles);
    const int b = blockIdx.z, split = first + blockIdx.x;
    const int T = min(max(lens[b], 0), Tmax);
    const int t0 = blockIdx.x * chunk, t1 = min(T, t0 + chunk);
    const long long hq0 = (long long)b * Hq + (long long)kvh * G;
    if (t0 >= t1) {
        empty_split(hq0, G, Hq, row0, min(32, G - row0), nsplit, split, ml);
        return;
    }
    A::run(lds, q, bf16 != 0, Hq, G, hq0, row0, G, cache_rows<BITS, D>(c, ((long long)b * Hkv + kvh) * Tmax), t0, t1,
           nsplit, split, ml, po, score, spad);
}

// (max, sum) over all splits of a row; every lane of the wave gets it.
__device__ __forceinline__ void row_stats(const float2* __restrict__ ml, int nsplit, int lane, float& M, float& L) {
    const float NEG = -__builtin_inff();
    float m = NEG, l = 0.0f;
    for (int j = lane; j < nsplit; j += 64) {
        const float2 v = ml[j];
        const float mn = fmaxf(m, v.x);
        if (mn != NEG) l = l * exp2_raw(m - mn) + v.y * exp2_raw(v.x - mn);
        m = mn;
    }
    M = m;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
    L = wave_sum(m == NEG ? 0.0f : l * exp2_raw(m - M));
}

// One block per query head of the batch: wave w adds up splits w, w + 4, ...; a row that saw no
// token gets zeros.
template <int BITS, int D>
__device__ __forceinline__ void merge_row(float (*part)[D], long long head, const float2* __restrict__ ml,
                                          const float* __restrict__ po, int nsplit, int bf16,
                                          uint16_t* __restrict__ out) {
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    constexpr int V = D / 64;                              // elements per lane
    const float2* mlr = ml + head * nsplit;
    float M, L;
    row_stats(mlr, nsplit, lane, M, L);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll 4
    for (int j = wave; j < nsplit; j += 4) {
        const float mj = mlr[j].x;
        const float w = mj == -__builtin_inff() ? 0.0f : exp2_raw(mj - M);
        const float* p = po + (head * nsplit + j) * D + lane * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float x = p[i];
            acc[i] = w > 0.0f ? fmaf(w, x, acc[i]) : acc[i];   // an empty split's output is not defined
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) part[wave][lane * V + i] = acc[i];
    __syncthreads();
    if (tid < D) {
        const float s = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        // 4-bit rows are stored in the order 0 4 1 5 2 6 3 7 of every eight elements
        const int e = BITS == 8 ? tid : (tid & ~7) + ((tid & 1) << 2) + ((tid & 7) >> 1);
        const float v = L > 0.0f ? s / L : 0.0f;
        out[head * D + e] = bf16 ? f2bf_bits(v) : f2h_bits(v);
    }
}

template <int BITS, int D>
__global__ __launch_bounds__(kThreads) void kv_merge_kernel(const float2* __restrict__ ml, const float* __restrict__ po,
                                                            int nsplit, int bf16, uint16_t* __restrict__ out) {
    __shared__ float part[4][D];
    merge_row<BITS, D>(part, blockIdx.x, ml, po, nsplit, bf16, out);
}

// Output and accumulated weights in one launch: the first `heads` blocks merge a query head each,
// the others turn kSpan scores of a (sequence, kv head) into weights.
constexpr int kSpan = 4 * kThreads;
template <int BITS, int D>
__global__ __launch_bounds__(kThreads) void kv_weights_kernel(const float2* __restrict__ ml,
                                                              const float* __restrict__ po, int nsplit, int bf16,
                                                              uint16_t* __restrict__ out, int heads, int Hq, int Hkv,
                                                              const int* __restrict__ lens, int Tmax, int spans,
                                                              const float* __restrict__ score, int spad,
                                                              const float* __restrict__ weights,
                                                              float* __restrict__ sums) {
    __shared__ float part[4][D];
    if (blockIdx.x < (unsigned)heads) {
        merge_row<BITS, D>(part, blockIdx.x, ml, po, nsplit, bf16, out);
        return;
    }
    const int i = blockIdx.x - heads;
    const int bh = i / spans, t0 = (i % spans) * kSpan;
    const int b = bh / Hkv, G = Hq / Hkv;
    const int T = min(max(lens[b], 0), Tmax);
    if (t0 >= T) return;
    const long long hq0 = (long long)b * Hq + (long long)(bh % Hkv) * G;
    const int t = t0 + 4 * threadIdx.x;
    float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int g = 0; g < G; ++g) {
        float M, L;
        row_stats(ml + (hq0 + g) * nsplit, nsplit, threadIdx.x & 63, M, L);
        const float inv = 1.0f / L;
        if (t < T) {
            const f32x4 s = *reinterpret_cast<const f32x4*>(score + (hq0 + g) * spad + t);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = fmaf(exp2_raw(s[j] - M), inv, w[j]);
        }
    }
    const long long at = (long long)bh * Tmax + t;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (t + j < T) sums[at + j] = (weights ? weights[at + j] : 0.0f) + w[j];
}

// ------------------------------------------------------------------------------- host side

constexpr long long kBlocks = 2048;      // blocks of the own caches' kernel to aim for
constexpr long long kPrefixBlocks = 1024;
constexpr int kMinChunk = 256;           // tokens of a split, at least

int divup(long long a, long long b) { return (int)((a + b - 1) / b); }

// tokens per split of a sequence's own cache (a multiple of the tile)
int own_chunk(long long B, long long Hq, long long Hkv, long long T) {
    const long long pairs = B * Hkv * ((Hq / Hkv + 31) / 32);
    const long long ns = kBlocks / pairs > 1 ? kBlocks / pairs : 1;
    const long long c = divup(divup(T, ns), 128) * 128;
    return (int)(c < kMinChunk ? kMinChunk : c);
}
int prefix_wq(long long R) { return R <= 32 ? 1 : R <= 64 ? 2 : 4; }
int prefix_chunk(long long B, long long Hq, long long Hkv, long long P) {
    const long long R = B * (Hq / Hkv);
    const long long tiles = Hkv * divup(R, 32 * prefix_wq(R));
    const long long ns = kPrefixBlocks / tiles > 1 ? kPrefixBlocks / tiles : 1;
    const long long c = divup(divup(P, ns), 128) * 128;
    return (int)(c < kMinChunk ? kMinChunk : c);
}

long long parts_floats(long long heads, long long ns, long long D) { return heads * ns * (D + 2); }

template <int BITS, int D>
hipError_t shared(const KvSharedArgs& a, float* work, hipStream_t st) {
    const int pc = prefix_chunk(a.B, a.Hq, a.Hkv, a.P), ps = divup(a.P, pc);
    const int oc = own_chunk(a.B, a.Hq, a.Hkv, a.Tmax), os = divup(a.Tmax, oc);
    const int ns = ps + os, G = a.Hq / a.Hkv;
    const long long heads = (long long)a.B * a.Hq;
    float* po = work;                                       // 16-byte aligned rows first
    float2* ml = reinterpret_cast<float2*>(work + heads * ns * D);
    const auto q = static_cast<const uint16_t*>(a.q);
    const int bf16 = a.dtype == DT_BF16;
    if (ps > 0) {
        const long long R = (long long)a.B * G;
        const int wq = prefix_wq(R), rtiles = divup(R, 32 * wq);
        const dim3 grid((unsigned)(8 * divup((long long)a.Hkv * ps, 8) * (long long)rtiles));
        if (wq == 1)
            hipLaunchKernelGGL((kv_prefix_kernel<BITS, D, 1>), grid, dim3(kThreads), 0, st, q, bf16, a.B, a.Hq, a.Hkv,
                               a.prefix, a.P, a.Pmax, pc, ps, ns, ml, po);
        else if (wq == 2)
            hipLaunchKernelGGL((kv_prefix_kernel<BITS, D, 2>), grid, dim3(kThreads), 0, st, q, bf16, a.B, a.Hq, a.Hkv,
                               a.prefix, a.P, a.Pmax, pc, ps, ns, ml, po);
        else
            hipLaunchKernelGGL((kv_prefix_kernel<BITS, D, 4>), grid, dim3(kThreads), 0, st, q, bf16, a.B, a.Hq, a.Hkv,
                               a.prefix, a.P, a.Pmax, pc, ps, ns, ml, po);
    }
    hipLaunchKernelGGL((kv_own_kernel<BITS, D, false>), dim3(os, a.Hkv * divup(G, 32), a.B), dim3(kThreads), 0, st, q,
                       bf16, a.Hq, a.Hkv, a.own, a.lens, a.Tmax, oc, ps, ns, ml, po, nullptr, 0);
    hipLaunchKernelGGL((kv_merge_kernel<BITS, D>), dim3((unsigned)heads), dim3(kThreads), 0, st, ml, po, ns, bf16,
                       static_cast<uint16_t*>(a.out));
    return hipGetLastError();
}

int score_pad(long long Tmax) { return (int)((Tmax + 3) / 4 * 4); }

template <int BITS, int D>
hipError_t weights(const KvWeightsArgs& a, float* work, hipStream_t st) {
    const int oc = own_chunk(a.B, a.Hq, a.Hkv, a.Tmax), ns = divup(a.Tmax, oc), G = a.Hq / a.Hkv;
    const long long heads = (long long)a.B * a.Hq;
    const int spad = score_pad(a.Tmax);
    float* score = work;
    float* po = work + heads * spad;
    float2* ml = reinterpret_cast<float2*>(po + heads * ns * D);
    const int bf16 = a.dtype == DT_BF16;
    hipLaunchKernelGGL((kv_own_kernel<BITS, D, true>), dim3(ns, a.Hkv * divup(G, 32), a.B), dim3(kThreads), 0, st,
                       static_cast<const uint16_t*>(a.q), bf16, a.Hq, a.Hkv, a.own, a.lens, a.Tmax, oc, 0, ns, ml, po,
                       score, spad);
    const int spans = divup(a.Tmax, kSpan);
    hipLaunchKernelGGL((kv_weights_kernel<BITS, D>), dim3((unsigned)(heads + (long long)a.B * a.Hkv * spans)),
                       dim3(kThreads), 0, st, ml, po, ns, bf16, static_cast<uint16_t*>(a.out), (int)heads, a.Hq, a.Hkv,
                       a.lens, a.Tmax, spans, score, spad, a.weights, a.sums);
    return hipGetLastError();
}

}  // namespace

long long kv_shared_workspace_floats(long long B, long long Hq, long long Hkv, long long P, long long Tmax,
                                     long long D) {
    return parts_floats(B * Hq, divup(P, prefix_chunk(B, Hq, Hkv, P)) + divup(Tmax, own_chunk(B, Hq, Hkv, Tmax)), D);
}

long long kv_weights_workspace_floats(long long B, long long Hq, long long Hkv, long long Tmax, long long D) {
    return B * Hq * score_pad(Tmax) + parts_floats(B * Hq, divup(Tmax, own_chunk(B, Hq, Hkv, Tmax)), D);
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
