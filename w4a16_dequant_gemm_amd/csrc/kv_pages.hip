// Rotary positions, appending to a paged 8-bit KV cache and reading it back.
//
// Rotation of a pair (x0, x1) of a head by its token's position: with a = position * f,
//   y0 = m (x0 cos a - x1 sin a),   y1 = m (x1 cos a + x0 sin a),
// pairs (i, i + R / 2) or (2 i, 2 i + 1) of the head's first R values; the rest passes through.
//
// Append: a page's scale is the largest |x| / top of the tokens written to it since its first, so it grows
// as the page fills; codes are rint(x / s) (or the nearest e4m3), those already there are rounded again where
// s has grown.  A block takes some heads of a page of one cache: rows into registers, rotated there in fp32, their
// largest value, the scale, the codes.  Bound by memory and by the latency of those steps: 12 chunks of up to 1024 tokens,
// 32 heads of K, V and queries, D = 128, pages of 32 (101 MB), take 27 us (3.8 TB/s); a token each of 128 sequences, 32 / 8
// heads, 6.2 - 7.8 us where no page's scale grows, 11.4 with new rows each step, of which some page grows nearly always
// (its codes are read, rounded and written by one wave), 12 where all do; of 4 sequences 3.2.
#include <algorithm>

#include "pages.h"

namespace w4a16 {

namespace {

// ---------------------------------------------------------------- rotations

// Which position a token has: given, or its place in its sequence's cache.  False for one of no sequence.
struct Places {
    const int *positions, *lens, *cu;
    int B, T;
};
__device__ __forceinline__ bool place_of(const Places& p, int token, int lane, int& place) {
    int b = token, end = token + 1;
    if (p.cu) {
        b = __builtin_amdgcn_readfirstlane(sequence_of(p.cu, p.B, p.T, token, lane));
        if (min(max(p.cu[b], 0), p.T) > token) return false;
        end = min(max(p.cu[b + 1], 0), p.T);
        if (end <= token) return false;
    }
    place = p.positions ? p.positions[token] : p.lens[b] - end + token;
    return true;
}

struct RopeView {
    const uint16_t* x;
    uint16_t* out;
    const long long* freqs;
    Places at;
    float m;
    int xs, os;             // elements from row to row
    int T, H, D, half;      // half: R / 2
    int inter, copy;        // copy: the values behind R too
};

constexpr int kRopePairs = 256;         // pairs of a head at most

// One token by one block: its angles' cos and sin once into LDS, then all heads, V pairs a thread at a time, two heads
// asked for at once.  The inputs pass the caches by: most are not read again, and the outputs, which are, find more room
// there (16384 tokens of 40 heads, D = 128: 70 -> 67 us when a block had four tokens, with the attention behind it
// 234 -> 230; outputs past the caches too: 64, but with the attention 237).  More tokens a block were slower (two 63 us,
// four 67, one 59: 5.7 TB/s).
template <int V>
struct Piece { typedef u32x4 type; };
template <>
struct Piece<1> { typedef uint16_t type; };

template <int DT, int V, int AT>
__device__ __forceinline__ void rope_token(const RopeView& r, int token, float* lc, float* ls) {
    typedef typename Piece<V>::type P;
    const int tid = threadIdx.x & 255, lane = tid & 63;
    int place = 0;
    if (!place_of(r.at, token, lane, place)) return;
    // (a copying step takes two pieces too, where they go into what is copied: 5001 tokens of 64 heads, 48 of 128
    // values turned, 35.4 -> 33.1 us)
    const bool two = V == 1 || (r.D - 2 * r.half) % (2 * V) == 0;
    const int step = two ? 2 * V : V, turns = r.half / V, units = turns + (r.copy ? (r.D - 2 * r.half) / step : 0);
    const int rows = 256 / units, unit = tid % units, row = tid / units;
    const bool turning = unit < turns;
    // the unit's values: two pieces (of V) of the rotation, or one to copy
    const int p = unit * V, e = 2 * r.half + (unit - turns) * step;
    const int at0 = turning ? (r.inter ? 2 * p : p) : e, at1 = turning ? (r.inter ? 2 * p + V : p + r.half) : two ? e + V : e;
    const uint16_t* x = r.x + (long long)token * r.xs;
    uint16_t* out = r.out + (long long)token * r.os;
    if (tid < r.half) position_cos_sin(place, r.freqs[tid], r.m, lc[tid], ls[tid]);
    __syncthreads();
    if (row >= rows) return;
    for (int h0 = row; h0 < r.H; h0 += AT * rows) {
        P lo[AT], hi[AT];
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            const int h = min(h0 + j * rows, r.H - 1);
            lo[j] = __builtin_nontemporal_load(reinterpret_cast<const P*>(x + h * r.D + at0));
            hi[j] = __builtin_nontemporal_load(reinterpret_cast<const P*>(x + h * r.D + at1));
        }
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            const int h = h0 + j * rows;
            if (h >= r.H) break;
            if (turning) {
                const float *c = lc + p, *s = ls + p;
                if constexpr (V == 8) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float x0 = in2f<DT>(lo[j][k] & 0xFFFFu), x1 = in2f<DT>(lo[j][k] >> 16);
                        float z0 = in2f<DT>(hi[j][k] & 0xFFFFu), z1 = in2f<DT>(hi[j][k] >> 16);
                        if (r.inter) {
                            turn_pair(x0, x1, c[k], s[k]);
                            turn_pair(z0, z1, c[k + 4], s[k + 4]);
                        } else {
                            turn_pair(x0, z0, c[2 * k], s[2 * k]);
                            turn_pair(x1, z1, c[2 * k + 1], s[2 * k + 1]);
                        }
                        lo[j][k] = pack2<DT>(x0, x1);
                        hi[j][k] = pack2<DT>(z0, z1);
                    }
                } else {
                    float x0 = in2f<DT>(lo[j]), x1 = in2f<DT>(hi[j]);
                    turn_pair(x0, x1, c[0], s[0]);
                    lo[j] = f2out<DT>(x0);
                    hi[j] = f2out<DT>(x1);
                }
            }
            uint16_t* po = out + h * r.D;
            *reinterpret_cast<P*>(po + at0) = lo[j];
            if (turning || two) *reinterpret_cast<P*>(po + at1) = hi[j];
        }
    }
}

template <int DT, int V>
__global__ __launch_bounds__(256) void rope_kernel(RopeView r) {
    __shared__ __attribute__((aligned(16))) float lc[kRopePairs], ls[kRopePairs];
    rope_token<DT, V, 2>(r, blockIdx.x, lc, ls);
}

bool rope_wide(const RopeView& r) {
    const auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    return r.half % 8 == 0 && r.D % 8 == 0 && r.xs % 8 == 0 && r.os % 8 == 0 && at16(r.x) && at16(r.out);
}

hipError_t rope(const RopeView& r, int dtype, hipStream_t st) {
    const dim3 grid((unsigned)r.T), block(256);
    if (rope_wide(r)) {
        if (dtype == DT_F16) hipLaunchKernelGGL((rope_kernel<DT_F16, 8>), grid, block, 0, st, r);
        else hipLaunchKernelGGL((rope_kernel<DT_BF16, 8>), grid, block, 0, st, r);
    } else {
        if (dtype == DT_F16) hipLaunchKernelGGL((rope_kernel<DT_F16, 1>), grid, block, 0, st, r);
        else hipLaunchKernelGGL((rope_kernel<DT_BF16, 1>), grid, block, 0, st, r);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------- append

__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp_mov<0xB1>(v));     // quad_perm [1,0,3,2]
    v = fmaxf(v, dpp_mov<0x4E>(v));     // quad_perm [2,3,0,1]
    v = fmaxf(v, dpp_mov<0x141>(v));    // row_half_mirror
    v = fmaxf(v, dpp_mov<0x140>(v));    // row_mirror
    const int i = __builtin_bit_cast(int, v);
    const auto at = [&](int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(i, l)); };
    return fmaxf(fmaxf(at(0), at(16)), fmaxf(at(32), at(48)));
}
// |x| where it is a number, else 0
__device__ __forceinline__ float size_of(float x) {
    const float a = fabsf(x);
    return a < __builtin_inff() ? a : 0.0f;
}

struct AppendView {
    KvPages c;
    const uint16_t *k, *v;
    const long long* freqs;
    const int* positions;
    float m;
    int ks, vs;             // elements from row to row
    int half, inter;        // half: R / 2 (0: no rotation)
};

// Heads h0 .. h1 - 1 of one page of K (ACROSS false: rows, rotated) or V (columns).  Thread units of eight values: of K
// four pairs (p .. p + 3 of the rotation, or eight adjacent values behind it), of V eight adjacent ones.  A thread's
// units are of the same tokens and pairs for every head: their angles are computed once.  (A head's rows asked for
// while the one before is worked on: no faster, and half as fast with pages of 128, for its registers.)
// Threads of a block: at most four units each.
constexpr int append_threads(int D, int page) { return page * D >= 8192 ? 512 : 256; }

template <int DT, int FMT, int D, int PAGE, bool ACROSS>
__device__ __forceinline__ void append_page(const AppendView& a, const PageTokens& p, int h0, int h1, uint8_t* lds,
                                            float (*red)[9]) {
    constexpr int NT = append_threads(D, PAGE);
    constexpr int UR = D / 8, UNITS = PAGE * UR > NT ? PAGE * UR / NT : 1;         // units of a row; of a thread
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int total = p.n * UR, j = tid % UR, t0 = tid / UR;       // unit i of a thread: token t0 + NT / UR i, values of j
    const uint16_t* src = ACROSS ? a.v : a.k;
    const int stride = ACROSS ? a.vs : a.ks;

    // a unit's values: of four pairs (first, second) in a word each, or eight in a row
    u32x4 raw[UNITS];
    const bool turns = !ACROSS && 4 * j < a.half;
    const bool halves = turns && !a.inter && a.half % 4 == 0;      // two pieces of four values
    const bool loose = turns && !a.inter && a.half % 4 != 0;       // value by value
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            if (NT * i >= total) break;
            const uint16_t* row = src + (long long)(p.token + min(t0 + NT / UR * i, p.n - 1)) * stride + h * D;
            if (halves) {
                const u32x2 lo = *reinterpret_cast<const u32x2*>(row + 4 * j);
                const u32x2 hi = *reinterpret_cast<const u32x2*>(row + a.half + 4 * j);
                raw[i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
            } else if (loose) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int q = 4 * j + e;
                    const bool turn = q < a.half;
                    raw[i][e] = row[turn ? q : 2 * q] | (uint32_t)row[turn ? q + a.half : 2 * q + 1] << 16;
                }
            } else raw[i] = *reinterpret_cast<const u32x4*>(row + 8 * j);
        }
    };
    load(h0);
    float cs[ACROSS ? 1 : UNITS][8];            // cos and sin of a unit's pairs
    if (!ACROSS && turns) {
        long long f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = a.freqs[min(4 * j + e, a.half - 1)];
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            if (NT * i >= total) break;
            const int t = min(t0 + NT / UR * i, p.n - 1);
            const int position = a.positions ? a.positions[p.token + t] : p.index * PAGE + p.off + t;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                cs[ACROSS ? 0 : i][2 * e] = 1.0f;
                cs[ACROSS ? 0 : i][2 * e + 1] = 0.0f;
                if (4 * j + e < a.half) position_cos_sin(position, f[e], a.m, cs[ACROSS ? 0 : i][2 * e], cs[ACROSS ? 0 : i][2 * e + 1]);
            }
        }
    }
    const int id = page_id(a.c.table, a.c.P, a.c.N, p.b, p.index);
    if (id < 0) return;
    float* scale = (ACROSS ? a.c.vs : a.c.ks) + (long long)id * a.c.Hkv + h0;

#pragma unroll 1
    for (int h = h0; h < h1; ++h, ++scale) {
        uint8_t* codes = (uint8_t*)(ACROSS ? a.c.vc : a.c.kc) + ((long long)id * a.c.Hkv + h) * (PAGE * D);
        float* r = red[h & 1];
        if (h > h0) load(h);
        if (tid == 0) r[8] = p.off > 0 ? *scale : 0.0f;         // (read by the thread that writes it)
        // (turned here for the largest, and again for the codes: that is less than holding them in 32 bits)
        auto values = [&](int i, float (&x)[8]) {
            const u32x4 w = halves ? u32x4{perm(raw[i][2], raw[i][0], 0x05040100u), perm(raw[i][2], raw[i][0], 0x07060302u),
                                           perm(raw[i][3], raw[i][1], 0x05040100u), perm(raw[i][3], raw[i][1], 0x07060302u)}
                                   : raw[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = in2f<DT>(w[e] & 0xFFFFu);
                x[2 * e + 1] = in2f<DT>(w[e] >> 16);
                if (!ACROSS && turns && 4 * j + e < a.half)
                    turn_pair(x[2 * e], x[2 * e + 1], cs[ACROSS ? 0 : i][2 * e], cs[ACROSS ? 0 : i][2 * e + 1]);
            }
        };
        uint32_t bits = 0;                      // the largest |x|, as its bits: at least those of infinity if one is no number
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            if (NT * i >= total) break;
            float x[8];
            values(i, x);
            if (t0 + NT / UR * i < p.n)
#pragma unroll
                for (int e = 0; e < 8; ++e) bits = max(bits, __builtin_bit_cast(uint32_t, x[e]) & 0x7FFFFFFFu);
        }
        float top = __builtin_bit_cast(float, bits);
        const bool odd = bits >= 0x7F800000u;
        if (odd) {
            top = 0.0f;
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                if (t0 + NT / UR * i >= p.n) break;
                float x[8];
                values(i, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, size_of(x[e]));
            }
        }
        top = wave_max(top);
        if (lane == 0) r[wave] = top;
        __syncthreads();
        const float old = r[8];
        top = r[0];
#pragma unroll
        for (int i = 1; i < NT / 64; ++i) top = fmaxf(top, r[i]);
        top /= kTop<FMT>;
        const float s = fmaxf(old, top);
        const bool grown = p.off > 0 && s > old;
        const float ratio = old / s;
        if (tid == 0 && (grown || p.off == 0)) *scale = s;
        const Divisor by(s);
        // eight values' codes, the first four and the last in the order a, b, c, d of `order`
        auto pack = [&](const float (&v)[8], int i0, int i1, int i2, int i3) {
            if (by.plain && !odd)
                return pack_numbers<FMT>(by.quotient(v[i0]), by.quotient(v[i1]), by.quotient(v[i2]), by.quotient(v[i3]));
            const auto q = [&](float y) { return s > 0.0f ? y / s : 0.0f; };
            return pack_codes<FMT>(q(v[i0]), q(v[i1]), q(v[i2]), q(v[i3]));
        };

        if constexpr (!ACROSS) {
            if (grown)
                for (int i = tid; i < p.off * D / 16; i += NT) {
                    u32x4 w = reinterpret_cast<u32x4*>(codes)[i];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = requantize<FMT>(w[e], ratio);
                    reinterpret_cast<u32x4*>(codes)[i] = w;
                }
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const int t = t0 + NT / UR * i;
                if (t >= p.n) break;
                uint8_t* row = codes + (p.off + t) * D;
                float x[8];
                values(i, x);
                if (halves) {
                    *reinterpret_cast<uint32_t*>(row + 4 * j) = pack(x, 0, 2, 4, 6);
                    *reinterpret_cast<uint32_t*>(row + a.half + 4 * j) = pack(x, 1, 3, 5, 7);
                } else {
                    const uint32_t w[2] = {pack(x, 0, 1, 2, 3), pack(x, 4, 5, 6, 7)};
                    if (!loose) *reinterpret_cast<u32x2*>(row + 8 * j) = u32x2{w[0], w[1]};
                    else
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int q = 4 * j + e;
                            const bool turn = q < a.half;
                            row[turn ? q : 2 * q] = (uint8_t)(w[e >> 1] >> (16 * (e & 1)));
                            row[turn ? q + a.half : 2 * q + 1] = (uint8_t)(w[e >> 1] >> (16 * (e & 1) + 8));
                        }
                }
            }
        } else {
            // through LDS, so that a dimension's tokens are stored together
            constexpr int pitch = PAGE + 4;
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const int t = t0 + NT / UR * i;
                if (t >= p.n) break;
                float x[8];
                values(i, x);
                const uint32_t w[2] = {pack(x, 0, 1, 2, 3), pack(x, 4, 5, 6, 7)};
#pragma unroll
                for (int e = 0; e < 8; ++e) lds[(8 * j + e) * pitch + p.off + t] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
            }
            __syncthreads();
            // pieces of 16 tokens of a dimension: the earlier tokens' codes (rounded again), the new ones, and what
            // lies behind them as it was
            const int first = grown ? 0 : p.off >> 4, pieces = ((p.off + p.n + 15) >> 4) - first;
            for (int i = tid; i < D * (PAGE / 16); i += NT) {
                const int d = i / (PAGE / 16), piece = i % (PAGE / 16), at = 16 * piece;
                if (piece < first || piece >= first + pieces) continue;
                u32x4* out = reinterpret_cast<u32x4*>(codes + d * PAGE + at);
                u32x4 w = {0, 0, 0, 0}, y;
                if (at >= p.off && at + 16 <= p.off + p.n) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[k] = *reinterpret_cast<const uint32_t*>(lds + d * pitch + at + 4 * k);
                } else {
                    w = *out;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t fresh = *reinterpret_cast<const uint32_t*>(lds + d * pitch + at + 4 * k);
                        const uint32_t again = grown && at + 4 * k < p.off ? requantize<FMT>(w[k], ratio) : w[k];
                        y[k] = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int slot = at + 4 * k + e;
                            const uint32_t from = slot < p.off ? again : slot < p.off + p.n ? fresh : w[k];
                            y[k] |= from & (255u << (8 * e));
                        }
                    }
                }
                *out = y;
            }
        }
    }
}

template <int DT, int FMT, int D, int PAGE>
__global__ __launch_bounds__(append_threads(D, PAGE)) void kv_append_kernel(AppendView a, int blocks, int groups, RopeView q) {
    constexpr int shift = PAGE == 16 ? 4 : PAGE == 32 ? 5 : PAGE == 64 ? 6 : 7;
    __shared__ __attribute__((aligned(16))) uint8_t lds[std::max(D * (PAGE + 4), 8 * kRopePairs * (append_threads(D, PAGE) / 256))];
    __shared__ float red[2][9];
    const int lane = threadIdx.x & 63;
    if ((int)blockIdx.x >= blocks) {            // the queries, a token 256 threads
        constexpr int TOKENS = append_threads(D, PAGE) / 256;
        const int mine = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
        float* cs = reinterpret_cast<float*>(lds) + 2 * kRopePairs * mine;
        const int token = ((int)blockIdx.x - blocks) * TOKENS + mine;
        if (token < q.T) rope_token<DT, 8, 1>(q, token, cs, cs + kRopePairs);
        return;
    }
    const int which = blockIdx.x & 1, group = (blockIdx.x >> 1) % groups, slot = (blockIdx.x >> 1) / groups;
    const int h0 = group * a.c.Hkv / groups, h1 = (group + 1) * a.c.Hkv / groups;
    PageTokens p;
    if (!page_tokens(a.c.lens, a.c.cu, a.c.B, a.c.T, shift, slot, lane, p) || p.index < 0) return;
    if (which) append_page<DT, FMT, D, PAGE, true>(a, p, h0, h1, lds, red);
    else append_page<DT, FMT, D, PAGE, false>(a, p, h0, h1, lds, red);
}

// A decode step: one token a sequence, a wave (sequence, head) of K or V, a lane a pair (or two adjacent values).
template <int DT, int FMT, int D>
__global__ __launch_bounds__(256, 8) void kv_append_step_kernel(AppendView a, int shift, int blocks, RopeView q) {
    __shared__ __attribute__((aligned(16))) float cs[2 * kRopePairs];
    const int tid = threadIdx.x, lane = tid & 63;
    if ((int)blockIdx.x >= blocks) {            // the queries
        rope_token<DT, 8, 1>(q, (int)blockIdx.x - blocks, cs, cs + kRopePairs);
        return;
    }
    const int item = 4 * blockIdx.x + __builtin_amdgcn_readfirstlane(tid >> 6);
    const int which = item & 1, h = (item >> 1) % a.c.Hkv, b = (item >> 1) / a.c.Hkv;
    if (b >= a.c.B) return;
    const int page = 1 << shift;
    const uint16_t* row = (which ? a.v + (long long)b * a.vs : a.k + (long long)b * a.ks) + h * D;
    const bool mine = lane < D / 2, turn = !which && lane < a.half;
    const int e0 = turn && !a.inter ? lane : 2 * lane, e1 = turn && !a.inter ? lane + a.half : 2 * lane + 1;
    float x0 = 0.0f, x1 = 0.0f;
    if (mine) {
        x0 = in2f<DT>(row[e0]);
        x1 = in2f<DT>(row[e1]);
    }
    const long long f = turn ? a.freqs[lane] : 0;
    const int place = a.c.lens[b] - 1;
    if (place < 0) return;
    const int id = page_id(a.c.table, a.c.P, a.c.N, b, place >> shift), off = place & (page - 1);
    if (id < 0) return;
    uint8_t* codes = (uint8_t*)(which ? a.c.vc : a.c.kc) + (((long long)id * a.c.Hkv + h) << shift) * D;
    float* scale = (which ? a.c.vs : a.c.ks) + (long long)id * a.c.Hkv + h;
    const float old = off > 0 ? *scale : 0.0f;
    if (turn) {
        float c, s;
        position_cos_sin(a.positions ? a.positions[b] : place, f, a.m, c, s);
        turn_pair(x0, x1, c, s);
    }
    const float top = wave_max(fmaxf(size_of(x0), size_of(x1))) / kTop<FMT>;
    const float s = fmaxf(old, top);
    if (off > 0 && s > old) {
        // earlier codes: of K the first off D bytes, of V the first off of every dimension's
        const float ratio = old / s;
        const int per = which ? (off + 15) >> 4 : D / 16, lines = which ? D : off;
        for (int i = lane; i < lines * per; i += 64) {
            u32x4* at = reinterpret_cast<u32x4*>(codes + (i / per) * (which ? page : D) + 16 * (i % per));
            u32x4 w = *at;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // (slots from the new one on are as they were: the new code is written below)
                const int keep = which ? min(max(off - 16 * (i % per) - 4 * k, 0), 4) : 4;
                const uint32_t mask = keep == 4 ? ~0u : (1u << (8 * keep)) - 1u;
                w[k] = (requantize<FMT>(w[k], ratio) & mask) | (w[k] & ~mask);
            }
            *at = w;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // (before other lanes' bytes of the same words)
    }
    if (lane == 0 && (off == 0 || s > old)) *scale = s;
    if (mine) {
        const uint32_t w = pack_codes<FMT>(s > 0.0f ? x0 / s : 0.0f, s > 0.0f ? x1 / s : 0.0f, 0.0f, 0.0f);
        codes[which ? e0 * page + off : off * D + e0] = (uint8_t)w;
        codes[which ? e1 * page + off : off * D + e1] = (uint8_t)(w >> 8);
    }
}

// ---------------------------------------------------------------- read

template <int FMT, int DT>
__device__ __forceinline__ uint32_t two_values(uint32_t w, int byte, float s) {
    return pack2<DT>(code_value<FMT>(w, byte) * s, code_value<FMT>(w, byte + 1) * s);
}

// One (page, head) of K and V as 16-bit rows; tokens without a page are zeros.  V's codes go through LDS, four
// dimensions by four tokens turned round in registers.  Bound by memory: 50300 tokens of 8 heads, D = 128 (309 MB),
// take 63 us, 4.9 TB/s (65.6 with the codes kept in the caches; the rows past the caches too: 59, but with the attention
// over 60000 rows behind it 208 against 200).
template <int DT, int FMT, int D, int PAGE>
__global__ __launch_bounds__(256) void kv_read_kernel(KvPages c, uint16_t* __restrict__ kout, uint16_t* __restrict__ vout) {
    constexpr int shift = PAGE == 16 ? 4 : PAGE == 32 ? 5 : PAGE == 64 ? 6 : 7, UR = D / 8;
    constexpr int NK = PAGE * UR > 256 ? PAGE * UR / 256 : 1, NV = PAGE * D > 4096 ? PAGE * D / 4096 : 1;
    constexpr int pitch = PAGE + 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[D * pitch];
    const int tid = threadIdx.x, lane = tid & 63;
    const int h = blockIdx.x % c.Hkv, slot = blockIdx.x / c.Hkv;
    PageTokens p;
    if (!page_tokens(c.lens, c.cu, c.B, c.T, shift, slot, lane, p)) return;
    const int id = page_id(c.table, c.P, c.N, p.b, p.index);
    const long long os = (long long)c.Hkv * D;
    uint16_t *ko = kout + p.token * os + h * D, *vo = vout + p.token * os + h * D;
    if (id < 0) {
        for (int u = tid; u < p.n * UR; u += 256) {
            *reinterpret_cast<u32x4*>(ko + (u / UR) * os + 8 * (u % UR)) = u32x4{0, 0, 0, 0};
            *reinterpret_cast<u32x4*>(vo + (u / UR) * os + 8 * (u % UR)) = u32x4{0, 0, 0, 0};
        }
        return;
    }
    const long long at = (long long)id * c.Hkv + h;
    const uint8_t *kc = (const uint8_t*)c.kc + at * (PAGE * D), *vc = (const uint8_t*)c.vc + at * (PAGE * D);
    const float ks = c.ks[at], vs = c.vs[at];
    u32x4 vw[NV];
    u32x2 kw[NK];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = tid + 256 * i, t = 16 * (u % (PAGE / 16));
        if (u < D * (PAGE / 16) && t + 16 > p.off && t < p.off + p.n) vw[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(vc + 16 * u));
    }
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int u = tid + 256 * i;
        if (u < p.n * UR) kw[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(kc + p.off * D + 8 * u));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = tid + 256 * i, d = u / (PAGE / 16), t = 16 * (u % (PAGE / 16));
        if (u < D * (PAGE / 16))
#pragma unroll
            for (int k = 0; k < 4; ++k) *reinterpret_cast<uint32_t*>(lds + d * pitch + t + 4 * k) = vw[i][k];
    }
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int u = tid + 256 * i;
        if (u < p.n * UR)
            *reinterpret_cast<u32x4*>(ko + (u / UR) * os + 8 * (u % UR)) =
                u32x4{two_values<FMT, DT>(kw[i][0], 0, ks), two_values<FMT, DT>(kw[i][0], 2, ks),
                      two_values<FMT, DT>(kw[i][1], 0, ks), two_values<FMT, DT>(kw[i][1], 2, ks)};
    }
    __syncthreads();
    // units of four tokens of eight dimensions
    for (int u = tid; u < (PAGE / 4) * UR; u += 256) {
        const int t4 = 4 * (u / UR), j = u % UR;
        if (t4 + 4 <= p.off || t4 >= p.off + p.n) continue;
        u32x4 lo, hi;                           // four tokens' codes of the first and of the last four dimensions
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint32_t*>(lds + (8 * j + 4 * k + e) * pitch + t4);
            const uint32_t a0 = perm(w[1], w[0], 0x05010400u), a1 = perm(w[1], w[0], 0x07030602u);
            const uint32_t b0 = perm(w[3], w[2], 0x05010400u), b1 = perm(w[3], w[2], 0x07030602u);
            (k ? hi : lo) = u32x4{perm(b0, a0, 0x05040100u), perm(b0, a0, 0x07060302u), perm(b1, a1, 0x05040100u),
                                  perm(b1, a1, 0x07060302u)};
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = t4 + e - p.off;
            if (t >= 0 && t < p.n)
                *reinterpret_cast<u32x4*>(vo + t * os + 8 * j) =
                    u32x4{two_values<FMT, DT>(lo[e], 0, vs), two_values<FMT, DT>(lo[e], 2, vs),
                          two_values<FMT, DT>(hi[e], 0, vs), two_values<FMT, DT>(hi[e], 2, vs)};
        }
    }
}

int shift_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }
// (page, group of heads, cache) blocks aimed at: 1024, and twice that of pages of 16, whose blocks have half the work.
// 512 / 1024 / 2048 / 4096, us: 12 prompts of 200 tokens, 32 heads of K, V and queries, D = 128, pages of 32
// 41 / 29 / 30 / 34, of 64 30 / 33 / 37 / 45, of 16 68 / 44 / 36 / 37; 8192 tokens, 32 / 8 heads, pages of 64 44 / 46 / 52 / 54.
constexpr unsigned kAppendBlocks = 1024;
// pages that a call may touch
unsigned page_slots(const KvPages& c) { return (unsigned)(c.cu ? (c.T >> shift_of(c.page)) + 2 * c.B : c.B); }

template <int DT, int FMT, int D>
hipError_t append(const AppendView& a, const RopeView& q, unsigned more, hipStream_t st) {
    const int page = a.c.page;
    if (!a.c.cu) {
        const unsigned blocks = ((unsigned)a.c.B * a.c.Hkv * 2 + 3) / 4;
        hipLaunchKernelGGL((kv_append_step_kernel<DT, FMT, D>), dim3(blocks + more), dim3(256), 0, st, a, shift_of(page),
                           (int)blocks, q);
        return hipGetLastError();
    }
    // heads in groups, as many as fill the GPU
    const unsigned slots = page_slots(a.c);
    const int groups = (int)std::min<unsigned>(a.c.Hkv, std::max(1u, kAppendBlocks * (page == 16 ? 2 : 1) / (2 * slots)));
    const unsigned blocks = slots * groups * 2;
#define W4A16_APPEND(PAGE) \
    hipLaunchKernelGGL((kv_append_kernel<DT, FMT, D, PAGE>), dim3(blocks + (append_threads(D, PAGE) == 512 ? (more + 1) / 2 : more)), \
                       dim3(append_threads(D, PAGE)), 0, st, a, (int)blocks, groups, q)
    if (page == 16) W4A16_APPEND(16);
    else if (page == 32) W4A16_APPEND(32);
    else if (page == 64) W4A16_APPEND(64);
    else W4A16_APPEND(128);
#undef W4A16_APPEND
    return hipGetLastError();
}

template <int DT, int FMT, int D>
hipError_t read(const KvPages& c, uint16_t* ko, uint16_t* vo, hipStream_t st) {
    const dim3 grid(page_slots(c) * c.Hkv), block(256);
    if (c.page == 16) hipLaunchKernelGGL((kv_read_kernel<DT, FMT, D, 16>), grid, block, 0, st, c, ko, vo);
    else if (c.page == 32) hipLaunchKernelGGL((kv_read_kernel<DT, FMT, D, 32>), grid, block, 0, st, c, ko, vo);
    else if (c.page == 64) hipLaunchKernelGGL((kv_read_kernel<DT, FMT, D, 64>), grid, block, 0, st, c, ko, vo);
    else hipLaunchKernelGGL((kv_read_kernel<DT, FMT, D, 128>), grid, block, 0, st, c, ko, vo);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t st) {
    RopeView r = {};
    r.x = static_cast<const uint16_t*>(a.x);
    r.out = static_cast<uint16_t*>(a.out);
    r.freqs = a.freqs;
    r.at.positions = a.positions;
    r.m = a.m;
    r.xs = a.xs;
    r.os = a.os;
    r.T = a.T;
    r.H = a.H;
    r.D = a.D;
    r.half = a.R / 2;
    r.inter = a.inter;
    r.copy = a.x != a.out;
    return rope(r, a.dtype, st);
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t st) {
    AppendView v = {};
    v.c = a.c;
    v.k = static_cast<const uint16_t*>(a.k);
    v.v = static_cast<const uint16_t*>(a.v);
    v.freqs = a.freqs;
    v.positions = a.positions;
    v.m = a.m;
    v.ks = a.ks;
    v.vs = a.vs;
    v.half = a.R / 2;
    v.inter = a.inter;
    RopeView r = {};
    unsigned more = 0;
    if (a.q) {
        r.x = static_cast<const uint16_t*>(a.q);
        r.out = static_cast<uint16_t*>(a.q_out);
        r.freqs = a.freqs;
        r.at = {a.positions, a.c.lens, a.c.cu, a.c.B, a.c.T};
        r.m = a.m;
        r.xs = a.qs;
        r.os = a.Hq * a.c.D;
        r.T = a.c.T;
        r.H = a.Hq;
        r.D = a.c.D;
        r.half = v.half;
        r.inter = a.inter;
        r.copy = 1;
        if (rope_wide(r)) {
            more = (unsigned)r.T;
        } else {
            const hipError_t e = rope(r, a.dtype, st);
            if (e != hipSuccess) return e;
        }
    }
#define W4A16_APPEND(DT, FMT) \
    (a.c.D == 64 ? append<DT, FMT, 64>(v, r, more, st) : append<DT, FMT, 128>(v, r, more, st))
    if (a.dtype == DT_F16) return a.c.fmt == FMT_INT8 ? W4A16_APPEND(DT_F16, FMT_INT8) : W4A16_APPEND(DT_F16, FMT_E4M3);
    return a.c.fmt == FMT_INT8 ? W4A16_APPEND(DT_BF16, FMT_INT8) : W4A16_APPEND(DT_BF16, FMT_E4M3);
#undef W4A16_APPEND
}

hipError_t launch_kv_read(const KvPages& c, int dtype, void* kout, void* vout, hipStream_t st) {
    uint16_t *ko = static_cast<uint16_t*>(kout), *vo = static_cast<uint16_t*>(vout);
#define W4A16_READ(DT, FMT) (c.D == 64 ? read<DT, FMT, 64>(c, ko, vo, st) : read<DT, FMT, 128>(c, ko, vo, st))
    if (dtype == DT_F16) return c.fmt == FMT_INT8 ? W4A16_READ(DT_F16, FMT_INT8) : W4A16_READ(DT_F16, FMT_E4M3);
    return c.fmt == FMT_INT8 ? W4A16_READ(DT_BF16, FMT_INT8) : W4A16_READ(DT_BF16, FMT_E4M3);
#undef W4A16_READ
}

}  // namespace w4a16
