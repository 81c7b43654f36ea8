// Rotary positions, appending to a paged 8-bit KV cache and reading it back.
//
// Rotation of a pair (x0, x1) of a head by its token's position: with a = position * f,
//   y0 = m (x0 cos a - x1 sin a),   y1 = m (x1 cos a + x0 sin a),
// pairs (i, i + R / 2) or (2 i, 2 i + 1) of the head's first R values; the rest passes through.
//
// Append: a page's scale is the largest |x| / top of the tokens written to it since its first, so it grows
// as the page fills; codes are rint(x / s) (or the nearest e4m3), those already there are rounded again where
// s has grown.  One block a (page, head) and cache: rows into registers, rotated there in fp32, their
// largest value, the scale, the codes.
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

constexpr int kRopePairs = 1024;        // (token, pair) angles of a block
constexpr int kRopeTokens = 4;          // tokens of a block at most

// Tokens t0 .. t0 + tb - 1 by one block: their angles' cos and sin once into LDS, then all heads, V pairs
// a thread at a time.
template <int DT, int V>
__device__ __forceinline__ void rope_block(const RopeView& r, int t0, int tb, float* lc, float* ls, int2* lp) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    tb = min(tb, r.T - t0);
    for (int i = wave; i < tb; i += 4) {
        int p = 0;
        const bool found = place_of(r.at, t0 + i, lane, p);
        if (lane == 0) lp[i] = make_int2(p, found);
    }
    __syncthreads();
    for (int i = tid; i < tb * r.half; i += 256) {
        const int t = i / r.half;
        position_cos_sin(lp[t].x, r.freqs[i - t * r.half], r.m, lc[i], ls[i]);
    }
    __syncthreads();
    constexpr int CP = V == 8 ? 8 : 2;                  // values of a copying step
    const int turns = r.half / V, units = turns + (r.copy ? (r.D - 2 * r.half) / CP : 0);
    const int rows = 256 / units, unit = tid % units, row = tid / units;
    if (row >= rows) return;
    int t = row / r.H, h = row - t * r.H;
    const uint16_t* x = r.x + (long long)t0 * r.xs;
    uint16_t* out = r.out + (long long)t0 * r.os;
    while (t < tb) {
        const uint16_t* px = x + (long long)t * r.xs + h * r.D;
        uint16_t* po = out + (long long)t * r.os + h * r.D;
        if (!lp[t].y) {
        } else if (unit < turns) {
            const int p = unit * V, a = r.inter ? 2 * p : p, b = r.inter ? 2 * p + V : p + r.half;
            const float *c = lc + t * r.half + p, *s = ls + t * r.half + p;
            if constexpr (V == 8) {
                const u32x4 lo = *reinterpret_cast<const u32x4*>(px + a), hi = *reinterpret_cast<const u32x4*>(px + b);
                u32x4 ylo, yhi;
                if (r.inter) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t w = i < 4 ? lo[i] : hi[i - 4];
                        const float x0 = in2f<DT>(w & 0xFFFFu), x1 = in2f<DT>(w >> 16);
                        const uint32_t y = pack2<DT>(x0 * c[i] - x1 * s[i], x1 * c[i] + x0 * s[i]);
                        if (i < 4) ylo[i] = y;
                        else yhi[i - 4] = y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float c0 = c[2 * i], s0 = s[2 * i], c1 = c[2 * i + 1], s1 = s[2 * i + 1];
                        const float a0 = in2f<DT>(lo[i] & 0xFFFFu), a1 = in2f<DT>(lo[i] >> 16);
                        const float b0 = in2f<DT>(hi[i] & 0xFFFFu), b1 = in2f<DT>(hi[i] >> 16);
                        ylo[i] = pack2<DT>(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
                        yhi[i] = pack2<DT>(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
                    }
                }
                *reinterpret_cast<u32x4*>(po + a) = ylo;
                *reinterpret_cast<u32x4*>(po + b) = yhi;
            } else {
                const float x0 = in2f<DT>(px[a]), x1 = in2f<DT>(px[b]);
                po[a] = f2out<DT>(x0 * c[0] - x1 * s[0]);
                po[b] = f2out<DT>(x1 * c[0] + x0 * s[0]);
            }
        } else {
            const int e = 2 * r.half + (unit - turns) * CP;
            if constexpr (V == 8) *reinterpret_cast<u32x4*>(po + e) = *reinterpret_cast<const u32x4*>(px + e);
            else {
                const uint16_t e0 = px[e], e1 = px[e + 1];
                po[e] = e0;
                po[e + 1] = e1;
            }
        }
        h += rows;
        while (h >= r.H) {
            h -= r.H;
            ++t;
        }
    }
}

template <int DT, int V>
__global__ __launch_bounds__(256) void rope_kernel(RopeView r, int tb) {
    __shared__ __attribute__((aligned(16))) float lc[kRopePairs], ls[kRopePairs];
    __shared__ int2 lp[kRopeTokens];
    rope_block<DT, V>(r, blockIdx.x * tb, tb, lc, ls, lp);
}

bool rope_wide(const RopeView& r) {
    const auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    return r.half % 8 == 0 && r.D % 8 == 0 && r.xs % 8 == 0 && r.os % 8 == 0 && at16(r.x) && at16(r.out);
}
// Tokens of a block.
int rope_tokens(const RopeView& r) { return std::max(1, std::min({kRopeTokens, kRopePairs / std::max(1, r.half), r.T / 1024})); }

hipError_t rope(const RopeView& r, int dtype, hipStream_t st) {
    const int tb = rope_tokens(r);
    const dim3 grid((unsigned)((r.T + tb - 1) / tb)), block(256);
    if (rope_wide(r)) {
        if (dtype == DT_F16) hipLaunchKernelGGL((rope_kernel<DT_F16, 8>), grid, block, 0, st, r, tb);
        else hipLaunchKernelGGL((rope_kernel<DT_BF16, 8>), grid, block, 0, st, r, tb);
    } else {
        if (dtype == DT_F16) hipLaunchKernelGGL((rope_kernel<DT_F16, 1>), grid, block, 0, st, r, tb);
        else hipLaunchKernelGGL((rope_kernel<DT_BF16, 1>), grid, block, 0, st, r, tb);
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

// One (page, head) of K (ACROSS false: rows, rotated) or V (columns).  Thread units of eight values: of K four
// pairs (p .. p + 3 of the rotation, or eight adjacent ones behind it), of V eight adjacent ones.
template <int DT, int FMT, int D, bool ACROSS>
__device__ __forceinline__ void append_page(const AppendView& a, const PageTokens& p, int id, int h, int shift,
                                            uint8_t* lds, float* red) {
    constexpr int UR = D / 8, UNITS = 128 * UR / 256;       // units of a row; of a thread at most
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int page = 1 << shift, total = p.n * UR;
    uint8_t* codes = (uint8_t*)(ACROSS ? a.c.vc : a.c.kc) + (((long long)id * a.c.Hkv + h) << shift) * D;
    float* scale = (ACROSS ? a.c.vs : a.c.ks) + (long long)id * a.c.Hkv + h;
    const uint16_t* src = (ACROSS ? a.v : a.k) + h * D;
    const int stride = ACROSS ? a.vs : a.ks;

    float x[UNITS][8];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int u = tid + 256 * i;
        if (256 * i >= total) break;
        if (u < total) {
            const int t = u / UR, j = u % UR;
            const uint16_t* row = src + (long long)(p.token + t) * stride;
            if (ACROSS || 4 * j >= a.half) {
                // (a rotation that ends inside the unit: pair by pair below)
                const u32x4 w = *reinterpret_cast<const u32x4*>(row + 8 * j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[i][2 * e] = in2f<DT>(w[e] & 0xFFFFu);
                    x[i][2 * e + 1] = in2f<DT>(w[e] >> 16);
                }
            } else {
                const int position = a.positions ? a.positions[p.token + t] : (p.index << shift) + p.off + t;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int q = 4 * j + e;
                    const bool turn = q < a.half;
                    const int e0 = a.inter || !turn ? 2 * q : q, e1 = a.inter || !turn ? 2 * q + 1 : q + a.half;
                    const float x0 = in2f<DT>(row[e0]), x1 = in2f<DT>(row[e1]);
                    float c = 1.0f, s = 0.0f;
                    if (turn) position_cos_sin(position, a.freqs[q], a.m, c, s);
                    x[i][2 * e] = x0 * c - x1 * s;
                    x[i][2 * e + 1] = x1 * c + x0 * s;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, size_of(x[i][e]));
        }
    }
    top = wave_max(top);
    if (lane == 0) red[wave] = top;
    if (tid == 0) red[4] = p.off > 0 ? *scale : 0.0f;      // (read by the thread that writes it)
    __syncthreads();
    const float old = red[4];
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])) / kTop<FMT>;
    const float s = fmaxf(old, top);
    const bool grown = p.off > 0 && s > old;
    const float ratio = old / s;
    if (tid == 0 && (grown || p.off == 0)) *scale = s;
    auto quotient = [&](float v) { return s > 0.0f ? v / s : 0.0f; };

    if constexpr (!ACROSS) {
        if (grown)
            for (int i = tid; i < p.off * D / 16; i += 256) {
                u32x4 w = reinterpret_cast<u32x4*>(codes)[i];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = requantize<FMT>(w[e], ratio);
                reinterpret_cast<u32x4*>(codes)[i] = w;
            }
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const int u = tid + 256 * i;
            if (u >= total) break;
            const int t = u / UR, j = u % UR;
            uint8_t* row = codes + (p.off + t) * D;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = quotient(x[i][e]);
            if (4 * j + 4 <= a.half && !a.inter) {
                const uint32_t lo = pack_codes<FMT>(y[0], y[2], y[4], y[6]), hi = pack_codes<FMT>(y[1], y[3], y[5], y[7]);
                *reinterpret_cast<uint32_t*>(row + 4 * j) = lo;
                if (a.half % 4 == 0) *reinterpret_cast<uint32_t*>(row + a.half + 4 * j) = hi;
                else
#pragma unroll
                    for (int e = 0; e < 4; ++e) row[a.half + 4 * j + e] = (uint8_t)(hi >> (8 * e));
            } else {
                const uint32_t w[2] = {pack_codes<FMT>(y[0], y[1], y[2], y[3]), pack_codes<FMT>(y[4], y[5], y[6], y[7])};
                if (a.inter || 4 * j >= a.half) *reinterpret_cast<u32x2*>(row + 8 * j) = u32x2{w[0], w[1]};
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
        const int pitch = page + 4;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const int u = tid + 256 * i;
            if (u >= total) break;
            const int t = u / UR, j = u % UR;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = quotient(x[i][e]);
            const uint32_t w[2] = {pack_codes<FMT>(y[0], y[1], y[2], y[3]), pack_codes<FMT>(y[4], y[5], y[6], y[7])};
#pragma unroll
            for (int e = 0; e < 8; ++e) lds[(8 * j + e) * pitch + p.off + t] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
        }
        __syncthreads();
        // pieces of 16 tokens of a dimension: the earlier tokens' codes (rounded again), the new ones, and what
        // lies behind them as it was
        const int first = grown ? 0 : p.off >> 4, pieces = ((p.off + p.n + 15) >> 4) - first;
        for (int i = tid; i < D * pieces; i += 256) {
            const int d = i / pieces, piece = first + i % pieces, t0 = 16 * piece;
            u32x4* at = reinterpret_cast<u32x4*>(codes + d * page + t0);
            u32x4 w = {0, 0, 0, 0};
            const bool whole = t0 >= p.off && t0 + 16 <= p.off + p.n;
            if (!whole) w = *at;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t fresh = *reinterpret_cast<const uint32_t*>(lds + d * pitch + t0 + 4 * j);
                const uint32_t again = grown && t0 + 4 * j < p.off ? requantize<FMT>(w[j], ratio) : w[j];
                uint32_t y = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int slot = t0 + 4 * j + e;
                    const uint32_t from = slot < p.off ? again : slot < p.off + p.n ? fresh : w[j];
                    y |= from & (255u << (8 * e));
                }
                w[j] = y;
            }
            *at = w;
        }
    }
}

template <int DT, int FMT, int D>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendView a, int shift, int blocks, RopeView q, int tb) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[std::max(D * 132, 8 * kRopePairs)];
    __shared__ float red[5];
    __shared__ int2 lp[kRopeTokens];
    const int lane = threadIdx.x & 63;
    if ((int)blockIdx.x >= blocks) {            // the queries
        float* cs = reinterpret_cast<float*>(lds);
        rope_block<DT, 8>(q, ((int)blockIdx.x - blocks) * tb, tb, cs, cs + kRopePairs, lp);
        return;
    }
    const int which = blockIdx.x & 1, h = (blockIdx.x >> 1) % a.c.Hkv, slot = (blockIdx.x >> 1) / a.c.Hkv;
    PageTokens p;
    if (!page_tokens(a.c.lens, a.c.cu, a.c.B, a.c.T, shift, slot, lane, p)) return;
    const int id = page_id(a.c.table, a.c.P, a.c.N, p.b, p.index);
    if (id < 0) return;
    if (which) append_page<DT, FMT, D, true>(a, p, id, h, shift, lds, red);
    else append_page<DT, FMT, D, false>(a, p, id, h, shift, lds, red);
}

// ---------------------------------------------------------------- read

template <int FMT, int DT>
__device__ __forceinline__ uint32_t two_values(uint32_t w, int byte, float s) {
    return pack2<DT>(code_value<FMT>(w, byte) * s, code_value<FMT>(w, byte + 1) * s);
}

// One (page, head) of K or V as 16-bit rows; tokens without a page are zeros.
template <int DT, int FMT, int D>
__global__ __launch_bounds__(256) void kv_read_kernel(KvPages c, int shift, uint16_t* __restrict__ kout,
                                                      uint16_t* __restrict__ vout) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[D * 132];
    const int tid = threadIdx.x, lane = tid & 63;
    const int across = blockIdx.x & 1, h = (blockIdx.x >> 1) % c.Hkv, slot = (blockIdx.x >> 1) / c.Hkv;
    PageTokens p;
    if (!page_tokens(c.lens, c.cu, c.B, c.T, shift, slot, lane, p)) return;
    const int id = page_id(c.table, c.P, c.N, p.b, p.index), page = 1 << shift;
    uint16_t* out = (across ? vout : kout) + ((long long)p.token * c.Hkv + h) * D;
    const long long os = (long long)c.Hkv * D;
    constexpr int UR = D / 8;
    if (id < 0) {
        for (int u = tid; u < p.n * UR; u += 256)
            *reinterpret_cast<u32x4*>(out + (u / UR) * os + 8 * (u % UR)) = u32x4{0, 0, 0, 0};
        return;
    }
    const uint8_t* codes = (const uint8_t*)(across ? c.vc : c.kc) + (((long long)id * c.Hkv + h) << shift) * D;
    const float s = (across ? c.vs : c.ks)[(long long)id * c.Hkv + h];
    if (!across) {
        for (int u = tid; u < p.n * UR; u += 256) {
            const int t = u / UR, j = u % UR;
            const u32x2 w = *reinterpret_cast<const u32x2*>(codes + (p.off + t) * D + 8 * j);
            *reinterpret_cast<u32x4*>(out + t * os + 8 * j) =
                u32x4{two_values<FMT, DT>(w[0], 0, s), two_values<FMT, DT>(w[0], 2, s), two_values<FMT, DT>(w[1], 0, s),
                      two_values<FMT, DT>(w[1], 2, s)};
        }
        return;
    }
    const int pitch = page + 4, first = p.off >> 4, pieces = ((p.off + p.n + 15) >> 4) - first;
    for (int i = tid; i < D * pieces; i += 256) {
        const int d = i / pieces, t0 = 16 * (first + i % pieces);
        const u32x4 w = *reinterpret_cast<const u32x4*>(codes + d * page + t0);
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(lds + d * pitch + t0 + 4 * j) = w[j];
    }
    __syncthreads();
    for (int u = tid; u < p.n * UR; u += 256) {
        const int t = u / UR, j = u % UR;
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e >> 2] |= (uint32_t)lds[(8 * j + e) * pitch + p.off + t] << (8 * (e & 3));
        *reinterpret_cast<u32x4*>(out + t * os + 8 * j) =
            u32x4{two_values<FMT, DT>(w[0], 0, s), two_values<FMT, DT>(w[0], 2, s), two_values<FMT, DT>(w[1], 0, s),
                  two_values<FMT, DT>(w[1], 2, s)};
    }
}

int shift_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }
// (page, head) blocks of K and of V
unsigned page_blocks(const KvPages& c) {
    return (unsigned)((c.cu ? (c.T >> shift_of(c.page)) + 2 * c.B : c.B) * c.Hkv) * 2u;
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
    const int shift = shift_of(a.c.page);
    RopeView r = {};
    int tb = 1;
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
        tb = rope_tokens(r);
        more = (unsigned)((r.T + tb - 1) / tb);
        if (!rope_wide(r)) {
            const hipError_t e = rope(r, a.dtype, st);
            if (e != hipSuccess) return e;
            more = 0;
        }
    }
    const unsigned blocks = page_blocks(a.c);
#define W4A16_APPEND(DT, FMT, D)                                                                                       \
    hipLaunchKernelGGL((kv_append_kernel<DT, FMT, D>), dim3(blocks + more), dim3(256), 0, st, v, shift, (int)blocks, r, tb)
#define W4A16_APPEND_D(DT, FMT) \
    if (a.c.D == 64) W4A16_APPEND(DT, FMT, 64); \
    else W4A16_APPEND(DT, FMT, 128)
    if (a.dtype == DT_F16) {
        if (a.c.fmt == FMT_INT8) { W4A16_APPEND_D(DT_F16, FMT_INT8); }
        else { W4A16_APPEND_D(DT_F16, FMT_E4M3); }
    } else {
        if (a.c.fmt == FMT_INT8) { W4A16_APPEND_D(DT_BF16, FMT_INT8); }
        else { W4A16_APPEND_D(DT_BF16, FMT_E4M3); }
    }
#undef W4A16_APPEND_D
#undef W4A16_APPEND
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvPages& c, int dtype, void* kout, void* vout, hipStream_t st) {
    const int shift = shift_of(c.page);
    uint16_t *ko = static_cast<uint16_t*>(kout), *vo = static_cast<uint16_t*>(vout);
#define W4A16_READ(DT, FMT, D) \
    hipLaunchKernelGGL((kv_read_kernel<DT, FMT, D>), dim3(page_blocks(c)), dim3(256), 0, st, c, shift, ko, vo)
#define W4A16_READ_D(DT, FMT) \
    if (c.D == 64) W4A16_READ(DT, FMT, 64); \
    else W4A16_READ(DT, FMT, 128)
    if (dtype == DT_F16) {
        if (c.fmt == FMT_INT8) { W4A16_READ_D(DT_F16, FMT_INT8); }
        else { W4A16_READ_D(DT_F16, FMT_E4M3); }
    } else {
        if (c.fmt == FMT_INT8) { W4A16_READ_D(DT_BF16, FMT_INT8); }
        else { W4A16_READ_D(DT_BF16, FMT_E4M3); }
    }
#undef W4A16_READ_D
#undef W4A16_READ
    return hipGetLastError();
}

}  // namespace w4a16
