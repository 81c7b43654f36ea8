// Causal attention of the sequences' last tokens over a paged 8-bit KV cache.
//
//   out[i, h] = softmax_j(q_i . k_j / sqrt(D)) v_j over the tokens j of i's sequence up to its own,
//   k_j = s_p c_j,  v_j = s'_p c'_j  (p: the page of j, one scale each for K and V and kv head)
//
// Query rows of a sequence and kv head are its new tokens times the G = Hq / Hkv heads that share the kv
// head, token by token; a tile is 16 of them.  A wave takes 64 cached tokens at a time, straight from
// memory into the operands of 16 x 16 x 32 matrix instructions, both products transposed:
//   S^T[token, row] = K Q^T,    O^T[d, row] = V^T P^T.
// The tokens of K's four 16-token operands are taken in the order 16 (m / 4) + 4 j + m % 4 (operand j,
// its row m), so that the results leave lane l with tokens 16 (l / 16) .. + 15 of row l % 16: one page's (no
// page is shorter), as 16 consecutive codes of a dimension are in the pool and as the second product's
// operand wants them.  Nothing passes through LDS until the waves are joined.
//
// Codes are exact in fp16 (values) and in the queries' type (keys); the scales stay out of the operands: K's
// multiplies the scores, V's the weights, which are held times 2^15 over the largest scale's power of two
// and rounded once to fp16 (relative 2^-11 down to 2^-29 of a row's largest).  Scores, maxima, sums and outputs are fp32.
#include <algorithm>

#include "pages.h"

namespace w4a16 {

namespace {

constexpr int kTile = 64;               // tokens of a wave's step
constexpr int kRowTile = 16;            // query rows of a block
constexpr int kWaves = 4;
constexpr int kWhole = 16;              // up to so many tiles a sequence is never split
constexpr int kLeast = 4;               // tiles of a chunk of a longer one
constexpr int kTargetBlocks = 1024;     // chunks x kv heads aimed at

template <int DT>
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
    if constexpr (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}

// Eight codes (two words) as 16-bit floats, exact.  int8 to fp16: the byte + 128 under the exponent of 1024 is
// 1152 + c, less 1152; to bf16 by way of fp32, whose upper half holds them.
template <int DT, int FMT>
__device__ __forceinline__ u32x4 widen(uint32_t w0, uint32_t w1) {
    u32x4 r;
    if constexpr (FMT == FMT_E4M3) {
        if constexpr (DT == DT_F16) {
            r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, false));
            r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, true));
            r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, false));
            r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, true));
        } else {
            r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false));
            r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true));
            r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false));
            r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true));
        }
    } else if constexpr (DT == DT_F16) {
        const uint32_t w[2] = {w0 ^ 0x80808080u, w1 ^ 0x80808080u};
        const f16x2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = perm(0x64646464u, w[i >> 1], i & 1 ? 0x04030402u : 0x04010400u);
            r[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, x) - bias);
        }
    } else {
        const uint32_t w[2] = {w0, w1};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = code_value<FMT>(w[i >> 1], 2 * (i & 1)), hi = code_value<FMT>(w[i >> 1], 2 * (i & 1) + 1);
            r[i] = perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
        }
    }
    return r;
}

// A value of lanes l % 16 + 0, 16, 32, 48 combined in all four.
__device__ __forceinline__ float max_groups(float x) {
    x = max_halves(x);
    const int i = __builtin_bit_cast(int, x);
    const auto r = __builtin_amdgcn_permlane16_swap(i, i, false, false);
    const int a = r[0], b = r[1];
    return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float sum_groups(float x) {
    x = sum_halves(x);
    const int i = __builtin_bit_cast(int, x);
    const auto r = __builtin_amdgcn_permlane16_swap(i, i, false, false);
    const int a = r[0], b = r[1];
    return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}

__device__ __forceinline__ bool any_lane(bool p) { return __builtin_amdgcn_ballot_w64(p) != 0; }
__device__ __forceinline__ int lanes_sum(int v) {
    v += __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);      // quad_perm [1,0,3,2]
    v += __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);      // quad_perm [2,3,0,1]
    v += __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);     // row_half_mirror
    v += __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);     // row_mirror
    return (__builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16)) +
           (__builtin_amdgcn_readlane(v, 32) + __builtin_amdgcn_readlane(v, 48));
}
__device__ __forceinline__ int wave_scan(int v, int lane) {     // inclusive
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __builtin_amdgcn_ds_bpermute(4 * (lane - d), v);
        if (lane >= d) v += o;
    }
    return v;
}

// What a block works on: 16 rows from `row0` of sequence b, its tiles [tile0, tile1), and where the outcome
// goes: chunk `part` of `parts` in the workspace from `slot`, or straight out if there is one.
struct Piece {
    int b, first, n, len, row0, tile0, tile1, part, parts, slot;
};
struct Sched {
    const int *lens, *cu;
    int B, T, G, tokens, W, most;       // tokens: of a table; W: chunks aimed at; most: a chunk's tiles if that decides
};
// A sequence's length, first new token, their count, row tiles and key tiles.
__device__ __forceinline__ void sequence(const Sched& s, int b, int& len, int& first, int& n, int& rts, int& tiles) {
    len = first = n = rts = tiles = 0;
    if (b >= s.B) return;
    len = min(max(s.lens[b], 0), s.tokens);
    if (s.cu) {
        first = min(max(s.cu[b], 0), s.T);
        n = min(max(s.cu[b + 1], first), s.T) - first;
    } else {
        first = b;
        n = 1;
    }
    rts = (int)(((long long)n * s.G + kRowTile - 1) / kRowTile);
    tiles = max((len + kTile - 1) / kTile, 1);
}
// Chunks are cut by the lengths: at most q tiles each, q so that about W chunks arise from all sequences'
// tiles.  Block `index` of a kv head is the index-th chunk; the walk is over 64 sequences at a time.
// MERGE: index counts the row tiles that were split (their chunks' outcomes are to be joined).
template <bool MERGE>
__device__ __forceinline__ bool find_piece(const Sched& s, int index, int lane, Piece& p) {
    int len, first, n, rts, tiles;
    int q = s.most;
    if (q == 0) {
        long long all = 0;
        for (int b0 = 0; b0 < s.B; b0 += 64) {
            sequence(s, b0 + lane, len, first, n, rts, tiles);
            const long long work = (long long)rts * tiles;
            all += lanes_sum((int)(work & 0xFFFF)) + ((long long)lanes_sum((int)(work >> 16)) << 16);
        }
        q = max(kLeast, (int)min((all + s.W - 1) / s.W, (long long)1 << 30));
    }
    int before = 0, slots = 0;
    for (int b0 = 0; b0 < s.B; b0 += 64) {
        sequence(s, b0 + lane, len, first, n, rts, tiles);
        const int parts = (tiles + q - 1) / q;
        const int mine = MERGE ? (parts > 1 ? rts : 0) : rts * parts, room = parts > 1 ? rts * parts : 0;
        const int upto = wave_scan(mine, lane), total = __builtin_amdgcn_readlane(upto, 63);
        const int sl = wave_scan(room, lane);
        if (index < before + total) {
            const unsigned long long m = __builtin_amdgcn_ballot_w64(before + upto > index);
            const int l = __builtin_ctzll(m);
            const auto at = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
            p.b = b0 + l;
            p.first = at(first);
            p.n = at(n);
            p.len = at(len);
            p.parts = at(parts);
            const int k = index - before - (at(upto) - at(mine));
            const int rt = MERGE ? k : k / p.parts;
            p.part = MERGE ? 0 : k - rt * p.parts;
            p.row0 = rt * kRowTile;
            const int t = at(tiles);
            p.tile0 = (int)((long long)t * p.part / p.parts);
            p.tile1 = (int)((long long)t * (p.part + 1) / p.parts);
            p.slot = slots + at(sl) - at(room) + rt * p.parts;
            return true;
        }
        before += total;
        slots += __builtin_amdgcn_readlane(sl, 63);
    }
    return false;
}

struct PagedView {
    KvPages c;
    Sched s;
    const uint16_t* q;
    uint16_t* out;
    float* work;
    int qs, Hq, shift;
};
// A chunk's outcome in the workspace: 16 rows of D sums, then (maximum, sum of weights) of each row.
template <int D>
constexpr int kPartFloats = kRowTile * (D + 2);

template <int DT, int D>
__device__ __forceinline__ void store_out(const PagedView& a, const Piece& p, int h, int row, int db, int g4,
                                          const f32x4& o, float inv) {
    const int token = row / a.s.G, head = h * a.s.G + row % a.s.G;
    uint16_t* at = a.out + ((long long)(p.first + token) * a.Hq + head) * D + 16 * db + 4 * g4;
    *reinterpret_cast<u32x2*>(at) = u32x2{pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv)};
}

template <int DT, int FMT, int D>
__global__ __launch_bounds__(64 * kWaves, 2) void kv_paged_kernel(PagedView a) {
    constexpr int KB = D / 32, DB = D / 16, KL = D / 64;
    __shared__ __attribute__((aligned(16))) f32x4 lo[kWaves][DB][64];
    __shared__ float lm[kWaves][kRowTile], ll[kWaves][kRowTile];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n16 = lane & 15, g4 = lane >> 4;
    const int h = blockIdx.x % a.c.Hkv;
    Piece p;
    if (!find_piece<false>(a.s, blockIdx.x / a.c.Hkv, lane, p)) return;
    const int shift = a.shift, page = 1 << shift;
    const int rows = min(kRowTile, p.n * a.s.G - p.row0), row = p.row0 + min(n16, rows - 1);
    // the last token that the lane's row sees, and the block's last row
    const int seen = p.len - p.n + row / a.s.G, most = p.len - p.n + (p.row0 + rows - 1) / a.s.G;

    u32x4 qf[KB];
    {
        const uint16_t* qp =
            a.q + (long long)(p.first + row / a.s.G) * a.qs + (h * a.s.G + row % a.s.G) * D + 16 * g4;
#pragma unroll
        for (int s = 0; s < KB; ++s) qf[s] = *reinterpret_cast<const u32x4*>(qp + 64 * (s >> 1) + 8 * (s & 1));
    }
    const float c = 1.4426950408889634f / sqrtf((float)D);
    f32x4 o[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // running maximum (base 2): -inf while the row has seen nothing, kLowest for scores of -inf alone
    constexpr float kLowest = -3.402823466e38f;
    float M = -__builtin_inff(), l = 0.0f;
    int unit = -200;                            // o counts 2^(unit - 15)

    const int* table = a.c.table + (long long)p.b * a.c.P;
    const int last_page = max(p.len - 1, 0) >> shift;
    const int end = min(p.tile1, most >= 0 ? most / kTile + 1 : 0);
    for (int t = p.tile0 + wave; t < end; t += kWaves) {
        const int kt = kTile * t + 16 * (n16 >> 2), vt = kTile * t + 16 * g4;      // tokens of the lane's K rows, V columns
        int kid = table[min(kt >> shift, last_page)], vid = table[min(vt >> shift, last_page)];
        const bool live = (unsigned)vid < (unsigned)a.c.N;
        kid = (unsigned)kid < (unsigned)a.c.N ? kid : 0;
        vid = live ? vid : 0;
        const uint8_t* kp = (const uint8_t*)a.c.kc +
                            ((((long long)kid * a.c.Hkv + h) << shift) + (kt & (page - 1)) + (n16 & 3)) * D + 16 * g4;
        const uint8_t* vp = (const uint8_t*)a.c.vc + (((long long)vid * a.c.Hkv + h) << shift) * D + (n16 << shift) +
                            (vt & (page - 1));
        u32x4 kw[4][KL], vw[DB];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < KL; ++i) kw[j][i] = *reinterpret_cast<const u32x4*>(kp + 4 * j * D + 64 * i);
#pragma unroll
        for (int i = 0; i < DB; ++i) vw[i] = *reinterpret_cast<const u32x4*>(vp + ((16 * i) << shift));
        const float ks = a.c.ks[(long long)vid * a.c.Hkv + h];
        const float vs = live && vt <= most ? a.c.vs[(long long)vid * a.c.Hkv + h] : 0.0f;

        f32x4 S[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            S[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < KL; ++i) {
                S[j] = mfma16<DT>(widen<DT, FMT>(kw[j][i][0], kw[j][i][1]), qf[2 * i], S[j]);
                S[j] = mfma16<DT>(widen<DT, FMT>(kw[j][i][2], kw[j][i][3]), qf[2 * i + 1], S[j]);
            }
        }
        const float sc = ks * c;
        const int limit = live ? seen - vt : -1;            // the lane's tokens 0 .. limit are seen
        float mt = limit >= 0 ? kLowest : -__builtin_inff();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                S[j][e] = 4 * j + e <= limit ? S[j][e] * sc : -__builtin_inff();
                mt = fmaxf(mt, S[j][e]);
            }
        const float Mn = fmaxf(M, max_groups(mt));
        float f = M != Mn ? exp2_raw(M - Mn) : 1.0f;
        M = Mn;
        l *= f;
        // V's largest scale so far gives the unit
        const float vmax = max_groups(vs);
        const int e = vmax > 0.0f ? __builtin_amdgcn_frexp_expf(vmax) : -200;
        if (e > unit) {
            f *= __builtin_amdgcn_ldexpf(1.0f, unit - e);
            unit = e;
        }
        if (any_lane(f != 1.0f)) {
#pragma unroll
            for (int i = 0; i < DB; ++i) o[i] *= f;
        }
        const float base = M == -__builtin_inff() ? 0.0f : M;
        const float vf = __builtin_amdgcn_ldexpf(vs, 15 - unit);
        u32x4 P[2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float p0 = exp2_raw(S[j][2 * k] - base), p1 = exp2_raw(S[j][2 * k + 1] - base);
                l += p0 + p1;
                P[j >> 1][2 * (j & 1) + k] = pack2<DT_F16>(p0 * vf, p1 * vf);
            }
        // stale codes may be no numbers, and weight 0 times them would not be 0
        if (FMT == FMT_E4M3 && (kTile * (t + 1) > p.len || any_lane(!live))) {
            const int keep = live ? p.len - vt : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = min(max(keep - 4 * j, 0), 4);
                const uint32_t mask = k == 4 ? ~0u : (1u << (8 * k)) - 1u;
#pragma unroll
                for (int i = 0; i < DB; ++i) vw[i][j] &= mask;
            }
        }
#pragma unroll
        for (int i = 0; i < DB; ++i) {
            o[i] = mfma16<DT_F16>(widen<DT_F16, FMT>(vw[i][0], vw[i][1]), P[0], o[i]);
            o[i] = mfma16<DT_F16>(widen<DT_F16, FMT>(vw[i][2], vw[i][3]), P[1], o[i]);
        }
    }
    // the waves' outcomes joined
    l = sum_groups(l);
    const float u = __builtin_amdgcn_ldexpf(1.0f, unit - 15);
#pragma unroll
    for (int i = 0; i < DB; ++i) lo[wave][i][lane] = o[i] * u;
    if (g4 == 0) {
        lm[wave][n16] = M;
        ll[wave][n16] = l;
    }
    __syncthreads();
    float Mt = lm[0][n16], lt = 0.0f, fw[kWaves];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) Mt = fmaxf(Mt, lm[w][n16]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float m = lm[w][n16];
        fw[w] = m == -__builtin_inff() ? 0.0f : exp2_raw(m - Mt);
        lt += ll[w][n16] * fw[w];
    }
    if (n16 >= rows) return;
    float* part = a.work + ((long long)(p.slot + p.part) * a.c.Hkv + h) * kPartFloats<D>;
    const float inv = Mt == -__builtin_inff() ? 0.0f : 1.0f / lt;
#pragma unroll
    for (int i = wave * (DB / kWaves); i < (wave + 1) * (DB / kWaves); ++i) {
        f32x4 s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += lo[w][i][lane] * fw[w];
        if (p.parts == 1) store_out<DT, D>(a, p, h, row, i, g4, s, inv);
        else *reinterpret_cast<f32x4*>(part + n16 * D + 16 * i + 4 * g4) = s;
    }
    if (p.parts > 1 && wave == 0 && g4 == 0) {
        part[kRowTile * D + 2 * n16] = Mt;
        part[kRowTile * D + 2 * n16 + 1] = lt;
    }
}

// Joins the chunks of row tiles that were split: a thread four values of a row.
template <int DT, int D>
__global__ __launch_bounds__(256) void kv_paged_join_kernel(PagedView a) {
    const int tid = threadIdx.x, lane = tid & 63, h = blockIdx.x % a.c.Hkv;
    Piece p;
    if (!find_piece<true>(a.s, blockIdx.x / a.c.Hkv, lane, p)) return;
    const int rows = min(kRowTile, p.n * a.s.G - p.row0);
    const long long step = (long long)a.c.Hkv * kPartFloats<D>;
    const float* part = a.work + ((long long)p.slot * a.c.Hkv + h) * kPartFloats<D>;
    for (int u = tid; u < rows * (D / 4); u += 256) {
        const int r = u / (D / 4), d = u % (D / 4);
        const float* stat = part + kRowTile * D + 2 * r;
        float Mt = -__builtin_inff();
        for (int i = 0; i < p.parts; ++i) Mt = fmaxf(Mt, stat[i * step]);
        float lt = 0.0f;
        f32x4 s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = 0; i < p.parts; ++i) {
            const float m = stat[i * step], f = m == -__builtin_inff() ? 0.0f : exp2_raw(m - Mt);
            lt += stat[i * step + 1] * f;
            s += *reinterpret_cast<const f32x4*>(part + i * step + r * D + 4 * d) * f;
        }
        store_out<DT, D>(a, p, h, p.row0 + r, d >> 2, d & 3, s, Mt == -__builtin_inff() ? 0.0f : 1.0f / lt);
    }
}

// chunks aimed at for each kv head
int chunks(long long Hkv) { return (int)((kTargetBlocks + Hkv - 1) / Hkv); }

template <int DT, int FMT, int D>
hipError_t paged(const PagedView& a, long long row_tiles, hipStream_t st) {
    const unsigned blocks = (unsigned)((row_tiles + (a.s.most ? 0 : a.s.W)) * a.c.Hkv);
    hipLaunchKernelGGL((kv_paged_kernel<DT, FMT, D>), dim3(blocks), dim3(64 * kWaves), 0, st, a);
    if (!a.s.most)
        hipLaunchKernelGGL((kv_paged_join_kernel<DT, D>), dim3((unsigned)(a.s.W * a.c.Hkv)), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace

long long kv_paged_workspace_floats(long long Hq, long long Hkv, long long D, long long tokens) {
    (void)Hq;
    if (tokens <= kWhole * kTile) return 0;
    return 2LL * chunks(Hkv) * Hkv * kRowTile * (D + 2);        // (row tiles that are split have at most 2 W chunks)
}

hipError_t launch_kv_paged(const KvPagedArgs& x, float* work, hipStream_t st) {
    PagedView a = {};
    a.c = x.c;
    a.q = static_cast<const uint16_t*>(x.q);
    a.out = static_cast<uint16_t*>(x.out);
    a.work = work;
    a.qs = x.qs;
    a.Hq = x.Hq;
    a.shift = x.c.page == 16 ? 4 : x.c.page == 32 ? 5 : x.c.page == 64 ? 6 : 7;
    const int G = x.Hq / x.c.Hkv, tokens = x.c.P << a.shift;
    a.s = {x.c.lens, x.c.cu, x.c.B, x.c.T, G, tokens, chunks(x.c.Hkv), tokens <= kWhole * kTile ? kWhole : 0};
    const long long row_tiles =
        x.c.cu ? (long long)x.c.T * G / kRowTile + x.c.B : (long long)x.c.B * ((G + kRowTile - 1) / kRowTile);
#define W4A16_PAGED_D(DT, FMT) (x.c.D == 64 ? paged<DT, FMT, 64>(a, row_tiles, st) : paged<DT, FMT, 128>(a, row_tiles, st))
    if (x.dtype == DT_F16)
        return x.c.fmt == FMT_INT8 ? W4A16_PAGED_D(DT_F16, FMT_INT8) : W4A16_PAGED_D(DT_F16, FMT_E4M3);
    return x.c.fmt == FMT_INT8 ? W4A16_PAGED_D(DT_BF16, FMT_INT8) : W4A16_PAGED_D(DT_BF16, FMT_E4M3);
#undef W4A16_PAGED_D
}

}  // namespace w4a16
