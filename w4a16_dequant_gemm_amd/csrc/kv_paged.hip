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
// multiplies the scores, V's the weights, which are held times 2^15 over the power of two above the largest scale of
// V that their row has seen, and go in as two fp16 numbers, rounded and the rest (relative 2^-22 down to 2^-18 of that
// scale times the row's largest softmax weight, below by 2^-39 of it).  The first alone would be off by as much as an fp16
// output's own rounding (1.4 times its error) and turn bf16 outputs over (8 sequences of up to 65536 tokens: 1.05e-3 of the
// norm off 32-bit weights' outputs, now 8e-5), in 0.4 to 3 % less time (bf16, 8 sequences of up to 40000 tokens, e4m3,
// 113.6 against 116.1 us; 128 of up to 8000, int8, 364 against 376).  Scores, maxima, sums and outputs are fp32.
//
// Bound by memory: one token each of 8 sequences of up to 65536 tokens, 32 / 8 heads, D = 128, e4m3 (801 MB), take
// 145 us with the joining (5.7 TB/s; vector units 28 % busy), of 16 of up to 4096, 32 heads, int8 (338 MB) 75 us; a few
// hundred tokens 6.4 us, of dependent latencies.
#include <algorithm>

#include "paged.h"

namespace w4a16 {

namespace {

constexpr int kRowTile = 16;            // query rows of a block
constexpr int kWaves = 4;
constexpr int kWhole = 16;              // up to so many tiles a sequence is never split
constexpr int kLeast = 4;               // tiles of a chunk of a longer one

template <int DT>
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
    if constexpr (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
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

template <bool ONCE>
__device__ __forceinline__ u32x4 codes(const uint8_t* at) {
    const u32x4* w = reinterpret_cast<const u32x4*>(at);
    return ONCE ? __builtin_nontemporal_load(w) : *w;
}

// ONCE: codes to read past the caches, K's (1), V's too (2).
template <int DT, int FMT, int D, int ONCE>
__global__ __launch_bounds__(64 * kWaves, 2) void kv_paged_kernel(PagedView a) {
    constexpr int KB = D / 32, DB = D / 16, KL = D / 64;
    __shared__ __attribute__((aligned(16))) f32x4 lo[kWaves][DB][64];
    __shared__ float lm[kWaves][kRowTile], ll[kWaves][kRowTile];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n16 = lane & 15, g4 = lane >> 4;
    const int h = blockIdx.x % a.c.Hkv;
    Piece p;
    const int q = cut<kRowTile>(a.s, lane);
    if (blockIdx.x == 0 && wave == 0 && !a.s.most) keep_cut<kRowTile>(a, q, lane);
    if (!find_piece<kRowTile, false>(a.s, q, blockIdx.x / a.c.Hkv, lane, p)) return;
    const int shift = a.shift, page = 1 << shift;
    const int rows = min(kRowTile, p.n * a.s.G - p.row0), row = p.row0 + min(n16, rows - 1);
    // the last token that the lane's row sees, and the block's last row
    const int seen = min(p.past + row / a.s.G, p.len - 1), most = min(p.past + (p.row0 + rows - 1) / a.s.G, p.len - 1);

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
    // tokens of the lane's K rows and V columns in a tile, and their pages, asked for a tile early
    const auto k_token = [&](int t) { return kTile * t + 16 * (n16 >> 2); };
    const auto v_token = [&](int t) { return kTile * t + 16 * g4; };
    const auto page_of = [&](int token) { return table[min(token >> shift, last_page)]; };
    const int t0 = p.tile0 + wave;
    int kid_next = page_of(k_token(t0)), vid_next = page_of(v_token(t0));
    for (int t = t0; t < end; t += kWaves) {
        const int kt = k_token(t), vt = v_token(t);
        int kid = kid_next, vid = vid_next;
        kid_next = page_of(k_token(t + kWaves));
        vid_next = page_of(v_token(t + kWaves));
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
            for (int i = 0; i < KL; ++i) kw[j][i] = codes<ONCE >= 1>(kp + 4 * j * D + 64 * i);
#pragma unroll
        for (int i = 0; i < DB; ++i) vw[i] = codes<ONCE >= 2>(vp + ((16 * i) << shift));
        const float ks = a.c.ks[(long long)vid * a.c.Hkv + h];
        // (0 where the row sees none of the 16 tokens: its unit below must not come from what it does not see)
        const float vs = live && vt <= seen ? a.c.vs[(long long)vid * a.c.Hkv + h] : 0.0f;

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
        // V's largest scale that the row has seen so far gives its unit
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
        u32x4 P[2], rest[2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float p0 = exp2_raw(S[j][2 * k] - base), p1 = exp2_raw(S[j][2 * k + 1] - base);
                l += p0 + p1;
                uint32_t word = pack2<DT_F16>(p0 * vf, p1 * vf);
                // (the rest is of the very bits that go in: rounded anew, from the exact product, one weight in thousands
                // came out a step of fp16 beside them)
                asm("" : "+v"(word));
                const f16x2 w = __builtin_bit_cast(f16x2, word);
                P[j >> 1][2 * (j & 1) + k] = word;
                rest[j >> 1][2 * (j & 1) + k] = pack2<DT_F16>(fmaf(p0, vf, -(float)w[0]), fmaf(p1, vf, -(float)w[1]));
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
            const u32x4 v0 = widen<DT_F16, FMT>(vw[i][0], vw[i][1]), v1 = widen<DT_F16, FMT>(vw[i][2], vw[i][3]);
            o[i] = mfma16<DT_F16>(v0, P[0], o[i]);
            o[i] = mfma16<DT_F16>(v1, P[1], o[i]);
            o[i] = mfma16<DT_F16>(v0, rest[0], o[i]);
            o[i] = mfma16<DT_F16>(v1, rest[1], o[i]);
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
    float* part = outcomes(a) + ((long long)(p.slot + p.part) * a.c.Hkv + h) * kPartFloats<kRowTile, D>;
    const float inv = Mt == -__builtin_inff() ? 0.0f : 1.0f / lt;
#pragma unroll
    for (int i = wave * (DB / kWaves); i < (wave + 1) * (DB / kWaves); ++i) {
        f32x4 s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += lo[w][i][lane] * fw[w];
        if (p.parts == 1) store_out<DT, D>(a, p, h, row, 16 * i + 4 * g4, s, inv);
        else *reinterpret_cast<f32x4*>(part + n16 * D + 16 * i + 4 * g4) = s;
    }
    if (p.parts > 1 && wave == 0 && g4 == 0) {
        part[kRowTile * D + 2 * n16] = Mt;
        part[kRowTile * D + 2 * n16 + 1] = lt;
    }
}

// Blocks that run at a time, for each kv head: three on a CU, four of D = 64.
int resident(long long Hkv, long long D) { return (int)(((D == 128 ? 768 : 1024) + Hkv - 1) / Hkv); }
// Chunks aimed at, at most (what is left over runs alone).
int chunks(long long Hkv, long long D) { return (4 * resident(Hkv, D) + 2) / 3; }

template <int DT, int FMT, int D>
hipError_t paged(const PagedView& a, long long row_tiles, hipStream_t st) {
    const unsigned blocks = (unsigned)((row_tiles + (a.s.most ? 0 : a.s.W)) * a.c.Hkv);
    // Caches that one row tile reads pass the GPU's caches by (8 sequences of up to 65536 tokens, 8 kv heads, e4m3:
    // 128 -> 119 us, 64 of up to 2048 51 -> 48), but not V in pages of 128, whose lines two waves share (162 -> 164).
    if (a.s.cu || a.s.G > kRowTile)
        hipLaunchKernelGGL((kv_paged_kernel<DT, FMT, D, 0>), dim3(blocks), dim3(64 * kWaves), 0, st, a);
    else if (a.c.page == 128)
        hipLaunchKernelGGL((kv_paged_kernel<DT, FMT, D, 1>), dim3(blocks), dim3(64 * kWaves), 0, st, a);
    else
        hipLaunchKernelGGL((kv_paged_kernel<DT, FMT, D, 2>), dim3(blocks), dim3(64 * kWaves), 0, st, a);
    if (a.s.most) return hipGetLastError();
    // few row tiles, of many chunks each: a row's chunks to four groups of threads (one sequence of 65536 tokens 56 -> 44 us)
    if (8 * row_tiles <= a.s.W) {
        const dim3 joins = join_grid<D, kRowTile, 4>(a, row_tiles);
        hipLaunchKernelGGL((kv_paged_join_kernel<DT, D, kRowTile, 4>), joins, dim3(256), 0, st, a);
    } else {
        const dim3 joins = join_grid<D, kRowTile, 1>(a, row_tiles);
        hipLaunchKernelGGL((kv_paged_join_kernel<DT, D, kRowTile, 1>), joins, dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace

long long kv_paged_workspace_floats(long long Hkv, long long D, long long tokens, bool many) {
    // (row tiles that are split have at most 2 W chunks)
    const long long few = tokens <= kWhole * kTile ? 0 : 2LL * chunks(Hkv, D) * Hkv * kRowTile * (D + 2) + kWorkHead;
    return many ? std::max(few, kv_paged_chunk_floats(Hkv, D, tokens)) : few;
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
    a.s = {x.c.lens, x.c.cu, x.c.B, x.c.T, G, tokens, chunks(x.c.Hkv, x.c.D), kLeast, tokens <= kWhole * kTile ? kWhole : 0,
           resident(x.c.Hkv, x.c.D), false};
    // many rows a sequence: 128 at a time
    if (x.c.cu && (long long)x.c.T * G > 32LL * x.c.B) return launch_kv_paged_chunk(a, x.dtype, st);
    const long long row_tiles =
        x.c.cu ? (long long)x.c.T * G / kRowTile + x.c.B : (long long)x.c.B * ((G + kRowTile - 1) / kRowTile);
#define W4A16_PAGED_D(DT, FMT) (x.c.D == 64 ? paged<DT, FMT, 64>(a, row_tiles, st) : paged<DT, FMT, 128>(a, row_tiles, st))
    if (x.dtype == DT_F16)
        return x.c.fmt == FMT_INT8 ? W4A16_PAGED_D(DT_F16, FMT_INT8) : W4A16_PAGED_D(DT_F16, FMT_E4M3);
    return x.c.fmt == FMT_INT8 ? W4A16_PAGED_D(DT_BF16, FMT_INT8) : W4A16_PAGED_D(DT_BF16, FMT_E4M3);
#undef W4A16_PAGED_D
}

}  // namespace w4a16
