// What the attention kernels over the paged cache share: codes as matrix operands, and how the work of
// sequences of any lengths, known on the device only, is cut into blocks of about equal work.
#pragma once

#include "pages.h"

namespace w4a16 {

constexpr int kTile = 64;               // cached tokens of a step

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

// What a block works on: ROWS rows from `row0` of sequence b, its tiles [tile0, tile1), and where the outcome
// goes: chunk `part` of `parts` in the workspace from `slot`, or straight out if there is one.
// Row r (a token times its G heads) is at place past + r / G and sees the tokens up to that, of the table's `len`.
struct Piece {
    int b, first, n, len, past, row0, tile0, tile1, part, parts, slot;
};
struct Sched {
    const int *lens, *cu;
    int B, T, G, tokens;        // tokens: of a table
    int W, least, most;         // W: chunks aimed at; least: their tiles; most: a chunk's tiles, if no split is wanted
    int R;                      // the blocks of a kv head that run at a time
    bool rounds;                // they are as many as there are chunks, nearly: a chunk more is a round more
};
// A sequence's length (its tokens behind the table among them), first new token, their count, row tiles and key tiles.
template <int ROWS>
__device__ __forceinline__ void sequence(const Sched& s, int b, int& len, int& first, int& n, int& rts, int& tiles) {
    len = first = n = rts = tiles = 0;
    if (b >= s.B) return;
    len = min(max(s.lens[b], 0), 1 << 25);      // (as in page_tokens: more than any table holds)
    if (s.cu) {
        first = min(max(s.cu[b], 0), s.T);
        n = min(max(s.cu[b + 1], first), s.T) - first;
    } else {
        first = b;
        n = 1;
    }
    rts = (int)(((long long)n * s.G + ROWS - 1) / ROWS);
    tiles = max((min(len, s.tokens) + kTile - 1) / kTile, 1);
}
// ceil(tiles / q) by the reciprocal, made whole
__device__ __forceinline__ int parts_of(int tiles, int q, float r) {
    int n = (int)((float)tiles * r);
    n += n * q < tiles;
    n -= (n - 1) * q >= tiles;
    return n;
}
// Chunks are cut by the lengths: at most q tiles each, so that about W chunks arise from all sequences' tiles.
template <int ROWS>
__device__ __forceinline__ int cut(const Sched& s, int lane) {
    if (s.most) return s.most;
    int len, first, n, rts = 0, tiles = 0;
    long long all = 0;
    for (int b0 = 0; b0 < s.B; b0 += 64) {
        sequence<ROWS>(s, b0 + lane, len, first, n, rts, tiles);
        const long long work = (long long)rts * tiles;
        all += lanes_sum((int)(work & 0xFFFF)) + ((long long)lanes_sum((int)(work >> 16)) << 16);
    }
    int q = max(s.least, (int)min((all + s.W - 1) / s.W, (long long)1 << 30));
    // Of a few cuts of up to 64 sequences the one whose blocks should be done first: all at a time if there are no
    // more than R, which then end with the largest; else in rounds, or one after another with the last of them a quarter
    // of a chunk late on average.  A block costs two tiles besides.  (8 sequences of up to 65536 tokens, 8 kv heads, a
    // token each: 120 -> 109 us.)
    if (s.B > 64 || all >= 1 << 24) return q;
    const float each = (float)all * __builtin_amdgcn_rcpf((float)s.R);
    const auto count = [&](int k) { return min(rts * parts_of(tiles, k, __builtin_amdgcn_rcpf((float)k)), 511); };
    if (s.rounds) {
        // (3 sequences' 80 tokens behind 20000, 32 / 8 heads: 155 -> 107 us)
        int n = lanes_sum(count(q));
        if (n <= s.R) return q;
        const int q0 = q;
        int best = (n + s.R - 1) / s.R * (q + 2);
#pragma unroll
        for (float f : {1.08f, 1.2f, 1.4f, 1.7f, 2.2f}) {
            const int k = max(q0, (int)(f * each) + 1);
            n = lanes_sum(count(k));
            const int c = (n + s.R - 1) / s.R * (k + 2);
            if (c < best) {
                best = c;
                q = k;
            }
        }
        return q;
    }
    const int q1 = max(q, (int)each + 1), q2 = max(q, (int)(1.07f * each) + 1), q3 = max(q, (int)(1.5f * each) + 1);
    // (two counts a sum: 64 times 511 are below 2^15)
    const int c01 = lanes_sum(count(q) | count(q1) << 16), c23 = lanes_sum(count(q2) | count(q3) << 16);
    const auto cost = [&](int k, int chunks) {
        return chunks <= s.R ? k + 2.0f : fmaf(2.0f, (float)chunks, (float)all) * __builtin_amdgcn_rcpf((float)s.R) + 0.25f * k;
    };
    float best = cost(q, c01 & 0xFFFF);
    const auto take = [&](int k, int chunks) {
        const float c = cost(k, chunks);
        if (c < best) {
            best = c;
            q = k;
        }
    };
    take(q1, c01 >> 16);
    take(q2, c23 & 0xFFFF);
    take(q3, c23 >> 16);
    return q;
}
// Block `index` of a kv head is the index-th chunk of a cut; the walk is over 64 sequences at a time.
// MERGE: index counts the row tiles that were split (their chunks' outcomes are to be joined).
template <int ROWS, bool MERGE>
__device__ __forceinline__ bool find_piece(const Sched& s, int q, int index, int lane, Piece& p) {
    int len, first, n, rts, tiles;
    const float rq = __builtin_amdgcn_rcpf((float)q);
    int before = 0, slots = 0;
    for (int b0 = 0; b0 < s.B; b0 += 64) {
        sequence<ROWS>(s, b0 + lane, len, first, n, rts, tiles);
        const int parts = parts_of(tiles, q, rq);
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
            p.len = min(at(len), s.tokens);
            p.past = at(len) - p.n;
            p.parts = at(parts);
            const int k = index - before - (at(upto) - at(mine));
            const int rt = MERGE ? k : k / p.parts;
            p.part = MERGE ? 0 : k - rt * p.parts;
            p.row0 = rt * ROWS;
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
// The workspace: the cut, then the chunks' outcomes.
constexpr int kWorkHead = 4;
__device__ __forceinline__ float* outcomes(const PagedView& a) { return a.work + kWorkHead; }
// A chunk's outcome in the workspace: ROWS rows of D sums, then (maximum, sum of weights) of each row.
template <int ROWS, int D>
constexpr int kPartFloats = ROWS * (D + 2);


// Four values of row `row` of a piece, from dimension d on, times inv.
template <int DT, int D>
__device__ __forceinline__ void store_out(const PagedView& a, const Piece& p, int h, int row, int d, const f32x4& o,
                                          float inv) {
    const int token = row / a.s.G, head = h * a.s.G + row % a.s.G;
    uint16_t* at = a.out + ((long long)(p.first + token) * a.Hq + head) * D + d;
    *reinterpret_cast<u32x2*>(at) = u32x2{pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv)};
}

// The cut for the joining; 0: no row tile is split.  By one wave of the attention's first block.
template <int ROWS>
__device__ __forceinline__ void keep_cut(const PagedView& a, int q, int lane) {
    bool any = false;
    for (int b0 = 0; b0 < a.s.B; b0 += 64) {
        int len, first, n, rts, tiles;
        sequence<ROWS>(a.s, b0 + lane, len, first, n, rts, tiles);
        any |= rts > 0 && tiles > q;
    }
    any = any_lane(any);
    if (lane == 0) *reinterpret_cast<int*>(a.work) = any ? q : 0;
}

// Joins the chunks of row tiles that were split: a block 1024 / (D GROUPS) rows (blockIdx.y), a thread four values of
// one and every GROUPS-th eight chunks, which are asked for at a time.
template <int DT, int D, int ROWS, int GROUPS>
__global__ __launch_bounds__(256) void kv_paged_join_kernel(PagedView a) {
    constexpr int AT = 8, RB = 1024 / (D * GROUPS);
    __shared__ __attribute__((aligned(16))) f32x4 ls[GROUPS][256 / GROUPS];
    __shared__ float lm[GROUPS][RB], ll[GROUPS][RB];
    const int tid = threadIdx.x, lane = tid & 63, h = blockIdx.x % a.c.Hkv;
    Piece p;
    const int q = __builtin_amdgcn_readfirstlane(*reinterpret_cast<const int*>(a.work));
    if (q == 0 || !find_piece<ROWS, true>(a.s, q, blockIdx.x / a.c.Hkv, lane, p)) return;
    const int rows = min(ROWS, p.n * a.s.G - p.row0), r0 = blockIdx.y * RB;
    if (r0 >= rows) return;
    const int group = tid / (256 / GROUPS), in = tid % (256 / GROUPS);
    const int rb = in / (D / 4), r = min(r0 + rb, rows - 1), d = 4 * (in % (D / 4));
    const long long step = (long long)a.c.Hkv * kPartFloats<ROWS, D>;
    const float* part = outcomes(a) + ((long long)p.slot * a.c.Hkv + h) * kPartFloats<ROWS, D>;
    float M = -__builtin_inff(), l = 0.0f;
    f32x4 s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = AT * group; i < p.parts; i += AT * GROUPS) {
        float m[AT], w[AT];
        f32x4 x[AT];
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            const float* at = part + min(i + j, p.parts - 1) * step;
            m[j] = at[ROWS * D + 2 * r];
            w[j] = at[ROWS * D + 2 * r + 1];
            x[j] = *reinterpret_cast<const f32x4*>(at + r * D + d);
        }
        float Mn = M;
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            if (i + j >= p.parts) m[j] = -__builtin_inff();
            Mn = fmaxf(Mn, m[j]);
        }
        if (Mn == -__builtin_inff()) continue;          // (rows that see nothing of these)
        const float f = exp2_raw(M - Mn);
        M = Mn;
        l *= f;
        s *= f;
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            const float e = exp2_raw(m[j] - M);
            l += w[j] * e;
            s += x[j] * e;
        }
    }
    if constexpr (GROUPS > 1) {
        ls[group][in] = s;
        if (d == 0) {
            lm[group][rb] = M;
            ll[group][rb] = l;
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 1; g < GROUPS; ++g) M = fmaxf(M, lm[g][rb]);
        l = 0.0f;
        s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const float m = lm[g][rb], e = m == -__builtin_inff() ? 0.0f : exp2_raw(m - M);
            l += ll[g][rb] * e;
            s += ls[g][in] * e;
        }
    }
    if (r0 + rb < rows) store_out<DT, D>(a, p, h, p.row0 + r, d, s, M == -__builtin_inff() ? 0.0f : 1.0f / l);
}
// Its grid: at most W row tiles are split, of a decode step's G rows.
template <int D, int ROWS, int GROUPS>
dim3 join_grid(const PagedView& a, long long row_tiles) {
    constexpr int RB = 1024 / (D * GROUPS);
    const int rows = a.s.cu || a.s.G > ROWS ? ROWS : a.s.G;
    return dim3((unsigned)((row_tiles < a.s.W ? row_tiles : a.s.W) * a.c.Hkv), (rows + RB - 1) / RB);
}

// Many rows a sequence (kv_paged_chunk.hip); the caller fills all of the view but how chunks are cut.
hipError_t launch_kv_paged_chunk(const PagedView& v, int dtype, hipStream_t st);
long long kv_paged_chunk_floats(long long Hkv, long long D, long long tokens);

}  // namespace w4a16
