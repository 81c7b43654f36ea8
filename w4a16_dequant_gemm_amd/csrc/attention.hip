// Causal attention over packed prompts: the attention that fills the cache which kv.hip
// quantizes and reads (16-bit queries, keys and values).
//
//   out[i, h] = sum_{j <= i} softmax_j(q_i . k_j / sqrt(D)) v_j      (j in the sequence of i,
//                                                                     kv head h / (Hq / Hkv))
//
// One block = 128 consecutive query rows of one sequence and one head, 32 per wave; it walks the
// keys in tiles of 64 with an online softmax (running maximum m, sum l, output O per row).
// Both products run on the matrix cores in transposed form,
//   S^T[key, row] = K Q^T   and   O^T[d, row] = V^T P^T,
// because in the 32 x 32 result a lane then holds one query row (its column) and the maximum,
// the exponentials and the rescaling of O are per-lane arithmetic: one exchange with lane ^ 32
// per tile completes the maximum, none is needed for the sum until the end.  The sixteen keys a
// lane holds of a 32-key block are, four by four, the keys that the second product wants from
// that lane if V's rows are taken in the same order, so P goes from registers to the matrix
// cores without a trip through LDS.
// P is rounded to the inputs' type (fp16 / bf16) for the second product, the only rounding
// besides the output's: relative 2^-11 / 2^-8 per weight, like the values themselves.  fp16 weights
// are held times 2^7 (kRaise), so that this holds down to 2^-21 of the largest and smaller ones are off by
// 2^-32 of it at most: taken as they are, weights below 2^-14 would lose bits and those below 2^-25
// vanish, which rows add up (one token of most of the weight beside 300 or 16384 of 2^-22 .. 2^-28: 2.3 and 1.6
// times what the rounding may cost).
// Scores, maxima, sums and outputs stay in fp32, and l sums the unrounded weights.
//
// Measured (32 heads, D = 128): one sequence of 16384 tokens, bf16, grouped heads: 1.96 ms, 1.12 PFLOP/s
// of the causal products' 2.2 TFLOP; a large library product of this card reaches 1.14.  The matrix
// cores are busy 60 % of the cycles at the clock that the power limit leaves (1.75 GHz), so what saves
// instructions, not what hides them, would shorten it: raised issue priorities, the maximum interleaved
// with the second product and stores of the output through LDS changed nothing.  12 packed prompts of
// up to 1024 tokens, fp16: 40 us (a block costs 5 us besides 1.9 a tile of keys); 6 of up to 96: 6.6 us, latency.
// One prompt of 128 / 512 / 1024 / 2048 / 4096 tokens: 8.8 / 16 / 24 / 51 / 154 us.  Before the loads went
// straight to LDS and the scores of the next tile under the weights of this one: 2313 and 49 us.  At D = 128 the
// kernel fills the registers and spills 14 vector ones, outside the loop over the tiles.
//
// Values that are no numbers: the matrix cores multiply a hidden key's value with its weight of 0, so an
// infinity or NaN among a row's later tokens of its last tile makes NaN of it.  Such rows are told by their
// outputs and computed again (rows_again).  Looking through the last tile first and keeping such values out
// of its product cost every call (12 packed prompts 39 -> 46 us, one of 1024 tokens 24 -> 31).
#include "attn.h"
#include "launch.h"

namespace w4a16 {

namespace {

constexpr int kRows = 128;      // query rows of a block
constexpr int kKeys = 64;       // keys of a tile
// exponent that a row's largest weight gets (2^15 with a maximum that lags by 8); l and O share the factor
template <int DT>
constexpr float kRaise = DT == DT_F16 ? 7.0f : 0.0f;

// The row tile that comes `rank`-th in order of work (tile j of a sequence has j + 1 times kRows keys,
// less the last one's shortfall): late tiles of all sequences first, so that the long blocks do not
// start last (12 prompts of up to 1024 tokens: 43.7 -> 41.0 us).  Lane b holds sequence b's tile count
// (B <= 64), F(j) = sum_b max(0, tiles_b - j) tiles are numbered j or later; j is the largest with
// F(j) > rank, found by bisection over the counts, and the sequences with more than j tiles follow in
// their order.  Returns false behind the last tile.
__device__ __forceinline__ int lanes_sum(int v) {
    v += __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);      // quad_perm [1,0,3,2]
    v += __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);      // quad_perm [2,3,0,1]
    v += __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);     // row_half_mirror
    v += __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);     // row_mirror
    return (__builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16)) +
           (__builtin_amdgcn_readlane(v, 32) + __builtin_amdgcn_readlane(v, 48));
}
__device__ __forceinline__ bool ranked_tile(const int* __restrict__ cu, int B, int T, int rank, int lane, int& s0,
                                            int& len, int& row0) {
    int first = 0, n = 0;
    if (lane < B) {
        first = min(max(cu[lane], 0), T);
        n = min(max(cu[lane + 1], first), T) - first;
    }
    const int tiles = (n + kRows - 1) / kRows;
    if (lanes_sum(tiles) <= rank) return false;
    int lo = 0, hi = T / kRows + 1;                 // F(lo) > rank >= F(hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (lanes_sum(max(0, tiles - mid)) > rank) lo = mid;
        else hi = mid;
    }
    int r = rank - lanes_sum(max(0, tiles - hi));   // among the sequences that have a tile lo
    unsigned long long m = __builtin_amdgcn_ballot_w64(tiles > lo);
    for (; r > 0; --r) m &= m - 1;
    const int b = __builtin_ctzll(m);
    s0 = __builtin_amdgcn_readlane(first, b);
    len = __builtin_amdgcn_readlane(n, b);
    row0 = lo * kRows;
    return true;
}

// With more sequences, the sequence of row tile `slot`.  Sequence b owns the slots first(b) = cu[b] /
// kRows + b and the following ceil(length / kRows) - 1; first() grows by at least that many per
// sequence, so the last b with first(b) <= slot is the only candidate.  64-way search, one load per
// level.  Returns false for a slot between two sequences.
__device__ __forceinline__ bool slot_tile(const int* __restrict__ cu, int B, int T, int slot, int lane, int& s0,
                                          int& len, int& row0) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) >> 6;
        const int b = lo + lane * step;
        const bool in = b < hi && min(max(cu[b], 0), T) / kRows + b <= slot;
        const int n = __builtin_popcountll(__builtin_amdgcn_ballot_w64(in));
        if (n == 0) break;
        lo += (n - 1) * step;
        hi = min(hi, lo + step);
    }
    s0 = __builtin_amdgcn_readfirstlane(min(max(cu[lo], 0), T));
    len = __builtin_amdgcn_readfirstlane(min(max(cu[lo + 1], s0), T)) - s0;
    row0 = (slot - (s0 / kRows + lo)) * kRows;
    return row0 >= 0 && row0 < len;
}

// A tile's rows straight to LDS: instruction i of the wave fills 1 KB, lane l 16 bytes at 16 l, which
// hold the piece that the tile's permutation puts there.
template <int D>
struct TileLoad {
    static constexpr int CH = D / 8;                    // 16-byte pieces of a row
    static constexpr int RI = 64 / CH;                  // rows per instruction
    static constexpr int NI = kKeys / RI / 4;           // instructions per wave
    __device__ static __forceinline__ int row(int wave, int lane, int i) { return (wave * NI + i) * RI + lane / CH; }
    __device__ static __forceinline__ void issue(const uint16_t* tile, const int (&off)[NI], uint16_t* lds, int wave) {
        const __amdgpu_buffer_rsrc_t r =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(tile), 0, -1, 0x00020000);
#pragma unroll
        for (int i = 0; i < NI; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                r, (__attribute__((address_space(3))) void*)(lds + (wave * NI + i) * RI * D), 16, off[i], 0, 0, 0);
    }
};

// A maximum as a reference: a row whose scores are -inf so far has none.
__device__ __forceinline__ float number_or_zero(float M) { return M == -__builtin_inff() ? 0.0f : M; }
__device__ __forceinline__ bool any_lane(bool p) { return __builtin_amdgcn_ballot_w64(p) != 0; }
// this wave's loads into LDS have landed, and its reads of LDS are in registers
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }

template <int DT>
__device__ __forceinline__ float value_of(uint16_t bits) {
    if constexpr (DT == DT_F16) return h2f(bits);
    else return bf2f(bits);
}
// Infinities and NaN among the two values of a word become 0: their exponents are all ones.
template <int DT>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
    constexpr uint32_t lo = DT == DT_F16 ? 0x7C00u : 0x7F80u, hi = lo << 16;
    if ((w & lo) == lo) w &= 0xFFFF0000u;
    if ((w & hi) == hi) w &= 0x0000FFFFu;
    return w;
}

// The index of the last of a tile's keys [first, end) (at most 64) whose values are not all numbers, or -1;
// behind the sequence's len keys the tile repeats its last one.
template <int DT, int D>
__device__ __forceinline__ int last_odd_key(const uint16_t* vb, int vs, int first, int end, int len, int lane) {
    const uint16_t* p = vb + (long long)min(first + lane, len - 1) * vs;
    uint32_t lost = 0;
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(p + 8 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) lost |= x[j] ^ finite_or_zero<DT>(x[j]);
    }
    const unsigned long long m = __builtin_amdgcn_ballot_w64(first + lane < end && lost != 0);
    return m ? first + 63 - __builtin_clzll(m) : -1;
}

// The rows wrow + r for the bits r of `which`, once more, by one wave from memory alone: the products and
// the softmax of the kernel below on 32 keys at a time, of which the last 32 are the rows' own tokens.  Among
// those a value that is no number stays out of the product (its weight is 0 in the rows before it, and 0
// times it would be NaN) and is added to the rows that see it.  One prompt of
// 8192 tokens, 8 heads, D = 64: 0.12 ms, with a NaN in the first token's value 0.12, in every 60th or every one's
// 0.74 - 0.77; of 16384, 32 heads, D = 128: 2.2 ms, 2.2, 16 - 17.
template <int DT, int D>
__device__ __forceinline__ void rows_again(const uint16_t* q, int qs, const uint16_t* kb, int ks, const uint16_t* vb,
                                           int vs, int wrow, int len, uint32_t which, int lane, uint16_t* out, int os) {
    asm("" : "+v"(lane), "+s"(wrow));       // (nothing of this is worked out, and held, before it is needed)
    const int n = lane & 31, h = lane >> 5, row = wrow + n;
    const float c = 1.4426950408889634f / sqrtf((float)D);
    u32x4 qf[D / 16];
    const uint16_t* qp = q + (long long)min(row, len - 1) * qs + 8 * h;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) qf[s] = *reinterpret_cast<const u32x4*>(qp + 16 * s);
    f32x16 o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    float M = -__builtin_inff(), l = 0.0f;
#pragma unroll 1
    for (int k0 = 0; k0 <= wrow; k0 += 32) {
        const bool own = k0 == wrow;                    // the rows' own tokens
        f32x16 S;
#pragma unroll
        for (int e = 0; e < 16; ++e) S[e] = 0.0f;
        const uint16_t* kp = kb + (long long)min(k0 + n, len - 1) * ks + 8 * h;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) S = mfma<DT>(*reinterpret_cast<const u32x4*>(kp + 16 * s), qf[s], S);
        float mt = -__builtin_inff();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            if (k0 + 8 * (e >> 2) + 4 * h + (e & 3) > row) S[e] = -__builtin_inff();
            mt = fmaxf(mt, S[e]);
        }
        const float Mn = fmaxf(M, max_halves(mt));
        const float f = M == Mn ? 1.0f : exp2_raw((M - Mn) * c), base = number_or_zero(Mn);
        M = Mn;
        l *= f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[i][e] *= f;
        u32x4 P[2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p0 = exp2_raw(fmaf(S[8 * s + 2 * j] - base, c, kRaise<DT>));
                const float p1 = exp2_raw(fmaf(S[8 * s + 2 * j + 1] - base, c, kRaise<DT>));
                l += p0 + p1;
                P[s][j] = pack2<DT>(p0, p1);
            }
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                u32x4 a;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = k0 + 16 * s + 4 * h + 2 * (j & 1) + 8 * (j >> 1);
                    const uint32_t lo = vb[(long long)min(key, len - 1) * vs + 32 * i + n];
                    const uint32_t hi = vb[(long long)min(key + 1, len - 1) * vs + 32 * i + n];
                    a[j] = own ? finite_or_zero<DT>(lo | hi << 16) : lo | hi << 16;
                }
                o[i] = mfma<DT>(a, P[s], o[i]);
            }
    }
    for (int key = wrow; key < min(wrow + 32, len); ++key) {
        const uint16_t* p = vb + (long long)key * vs + 4 * h;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const u32x2 x = *reinterpret_cast<const u32x2*>(p + 32 * i + 8 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = value_of<DT>((uint16_t)(x[e >> 1] >> (16 * (e & 1))));
                    o[i][4 * g + e] += key <= row && !(fabsf(v) < __builtin_inff()) ? v : -0.0f;
                }
            }
    }
    l = sum_halves(l);
    if (which >> n & 1) {
        uint16_t* op = out + (long long)row * os + 4 * h;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<u32x2*>(op + 32 * i + 8 * g) = u32x2{pack2<DT>(o[i][4 * g] / l, o[i][4 * g + 1] / l),
                                                                       pack2<DT>(o[i][4 * g + 2] / l, o[i][4 * g + 3] / l)};
    }
}

// Pipeline: in iteration t a wave turns the scores of tile t into weights while the matrix cores work
// on the scores of tile t + 1 (independent instructions, interleaved), then multiplies the weights
// with V(t).  One barrier an iteration: at its top every wave has waited for its own loads of the
// previous one, so K(t + 1) and V(t) are complete, and K(t) and V(t - 1) have been read; K(t + 2) and
// V(t + 1) are loaded over them.  The first two tiles are asked for at once (1 - 6 % for short prompts).
// The two buffers of K and of V are four LDS objects, so that the compiler does not make a read of one
// wait for loads into another.
//
// GROUPS == 2: eight waves, the first four take the first half of the keys and the others the rest, each
// with buffers of its own; the second four leave their outputs in LDS and the first add them to theirs.
template <int DT, int D, int GROUPS>
__global__ __launch_bounds__(256 * GROUPS, 2) void attention_prompt_kernel(
    const uint16_t* __restrict__ q, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
    const int* __restrict__ cu, int B, int T, int Hq, int Hkv, int qs, int ks, int vs, int tiles,
    uint16_t* __restrict__ out) {
    using L = TileLoad<D>;
    constexpr int TILE = kKeys * D;
    __shared__ __attribute__((aligned(16))) uint16_t lK0[GROUPS * TILE], lK1[GROUPS * TILE], lV0[GROUPS * TILE],
        lV1[GROUPS * TILE];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3, grp = __builtin_amdgcn_readfirstlane(tid >> 8);
    uint16_t *K0 = lK0 + grp * TILE, *K1 = lK1 + grp * TILE, *V0 = lV0 + grp * TILE, *V1 = lV1 + grp * TILE;
    const int n = lane & 31, h = lane >> 5;
    // the tiles with most keys first; heads vary fastest
    const int head = blockIdx.x % Hq, tile = blockIdx.x / Hq;
    int s0, len, row0;
    if (!(B <= 64 ? ranked_tile(cu, B, T, tile, lane, s0, len, row0)
                  : slot_tile(cu, B, T, tiles - 1 - tile, lane, s0, len, row0)))
        return;
    const int kvh = head / (Hq / Hkv);

    const int alltiles = (min(row0 + kRows, len) + kKeys - 1) / kKeys;
    // the group's tiles are tile0, tile0 + 1, ...; tiles, keys and rows count from there on below
    const int half = GROUPS == 2 ? (alltiles + 1) / 2 : alltiles;
    const int tile0 = grp * half, ntiles = grp ? alltiles - half : half, turns = half;
    const int key0 = tile0 * kKeys;
    const uint16_t* kb = k + (long long)(s0 + key0) * ks + kvh * D;
    const uint16_t* vb = v + (long long)(s0 + key0) * vs + kvh * D;
    const int keys = len - key0;
    int koff[L::NI], voff[L::NI];                   // byte offsets in a tile
    // rows behind the sequence are replaced by its last one: they may hold anything
    auto k_offsets = [&](int last) {
#pragma unroll
        for (int i = 0; i < L::NI; ++i) {
            const int r = L::row(wave, lane, i);
            koff[i] = (min(r, last) * ks + 8 * swz_k<D>(r, lane % L::CH)) * 2;
        }
    };
    auto v_offsets = [&](int last) {
#pragma unroll
        for (int i = 0; i < L::NI; ++i) {
            const int r = L::row(wave, lane, i);
            voff[i] = (min(r, last) * vs + 8 * swz_v<D>(r, lane % L::CH)) * 2;
        }
    };
    k_offsets(keys - 1);
    v_offsets(keys - 1);
    auto load_k = [&](int t, uint16_t* lds) {
        if (t >= ntiles) return;
        if (t > 0 && (t + 1) * kKeys > keys) k_offsets(keys - 1 - t * kKeys);     // the last tile
        L::issue(kb + (long long)t * kKeys * ks, koff, lds, wave);
    };
    auto load_v = [&](int t, uint16_t* lds) {
        if (t >= ntiles) return;
        if (t > 0 && (t + 1) * kKeys > keys) v_offsets(keys - 1 - t * kKeys);
        L::issue(vb + (long long)t * kKeys * vs, voff, lds, wave);
    };
    load_k(0, K0);
    load_v(0, V0);
    load_k(1, K1);
    load_v(1, V1);

    const int wrow = row0 + 32 * wave;              // first row of the wave
    const int row = wrow + n;                       // the lane's row (behind the sequence: not stored)
    u32x4 qf[D / 16];
    {
        const uint16_t* qp = q + (long long)(s0 + min(row, len - 1)) * qs + head * D + 8 * h;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) qf[s] = *reinterpret_cast<const u32x4*>(qp + 16 * s);
    }
    // tiles with a key that some row of the wave sees; only the last of them needs a mask
    const int own = wrow < len ? min(max(min(wrow + 31, len - 1) / kKeys + 1 - tile0, 0), ntiles) : 0;

    f32x16 o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    // softmax in base 2: weight = 2^(c (S - M) + kRaise), M the row's running maximum (of raw scores)
    float M = -__builtin_inff(), l = 0.0f;
    float m = -kRaise<DT>;                          // c M - kRaise, with 0 for an M of -inf: all weights are 0
    bool big = false;                               // wave-uniform: some |m| is above 2^20
    const float c = 1.4426950408889634f / sqrtf((float)D);

    // running maximum of tile t; where it rises O and l are rescaled
    auto maximum = [&](f32x16 (&S)[2], float& sub) {
        float mt = S[0][0];
#pragma unroll
        for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
            for (int e = 0; e < 16; ++e) mt = fmaxf(mt, S[kb2][e]);
        mt = max_halves(mt);
        // O and l follow a maximum that may lag the true one by 8 / c (weights up to 2^8 more): the
        // rescaling of O is then rare, and exact either way
        if (any_lane(mt > M + 8.0f / c)) {
            const float Mn = fmaxf(M, mt);
            const float f = M == Mn ? 1.0f : exp2_raw((M - Mn) * c);
            M = Mn;
            m = fmaf(number_or_zero(M), c, -kRaise<DT>);
            l *= f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[i][e] *= f;
            big = any_lane(fabsf(m) > 1048576.0f);
        }
        // c S - m in one fused operation, exact up to the rounding of m, which all weights of a
        // row share and which cancels; where it could pass the exponent range, S - M first
        sub = m;
        if (big) {
            sub = -kRaise<DT>;
            const float ref = number_or_zero(M);
#pragma unroll
            for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
                for (int e = 0; e < 16; ++e) S[kb2][e] -= ref;
        }
    };
    auto weights = [&](const f32x16 (&S)[2], float sub, u32x4 (&P)[4]) {
#pragma unroll
        for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p0 = exp2_raw(fmaf(S[kb2][8 * s + 2 * j], c, -sub));
                    const float p1 = exp2_raw(fmaf(S[kb2][8 * s + 2 * j + 1], c, -sub));
                    l += p0 + p1;
                    P[2 * kb2 + s][j] = pack2<DT>(p0, p1);
                }
    };
    auto values = [&](const uint16_t* V, const u32x4 (&P)[4]) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int r = 16 * s + 4 * h + ((lane & 15) >> 2);
                const int ch = 4 * i + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
                const u32x2 a0 = lds_read_tr(V + r * D + 8 * swz_v<D>(r, ch) + 4 * (lane & 1));
                const u32x2 a1 = lds_read_tr(V + (r + 8) * D + 8 * swz_v<D>(r + 8, ch) + 4 * (lane & 1));
                o[i] = mfma<DT>(u32x4{a0.x, a0.y, a1.x, a1.y}, P[s], o[i]);
            }
    };
    // piece 2 s + h of key 32 kb2 + n: the permutation is an exclusive or, so one register and one
    // operation a read do (kept opaque, or the compiler holds an address per piece)
    auto key_piece = [&](const uint16_t* K, int kb2, int s) {
        int at = n * D + 8 * swz_k<D>(n, h);
        asm("" : "+v"(at));
        return *reinterpret_cast<const u32x4*>(K + 32 * kb2 * D + (at ^ (16 * s)));
    };
    auto scores = [&](const uint16_t* K, f32x16 (&S)[2]) {
#pragma unroll
        for (int kb2 = 0; kb2 < 2; ++kb2) {
#pragma unroll
            for (int e = 0; e < 16; ++e) S[kb2][e] = 0.0f;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) S[kb2] = mfma<DT>(key_piece(K, kb2, s), qf[s], S[kb2]);
        }
    };
    // weights of S and scores of the next tile, a k-step's products and its share of the weights at a
    // time, the fragments one k-step ahead
    auto weights_and_scores = [&](const f32x16 (&S)[2], float sub, u32x4 (&P)[4], const uint16_t* K, f32x16 (&Sn)[2]) {
        constexpr int KS = D / 16, PW = 16 / KS;    // k-steps; pairs of weights per k-step
        u32x4 a0 = key_piece(K, 0, 0), a1 = key_piece(K, 1, 0);
#pragma unroll
        for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
            for (int e = 0; e < 16; ++e) Sn[kb2][e] = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            u32x4 n0, n1;
            if (s + 1 < KS) {
                n0 = key_piece(K, 0, s + 1);
                n1 = key_piece(K, 1, s + 1);
            }
            Sn[0] = mfma<DT>(a0, qf[s], Sn[0]);
            Sn[1] = mfma<DT>(a1, qf[s], Sn[1]);
#pragma unroll
            for (int i = 0; i < PW; ++i) {
                const int pr = PW * s + i, kb2 = pr >> 3, e = 2 * (pr & 7);
                const float p0 = exp2_raw(fmaf(S[kb2][e], c, -sub));
                const float p1 = exp2_raw(fmaf(S[kb2][e + 1], c, -sub));
                l += p0 + p1;
                P[pr >> 2][pr & 3] = pack2<DT>(p0, p1);
            }
            __builtin_amdgcn_sched_barrier(0);
            a0 = n0;
            a1 = n1;
        }
    };
    // top of iteration t: Kl takes K(t + 2), Vl takes V(t + 1) (V(1) is there from the start)
    auto turn = [&](int t, uint16_t* Kl, uint16_t* Vl) {
        wait_loads();
        __syncthreads();
        load_k(t + 2, Kl);
        if (t > 0) load_v(t + 1, Vl);
    };
    // iteration t where the wave sees tile t + 1 too: Kn = K(t + 1), Vc = V(t)
    auto full_step = [&](int t, const uint16_t* Kn, uint16_t* Kl, const uint16_t* Vc, uint16_t* Vl, f32x16 (&S)[2],
                         f32x16 (&Sn)[2]) {
        turn(t, Kl, Vl);
        u32x4 P[4];
        float sub;
        maximum(S, sub);
        weights_and_scores(S, sub, P, Kn, Sn);
        values(Vc, P);
    };
    // the wave's last tile, the only one with a key behind one of its rows
    auto last_step = [&](int t, uint16_t* Kl, const uint16_t* Vc, uint16_t* Vl, f32x16 (&S)[2]) {
        turn(t, Kl, Vl);
        const int seen = row - key0 - 4 * h - t * kKeys;       // (one register to compare constants with)
#pragma unroll
        for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (32 * kb2 + 8 * (e >> 2) + (e & 3) > seen) S[kb2][e] = -__builtin_inff();
        u32x4 P[4];
        float sub;
        maximum(S, sub);
        weights(S, sub, P);
        values(Vc, P);
    };

    f32x16 Sa[2], Sb[2];
    wait_loads();
    __syncthreads();
    // A block's rows begin at a multiple of two tiles, so its waves 0 and 1 end in an even tile and
    // waves 2 and 3 in the odd one after it; a wave without rows only keeps the barriers.
    int t = 0;
    if (own > 0) {
        scores(K0, Sa);
        for (; t + 2 < own; t += 2) {
            full_step(t, K1, K0, V0, V1, Sa, Sb);
            full_step(t + 1, K0, K1, V1, V0, Sb, Sa);
        }
        if (t + 1 < own) {
            full_step(t, K1, K0, V0, V1, Sa, Sb);
            last_step(t + 1, K1, V1, V0, Sb);
            t += 2;
        } else {
            last_step(t, K0, V0, V1, Sa);
            t += 1;
        }
    }
    for (; t < turns; ++t) turn(t, t & 1 ? K1 : K0, t & 1 ? V0 : V1);

    l = sum_halves(l);
    if constexpr (GROUPS == 2) {
        __shared__ float2 stat[4][64];
        float* joint = reinterpret_cast<float*>(wave == 0 ? lK0 : wave == 1 ? lK1 : wave == 2 ? lV0 : lV1) + 4 * lane;
        static_assert(GROUPS * TILE * 2 >= 32 * D * 4, "a wave's output");
        __syncthreads();                            // everyone is done with K and V
        if (grp == 1) {
            stat[wave][lane] = make_float2(M, l);
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<f32x4*>(joint + 256 * (4 * i + g)) =
                        f32x4{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]};
        }
        __syncthreads();
        if (grp == 1) return;
        const float2 other = stat[wave][lane];
        const float Mn = fmaxf(M, other.x), f0 = exp2_raw((M - Mn) * c), f1 = exp2_raw((other.x - Mn) * c);
        l = l * f0 + other.y * f1;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(joint + 256 * (4 * i + g));
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][4 * g + j] = fmaf(o[i][4 * g + j], f0, x[j] * f1);
            }
    }
    // A key behind a row has weight 0, but the matrix cores multiply that with the key's value: a row
    // without numbers whose sum is one may owe that to an infinity or NaN behind it in its last tile.
    bool odd = false;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; e += 2) odd |= __builtin_isunordered(o[i][e], o[i][e + 1]);
    const unsigned long long om = __builtin_amdgcn_ballot_w64(odd && l == l && row < len);
    uint32_t again = (uint32_t)om | (uint32_t)(om >> 32);
    if (__builtin_expect(again != 0, 0)) {
        const uint16_t* vall = v + (long long)s0 * vs + kvh * D;
        const int late = last_odd_key<DT, D>(vall, vs, wrow + 1, (wrow & -kKeys) + kKeys, len, lane) - wrow;
        again = late < 0 ? 0 : late < 32 ? again & ((1u << late) - 1u) : again;     // (rows before that key)
    }
    if (row < len && !(again >> n & 1)) {
        const float inv = 1.0f / l;
        uint16_t* op = out + (long long)(s0 + row) * Hq * D + head * D + 4 * h;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<u32x2*>(op + 32 * i + 8 * g) =
                    u32x2{pack2<DT>(o[i][4 * g] * inv, o[i][4 * g + 1] * inv),
                          pack2<DT>(o[i][4 * g + 2] * inv, o[i][4 * g + 3] * inv)};
    }
    if (__builtin_expect(again != 0, 0))
        rows_again<DT, D>(q + (long long)s0 * qs + head * D, qs, k + (long long)s0 * ks + kvh * D, ks,
                          v + (long long)s0 * vs + kvh * D, vs, wrow, len, again, lane,
                          out + (long long)s0 * Hq * D + head * D, Hq * D);
}

// Two groups of waves a block where the blocks leave the GPU half empty and most have many tiles.  One /
// two groups, us: 8 heads, D = 64, one prompt of 512 / 1024 / 4096 tokens 11.3 / 11.1, 17.5 / 15.7, 53.1 / 41.6;
// 32 heads, D = 128, of 512 / 1024 / 1536 / 2048 / 3000 16.2 / 16.7, 26.0 / 24.4, 37.1 / 35.6, 51.4 / 51.3,
// 89.6 / 102.6; 12 of up to 1024, 8 heads 17.0 / 20.3.
bool split_keys(const PromptArgs& a) {
    return (a.T / kRows + a.B) * (long long)a.Hq <= 448 && a.T >= 1024LL * a.B;
}

template <int DT, int D>
hipError_t prompt(const PromptArgs& a, hipStream_t st) {
    const int tiles = a.T / kRows + a.B;
#define W4A16_PROMPT(GROUPS)                                                                                          \
    hipLaunchKernelGGL((attention_prompt_kernel<DT, D, GROUPS>), dim3((unsigned)tiles * a.Hq), dim3(256 * GROUPS), 0,  \
                       st, static_cast<const uint16_t*>(a.q), static_cast<const uint16_t*>(a.k),                       \
                       static_cast<const uint16_t*>(a.v), a.cu, a.B, a.T, a.Hq, a.Hkv, a.qs, a.ks, a.vs, tiles,        \
                       static_cast<uint16_t*>(a.out))
    if (split_keys(a)) W4A16_PROMPT(2);
    else W4A16_PROMPT(1);
#undef W4A16_PROMPT
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_prompt(const PromptArgs& a, hipStream_t st) {
    if (a.dtype == DT_F16) return a.D == 64 ? prompt<DT_F16, 64>(a, st) : prompt<DT_F16, 128>(a, st);
    return a.D == 64 ? prompt<DT_BF16, 64>(a, st) : prompt<DT_BF16, 128>(a, st);
}

}  // namespace w4a16
