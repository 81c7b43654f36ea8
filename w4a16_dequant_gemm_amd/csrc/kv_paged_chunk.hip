// Causal attention over a paged 8-bit KV cache for many query rows at a time: chunks of prompts behind what is
// cached already (kv_paged.hip has the operator and takes few rows).
//
// One block = 128 or 256 rows (tokens times the heads of a kv head, token by token), 32 a wave; it walks the cached
// tokens in tiles of 64.  Both products run transposed on 32 x 32 x 16 tiles (attn.h).  A tile's codes are read
// two tiles ahead into registers, widened to 16 bits (exact) once for the block's rows and put into LDS while the
// products of the tile before run.
//
// K's 32-row operands take the tokens with bits 2 and 3 of their index exchanged, so that a lane's scores of
// registers 8 s .. 8 s + 7 are the consecutive tokens 16 s + 8 (l / 32) .. + 7, which V, whose tokens are
// consecutive in memory, then has as 16 bytes.
//
// Scales: a tile is four groups of 16 tokens, each of one page.  K's scale and 1 / sqrt(D) ride on the multiply-add
// before the exponential; V's does too, as its logarithm: the weights come out times scale / 2^unit, as they
// enter the second product, and a group's sum is divided by that again.  2^unit is the power of two above the largest
// scale of V that the row has seen.  Weights are held times 2^11 and rounded once to fp16 (relative 2^-11 down to
// 2^-25 of 2^unit, below that by 2^-36 of it, and by as much again where 2^unit or the maximum rises before they are
// used).  For fp16 outputs, where that counts beside their own rounding, the sum is taken of the rounded weights, so that
// a row that few tokens make up is off by less (19 cases: 1.41 -> 1.14 times the error of the output's rounding alone; the
// roundings in a second fp16 operand 1.00, but 2048 tokens behind 30000 1078 -> 1458 us).  The running maximum may lag by
// 4 (base 2), so that O is rarely rescaled.
//
// Bound by the vector units (60 % busy: softmax, widening) beside the matrix cores (46 %), at the power limit: 2048 tokens
// behind 30000, 32 / 8 heads, D = 128, int8, take 1050 - 1070 us in passes after one another (0.98 PFLOP/s); 128 behind
// 8000 39 us.
#include <algorithm>

#include "paged.h"

namespace w4a16 {

namespace {

constexpr float kLag = 4.0f;            // the maximum may lag by so much (base 2)
constexpr int kRaise = 11;              // weights are held times 2^kRaise; 2^(kLag + kRaise) < 65504
constexpr int kDeepest = -60;           // scales below 2^kDeepest of the largest count as that (their share is nothing)
constexpr int kThin = -8;               // scales below 2^kThin of the largest have their weights summed in fp32
constexpr float kLowest = -3.402823466e38f;

// 64 pages of a sequence from page `base` on, one a lane.
struct Window {
    int base;
    int id;                             // -1: no page
    float kc;                           // K's scale times log2(e) / sqrt(D)
    float lm, im;                       // logarithm (base 2) and reciprocal of V's scale's mantissa
    int e;                              // its exponent; kNone: V's scale is 0, or there is no page
};
constexpr int kNone = -10000;

__device__ __forceinline__ int lane_of(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ float lane_of(float v, int l) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// In iteration t the scores of tile t are computed beside the widening of K(t + 1) and V(t + 1), whose codes were
// asked for an iteration before, and its softmax beside the second product of tile t - 1; one barrier an
// iteration (eight waves: K(t + 2) and V(t + 2), a barrier every other iteration: 1026 -> 1008 us).  (The scores of tile
// t + 1 beside the softmax of tile t, as in attention.hip, need 32 registers more than there are with the codes on their way.)
//
// ONE: pages of at least a tile, so that its four groups are of one page.
template <int DT, int FMT, int D, bool ONE, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void kv_paged_chunk_kernel(PagedView a) {
    constexpr int THREADS = 64 * WAVES, kRows = 32 * WAVES, TILE = kTile * D, PR = D / 16, NL = kTile * PR / THREADS;
    static_assert(NL >= 1, "a piece a thread");         // PR: 16-code pieces of a K row; NL: loads of a thread
    constexpr int NG = ONE ? 1 : 4;
    constexpr bool kRounded = DT == DT_F16;     // sums are of rounded weights
    // tiles staged ahead, and how many of K and V there is room for
    constexpr int AHEAD = WAVES == 8 ? 2 : 1, KR = 2 * AHEAD, VR = 2 * AHEAD + 1;
    __shared__ __attribute__((aligned(16))) uint16_t lK[KR * TILE], lV[VR * TILE];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const int h = blockIdx.x % a.c.Hkv;
    Piece p;
    const int q = cut<kRows>(a.s, lane);
    if (blockIdx.x == 0 && wave == 0 && !a.s.most) keep_cut<kRows>(a, q, lane);
    if (!find_piece<kRows, false>(a.s, q, blockIdx.x / a.c.Hkv, lane, p)) return;
    const int shift = a.shift, page = 1 << shift, G = a.s.G;
    const int rows = min(kRows, p.n * G - p.row0);
    // the last token that a row sees
    const auto upto = [&](int row) { return min(p.past + row / G, p.len - 1); };
    const int wrow = p.row0 + 32 * wave, row = p.row0 + min(32 * wave + n, rows - 1);
    const int seen = upto(row), most = upto(p.row0 + rows - 1);                 // of the lane's row, of the block
    const bool idle = 32 * wave >= rows;
    const int tile0 = p.tile0;
    const int tile1 = min(p.tile1, most >= 0 ? most / kTile + 1 : 0);           // the block's tiles: [tile0, tile1)
    const int first = upto(min(wrow, p.row0 + rows - 1)), last = upto(min(wrow + 31, p.row0 + rows - 1));
    const int own1 = idle || last < 0 ? 0 : min(tile1, last / kTile + 1);       // the wave's tiles end there,
    const int clear1 = first < 0 ? 0 : (first + 1) / kTile;                     // and those before need no mask

    u32x4 qf[D / 16];
    {
        const uint16_t* qp = a.q + (long long)(p.first + row / G) * a.qs + (h * G + row % G) * D + 8 * hf;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) qf[s] = *reinterpret_cast<const u32x4*>(qp + 16 * s);
    }
    f32x16 o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    float M = -__builtin_inff(), l = 0.0f;
    // o counts 2^(unit - low - kRaise): unit is the exponent of V's largest scale that the wave has met, that of what
    // the row itself has seen lies `low` below it
    int unit = -200, low = 0;
    const float c = 1.4426950408889634f / sqrtf((float)D);

    const int* table = a.c.table + (long long)p.b * a.c.P;
    const int last_page = max(p.len - 1, 0) >> shift;
    Window w;
    auto refresh = [&](int base) {
        w.base = base;
        const int id = table[min(base + lane, last_page)];
        const bool live = (unsigned)id < (unsigned)a.c.N;
        w.id = live ? id : -1;
        const long long at = (long long)(live ? id : 0) * a.c.Hkv + h;
        const float ks = a.c.ks[at], vs = live ? a.c.vs[at] : 0.0f;
        w.kc = live ? fmaxf(ks * c, 1e-37f) : 1.0f;     // (not 0: hidden scores are -inf)
        const bool any = vs > 0.0f;
        const float m = any ? __builtin_amdgcn_frexp_mantf(vs) : 1.0f;
        w.lm = __builtin_amdgcn_logf(m);
        w.im = __builtin_amdgcn_rcpf(m);
        w.e = any ? __builtin_amdgcn_frexp_expf(vs) : kNone;
    };
    // (tiles behind the last are taken for it: they are loaded, but nothing of them is used)
    auto group_page = [&](int t, int g) { return min((kTile * t + 16 * g) >> shift, last_page) - w.base; };

    // a thread's pieces of a tile: of K token tid / PR + (THREADS / PR) i, codes 16 (tid % PR) and on; of V
    // dimension tid / 4 + 64 i, tokens 16 (tid % 4) and on
    u32x4 kw[NL], vw[NL];
    const int kr = tid / PR, kj = tid % PR, vd = tid >> 2, vg = tid & 3;
    // where tile t's pieces lie, and their loads
    const uint8_t *kat[NL], *vat;
    auto locate = [&](int t) {
        t = min(t, tile1 - 1);
        int id[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) id[g] = max(lane_of(w.id, group_page(t, g)), 0);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int r = kr + (THREADS / PR) * i, g = r >> 4;          // (g is the same for a wave)
            int pg = id[0];
            if constexpr (!ONE) pg = __builtin_amdgcn_readfirstlane(g == 0 ? id[0] : g == 1 ? id[1] : g == 2 ? id[2] : id[3]);
            const uint8_t* base = (const uint8_t*)a.c.kc + (((long long)pg * a.c.Hkv + h) << shift) * D;
            kat[i] = base + ((kTile * t + r) & (page - 1)) * D + 16 * kj;
        }
        int pv = id[0];
        if constexpr (!ONE) pv = vg == 0 ? id[0] : vg == 1 ? id[1] : vg == 2 ? id[2] : id[3];
        vat = (const uint8_t*)a.c.vc + (((long long)pv * a.c.Hkv + h) << shift) * D + ((kTile * t + 16 * vg) & (page - 1)) +
              (vd << shift);
    };
    auto load_k = [&](int i) { kw[i] = *reinterpret_cast<const u32x4*>(kat[i]); };
    auto load_v = [&](int i) { vw[i] = *reinterpret_cast<const u32x4*>(vat + ((THREADS / 4 * i) << shift)); };
    // V's codes where the weights do not hold its scale, and stale ones that may be no numbers, become 0
    auto clean_v = [&](int t) {
        t = min(t, tile1 - 1);
        bool none = false;
#pragma unroll
        for (int g = 0; g < NG; ++g) none |= lane_of(w.e, group_page(t, g)) == kNone;
        if (none || (FMT == FMT_E4M3 && kTile * (t + 1) > p.len)) {
            bool mine = false;
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (vg == g) mine = lane_of(w.e, group_page(t, g)) == kNone;
            const int keep = mine ? 0 : p.len - kTile * t - 16 * vg;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = min(max(keep - 4 * j, 0), 4);
                const uint32_t mask = k == 4 ? ~0u : (1u << (8 * k)) - 1u;
#pragma unroll
                for (int i = 0; i < NL; ++i) vw[i][j] &= mask;
            }
        }
    };
    // half `part` of piece i: registers to LDS as 16-bit values
    auto put_k = [&](uint16_t* K, int i, int part) {
        const int r = kr + (THREADS / PR) * i;
        // (not to be widened, and held, before it is needed)
        asm volatile("" : "+v"(kw[i][2 * part]), "+v"(kw[i][2 * part + 1]));
        *reinterpret_cast<u32x4*>(K + r * D + 8 * swz_k<D>(r, 2 * kj + part)) =
            widen<DT, FMT>(kw[i][2 * part], kw[i][2 * part + 1]);
    };
    auto put_v = [&](uint16_t* V, int i, int part) {
        const int d = vd + THREADS / 4 * i;
        asm volatile("" : "+v"(vw[i][2 * part]), "+v"(vw[i][2 * part + 1]));
        *reinterpret_cast<u32x4*>(V + d * kTile + 8 * swz_k<64>(d, 2 * vg + part)) =
            widen<DT_F16, FMT>(vw[i][2 * part], vw[i][2 * part + 1]);
    };
    const int kn = (n & ~12) | ((n & 4) << 1) | ((n & 8) >> 1);        // the token that row n of an operand holds
    auto key_piece = [&](const uint16_t* K, int kb, int s) {
        int at = kn * D + 8 * swz_k<D>(kn, hf);
        asm("" : "+v"(at));
        return *reinterpret_cast<const u32x4*>(K + 32 * kb * D + (at ^ (16 * s)));
    };
    auto value_piece = [&](const uint16_t* V, int g, int i) {
        int at = n * kTile + 8 * swz_k<64>(n, hf);
        asm("" : "+v"(at));
        return *reinterpret_cast<const u32x4*>(V + 32 * i * kTile + (at ^ (16 * g)));
    };
    // the scores of a tile, half a piece of the next codes to LDS beside the two products of a k-step; K's operands are
    // read kAhead steps early
    auto scores_and_stage = [&](const uint16_t* K, f32x16 (&S)[2], uint16_t* Kn, uint16_t* Vn) {
        constexpr int KS = D / 16, kAhead = 2;
        constexpr int EVERY = KS / (4 * NL);        // half a piece every so many k-steps
        u32x4 k[kAhead][2];
#pragma unroll
        for (int s = 0; s < kAhead; ++s) {
            k[s][0] = key_piece(K, 0, s);
            k[s][1] = key_piece(K, 1, s);
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int e = 0; e < 16; ++e) S[kb][e] = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const u32x4 a0 = k[s % kAhead][0], a1 = k[s % kAhead][1];
            S[0] = mfma<DT>(a0, qf[s], S[0]);
            S[1] = mfma<DT>(a1, qf[s], S[1]);
            if (s + kAhead < KS) {
                k[s % kAhead][0] = key_piece(K, 0, s + kAhead);
                k[s % kAhead][1] = key_piece(K, 1, s + kAhead);
            }
            if (s % EVERY == 0) {
                const int i = s / EVERY;
                if (i & 2) put_v(Vn, i >> 2, i & 1);
                else put_k(Kn, i >> 2, i & 1);
                // the registers of a whole piece take the tile after the next
                if ((i & 3) == 1) load_k(i >> 2);
                if ((i & 3) == 3) load_v(i >> 2);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // the weights of the tile before, whose second product is still to come: none at first
    u32x4 P[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) P[g] = u32x4{0, 0, 0, 0};
    // masks, the running maximum and what the weights of tile t need; where the maximum or the unit rises, o, l and
    // P are rescaled.  The maximum is held rounded up to a whole number, so that this is by powers of two and exact
    float kc[NG], sub[NG], inv[NG];
    auto prepare = [&](int t, f32x16 (&S)[2]) {
        float lv[NG];
        int ge[NG], top = kNone, dead = 0;
        bool thin = false;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int i = group_page(t, g);
            kc[g] = lane_of(w.kc, i);
            lv[g] = lane_of(w.lm, i);
            inv[g] = lane_of(w.im, i);
            ge[g] = lane_of(w.e, i);
            if (!ONE && kTile * t + 16 * g > most) ge[g] = kNone;       // (no row sees it)
            if (lane_of(w.id, i) < 0) dead |= 1 << g;
            top = max(top, ge[g]);
        }
        float f = 1.0f;
        const int before = unit - low;
        if (top > unit) {
            f = __builtin_amdgcn_ldexpf(1.0f, unit - top);
            unit = top;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int e = ge[g] == kNone ? 0 : max(ge[g] - unit, kDeepest) + kRaise;
            lv[g] = ge[g] == kNone ? 0.0f : lv[g] + (float)e;
            inv[g] = ge[g] == kNone ? 1.0f : __builtin_amdgcn_ldexpf(inv[g], -e);
            thin |= kRounded && e < kThin + kRaise;
        }
        unsigned long long thins = thin ? ~0ull : 0;        // rows whose weights lose bits
        // In the last tiles a wave's rows see different groups: there each row's unit is of what it sees itself, so that V's
        // scales behind it change no bit of its outcome.  (The wave's largest for all its rows: 0.4 % faster with pages of
        // 64, up to 4 % with pages of 16, but a page of 2^12 times the scale behind a row cost its weights bits, 2^40 all.)
        if (t >= clear1) {
            int mine = before;
#pragma unroll
            for (int g = 0; g < NG; ++g)
                if (kTile * t + 16 * g <= seen) mine = max(mine, ge[g]);
            low = unit - mine;
            f = __builtin_amdgcn_ldexpf(1.0f, before - mine);
            thin = false;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int i = group_page(t, g);
                const bool any = ge[g] != kNone && kTile * t + 16 * g <= seen;
                const int e = any ? max(ge[g] - mine, kDeepest) + kRaise : 0;
                lv[g] = any ? lane_of(w.lm, i) + (float)e : 0.0f;
                inv[g] = any ? __builtin_amdgcn_ldexpf(lane_of(w.im, i), -e) : 1.0f;
                thin |= e < kThin + kRaise;
            }
            thins = kRounded ? __builtin_amdgcn_ballot_w64(thin) : 0;
        }
        const bool masked = t >= clear1 || dead;
        if (masked) {
            const int upto = seen - kTile * t - 8 * hf;
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (16 * g + e > upto || (dead >> (ONE ? 0 : g) & 1)) S[g >> 1][8 * (g & 1) + e] = -__builtin_inff();
        }
        float mt = -__builtin_inff();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float mg = S[g >> 1][8 * (g & 1)];
#pragma unroll
            for (int e = 1; e < 8; ++e) mg = fmaxf(mg, S[g >> 1][8 * (g & 1) + e]);
            mt = fmaxf(mt, ONE ? mg : mg * kc[ONE ? 0 : g]);
        }
        if (ONE) mt *= kc[0];
        // what is seen at all counts as kLowest
        if (masked) {
            bool any = false;
#pragma unroll
            for (int g = 0; g < 4; ++g) any |= !(dead >> (ONE ? 0 : g) & 1) && 16 * g <= seen - kTile * t - 8 * hf;
            mt = any ? fmaxf(mt, kLowest) : -__builtin_inff();
        } else mt = fmaxf(mt, kLowest);
        mt = max_halves(mt);
        if (any_lane(mt > M + kLag)) {
            const float Mn = __builtin_ceilf(fmaxf(M, mt)), r = M == Mn ? 1.0f : exp2_raw(M - Mn);
            M = Mn;
            l *= r;
            f *= r;
        }
        if (any_lane(f != 1.0f)) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[i][e] *= f;
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    P[g][j] = pack2<DT_F16>(h2f((uint16_t)P[g][j]) * f, h2f((uint16_t)(P[g][j] >> 16)) * f);
        }
        const float base = M == -__builtin_inff() ? 0.0f : M;
        // the multiply-add of the weights is exact but for the rounding of base - lv; rows of scores so large that
        // this would count have the maximum taken off first
        const bool big = fabsf(base) > 1048576.0f;
#pragma unroll
        for (int g = 0; g < NG; ++g) sub[g] = big ? -lv[g] : base - lv[g];
        if (any_lane(big)) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float k = kc[ONE ? 0 : g], back = 1.0f / k;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // (rounded as the maximum was: a difference from the exact product could be above 0 by far)
                    float x = S[g >> 1][8 * (g & 1) + e] * k;
                    asm("" : "+v"(x));
                    if (big) S[g >> 1][8 * (g & 1) + e] = (x - base) * back;
                }
            }
        }
        if (thins) {
            // weights of so small a scale lose their last bits: they are summed before that
            const bool mine = thins >> lane & 1;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int gg = ONE ? 0 : g;
                float s = 0.0f, off = sub[gg];
                asm volatile("" : "+v"(off));           // (else these are taken for the weights below and all kept)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s += exp2_raw(fmaf(S[g >> 1][8 * (g & 1) + e], kc[gg], -off));
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (mine) l = fmaf(s, inv[gg], l);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) inv[g] = mine ? 0.0f : inv[g];
        }
    };
    float sum = 0.0f;                           // of the weights of a group (ONE: of a tile)
    auto weight_pair = [&](const f32x16 (&S)[2], int pr) {
        const int g = pr >> 2, j = pr & 3, gg = ONE ? 0 : g;
        const float p0 = exp2_raw(fmaf(S[g >> 1][8 * (g & 1) + 2 * j], kc[gg], -sub[gg]));
        const float p1 = exp2_raw(fmaf(S[g >> 1][8 * (g & 1) + 2 * j + 1], kc[gg], -sub[gg]));
        P[g][j] = pack2<DT_F16>(p0, p1);
        if (kRounded) {
            const f16x2 ones = {(_Float16)1.0f, (_Float16)1.0f};
            sum = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, (uint32_t)P[g][j]), ones, sum, false);
        } else sum += p0 + p1;
        if (ONE ? pr == 15 : j == 3) {
            l = fmaf(sum, inv[gg], l);
            sum = 0.0f;
        }
    };
    // the second product of tile t - 1
    auto values = [&](const uint16_t* V) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < D / 32; ++i) o[i] = mfma<DT_F16>(value_piece(V, g, i), P[g], o[i]);
    };
    // ... with the weights of tile t beside it, a group's in place of those of the group that has gone in before; the
    // first kEarly operands are read by the caller, the others as many products early
    constexpr int kEarly = 4;
    u32x4 v[kEarly];
    auto first_values = [&](const uint16_t* V) {
#pragma unroll
        for (int s = 0; s < kEarly; ++s) v[s] = value_piece(V, s / (D / 32), s % (D / 32));
    };
    auto values_and_weights = [&](const uint16_t* V, const f32x16 (&S)[2]) {
        constexpr int DB = D / 32, STEPS = 4 * DB, PW = 16 / STEPS;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            o[s % DB] = mfma<DT_F16>(v[s % kEarly], P[s / DB], o[s % DB]);
            if (s + kEarly < STEPS) v[s % kEarly] = value_piece(V, (s + kEarly) / DB, (s + kEarly) % DB);
            if (s >= DB)
#pragma unroll
                for (int i = 0; i < PW; ++i) weight_pair(S, PW * (s - DB) + i);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int pr = 12; pr < 16; ++pr) weight_pair(S, pr);
    };
    auto stage = [&](uint16_t* Kn, uint16_t* Vn) {
#pragma unroll
        for (int i = 0; i < NL; ++i)
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                put_k(Kn, i, part);
                put_v(Vn, i, part);
            }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            load_k(i);
            load_v(i);
        }
    };
    if (tile0 < tile1) {
        refresh(min((kTile * tile0) >> shift, last_page));
        locate(tile0);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            load_k(i);
            load_v(i);
        }
        // (what the weights of no tile are multiplied with has to be numbers)
        for (int i = tid; i < TILE / 8; i += THREADS)
            *reinterpret_cast<u32x4*>(lV + (VR - 1) * TILE + 8 * i) = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            clean_v(tile0 + i);
            locate(tile0 + i + 1);
            stage(lK + i * TILE, lV + i * TILE);
        }
        // where K(t), V(t - 1) and what is staged for t + AHEAD lie
        int kc_at = 0, kn_at = AHEAD * TILE, vp_at = (VR - 1) * TILE, vn_at = AHEAD * TILE;
        // the top of iteration t; where there is a barrier, K and V of the AHEAD tiles from t on are in LDS, and what the
        // iterations up to the next one stage over has been read
        auto top = [&](int t) {
            // tiles t .. t + AHEAD + 1 have to be in the window
            if (min((kTile * (t + AHEAD + 2) - 1) >> shift, last_page) - w.base > 63) refresh((kTile * t) >> shift);
            if (AHEAD == 1 || ((t - tile0) & 1) == 0) {
                wait_lds();
                __syncthreads();
            }
            clean_v(t + AHEAD);
            locate(t + AHEAD + 1);
        };
        auto turn = [&] {
            kc_at = kc_at == (KR - 1) * TILE ? 0 : kc_at + TILE;
            kn_at = kn_at == (KR - 1) * TILE ? 0 : kn_at + TILE;
            vp_at = vp_at == (VR - 1) * TILE ? 0 : vp_at + TILE;
            vn_at = vn_at == (VR - 1) * TILE ? 0 : vn_at + TILE;
        };
        int t = tile0;
#pragma unroll 1
        for (; t < own1; ++t) {
            top(t);
            f32x16 S[2];
            // a SIMD's other wave gives way up to the maxima, so that the two do not go in step: one's second product
            // and exponentials beside the other's scores and masks (2048 tokens behind 30000 1040 -> 1016 us, 4 of 512
            // behind 8000 in pages of 32 342 -> 323, 8 of 128 of D = 64 115 -> 106; the second half first: no gain)
            __builtin_amdgcn_s_setprio(1);
            scores_and_stage(lK + kc_at, S, lK + kn_at, lV + vn_at);
            first_values(lV + vp_at);
            prepare(t, S);
            __builtin_amdgcn_s_setprio(0);
            values_and_weights(lV + vp_at, S);
            turn();
        }
        if (t > tile0) values(lV + vp_at);
        // tiles that only other waves' rows see
#pragma unroll 1
        for (; t < tile1; ++t) {
            top(t);
            stage(lK + kn_at, lV + vn_at);
            turn();
        }
    }

    l = sum_halves(l);
    const float u = __builtin_amdgcn_ldexpf(1.0f, unit - low - kRaise);
    if (32 * wave + n >= rows) return;
    if (p.parts == 1) {
        const float inv = M == -__builtin_inff() ? 0.0f : u / l;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                store_out<DT, D>(a, p, h, row, 32 * i + 8 * g + 4 * hf,
                                 f32x4{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]}, inv);
    } else {
        float* part = outcomes(a) + ((long long)(p.slot + p.part) * a.c.Hkv + h) * kPartFloats<kRows, D>;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4*>(part + (32 * wave + n) * D + 32 * i + 8 * g + 4 * hf) =
                    f32x4{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]} * u;
        if (hf == 0) {
            part[kRows * D + 2 * (32 * wave + n)] = M;
            part[kRows * D + 2 * (32 * wave + n) + 1] = l;
        }
    }
}

constexpr int kWhole = 16;              // up to so many tiles a sequence is never split
constexpr int kLeast = 8;               // tiles of a chunk of a longer one

// chunks aimed at for each kv head: a block of eight waves a CU, or two of four
int chunks(long long Hkv, int waves) {
    const int blocks = waves == 8 ? 256 : 512;
    return (int)((blocks + Hkv - 1) / Hkv);
}

template <int DT, int FMT, int D, bool ONE, int WAVES>
hipError_t chunk(PagedView a, hipStream_t st) {
    constexpr int ROWS = 32 * WAVES;
    a.s.W = chunks(a.c.Hkv, WAVES);
    a.s.R = a.s.W;
    a.s.rounds = true;
    a.s.least = kLeast;
    a.s.most = a.s.tokens <= kWhole * kTile ? kWhole : 0;
    const long long row_tiles = (long long)a.c.T * a.s.G / ROWS + a.c.B;
    const unsigned blocks = (unsigned)((row_tiles + (a.s.most ? 0 : a.s.W)) * a.c.Hkv);
    hipLaunchKernelGGL((kv_paged_chunk_kernel<DT, FMT, D, ONE, WAVES>), dim3(blocks), dim3(64 * WAVES), 0, st, a);
    if (!a.s.most) {
        const dim3 joins = join_grid<D, ROWS, 1>(a, row_tiles);
        hipLaunchKernelGGL((kv_paged_join_kernel<DT, D, ROWS, 1>), joins, dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

// Eight waves of 256 rows where there are many: a widened code serves twice the rows.  Four / eight waves, us (32 / 8
// heads, int8, pages of 64): a chunk of 64 / 128 / 512 tokens behind 8000 29.6 / 32.6, 39.1 / 39.2, 94 / 91, of 128 / 2048 behind
// 30000 85 / 81, 1090 / 1012; 8 of 32 / 40 / 64 / 128 behind 8000 57.5 / 59.7, 81 / 73.6, 92.3 / 89.4, 165 / 158; 3 of 80
// behind 20000 108 / 126.  Short tables are not split over blocks, and four waves leave fewer CUs idle: 512 tokens alone
// 20 / 25, 64 times 1000 alone 838 / 873.
bool wide(const PagedView& a) {
    const long long rows = (long long)a.c.T * a.s.G;
    return a.s.tokens > kWhole * kTile && (rows >= 512LL * a.c.B || (rows >= 160LL * a.c.B && rows * a.c.Hkv >= 8192));
}

template <int DT, int FMT, bool ONE>
hipError_t chunk(const PagedView& a, hipStream_t st) {
    if (a.c.D == 64) return chunk<DT, FMT, 64, ONE, 4>(a, st);
    return wide(a) ? chunk<DT, FMT, 128, ONE, 8>(a, st) : chunk<DT, FMT, 128, ONE, 4>(a, st);
}
template <int DT, int FMT>
hipError_t chunk(const PagedView& a, hipStream_t st) {
    return a.c.page >= kTile ? chunk<DT, FMT, true>(a, st) : chunk<DT, FMT, false>(a, st);
}

}  // namespace

long long kv_paged_chunk_floats(long long Hkv, long long D, long long tokens) {
    // (row tiles that are split have at most 2 W chunks; W times the rows is the same for both kernels up to rounding)
    const long long rows = std::max(128LL * chunks(Hkv, 4), 256LL * chunks(Hkv, 8));
    return tokens <= kWhole * kTile ? 0 : 2 * rows * Hkv * (D + 2) + kWorkHead;
}

hipError_t launch_kv_paged_chunk(const PagedView& a, int dtype, hipStream_t st) {
    if (dtype == DT_F16) return a.c.fmt == FMT_INT8 ? chunk<DT_F16, FMT_INT8>(a, st) : chunk<DT_F16, FMT_E4M3>(a, st);
    return a.c.fmt == FMT_INT8 ? chunk<DT_BF16, FMT_INT8>(a, st) : chunk<DT_BF16, FMT_E4M3>(a, st);
}

}  // namespace w4a16
