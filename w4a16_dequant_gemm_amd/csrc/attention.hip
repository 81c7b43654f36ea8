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
// besides the output's: relative 2^-11 / 2^-8 per weight, like the values themselves; scores,
// maxima, sums and outputs stay in fp32, and l sums the unrounded weights.
#include "attn.h"
#include "launch.h"

namespace w4a16 {

namespace {

constexpr int kRows = 128;      // query rows of a block
constexpr int kKeys = 64;       // keys of a tile

// The sequence of row tile `slot`.  Sequence b owns the slots first(b) = cu[b] / kRows + b and the
// following ceil(length / kRows) - 1; first() grows by at least that many per sequence, so the
// last b with first(b) <= slot is the only candidate.  64-way search, one load per level.
__device__ __forceinline__ int find_sequence(const int* __restrict__ cu, int B, int T, int slot, int lane) {
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
    return lo;
}

template <int DT, int D>
__global__ __launch_bounds__(256, 2) void attention_prompt_kernel(
    const uint16_t* __restrict__ q, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
    const int* __restrict__ cu, int B, int T, int Hq, int Hkv, int qs, int ks, int vs, int tiles,
    uint16_t* __restrict__ out) {
    constexpr int CH = D / 8;                       // 16-byte pieces of a row
    constexpr int PT = kKeys * CH / 256;            // pieces a thread stages per tile
    __shared__ __attribute__((aligned(16))) uint16_t Ks[2][kKeys * D], Vs[2][kKeys * D];

    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int n = lane & 31, h = lane >> 5;
    // late row tiles (the ones with most keys) first; heads vary fastest
    const int head = blockIdx.x % Hq;
    const int slot = tiles - 1 - blockIdx.x / Hq;
    const int b = find_sequence(cu, B, T, slot, lane);
    const int s0 = min(max(cu[b], 0), T);
    const int len = min(max(cu[b + 1], s0), T) - s0;
    const int row0 = (slot - (s0 / kRows + b)) * kRows;
    if (row0 < 0 || row0 >= len) return;            // a slot between two sequences
    const int kvh = head / (Hq / Hkv);

    const int wrow = row0 + 32 * wave;              // first row of the wave
    const int row = wrow + n;                       // the lane's row (behind the sequence: not stored)
    u32x4 qf[D / 16];
    {
        const uint16_t* qp = q + (long long)(s0 + min(row, len - 1)) * qs + head * D + 8 * h;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) qf[s] = *reinterpret_cast<const u32x4*>(qp + 16 * s);
    }

    f32x16 o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    // softmax in base 2: weight = 2^(c (S - M)), M the row's running maximum (of raw scores)
    float M = -__builtin_inff(), m = M, l = 0.0f;
    bool big = false;                               // wave-uniform: some |c M| is above 2^20
    const float c = 1.4426950408889634f / sqrtf((float)D);

    const int ntiles = (min(row0 + kRows, len) + kKeys - 1) / kKeys;
    const uint16_t* kb = k + (long long)s0 * ks + kvh * D;
    const uint16_t* vb = v + (long long)s0 * vs + kvh * D;
    u32x4 kr[PT], vr[PT];
    // rows behind the sequence are replaced by its last one: they may hold anything
    auto load = [&](int t) {
        const uint16_t* kt = kb + (long long)t * kKeys * ks;
        const uint16_t* vt = vb + (long long)t * kKeys * vs;
        const int last = len - 1 - t * kKeys;
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            const int p = tid + 256 * i, r = min(p / CH, last), ch = p % CH;
            kr[i] = *reinterpret_cast<const u32x4*>(kt + r * ks + 8 * ch);
            vr[i] = *reinterpret_cast<const u32x4*>(vt + r * vs + 8 * ch);
        }
    };
    auto store = [&](int buf) {
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            const int p = tid + 256 * i, r = p / CH, ch = p % CH;
            *reinterpret_cast<u32x4*>(&Ks[buf][r * D + 8 * swz_k<D>(r, ch)]) = kr[i];
            *reinterpret_cast<u32x4*>(&Vs[buf][r * D + 8 * swz_v<D>(r, ch)]) = vr[i];
        }
    };

    load(0);
    store(0);
    __syncthreads();
    for (int t = 0; t < ntiles; ++t) {
        if (t + 1 < ntiles) load(t + 1);
        const uint16_t* K = Ks[t & 1];
        const uint16_t* V = Vs[t & 1];
        const int key0 = t * kKeys;
        if (key0 <= wrow + 31) {                    // wave-uniform: some key is visible to some row
            f32x16 S[2];
#pragma unroll
            for (int kb2 = 0; kb2 < 2; ++kb2) {
#pragma unroll
                for (int e = 0; e < 16; ++e) S[kb2][e] = 0.0f;
                const int r = 32 * kb2 + n;
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const u32x4 a = *reinterpret_cast<const u32x4*>(K + r * D + 8 * swz_k<D>(r, 2 * s + h));
                    S[kb2] = mfma<DT>(a, qf[s], S[kb2]);
                }
            }
            if (key0 + kKeys - 1 > wrow) {
#pragma unroll
                for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (key0 + 32 * kb2 + 8 * (e >> 2) + 4 * h + (e & 3) > row) S[kb2][e] = -__builtin_inff();
            }
            float mt = S[0][0];
#pragma unroll
            for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
                for (int e = 0; e < 16; ++e) mt = fmaxf(mt, S[kb2][e]);
            mt = max_halves(mt);
            // O and l follow a maximum that may lag the true one by 8 / c (weights up to 2^8): the
            // rescaling of O is then rare, and exact either way
            if (__builtin_amdgcn_ballot_w64(mt > M + 8.0f / c)) {
                const float Mn = fmaxf(M, mt);
                const float f = exp2_raw((M - Mn) * c);
                M = Mn;
                m = M * c;
                l *= f;
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[i][e] *= f;
                big = __builtin_amdgcn_ballot_w64(fabsf(m) > 1048576.0f) != 0;
            }
            // c S - m in one fused operation, exact up to the rounding of m, which all weights of a
            // row share and which cancels; where it could pass the exponent range, S - M first
            float sub = m;
            if (big) {
                sub = 0.0f;
#pragma unroll
                for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
                    for (int e = 0; e < 16; ++e) S[kb2][e] -= M;
            }
            u32x4 P[4];
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
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int r = 16 * s + 4 * h + ((lane & 15) >> 2);
                    const int ch = 4 * i + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
                    const u32x2 a0 = lds_read_tr(V + r * D + 8 * swz_v<D>(r, ch) + 4 * (lane & 1));
                    const u32x2 a1 = lds_read_tr(V + (r + 8) * D + 8 * swz_v<D>(r + 8, ch) + 4 * (lane & 1));
                    o[i] = mfma<DT>(u32x4{a0.x, a0.y, a1.x, a1.y}, P[s], o[i]);
                }
        }
        if (t + 1 < ntiles) store((t + 1) & 1);
        __syncthreads();
    }

    l = sum_halves(l);
    if (row < len) {
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
}

template <int DT, int D>
hipError_t prompt(const PromptArgs& a, hipStream_t st) {
    const int tiles = a.T / kRows + a.B;
    hipLaunchKernelGGL((attention_prompt_kernel<DT, D>), dim3((unsigned)tiles * a.Hq), dim3(256), 0, st,
                       static_cast<const uint16_t*>(a.q), static_cast<const uint16_t*>(a.k),
                       static_cast<const uint16_t*>(a.v), a.cu, a.B, a.T, a.Hq, a.Hkv, a.qs, a.ks, a.vs, tiles,
                       static_cast<uint16_t*>(a.out));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_prompt(const PromptArgs& a, hipStream_t st) {
    if (a.dtype == DT_F16) return a.D == 64 ? prompt<DT_F16, 64>(a, st) : prompt<DT_F16, 128>(a, st);
    return a.D == 64 ? prompt<DT_BF16, 64>(a, st) : prompt<DT_BF16, 128>(a, st);
}

}  // namespace w4a16
