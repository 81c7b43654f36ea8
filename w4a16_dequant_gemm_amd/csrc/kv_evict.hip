// Eviction from a quantized cache by accumulated attention weight: every (sequence, kv head) keeps
// its most recent tokens and, of the older ones, those with the largest accumulated weight
// (kv_attend.hip adds it up), in their order, in a cache of their own.
//
// Two launches.  Select (one block per sequence and kv head): the budget-th largest weight by radix
// selection on order-preserving integer keys, eight bits a pass, then one ordered pass that writes
// the kept tokens' indices and weights; ties go to the earlier token.  Gather: the kept rows' codes
// and parameters, 16 bytes per thread.  Nothing is dequantized, so the kept rows are the same bits.
// Both are bound by memory: the weights once, the kept rows in and out once.
#include "common.h"
#include "launch.h"

namespace w4a16 {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kCopies = 32;       // histogram copies: lanes of a wave that share a bin do not collide

// Order of floats as unsigned integers; -0 = +0, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float w) {
    const uint32_t u = __builtin_bit_cast(uint32_t, w + 0.0f);
    if (w != w) return 0xFFFFFFFFu;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int lanes_below(unsigned long long mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

__global__ __launch_bounds__(kSelThreads) void kv_select_kernel(const float* __restrict__ weights,
                                                                const int* __restrict__ lens, int Hkv, int Tmax,
                                                                int budget, int recent, int Tout,
                                                                float* __restrict__ weights_out,
                                                                int* __restrict__ lens_out, int* __restrict__ kept) {
    __shared__ uint32_t hist[256][kCopies];
    __shared__ uint32_t total[256];
    __shared__ uint32_t s_prefix, s_need;
    __shared__ int s_gt[kSelWaves], s_eq[kSelWaves];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const long long bh = blockIdx.x;
    const int b = blockIdx.x / Hkv;
    const int n = min(max(lens[b], 0), Tmax);
    const int count = min(n, budget);
    const float* w = weights + bh * Tmax;
    float* wo = weights_out + bh * Tout;
    int* ko = kept + bh * budget;
    if (tid == 0 && blockIdx.x % Hkv == 0) lens_out[b] = count;
    for (int i = count + tid; i < budget; i += kSelThreads) ko[i] = -1;
    for (int i = count + tid; i < Tout; i += kSelThreads) wo[i] = 0.0f;
    if (n <= budget) {
        for (int i = tid; i < n; i += kSelThreads) {
            ko[i] = i;
            wo[i] = w[i];
        }
        return;
    }
    // of the `old` earlier tokens keep the `need` largest (0 <= need < old)
    const int old = n - recent, need = budget - recent;
    uint32_t prefix = 0, mask = 0;
    int rem = need;
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256 * kCopies; i += kSelThreads) hist[0][i] = 0;
            __syncthreads();
            for (int t = tid; t < old; t += kSelThreads) {
                const uint32_t k = order_key(w[t]);
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255][lane % kCopies], 1u);
            }
            __syncthreads();
            if (tid < 256) {
                uint32_t s = 0;
                for (int c = 0; c < kCopies; ++c) s += hist[tid][(c + tid) % kCopies];
                total[tid] = s;
            }
            __syncthreads();
            // the highest digit with `rem` or more keys at or above it: lane l of wave 0 adds up the
            // digits 4 l .. 4 l + 3, a suffix sum over the lanes finds the lane
            if (wave == 0) {
                const int c0 = total[4 * lane], c1 = total[4 * lane + 1], c2 = total[4 * lane + 2],
                          c3 = total[4 * lane + 3];
                int suf = c0 + c1 + c2 + c3;
                const int mine = suf;
#pragma unroll
                for (int off = 1; off < 64; off <<= 1) {
                    const int o = __shfl_down(suf, off, 64);
                    suf += lane + off < 64 ? o : 0;
                }
                int above = suf - mine;
                if (above < rem && suf >= rem) {
                    int d = 3;
                    if (above + c3 < rem) { above += c3; d = 2; }
                    if (d == 2 && above + c2 < rem) { above += c2; d = 1; }
                    if (d == 1 && above + c1 < rem) { above += c1; d = 0; }
                    s_prefix = prefix | ((uint32_t)(4 * lane + d) << shift);
                    s_need = rem - above;
                }
            }
            __syncthreads();
            prefix = s_prefix;
            rem = s_need;
            mask |= 255u << shift;
        }
    } else {
        prefix = 0xFFFFFFFFu;            // nothing old is kept: no key is above, and no tie is taken
    }
    // wave w owns the tokens [lo, hi); how many of them are above the threshold, and at it
    const int per = ((n + kSelWaves - 1) / kSelWaves + 63) / 64 * 64;
    const int lo = min(wave * per, n), hi = min(lo + per, n);
    int gt = 0, eq = 0;
    for (int t = lo + lane; t < min(hi, old); t += 64) {
        const uint32_t k = order_key(w[t]);
        gt += k > prefix;
        eq += k == prefix;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        gt += __shfl_xor(gt, off, 64);
        eq += __shfl_xor(eq, off, 64);
    }
    if (lane == 0) {
        s_gt[wave] = gt;
        s_eq[wave] = eq;
    }
    __syncthreads();
    int ties = 0, pos = 0;               // ties seen and tokens kept before this wave's
    for (int i = 0; i < wave; ++i) {
        const int take = min(max(rem - ties, 0), s_eq[i]);
        const int ihi = min(min(i * per, n) + per, n);
        pos += s_gt[i] + take + max(0, ihi - max(min(i * per, n), old));
        ties += s_eq[i];
    }
    for (int t0 = lo; t0 < hi; t0 += 64) {
        const int t = t0 + lane;
        const float x = t < hi ? w[t] : 0.0f;
        const uint32_t k = order_key(x);
        const bool is_eq = t < hi && t < old && k == prefix;
        const unsigned long long eqm = __builtin_amdgcn_ballot_w64(is_eq);
        const bool keep = t < hi && (t >= old || k > prefix || (is_eq && ties + lanes_below(eqm) < rem));
        const unsigned long long km = __builtin_amdgcn_ballot_w64(keep);
        if (keep) {
            const int p = pos + lanes_below(km);
            ko[p] = t;
            wo[p] = x;
        }
        ties += __builtin_popcountll(eqm);
        pos += __builtin_popcountll(km);
    }
}

// Rows of 16 PR bytes: block = 64 kept rows of one (sequence, kv head), K and V with their
// parameters.  Z: with zero points (4-bit codes).
constexpr int kGatherRows = 64;
template <int PR, bool Z>
__global__ __launch_bounds__(256) void kv_gather_kernel(const int* __restrict__ lens, int Hkv, int Tmax, int budget,
                                                        int Tout, int groups, const int* __restrict__ kept, KvCache in,
                                                        KvCacheOut out) {
    const long long bh = blockIdx.x / groups;
    const int n = min(max(lens[(int)bh / Hkv], 0), Tmax);
    const int count = min(n, budget);
    const int r0 = blockIdx.x % groups * kGatherRows;
    if (r0 >= count) return;
    const int rows = min(kGatherRows, count - r0);
    const int* ko = kept + bh * budget + r0;
    const long long src = bh * Tmax, dst = bh * Tout + r0;
    const u32x4* kc = static_cast<const u32x4*>(in.kc);
    const u32x4* vc = static_cast<const u32x4*>(in.vc);
    u32x4* kd = static_cast<u32x4*>(out.kc);
    u32x4* vd = static_cast<u32x4*>(out.vc);
    for (int p = threadIdx.x; p < rows * PR; p += 256) {
        const int r = p / PR, c = p % PR;
        const long long s = (src + ko[r]) * PR + c, d = (dst + r) * PR + c;
        kd[d] = kc[s];
        vd[d] = vc[s];
    }
    if ((int)threadIdx.x < rows) {
        const long long s = src + ko[threadIdx.x], d = dst + threadIdx.x;
        out.ks[d] = in.ks[s];
        out.vs[d] = in.vs[s];
        if constexpr (Z) {
            out.kz[d] = in.kz[s];
            out.vz[d] = in.vz[s];
        }
    }
}

template <int PR, bool Z>
void gather(const KvEvictArgs& a, hipStream_t st) {
    const int rows = a.budget < a.Tmax ? a.budget : a.Tmax;
    const int groups = (rows + kGatherRows - 1) / kGatherRows;
    hipLaunchKernelGGL((kv_gather_kernel<PR, Z>), dim3((unsigned)groups * a.B * a.Hkv), dim3(256), 0, st, a.lens, a.Hkv,
                       a.Tmax, a.budget, a.Tout, groups, a.kept, a.in, a.out);
}

}  // namespace

hipError_t launch_kv_evict(const KvEvictArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(kv_select_kernel, dim3(a.B * a.Hkv), dim3(kSelThreads), 0, st, a.weights, a.lens, a.Hkv, a.Tmax,
                       a.budget, a.recent, a.Tout, a.weights_out, a.lens_out, a.kept);
    if (a.bits == 8) a.D == 64 ? gather<4, false>(a, st) : gather<8, false>(a, st);
    else a.D == 64 ? gather<2, true>(a, st) : gather<4, true>(a, st);
    return hipGetLastError();
}

}  // namespace w4a16
