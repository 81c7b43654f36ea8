// Eviction from a quantized cache by accumulated attention weight: every (sequence, kv head) keeps
// its most recent tokens and, of the older ones, those with the largest accumulated weight
// (kv_attend.hip adds it up), in their order, in a cache of their own.
//
// Select finds the budget-th largest weight by radix selection on order-preserving integer keys,
// digits of 11, 11 and 10 bits, and writes the kept tokens' indices and weights in order; ties go to
// the earlier token.  Up to kBatch tokens are one block per (sequence, kv head), the weights in
// registers from the first digit to the end.  Longer ones are cut into chunks, one block each, and
// take four launches: one per digit, in which a block adds up the chunks' histograms of the previous
// digit for itself, and the ordered write, where the same histograms tell how much the chunks before
// this one keep.  (One block walking 100001 weights of each of 8 heads took 142 us; these launches 31.)
// Gather copies the kept rows' codes and parameters, 16 bytes per thread; nothing is dequantized, so
// the kept rows are the same bits.  Where a head keeps few rows the selecting block copies them.
// All of it is bound by memory: the weights, the kept rows in and out.
// Measured: 16 x 32 heads of up to 4096 KV8 tokens, D = 128, halved: select 15.7 us, gather 93 us (533
// MB, 5.7 TB/s); 8 heads of 100001 KV4 tokens to 16384: select 4.5 + 7.6 + 7.8 + 11 us, each launch the
// latency of its chain (length, earlier histograms, scan, weights; fetching the weights first did not
// shorten it), gather 9.8 us; 2 x 2 heads of 300 to 128: 8 us, one launch.
#include <algorithm>

#include "common.h"
#include "launch.h"

namespace w4a16 {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kPer = 8;                          // tokens of a thread and batch
constexpr int kBatch = kSelThreads * kPer;
constexpr int kChunks = 64;                      // chunks of a sequence, at most
constexpr int kBins = 2048;
constexpr int kCopies = 4;                       // of the histogram: lanes that share a digit collide less
constexpr int kShift[3] = {21, 10, 0};

// Order of floats as unsigned integers; -0 = +0, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float w) {
    const uint32_t u = __builtin_bit_cast(uint32_t, w + 0.0f);
    if (w != w) return 0xFFFFFFFFu;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int lanes_below(unsigned long long mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// Inclusive sum over the lanes 0 .. l of a wave (row shifts, then the rows' totals onto the next ones).
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
    v = dpp_add<0x111, 0xF>(v);                  // row_shr 1, 2, 4, 8
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);                  // row_bcast 15 into rows 1 and 3
    return dpp_add<0x143, 0xC>(v);               // row_bcast 31 into rows 2 and 3
}
__device__ __forceinline__ int last_lane(int v) { return __builtin_amdgcn_readlane(v, 63); }
// The sum of sixteen values v[0 .. 15], and of those before index `upto`.
__device__ __forceinline__ int sum16(const int* v, int upto, int& before) {
    const int lane = threadIdx.x & 63;
    const int s = wave_scan(lane < 16 ? v[lane] : 0);
    before = upto > 0 ? __builtin_amdgcn_readlane(s, upto - 1) : 0;
    return __builtin_amdgcn_readlane(s, 15);
}

struct SelectLds {
    __attribute__((aligned(16))) uint32_t hist[2][kBins * kCopies];    // of this digit, and cleared for the next
    int sum[kSelWaves], before[kSelWaves];
    int digit, rem, whole, at;
    int gt[kSelWaves], eq[kSelWaves];
};

// What is known of the threshold key: its leading digits, and how many of the tokens that agree with
// them are kept (the largest).
struct Threshold {
    uint32_t prefix, mask;
    int rem;
    // every token that agrees so far is kept: no further digit is needed
    __device__ __forceinline__ void close() {
        prefix -= 1;                             // (rem > 0 tokens have that key or a larger one: not 0)
        rem = 0;
    }
};

// A batch's weights: token base + 512 wave + 64 j + lane in x[j]; a wave's tokens are consecutive.
__device__ __forceinline__ int token(int base, int j) {
    return base + (int)(threadIdx.x >> 6) * 64 * kPer + 64 * j + (int)(threadIdx.x & 63);
}
__device__ __forceinline__ void load_batch(const float* __restrict__ w, int base, int n, float x[kPer]) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int t = token(base, j);
        x[j] = t < n ? w[t] : 0.0f;
    }
}

__device__ __forceinline__ void clear_hist(SelectLds& s, int buf) {
    u32x4* h = reinterpret_cast<u32x4*>(s.hist[buf]);
    for (int i = threadIdx.x; i < kBins * kCopies / 4; i += kSelThreads) h[i] = u32x4{0, 0, 0, 0};
}
__device__ __forceinline__ void count_batch(SelectLds& s, int buf, const float x[kPer], int base, int old,
                                            const Threshold& th, int level) {
    const uint32_t bins = level == 2 ? 1023u : 2047u;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const uint32_t k = order_key(x[j]);
        if (token(base, j) < old && (k & th.mask) == th.prefix)
            atomicAdd(&s.hist[buf][((k >> kShift[level]) & bins) * kCopies + (threadIdx.x & (kCopies - 1))], 1u);
    }
}
// This thread's two digits, 2047 - 2 tid and 2046 - 2 tid.
__device__ __forceinline__ void counts(const SelectLds& s, int buf, int& c0, int& c1) {
    const u32x4* h = reinterpret_cast<const u32x4*>(s.hist[buf]) + (kBins - 2 - 2 * (int)threadIdx.x);
    const u32x4 lo = h[0], hi = h[1];
    c0 = (int)(hi.x + hi.y + hi.z + hi.w);
    c1 = (int)(lo.x + lo.y + lo.z + lo.w);
}
static_assert(kCopies == 4, "a digit's copies are one 16-byte load");

// The next digit of the threshold from the counts c0, c1 of this thread's two digits: the highest with
// th.rem or more tokens at or above it.  Returns whether all tokens at it are kept.
__device__ __forceinline__ bool next_digit(SelectLds& s, int c0, int c1, int level, Threshold& th) {
    const int tid = threadIdx.x, wave = tid >> 6;
    int inc = wave_scan(c0 + c1), before;
    if ((tid & 63) == 63) s.sum[wave] = inc;
    __syncthreads();
    sum16(s.sum, wave, before);
    inc += before;
    const int higher = inc - c0 - c1;                // tokens at the digits above this thread's
    if (higher < th.rem && inc >= th.rem) {
        const bool first = higher + c0 >= th.rem;
        s.digit = kBins - 1 - 2 * tid - (first ? 0 : 1);
        s.rem = th.rem - higher - (first ? 0 : c0);
        s.whole = s.rem == (first ? c0 : c1);
    }
    __syncthreads();
    th.rem = s.rem;
    th.prefix |= (uint32_t)s.digit << kShift[level];
    th.mask |= (level == 2 ? 1023u : 2047u) << kShift[level];
    return s.whole != 0;
}
// Of the counts p0, p1 of this thread's two digits: the sum over the digits above the threshold's, and
// the count at it.
__device__ __forceinline__ int above_digit(SelectLds& s, int p0, int p1, int& at) {
    const int tid = threadIdx.x, d = s.digit, mine = kBins - 1 - 2 * tid;
    const int gt = last_lane(wave_scan((mine > d ? p0 : 0) + (mine - 1 > d ? p1 : 0)));
    if ((tid & 63) == 0) s.before[tid >> 6] = gt;
    if (mine == d || mine - 1 == d) s.at = mine == d ? p0 : p1;
    __syncthreads();
    at = s.at;
    int unused;
    return sum16(s.before, 0, unused);
}

// Writes the kept tokens of one batch in order, from position `pos` on with `ties` tokens at the
// threshold seen before; both move on.  kt.prefix is the whole key (nothing is above it and no tie
// is taken when no old token is kept).
__device__ __forceinline__ void write_batch(SelectLds& s, const float x[kPer], int base, int old, int n,
                                            const Threshold& kt, int& pos, int& ties, int* __restrict__ ko,
                                            float* __restrict__ wo) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    unsigned long long gtm[kPer], eqm[kPer];
    int gt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int t = token(base, j);
        const uint32_t k = order_key(x[j]);
        const unsigned long long lm = __builtin_amdgcn_ballot_w64(t >= old && t < n);
        gtm[j] = __builtin_amdgcn_ballot_w64(t < old && k > kt.prefix) | lm;
        eqm[j] = __builtin_amdgcn_ballot_w64(t < old && k == kt.prefix);
        gt += __builtin_popcountll(gtm[j]);
        eq += __builtin_popcountll(eqm[j]);
    }
    if (lane == 0) {
        s.gt[wave] = gt;
        s.eq[wave] = eq;
    }
    __syncthreads();
    // kept and tied tokens of the waves before this one, and of all
    int eq_before, gt_before;
    const int eq_all = sum16(s.eq, wave, eq_before), gt_all = sum16(s.gt, wave, gt_before);
    const auto taken = [&](int e) { return min(max(kt.rem - ties, 0), e); };     // of the first e ties
    int p = pos + gt_before + taken(eq_before), q = ties + eq_before;
    pos += gt_all + taken(eq_all);
    ties += eq_all;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const bool keep = (gtm[j] >> lane & 1) || ((eqm[j] >> lane & 1) && q + lanes_below(eqm[j]) < kt.rem);
        const unsigned long long km = __builtin_amdgcn_ballot_w64(keep);
        if (keep) {
            const int at = p + lanes_below(km);
            ko[at] = token(base, j);
            wo[at] = x[j];
        }
        p += __builtin_popcountll(km);
        q += __builtin_popcountll(eqm[j]);
    }
    __syncthreads();                                 // before the next batch's counts
}

// Behind the kept tokens: index -1, weight 0 (threads first, first + step, ... of the sequence).
__device__ __forceinline__ void fill_rest(int count, int budget, int Tout, int first, int step, int* ko, float* wo) {
    for (int i = count + first; i < budget; i += step) ko[i] = -1;
    for (int i = count + first; i < Tout; i += step) wo[i] = 0.0f;
}

// The rows src + ko[0 .. rows) of the caches to dst, dst + 1, ...: 16 PR bytes of codes each of K and V,
// with their parameters.  Z: with zero points (4-bit codes).  ONCE: so much that the GPU's caches would not
// keep it; they are passed by.
template <int PR, bool Z, int THREADS, bool ONCE>
__device__ __forceinline__ void copy_rows(const KvCache& in, const KvCacheOut& out, const int* ko, long long src,
                                          long long dst, int rows) {
    const u32x4* kc = static_cast<const u32x4*>(in.kc);
    const u32x4* vc = static_cast<const u32x4*>(in.vc);
    u32x4* kd = static_cast<u32x4*>(out.kc);
    u32x4* vd = static_cast<u32x4*>(out.vc);
    for (int p = threadIdx.x; p < rows * PR; p += THREADS) {
        const int r = p / PR, c = p % PR;
        const long long s = (src + ko[r]) * PR + c, d = (dst + r) * PR + c;
        if constexpr (ONCE) {
            __builtin_nontemporal_store(__builtin_nontemporal_load(kc + s), kd + d);
            __builtin_nontemporal_store(__builtin_nontemporal_load(vc + s), vd + d);
        } else {
            kd[d] = kc[s];
            vd[d] = vc[s];
        }
    }
    for (int r = threadIdx.x; r < rows; r += THREADS) {
        const long long s = src + ko[r], d = dst + r;
        out.ks[d] = in.ks[s];
        out.vs[d] = in.vs[s];
        if constexpr (Z) {
            out.kz[d] = in.kz[s];
            out.vz[d] = in.vz[s];
        }
    }
}

// One block per (sequence, kv head) of up to kBatch tokens; PR > 0: it copies the kept rows too.
template <int PR, bool Z>
__global__ __launch_bounds__(kSelThreads) void kv_select_kernel(const float* __restrict__ weights,
                                                                const int* __restrict__ lens, int Hkv, int Tmax,
                                                                int budget, int recent, int Tout,
                                                                float* __restrict__ weights_out,
                                                                int* __restrict__ lens_out, int* kept, KvCache in,
                                                                KvCacheOut out) {
    __shared__ SelectLds s;
    const long long bh = blockIdx.x;
    const int b = blockIdx.x / Hkv;
    const int n = min(max(lens[b], 0), Tmax), count = min(n, budget);
    const float* w = weights + bh * Tmax;
    float* wo = weights_out + bh * Tout;
    int* ko = kept + bh * budget;
    float x[kPer];
    load_batch(w, 0, n, x);
    if (threadIdx.x == 0 && blockIdx.x % Hkv == 0) lens_out[b] = count;
    fill_rest(count, budget, Tout, threadIdx.x, kSelThreads, ko, wo);
    // n <= budget: every token is "recent"
    const int old = n <= budget ? 0 : n - recent;
    Threshold th = {0, 0, n <= budget ? 0 : budget - recent};
    if (th.rem > 0) {
        clear_hist(s, 0);
        __syncthreads();
        for (int level = 0; level < 3; ++level) {
            count_batch(s, level & 1, x, 0, old, th, level);
            if (level < 2) clear_hist(s, (level + 1) & 1);
            __syncthreads();
            int c0, c1;
            counts(s, level & 1, c0, c1);
            if (next_digit(s, c0, c1, level, th)) {
                th.close();
                break;
            }
        }
    } else {
        th.prefix = 0xFFFFFFFFu;
    }
    int pos = 0, ties = 0;
    write_batch(s, x, 0, old, n, th, pos, ties, ko, wo);       // (ends with a barrier)
    if constexpr (PR > 0) copy_rows<PR, Z, kSelThreads, false>(in, out, ko, bh * Tmax, bh * Tout, count);
}

// Longer sequences, one launch per digit (LEVEL 0 .. 2) and the ordered write (LEVEL 3).  Workspace of a
// (sequence, kv head): per chunk its three histograms and its state after the previous launch (the
// threshold so far, and how many tokens above it the chunks before this one hold).
struct ChunkState {
    uint32_t prefix, mask;
    int rem, above;
};
constexpr int kChunkWords = 3 * kBins + 4;
template <int LEVEL>
__global__ __launch_bounds__(kSelThreads) void kv_select_chunk_kernel(
    const float* __restrict__ weights, const int* __restrict__ lens, int Hkv, int Tmax, int budget, int recent,
    int Tout, int chunks, int chunk, uint32_t* __restrict__ work, float* __restrict__ weights_out,
    int* __restrict__ lens_out, int* __restrict__ kept) {
    __shared__ SelectLds s;
    const int tid = threadIdx.x;
    const long long bh = blockIdx.x / chunks;
    const int me = blockIdx.x % chunks, b = (int)(bh / Hkv);
    const int n = min(max(lens[b], 0), Tmax), count = min(n, budget);
    const float* w = weights + bh * Tmax;
    const int old = n <= budget ? 0 : n - recent;
    const int need = n <= budget ? 0 : budget - recent;
    const int lo = me * chunk, hi = min(n, lo + chunk);
    uint32_t* all = work + bh * chunks * kChunkWords;
    uint32_t* own = all + me * kChunkWords;
    ChunkState* state = reinterpret_cast<ChunkState*>(own + 3 * kBins);
    const int live = (old + chunk - 1) / chunk;      // chunks with old tokens: the ones with histograms
    if (LEVEL < 3 && (need == 0 || me >= live)) return;
    Threshold th = {0, 0, need};
    int above = 0, at = 0;
    if constexpr (LEVEL < 3) clear_hist(s, 0);
    if constexpr (LEVEL > 0) {
        if (need > 0) {
            if (LEVEL > 1 && me < live) {
                th = {state->prefix, state->mask, state->rem};
                above = state->above;
            } else if (LEVEL > 1) {                  // (LEVEL 3, a chunk of recent tokens only)
                const ChunkState* last = reinterpret_cast<const ChunkState*>(all + (live - 1) * kChunkWords + 3 * kBins);
                th = {last->prefix, last->mask, last->rem};
            }
            int c0 = 0, c1 = 0, p0 = 0, p1 = 0;
#pragma unroll 8
            for (int c = 0; c < live; ++c) {
                const uint2 v = *reinterpret_cast<const uint2*>(all + c * kChunkWords + (LEVEL - 1) * kBins + 2 * tid);
                c0 += (int)v.x;
                c1 += (int)v.y;
                p0 += c < me ? (int)v.x : 0;
                p1 += c < me ? (int)v.y : 0;
            }
            next_digit(s, c0, c1, LEVEL - 1, th);
            above += above_digit(s, p0, p1, at);
            if (LEVEL < 3 && tid == 0) *state = {th.prefix, th.mask, th.rem, above};
        } else {
            th.prefix = 0xFFFFFFFFu;
        }
    }
    float x[kPer];
    if constexpr (LEVEL < 3) {
        for (int base = lo; base < min(hi, old); base += kBatch) {
            load_batch(w, base, min(hi, old), x);
            if (base == lo) __syncthreads();             // (the cleared histogram)
            count_batch(s, 0, x, base, min(hi, old), th, LEVEL);
        }
        __syncthreads();
        int c0, c1;
        counts(s, 0, c0, c1);
        *reinterpret_cast<uint2*>(own + LEVEL * kBins + 2 * tid) = make_uint2((uint32_t)c0, (uint32_t)c1);
    } else {
        float* wo = weights_out + bh * Tout;
        int* ko = kept + bh * budget;
        if (tid == 0 && me == 0 && bh % Hkv == 0) lens_out[b] = count;
        fill_rest(count, budget, Tout, me * kSelThreads + tid, chunks * kSelThreads, ko, wo);
        // before this chunk: what is above the threshold, the ties that are taken, and recent tokens
        int ties = at, pos;
        if (me >= live) pos = need + max(0, lo - old);          // (all old tokens come before)
        else pos = above + min(ties, th.rem) + max(0, lo - old);
        for (int base = lo; base < hi; base += kBatch) {
            load_batch(w, base, hi, x);
            write_batch(s, x, base, old, hi, th, pos, ties, ko, wo);
        }
    }
}

// Rows of 16 PR bytes: block = 64 kept rows of one (sequence, kv head).  `first`: the launch's first
// block (a launch has fewer than 2^32 threads, so 2^30 rows take a second one).
constexpr int kGatherRows = 64;
constexpr long long kGatherBlocks = (1 << 24) - 1;
template <int PR, bool Z, bool ONCE>
__global__ __launch_bounds__(256) void kv_gather_kernel(const int* __restrict__ lens, int Hkv, int Tmax, int budget,
                                                        int Tout, int groups, int first,
                                                        const int* __restrict__ kept, KvCache in, KvCacheOut out) {
    const int id = first + (int)blockIdx.x;
    const long long bh = id / groups;
    const int n = min(max(lens[(int)bh / Hkv], 0), Tmax);
    const int count = min(n, budget);
    const int r0 = id % groups * kGatherRows;
    if (r0 >= count) return;
    copy_rows<PR, Z, 256, ONCE>(in, out, kept + bh * budget + r0, bh * Tmax, bh * Tout + r0, min(kGatherRows, count - r0));
}

template <int PR, bool Z>
void gather(const KvEvictArgs& a, hipStream_t st) {
    const int rows = a.budget < a.Tmax ? a.budget : a.Tmax;
    const int groups = (rows + kGatherRows - 1) / kGatherRows;
    const long long blocks = (long long)groups * a.B * a.Hkv;
    // 512 heads of up to 4096 KV8 tokens halved (268 MB of kept rows): 100 -> 92 us; 8 heads to 16384 KV4 ones
    // (17 MB) 9.8 -> 10.5
    const bool once = 32LL * PR * rows * a.B * a.Hkv >= (64 << 20);
#define W4A16_GATHER(ONCE)                                                                                             \
    hipLaunchKernelGGL((kv_gather_kernel<PR, Z, ONCE>), dim3((unsigned)std::min(blocks - first, kGatherBlocks)),       \
                       dim3(256), 0, st, a.lens, a.Hkv, a.Tmax, a.budget, a.Tout, groups, (int)first, a.kept, a.in,    \
                       a.out)
    for (long long first = 0; first < blocks; first += kGatherBlocks)
        if (once) W4A16_GATHER(true);
        else W4A16_GATHER(false);
#undef W4A16_GATHER
}

}  // namespace

// Tokens of a chunk: whole batches, at most kChunks chunks.
static int chunk_tokens(long long Tmax) { return (int)((Tmax + (long long)kBatch * kChunks - 1) / (kBatch * kChunks)) * kBatch; }

long long kv_evict_call_words(long long B, long long Hkv, long long Tmax) {
    if (Tmax <= kBatch) return 0;
    const int chunk = chunk_tokens(Tmax);
    return B * Hkv * ((Tmax + chunk - 1) / chunk) * kChunkWords;
}

// What any call of at most B sequences and Tmax tokens uses: past kBatch kChunks tokens the chunks become
// longer, and fewer than kChunks again.
long long kv_evict_workspace_words(long long B, long long Hkv, long long Tmax) {
    if (Tmax <= kBatch) return 0;
    return B * Hkv * std::min<long long>((Tmax + kBatch - 1) / kBatch, kChunks) * kChunkWords;
}

// Kept rows that the selecting block copies itself: up to 64 KB of K's codes.  Against a launch of its own,
// us in a graph (a call by itself saves 3 us of submission besides): 8 heads of 1000 KV4 tokens to 125 / 500
// (D = 128) 8.7 / 9.5 against 9.9 / 10.0, 512 heads 17.7 / 26.5 against 20.2 / 31.3; of 4096 to 512 / 2048
// 10.2 / 14.6 against 10.9 / 11.1 and 30.1 / 88.1 against 35.9 / 81.7.
constexpr long long kWholeBytes = 65536;

template <int PR, bool Z>
static void evict(const KvEvictArgs& a, uint32_t* work, hipStream_t st) {
    if (a.Tmax <= kBatch) {
        const bool whole = std::min(a.budget, a.Tmax) * 16LL * PR <= kWholeBytes;
#define W4A16_SELECT(ROWS)                                                                                            \
    hipLaunchKernelGGL((kv_select_kernel<ROWS, Z>), dim3(a.B * a.Hkv), dim3(kSelThreads), 0, st, a.weights, a.lens,    \
                       a.Hkv, a.Tmax, a.budget, a.recent, a.Tout, a.weights_out, a.lens_out, a.kept, a.in, a.out)
        if (whole) {
            W4A16_SELECT(PR);
            return;
        }
        W4A16_SELECT(0);
#undef W4A16_SELECT
    } else {
        const int chunk = chunk_tokens(a.Tmax), chunks = (a.Tmax + chunk - 1) / chunk;
        const dim3 grid((unsigned)chunks * a.B * a.Hkv);
#define W4A16_SELECT(L)                                                                                               \
    hipLaunchKernelGGL(kv_select_chunk_kernel<L>, grid, dim3(kSelThreads), 0, st, a.weights, a.lens, a.Hkv, a.Tmax,    \
                       a.budget, a.recent, a.Tout, chunks, chunk, work, a.weights_out, a.lens_out, a.kept)
        W4A16_SELECT(0);
        W4A16_SELECT(1);
        W4A16_SELECT(2);
        W4A16_SELECT(3);
#undef W4A16_SELECT
    }
    gather<PR, Z>(a, st);
}

hipError_t launch_kv_evict(const KvEvictArgs& a, uint32_t* work, hipStream_t st) {
    if (a.bits == 8) a.D == 64 ? evict<4, false>(a, work, st) : evict<8, false>(a, work, st);
    else a.D == 64 ? evict<2, true>(a, work, st) : evict<4, true>(a, work, st);
    return hipGetLastError();
}

}  // namespace w4a16
