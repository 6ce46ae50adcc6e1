// Drawing the next tokens with temperature, top-k, top-p and min-p from given
// random numbers (qlin_sample).
//
// With x the logits of a row, M their largest and T the temperature, a word's
// weight is w_v = exp((x_v - M) / T).  The words in the order of their logits
// (equal ones by their number) are cut behind the k-th, then behind the first
// of them whose running sum reaches p times the sum of what top-k left, then
// where w < min_p.  The token is the first word, by number, at which the
// running sum of the weights left exceeds u times their sum.
//
// The sums decide between neighbouring words, whose weights are 10^-6 of the
// sum and less, so a float's 2^-24 would take the wrong one often.  A weight is
// a whole number of 2^-44 (2^44 for the largest; fewer bits above 2^18 words),
// good to about 2^-38 of itself, and sums of whole numbers do not depend on
// their order.  2^-y: y as a pair of floats in units of 1/32, its whole part
// split into an exponent and one of 32 numbers 2^(-j/32), which the lanes of a
// warp hold and hand over by shuffles, and a series of four terms.
//
// One cluster of CTAs per row, whose shared memory holds the row: it is read
// once.  A cut is found with a histogram of 2048 bins over y (counts for
// top-k, weights for top-p; a CTA sums a share of the bins over the cluster's),
// then among the words of one bin, which go to a list in the first CTA.  Where
// few words are left the first CTA does the rest alone.
#include <cmath>

#include "launch.cuh"
#include "stream.cuh"
#include "tcgen05.cuh"

namespace qlin {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kLocalBins = 512;
constexpr int kList = 1536;
constexpr int kMaxCluster = 16;
constexpr int kMaxVocab = 1 << 24;
constexpr float kInf = __builtin_huge_valf();
constexpr float kPart = 32.0f;               // units of y to a factor of two
constexpr float kNoWeight = 46.0f * kPart;   // y from which a weight is 0
constexpr float kMagic = 12582912.0f;        // 1.5 * 2^23: adding it rounds to a whole number
constexpr int kMagicBits = 0x4B400000;

struct SampleArgs {
    const float *logits;
    int64_t row_stride;
    const float *u, *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p;
    int vocab;
    int32_t *tokens;
    float *probs;
    int32_t *kept;
    int cluster, slice;  // CTAs of a row, words of a CTA (a multiple of 4)
    int cached;          // of them in shared memory (a multiple of 4)
    int drop;            // bits of a weight that are left out, so that a row's sum stays below 2^63
    int wide;            // rows are 16-byte aligned
};

struct Shared {
    union {
        struct {
            u64 mass[kBins];
            uint32_t count[kBins];
        } hist;
        struct {
            u64 mass[kList];
            uint32_t key[kList], idx[kList];
        } list;
    };
    u64 lmass[kLocalBins];  // the first CTA's own histograms
    u64 scan[kWarps];
    u64 pub[2];             // what the CTAs tell each other, in turn
    u64 peer[kMaxCluster];
    u64 found[4];           // what a search ends with
    uint32_t n_list;
    double thr;             // the least logit that min-p keeps, less the largest
    float ch, cl;
};

// 2^(24 - j/32) as a pair
__device__ const float2 kPow[32] = {
    {16777216.0f, 0.e+00f}, {16417715.0f, -1.4278924e-01f}, {16065917.0f, 8.25886e-02f}, {15721658.0f, -3.9116126e-01f},
    {15384775.0f, -9.42819e-02f}, {15055111.0f, -9.575634e-02f}, {14732511.0f, -7.747526e-02f}, {14416824.0f, -4.068154e-01f},
    {14107901.0f, -2.0766273e-01f}, {13805598.0f, -4.2991382e-01f}, {13509772.0f, 8.251217e-02f}, {13220286.0f, -4.7488123e-01f},
    {12937002.0f, 6.770366e-02f}, {12659789.0f, -2.093744e-01f}, {12388516.0f, -3.7756276e-01f}, {12123055.0f, 2.788541e-01f},
    {11863283.0f, 2.0303145e-01f}, {11609078.0f, -4.9287915e-01f}, {11360319.0f, -8.492081e-02f}, {11116891.0f, -2.9329705e-01f},
    {10878679.0f, -3.3713812e-01f}, {10645571.0f, 1.1906231e-02f}, {10417458.0f, 3.7722212e-01f}, {10194234.0f, -2.7408895e-01f},
    {9975792.0f, 3.1856874e-01f}, {9762032.0f, -3.3985955e-01f}, {9552851.0f, 4.5182908e-01f}, {9348154.0f, -4.5596614e-01f},
    {9147842.0f, -1.09702356e-01f}, {8951823.0f, -4.977592e-01f}, {8760003.0f, 4.0546086e-01f}, {8572295.0f, -4.036229e-01f},
};

// An fp32 number's place in the order of numbers, equal for both zeros.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // key_of(-inf)

template <typename T>
__device__ __forceinline__ T ld_peer(const T *local, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    if constexpr (sizeof(T) == 8) {
        u64 v;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
        return (T)v;
    } else {
        uint32_t v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
        return (T)v;
    }
}
__device__ __forceinline__ void st_peer(uint32_t *local, uint32_t rank, uint32_t v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_peer(uint32_t *local, uint32_t rank, uint32_t v) {
    uint32_t a, old;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(a), "r"(v) : "memory");
    return old;
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// floor(a * b) of a number b in 0 .. 1 and a < 2^63, and whether that is all of it
__device__ __forceinline__ u64 times(u64 a, float b, bool &exact) {
    exact = true;
    if (!(b > 0.0f)) return 0;
    if (b >= 1.0f) return a;
    const uint32_t bits = __float_as_uint(b);
    const int e = (int)(bits >> 23);
    const u64 m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int sh = 150 - (e ? e : 1);  // b = m 2^-sh, sh >= 24
    const u64 lo = a * m, hi = __umul64hi(a, m);
    if (sh >= 128) {
        exact = lo == 0 && hi == 0;
        return 0;
    }
    if (sh >= 64) {
        exact = lo == 0 && (sh == 64 || (hi << (128 - sh)) == 0);
        return sh == 64 ? hi : hi >> (sh - 64);
    }
    exact = (lo << (64 - sh)) == 0;
    return hi << (64 - sh) | lo >> sh;
}

struct Row {
    const SampleArgs &A;
    Shared &S;
    float *words;  // the CTA's words, filled up with minus infinity to a multiple of 4
    const float *from;
    int rank, n;   // n words of its own, from word `first` on
    int first;
    float M, ch, cl;  // the largest logit; y = (M - x) (ch + cl)
    float th, tl;     // this lane's number 2^(-lane/32), times 2^24
    uint32_t kt, it;  // kept: a key above kt, or equal and a word number up to it (first: all finite ones)
    int turn = 0;

    __device__ __forceinline__ bool keeps(uint32_t k, uint32_t i) const { return k > kt || (k == kt && i <= it); }
    __device__ __forceinline__ float y_of(float x) const { return __fmul_rn(__fsub_rn(M, x), ch); }
    __device__ __forceinline__ int bin_of(float y) const {
        return y < kNoWeight ? __float_as_int(__fmaf_rn(y, 1.375f, kMagic)) - kMagicBits : kBins - 1;
    }
    // A word's weight; all lanes of the warp at once.
    __device__ __forceinline__ u64 weight(float x, bool on) const {
        const float s = __fsub_rn(M, x), bb = __fsub_rn(s, M);
        const float e = __fsub_rn(__fsub_rn(M, __fsub_rn(s, bb)), __fadd_rn(x, bb));
        const float yh = __fmul_rn(s, ch);
        on = on && yh < kNoWeight;
        const float t = __fadd_rn(yh, kMagic), f = __fsub_rn(yh, __fsub_rn(t, kMagic));  // -1/2 .. 1/2, exact
        const int n = __float_as_int(t) - kMagicBits;
        const float yl = __fmaf_rn(e, ch, __fmaf_rn(s, cl, __fmaf_rn(s, ch, -yh)));
        // z = (f + yl) log(2) / 32 as a pair
        const float zh = __fmul_rn(f, kL), zl = __fmaf_rn(yl, kL, __fmaf_rn(f, kLl, __fmaf_rn(f, kL, -zh)));
        // exp(-z) = 1 - zh + b
        const float b = __fmaf_rn(__fmul_rn(zh, zh),
                                  __fmaf_rn(zh, __fmaf_rn(zh, 1.0f / 24.0f, -1.0f / 6.0f), 0.5f), -zl);
        const float a = __shfl_sync(0xffffffffu, th, n & 31), al = __shfl_sync(0xffffffffu, tl, n & 31);
        const float ph = __fmul_rn(a, zh), pl = __fmaf_rn(a, zh, -ph), hi = __fsub_rn(a, ph);
        float lo = __fsub_rn(__fsub_rn(__fsub_rn(a, hi), ph), pl);
        lo = __fadd_rn(__fmaf_rn(a, b, lo), __fmaf_rn(-al, zh, al));
        if (!on) return 0;
        // (hi is a whole number of halves up to 2^24 and a little, lo below 2^10)
        const int64_t v = (int64_t)__float2int_rn(__fmul_rn(hi, 2.0f)) * (1 << 19) + __float2int_rn(__fmul_rn(lo, 1048576.0f));
        const int sh = (n >> 5) + A.drop;
        return sh ? (u64)(v + ((int64_t)1 << (sh - 1))) >> sh : (u64)v;
    }
    // log(2) / 32
    static constexpr float kL = 0.021660849452018738f, kLl = -5.9520444e-11f;

    // f(logit, word number) of the CTA's words, warp by warp in runs of `run` words from r0 on; all lanes of a warp at
    // once (words that are not there are minus infinity)
    template <typename F>
    __device__ __forceinline__ void words_of_warp(F f) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, run = (A.slice + 128 * kWarps - 1) / (128 * kWarps) * 128;
        const int r0 = min(n, warp * run), r1 = min(n, r0 + run);
        for (int b = r0; b < r1; b += 128) {
            const int i = b + 4 * lane;
            float4 v = make_float4(-kInf, -kInf, -kInf, -kInf);
            if (i < r1) v = quad(i);
            f(v.x, (uint32_t)(first + i)), f(v.y, (uint32_t)(first + i + 1)), f(v.z, (uint32_t)(first + i + 2)),
                f(v.w, (uint32_t)(first + i + 3));
        }
    }
    // words i .. i + 3 (i a multiple of 4), minus infinity behind the last
    __device__ __forceinline__ float4 quad(int i) const {
        if (i < A.cached) return *reinterpret_cast<const float4 *>(words + i);
        float4 v;
        v.x = __ldg(from + i);
        v.y = i + 1 < n ? __ldg(from + i + 1) : -kInf;
        v.z = i + 2 < n ? __ldg(from + i + 2) : -kInf;
        v.w = i + 3 < n ? __ldg(from + i + 3) : -kInf;
        return v;
    }

    // thread 0's v of every CTA of the cluster, in S.peer
    __device__ __forceinline__ void tell(u64 v) {
        if (threadIdx.x == 0) S.pub[turn & 1] = v;
        cluster_sync();
        if (threadIdx.x < A.cluster) S.peer[threadIdx.x] = ld_peer(&S.pub[turn & 1], threadIdx.x);
        turn++;
        __syncthreads();
    }
    // the sums of v over the threads before this one, and over all
    __device__ __forceinline__ u64 before(u64 v, u64 &total) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        u64 in = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const u64 o = __shfl_up_sync(0xffffffffu, in, off);
            if (lane >= off) in += o;
        }
        __syncthreads();
        if (lane == 31) S.scan[warp] = in;
        __syncthreads();
        u64 w = 0, all = 0;
#pragma unroll
        for (int k = 0; k < kWarps; k++) {
            const u64 x = S.scan[k];
            if (k < warp) w += x;
            all += x;
        }
        total = all;
        return w + in - v;
    }

    // The first word, by number, at which the running sum of f(logit, number) exceeds want(sum over all).  f is called
    // by whole warps.  On every CTA: S.found = {number, its f, the sum, the words with one} of the CTA that has it in
    // owner's shared memory; the sum's owner is returned, or -1 if the sum is 0.
    template <typename F, typename W>
    __device__ __forceinline__ int search(F f, W want, u64 &sum) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        u64 mine = 0;
        words_of_warp([&](float x, uint32_t i) { mine += f(x, i); });
        mine = warp_sum(mine);
        __syncthreads();
        if (lane == 0) S.scan[warp] = mine;
        __syncthreads();
        u64 all = 0;
        for (int k = 0; k < kWarps; k++) all += S.scan[k];
        tell(all);
        sum = 0;
        for (int k = 0; k < A.cluster; k++) sum += S.peer[k];
        if (sum == 0) return -1;
        const u64 target = want(sum);
        u64 low = 0;
        int owner = 0;
        while (owner < A.cluster - 1 && low + S.peer[owner] <= target) low += S.peer[owner++];
        if (owner == rank) {
            int w = 0;
            while (w < kWarps - 1 && low + S.scan[w] <= target) low += S.scan[w++];
            // the run of warp w, a stretch of words per thread
            const int run = (A.slice + 128 * kWarps - 1) / (128 * kWarps) * 128, r0 = min(n, w * run), r1 = min(n, r0 + run);
            const int per = (r1 - r0 + kThreads - 1) / kThreads, a = r0 + (int)threadIdx.x * per;
            u64 v = 0, total;
            for (int k = 0; k < per; k++) {
                const int i = a + k;
                const float x = i < r1 ? (i < A.cached ? words[i] : __ldg(from + i)) : -kInf;
                v += f(x, (uint32_t)(first + i));
            }
            u64 at = low + before(v, total);
            const bool here = at <= target && target < at + v;
            // (whole warps again, for f)
            for (int k = 0; k < per; k++) {
                const int i = a + k;
                const float x = i < r1 ? (i < A.cached ? words[i] : __ldg(from + i)) : -kInf;
                const u64 g = f(x, (uint32_t)(first + i));
                if (here && at <= target && target < at + g) S.found[0] = (u64)(first + i), S.found[1] = g;
                at += g;
            }
            __syncthreads();
        }
        return owner;
    }

    // ---------------------------------------------------------------- a cut, by the whole cluster
    struct Cut {
        int bin;
        u64 above, above_n;  // what the words in the bins before hold, and how many they are
        u64 in_n, total;     // words in the bin; the sum over all bins
    };
    // A histogram is filled: the bin at which the running sum reaches want(total) (by weights, or by counts).
    template <bool MASS, typename W>
    __device__ __forceinline__ Cut find_bin(W want) {
        const int tid = threadIdx.x, C = A.cluster, per = (kBins + C - 1) / C, b0 = rank * per;
        const int mine = max(0, min(per, kBins - b0)), each = (mine + kThreads - 1) / kThreads;  // bins of a thread: 4 at most
        cluster_sync();
        u64 m[4] = {}, c[4] = {}, ms = 0, cs = 0;
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int b = b0 + tid * each + k;
            if (k >= each || tid * each + k >= mine) continue;
            for (int r = 0; r < C; r++) {
                if (MASS) m[k] += ld_peer(&S.hist.mass[b], (uint32_t)r);
                c[k] += ld_peer(&S.hist.count[b], (uint32_t)r);
            }
            ms += m[k], cs += c[k];
        }
        u64 mt = 0, ct;
        u64 mb = MASS ? before(ms, mt) : 0;
        u64 cb = before(cs, ct);
        // the CTAs' sums
        Cut r;
        u64 mlow = 0, clow = 0;
        r.total = 0;
        if (MASS) {
            tell(mt);
            for (int k = 0; k < C; k++) {
                if (k < rank) mlow += S.peer[k];
                r.total += S.peer[k];
            }
            __syncthreads();
        }
        tell(ct);
        u64 call = 0;
        for (int k = 0; k < C; k++) {
            if (k < rank) clow += S.peer[k];
            call += S.peer[k];
        }
        if (!MASS) r.total = call;
        const u64 target = want(r.total);
        mb += mlow, cb += clow;
        if (tid < 4) S.found[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const u64 a = MASS ? mb : cb, v = MASS ? m[k] : c[k];
            if (a < target && target <= a + v)
                S.found[0] = (u64)(b0 + tid * each + k) + 1, S.found[1] = a, S.found[2] = cb, S.found[3] = c[k];
            mb += m[k], cb += c[k];
        }
        cluster_sync();
        // (one CTA has it; the others' are zeros)
        u64 x[4] = {0, 0, 0, 0};
        for (int k = 0; k < C; k++)
            if (ld_peer(&S.found[0], (uint32_t)k))
                for (int e = 0; e < 4; e++) x[e] = ld_peer(&S.found[e], (uint32_t)k);
        r.bin = (int)x[0] - 1, r.above = x[1], r.above_n = x[2], r.in_n = x[3];
        cluster_sync();  // (before anyone writes found or the histogram again)
        return r;
    }
    __device__ __forceinline__ void clear_hist() {
        __syncthreads();
        for (int b = threadIdx.x; b < kBins; b += kThreads) S.hist.mass[b] = 0, S.hist.count[b] = 0;
        __syncthreads();
    }
    // the words that are kept so far, by y
    template <bool MASS>
    __device__ __forceinline__ void fill_by_y() {
        clear_hist();
        uint32_t rest = 0;
        words_of_warp([&](float x, uint32_t i) {
            const bool on = keeps(key_of(x), i);
            const u64 w = MASS ? weight(x, on) : 0;
            const int b = bin_of(y_of(x));
            if (!on) return;
            if (b == kBins - 1) {
                rest++;  // (those of no weight, which may be most)
                return;
            }
            if (MASS) atomicAdd(&S.hist.mass[b], w);
            atomicAdd(&S.hist.count[b], 1u);
        });
        rest = __reduce_add_sync(0xffffffffu, rest);
        if ((threadIdx.x & 31) == 0 && rest) atomicAdd(&S.hist.count[kBins - 1], rest);
    }
    // the kept words that sel(key, y) takes to the first CTA's list
    template <typename F>
    __device__ __forceinline__ void gather(F sel) {
        if (threadIdx.x == 0 && rank == 0) S.n_list = 0;
        cluster_sync();
        words_of_warp([&](float x, uint32_t i) {
            const uint32_t k = key_of(x);
            if (!keeps(k, i) || !sel(k, x)) return;
            const uint32_t at = add_peer(&S.n_list, 0, 1);
            if (at < kList) st_peer(&S.list.key[at], 0, k), st_peer(&S.list.idx[at], 0, i);
        });
        cluster_sync();
    }

    // ---------------------------------------------------------------- the first CTA alone
    // Of the n list entries with on(e): the key at which the running sum of val(e), from the largest key down, reaches
    // target (0 < target <= the sum); above: the sum of the entries with larger keys.
    template <typename K, typename V, typename O>
    __device__ __forceinline__ uint32_t local_cut(int n, K key, V val, O on, u64 target, u64 &above) {
        const int tid = threadIdx.x;
        uint32_t hi = 0xffffffffu;
        int s = 23;  // bins of 2^s keys from hi down
        above = 0;
        for (;;) {
            __syncthreads();
            S.lmass[tid] = 0;
            __syncthreads();
            for (int e = tid; e < n; e += kThreads) {
                const uint32_t d = hi - key(e);
                if (on(e) && key(e) <= hi && (d >> s) < kLocalBins) atomicAdd(&S.lmass[d >> s], val(e));
            }
            __syncthreads();
            const u64 v = S.lmass[tid];
            u64 total;
            const u64 b = above + before(v, total);
            if (b < target && target <= b + v) S.found[0] = (u64)tid, S.found[1] = b;
            __syncthreads();
            hi -= (uint32_t)S.found[0] << s;
            above = S.found[1];
            if (s == 0) return hi;
            s = s > 9 ? s - 9 : 0;
        }
    }
    // Cuts the list's kept words behind the first `target` of the sum, by counts or weights: kt and it.
    template <bool MASS>
    __device__ __forceinline__ void cut_list(int n, u64 target) {
        u64 above;
        const uint32_t k = local_cut(
            n, [&](int e) { return S.list.key[e]; }, [&](int e) { return MASS ? S.list.mass[e] : (u64)1; },
            [&](int e) { return keeps(S.list.key[e], S.list.idx[e]); }, target, above);
        // of the words with this key, the first ones that reach the target
        u64 a2;
        const uint32_t last = local_cut(
            n, [&](int e) { return ~S.list.idx[e]; }, [&](int e) { return MASS ? S.list.mass[e] : (u64)1; },
            [&](int e) { return S.list.key[e] == k && keeps(k, S.list.idx[e]); }, target - above, a2);
        __syncthreads();
        kt = k, it = ~last;
    }
    __device__ __forceinline__ u64 sum_list(int n, uint32_t &count) {
        u64 v = 0, total, many;
        u64 c = 0;
        for (int e = threadIdx.x; e < n; e += kThreads)
            if (keeps(S.list.key[e], S.list.idx[e])) v += S.list.mass[e], c++;
        before(v, total);
        before(c, many);
        count = (uint32_t)many;
        return total;
    }
    __device__ __forceinline__ void weigh_list(int n) {
        for (int e = threadIdx.x; e - (int)(threadIdx.x & 31) < n; e += kThreads) {
            const u64 w = weight(e < n ? of_key(S.list.key[e]) : -kInf, e < n);
            if (e < n) S.list.mass[e] = w;
        }
        __syncthreads();
    }

    // ---------------------------------------------------------------- the parts of a row
    // min-p's cut
    __device__ __forceinline__ void cut_min_p(float min_p) {
        if (!(min_p > 0.0f) || ch == 0.0f) return;  // (at an infinite temperature all weigh the same)
        const double t = (double)M + S.thr;
        float x = (float)t;
        if ((double)x < t) x = nextafterf(x, kInf);
        const uint32_t k = key_of(fminf(x, M));
        if (k > kt) kt = k, it = 0xffffffffu;
    }
    // In a bin of `in_n` kept words (those that sel takes), the cut where the running sum reaches target.
    template <bool MASS, typename F>
    __device__ __forceinline__ void cut_in_bin(F sel, u64 in_n, u64 target) {
        uint32_t prefix = 0;
        int known = 0;  // of a key's bits
        auto in = [&](uint32_t k, float x) { return sel(k, x) && (known == 0 || (k >> (32 - known)) == prefix); };
        while (in_n > kList && known < 32) {
            const int bits = known == 22 ? 10 : 11, sh = 32 - known - bits;
            clear_hist();
            words_of_warp([&](float x, uint32_t i) {
                const uint32_t k = key_of(x);
                const bool on = keeps(k, i) && in(k, x);
                const u64 w = MASS ? weight(x, on) : 0;
                if (!on) return;
                const int b = (1 << bits) - 1 - (int)((k >> sh) & ((1u << bits) - 1));
                if (MASS) atomicAdd(&S.hist.mass[b], w);
                atomicAdd(&S.hist.count[b], 1u);
            });
            const Cut c = find_bin<MASS>([&](u64) { return target; });
            target -= c.above, in_n = c.in_n;
            prefix = prefix << bits | (uint32_t)((1 << bits) - 1 - c.bin), known += bits;
        }
        if (in_n > kList) {  // one logit, many words: the target's word by its number
            u64 sum;
            const int owner = search([&](float x, uint32_t i) -> u64 {
                const uint32_t k = key_of(x);
                const bool on = keeps(k, i) && in(k, x);
                return MASS ? weight(x, on) : (u64)on;
            }, [&](u64) { return target - 1; }, sum);
            cluster_sync();
            const uint32_t last = (uint32_t)ld_peer(&S.found[0], (uint32_t)owner);
            cluster_sync();
            kt = prefix, it = last;
            return;
        }
        gather(in);
        if (rank == 0) {
            const int n = (int)min(S.n_list, (uint32_t)kList);
            if (MASS) weigh_list(n);
            cut_list<MASS>(n, target);
            if (threadIdx.x == 0) S.found[2] = kt, S.found[3] = it;
        }
        cluster_sync();
        kt = (uint32_t)ld_peer(&S.found[2], 0), it = (uint32_t)ld_peer(&S.found[3], 0);
        cluster_sync();
    }
    __device__ __forceinline__ void write(int row, int64_t token, u64 mass, u64 sum, uint32_t kept) {
        A.tokens[row] = (int32_t)token;
        if (A.probs) A.probs[row] = sum ? (float)((double)mass / (double)sum) : 0.0f;
        if (A.kept) A.kept[row] = (int32_t)kept;
    }
    // The first CTA's list holds every word that is left and maybe more: the rest of the row.
    __device__ __forceinline__ void finish_list(int row, u64 k, float p, u64 p_target, float min_p, float u) {
        const int n = (int)min(S.n_list, (uint32_t)kList);
        weigh_list(n);
        uint32_t count;
        if (k) cut_list<false>(n, k);
        if (p < 1.0f) {
            if (!p_target) {
                bool exact;
                const u64 t = times(sum_list(n, count), p, exact);
                p_target = max((u64)1, t + !exact);
            }
            cut_list<true>(n, p_target);
        }
        cut_min_p(min_p);
        const u64 sum = sum_list(n, count);
        bool exact;
        const u64 target = min(times(sum, u, exact), sum - 1);
        u64 above;
        const uint32_t idx = ~local_cut(
            n, [&](int e) { return ~S.list.idx[e]; }, [&](int e) { return S.list.mass[e]; },
            [&](int e) { return keeps(S.list.key[e], S.list.idx[e]); }, target + 1, above);
        for (int e = threadIdx.x; e < n; e += kThreads)
            if (S.list.idx[e] == idx) write(row, idx, S.list.mass[e], sum, count);
    }
};

__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleArgs A) {
    extern __shared__ __align__(16) float words[];
    __shared__ Shared S;
    __shared__ float red[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_rank(), row = blockIdx.x / A.cluster, first = rank * A.slice;
    const int n = max(0, min(A.slice, A.vocab - first));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const float *from = A.logits + (int64_t)row * A.row_stride + first;
    const float T = A.temperature ? A.temperature[row] : 1.0f, p = A.top_p ? A.top_p[row] : 1.0f;
    const float min_p = A.min_p ? A.min_p[row] : 0.0f, u = A.u ? A.u[row] : 0.0f;
    const int64_t k = A.top_k ? A.top_k[row] : 0;
    const float2 pow = kPow[lane];
    // the words into shared memory, and their largest
    float top = -kInf;
    bool bad = false;
    const int in_smem = min(n, A.cached);
    if (A.wide) {
#pragma unroll 8
        for (int i = 4 * tid; i + 3 < in_smem; i += 4 * kThreads) {
            const uint4 b = ld_stream_v4(from + i);
            const float4 v = make_float4(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w));
            *reinterpret_cast<float4 *>(words + i) = v;
            bad = bad || !(v.x < kInf && v.y < kInf && v.z < kInf && v.w < kInf);
            top = fmaxf(fmaxf(top, fmaxf(v.x, v.y)), fmaxf(v.z, v.w));
        }
    }
#pragma unroll 4
    for (int i = (A.wide ? in_smem / 4 * 4 : 0) + tid; i < in_smem; i += kThreads) {
        const float x = __ldg(from + i);
        words[i] = x;
        bad = bad || !(x < kInf);
        top = fmaxf(top, x);
    }
    for (int i = in_smem + tid; i < (in_smem + 3) / 4 * 4; i += kThreads) words[i] = -kInf;
#pragma unroll 4
    for (int i = A.cached + tid; i < n; i += kThreads) {
        const float x = __ldg(from + i);
        bad = bad || !(x < kInf);
        top = fmaxf(top, x);
    }
    if (tid == 0) {
        // y's factor, 32 / (T log(2)), as a pair; a temperature next to 0 leaves the largest logits only
        constexpr float C = 46.16624069213867f, Cl = 6.1630817e-07f;
        const float c = fminf(__fdiv_rn(C, T), 3e38f);
        const float rest = c < 3e38f ? __fdiv_rn(__fadd_rn(__fmaf_rn(-c, T, C), Cl), T) : 0.0f;
        S.ch = c, S.cl = rest == rest ? rest : 0.0f;
    }
    if (tid == 32 && min_p > 0.0f) S.thr = (double)T * log((double)fminf(min_p, 1.0f));
    top = warp_max(top);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) red[warp] = bad ? kInf : top;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kWarps; e++) top = fmaxf(top, red[e]);
    Row R{A, S, words, from, rank, n, first, 0.0f, S.ch, S.cl, pow.x, pow.y, kKeyNegInf + 1, 0xffffffffu};
    R.tell((u64)key_of(top));
    uint32_t best = 0;
    for (int e = 0; e < A.cluster; e++) best = max(best, (uint32_t)S.peer[e]);
    R.M = of_key(best);
    const float M = R.M;
    if (!(M < kInf) || !(M > -kInf) || !(T == T)) {  // a NaN or plus infinity, or no word at all
        if (rank == 0 && tid == 0) R.write(row, -1, 0, 0, 0);
        cluster_sync();
        return;
    }
    u64 sum = 0;
    if (!(T > 0.0f)) {  // the first of the largest
        const int owner = R.search([&](float x, uint32_t) { return (u64)(x == M); }, [](u64) { return (u64)0; }, sum);
        if (owner == rank && tid == 0) R.write(row, (int64_t)S.found[0], 1, 1, 1);
        cluster_sync();
        return;
    }
    const bool by_k = k > 0 && k < A.vocab, by_p = p < 1.0f;
    u64 k_left = 0;
    if (by_k) {
        R.fill_by_y<false>();
        const Row::Cut c = R.find_bin<false>([&](u64 total) { return min((u64)k, total); });
        k_left = min((u64)k, c.total);
        if (c.above_n + c.in_n <= kList) {
            R.gather([&](uint32_t, float x) { return R.bin_of(R.y_of(x)) <= c.bin; });
            if (rank == 0) R.finish_list(row, k_left, p, 0, min_p, u);
            return;
        }
        R.cut_in_bin<false>([&](uint32_t, float x) { return R.bin_of(R.y_of(x)) == c.bin; }, c.in_n, k_left - c.above);
    }
    if (by_p) {
        R.fill_by_y<true>();
        u64 target = 0;
        const Row::Cut c = R.find_bin<true>([&](u64 total) {
            bool exact;
            const u64 t = times(total, p, exact);
            return target = max((u64)1, t + !exact);
        });
        if (c.above_n + c.in_n <= kList) {
            R.gather([&](uint32_t, float x) { return R.bin_of(R.y_of(x)) <= c.bin; });
            if (rank == 0) R.finish_list(row, 0, p, target, min_p, u);
            return;
        }
        R.cut_in_bin<true>([&](uint32_t, float x) { return R.bin_of(R.y_of(x)) == c.bin; }, c.in_n, target - c.above);
    }
    R.cut_min_p(min_p);
    uint32_t mine = 0;
    const int owner = R.search(
        [&](float x, uint32_t i) { return R.weight(x, R.keeps(key_of(x), i)); },
        [&](u64 total) {
            bool exact;
            return min(times(total, u, exact), total - 1);
        },
        sum);
    R.words_of_warp([&](float x, uint32_t i) { mine += R.keeps(key_of(x), i); });
    mine = __reduce_add_sync(0xffffffffu, mine);
    u64 many;
    R.before(lane == 0 ? (u64)mine : 0, many);
    R.tell(many);
    many = 0;
    for (int e = 0; e < A.cluster; e++) many += S.peer[e];
    if (owner == rank && tid == 0) R.write(row, (int64_t)S.found[0], S.found[1], sum, (uint32_t)many);
    cluster_sync();  // nobody leaves while its numbers are read
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

qlin_status qlin_sample(const float *logits, int64_t row_stride, const float *u, const float *temperature,
                        const int32_t *top_k, const float *top_p, const float *min_p, int n_rows, int vocab,
                        int32_t *tokens, float *probs, int32_t *kept, qlin_stream_t stream) {
    qlin::clear_error();
    const char *fn = "qlin_sample";
    QLIN_REQUIRE(logits && u && tokens, QLIN_ERR_INVALID_ARG, "%s: null pointer", fn);
    QLIN_REQUIRE(n_rows >= 1 && vocab >= 1 && row_stride >= vocab, QLIN_ERR_INVALID_ARG,
                 "%s: n_rows %d, vocab %d, row_stride %lld", fn, n_rows, vocab, (long long)row_stride);
    QLIN_REQUIRE(n_rows <= 65535 && vocab <= kMaxVocab && row_stride < (int64_t)1 << 40, QLIN_ERR_UNSUPPORTED,
                 "%s: more than 65535 rows (%d) or 2^24 words (%d), or a row_stride of 2^40", fn, n_rows, vocab);
    QLIN_REQUIRE(aligned4(logits) && aligned4(u) && aligned4(temperature) && aligned4(top_k) && aligned4(top_p) &&
                     aligned4(min_p) && aligned4(tokens) && aligned4(probs) && aligned4(kept),
                 QLIN_ERR_INVALID_ARG, "%s: pointer not 4-byte aligned", fn);
    SampleArgs A{logits, row_stride, u, temperature, top_k, top_p, min_p, vocab, tokens, probs, kept};
    const void *kern = (const void *)sample_kernel;
    const int room = (max_smem_optin() - (int)sizeof(Shared) - 1024) / 4 / 4 * 4;  // words of a CTA in shared memory
    int c = 1;
    while (c < kMaxCluster && (vocab + c - 1) / c > 16384) c *= 2;
    size_t smem = 0;
    for (;; c /= 2) {
        A.cluster = c;
        A.slice = ((vocab + c - 1) / c + 3) / 4 * 4;
        A.cached = A.slice < room ? A.slice : room;
        smem = (size_t)A.cached * 4;
        if (c == 1) {
            blocks_per_sm(kern, smem);
            break;
        }
        if (max_clusters(kern, smem, kThreads, c) >= 1) break;
    }
    A.drop = 0;
    while (A.drop < 20 && ((int64_t)vocab >> A.drop) > 1 << 18) A.drop++;
    A.wide = aligned16(logits) && row_stride % 4 == 0;
    void *args[] = {(void *)&A};
    return launch_pdl(kern, dim3((unsigned)(n_rows * c)), dim3(kThreads), smem, (cudaStream_t)stream, args, "sample_kernel", c);
}

}  // extern "C"
