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
// rounded to nearest from what is good to 2^-29 of itself, each word's error its
// own, and sums of whole numbers do not depend on their order.  2^-y: y as a
// pair of floats in units of 1/32, its whole part split into an exponent and one
// of 32 numbers 2^(-j/32), a pair each, which the lanes of a warp hold and hand
// over by shuffles, and a series of four terms for the rest: some 35
// instructions a word.  (Two words at a time in packed fp32 took more: packed
// operations have no immediate operands, and their constants no registers left.)
//
// One cluster of CTAs per row.  The logits come from memory once: a CTA keeps its
// first 16384 words in shared memory, and those behind them, where a row is dealt
// to few CTAs, come from L2 again in every pass (three quarters of 64 rows of
// 262144 by fours, half of 256 rows of 32000).  A histogram of 2048 bins over y counts the words, or adds up their
// weights by a line through the bin, good to 10^-5; a CTA sums a share of the
// bins over the cluster's.  So top-k's
// border is known to a bin and top-p's to one or two.  Their words go to a list
// in the first CTA, which sorts it, while every thread adds up the exact weights
// of the words before them (and of all) in registers; the border is then a place
// in the list.  Where all words up to the border fit the list the first CTA does
// the rest alone.  Where a list does not hold the border (many equal logits, a
// top_p next to 1) a histogram of exact weights, and more of them over the bits
// of the logits of one bin, narrow it down.  A min-p border before top-p's ends
// the search for that.
//
// Instructions bound it, not memory: 64 rows of 262144 words with a top_p of 0.9
// take 100 us for 67 MB, about half of it the exact weights (some 60 instructions
// a word); counting, one addition to shared memory a word (8 cycles a warp), is
// the next.  256 rows of 32000 with no bound, one pass, take 30 us.  One row of
// 262144 with a top_k of 64 takes 16 us, some 32,500 cycles of its first CTA:
// 3,100 to load, 2,100 for the first meeting, 4,900 to count, 7,500 for the border
// with three meetings, 6,000 until the list is there, 8,900 to sort it and draw.
// Where a row has only a few different logits most words meet in a few bins, and
// the additions to them queue: 64 rows of 262144 words on eight levels take 4.4 ms.
#include <cmath>

#include "launch.cuh"
#include "stream.cuh"
#include "tcgen05.cuh"

namespace qlin {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 2048, kEach = kList / kThreads;  // words of the list, and of a thread
constexpr int kMaxCluster = 16;
constexpr int kCached = 16384;  // words of a CTA in shared memory, so that an SM has room for two CTAs
constexpr int kMaxVocab = 1 << 24;
constexpr float kInf = __builtin_huge_valf();
constexpr float kPart = 32.0f;               // units of y to a factor of two
constexpr float kNoWeight = 46.0f * kPart;   // y from which a weight is 0
constexpr float kMagic = 12582912.0f;        // 1.5 * 2^23: adding it rounds to a whole number
constexpr int kMagicBits = 0x4B400000;
constexpr float kMagicHi = 50331648.0f, kMagicLo = 12.0f;    // 1.5 * 2^25 and 1.5 * 2^3: to fours, and to 2^-20
constexpr int kMagicHiBits = 0x4C400000, kMagicLoBits = 0x41400000;
constexpr float kBinsPer = 1.375f;           // bins to a unit of y
constexpr float kBinPart = 0.69314718f / (kPart * kBinsPer);  // what a bin takes from a weight, as a part of it
// Logits' differences overflow fp32, and what their factor's second part is becomes too small for it, only beside a largest
// one of kFarLogit or at a temperature of kFarT and more: there everything is taken times kFar.
constexpr float kFar = 0x1p-24f, kFarLogit = 0x1p102f, kFarT = 0x1p100f;
constexpr float kNear = 2e-5f;               // how far the bins' weights may be off as a part of the sum, beside rounding

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
    float unit;          // a bin's weights as whole numbers: what the one at its middle counts
};

struct Shared {
    union {
        struct {
            u64 mass[kBins];
            uint32_t count[kBins];
        } hist;
        struct {
            u64 word[kList];  // key << 32 | ~number, so that the larger one comes first
            u64 mass[kList];
        } list;
    };
    uint32_t mine[kList];   // the CTA's own words in the list
    u64 scan[kWarps];
    u64 certain[kWarps];    // weights before the list's words
    u64 peer[2][2][kMaxCluster];  // what the CTAs tell each other, in turn
    u64 found[4];           // what a search in this CTA ends with
    u64 result[4];          // and what some CTA's ended with
    uint32_t n_list, n_mine;
    double thr;             // the least logit that min-p keeps, less the largest
    float ch[2], cl[2];     // y's factor as a pair, for h = 1 and h = kFar
    float top;              // the largest logit
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

__device__ __forceinline__ uint32_t peer_addr(const void *local, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    return a;
}
template <typename T>
__device__ __forceinline__ T ld_peer(const T *local, uint32_t rank) {
    if constexpr (sizeof(T) == 8) {
        u64 v;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer_addr(local, rank)) : "memory");
        return (T)v;
    } else {
        uint32_t v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_addr(local, rank)) : "memory");
        return (T)v;
    }
}
__device__ __forceinline__ void st_peer(u64 *local, uint32_t rank, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer_addr(local, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_peer(uint32_t *local, uint32_t rank, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(peer_addr(local, rank)), "r"(v) : "memory");
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
    float M, ch, cl;  // the largest logit, times h; y = (M - h x) (ch + cl)
    float h;          // a power of two that keeps the differences in range
    float th, tl;     // this lane's number 2^(-lane/32), times 2^24
    uint32_t kt, it;  // kept: a key above kt, or equal and a word number up to it (first: all finite ones)
    int turn = 0;

    __device__ __forceinline__ bool keeps(uint32_t k, uint32_t i) const { return k > kt || (k == kt && i <= it); }
    // (the lowest finite number may be a word's, and the cut among its equals)
    __device__ __forceinline__ bool is_cut() const { return kt != kKeyNegInf + 1 || it != 0xffffffffu; }
    __device__ __forceinline__ float y_of(float x) const { return __fmul_rn(__fmaf_rn(-h, x, M), ch); }
    __device__ __forceinline__ int bin_of(float y) const {
        return y < kNoWeight ? __float_as_int(__fmaf_rn(y, kBinsPer, kMagic)) - kMagicBits : kBins - 1;
    }
    // A word's weight and y, all lanes of the warp at once: w = (q - kMagicHiBits) 2^22 + r - kMagicLoBits.  Where y is
    // kNoWeight or more, or not a number, q and r say nothing.  value: w 2^-20 as a float.
    __device__ __forceinline__ void weigh(float x, int &q, int &r, float &y, float *value = nullptr) const {
        const float s = __fmaf_rn(-h, x, M), bb = __fsub_rn(s, M);
        const float e = __fsub_rn(__fsub_rn(M, __fsub_rn(s, bb)), __fmaf_rn(h, x, bb));  // M - h x is s + e
        y = __fmul_rn(s, ch);
        const float yl = __fmaf_rn(e, ch, __fmaf_rn(s, cl, __fmaf_rn(s, ch, -y)));
        const float t = __fadd_rn(y, kMagic);
        const float f = __fadd_rn(__fsub_rn(y, __fsub_rn(t, kMagic)), yl);  // what is left of y, up to 1/2 and a little
        const int n = __float_as_int(t);  // (kMagic's bits end in 22 zeros: n's last five are j, those before the exponent)
        const float a = __shfl_sync(0xffffffffu, th, n), al = __shfl_sync(0xffffffffu, tl, n);
        // a + al times 2^(-f/32) = 1 - g
        constexpr float k1 = 0.021660849392498290f, k2 = -k1 * k1 / 2.0f, k3 = k1 * k1 * k1 / 6.0f, k4 = -k1 * k1 * k1 * k1 / 24.0f;
        const float g = __fmul_rn(f, __fmaf_rn(f, __fmaf_rn(f, __fmaf_rn(f, k4, k3), k2), k1));
        const float lo = __fmaf_rn(-a, g, al);
        // times the power of two, in fours and the rest
        const float scale = __int_as_float(0x3f800000 - (A.drop << 23) - ((n & ~31) << 18));
        const float u = __fmul_rn(a, scale), v = __fmaf_rn(lo, scale, u), top = __fadd_rn(v, kMagicHi);
        if (value) *value = v;
        q = __float_as_int(top);
        r = __float_as_int(__fadd_rn(__fmaf_rn(lo, scale, __fsub_rn(u, __fsub_rn(top, kMagicHi))), kMagicLo));
    }
    static __device__ __forceinline__ u64 whole(int q, int r) { return (u64)((int64_t)(q - kMagicHiBits) * (1 << 22) + (r - kMagicLoBits)); }
    // one word's weight; 0 where it is not on
    __device__ __forceinline__ u64 weight(float x, bool on) const {
        int q, r;
        float y;
        weigh(x, q, r, y);
        return on && y < kNoWeight ? whole(q, r) : 0;
    }

    // f(four logits, the first one's number) of the CTA's words, warp by warp in runs of run_length words; all lanes of a
    // warp at once (words that are not there are minus infinity).  The next four are on their way meanwhile.
    template <typename F>
    __device__ __forceinline__ void words_of_warp(F f) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, run = run_length();
        const int r0 = min(n, warp * run), r1 = min(n, r0 + run);
        auto at = [&](int i) { return i < r1 ? quad(i) : make_float4(-kInf, -kInf, -kInf, -kInf); };
        float4 next = at(r0 + 4 * lane);
        for (int b = r0; b < r1; b += 128) {
            const float4 v = next;
            const int i = b + 4 * lane;
            next = at(i + 128);
            const float x[4] = {v.x, v.y, v.z, v.w};
            f(x, (uint32_t)(first + i));
        }
    }
    // A sum of weights in two parts, of up to 512 words.
    struct Sum {
        uint32_t q = 0, r = 0, n = 0;
        u64 all = 0;
        __device__ __forceinline__ void add(bool on, int qq, int rr) {
            if (on) q += (uint32_t)qq, r += (uint32_t)rr, n++;
        }
        // (behind 512 words, and before all is read)
        __device__ __forceinline__ void flush() {
            all += (u64)(q - n * (uint32_t)kMagicHiBits) * (1 << 22) + (u64)(int64_t)(int32_t)(r - n * (uint32_t)kMagicLoBits);
            q = r = n = 0;
        }
    };
    // the same with every word's weight and y: f(logit, number, kept, weighs, q, r, y); flush() every 512 words
    template <typename F, typename G>
    __device__ __forceinline__ void weights_of_warp(F f, G flush) const {
        const bool cut = is_cut();
        int left = 128;
        words_of_warp([&](const float (&x)[4], uint32_t i) {
            int q[4], r[4];
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; k++) weigh(x[k], q[k], r[k], y[k]);
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const bool on = cut ? keeps(key_of(x[k]), i + k) : x[k] > -kInf;
                f(x[k], i + k, on, on && y[k] < kNoWeight, q[k], r[k], y[k]);
            }
            if (--left == 0) flush(), left = 128;
        });
        flush();
    }
    // words i .. i + 3 (i a multiple of 4), minus infinity behind the last
    __device__ __forceinline__ float4 quad(int i) const {
        if (i < A.cached) return *reinterpret_cast<const float4 *>(words + i);
        if (A.wide && i + 3 < n) return __ldg(reinterpret_cast<const float4 *>(from + i));
        float4 v;
        v.x = __ldg(from + i);
        v.y = i + 1 < n ? __ldg(from + i + 1) : -kInf;
        v.z = i + 2 < n ? __ldg(from + i + 2) : -kInf;
        v.w = i + 3 < n ? __ldg(from + i + 3) : -kInf;
        return v;
    }

    // The CTAs tell each other two numbers (the same in all of a CTA's threads): told(0, r) and told(1, r) are CTA r's.
    // Nobody reads another's memory afterwards.  (A CTA is at most one such meeting ahead: two places in turn.)
    __device__ __forceinline__ void tell(u64 v, u64 w = 0) {
        turn++;
        if (threadIdx.x < 2 * A.cluster)
            st_peer(&S.peer[turn & 1][threadIdx.x & 1][rank], threadIdx.x >> 1, threadIdx.x & 1 ? w : v);
        cluster_sync();
    }
    __device__ __forceinline__ u64 told(int what, int r) const { return S.peer[turn & 1][what][r]; }
    // words q .. q + many - 1 of found, where this CTA has them, become result's on every CTA (behind the next meeting)
    __device__ __forceinline__ void give(bool has, int q, int many) {
        for (int e = threadIdx.x; e < many * A.cluster; e += kThreads)
            if (has) st_peer(&S.result[q + e % many], e / many, S.found[q + e % many]);
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

    __device__ __forceinline__ int run_length() const { return (A.slice + 128 * kWarps - 1) / (128 * kWarps) * 128; }
    // The first word, by number, at which the running sum of f(logit, number) exceeds want(sum over all), f called by
    // whole warps.  sums: each warp's sum of its words, in S.scan; count: words to add up beside.  Returns the CTA in
    // whose S.found the word's number is, or -1 if the sum is 0.
    template <typename F, typename W>
    __device__ __forceinline__ int find(F f, W want, u64 &sum, u64 &count) {
        u64 all = 0;
        for (int k = 0; k < kWarps; k++) all += S.scan[k];
        tell(all, count);
        sum = count = 0;
        for (int k = 0; k < A.cluster; k++) sum += told(0, k), count += told(1, k);
        if (sum == 0) return -1;
        const u64 target = want(sum);
        u64 low = 0;
        int owner = 0;
        while (owner < A.cluster - 1 && low + told(0, owner) <= target) low += told(0, owner++);
        if (owner == rank) {
            int w = 0;
            while (w < kWarps - 1 && low + S.scan[w] <= target) low += S.scan[w++];
            // the run of warp w, a stretch of words per thread
            const int run = run_length(), r0 = min(n, w * run), r1 = min(n, r0 + run);
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
                if (here && at <= target && target < at + g) S.found[0] = (u64)(first + i);
                at += g;
            }
            __syncthreads();
        }
        return owner;
    }
    // the same, the sums made first: of the weights of the kept words (and how many they are), or of f
    template <typename W>
    __device__ __forceinline__ int search_weights(W want, u64 &sum, u64 &count) {
        Sum mine;
        uint32_t many = 0;
        weights_of_warp([&](float, uint32_t, bool on, bool weighs, int q, int r, float) { mine.add(weighs, q, r), many += on; },
                        [&]() { mine.flush(); });
        sum_up(mine.all, many, count);
        return find([&](float x, uint32_t i) { return weight(x, keeps(key_of(x), i)); }, want, sum, count);
    }
    template <typename F, typename W>
    __device__ __forceinline__ int search(F f, W want, u64 &sum, u64 &count) {
        u64 mine = 0;
        words_of_warp([&](const float (&x)[4], uint32_t i) {
#pragma unroll
            for (int q = 0; q < 4; q++) mine += f(x[q], i + q);
        });
        sum_up(mine, 0, count);
        return find(f, want, sum, count);
    }
    // the warps' sums into S.scan, the CTA's words into count
    __device__ __forceinline__ void sum_up(u64 mine, uint32_t many, u64 &count) {
        mine = warp_sum(mine);
        many = __reduce_add_sync(0xffffffffu, many);
        before((threadIdx.x & 31) == 0 ? (u64)many : 0, count);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) S.scan[threadIdx.x >> 5] = mine;
        __syncthreads();
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
        const int tid = threadIdx.x, C = A.cluster, per = kBins / C, b0 = rank * per;
        // bins of a thread (four at most), or threads to a bin, each for some of the CTAs
        const int each = max(1, per / kThreads), share = max(1, kThreads / per), sub = tid & (share - 1);
        cluster_sync();
        u64 m[4], c[4], ms = 0, cs = 0;
#pragma unroll
        for (int k = 0; k < 4; k++) {
            m[k] = c[k] = 0;
            if (k >= each) continue;
            const int b = b0 + tid / share * each + k;
#pragma unroll 4
            for (int r = sub; r < C; r += share) {
                if (MASS) m[k] += ld_peer(&S.hist.mass[b], (uint32_t)r);
                c[k] += ld_peer(&S.hist.count[b], (uint32_t)r);
            }
            for (int off = 1; off < share; off <<= 1) {
                if (MASS) m[k] += __shfl_xor_sync(0xffffffffu, m[k], off);
                c[k] += __shfl_xor_sync(0xffffffffu, c[k], off);
            }
            if (sub) m[k] = c[k] = 0;
            ms += m[k], cs += c[k];
        }
        u64 mt = 0, ct;
        u64 mb = MASS ? before(ms, mt) : 0;
        u64 cb = before(cs, ct);
        tell(MASS ? mt : ct, ct);
        Cut r;
        r.total = 0;
        for (int k = 0; k < C; k++) {
            if (k < rank) mb += told(0, k), cb += told(1, k);
            r.total += told(0, k);
        }
        const u64 target = want(r.total);
        if (tid < 4) S.found[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const u64 a = MASS ? mb : cb, v = MASS ? m[k] : c[k];
            if (a < target && target <= a + v)
                S.found[0] = (u64)(b0 + tid / share * each + k) + 1, S.found[1] = a, S.found[2] = cb, S.found[3] = c[k];
            mb += m[k], cb += c[k];
        }
        __syncthreads();
        give(S.found[0] != 0, 0, 4);
        if (tid == 0) S.n_list = S.n_mine = 0;
        cluster_sync();
        r.bin = (int)S.result[0] - 1, r.above = S.result[1], r.above_n = S.result[2], r.in_n = S.result[3];
        return r;
    }
    // The bins of the words as they are counted by count_by_y: lo and hi, between which top-k's border (k > 0) or top-p's
    // must be, and the words up to hi and between; for top-p, `between` is a bound and `upto` says nothing.  Counts are
    // exact.  p is 0 .. 1, so that both borders of it are in a bin.  A word's weight is off by kBinPart^2 / 16 of itself (a line in place of 2^-y) and by half a unit, which
    // moves the border by half as much of the sum at most: what lies before it counts 1 - p times, the rest p times.
    struct Border {
        int lo, hi;
        uint32_t upto, between;
    };
    __device__ __forceinline__ Border find_border(u64 k, float p) {
        const int tid = threadIdx.x, C = A.cluster, per = kBins / C, b0 = rank * per;
        const int each = max(1, per / kThreads), share = max(1, kThreads / per), sub = tid & (share - 1);
        cluster_sync();
        u64 c[4], m[4], cs = 0, ms = 0;  // words, and weights as whole numbers of 2^-32, so that every CTA adds up the same
#pragma unroll
        for (int q = 0; q < 4; q++) {
            m[q] = c[q] = 0;
            if (q >= each) continue;
            const int b = b0 + tid / share * each + q;
            u64 v = 0;
#pragma unroll 4
            for (int r = sub; r < C; r += share) v += ld_peer(&S.hist.count[b], (uint32_t)r);
            for (int off = 1; off < share; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            if (sub || !v) continue;
            if (k) {
                c[q] = v;
            } else {
                const float units = __fdiv_rn((float)v, A.unit);
                c[q] = (u64)(units * (1.0f + kBinPart)) + 1;  // (a word counts at least 1 - kBinPart / 2)
                m[q] = (u64)(units * exp2f((float)-b / (kBinsPer * kPart)) * 4294967296.0f);
            }
            cs += c[q], ms += m[q];
        }
        u64 ct, mt = 0, mb = 0;
        u64 cb = before(cs, ct);
        if (!k) mb = before(ms, mt);
        tell(mt, ct);
        u64 mall = 0, call = 0;
        for (int q = 0; q < C; q++) {
            if (q < rank) mb += told(0, q), cb += told(1, q);
            mall += told(0, q), call += told(1, q);
        }
        k = min(k, call);
        const float want = p * (float)mall, off = (kNear + __fdiv_rn(0.5f, A.unit)) * (float)mall;
        const u64 lo_t = k ? k : (u64)fmaxf(want - off, 1.0f), hi_t = k ? k : min(mall, (u64)(want + off));
        if (tid < 4) S.found[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const u64 a = k ? cb : mb, v = k ? c[q] : m[q];
            const int b = b0 + tid / share * each + q;
            if (a < lo_t && lo_t <= a + v) S.found[0] = (u64)b + 1, S.found[1] = cb;
            if (a < hi_t && hi_t <= a + v) S.found[2] = (u64)b + 1, S.found[3] = cb + c[q];
            mb += m[q], cb += c[q];
        }
        __syncthreads();
        give(S.found[0] != 0, 0, 2);
        give(S.found[2] != 0, 2, 2);
        if (tid == 0) S.n_list = S.n_mine = 0;
        cluster_sync();
        Border r{(int)S.result[0] - 1, (int)S.result[2] - 1, 0, 0};
        r.upto = (uint32_t)S.result[3], r.between = (uint32_t)(S.result[3] - S.result[1]);
        return r;
    }
    template <bool MASS, bool COUNT>
    __device__ __forceinline__ void clear_hist() {
        __syncthreads();
        for (int b = threadIdx.x; b < kBins; b += kThreads) {
            if (MASS) S.hist.mass[b] = 0;
            if (COUNT) S.hist.count[b] = 0;
        }
        __syncthreads();
    }
    // The kept words by y: a bin's count, or the sum of its words' weights (a line through the bin) in A.unit to one at
    // its middle.  Either is one addition to shared memory, which is what bounds this.
    template <bool MASS>
    __device__ __forceinline__ void count_by_y() {
        clear_hist<false, true>();
        uint32_t rest = 0;
        const bool cut = is_cut();
        const float slope = -kBinPart * A.unit, middle = kMagic + rintf(A.unit * (1.0f + kBinPart * kBinPart / 16.0f));
        words_of_warp([&](const float (&x)[4], uint32_t i) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const bool on = cut ? keeps(key_of(x[q]), i + q) : x[q] > -kInf;
                const float y = y_of(x[q]);
                if (!on || !(y < kNoWeight)) {
                    rest += on;  // (those of no weight, which may be most)
                    continue;
                }
                const float t = __fmaf_rn(y, kBinsPer, kMagic);  // (as bin_of)
                const int b = __float_as_int(t) - kMagicBits;
                if (MASS) {
                    const float g = __fmaf_rn(y, kBinsPer, -__fsub_rn(t, kMagic));  // -1/2 .. 1/2 of the bin
                    atomicAdd(&S.hist.count[b], (uint32_t)(__float_as_int(__fmaf_rn(g, slope, middle)) - kMagicBits));
                } else {
                    atomicAdd(&S.hist.count[b], 1u);
                }
            }
        });
        if (MASS) return;
        rest = __reduce_add_sync(0xffffffffu, rest);
        if ((threadIdx.x & 31) == 0 && rest) atomicAdd(&S.hist.count[kBins - 1], rest);
    }
    // the kept words' exact weights by y
    __device__ __forceinline__ void weigh_by_y() {
        clear_hist<true, true>();
        uint32_t rest = 0;
        weights_of_warp([&](float, uint32_t, bool on, bool weighs, int q, int r, float y) {
            if (weighs) {
                const int b = bin_of(y);
                atomicAdd(&S.hist.mass[b], whole(q, r));
                atomicAdd(&S.hist.count[b], 1u);
            } else {
                rest += on;
            }
        }, []() {});
        rest = __reduce_add_sync(0xffffffffu, rest);
        if ((threadIdx.x & 31) == 0 && rest) atomicAdd(&S.hist.count[kBins - 1], rest);
    }
    // A word of this CTA's into the first CTA's list.  (find_bin and find_border leave the list empty, and the histogram's
    // place free; a meeting of the CTAs closes it.)
    __device__ __forceinline__ void enlist(uint32_t k, uint32_t i) {
        const uint32_t at = add_peer(&S.n_list, 0, 1), own = atomicAdd(&S.n_mine, 1u);
        if (at < kList) st_peer(&S.list.word[at], 0, (u64)k << 32 | (uint32_t)~i);
        if (own < kList) S.mine[own] = i;
    }
    // the kept words that sel(key, logit) takes
    template <typename F>
    __device__ __forceinline__ void gather(F sel) {
        words_of_warp([&](const float (&x)[4], uint32_t i) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const uint32_t k = key_of(x[q]);
                if (keeps(k, i + q) && sel(k, x[q])) enlist(k, i + q);
            }
        });
        cluster_sync();
    }

    // ---------------------------------------------------------------- the first CTA's list
    // n words, all different, sorted, the largest first.  Up to 128 every word's place is counted, by four threads; more go through a network, in which a
    // warp's 32 pairs of a step up to 32 words apart lie in 64 words of its own.  (70 words: 0.3 us against 1.4.)
    __device__ __forceinline__ void sort(u64 *w, int n) const {
        const int tid = threadIdx.x;
        __syncthreads();
        if (n <= 128) {
            const int e = tid >> 2;
            const u64 mine = e < n ? w[e] : 0;
            int place = 0;
            for (int i = tid & 3; i < n; i += 4) place += w[i] > mine;
            place += __shfl_xor_sync(0xffffffffu, place, 1);
            place += __shfl_xor_sync(0xffffffffu, place, 2);
            __syncthreads();
            if (e < n && (tid & 3) == 0) w[place] = mine;
            __syncthreads();
            return;
        }
        const int P = 1 << (32 - __clz(n - 1));
        for (int e = n + tid; e < P; e += kThreads) w[e] = 0;  // (behind every word)
        for (int k = 2; k <= P; k <<= 1)
            for (int j = k >> 1; j > 0; j >>= 1) {
                if (j >= 32 || (k == 2))
                    __syncthreads();
                else
                    __syncwarp();
                for (int t = tid; t < P / 2; t += kThreads) {
                    const int a = ((t & ~(j - 1)) << 1) | (t & (j - 1)), b = a | j;
                    const u64 x = w[a], y = w[b];
                    if ((x < y) == ((a & k) == 0)) w[a] = y, w[b] = x;
                }
            }
        __syncthreads();
    }
    // The first n words of the list sorted; returns n.
    __device__ __forceinline__ int sort_list() {
        const int n = (int)min(S.n_list, (uint32_t)kList);
        sort(S.list.word, n);
        return n;
    }
    // The weights of the sorted list's first `n` words, and the sums up to and with each, in S.list.mass.
    __device__ __forceinline__ u64 sums_of_list(int n) {
        const int e = kEach * threadIdx.x;
        u64 w[kEach] = {}, mine = 0, total;
        if (kEach * (threadIdx.x & ~31) < n)  // (whole warps)
#pragma unroll
            for (int q = 0; q < kEach; q++) {
                w[q] = weight(e + q < n ? of_key((uint32_t)(S.list.word[e + q] >> 32)) : -kInf, e + q < n);
                mine += w[q];
            }
        u64 at = before(mine, total);
#pragma unroll
        for (int q = 0; q < kEach; q++) S.list.mass[e + q] = at += w[q];
        __syncthreads();
        return total;
    }
    // how many of the list's first n sums are below target
    __device__ __forceinline__ int below(int n, u64 target) {
        const int e = kEach * threadIdx.x;
        u64 mine = 0, total;
#pragma unroll
        for (int q = 0; q < kEach; q++) mine += e + q < n && S.list.mass[e + q] < target;
        before(mine, total);
        return (int)total;
    }

    // ---------------------------------------------------------------- the parts of a row
    // the least logit that min-p keeps
    __device__ __forceinline__ float floor_of(float min_p) const {
        if (!(min_p > 0.0f) || ch == 0.0f) return -kInf;  // (at an infinite temperature all weigh the same)
        const float top = S.top;
        const double t = (double)top + S.thr;
        float x = (float)t;
        if ((double)x < t) x = nextafterf(x, kInf);
        return fminf(x, top);
    }
    // min-p's cut
    __device__ __forceinline__ void cut_min_p(float min_p) {
        const uint32_t k = key_of(floor_of(min_p));
        if (k > kt) kt = k, it = 0xffffffffu;
    }
    // kt and it from the place in the first CTA's list behind which it is cut, on every CTA; a place below 0: not there
    __device__ __forceinline__ bool cut_at(int place) {
        if (rank == 0) {
            if (threadIdx.x == 0) {
                const u64 w = place >= 0 ? S.list.word[place] : 0;
                S.found[0] = w >> 32, S.found[1] = (uint32_t)~w;
            }
            __syncthreads();
            give(true, 0, 2);
        }
        cluster_sync();
        const uint32_t k = (uint32_t)S.result[0], i = (uint32_t)S.result[1];
        if (!k) return false;
        kt = k, it = i;
        return true;
    }
    // In a bin of `in_n` kept words (those that sel takes), the cut where the running sum reaches target.
    template <bool MASS, typename F>
    __device__ __forceinline__ void cut_in_bin(F sel, u64 in_n, u64 target) {
        uint32_t prefix = 0;
        int known = 0;  // of a key's bits
        auto in = [&](uint32_t k, float x) { return sel(k, x) && (known == 0 || (k >> (32 - known)) == prefix); };
        while (in_n > kList && known < 32) {
            const int bits = known == 22 ? 10 : 11, sh = 32 - known - bits;
            clear_hist<true, true>();
            weights_of_warp([&](float x, uint32_t, bool on, bool weighs, int q, int r, float) {
                const uint32_t k = key_of(x);
                if (!on || !in(k, x)) return;
                const int b = (1 << bits) - 1 - (int)((k >> sh) & ((1u << bits) - 1));
                if (MASS && weighs) atomicAdd(&S.hist.mass[b], whole(q, r));
                atomicAdd(&S.hist.count[b], 1u);
            }, []() {});
            const Cut c = find_bin<MASS>([&](u64) { return target; });
            target -= c.above, in_n = c.in_n;
            prefix = prefix << bits | (uint32_t)((1 << bits) - 1 - c.bin), known += bits;
        }
        if (in_n > kList) {  // one logit, many words: the target's word by its number
            u64 sum, many;
            const int owner = search([&](float x, uint32_t i) -> u64 {
                const uint32_t k = key_of(x);
                const bool on = keeps(k, i) && in(k, x);
                return MASS ? weight(x, on) : (u64)on;
            }, [&](u64) { return target - 1; }, sum, many);
            give(owner == rank, 0, 1);
            cluster_sync();
            kt = prefix, it = (uint32_t)S.result[0];
            return;
        }
        gather(in);
        int place = -1;
        if (rank == 0) {
            const int n = sort_list();
            if (MASS) sums_of_list(n);
            place = MASS ? below(n, target) : (int)target - 1;
        }
        cut_at(place);
    }
    __device__ __forceinline__ void write(int row, int64_t token, float prob, u64 kept) const {
        if (threadIdx.x) return;
        A.tokens[row] = (int32_t)token;
        if (A.probs) A.probs[row] = prob;
        if (A.kept) A.kept[row] = (int32_t)kept;
    }
    // the token, the logit x of it, the sum of the weights and the words left; whole warps
    __device__ __forceinline__ void write(int row, int64_t token, float x, u64 sum, u64 kept) const {
        int q, r;
        float y, v;
        weigh(x, q, r, y, &v);  // (a small weight has few bits as a whole number)
        v = __fmul_rn(v, 1048576.0f);
        const float hi = __ull2float_rn(sum), lo = (float)((int64_t)sum - (int64_t)hi), p = __fdiv_rn(v, hi);
        write(row, token, __fadd_rn(p, __fdiv_rn(__fmaf_rn(-p, lo, __fmaf_rn(-p, hi, v)), hi)), kept);
    }
    // The first CTA's list holds top-k's k words (or all there are) and maybe more: the rest of the row.
    __device__ __forceinline__ void finish_list(int row, u64 k, float p, float min_p, float u) {
        int n = sort_list();
        if (k < (u64)n) n = (int)k;
        u64 total = sums_of_list(n);
        bool exact;
        if (p < 1.0f) {
            const u64 t = times(total, p, exact);
            n = min(n, below(n, max((u64)1, t + !exact)) + 1);
        }
        cut_min_p(min_p);
        if (min_p > 0.0f) {
            u64 mine = 0, many;
#pragma unroll
            for (int q = 0; q < kEach; q++) {
                const int at = kEach * threadIdx.x + q;
                const u64 w = at < n ? S.list.word[at] : 0;
                mine += at < n && keeps((uint32_t)(w >> 32), (uint32_t)~w);
            }
            before(mine, many);
            n = (int)many;
        }
        const u64 sum = S.list.mass[n - 1], target = min(times(sum, u, exact), sum - 1);
        // the words that are left in the order of their numbers: ~number << 32 | place
        const int e = kEach * threadIdx.x;
        u64 *const order = S.list.word;
        u64 o[kEach];
#pragma unroll
        for (int q = 0; q < kEach; q++) o[q] = e + q < n ? S.list.word[e + q] << 32 | (uint32_t)(e + q) : 0;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kEach; q++)
            if (e + q < n) order[e + q] = o[q];
        sort(order, n);
        u64 mine = 0;
#pragma unroll
        for (int q = 0; q < kEach; q++) {
            o[q] = 0;  // (the word's weight)
            if (e + q < n) {
                const int at = (int)(uint32_t)order[e + q];
                o[q] = S.list.mass[at] - (at ? S.list.mass[at - 1] : 0);
            }
            mine += o[q];
        }
        u64 at = before(mine, total);
#pragma unroll
        for (int q = 0; q < kEach; q++) {
            if (at <= target && target < at + o[q]) S.found[0] = (uint32_t)~(uint32_t)(order[e + q] >> 32);
            at += o[q];
        }
        __syncthreads();
        write(row, (int64_t)S.found[0], __ldg(from + S.found[0]), sum, (u64)n);  // (the first CTA's words are the row's)
    }
};

__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs A) {
    extern __shared__ __align__(16) float words[];
    __shared__ Shared S;
    __shared__ float red[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_rank(), row = blockIdx.x / A.cluster, first = rank * A.slice;
    const int n = max(0, min(A.slice, A.vocab - first));
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (this CTA is there)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const float *from = A.logits + (int64_t)row * A.row_stride + first;
    const float T = A.temperature ? A.temperature[row] : 1.0f, given_p = A.top_p ? A.top_p[row] : 1.0f;
    const float p = given_p < 0.0f ? 0.0f : given_p;  // (the border is then at the first word; a NaN stays one: no border)
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
    const int vectors = A.wide && n > A.cached ? A.cached + (n - A.cached) / 4 * 4 : A.cached;
#pragma unroll 8
    for (int i = A.cached + 4 * tid; i < vectors; i += 4 * kThreads) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(from + i));
        bad = bad || !(v.x < kInf && v.y < kInf && v.z < kInf && v.w < kInf);
        top = fmaxf(fmaxf(top, fmaxf(v.x, v.y)), fmaxf(v.z, v.w));
    }
#pragma unroll 4
    for (int i = vectors + tid; i < n; i += kThreads) {
        const float x = __ldg(from + i);
        bad = bad || !(x < kInf);
        top = fmaxf(top, x);
    }
    if (tid < 2) {
        // y's factor, 32 / (T log(2)), as a pair; a temperature next to 0 leaves the largest logits only
        constexpr float C = 46.16624069213867f, Cl = 6.1630817e-07f;
        const float Th = tid ? __fmul_rn(T, kFar) : T, c = fminf(__fdiv_rn(C, Th), 3e38f);
        const float rest = c < 3e38f ? __fdiv_rn(__fadd_rn(__fmaf_rn(-c, Th, C), Cl), Th) : 0.0f;
        S.ch[tid] = c, S.cl[tid] = rest == rest ? rest : 0.0f;
    }
    if (tid == 32 && min_p > 0.0f) S.thr = (double)T * log((double)fminf(min_p, 1.0f));
    top = warp_max(top);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) red[warp] = bad ? kInf : top;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kWarps; e++) top = fmaxf(top, red[e]);
    Row R{A, S, words, from, rank, n, first, 0.0f, 0.0f, 0.0f, 0.0f, pow.x, pow.y, kKeyNegInf + 1, 0xffffffffu};
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // (all are: their memory may be written)
    R.tell((u64)key_of(top));
    uint32_t best = 0;
    for (int e = 0; e < A.cluster; e++) best = max(best, (uint32_t)R.told(0, e));
    const float M = of_key(best);
    S.top = M;  // (all threads the same)
    const int far = M > kFarLogit || T > kFarT;
    R.h = far ? kFar : 1.0f;
    R.M = __fmul_rn(M, R.h), R.ch = S.ch[far], R.cl = S.cl[far];
    if (!(M < kInf) || !(M > -kInf) || !(T == T)) {  // a NaN or plus infinity, or no word at all
        if (rank == 0) R.write(row, -1, 0.0f, 0);
        return;
    }
    u64 sum = 0, many = 0;
    bool exact;
    auto drawn = [&](u64 total) { return min(times(total, u, exact), total - 1); };
    if (!(T > 0.0f)) {  // the first of the largest
        const int owner = R.search([&](float x, uint32_t) { return (u64)(x == M); }, [](u64) { return (u64)0; }, sum, many);
        if (owner == rank) R.write(row, (int64_t)S.found[0], 1.0f, 1);
        return;
    }
    const bool by_k = k > 0 && k < A.vocab, by_p = p < 1.0f;
    if (by_k) {
        R.count_by_y<false>();
        const Row::Border c = R.find_border((u64)k, 0.0f);
        auto bin = [&](float x) { return R.bin_of(R.y_of(x)); };
        if (c.upto <= kList) {
            R.gather([&](uint32_t, float x) { return bin(x) <= c.hi; });
            if (rank == 0) R.finish_list(row, (u64)k, p, min_p, u);
            return;
        }
        // (fewer words than k: all of them stay)
        const u64 above = c.upto - c.between;
        if (c.upto >= k) R.cut_in_bin<false>([&](uint32_t, float x) { return bin(x) == c.hi; }, c.between, (u64)k - above);
    }
    auto kept_weight = [&](float x, uint32_t i) { return R.weight(x, R.keeps(key_of(x), i)); };
    bool summed = false;  // S.scan holds the warps' sums of what is left, many the CTA's words
    if (by_p) {
        R.count_by_y<true>();
        const float floor_x = R.floor_of(min_p);
        const Row::Border c = R.find_border(0, p);
        // (where min-p keeps words of bins before the border's only, top-p takes none of them)
        bool done = floor_x > -kInf && R.bin_of(R.y_of(floor_x)) < c.lo;
        if (!done && c.between <= kList) {
            // the exact weights of the words before the list's, and of all
            Row::Sum before, all;
            u64 total, ahead;
            uint32_t ahead_n = 0;
            R.weights_of_warp([&](float x, uint32_t i, bool, bool weighs, int q, int r, float y) {
                const int b = R.bin_of(y);
                all.add(weighs, q, r);
                before.add(weighs && b < c.lo, q, r);
                if (weighs && (uint32_t)(b - c.lo) <= (uint32_t)(c.hi - c.lo)) R.enlist(key_of(x), i);
            }, [&]() { all.flush(), ahead_n += before.n, before.flush(); });
            cluster_sync();
            const u64 ahead_w = warp_sum(before.all);
            if (lane == 0) S.certain[warp] = ahead_w;
            ahead_n = __reduce_add_sync(0xffffffffu, ahead_n);
            u64 counted;
            R.before(all.all, total);
            R.before(lane == 0 ? (u64)ahead_n : 0, counted);
            u64 own = 0;
            for (int e = 0; e < kWarps; e++) own += S.certain[e];
            R.tell(total, own);
            total = ahead = 0;
            for (int e = 0; e < A.cluster; e++) total += R.told(0, e), ahead += R.told(1, e);
            const u64 t = times(total, p, exact), target = max((u64)1, t + !exact);
            int place = -1;
            if (rank == 0) {
                const int m = R.sort_list();
                const u64 in_list = R.sums_of_list(m);
                if (ahead < target && target <= ahead + in_list) place = R.below(m, target - ahead);
            }
            done = R.cut_at(place);
            if (done) {
                // the warps' sums of what is left: the words before, and those of the CTA's own in the list
                summed = floor_x == -kInf || R.bin_of(R.y_of(floor_x)) > c.hi;
                if (summed) {
                    const int run = R.run_length(), own_n = (int)min(S.n_mine, (uint32_t)kList);
                    __syncthreads();
                    if (tid < kWarps) S.scan[tid] = S.certain[tid];
                    __syncthreads();
                    u64 left = 0;
                    for (int e = tid; e - lane < own_n; e += kThreads) {
                        const uint32_t i = e < own_n ? S.mine[e] : 0;
                        const int at = (int)(i - (uint32_t)first);
                        const float x = e < own_n ? (at < A.cached ? words[at] : __ldg(from + at)) : -kInf;
                        const bool on = e < own_n && R.keeps(key_of(x), i);
                        const u64 w = R.weight(x, on);
                        if (on) atomicAdd(&S.scan[at / run], w), left++;
                    }
                    u64 in_list;
                    // (before() uses S.scan)
                    __syncthreads();
                    const u64 mine = tid < kWarps ? S.scan[tid] : 0;
                    R.before(left, in_list);
                    __syncthreads();
                    if (tid < kWarps) S.scan[tid] = mine;
                    __syncthreads();
                    many = counted + in_list;
                }
            }
        }
        if (!done) {
            R.weigh_by_y();
            u64 target = 0;
            const Row::Cut b = R.find_bin<true>([&](u64 total) {
                const u64 t = times(total, p, exact);
                return target = max((u64)1, t + !exact);
            });
            R.cut_in_bin<true>([&](uint32_t, float x) { return R.bin_of(R.y_of(x)) == b.bin; }, b.in_n, target - b.above);
        }
    }
    R.cut_min_p(min_p);
    const int owner = summed ? R.find(kept_weight, drawn, sum, many) : R.search_weights(drawn, sum, many);
    if (owner == rank) R.write(row, (int64_t)S.found[0], __ldg(from + (S.found[0] - (u64)first)), sum, many);
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
    // As many CTAs to a row as give two to every SM, for no fewer than 4096 words each.  (Rows past what the cluster's
    // shared memory holds come from L2 again in every pass: 64 rows of 262144 words take 100 us by fours and 200
    // by sixteens, of which 11 run at a time, one after the other.)
    int c = 1;
    while (c < kMaxCluster && (int64_t)n_rows * c * 2 <= 2 * sm_count() && vocab / c > 4096) c *= 2;
    size_t smem = 0;
    for (;; c /= 2) {
        A.cluster = c;
        A.slice = ((vocab + c - 1) / c + 3) / 4 * 4;
        A.cached = A.slice < kCached ? A.slice : kCached;
        smem = (size_t)A.cached * 4;
        if (c == 1) {
            blocks_per_sm(kern, smem);
            break;
        }
        if (max_clusters(kern, smem, kThreads, c) >= 1) break;
    }
    A.drop = 0;
    while (((int64_t)(vocab - 1) >> A.drop) >= 1 << 18) A.drop++;
    A.wide = aligned16(logits) && row_stride % 4 == 0;
    A.unit = (float)std::fmin(65000.0, std::floor(4.2e9 / A.slice));  // all of a CTA's words in one bin fit 32 bits
    void *args[] = {(void *)&A};
    return launch_pdl(kern, dim3((unsigned)(n_rows * c)), dim3(kThreads), smem, (cudaStream_t)stream, args, "sample_kernel", c);
}

}  // extern "C"
