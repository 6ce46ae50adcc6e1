// Beam search over many sequences: the selection over beams and vocabulary
// (qlin_beam_select) and the reordering of the beams' states that follows it
// (qlin_beam_reorder).
//
// Selection.  A live beam b of a group with running score s_b and logits x_b
// offers the candidates c(b, v) = s_b + x_b[v] - lse_b, lse_b = log sum_v
// exp(x_b[v]); a finished beam offers itself alone, with its score and the
// end token.  The n largest of a group come out in descending order, ties to
// the lower b * vocab + v.
//
// Two launches.  beam_slice_kernel reads every logit once: a CTA walks a slice
// of one beam's row, a few thousand values in registers at a time with the next
// ones in flight, sums the exponentials and keeps the values that can be among
// the slice's n largest logits (inside a beam the order of the candidates is
// the order of the logits).  What can be is told by a threshold from the
// largest values of a warp's threads so far, in order (sel_kth).
// beam_merge_kernel, one CTA per group, adds the sums up and takes the n best
// of the slices' sorted lists, again by a threshold (on the lists' heads)
// first.
//
// 4 beams of 262144 words (4.2 MB): 10.1 us; the slices' two tiles each and
// the merge are 4 us each, chains of a few dozen steps.  8 groups of 8 beams (59
// MB): 24 us from L2, 26 from memory (2.2 TB/s, a third of a measured copy).  The
// slices take 18 of them, and nothing is full: half of the issue slots (330
// instructions per warp and 512 values), a third of the memory's rate, the warps
// mostly waiting for their next values (a ring in shared memory with two tiles on
// their way gave 0.5 us here and cost 1 us on the small case, prefetching to L2
// nothing).  Slices are dealt out over all rows: those of dead and finished beams
// end at once, and the others get no more for it.
//
// Masks of minus infinity cost nothing (64 rows with 40 words left: 19 to 26 us).
// With finite ones, the type's lowest value or -1e4, every masked word of a slice
// without n others is a candidate as good as the next: the buffer overflows, the
// slice is walked again with care, and the same 64 rows take 450 to 870 us.
//
// Two beams' candidates can lie closer together than fp32 resolves, so lse
// and the candidates are held as pairs of floats (48 bits; fp64 instructions
// take 16 cycles per warp here), and in fp64 only where a beam's numbers are
// too large for pairs.  The sum's parts are exact to scale: a
// slice sums 2^(x log2(e) - e) with a whole number e that follows from its
// largest logit, so slices are brought to one scale by powers of two.  (Logits
// beyond 2^24, where masks of the type's lowest value lie, take the slice's
// largest logit itself as the scale.)  Each term is one fp32 exp2 (relative error
// about 2^-22); the terms of a thread's tile, 16 at most, are summed in fp32 (2^-21
// at most) and pairs from there, since equal terms all round the same way and a
// longer sum would be off the more the longer it is.
//
// Reordering.  new[b] = old[parent[b]] for every beam that does not keep its
// place, in place: a CTA brings the same stretch of every beam that is wanted
// elsewhere into shared memory by bulk copies, and once all have landed writes
// it to every beam that takes it by bulk stores.  Stretches are disjoint, so
// the order in which CTAs run does not matter, each wanted byte is read once,
// and beams that stay cost nothing.  64 beams of 13 MB in four groups (1.22 GB
// read and written): 194 us, 6.3 TB/s, 94% of a measured copy; four beams of 2.7
// MB, three of them moved (10.6 MB, from L2): 4.2 us.
#include "launch.cuh"
#include "stream.cuh"
#include "tcgen05.cuh"

namespace qlin {
namespace {

constexpr int kMaxBeams = 64;
constexpr int kMaxOut = 128;

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 256, kSelPerSm = 3;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBuf = 1024;  // candidates of a slice in shared memory

// fp32 as an unsigned whole number in the same order
__device__ __forceinline__ uint32_t ord32(float v) {
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unord32(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// larger value first, then the lower index (+ 0: no negative zeros)
__device__ __forceinline__ uint64_t cand_key(float v, uint32_t idx) {
    return ((uint64_t)ord32(__fadd_rn(v, 0.0f)) << 32) | (uint32_t)~idx;
}

constexpr uint32_t kOrdNegInf = 0x007fffffu;  // ord32(-inf); anything above it is a candidate

struct SelPart {  // a slice's part of its beam's sum of exponentials
    float sum, lo;  // sum + lo, times 2^sel_exp(m), or times exp(m) where sel_wide(m)
    float m;        // the slice's largest logit
    int count;      // candidates listed
};
static_assert(sizeof(SelPart) == 16, "read as one vector");
constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654323148236e-9f;
constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.9259629911266175e-8f;
__device__ __forceinline__ bool sel_wide(float m) { return !(fabsf(m) <= 16777216.0f); }
__device__ __forceinline__ float sel_exp(float m) { return ceilf(__fmul_rn(m, kLog2eHi)); }

struct SelWs {
    SelPart *part;  // [rows][S]
    uint64_t *cand; // [rows][S][n], descending keys
    size_t bytes;
};

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

SelWs carve_sel(int rows, int S, int n, char *base) {
    SelWs w{};
    const size_t a = align256(sizeof(SelPart) * (size_t)rows * S);
    w.part = (SelPart *)base;
    w.cand = (uint64_t *)(base ? base + a : nullptr);
    w.bytes = a + align256(8 * (size_t)rows * S * n);
    return w;
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two at once
__device__ __forceinline__ uint64_t bits2(float2 v) {
    return (uint64_t)__float_as_uint(v.y) << 32 | __float_as_uint(v.x);
}
__device__ __forceinline__ float2 floats2(uint64_t b) {
    return make_float2(__uint_as_float((uint32_t)b), __uint_as_float((uint32_t)(b >> 32)));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return floats2(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
    return floats2(d);
}

__device__ __forceinline__ bool beam_live(const float *scores, const uint8_t *finished, int row) {
    return !(finished && finished[row]) && scores[row] > -__int_as_float(0x7f800000);
}

// Two floats as one number of twice the digits: h + l += oh + ol, with the
// rounding of h + oh kept in l (fp64 costs 16 cycles per instruction and warp
// here, and stalls what depends on it for longer).
__device__ __forceinline__ void pair_add(float &h, float &l, float oh, float ol) {
    const float t = __fadd_rn(h, oh), z = __fsub_rn(t, h);
    l = __fadd_rn(__fadd_rn(l, ol), __fadd_rn(__fsub_rn(h, __fsub_rn(t, z)), __fsub_rn(oh, z)));
    h = t;
}
__device__ __forceinline__ void pair_warp_sum(float &h, float &l) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        pair_add(h, l, __shfl_xor_sync(0xffffffffu, h, off), __shfl_xor_sync(0xffffffffu, l, off));
}

// A slice's candidates so far, in shared memory.
struct SelBuf {
    uint64_t key[kSelBuf];
    int count;
};

// The place of key `mine` (and `tie`, smaller first) among c keys: the number
// of larger ones (self: it is among them).  The high words tell nearly all of
// them apart.
template <typename Tie>
__device__ __forceinline__ int place_of(uint64_t mine, Tie tie, bool self, const uint64_t *key, const Tie *ties, int c) {
    const uint32_t hi = (uint32_t)(mine >> 32);
    const uint32_t *his = reinterpret_cast<const uint32_t *>(key) + 1;
    int r = 0, eq = 0;
#pragma unroll 8
    for (int q = 0; q < c; q++) {
        const uint32_t h = his[2 * q];
        r += h > hi;
        eq += h == hi;
    }
    if (eq > (int)self)
        for (int q = 0; q < c; q++) {
            const uint64_t k = key[q];
            if ((uint32_t)(k >> 32) == hi && (k > mine || (k == mine && ties[q] < tie))) r++;  // (not itself)
        }
    return r;
}

// The n largest of the c (<= kSelBuf) keys of b to out, in descending order
// (keys are unique); four threads count for a key.
__device__ __forceinline__ void sel_rank(const SelBuf &b, int c, int n, uint64_t *out) {
    const int part = threadIdx.x & 3, per = (c + 3) / 4, j0 = min(part * per, c), j1 = min(j0 + per, c);
    for (int i0 = 0; i0 < c; i0 += kSelThreads / 4) {
        const int i = i0 + ((int)threadIdx.x >> 2);
        uint64_t key = 0;
        int r = 0;
        if (i < c) {
            key = b.key[i];
            r = place_of<uint64_t>(key, 0, i >= j0 && i < j1, b.key + j0, b.key, j1 - j0);
        }
        r += __shfl_xor_sync(0xffffffffu, r, 1);
        r += __shfl_xor_sync(0xffffffffu, r, 2);
        if (i < c && part == 0 && r < n) out[r] = key;
    }
}

// A value that n of the block's threads' `mine` are no smaller than: with
// k = ceil(n / warps) and j = ceil(n / k), the j-th largest of the warps' k-th
// largest.  A warp's k-th largest only grows, so any of its
// published values will do (one of an earlier walk over the slice would too).
__device__ __forceinline__ void sel_kth(uint32_t mine, int k, uint32_t *wkth) {
    const int lane = threadIdx.x & 31;
    uint32_t kth = 0;
    for (int r = 0; r < k; r++) {
        kth = __reduce_max_sync(0xffffffffu, mine);
        const uint32_t who = __ballot_sync(0xffffffffu, mine == kth);
        if (lane == __ffs(who) - 1) mine = 0;
    }
    if (lane == 0) *(volatile uint32_t *)&wkth[threadIdx.x >> 5] = kth;
}
__device__ __forceinline__ uint32_t sel_threshold(const uint32_t *wkth, int j) {
    const int own = threadIdx.x & (kSelWarps - 1);
    // (other warps may be writing: each value is read once)
    const uint32_t mine = *(volatile const uint32_t *)&wkth[own];
    int above = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; w++) {
        const uint32_t other = __shfl_sync(0xffffffffu, mine, w);
        above += other > mine || (other == mine && w < own);
    }
    const uint32_t who = __ballot_sync(0xffffffffu, above == j - 1);
    return __shfl_sync(0xffffffffu, mine, __ffs(who) - 1);
}

// grid (S, rows): slice blockIdx.x of a row is the values from blockIdx.x * len
// on, `len` of them (a multiple of 4), taken in tiles of 256 VPT: thread t
// holds 16-byte groups t, t + 256, ... with VEC (rows 16-byte aligned), single
// values t, t + 256, ... without.
template <int VPT, bool VEC>
__global__ void __launch_bounds__(kSelThreads, kSelPerSm)
    beam_slice_kernel(const float *__restrict__ logits, int64_t row_stride, const float *__restrict__ scores,
                      const uint8_t *__restrict__ finished, int V, int len, int n, SelPart *part, uint64_t *cand) {
    constexpr int kTile = kSelThreads * VPT;
    __shared__ float wmax[kSelWarps];
    __shared__ float2 wsum[kSelWarps];
    __shared__ uint32_t wkth[kSelWarps];
    __shared__ SelBuf buf, last;
    __shared__ uint64_t best[kMaxOut];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.y, S = gridDim.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!beam_live(scores, finished, row)) return;  // (the merge skips its parts)
    const float ninf = -__int_as_float(0x7f800000);
    const int v0 = blockIdx.x * len, v1 = min(v0 + len, V);
    const float *x = logits + (int64_t)row * row_stride;
    auto index = [&](int j) { return VEC ? ((j >> 2) * kSelThreads + tid) * 4 + (j & 3) : j * kSelThreads + tid; };
    auto load = [&](int at, float (&v)[VPT]) {
        // (the loads of a whole tile are predicated, not branched to: none is waited for before the next is out)
        const bool whole = at + kTile <= v1;
        if (!whole)
#pragma unroll
            for (int j = 0; j < VPT; j++) {
                const int i = at + index(j);
                v[j] = i < v1 ? x[i] : ninf;
            }
#pragma unroll
        for (int j = 0; j < VPT; j += VEC ? 4 : 1) {
            if constexpr (VEC)
                asm volatile(
                    "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p ld.global.cs.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
                    : "+f"(v[j]), "+f"(v[j + 1]), "+f"(v[j + 2]), "+f"(v[j + 3])
                    : "l"(x + at + index(j)), "r"((uint32_t)whole));
            else
                asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.cs.f32 %0, [%1];\n\t}"
                             : "+f"(v[j])
                             : "l"(x + at + index(j)), "r"((uint32_t)whole));
        }
    };
    float v[VPT], nx[VPT];
    float m, sum, rest;  // this thread's largest value and its sum (sum + rest) times 2^e
    int e, c;
    uint32_t thr;  // n values of the slice so far are no smaller (minus infinity is no candidate)
    const int k = (n + kSelWarps - 1) / kSelWarps, jw = (n + k - 1) / k;  // k at most 16
    const bool many = n > 32;
    if (tid == 0) last.count = 0;
    // Once without looking at the buffer after every tile; where that let it
    // overflow (many equal values) once more, carefully.
    for (bool careful = false;; careful = true) {
        load(v0, v);
        if (tid == 0) buf.count = 0;
        m = ninf, sum = rest = 0.0f, e = -(1 << 28);
        thr = kOrdNegInf + 1;
        bool over = false;
        int tile = 0;
        for (int at = v0; at < v1 && !over; at += kTile, tile++) {
            if (at + kTile < v1) load(at + kTile, nx);
            float tmax = ninf, gmax[VPT / 4];
#pragma unroll
            for (int u = 0; u < VPT / 4; u++) {
                gmax[u] = fmaxf(fmaxf(v[4 * u], v[4 * u + 1]), fmaxf(v[4 * u + 2], v[4 * u + 3]));
                tmax = fmaxf(tmax, gmax[u]);
            }
            if (tmax > m) {
                m = tmax;
                // a whole-number scale at or above the largest term's exponent
                const int ne = (int)fminf(fmaxf(sel_exp(m), -1e8f), 1e8f);
                if (ne > e) {
                    const float f = pow2i(max(e - ne, -126));
                    sum *= f, rest *= f, e = ne;
                }
            }
            // x log2(e) - e with log2(e) in two parts: the rounding of one would be the same for a whole beam (NaN
            // stays in the sum; where a logit is beyond 2^24 the sum is made again)
            const float2 ef = make_float2(-(float)e, -(float)e);
            float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < VPT; j += 2) {
                const float2 y = fma2(make_float2(v[j], v[j + 1]), make_float2(kLog2eLo, kLog2eLo),
                                      fma2(make_float2(v[j], v[j + 1]), make_float2(kLog2eHi, kLog2eHi), ef));
                acc = add2(acc, make_float2(ex2_approx(y.x), ex2_approx(y.y)));
            }
            pair_add(sum, rest, __fadd_rn(acc.x, acc.y), 0.0f);
            // the threshold: from the threads' maxima so far, after tiles 1, 2, 4, 8, ... (a tile's share of the values
            // is halved from one to the next, so each part of the slice leaves about as many candidates).  What a warp
            // last published holds from then on, so without many candidates only the first tile needs a barrier, and
            // the tile behind each takes in what the other warps published late.
            const bool publish = careful || (tile & (tile + 1)) == 0;
            if (publish) sel_kth(ord32(m), k, wkth);
            if (publish && (careful || tile == 0 || many)) {
                __syncthreads();
                thr = max(thr, sel_threshold(wkth, jw));
                c = buf.count;
                __syncthreads();
                over = c > kSelBuf;
                if (!over && c > kSelBuf / 2) {  // keep the n best
                    sel_rank(buf, c, n, best);
                    __syncthreads();
                    c = min(c, n);
                    for (int i = tid; i < c; i += kSelThreads) buf.key[i] = best[i];
                    if (c == n) thr = max(thr, (uint32_t)(best[n - 1] >> 32));
                    if (tid == 0) buf.count = c;
                    __syncthreads();
                }
            } else if (publish || (tile & (tile - 1)) == 0) {
                thr = max(thr, sel_threshold(wkth, jw));
            }
            const float low = unord32(thr);
            if (tmax >= low && !over)  // (NaN is not)
#pragma unroll
                for (int u = 0; u < VPT / 4; u++)  // (a warp passes over the fours that none of its threads has one in)
                    if (gmax[u] >= low) {
                        int p = 0;
#pragma unroll
                        for (int j = 4 * u; j < 4 * u + 4; j++) p += v[j] >= low;
                        p = atomicAdd(&buf.count, p);
#pragma unroll
                        for (int j = 4 * u; j < 4 * u + 4; j++)
                            if (v[j] >= low) {
                                if (p < kSelBuf) buf.key[p] = cand_key(v[j], (uint32_t)(at + index(j)));
                                p++;
                            }
                    }
            if (careful) {
                __syncthreads();
                if (buf.count > kSelBuf) {
                    // the tile's n-th largest key bit by bit, then the n keys no smaller
                    uint64_t t = 0;
                    for (int bit = 63; bit >= 0; bit--) {
                        const uint64_t tt = t | (1ull << bit);
                        int nn = 0;
#pragma unroll
                        for (int j = 0; j < VPT; j++)
                            nn += v[j] == v[j] && cand_key(v[j], (uint32_t)(at + index(j))) >= tt;
                        nn = (int)__reduce_add_sync(0xffffffffu, (unsigned)nn);
                        __syncthreads();
                        if (lane == 0) wkth[warp] = (uint32_t)nn;
                        __syncthreads();
                        nn = 0;
#pragma unroll
                        for (int w = 0; w < kSelWarps; w++) nn += (int)wkth[w];
                        if (nn >= n) t = tt;
                    }
                    __syncthreads();
                    if (tid == 0) buf.count = c;
                    __syncthreads();
#pragma unroll
                    for (int j = 0; j < VPT; j++) {
                        const uint64_t key = cand_key(v[j], (uint32_t)(at + index(j)));
                        if (v[j] == v[j] && key >= t) buf.key[atomicAdd(&buf.count, 1)] = key;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < VPT; j++) v[j] = nx[j];
        }
        sel_kth(ord32(m), k, wkth);
        const float wtop = warp_max(m);
        if (lane == 0) wmax[warp] = wtop;
        __syncthreads();
        c = buf.count;
        if (careful || (!over && c <= kSelBuf)) break;
        __syncthreads();
    }
    // the ones below the last threshold are out
    thr = max(thr, sel_threshold(wkth, jw));
    for (int i = tid; i < c; i += kSelThreads) {
        const uint64_t key = buf.key[i];
        if ((uint32_t)(key >> 32) >= thr) last.key[atomicAdd(&last.count, 1)] = key;
    }
    // the block's largest value, and the sum on its scale (no thread's is above it)
    float top = wmax[0];
#pragma unroll
    for (int w = 1; w < kSelWarps; w++) top = fmaxf(top, wmax[w]);
    float d, dl;
    if (sel_wide(top)) {
        // logits beyond 2^24 (or none at all): once more, relative to the largest
        // (a NaN is no smaller than anything and stays in the sum, plus infinity less itself is one; the first sum says
        // nothing here: its scale ends at 1e8)
        d = dl = 0.0f;
        for (int i = v0 + tid; i < v1; i += kSelThreads) {
            const float xi = x[i];
            if (!(xi == ninf)) pair_add(d, dl, ex2_approx(__fmul_rn(__fsub_rn(xi, top), kLog2eHi)), 0.0f);
        }
    } else {
        const float f = pow2i(max(e - (int)sel_exp(top), -126));
        d = __fmul_rn(sum, f), dl = __fmul_rn(rest, f);
    }
    pair_warp_sum(d, dl);
    if (lane == 0) wsum[warp] = make_float2(d, dl);
    __syncthreads();
    c = last.count;
    const int64_t ps = (int64_t)row * S + blockIdx.x;
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kSelWarps; w++) pair_add(d, dl, wsum[w].x, wsum[w].y);
        part[ps] = SelPart{d, dl, top, min(c, n)};
    }
    sel_rank(last, c, n, cand + ps * n);
}

constexpr int kMergeThreads = 512, kMergeWarps = kMergeThreads / 32;
constexpr int kMergeBuf = 2048;    // candidates ranked in shared memory
constexpr int kMergeStage = 4096;  // listed candidates read at once

// fp64 as an unsigned whole number in the same order, above 0 for all but NaN
__device__ __forceinline__ uint64_t ord64(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double unord64(uint64_t k) {
    return __longlong_as_double((long long)((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}
__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

// log (h + l) as a pair, to about 1e-9 (the sums it is taken of are good to
// 7e-7): h + l = 2^k f with f in [2/3, 4/3] and log f =
// 2 (w + w^3 / 3 + w^5 / 5 + ...), w = (f - 1) / (f + 1).  |w| <= 1/5: the
// first term left out is below 1e-9, and behind w itself, which is a pair, one
// float's digits do.  h is 0, positive or NaN.
__device__ __forceinline__ float2 log_of_sum(float h, float l) {
    if (!(h > 0.0f)) return make_float2(h == 0.0f ? -__int_as_float(0x7f800000) : h, 0.0f);
    int k = (int)(__float_as_uint(h) >> 23) - 127;
    float sc = pow2i(-k);
    if (__fmul_rn(h, sc) > 1.3333334f) sc = __fmul_rn(sc, 0.5f), k++;
    const float f = __fmul_rn(h, sc), fl = __fmul_rn(l, sc);
    const float nh = __fsub_rn(f, 1.0f);  // (exact)
    float dh = f, dl = fl;
    pair_add(dh, dl, 1.0f, 0.0f);
    const float w = __fdiv_rn(nh, dh);
    const float wl = __fdividef(__fmaf_rn(-w, dl, __fadd_rn(__fmaf_rn(-w, dh, nh), fl)), dh);
    const float z = __fmul_rn(w, w);
    float t = 1.0f / 13;
#pragma unroll
    for (int c = 11; c >= 3; c -= 2) t = __fmaf_rn(z, t, 1.0f / (float)c);
    t = __fmul_rn(z, t);
    float rh = 2.0f * w, rl = 2.0f * __fmaf_rn(w, t, wl);
    const float kf = (float)k, ph = __fmul_rn(kf, kLn2Hi);
    pair_add(rh, rl, ph, __fmaf_rn(kf, kLn2Lo, __fmaf_rn(kf, kLn2Hi, -ph)));
    return make_float2(rh, rl);
}

struct MergeSmem {
    float2 lse[kMaxBeams];  // a beam's sum of exponentials, then its log less top
    float2 shift[kMaxBeams];  // its score less that log
    float top[kMaxBeams];   // the beam's largest logit
    float base[kMaxBeams];  // its score
    int kind[kMaxBeams];    // 0: dead, 1: live, 2: finished
    int wild;               // a live beam's numbers are beyond what pairs of floats hold
    int count, passing;
    uint64_t sharp;
    uint64_t kth[kMergeWarps], wkey[kMergeWarps];
    int64_t wat[kMergeWarps];
    int wlist[kMergeWarps];
    SelPart part[kMergeThreads];
    uint64_t key[kMergeBuf];
    int64_t at[kMergeBuf];
    uint64_t stage[kMergeStage];
    uint64_t heads[kMergeThreads + 32];  // (an odd stride between a warp's)
    uint16_t list[kMergeThreads];
    uint8_t beam[kMergeThreads];  // of each list
    uint8_t next[kMergeThreads];  // the next entry of each list
};

// Entry h of list i as a whole number in the order of the candidates (key 0:
// there is none; NaN gives nothing of this beam), and what settles equal ones:
// the beam, the logit (the larger first: offers are only equal as rounded) and
// the word, in 6, 32 and 24 bits.
struct MergeEntry {
    uint64_t key;
    int64_t at;
};
__device__ __noinline__ MergeEntry merge_entry(const MergeSmem &M, const uint64_t *list, int i, int h, int eos) {
    MergeEntry e{0, 0};
    const int b = M.beam[i], kind = M.kind[b];
    const float ninf = -__int_as_float(0x7f800000);
    if (kind == 1) {
        if (h >= M.part[i].count) return e;
        const uint64_t k = list[h];
        const float x = unord32((uint32_t)(k >> 32)), top = M.top[b], base = M.base[b];
        const float2 lse = M.lse[b];
        e.at = (int64_t)b << 56 | (int64_t)(uint32_t)~(uint32_t)(k >> 32) << 24 | (uint32_t)~(uint32_t)k;
        if (M.wild) {
            const double c = (double)base + (((double)x - (double)top) - ((double)lse.x + (double)lse.y));
            if (c > (double)ninf) e.key = ord64(c);
        } else {
            // (one rounding, of the low part: a beam's candidates keep the order of its logits)
            const float2 shift = M.shift[b];
            float c = x, l = 0.0f;
            pair_add(c, l, shift.x, shift.y);
            // the nearest float and the rest of it (+ 0: no negative zeros)
            float hi = l, lo = 0.0f;
            pair_add(hi, lo, c, 0.0f);
            if (fabsf(lo) < fabsf(hi) * 0x1p-53f) lo = 0.0f;  // (candidates near the type's lowest value are equal)
            if (hi > ninf) e.key = (uint64_t)ord32(__fadd_rn(hi, 0.0f)) << 32 | ord32(__fadd_rn(lo, 0.0f));
        }
    } else if (kind == 2 && h == 0 && (i == 0 || M.beam[i - 1] != b)) {
        const float c = __fadd_rn(M.base[b], 0.0f);
        e.at = (int64_t)b << 56 | (uint32_t)eos;
        if (c > ninf) e.key = M.wild ? ord64((double)c) : (uint64_t)ord32(c) << 32 | ord32(0.0f);
    }
    return e;
}

// One CTA per group: lse of every live beam, then the n best of the beams'
// sorted lists (S lists per live beam, one entry for a finished one).  What it
// reads is on its way at once; candidates are pairs of floats (48 bits), or
// fp64 where a beam's numbers are too large for that, and compared as whole
// numbers in the same order.
__global__ void __launch_bounds__(kMergeThreads)
    beam_merge_kernel(const SelPart *__restrict__ part, const uint64_t *__restrict__ cand,
                      const float *__restrict__ scores, const uint8_t *__restrict__ finished, int eos, int beams,
                      int S, int n, float *out_scores, int32_t *parents, int32_t *tokens) {
    extern __shared__ __align__(16) uint8_t mg_raw[];
    MergeSmem &M = *reinterpret_cast<MergeSmem *>(mg_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = blockIdx.x, lists = beams * S;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float ninf = -__int_as_float(0x7f800000);
    part += (int64_t)g * lists;
    cand += (int64_t)g * lists * n;
    const bool staged = lists * n <= kMergeStage;
    {
        // (a dead or finished beam's parts and a list's end hold anything: read, and not used)
        uint64_t w[kMergeStage / kMergeThreads];
        if (staged)
#pragma unroll
            for (int u = 0; u < kMergeStage / kMergeThreads; u++)
                if (u * kMergeThreads + tid < lists * n) w[u] = __ldcg(&cand[u * kMergeThreads + tid]);
        if (tid < lists) {
            const int4 p = __ldcg((const int4 *)&part[tid]);
            M.part[tid] = SelPart{__int_as_float(p.x), __int_as_float(p.y), __int_as_float(p.z), p.w};
        }
        if (tid < lists) M.beam[tid] = (uint8_t)(tid / S);
        if (tid < beams) {
            const float score = scores[g * beams + tid];
            M.base[tid] = score;
            M.kind[tid] = finished && finished[g * beams + tid] ? 2 : score > ninf ? 1 : 0;
        }
        if (tid == 0) M.count = M.wild = 0, M.sharp = 0;
        if (staged)
#pragma unroll
            for (int u = 0; u < kMergeStage / kMergeThreads; u++)
                if (u * kMergeThreads + tid < lists * n) M.stage[u * kMergeThreads + tid] = w[u];
    }
    __syncthreads();
    for (int b = warp; b < beams; b += kMergeWarps) {
        if (M.kind[b] != 1) continue;
        const SelPart *p = M.part + b * S;
        float big = ninf;
        for (int i = lane; i < S; i += 32) big = fmaxf(big, p[i].m);
        big = unord32(__reduce_max_sync(0xffffffffu, ord32(big)));
        float h = 0.0f, l = 0.0f;
        if (!sel_wide(big)) {
            for (int i = lane; i < S; i += 32) {
                // (a wide slice is far below the others here: nothing, or NaN)
                const float sh = sel_wide(p[i].m) ? ninf : sel_exp(p[i].m) - sel_exp(big);
                const float f = sh >= -126.0f ? pow2i((int)sh) : 0.0f;
                pair_add(h, l, __fmul_rn(p[i].sum, f), __fmul_rn(p[i].lo, f));
            }
        } else {
            for (int i = lane; i < S; i += 32) {
                // (0, or NaN, where there is no logit)
                const double mi = (double)p[i].m, si = (double)p[i].sum + (double)p[i].lo;
                const double v = p[i].m > ninf
                                     ? si * exp((sel_wide(p[i].m) ? mi : (double)sel_exp(p[i].m) * 0.69314718055994530942) -
                                                (double)big)
                                     : si;
                pair_add(h, l, (float)v, (float)(v - (double)(float)v));
            }
        }
        pair_warp_sum(h, l);
        if (lane == 0) {
            float hi = l, lo = 0.0f;
            pair_add(hi, lo, h, 0.0f);
            M.lse[b] = make_float2(hi, lo), M.top[b] = big;
        }
    }
    __syncthreads();
    if (tid < beams && M.kind[tid] == 1) {  // (one warp or two)
        const float big = M.top[tid];
        float2 l = log_of_sum(M.lse[tid].x, M.lse[tid].y);
        const bool wide = sel_wide(big);
        if (!wide) {
            const float e = sel_exp(big), p = __fmul_rn(e, kLn2Hi);
            pair_add(l.x, l.y, p, __fmaf_rn(e, kLn2Lo, __fmaf_rn(e, kLn2Hi, -p)));
            pair_add(l.x, l.y, -big, 0.0f);
        }
        M.lse[tid] = l;
        // what a candidate is above its logit: score - lse
        l.x = -l.x, l.y = -l.y;
        pair_add(l.x, l.y, -big, 0.0f);
        pair_add(l.x, l.y, M.base[tid], 0.0f);
        float hi = l.y, lo = 0.0f;
        pair_add(hi, lo, l.x, 0.0f);
        M.shift[tid] = make_float2(hi, lo);
        if (wide || !(fabsf(M.base[tid]) <= 1e30f)) M.wild = 1;
    }
    __syncthreads();
    auto entry = [&](int i, int h) {
        return merge_entry(M, staged ? M.stage + i * n : cand + (int64_t)i * n, i, h, eos);
    };
    // The lists are dealt out to the warps evenly.  With the q-th entries of
    // ceil(n / (warps q)) lists in every warp no smaller than a threshold, n
    // candidates are not.
    const int W = min(kMergeWarps, lists), q = (n + lists - 1) / lists, k = (n + W * q - 1) / (W * q);
    const int mylist = lane * kMergeWarps + warp;
    M.heads[tid + tid / kMergeWarps] = tid < lists ? entry(tid, q - 1).key : 0;
    __syncthreads();
    const uint64_t head = M.heads[mylist + lane];
    uint64_t mine = head, kth = 0;
    for (int r = 0; r < k; r++) {
        kth = warp_max64(mine);
        const uint32_t who = __ballot_sync(0xffffffffu, mine == kth);
        if (lane == __ffs(who) - 1) mine = 0;
    }
    if (lane == 0) M.kth[warp] = kth;
    __syncthreads();
    uint64_t thr = ~warp_max64(lane < W ? ~M.kth[lane] : 0);
    // sharper: the ceil(n / q)-th of the heads that pass (beams differ: a warp may hold poor ones only); eight threads
    // count for a head
    if (head && head >= thr) M.key[atomicAdd(&M.count, 1)] = head;
    __syncthreads();
    const int heads = M.count, want = (n + q - 1) / q;
    for (int i0 = 0; i0 < heads; i0 += kMergeThreads / 8) {
        const int i = i0 + (tid >> 3);
        const uint64_t key = i < heads ? M.key[i] : 0;
        int above = 0, same = 0;
#pragma unroll 4
        for (int j = tid & 7; j < heads; j += 8) above += M.key[j] > key, same += M.key[j] == key;
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) {
            above += __shfl_xor_sync(0xffffffffu, above, off);
            same += __shfl_xor_sync(0xffffffffu, same, off);
        }
        if (i < heads && above < want && above + same >= want) M.sharp = key;  // (all that write it write the same)
    }
    __syncthreads();
    thr = max(thr, M.sharp);
    // the lists whose head passes, then all of their entries at once
    if (tid == 0) M.count = M.passing = 0;
    __syncthreads();
    if (mylist < lists && (q > 1 || (head && head >= thr))) M.list[atomicAdd(&M.passing, 1)] = (uint16_t)mylist;
    __syncthreads();
    const int pairs = M.passing * n;
    for (int i = tid; i < pairs; i += kMergeThreads) {
        const int l = i / n;
        const MergeEntry e = entry(M.list[l], i - l * n);
        if (e.key && e.key >= thr) {
            const int p = atomicAdd(&M.count, 1);
            if (p < kMergeBuf) M.key[p] = e.key, M.at[p] = e.at;
        }
    }
    __syncthreads();
    const int total = M.count;
    auto write = [&](int r, uint64_t key, int64_t at) {
        const int64_t o = (int64_t)g * n + r;
        out_scores[o] = M.wild ? (float)unord64(key) : unord32((uint32_t)(key >> 32));
        parents[o] = (int)(at >> 56);
        tokens[o] = (int)(at & 0xffffff);
    };
    const int found = min(total, n);
    if (total <= kMergeBuf) {
        // four threads count for a candidate
        const int part4 = tid & 3, per = (total + 3) / 4, j0 = min(part4 * per, total), j1 = min(j0 + per, total);
        for (int i0 = 0; i0 < total; i0 += kMergeThreads / 4) {
            const int i = i0 + (tid >> 2);
            uint64_t key = 0;
            int64_t at = 0;
            int r = 0;
            if (i < total) {
                key = M.key[i], at = M.at[i];
                r = place_of<int64_t>(key, at, i >= j0 && i < j1, M.key + j0, M.at + j0, j1 - j0);
            }
            r += __shfl_xor_sync(0xffffffffu, r, 1);
            r += __shfl_xor_sync(0xffffffffu, r, 2);
            if (i < total && part4 == 0 && r < n) write(r, key, at);
        }
    } else {
        // too many equal candidates: n rounds of taking the best head of the lists
        if (tid < lists) M.next[tid] = 0;
        __syncthreads();
        auto better = [](uint64_t key, int64_t at, uint64_t bkey, int64_t bat) {
            return key > bkey || (key == bkey && at < bat);
        };
        for (int r = 0; r < n; r++) {
            const MergeEntry e = tid < lists ? entry(tid, M.next[tid]) : MergeEntry{0, 0};
            uint64_t key = e.key;
            int64_t at = key ? e.at : INT64_MAX;
            int li = tid;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const uint64_t ok = __shfl_xor_sync(0xffffffffu, key, off);
                const int64_t oat = __shfl_xor_sync(0xffffffffu, at, off);
                const int ol = __shfl_xor_sync(0xffffffffu, li, off);
                if (better(ok, oat, key, at)) key = ok, at = oat, li = ol;
            }
            if (lane == 0) M.wkey[warp] = key, M.wat[warp] = at, M.wlist[warp] = li;
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w < kMergeWarps; w++)
                    if (better(M.wkey[w], M.wat[w], key, at)) key = M.wkey[w], at = M.wat[w], li = M.wlist[w];
                write(r, key, at);  // (there are more than n)
                M.next[li]++;
            }
            __syncthreads();
        }
    }
    for (int r = found + tid; r < n; r += kMergeThreads) {
        const int64_t o = (int64_t)g * n + r;
        out_scores[o] = ninf;
        parents[o] = tokens[o] = -1;
    }
}

// ---------------------------------------------------------------- reordering
constexpr int kRoStages = 3;
constexpr int kRoSmem = 192 * 1024;  // the stages' bytes
constexpr int kRoMaxChunk = 16384, kRoMinChunk = 1024;

struct RoArgs {
    char *cache;
    int64_t seq_stride, plane_stride;
    int n_planes;
    int64_t row_bytes;
    int max_rows;
    const int32_t *parents;
    const int32_t *rows;
    int n_groups, beams;
    int32_t *status;
};

// One warp per CTA: the copies need no other threads.  CTA c takes the items
// c, c + grid, ... of every group; an item is one stretch of at most `chunk`
// bytes of one plane, of every beam.
__global__ void __launch_bounds__(32) beam_reorder_kernel(RoArgs A) {
    extern __shared__ __align__(128) uint8_t ro_smem[];
    __shared__ uint64_t full[kRoStages];
    __shared__ int src[kMaxBeams];        // slot -> source beam
    __shared__ int slot_of[kMaxBeams];    // source beam -> slot
    __shared__ int dst[kMaxBeams];        // moved beams
    __shared__ int dst_slot[kMaxBeams];
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int s = 0; s < kRoStages; s++) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    __syncwarp();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int filled = 0;  // stages filled so far: fill f uses stage f % kRoStages
    bool ok = true;
    int64_t skip = blockIdx.x;  // items until this CTA's next one
    for (int g = 0; g < A.n_groups && ok; g++) {
        const int nrows = A.rows ? min(max(A.rows[g], 0), A.max_rows) : A.max_rows;
        // moved beams and the distinct beams they take
        uint64_t want = 0;
        int nd = 0;
        for (int b0 = 0; b0 < A.beams; b0 += 32) {
            const int b = b0 + lane;
            const int p = b < A.beams ? A.parents[(int64_t)g * A.beams + b] : -1;
            const bool moved = p >= 0 && p < A.beams && p != b;
            const uint32_t bal = __ballot_sync(0xffffffffu, moved);
            if (moved) {
                const int at = nd + __popc(bal & ((1u << lane) - 1u));
                dst[at] = b;
                dst_slot[at] = p;  // the beam for now
            }
            nd += __popc(bal);
            uint64_t w = moved ? 1ull << p : 0ull;
            w = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)w) |
                (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(w >> 32)) << 32;
            want |= w;
        }
        const int ns = __popcll(want);
        if (ns == 0 || nrows == 0) continue;
        __syncwarp();
        for (int b = lane; b < A.beams; b += 32)
            if (want >> b & 1) {
                const int sidx = __popcll(want & ((1ull << b) - 1ull));
                src[sidx] = b;
                slot_of[b] = sidx;
            }
        __syncwarp();
        for (int i = lane; i < nd; i += 32) dst_slot[i] = slot_of[dst_slot[i]];
        __syncwarp();
        const int64_t plane = (int64_t)nrows * A.row_bytes;
        // as much of a stage as the sources fill, but enough items for every CTA
        const int64_t even = (plane * A.n_planes / gridDim.x + 127) / 128 * 128;
        const int cap = (int)min((int64_t)min(kRoMaxChunk, kRoSmem / kRoStages / ns / 128 * 128),
                                 max(even, (int64_t)kRoMinChunk));
        const int64_t parts = (plane + cap - 1) / cap;
        const int chunk = (int)((plane + parts * 16 - 1) / (parts * 16) * 16);
        const int64_t per = (plane + chunk - 1) / chunk;
        const int64_t items = (int64_t)A.n_planes * per;
        char *base = A.cache + (int64_t)g * A.beams * A.seq_stride;
        if (skip >= items) {
            skip -= items;
            continue;
        }
        const int64_t mine = (items - skip + gridDim.x - 1) / gridDim.x;
        auto where = [&](int64_t k, int64_t &off, uint32_t &bytes) {
            const int64_t it = skip + k * gridDim.x, pl = it / per, at = (it - pl * per) * chunk;
            off = pl * A.plane_stride + at;
            bytes = (uint32_t)min((int64_t)chunk, plane - at);
        };
        auto load = [&](int64_t k, int f) {
            int64_t off;
            uint32_t bytes;
            where(k, off, bytes);
            const int st = f % kRoStages;
            uint8_t *to = ro_smem + (size_t)st * (kRoSmem / kRoStages);
            if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes * (uint32_t)ns);
            __syncwarp();
            for (int i = lane; i < ns; i += 32)
                bulk_g2s_l2(to + (size_t)i * chunk, base + (int64_t)src[i] * A.seq_stride + off, bytes, &full[st]);
        };
        const int f0 = filled;
        for (int64_t k = 0; k < min((int64_t)kRoStages - 1, mine); k++) load(k, f0 + (int)k);
        for (int64_t k = 0; k < mine; k++) {
            const int f = f0 + (int)k, st = f % kRoStages;
            if (__any_sync(0xffffffffu, !mbar_wait(&full[st], (uint32_t)(f / kRoStages) & 1u))) {
                if (lane == 0) raise_status(A.status, kStatusTimeout);
                for (int64_t j = k + 1; j < min(k + kRoStages - 1, mine); j++)  // the copies behind it
                    mbar_wait(&full[(f0 + (int)j) % kRoStages], (uint32_t)((f0 + (int)j) / kRoStages) & 1u);
                ok = false;
                break;
            }
            int64_t off;
            uint32_t bytes;
            where(k, off, bytes);
            const uint8_t *from = ro_smem + (size_t)st * (kRoSmem / kRoStages);
            for (int i = lane; i < nd; i += 32)
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                 base + (int64_t)dst[i] * A.seq_stride + off),
                             "r"(smem_addr(from + (size_t)dst_slot[i] * chunk)), "r"(bytes)
                             : "memory");
            bulk_commit_group();
            // the stage of item k - 1 takes item k + stages - 1 once its stores have read it
            if (k + kRoStages - 1 < mine) {
                asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                __syncwarp();
                load(k + kRoStages - 1, f + kRoStages - 1);
            }
        }
        filled = f0 + (int)mine;
        bulk_wait_read_all();
        __syncwarp();
        skip = (skip + mine * gridDim.x) - items;
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Slices of a row: one wave of CTAs over all rows, but a thousand values each.
constexpr int kSelCtas = kSelPerSm * 152;
int sel_len(int rows, int V) {
    int S = kSelCtas / rows;
    if (S > (V + 1023) / 1024) S = (V + 1023) / 1024;
    if (S < 1) S = 1;
    return ((V + S - 1) / S + 3) / 4 * 4;
}
int sel_slices(int rows, int V) {
    const int len = sel_len(rows, V);
    return (V + len - 1) / len;
}
static_assert(kSelCtas <= kMergeThreads && kMaxBeams <= kMergeThreads, "a thread for each of a group's lists");

template <int VPT>
const void *slice_kernel(bool vec) {
    return vec ? (const void *)beam_slice_kernel<VPT, true> : (const void *)beam_slice_kernel<VPT, false>;
}

bool sel_sizes_ok(int n_groups, int beams, int vocab, int n_out) {
    return n_groups >= 1 && beams >= 1 && beams <= kMaxBeams && vocab >= 1 && vocab <= (1 << 24) && n_out >= 1 &&
           n_out <= kMaxOut && (int64_t)n_groups * beams <= 65535;
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

size_t qlin_beam_select_workspace_size(int n_groups, int beams, int vocab, int n_out) {
    if (!sel_sizes_ok(n_groups, beams, vocab, n_out)) return 0;
    const int rows = n_groups * beams;
    return carve_sel(rows, sel_slices(rows, vocab), n_out, nullptr).bytes;
}

qlin_status qlin_beam_select(const float *logits, int64_t row_stride, const float *scores, const uint8_t *finished,
                             int eos, int n_groups, int beams, int vocab, int n_out, float *out_scores,
                             int32_t *parents, int32_t *tokens, void *workspace, size_t workspace_bytes,
                             qlin_stream_t stream) {
    qlin::clear_error();
    QLIN_REQUIRE(logits && scores && out_scores && parents && tokens && workspace, QLIN_ERR_INVALID_ARG,
                 "qlin_beam_select: null pointer");
    QLIN_REQUIRE(n_groups >= 1 && beams >= 1 && vocab >= 1 && n_out >= 1, QLIN_ERR_INVALID_ARG,
                 "qlin_beam_select: n_groups %d, beams %d, vocab %d, n_out %d", n_groups, beams, vocab, n_out);
    QLIN_REQUIRE(sel_sizes_ok(n_groups, beams, vocab, n_out), QLIN_ERR_UNSUPPORTED,
                 "qlin_beam_select: at most %d beams, %d outputs, %d words and 65535 rows (%d groups of %d, %d, %d)",
                 kMaxBeams, kMaxOut, 1 << 24, n_groups, beams, n_out, vocab);
    QLIN_REQUIRE(row_stride >= vocab, QLIN_ERR_INVALID_ARG, "qlin_beam_select: row_stride %lld < vocab %d",
                 (long long)row_stride, vocab);
    QLIN_REQUIRE(!finished || (eos >= 0 && eos < vocab), QLIN_ERR_INVALID_ARG,
                 "qlin_beam_select: eos %d outside the vocabulary", eos);
    QLIN_REQUIRE(aligned4(logits) && aligned4(scores) && aligned4(out_scores) && aligned4(parents) && aligned4(tokens),
                 QLIN_ERR_INVALID_ARG, "qlin_beam_select: pointer not 4-byte aligned");
    QLIN_REQUIRE(aligned16(workspace), QLIN_ERR_INVALID_ARG, "qlin_beam_select: workspace not 16-byte aligned");
    const int rows = n_groups * beams, S = sel_slices(rows, vocab);
    const SelWs w = carve_sel(rows, S, n_out, (char *)workspace);
    QLIN_REQUIRE(workspace_bytes >= w.bytes, QLIN_ERR_INVALID_ARG, "qlin_beam_select: workspace %zu < %zu bytes",
                 workspace_bytes, w.bytes);
    const bool vec = aligned16(logits) && row_stride % 4 == 0;
    const int len = sel_len(rows, vocab);
    const void *k = len <= 1024 ? slice_kernel<4>(vec) : len <= 4096 ? slice_kernel<8>(vec) : slice_kernel<16>(vec);
    void *a0[] = {(void *)&logits, (void *)&row_stride, (void *)&scores, (void *)&finished, (void *)&vocab,
                  (void *)&len, (void *)&n_out, (void *)&w.part, (void *)&w.cand};
    if (qlin_status st = launch_pdl(k, dim3(S, rows), dim3(kSelThreads), 0, (cudaStream_t)stream, a0,
                                    "beam_slice_kernel"))
        return st;
    void *a1[] = {(void *)&w.part, (void *)&w.cand, (void *)&scores, (void *)&finished, (void *)&eos, (void *)&beams,
                  (void *)&S, (void *)&n_out, (void *)&out_scores, (void *)&parents, (void *)&tokens};
    const size_t smem = sizeof(MergeSmem);
    blocks_per_sm((const void *)beam_merge_kernel, smem);  // raises the dynamic shared-memory limit once
    return launch_pdl((const void *)beam_merge_kernel, dim3(n_groups), dim3(kMergeThreads), smem, (cudaStream_t)stream,
                      a1, "beam_merge_kernel");
}

qlin_status qlin_beam_reorder(void *cache, int64_t seq_stride, int64_t plane_stride, int n_planes, int64_t row_bytes,
                              int max_rows, const int32_t *parents, const int32_t *n_rows, int n_groups, int beams,
                              int32_t *status_word, qlin_stream_t stream) {
    qlin::clear_error();
    QLIN_REQUIRE(cache && parents, QLIN_ERR_INVALID_ARG, "qlin_beam_reorder: null pointer");
    QLIN_REQUIRE(n_planes >= 1 && max_rows >= 1 && n_groups >= 1 && beams >= 1 && row_bytes >= 16, QLIN_ERR_INVALID_ARG,
                 "qlin_beam_reorder: n_planes %d, max_rows %d, n_groups %d, beams %d, row_bytes %lld", n_planes,
                 max_rows, n_groups, beams, (long long)row_bytes);
    QLIN_REQUIRE(beams <= kMaxBeams, QLIN_ERR_UNSUPPORTED, "qlin_beam_reorder: %d beams, at most %d", beams, kMaxBeams);
    QLIN_REQUIRE(aligned16(cache) && row_bytes % 16 == 0 && seq_stride % 16 == 0 && plane_stride % 16 == 0,
                 QLIN_ERR_INVALID_ARG, "qlin_beam_reorder: cache, row_bytes and strides are multiples of 16 bytes");
    QLIN_REQUIRE(row_bytes <= (int64_t)1 << 40 && seq_stride >= 0 && seq_stride <= (int64_t)1 << 46 &&
                     plane_stride >= 0 && plane_stride <= (int64_t)1 << 46,
                 QLIN_ERR_INVALID_ARG, "qlin_beam_reorder: a stride is out of range");
    // every beam's rows are its own: planes inside a sequence, or sequences inside a plane
    const __int128 plane = (__int128)row_bytes * max_rows, seqs = (__int128)n_groups * beams;
    const bool seq_major = (n_planes == 1 || plane_stride >= plane) &&
                           (seqs == 1 || seq_stride >= (__int128)plane_stride * (n_planes - 1) + plane);
    const bool plane_major = (seqs == 1 || seq_stride >= plane) &&
                             (n_planes == 1 || plane_stride >= (__int128)seq_stride * (seqs - 1) + plane);
    QLIN_REQUIRE(seq_major || plane_major, QLIN_ERR_INVALID_ARG, "qlin_beam_reorder: the beams' rows overlap");
    QLIN_REQUIRE(aligned4(parents) && aligned4(n_rows) && aligned4(status_word), QLIN_ERR_INVALID_ARG,
                 "qlin_beam_reorder: pointer not 4-byte aligned");
    QLIN_REQUIRE(kRoSmem + 1024 <= max_smem_optin(), QLIN_ERR_UNSUPPORTED, "qlin_beam_reorder: shared memory");
    blocks_per_sm((const void *)beam_reorder_kernel, kRoSmem);  // raises the limit once
    RoArgs A{(char *)cache, seq_stride, plane_stride, n_planes, row_bytes, max_rows, parents, n_rows, n_groups, beams,
             status_word};
    void *args[] = {(void *)&A};
    return launch_pdl((const void *)beam_reorder_kernel, dim3(sm_count()), dim3(32), kRoSmem, (cudaStream_t)stream, args,
                      "beam_reorder_kernel");
}

}  // extern "C"
