// Attention over lanes with a sliding window and first tokens that reads the
// paged cache of 4 bits a value (qlin_attention_kv4).
//
// Lane i, at position p of its sequence, sees the keys at positions j <= p
// with j > p - window or j < sinks (every j <= p without a window); its query
// head h takes KV head h / (n_heads / n_kv) and gives
//   o = sum_j w_j v_j,  w = softmax_j(q . k_j / sqrt(head_dim)),
// zeros where no key is seen.
//
// A softmax over keys in any order: with m a number no smaller than some score,
// weights 2^(s_j - m) (s in units of log(2), the factor log2(e) / sqrt(head_dim)
// goes into the queries), their sum l and the sum of w_j v_j; parts of the keys
// are joined by 2^(m_part - m).  Little work goes to CUDA cores (below), the
// rest to the tensor cores (further down); few_fits tells them apart.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>

#include "attention_lanes.cuh"
#include "kv4.cuh"

namespace qlin {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSplits = 1024;
constexpr int kMergeDims = 64;     // dims of a head per merging CTA
constexpr int kCluster = 16;       // CTAs of a cluster at most

struct Kv4Args {
    const float *q;
    qlin_kv4 kv;
    const int32_t *positions, *seqs;
    int n_lanes, n_heads, n_kv, hd, window, sinks;
    float *out;
    int32_t *status;
    int group;  // query heads per KV head
    float c;    // log2(e) / sqrt(hd)
};

constexpr float kInf = __builtin_huge_valf();

// What lane i sees: keys j < sk and lo <= j <= p (sk <= lo), `count` of them; 0 if it is none.
struct LaneKeys {
    int count, sk, lo, seq;
    bool bad;
    __device__ __forceinline__ LaneKeys(const Kv4Args &A, int i) {
        const int p = A.positions[i];
        seq = A.seqs[i];
        const bool ok = seq >= 0 && seq < A.kv.n_seqs && p / A.kv.page_rows < A.kv.max_pages;
        bad = p >= 0 && !ok;
        lo = A.window && p >= A.window ? p - A.window + 1 : 0;
        sk = min(A.sinks, lo);
        count = p >= 0 && ok ? sk + p + 1 - lo : 0;
    }
    __device__ __forceinline__ int key(int x) const { return x < sk ? x : lo + x - sk; }
};

__device__ __forceinline__ void decode8f(uint32_t w, __half2 s, __half2 m24, float (&f)[8]) {
    uint32_t o[4];
    kv4_decode8(w, s, m24, o);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&o[i]));
        f[2 * i] = x.x, f[2 * i + 1] = x.y;
    }
}

// Shared memory of a CTA of the kernel for little work: the keys' and values'
// rows, later the sums of the groups of keys; then the scales.
template <int HD, bool CL>
struct FewCfg {
    static constexpr int kKeys = CL ? 128 : 64;            // of a CTA at most
    static constexpr int kParts = kThreads / kKeys;        // threads to a key
    static constexpr int kRow = HD / 2 + 16;               // bytes between rows of codes
    static constexpr int kPer = HD / 32;                   // 16-byte groups of a row, and scales
    static constexpr int kWords = HD / 8, kGroups = kThreads / kWords;
    static constexpr int kRows = kKeys * kRow;
    static constexpr size_t bytes(int gh) {
        const size_t rows = 2 * (kRows + kKeys * kPer), sums = (size_t)kGroups * gh * HD * 4;
        return rows > sums ? rows : sums;
    }
};

// Little work: a CTA takes up to 64 or 128 of a lane's keys for one KV head and
// up to eight of its query heads.  Scores: the threads of a key share its dims,
// each decoding its 16 bytes at a time for all heads at once; outputs: a thread
// per word of eight dims and group of keys.  Decoding is in fp16 (exact), the
// rest in fp32.  Latency bounds it: the copy of the rows, one pass for the
// scores, one for the outputs, and the merge.  Where the CTAs of a (lane, head
// block) fit one cluster they merge through each other's shared memory, so that
// there is one launch: a call for one token of 4 heads on one KV head of 256 and
// 1024 keys takes 8.6 us, and 12.9 with the merge as a launch of its own.
//
// grid (splits, KV heads x blocks of GH query heads, lanes); span: keys of a
// CTA.  CL: the CTAs of a (lane, head block) are one cluster and merge among
// themselves.
template <int HD, int GH, bool CL>
__global__ void __launch_bounds__(kThreads) kv4_few_kernel(const __grid_constant__ Kv4Args A, float2 *ml, float *part,
                                                           int splits, int span) {
    using C = FewCfg<HD, CL>;
    constexpr int KM = C::kKeys, PER = C::kPer;
    extern __shared__ __align__(16) uint8_t few_smem[];
    __shared__ __align__(16) float qs[GH][HD];
    __shared__ __align__(16) float ws[KM][GH];
    __shared__ float inv[GH];
    __shared__ float4 stat[GH];  // a cluster's: the largest score and the sum of the weights here
    __shared__ int ok[KM];
    uint8_t *const rows[2] = {few_smem, few_smem + C::kRows};
    uint8_t *const scales[2] = {few_smem + 2 * C::kRows, few_smem + 2 * C::kRows + KM * PER};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int s = blockIdx.x, blocks = (A.group + GH - 1) / GH, kvh = blockIdx.y / blocks, h0 = (blockIdx.y % blocks) * GH;
    const int lane_i = blockIdx.z, heads = min(GH, A.group - h0), head0 = kvh * A.group + h0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const LaneKeys L(A, lane_i);
    if (L.bad && s == 0 && blockIdx.y == 0 && tid == 0) raise_status(A.status, kStatusKv4Lane);
    const int n = min(span, L.count - s * span);
    if (CL ? L.count <= 0 : n <= 0) {
        if (s == 0)
            for (int e = tid; e < heads * HD; e += kThreads) A.out[((int64_t)lane_i * A.n_heads + head0) * HD + e] = 0.0f;
        return;
    }
    // a thread to 16 bytes of a key's codes and of its value's, and their scales
    for (int e = tid; e < n * PER; e += kThreads) {
        const int r = e / PER, c = e % PER;
        const int64_t at = kv4_row(A.kv, A.n_kv, L.key(s * span + r), L.seq);
        if (c == 0) ok[r] = at >= 0;
        if (at < 0) continue;
        const int64_t row = at + (int64_t)kvh * A.kv.page_rows;
        cp_async16(rows[0] + r * C::kRow + c * 16, static_cast<const uint8_t *>(A.kv.k) + row * (HD / 2) + c * 16, 16);
        cp_async16(rows[1] + r * C::kRow + c * 16, static_cast<const uint8_t *>(A.kv.v) + row * (HD / 2) + c * 16, 16);
        scales[0][r * PER + c] = static_cast<const uint8_t *>(A.kv.k_scale)[row * PER + c];
        scales[1][r * PER + c] = static_cast<const uint8_t *>(A.kv.v_scale)[row * PER + c];
    }
    cp_async_commit();
    if (CL && tid < GH) stat[tid] = make_float4(-kInf, 0.0f, 0.0f, 0.0f);  // (no key)
    for (int e = tid; e < GH * HD; e += kThreads)
        qs[e / HD][e % HD] = e / HD < heads ? A.q[((int64_t)lane_i * A.n_heads + head0) * HD + e] * A.c : 0.0f;
    cp_async_wait_pending<0>();
    __syncthreads();
    // scores: kParts threads share a key, 32 dims of it in turn
    const int key = tid / C::kParts, pt = tid % C::kParts;
    float sc[GH];
#pragma unroll
    for (int h = 0; h < GH; h++) sc[h] = 0.0f;
    const bool seen = key < n && ok[key];
    if (seen)
        for (int c = pt; c < PER; c += C::kParts) {
            const uint4 u = lds128(rows[0] + key * C::kRow + c * 16);
            __half2 sc2, m24;
            kv4_scale2(scales[0][key * PER + c], sc2, m24);
            const uint32_t words[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float f[8];
                decode8f(words[i], sc2, m24, f);
#pragma unroll
                for (int h = 0; h < GH; h++)
#pragma unroll
                    for (int d = 0; d < 8; d += 4) {
                        const float4 q = *reinterpret_cast<const float4 *>(&qs[h][c * 32 + i * 8 + d]);
                        sc[h] = __fmaf_rn(q.x, f[d], sc[h]);
                        sc[h] = __fmaf_rn(q.y, f[d + 1], sc[h]);
                        sc[h] = __fmaf_rn(q.z, f[d + 2], sc[h]);
                        sc[h] = __fmaf_rn(q.w, f[d + 3], sc[h]);
                    }
            }
        }
    if (key < n && pt == 0 && !seen) raise_status(A.status, kStatusKv4Lane);
#pragma unroll
    for (int off = 1; off < C::kParts; off <<= 1)
#pragma unroll
        for (int h = 0; h < GH; h++) sc[h] = __fadd_rn(sc[h], __shfl_xor_sync(0xffffffffu, sc[h], off));
    if (pt == 0)
#pragma unroll
        for (int h = 0; h < GH; h++) ws[key][h] = seen ? sc[h] : -kInf;
    __syncthreads();
    // weights: a warp per head
    const bool alone = !CL && L.count <= span;
    const int64_t id0 = (int64_t)lane_i * A.n_heads + head0;
    if (warp < GH && n > 0) {
        float x[KM / 32], m = -kInf, l = 0.0f;
#pragma unroll
        for (int u = 0; u < KM / 32; u++) x[u] = ws[lane + 32 * u][warp], m = fmaxf(m, x[u]);
        m = warp_max(m);
        const bool some = m > -kInf;
        if (!some) m = 0.0f;  // (nothing seen, scores of minus infinity or NaN alone)
#pragma unroll
        for (int u = 0; u < KM / 32; u++) {
            x[u] = al_ex2(__fsub_rn(x[u], m));
            l += x[u];
            ws[lane + 32 * u][warp] = x[u];
        }
        l = warp_psum(l);
        if (!some && l == 0.0f) m = -kInf;  // (no say in what the other pieces are relative to)
        if (lane == 0) {
            inv[warp] = !alone ? 1.0f : l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
            if (CL)
                stat[warp] = make_float4(m, l, 0.0f, 0.0f);
            else if (!alone && warp < heads)
                ml[(id0 + warp) * splits + s] = make_float2(m, l);
        }
    }
    __syncthreads();
    // values: a word of eight dims of every kGroups-th key per thread
    const int w = tid % C::kWords, gi = tid / C::kWords;
    float acc[GH][8];
#pragma unroll
    for (int h = 0; h < GH; h++)
#pragma unroll
        for (int d = 0; d < 8; d++) acc[h][d] = 0.0f;
#pragma unroll 2
    for (int j = gi; j < n; j += C::kGroups) {
        if (!ok[j]) continue;
        __half2 sc2, m24;
        kv4_scale2(scales[1][j * PER + w / 4], sc2, m24);
        float f[8];
        decode8f(*reinterpret_cast<const uint32_t *>(rows[1] + j * C::kRow + w * 4), sc2, m24, f);
#pragma unroll
        for (int h = 0; h < GH; h++) {
            const float x = ws[j][h];
#pragma unroll
            for (int d = 0; d < 8; d++) acc[h][d] = __fmaf_rn(x, f[d], acc[h][d]);
        }
    }
    __syncthreads();  // the rows' place takes the groups' sums, [kGroups][GH][HD]
    float *const red = reinterpret_cast<float *>(few_smem);
#pragma unroll
    for (int h = 0; h < GH; h++)
#pragma unroll
        for (int d = 0; d < 8; d += 4)
            *reinterpret_cast<float4 *>(red + (gi * GH + h) * HD + w * 8 + d) =
                make_float4(acc[h][d], acc[h][d + 1], acc[h][d + 2], acc[h][d + 3]);
    __syncthreads();
    constexpr int NV = HD / 4;
    for (int e = tid; e < heads * NV; e += kThreads) {
        const int h = e / NV, dd = (e % NV) * 4;
        float4 a = *reinterpret_cast<const float4 *>(red + h * HD + dd);
        for (int u = 1; u < C::kGroups; u++) {
            const float4 b = *reinterpret_cast<const float4 *>(red + (u * GH + h) * HD + dd);
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
        }
        if constexpr (CL) {
            *reinterpret_cast<float4 *>(red + h * HD + dd) = a;
            continue;
        }
        const float f = inv[h];
        float *to = alone ? A.out + (id0 + h) * HD : part + ((id0 + h) * splits + s) * HD;
        *reinterpret_cast<float4 *>(to + dd) = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
    }
    if constexpr (CL) {
        // the cluster's CTAs share the outputs out: as many threads to four dims as there are CTAs (2, 4, 8 or 16), one
        // for each one's sums
        cluster_sync();
        const int lg = splits <= 2 ? 1 : splits <= 4 ? 2 : splits <= 8 ? 3 : 4, r = tid & ((1 << lg) - 1);
        const int items = heads * NV, share = (items + splits - 1) / splits;
        for (int i0 = 0; i0 < share; i0 += kThreads >> lg) {
            const int at = i0 + (tid >> lg), i = s * share + at, h = min(i, items - 1) / NV, dd = (i - h * NV) * 4;
            const bool on = at < share && i < items;
            float4 st = make_float4(-kInf, 0.0f, 0.0f, 0.0f), v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (on && r < splits) st = ld_peer_f4(&stat[h], (uint32_t)r);
            const bool some = st.x > -kInf;
            if (some) v = ld_peer_f4(red + h * HD + dd, (uint32_t)r);
            float m = st.x;
            for (int off = 1 << lg >> 1; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            const float x = some ? al_ex2(__fsub_rn(st.x, m)) : 0.0f;
            float l = x * st.y;
            v.x *= x, v.y *= x, v.z *= x, v.w *= x;
            for (int off = 1 << lg >> 1; off > 0; off >>= 1) {
                l += __shfl_xor_sync(0xffffffffu, l, off);
                v.x += __shfl_xor_sync(0xffffffffu, v.x, off), v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
                v.z += __shfl_xor_sync(0xffffffffu, v.z, off), v.w += __shfl_xor_sync(0xffffffffu, v.w, off);
            }
            const float f = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
            if (on && r == 0)
                *reinterpret_cast<float4 *>(A.out + (id0 + h) * HD + dd) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
        }
        cluster_sync();  // nobody leaves while its sums are read
    }
}

// grid (heads, lanes, dims / kMergeDims): the partial sums of one (lane, head)
// by the weights 2^(maximum - largest maximum).
__global__ void __launch_bounds__(kThreads) kv4_few_merge_kernel(const __grid_constant__ Kv4Args A, const float2 *ml,
                                                                 const float *part, int splits, int span) {
    __shared__ float w[kMaxSplits];
    __shared__ float red[8];
    __shared__ float4 acc[kThreads];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hd = A.hd;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const LaneKeys L(A, blockIdx.y);
    const int n = (L.count + span - 1) / span;
    if (n <= 1) return;  // done already
    const int64_t id = (int64_t)blockIdx.y * A.n_heads + blockIdx.x, row0 = id * splits;
    float m = -kInf;
    for (int k = tid; k < n; k += kThreads) m = fmaxf(m, __ldcg(&ml[row0 + k]).x);
    m = warp_max(m);
    if (lane == 0) red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; k++) m = fmaxf(m, red[k]);
    __syncthreads();
    if (!(m > -kInf)) m = 0.0f;
    float l = 0.0f;
    for (int k = tid; k < n; k += kThreads) {
        const float2 v = __ldcg(&ml[row0 + k]);
        w[k] = al_ex2(__fsub_rn(v.x, m));
        l += w[k] * v.y;
    }
    l = warp_psum(l);
    if (lane == 0) red[warp] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++) l += red[k];
    constexpr int nv = kMergeDims / 4, groups = kThreads / nv;
    const int gi = tid / nv, dv = blockIdx.z * nv + tid % nv;  // four dims, every 16th piece
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int k = gi; k < n; k += groups) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(part + (row0 + k) * hd) + dv);
        const float x = w[k];
        a.x += v.x * x, a.y += v.y * x, a.z += v.z * x, a.w += v.w * x;
    }
    acc[tid] = a;
    __syncthreads();
    if (tid < nv) {
        for (int k = 1; k < min(groups, n); k++) {
            const float4 v = acc[k * nv + tid];
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
        const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
        reinterpret_cast<float4 *>(A.out + id * hd)[dv] = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    }
}

// ------------------------------------------------------------------ the product
// A tile is up to 32 rows (the query heads of one KV head, of lanes of one
// sequence on end); the tiles' chunks of 128 keys are dealt to one CTA per SM in
// equal runs, a run's parts of a tile joined by a merging launch: the plan and
// its order are attention_lanes.cuh's.  Per chunk
//   S^T [128 keys x rows] = K [128 x hd] q^T,   O^T [hd x rows] += V^T [hd x 128] P^T
// with the codes decoded to fp16, which is exact: an fp16 has 11 bits and the
// range of every code times its scale.  Queries and weights are two fp16 terms
// each (22 bits; a row's queries times a power of two that puts the largest at
// 2^13 .. 2^14), side by side as columns of one operand, so that the products
// are good to fp32's rounding.  The keys are the products' rows because there
// are 128 of them and few queries: the decoded operand is then the A of both, K
// from tensor memory (written straight from registers) and V from shared memory
// with the keys as its rows.
//
// Roles: one warp walks over the plan, one looks up pages and copies codes and
// scales (2-D tensor copies, a page at a time, with the copy engine's swizzle),
// 16 warps decode, a thread issues the MMAs, two warpgroups turn S^T into
// weights and add up O^T, which is taken out of tensor memory after every chunk.
// With up to 16 rows the warpgroups take the chunks in turn, each with running
// maxima and outputs of its own, joined at the end of a tile; with more they
// share the rows.  A maximum is only raised when a score exceeds it by kStale.
//
// Measured (4 query heads on one KV head of 256 unless said): 64 lanes of up to
// 8192 keys 50 us for 106 MB of cache, 2.1 TB/s; 16 lanes of up to 32768 keys,
// 8 heads on each of two of 128, 60 us for 111 MB; 64 lanes with a window of 1024
// 25 us; two prompts of 1024 lanes with that window 70 us.  A chunk takes some
// 3200 cycles, of which DRAM is busy 28% and the tensor cores 12%: the decoding
// threads' instructions (60% of the issue slots, 7 us of the 51 without the
// arithmetic) and the hand-overs from step to step bound it.  Around that a
// start of 4 us, 5 us where a CTA goes from one tile to the next, and the merge
// of 4 us, which is most of the window's 25.  Taken back after timing: the
// decode with a packed add and multiply in place of three of the shifts (6 us
// more), K's and V's slices by all producers in one order (slower), the next
// tile's queries loaded under the last products (1 us more).
constexpr int kR = 32;                // rows of a tile at most
constexpr int kProd = 16;             // producer warps, in groups of four
constexpr int kProd0 = 8;             // behind two warpgroups of the weights
constexpr int kMma = kProd0 + kProd;  // the warp that issues the MMAs; then the ones that describe pieces and copy
constexpr int kWalk = kMma + 1, kCopy = kMma + 2;
constexpr int kTcThreads = 32 * (kMma + 4);
constexpr int kVSlot = 16384;         // 64 keys x 128 dims of V
constexpr int kVRing = 6 * kVSlot;    // half chunks
constexpr int kMaxStages = 4;         // chunks of codes of K, and of V
constexpr int kBadRing = 64;
// tensor memory: S^T twice [2 kR], O^T [4 kR], K of two chunks
constexpr uint32_t kTmS = 0, kTmO = 4 * kR, kTmK = 8 * kR, kTmCols = 512;
constexpr float kStale = 4.0f;        // how far a score may exceed the maximum in use
constexpr float kUp = 2048.0f;        // weights are multiplied by this: below 2^15, and steps of 2^-35 of the largest

struct KvMaps {
    CUtensorMap k, v;
};

template <int HD>
struct KvCfg {
    static constexpr int nK = HD / 64;               // slices of 64 dims of a chunk's K
    static constexpr int nDH = (HD + 127) / 128, nV = 2 * nDH;  // slices of 64 keys x 128 dims of V
    static constexpr int kCodes = kChunk * HD / 2, kScales = kChunk * HD / 32, kStage = kCodes + kScales;
    // The producer groups' slices of every chunk: with 256 dims one of K and one of V each, else groups 0 (and 1, with
    // 128) K's, groups 2 and 3 V's
    static constexpr bool kBoth = HD == 256;
    static constexpr int kKWarps = 4 * nK, kVWarps = 4 * nV;  // warps that read a chunk's codes
    static constexpr int kHalf = nDH * kVSlot, kHalves = kVRing / kHalf;  // half a chunk of V in the ring, and how many
    static constexpr uint32_t kKCols = 32 * nK;               // tensor memory columns of a chunk's K
    static_assert(kTmK + 2 * kKCols <= kTmCols, "tensor memory");
};

struct KvCtl {
    uint64_t kfull[2], vfull[6], vempty[6];
    uint64_t kst_full[kMaxStages], kst_empty[kMaxStages], vst_full[kMaxStages], vst_empty[kMaxStages];
    uint64_t s_full[2], s_free[2], p_ready[2], pv_done[2], q_ready, drain;
    uint64_t pc_full[kPieceRing], pc_empty[kPieceRing];
    uint32_t bad[kBadRing];   // per chunk: pages that are out of range
    int rowid[kR];            // lane * n_heads + head
    int rowlo[kR], rowhi[kR]; // a row sees the keys <= rowhi that are > rowlo or first ones
    float qf[kR];             // what a row's scores are multiplied by
    float mc[kR], sum[kR], alpha[kR];  // of a warpgroup's 16 rows each
    float red[4][kR];
    float *optr[kR];
    AlSelfPlan plan;
    AlPiece piece[kPieceRing];
    int chunks;               // all of them, once that is known
    uint32_t tmem;
    int abort;
};

// In shared memory: the ring of V, the rows' q (per 64 dims the two terms'
// rows), the weights P, the stages' codes (K's, V's), their scales.
template <int HD>
struct KvLayout {
    using C = KvCfg<HD>;
    int q, qslice, p, codes, scales, nks, nvs;
    __device__ __forceinline__ KvLayout(int rmax) {
        qslice = 2 * (rmax <= 16 ? 16 : 32) * 128;
        q = kVRing;
        p = q + C::nK * qslice;
        codes = p + 2 * kChunk * 64;
        const int n = min((kAlSmem - 1024 - (int)sizeof(KvCtl) - 16 - codes) / C::kStage, 2 * kMaxStages);
        nks = (n + 1) / 2, nvs = n / 2;
        scales = codes + n * C::kCodes;
    }
};
static_assert(kAlSmem - 1024 - (int)sizeof(KvCtl) - 16 - kVRing - 4 * 2 * 32 * 128 - 2 * kChunk * 64 >=
                  4 * KvCfg<256>::kStage,
              "two stages of K and two of V");

// D (tensor memory) (+)= A (tensor memory) x B (shared memory)
__device__ __forceinline__ void kv_mma_ta(uint32_t d, uint32_t a, uint32_t blo, uint32_t bhi, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(blo), "r"(bhi), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void kv_tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint32_t f16x2(float a, float b) {  // a in the low half
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// two values as two pairs of fp16 terms: hi + lo is 22 bits of them, and steps of 2^-25 at least
__device__ __forceinline__ void kv_split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = f16x2(a, b);
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    lo = f16x2(__fsub_rn(a, h.x), __fsub_rn(b, h.y));
}
// a barrier of both warpgroups of the weights, and whether v holds anywhere
__device__ __forceinline__ bool kv_bar_or(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 3, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

// A wait of a whole warp: its lanes go on, or give up, together.
__device__ __forceinline__ bool kv_wait_all(uint64_t *bar, uint32_t parity, int *abort) {
    return __all_sync(0xffffffffu, al_wait(bar, parity, abort));
}

template <int HD>
__global__ void __launch_bounds__(kTcThreads, 1)
    kv4_attn_kernel(const __grid_constant__ KvMaps maps, const __grid_constant__ AlArgs A, const __grid_constant__ AlDims D,
                    const __grid_constant__ AlWs W, const __grid_constant__ qlin_kv4 kv) {
    using C = KvCfg<HD>;
    constexpr int nK = C::nK, nDH = C::nDH;
    extern __shared__ uint8_t kv_raw[];
    uint8_t *const smem = kv_raw + ((1024u - (smem_addr(kv_raw) & 1023u)) & 1023u);  // the swizzled operands' alignment
    KvCtl &S = *reinterpret_cast<KvCtl *>(smem + (kAlSmem - 1024 - sizeof(KvCtl)) / 16 * 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == kMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&S.tmem)),
                     "r"(kTmCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
        for (int s = 0; s < 2; s++) mbar_init(&S.kfull[s], C::kKWarps);
        for (int s = 0; s < C::kHalves; s++) mbar_init(&S.vfull[s], C::kVWarps / 2), mbar_init(&S.vempty[s], 1);
        for (int s = 0; s < kMaxStages; s++) {
            mbar_init(&S.kst_full[s], 1), mbar_init(&S.kst_empty[s], C::kKWarps);
            mbar_init(&S.vst_full[s], 1), mbar_init(&S.vst_empty[s], C::kVWarps);
        }
        // (a chunk's weights come from both warpgroups, a warp's first lane arriving, or from one, its first two)
        for (int s = 0; s < 2; s++)
            mbar_init(&S.s_full[s], 1), mbar_init(&S.s_free[s], 8), mbar_init(&S.p_ready[s], 8), mbar_init(&S.pv_done[s], 1);
        mbar_init(&S.q_ready, 8), mbar_init(&S.drain, 1);
        for (int s = 0; s < kPieceRing; s++) mbar_init(&S.pc_full[s], 1), mbar_init(&S.pc_empty[s], 8 + 2);
        S.chunks = INT_MAX;
        S.abort = 0;
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan, and what the kernels before wrote
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    AlPlan P{W.head, W.first + blockIdx.x, W.tile_of, W.tiles};
    if (A.n_lanes <= kSelfPlan) {
        AlSelfScratch &x = *reinterpret_cast<AlSelfScratch *>(smem);  // (the ring is not in use yet)
        if (tid < kSelfPlan) {
            make_plan<kSelfPlan>(A, D, x.lane, x.red, &S.plan.head, &S.plan.first, blockIdx.x, x.tile_of, S.plan.tiles,
                                 blockIdx.x == 0 ? A.status : nullptr);
            fence_proxy_async_smem();
        }
        P = AlPlan{&S.plan.head, &S.plan.first, nullptr, S.plan.tiles};
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    const KvLayout<HD> L(P.head->rmax);
    uint8_t *const ring = smem, *const qs = ring + L.q, *const ps = ring + L.p;
    uint8_t *const codes = ring + L.codes, *const scales = ring + L.scales;  // K's stages, then V's
    auto give_up = [&]() {
        S.abort = 1;
        raise_status(A.status, kStatusTimeout);
    };

    if (warp >= kProd0 && warp < kMma) {
        // ---------------------------------------------------------- producers: a slice of K or V per group of four warps,
        // 64 dims of a key per thread
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const int pg = (warp - kProd0) >> 2, t = tid & 127;
        const bool does_k = C::kBoth || pg < nK, does_v = C::kBoth || pg >= 2;
        const int ev = C::kBoth ? pg : pg - 2, kh = ev / nDH, dh = ev % nDH;  // (a slice of V: half the keys, 128 dims)
        const bool v_dims = nDH * 128 == HD || t < 64;
        auto place = [&](int row, int group) {  // of a group of 32 dims in a stage (the copies' swizzle)
            const int x = HD == 256 ? row & 7 : HD == 128 ? (row >> 1) & 3 : (row >> 2) & 1;
            return (uint32_t)(row * (HD / 2) + ((group ^ x) << 4));
        };
        // where this thread's codes and scales lie in a stage of K and of V
        const int vrow = 64 * kh + (t & 63), vg = 4 * dh + 2 * (t >> 6);
        const uint32_t k0 = place(t, 2 * pg), k1 = place(t, 2 * pg + 1), ks = (uint32_t)(t * (HD / 32) + 2 * pg);
        const uint32_t v0 = place(vrow, vg), v1 = place(vrow, vg + 1), vs = (uint32_t)(vrow * (HD / 32) + vg);
        const uint32_t to_v = smem_addr(ring) + (uint32_t)(dh * kVSlot + (t >> 6) * 8192 + (t & 63) * 128);
        const uint32_t to_k = tmem + kTmK + 32u * (uint32_t)pg + ((uint32_t)(32 * (warp & 3)) << 16);
        int kst = 0, vst = 0;
        uint32_t kpar = 0, vpar = 0;
        int vslot = kh;
        uint32_t vround = 0;
        bool ok = true;
        for (int c = 0; ok && (does_k || does_v); c++) {
            bool end = false;
            if (does_k) {
                if (!(ok = kv_wait_all(&S.kst_full[kst], kpar, &S.abort))) break;
                end = c >= *(volatile int *)&S.chunks;
                if (!end) {
                    const uint8_t *from = codes + kst * C::kCodes;
                    const uint4 a = lds128(from + k0), b = lds128(from + k1);
                    const uint32_t sc = *reinterpret_cast<const uint16_t *>(scales + kst * C::kScales + ks);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.kst_empty[kst]);
                    if (++kst == L.nks) kst = 0, kpar ^= 1u;
                    const int slot = c & 1, round = c >> 1;
                    if (round && !(ok = kv_wait_all(&S.s_full[slot], (uint32_t)(round - 1) & 1u, &S.abort))) break;
                    __syncwarp();
                    tc_fence_after();  // (the scores that read what lay there)
                    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        __half2 s2, m2;
                        kv4_scale2(h ? sc >> 8 : sc & 255u, s2, m2);
                        uint32_t o[16];
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            uint32_t x[4];
                            kv4_decode8(w[4 * h + i], s2, m2, x);
                            o[4 * i] = x[0], o[4 * i + 1] = x[1], o[4 * i + 2] = x[2], o[4 * i + 3] = x[3];
                        }
                        tm_st16(to_k + C::kKCols * (uint32_t)slot + 16u * h, o);
                    }
                    tm_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.kfull[slot]);
                }
            }
            if (does_v && (!does_k || c > 0)) {
                if (!(ok = kv_wait_all(&S.vst_full[vst], vpar, &S.abort))) break;
                if (!does_k && (end = c >= *(volatile int *)&S.chunks)) break;
                uint4 a, b;
                uint32_t sc = 0;
                if (v_dims) {
                    const uint8_t *from = codes + (L.nks + vst) * C::kCodes;
                    a = lds128(from + v0), b = lds128(from + v1);
                    sc = *reinterpret_cast<const uint16_t *>(scales + (L.nks + vst) * C::kScales + vs);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.vst_empty[vst]);
                if (++vst == L.nvs) vst = 0, vpar ^= 1u;
                if (vround && !(ok = kv_wait_all(&S.vempty[vslot], (vround - 1) & 1u, &S.abort))) break;
                if (v_dims) {
                    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        __half2 s2, m2;
                        kv4_scale2(h ? sc >> 8 : sc & 255u, s2, m2);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            uint32_t o[4];
                            kv4_decode8(w[4 * h + i], s2, m2, o);
                            sts128(to_v + (uint32_t)(vslot * C::kHalf + (((4 * h + i) ^ (t & 7)) << 4)),
                                   make_uint4(o[0], o[1], o[2], o[3]));
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.vfull[vslot]);
                vslot += 2;
                if (vslot >= C::kHalves) vslot -= C::kHalves, vround++;
            }
            if (end) break;
        }
        if (!ok) give_up();
    } else if (warp >= kMma) {
        // 896 threads are launched with 72 registers (64512 in all): 128 x 40 here, 256 x 120 for the weights and
        // 512 x 56 for the producers are as many.  (With 40, 104 and 64 the weights spilled more: 64 lanes of up to 8192
        // keys took 51.4 us, 50.3 now, two prompts 73.3, 70.6 now.  56, 128 and 48: 50.7 and 70.2.)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == kWalk && al_elect()) {
            // ------------------------------------------------------ describes the pieces
            Walker w(P, D);
            for (int k = 0;; k++) {
                const int r = k % kPieceRing;
                if (k >= kPieceRing && !al_wait(&S.pc_empty[r], (uint32_t)(k / kPieceRing - 1) & 1u, &S.abort)) {
                    give_up();
                    break;
                }
                w.next(S.piece[r], A, D);
                const bool end = S.piece[r].n == 0;
                mbar_arrive(&S.pc_full[r]);
                if (end) break;
            }
        }
        if (warp == kCopy) {
            // ------------------------------------------------------ copies the chunks' codes and scales: a lane per page of
            // a chunk, four chunks' pages looked up at a time
            PieceRef ref;
            int it = 0, kst = 0, vst = 0;  // chunks so far, the next stages
            uint32_t kround = 0, vround = 0;
            int ks_n = 0, vs_n = 0;        // stages filled
            bool ok = true;
            const int lp = 31 - __clz(kv.page_rows), per = max(1, kChunk >> lp), e = lane & 7, rows = min(kChunk, kv.page_rows);
            // a chunk whose pages lie at the rows `row` of the pool (lanes 0 .. 7; -1: nothing to read)
            auto fill = [&](bool v, int row) -> bool {
                int &st = v ? vst : kst;
                uint32_t &round = v ? vround : kround;
                uint64_t *const full = v ? &S.vst_full[st] : &S.kst_full[st];
                if (round && !kv_wait_all(v ? &S.vst_empty[st] : &S.kst_empty[st], (round - 1) & 1u, &S.abort))
                    return false;
                const bool on = lane < per && row >= 0;
                const int pages = __popc(__ballot_sync(0xffffffffu, on));
                if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(pages * rows * (HD / 2 + HD / 32)));
                __syncwarp();
                if (on) {
                    const int s = (v ? L.nks : 0) + st;
                    kv_tma_2d(smem_addr(codes + s * C::kCodes + lane * rows * (HD / 2)), v ? &maps.v : &maps.k, 0, row,
                              smem_addr(full));
                    bulk_g2s_l2(scales + s * C::kScales + lane * rows * (HD / 32),
                                static_cast<const uint8_t *>(v ? kv.v_scale : kv.k_scale) + (int64_t)row * (HD / 32),
                                (uint32_t)(rows * (HD / 32)), full);
                }
                __syncwarp();
                if (++st == (v ? L.nvs : L.nks)) st = 0, round++;
                (v ? vs_n : ks_n)++;
                return true;
            };
            while (ok) {
                const AlPiece *p = ref.next(S);
                if (!(ok = __all_sync(0xffffffffu, p != nullptr))) break;
                const int n = p->n;
                if (n == 0) {
                    if (lane == 0) *(volatile int *)&S.chunks = it;
                    ok = fill(false, -1) && fill(true, -1);  // (empty ones, behind the last)
                    break;
                }
                const int kvh = p->kvh;
                const int32_t *table = kv.table + (int64_t)p->slot * kv.table_stride;
                int row4 = -1, prev = -1;  // of this lane's page: in the four chunks, in the chunk before
                for (int i = 0; i <= n && ok; i++) {
                    if (i < n && (i & 3) == 0) {
                        const int c = i + (lane >> 3), b = c < n ? p->row0(c) : 0, k0 = b + (e << lp);
                        row4 = -1;
                        bool miss = false;
                        if (c < n && e < per && p->any_in(k0, k0 + rows)) {
                            const int id = __ldg(table + (k0 >> lp));
                            miss = id < 0 || id >= kv.n_pages;
                            if (!miss) row4 = ((id * A.n_kv + kvh) << lp) + (k0 & ((1 << lp) - 1));
                        }
                        const uint32_t bad = __ballot_sync(0xffffffffu, miss);
                        if (bad && lane == 0) raise_status(A.status, kStatusBadLane);
                        if (e == 0 && c < n) S.bad[(it + c) % kBadRing] = bad >> (lane & 24) & 255u;
                        __syncwarp();
                    }
                    const int row = __shfl_sync(0xffffffffu, row4, (i & 3) * 8 + e);
                    if (i < n) ok = fill(false, row);
                    if (ok && i > 0) ok = fill(true, prev);
                    prev = row;
                }
                it += n;
                if (ok && lane == 0) ref.done(S);
            }
            if (!ok) {
                give_up();
                // the copies in flight
                for (int k = max(0, ks_n - L.nks); k < ks_n; k++) mbar_wait(&S.kst_full[k % L.nks], (uint32_t)(k / L.nks) & 1u);
                for (int k = max(0, vs_n - L.nvs); k < vs_n; k++) mbar_wait(&S.vst_full[k % L.nvs], (uint32_t)(k / L.nvs) & 1u);
            }
        }
        if (warp == kMma && al_elect()) {
            // ------------------------------------------------------ the MMAs
            PieceRef ref;
            int it = 0;  // chunks so far
            bool ok = true;
            const uint32_t qs_a = smem_addr(qs), ps_a = smem_addr(ps), qstep = (uint32_t)L.qslice >> 4;
            const uint32_t ring_d = al_desc_lo(smem_addr(ring), 8192);
            const uint32_t hi128 = al_desc_hi(1024, 2), hip = al_desc_hi(512, 4);
            int vslot = 0;
            uint32_t vpar = 0;
            while (ok) {
                const AlPiece *p = ref.next(S);
                if (!(ok = p != nullptr)) break;
                const int n = p->n;
                if (n == 0) break;
                const uint32_t nr = p->nrows <= 16 ? 16 : 32;
                const bool turns = nr == 16;  // the warpgroups take chunks in turn, each with weights and outputs of its own
                // fp32 accumulator, fp16 operands, N = the two terms' rows; S^T: q K-major, O^T: both with the keys as rows
                const uint32_t ids = (1u << 4) | (128u >> 4) << 24 | (2 * nr >> 3) << 17, idp = ids | (1u << 15) | (1u << 16);
                if (!(ok = al_wait(&S.q_ready, (uint32_t)ref.k & 1u, &S.abort))) break;
                for (int i = 0; i <= n; i++) {
                    if (i < n) {
                        const int g = it + i;
                        if (g >= 2 && !(ok = al_wait(&S.s_free[g & 1], (uint32_t)((g >> 1) - 1) & 1u, &S.abort))) break;
                        const uint32_t d = tmem + kTmS + (uint32_t)(g & 1) * 2 * kR;
                        const uint32_t b0 = al_desc_lo(qs_a, 16);
                        if (!(ok = al_wait(&S.kfull[g & 1], (uint32_t)(g >> 1) & 1u, &S.abort))) break;
                        tc_fence_after();
                        const uint32_t a = tmem + kTmK + C::kKCols * (uint32_t)(g & 1);
#pragma unroll
                        for (int kk = 0; kk < 4 * nK; kk++)
                            kv_mma_ta(d, a + 8u * kk, b0 + qstep * (kk / 4) + 2u * (kk % 4), hi128, ids, kk > 0);
                        tc_commit(&S.s_full[g & 1]);
                    }
                    if (i >= 1) {
                        const int g = it + i - 1;
                        if (!(ok = al_wait(&S.p_ready[g & 1], (uint32_t)(g >> 1) & 1u, &S.abort))) break;
                        const uint32_t d = tmem + kTmO + (turns ? (uint32_t)(g & 1) * 64u : 0u);
                        const uint32_t pa = ps_a + (turns ? (uint32_t)(g & 1) * (kChunk * 64) : 0u);
#pragma unroll
                        for (int kh = 0; kh < 2; kh++) {
                            if (!(ok = al_wait(&S.vfull[vslot], vpar, &S.abort))) break;
                            tc_fence_after();
                            const uint32_t a0 = ring_d + (uint32_t)(vslot * (C::kHalf / 16));
                            const uint32_t b0 = al_desc_lo(pa + kh * 64 * 64, kChunk * 64);
#pragma unroll
                            for (int dh = 0; dh < nDH; dh++)
#pragma unroll
                                for (int k4 = 0; k4 < 4; k4++)
                                    al_mma(d + (uint32_t)dh * 2 * nr, a0 + (uint32_t)(dh * (kVSlot / 16)) + 128u * k4, hi128,
                                           b0 + 64u * k4, hip, idp, k4 > 0 || kh > 0);
                            tc_commit(&S.vempty[vslot]);
                            if (++vslot == C::kHalves) vslot = 0, vpar ^= 1u;
                        }
                        if (!ok) break;
                        tc_commit(&S.pv_done[g & 1]);
                    }
                }
                it += n;
                if (ok) ref.done(S);
            }
            if (!ok) give_up();
            tc_commit(&S.drain);  // the MMAs in flight (others may have given up)
            mbar_wait(&S.drain, 0);
        }
    } else {
        // ---------------------------------------------------------- weights and sums: thread t of a warpgroup owns key t of a
        // chunk, and of the outputs dims t and t + 128.  Up to 16 rows the warpgroups take the chunks in turn and add up at
        // the end; more, and warpgroup wg owns rows 16 wg .. 16 wg + 15 of every chunk.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
        const int wg = warp >> 2, t = tid & 127, own = 16 * wg;  // own: this warpgroup's place in what both have 16 of
        PieceRef ref;
        int it = 0;  // chunks so far
        const int lp = kv.page_rows >= kChunk ? 7 : 31 - __clz(kv.page_rows);
        bool ok = true;
        while (true) {
            const AlPiece *p = ref.next(S);
            __syncwarp();
            if (p == nullptr) give_up();
            if (kv_bar_or(p == nullptr || !ok)) break;  // (and the rows of the last piece are no longer needed)
            const int n = p->n, nrows = p->nrows, nr = nrows <= 16 ? 16 : 32;
            if (n == 0) break;
            const bool turns = nr == 16;
            const int r0 = turns ? 0 : own;
            if (t < 16) {
                const int r = r0 + t, gs = p->gs, ln = p->lane0 + r / gs;
                const bool in = r < nrows;
                const int pl = in ? A.positions[ln] - p->base : -1;
                S.rowid[r] = in ? ln * A.n_heads + p->head0 + r % gs : -1;  // (in turns: both write the same)
                S.rowhi[r] = max(-1, min(pl, p->lim - 1));
                S.rowlo[r] = A.window && pl >= A.window ? pl - A.window : -1;
                S.mc[own + t] = in ? kNoKey : kInf;  // (what lies in the place of a row that is not there gets no weight)
            }
            kv_bar_or(false);
            // the rows' q with the softmax's scale, multiplied by a power of two that brings the largest value of the row
            // to 2^13 .. 2^14, as two fp16 terms
            constexpr int per = HD / 8;  // threads to a row
#pragma unroll 2
            for (int e = tid; e < nr * per; e += 256) {
                const int r = e / per, d8 = e % per;
                const bool in = r < nrows;
                uint4 a, b;
                al_ld32(A.q + (in ? (int64_t)S.rowid[r] * HD + 8 * d8 : 0), in, a, b);
                float x[8] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
                              __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; k++) x[k] = __fmul_rn(x[k], D.c), top = fmaxf(top, fabsf(x[k]));
#pragma unroll
                for (int off = 1; off < per; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const int k2 = top < kInf ? min(126, 140 - (int)(__float_as_uint(top) >> 23)) : 0;
                const float f = __uint_as_float((uint32_t)(k2 + 127) << 23);
                if (d8 == 0) S.qf[r] = __uint_as_float((uint32_t)(127 - k2) << 23);
#pragma unroll
                for (int k = 0; k < 8; k++) x[k] = __fmul_rn(x[k], f);
                uint4 h, l;
                kv_split2(x[0], x[1], h.x, l.x), kv_split2(x[2], x[3], h.y, l.y);
                kv_split2(x[4], x[5], h.z, l.z), kv_split2(x[6], x[7], h.w, l.w);
                const uint32_t at = smem_addr(qs) + (uint32_t)((d8 >> 3) * L.qslice + r * 128 + (((d8 & 7) ^ (r & 7)) << 4));
                sts128(at, h);
                sts128(at + nr * 128, l);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.q_ready);
            kv_bar_or(false);  // (the rows' factors)
            const int arrivals = turns ? 2 : 1;
            const uint32_t half = 2 * nr;  // columns of O^T's second half of dims behind the first
            const uint32_t lanes_at = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
            const uint32_t at_o = lanes_at + kTmO + (turns ? 64u * wg : (uint32_t)r0);
            const uint32_t at_p = smem_addr(ps) + (turns ? (uint32_t)wg * (kChunk * 64) : 0u) + (uint32_t)t * 64;
            float lsum[16], acc[nDH][16];
#pragma unroll
            for (int j = 0; j < 16; j++) {
                lsum[j] = 0.0f;
#pragma unroll
                for (int h = 0; h < nDH; h++) acc[h][j] = 0.0f;
            }
            // 16 columns' terms of the products
            auto sum2 = [&](uint32_t at, float (&o)[16]) {
                uint32_t h[16], l[16];
                tm_ld16_nw(at, h);
                tm_ld16_nw(at + nr, l);
                tm_wait_ld(h);
                tm_wait_ld(l);
#pragma unroll
                for (int j = 0; j < 16; j++) o[j] = __fadd_rn(__uint_as_float(h[j]), __uint_as_float(l[j]));
            };
            // adds a chunk's products to the outputs
            auto take = [&]() {
#pragma unroll
                for (int h = 0; h < nDH; h++) {
                    float o[16];
                    sum2(at_o + h * half, o);
#pragma unroll
                    for (int j = 0; j < 16; j++) acc[h][j] = __fadd_rn(acc[h][j], o[j]);
                }
            };

            const int step = turns ? 2 : 1, i0 = turns ? (it ^ wg) & 1 : 0;  // this warpgroup's chunks
            int last = -1;  // the last one
            for (int i = i0; i < n; i += step) {
                const int g = it + i, cr = p->row0(i), sk = p->sk, key = cr + t;
                const bool fail = !al_wait(&S.s_full[g & 1], (uint32_t)(g >> 1) & 1u, &S.abort);
                __syncwarp();  // (the tensor-memory loads are for whole warps)
                tc_fence_after();
                const uint32_t bad = S.bad[g % kBadRing];
                const bool edge = p->edge_in(cr, cr + kChunk) || bad;
                float s[16];
                sum2(lanes_at + kTmS + (uint32_t)(g & 1) * 2 * kR + (uint32_t)r0, s);
                tc_fence_before();
                __syncwarp();
                if (lane < arrivals) mbar_arrive(&S.s_free[g & 1]);
                // whether row r of the tile sees this thread's key
                const bool there = !(bad >> (t >> lp) & 1u);
                auto sees = [&](int r) { return there && key <= S.rowhi[r] && (key > S.rowlo[r] || key < sk); };
                if (edge)
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (!sees(r0 + j)) s[j] = -kInf;
                bool big = last < 0;
                // (a power of two times a score is exact: one rounding)
                auto over = [&](int j) { return __fmaf_rn(s[j], S.qf[r0 + j], -S.mc[own + j]); };
                float e[16];
                if (last >= 0)
#pragma unroll
                    for (int j = 0; j < 16; j++) e[j] = over(j), big |= e[j] > kStale;
                const bool update = al_bar_or(wg, big || fail);
                if (update) {
                    if (al_bar_or(wg, fail)) {
                        if (fail) give_up();
                        ok = false;
                        break;
                    }
                    // new maxima
                    float m[16];
#pragma unroll
                    for (int j = 0; j < 16; j++) m[j] = __fmul_rn(s[j], S.qf[r0 + j]);
                    const float top = al_reduce16<true>(m, lane);
                    if (lane < 16) S.red[warp & 3][own + lane] = top;
                    al_bar(wg);
                    if (t < 16) {
                        const int r = own + t;
                        const float mx = fmaxf(fmaxf(S.red[0][r], S.red[1][r]), fmaxf(S.red[2][r], S.red[3][r]));
                        const float old = S.mc[r], mc = mx > -kInf ? fmaxf(mx, old) : old;
                        S.mc[r] = mc;
                        S.alpha[r] = old == kNoKey ? 0.0f : al_ex2(__fsub_rn(old, mc));
                    }
                    al_bar(wg);
#pragma unroll
                    for (int j = 0; j < 16; j++) lsum[j] = __fmul_rn(lsum[j], S.alpha[own + j]), e[j] = over(j);
                }
                // (a masked score stays minus infinity, the weight 0)
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    s[j] = __fmul_rn(al_ex2(e[j]), kUp);
                    lsum[j] = __fadd_rn(lsum[j], s[j]);
                }
                if (last >= 0) {  // the products of the chunk before: P is read, and O^T is there
                    if (!al_wait(&S.pv_done[last & 1], (uint32_t)(last >> 1) & 1u, &S.abort)) S.abort = 1;
                    __syncwarp();
                }
                // the weights, as two fp16 terms, a key's rows side by side
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    uint4 w2[2];
                    kv_split2(s[8 * q], s[8 * q + 1], w2[0].x, w2[1].x);
                    kv_split2(s[8 * q + 2], s[8 * q + 3], w2[0].y, w2[1].y);
                    kv_split2(s[8 * q + 4], s[8 * q + 5], w2[0].z, w2[1].z);
                    kv_split2(s[8 * q + 6], s[8 * q + 7], w2[0].w, w2[1].w);
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const int c = u * nr + r0 + 8 * q;
                        sts128(at_p + (uint32_t)((c >> 5) * (kChunk * 64) + ((((c >> 3) & 3) ^ ((t >> 1) & 3)) << 4)), w2[u]);
                    }
                }
                if (last >= 0) {
                    tc_fence_after();
                    take();
                    if (update)
#pragma unroll
                        for (int j = 0; j < 16; j++) {
                            const float al = S.alpha[own + j];
#pragma unroll
                            for (int h = 0; h < nDH; h++) acc[h][j] = __fmul_rn(acc[h][j], al);
                        }
                }
                last = g;
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane < arrivals) mbar_arrive(&S.p_ready[g & 1]);
            }
            it += n;
            if (ok && last >= 0) {
                if (!(ok = al_wait(&S.pv_done[last & 1], (uint32_t)(last >> 1) & 1u, &S.abort))) S.abort = 1;
                __syncwarp();
                tc_fence_after();
                take();
                tc_fence_before();
            }
            // the sums over the keys
            const float l4 = al_reduce16<false>(lsum, lane);
            if (lane < 16) S.red[warp & 3][own + lane] = l4;
            if (kv_bar_or(!ok)) break;  // (the weights' place is free as well)
            if (t < 16) {
                const int r = own + t;
                S.sum[r] = (S.red[0][r] + S.red[1][r]) + (S.red[2][r] + S.red[3][r]);
            }
            // in turns: the warpgroups' halves of the rows change places, [half of dims][8 rows][128] in the weights' place
            float *const other = reinterpret_cast<float *>(ps) + (wg ^ 1) * 1024 * nDH, *const mine = reinterpret_cast<float *>(ps) + wg * 1024 * nDH;
            if (turns)
#pragma unroll
                for (int h = 0; h < nDH; h++)
#pragma unroll
                    for (int j = 0; j < 8; j++) other[(h * 8 + j) * 128 + t] = wg ? acc[h][j] : acc[h][8 + j];
            kv_bar_or(false);
            if (t < 16) {
                const int r = r0 + t;
                float *o = nullptr;
                float f0 = 1.0f, f1 = 0.0f;  // the factors of this warpgroup's sums and of the other's
                if (r < nrows) {
                    float l = S.sum[own + t], mc = S.mc[own + t];
                    if (turns) {
                        const float m1 = S.mc[(own ^ 16) + t], m = fmaxf(mc, m1);
                        f0 = mc == kNoKey ? 0.0f : al_ex2(__fsub_rn(mc, m));
                        f1 = m1 == kNoKey ? 0.0f : al_ex2(__fsub_rn(m1, m));
                        l = f0 * l + f1 * S.sum[(own ^ 16) + t];
                        mc = m;
                    }
                    if (mc == kInf) l = __int_as_float(0x7fc00000);  // (a score past fp32's range)
                    const int64_t id = S.rowid[r];
                    float inv = 1.0f;
                    if (p->whole) {
                        o = A.out + id * HD;
                        inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
                    } else {
                        const int64_t row = (int64_t)(2 * blockIdx.x + p->begins) * D.cap + r;
                        o = W.part + row * HD;
                        if (!turns || wg == 0) W.ml[row] = make_float2(mc, l);
                    }
                    f0 *= inv, f1 *= inv;
                }
                S.optr[own + t] = o;
                S.alpha[own + t] = f0;
                S.red[0][own + t] = f1;
            }
            al_bar(wg);
            if (lane == 0) ref.done(S);
            if (turns) {
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    float *o = S.optr[own + 8 * wg + j];
                    if (o) {
                        const float f0 = S.alpha[own + 8 * wg + j], f1 = S.red[0][own + 8 * wg + j];
#pragma unroll
                        for (int h = 0; h < nDH; h++)
                            if (HD >= 128 || t < HD)
                                o[t + 128 * h] = __fmaf_rn(wg ? acc[h][8 + j] : acc[h][j], f0, __fmul_rn(mine[(h * 8 + j) * 128 + t], f1));
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    float *o = S.optr[own + j];
                    if (o) {
                        const float f0 = S.alpha[own + j];
#pragma unroll
                        for (int h = 0; h < nDH; h++)
                            if (HD >= 128 || t < HD) o[t + 128 * h] = __fmul_rn(acc[h][j], f0);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && S.abort) raise_status(A.status, kStatusTimeout);  // (whoever saw it)
    if (warp == kMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmCols) : "memory");
}

// ------------------------------------------------------------------ host
int few_heads(int group) { return group <= 1 ? 1 : group <= 2 ? 2 : group <= 4 ? 4 : 8; }

bool sizes_ok(int n_lanes, int n_heads, int n_kv, int hd) {
    return n_lanes >= 1 && n_lanes <= kMaxLanes && n_kv >= 1 && n_heads >= n_kv && n_heads % n_kv == 0 &&
           n_heads <= 65535 && (hd == 64 || hd == 128 || hd == 256);
}

template <int HD, bool CL>
const void *few_kernel(int gh, size_t &smem) {
    smem = FewCfg<HD, CL>::bytes(gh);
    switch (gh) {
        case 1: return (const void *)kv4_few_kernel<HD, 1, CL>;
        case 2: return (const void *)kv4_few_kernel<HD, 2, CL>;
        case 4: return (const void *)kv4_few_kernel<HD, 4, CL>;
        default: return (const void *)kv4_few_kernel<HD, 8, CL>;
    }
}
template <bool CL>
const void *few_kernel(int hd, int gh, size_t &smem) {
    return hd == 64 ? few_kernel<64, CL>(gh, smem) : hd == 128 ? few_kernel<128, CL>(gh, smem) : few_kernel<256, CL>(gh, smem);
}

// The keys that a lane can see at most.
int64_t most_keys(const Kv4Args &A) {
    const int64_t rows = (int64_t)A.kv.max_pages * A.kv.page_rows;
    return A.window && (int64_t)A.window + A.sinks < rows ? (int64_t)A.window + A.sinks : rows;
}

// Whether a call is little work, by the caches' sizes (the positions are on the
// device): the multiply-adds of all its lanes at most, and partial sums that the
// workspace holds.  us per call here / on the tensor cores, whole caches in use:
// 4 query heads on one KV head of 256: one lane of 1024 8.2 / 13.7, 16 of 1024
// (34 M) 12.8 / 17.0, 16 of 2048 (67 M) 18.7 / 18.1, 16 of 4096 47 / 21; 8 on
// each of two of 128: 16 of 512 (34 M) 10.4 / 14.4, 16 of 1024 (67 M) 30.0 /
// 16.3; one on each of eight of 128: 16 of 1024 (34 M) 18.8 / 22.7, 64 of 1024
// (134 M) 59 / 60, 64 of 2048 100 / 84; one on each of four of 64: 64 of 2048
// (67 M) 32 / 43, 16 of 16384 (134 M) 63 / 58.
bool few_fits(const Kv4Args &A) {
    const int64_t keys = most_keys(A), splits = (keys + 63) / 64;
    const int gh = few_heads(A.group);
    int64_t rows;
    carve(A.n_lanes, A.n_heads, A.n_kv, A.hd, nullptr, &rows);
    return splits <= kMaxSplits && splits * A.n_lanes * A.n_heads <= rows &&
           (double)keys * A.n_lanes * A.n_heads * A.hd * 2 <= (gh >= 8 ? 40e6 : gh == 4 ? 55e6 : gh == 2 ? 80e6 : 110e6);
}

// The checks of a call's sizes, and what they make of its arguments.
qlin_status describe(const char *fn, const qlin_kv4 *kv, int n_lanes, int n_heads, int n_kv, int hd, int window, int sinks,
                     Kv4Args &A) {
    if (qlin_status st = check_kv4(fn, kv, n_kv, hd)) return st;
    QLIN_REQUIRE(n_lanes >= 1 && n_heads >= 1 && n_heads % n_kv == 0 && window >= 0 && sinks >= 0, QLIN_ERR_INVALID_ARG,
                 "%s: n_lanes %d, n_heads %d, n_kv %d, window %d, sinks %d", fn, n_lanes, n_heads, n_kv, window, sinks);
    QLIN_REQUIRE(sizes_ok(n_lanes, n_heads, n_kv, hd), QLIN_ERR_UNSUPPORTED, "%s: more than %d lanes (%d) or 65535 heads", fn,
                 kMaxLanes, n_lanes);
    A.kv = *kv, A.n_lanes = n_lanes, A.n_heads = n_heads, A.n_kv = n_kv, A.hd = hd, A.window = window, A.sinks = sinks;
    A.group = n_heads / n_kv;
    A.c = (float)(1.4426950408889634 / std::sqrt((double)hd));
    return QLIN_OK;
}

qlin_status attend_few(const Kv4Args &A, const AlWs &w, cudaStream_t st) {
    const int64_t keys = most_keys(A);
    const int gh = few_heads(A.group);
    int splits = (int)((keys + 63) / 64), span = 64;
    size_t smem;
    void *args[] = {(void *)&A, (void *)&w.ml, (void *)&w.part, (void *)&splits, (void *)&span};
    dim3 grid(splits, A.n_kv * ((A.group + gh - 1) / gh), A.n_lanes);
    // One launch if the CTAs of every (lane, head block) can be a cluster and no cluster has to wait for another's SMs.
    if (splits > 1 && keys <= kCluster * 128) {
        const int c = splits < kCluster ? splits : kCluster;
        const void *kern = few_kernel<true>(A.hd, gh, smem);
        if (max_clusters(kern, smem, kThreads, c) >= (int64_t)grid.y * grid.z) {
            splits = c, span = (int)((keys + c - 1) / c);
            grid.x = c;
            return launch_pdl(kern, grid, dim3(kThreads), smem, st, args, "kv4_few_kernel", c);
        }
    }
    const void *kern = few_kernel<false>(A.hd, gh, smem);
    blocks_per_sm(kern, smem);  // raises the dynamic shared-memory limit once
    if (qlin_status e = launch_pdl(kern, grid, dim3(kThreads), smem, st, args, "kv4_few_kernel")) return e;
    if (splits == 1) return QLIN_OK;
    return launch_pdl((const void *)kv4_few_merge_kernel, dim3(A.n_heads, A.n_lanes, A.hd / kMergeDims), dim3(kThreads), 0,
                      st, args, "kv4_few_merge_kernel");
}

// The tensor map of a pool's codes: its rows, boxes of a page or 128 of its
// rows, swizzled so that the 16 bytes of eight rows on end meet all banks.
qlin_status codes_map(const void *p, const qlin_kv4 &c, int n_kv, int hd, CUtensorMap *out) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)fn;
    }();
    QLIN_REQUIRE(encode, QLIN_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t gdim[2] = {(cuuint64_t)hd / 2, (cuuint64_t)c.n_pages * n_kv * c.page_rows}, gstride[1] = {(cuuint64_t)hd / 2};
    const cuuint32_t box[2] = {(cuuint32_t)hd / 2, (cuuint32_t)(c.page_rows < kChunk ? c.page_rows : kChunk)}, estride[2] = {1, 1};
    const CUtensorMapSwizzle swizzle = hd == 256   ? CU_TENSOR_MAP_SWIZZLE_128B
                                       : hd == 128 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                   : CU_TENSOR_MAP_SWIZZLE_32B;
    const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), gdim, gstride, box, estride,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    QLIN_REQUIRE(r == CUDA_SUCCESS, QLIN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return QLIN_OK;
}

qlin_status attend_tc(const Kv4Args &K, const AlWs &w, cudaStream_t st) {
    AlArgs A{};
    A.q = K.q, A.positions = K.positions, A.seqs = K.seqs, A.out = K.out, A.status = K.status;
    A.n_lanes = K.n_lanes, A.n_heads = K.n_heads, A.n_kv = K.n_kv, A.hd = K.hd, A.window = K.window, A.sinks = K.sinks;
    A.own.n_seqs = K.kv.n_seqs, A.own.rows = K.kv.max_pages * K.kv.page_rows;  // (what the plan goes by)
    AlDims D{};
    D.group = K.group, D.R = kR;
    D.LT = D.group < D.R ? D.R / D.group : 1;
    D.HB = (D.group + D.R - 1) / D.R;
    D.cap = (int64_t)A.n_lanes * D.group < D.R ? A.n_lanes * D.group : D.R;
    D.streams = 1;
    D.grid = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
    D.merge = A.n_lanes <= kSelfPlan ? 1 : 16;
    D.setup = 4;
    D.c = K.c;
    const void *kern = A.hd == 64    ? (const void *)kv4_attn_kernel<64>
                       : A.hd == 128 ? (const void *)kv4_attn_kernel<128>
                                     : (const void *)kv4_attn_kernel<256>;
    const size_t plan_smem = 6 * sizeof(int) * (size_t)A.n_lanes;
    QLIN_REQUIRE(kAlSmem <= max_smem_optin(), QLIN_ERR_UNSUPPORTED, "qlin_attention_kv4: shared memory");
    blocks_per_sm(kern, kAlSmem);  // raises the dynamic shared-memory limit once
    blocks_per_sm((const void *)al_plan_kernel, plan_smem);
    void *pargs[] = {(void *)&A, (void *)&D, (void *)&w};
    if (A.n_lanes > kSelfPlan)
        if (qlin_status e = launch_pdl((const void *)al_plan_kernel, dim3(1), dim3(kPlanThreads), plan_smem, st, pargs,
                                       "al_plan_kernel"))
            return e;
    KvMaps maps;
    if (qlin_status e = codes_map(K.kv.k, K.kv, A.n_kv, A.hd, &maps.k)) return e;
    if (qlin_status e = codes_map(K.kv.v, K.kv, A.n_kv, A.hd, &maps.v)) return e;
    void *args[] = {(void *)&maps, (void *)&A, (void *)&D, (void *)&w, (void *)&K.kv};
    if (qlin_status e = launch_pdl(kern, dim3(D.grid), dim3(kTcThreads), kAlSmem, st, args, "kv4_attn_kernel")) return e;
    const int64_t total = (int64_t)A.n_lanes * A.n_heads, blocks = (total + D.merge - 1) / D.merge;
    return launch_pdl((const void *)al_merge_kernel, dim3((unsigned)(blocks < 8 * D.grid ? blocks : 8 * D.grid)),
                      dim3(kMergeThreads), 0, st, pargs, "al_merge_kernel");
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

size_t qlin_attention_kv4_workspace_size(int n_lanes, int n_heads, int n_kv, int head_dim) {
    return sizes_ok(n_lanes, n_heads, n_kv, head_dim) ? carve(n_lanes, n_heads, n_kv, head_dim, nullptr).bytes : 0;
}

int qlin_attention_kv4_on_tensor_cores(const qlin_kv4 *kv, int n_lanes, int n_heads, int n_kv, int head_dim, int window,
                                       int sinks) {
    qlin::clear_error();
    const char *fn = "qlin_attention_kv4_on_tensor_cores";
    Kv4Args A{};
    if (qlin_status st = describe(fn, kv, n_lanes, n_heads, n_kv, head_dim, window, sinks, A)) return -(int)st;
    return few_fits(A) ? 0 : 1;
}

qlin_status qlin_attention_kv4(const float *q, const qlin_kv4 *kv, const int32_t *positions, const int32_t *seqs,
                               int n_lanes, int n_heads, int n_kv, int head_dim, int window, int sinks, float *out,
                               int32_t *status_word, void *workspace, size_t workspace_bytes, qlin_stream_t stream) {
    qlin::clear_error();
    const char *fn = "qlin_attention_kv4";
    Kv4Args A{};
    if (qlin_status st = describe(fn, kv, n_lanes, n_heads, n_kv, head_dim, window, sinks, A)) return st;
    QLIN_REQUIRE(q && positions && seqs && out && workspace, QLIN_ERR_INVALID_ARG, "%s: null pointer", fn);
    QLIN_REQUIRE(aligned16(q) && aligned16(out) && aligned16(workspace) && aligned4(positions) && aligned4(seqs) &&
                     aligned4(status_word),
                 QLIN_ERR_INVALID_ARG, "%s: q, out and workspace are 16-byte aligned (positions, seqs, status_word: 4)", fn);
    const AlWs w = carve(n_lanes, n_heads, n_kv, head_dim, (char *)workspace);
    QLIN_REQUIRE(workspace_bytes >= w.bytes, QLIN_ERR_INVALID_ARG, "%s: workspace %zu < %zu bytes", fn, workspace_bytes,
                 w.bytes);
    A.q = q, A.positions = positions, A.seqs = seqs, A.out = out, A.status = status_word;
    return few_fits(A) ? attend_few(A, w, (cudaStream_t)stream) : attend_tc(A, w, (cudaStream_t)stream);
}

}  // extern "C"
