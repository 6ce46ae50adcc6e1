// Attention over lanes with a sliding window and first tokens that reads the
// paged cache of 4 bits a value (qlin_attention_kv4).
//
// Lane i, at position p of its sequence, sees the keys at positions j <= p
// with j > p - window or j < sinks (every j <= p without a window); its query
// head h takes KV head h / (n_heads / n_kv) and gives
//   o = sum_j w_j v_j,  w = softmax_j(q . k_j / sqrt(head_dim)),
// zeros where no key is seen.
//
// A CTA takes one lane, up to GH query heads of one KV head and a run of the
// keys that the lane sees, counted without gaps (first tokens, then the
// window).  It goes through them 64 at a time with a running maximum and sum:
// their codes and scales into shared memory, scores and weighted values in
// fp32 on the CUDA cores.  The runs of one lane leave partial sums that a
// second kernel joins by the weights 2^(maximum - largest maximum).
#include <cmath>

#include "kv4.cuh"
#include "launch.cuh"
#include "stream.cuh"
#include "tcgen05.cuh"

namespace qlin {
namespace {

constexpr int kMaxLanes = 4096;
constexpr int kThreads = 256;
constexpr int kKeys = 64;          // keys of a step
constexpr int kParts = kThreads / kKeys;
constexpr int kMaxSplits = 1024;
constexpr int kMergeDims = 64;     // dims of a head per merging CTA

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

__device__ __forceinline__ float kv4_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
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

// grid (splits, KV heads x blocks of GH query heads, lanes); span: keys of a CTA
template <int HD, int GH>
__global__ void __launch_bounds__(kThreads) kv4_few_kernel(const __grid_constant__ Kv4Args A, float2 *ml, float *part,
                                                           int splits, int span) {
    constexpr int kRow = HD / 2 + 16, kPer = HD / 32;  // bytes between rows of codes; 16-byte groups, and scales, of a row
    constexpr int kWords = HD / 8, kGroups = kThreads / kWords;
    constexpr int kSums = kGroups * HD * 4, kBuf = 2 * kKeys * kRow > kSums ? 2 * kKeys * kRow : kSums;
    __shared__ __align__(16) uint8_t buf[kBuf];  // the keys' and the values' rows, then sums
    uint8_t *const rows[2] = {buf, buf + kKeys * kRow};
    __shared__ __align__(16) uint8_t scales[2][kKeys * kPer];
    __shared__ __align__(16) float qs[GH][HD];
    __shared__ __align__(16) float ws[kKeys][GH];
    __shared__ float sm[GH], sl[GH], sa[GH];  // running maximum and sum, the last step's factor
    __shared__ int ok[kKeys];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int s = blockIdx.x, blocks = (A.group + GH - 1) / GH, kvh = blockIdx.y / blocks, h0 = (blockIdx.y % blocks) * GH;
    const int lane_i = blockIdx.z, heads = min(GH, A.group - h0), head0 = kvh * A.group + h0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const LaneKeys L(A, lane_i);
    if (L.bad && s == 0 && blockIdx.y == 0 && tid == 0) raise_status(A.status, kStatusKv4Lane);
    const int n = min(span, L.count - s * span);
    if (n <= 0) {
        if (s == 0)
            for (int e = tid; e < heads * HD; e += kThreads) A.out[((int64_t)lane_i * A.n_heads + head0) * HD + e] = 0.0f;
        return;
    }
    for (int e = tid; e < GH * HD; e += kThreads)
        qs[e / HD][e % HD] = e / HD < heads ? A.q[((int64_t)lane_i * A.n_heads + head0) * HD + e] * A.c : 0.0f;
    if (tid < GH) sm[tid] = -kInf, sl[tid] = 0.0f;
    float acc[GH][8];
#pragma unroll
    for (int h = 0; h < GH; h++)
#pragma unroll
        for (int d = 0; d < 8; d++) acc[h][d] = 0.0f;
    const int w = tid % kWords, gi = tid / kWords;
    for (int x0 = 0; x0 < n; x0 += kKeys) {
        const int m = min(kKeys, n - x0);
        __syncthreads();
        for (int e = tid; e < m * kPer; e += kThreads) {
            const int r = e / kPer, c = e % kPer;
            const int64_t at = kv4_row(A.kv, A.n_kv, L.key(s * span + x0 + r), L.seq);
            if (c == 0) ok[r] = at >= 0;
            if (at < 0) continue;
            const int64_t row = at + (int64_t)kvh * A.kv.page_rows;
            cp_async16(rows[0] + r * kRow + c * 16, static_cast<const uint8_t *>(A.kv.k) + row * (HD / 2) + c * 16, 16);
            cp_async16(rows[1] + r * kRow + c * 16, static_cast<const uint8_t *>(A.kv.v) + row * (HD / 2) + c * 16, 16);
            scales[0][r * kPer + c] = static_cast<const uint8_t *>(A.kv.k_scale)[row * kPer + c];
            scales[1][r * kPer + c] = static_cast<const uint8_t *>(A.kv.v_scale)[row * kPer + c];
        }
        cp_async_commit();
        cp_async_wait_pending<0>();
        __syncthreads();
        // scores: kParts threads share a key, 32 dims of it in turn
        const int key = tid / kParts, pt = tid % kParts;
        float sc[GH];
#pragma unroll
        for (int h = 0; h < GH; h++) sc[h] = 0.0f;
        const bool seen = key < m && ok[key];
        if (seen)
            for (int c = pt; c < kPer; c += kParts) {
                const uint4 u = lds128(rows[0] + key * kRow + c * 16);
                __half2 sc2, m24;
                kv4_scale2(scales[0][key * kPer + c], sc2, m24);
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
        if (key < m && pt == 0 && !seen) raise_status(A.status, kStatusKv4Lane);
#pragma unroll
        for (int off = 1; off < kParts; off <<= 1)
#pragma unroll
            for (int h = 0; h < GH; h++) sc[h] = __fadd_rn(sc[h], __shfl_xor_sync(0xffffffffu, sc[h], off));
        if (pt == 0)
#pragma unroll
            for (int h = 0; h < GH; h++) ws[key][h] = seen ? sc[h] : -kInf;
        __syncthreads();
        // weights: a warp per head
        if (warp < GH) {
            const float a = ws[lane][warp], b = ws[lane + 32][warp], old = sm[warp];
            const float top = fmaxf(old, warp_max(fmaxf(a, b)));
            const float base = top > -kInf ? top : 0.0f;  // (nothing seen yet)
            const float ea = kv4_ex2(__fsub_rn(a, base)), eb = kv4_ex2(__fsub_rn(b, base));
            const float sum = warp_psum(__fadd_rn(ea, eb));
            ws[lane][warp] = ea, ws[lane + 32][warp] = eb;
            if (lane == 0) {
                const float f = old > -kInf ? kv4_ex2(__fsub_rn(old, base)) : 0.0f;
                sl[warp] = __fmaf_rn(sl[warp], f, sum);
                sm[warp] = top, sa[warp] = f;
            }
        }
        __syncthreads();
        // values: a word of eight dims of every kGroups-th key per thread
#pragma unroll
        for (int h = 0; h < GH; h++)
#pragma unroll
            for (int d = 0; d < 8; d++) acc[h][d] = __fmul_rn(acc[h][d], sa[h]);
        for (int j = gi; j < m; j += kGroups) {
            if (!ok[j]) continue;
            __half2 sc2, m24;
            kv4_scale2(scales[1][j * kPer + w / 4], sc2, m24);
            float f[8];
            decode8f(*reinterpret_cast<const uint32_t *>(rows[1] + j * kRow + w * 4), sc2, m24, f);
#pragma unroll
            for (int h = 0; h < GH; h++) {
                const float x = ws[j][h];
#pragma unroll
                for (int d = 0; d < 8; d++) acc[h][d] = __fmaf_rn(x, f[d], acc[h][d]);
            }
        }
    }
    // the sum over the groups of keys: [kGroups][HD] for one head after the other, in the rows' place
    __syncthreads();
    float *red = reinterpret_cast<float *>(buf);
    const bool alone = L.count <= span;
#pragma unroll
    for (int h = 0; h < GH; h++) {
        if (h >= heads) break;
#pragma unroll
        for (int d = 0; d < 8; d += 4)
            *reinterpret_cast<float4 *>(red + gi * HD + w * 8 + d) =
                make_float4(acc[h][d], acc[h][d + 1], acc[h][d + 2], acc[h][d + 3]);
        __syncthreads();
        const int64_t id = (int64_t)lane_i * A.n_heads + head0 + h, row = id * splits + s;
        const float l = sl[h], inv = !alone ? 1.0f : l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
        for (int d = tid; d < HD; d += kThreads) {
            float a = red[d];
            for (int g = 1; g < kGroups; g++) a = __fadd_rn(a, red[g * HD + d]);
            (alone ? A.out + id * HD : part + row * HD)[d] = a * inv;
        }
        if (!alone && tid == 0) ml[row] = make_float2(sm[h], l);
        __syncthreads();
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
        w[k] = kv4_ex2(__fsub_rn(v.x, m));
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

// ------------------------------------------------------------------ host
size_t align256(size_t b) { return (b + 255) / 256 * 256; }

int few_heads(int group) { return group <= 1 ? 1 : group <= 2 ? 2 : group <= 4 ? 4 : 8; }

bool sizes_ok(int n_lanes, int n_heads, int n_kv, int hd) {
    return n_lanes >= 1 && n_lanes <= kMaxLanes && n_kv >= 1 && n_heads >= n_kv && n_heads % n_kv == 0 &&
           n_heads <= 65535 && (hd == 64 || hd == 128 || hd == 256);
}

struct Kv4Ws {
    float2 *ml;
    float *part;
    int splits;  // at most
    size_t bytes;
};

// CTAs of about four to an SM, whatever the lanes
Kv4Ws carve(int n_lanes, int n_heads, int n_kv, int hd, char *base) {
    Kv4Ws w{};
    const int group = n_heads / n_kv, gh = few_heads(group), blocks = n_kv * ((group + gh - 1) / gh);
    const int64_t ctas = (int64_t)n_lanes * blocks;
    w.splits = (int)(ctas >= 1024 ? 1 : 1024 / ctas);
    const size_t rows = (size_t)w.splits * n_lanes * n_heads;
    w.ml = (float2 *)base;
    w.bytes = align256(rows * sizeof(float2));
    w.part = (float *)(base ? base + w.bytes : nullptr);
    w.bytes += align256(rows * hd * sizeof(float));
    return w;
}

template <int HD>
const void *few_kernel(int gh) {
    switch (gh) {
        case 1: return (const void *)kv4_few_kernel<HD, 1>;
        case 2: return (const void *)kv4_few_kernel<HD, 2>;
        case 4: return (const void *)kv4_few_kernel<HD, 4>;
        default: return (const void *)kv4_few_kernel<HD, 8>;
    }
}

qlin_status attend_few(const Kv4Args &A, const Kv4Ws &w, cudaStream_t st) {
    const int64_t rows = (int64_t)A.kv.max_pages * A.kv.page_rows;
    const int64_t keys = A.window && (int64_t)A.window + A.sinks < rows ? (int64_t)A.window + A.sinks : rows;
    int64_t span = (keys + w.splits - 1) / w.splits;
    span = (span + kKeys - 1) / kKeys * kKeys;
    int splits = (int)((keys + span - 1) / span), ispan = (int)span;
    const int gh = few_heads(A.group);
    void *args[] = {(void *)&A, (void *)&w.ml, (void *)&w.part, (void *)&splits, (void *)&ispan};
    const void *kern = A.hd == 64 ? few_kernel<64>(gh) : A.hd == 128 ? few_kernel<128>(gh) : few_kernel<256>(gh);
    if (qlin_status e = launch_pdl(kern, dim3(splits, A.n_kv * ((A.group + gh - 1) / gh), A.n_lanes), dim3(kThreads), 0, st,
                                   args, "kv4_few_kernel"))
        return e;
    if (splits == 1) return QLIN_OK;
    return launch_pdl((const void *)kv4_few_merge_kernel, dim3(A.n_heads, A.n_lanes, A.hd / kMergeDims), dim3(kThreads), 0,
                      st, args, "kv4_few_merge_kernel");
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

size_t qlin_attention_kv4_workspace_size(int n_lanes, int n_heads, int n_kv, int head_dim) {
    return sizes_ok(n_lanes, n_heads, n_kv, head_dim) ? carve(n_lanes, n_heads, n_kv, head_dim, nullptr).bytes : 0;
}

qlin_status qlin_attention_kv4(const float *q, const qlin_kv4 *kv, const int32_t *positions, const int32_t *seqs,
                               int n_lanes, int n_heads, int n_kv, int head_dim, int window, int sinks, float *out,
                               int32_t *status_word, void *workspace, size_t workspace_bytes, qlin_stream_t stream) {
    qlin::clear_error();
    const char *fn = "qlin_attention_kv4";
    if (qlin_status st = check_kv4(fn, kv, n_kv, head_dim)) return st;
    QLIN_REQUIRE(q && positions && seqs && out && workspace, QLIN_ERR_INVALID_ARG, "%s: null pointer", fn);
    QLIN_REQUIRE(n_lanes >= 1 && n_heads >= 1 && n_heads % n_kv == 0 && window >= 0 && sinks >= 0, QLIN_ERR_INVALID_ARG,
                 "%s: n_lanes %d, n_heads %d, n_kv %d, window %d, sinks %d", fn, n_lanes, n_heads, n_kv, window, sinks);
    QLIN_REQUIRE(sizes_ok(n_lanes, n_heads, n_kv, head_dim), QLIN_ERR_UNSUPPORTED, "%s: more than %d lanes (%d) or 65535 heads",
                 fn, kMaxLanes, n_lanes);
    QLIN_REQUIRE(aligned16(q) && aligned16(out) && aligned16(workspace) && aligned4(positions) && aligned4(seqs) &&
                     aligned4(status_word),
                 QLIN_ERR_INVALID_ARG, "%s: q, out and workspace are 16-byte aligned (positions, seqs, status_word: 4)", fn);
    const Kv4Ws w = carve(n_lanes, n_heads, n_kv, head_dim, (char *)workspace);
    QLIN_REQUIRE(workspace_bytes >= w.bytes, QLIN_ERR_INVALID_ARG, "%s: workspace %zu < %zu bytes", fn, workspace_bytes,
                 w.bytes);
    Kv4Args A{q, *kv, positions, seqs, n_lanes, n_heads, n_kv, head_dim, window, sinks, out, status_word, n_heads / n_kv,
              (float)(1.4426950408889634 / std::sqrt((double)head_dim))};
    return attend_few(A, w, (cudaStream_t)stream);
}

}  // extern "C"
