// Attention over lanes with a sliding window and first tokens, over caches of
// their own (qlin_attention_lanes) and behind shared prompts kept once
// (qlin_attention_prefix).
//
// Lane i, at position p of its sequence, sees the keys at positions j <= p
// with j > p - window or j < sinks (every j <= p without a window); its query
// head h takes KV head h / (n_heads / n_kv) and gives
//   o = sum_j w_j v_j,  w = softmax_j(q . k_j / sqrt(head_dim)),
// zeros where no key is seen.
#include "common.cuh"
#include "stream.cuh"

namespace qlin {
namespace {

constexpr int kMaxLanes = 4096;
constexpr int kStatusBadLane = 1;

struct AlArgs {
    const float *q;
    qlin_kv own, pre;  // pre.k null: no prompts
    const int32_t *positions, *seqs, *prefix_len, *prefix_of;
    int n_lanes, n_heads, n_kv, hd, window, sinks;
    float *out;
    int32_t *status;
};

template <typename T>
__device__ __forceinline__ float kv_at(const void *p, int64_t i);
template <>
__device__ __forceinline__ float kv_at<float>(const void *p, int64_t i) {
    return static_cast<const float *>(p)[i];
}
template <>
__device__ __forceinline__ float kv_at<uint16_t>(const void *p, int64_t i) {
    return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
}

// grid (n_heads, n_lanes), 128 threads: 128 keys at a time, thread t scoring
// key t and summing dims t and t + 128, with the running maximum and sum.
template <typename T>
__global__ void __launch_bounds__(128) attn_simple_kernel(AlArgs A) {
    __shared__ float qs[256], ps[128], red[4];
    const int h = blockIdx.x, i = blockIdx.y, t = threadIdx.x, hd = A.hd;
    const int g = h / (A.n_heads / A.n_kv);
    const float ninf = -__int_as_float(0x7f800000);
    float *o = A.out + ((int64_t)i * A.n_heads + h) * hd;
    const int p = A.positions[i], s = A.seqs[i];
    const int f = A.pre.k ? (A.prefix_of ? A.prefix_of[i] : 0) : 0;
    bool ok = s >= 0 && s < A.own.n_seqs;
    int P = 0;
    if (A.pre.k) {
        ok = ok && f >= 0 && f < A.pre.n_seqs;
        P = ok ? A.prefix_len[f] : 0;
        ok = ok && P >= 0 && P <= A.pre.rows;
    }
    ok = ok && p - P < A.own.rows;
    if (p < 0 || !ok) {
        if (p >= 0 && t == 0 && h == 0) raise_status(A.status, kStatusBadLane);
        for (int d = t; d < hd; d += 128) o[d] = 0.0f;
        return;
    }
    for (int d = t; d < hd; d += 128) qs[d] = A.q[((int64_t)i * A.n_heads + h) * hd + d];
    float m = ninf, l = 0.0f, acc0 = 0.0f, acc1 = 0.0f;
    const float c = 1.0f / sqrtf((float)hd);
    const int lo = A.window ? max(0, p - A.window + 1) : 0;
    for (int j0 = 0; j0 <= p; j0 += 128) {
        if (j0 + 127 < lo && j0 >= A.sinks) continue;
        __syncthreads();
        const int j = j0 + t;
        const bool seen = j <= p && (j >= lo || j < A.sinks);
        const bool in = j < P;
        const int64_t row = in ? (int64_t)f * A.pre.seq_stride + (int64_t)j * A.pre.row_stride
                               : (int64_t)s * A.own.seq_stride + (int64_t)(j - P) * A.own.row_stride;
        float x = ninf;
        if (seen) {
            x = 0.0f;
            for (int d = 0; d < hd; d++) x += qs[d] * kv_at<T>(in ? A.pre.k : A.own.k, row + g * hd + d);
            x *= c;
        }
        float mx = warp_max(x);
        if ((t & 31) == 0) red[t >> 5] = mx;
        __syncthreads();
        mx = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float al = m > ninf ? expf(m - mx) : 0.0f;
        ps[t] = seen ? expf(x - mx) : 0.0f;
        m = mx;
        __syncthreads();
        l *= al, acc0 *= al, acc1 *= al;
        for (int u = 0; u < 128 && j0 + u <= p; u++) {
            const int ju = j0 + u;
            if (!(ju >= lo || ju < A.sinks)) continue;
            const bool iu = ju < P;
            const int64_t r = iu ? (int64_t)f * A.pre.seq_stride + (int64_t)ju * A.pre.row_stride
                                 : (int64_t)s * A.own.seq_stride + (int64_t)(ju - P) * A.own.row_stride;
            const void *v = iu ? A.pre.v : A.own.v;
            l += ps[u];
            if (t < hd) acc0 += ps[u] * kv_at<T>(v, r + g * hd + t);
            if (t + 128 < hd) acc1 += ps[u] * kv_at<T>(v, r + g * hd + t + 128);
        }
    }
    if (t < hd) o[t] = acc0 / l;
    if (t + 128 < hd) o[t + 128] = acc1 / l;
}

qlin_status check_kv(const char *fn, const char *what, const qlin_kv *c, int n_kv, int hd) {
    QLIN_REQUIRE(c && c->k && c->v, QLIN_ERR_INVALID_ARG, "%s: %s: null pointer", fn, what);
    QLIN_REQUIRE(c->type == QLIN_KV_F32 || c->type == QLIN_KV_BF16, QLIN_ERR_UNSUPPORTED, "%s: %s: type %d", fn, what,
                 (int)c->type);
    const int e = c->type == QLIN_KV_F32 ? 4 : 2;
    QLIN_REQUIRE(c->n_seqs >= 1 && c->rows >= 1, QLIN_ERR_INVALID_ARG, "%s: %s: %d sequences of %d rows", fn, what,
                 (int)c->n_seqs, (int)c->rows);
    QLIN_REQUIRE(c->row_stride >= (int64_t)n_kv * hd && c->seq_stride >= 0, QLIN_ERR_INVALID_ARG,
                 "%s: %s: row_stride %lld below n_kv * head_dim, or a negative seq_stride", fn, what,
                 (long long)c->row_stride);
    QLIN_REQUIRE(aligned16(c->k) && aligned16(c->v) && c->row_stride * e % 16 == 0 && c->seq_stride * e % 16 == 0,
                 QLIN_ERR_INVALID_ARG, "%s: %s: k, v and the strides are multiples of 16 bytes", fn, what);
    QLIN_REQUIRE(c->row_stride * e < (int64_t)1 << 40 && c->seq_stride * e < (int64_t)1 << 40, QLIN_ERR_UNSUPPORTED,
                 "%s: %s: a stride of 2^40 bytes or more", fn, what);
    return QLIN_OK;
}

bool sizes_ok(int n_lanes, int n_heads, int n_kv, int hd) {
    return n_lanes >= 1 && n_lanes <= kMaxLanes && n_kv >= 1 && n_heads >= n_kv && n_heads % n_kv == 0 &&
           n_heads <= 65535 && hd >= 16 && hd <= 256 && hd % 16 == 0;
}

qlin_status attend(const char *fn, const AlArgs &A, void *workspace, size_t workspace_bytes, qlin_stream_t stream) {
    QLIN_REQUIRE(A.q && A.positions && A.seqs && A.out && workspace, QLIN_ERR_INVALID_ARG, "%s: null pointer", fn);
    QLIN_REQUIRE(A.n_lanes >= 1 && A.n_heads >= 1 && A.n_kv >= 1 && A.n_heads % A.n_kv == 0 && A.window >= 0 &&
                     A.sinks >= 0,
                 QLIN_ERR_INVALID_ARG, "%s: n_lanes %d, n_heads %d, n_kv %d, window %d, sinks %d", fn, A.n_lanes,
                 A.n_heads, A.n_kv, A.window, A.sinks);
    QLIN_REQUIRE(sizes_ok(A.n_lanes, A.n_heads, A.n_kv, A.hd), QLIN_ERR_UNSUPPORTED,
                 "%s: head_dim %d is not a multiple of 16 in 16..256, or more than %d lanes (%d) or 65535 heads", fn, A.hd,
                 kMaxLanes, A.n_lanes);
    QLIN_REQUIRE(aligned16(A.q) && aligned16(A.out) && aligned16(workspace), QLIN_ERR_INVALID_ARG,
                 "%s: q, out and workspace are 16-byte aligned", fn);
    QLIN_REQUIRE(aligned4(A.positions) && aligned4(A.seqs) && aligned4(A.prefix_len) && aligned4(A.prefix_of) &&
                     aligned4(A.status),
                 QLIN_ERR_INVALID_ARG, "%s: pointer not 4-byte aligned", fn);
    const size_t need = qlin_attention_lanes_workspace_size(A.n_lanes, A.n_heads, A.n_kv, A.hd);
    QLIN_REQUIRE(workspace_bytes >= need, QLIN_ERR_INVALID_ARG, "%s: workspace %zu < %zu bytes", fn, workspace_bytes, need);
    const dim3 grid(A.n_heads, A.n_lanes);
    if (A.own.type == QLIN_KV_F32)
        attn_simple_kernel<float><<<grid, 128, 0, (cudaStream_t)stream>>>(A);
    else
        attn_simple_kernel<uint16_t><<<grid, 128, 0, (cudaStream_t)stream>>>(A);
    QLIN_LAUNCHED("attn_simple_kernel");
    return QLIN_OK;
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

size_t qlin_attention_lanes_workspace_size(int n_lanes, int n_heads, int n_kv, int head_dim) {
    return sizes_ok(n_lanes, n_heads, n_kv, head_dim) ? 256 : 0;
}

qlin_status qlin_attention_lanes(const float *q, const qlin_kv *kv, const int32_t *positions, const int32_t *seqs,
                                 int n_lanes, int n_heads, int n_kv, int head_dim, int window, int sinks, float *out,
                                 int32_t *status_word, void *workspace, size_t workspace_bytes, qlin_stream_t stream) {
    qlin::clear_error();
    if (qlin_status st = check_kv("qlin_attention_lanes", "kv", kv, n_kv, head_dim)) return st;
    AlArgs A{q, *kv, qlin_kv{}, positions, seqs, nullptr, nullptr, n_lanes, n_heads, n_kv, head_dim, window, sinks,
             out, status_word};
    return attend("qlin_attention_lanes", A, workspace, workspace_bytes, stream);
}

qlin_status qlin_attention_prefix(const float *q, const qlin_kv *prefix, const int32_t *prefix_len,
                                  const int32_t *prefix_of, const qlin_kv *kv, const int32_t *positions,
                                  const int32_t *seqs, int n_lanes, int n_heads, int n_kv, int head_dim, int window,
                                  int sinks, float *out, int32_t *status_word, void *workspace,
                                  size_t workspace_bytes, qlin_stream_t stream) {
    qlin::clear_error();
    if (qlin_status st = check_kv("qlin_attention_prefix", "prefix", prefix, n_kv, head_dim)) return st;
    if (qlin_status st = check_kv("qlin_attention_prefix", "kv", kv, n_kv, head_dim)) return st;
    QLIN_REQUIRE(prefix->type == kv->type, QLIN_ERR_INVALID_ARG, "qlin_attention_prefix: the caches' types differ");
    QLIN_REQUIRE(prefix_len, QLIN_ERR_INVALID_ARG, "qlin_attention_prefix: null pointer");
    AlArgs A{q, *kv, *prefix, positions, seqs, prefix_len, prefix_of, n_lanes, n_heads, n_kv, head_dim, window, sinks,
             out, status_word};
    return attend("qlin_attention_prefix", A, workspace, workspace_bytes, stream);
}

}  // extern "C"
