// Appending keys and values to the paged cache of 4 bits a value, with the
// position's rotation applied on the way (qlin_kv4_append), and reading rows
// back as the values that they stand for (qlin_kv4_read).
//
// A head's row x of a lane at position p turns as
//   x'[i] = x[i] cos_p[i] - x[i+h] sin_p[i],  x'[i+h] = x[i] sin_p[i] + x[i+h] cos_p[i],  h = head_dim / 2
// and every 32 dims of a key or value are rounded to codes of one scale s, the
// least number (8 + m) 2^(e-24) that is at least max|x'| / 7.
//
// Everything is read once and written once, so memory bounds it, and a launch
// where there is little: 4096 lanes of 8 + 2 + 2 heads of 128 take 10.4 us (47
// MB, in good part in L2) and the reading back 4.6; one lane 2.6 and 1.7.  A
// thread takes four dims i .. i+3 and their partners
// i+h .. i+h+3, so that a rotation needs no other thread and may be in place;
// the eight threads of four low dims each are the 32 of one scale, as are their
// eight partners, and two neighbours' codes make a word.
#include "kv4.cuh"
#include "launch.cuh"
#include "stream.cuh"

namespace qlin {
namespace {

constexpr int kKv4Threads = 256;
constexpr int kKv4MaxLanes = 65536, kKv4MaxRead = 1 << 20;

struct AppendArgs {
    qlin_kv4 kv;
    const float *k, *v, *q;
    int64_t kv_stride, q_stride;
    float *q_out;
    const float *cos_t, *sin_t;
    int rope_rows;
    const int32_t *positions, *seqs;
    int n_heads, n_kv;
    int32_t *status;
};

// Four dims as codes: bits 0 .. 15 of the low and of the high halves' nibbles
// that these four have in their word (the first four dims of the word in the
// low byte of each half; the other thread's are shifted by 8).
__device__ __forceinline__ uint32_t code4(const float (&x)[4], float s) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        float r = rintf(__fdiv_rn(x[j], s));
        r = fminf(fmaxf(r, -7.0f), 7.0f);
        const uint32_t c = x[j] != x[j] ? 8u : (uint32_t)((int)r + 8);
        w |= c << (4 * (j >> 1) + 16 * (j & 1));
    }
    return w;
}

__device__ __forceinline__ float top8(const float (&x)[4]) {
    // (fmaxf passes over a NaN)
    float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m == m ? m : 0.0f;
}

__device__ __forceinline__ bool finite4(const float (&x)[4]) {
    bool ok = true;
#pragma unroll
    for (int j = 0; j < 4; j++) ok = ok && fabsf(x[j]) < __int_as_float(0x7f800000);
    return ok;
}

// Block x: a lane; y: its rows, PER threads to a head's row and ROWS rows to
// them, whose loads are on their way together.  The rows of a lane: the
// queries', then the keys', then the values'.
template <int PER, int ROWS>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(const __grid_constant__ AppendArgs A) {
    constexpr int HD = 8 * PER;
    const int heads = A.q ? A.n_heads : 0, rows = heads + 2 * A.n_kv, lane = blockIdx.x, j = threadIdx.x % PER;
    const int step = blockDim.x / PER, row0 = blockIdx.y * step * ROWS + threadIdx.x / PER;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int p = A.positions[lane];
    int64_t place = kv4_row(A.kv, A.n_kv, p, A.seqs[lane]);
    if (place >= 0 && A.cos_t && p >= A.rope_rows) place = -2;
    const bool live = place >= 0;
    if (place == -2 && row0 == 0 && j == 0) raise_status(A.status, kStatusKv4Lane);
    float lo[ROWS][4] = {}, hi[ROWS][4] = {}, c[4] = {}, s[4] = {};
    if (live) {
#pragma unroll
        for (int i = 0; i < ROWS; i++) {
            const int row = row0 + i * step, kv = row - heads, head = kv < 0 ? row : kv < A.n_kv ? kv : kv - A.n_kv;
            if (row >= rows) continue;
            const float *src = kv < 0 ? A.q + lane * A.q_stride : (kv < A.n_kv ? A.k : A.v) + lane * A.kv_stride;
            src += head * HD + 4 * j;
            const float4 a = *reinterpret_cast<const float4 *>(src), b = *reinterpret_cast<const float4 *>(src + HD / 2);
            lo[i][0] = a.x, lo[i][1] = a.y, lo[i][2] = a.z, lo[i][3] = a.w;
            hi[i][0] = b.x, hi[i][1] = b.y, hi[i][2] = b.z, hi[i][3] = b.w;
        }
        if (A.cos_t && row0 < rows - A.n_kv) {
            const int64_t o = (int64_t)p * (HD / 2) + 4 * j;
            const float4 c4 = __ldg(reinterpret_cast<const float4 *>(A.cos_t + o));
            const float4 s4 = __ldg(reinterpret_cast<const float4 *>(A.sin_t + o));
            c[0] = c4.x, c[1] = c4.y, c[2] = c4.z, c[3] = c4.w, s[0] = s4.x, s[1] = s4.y, s[2] = s4.z, s[3] = s4.w;
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS; i++) {
        const int row = row0 + i * step;
        if (row0 + i * step - (int)threadIdx.x / PER >= rows) break;  // (nobody's row)
        const int what = row < heads ? 0 : row < heads + A.n_kv ? 1 : 2;  // query, key, value (behind the last row: of no use)
        const int head = what == 0 ? row : row - heads - (what - 1) * A.n_kv;
        const bool on = row < rows;
        if (live && A.cos_t && what < 2)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float x = lo[i][e], y = hi[i][e];
                lo[i][e] = __fsub_rn(__fmul_rn(x, c[e]), __fmul_rn(y, s[e]));
                hi[i][e] = __fadd_rn(__fmul_rn(x, s[e]), __fmul_rn(y, c[e]));
            }
        if (on && what == 0) {
            float *to = A.q_out + ((int64_t)lane * A.n_heads + head) * HD + 4 * j;
            *reinterpret_cast<float4 *>(to) = make_float4(lo[i][0], lo[i][1], lo[i][2], lo[i][3]);
            *reinterpret_cast<float4 *>(to + HD / 2) = make_float4(hi[i][0], hi[i][1], hi[i][2], hi[i][3]);
        }
        if (!__any_sync(0xffffffffu, on && what > 0)) continue;
        // (whole warps from here on: a row's threads are 8, 16 or 32 of one warp)
        const uint32_t bl = kv4_scale_byte(__fdiv_rn(top8(lo[i]), 7.0f)), bh = kv4_scale_byte(__fdiv_rn(top8(hi[i]), 7.0f));
        const uint32_t l = code4(lo[i], kv4_scale(bl)), h = code4(hi[i], kv4_scale(bh));
        // the even thread writes the low dims' word, the odd one the high dims'
        const bool odd = j & 1;
        const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? l : h, 1);
        const uint32_t word = odd ? other | h << 8 : l | other << 8;
        if (live && on && what > 0) {
            const int64_t r = place + (int64_t)head * A.kv.page_rows;
            uint8_t *code = static_cast<uint8_t *>(what == 1 ? A.kv.k : A.kv.v) + r * (HD / 2);
            uint8_t *sc = static_cast<uint8_t *>(what == 1 ? A.kv.k_scale : A.kv.v_scale) + r * (HD / kKv4Group);
            *reinterpret_cast<uint32_t *>(code + (odd ? HD / 4 : 0) + (j >> 1) * 4) = word;
            if ((j & 7) < 2) sc[(odd ? HD / 64 : 0) + (j >> 3)] = (uint8_t)(odd ? bh : bl);
            if (!finite4(lo[i]) || !finite4(hi[i])) raise_status(A.status, kStatusKv4NotFinite);
        }
    }
}

struct ReadArgs {
    qlin_kv4 kv;
    const int32_t *positions, *seqs;
    int n_kv;
    float *k_out, *v_out;
    int32_t *status;
};

// Block x: a lane; y: its rows, the keys' and then the values'; a thread to a
// word of eight codes.
template <int PER>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const __grid_constant__ ReadArgs A) {
    constexpr int HD = 8 * PER;
    const int lane = blockIdx.x, row = blockIdx.y * (blockDim.x / PER) + threadIdx.x / PER, w = threadIdx.x % PER;
    if (row >= 2 * A.n_kv) return;
    const int which = row >= A.n_kv, head = row - which * A.n_kv;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t place = kv4_row(A.kv, A.n_kv, A.positions[lane], A.seqs[lane]);
    if (place == -2 && row == 0 && w == 0) raise_status(A.status, kStatusKv4Lane);
    float *to = which ? A.v_out : A.k_out;
    if (!to) return;
    float x[8] = {};
    if (place >= 0) {
        const int64_t r = place + (int64_t)head * A.kv.page_rows;
        const uint32_t word = *reinterpret_cast<const uint32_t *>(
            static_cast<const uint8_t *>(which ? A.kv.v : A.kv.k) + r * (HD / 2) + 4 * w);
        const float s = kv4_scale(static_cast<const uint8_t *>(which ? A.kv.v_scale : A.kv.k_scale)[r * (HD / kKv4Group) + w / 4]);
#pragma unroll
        for (int d = 0; d < 8; d++) x[d] = __fmul_rn((float)((int)(word >> (4 * (d >> 1) + 16 * (d & 1)) & 15u) - 8), s);
    }
    to += ((int64_t)lane * A.n_kv + head) * HD + 8 * w;
    *reinterpret_cast<float4 *>(to) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(to + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// The launch of one of the two for `rows` rows of every lane, `each` of them to
// a thread; the kernel by the threads to a row.
template <typename Args>
qlin_status launch_rows(const void *k8, const void *k16, const void *k32, const char *name, const Args &A, int n_lanes,
                        int rows, int each, int hd, cudaStream_t st) {
    const int per = hd / 8, most = ((rows + each - 1) / each * per + 31) / 32 * 32;
    const int threads = most < kKv4Threads ? most : kKv4Threads, block = threads / per * each;
    const int blocks = (rows + block - 1) / block;
    QLIN_REQUIRE(blocks <= 65535, QLIN_ERR_UNSUPPORTED, "%s: too many heads", name);
    void *args[] = {(void *)&A};
    return launch_pdl(per == 8 ? k8 : per == 16 ? k16 : k32, dim3((unsigned)n_lanes, (unsigned)blocks), dim3(threads), 0, st,
                      args, name);
}
template <int ROWS>
qlin_status launch_append(const AppendArgs &A, int n_lanes, int hd, cudaStream_t st) {
    return launch_rows((const void *)kv4_append_kernel<8, ROWS>, (const void *)kv4_append_kernel<16, ROWS>,
                       (const void *)kv4_append_kernel<32, ROWS>, "kv4_append_kernel", A, n_lanes,
                       (A.q ? A.n_heads : 0) + 2 * A.n_kv, ROWS, hd, st);
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

qlin_status qlin_kv4_append(const qlin_kv4 *kv, const float *k, const float *v, int64_t kv_stride, const float *q,
                            int64_t q_stride, float *q_out, const float *cos_t, const float *sin_t, int rope_rows,
                            const int32_t *positions, const int32_t *seqs, int n_lanes, int n_heads, int n_kv,
                            int head_dim, int32_t *status_word, qlin_stream_t stream) {
    qlin::clear_error();
    const char *fn = "qlin_kv4_append";
    if (qlin_status st = check_kv4(fn, kv, n_kv, head_dim)) return st;
    QLIN_REQUIRE(k && v && positions && seqs && !q == !q_out && !cos_t == !sin_t, QLIN_ERR_INVALID_ARG,
                 "%s: null pointer (q and q_out, cos_t and sin_t go together)", fn);
    QLIN_REQUIRE(n_lanes >= 1 && (!q || n_heads >= 1) && (!cos_t || rope_rows >= 1), QLIN_ERR_INVALID_ARG,
                 "%s: n_lanes %d, n_heads %d, rope_rows %d", fn, n_lanes, n_heads, rope_rows);
    QLIN_REQUIRE(n_lanes <= kKv4MaxLanes && (!q || n_heads <= 65535) && n_kv <= 65535, QLIN_ERR_UNSUPPORTED,
                 "%s: more than %d lanes (%d) or 65535 heads", fn, kKv4MaxLanes, n_lanes);
    QLIN_REQUIRE(aligned16(k) && aligned16(v) && aligned16(q) && aligned16(q_out) && aligned16(cos_t) && aligned16(sin_t) &&
                     aligned4(positions) && aligned4(seqs) && aligned4(status_word),
                 QLIN_ERR_INVALID_ARG, "%s: a pointer is not 16-byte aligned (positions, seqs, status_word: 4)", fn);
    const int64_t most = (int64_t)1 << 40;
    QLIN_REQUIRE(kv_stride >= (int64_t)n_kv * head_dim && kv_stride % 4 == 0 && kv_stride < most &&
                     (!q || (q_stride >= (int64_t)n_heads * head_dim && q_stride % 4 == 0 && q_stride < most)),
                 QLIN_ERR_INVALID_ARG, "%s: kv_stride %lld, q_stride %lld: a lane's rows at least, multiples of 4", fn,
                 (long long)kv_stride, (long long)q_stride);
    QLIN_REQUIRE(!q || q != q_out || q_stride == (int64_t)n_heads * head_dim, QLIN_ERR_INVALID_ARG,
                 "%s: in place with a q_stride of %lld", fn, (long long)q_stride);
    AppendArgs A{*kv, k, v, q, kv_stride, q_stride, q_out, cos_t, sin_t, rope_rows, positions, seqs, n_heads, n_kv, status_word};
    // One row to a thread where there are few lanes, for the shorter way, and four where there are many, for more loads
    // in flight.  us with one / with four: 8 + 2 + 2 heads of 128, 64 lanes 2.7 / 2.9, 608 3.2 / 3.3, 1216 4.1 / 3.9, 2432
    // 6.8 / 5.3, 4864 12.5 / 10.1; 16 + 16 + 16 heads of 128, 64 lanes 3.0 / 4.8, 608 7.4 / 7.5, 1216 13.6 / 12.9, 4864
    // 49 / 45.
    return n_lanes <= 4 * sm_count() ? launch_append<1>(A, n_lanes, head_dim, (cudaStream_t)stream)
                                     : launch_append<4>(A, n_lanes, head_dim, (cudaStream_t)stream);
}

qlin_status qlin_kv4_read(const qlin_kv4 *kv, const int32_t *positions, const int32_t *seqs, int n_lanes, int n_kv,
                          int head_dim, float *k_out, float *v_out, int32_t *status_word, qlin_stream_t stream) {
    qlin::clear_error();
    const char *fn = "qlin_kv4_read";
    if (qlin_status st = check_kv4(fn, kv, n_kv, head_dim)) return st;
    QLIN_REQUIRE(positions && seqs, QLIN_ERR_INVALID_ARG, "%s: null pointer", fn);
    QLIN_REQUIRE(n_lanes >= 1, QLIN_ERR_INVALID_ARG, "%s: n_lanes %d", fn, n_lanes);
    QLIN_REQUIRE(n_lanes <= kKv4MaxRead && n_kv <= 65535, QLIN_ERR_UNSUPPORTED, "%s: more than %d lanes (%d) or 65535 heads",
                 fn, kKv4MaxRead, n_lanes);
    QLIN_REQUIRE(aligned16(k_out) && aligned16(v_out) && aligned4(positions) && aligned4(seqs) && aligned4(status_word),
                 QLIN_ERR_INVALID_ARG, "%s: a pointer is not 16-byte aligned (positions, seqs, status_word: 4)", fn);
    ReadArgs A{*kv, positions, seqs, n_kv, k_out, v_out, status_word};
    return launch_rows((const void *)kv4_read_kernel<8>, (const void *)kv4_read_kernel<16>, (const void *)kv4_read_kernel<32>,
                       "kv4_read_kernel", A, n_lanes, 2 * n_kv, 1, head_dim, (cudaStream_t)stream);
}

}  // extern "C"
