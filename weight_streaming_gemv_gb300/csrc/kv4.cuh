// The cache of 4 bits a value on pages (qlin_kv4): where a position lies, what
// its bits stand for, and the host's checks of a description.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace qlin {

constexpr int kKv4Group = 32;  // dims that share a scale
constexpr int kStatusKv4Lane = 1, kStatusKv4NotFinite = 4;

// Where a lane's row lies: its number among all rows of the pool for KV head
// 0 (head h: + h * page_rows), or -1 (padding), or -2 (out of range).
__device__ __forceinline__ int64_t kv4_row(const qlin_kv4 &c, int n_kv, int p, int s) {
    if (p < 0) return -1;
    if (s < 0 || s >= c.n_seqs || p / c.page_rows >= c.max_pages) return -2;
    const int page = c.table[(int64_t)s * c.table_stride + p / c.page_rows];
    return page < 0 || page >= c.n_pages ? -2 : (int64_t)page * n_kv * c.page_rows + p % c.page_rows;
}

// A scale byte's number: its bits are an fp32 number's exponent, less a bias,
// and first three bits of mantissa.
__device__ __forceinline__ float kv4_scale(uint32_t b) { return __uint_as_float((b + (106u << 3)) << 20); }
// The byte of the least scale that is at least `need` (0 or more, or infinite).
__device__ __forceinline__ uint32_t kv4_scale_byte(float need) {
    const int b = (int)((__float_as_uint(need) + 0xFFFFFu) >> 20) - (106 << 3);
    return (uint32_t)min(max(b, 0), 255);
}

// Eight codes (a word) as four pairs of fp16 values in the dims' order: a
// nibble at bits 9 .. 6 of 0x4C00 is 16 + c, and (16 + c) s - 24 s = (c - 8) s
// in one instruction.  Exact: s has 4 significant bits, so 24 s has at most 5,
// the result at most 7, and all are multiples of 2^-24 below 2^16.
__device__ __forceinline__ void kv4_decode8(uint32_t w, __half2 s, __half2 m24, uint32_t (&o)[4]) {
    const uint32_t n[4] = {w << 6, w << 2, w >> 2, w >> 6};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t x = (n[i] & 0x03C003C0u) | 0x4C004C00u;
        const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&x), s, m24);
        o[i] = *reinterpret_cast<const uint32_t *>(&r);
    }
}
// s and -24 s of a scale byte, for kv4_decode8
__device__ __forceinline__ void kv4_scale2(uint32_t b, __half2 &s, __half2 &m24) {
    s = __float2half2_rn(kv4_scale(b));
    m24 = __hmul2(s, __float2half2_rn(-24.0f));
}

inline qlin_status check_kv4(const char *fn, const qlin_kv4 *c, int n_kv, int head_dim) {
    QLIN_REQUIRE(c && c->k && c->v && c->k_scale && c->v_scale && c->table, QLIN_ERR_INVALID_ARG, "%s: kv: null pointer", fn);
    QLIN_REQUIRE((((uintptr_t)c->k | (uintptr_t)c->v) & 31u) == 0 && aligned16(c->k_scale) && aligned16(c->v_scale) &&
                     aligned4(c->table),
                 QLIN_ERR_INVALID_ARG, "%s: kv: codes are 32-byte aligned, scales 16-byte, the table 4-byte", fn);
    QLIN_REQUIRE(c->n_pages >= 1 && c->n_seqs >= 1 && c->max_pages >= 1 && n_kv >= 1, QLIN_ERR_INVALID_ARG,
                 "%s: kv: %d pages, %d sequences of %d pages, %d KV heads", fn, (int)c->n_pages, (int)c->n_seqs,
                 (int)c->max_pages, n_kv);
    QLIN_REQUIRE(c->page_rows >= 16 && c->page_rows <= 256 && (c->page_rows & (c->page_rows - 1)) == 0,
                 QLIN_ERR_UNSUPPORTED, "%s: kv: %d rows to a page are not 16, 32, 64, 128 or 256", fn, (int)c->page_rows);
    QLIN_REQUIRE(head_dim == 64 || head_dim == 128 || head_dim == 256, QLIN_ERR_UNSUPPORTED,
                 "%s: head_dim %d is not 64, 128 or 256", fn, head_dim);
    QLIN_REQUIRE(c->table_stride >= c->max_pages && c->table_stride < (int64_t)1 << 40, QLIN_ERR_INVALID_ARG,
                 "%s: kv: table_stride %lld, %d pages of a sequence", fn, (long long)c->table_stride, (int)c->max_pages);
    QLIN_REQUIRE((int64_t)c->max_pages * c->page_rows <= 1 << 30 &&
                     (double)c->n_pages * n_kv * c->page_rows < 2147483648.0,
                 QLIN_ERR_UNSUPPORTED, "%s: kv: %d pages of %d rows, %d to a sequence, %d KV heads", fn, (int)c->n_pages,
                 (int)c->page_rows, (int)c->max_pages, n_kv);
    return QLIN_OK;
}

}  // namespace qlin
