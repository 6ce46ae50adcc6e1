// Attention over lanes with a sliding window and first tokens, over caches of
// their own (qlin_attention_lanes) and behind shared prompts kept once
// (qlin_attention_prefix).
//
// Lane i, at position p of its sequence, sees the keys at positions j <= p
// with j > p - window or j < sinks (every j <= p without a window); its query
// head h takes KV head h / (n_heads / n_kv) and gives
//   o = sum_j w_j v_j,  w = softmax_j(q . k_j / sqrt(head_dim)),
// zeros where no key is seen.
//
// One product for every use.  The rows of a tile are the query heads of one KV
// head for the lanes that read the same sequence, 48 rows at most (32 with fp32
// caches): lanes of a prompt chunk, beams of a prompt, or one lane alone.  The
// keys and values are the large operand, so they take the tensor cores' 128
// rows and the tile's rows the columns:
//   S^T [128 keys][rows]      = K [keys][dims] . Q^T
//   O^T [head_dim][rows]     += V^T [dims][keys] . P^T
// (tcgen05.mma kind::f16, fp32 accumulators in tensor memory).  A few rows
// cost a few columns; nothing is padded to 128 rows.
//
// fp32 accuracy from bf16 operands: q, the weights P and an fp32 cache's
// values enter as three bf16 terms x = hi + mid + lo (24 bits), a bf16 cache's
// as they are; the products of terms whose orders add to at most two are
// accumulated: three for a bf16 cache, which are all there are, six for an fp32
// one, where mid lo + lo mid + lo lo is left out.  With mid at most 2^-7 and lo
// at most 2^-16 of a value's leading bit that is at most 2^-22 of the product, of
// either sign, and some 2^-26 on average.  The rows' terms stand side by side as
// the columns of one product, in the order of their size, so that a cached term
// is read once for all of them and each order has a sum of its own.
//
// A pass over the keys with a running maximum: q is multiplied by log2(e) /
// sqrt(head_dim) before it is cut into terms, so a weight is 2^(score - maximum)
// with one subtraction, which is exact for scores near the maximum however large
// they are.  The rows go to warpgroups, 16 each, and thread t of one owns key t
// of a 128-key chunk (a tensor-memory lane).  The maximum of a row is over
// threads, so it is only taken when some score exceeds the one in use by 8 (and
// for a tile's first chunk): otherwise weights relative to the maximum in use
// stay below 2^8 and nothing needs rescaling.  The sums stay in each thread's
// registers until the end, and so do the outputs: the tensor cores' accumulation
// rounds toward zero, so they sum over one chunk only.
//
// Work is dealt out by 128-key chunks: every CTA (one per SM) takes an equal
// run of the (tile, KV head, chunk) units, so a long sequence is split over
// many SMs and many short ones are packed, whatever the lengths, which are
// read on the device.  A tile that lies in one CTA is finished there; the
// others leave partial sums that a second kernel merges.  Up to 64 lanes every
// CTA plans for itself (two warps, a thread per lane); from there a kernel of
// one CTA plans once for all (15 us at 4096 lanes).  A tile's start (the rows'
// q, the first scores and maxima, the outputs) takes as long as four chunks of a
// bf16 cache or two of an fp32 one and is dealt out as that many.  Tiles of one
// sequence read the same chunks; each CTA takes its own in the order of their
// number modulo a CTA's units, so that they are read from memory once.
//
// Keys and values go through a ring of 16 KB slots (x 3 terms for an fp32
// cache): 128 keys x 64 dims of K, 64 keys x 128 dims of V.  The shared memory
// that the plan's widest tile leaves is ring.  A bf16 cache's are tensor
// copies (TMA, 128-byte swizzle) straight from the cache, issued by two warps;
// an fp32 cache's are loaded, split and stored by 16 warps.
//
// Rows that nobody in the tile may see (behind the last position, before the
// window) are set to zero before their product, and a value that only some
// rows of a tile may see is replaced by zero where it is not finite, with the
// sums of the rows that do see it made NaN: 0 x NaN would reach the others.
//
// What bounds it, at 256 dims and 4 query heads on one KV head in bf16 (us of a
// call in a graph; GB300):
//   64 lanes of their own, 4100 keys each: 57 (270 MB: 4.7 TB/s, 71% of a
//     measured copy; without any product 43: the tiles' starts are the rest);
//   64 lanes behind one prompt of 131072: 102.  Each 128-key chunk takes 4000
//     cycles: 2640 for the products' columns at the full rate, the rest
//     hand-overs between the thread that issues them and the warpgroups (with a
//     quarter of the products and no copies it is 93).  Caches are read once
//     (147 MB), the tensor pipe is busy half of the time;
//   two chunks of 2048 lanes, a window of 1024: 89 (98 to 102 where the inputs
//     change from call to call), of which 15 plan and 6 merge; a tile has 10
//     chunks, 3 of them with keys that some rows do not see (5000 cycles and
//     more), and a start;
// and 16 lanes of 32768 keys on fp32 caches, 8 heads on each of two KV heads of
// 128: 192 (836 MB, 4.4 TB/s: 65% of a measured copy; the producers wait for
// their loads two thirds of the time, with the 64 KB in flight that their
// registers hold, and split and store for a sixth; at these 16 rows of 128 dims
// 46 KB of shared memory are left over, as the ring's slots are 48).  On fp32
// caches two chunks of 512 lanes, a window of 1024, 4 heads on one of 256, take
// 87 (floor 11: six products of 3.6 GFLOP), 32 lanes behind one prompt of 32768,
// 4 heads on each of two of 128, 80 (floor 13, the same).
// Few keys per lane take another kernel, below.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <cmath>

#include "attention_lanes.cuh"

namespace qlin {
namespace {

// ------------------------------------------------------------------ the product
// NT: bf16 terms of a cached value (1: bf16 cache, 3: fp32 cache)
template <int NT>
struct AlCfg {
    static constexpr int R = NT == 1 ? 48 : 32;     // rows of a tile at most
    static constexpr int kWg = R / 16;              // warpgroups, 16 rows each
    static constexpr int kTerm = 16384;             // 128 keys x 64 dims, or 64 keys x 128 dims, in bf16
    static constexpr int kSlot = NT * kTerm;
    static constexpr int kProd = NT == 1 ? 2 : 16;  // producer warps (arrivals of a slot)
    // after the warpgroups, and the producers of an fp32 cache: a warp that issues the MMAs, one that describes the
    // pieces, two that copy the slices of a bf16 cache (half a slice each: one thread issues a copy in some 200 cycles,
    // 500 with all that goes with a slice) or one that describes those of an fp32 cache to the producers (registers are
    // dealt out by warpgroup)
    static constexpr int kProd0 = 4 * kWg;
    static constexpr int kMma = 4 * kWg + (NT == 1 ? 0 : kProd), kWalk = kMma + 1, kCopy = kMma + 2;
    static constexpr int kCopies = NT == 1 ? 2 : 1;
    static constexpr int kThreads = 32 * (kMma + 4);
    static constexpr uint32_t kCols = 512;          // S^T [3 R], then O^T's two halves of dims [3 R] each
    static constexpr uint32_t kO = 3 * R;
    static constexpr int kMaxSlots = NT == 1 ? 12 : 3;  // (bf16: at least six, more than a chunk's four slices of V)
};

// What a producer warp needs to load a slice of an fp32 cache.
struct __align__(16) AlSlice {
    const float *src;  // its first row and dim; null: no more slices
    int64_t stride;    // floats between rows
    int y0, any_lo, any_hi, sk;  // its first row; the rows that are seen
    int v, dims;       // a slice of V; dims from src on
    int64_t pad;
};
constexpr int kSliceRing = 4;

template <int NT>
struct AlCtl {
    using C = AlCfg<NT>;
    uint64_t full[C::kMaxSlots], empty[C::kMaxSlots];
    uint64_t s_full, s_free, p_ready, q_ready, pv_done, fix_go, fixed, drain;
    int rowid[C::R];  // lane * n_heads + head
    int rowlo[C::R], rowhi[C::R];  // a row sees the keys <= rowhi that are > rowlo or first ones
    int nan[C::R];    // it sees a value that is not finite and was replaced
    float mc[C::R], alpha[C::R];
    float red[4][C::R];
    AlSelfPlan plan;
    AlPiece piece[kPieceRing];
    uint64_t pc_full[kPieceRing], pc_empty[kPieceRing];
    float *optr[C::R];  // a row's outputs
    AlSlice slice[kSliceRing];
    uint64_t sl_full[kSliceRing], sl_empty[kSliceRing];
    uint32_t tmem;
    int abort;
};

// Shared memory: ring slots, then the rows' q (per 64 dims the three terms'
// rows, of 128 swizzled bytes), then the weights P (the terms' rows in blocks
// of 32, each [128 keys][64 swizzled bytes]), then the control block.  Rc: the
// widest tile's rows, rounded up to 16s.
template <int NT>
struct AlLayout {
    int q, qslice, p, slots;
    __device__ __forceinline__ AlLayout(int rmax, int hd) {
        const int Rc = max(16, (rmax + 15) / 16 * 16);
        qslice = 3 * Rc * 128;
        const int qb = (hd + 63) / 64 * qslice, pb = (3 * Rc + 31) / 32 * (kChunk * 64);
        slots = min((kAlSmem - 1024 - (int)sizeof(AlCtl<NT>) - qb - pb) / AlCfg<NT>::kSlot, AlCfg<NT>::kMaxSlots);
        q = slots * AlCfg<NT>::kSlot;
        p = q + qb;
    }
};
static_assert(kAlSmem - 1024 - (int)sizeof(AlCtl<1>) - 4 * 3 * 48 * 128 - 5 * 128 * 64 >= 6 * 16384, "ring of six");
static_assert(kAlSmem - 1024 - (int)sizeof(AlCtl<3>) - 4 * 3 * 32 * 128 - 3 * 128 * 64 >= 3 * 49152, "ring of three");

__device__ __forceinline__ void al_tma(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}


// Two values as three pairs of bf16 terms (the first value in the low half).
// The first term is cut off, so that the largest values stay finite, the second
// rounded to nearest: what is left then has either sign, is at most 2^-16 of the
// value's leading bit and fits the third, and the three add up to the value
// exactly (an infinity or NaN gives a NaN below itself).  With the second term
// cut off as well the products that are left out (al_attn_kernel) would all have
// the sign of those that are not, and be twice as large.
__device__ __forceinline__ void al_split2(float a, float b, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    hi = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    a = __fsub_rn(a, __uint_as_float(__float_as_uint(a) & 0xffff0000u));
    b = __fsub_rn(b, __uint_as_float(__float_as_uint(b) & 0xffff0000u));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(mid) : "f"(b), "f"(a));
    a = __fsub_rn(a, __uint_as_float(mid << 16));
    b = __fsub_rn(b, __uint_as_float(mid & 0xffff0000u));
    lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
// eight values as three 16-byte groups of bf16 terms
__device__ __forceinline__ void al_split8(const uint4 &a, const uint4 &b, uint4 &h, uint4 &m, uint4 &l) {
    al_split2(__uint_as_float(a.x), __uint_as_float(a.y), h.x, m.x, l.x);
    al_split2(__uint_as_float(a.z), __uint_as_float(a.w), h.y, m.y, l.y);
    al_split2(__uint_as_float(b.x), __uint_as_float(b.y), h.z, m.z, l.z);
    al_split2(__uint_as_float(b.z), __uint_as_float(b.w), h.w, m.w, l.w);
}

struct AlMaps {
    CUtensorMap k[2], v[2];  // stream 0 (prompts), stream 1 (own)
};

// The slices of a piece in the order in which they pass through the ring: K of
// chunk 0, then for every chunk K of the next one and its own V.  f(v, row,
// dim): a slice of V or K from that row and dim on; it returns false to stop.
// (One thread runs this among busy warps: what a piece's slices share is in
// registers.)
template <typename F>
__device__ __forceinline__ bool for_slices(const AlPiece &p, int nK, int nDH, F f) {
    const int n = p.n, c1 = p.c1, nsink = p.nsink, skip = p.cfirst - nsink;
    int c = p.first, prev = 0;
    for (int i = 0; i <= n; i++) {
        const int row = (c < nsink ? c : c + skip) * kChunk;
        if (++c == c1) c -= n;
        if (i < n)
            for (int sl = 0; sl < nK; sl++)
                if (!f(false, row, 64 * sl)) return false;
        if (i >= 1)
            for (int kh = 0; kh < 2; kh++)
                for (int dh = 0; dh < nDH; dh++)
                    if (!f(true, prev + 64 * kh, 128 * dh)) return false;
        prev = row;
    }
    return true;
}


// 64 dims of one key's values in a slice (row: their 128 swizzled bytes, of the slice's t-th key), a key that not every
// row sees: zeros where no row does, or where one is not finite; then the rows that see it are marked.
template <int NT>
__device__ __forceinline__ void al_look(AlCtl<NT> &S, const AlPiece &p, int key, uint32_t row, int t, int dims) {
    if (p.any_in(key, key + 1)) {
        uint32_t bad = 0;
#pragma unroll 4
        for (int q = 0; q < 8; q++)
            if (8 * q < dims) {
                const uint4 v = lds128_a(row + ((q ^ (t & 7)) << 4));
                // an exponent of all ones runs over into the sign's place
                bad |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                       ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
            }
        if (!(bad & 0x80008000u)) return;
        for (int r = 0; r < p.nrows; r++)
            if (key <= S.rowhi[r] && (key > S.rowlo[r] || key < p.sk)) S.nan[r] = 1;
    }
    for (int tt = 0; tt < NT; tt++)
#pragma unroll 4
        for (int q = 0; q < 8; q++) sts128(row + tt * AlCfg<NT>::kTerm + ((q ^ (t & 7)) << 4), make_uint4(0, 0, 0, 0));
}

template <int NT>
__global__ void __launch_bounds__(AlCfg<NT>::kThreads, 1)
    al_attn_kernel(const __grid_constant__ AlMaps maps, AlArgs A, AlDims D, AlWs W) {
    using C = AlCfg<NT>;
    constexpr int R = C::R;
    extern __shared__ uint8_t al_raw[];
    uint8_t *const smem = al_raw + ((1024u - (smem_addr(al_raw) & 1023u)) & 1023u);  // the swizzled operands' alignment
    AlCtl<NT> &S = *reinterpret_cast<AlCtl<NT> *>(smem + (kAlSmem - 1024 - sizeof(AlCtl<NT>)) / 16 * 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hd = A.hd;
    const int nK = (hd + 63) / 64, nDH = (hd + 127) / 128, nV = 2 * nDH;
    if (warp == C::kMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&S.tmem)),
                     "r"(C::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
        for (int s = 0; s < C::kMaxSlots; s++) {
            mbar_init(&S.full[s], C::kProd);
            mbar_init(&S.empty[s], 1);
        }
        mbar_init(&S.s_full, 1);
        mbar_init(&S.s_free, 4 * C::kWg);
        // every warpgroup's warps arrive for every chunk and piece, with rows in it or not: no wait can then be
        // two phases behind
        mbar_init(&S.p_ready, 4 * C::kWg);
        mbar_init(&S.q_ready, 4 * C::kWg);
        for (int s = 0; s < kSliceRing; s++) {
            mbar_init(&S.sl_full[s], 1);
            mbar_init(&S.sl_empty[s], C::kProd);
        }
        for (int s = 0; s < kPieceRing; s++) {
            mbar_init(&S.pc_full[s], 1);
            mbar_init(&S.pc_empty[s], 4 * C::kWg + 1 + C::kCopies);  // the warpgroups' warps, MMA and copy warps
        }
        mbar_init(&S.pv_done, 1);
        mbar_init(&S.fix_go, 1);
        mbar_init(&S.fixed, 4);
        mbar_init(&S.drain, 1);
        S.abort = 0;
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan, and what the kernels before wrote
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    AlPlan P{W.head, W.first + blockIdx.x, W.tile_of, W.tiles};
    if (A.n_lanes <= kSelfPlan) {
        AlSelfScratch &x = *reinterpret_cast<AlSelfScratch *>(smem);  // (the ring is not in use yet)
        if (tid < kSelfPlan) {
            make_plan<kSelfPlan>(A, D, x.lane, x.red, &S.plan.head, &S.plan.first, blockIdx.x,
                                          x.tile_of, S.plan.tiles, blockIdx.x == 0 ? A.status : nullptr);
            fence_proxy_async_smem();
        }
        P = AlPlan{&S.plan.head, &S.plan.first, nullptr, S.plan.tiles};
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    const AlLayout<NT> L(P.head->rmax, hd);
    const int slots = L.slots;
    uint8_t *const ring = smem, *const qs = ring + L.q, *const ps = ring + L.p;

    if (NT == 3 && warp >= C::kProd0 && warp < C::kProd0 + C::kProd) {
        // ---------------------------------------------------------- producers of an fp32 cache's slices
        if constexpr (NT == 3) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // 64 rows at a time: eight threads take dims 4 pc .. + 3 of a row and the same 32 dims on (they read 128 bytes
        // of it at once); two such passes are a slice's 128 rows (a V slice's rows 64 .. 127 are the second 64 dims of
        // its 64 keys)
        // (a warp's four rows are 0, 4, 1, 5 or 2, 6, 3, 7 of eight: their swizzled halves fill all banks)
        const int pw = warp - C::kProd0, pj = lane >> 3, pc = lane & 7;
        const int pr = (pw >> 1) * 8 + (pw & 1) * 2 + (pj & 1) * 4 + (pj >> 1);
        uint4 buf[2][4];
        int ds = 0;
        uint32_t dpar = 0;
        bool ok = true, have[2];
        // the next slice of the ring of descriptions; false when there is none
        auto load = [&](uint4 (&o)[4]) -> bool {
            if (!(ok = al_wait(&S.sl_full[ds], dpar, &S.abort))) return false;
            const AlSlice &q = S.slice[ds];
            // (no branch around the loads: the registers would be waited for behind it)
            const bool more = q.src != nullptr;
            const int key0 = q.y0 + pr, dims = q.dims - 4 * pc, v = q.v;
            const float *a = q.src + pr * q.stride + 4 * pc;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                // K: 64 rows on; V: 64 dims on
                const int key = key0 + (v ? 0 : e * 64), d = v ? e * 64 : 0;
                const bool any = more && key <= q.any_hi && (key > q.any_lo || key < q.sk);
                al_ld16(a, any && d < dims, o[2 * e]);
                al_ld16(a + 32, any && d + 32 < dims, o[2 * e + 1]);
                a += v ? 64 : 64 * q.stride;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.sl_empty[ds]);
            if (++ds == kSliceRing) ds = 0, dpar ^= 1u;
            return more;
        };
        have[0] = load(buf[0]);
        have[1] = have[0] && load(buf[1]);
        RingPos at;
        while (ok && have[0]) {
#pragma unroll
            for (int k = 0; k < 2; k++) {
                if (!have[k]) break;
                const int s = at.s;
                if (at.round && !al_wait(&S.empty[s], (at.round - 1) & 1u, &S.abort)) {
                    S.abort = 1;
                    raise_status(A.status, kStatusTimeout);
                    ok = false;
                    break;
                }
                const uint32_t to = smem_addr(ring + s * C::kSlot);
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int r = e * 64 + pr;
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        const uint4 v = buf[k][2 * e + q];
                        uint2 h, m, l;
                        al_split2(__uint_as_float(v.x), __uint_as_float(v.y), h.x, m.x, l.x);
                        al_split2(__uint_as_float(v.z), __uint_as_float(v.w), h.y, m.y, l.y);
                        const uint32_t a = to + (uint32_t)(r * 128 + (((4 * q + (pc >> 1)) ^ (r & 7)) << 4) + (pc & 1) * 8);
                        sts64(a, h);
                        sts64(a + C::kTerm, m);
                        sts64(a + 2 * C::kTerm, l);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.full[s]);
                at.step(slots);
                have[k] = have[k ^ 1] && load(buf[k]);
            }
        }
    } else if (warp >= C::kMma) {
        // 896 threads are launched with 72 registers (64512 in all): 128 x 40 here, 256 x 104 for the weights and
        // 512 x 64 for the producers are as many
        if constexpr (NT == 3) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == C::kWalk && al_elect()) {
            // ------------------------------------------------------ describes the pieces
            Walker w(P, D);
            for (int k = 0;; k++) {
                const int r = k % kPieceRing;
                if (k >= kPieceRing && !al_wait(&S.pc_empty[r], (uint32_t)(k / kPieceRing - 1) & 1u, &S.abort)) {
                    S.abort = 1;
                    raise_status(A.status, kStatusTimeout);
                    break;
                }
                w.next(S.piece[r], A, D);
                const bool end = S.piece[r].n == 0;
                mbar_arrive(&S.pc_full[r]);
                if (end) break;
            }
        }
        if (NT == 1 && warp >= C::kCopy && al_elect()) {
            const int half = warp - C::kCopy;
            // ------------------------------------------------------ copies the slices of a bf16 cache
            PieceRef ref;
            RingPos at;
            int g = 0;
            bool ok = true;
            while (ok) {
                const AlPiece *p = ref.next(S);
                if (!(ok = p != nullptr) || p->n == 0) break;
                const CUtensorMap *mk = &maps.k[p->stream], *mv = &maps.v[p->stream];
                const int z = (p->stream ? A.own : A.pre).seq_stride ? p->slot : 0, x0 = p->kvh * hd;
                const int any_lo = p->any_lo, any_hi = p->any_hi, sk = p->sk;
                // a box of 64 keys x 64 dims, left out if nobody sees it: K's are the halves of the chunk, V's (of half
                // a chunk) the halves of 128 dims
                ok = for_slices(*p, nK, nDH, [&](bool v, int row, int dim) {
                    const int s = at.s, y = row + (v ? 0 : 64 * half), x = dim + (v ? 64 * half : 0);
                    if (at.round && !al_wait(&S.empty[s], (at.round - 1) & 1u, &S.abort)) return false;
                    const bool on = x < hd && y <= any_hi && (y + 63 > any_lo || y < sk);
                    mbar_arrive_expect_tx(&S.full[s], on ? 8192u : 0u);
                    if (on)
                        al_tma(smem_addr(ring + s * C::kSlot) + 8192u * half, v ? mv : mk, x0 + x, y, z, smem_addr(&S.full[s]));
                    at.step(slots);
                    g++;
                    return true;
                });
                if (ok) ref.done(S);
            }
            if (!ok) {
                S.abort = 1;
                raise_status(A.status, kStatusTimeout);
                for (int k = max(0, g - slots); k < g; k++)  // the copies in flight
                    mbar_wait(&S.full[k % slots], (uint32_t)(k / slots) & 1u);
            }
        }
        if (NT == 3 && warp == C::kCopy && al_elect()) {
            // ------------------------------------------------------ describes the slices of an fp32 cache
            PieceRef ref;
            int ds = 0;
            uint32_t dround = 0;
            bool ok = true;
            // the next entry of the ring of descriptions; null: gave up
            auto entry = [&]() -> AlSlice * {
                return dround && !al_wait(&S.sl_empty[ds], (dround - 1) & 1u, &S.abort) ? nullptr : &S.slice[ds];
            };
            auto publish = [&]() {
                mbar_arrive(&S.sl_full[ds]);
                if (++ds == kSliceRing) ds = 0, dround++;
            };
            while (ok) {
                const AlPiece *p = ref.next(S);
                if (!(ok = p != nullptr)) break;
                if (p->n == 0) {
                    AlSlice *q = entry();
                    if ((ok = q != nullptr)) {
                        q->src = nullptr;
                        publish();
                    }
                    break;
                }
                const qlin_kv &kv = p->stream ? A.own : A.pre;
                const int64_t off = (int64_t)p->slot * kv.seq_stride + p->kvh * hd, stride = kv.row_stride;
                const float *ksrc = static_cast<const float *>(kv.k) + off, *vsrc = static_cast<const float *>(kv.v) + off;
                const int any_lo = p->any_lo, any_hi = p->any_hi, sk = p->sk;
                ok = for_slices(*p, nK, nDH, [&](bool v, int row, int dim) {
                    AlSlice *q = entry();
                    if (!q) return false;
                    q->src = (v ? vsrc : ksrc) + row * stride + dim;
                    q->stride = stride;
                    q->y0 = row, q->any_lo = any_lo, q->any_hi = any_hi, q->sk = sk;
                    q->v = v, q->dims = hd - dim;
                    publish();
                    return true;
                });
                if (ok) ref.done(S);
            }
            if (!ok) {
                S.abort = 1;
                raise_status(A.status, kStatusTimeout);
            }
        }
        if (warp == C::kMma && al_elect()) {
            // ------------------------------------------------------ the MMAs
            // One thread paces a chunk.  What it needs is in registers, whether the next slice has landed is asked while
            // the products of this one are issued (the answer takes 70 cycles), and a chunk is one run of instructions:
            // a jump back takes 200 cycles here, the other warps having pushed its target out of the instruction cache.
            PieceRef ref;
            int it = 0;           // chunks so far
            uint32_t fixes = 0;   // slices of V of an fp32 cache handed to the first warpgroup so far
            bool ok = true;
            const uint32_t qs_a = smem_addr(qs), ps_a = smem_addr(ps);
            // (K slices have no leading byte offset to speak of, V's 64-dim blocks are 8 KB apart)
            const uint32_t ring_d = al_desc_lo(smem_addr(ring), 16), vlbo = ((8192u - 16u) >> 4) << 16;
            const uint32_t hi128 = al_desc_hi(1024, 2), hip = al_desc_hi(512, 4), qstep = (uint32_t)L.qslice >> 4;
            const uint32_t full0 = smem_addr(&S.full[0]), empty0 = smem_addr(&S.empty[0]) - full0;
            const uint32_t end = full0 + 8u * slots, s_free = smem_addr(&S.s_free), p_ready = smem_addr(&S.p_ready);
            uint32_t full = full0, par = 0, slot_d = ring_d;  // the next slice: its barrier, its phase, its place
            bool landed = false;                              // it has
            // the barrier to commit to when the slice's products are issued; on to the next one
            auto step = [&]() {
                const uint32_t done = full + empty0;
                full += 8, slot_d += C::kSlot / 16;
                if (full == end) full = full0, slot_d = ring_d, par ^= 1u;
                landed = al_test(full, par);
                return done;
            };
            auto arrived = [&]() { return landed || al_wait_at(full, par, &S.abort); };
            while (ok) {
                const AlPiece *p = ref.next(S);
                if (!(ok = p != nullptr)) break;
                const int n = p->n;
                if (n == 0) break;
                const uint32_t nr = (uint32_t)(p->nrows + 15) / 16 * 16;
                // fp32 accumulator, bf16 operands, N = the terms' rows; S^T: both operands K-major, O^T: both with
                // the keys as rows.  Term t of a cached value meets the 3 - t first terms of the rows, whose columns
                // start at the products' order t.
                uint32_t ids[NT], idp[NT];
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    ids[t] = (1u << 4) | (1u << 7) | (1u << 10) | (128u >> 4) << 24 | ((3 - t) * nr >> 3) << 17;
                    idp[t] = ids[t] | (1u << 15) | (1u << 16);
                }
                uint32_t edge = 0, edge_next = 0;  // bit kh: of half kh of the chunk whose products are next; of the one behind
                if (!(ok = al_wait(&S.q_ready, (uint32_t)ref.k & 1u, &S.abort))) break;
                for (int i = 0; ok && i <= n; i++) {
                    if (i < n) {
                        if (it + i > 0 && !(ok = al_wait_at(s_free, (uint32_t)(it + i - 1) & 1u, &S.abort))) break;
                        if (NT == 3) {
                            const int row = p->row0(i);
                            edge = edge_next;
                            edge_next = (uint32_t)p->edge_in(row, row + 64) | (uint32_t)p->edge_in(row + 64, row + 128) << 1;
                        }
                        uint32_t b0 = al_desc_lo(qs_a, 16);
#pragma unroll
                        for (int sl = 0; sl < 4; sl++, b0 += qstep) {
                            const int dims = hd - 64 * sl;
                            if (dims <= 0 || !(ok = arrived())) break;
                            tc_fence_after();
#pragma unroll
                            for (int kk = 0; kk < 4; kk++)
                                if (16 * kk < dims)
#pragma unroll
                                    for (int t = 0; t < NT; t++)
                                        al_mma(tmem + t * nr, slot_d + (uint32_t)(t * C::kTerm / 16 + 2 * kk), hi128, b0 + 2u * kk,
                                               hi128, ids[t], kk > 0 || t > 0 || sl > 0);
                            al_commit(step());
                        }
                        if (!ok) break;
                        tc_commit(&S.s_full);
                    } else {
                        edge = edge_next;
                    }
                    if (i >= 1) {
                        if (!(ok = al_wait_at(p_ready, (uint32_t)(it + i - 1) & 1u, &S.abort))) break;
#pragma unroll
                        for (int kh = 0; kh < 2; kh++) {
                            const uint32_t b0 = al_desc_lo(ps_a + kh * 64 * 64, kChunk * 64);
                            uint32_t d = tmem + C::kO;
#pragma unroll
                            for (int dh = 0; dh < 2; dh++, d += 3 * R) {
                                if (dh >= nDH || !(ok = arrived())) break;
                                if (NT == 3 && (edge >> kh & 1u)) {
                                    mbar_arrive(&S.fix_go);
                                    if (!(ok = al_wait(&S.fixed, fixes & 1u, &S.abort))) break;
                                    fixes++;
                                }
                                tc_fence_after();
                                const uint32_t a0 = slot_d + vlbo;
#pragma unroll
                                for (int ks = 0; ks < 4; ks++)
#pragma unroll
                                    for (int t = 0; t < NT; t++)
                                        al_mma(d + t * nr, a0 + (uint32_t)(t * C::kTerm / 16 + 128 * ks), hi128, b0 + 64u * ks,
                                               hip, idp[t], ks > 0 || t > 0 || kh > 0);
                                al_commit(step());
                            }
                            if (!ok) break;
                        }
                        if (!ok) break;
                        tc_commit(&S.pv_done);
                    }
                }
                it += n;
                if (ok) ref.done(S);
            }
            if (!ok) {
                S.abort = 1;
                raise_status(A.status, kStatusTimeout);
            }
            tc_commit(&S.drain);  // the MMAs in flight (others may have given up)
            mbar_wait(&S.drain, 0);
        }
    } else {
        // ---------------------------------------------------------- weights and sums: warpgroup wg owns rows
        // 16 wg .. 16 wg + 15, its thread t key t of a chunk, and of the outputs dims t and t + 128
        if constexpr (NT == 3) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int wg = warp >> 2, t = tid & 127, r0 = 16 * wg;
        PieceRef ref;
        int g = 0, it = 0;   // slices and chunks so far
        uint32_t fixes = 0;  // slices of V of an fp32 cache looked through
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)r0;
        const float ninf = -__int_as_float(0x7f800000);
        bool ok = true;
        while (ok) {
            const AlPiece *p = ref.next(S);
            __syncwarp();
            if (p == nullptr) {
                S.abort = 1;
                raise_status(A.status, kStatusTimeout);
            }
            if (al_bar_or(wg, p == nullptr)) break;  // (and the rows of the last piece are no longer needed)
            const int n = p->n, nrows = p->nrows, nr = (nrows + 15) / 16 * 16;
            if (n == 0) break;
            if (r0 >= nrows) {  // (the first warpgroup always has rows)
                if (lane == 0) mbar_arrive(&S.q_ready);
                for (int i = 0; i < n && ok; i++, it++) {
                    ok = al_wait(&S.s_full, (uint32_t)it & 1u, &S.abort);
                    if (lane == 0) mbar_arrive(&S.s_free), mbar_arrive(&S.p_ready);
                    // (a second arrival must not meet the same phase)
                    ok = ok && al_wait(&S.pv_done, (uint32_t)it & 1u, &S.abort);
                    __syncwarp();
                }
                if (!ok) S.abort = 1;
                ok = !al_bar_or(wg, !ok);
                g += n * (nK + nV);
                if (lane == 0) ref.done(S);
                continue;
            }
            if (t < 16) {
                const int r = r0 + t, gs = p->gs, ln = p->lane0 + r / gs;
                const bool in = r < nrows;
                const int pl = in ? A.positions[ln] - p->base : -1;
                S.rowid[r] = in ? ln * A.n_heads + p->head0 + r % gs : -1;
                S.rowhi[r] = max(-1, min(pl, p->lim - 1));
                S.rowlo[r] = A.window && pl >= A.window ? pl - A.window : -1;
                S.mc[r] = in ? kNoKey : -ninf;  // (what lies in the place of a row that is not there gets no weight)
                S.nan[r] = 0;
            }
            al_bar(wg);
            // the rows' q, with the softmax's scale, as three bf16 terms
#pragma unroll 4
            for (int e = t; e < min(16, nrows - r0) * (hd / 8); e += 128) {
                const int rr = e / (hd / 8), d8 = e - rr * (hd / 8), r = r0 + rr;
                uint4 a, b, h, m, l;
                al_ld32(A.q + (int64_t)S.rowid[r] * hd + 8 * d8, true, a, b);
                auto scale = [&](uint32_t &u) { u = __float_as_uint(__fmul_rn(__uint_as_float(u), D.c)); };
                scale(a.x), scale(a.y), scale(a.z), scale(a.w), scale(b.x), scale(b.y), scale(b.z), scale(b.w);
                al_split8(a, b, h, m, l);
                const uint32_t at = smem_addr(qs) + (uint32_t)((d8 >> 3) * L.qslice + r * 128 + (((d8 & 7) ^ (r & 7)) << 4));
                sts128(at, h);
                sts128(at + nr * 128, m);
                sts128(at + 2 * nr * 128, l);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.q_ready);
            float lsum[16], acc[2][16];
#pragma unroll
            for (int j = 0; j < 16; j++) lsum[j] = acc[0][j] = acc[1][j] = 0.0f;
            // 16 columns' terms of the products: (lo + mid) + hi
            auto sum3 = [&](uint32_t at, float (&o)[16]) {
                uint32_t h[16], m[16];
                tm_ld16_nw(at + 2 * nr, h);
                tm_ld16_nw(at + nr, m);
                tm_wait_ld(h);
                tm_wait_ld(m);
#pragma unroll
                for (int j = 0; j < 16; j++) o[j] = __fadd_rn(__uint_as_float(h[j]), __uint_as_float(m[j]));
                tm_ld16(at, h);
#pragma unroll
                for (int j = 0; j < 16; j++) o[j] = __fadd_rn(o[j], __uint_as_float(h[j]));
            };
            // adds a chunk's products to the outputs
            auto take = [&]() {
                float o[16];
                sum3(tl + C::kO, o);
#pragma unroll
                for (int j = 0; j < 16; j++) acc[0][j] = __fadd_rn(acc[0][j], o[j]);
                if (nDH == 2) {
                    sum3(tl + C::kO + 3 * R, o);
#pragma unroll
                    for (int j = 0; j < 16; j++) acc[1][j] = __fadd_rn(acc[1][j], o[j]);
                }
            };

            for (int i = 0; i < n; i++, it++) {
                const int cr = p->row0(i), sk = p->sk, key = cr + t;
                const bool edge = p->edge_in(cr, cr + kChunk);
                const bool fail = !al_wait(&S.s_full, (uint32_t)it & 1u, &S.abort);
                __syncwarp();  // (the tensor-memory loads are for whole warps)
                tc_fence_after();
                float s[16];
                sum3(tl, s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.s_free);
                // whether row r of the tile sees this thread's key
                auto sees = [&](int r) { return key <= S.rowhi[r] && (key > S.rowlo[r] || key < sk); };
                if (edge)
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (!sees(r0 + j)) s[j] = ninf;
                bool big = i == 0;
                if (i > 0)
#pragma unroll
                    for (int j = 0; j < 16; j++) big |= __fsub_rn(s[j], S.mc[r0 + j]) > 8.0f;
                const bool update = al_bar_or(wg, big || fail);
                if (update) {
                    if (al_bar_or(wg, fail)) {
                        if (fail) {
                            S.abort = 1;
                            raise_status(A.status, kStatusTimeout);
                        }
                        ok = false;
                        break;
                    }
                    // new maxima
                    float m[16];
#pragma unroll
                    for (int j = 0; j < 16; j++) m[j] = s[j];
                    const float top = al_reduce16<true>(m, lane);
                    if (lane < 16) S.red[warp & 3][r0 + lane] = top;
                    al_bar(wg);
                    if (t < 16) {
                        const int r = r0 + t;
                        const float mx = fmaxf(fmaxf(S.red[0][r], S.red[1][r]), fmaxf(S.red[2][r], S.red[3][r]));
                        const float old = S.mc[r], mc = mx > ninf ? fmaxf(mx, old) : old;
                        S.mc[r] = mc;
                        S.alpha[r] = old == kNoKey ? 0.0f : al_ex2(__fsub_rn(old, mc));
                    }
                    al_bar(wg);
#pragma unroll
                    for (int j = 0; j < 16; j++) lsum[j] = __fmul_rn(lsum[j], S.alpha[r0 + j]);
                }
                // (a masked score stays minus infinity, the weight 0)
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    s[j] = al_ex2(__fsub_rn(s[j], S.mc[r0 + j]));
                    lsum[j] = __fadd_rn(lsum[j], s[j]);
                }
                if (i > 0) {  // the products of the chunk before: P is read, and O^T is there
                    if (!al_wait(&S.pv_done, (uint32_t)(it - 1) & 1u, &S.abort)) S.abort = 1;
                    __syncwarp();
                }
                // the weights, as three bf16 terms, a key's rows side by side
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    uint4 w3[3];
                    al_split2(s[8 * q], s[8 * q + 1], w3[0].x, w3[1].x, w3[2].x);
                    al_split2(s[8 * q + 2], s[8 * q + 3], w3[0].y, w3[1].y, w3[2].y);
                    al_split2(s[8 * q + 4], s[8 * q + 5], w3[0].z, w3[1].z, w3[2].z);
                    al_split2(s[8 * q + 6], s[8 * q + 7], w3[0].w, w3[1].w, w3[2].w);
#pragma unroll
                    for (int u = 0; u < 3; u++) {
                        const int c = u * nr + r0 + 8 * q;
                        sts128(smem_addr(ps) + (uint32_t)((c >> 5) * (kChunk * 64) + t * 64 +
                                                          ((((c >> 3) & 3) ^ ((t >> 1) & 3)) << 4)),
                               w3[u]);
                    }
                }
                if (i > 0) {
                    tc_fence_after();
                    take();
                    if (update)
#pragma unroll
                        for (int j = 0; j < 16; j++) {
                            const float al = S.alpha[r0 + j];
                            acc[0][j] = __fmul_rn(acc[0][j], al);
                            acc[1][j] = __fmul_rn(acc[1][j], al);
                        }
                }
                if (NT == 1 && edge) {
                    // Values of keys that not every row sees: the weight of a hidden one is zero, but zero times an
                    // infinity or NaN is not.  The slices are dealt out to the warpgroups, half a key's values to a
                    // thread.  (With the scores of the next chunk there, what lay in these slots before is read, and
                    // what lies in them now stays until the weights are ready: the barriers' phases are the next ones.)
                    if (i + 1 < n && !al_wait(&S.s_full, (uint32_t)(it + 1) & 1u, &S.abort)) S.abort = 1;
                    const int gv = g + min(i + 2, n) * nK + i * nV;
                    for (int vs = wg; vs < nV; vs += (nrows + 15) / 16) {
                        const int sl = (gv + vs) % slots, k0 = cr + 64 * (vs / nDH), y = k0 + (t & 63);
                        if (!p->edge_in(k0, k0 + 64)) continue;
                        if (!al_wait(&S.full[sl], (uint32_t)((gv + vs) / slots) & 1u, &S.abort)) S.abort = 1;
                        if (p->edge_in(y, y + 1))
                            al_look<NT>(S, *p, y, smem_addr(ring + sl * C::kSlot) + (uint32_t)((t >> 6) * 8192 + (t & 63) * 128),
                                        t, hd - (vs % nDH) * 128 - (t >> 6) * 64);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.p_ready);
                if (NT == 3 && wg == 0 && edge) {
                    // the same slice by slice, as each has landed and its product waits (the ring of an fp32 cache may
                    // be shorter than a chunk's slices of V)
                    const int gv = g + min(i + 2, n) * nK + i * nV;
                    for (int vs = 0; vs < nV; vs++) {
                        const int sl = (gv + vs) % slots, k0 = cr + 64 * (vs / nDH), y = k0 + (t & 63);
                        if (!p->edge_in(k0, k0 + 64)) continue;
                        if (!al_wait(&S.fix_go, fixes & 1u, &S.abort)) S.abort = 1;
                        fixes++;
                        if (p->edge_in(y, y + 1))
                            al_look<NT>(S, *p, y, smem_addr(ring + sl * C::kSlot) + (uint32_t)((t >> 6) * 8192 + (t & 63) * 128),
                                        t, hd - (vs % nDH) * 128 - (t >> 6) * 64);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&S.fixed);
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            g += n * (nK + nV);
            // the sums over the keys
            const float l4 = al_reduce16<false>(lsum, lane);
            if (lane < 16) S.red[warp & 3][r0 + lane] = l4;
            const bool gone = !al_wait(&S.pv_done, (uint32_t)(it - 1) & 1u, &S.abort);
            if (gone) S.abort = 1;
            if (al_bar_or(wg, gone)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const bool direct = p->whole && D.streams == 1;
            const int rows = min(16, nrows - r0);
            if (t < 16) {
                const int r = r0 + t;
                float *o = nullptr;
                if (t < rows) {
                    float l = (S.red[0][r] + S.red[1][r]) + (S.red[2][r] + S.red[3][r]);
                    if (S.nan[r]) l = __int_as_float(0x7fc00000);
                    const int64_t id = S.rowid[r];
                    if (direct) {
                        o = A.out + id * hd;
                        l = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
                    } else {
                        const int64_t row = p->whole ? (int64_t)2 * D.grid * D.cap + (int64_t)p->stream * A.n_lanes * A.n_heads + id
                                                     : (int64_t)(2 * blockIdx.x + p->begins) * D.cap + r;
                        o = W.part + row * hd;
                        W.ml[row] = make_float2(S.mc[r], l);
                        l = 1.0f;
                    }
                    S.alpha[r] = l;
                }
                S.optr[r] = o;
            }
            take();
            tc_fence_before();
            al_bar(wg);
            if (lane == 0) ref.done(S);
#pragma unroll
            for (int j = 0; j < 16; j++) {
                float *o = S.optr[r0 + j];
                if (o) {
                    const float al = S.alpha[r0 + j];
                    if (t < hd) o[t] = __fmul_rn(acc[0][j], al);
                    if (t + 128 < hd) o[t + 128] = __fmul_rn(acc[1][j], al);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && S.abort) raise_status(A.status, kStatusTimeout);  // (whoever saw it)
    if (warp == C::kMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
}

// ------------------------------------------------------------------ little work
// A few lanes over short stretches are over before the product kernel's plan,
// pieces and rings are set up.  Here every CTA takes one lane, up to GH query
// heads of one KV head and kKeys of the keys that the lane sees, counted
// without gaps (first tokens, then the window): it copies their k and v rows
// into shared memory, all of them at once, and computes in fp32 on the CUDA
// cores.  Nothing is shared between lanes.  The CTA s of a (lane, head)
// leaves partial sums for al_few_merge_kernel, or the result if it is alone;
// few enough CTAs are a cluster, which merges through its shared memory.  One
// lane of 516 keys (4 heads, 256 dims, fp32: 1.06 MB) takes 6.8 us as a cluster
// of 16, 7.3 with a merging launch, and 16.7 in the product kernel: a launch, a
// trip to memory, and the chain from a key's dot product to the sum.
constexpr int kFewThreads = 256, kFewMaxSplits = 1024;
constexpr int kFewDims = 64;  // dims of a head per merging CTA

// CL: the CTAs of a (lane, head) are one cluster and merge among themselves
template <typename T, bool CL = false>
struct FewCfg {
    static constexpr int kKeys = (sizeof(T) == 4 ? 32 : 64) * (CL ? 2 : 1);  // 32 KB of k and of v rows at most, 64 of a cluster's
    static constexpr int kParts = kFewThreads / kKeys;           // threads that share a key's dot products
    static constexpr int kVec = 16 / (int)sizeof(T);             // values of 16 bytes
};

// What lane i sees: keys j < sk and lo <= j <= p (sk <= lo), `count` of them; -1 if it is none.
struct FewLane {
    int count, sk, lo, len, seq, pre;
    bool bad;
    __device__ __forceinline__ FewLane(const AlArgs &A, int i) {
        const int p = A.positions[i];
        seq = A.seqs[i];
        pre = 0, len = 0;
        bool ok = seq >= 0 && seq < A.own.n_seqs;
        if (A.pre.k) {
            pre = A.prefix_of ? A.prefix_of[i] : 0;
            ok = ok && pre >= 0 && pre < A.pre.n_seqs;
            len = ok ? A.prefix_len[pre] : 0;
            ok = ok && len >= 0 && len <= A.pre.rows;
        }
        ok = ok && p - len < A.own.rows;
        bad = p >= 0 && !ok;
        lo = A.window && p >= A.window ? p - A.window + 1 : 0;
        sk = min(A.sinks, lo);
        count = p >= 0 && ok ? sk + p + 1 - lo : 0;
    }
};

__device__ __forceinline__ void few_unpack(const uint4 &u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void few_unpack(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; k++) f[2 * k] = __uint_as_float(w[k] << 16), f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
}

// grid (splits, KV heads x blocks of GH query heads, lanes); K: keys of a CTA
template <typename T, int GH, bool CL>
__global__ void __launch_bounds__(kFewThreads)
    al_few_kernel(AlArgs A, AlDims D, float2 *ml, float *part, int splits, int K) {
    using C = FewCfg<T, CL>;
    constexpr int KM = C::kKeys, V = C::kVec;
    extern __shared__ __align__(16) uint8_t few_smem[];
    __shared__ __align__(16) float qs[GH][256];
    __shared__ __align__(16) float ws[KM][GH];
    __shared__ float4 stat[GH];  // a cluster's: the largest score and the sum of the weights here
    const int tid = threadIdx.x, hd = A.hd, pitch = hd * (int)sizeof(T) + 16;
    const int s = blockIdx.x, blocks = (D.group + GH - 1) / GH, kvh = blockIdx.y / blocks, h0 = (blockIdx.y % blocks) * GH;
    const int lane_i = blockIdx.z, heads = min(GH, D.group - h0), head0 = kvh * D.group + h0;
    uint8_t *ks = few_smem, *vs = few_smem + (CL ? K : KM) * pitch;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const FewLane L(A, lane_i);
    if (L.bad && s == 0 && blockIdx.y == 0 && tid == 0) raise_status(A.status, kStatusBadLane);
    const int n = min(K, L.count - s * K);  // this CTA's keys
    if (CL ? L.count <= 0 : n <= 0) {
        if (s == 0)
            for (int e = tid; e < heads * hd; e += kFewThreads) A.out[((int64_t)lane_i * A.n_heads + head0) * hd + e] = 0.0f;
        return;
    }
    const int per = hd / V;  // 16-byte groups of a row
    for (int e = tid; e < n * per; e += kFewThreads) {
        const int r = e / per, c = e - r * per, x = s * K + r, j = x < L.sk ? x : L.lo + x - L.sk;
        const bool in = j < L.len;
        const qlin_kv &kv = in ? A.pre : A.own;
        const int64_t off = (int64_t)(in ? L.pre : L.seq) * kv.seq_stride + (int64_t)(in ? j : j - L.len) * kv.row_stride +
                            kvh * hd + c * V;
        cp_async16(ks + r * pitch + c * 16, static_cast<const T *>(kv.k) + off, 16);
        cp_async16(vs + r * pitch + c * 16, static_cast<const T *>(kv.v) + off, 16);
    }
    cp_async_commit();
    if (CL && tid < GH) stat[tid] = make_float4(-__int_as_float(0x7f800000), 0.0f, 0.0f, 0.0f);  // (no key)
    for (int e = tid; e < GH * hd; e += kFewThreads) {
        const int h = e / hd;
        qs[h][e - h * hd] = h < heads ? A.q[((int64_t)lane_i * A.n_heads + head0) * hd + e] : 0.0f;
    }
    cp_async_wait_pending<0>();
    __syncthreads();
    // scores: kParts threads share a key, 16 bytes of its row in turn
    const int key = tid / C::kParts, pt = tid % C::kParts;
    float sc[GH];
#pragma unroll
    for (int h = 0; h < GH; h++) sc[h] = 0.0f;
    if (key < n)
        for (int c = pt; c < per; c += C::kParts) {
            float k[V];
            few_unpack(lds128(ks + key * pitch + c * 16), k);
#pragma unroll
            for (int h = 0; h < GH; h++)
#pragma unroll
                for (int v = 0; v < V; v += 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(&qs[h][c * V + v]);
                    sc[h] = __fmaf_rn(q.x, k[v], sc[h]);
                    sc[h] = __fmaf_rn(q.y, k[v + 1], sc[h]);
                    sc[h] = __fmaf_rn(q.z, k[v + 2], sc[h]);
                    sc[h] = __fmaf_rn(q.w, k[v + 3], sc[h]);
                }
        }
#pragma unroll
    for (int off = 1; off < C::kParts; off <<= 1)
#pragma unroll
        for (int h = 0; h < GH; h++) sc[h] = __fadd_rn(sc[h], __shfl_xor_sync(0xffffffffu, sc[h], off));
    if (pt == 0)
#pragma unroll
        for (int h = 0; h < GH; h++) ws[key][h] = key < n ? __fmul_rn(sc[h], D.c) : -__int_as_float(0x7f800000);
    __syncthreads();
    // weights: a warp per head
    const int warp = tid >> 5, lane = tid & 31;
    const bool alone = !CL && L.count <= K;
    const int64_t row0 = ((int64_t)lane_i * A.n_heads + head0) * splits + s;  // head h: row0 + h splits
    __shared__ float inv[GH];
    if (warp < GH && n > 0) {
        float x[KM / 32], m = -__int_as_float(0x7f800000), l = 0.0f;
#pragma unroll
        for (int u = 0; u < KM / 32; u++) x[u] = ws[lane + 32 * u][warp], m = fmaxf(m, x[u]);
        m = warp_max(m);
        const bool some = m > -__int_as_float(0x7f800000);
        if (!some) m = 0.0f;  // (scores of minus infinity or NaN alone)
#pragma unroll
        for (int u = 0; u < KM / 32; u++) {
            x[u] = al_ex2(__fsub_rn(x[u], m));
            l += x[u];
            ws[lane + 32 * u][warp] = x[u];
        }
        l = warp_psum(l);
        // (scores beyond fp32's range have no weight, and no say in what the other pieces are relative to)
        if (!some && l == 0.0f) m = -__int_as_float(0x7f800000);
        if (lane == 0) {
            inv[warp] = alone ? __fdiv_rn(1.0f, l) : 1.0f;
            if (CL)
                stat[warp] = make_float4(m, l, 0.0f, 0.0f);
            else if (!alone && warp < heads)
                ml[row0 + (int64_t)warp * splits] = make_float2(m, l);
        }
    }
    __syncthreads();
    // outputs: four dims of every `groups`-th key per thread, then the sum over the groups
    const int nv = hd / 4, groups = kFewThreads / nv, gi = tid / nv, d = (tid - gi * nv) * 4;
    float4 o[GH];
#pragma unroll
    for (int h = 0; h < GH; h++) o[h] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (gi < groups)
#pragma unroll 4
        for (int j = gi; j < n; j += groups) {
            float4 v;
            if constexpr (sizeof(T) == 4) {
                v = *reinterpret_cast<const float4 *>(vs + j * pitch + d * 4);
            } else {
                const uint2 u = *reinterpret_cast<const uint2 *>(vs + j * pitch + d * 2);
                v = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                                __uint_as_float(u.y & 0xffff0000u));
            }
#pragma unroll
            for (int h = 0; h < GH; h++) {
                const float w = ws[j][h];
                o[h].x = __fmaf_rn(w, v.x, o[h].x), o[h].y = __fmaf_rn(w, v.y, o[h].y);
                o[h].z = __fmaf_rn(w, v.z, o[h].z), o[h].w = __fmaf_rn(w, v.w, o[h].w);
            }
        }
    __syncthreads();  // the k rows' place takes the groups' sums: [groups][GH][hd], at most 32 KB
    float *red = reinterpret_cast<float *>(few_smem);
    if (gi < groups)
#pragma unroll
        for (int h = 0; h < GH; h++) *reinterpret_cast<float4 *>(red + (gi * GH + h) * hd + d) = o[h];
    __syncthreads();
    for (int e = tid; e < heads * nv; e += kFewThreads) {
        const int h = e / nv, dd = (e - h * nv) * 4;
        float4 a = *reinterpret_cast<const float4 *>(red + h * hd + dd);
        for (int u = 1; u < groups; u++) {
            const float4 b = *reinterpret_cast<const float4 *>(red + (u * GH + h) * hd + dd);
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
        }
        if constexpr (CL) {
            *reinterpret_cast<float4 *>(red + h * hd + dd) = a;
            continue;
        }
        const float f = inv[h];
        float *to = alone ? A.out + ((int64_t)lane_i * A.n_heads + head0 + h) * hd : part + (row0 + (int64_t)h * splits) * hd;
        *reinterpret_cast<float4 *>(to + dd) = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
    }
    if constexpr (CL) {
        // the cluster's CTAs share the outputs out: as many threads to four dims as there are CTAs (2, 4, 8 or 16), one
        // for each one's sums
        cluster_sync();
        const int lg = splits <= 2 ? 1 : splits <= 4 ? 2 : splits <= 8 ? 3 : 4, r = tid & ((1 << lg) - 1);
        const int items = heads * nv, share = (items + splits - 1) / splits;
        for (int i0 = 0; i0 < share; i0 += kFewThreads >> lg) {
            const int at = i0 + (tid >> lg), i = s * share + at, h = min(i, items - 1) / nv, dd = (i - h * nv) * 4;
            const bool on = at < share && i < items;
            float4 st = make_float4(-__int_as_float(0x7f800000), 0.0f, 0.0f, 0.0f), v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (on && r < splits) st = ld_peer_f4(&stat[h], (uint32_t)r);
            const bool some = st.x > -__int_as_float(0x7f800000);
            if (some) v = ld_peer_f4(red + h * hd + dd, (uint32_t)r);
            float m = st.x;
            for (int off = 1 << lg >> 1; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            const float w = some ? al_ex2(__fsub_rn(st.x, m)) : 0.0f;
            float l = w * st.y;
            v.x *= w, v.y *= w, v.z *= w, v.w *= w;
            for (int off = 1 << lg >> 1; off > 0; off >>= 1) {
                l += __shfl_xor_sync(0xffffffffu, l, off);
                v.x += __shfl_xor_sync(0xffffffffu, v.x, off), v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
                v.z += __shfl_xor_sync(0xffffffffu, v.z, off), v.w += __shfl_xor_sync(0xffffffffu, v.w, off);
            }
            const float f = __fdiv_rn(1.0f, l);
            if (on && r == 0)
                *reinterpret_cast<float4 *>(A.out + ((int64_t)lane_i * A.n_heads + head0 + h) * hd + dd) =
                    make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
        }
        cluster_sync();  // nobody leaves while its sums are read
    }
}

// grid (heads, lanes, dims / kFewDims): the partial sums of one (lane, head) by
// the weights 2^(maximum - largest maximum).
__global__ void __launch_bounds__(kFewThreads) al_few_merge_kernel(AlArgs A, const float2 *ml, const float *part, int splits,
                                                                 int keys) {
    __shared__ float w[kFewMaxSplits];
    __shared__ float red[8];
    __shared__ float4 acc[kFewThreads];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hd = A.hd;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // (the lanes' places were there before the kernel before began)
    const FewLane L(A, blockIdx.y);
    const int n = (L.count + keys - 1) / keys;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n <= 1) return;  // done already
    const int64_t id = (int64_t)blockIdx.y * A.n_heads + blockIdx.x, row0 = id * splits;
    float m = -__int_as_float(0x7f800000);
    for (int k = tid; k < n; k += kFewThreads) m = fmaxf(m, __ldcg(&ml[row0 + k]).x);
    m = warp_max(m);
    if (lane == 0) red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; k++) m = fmaxf(m, red[k]);
    __syncthreads();
    float l = 0.0f;
    for (int k = tid; k < n; k += kFewThreads) {
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
    constexpr int nv = kFewDims / 4, groups = kFewThreads / nv;
    const int gi = tid / nv, dv = blockIdx.z * nv + tid % nv;  // four dims, every 16th piece
    const bool in = dv < hd / 4;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (in)
#pragma unroll 8
        for (int k = gi; k < n; k += groups) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(part + (row0 + k) * hd) + dv);
            const float x = w[k];
            a.x += v.x * x, a.y += v.y * x, a.z += v.z * x, a.w += v.w * x;
        }
    acc[tid] = a;
    __syncthreads();
    if (tid < nv && in) {
        for (int k = 1; k < min(groups, n); k++) {
            const float4 v = acc[k * nv + tid];
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
        const float inv = __fdiv_rn(1.0f, l);
        reinterpret_cast<float4 *>(A.out + id * hd)[dv] = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    }
}

// ------------------------------------------------------------------ host

// The tensor maps of a bf16 cache: [n_seqs][rows][n_kv hd], boxes of 64 rows x
// 64 values, 128-byte swizzle, zeros out of range.
qlin_status kv_map(const void *p, const qlin_kv &c, int kvd, CUtensorMap *out) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)fn;
    }();
    QLIN_REQUIRE(encode, QLIN_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    // (sequences that all start at one place are read as the first)
    const cuuint64_t gdim[3] = {(cuuint64_t)kvd, (cuuint64_t)c.rows, (cuuint64_t)(c.seq_stride ? c.n_seqs : 1)};
    const cuuint64_t gstride[2] = {(cuuint64_t)c.row_stride * 2, (cuuint64_t)(c.seq_stride ? c.seq_stride : c.row_stride) * 2};
    const cuuint32_t box[3] = {64, 64, 1}, estride[3] = {1, 1, 1};
    const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), gdim, gstride, box, estride,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    QLIN_REQUIRE(r == CUDA_SUCCESS, QLIN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return QLIN_OK;
}

// The keys that a lane can see at most, and the splits they make.
int64_t few_keys(const AlArgs &A) {
    const int64_t keys = (int64_t)A.own.rows + (A.pre.k ? A.pre.rows : 0);
    return A.window && (int64_t)A.window + A.sinks < keys ? (int64_t)A.window + A.sinks : keys;
}
int64_t few_splits(const AlArgs &A, bool f32) {
    const int64_t keys = few_keys(A);
    const int per = f32 ? FewCfg<float>::kKeys : FewCfg<uint16_t>::kKeys;
    return (keys + per - 1) / per;
}
int few_heads(const AlDims &D) { return D.group <= 1 ? 1 : D.group <= 2 ? 2 : D.group <= 4 ? 4 : 8; }

// Whether the call is little work, by the caches' sizes (the positions are on
// the device): the multiply-adds of all its CTAs at most, with every lane and
// block of GH heads counted for itself.  Measured with every position of the
// caches in use, us per call here / by the product kernel: fp32, 4 query heads
// on one KV head of 256: one lane of 512 6.8 / 16.7, 64 of 2048 (268 MB, 268 M
// multiply-adds) 56.1 / 63.9; 8 on each of two of 128: 16 of 512 (34 M) 11.4 /
// 20.5, 16 of 2048 (134 M) 28.7 / 29.0; bf16, 4 on one of 256: 16 of 2048 (67
// M) 14.0 / 18.9, 64 of 2048 (268 M) 41.4 / 27.4; 8 on each of two of 128: 16
// of 512 (34 M) 12.9 / 15.3, 16 of 2048 (134 M) 21.8 / 17.9; one on each of
// four of 64: 64 of 2048 (67 M) 34.8 / 41.4.
//
// Where lanes share a sequence or a prompt (at least two to each, by the
// caches' sizes), the product kernel reads its rows once and this one once per
// lane, so the rows' bytes count too, some 256 more for a row's handling,
// against a product kernel that takes longer for more tiles.  fp32, 32 beams of
// one prompt: two heads on each of four KV heads of 128, 1250 rows (168 MB) 44.6
// / 30.1, 300 rows (44 MB) 16.9 / 26.4; on three of 64, 2500 rows (124 MB) 50.6
// / 24.9; 32 on each of six prompts of 300 (98 MB, 576 tiles) 39.3 / 64.7; four
// on one of 256, 620 rows (43 MB) 18.5 / 25.6, 2500 (166 MB) 43.9 / 34.1; bf16,
// two on each of four of 128, 1250 (84 MB) 26.2 / 21.5 (just inside the limit, so
// it goes the slower way), 620 (43 MB) 16.6 / 21.5; a chunk of 64 lanes, window
// 512, fp32, two on each of four of 128: 38.1 / 21.6.
//
// Caches larger than what is seen count as if all of them were: 16 lanes at
// position 500 (fp32, 8 on each of two of 128) take 13.2 us in caches of 512 rows
// and 20.8 in caches of 32768, by the product kernel; four beams behind a prompt
// of 300 (4 on one of 256) 7.4 where the prompts' cache has 300 rows and 21.6 at
// 32768.
bool few_fits(const AlArgs &A, const AlDims &D, bool f32, int64_t rows) {
    const int64_t s = few_splits(A, f32);
    const int gh = few_heads(D);
    const double fma = (double)s * (f32 ? FewCfg<float>::kKeys : FewCfg<uint16_t>::kKeys) * A.n_lanes * A.n_kv *
                       ((D.group + gh - 1) / gh) * gh * A.hd * 2;
    if (s > kFewMaxSplits || s * A.n_lanes * A.n_heads > rows || fma > (!f32 ? 90e6 : gh < 8 ? 300e6 : 140e6)) return false;
    const qlin_kv &from = A.pre.k ? A.pre : A.own;
    if (A.n_lanes < 2 * (int64_t)from.n_seqs) return true;
    // several lanes to a sequence
    const double bytes = (double)A.n_lanes * A.n_kv * ((D.group + gh - 1) / gh) * few_keys(A) *
                         (A.hd * 2 * (f32 ? 4 : 2) + 256);
    const double tiles = (double)A.n_kv * (A.pre.k ? A.n_lanes : (A.n_lanes + D.LT - 1) / D.LT);
    return bytes <= (f32 ? 106e6 : 90e6) + 0.3e6 * tiles && !(f32 && gh == 8 && fma > 100e6);
}

// CTAs of a cluster for keys that make `splits` CTAs; 0: no cluster.
constexpr int kFewCluster = 16;
int few_cluster(int splits) {
    return splits > 1 && splits <= kFewCluster * 5 / 4 ? (splits < kFewCluster ? splits : kFewCluster) : 0;
}
constexpr qlin_status kNoCluster = (qlin_status)-1;

template <typename T, int GH, bool CL>
qlin_status launch_few(const AlArgs &A, const AlDims &D, const AlWs &w, int splits, int keys, cudaStream_t st) {
    const void *kern = (const void *)al_few_kernel<T, GH, CL>;
    const size_t rowbytes = (size_t)2 * keys * (A.hd * sizeof(T) + 16);
    const size_t sums = (size_t)(kFewThreads / (A.hd / 4)) * GH * A.hd * sizeof(float);
    const size_t smem = rowbytes > sums ? rowbytes : sums;
    blocks_per_sm(kern, smem);  // raises the dynamic shared-memory limit once
    void *args[] = {(void *)&A, (void *)&D, (void *)&w.ml, (void *)&w.part, (void *)&splits, (void *)&keys};
    const dim3 grid(splits, A.n_kv * ((D.group + GH - 1) / GH), A.n_lanes);
    if (CL && max_clusters(kern, smem, kFewThreads, splits) < (int64_t)grid.y * grid.z) return kNoCluster;
    return launch_pdl(kern, grid, dim3(kFewThreads), smem, st, args, "al_few_kernel", CL ? splits : 0);
}
template <typename T, bool CL>
qlin_status launch_few(const AlArgs &A, const AlDims &D, const AlWs &w, int splits, int keys, cudaStream_t st) {
    switch (few_heads(D)) {
        case 1: return launch_few<T, 1, CL>(A, D, w, splits, keys, st);
        case 2: return launch_few<T, 2, CL>(A, D, w, splits, keys, st);
        case 4: return launch_few<T, 4, CL>(A, D, w, splits, keys, st);
        default: return launch_few<T, 8, CL>(A, D, w, splits, keys, st);
    }
}
qlin_status attend_few(const AlArgs &A, const AlDims &D, const AlWs &w, bool f32, cudaStream_t st) {
    const int splits = (int)few_splits(A, f32), keys = f32 ? FewCfg<float>::kKeys : FewCfg<uint16_t>::kKeys;
    // One launch if the CTAs of every (lane, head block) can be a cluster and no cluster has to wait for another's SMs.
    // us per call with a cluster / with two launches: fp32, 4 query heads on one KV head of 256: one lane of 512 6.8 /
    // 7.5, four 7.0 / 8.6, 16 of 200 8.6 / 9.5; one on each of four of 64: one lane of 512 4.4 / 5.8; bf16: one lane of
    // 1024 7.2 / 8.2, eight of 512 7.8 / 11.1.  With more keys to a CTA than a quarter above its own number it does not
    // pay (fp32, one lane of 1024 in 16 CTAs: 8.7 / 7.4).
    if (const int c = few_cluster(splits)) {
        const int share = (int)((few_keys(A) + c - 1) / c);
        const qlin_status e = f32 ? launch_few<float, true>(A, D, w, c, share, st) : launch_few<uint16_t, true>(A, D, w, c, share, st);
        if (e != kNoCluster) return e;
    }
    if (qlin_status e = f32 ? launch_few<float, false>(A, D, w, splits, keys, st)
                            : launch_few<uint16_t, false>(A, D, w, splits, keys, st))
        return e;
    if (splits == 1) return QLIN_OK;
    void *args[] = {(void *)&A, (void *)&w.ml, (void *)&w.part, (void *)&splits, (void *)&keys};
    return launch_pdl((const void *)al_few_merge_kernel, dim3(A.n_heads, A.n_lanes, (A.hd + kFewDims - 1) / kFewDims),
                      dim3(kFewThreads), 0, st, args, "al_few_merge_kernel");
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
    QLIN_REQUIRE(c->rows <= 1 << 30, QLIN_ERR_UNSUPPORTED, "%s: %s: more than 2^30 rows", fn, what);
    QLIN_REQUIRE(c->row_stride < (int64_t)1 << 40 && c->seq_stride < (int64_t)1 << 40 && c->row_stride * e < (int64_t)1 << 40 && c->seq_stride * e < (int64_t)1 << 40, QLIN_ERR_UNSUPPORTED,
                 "%s: %s: a stride of 2^40 bytes or more", fn, what);
    return QLIN_OK;
}

qlin_status same_types(const char *fn, const qlin_kv *prefix, const qlin_kv *kv) {
    QLIN_REQUIRE(!prefix || prefix->type == kv->type, QLIN_ERR_INVALID_ARG, "%s: the caches' types differ", fn);
    return QLIN_OK;
}

bool sizes_ok(int n_lanes, int n_heads, int n_kv, int hd) {
    return n_lanes >= 1 && n_lanes <= kMaxLanes && n_kv >= 1 && n_heads >= n_kv && n_heads % n_kv == 0 &&
           n_heads <= 65535 && hd >= 16 && hd <= 256 && hd % 16 == 0;
}

AlDims al_dims(const AlArgs &A) {
    const bool f32 = A.own.type == QLIN_KV_F32;
    AlDims D{};
    D.group = A.n_heads / A.n_kv;
    D.R = f32 ? AlCfg<3>::R : AlCfg<1>::R;
    D.LT = D.group < D.R ? D.R / D.group : 1;
    D.HB = (D.group + D.R - 1) / D.R;
    D.cap = (int64_t)A.n_lanes * D.group < D.R ? A.n_lanes * D.group : D.R;
    D.streams = A.pre.k ? 2 : 1;
    D.grid = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
    D.merge = A.n_lanes <= kSelfPlan ? 1 : 16;
    // (measured: tiles of 2 to 33 chunks of 128 keys in bf16 want 3 to 5, the longer chunks of fp32 caches 2)
    D.setup = f32 ? 2 : 4;
    D.c = (float)(1.4426950408889634 / std::sqrt((double)A.hd));
    return D;
}

qlin_status check_sizes(const char *fn, const AlArgs &A) {
    QLIN_REQUIRE(A.n_lanes >= 1 && A.n_heads >= 1 && A.n_kv >= 1 && A.n_heads % A.n_kv == 0 && A.window >= 0 &&
                     A.sinks >= 0,
                 QLIN_ERR_INVALID_ARG, "%s: n_lanes %d, n_heads %d, n_kv %d, window %d, sinks %d", fn, A.n_lanes,
                 A.n_heads, A.n_kv, A.window, A.sinks);
    QLIN_REQUIRE(sizes_ok(A.n_lanes, A.n_heads, A.n_kv, A.hd), QLIN_ERR_UNSUPPORTED,
                 "%s: head_dim %d is not a multiple of 16 in 16..256, or more than %d lanes (%d) or 65535 heads", fn, A.hd,
                 kMaxLanes, A.n_lanes);
    return QLIN_OK;
}

qlin_status attend(const char *fn, const AlArgs &A, void *workspace, size_t workspace_bytes, qlin_stream_t stream) {
    QLIN_REQUIRE(A.q && A.positions && A.seqs && A.out && workspace, QLIN_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (qlin_status e = check_sizes(fn, A)) return e;
    QLIN_REQUIRE(aligned16(A.q) && aligned16(A.out) && aligned16(workspace), QLIN_ERR_INVALID_ARG,
                 "%s: q, out and workspace are 16-byte aligned", fn);
    QLIN_REQUIRE(aligned4(A.positions) && aligned4(A.seqs) && aligned4(A.prefix_len) && aligned4(A.prefix_of) &&
                     aligned4(A.status),
                 QLIN_ERR_INVALID_ARG, "%s: pointer not 4-byte aligned", fn);
    int64_t rows;
    const AlWs w = carve(A.n_lanes, A.n_heads, A.n_kv, A.hd, (char *)workspace, &rows);
    QLIN_REQUIRE(workspace_bytes >= w.bytes, QLIN_ERR_INVALID_ARG, "%s: workspace %zu < %zu bytes", fn, workspace_bytes,
                 w.bytes);
    const bool f32 = A.own.type == QLIN_KV_F32;
    const AlDims D = al_dims(A);
    if (few_fits(A, D, f32, rows)) return attend_few(A, D, w, f32, (cudaStream_t)stream);
    const void *kern = f32 ? (const void *)al_attn_kernel<3> : (const void *)al_attn_kernel<1>;
    const size_t smem = kAlSmem, plan_smem = 6 * sizeof(int) * (size_t)A.n_lanes;
    QLIN_REQUIRE((int)smem <= max_smem_optin(), QLIN_ERR_UNSUPPORTED, "%s: shared memory", fn);
    blocks_per_sm(kern, smem);  // raises the dynamic shared-memory limit once
    blocks_per_sm((const void *)al_plan_kernel, plan_smem);
    AlMaps maps{};
    if (!f32)
        for (int st = 2 - D.streams; st < 2; st++) {
            const qlin_kv &c = st ? A.own : A.pre;
            if (qlin_status e = kv_map(c.k, c, A.n_kv * A.hd, &maps.k[st])) return e;
            if (qlin_status e = kv_map(c.v, c, A.n_kv * A.hd, &maps.v[st])) return e;
        }
    cudaStream_t st = (cudaStream_t)stream;
    void *pargs[] = {(void *)&A, (void *)&D, (void *)&w};
    if (A.n_lanes > kSelfPlan)
        if (qlin_status e = launch_pdl((const void *)al_plan_kernel, dim3(1), dim3(kPlanThreads), plan_smem, st, pargs,
                                       "al_plan_kernel"))
            return e;
    void *args[] = {(void *)&maps, (void *)&A, (void *)&D, (void *)&w};
    if (qlin_status e = launch_pdl(kern, dim3(D.grid), dim3(f32 ? AlCfg<3>::kThreads : AlCfg<1>::kThreads), smem, st, args,
                                   "al_attn_kernel"))
        return e;
    const int64_t total = (int64_t)A.n_lanes * A.n_heads, blocks = (total + D.merge - 1) / D.merge;
    return launch_pdl((const void *)al_merge_kernel, dim3((unsigned)(blocks < 8 * D.grid ? blocks : 8 * D.grid)),
                      dim3(kMergeThreads), 0, st, pargs, "al_merge_kernel");
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

size_t qlin_attention_lanes_workspace_size(int n_lanes, int n_heads, int n_kv, int head_dim) {
    return sizes_ok(n_lanes, n_heads, n_kv, head_dim) ? carve(n_lanes, n_heads, n_kv, head_dim, nullptr).bytes : 0;
}

int qlin_attention_on_tensor_cores(const qlin_kv *prefix, const qlin_kv *kv, int n_lanes, int n_heads, int n_kv,
                                   int head_dim, int window, int sinks) {
    qlin::clear_error();
    const char *fn = "qlin_attention_on_tensor_cores";
    if (prefix)
        if (qlin_status st = check_kv(fn, "prefix", prefix, n_kv, head_dim)) return -(int)st;
    if (qlin_status st = check_kv(fn, "kv", kv, n_kv, head_dim)) return -(int)st;
    if (qlin_status st = same_types(fn, prefix, kv)) return -(int)st;
    AlArgs A{};
    A.own = *kv;
    if (prefix) A.pre = *prefix;
    A.n_lanes = n_lanes, A.n_heads = n_heads, A.n_kv = n_kv, A.hd = head_dim, A.window = window, A.sinks = sinks;
    if (qlin_status st = check_sizes(fn, A)) return -(int)st;
    int64_t rows;
    carve(n_lanes, n_heads, n_kv, head_dim, nullptr, &rows);
    return few_fits(A, al_dims(A), kv->type == QLIN_KV_F32, rows) ? 0 : 1;
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
    if (qlin_status st = same_types("qlin_attention_prefix", prefix, kv)) return st;
    QLIN_REQUIRE(prefix_len, QLIN_ERR_INVALID_ARG, "qlin_attention_prefix: null pointer");
    AlArgs A{q, *kv, *prefix, positions, seqs, prefix_len, prefix_of, n_lanes, n_heads, n_kv, head_dim, window, sinks,
             out, status_word};
    return attend("qlin_attention_prefix", A, workspace, workspace_bytes, stream);
}

}  // extern "C"
