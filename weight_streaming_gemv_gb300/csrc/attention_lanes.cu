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
// head for up to 64 lanes (32 with fp32 caches) that read the same sequence:
// the lanes of a prompt chunk, the beams of a prompt, or one lane alone.  The
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
// accumulated (three for a bf16 cache, six for an fp32 one; what is left out
// is below 2^-24 of the product).
//
// A pass over the keys with a running maximum: thread t of four warps owns key
// t of a 128-key chunk (a tensor-memory lane).  The maximum of a row is over
// threads, so it is only taken when some score exceeds the one in use by 2^8
// (and for a tile's first chunk): otherwise weights relative to the maximum in
// use stay below 2^8 and nothing needs rescaling.  The sums stay in each
// thread's registers until the end.
//
// Work is dealt out by 128-key chunks: every CTA (one per SM) takes an equal
// run of the (tile, KV head, chunk) units, so a long sequence is split over
// many SMs and many short ones are packed, whatever the lengths, which are
// read on the device.  A tile that lies in one CTA is finished there; the
// others leave partial sums that a second kernel merges.  A planning kernel
// finds the tiles first.
//
// Keys and values go through a ring of 16 KB slots (x 3 terms): 128 keys x 64
// dims of K, 64 keys x 128 dims of V.  A bf16 cache's are tensor copies (TMA,
// 128-byte swizzle) straight from the cache; an fp32 cache's are loaded, split
// and stored by eight warps.
//
// Rows that nobody in the tile may see (behind the last position, before the
// window) are set to zero before their product, and a value that only some
// rows of a tile may see is replaced by zero where it is not finite, with the
// sums of the rows that do see it made NaN: 0 x NaN would reach the others.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <cmath>

#include "common.cuh"
#include "stream.cuh"
#include "tcgen05.cuh"

namespace qlin {
namespace {

constexpr int kMaxLanes = 4096;
constexpr int kStatusBadLane = 1;
constexpr int kMaxCtas = 160;  // the workspace holds two partial tiles for each
constexpr int kChunk = 128;    // keys per unit (MMA M)
constexpr float kNoKey = -1e30f;  // the running maximum of a row that has seen no key

struct AlArgs {
    const float *q;
    qlin_kv own, pre;  // pre.k null: no prompts
    const int32_t *positions, *seqs, *prefix_len, *prefix_of;
    int n_lanes, n_heads, n_kv, hd, window, sinks;
    float *out;
    int32_t *status;
};

// A tile: lanes lane0 .. lane0 + nl - 1, all of one sequence of one stream
// (stream 0: prompts, stream 1: the lanes' own caches).  Its chunks of that
// sequence's rows are 0 .. nsink - 1 and then cfirst, cfirst + 1, ...
struct __align__(16) AlTile {
    int64_t unit0;  // its first unit; units go (KV head, head block, chunk), chunk fastest
    int lane0, nl, stream, nch, nsink, cfirst;
    int slot;        // sequence (or prompt) in the stream's caches
    int base;        // position of the sequence's row 0
    int lim;         // its rows
    int pmin, pmax;  // the lanes' positions
    int pad;
};
static_assert(sizeof(AlTile) == 64, "tiles are loaded 16 bytes at a time");

struct AlPlanHead {
    int64_t units;
    int64_t grid;  // CTAs with work: the launch's, or one per unit if there are fewer
};

struct AlWs {
    AlPlanHead *head;
    int *first;    // [kMaxCtas]: the tile of a CTA's first unit
    int *tile_of;  // [2][n_lanes]
    AlTile *tiles; // [2 n_lanes]
    float2 *ml;    // per partial row: maximum (log2) and sum
    float *part;   // [rows][hd]: partial rows, 2 grid cap, then whole tiles' [2][n_lanes][n_heads]
    size_t bytes;
};

// What the kernels share besides the arguments.
struct AlDims {
    int group;  // query heads per KV head
    int R;      // row capacity of a tile
    int LT;     // lanes of a tile
    int HB;     // head blocks per KV head (1 unless group > R)
    int cap;    // partial rows per slot
    int streams;  // 1: own caches only, 2
    int grid;
    float c;    // log2(e) / sqrt(hd)
};

__device__ __forceinline__ float al_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------------ the plan
constexpr int kPlanThreads = 1024, kPlanPer = kMaxLanes / kPlanThreads;

// Inclusive scans over the block (every thread calls them).
__device__ __forceinline__ int plan_scan_max(int v, int *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v = max(v, o);
    }
    __syncthreads();
    if (lane == 31) red[warp] = v;
    __syncthreads();
    int before = -1;
    for (int w = 0; w < warp; w++) before = max(before, red[w]);
    return max(v, before);
}
__device__ __forceinline__ int64_t plan_scan_sum(int64_t v, int64_t *red, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    __syncthreads();
    if (lane == 31) red[warp] = v;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int w = 0; w < kPlanThreads / 32; w++) {
        if (w < warp) before += red[w];
        total += red[w];
    }
    return v + before;
}

// One CTA: checks the lanes, cuts them into tiles and deals the units out.
__global__ void __launch_bounds__(kPlanThreads) al_plan_kernel(AlArgs A, AlDims D, AlWs W) {
    extern __shared__ int pl_smem[];  // [3][n]: position (-1: no lane), sequence, prompt
    __shared__ int redi[32];
    __shared__ int64_t redl[32];
    const int tid = threadIdx.x, n = A.n_lanes;
    int *spos = pl_smem, *sseq = spos + n, *spre = sseq + n;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = tid; i < n; i += kPlanThreads) {
        const int p = A.positions[i], s = A.seqs[i];
        int f = 0, P = 0;
        bool ok = s >= 0 && s < A.own.n_seqs;
        if (A.pre.k) {
            f = A.prefix_of ? A.prefix_of[i] : 0;
            ok = ok && f >= 0 && f < A.pre.n_seqs;
            P = ok ? A.prefix_len[f] : 0;
            ok = ok && P >= 0 && P <= A.pre.rows;
        }
        ok = ok && p - P < A.own.rows;
        if (p >= 0 && !ok) raise_status(A.status, kStatusBadLane);
        spos[i] = p >= 0 && ok ? p : -1;
        sseq[i] = s;
        spre[i] = f;
    }
    __syncthreads();
    int64_t units = 0, tu0[2][kPlanPer], tun[2][kPlanPer];
    int tiles = 0, tix[2][kPlanPer];
    const int i0 = tid * kPlanPer;
    for (int st = 0; st < 2; st++) {
#pragma unroll
        for (int e = 0; e < kPlanPer; e++) tun[st][e] = 0;
        if (st == 0 && D.streams == 1) continue;
        auto same = [&](int a, int b) { return spre[a] == spre[b] && (st == 0 || sseq[a] == sseq[b]); };
        // where each lane's run of lanes of one sequence starts
        int rs[kPlanPer], last = -1;
        for (int e = 0; e < kPlanPer; e++) {
            const int i = i0 + e;
            if (i < n && spos[i] >= 0 && (i == 0 || spos[i - 1] < 0 || !same(i, i - 1))) last = i;
            rs[e] = last;
        }
        int before = plan_scan_max(last, redi);
        before = __shfl_up_sync(0xffffffffu, before, 1);
        if ((tid & 31) == 0) {
            before = -1;
            for (int w = 0; w < (tid >> 5); w++) before = max(before, redi[w]);
        }
        AlTile t[kPlanPer];
        int64_t mine = 0;  // tiles << 40 | units would overflow: two scans
        int nt = 0;
        for (int e = 0; e < kPlanPer; e++) {
            const int i = i0 + e;
            if (rs[e] < 0) rs[e] = before;
            const bool start = i < n && spos[i] >= 0 && (i - rs[e]) % D.LT == 0;
            t[e].nl = 0;
            if (!start) continue;
            int nl = 0, pmin = INT_MAX, pmax = -1;
            for (int j = i; j < n && nl < D.LT && spos[j] >= 0 && same(i, j); j++, nl++) {
                pmin = min(pmin, spos[j]);
                pmax = max(pmax, spos[j]);
            }
            const int P = A.pre.k ? A.prefix_len[spre[i]] : 0;
            const int64_t base = st == 0 ? 0 : P, lim = st == 0 ? P : A.own.rows;
            const int64_t hi = min((int64_t)pmax - base, lim - 1);
            const int64_t lo = A.window ? max((int64_t)0, (int64_t)pmin - A.window + 1 - base) : 0;
            const int64_t sk = max((int64_t)0, min((int64_t)A.sinks - base, hi + 1));
            const int64_t cf = lo / kChunk, main = lo <= hi ? hi / kChunk - cf + 1 : 0;
            int64_t ns = A.window ? (sk + kChunk - 1) / kChunk : 0;
            if (main > 0) ns = min(ns, cf);
            t[e].lane0 = i, t[e].nl = nl, t[e].stream = st, t[e].nch = (int)(ns + main), t[e].nsink = (int)ns;
            t[e].cfirst = (int)cf, t[e].slot = st == 0 ? spre[i] : sseq[i], t[e].base = (int)base, t[e].lim = (int)lim;
            t[e].pmin = pmin, t[e].pmax = pmax, t[e].pad = 0;
            nt++;
            tun[st][e] = (ns + main) * A.n_kv * D.HB;
            mine += tun[st][e];
        }
        int64_t tot_t, tot_u;
        int ti = tiles + (int)(plan_scan_sum(nt, redl, tot_t) - nt);
        int64_t u = units + plan_scan_sum(mine, redl, tot_u) - mine;
        for (int e = 0; e < kPlanPer; e++) {
            const int i = i0 + e;
            if (t[e].nl) {
                t[e].unit0 = u;
                W.tiles[ti] = t[e];
                tu0[st][e] = u;
                tix[st][e] = ti;
                u += tun[st][e];
                ti++;
            }
            if (i < n) W.tile_of[(int64_t)st * n + i] = spos[i] >= 0 ? ti - 1 : -1;
        }
        tiles += (int)tot_t;
        units += tot_u;
    }
    if (D.streams == 1)
        for (int i = tid; i < n; i += kPlanThreads) W.tile_of[i] = -1;
    // CTA b takes the units [U b / grid, U (b + 1) / grid): at least one each
    const int64_t grid = min((int64_t)D.grid, units);
    if (tid == 0) W.head->units = units, W.head->grid = grid;
    for (int st = 0; st < 2; st++)
        for (int e = 0; e < kPlanPer; e++)
            if (tun[st][e] > 0) {
                const int64_t u0 = tu0[st][e], u1 = u0 + tun[st][e];
                for (int64_t b = (u0 * grid + units - 1) / units; b < grid && units * b / grid < u1; b++)
                    W.first[b] = tix[st][e];
            }
}

// ------------------------------------------------------------------ the walk over a CTA's units
struct Piece {
    AlTile t;
    int kvh, hb, c0, c1;  // chunks c0 .. c1 - 1 of the tile for KV head kvh, head block hb
    int nrows, gs;        // rows, and rows per lane
    bool whole, head;     // all of its chunks; it is where the CTA's units start
};

struct Walker {
    int64_t u0, u, hi;
    int ti;
    AlTile t;
    __device__ __forceinline__ void load(const AlWs &W) {
        const int4 *p = reinterpret_cast<const int4 *>(W.tiles + ti);
        int4 *o = reinterpret_cast<int4 *>(&t);
#pragma unroll
        for (int k = 0; k < 4; k++) o[k] = __ldcg(p + k);
    }
    __device__ __forceinline__ explicit Walker(const AlWs &W) {
        const int64_t U = __ldcg(&W.head->units), G = __ldcg(&W.head->grid);
        u0 = u = hi = 0;
        if (blockIdx.x < G) {
            u0 = u = U * blockIdx.x / G;
            hi = U * (blockIdx.x + 1) / G;
            ti = __ldcg(&W.first[blockIdx.x]);
            load(W);
        }
    }
    __device__ __forceinline__ bool next(Piece &p, const AlArgs &A, const AlWs &W, const AlDims &D) {
        if (u >= hi) return false;
        while (u >= t.unit0 + (int64_t)t.nch * A.n_kv * D.HB) {
            ti++;
            load(W);
        }
        const int64_t r = u - t.unit0, sub = r / t.nch;
        p.t = t;
        p.kvh = (int)(sub / D.HB);
        p.hb = (int)(sub - (int64_t)p.kvh * D.HB);
        p.c0 = (int)(r - sub * t.nch);
        p.c1 = (int)min((int64_t)t.nch, p.c0 + (hi - u));
        p.gs = D.HB == 1 ? D.group : min(D.R, D.group - p.hb * D.R);
        p.nrows = t.nl * p.gs;
        p.whole = p.c0 == 0 && p.c1 == t.nch;
        p.head = u == u0;
        u += p.c1 - p.c0;
        return true;
    }
};

// The keys of chunk c of a piece, as rows of its sequence.
struct ChunkView {
    int r0;                       // its first row
    int any_lo, any_hi, sk;       // rows > any_lo or < sk, and <= any_hi, may be seen by some row of the tile
    int all_lo, all_hi;           // rows <= all_hi that are > all_lo or < sk are seen by every one
    bool edge;                    // not all of its keys are
    __device__ __forceinline__ ChunkView(const Piece &p, int c, const AlArgs &A) {
        r0 = (c < p.t.nsink ? c : p.t.cfirst + c - p.t.nsink) * kChunk;
        any_hi = (int)min((int64_t)p.t.pmax - p.t.base, (int64_t)p.t.lim - 1);
        all_hi = (int)min((int64_t)p.t.pmin - p.t.base, (int64_t)p.t.lim - 1);
        any_lo = all_lo = -1;
        sk = 0;
        if (A.window) {
            any_lo = (int)max((int64_t)-1, (int64_t)p.t.pmin - A.window - p.t.base);
            all_lo = (int)max((int64_t)-1, (int64_t)p.t.pmax - A.window - p.t.base);
            sk = max(0, A.sinks - p.t.base);
        }
        edge = !(r0 + kChunk - 1 <= all_hi && (r0 > all_lo || r0 + kChunk - 1 < sk));
    }
    __device__ __forceinline__ bool any(int r) const { return r <= any_hi && (r > any_lo || r < sk); }
    __device__ __forceinline__ bool all(int r) const { return r <= all_hi && (r > all_lo || r < sk); }
    // whether some row of the tile may see one of the rows [a, b)
    __device__ __forceinline__ bool any_in(int a, int b) const {
        return a <= any_hi && (b - 1 > any_lo || a < sk);
    }
};

// ------------------------------------------------------------------ the product
// NT: bf16 terms of a cached value (1: bf16 cache, 3: fp32 cache)
template <int NT>
struct AlCfg {
    static constexpr int R = NT == 1 ? 64 : 32;     // rows of a tile
    static constexpr int kSlots = NT == 1 ? 4 : 3;
    static constexpr int kTerm = 16384;             // 128 keys x 64 dims, or 64 keys x 128 dims, in bf16
    static constexpr int kSlot = NT * kTerm;
    static constexpr int kQBlock = R * 128;         // one term of 64 dims of the rows
    static constexpr int kQ = 4 * 3 * kQBlock;
    static constexpr int kPPitch = 2 * R;           // a key's weights, one term
    static constexpr int kPTerm = kChunk * kPPitch;
    static constexpr int kP = 3 * kPTerm;
    static constexpr int kProd = NT == 1 ? 1 : 8;   // producer warps
    static constexpr int kThreads = 32 * (4 + 1 + kProd);
    static constexpr uint32_t kCols = 4 * R;        // two S^T, two halves of O^T
};

template <int NT>
struct AlCtl {
    using C = AlCfg<NT>;
    uint64_t full[C::kSlots], empty[C::kSlots], fixed[C::kSlots];
    uint64_t s_full[2], p_ready, pv_done, q_ready, drain;
    int rowid[C::R];  // lane * n_heads + head
    int rowlo[C::R], rowhi[C::R];  // a row sees the keys <= rowhi that are > rowlo or first ones
    float mc[C::R], alpha[C::R];
    float red[4][C::R];
    uint32_t tmem;
    int abort;
};

template <int NT>
constexpr int al_smem() {
    using C = AlCfg<NT>;
    return 1024 + C::kSlots * C::kSlot + C::kQ + C::kP + (int)sizeof(AlCtl<NT>);
}
static_assert(al_smem<1>() <= 227 * 1024 && al_smem<3>() <= 227 * 1024, "shared memory of one CTA per SM");

// descriptor version 1; layout 2: 128-byte swizzle, 4: 64-byte
__device__ __forceinline__ uint64_t al_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)layout << 61;
}
__device__ __forceinline__ void al_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void al_tma(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// Bounded wait that also ends when another role gave up.
__device__ __forceinline__ bool al_wait(uint64_t *bar, uint32_t parity, int *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 0; i < (1u << 26); i++) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 63u && (*(volatile int *)abort || global_ns() - t0 > kWaitLimitNs)) return false;
    }
    return false;
}

// Two values as three pairs of bf16 terms (the first value in the low half).
__device__ __forceinline__ uint32_t al_pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void al_split2(float a, float b, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    hi = al_pack(a, b);
    a = __fsub_rn(a, __uint_as_float(hi << 16)), b = __fsub_rn(b, __uint_as_float(hi & 0xffff0000u));
    mid = al_pack(a, b);
    a = __fsub_rn(a, __uint_as_float(mid << 16)), b = __fsub_rn(b, __uint_as_float(mid & 0xffff0000u));
    lo = al_pack(a, b);
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Every lane's values of 32 columns -> lane l the reduction of column l over the warp.
template <bool MAX>
__device__ __forceinline__ float al_reduce32(float (&v)[32], int lane) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < off; i++) {
            const float send = (lane & off) ? v[i] : v[i + off], keep = (lane & off) ? v[i + off] : v[i];
            const float recv = __shfl_xor_sync(0xffffffffu, send, off);
            v[i] = MAX ? fmaxf(keep, recv) : __fadd_rn(keep, recv);
        }
    return v[0];
}

__device__ __forceinline__ void al_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool al_bar_or(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

struct AlMaps {
    CUtensorMap k[2], v[2];  // stream 0 (prompts), stream 1 (own)
};

// The slices of a CTA's pieces in the order in which they pass through the
// ring: K of chunk 0, then for every chunk K of the next one and its own V.
struct SliceGen {
    Walker w;
    Piece p;
    int n, i, sl;
    bool v, more;
    __device__ __forceinline__ SliceGen(const AlArgs &A, const AlWs &W, const AlDims &D) : w(W) { piece(A, W, D); }
    __device__ __forceinline__ void piece(const AlArgs &A, const AlWs &W, const AlDims &D) {
        more = w.next(p, A, W, D);
        n = p.c1 - p.c0;
        i = sl = 0;
        v = false;
    }
    __device__ __forceinline__ int chunk() const { return p.c0 + (v ? i - 1 : i); }
    __device__ __forceinline__ void step(const AlArgs &A, const AlWs &W, const AlDims &D, int nK, int nV) {
        if (++sl < (v ? nV : nK)) return;
        sl = 0;
        // step i: K of chunk i (if there is one), then V of chunk i - 1 (if there is one)
        if (!v && i >= 1) {
            v = true;
        } else if (!v && n == 1) {
            v = true, i = 1;
        } else {
            i++;
            v = i >= n;
            if (i > n) piece(A, W, D);
        }
    }
};

template <int NT>
__global__ void __launch_bounds__(AlCfg<NT>::kThreads, 1)
    al_attn_kernel(const __grid_constant__ AlMaps maps, AlArgs A, AlDims D, AlWs W) {
    using C = AlCfg<NT>;
    constexpr int R = C::R;
    extern __shared__ uint8_t al_raw[];
    uint8_t *const smem = al_raw + ((1024u - (smem_addr(al_raw) & 1023u)) & 1023u);  // the swizzled operands' alignment
    uint8_t *const ring = smem, *const qs = ring + C::kSlots * C::kSlot, *const ps = qs + C::kQ;
    AlCtl<NT> &S = *reinterpret_cast<AlCtl<NT> *>(ps + C::kP);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hd = A.hd;
    const int nK = (hd + 63) / 64, nDH = (hd + 127) / 128, nV = 2 * nDH;
    if (warp == 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&S.tmem)),
                     "r"(C::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int s = 0; s < C::kSlots; s++) {
            mbar_init(&S.full[s], C::kProd);
            mbar_init(&S.empty[s], 1);
            mbar_init(&S.fixed[s], 128);
        }
        mbar_init(&S.s_full[0], 1);
        mbar_init(&S.s_full[1], 1);
        mbar_init(&S.p_ready, 128);
        mbar_init(&S.pv_done, 1);
        mbar_init(&S.q_ready, 128);
        mbar_init(&S.drain, 1);
        S.abort = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan, and what the kernels before it wrote

    if (warp >= 5) {
        // ---------------------------------------------------------- producers
        if constexpr (NT == 1) {
            if (lane == 0) {
                SliceGen sg(A, W, D);
                int g = 0;
                for (; sg.more; g++) {
                    const int s = g % C::kSlots;
                    if (g >= C::kSlots && !al_wait(&S.empty[s], (uint32_t)(g / C::kSlots - 1) & 1u, &S.abort)) {
                        S.abort = 1;
                        raise_status(A.status, kStatusTimeout);
                        break;
                    }
                    const Piece &p = sg.p;
                    const ChunkView cv(p, sg.chunk(), A);
                    const CUtensorMap *map = sg.v ? &maps.v[p.t.stream] : &maps.k[p.t.stream];
                    const qlin_kv &kv = p.t.stream ? A.own : A.pre;
                    const int z = kv.seq_stride ? p.t.slot : 0;
                    uint8_t *to = ring + s * C::kSlot;
                    // two boxes of 64 keys x 64 dims, those that nobody sees left out: K's are the two halves of
                    // the chunk, V's (of one half) the two halves of 128 dims
                    int x[2], y[2];
                    bool on[2];
#pragma unroll
                    for (int b = 0; b < 2; b++) {
                        const int d = sg.v ? (sg.sl % nDH) * 128 + b * 64 : sg.sl * 64;
                        x[b] = p.kvh * hd + d;
                        y[b] = cv.r0 + (sg.v ? sg.sl / nDH : b) * 64;
                        on[b] = d < hd && cv.any_in(y[b], y[b] + 64);
                    }
                    mbar_arrive_expect_tx(&S.full[s], 8192u * ((uint32_t)on[0] + (uint32_t)on[1]));
#pragma unroll
                    for (int b = 0; b < 2; b++)
                        if (on[b]) al_tma(to + b * 8192, map, x[b], y[b], z, &S.full[s]);
                    sg.step(A, W, D, nK, nV);
                }
                if (S.abort)  // the copies in flight
                    for (int k = max(0, g - C::kSlots); k < g; k++)
                        mbar_wait(&S.full[k % C::kSlots], (uint32_t)(k / C::kSlots) & 1u);
            }
        } else {
            // 32 rows of 8 dims at a time: thread t takes row t / 8, dims 8 (t % 8) ..; four such passes are a
            // slice's 128 rows (a V slice's rows 64 .. 127 are the second 64 dims of its 64 keys)
            const int pt = tid - 160, pr = pt >> 3, pc = pt & 7;
            float4 buf[2][8];
            auto load = [&](SliceGen &sg, float4 (&o)[8]) {
                const Piece &p = sg.p;
                const ChunkView cv(p, sg.chunk(), A);
                const qlin_kv &kv = p.t.stream ? A.own : A.pre;
                const float *src = static_cast<const float *>(sg.v ? kv.v : kv.k) + (int64_t)p.t.slot * kv.seq_stride +
                                   p.kvh * hd + 8 * pc;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int r = e * 32 + pr;
                    const int key = cv.r0 + (sg.v ? (sg.sl / nDH) * 64 + (r & 63) : r);
                    const int d = sg.v ? (sg.sl % nDH) * 128 + (r >> 6) * 64 : sg.sl * 64;
                    o[2 * e] = o[2 * e + 1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (d + 8 * pc < hd && cv.any(key)) {
                        const float *a = src + (int64_t)key * kv.row_stride + d;
                        const uint4 u = ld_stream_v4(a), w = ld_stream_v4(a + 4);
                        o[2 * e] = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                                               __uint_as_float(u.w));
                        o[2 * e + 1] = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                                                   __uint_as_float(w.w));
                    }
                }
            };
            SliceGen sg(A, W, D);
            bool have[2] = {false, false};
#pragma unroll
            for (int k = 0; k < 2; k++)
                if (sg.more) {
                    load(sg, buf[k]);
                    have[k] = true;
                    sg.step(A, W, D, nK, nV);
                }
            bool ok = true;
            for (int g = 0; ok && have[0]; g += 2) {
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    if (!have[k]) break;
                    const int gg = g + k, s = gg % C::kSlots;
                    if (gg >= C::kSlots && !al_wait(&S.empty[s], (uint32_t)(gg / C::kSlots - 1) & 1u, &S.abort)) {
                        S.abort = 1;
                        raise_status(A.status, kStatusTimeout);
                        ok = false;
                        break;
                    }
                    const uint32_t to = smem_addr(ring + s * C::kSlot);
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int r = e * 32 + pr;
                        const float4 a = buf[k][2 * e], b = buf[k][2 * e + 1];
                        uint4 h, m, l;
                        al_split2(a.x, a.y, h.x, m.x, l.x);
                        al_split2(a.z, a.w, h.y, m.y, l.y);
                        al_split2(b.x, b.y, h.z, m.z, l.z);
                        al_split2(b.z, b.w, h.w, m.w, l.w);
                        const uint32_t at = to + (uint32_t)(r * 128 + ((pc ^ (r & 7)) << 4));
                        sts128(at, h);
                        sts128(at + C::kTerm, m);
                        sts128(at + 2 * C::kTerm, l);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.full[s]);
                    have[k] = sg.more;
                    if (sg.more) {
                        load(sg, buf[k]);
                        sg.step(A, W, D, nK, nV);
                    }
                }
            }
        }
    } else if (warp == 4) {
        // ---------------------------------------------------------- the MMAs
        if (lane == 0) {
            Walker w(W);
            Piece p;
            int g = 0, it = 0;  // slices and chunks so far
            uint32_t fixpar = 0;
            bool ok = true;
            const uint32_t ring_a = smem_addr(ring), qs_a = smem_addr(qs), ps_a = smem_addr(ps);
            constexpr uint32_t kPLayout = R == 64 ? 2u : 4u;
            for (int np = 0; ok && w.next(p, A, W, D); np++) {
                const int n = p.c1 - p.c0;
                const uint32_t N = (uint32_t)(p.nrows + 15) / 16 * 16;
                // fp32 accumulator, bf16 operands; S^T: both K-major, O^T: both with the keys as rows
                const uint32_t ids = (1u << 4) | (1u << 7) | (1u << 10) | (N >> 3) << 17 | (128u >> 4) << 24;
                const uint32_t idp = ids | (1u << 15) | (1u << 16);
                if (!(ok = al_wait(&S.q_ready, (uint32_t)np & 1u, &S.abort))) break;
                for (int i = 0; ok && i <= n; i++) {
                    if (i < n) {
                        const uint32_t d = tmem + (uint32_t)((it + i) & 1) * R;
                        for (int sl = 0; sl < nK; sl++, g++) {
                            const int s = g % C::kSlots;
                            if (!(ok = al_wait(&S.full[s], (uint32_t)(g / C::kSlots) & 1u, &S.abort))) break;
                            tc_fence_after();
                            const int steps = min(64, hd - sl * 64) / 16;
                            for (int kk = 0; kk < steps; kk++)
#pragma unroll
                                for (int t = 0; t < NT; t++)
#pragma unroll
                                    for (int u = 0; u < 3 - t; u++)
                                        al_mma(d, al_desc(ring_a + s * C::kSlot + t * C::kTerm + 32 * kk, 16, 1024, 2),
                                               al_desc(qs_a + (sl * 3 + u) * C::kQBlock + 32 * kk, 16, 1024, 2), ids,
                                               sl > 0 || kk > 0 || t > 0 || u > 0);
                            tc_commit(&S.empty[s]);
                        }
                        if (!ok) break;
                        tc_commit(&S.s_full[(it + i) & 1]);
                    }
                    if (i >= 1) {
                        const ChunkView cv(p, p.c0 + i - 1, A);
                        if (!(ok = al_wait(&S.p_ready, (uint32_t)(it + i - 1) & 1u, &S.abort))) break;
                        for (int vs = 0; vs < nV; vs++, g++) {
                            const int s = g % C::kSlots, kh = vs / nDH, dh = vs % nDH;
                            if (!(ok = al_wait(&S.full[s], (uint32_t)(g / C::kSlots) & 1u, &S.abort))) break;
                            if (cv.edge) {
                                if (!(ok = al_wait(&S.fixed[s], (fixpar >> s) & 1u, &S.abort))) break;
                                fixpar ^= 1u << s;
                            }
                            tc_fence_after();
                            const uint32_t d = tmem + (uint32_t)(2 + dh) * R;
                            for (int ks = 0; ks < 4; ks++)
#pragma unroll
                                for (int t = 0; t < NT; t++)
#pragma unroll
                                    for (int u = 0; u < 3 - t; u++)
                                        al_mma(d, al_desc(ring_a + s * C::kSlot + t * C::kTerm + 2048 * ks, 8192, 1024, 2),
                                               al_desc(ps_a + u * C::kPTerm + (kh * 64 + ks * 16) * C::kPPitch, 16,
                                                       8 * C::kPPitch, kPLayout),
                                               idp, i > 1 || kh > 0 || ks > 0 || t > 0 || u > 0);
                            tc_commit(&S.empty[s]);
                        }
                        if (!ok) break;
                        tc_commit(&S.pv_done);
                    }
                }
                it += n;
            }
            if (!ok) {
                S.abort = 1;
                raise_status(A.status, kStatusTimeout);
                tc_commit(&S.drain);  // the MMAs in flight
                mbar_wait(&S.drain, 0);
            }
        }
    } else {
        // ---------------------------------------------------------- weights: thread t owns key t of a chunk
        Walker w(W);
        Piece p;
        int g = 0, it = 0;
        const uint32_t tl = tmem + ((uint32_t)(32 * warp) << 16);
        const float ninf = -__int_as_float(0x7f800000);
        bool ok = true;
        while (ok && w.next(p, A, W, D)) {
            const int n = p.c1 - p.c0, nr = (p.nrows + 15) / 16 * 16;
            al_bar();  // the rows of the last piece are no longer needed
            if (tid < nr) {
                const int r = tid, ln = p.t.lane0 + r / p.gs;
                const bool in = r < p.nrows;
                const int64_t pl = in ? (int64_t)A.positions[ln] - p.t.base : -1;
                S.rowid[r] = in ? ln * A.n_heads + p.kvh * D.group + p.hb * R + r % p.gs : -1;
                S.rowhi[r] = (int)max((int64_t)-1, min(pl, (int64_t)p.t.lim - 1));
                S.rowlo[r] = A.window ? (int)max((int64_t)-1, pl - A.window) : -1;
                S.mc[r] = kNoKey;
            }
            al_bar();
            // the rows' q as three bf16 terms, 64 dims after 64 dims, rows of 128 swizzled bytes
            for (int e = tid; e < nr * (hd / 8); e += 128) {
                const int r = e / (hd / 8), d8 = e - r * (hd / 8), id = S.rowid[r];
                float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
                if (id >= 0) {
                    const float4 *src = reinterpret_cast<const float4 *>(A.q + (int64_t)id * hd + 8 * d8);
                    a = __ldg(src), b = __ldg(src + 1);
                }
                uint4 h, m, l;
                al_split2(a.x, a.y, h.x, m.x, l.x);
                al_split2(a.z, a.w, h.y, m.y, l.y);
                al_split2(b.x, b.y, h.z, m.z, l.z);
                al_split2(b.z, b.w, h.w, m.w, l.w);
                const uint32_t at = smem_addr(qs) + (uint32_t)((d8 >> 3) * 3 * C::kQBlock + r * 128 +
                                                               (((d8 & 7) ^ (r & 7)) << 4));
                sts128(at, h);
                sts128(at + C::kQBlock, m);
                sts128(at + 2 * C::kQBlock, l);
            }
            fence_proxy_async_smem();
            mbar_arrive(&S.q_ready);
            float lsum[R];
#pragma unroll
            for (int r = 0; r < R; r++) lsum[r] = 0.0f;

            for (int i = 0; i < n; i++, it++) {
                const ChunkView cv(p, p.c0 + i, A);
                const int key = cv.r0 + tid;
                bool fail = !al_wait(&S.s_full[it & 1], (uint32_t)(it >> 1) & 1u, &S.abort);
                __syncwarp();  // (the tensor-memory loads are for whole warps)
                tc_fence_after();
                const uint32_t ts = tl + (uint32_t)(it & 1) * R;
                // whether this row of the tile sees this thread's key
                auto sees = [&](int r) {
                    return key <= S.rowhi[r] && (key > S.rowlo[r] || key < cv.sk);
                };
                bool big = i == 0;
                if (i > 0) {
#pragma unroll
                    for (int b = 0; b < R / 16; b++)
                        if (b * 16 < nr) {
                            uint32_t v[16];
                            tm_ld16(ts + 16 * b, v);
#pragma unroll
                            for (int j = 0; j < 16; j++) {
                                const float x = __fmaf_rn(__uint_as_float(v[j]), D.c, -S.mc[16 * b + j]);
                                if (!cv.edge || sees(16 * b + j)) big |= x > 8.0f;
                            }
                        }
                }
                if (al_bar_or(fail)) {
                    if (fail) {
                        S.abort = 1;
                        raise_status(A.status, kStatusTimeout);
                    }
                    ok = false;
                    break;
                }
                if (al_bar_or(big)) {
                    // new maxima
#pragma unroll
                    for (int b = 0; b < R / 32; b++)
                        if (b * 32 < nr) {
                            uint32_t v0[16], v1[16];
                            float m[32];
                            tm_ld16(ts + 32 * b, v0);
                            tm_ld16(ts + 32 * b + 16, v1);
#pragma unroll
                            for (int j = 0; j < 16; j++) {
                                const int r = 32 * b + j;
                                m[j] = !cv.edge || sees(r) ? __uint_as_float(v0[j]) : ninf;
                                m[j + 16] = r + 16 < nr && (!cv.edge || sees(r + 16)) ? __uint_as_float(v1[j]) : ninf;
                            }
                            const float top = al_reduce32<true>(m, lane);
                            S.red[warp][32 * b + lane] = top;
                        }
                    al_bar();
                    if (tid < nr) {
                        const float m = fmaxf(fmaxf(S.red[0][tid], S.red[1][tid]), fmaxf(S.red[2][tid], S.red[3][tid]));
                        const float old = S.mc[tid];
                        const float mc = m > ninf ? fmaxf(__fmul_rn(m, D.c), old) : old;
                        S.mc[tid] = mc;
                        S.alpha[tid] = old == kNoKey ? 0.0f : al_ex2(__fsub_rn(old, mc));
                    }
                    al_bar();
                    if (i > 0) {
#pragma unroll
                        for (int r = 0; r < R; r++)
                            if (r < nr) lsum[r] = __fmul_rn(lsum[r], S.alpha[r]);
                        // O^T: the products of the chunk before are in
                        al_wait(&S.pv_done, (uint32_t)(it - 1) & 1u, &S.abort);
                        __syncwarp();
                        tc_fence_after();
                        for (int dh = 0; dh < nDH; dh++)
                            for (int b = 0; b * 16 < nr; b++) {
                                uint32_t v[16];
                                const uint32_t to = tl + (uint32_t)((2 + dh) * R + 16 * b);
                                tm_ld16(to, v);
#pragma unroll
                                for (int j = 0; j < 16; j++)
                                    v[j] = __float_as_uint(__fmul_rn(__uint_as_float(v[j]), S.alpha[16 * b + j]));
                                tm_st16(to, v);
                            }
                        tm_wait_st();
                    }
                }
                // the weights, as three bf16 terms, a key's rows side by side
                if (i > 0) al_wait(&S.pv_done, (uint32_t)(it - 1) & 1u, &S.abort);  // P is read
                __syncwarp();
                const uint32_t prow = smem_addr(ps) + (uint32_t)(tid * C::kPPitch);
                const uint32_t px = R == 64 ? (uint32_t)(tid & 7) : (uint32_t)((tid >> 1) & 3);
#pragma unroll
                for (int b = 0; b < R / 16; b++)
                    if (b * 16 < nr) {
                        uint32_t v[16];
                        tm_ld16(ts + 16 * b, v);
                        float w16[16];
#pragma unroll
                        for (int j = 0; j < 16; j++) {
                            const float x = __fmaf_rn(__uint_as_float(v[j]), D.c, -S.mc[16 * b + j]);
                            w16[j] = !cv.edge || sees(16 * b + j) ? al_ex2(x) : 0.0f;
                            lsum[16 * b + j] = __fadd_rn(lsum[16 * b + j], w16[j]);
                        }
#pragma unroll
                        for (int q = 0; q < 2; q++) {
                            uint4 h, m, l;
                            al_split2(w16[8 * q], w16[8 * q + 1], h.x, m.x, l.x);
                            al_split2(w16[8 * q + 2], w16[8 * q + 3], h.y, m.y, l.y);
                            al_split2(w16[8 * q + 4], w16[8 * q + 5], h.z, m.z, l.z);
                            al_split2(w16[8 * q + 6], w16[8 * q + 7], h.w, m.w, l.w);
                            const uint32_t at = prow + ((((uint32_t)(2 * b + q)) ^ px) << 4);
                            sts128(at, h);
                            sts128(at + C::kPTerm, m);
                            sts128(at + 2 * C::kPTerm, l);
                        }
                    }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&S.p_ready);
                if (cv.edge) {
                    // the values of keys that not every row sees
                    const int gv = g + min(i + 2, n) * nK + i * nV;
                    const bool any = cv.any(key), all = cv.all(key);
                    bool bad = false;
                    for (int vs = 0; vs < nV; vs++) {
                        const int s = (gv + vs) % C::kSlots;
                        al_wait(&S.full[s], (uint32_t)((gv + vs) / C::kSlots) & 1u, &S.abort);
                        if (!all && (tid >> 6) == vs / nDH) {
                            const uint32_t row = smem_addr(ring + s * C::kSlot) + (uint32_t)((tid & 63) * 128);
                            bool nf = !any;
                            if (any)
                                for (int q = 0; q < 16; q++) {
                                    const int d = (vs % nDH) * 128 + 8 * q;
                                    // a row of 64 dims is 8 groups of 16 bytes, swizzled by the row
                                    const uint32_t at = row + (q >> 3) * 8192 + (((q & 7) ^ (tid & 7)) << 4);
                                    if (d < hd) {
                                        uint4 v;
                                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                                     : "r"(at));
                                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                        for (int k = 0; k < 4; k++)
                                            nf |= (u[k] & 0x7f80u) == 0x7f80u || (u[k] & 0x7f800000u) == 0x7f800000u;
                                    }
                                }
                            if (nf) {
                                bad |= any;
                                for (int t = 0; t < NT; t++)
                                    for (int q = 0; q < 16; q++)
                                        sts128(row + t * C::kTerm + (q >> 3) * 8192 + ((q & 7) << 4), make_uint4(0, 0, 0, 0));
                            }
                        }
                        fence_proxy_async_smem();
                        mbar_arrive(&S.fixed[s]);
                    }
                    if (bad)
#pragma unroll
                        for (int r = 0; r < R; r++)
                            if (r < nr && sees(r)) lsum[r] = __int_as_float(0x7fc00000);
                }
            }
            if (!ok) break;
            g += n * (nK + nV);
            // the sums over the keys
#pragma unroll
            for (int b = 0; b < R / 32; b++)
                if (b * 32 < nr) {
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; j++) v[j] = lsum[32 * b + j];
                    const float l = al_reduce32<false>(v, lane);
                    S.red[warp][32 * b + lane] = l;
                }
            if (al_bar_or(!al_wait(&S.pv_done, (uint32_t)(it - 1) & 1u, &S.abort))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const bool direct = p.whole && D.streams == 1;
            const int64_t prow0 = p.whole ? (int64_t)2 * D.grid * D.cap + (int64_t)p.t.stream * A.n_lanes * A.n_heads
                                          : (int64_t)(2 * blockIdx.x + (p.head ? 0 : 1)) * D.cap;
            if (tid < p.nrows) {
                const float l = S.red[0][tid] + S.red[1][tid] + S.red[2][tid] + S.red[3][tid];
                S.alpha[tid] = direct ? (l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l)) : 1.0f;
                if (!direct) W.ml[prow0 + (p.whole ? S.rowid[tid] : tid)] = make_float2(S.mc[tid], l);
            }
            al_bar();
            for (int dh = 0; dh < nDH; dh++) {
                const int d = dh * 128 + tid;
                for (int b = 0; b * 16 < p.nrows; b++) {
                    uint32_t v[16];
                    tm_ld16(tl + (uint32_t)((2 + dh) * R + 16 * b), v);
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        const int r = 16 * b + j;
                        if (r < p.nrows && d < hd) {
                            const int64_t id = S.rowid[r];
                            float *o = direct ? A.out + id * hd : W.part + (prow0 + (p.whole ? id : r)) * hd;
                            o[d] = __fmul_rn(__uint_as_float(v[j]), S.alpha[r]);
                        }
                    }
                }
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
}

// ------------------------------------------------------------------ merging partial tiles
constexpr int kMergeThreads = 256;

// One (lane, head) after the other: the pieces of its tiles by the weights
// 2^(maximum - largest maximum); zeros where there are none.
__global__ void __launch_bounds__(kMergeThreads) al_merge_kernel(AlArgs A, AlDims D, AlWs W) {
    __shared__ float w[2 * kMaxCtas];
    __shared__ int64_t row[2 * kMaxCtas];
    __shared__ float red[8];
    __shared__ float4 acc[kMergeThreads];
    const int tid = threadIdx.x, warp = tid >> 5, lane_t = tid & 31, hd = A.hd;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t U = __ldcg(&W.head->units), G = __ldcg(&W.head->grid);
    const int total = A.n_lanes * A.n_heads;
    for (int idx = blockIdx.x; idx < total; idx += gridDim.x) {
        const int lane = idx / A.n_heads, h = idx - lane * A.n_heads;
        const int kvh = h / D.group, hg = h - kvh * D.group, hb = hg / D.R;
        int n = 0;
        bool done = false;
        __syncthreads();
        for (int st = 2 - D.streams; st < 2; st++) {
            const int ti = __ldcg(&W.tile_of[(int64_t)st * A.n_lanes + lane]);
            if (ti < 0) continue;
            const AlTile *t = W.tiles + ti;
            const int nch = __ldcg(&t->nch);
            if (nch == 0) continue;
            const int gs = D.HB == 1 ? D.group : min(D.R, D.group - hb * D.R);
            const int r = (lane - __ldcg(&t->lane0)) * gs + hg - hb * D.R;
            const int64_t u0 = __ldcg(&t->unit0) + (int64_t)(kvh * D.HB + hb) * nch, u1 = u0 + nch;
            const int b0 = (int)(((u0 + 1) * G - 1) / U), b1 = (int)((u1 * G - 1) / U);
            if (b0 == b1 && D.streams == 1) {
                done = true;
                break;
            }
            for (int b = b0 + tid; b <= b1; b += kMergeThreads) {
                const bool head = U * b / G >= u0;
                row[n + b - b0] = b0 == b1 ? (int64_t)2 * D.grid * D.cap + (int64_t)st * total + idx
                                           : (int64_t)(2 * b + (head ? 0 : 1)) * D.cap + r;
            }
            n += b1 - b0 + 1;
        }
        if (done) continue;
        float *o = A.out + (int64_t)idx * hd;
        if (n == 0) {
            for (int d = tid; d < hd; d += kMergeThreads) o[d] = 0.0f;
            continue;
        }
        __syncthreads();
        float m = kNoKey, l[2] = {0.0f, 0.0f}, mi[2];
#pragma unroll
        for (int k = 0; k < 2; k++)
            if (tid + k * kMergeThreads < n) {
                const float2 v = __ldcg(&W.ml[row[tid + k * kMergeThreads]]);
                mi[k] = v.x, l[k] = v.y;
                m = fmaxf(m, v.x);
            }
        m = warp_max(m);
        if (lane_t == 0) red[warp] = m;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; k++) m = fmaxf(m, red[k]);
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; k++)
            if (tid + k * kMergeThreads < n) {
                const float x = mi[k] == kNoKey ? 0.0f : al_ex2(__fsub_rn(mi[k], m));
                w[tid + k * kMergeThreads] = x;
                sum += x * l[k];
            }
        sum = warp_psum(sum);
        __syncthreads();
        if (lane_t == 0) red[warp] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; k++) sum += red[k];
        // thread: four dims, every `groups`-th piece
        const int nv = hd / 4, groups = kMergeThreads / nv, gi = tid / nv, dv = tid - gi * nv;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (gi < groups)
#pragma unroll 4
            for (int k = gi; k < n; k += groups) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(W.part + row[k] * hd) + dv);
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
            const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
            reinterpret_cast<float4 *>(o)[tid] = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        }
    }
}

// ------------------------------------------------------------------ host
size_t align256(size_t b) { return (b + 255) / 256 * 256; }

AlWs carve(int n_lanes, int n_heads, int n_kv, int hd, char *base) {
    AlWs w{};
    size_t off = 0;
    auto take = [&](size_t b) {
        char *p = base ? base + off : nullptr;
        off += align256(b);
        return p;
    };
    const int64_t group = n_heads / n_kv;
    const int64_t rows = (int64_t)2 * kMaxCtas * (n_lanes * group < 64 ? n_lanes * group : 64) +
                         (int64_t)2 * n_lanes * n_heads;
    w.head = (AlPlanHead *)take(sizeof(AlPlanHead));
    w.first = (int *)take(sizeof(int) * kMaxCtas);
    w.tile_of = (int *)take(sizeof(int) * 2 * (size_t)n_lanes);
    w.tiles = (AlTile *)take(sizeof(AlTile) * 2 * (size_t)n_lanes);
    w.ml = (float2 *)take(sizeof(float2) * (size_t)rows);
    w.part = (float *)take(sizeof(float) * (size_t)rows * hd);
    w.bytes = off;
    return w;
}

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
    const AlWs w = carve(A.n_lanes, A.n_heads, A.n_kv, A.hd, (char *)workspace);
    QLIN_REQUIRE(workspace_bytes >= w.bytes, QLIN_ERR_INVALID_ARG, "%s: workspace %zu < %zu bytes", fn, workspace_bytes,
                 w.bytes);
    const bool f32 = A.own.type == QLIN_KV_F32;
    AlDims D{};
    D.group = A.n_heads / A.n_kv;
    D.R = f32 ? AlCfg<3>::R : AlCfg<1>::R;
    D.LT = D.group < D.R ? D.R / D.group : 1;
    D.HB = (D.group + D.R - 1) / D.R;
    D.cap = (int64_t)A.n_lanes * D.group < D.R ? A.n_lanes * D.group : D.R;
    D.streams = A.pre.k ? 2 : 1;
    D.grid = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
    D.c = (float)(1.4426950408889634 / std::sqrt((double)A.hd));
    const void *kern = f32 ? (const void *)al_attn_kernel<3> : (const void *)al_attn_kernel<1>;
    const size_t smem = f32 ? al_smem<3>() : al_smem<1>(), plan_smem = 3 * sizeof(int) * (size_t)A.n_lanes;
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
    if (qlin_status e = launch_pdl((const void *)al_plan_kernel, dim3(1), dim3(kPlanThreads), plan_smem, st, pargs,
                                   "al_plan_kernel"))
        return e;
    void *args[] = {(void *)&maps, (void *)&A, (void *)&D, (void *)&w};
    if (qlin_status e = launch_pdl(kern, dim3(D.grid), dim3(f32 ? AlCfg<3>::kThreads : AlCfg<1>::kThreads), smem, st, args,
                                   "al_attn_kernel"))
        return e;
    const int64_t total = (int64_t)A.n_lanes * A.n_heads;
    return launch_pdl((const void *)al_merge_kernel, dim3((unsigned)(total < 8 * D.grid ? total : 8 * D.grid)),
                      dim3(kMergeThreads), 0, st, pargs, "al_merge_kernel");
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

size_t qlin_attention_lanes_workspace_size(int n_lanes, int n_heads, int n_kv, int head_dim) {
    return sizes_ok(n_lanes, n_heads, n_kv, head_dim) ? carve(n_lanes, n_heads, n_kv, head_dim, nullptr).bytes : 0;
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
