// What the attention over lanes on the tensor cores is made of, whatever holds
// its keys and values: lanes are cut into tiles and tiles into units (the plan),
// every CTA walks over its own (the pieces), and partial tiles are merged.
#pragma once
#include <climits>

#include "launch.cuh"
#include "stream.cuh"
#include "tcgen05.cuh"

namespace qlin {
namespace {

constexpr int kMaxLanes = 4096;
constexpr int kStatusBadLane = 1;
constexpr int kMaxCtas = 160;  // the workspace holds two partial tiles for each
constexpr int kChunk = 128;    // keys per unit (MMA M)
constexpr float kNoKey = -3.402823466e38f;  // the running maximum of a row that has seen no key: no score is below it

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
    int64_t unit0;  // its first unit; units go (KV head, head block, AlDims::setup and then the chunks)
    uint16_t lane0;
    uint8_t nl, stream;
    int nch, nsink, cfirst;
    int slot;        // sequence (or prompt) in the stream's caches
    int base;        // position of the sequence's row 0
    int lim;         // its rows
    int pmin, pmax;  // the lanes' positions
    int pad;
};
static_assert(sizeof(AlTile) == 48 && kMaxLanes <= 65536, "tiles in shared memory");

struct AlPlanHead {
    int64_t units;
    int grid;  // CTAs with work: the launch's, or one per unit if there are fewer
    int rmax;  // rows of the widest tile
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
    int merge;  // (lane, head)s per block of the merging kernel
    int setup;  // units that a tile's start is counted as (its rows' q, the first scores, the outputs)
    float c;    // log2(e) / sqrt(hd)
};

__device__ __forceinline__ float al_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------------ the plan
constexpr int kPlanThreads = 1024;
constexpr int kSelfPlan = 64;  // lanes up to which every CTA plans for itself, a thread for each

struct AlSelfPlan {  // in shared memory
    AlPlanHead head;
    AlTile tiles[2 * kSelfPlan];
    int first;
};

// The first unit of CTA b of the `grid` that have work: units * b / grid (in 32
// bits where that is enough: it stands at the head of every CTA's work).
__device__ __forceinline__ int64_t unit_of(int64_t units, int b, int grid, const AlDims &D) {
    if (units <= D.grid) return b;
    const uint64_t p = (uint64_t)units * (uint32_t)b;
    return (p >> 32) ? (int64_t)(p / (uint32_t)grid) : (int64_t)((uint32_t)p / (uint32_t)grid);
}

__device__ __forceinline__ int64_t tile_units(int nch, const AlArgs &A, const AlDims &D) {
    return nch ? (int64_t)(nch + D.setup) * A.n_kv * D.HB : 0;
}

struct PlanRed {
    int64_t sum[32];
    int last[32];
};
struct AlSelfScratch {
    int tile_of[2 * kSelfPlan];
    int lane[6 * kSelfPlan];
    PlanRed red;
};

// Checks the lanes, cuts them into tiles and deals the units out.  T threads
// of the block, the first ones, take T lanes at a time (barrier 1 among them);
// scratch: [6 n_lanes].  first: the first tile of CTA `cta`, or of every CTA
// if that is negative.
template <int T>
__device__ __forceinline__ void make_plan(const AlArgs &A, const AlDims &D, int *scratch, PlanRed &red, AlPlanHead *head,
                                          int *first, int cta, int *tile_of, AlTile *tiles_out, int32_t *status) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = A.n_lanes;
    // per lane: position (-1: no lane), sequence, prompt; of the tile that starts at it: lanes, least and largest position
    int *spos = scratch, *sseq = spos + n, *spre = sseq + n, *snl = spre + n, *smin = snl + n, *smax = smin + n;
    auto bar = [] { asm volatile("bar.sync 1, %0;" ::"n"(T) : "memory"); };
#pragma unroll 1
    for (int i = tid; i < n; i += T) {
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
        if (p >= 0 && !ok) raise_status(status, kStatusBadLane);
        spos[i] = p >= 0 && ok ? p : -1;
        sseq[i] = s;
        spre[i] = f;
    }
    int64_t units = 0;
    int tiles = 0, rmax = 0;
#pragma unroll 1
    for (int st = 2 - D.streams; st < 2; st++) {
        auto same = [&](int a, int b) { return spre[a] == spre[b] && (st == 0 || sseq[a] == sseq[b]); };
        int run = -1;  // where the latest run of lanes of one sequence starts
#pragma unroll 1
        for (int i = tid; i < n; i += T) snl[i] = 0, smin[i] = INT_MAX, smax[i] = -1;
#pragma unroll 1
        for (int base = 0; base < n; base += T) {
            bar();
            const int i = base + tid;
            const bool valid = i < n && spos[i] >= 0;
            const uint32_t starts =
                __ballot_sync(0xffffffffu, valid && (i == 0 || spos[i - 1] < 0 || !same(i, i - 1)));
            if (lane == 0) red.last[warp] = starts ? i + 31 - __clz(starts) : -1;
            bar();
            int rs = run;
            if (T == 64) {
                if (warp == 1) rs = max(rs, red.last[0]);
                run = max(run, max(red.last[0], red.last[1]));
            } else {
                const int lw = lane < T / 32 ? red.last[lane] : -1;
                rs = max(run, __reduce_max_sync(0xffffffffu, lane < warp ? lw : -1));
                run = max(run, __reduce_max_sync(0xffffffffu, lw));
            }
            const uint32_t upto = starts & (0xffffffffu >> (31 - lane));
            if (upto) rs = i - lane + 31 - __clz(upto);
            const int in_tile = valid ? (i - rs) % D.LT : 0;
            const bool start = valid && in_tile == 0;
            if (valid) {
                atomicAdd(&snl[i - in_tile], 1);
                atomicMin(&smin[i - in_tile], spos[i]);
                atomicMax(&smax[i - in_tile], spos[i]);
            }
            // (a tile that reaches the last of these lanes may go on behind them: its first lane looks)
            bar();
            AlTile t;
            int64_t tu = 0;
            if (start) {
                int nl = snl[i], pmin = smin[i], pmax = smax[i];
                if (i + nl == base + T)
                    for (int j = base + T; j < n && j < i + D.LT && spos[j] >= 0 && same(i, j); j++, nl++) {
                        pmin = min(pmin, spos[j]);
                        pmax = max(pmax, spos[j]);
                    }
                // positions and rows are below 2^31, so differences fit
                const int P = A.pre.k ? A.prefix_len[spre[i]] : 0;
                const int org = st == 0 ? 0 : P, lim = st == 0 ? P : A.own.rows;
                const int hi = min(pmax - org, lim - 1);
                const int lo = A.window && pmin - org >= A.window ? pmin - org - A.window + 1 : 0;
                const int sk = A.window ? max(0, min(A.sinks - org, hi + 1)) : 0;
                const int cf = lo / kChunk, main = lo <= hi ? hi / kChunk - cf + 1 : 0;
                int ns = (sk + kChunk - 1) / kChunk;
                if (main > 0) ns = min(ns, cf);
                t.lane0 = (uint16_t)i, t.nl = (uint8_t)nl, t.stream = (uint8_t)st, t.nch = ns + main, t.nsink = ns, t.cfirst = cf;
                t.slot = st == 0 ? spre[i] : sseq[i], t.base = org, t.lim = lim;
                t.pmin = pmin, t.pmax = pmax, t.pad = 0;
                tu = tile_units(t.nch, A, D);
                if (t.nch > 0) rmax = max(rmax, nl * min(D.group, D.R));
            }
            // tiles and units before this lane's, in one sum
            const int64_t mine = ((int64_t)start << 48) | tu;
            int64_t in = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, in, off);
                if (lane >= off) in += o;
            }
            if (lane == 31) red.sum[warp] = in;
            bar();
            int64_t total, before;
            if (T == 64) {
                before = warp ? red.sum[0] : 0;
                total = red.sum[0] + red.sum[1];
            } else {
                total = lane < T / 32 ? red.sum[lane] : 0, before = lane < warp ? total : 0;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) {
                    total += __shfl_xor_sync(0xffffffffu, total, off);
                    before += __shfl_xor_sync(0xffffffffu, before, off);
                }
            }
            before += in - mine;
            const int ti = tiles + (int)(before >> 48);
            if (start) {
                t.unit0 = units + (before & 0xffffffffffffll);
                tiles_out[ti] = t;
            }
            if (i < n) tile_of[(int64_t)st * n + i] = valid ? ti - (start ? 0 : 1) : -1;
            tiles += (int)(total >> 48);
            units += total & 0xffffffffffffll;
        }
    }
    if (D.streams == 1)
        for (int i = tid; i < n; i += T) tile_of[i] = -1;
    rmax = __reduce_max_sync(0xffffffffu, rmax);
    if (lane == 0) red.last[warp] = rmax;
    bar();
    for (int w = 0; w < T / 32; w++) rmax = max(rmax, red.last[w]);
    // CTA b takes the units [U b / grid, U (b + 1) / grid): at least one each
    const int grid = (int)min((int64_t)D.grid, units);
    if (tid == 0) head->units = units, head->grid = grid, head->rmax = rmax;
    const int64_t own = cta >= 0 && cta < grid ? unit_of(units, cta, grid, D) : -1;
#pragma unroll 1
    for (int i = tid; i < tiles; i += T) {
        const int64_t u0 = tiles_out[i].unit0, u1 = u0 + tile_units(tiles_out[i].nch, A, D);
        if (cta >= 0) {
            if (own >= u0 && own < u1) *first = i;
        } else if (u0 < u1) {
            for (int64_t b = (u0 * grid + units - 1) / units; b < grid && unit_of(units, (int)b, grid, D) < u1; b++)
                first[b] = i;
        }
    }
}

// One CTA plans for all.
__global__ void __launch_bounds__(kPlanThreads) al_plan_kernel(AlArgs A, AlDims D, AlWs W) {
    extern __shared__ int pl_smem[];  // [6][n_lanes]
    __shared__ PlanRed red;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    make_plan<kPlanThreads>(A, D, pl_smem, red, W.head, W.first, -1, W.tile_of, W.tiles, A.status);
}

// The plan as the other kernels see it: in the workspace, or in shared memory.
struct AlPlan {
    const AlPlanHead *head;
    const int *first;  // of this CTA
    const int *tile_of;
    const AlTile *tiles;
};

// ------------------------------------------------------------------ the pieces of a CTA
// A run of chunks of one tile for one KV head and head block, as one thread
// hands it to the others.
struct __align__(16) AlPiece {
    int n;                 // its chunks; 0: there are no more pieces
    int first, c1;         // they are first, first + 1, ... and from c1 on around
    int nsink, cfirst;     // the tile's chunks as rows (AlTile)
    int any_lo, any_hi, sk;  // rows that some row of the tile may see: > any_lo or < sk, and <= any_hi
    int all_lo, all_hi;      // rows that all of them see: > all_lo or < sk, and <= all_hi
    int stream, slot, kvh;
    int nrows, gs;         // rows, and rows per lane
    int lane0, head0;      // the first lane, and the first head
    int base, lim;         // AlTile
    int whole, begins;     // all of the tile's chunks; its first one

    __device__ __forceinline__ int row0(int i) const {
        int c = first + i;
        if (c >= c1) c -= n;
        return (c < nsink ? c : cfirst + c - nsink) * kChunk;
    }
    // whether some row of the tile may see one of the rows [a, b), and whether some may not
    __device__ __forceinline__ bool any_in(int a, int b) const { return a <= any_hi && (b - 1 > any_lo || a < sk); }
    __device__ __forceinline__ bool edge_in(int a, int b) const { return !(b - 1 <= all_hi && (a > all_lo || b - 1 < sk)); }
};

// Walks over a CTA's units and writes its pieces down.  Tiles of one sequence
// read the same chunks.  So that they read them at the same time, once from
// memory and then from L2, every CTA takes its chunks in the order of their
// number modulo the units of a CTA.
struct Walker {
    int64_t u, hi;
    int turn;  // units of a CTA
    const AlTile *at;
    __device__ __forceinline__ Walker(const AlPlan &P, const AlDims &D) {
        const int64_t U = P.head->units;
        const int G = P.head->grid;
        u = hi = 0;
        turn = 1;
        if ((int)blockIdx.x < G) {
            u = unit_of(U, (int)blockIdx.x, G, D);
            hi = (int)blockIdx.x + 1 == G ? U : unit_of(U, (int)blockIdx.x + 1, G, D);
            turn = (int)min(unit_of(U, 1, G, D) + 1, (int64_t)INT_MAX);
            at = P.tiles + *P.first;
        }
    }
    __device__ __forceinline__ void next(AlPiece &p, const AlArgs &A, const AlDims &D) {
        while (u < hi) {
            while (u >= at->unit0 + tile_units(at->nch, A, D)) at++;
            const int nch = at->nch, per = nch + D.setup;
            const int64_t r = u - at->unit0;
            const int64_t sub = r < per ? 0 : (r >> 31) ? r / per : (int64_t)((uint32_t)r / (uint32_t)per);
            const int v0 = (int)(r - sub * per), v1 = (int)min((int64_t)per, v0 + (hi - u));
            u += v1 - v0;
            if (v1 <= D.setup) continue;  // the next CTA starts it
            const int kvh = D.HB == 1 ? (int)sub : (int)(sub / D.HB), hb = (int)sub - kvh * D.HB;
            const int c0 = max(v0 - D.setup, 0), c1 = v1 - D.setup;
            const int over = c0 < turn ? c0 : c0 % turn;
            p.first = c0 + (over && turn - over < c1 - c0 ? turn - over : 0), p.c1 = c1;
            p.nsink = at->nsink, p.cfirst = at->cfirst;
            const int base = at->base, lim = at->lim, pmin = at->pmin - base, pmax = at->pmax - base;
            p.any_hi = min(pmax, lim - 1), p.all_hi = min(pmin, lim - 1);
            p.any_lo = A.window && pmin >= A.window ? pmin - A.window : -1;
            p.all_lo = A.window && pmax >= A.window ? pmax - A.window : -1;
            p.sk = A.window ? max(0, A.sinks - base) : 0;
            p.stream = at->stream, p.slot = at->slot, p.kvh = kvh;
            p.gs = D.HB == 1 ? D.group : min(D.R, D.group - hb * D.R);
            p.nrows = at->nl * p.gs;
            p.lane0 = at->lane0, p.head0 = kvh * D.group + hb * D.R;
            p.base = base, p.lim = lim;
            p.whole = c0 == 0 && c1 == nch, p.begins = c0 == 0;
            p.n = c1 - c0;
            return;
        }
        p.n = 0;
    }
};

// ------------------------------------------------------------------ instructions and barriers
constexpr int kAlSmem = 227 * 1024;  // all of an SM's: one CTA per SM
constexpr int kPieceRing = 2;

// Shared-memory matrix descriptors as two words, so that a step inside an
// operand is one 32-bit addition.  Low: address and leading byte offset (both
// in 16 bytes); high: stride byte offset, version 1, layout (2: 128-byte
// swizzle, 4: 64-byte).
__device__ __forceinline__ uint32_t al_desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | (lbo >> 4) << 16; }
__device__ __forceinline__ uint32_t al_desc_hi(uint32_t sbo, uint32_t layout) { return (sbo >> 4) | 1u << 14 | layout << 29; }
__device__ __forceinline__ void al_mma(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                       bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.u32 p, %6, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// One thread of the (converged) warp, chosen so that the compiler knows it is
// one: behind a test of the lane number it wraps every MMA, whose operands are
// uniform registers, in a loop over lanes (about 100 cycles each).
__device__ __forceinline__ bool al_elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void al_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// whether the phase is over by now
__device__ __forceinline__ bool al_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait that also ends when another role gave up.
__device__ __forceinline__ bool al_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool al_wait_at(uint32_t bar, uint32_t parity, int *abort) {
    if (al_try(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 0; i < (1u << 26); i++) {
        if (al_try(bar, parity)) return true;
        if ((i & 63u) == 63u && (*(volatile int *)abort || global_ns() - t0 > kWaitLimitNs)) return false;
    }
    return false;
}
__device__ __forceinline__ bool al_wait(uint64_t *bar, uint32_t parity, int *abort) {
    return al_wait_at(smem_addr(bar), parity, abort);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 lds128_a(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void sts64(uint32_t addr, uint2 v) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

// Every lane's values of 16 columns -> lane l the reduction of column l % 16 over the warp.
template <bool MAX>
__device__ __forceinline__ float al_reduce16(float (&v)[16], int lane) {
#pragma unroll
    for (int off = 8; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < off; i++) {
            const float send = (lane & off) ? v[i] : v[i + off], keep = (lane & off) ? v[i + off] : v[i];
            const float recv = __shfl_xor_sync(0xffffffffu, send, off);
            v[i] = MAX ? fmaxf(keep, recv) : __fadd_rn(keep, recv);
        }
    const float o = __shfl_xor_sync(0xffffffffu, v[0], 16);
    return MAX ? fmaxf(v[0], o) : __fadd_rn(v[0], o);
}

// barriers of one warpgroup
__device__ __forceinline__ void al_bar(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(wg + 1) : "memory"); }
__device__ __forceinline__ bool al_bar_or(int wg, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(wg + 1)
        : "memory");
    return r != 0;
}

// 32 bytes if on, else zeros: both loads are in flight before either is used
__device__ __forceinline__ void al_ld32(const float *p, bool on, uint4 &a, uint4 &b) {
    a = b = make_uint4(0, 0, 0, 0);
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %9, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%8];\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.u32 {%4,%5,%6,%7}, [%8+16];\n\t}"
        : "+r"(a.x), "+r"(a.y), "+r"(a.z), "+r"(a.w), "+r"(b.x), "+r"(b.y), "+r"(b.z), "+r"(b.w)
        : "l"(p), "r"((uint32_t)on));
}
__device__ __forceinline__ void al_ld16(const float *p, bool on, uint4 &a) {
    a = make_uint4(0, 0, 0, 0);
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "+r"(a.x), "+r"(a.y), "+r"(a.z), "+r"(a.w)
        : "l"(p), "r"((uint32_t)on));
}

// A place in the ring: slot and the parity of its round.
struct RingPos {
    int s = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void step(int slots) {
        if (++s == slots) s = 0, round++;
    }
};

// A reader's place in the ring of pieces.
struct PieceRef {
    int k = -1;
    template <typename Ctl>
    __device__ __forceinline__ const AlPiece *next(Ctl &S) {  // null: gave up
        k++;
        if (!al_wait(&S.pc_full[k % kPieceRing], (uint32_t)(k / kPieceRing) & 1u, &S.abort)) return nullptr;
        return &S.piece[k % kPieceRing];
    }
    template <typename Ctl>
    __device__ __forceinline__ void done(Ctl &S) {
        mbar_arrive(&S.pc_empty[k % kPieceRing]);
    }
};

// ------------------------------------------------------------------ merging partial tiles
constexpr int kMergeThreads = 256;

// The (lane, head)s in blocks of up to 256: first every thread finds out
// whether its own is finished already, then the block takes the others: the pieces of their tiles by the weights 2^(maximum - largest
// maximum), zeros where there are none.  All but the partial sums themselves
// is read while the kernel before still runs.
__global__ void __launch_bounds__(kMergeThreads) al_merge_kernel(AlArgs A, AlDims D, AlWs W) {
    __shared__ float w[2 * kMaxCtas];
    __shared__ float red[8];
    __shared__ float4 acc[kMergeThreads];
    __shared__ int todo[kMergeThreads];
    __shared__ int4 what[kMergeThreads][2];  // per stream: pieces, first CTA, row of its partial rows
    __shared__ int count;
    __shared__ AlSelfPlan plan;
    __shared__ AlSelfScratch x;
    const int tid = threadIdx.x, warp = tid >> 5, lane_t = tid & 31, hd = A.hd;
    const int total = A.n_lanes * A.n_heads;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    AlPlan P{W.head, nullptr, W.tile_of, W.tiles};
    if (A.n_lanes <= kSelfPlan) {
        if (tid < kSelfPlan)
            make_plan<kSelfPlan>(A, D, x.lane, x.red, &plan.head, &plan.first, kMaxCtas, x.tile_of, plan.tiles, nullptr);
        P = AlPlan{&plan.head, nullptr, x.tile_of, plan.tiles};
        __syncthreads();
    }
    const int64_t U = P.head->units, G = P.head->grid;
    // the partial row of piece q: the second slot of the CTA that starts the tile, the first of the ones behind it
    auto piece_row = [&](const int4 &a0, const int4 &a1, int q, int idx) -> int64_t {
        const int st = q < a0.x ? 0 : 1;
        const int4 x = st ? a1 : a0;
        const int b = st ? q - a0.x : q;
        return x.y < 0 ? (int64_t)2 * D.grid * D.cap + (int64_t)st * total + idx
                       : (int64_t)(2 * (x.y + b) + (b == 0 ? 1 : 0)) * D.cap + x.z;
    };
    bool waited = false;
    for (int base = blockIdx.x * D.merge; base < total; base += gridDim.x * D.merge) {
        __syncthreads();
        if (tid == 0) count = 0;
        __syncthreads();
        const int mine = base + tid;
        if (tid < D.merge && mine < total) {
            const int lane = mine / A.n_heads, h = mine - lane * A.n_heads;
            const int kvh = h / D.group, hg = h - kvh * D.group, hb = hg / D.R;
            bool done = false;
            int4 y[2];
#pragma unroll
            for (int st = 0; st < 2; st++) {
                y[st] = make_int4(0, 0, 0, 0);
                if (st < 2 - D.streams) continue;
                const int ti = P.tile_of[(int64_t)st * A.n_lanes + lane];
                if (ti < 0) continue;
                const AlTile *t = P.tiles + ti;
                const int nch = t->nch;
                if (nch == 0) continue;
                const int gs = D.HB == 1 ? D.group : min(D.R, D.group - hb * D.R);
                const int r = (lane - t->lane0) * gs + hg - hb * D.R;
                // from the unit of its first chunk
                const int64_t u1 = t->unit0 + (int64_t)(kvh * D.HB + hb + 1) * (nch + D.setup), u0 = u1 - nch;
                const int b0 = (int)(((u0 + 1) * G - 1) / U), b1 = (int)((u1 * G - 1) / U);
                if (b0 == b1)
                    done = D.streams == 1, y[st] = make_int4(1, -1, 0, 0);
                else
                    y[st] = make_int4(b1 - b0 + 1, b0, r, 0);
            }
            if (!done) {
                const int k = atomicAdd(&count, 1);
                todo[k] = mine;
                what[k][0] = y[0], what[k][1] = y[1];
            }
        }
        __syncthreads();
        if (!waited) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            waited = true;
        }
        // up to 32 pieces: a warp each, a lane per piece for the weights, then four dims each
        for (int k = warp; k < count; k += kMergeThreads / 32) {
            const int idx = todo[k];
            const int4 a0 = what[k][0], a1 = what[k][1];
            const int n = a0.x + a1.x;
            if (n > 32) continue;
            float4 *o = reinterpret_cast<float4 *>(A.out + (int64_t)idx * hd);
            int64_t row = 0;
            float m = kNoKey, l = 0.0f;
            if (lane_t < n) {
                row = piece_row(a0, a1, lane_t, idx);
                const float2 v = __ldcg(&W.ml[row]);
                m = v.x, l = v.y;
            }
            const float top = warp_max(m);
            const float x = m == kNoKey ? 0.0f : al_ex2(__fsub_rn(m, top));
            const float sum = warp_psum(lane_t < n ? x * l : 0.0f);
            const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
            float4 a[2] = {};
#pragma unroll 4
            for (int q = 0; q < n; q++) {
                const float xq = __shfl_sync(0xffffffffu, x, q);
                const float4 *src = reinterpret_cast<const float4 *>(W.part + __shfl_sync(0xffffffffu, row, q) * hd);
#pragma unroll
                for (int e = 0; e < 2; e++)
                    if (lane_t + 32 * e < hd / 4) {
                        const float4 v = __ldcg(src + lane_t + 32 * e);
                        a[e].x += v.x * xq, a[e].y += v.y * xq, a[e].z += v.z * xq, a[e].w += v.w * xq;
                    }
            }
#pragma unroll
            for (int e = 0; e < 2; e++)
                if (lane_t + 32 * e < hd / 4)
                    o[lane_t + 32 * e] = make_float4(a[e].x * inv, a[e].y * inv, a[e].z * inv, a[e].w * inv);
        }
        // more: the whole block
        for (int k = 0; k < count; k++) {
            const int idx = todo[k];
            const int4 a0 = what[k][0], a1 = what[k][1];
            const int n = a0.x + a1.x;
            if (n <= 32) continue;
            float4 *o = reinterpret_cast<float4 *>(A.out + (int64_t)idx * hd);
            __syncthreads();
            float m = kNoKey, l[2] = {0.0f, 0.0f}, mi[2];
#pragma unroll
            for (int e = 0; e < 2; e++)
                if (tid + e * kMergeThreads < n) {
                    const float2 v = __ldcg(&W.ml[piece_row(a0, a1, tid + e * kMergeThreads, idx)]);
                    mi[e] = v.x, l[e] = v.y;
                    m = fmaxf(m, v.x);
                }
            m = warp_max(m);
            if (lane_t == 0) red[warp] = m;
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; e++) m = fmaxf(m, red[e]);
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; e++)
                if (tid + e * kMergeThreads < n) {
                    const float x = mi[e] == kNoKey ? 0.0f : al_ex2(__fsub_rn(mi[e], m));
                    w[tid + e * kMergeThreads] = x;
                    sum += x * l[e];
                }
            sum = warp_psum(sum);
            __syncthreads();
            if (lane_t == 0) red[warp] = sum;
            __syncthreads();
            sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; e++) sum += red[e];
            // thread: four dims, every `groups`-th piece
            const int nv = hd / 4, groups = kMergeThreads / nv, gi = tid / nv, dv = tid - gi * nv;
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (gi < groups)
#pragma unroll 8
                for (int q = gi; q < n; q += groups) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(W.part + piece_row(a0, a1, q, idx) * hd) + dv);
                    const float x = w[q];
                    a.x += v.x * x, a.y += v.y * x, a.z += v.z * x, a.w += v.w * x;
                }
            acc[tid] = a;
            __syncthreads();
            if (tid < nv) {
                for (int e = 1; e < min(groups, n); e++) {
                    const float4 v = acc[e * nv + tid];
                    a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
                }
                const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
                o[tid] = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
            }
        }
    }
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ the workspace
constexpr int kFewRows = 16384;  // partial rows at least, for the kernels of little work

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

AlWs carve(int n_lanes, int n_heads, int n_kv, int hd, char *base, int64_t *n_rows = nullptr) {
    AlWs w{};
    size_t off = 0;
    auto take = [&](size_t b) {
        char *p = base ? base + off : nullptr;
        off += align256(b);
        return p;
    };
    const int64_t group = n_heads / n_kv;
    int64_t rows = (int64_t)2 * kMaxCtas * (n_lanes * group < 48 ? n_lanes * group : 48) + (int64_t)2 * n_lanes * n_heads;
    if (rows < kFewRows) rows = kFewRows;
    if (n_rows) *n_rows = rows;
    w.head = (AlPlanHead *)take(sizeof(AlPlanHead));
    w.first = (int *)take(sizeof(int) * kMaxCtas);
    w.tile_of = (int *)take(sizeof(int) * 2 * (size_t)n_lanes);
    w.tiles = (AlTile *)take(sizeof(AlTile) * 2 * (size_t)n_lanes);
    w.ml = (float2 *)take(sizeof(float2) * (size_t)rows);
    w.part = (float *)take(sizeof(float) * (size_t)rows * hd);
    w.bytes = off;
    return w;
}

}  // namespace
}  // namespace qlin
