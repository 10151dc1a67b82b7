// prefix_attn.cu -- attention of a batch of draft trees (or single tokens)
// over a paged cache whose sequences share a prefix, on the 5th-generation
// tensor cores (tcgen05 + tensor memory), bf16 or fp16, head sizes 64, 128, 256.
//
// The mathematics: softmax(scale q K^T) V over the union of the prefix's keys,
// the sequence's own keys and the node's ancestors-or-self.  A softmax over a
// union is joined from softmaxes over its parts by their maxima and sums, so
// the work is cut into units:
//   * prefix units: a tile of query rows of ALL sequences (rows of one KV head:
//     sequence, node, head of the group) against the prefix.  No row is masked
//     there, so rows of different sequences share a matrix product and the
//     prefix is read once per row tile instead of once per sequence;
//   * own units: the rows of one sequence against its own tokens and tree.
// A unit is a row of 64-key tiles.  All tiles of all units form one line that
// is cut into equal shares, one per CTA (persistent, one per SM), so the load
// is even whatever the lengths are (a unit starts with some places for its query
// load and result store); a share is a few segments (consecutive
// tiles of a unit), each segment leaves (max, sum, O) of its rows in the
// workspace, and a second kernel joins them.  The lengths are read on the
// device: nothing on the host depends on them.
//
// Inside a CTA (every wait bounded):
//   * the load warp: TMA boxes (64 elements x a page's rows, 128-byte swizzle)
//     from the pages of a tile into rings of K and V tiles;
//   * the fix warp: rows of V past the length become zero (0 x NaN is NaN), and
//     so do values of tree rows that are not finite: the softmax warps add those
//     to the rows that may see them when they store O;
//   * the MMA warps, one an accumulator: S = Q K^T into score buffers, O += P V
//     with P written over its scores.  Step i uses buffer i % kBufs and its
//     products are issued as PV(i) QK(i + kBufs), in one thread, so the scores need
//     no wait for the products that read the buffer before.  The tensor core's
//     queue is short (about four instructions), so what the issuing thread does
//     between two steps leaves it idle: one barrier stands for all that a step
//     needs (its weights, its V tile, the K tile of the scores it issues), and
//     with two accumulators the other warp's step fills the gap;
//   * softmax warps (one thread per query row): online softmax with a lazily
//     updated maximum (O is rescaled only when a row's maximum grows by more
//     than 2^8), P rounded to the 16-bit type, sums in fp32 of the unrounded P.
//     The rounding is what the product with V takes (its operands have one type,
//     and V is 16-bit); a second product with the remainder of P would double that
//     half of the matrix work.  Each weight is off by half a step of the type at
//     most, in either direction, so their weighted mean of the values, itself
//     rounded to the type, has 1.2 to 1.4 times the error of a result that is
//     rounded once.
// Head sizes 64 and 128 have room for two accumulators in tensor memory and
// run two softmax groups: on two halves of the rows with the same key tiles
// when a unit has more than 128 rows, else on the same rows with alternating
// key tiles.  Head size 256 has one accumulator; its two groups take half of
// each tile's keys and half of O's columns.
//
// What bounds it.  Many rows on a long prefix: the matrix products, which wait
// for the softmax between a tile's two and for their operands from shared memory
// (trees of 22 nodes, 16,384 shared tokens: 16 trees, 24/4 heads of 256, 106 us, 1.09
// PFLOP/s; 64 trees, 32/8 heads of 128, 283 us, 1.03; 103 and 250 us where the keys
// are in the L2).  Single tokens: the latency of a unit's start and end, some 8 K
// cycles a segment, of which half is hidden (64 sequences of 8,192 shared and 512 to
// 1,024 own tokens, 32/8 heads of 128: 69 us, this kernel 61 of them, 239 MB at 3.9
// TB/s).  A handful of sequences: plan, first tiles, one segment and the join, one
// after the other (16 us).  (Times without the host's, from a cold L2.)
#include <cuda.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace dflv {

namespace {

constexpr int kKT = 64;          // keys per tile
// Places on the line that a unit's query load and result store are worth, by
// rows of a unit (R = 128: head size 256, else 256).  Where the CTAs get fewer
// tiles than that each, a unit is better cut into segments than kept whole, and
// the set-up counts as much as a CTA's tiles.  Measured, in us, the keys in the L2:
//   head size 128, places                                   5    8   12   16
//     64 sequences of a token, 8,192 shared, 1,024 own     62   60   62   65
//     their own tokens alone                               55   55   56   56
//     64 trees of 22 nodes, 16,384 shared                 394  285  250  248
//   head size 256, places                                   4    8   12
//     16 trees of 22 nodes, 16,384 shared, 2,048 own      130  122  113
//     their shared tokens alone                           154  103  105
// (Head size 256 has 8: 12 gains 9 us on the one and loses 2 on the other.)
template <int R>
__host__ __device__ constexpr int most_setup() { return R == 128 ? 8 : 12; }
constexpr int kMaxB = 1024;
constexpr int kBlockBytes = kKT * 128;  // one 64-column block of a K or V tile

template <int D>
struct Cfg {
    static constexpr int kStreams = D == 256 ? 1 : 2;      // accumulators
    static constexpr int kRows = 128 * kStreams;           // query rows of a unit
    static constexpr int kBufs = 2 * kStreams;             // score buffers; step i uses buffer i % kBufs
    // Two softmax groups: with two accumulators step i is group i % 2's, with one
    // each group takes half of a step's keys.
    static constexpr int kSoftWarps = 8;
    static constexpr int kCols = kStreams == 2 ? kKT : kKT / 2;  // keys of a step that a thread takes
    // An MMA warp an accumulator, the load warp, the fix warp.
    static constexpr int kMmaWarp = kSoftWarps, kLoadWarp = kSoftWarps + kStreams, kFixWarp = kLoadWarp + 1;
    static constexpr int kWarps = kFixWarp + 1, kThreads = kWarps * 32;
    static constexpr bool kQSmem = D != 256;               // Q in shared or in tensor memory
    static constexpr int kQTile = 128 * D * 2;             // bytes of a stream's Q
    static constexpr int kTile = kKT * D * 2;              // bytes of a K or V tile
    static constexpr int kStages = D == 256 ? 6 : D == 128 ? 8 : 16;  // of the ring of K and V tiles
    // tensor-memory columns: O at 0, the score buffers behind 256, Q (D = 256)
    static constexpr uint32_t kOcol = 0, kScol = 256, kQcol = 384, kOstep = kStreams == 1 ? 0 : D;
    static constexpr int kOwnCols = kStreams == 1 ? D / 2 : D;       // columns of O that a group looks after
    static_assert(kScol + kBufs * kKT <= (kQSmem ? 512 : kQcol), "score buffers");
    static constexpr size_t kPlan = (size_t)4 * (kMaxB + 1) * 4;
    static constexpr size_t kHead = 6144;
    static constexpr size_t kOffPlan = kHead;
    static constexpr size_t kOffQ = (kOffPlan + kPlan + 1023) / 1024 * 1024;
    static constexpr size_t kOffRing = kOffQ + (kQSmem ? (size_t)kStreams * kQTile : 0);
    static constexpr size_t kSmem = kOffRing + (size_t)kStages * kTile + 1024;  // + alignment of the base
    static_assert(kSmem <= 227 * 1024, "fits in shared memory");
};

// ---------------------------------------------------------------- the plan
// What follows from the lengths, the same in every CTA.
struct Plan {
    int rows;        // query rows of a KV head over all sequences
    int prefix;      // prefix keys
    int p_tiles;     // key tiles of the prefix
    int p_units;     // row tiles of the prefix per KV head
    int p_rows;      // rows of such a tile
    int p_steps;     // places of a prefix unit on the line: its set-up, then its key tiles
    int own_steps;   // per KV head, over the sequences: the places of its units
    int own_units;   // per KV head: sum of row tiles
    int ctas;        // shares
    int setup;       // places of a unit before its tiles
    long long total; // places in all
};

// Workspace: the plan and the prefix sums for the joining kernel, then the
// segments' (max, sum) and O.
struct Layout {
    int G, max_rows;               // rows of a sequence
    int p_units, own_units;        // most units over all KV heads
    int ctas, half_p, half_own;    // rows between a segment's two groups
    int p_seg_rows, own_seg_rows;
    size_t off_ml, off_o, bytes;
    size_t own_row0;               // first row of the own segments
};

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

__host__ inline Layout make_layout(const PrefixAttnArgs& a, int ctas) {
    Layout l;
    const int R = a.D == 256 ? 128 : 256;
    l.G = a.Hq / a.Hkv;
    l.max_rows = a.N_max * l.G;
    l.p_units = a.Hkv * (int)(((long long)a.B * l.max_rows + R - 1) / R);
    l.own_units = a.Hkv * a.B * ceil_div(l.max_rows, R);
    l.ctas = ctas;
    const long long all = (long long)a.B * l.max_rows;
    l.half_p = all < 128 ? (int)all : 128;
    l.half_own = l.max_rows < 128 ? l.max_rows : 128;
    const int groups = R / 128;
    l.p_seg_rows = l.half_p * groups;
    l.own_seg_rows = l.half_own * groups;
    const size_t p_rows = (size_t)(l.p_units + ctas) * l.p_seg_rows;
    const size_t rows = p_rows + (size_t)(l.own_units + ctas) * l.own_seg_rows;
    l.own_row0 = p_rows;
    l.off_ml = (sizeof(Plan) + 3 * (kMaxB + 1) * 4 + 255) / 256 * 256;
    l.off_o = (l.off_ml + rows * 8 + 255) / 256 * 256;
    l.bytes = l.off_o + rows * a.D * 4;
    return l;
}

// The ring holds a segment's K and V tiles in the order in which the products
// take them: the scores run kBufs steps ahead, `ahead` tiles, so K0 ..
// K(ahead-1) V0 K(ahead) V1 K(ahead+1) .., and the V tiles that are left.  Every
// role walks it with a cursor of its own.
template <int N>
struct Cursor {
    int slot = 0;
    uint32_t phase = 0;
    DFLV_DEVINL void step() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1;
        }
    }
};
DFLV_DEVINL int k_place(int t, int ahead) { return t < ahead ? t : 2 * t - ahead + 1; }
DFLV_DEVINL int v_place(int t, int ahead, int nt) { return t <= nt - ahead ? 2 * t + ahead : nt + t; }

// Parities of the uses of the score buffers in all segments before this one, a
// bit a buffer; use k of a buffer within the segment completes phase
// (parity + k) of its barriers.
template <int N>
DFLV_DEVINL uint32_t add_uses(uint32_t parities, int steps) {
#pragma unroll
    for (int b = 0; b < N; ++b) parities ^= (uint32_t)((steps - b + N - 1) / N & 1) << b;
    return parities;
}

struct Segment {
    int h, rows, keys;        // KV head, query rows, keys of the unit
    int t0, nt;               // tiles [t0, t0 + nt)
    int steps;                // places on the line
    int per;                  // rows of the units of this kind (the last one may have fewer)
    int row0;                 // first row of the unit (in the prefix's row line, or the sequence's)
    int b;                    // sequence, -1: prefix
    long long unit;           // index among the units of its kind
};

// A unit with more than 128 rows works two steps off a tile: two places each.
// A tile belongs to the share that its first place is in.
template <int R>
DFLV_DEVINL int tile_places(int rows) { return R == 256 && rows > 128 ? 2 : 1; }
DFLV_DEVINL int first_tile(int place, int setup, int wt) { return place <= setup ? 0 : ceil_div(place - setup, wt); }

// a / b; 64-bit division takes a hundred instructions.
DFLV_DEVINL long long div_small(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// First index i in [0, n) with c[i + 1] > x (c ascending, c[n] > x).
DFLV_DEVINL int find_in(const int* c, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (c[mid + 1] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// The segment that starts at place w of a share ending at w_end, and the places
// it covers (`steps`; its tiles may be none).  cn, ct, cu: sums over the
// sequences of nodes, places and row tiles.
template <int R>
DFLV_DEVINL Segment segment_at(const PrefixAttnArgs& a, const Plan& p, const int* cn, const int* ct, const int* cu,
                               const int* cp, long long w, long long w_end) {
    Segment s;
    const int G = a.Hq / a.Hkv;
    const long long wp = (long long)a.Hkv * p.p_units * p.p_steps;
    int places, v;  // of the unit; the first one here
    if (w < wp) {
        s.unit = div_small(w, p.p_steps);
        v = (int)(w - s.unit * p.p_steps);
        places = p.p_steps;
        s.h = (int)div_small(s.unit, p.p_units);
        s.row0 = (int)(s.unit - (long long)s.h * p.p_units) * p.p_rows;
        s.per = p.p_rows;
        s.rows = min(s.per, p.rows - s.row0);
        s.keys = p.prefix;
        s.b = -1;
    } else {
        w -= wp;
        w_end -= wp;
        s.h = (int)div_small(w, p.own_steps);
        const int x = (int)(w - (long long)s.h * p.own_steps);
        s.b = find_in(ct, a.B, x);
        const int n = cn[s.b + 1] - cn[s.b], units = cu[s.b + 1] - cu[s.b];
        places = (ct[s.b + 1] - ct[s.b]) / units;
        const int y = x - ct[s.b], rt = y / places;
        v = y - rt * places;
        s.per = ceil_div(n * G, units);
        s.row0 = rt * s.per;
        s.rows = min(s.per, n * G - s.row0);
        s.keys = cp[s.b] + n;
        s.unit = (long long)s.h * p.own_units + cu[s.b] + rt;
    }
    s.steps = (int)min((long long)(places - v), w_end - w);
    const int wt = tile_places<R>(s.per);
    s.t0 = first_tile(v, p.setup, wt);
    s.nt = first_tile(v + s.steps, p.setup, wt) - s.t0;
    return s;
}

// All threads of the block.  A sequence whose lengths do not fit takes no part.
template <int R>
DFLV_DEVINL void make_plan(const PrefixAttnArgs& a, Plan* plan, int* cn, int* ct, int* cu, int* cp, int (*red)[4],
                           int ctas, bool report) {
    const int G = a.Hq / a.Hkv, B = a.B;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int prefix_len = __ldg(a.prefix_len);
    int carry[3] = {0, 0, 0};  // nodes, places, row tiles of the sequences before
    long long places = 0;
    for (int b0 = 0; b0 < B; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        int v[3] = {0, 0, 0};
        if (b < B) {
            int n = __ldg(a.n_nodes + b);
            const int past = __ldg(a.n_past + b);
            if (n < 0 || n > a.N_max) {
                if (report) raise_status(a.status, DFLV_DEV_TOPOLOGY);
                n = 0;
            } else if (past < 0 || (long long)past + n > (long long)a.max_pages * a.page) {
                if (report && n > 0) raise_status(a.status, DFLV_DEV_CAPACITY);
                n = 0;
            }
            const int u = n ? ceil_div(n * G, R) : 0;
            v[0] = n;
            v[1] = n ? u * ceil_div(past + n, kKT) * tile_places<R>(ceil_div(n * G, u)) : 0;
            v[2] = u;
            cp[b] = past;
        }
        // exclusive sums over the block
        int x[3] = {v[0], v[1], v[2]};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const int y = __shfl_up_sync(0xffffffffu, x[k], o);
                // (places stop at 2^31 - 1: the sum below then says so)
                if (lane >= o) x[k] = (int)min((unsigned)x[k] + (unsigned)y, 0x7fffffffu);
            }
        __syncthreads();
        if (lane == 31)
#pragma unroll
            for (int k = 0; k < 3; ++k) red[warp][k] = x[k];
        __syncthreads();
        int before[3] = {carry[0], carry[1], carry[2]};
        for (int w = 0; w < warps; ++w)
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const int y = red[w][k];
                if (w < warp) before[k] += y;
                carry[k] = (int)((unsigned)carry[k] + (unsigned)y);
                if (k == 1) places += y;
            }
        if (b < B) {
            cn[b] = before[0] + x[0] - v[0];
            ct[b] = before[1] + x[1] - v[1];
            cu[b] = before[2] + x[2] - v[2];
        }
    }
    if (threadIdx.x == 0) {
        cn[B] = carry[0];
        ct[B] = carry[1];
        cu[B] = carry[2];
        Plan p;
        p.prefix = prefix_len;
        if (p.prefix < 0 || p.prefix > a.max_prefix_pages * a.page) {
            if (report) raise_status(a.status, DFLV_DEV_CAPACITY);
            p.prefix = 0;
        }
        p.rows = carry[0] * G;
        p.p_tiles = ceil_div(p.prefix, kKT);
        p.p_units = ceil_div(p.rows, R);
        p.p_rows = p.p_units ? ceil_div(p.rows, p.p_units) : 0;
        const int p_places = p.p_tiles * tile_places<R>(p.p_rows);
        const long long tiles = (long long)a.Hkv * ((long long)p.p_units * p_places + carry[1]);
        p.setup = (int)max(1ll, min((long long)most_setup<R>(), div_small(tiles, ctas)));
        p.p_steps = p.p_tiles ? p.setup + p_places : 0;
        p.own_steps = carry[1] + p.setup * carry[2];
        p.own_units = carry[2];
        p.total = (long long)a.Hkv * ((long long)p.p_units * p.p_steps + p.own_steps);
        if (places + (long long)p.setup * carry[2] >= (1ll << 31)) {
            // more tokens than 32-bit sums of tiles hold (tables that name the
            // same pages again and again): nothing is computed
            if (report) raise_status(a.status, DFLV_DEV_CAPACITY);
            p.rows = p.p_units = 0;
            p.total = 0;
        }
        // (at least two places a share: one between two of a unit's segments
        // then holds the first place of a tile)
        p.ctas = (int)min((long long)ctas, p.total / 2);
        *plan = p;
    }
    __syncthreads();
    // ct: now with the units' set-up places
    const int setup = plan->setup;
    for (int b = threadIdx.x; b <= B; b += blockDim.x) ct[b] += setup * cu[b];
    __syncthreads();
}

// ---------------------------------------------------------------- helpers
// Descriptors of 128-byte-swizzled operands in 64-column blocks of kKT rows
// (8192 bytes): K-major (rows = N, the scores' K tile): 8-row groups 1024
// bytes apart; MN-major (rows = K, the values): the same groups along K, and
// the next 64 columns kBlockBytes on.
DFLV_DEVINL uint64_t desc_sw128(uint32_t addr, uint32_t lbo) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

template <bool kBf16>
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_mn) {
    return (1u << 4) | ((kBf16 ? 1u : 0u) << 7) | ((kBf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

DFLV_DEVINL void tma_box(void* dst, const CUtensorMap* map, int x, int row, int h, int page, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];\n" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(row), "r"(h), "r"(page), "r"(smem_u32(bar))
        : "memory");
}

// 2^x by the hardware's approximate base-2 exponential.
DFLV_DEVINL float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

template <bool kBf16>
DFLV_DEVINL uint32_t pack2(float lo, float hi) {
    return kBf16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}
// The type's largest exponent field: not finite.
template <bool kBf16>
DFLV_DEVINL bool not_finite(uint32_t b16) {
    return kBf16 ? (b16 & 0x7f80u) == 0x7f80u : (b16 & 0x7c00u) == 0x7c00u;
}
template <bool kBf16>
DFLV_DEVINL float to_f32(uint32_t b16) {
    return kBf16 ? __uint_as_float(b16 << 16) : __half2float(__ushort_as_half((unsigned short)b16));
}

// One thread of a converged warp, the same one every time: what follows stays
// in uniform registers, which tcgen05.mma takes its operands from.
DFLV_DEVINL bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// 16 consecutive columns of this thread's tensor-memory lane, without the wait.
DFLV_DEVINL void st16_nowait(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// In the place of a row's sum where the segment reaches a malformed tree, as the
// last one of every row of that sequence does: the join writes nothing for it.
constexpr float kMalformed = -1.0f;

constexpr int kMaxStages = 16;
constexpr int kMaxBufs = 4;
constexpr int kBadSlots = 16;  // segments the fix warp can be ahead of the softmax: fewer than half the stages + 1

struct Head {
    uint64_t full[kMaxStages], ready[kMaxStages], freed[kMaxStages];  // ready: values looked over by the fix warp
    // go: a step's weights are written (an arrival a softmax warp) and its tiles
    // are there (one of the fix warp)
    uint64_t s_full[kMaxBufs], go[kMaxBufs], pv_done[kMaxBufs], m_ready[4], o_fin, q_ready, l_ready, drain;
    unsigned long long bad[kBadSlots];  // tree nodes with values that are not finite, per segment
    uint32_t tmem;
    int fail;
    int red[32][4];
    int par[8][64];  // per softmax warp: the tree of its segment's sequence
    float m[2][2][128], l[128];  // head size 256: a step's maxima by group; the second group's sums
    Plan plan;
};
static_assert(sizeof(Head) <= 6144, "header");

// One arrival for a warp whose lanes are all done (128 single arrivals at a
// barrier take hundreds of cycles).
DFLV_DEVINL void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Bounded wait of a whole warp, with one answer for all of its lanes; gives up
// early once another role has.
__device__ __noinline__ bool wait_bar_slow(Head* hd, uint64_t* bar, uint32_t parity, int32_t* status) {
    bool done = false;
    for (uint32_t it = 0; it < kWaitLimit && !done; ++it) {
        done = mbar_try_wait(bar, parity);
        if (!done && (it & 255) == 255 && *(volatile int*)&hd->fail) break;
    }
    if (__all_sync(0xffffffffu, done)) return true;
    if (*(volatile int*)&hd->fail == 0) {
        *(volatile int*)&hd->fail = 1;
        raise_status(status, DFLV_DEV_TIMEOUT);
    }
    return false;
}
DFLV_DEVINL bool wait_bar(Head* hd, uint64_t* bar, uint32_t parity, int32_t* status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_bar_slow(hd, bar, parity, status);
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    prefix_attn_kernel(const PrefixAttnArgs a, const Layout lay, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map) {
    using C = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Head* hd = reinterpret_cast<Head*>(smem);
    int* cn = reinterpret_cast<int*>(smem + C::kOffPlan);
    int *ct = cn + kMaxB + 1, *cu = ct + kMaxB + 1;
    int* cp = cu + kMaxB + 1;  // own committed tokens
    unsigned char* ring = smem + C::kOffRing;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&hd->full[s], 1);
            mbar_init(&hd->ready[s], 1);
            mbar_init(&hd->freed[s], C::kStreams);
        }
        for (int s = 0; s < C::kBufs; ++s) {
            mbar_init(&hd->s_full[s], 1);
            mbar_init(&hd->go[s], (C::kStreams == 2 ? 4 : 8) + 1);
            mbar_init(&hd->pv_done[s], 1);
        }
        mbar_init(&hd->o_fin, C::kStreams);
        mbar_init(&hd->drain, C::kStreams);
        mbar_init(&hd->q_ready, 8);
        mbar_init(&hd->l_ready, 4);
        for (int s = 0; s < 4; ++s) mbar_init(&hd->m_ready[s], 2);
        hd->fail = 0;
        for (int s = 0; s < kBadSlots; ++s) hd->bad[s] = 0;
        fence_mbar_init();
    }
    if (warp == C::kMmaWarp) tc::alloc(&hd->tmem, 512);
    if (warp == C::kLoadWarp && lane < 2) {
        const CUtensorMap* m = lane ? &v_map : &k_map;
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(m) : "memory");
    }
    grid_dependency_wait();
    make_plan<C::kRows>(a, &hd->plan, cn, ct, cu, cp, hd->red, lay.ctas, blockIdx.x == 0);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const Plan plan = hd->plan;
    const uint32_t tmem = hd->tmem;
    if (blockIdx.x == 0) {  // for the joining kernel
        int* out = reinterpret_cast<int*>(static_cast<unsigned char*>(a.ws) + sizeof(Plan));
        for (int i = tid; i <= a.B; i += C::kThreads) {
            out[i] = cn[i];
            out[kMaxB + 1 + i] = ct[i];
            out[2 * (kMaxB + 1) + i] = cu[i];
        }
        if (tid == 0) *reinterpret_cast<Plan*>(a.ws) = plan;
    }
    const bool busy = (int)blockIdx.x < plan.ctas;
    const long long w0 = busy ? div_small(plan.total * blockIdx.x, plan.ctas) : 0;
    const long long w1 = busy ? div_small(plan.total * (blockIdx.x + 1), plan.ctas) : 0;
    const int G = a.Hq / a.Hkv;
    int32_t* const status = a.status;
    bool ok = true;

    if (warp == C::kLoadWarp) {
        // ------------------------------------------------ loads
        Cursor<C::kStages> at;
        uint32_t loaded = 0;
        const int box_rows = min(a.page, kKT), per_tile = kKT / box_rows;
        const int mine = lane % per_tile, blk = lane / per_tile;   // this lane's box: page of the tile, 64-column block
        const bool has_box = blk < D / 64;
        unsigned char* const box = ring + (size_t)blk * kBlockBytes + (size_t)mine * box_rows * 128;
        for (long long w = w0; w < w1 && ok;) {
            const Segment s = segment_at<C::kRows>(a, plan, cn, ct, cu, cp, w, w1);
            w += s.steps;
            if (s.nt == 0) continue;
            const bool two = C::kStreams == 2 && s.per > 128;
            const int32_t* table = s.b < 0 ? a.prefix_table : a.table + (size_t)s.b * a.max_pages;
            const int n_pages = (s.keys + a.page - 1) >> a.page_shift;  // pages in use
            // the page of this lane's box in tile t (its pages that hold no key
            // are not loaded)
            auto page_of = [&](int t) {
                const int p = ((s.t0 + t) * kKT >> a.page_shift) + mine;
                if (t >= s.nt || p >= n_pages) return -1;
                const int id = __ldg(table + p);
                if ((unsigned)id < (unsigned)a.n_pages) return id;
                raise_status(status, DFLV_DEV_PAGE);
                return 0;
            };
            auto load = [&](const CUtensorMap* map, int t, int page) {
                ok = ok && wait_bar(hd, &hd->freed[at.slot], at.phase ^ 1, status);
                if (!ok) return;
                uint64_t* full = &hd->full[at.slot];
                const int p0 = (s.t0 + t) * kKT >> a.page_shift;
                if (lane == 0)
                    mbar_arrive_expect_tx(full, (uint32_t)(min(per_tile, n_pages - p0) * box_rows * D * 2));
                __syncwarp();
                if (has_box && page >= 0)
                    tma_box(box + (size_t)at.slot * C::kTile, map, blk * 64,
                            a.page > kKT ? ((s.t0 + t) * kKT) & (a.page - 1) : 0, s.h, page, full);
                at.step();
                ++loaded;
            };
            const int ahead = C::kBufs >> two;
            for (int t = 0; t < ahead && t < s.nt; ++t) load(&k_map, t, page_of(t));
            for (int t = 0; t < s.nt && ok; ++t) {
                const int k_page = page_of(t + ahead);  // (its latency passes under the wait for V's place)
                load(&v_map, t, page_of(t));
                if (t + ahead < s.nt) load(&k_map, t + ahead, k_page);
            }
        }
        // no box is in flight when the CTA leaves, even after a failure
        for (uint32_t e = loaded < (uint32_t)C::kStages ? 0 : loaded - C::kStages; e < loaded; ++e)
            for (uint32_t it = 0; it < kWaitLimit; ++it)
                if (mbar_try_wait(&hd->full[e % C::kStages], (e / C::kStages) & 1)) break;
    } else if (warp == C::kFixWarp) {
        // ------------------------------------------------ V rows no one may see
        Cursor<C::kStages> at;
        uint32_t n_seg = 0, uses = 0;
        for (long long w = w0; w < w1 && ok;) {
            const Segment s = segment_at<C::kRows>(a, plan, cn, ct, cu, cp, w, w1);
            w += s.steps;
            if (s.nt == 0) continue;
            const bool two = C::kStreams == 2 && s.per > 128;
            const int n = s.b < 0 ? 0 : cn[s.b + 1] - cn[s.b];
            const int past = s.keys - n;
            unsigned long long* bad_nodes = &hd->bad[n_seg++ % kBadSlots];
            if (lane == 0) *bad_nodes = 0;
            __syncwarp();
            auto pass = [&] {
                if (lane == 0) mbar_arrive(&hd->ready[at.slot]);
                at.step();
            };
            const int ahead = C::kBufs >> two, steps = s.nt << two;
            // The next tile of the ring is there.
            auto arrived = [&] {
                ok = ok && wait_bar(hd, &hd->full[at.slot], at.phase, status);
                return ok;
            };
            for (int t = 0; t < ahead && t < s.nt; ++t) {  // the first K tiles
                if (!arrived()) break;
                if (lane == 0) mbar_arrive(&hd->ready[at.slot]);
                at.step();
            }
            for (int t = 0; t < s.nt && ok; ++t) {
                if (!arrived()) break;
                const int j0 = (s.t0 + t) * kKT;
                unsigned char* tile = ring + (size_t)at.slot * C::kTile;
                bool wrote = false;
                // a row is 8 pieces of 16 bytes in each of D / 64 blocks (the
                // swizzle permutes pieces inside a row)
                if (j0 + kKT > s.keys) {
                    const int r0 = s.keys - j0;
                    for (int q = lane; q < (kKT - r0) * (D / 8); q += 32) {
                        const int r = r0 + q / (D / 8), c = q % (D / 8);
                        *reinterpret_cast<uint4*>(tile + (c >> 3) * kBlockBytes + r * 128 + (c & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    wrote = true;
                }
                if (n > 1 && j0 + kKT > past) {
                    const int r0 = max(0, past - j0), r1 = min(kKT, s.keys - j0);
                    for (int q = lane; q < (r1 - r0) * (D / 8); q += 32) {
                        const int r = r0 + q / (D / 8), c = q % (D / 8);
                        uint32_t* at = reinterpret_cast<uint32_t*>(tile + (c >> 3) * kBlockBytes + r * 128 + (c & 7) * 16);
                        bool bad = false;
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            uint32_t x = at[y];
                            const bool lo = not_finite<kBf16>(x & 0xffffu), hi = not_finite<kBf16>(x >> 16);
                            if (lo || hi) {
                                if (lo) x &= 0xffff0000u;
                                if (hi) x &= 0x0000ffffu;
                                at[y] = x;
                                bad = true;
                            }
                        }
                        if (bad) atomicOr(bad_nodes, 1ull << (j0 + r - past));
                    }
                    wrote = true;
                }
                if (wrote) fence_proxy_async_smem();
                __syncwarp();
                at.step();
                if (t + ahead < s.nt) {  // the K tile that goes with it
                    if (!arrived()) break;
                    at.step();
                }
                for (int i = t << two; i < (t + 1) << two && ok; ++i) {
                    // (the buffer's last use has gone, or the arrival would count for it)
                    const int buf = i & (C::kBufs - 1);
                    if (i >= C::kBufs)
                        ok = wait_bar(hd, &hd->go[buf], ((uses >> buf) + i / C::kBufs - 1) & 1, status);
                    if (ok && lane == 0) mbar_arrive(&hd->go[buf]);
                }
            }
            // (nor has the next segment's first arrival anything to wait for:
            // it comes after this segment's last step)
            for (int b = 0; b < C::kBufs && ok; ++b) {
                const int n_uses = (steps - b + C::kBufs - 1) / C::kBufs;
                if (n_uses > 0) ok = wait_bar(hd, &hd->go[b], ((uses >> b) + n_uses - 1) & 1, status);
            }
            uses = add_uses<C::kBufs>(uses, steps);
        }
    } else if (warp >= C::kMmaWarp && warp < C::kMmaWarp + C::kStreams) {
        // ------------------------------------------------ matrix products
        constexpr uint32_t id_qk = idesc<kBf16>(128, kKT, false), id_pv = idesc<kBf16>(128, D, true);
        const int stream = warp - C::kMmaWarp;
        // operands the same in every lane, so that they stay in uniform registers
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t ring_at = __shfl_sync(0xffffffffu, smem_u32(ring), 0);
        const uint64_t k_desc = desc_sw128(ring_at, 16), v_desc = desc_sw128(ring_at, kBlockBytes);
        const uint64_t q_desc =
            desc_sw128(__shfl_sync(0xffffffffu, smem_u32(smem + C::kOffQ), 0) + stream * C::kQTile, 16);
        const uint32_t o_tm = tm + C::kOcol + stream * C::kOstep;
        int base = 0;                   // first place of the segment in the ring
        uint32_t uses = 0, q_ph = 0, ready_ph = 0;
        for (long long w = w0; w < w1 && ok;) {
            const Segment s = segment_at<C::kRows>(a, plan, cn, ct, cu, cp, w, w1);
            w += s.steps;
            if (s.nt == 0) continue;
            const bool two = C::kStreams == 2 && s.per > 128;  // two row halves on each tile
            const int steps = s.nt << two, ahead = C::kBufs >> two;
            auto slot_of = [&](int place) { return (base + place) % C::kStages; };
            // A tile is freed by both streams, or twice by its only one. (One thread.)
            auto free_tile = [&](int slot) {
                tc::commit(&hd->freed[slot]);
                if (C::kStreams == 2 && !two) tc::commit(&hd->freed[slot]);
            };
            auto qk = [&](int buf, int slot) {
                const uint64_t kb = k_desc + (uint32_t)(slot * (C::kTile >> 4));
                const uint32_t d = tm + C::kScol + buf * kKT;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t b = kb + ((kk >> 2) * kBlockBytes + (kk & 3) * 32) / 16;
                    if (C::kQSmem) tc::mma_f16(d, q_desc + ((kk >> 2) * 128 * 128 + (kk & 3) * 32) / 16, b, id_qk, kk > 0);
                    else tc::mma_f16_ts(d, tm + C::kQcol + kk * 8, b, id_qk, kk > 0);
                }
                tc::commit(&hd->s_full[buf]);
                free_tile(slot);
            };
            ok = wait_bar(hd, &hd->q_ready, q_ph, status);
            q_ph ^= 1;
            // the first K tiles: their barriers complete a phase a segment that
            // uses the slot for one of them
            for (int t = 0; t < ahead && t < s.nt && ok; ++t) {
                const int slot = slot_of(t);
                if (two || (t & (C::kStreams - 1)) == stream) {
                    ok = wait_bar(hd, &hd->ready[slot], (ready_ph >> slot) & 1, status);
                    const int buf = two ? 2 * t + stream : t;
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (elect_one()) qk(buf, slot);
                    __syncwarp();
                }
                ready_ph ^= 1u << slot;
            }
            for (int i = stream; i < steps && ok; i += C::kStreams) {
                // Step i: its products with V, then the scores of step i + kBufs.
                const int buf = i & (C::kBufs - 1), t = i >> two;
                const bool more = i + C::kBufs < steps;
                const int v_slot = slot_of(v_place(t, ahead, s.nt)), k_slot = slot_of(k_place(t + ahead, ahead));
                const uint64_t vb = v_desc + (uint32_t)(v_slot * (C::kTile >> 4));
                const uint32_t p = tm + C::kScol + buf * kKT;
                ok = wait_bar(hd, &hd->go[buf], ((uses >> buf) + i / C::kBufs) & 1, status);
                if (!ok) break;
                tc::fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kKT / 16; ++kk)
                        tc::mma_f16_ts(o_tm, p + kk * 8, vb + kk * 2048 / 16, id_pv, kk > 0 || i >= C::kStreams);
                    tc::commit(&hd->pv_done[buf]);
                    free_tile(v_slot);
                    if (more) qk(buf, k_slot);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (elect_one()) tc::commit(&hd->o_fin);
            __syncwarp();
            uses = add_uses<C::kBufs>(uses, steps);
            base = (base + 2 * s.nt) % C::kStages;
        }
        // no product is in flight when tensor memory is given back
        if (elect_one()) tc::commit(&hd->drain);
        for (uint32_t it = 0; it < kWaitLimit; ++it)
            if (mbar_try_wait(&hd->drain, 0)) break;
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax
        const int grp = warp >> 2, row = tid & 127;
        const uint32_t lane_base = (uint32_t)(warp & 3) * 32u << 16;
        // (a scale of zero still has to mask, as -infinity x 0 is NaN: with the
        // smallest float no finite score comes to more than 2^-21)
        const float c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 0x1p-149f);
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;  // q negated for a negative scale
        // fp16 weights are scaled by 2^6 (they stay below 2^14): fewer of them
        // are subnormal.  Sums and O carry the factor alike.
        const float bias = kBf16 ? 0.0f : 6.0f;
        uint32_t uses = 0, fin_ph = 0, n_seg = 0, steps_before = 0;
        const uint32_t o_tm = tmem + lane_base + C::kOcol + grp * C::kOwnCols;  // this group's columns of O
        long long w = w0;
        // The next segment of the share that has tiles (nt = 0: none).
        auto next_segment = [&] {
            Segment s = {};
            while (w < w1 && s.nt == 0) {
                s = segment_at<C::kRows>(a, plan, cn, ct, cu, cp, w, w1);
                w += s.steps;
            }
            return s;
        };
        // The row's query of a segment goes to where the products take it from;
        // returns its node.
        auto load_query = [&](const Segment& s) {
            const bool two = C::kStreams == 2 && s.per > 128;
            const int half = two ? (s.rows + 1) >> 1 : 0;
            const int my_rows = two ? (grp ? s.rows - half : half) : s.rows;
            const bool has_row = row < my_rows, any_row = (row & ~31) < my_rows;
            const int r = s.row0 + grp * half + row;
            int node = 0;
            size_t at = 0;
            if (has_row) {
                int b = s.b, ln = r / G;
                const int g = r - ln * G;
                if (b < 0) {
                    b = find_in(cn, a.B, ln);
                    ln -= cn[b];
                }
                node = ln;
                at = ((size_t)b * a.N_max + ln) * a.q_stride + (size_t)(s.h * G + g) * D;
            }
            const uint4* src = reinterpret_cast<const uint4*>(a.q + at);
            if constexpr (C::kQSmem) {
                // rows of 64 columns in 128-byte lines, pieces of 16 bytes
                // swizzled as the descriptors have it
                if (any_row) {
                    uint4 y[D / 8];  // all loads in flight
#pragma unroll
                    for (int e = 0; e < D / 8; ++e) y[e] = has_row ? __ldg(src + e) : make_uint4(0, 0, 0, 0);
                    unsigned char* q_row = smem + C::kOffQ + grp * C::kQTile + row * 128;
#pragma unroll
                    for (int e = 0; e < D / 8; ++e)
                        *reinterpret_cast<uint4*>(q_row + (e >> 3) * 128 * 128 + ((e & 7) ^ (row & 7)) * 16) =
                            make_uint4(y[e].x ^ flip, y[e].y ^ flip, y[e].z ^ flip, y[e].w ^ flip);
                }
                fence_proxy_async_smem();
            } else {
                // each group half of the row, into tensor memory
                if (any_row) {
                    uint4 y[D / 16];
#pragma unroll
                    for (int e = 0; e < D / 16; ++e) y[e] = has_row ? __ldg(src + grp * (D / 16) + e) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int q0 = 0; q0 < D / 4; q0 += 32) {
                        uint32_t x[32];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            x[4 * e] = y[q0 / 4 + e].x ^ flip;
                            x[4 * e + 1] = y[q0 / 4 + e].y ^ flip;
                            x[4 * e + 2] = y[q0 / 4 + e].z ^ flip;
                            x[4 * e + 3] = y[q0 / 4 + e].w ^ flip;
                        }
                        tc::st32u(tmem + lane_base + C::kQcol + grp * (D / 4) + q0, x);
                    }
                }
                tc::fence_before_sync();
            }
            warp_arrive(&hd->q_ready);
            return node;
        };
        Segment upcoming = next_segment();
        int upcoming_node = upcoming.nt > 0 ? load_query(upcoming) : 0;
        while (upcoming.nt > 0 && ok) {
            const Segment s = upcoming;
            const int node = upcoming_node;
            const bool two = C::kStreams == 2 && s.per > 128;
            const int steps = s.nt << two;
            const int half = two ? (s.rows + 1) >> 1 : 0;             // rows of the first group
            const int my_rows = two ? (grp ? s.rows - half : half) : s.rows;
            const bool live = row < my_rows;
            const bool warp_live = (row & ~31) < my_rows;
            const int n = s.b < 0 ? 0 : cn[s.b + 1] - cn[s.b];
            const int past = s.keys - n;
            const unsigned long long* bad_nodes = &hd->bad[n_seg++ % kBadSlots];
            // ---- the row's ancestors, when the segment reaches the tree
            unsigned long long anc = 0;
            bool malformed = false;
            if (n > 0 && (s.t0 + s.nt) * kKT > past) {
                int* par = hd->par[warp];  // a copy per warp: no barrier between warps
                __syncwarp();
                for (int x = lane; x < n; x += 32) {
                    int p = x - 1;
                    if (a.parent) {
                        const int q = __ldg(a.parent + (size_t)s.b * a.N_max + x);
                        if (x == 0 ? q != -1 : (q < 0 || q >= x)) malformed = true;
                        else p = q;
                    }
                    par[x] = p;
                }
                malformed = __any_sync(0xffffffffu, malformed);
                if (malformed && lane == 0) raise_status(status, DFLV_DEV_TOPOLOGY);
                __syncwarp();
                if (live)
                    for (int x = node; x >= 0; x = par[x]) anc |= 1ull << x;
            }
            // ---- the tiles
            float m = -INFINITY, l = 0.0f;
            constexpr int kCols = C::kCols;
            const int e0 = C::kStreams == 2 ? 0 : grp * kCols;   // this thread's first key of a tile
            for (int i = C::kStreams == 2 ? grp : 0; i < steps; i += C::kStreams) {
                const int buf = i & (C::kBufs - 1), j0 = (s.t0 + (i >> two)) * kKT + e0;
                ok = wait_bar(hd, &hd->s_full[buf], ((uses >> buf) + i / C::kBufs) & 1, status);
                if (!ok) break;
                tc::fence_after_sync();
                if (warp_live) {
                    const uint32_t s_tm = tmem + lane_base + C::kScol + buf * kKT;
                    uint32_t x[kCols];
#pragma unroll
                    for (int e = 0; e < kCols; e += 32) tc::ld32_nowait(s_tm + e0 + e, *reinterpret_cast<uint32_t(*)[32]>(x + e));
                    unsigned long long vis = ~0ull;
                    if (s.b < 0) {
                        const int left = s.keys - j0;
                        if (left < kCols) vis = left > 0 ? (1ull << left) - 1 : 0ull;
                    } else if (j0 + kCols > past) {
                        const int d = past - j0;  // < 64
                        vis = d >= 0 ? ((1ull << d) - 1) | (anc << d) : (-d < 64 ? anc >> -d : 0ull);
                    }
                    tc::wait_ld();
                    if (__any_sync(0xffffffffu, vis != ~0ull)) {
                        const uint32_t v[2] = {(uint32_t)vis, (uint32_t)(vis >> 32)};
#pragma unroll
                        for (int e = 0; e < kCols; ++e)
                            if (!((v[e >> 5] >> (e & 31)) & 1)) x[e] = 0xff800000u;
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < kCols; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(x[e]));
                    float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (C::kStreams == 1) {
                        // the row's other half is in the other group's thread.
                        // (Past this point both have read their scores, which
                        // the weights overwrite.)
                        hd->m[i & 1][grp][row] = top;
                        warp_arrive(&hd->m_ready[warp & 3]);
                        ok = wait_bar(hd, &hd->m_ready[warp & 3], (steps_before + i) & 1, status);
                        top = fmaxf(top, hd->m[i & 1][grp ^ 1][row]);
                    }
                    const bool raise = top > m && (m == -INFINITY || (top - m) * c > 8.0f);
                    if (i < C::kStreams) {
                        m = top;
                    } else if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? (m == -INFINITY ? 0.0f : ex2((m - top) * c)) : 1.0f;
                        if (raise) m = top;
                        l *= f;
                        // the last products that add to O have to be through
                        const int ip = i - C::kStreams, pb = ip & (C::kBufs - 1);
                        ok = wait_bar(hd, &hd->pv_done[pb], ((uses >> pb) + ip / C::kBufs) & 1, status);
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int q0 = 0; q0 < C::kOwnCols; q0 += 16) {
                            uint32_t o[16];
                            tc::ld16_nowait(o_tm + q0, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc::st16u(o_tm + q0, o);
                        }
                    }
                    const float mc = m == -INFINITY ? 0.0f : m * c - bias;
                    const uint64_t c2 = pair(c, c), mc2 = pair(-mc, -mc);
                    uint64_t sum2[2] = {0, 0};
#pragma unroll
                    for (int hf = 0; hf < kCols / 32; ++hf) {
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const uint64_t t = fma2(pair(x[hf * 32 + e], x[hf * 32 + e + 1]), c2, mc2);
                            float t0, t1;
                            unpair(t, t0, t1);
                            t0 = ex2(t0);
                            t1 = ex2(t1);
                            sum2[(e >> 1) & 1] = add2(sum2[(e >> 1) & 1], pair(t0, t1));
                            p[e >> 1] = pack2<kBf16>(t0, t1);
                        }
                        st16_nowait(s_tm + e0 / 2 + hf * 16, p);
                    }
                    float s0, s1;
                    unpair(add2(sum2[0], sum2[1]), s0, s1);
                    l += s0 + s1;
                    asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
                }
                tc::fence_before_sync();
                warp_arrive(&hd->go[buf]);
            }
            if (!ok) break;
            // All scores of the segment are there, so its query has been read: the
            // next segment's takes its place while the last products run, and its
            // first scores are computed while O is stored.  (Its products with V
            // wait for weights, which each warp writes after it has read O.)  Not so
            // where the group has no step in this segment or in the next one: in
            // this one, its arrival could count for this segment's query, which the
            // other group may still be loading; in the next one, its products could
            // be done with that one, and say so, before the other's are with this.
            upcoming = next_segment();
            const int next_steps = upcoming.nt << (C::kStreams == 2 && upcoming.per > 128);
            const bool early = C::kStreams == 1 || (grp < steps && grp < next_steps);
            if (early && upcoming.nt > 0) upcoming_node = load_query(upcoming);
            // ---- (max, sum, O) of the segment
            ok = wait_bar(hd, &hd->o_fin, fin_ph, status);
            fin_ph ^= 1;
            if (!ok) break;
            if (!early && upcoming.nt > 0) upcoming_node = load_query(upcoming);
            tc::fence_after_sync();
            // With one accumulator the groups' sums are joined here, and each
            // group stores half of the columns.
            constexpr bool kOne = C::kStreams == 1;
            if (kOne) {
                if (warp_live) steps_before += steps;  // (idle warps exchange nothing)
                if (grp == 1) {
                    hd->l[row] = l;
                    warp_arrive(&hd->l_ready);
                } else {
                    ok = wait_bar(hd, &hd->l_ready, fin_ph ^ 1, status);
                    if (!ok) break;
                    l += hd->l[row];
                }
            }
            uses = add_uses<C::kBufs>(uses, steps);
            if (warp_live) {
                const int which = kOne ? 0 : grp;
                const size_t seg0 = s.b < 0 ? (size_t)(s.unit + blockIdx.x) * lay.p_seg_rows
                                            : lay.own_row0 + (size_t)(s.unit + blockIdx.x) * lay.own_seg_rows;
                const int seg_rows = s.b < 0 ? lay.p_seg_rows : lay.own_seg_rows;
                const int in_seg = which * (s.b < 0 ? lay.half_p : lay.half_own) + row;
                // O as [D][rows of the segment]: a warp's store of a column is
                // one line
                float2* ml = reinterpret_cast<float2*>(static_cast<unsigned char*>(a.ws) + lay.off_ml) + seg0 + in_seg;
                float* po = reinterpret_cast<float*>(static_cast<unsigned char*>(a.ws) + lay.off_o) + seg0 * D + in_seg;
                if (live && (!kOne || grp == 0)) *ml = make_float2(m * c, malformed ? kMalformed : l);
                const unsigned long long bad = s.b < 0 ? 0ull : *bad_nodes & anc;
                const int d0 = kOne ? grp * C::kOwnCols : 0;
                if (kOne || grp < steps) {  // (a group without a tile has no O)
                    float* to = po + (size_t)d0 * seg_rows;
#pragma unroll
                    for (int q0 = 0; q0 < C::kOwnCols; q0 += 32) {
                        uint32_t o[32];
                        tc::ld32_nowait(o_tm + q0, o);
                        tc::wait_ld();
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 32; ++e, to += seg_rows) *to = __uint_as_float(o[e]);
                        }
                    }
                }
                for (unsigned long long left = live ? bad : 0ull; left; left &= left - 1) {
                    // a visible node's values that are not finite: the fix warp
                    // left them out of the product (only a tile of this group's)
                    const int j = past + ffs64(left), t = j / kKT - s.t0;
                    if (t < 0 || t >= s.nt || (!kOne && !two && (t & 1) != grp)) continue;
                    int id = __ldg(a.table + (size_t)s.b * a.max_pages + (j >> a.page_shift));
                    if ((unsigned)id >= (unsigned)a.n_pages) id = 0;
                    const uint16_t* v = static_cast<const uint16_t*>(a.vp) +
                                        ((((size_t)id * a.Hkv + s.h) << a.page_shift) + (j & (a.page - 1))) * D;
#pragma unroll 1
                    for (int e = d0; e < d0 + C::kOwnCols; ++e)
                        if (not_finite<kBf16>(v[e])) po[(size_t)e * seg_rows] += to_f32<kBf16>(v[e]);
                }
                // O is read before the next segment's products write it
                tc::fence_before_sync();
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    // (not earlier: joining CTAs that wait on the SMs all the while cost 2 to 12 us)
    grid_launch_dependents();
    if (warp == C::kMmaWarp) tc::dealloc(tmem, 512);
}

// ---------------------------------------------------------------- join
constexpr int kJoinWarps = 8;

// grid (blocks of 32 rows, KV heads, column blocks): lane = row of the head's
// row line (sequence, node, head of the group).  Every segment that holds the
// row is read column by column, 32 rows a load, four segments of 8 columns in
// flight.  kSplit = 1: a warp per 8 columns; kSplit = 8: the 8 warps share 8
// columns and take every eighth segment (few units are cut into many).
template <int D, bool kBf16, int kSplit>
__global__ void __launch_bounds__(kJoinWarps * 32) prefix_attn_join_kernel(const PrefixAttnArgs a, const Layout lay) {
    constexpr int E = 8, U = 4, kStreams = Cfg<D>::kStreams;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
    // the plan and the sums over the sequences, in one round trip
    __shared__ int cn[kMaxB + 1], ct[kMaxB + 1], cu[kMaxB + 1];
    const int* sums = reinterpret_cast<const int*>(static_cast<const unsigned char*>(a.ws) + sizeof(Plan));
    for (int i = threadIdx.x; i <= a.B; i += kJoinWarps * 32) {
        const int x = sums[i], y = sums[kMaxB + 1 + i], z = sums[2 * (kMaxB + 1) + i];
        cn[i] = x;
        ct[i] = y;
        cu[i] = z;
    }
    const Plan p = *reinterpret_cast<const Plan*>(a.ws);
    const int line = blockIdx.x * 32 + lane;
    if (blockIdx.x * 32 >= p.rows) return;
    const bool live = line < p.rows;
    __syncthreads();
    const float2* ml = reinterpret_cast<const float2*>(static_cast<const unsigned char*>(a.ws) + lay.off_ml);
    const float* po = reinterpret_cast<const float*>(static_cast<const unsigned char*>(a.ws) + lay.off_o);
    const int G = lay.G, at = live ? line : p.rows - 1;
    const int b = find_in(cn, a.B, at / G), n = cn[b + 1] - cn[b];
    const int own_line = at - cn[b] * G;

    // the two units of the row, [0] prefix and [1] own: first segment, the row
    // in it, segments, partial results
    size_t seg0[2];
    int row[2], n_part[2], two[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        long long w, unit;
        int tiles, per, r, places;
        if (k == 0) {
            per = p.p_rows;
            const int rt = at / per;
            r = at - rt * per;
            unit = (long long)h * p.p_units + rt;
            places = p.p_steps;
            w = unit * places;
            tiles = p.p_tiles;
        } else {
            const int units = cu[b + 1] - cu[b];
            per = ceil_div(n * G, units);
            const int rt = own_line / per;
            r = own_line - rt * per;
            unit = (long long)h * p.own_units + cu[b] + rt;
            places = (ct[b + 1] - ct[b]) / units;
            w = (long long)a.Hkv * p.p_units * p.p_steps + (long long)h * p.own_steps + ct[b] + (long long)rt * places;
            tiles = (places - p.setup) / tile_places<Cfg<D>::kRows>(per);
        }
        const int seg_rows = k == 0 ? lay.p_seg_rows : lay.own_seg_rows, half = k == 0 ? lay.half_p : lay.half_own;
        two[k] = kStreams == 2 && per > 128;
        if (two[k]) {
            const int rows = min(per, k == 0 ? p.rows - (at - r) : n * G - (own_line - r)), h1 = (rows + 1) >> 1;
            if (r >= h1) r += half - h1;
        }
        row[k] = r;
        n_part[k] = 0;
        seg0[k] = 0;
        if (tiles > 0) {
            // share of place x: the largest c with floor(c total / ctas) <= x;
            // the tiles' first places run from w + p.setup on (the last tile's may
            // be one before the unit's end)
            const int wt = tile_places<Cfg<D>::kRows>(per);
            const long long x0 = w + p.setup, x1 = w + p.setup + (long long)(tiles - 1) * wt;
            const long long c0 = div_small((x0 + 1) * p.ctas - 1, p.total), c1 = div_small((x1 + 1) * p.ctas - 1, p.total);
            n_part[k] = (int)(c1 - c0 + 1) * (kStreams == 2 && !two[k] ? 2 : 1);
            seg0[k] = (k == 0 ? 0 : lay.own_row0) + (size_t)(unit + c0) * seg_rows;
        }
    }
    const int n0 = n_part[0], n_all = live ? n0 + n_part[1] : 0;
    // partial result i: where its (max, sum) and its first column lie
    auto where = [&](int i, size_t& m_at, size_t& o_at, int& stride) {
        const int k = i >= n0, j = i - (k ? n0 : 0);
        const int half = k ? lay.half_own : lay.half_p;
        stride = k ? lay.own_seg_rows : lay.p_seg_rows;
        const bool pair = kStreams == 2 && !two[k];
        const size_t s0 = seg0[k] + (size_t)(pair ? j >> 1 : j) * stride;
        const int r = row[k] + (pair && (j & 1) ? half : 0);
        m_at = s0 + r;
        o_at = s0 * D + r;
    };
    const int part = kSplit == 1 ? 0 : warp;
    // A running maximum: (max, sum) and O are asked for together.
    float top = -INFINITY, sum = 0.0f, acc[E];
    bool drop = false;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    const int c0 = (kSplit == 1 ? blockIdx.z * kJoinWarps + warp : blockIdx.z) * E;
    for (int i0 = part; i0 < n_all; i0 += U * kSplit) {
        float v[U][E];
        float2 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            size_t m_at, o_at;
            int stride;
            where(min(i0 + u * kSplit, n_all - 1), m_at, o_at, stride);
            x[u] = ml[m_at];
            const float* col = po + o_at + (size_t)c0 * stride;
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = __ldcg(col + (size_t)e * stride);
        }
        // (a sum of zero: nothing seen there, its O was not written)
        float next = top;
#pragma unroll
        for (int u = 0; u < U; ++u) drop |= x[u].y == kMalformed;
        bool use[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            use[u] = i0 + u * kSplit < n_all && !(x[u].y == 0.0f);
            if (use[u]) next = fmaxf(next, x[u].x);
        }
        const float old = next == top ? 1.0f : ex2(top - next);
        top = next;
        sum *= old;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= old;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float f = use[u] ? ex2(x[u].x - top) : 0.0f;
            sum = use[u] ? fmaf(f, x[u].y, sum) : sum;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = use[u] ? fmaf(f, v[u][e], acc[e]) : acc[e];
        }
    }
    if constexpr (kSplit > 1) {
        __shared__ float red[kSplit][E + 2][32];
#pragma unroll
        for (int e = 0; e < E; ++e) red[warp][e][lane] = acc[e];
        red[warp][E][lane] = drop ? kMalformed : sum;
        red[warp][E + 1][lane] = top;
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int q = 1; q < kSplit; ++q) top = fmaxf(top, red[q][E + 1][lane]);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
        sum = 0.0f;
#pragma unroll
        for (int q = 0; q < kSplit; ++q) {
            const float l = red[q][E][lane], f = l == 0.0f ? 0.0f : ex2(red[q][E + 1][lane] - top);
            drop |= l == kMalformed;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = l == 0.0f ? acc[e] : fmaf(f, red[q][e][lane], acc[e]);
            sum = l == 0.0f ? sum : fmaf(f, l, sum);
        }
    }
    if (!live || drop) return;
    const float inv = 1.0f / sum;
    uint32_t out[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) out[e / 2] = pack2<kBf16>(acc[e] * inv, acc[e + 1] * inv);
    const int node = own_line / G, g = own_line - node * G;
    uint4* dst = reinterpret_cast<uint4*>(a.out + (((size_t)b * a.N_max + node) * a.Hq + h * G + g) * D + c0);
    *dst = make_uint4(out[0], out[1], out[2], out[3]);
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::atomic<EncodeTiled> cached{nullptr};
    EncodeTiled f = cached.load(std::memory_order_relaxed);
    if (f) return f;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    f = reinterpret_cast<EncodeTiled>(p);
    cached.store(f, std::memory_order_relaxed);
    return f;
}

// A plane as [n_pages][Hkv][page][D]; boxes of 64 elements x a page's rows (at
// most a tile's), 128-byte swizzle.
bool plane_map(const PrefixAttnArgs& a, const void* plane, CUtensorMap* m) {
    EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dim[4] = {(cuuint64_t)a.D, (cuuint64_t)a.page, (cuuint64_t)a.Hkv, (cuuint64_t)a.n_pages};
    const cuuint64_t row = (cuuint64_t)a.D * 2;
    const cuuint64_t stride[3] = {row, row * a.page, row * a.page * a.Hkv};
    const cuuint32_t box[4] = {64, (cuuint32_t)(a.page < kKT ? a.page : kKT), 1, 1}, one[4] = {1, 1, 1, 1};
    return f(m, a.type == DFLV_KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void*>(plane), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kBf16>
cudaError_t launch_typed(const PrefixAttnArgs& a, cudaStream_t stream) {
    using C = Cfg<D>;
    const Layout lay = make_layout(a, sm_count_cached());
    CUtensorMap k_map, v_map;
    if (!plane_map(a, a.kp, &k_map) || !plane_map(a, a.vp, &v_map)) return cudaErrorNotSupported;
    cudaError_t e = ensure_smem(prefix_attn_kernel<D, kBf16>, C::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(prefix_attn_kernel<D, kBf16>, dim3(lay.ctas), dim3(C::kThreads), C::kSmem, stream, 1, a, lay, k_map,
                   v_map);
    if (e != cudaSuccess) return e;
    // A unit is cut into 1 + ctas / units segments on average; from three on, the
    // join's warps share them.  (56 + 8 units over 152 CTAs, 7 trees of 13 nodes:
    // 18.5 us shared, 22.0 not; 128 + 68 units, 16 trees of 22 nodes: 161 us
    // shared, 111 not.)
    const int rows = a.B * lay.max_rows;  // of a KV head, at most
    const dim3 grid((rows + 31) / 32, a.Hkv, D / 64), grid_split(grid.x, grid.y, D / 8), block(kJoinWarps * 32);
    if (2 * (lay.p_units + lay.own_units) <= lay.ctas)
        return launch_pdl(prefix_attn_join_kernel<D, kBf16, 8>, grid_split, block, 0, stream, 1, a, lay);
    return launch_pdl(prefix_attn_join_kernel<D, kBf16, 1>, grid, block, 0, stream, 1, a, lay);
}

}  // namespace

size_t prefix_attn_workspace_bytes(const PrefixAttnArgs& a) { return make_layout(a, sm_count_cached()).bytes; }

cudaError_t launch_prefix_attn(const PrefixAttnArgs& a, cudaStream_t stream) {
    const bool bf = a.type == DFLV_KV_BF16;
    switch (a.D) {
        case 64: return bf ? launch_typed<64, true>(a, stream) : launch_typed<64, false>(a, stream);
        case 128: return bf ? launch_typed<128, true>(a, stream) : launch_typed<128, false>(a, stream);
        case 256: return bf ? launch_typed<256, true>(a, stream) : launch_typed<256, false>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace dflv
