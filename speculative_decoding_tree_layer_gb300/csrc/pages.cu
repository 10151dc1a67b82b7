// pages.cu -- the page bookkeeping of a paged cache (block tables, slot maps,
// the free list) and the writes into its pages (new tokens, accepted paths).
//
// The pages of a call are numbered by an exclusive sum of the sequences'
// demands, so every sequence knows its pages without an atomic and the
// result does not depend on the order of execution.  Every CTA sums the
// demands before its own sequences itself: three int32 per sequence from the
// L2, far cheaper than a grid-wide exchange; the in-place counters are
// then updated by a second, dependent launch (by the same one when a single
// CTA does the work), after every CTA has read them.
//
// A slot costs 4 bytes written, a page 4 bytes read and 4 written, a cache row is
// read and written once.  Small calls are bound by the host and the launches (8
// sequences of 22 nodes: grow and release 12 us, 7 of them on the GPU; the accepted
// path of 16 layers 21 us, 4.5 of them on the GPU).  1024 prompts of 4096 tokens, grow
// and release: 16.4 us for 20 MB, four launches that wait for one another (17 us in
// a replayed graph too).  Prompts of 16 x 2048 tokens into the cache: 201 MB in 36.9
// us, 5.4 TB/s.
#include "common.cuh"
#include "kernels.h"

namespace dflv {

namespace {

constexpr int kTabThreads = 256;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kSlotChunk = 4096;  // slots of one sequence per CTA

// Sums of pages: a batch's tables have fewer than 2^31 entries.

// Sum of v over the block, for every thread.
DFLV_DEVINL int block_sum(int v, int* red) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < warps ? red[lane] : 0);
}

// Exclusive sum of v over the block's threads; total receives the sum.
DFLV_DEVINL int block_exclusive(int v, int* red, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    const int r = lane < warps ? red[lane] : 0;
    total = __reduce_add_sync(0xffffffffu, r);
    return __reduce_add_sync(0xffffffffu, lane < warp ? r : 0) + x - v;
}

struct Demand {
    int held, past, nw, more;
    bool bad;
};

DFLV_DEVINL Demand grow_demand(const PageTableArgs& a, int b) {
    Demand d;
    d.past = a.len[b];
    d.nw = a.n_new[b];
    d.held = a.n_held[b];
    const uint32_t need = ((uint32_t)d.past + (uint32_t)d.nw + a.page - 1) >> a.page_shift;
    d.bad = d.past < 0 || (uint32_t)d.nw > (uint32_t)a.N_max || (uint32_t)d.held > (uint32_t)a.max_pages ||
            need > (uint32_t)a.max_pages;
    d.more = d.bad ? 0 : max((int)need - d.held, 0);
    return d;
}

// Pages that sequence b gives back, 0 if its lengths do not fit.
DFLV_DEVINL int release_back(const PageTableArgs& a, int b, bool& bad) {
    const int len = a.len[b], held = a.n_held[b];
    const int keep = (int)(((uint32_t)len + a.page - 1) >> a.page_shift);
    bad = len < 0 || held < 0 || held > a.max_pages || keep > held;
    return bad ? 0 : held - keep;
}

DFLV_DEVINL bool in_pool(const PageTableArgs& a, int id) { return (unsigned)id < (unsigned)a.n_pages; }
constexpr int kNoSlots = -(1 << 30);  // negative with any place in a page added

DFLV_DEVINL int free_count(const PageTableArgs& a) {
    const int f = *a.n_free;
    return f < 0 || f > a.n_pages ? 0 : f;
}

// Updates n_held and n_free for the whole batch (one CTA).  Demands are
// served in order while their running sum fits.
template <bool kGrow>
DFLV_DEVINL void update_counts(const PageTableArgs& a, int* red) {
    const int tid = threadIdx.x, T = blockDim.x;
    const int n_free = free_count(a);
    int total = 0;
    if (!kGrow) {
        for (int b = tid; b < a.B; b += T) {
            bool bad;
            total += release_back(a, b, bad);
        }
        total = block_sum(total, red);
        if ((long long)n_free + total > a.n_pages) return;  // reported by the fill
        for (int b = tid; b < a.B; b += T) {
            bool bad;
            const int back = release_back(a, b, bad);
            if (back) a.n_held[b] -= back;
        }
    } else {
        int carry = 0;
        for (int b0 = 0; b0 < a.B; b0 += T) {
            const int b = b0 + tid;
            Demand d = {};
            if (b < a.B) d = grow_demand(a, b);
            int sum;
            const int start = carry + block_exclusive(d.more, red, sum);
            carry += sum;
            const bool served = d.more > 0 && start + d.more <= n_free;
            if (served) {
                a.n_held[b] = d.held + d.more;
                total -= d.more;
            }
        }
        total = block_sum(total, red);
    }
    __syncthreads();
    if (tid == 0 && total != 0) *a.n_free = n_free + total;
}

// move(s, first, step) for the rows of the CTA's nb sequences: a warp a row, or
// several where there are fewer rows than warps; the row's pages first, first +
// step, ..
template <typename F>
DFLV_DEVINL void for_rows(int nb, F move) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_row = max(1, kTabWarps / nb);
    for (int s = warp / per_row; s < nb; s += kTabWarps / per_row)
        move(s, warp % per_row * 32 + lane, per_row * 32);
}
// Copies pages first, first + step, .. below n, eight loads in flight.
template <typename Load, typename Store>
DFLV_DEVINL void copy_pages(int first, int step, int n, Load load, Store store) {
    constexpr int U = 8;
    for (int t0 = first; t0 < n; t0 += U * step) {
        int id[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t0 + u * step < n) id[u] = load(t0 + u * step);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t0 + u * step < n) store(t0 + u * step, id[u]);
    }
}

// grid (sequence ranges, slot chunks).  CTA x owns `per` <= 256 consecutive
// sequences; chunk y owns slots [y * kSlotChunk, +kSlotChunk) of each, and
// chunk 0 their table entries.
template <bool kFuse>
__global__ void __launch_bounds__(kTabThreads) tables_grow_kernel(const PageTableArgs a, int per) {
    __shared__ int red[kTabWarps];
    __shared__ int start_s[kTabThreads], held_s[kTabThreads], more_s[kTabThreads], past_s[kTabThreads], new_s[kTabThreads];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x;
    const int b0 = blockIdx.x * per, nb = min(per, a.B - b0);
    const int n_free = free_count(a);
    // The loads of the CTA's own sequences and of those before it go out
    // together.
    Demand d = {};
    if (tid < nb) d = grow_demand(a, b0 + tid);
    int before = 0, own;
    for (int b = tid; b < b0; b += kTabThreads) before += grow_demand(a, b).more;
    before = b0 ? block_sum(before, red) : 0;
    const int start = before + block_exclusive(d.more, red, own);
    if (tid < nb) {
        const bool refused = d.bad || (d.more > 0 && start + d.more > n_free);
        if (refused && blockIdx.y == 0) raise_status(a.status, DFLV_DEV_CAPACITY);
        start_s[tid] = refused ? 0 : min(start, n_free);
        held_s[tid] = d.held;
        more_s[tid] = refused ? 0 : d.more;
        past_s[tid] = d.past;
        new_s[tid] = refused ? 0 : d.nw;
        if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0 && n_free != *a.n_free)
            raise_status(a.status, DFLV_DEV_CAPACITY);
    }
    __syncthreads();
    bool bad_id = false;
    if (blockIdx.y == 0)
        for_rows(nb, [&](int s, int first, int step) {
            int32_t* row = a.table + (size_t)(b0 + s) * a.max_pages + held_s[s];
            const int32_t* top = a.free_list + (n_free - 1 - start_s[s]);
            copy_pages(first, step, more_s[s], [&](int t) { return top[-t]; }, [&](int t, int id) {
                bad_id |= !in_pool(a, id);
                row[t] = id;
            });
        });
    const int shift = a.page_shift, mask = a.page - 1;
    const int i0 = blockIdx.y * kSlotChunk, i1 = min(a.N_max, i0 + kSlotChunk), w = i1 - i0;
    // page q of sequence s: one it held, or one of the new ones
    auto page_of = [&](int s, int q) {
        const int32_t* at = q < held_s[s] ? a.table + ((size_t)(b0 + s) * a.max_pages + q)
                                          : a.free_list + (n_free - 1 - (start_s[s] + q - held_s[s]));
        return *at;
    };
    // An id outside the pool gives no slots: shifted, it could name a slot of any page.
    auto first_slot = [&](int id) {
        const bool ok = in_pool(a, id);
        bad_id |= !ok;
        return ok ? id << shift : kNoSlots;
    };
    if ((a.N_max & 3) == 0 && (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0) {
        // Four slots a thread and one 16-byte store: `here` of them lie in one
        // page, the others in the next.  Four such pieces in flight, as the page
        // ids come from the L2.
        constexpr int U = 4;
        const int w4 = w >> 2, all = nb * w4;
        const uint32_t inv = 0xffffffffu / (uint32_t)w4 + 1;  // e / w4 is the upper half of e inv: e w4 < 2^32
        static_assert(kTabThreads * (kSlotChunk / 4) * (long long)(kSlotChunk / 4) < 1ll << 32, "exact quotients");
        for (int e0 = tid; e0 < all; e0 += U * kTabThreads) {
            int s[U], i[U], first[U], second[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = e0 + u * kTabThreads;
                if (e >= all) break;
                s[u] = w4 == 1 ? e : (int)__umulhi((uint32_t)e, inv);
                i[u] = (e - s[u] * w4) * 4 + i0;
                first[u] = second[u] = 0;
                if (i[u] < new_s[s[u]]) {
                    const int t = past_s[s[u]] + i[u], here = a.page - (t & mask);
                    first[u] = page_of(s[u], t >> shift);
                    if (here < 4 && i[u] + here < new_s[s[u]]) second[u] = page_of(s[u], (t >> shift) + 1);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (e0 + u * kTabThreads >= all) break;
                const int off = (past_s[s[u]] + i[u]) & mask, here = a.page - off, left = new_s[s[u]] - i[u];
                const int x0 = first_slot(first[u]) + off, x1 = first_slot(second[u]) - here;
                int x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = k < left ? max((k < here ? x0 : x1) + k, -1) : -1;
                *reinterpret_cast<int4*>(a.slots + (size_t)(b0 + s[u]) * a.N_max + i[u]) = make_int4(x[0], x[1], x[2], x[3]);
            }
        }
    } else {
        for (int e = tid; e < nb * w; e += kTabThreads) {
            const int s = e / w, i = i0 + (e - s * w), t = past_s[s] + i;
            a.slots[(size_t)(b0 + s) * a.N_max + i] =
                i < new_s[s] ? max(first_slot(page_of(s, t >> shift)) + (t & mask), -1) : -1;
        }
    }
    // (once a thread: raised where each is found, 1024 prompts take 17.1 us, not 16.4)
    if (bad_id) raise_status(a.status, DFLV_DEV_PAGE);
    if (kFuse) {
        __syncthreads();
        update_counts<true>(a, red);
    }
}

template <bool kFuse>
__global__ void __launch_bounds__(kTabThreads) tables_release_kernel(const PageTableArgs a, int per) {
    __shared__ int red[kTabWarps];
    __shared__ int start_s[kTabThreads], back_s[kTabThreads], keep_s[kTabThreads];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x;
    const int b0 = blockIdx.x * per, nb = min(per, a.B - b0);
    const int n_free = free_count(a);
    int before = 0, total = 0, own;
    int back = 0;
    bool bad = false;
    for (int b = tid; b < a.B; b += kTabThreads) {
        bool x;
        const int r = release_back(a, b, x);
        total += r;
        if (b < b0) before += r;
    }
    if (tid < nb) back = release_back(a, b0 + tid, bad);
    total = block_sum(total, red);
    before = b0 ? block_sum(before, red) : 0;
    const int start = before + block_exclusive(back, red, own);
    const bool full = (long long)n_free + total > a.n_pages || n_free != *a.n_free;
    if (bad || (full && tid == 0)) raise_status(a.status, DFLV_DEV_CAPACITY);
    if (!full) {
        if (tid < nb) {
            start_s[tid] = start;
            back_s[tid] = back;
            keep_s[tid] = back ? a.n_held[b0 + tid] - back : 0;
        }
        __syncthreads();
        int32_t* top = a.free_list + n_free + total - 1;
        for_rows(nb, [&](int s, int first, int step) {
            const int32_t* row = a.table + (size_t)(b0 + s) * a.max_pages + keep_s[s];
            copy_pages(first, step, back_s[s], [&](int t) { return row[t]; }, [&](int t, int id) {
                if (!in_pool(a, id)) raise_status(a.status, DFLV_DEV_PAGE);
                *(top - (start_s[s] + t)) = id;
            });
        });
    }
    if (kFuse) {
        __syncthreads();
        if (!full) update_counts<false>(a, red);
    }
}

constexpr int kCountThreads = 1024;

template <bool kGrow>
__global__ void __launch_bounds__(kCountThreads) tables_update_kernel(const PageTableArgs a) {
    __shared__ int red[kCountThreads / 32];
    // The whole preceding launch has read the counters and written its pages.
    grid_dependency_wait();
    if (!kGrow && free_count(a) != *a.n_free) return;
    update_counts<kGrow>(a, red);
}

// ---------------------------------------------------------------- writes
constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;

// One 16-byte piece of k_new and of v_new per item, kAppendUnroll items in
// flight per thread; pieces of a row are consecutive, so loads and stores of
// a warp cover whole rows.
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const PagedAppendArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int dp = a.D >> 3, dshift = a.d_shift;      // pieces of a head's row
    const int row_pieces = a.Hkv << dshift;           // pieces of a token
    const long long total = (long long)a.rows * row_pieces;
    const long long step = (long long)gridDim.x * kAppendThreads;
    const long long slots_end = (long long)a.n_pages << a.page_shift;
    for (long long e0 = (long long)blockIdx.x * kAppendThreads + threadIdx.x; e0 < total; e0 += step * kAppendUnroll) {
        uint4 kx[kAppendUnroll], vx[kAppendUnroll];
        long long dst[kAppendUnroll];
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u) {
            const long long e = e0 + u * step;
            dst[u] = -1;
            if (e >= total) continue;
            const int row = (int)(e / row_pieces), piece = (int)(e - (long long)row * row_pieces);
            const int slot = __ldg(a.slots + row);
            if (slot < 0 || slot >= slots_end) {
                if (slot != -1 && piece == 0) raise_status(a.status, DFLV_DEV_PAGE);
                continue;
            }
            const int h = piece >> dshift, c = piece & (dp - 1);
            const size_t src = (size_t)row * a.kv_stride + (size_t)piece * 8;
            kx[u] = __ldcs(reinterpret_cast<const uint4*>(a.k_new + src));
            vx[u] = __ldcs(reinterpret_cast<const uint4*>(a.v_new + src));
            const long long page = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
            dst[u] = ((((page * a.Hkv + h) << a.page_shift) + off) << dshift) + c;
        }
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u)
            if (dst[u] >= 0) {
                reinterpret_cast<uint4*>(a.kp)[dst[u]] = kx[u];
                reinterpret_cast<uint4*>(a.vp)[dst[u]] = vx[u];
            }
    }
}

constexpr int kMoveThreads = 128;
constexpr int kMoveBatch = 8;

// grid (B * Hkv, layers).  A thread owns 16-byte columns of the head's K and V
// rows and moves them path entry by path entry: the path ascends, so entry
// m's destination (node m) is the source of no later entry, and a batch of
// kMoveBatch rows is read before it is written.
__global__ void __launch_bounds__(kMoveThreads) paged_commit_kernel(const __grid_constant__ PagedCommitArgs a) {
    __shared__ long long src_s[64], dst_s[64];
    grid_dependency_wait();
    const int tid = threadIdx.x, N = a.N_max;
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x - b * a.Hkv, layer = blockIdx.y;
    const bool first = h == 0 && layer == 0;
    const int L = __ldg(a.path_len + b);
    const bool L_ok = L >= 0 && L <= N;
    bool bad_path = !L_ok, bad_slot = false;
    const long long slots_end = (long long)a.n_pages << a.page_shift;
    const int mask = (1 << a.page_shift) - 1;
    if (L_ok && tid < L) {
        const int p = __ldg(a.path + (size_t)b * N + tid);
        const int prev = tid ? __ldg(a.path + (size_t)b * N + tid - 1) : -1;
        if (p < 0 || p >= N || p <= prev) {
            bad_path = true;
        } else {
            const int s = __ldg(a.slots + (size_t)b * N + p), t = __ldg(a.slots + (size_t)b * N + tid);
            bad_slot = s < 0 || s >= slots_end || t < 0 || t >= slots_end;
            // the head's row of a slot, in rows of D
            src_s[tid] = (((long long)(s >> a.page_shift) * a.Hkv + h) << a.page_shift) + (s & mask);
            dst_s[tid] = (((long long)(t >> a.page_shift) * a.Hkv + h) << a.page_shift) + (t & mask);
        }
    }
    bad_path = __syncthreads_or(bad_path);
    bad_slot = __syncthreads_or(bad_slot);
    if (bad_path || bad_slot) {
        if (first && tid == 0) raise_status(a.status, bad_path ? DFLV_DEV_PATH : DFLV_DEV_PAGE);
        return;
    }
    const int dp = a.D >> 3;
    // half of the threads take the keys, the other half the values
    uint4* plane = reinterpret_cast<uint4*>(tid < kMoveThreads / 2 ? a.k[layer] : a.v[layer]);
    const int c = tid & (kMoveThreads / 2 - 1), lanes = (kMoveThreads / 2) / dp;  // dp <= 32
    if (c < lanes * dp) {
        // `lanes` entries side by side: the batch is lanes * kMoveBatch rows
        const int col = c % dp, l = c / dp;
        for (int m0 = 0; m0 < L; m0 += kMoveBatch * lanes) {
            uint4 x[kMoveBatch];
#pragma unroll
            for (int u = 0; u < kMoveBatch; ++u) {
                const int m = m0 + u * lanes + l;
                if (m < L && src_s[m] != dst_s[m]) x[u] = plane[src_s[m] * dp + col];
            }
            // (the threads of a column group sit in different warps for
            // D = 64 only within the same half: order the batch)
            asm volatile("bar.sync %0, %1;\n" ::"r"(1 + (tid >= kMoveThreads / 2)), "r"(kMoveThreads / 2) : "memory");
#pragma unroll
            for (int u = 0; u < kMoveBatch; ++u) {
                const int m = m0 + u * lanes + l;
                if (m < L && src_s[m] != dst_s[m]) plane[dst_s[m] * dp + col] = x[u];
            }
        }
    }
    if (first && tid == 0 && a.n_past != nullptr) a.n_past[b] += L;
}

}  // namespace

template <bool kGrow>
static cudaError_t launch_tables(const PageTableArgs& a, cudaStream_t stream) {
    const int sms = sm_count_cached();
    // Enough CTAs for two per SM, at most 256 sequences each.
    const int chunks = kGrow ? (a.N_max + kSlotChunk - 1) / kSlotChunk : 1;
    int gx = (a.B + kTabThreads - 1) / kTabThreads;
    // A CTA works off about 2048 slots (or table rows of 8 sequences) before
    // a second one pays for its own sums.
    const long long work = kGrow ? (long long)a.B * a.N_max : (long long)a.B * 256;
    long long want = work / 2048;
    // (1024 sequences of 4096 new slots: grow and release take as long with two,
    // four or eight CTAs an SM)
    if (want > 2L * sms) want = 2L * sms;
    if (want > a.B) want = a.B;
    if (want > gx) gx = (int)want;
    const int per = (a.B + gx - 1) / gx;
    gx = (a.B + per - 1) / per;
    const dim3 grid(gx, chunks);
    const bool fuse = gx == 1 && chunks == 1;
    cudaError_t e;
    if (kGrow)
        e = fuse ? launch_pdl(tables_grow_kernel<true>, grid, dim3(kTabThreads), 0, stream, 1, a, per)
                 : launch_pdl(tables_grow_kernel<false>, grid, dim3(kTabThreads), 0, stream, 1, a, per);
    else
        e = fuse ? launch_pdl(tables_release_kernel<true>, grid, dim3(kTabThreads), 0, stream, 1, a, per)
                 : launch_pdl(tables_release_kernel<false>, grid, dim3(kTabThreads), 0, stream, 1, a, per);
    if (e != cudaSuccess || fuse) return e;
    return launch_pdl(tables_update_kernel<kGrow>, dim3(1), dim3(kCountThreads), 0, stream, 1, a);
}

cudaError_t launch_tables_grow(const PageTableArgs& a, cudaStream_t stream) { return launch_tables<true>(a, stream); }
cudaError_t launch_tables_release(const PageTableArgs& a, cudaStream_t stream) {
    return launch_tables<false>(a, stream);
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
    const long long items = (long long)a.rows * (a.Hkv << a.d_shift);
    const long long per_cta = (long long)kAppendThreads * kAppendUnroll;
    long long ctas = (items + kAppendThreads - 1) / kAppendThreads;
    // small calls: one item a thread (latency); large ones: eight CTAs an SM
    const long long cap = 8L * sm_count_cached();
    if (ctas > cap) ctas = (items + per_cta - 1) / per_cta;
    if (ctas > cap) ctas = cap;
    return launch_pdl(paged_append_kernel, dim3((unsigned)ctas), dim3(kAppendThreads), 0, stream, 1, a);
}

cudaError_t launch_paged_commit(const PagedCommitArgs& a, cudaStream_t stream) {
    return launch_pdl(paged_commit_kernel, dim3((unsigned)(a.B * a.Hkv), (unsigned)a.n_layers), dim3(kMoveThreads), 0,
                      stream, 1, a);
}

}  // namespace dflv
