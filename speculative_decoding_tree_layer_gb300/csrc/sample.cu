// sample.cu -- one token per row drawn from the target's logits with
// temperature, top-k, top-p and min-p (include/dflv.h states the rule).
//
// Every filter keeps a leading part of the row's tokens in descending order
// (ties by index), so what is kept is described by one threshold: the key of
// the last kept token and how many tokens of that key are kept.  A
// thread-block cluster holds a row in its CTAs' shared memory, so the logits
// are read once from HBM; every later pass over them is on chip.
//   * no filter: one pass sums the masses, one exchange finds the CTA and
//     thread whose tokens hold the draw.
//   * a filter: the tokens are counted in 2048 bins, linear in the logit below
//     the maximum (a small top-k: only the lanes' largest tokens, in 512).  Counts
//     say in which bin the top-k cut lies, and, with their tokens' mean position
//     in the bin, between which bins the top-p cut lies.  If all that can be
//     kept is at most kList tokens (the usual case), they go to one CTA, which
//     ranks them and decides.  Else one pass sums the masses and collects the
//     tokens of the cut's bins, a finer count and a comparison of the few left
//     find the last kept token (many copies of one logit: an interval of
//     sortable keys is narrowed, eight parts a round), and what each warp keeps
//     follows from the collected tokens.
//
// What bounds it: one row, the exchanges between the CTAs (about 1.1 K cycles
// each, and 3 to 5 K where they read each other's bins); many rows, the
// instructions, as a mass takes about 30 and the loads are done after a third of
// a row's time.  151,936 fp32 logits from a cold L2, in us without the host's time,
// with 1 / 64 / 264 rows: argmax (T = 0) 5.4 / 17 / 52, top-k 50 and top-p 0.9 11.5 /
// 29 / 99, no filter 12.3 / 38 / 125, min-p 0.05 15 / 42 / 140, top-p 0.95 alone 44 / 95
// / 328.
//
// A token's mass e^{(x - max) / T} is computed to 2^-30 of itself as a pair of
// floats, summed per thread in such pairs and from there on as 64-bit integers
// in units of 2^-44, whose sums are exact.  A draw compares a running sum over
// up to 400,000 tokens with u times the total: with masses rounded to 2^-24 a
// flat row would be decided by rounding in one draw of a hundred.  (64-bit
// floating point would do, but this GPU has two FP64 lanes an SM.)
#include <cstddef>
#include <type_traits>

#include "cluster.cuh"
#include "common.cuh"
#include "kernels.h"

namespace dflv {

namespace {

constexpr int kSampThreads = 512;
constexpr int kSampWarps = kSampThreads / 32;
constexpr int kSampMaxCluster = 8;
constexpr int kCuts = 8;
constexpr int kMassBits = 44;
constexpr int kTab = 64;    // 2^(j/64), j in [-32, 32]
constexpr int kBins = 2048;  // four a thread
constexpr int kList = 1024;  // candidates one CTA decides on: two a thread
constexpr float kOctaves = 46.5f;  // below 2^-46 a token has no mass
static_assert(kBins == 4 * kSampThreads && kList == 2 * kSampThreads, "bins and candidates per thread");

// 2^(j/64) as pairs of floats, by the exponential series.
struct ExpTable {
    float hi[kTab + 1], lo[kTab + 1];
};
constexpr ExpTable make_exp_table() {
    ExpTable t = {};
    for (int j = 0; j <= kTab; ++j) {
        const double z = (j - kTab / 2) * 0.69314718055994530942 / kTab;
        double v = 1.0, term = 1.0;
        for (int i = 1; i < 24; ++i) {
            term *= z / i;
            v += term;
        }
        t.hi[j] = (float)v;
        t.lo[j] = (float)(v - (double)(float)v);
    }
    return t;
}
__device__ constexpr ExpTable kExpTable = make_exp_table();

typedef unsigned long long u64;

// Floats in an order-preserving 32-bit key; -infinity has the lowest key of
// the values that occur (NaN has been replaced).
DFLV_DEVINL uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
DFLV_DEVINL float float_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // key_of(-infinity)

template <typename T>
DFLV_DEVINL float to_float(T x);
template <>
DFLV_DEVINL float to_float<float>(float x) { return x; }
template <>
DFLV_DEVINL float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
DFLV_DEVINL float to_float<__half>(__half x) { return __half2float(x); }

// NaN counts as -infinity; -0 becomes +0, so that equal values have one key.
DFLV_DEVINL float canonical(float x) { return x != x ? -INFINITY : x + 0.0f; }

struct Scale {
    float mx, ch, cl;  // row maximum, log2(e) / T as a pair
};

// e^{(x - mx) / T} as hi + lo; tab[j + 32] = 2^(j/64) as (hi, lo).
//   d = x - mx exactly (two-sum), t = d log2(e) / T as a pair, t = n + j/64 + g
//   with |g| <= 1/128; 2^g - 1 = z + z^2/2 + z^3/6 with z = g ln 2, whose next
//   term is below 2^-34.  n and j come from adding 1.5 2^23 (the sum's last bits
//   are the rounded value).  The terms left out (products of two rounding
//   errors) are below 2^-31 and of either sign.
// Two tokens at a time, as packed operations: the passes over masses are bound
// by the instructions they issue (151,936 logits on 8 CTAs: a pass over all masses
// 7.2 K cycles, one token at a time 9.0 K).
struct Mass {
    float hi, lo;
};
struct Mass2 {
    uint64_t hi, lo;
};
DFLV_DEVINL uint64_t twice(float v) { return pair(v, v); }
DFLV_DEVINL Mass2 mass_pair2(float x0, float x1, const Scale& s, const float2* tab) {
    constexpr float kMagic = 12582912.0f, kLn2 = 0.693147182464599609375f;  // 1.5 2^23
    constexpr int kMagicBits = 0x4B400000;
    const uint64_t x = pair(x0, x1), minus = twice(-1.0f), ch = twice(s.ch), nmx = twice(-s.mx);
    const uint64_t dh = add2(x, nmx);
    const uint64_t bb = fma2(x, minus, dh);  // (a - b is fma(b, -1, a))
    const uint64_t dl = add2(fma2(fma2(bb, minus, dh), minus, x), fma2(bb, minus, nmx));
    const uint64_t t = mul2(dh, ch);
    const uint64_t tl2 = fma2(dl, ch, fma2(dh, twice(s.cl), fma2(dh, ch, mul2(dh, twice(-s.ch)))));
    float th0, th1, tl0, tl1;
    unpair(t, th0, th1);
    unpair(tl2, tl0, tl1);
    const bool ok0 = th0 > -46.0f, ok1 = th1 > -46.0f;  // else below half a unit (or x is -infinity)
    const uint64_t th = pair(ok0 ? th0 : -46.0f, ok1 ? th1 : -46.0f), tl = pair(ok0 ? tl0 : 0.0f, ok1 ? tl1 : 0.0f);
    const uint64_t magic = twice(kMagic), nm = add2(th, magic);
    const uint64_t f = add2(th, fma2(nm, minus, magic));   // exact
    const uint64_t fs = add2(f, tl);
    const uint64_t fl = fma2(fma2(f, minus, fs), minus, tl);
    const uint64_t jm = fma2(fs, twice((float)kTab), magic);
    const uint64_t g = fma2(add2(jm, twice(-kMagic)), twice(-1.0f / kTab), fs);  // exact
    const uint64_t z = mul2(g, twice(kLn2));
    const uint64_t p = fma2(fma2(z, twice(1.0f / 6.0f), twice(0.5f)), mul2(z, z), z);
    float q0, q1, jm0, jm1, nm0, nm1;
    unpair(fma2(fl, twice(kLn2), p), q0, q1);
    unpair(jm, jm0, jm1);
    unpair(nm, nm0, nm1);
    const float2 a = tab[__float_as_int(jm0) - kMagicBits + kTab / 2], b = tab[__float_as_int(jm1) - kMagicBits + kTab / 2];
    // 2^n: the last bits of nm become the exponent
    const float sc0 = ok0 ? __int_as_float((__float_as_int(nm0) << 23) + 0x3f800000) : 0.0f;
    const float sc1 = ok1 ? __int_as_float((__float_as_int(nm1) << 23) + 0x3f800000) : 0.0f;
    return {pair(a.x * sc0, b.x * sc1), pair(fmaf(a.x, q0, a.y) * sc0, fmaf(b.x, q1, b.y) * sc1)};
}

// Sums of masses, two side by side.  They start at one, which no mass exceeds, so
// a sum's rounding error is what the new mass less the sum's growth leaves.
struct MassSum {
    uint64_t hi, lo;
};
DFLV_DEVINL MassSum no_mass() { return {twice(1.0f), twice(0.0f)}; }
DFLV_DEVINL void add_mass(MassSum& a, const Mass2& m) {
    const uint64_t minus = twice(-1.0f), s = add2(a.hi, m.hi);
    a.lo = add2(a.lo, add2(fma2(fma2(a.hi, minus, s), minus, m.hi), m.lo));
    a.hi = s;
}
// In units of 2^-44: the multiple of 2^-20, then the rest.
DFLV_DEVINL u64 to_units(const Mass& m) {
    const float s = m.hi + m.lo, l = (m.hi - s) + m.lo;
    const int n1 = __float2int_rn(s * 0x1p20f);
    const int n2 = __float2int_rn((fmaf((float)n1, -0x1p-20f, s) + l) * 0x1p44f);
    return (u64)max(((long long)n1 << 24) + n2, 0ll);
}
static_assert(kMassBits == 44, "units of a mass");
DFLV_DEVINL u64 to_units(const MassSum& m) {
    Mass a, b;
    unpair(m.hi, a.hi, b.hi);
    unpair(m.lo, a.lo, b.lo);
    a.hi -= 1.0f;
    b.hi -= 1.0f;
    return to_units(a) + to_units(b);
}
// One token's.  (With an infinite maximum: one, or nothing.)
DFLV_DEVINL u64 mass_of(float x, const Scale& s, const float2* tab) {
    if (x == s.mx) return 1ull << kMassBits;
    const Mass2 m = mass_pair2(x, x, s, tab);
    Mass a;
    float other;
    unpair(m.hi, a.hi, other);
    unpair(m.lo, a.lo, other);
    return to_units(a);
}

// (x - mx) / T - ln(total 2^-44), 1 / T = inv_h + inv_l, rounded once: with y the
// float next to the logarithm, ln(t) = y + (t e^-y - 1) but for 2^-47.  (64-bit
// floating point would take 3 K cycles.)
__device__ __noinline__ float log_share(float x, const Scale& s, float inv_h, float inv_l, u64 total, const float2* tab) {
    const float th = __ull2float_rn(total), tl = __ll2float_rn((long long)(total - (u64)th));
    const float t_h = th * 0x1p-44f, t_l = tl * 0x1p-44f, y = logf(t_h);
    const Mass2 m = mass_pair2(-y, -y, Scale{0.0f, 1.44269502162933349609375f, 1.92596299112661746887e-8f}, tab);
    float e_h, e_l, other;
    unpair(m.hi, e_h, other);
    unpair(m.lo, e_l, other);
    const float p = t_h * e_h;
    const float r = ((p - 1.0f) + fmaf(t_h, e_h, -p)) + fmaf(t_h, e_l, t_l * (e_h + e_l));
    float zh = 0.0f, zl = 0.0f;
    if (x != s.mx) {
        const float dh = x - s.mx, bb = dh - x, dl = (x - (dh - bb)) + (-s.mx - bb);
        zh = dh * inv_h;
        zl = fmaf(dl, inv_h, fmaf(dh, inv_l, fmaf(dh, inv_h, -zh)));
    }
    const float v = zh - y, vb = v - zh, vl = (zh - (v - vb)) + (-y - vb);
    return v + (vl + (zl - r));
}

// Largest of the values of lanes 0 .. 2 kFirst - 1, for every lane.
template <int kFirst>
DFLV_DEVINL u64 max_of(u64 v) {
#pragma unroll
    for (int o = kFirst; o; o >>= 1) {
        const u64 y = __shfl_xor_sync(0xffffffffu, v, o);
        v = y > v ? y : v;
    }
    return __shfl_sync(0xffffffffu, v, 0);
}

DFLV_DEVINL u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A row's parameters, checked and prepared by one thread while the row loads.
struct Params {
    float T, top_p, min_p;
    int top_k, valid;
    float ch, cl;
    u64 w_min, p64, u64_;  // min_p in mass units; top_p and u in units of 2^-64
    float inv_h, inv_l;  // 1 / T as a pair
};

// ceil(m * f) and floor(m * f) of a mass and a fraction in units of 2^-64.
DFLV_DEVINL u64 part_up(u64 m, u64 f) { return __umul64hi(m, f) + (m * f != 0); }
DFLV_DEVINL u64 part_down(u64 m, u64 f) { return __umul64hi(m, f); }

struct Shared {
    uint32_t hist[kBins];  // this CTA's tokens per bin
    u64 list[kList];       // first CTA: candidates, key above, complement of the index below
    u64 mass[kList];       // this CTA's candidates; their masses; the tokens around a cut
    Params par;
    uint32_t n_own, n_tok;
    uint32_t pick_key;
    u64 pick;
    int cut[3];            // bins found: top-k, top-p from, top-p to
    uint32_t cum[3];       // tokens before and up to the top-k bin, up to the last bin
    float scan[kSampWarps][2];
    u64 xchg[2][kSampMaxCluster][kCuts];  // per exchange parity: every CTA's values
    u64 red[kSampWarps][kCuts];
    u64 best[kSampWarps];
    uint32_t least[kSampWarps];
    float2 tab[kTab + 1];
};

DFLV_DEVINL void st_dsmem_u64(uint32_t addr, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;\n" ::"r"(addr), "l"(v) : "memory");
}
DFLV_DEVINL void st_dsmem_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;\n" : : "r"(addr), "r"(v) : "memory");
}
DFLV_DEVINL void st_dsmem_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(addr), "f"(v) : "memory");
}

// The bin of a token: monotone in x, so the bins are in the tokens' order.
struct Bins {
    float mx, scale;
};
DFLV_DEVINL int bin_of(float x, const Bins& bn) {
    if (x == bn.mx) return 0;
    const float t = (bn.mx - x) * bn.scale;
    return t < (float)(kBins - 1) ? (int)t : kBins - 1;
}

// Every CTA contributes K values (the same in all threads below CS); afterwards
// sh.xchg[par][r][k] holds CTA r's value k in every CTA.  Two exchanges in a
// row use different halves, and the barrier of the second separates a half's
// readers from its next writers.
template <int K>
DFLV_DEVINL void exchange(Shared& sh, int& par, const u64 (&v)[K], int CS, int rank) {
    par ^= 1;
    if (CS == 1) {
        if (threadIdx.x == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) sh.xchg[par][0][k] = v[k];
        __syncthreads();
        return;
    }
    if ((int)threadIdx.x < CS) {
        const uint32_t at = map_to_rank(smem_u32(&sh.xchg[par][rank][0]), threadIdx.x);
#pragma unroll
        for (int k = 0; k < K; ++k) st_dsmem_u64(at + 8 * k, v[k]);
    }
    cluster_sync_all();
}

// Sum of the values of lanes 0 .. 7 (16), for every lane.
DFLV_DEVINL u64 sum8(u64 v) {
#pragma unroll
    for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return __shfl_sync(0xffffffffu, v, 0);
}
DFLV_DEVINL u64 sum16(u64 v) {
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return __shfl_sync(0xffffffffu, v, 0);
}
static_assert(kSampWarps == 16 && kSampMaxCluster == 8, "sums over warps and CTAs");

// Block sums of K values, for every thread (order-free: integers).
template <int K>
DFLV_DEVINL void block_sums(Shared& sh, u64 (&v)[K]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = warp_sum(v[k]);
        if (lane == 0) sh.red[warp][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = sum16(lane < kSampWarps ? sh.red[lane][k] : 0ull);
}

template <int K>
DFLV_DEVINL void cluster_sums(Shared& sh, int& par, u64 (&v)[K], int CS, int rank) {
    const int lane = threadIdx.x & 31;
    block_sums(sh, v);
    exchange(sh, par, v, CS, rank);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = sum8(lane < CS ? sh.xchg[par][lane][k] : 0ull);
}

// Turns K values per warp (the same in its lanes) into the sums over the warps of
// the cluster before it, in row order; totals.
template <int K>
DFLV_DEVINL void cluster_exclusive(Shared& sh, int& par, u64 (&v)[K], u64 (&total)[K], int CS, int rank) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane < K) {
        u64 x = v[0];
#pragma unroll
        for (int k = 1; k < K; ++k) x = lane == k ? v[k] : x;
        sh.red[warp][lane] = x;
    }
    __syncthreads();
    u64 all[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const u64 r = lane < kSampWarps ? sh.red[lane][k] : 0ull;
        all[k] = sum16(r);
        v[k] = sum16(lane < warp ? r : 0ull);
    }
    exchange(sh, par, all, CS, rank);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const u64 y = lane < CS ? sh.xchg[par][lane][k] : 0ull;
        total[k] = sum8(y);
        v[k] += sum8(lane < rank ? y : 0ull);
    }
}

// Exclusive sum over the block's threads; total receives the sum.
DFLV_DEVINL u64 block_exclusive(Shared& sh, u64 v, u64& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sh.red[warp][0] = x;
    __syncthreads();
    const u64 r = lane < kSampWarps ? sh.red[lane][0] : 0ull;
    total = sum16(r);
    const u64 base = sum16(lane < warp ? r : 0ull);
    return base + x - v;
}

DFLV_DEVINL uint32_t block_exclusive32(Shared& sh, uint32_t v, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sh.least[warp] = x;
    __syncthreads();
    const uint32_t r = lane < kSampWarps ? sh.least[lane] : 0;
    total = __reduce_add_sync(0xffffffffu, r);
    const uint32_t base = __reduce_add_sync(0xffffffffu, lane < warp ? r : 0);
    return base + x - v;
}

// What is kept: keys above `key`, and of the tokens of that key the first
// `ties` by index (`base`: how many of them lie before this warp's tokens).
struct Keep {
    uint32_t key;
    u64 ties, base;
};

// Which of a lane's four tokens are kept.  The warp's tokens come in row order
// (four a lane, lane by lane); rk counts its tokens of the last key so far.
DFLV_DEVINL void kept4(const float (&x)[4], const Keep& keep, u64& rk, bool (&in)[4]) {
    bool eq[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t key = key_of(x[e]);
        in[e] = key > keep.key;
        eq[e] = key == keep.key;
    }
    if (__any_sync(0xffffffffu, eq[0] || eq[1] || eq[2] || eq[3])) {
        const uint32_t below = (1u << (threadIdx.x & 31)) - 1;
        uint32_t before = 0, all = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t m = __ballot_sync(0xffffffffu, eq[e]);
            before += __popc(m & below);
            all += __popc(m);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (eq[e]) in[e] = rk + before++ < keep.ties;
        rk += all;
    }
}

DFLV_DEVINL void load4(const float* p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
}

// The mass of all of a lane's tokens.
DFLV_DEVINL u64 row_mass(const float* mine, int J, const Scale& sc, const float2* tab) {
    if (isinf(sc.mx)) {
        u64 n = 0;
        for (int j = 0; j < J; ++j) {
            float x[4];
            load4(mine + j * 128, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) n += x[e] == sc.mx;
        }
        return n << kMassBits;
    }
    MassSum m = no_mass();
#pragma unroll 2
    for (int j = 0; j < J; ++j) {
        float x[4];
        load4(mine + j * 128, x);
#pragma unroll
        for (int e = 0; e < 4; e += 2) add_mass(m, mass_pair2(x[e], x[e + 1], sc, tab));
    }
    return to_units(m);
}

// Ascending bitonic sort of a power of two of 64-bit values (all threads).
DFLV_DEVINL void sort_block(u64* v, int n) {
    for (int k = 2; k <= n; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            __syncthreads();
            for (int t = threadIdx.x; t < n >> 1; t += kSampThreads) {
                const int i = ((t & ~(j - 1)) << 1) | (t & (j - 1));
                const u64 a = v[i], b = v[i + j];
                if ((a > b) == ((i & k) == 0)) {
                    v[i] = b;
                    v[i + j] = a;
                }
            }
        }
    __syncthreads();
}

// Narrows [lo, hi] to the key of the last kept token: the largest key whose
// tokens, with `above` (all that come before the interval's), reach `target`
// (a count, or a mass).  Returns the key; `above` becomes the sum over the
// keys strictly above it.  The tokens come from each(f): f(x) for every token
// of this thread that may lie in the interval.
template <bool kMass, typename Each>
DFLV_DEVINL uint32_t find_key(Shared& sh, int& par, const Scale& sc, uint32_t lo, uint32_t hi, u64 target, u64& above,
                              int CS, int rank, Each each) {
    while (lo < hi) {
        const uint32_t step = (hi - lo) / kCuts + 1;  // kCuts * step > hi - lo
        u64 a[kCuts];
#pragma unroll
        for (int k = 0; k < kCuts; ++k) a[k] = 0;
        each([&](float x) {
            const uint32_t key = key_of(x);
            if (key < lo || key > hi) return;
            const u64 w = kMass ? mass_of(x, sc, sh.tab) : 1ull;
            const uint32_t off = hi - key;
            // a[k]: tokens with key > hi - (k + 1) step
#pragma unroll
            for (int k = 0; k < kCuts; ++k) a[k] += (u64)off < (u64)(k + 1) * step ? w : 0ull;
        });
        cluster_sums(sh, par, a, CS, rank);
        int k = 0;
        u64 under = 0;  // sum above part k
#pragma unroll
        for (int q = 0; q < kCuts; ++q)
            if (q < kCuts - 1 && (u64)(q + 1) * step <= (u64)(hi - lo) && above + a[q] < target) {
                k = q + 1;
                under = a[q];
            }
        above += under;
        const u64 bottom = (u64)(k + 1) * step;
        const uint32_t nlo = bottom > (u64)(hi - lo) ? lo : hi - (uint32_t)bottom + 1;
        hi -= (uint32_t)k * step;
        lo = nlo;
    }
    return lo;
}

// What the CTAs of a cluster read of each other's counts takes time (64 KB of
// them 3 K cycles), so a CTA sums a part of the bins and tells the others.

// A bin's tokens, and their mean position in it in units of 2^-13, rounded down.
constexpr int kPosBits = 13;
struct BinCount {
    uint32_t n, pos;
};
DFLV_DEVINL uint32_t pack_bin(uint32_t n, uint32_t q, float inv_q) {
    const float f = n ? (float)q * inv_q / (float)n : 0.0f;
    return n | ((uint32_t)(f * ((1 << kPosBits) * (1.0f - 0x1p-20f))) << (32 - kPosBits));
}
static_assert(400000 + kSampMaxCluster * kSampWarps * 128 < 1 << (32 - kPosBits), "tokens of a row");

// The cluster's tokens in this thread's four bins, once every CTA has counted.
// A CTA's counts hold the tokens below and the sum of their positions (inv_q
// each) above bit 16.
DFLV_DEVINL void read_hist(Shared& sh, int CS, int rank, float inv_q, BinCount (&out)[4]) {
    const int tid = threadIdx.x;
    uint32_t* sums = reinterpret_cast<uint32_t*>(sh.mass);
    static_assert(sizeof(sh.mass) == kBins * 4, "a sum a bin");
    uint4 v;
    if (CS > 1) {
        cluster_sync_all();
        const int per = kBins / CS;  // (CS is a power of two)
        for (int t = rank * per + tid; t < (rank + 1) * per; t += kSampThreads) {
            const uint32_t here = smem_u32(&sh.hist[t]), there = smem_u32(&sums[t]);
            uint32_t part[kSampMaxCluster], n = 0, q = 0;
#pragma unroll
            for (int r = 0; r < kSampMaxCluster; ++r) part[r] = (uint32_t)ld_dsmem_s32(map_to_rank(here, r & (CS - 1)));
#pragma unroll
            for (int r = 0; r < kSampMaxCluster; ++r)
                if (r < CS) {
                    n += part[r] & 0xffffu;
                    q += part[r] >> 16;
                }
            n = pack_bin(n, q, inv_q);
            for (int r = 0; r < CS; ++r) st_dsmem_u32(map_to_rank(there, r), n);
        }
        cluster_sync_all();
        v = *reinterpret_cast<const uint4*>(&sums[4 * tid]);
    } else {
        __syncthreads();
        v = *reinterpret_cast<const uint4*>(&sh.hist[4 * tid]);
        v = make_uint4(pack_bin(v.x & 0xffffu, v.x >> 16, inv_q), pack_bin(v.y & 0xffffu, v.y >> 16, inv_q),
                       pack_bin(v.z & 0xffffu, v.z >> 16, inv_q), pack_bin(v.w & 0xffffu, v.w >> 16, inv_q));
    }
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) out[k] = {x[k] & ((1u << (32 - kPosBits)) - 1), x[k] >> (32 - kPosBits)};
}

// As many counts as threads: the cluster's tokens in this thread's.  (A CTA's
// counts are next written or left after a later barrier.)
DFLV_DEVINL uint32_t read_counts(Shared& sh, int CS) {
    const int tid = threadIdx.x;
    if (CS == 1) {
        __syncthreads();
        return sh.hist[tid];
    }
    cluster_sync_all();
    const uint32_t here = smem_u32(&sh.hist[tid]);
    uint32_t part[kSampMaxCluster], n = 0;
#pragma unroll
    for (int q = 0; q < kSampMaxCluster; ++q) part[q] = (uint32_t)ld_dsmem_s32(map_to_rank(here, q & (CS - 1)));
#pragma unroll
    for (int q = 0; q < kSampMaxCluster; ++q) n += q < CS ? part[q] : 0;
    return n;
}

// Turns a thread's two values into the sums of the threads before it; totals.
DFLV_DEVINL void scan_pair(Shared& sh, float& lo, float& hi, float& lo_all, float& hi_all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float lo_x = lo, hi_x = hi;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, lo_x, o), z = __shfl_up_sync(0xffffffffu, hi_x, o);
        if (lane >= o) {
            lo_x += y;
            hi_x += z;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sh.scan[warp][0] = lo_x;
        sh.scan[warp][1] = hi_x;
    }
    __syncthreads();
    // (the same order of additions in every thread)
    float lo_w = lane < kSampWarps ? sh.scan[lane][0] : 0.0f, hi_w = lane < kSampWarps ? sh.scan[lane][1] : 0.0f;
#pragma unroll
    for (int o = 1; o < kSampWarps; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, lo_w, o), z = __shfl_up_sync(0xffffffffu, hi_w, o);
        if (lane >= o) {
            lo_w += y;
            hi_w += z;
        }
    }
    lo_all = __shfl_sync(0xffffffffu, lo_w, kSampWarps - 1);
    hi_all = __shfl_sync(0xffffffffu, hi_w, kSampWarps - 1);
    const float lo_p = __shfl_sync(0xffffffffu, lo_w, max(warp - 1, 0)), hi_p = __shfl_sync(0xffffffffu, hi_w, max(warp - 1, 0));
    const float lo_b = warp ? lo_p : 0.0f, hi_b = warp ? hi_p : 0.0f;
    lo = lo_b + (lo_x - lo);
    hi = hi_b + (hi_x - hi);
}

// grid rows * CS, clusters of CS CTAs: a cluster per row.  Warp w of CTA r
// owns the 128 J consecutive tokens from (r * 16 + w) * 128 J, four a lane at a
// time, so a pass is conflict-free 16-byte reads and sums are in row order by
// warp.
template <typename T>
__global__ void __launch_bounds__(kSampThreads, 2) sample_kernel(const SampleArgs a, int CS, int J, int ahead) {
    extern __shared__ __align__(16) float row_s[];
    __shared__ __align__(16) Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = CS > 1 ? (int)cluster_ctarank() : 0;
    if (CS > 1) cluster_arrive_relaxed();  // paired with the wait before the first exchange
    const long long r = blockIdx.x / CS;
    const int b = (int)(r / a.N_max), node = (int)(r - (long long)b * a.N_max);
    if (tid <= kTab) sh.tab[tid] = make_float2(kExpTable.hi[tid], kExpTable.lo[tid]);
    *reinterpret_cast<uint4*>(&sh.hist[4 * tid]) = make_uint4(0, 0, 0, 0);
    if (tid == 0) {
        sh.n_own = 0;
        sh.cut[1] = sh.cut[2] = kBins - 1;
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (a.n_nodes) {  // uniform over the cluster
        const int n = __ldg(a.n_nodes + b);
        const bool bad = n < 0 || n > a.N_max;
        if (bad || node >= n) {
            if (bad && node == 0 && rank == 0 && tid == 0) raise_status(a.status, DFLV_DEV_TOPOLOGY);
            if (CS > 1) cluster_wait();
            return;
        }
    }
    if (tid == kSampThreads - 1) {
        Params q;
        q.T = __ldg(a.temperature + b);
        q.top_p = __ldg(a.top_p + b);
        q.min_p = __ldg(a.min_p + b);
        const float u = __ldg(a.u + r);
        q.top_k = __ldg(a.top_k + b);
        q.valid = q.T >= 0.0f && q.T < INFINITY && q.top_p >= 0.0f && q.min_p >= 0.0f && q.min_p <= 1.0f &&
                  u >= 0.0f && u < 1.0f;
        // (log2(e) 2^127 is the largest that a float holds of it)
        const double inv = 1.0 / fmax((double)q.T, 0x1p-127), c = 1.4426950408889634074 * inv;
        q.inv_h = (float)inv;
        q.inv_l = (float)(inv - (double)q.inv_h);
        q.ch = (float)c;
        q.cl = (float)(c - (double)q.ch);
        q.w_min = (u64)ceil((double)q.min_p * (double)(1ull << kMassBits));
        q.p64 = q.valid && q.top_p < 1.0f ? __float2ull_rz(q.top_p * 18446744073709551616.0f) : 0;
        q.u64_ = q.valid ? __float2ull_rz(u * 18446744073709551616.0f) : 0;
        sh.par = q;
    }
    // ---- the row into shared memory, its largest logit and its smallest
    // above -infinity
    const int w_len = 128 * J, c0 = rank * kSampWarps * w_len;
    const int first = c0 + warp * w_len;                       // of this warp
    const int n_own = max(0, min(a.V - first, w_len));
    float* xs = row_s + warp * w_len;
    const T* row = reinterpret_cast<const T*>(a.logits) + r * a.ld + first;
    if (ahead && lane == 0 && n_own > 0 && r + ahead < (long long)a.B * a.N_max) {
        // the row this cluster's successor on the SMs will read goes to the L2
        const T* next = row + (long long)ahead * a.ld;
        const uint32_t bytes = (uint32_t)(n_own * sizeof(T)) & ~15u;
        if ((reinterpret_cast<uintptr_t>(next) & 15) == 0 && bytes) prefetch_l2_bulk(next, bytes);
    }
    float bv = -INFINITY, lv = INFINITY;
    int bi = 0x7fffffff;
    auto take = [&](float v, int i) {
        v = canonical(v);
        if (v > bv) {  // indices ascend: the first of equals stays
            bv = v;
            bi = first + i;
        }
        if (v > -INFINITY) lv = fminf(lv, v);
        return v;
    };
    if ((reinterpret_cast<uintptr_t>(row) & (4 * sizeof(T) - 1)) == 0) {
        struct alignas(4 * sizeof(T)) Four {
            T v[4];
        };
        constexpr int U = 5;
        for (int j0 = 0; j0 < J; j0 += U) {
            Four x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = (j0 + u) * 128 + lane * 4;
                if (i + 4 <= n_own) {
                    if constexpr (sizeof(T) == 4) {
                        const float4 y = __ldcs(reinterpret_cast<const float4*>(row + i));
                        x[u] = *reinterpret_cast<const Four*>(&y);
                    } else {
                        const uint2 y = __ldcs(reinterpret_cast<const uint2*>(row + i));
                        x[u] = *reinterpret_cast<const Four*>(&y);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = (j0 + u) * 128 + lane * 4;
                if (j0 + u >= J) break;
                float4 y = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (i + 4 <= n_own) {
                    y.x = take(to_float<T>(x[u].v[0]), i);
                    y.y = take(to_float<T>(x[u].v[1]), i + 1);
                    y.z = take(to_float<T>(x[u].v[2]), i + 2);
                    y.w = take(to_float<T>(x[u].v[3]), i + 3);
                } else {
                    if (i < n_own) y.x = take(to_float<T>(row[i]), i);
                    if (i + 1 < n_own) y.y = take(to_float<T>(row[i + 1]), i + 1);
                    if (i + 2 < n_own) y.z = take(to_float<T>(row[i + 2]), i + 2);
                }
                *reinterpret_cast<float4*>(xs + i) = y;
            }
        }
    } else {
        // One token at a time, without the loads in flight above: three rows of four
        // where V is odd.  64 rows of bf16, no filter: 24.0 us with 50,257 tokens, 15.0
        // with 50,256; fp32 27.6 and 16.0.
        for (int i = lane; i < w_len; i += 32) xs[i] = i < n_own ? take(to_float<T>(row[i]), i) : -INFINITY;
    }
    // largest key, then lowest index
    u64 best = ((u64)key_of(bv) << 32) | (uint32_t)~bi;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const u64 y = __shfl_xor_sync(0xffffffffu, best, o);
        best = y > best ? y : best;
    }
    const uint32_t least = __reduce_min_sync(0xffffffffu, key_of(lv));
    if (lane == 0) {
        sh.best[warp] = best;
        sh.least[warp] = least;
    }
    __syncthreads();
    u64 one[2] = {max_of<8>(lane < kSampWarps ? sh.best[lane] : 0ull),
                  __reduce_min_sync(0xffffffffu, lane < kSampWarps ? sh.least[lane] : 0xffffffffu)};
    int par = 0;
    if (CS > 1) cluster_wait();  // every CTA has started: its shared memory exists
    exchange(sh, par, one, CS, rank);
    best = max_of<4>(lane < CS ? sh.xchg[par][lane][0] : 0ull);
    const uint32_t key_min = __reduce_min_sync(0xffffffffu, lane < CS ? (uint32_t)sh.xchg[par][lane][1] : 0xffffffffu);
    const uint32_t key_max = (uint32_t)(best >> 32);
    const float mx = float_of(key_max);

    const Params& pr = sh.par;
    const bool valid = pr.valid && key_max > kKeyNegInf;
    if (!valid || pr.T == 0.0f) {
        if (rank == 0 && tid == 0) {
            if (!valid) raise_status(a.status, DFLV_DEV_SAMPLE);
            a.drawn[r] = key_max > kKeyNegInf ? (int)~(uint32_t)best : 0;
            if (a.logp) a.logp[r] = 0.0f;
        }
        return;  // uniform over the cluster
    }
    const Scale sc = {mx, pr.ch, pr.cl};
    const int top_k = pr.top_k;
    const float top_p = pr.top_p;
    const u64 w_min = pr.w_min;
    const float* mine = xs + lane * 4;
    auto store = [&](int t, float x, u64 total) {
        a.drawn[r] = t;
        if (a.logp) {
            a.logp[r] = log_share(x, sc, pr.inv_h, pr.inv_l, total, sh.tab);
        }
    };

    // ---- thresholds
    Keep keep = {kKeyNegInf + 1, ~0ull, 0};  // everything above -infinity
    // `ties` of the tokens of `key` are kept: count those before this warp
    auto set_keep = [&](uint32_t key, u64 ties) {
        uint32_t n = 0;
        for (int j = 0; j < J; ++j) {
            float x[4];
            load4(mine + j * 128, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) n += key_of(x[e]) == key;
        }
        u64 base[1] = {__reduce_add_sync(0xffffffffu, n)}, all[1];
        cluster_exclusive(sh, par, base, all, CS, rank);
        if (key == keep.key && keep.ties < ties) ties = keep.ties;
        keep = {key, ties, base[0]};
    };
    // Few candidates: those of bins up to b_end go to one CTA, which decides.
    // False (in all threads) if they are more than kList.  want_all: the mass of
    // the whole row is what top-p takes its part of; cut_k: top_k counts.
    auto compact = [&](int b_end, bool want_all, bool cut_k, const Bins& bn) -> bool {
        const bool cut_p = top_p < 1.0f;
        const float lim = b_end == kBins - 1 ? INFINITY : (float)(b_end + 1);
        // each CTA's own, in its shared memory
#pragma unroll 2
        for (int j = 0; j < J; ++j) {
            float x[4];
            load4(mine + j * 128, x);
            uint32_t n = 0;
            bool in[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // (bin_of(x) <= b_end; NaN: x and the maximum both infinite)
                in[e] = x[e] > -INFINITY && !((mx - x[e]) * bn.scale >= lim);
                n += in[e];
            }
            if (n) {
                uint32_t at = atomicAdd(&sh.n_own, n);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    // descending logit, then ascending index
                    if (in[e]) {
                        if (at < (uint32_t)kList)
                            sh.mass[at] = ((u64)~key_of(x[e]) << 32) | (uint32_t)(first + j * 128 + lane * 4 + e);
                        ++at;
                    }
            }
        }
        u64 all[1] = {0};
        if (want_all) {
            all[0] = row_mass(mine, J, sc, sh.tab);
            block_sums(sh, all);
        } else {
            __syncthreads();
        }
        // ... then to the first CTA, each to its part of the list, with the
        // counts and masses to all
        constexpr uint32_t kPart = kList / kSampMaxCluster;
        const uint32_t own = sh.n_own;
        if (CS > 1) {
            if (own <= kPart) {
                const uint32_t l0 = map_to_rank(smem_u32(&sh.list[rank * kPart]), 0);
                if (tid < (int)own) st_dsmem_u64(l0 + 8 * tid, sh.mass[tid]);
            }
        } else {
            for (uint32_t i = tid; i < min(own, (uint32_t)kList); i += kSampThreads) sh.list[i] = sh.mass[i];
        }
        const u64 mine2[2] = {own, all[0]};
        exchange(sh, par, mine2, CS, rank);
        const uint32_t n_q = lane < CS ? (uint32_t)sh.xchg[par][lane][0] : 0;
        if (__any_sync(0xffffffffu, n_q > (CS > 1 ? kPart : (uint32_t)kList))) return false;  // the same in all CTAs
        all[0] = sum8(lane < CS ? sh.xchg[par][lane][1] : 0ull);
        const int n = (int)__reduce_add_sync(0xffffffffu, n_q);
        if (CS > 1) {
            // (a CTA leaves only after the others have read its bins: their
            // arrival at the exchange says so)
            if (rank != 0) return true;
            // the parts close up
            u64 mine1[2];
            int to[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int i = tid + q * kSampThreads, r1 = i / (int)kPart, k = i % (int)kPart;
                const uint32_t before = __reduce_add_sync(0xffffffffu, lane < r1 ? n_q : 0);
                to[q] = k < (int)__shfl_sync(0xffffffffu, n_q, r1) ? (int)before + k : -1;
                mine1[q] = to[q] >= 0 ? sh.list[i] : 0ull;
            }
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (to[q] >= 0) sh.list[to[q]] = mine1[q];
        }
        __syncthreads();
        if (n <= kSampThreads / 2) {
            // each candidate against all others: its rank, the mass before
            // it, then the kept mass before it by index.  G threads share
            // a candidate.
            int G = 1;
            while (G < 32 && G * 2 * n <= kSampThreads) G *= 2;
            const int i = tid / G, part = tid % G;
            const bool live = i < n;
            const u64 e = live ? sh.list[i] : ~0ull;
            const float x = float_of(~(uint32_t)(e >> 32));
            const u64 w = live ? mass_of(x, sc, sh.tab) : 0ull;
            if (live && part == 0) sh.mass[i] = w;
            __syncthreads();
            uint32_t rk = 0;
            u64 before = 0;
            if (live)
                for (int q = part; q < n; q += G)
                    if (sh.list[q] < e) {
                        ++rk;
                        before += sh.mass[q];
                    }
            for (int o = G >> 1; o; o >>= 1) {
                rk += __shfl_xor_sync(0xffffffffu, rk, o);
                before += __shfl_xor_sync(0xffffffffu, before, o);
            }
            u64 total[1] = {live && part == 0 && (!cut_k || rk < (uint32_t)top_k) ? w : 0ull};
            bool kept = live && (!cut_k || rk < (uint32_t)top_k) && w >= w_min && w > 0;
            if (cut_p) {
                if (!want_all) block_sums(sh, total);
                const u64 target = part_up(want_all ? all[0] : total[0], pr.p64);
                kept = kept && before < (target < 1 ? 1 : target);
            }
            total[0] = kept && part == 0 ? w : 0ull;
            block_sums(sh, total);  // (everyone has read the masses)
            if (live && part == 0 && !kept) sh.mass[i] = 0;
            __syncthreads();
            u64 at = 0;
            if (live)
                for (int q = part; q < n; q += G)
                    if ((uint32_t)sh.list[q] < (uint32_t)e) at += sh.mass[q];
            for (int o = G >> 1; o; o >>= 1) at += __shfl_xor_sync(0xffffffffu, at, o);
            const u64 draw = part_down(total[0], pr.u64_);
            if (kept && part == 0 && at <= draw && draw < at + w) store((int)(uint32_t)e, x, total[0]);
            return true;
        }
        int n2 = 32;
        while (n2 < n) n2 <<= 1;
        for (int i = n + tid; i < n2; i += kSampThreads) sh.list[i] = ~0ull;
        sort_block(sh.list, n2);
        // two ranks a thread: masses and their running sums
        u64 e[2], w[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int i = 2 * tid + q;
            e[q] = i < n ? sh.list[i] : ~0ull;
            w[q] = i < n && (!cut_k || i < top_k) ? mass_of(float_of(~(uint32_t)(e[q] >> 32)), sc, sh.tab) : 0ull;
        }
        u64 total;
        const u64 before = block_exclusive(sh, w[0] + w[1], total);
        u64 target = ~0ull;
        if (cut_p) {
            target = part_up(want_all ? all[0] : total, pr.p64);
            if (target < 1) target = 1;
        }
        if (w[1] < w_min || before + w[0] >= target) w[1] = 0;
        if (w[0] < w_min || before >= target) w[0] = 0;
        // the kept tokens by index; the keys stay with the masses' places
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int i = 2 * tid + q;
            if (i < n2) {
                sh.mass[i] = w[q];
                sh.hist[i] = ~(uint32_t)(e[q] >> 32);
                sh.list[i] = w[q] ? ((u64)(uint32_t)e[q] << 32) | (uint32_t)i : ~0ull;
            }
        }
        sort_block(sh.list, n2);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int i = 2 * tid + q;
            e[q] = i < n2 ? sh.list[i] : ~0ull;
            w[q] = e[q] != ~0ull ? sh.mass[(uint32_t)e[q]] : 0ull;
        }
        u64 at = block_exclusive(sh, w[0] + w[1], total);
        const u64 draw = part_down(total, pr.u64_);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (w[q] && at <= draw && draw < at + w[q])
                store((int)(e[q] >> 32), float_of(sh.hist[(uint32_t)e[q]]), total);
            at += w[q];
        }
        return true;
    };
    bool found = false;  // the draw's warp is known
    u64 at = 0, own = 0, total = 0;
    Bins bn = {mx, 0.0f};
    if ((top_k > 0 && top_k < a.V) || top_p < 1.0f || pr.min_p > 0.0f) {
        // ---- tokens per bin.  The bins span the row's finite logits, at most
        // kOctaves of mass.
        const float c = sc.ch, range = mx - float_of(key_min);
        bn.scale = c * ((kBins - 1) / kOctaves);
        if (range > 0.0f && range < INFINITY) bn.scale = fmaxf(bn.scale, (kBins - 1) / range);
        // (four times it is finite: the count and the later passes bin alike)
        bn.scale = fminf(bn.scale, 0x1p125f);
        const bool cut_p = top_p < 1.0f;
        // The bin of the last wanted maximum and what min_p leaves of it.
        auto cut_min_p = [&](int b_end) {
            const float e = -log2f(pr.min_p) * bn.scale / c * (1.0f + 1e-4f) + 1.0f;
            return pr.min_p > 0.0f && e < (float)b_end ? (int)e : b_end;
        };
        if (top_k > 0 && top_k <= kList / 2 && top_k * 4 <= CS * kSampThreads) {
            // A small top_k: the lanes' own maxima alone, four bins in one.  The
            // bin that holds the top_k-th largest of them holds the top_k-th
            // largest token or one below it.
            if (bv > -INFINITY) atomicAdd(&sh.hist[bin_of(bv, bn) >> 2], 1u);
            if (tid == 0) sh.cut[0] = -1;
            uint32_t lanes;
            const uint32_t n = read_counts(sh, CS);
            const uint32_t before = block_exclusive32(sh, n, lanes);
            if (before < (uint32_t)top_k && before + n >= (uint32_t)top_k) sh.cut[0] = 4 * tid + 3;
            __syncthreads();
            const int b_k = sh.cut[0];
            if (b_k >= 0 && compact(cut_p ? b_k : cut_min_p(b_k), false, true, bn)) return;
            // too many of them, or too few lanes: all tokens
            if (CS > 1) cluster_sync_all();
            *reinterpret_cast<uint4*>(&sh.hist[4 * tid]) = make_uint4(0, 0, 0, 0);
            if (tid == 0) sh.n_own = 0;
            __syncthreads();
        }
        // With its count a bin sums, in its upper half, the quarter of the bin
        // that each token lies in (the half of it where a CTA has more tokens than
        // 16 bits hold the quarters of).
        const int q_bits = J <= 10 ? 2 : 1;
        static_assert(10 * kSampWarps * 128 * 3 < 65536 && 400000 / kSampMaxCluster + kSampWarps * 128 < 65536, "16 bits");
        {
            const float fine = bn.scale * (float)(1 << q_bits);  // (a power of two: no other rounding)
            const int last = (kBins - 1) << q_bits;
#pragma unroll 2
            for (int j = 0; j < J; ++j) {
                float x[4];
                load4(mine + j * 128, x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float t = x[e] == mx ? 0.0f : (mx - x[e]) * fine;
                    const int i = t < (float)last ? (int)t : last;
                    if (x[e] > -INFINITY)
                        atomicAdd(&sh.hist[i >> q_bits], 1u + ((uint32_t)(i & ((1 << q_bits) - 1)) << 16));
                }
            }
        }
        BinCount bins4[4];
        uint32_t n4[4], n_all;
        read_hist(sh, CS, rank, 1.0f / (float)(1 << q_bits), bins4);
#pragma unroll
        for (int q = 0; q < 4; ++q) n4[q] = bins4[q].n;
        const uint32_t n_before = block_exclusive32(sh, n4[0] + n4[1] + n4[2] + n4[3], n_all);
        const bool cut_k = top_k > 0 && (uint32_t)top_k < n_all;
        // the top-k bin, and what the bins hold after that cut
        uint32_t left[4];
        {
            uint32_t before = n_before;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                left[q] = n4[q];
                if (cut_k) {
                    if (before < (uint32_t)top_k && before + n4[q] >= (uint32_t)top_k) {
                        sh.cut[0] = 4 * tid + q;
                        sh.cum[0] = before;
                        sh.cum[1] = before + n4[q];
                    }
                    left[q] = before >= (uint32_t)top_k ? 0 : min(n4[q], (uint32_t)top_k - before);
                }
                before += n4[q];
            }
        }
        if (cut_k) __syncthreads();
        const int b_k = cut_k ? sh.cut[0] : kBins - 1;
        bool few = cut_k && sh.cum[1] <= (uint32_t)kList;  // (the same in all threads)
        const bool bounds = cut_p && !few;
        if (bounds) {
            // Mass of a bin of n tokens that lie at f_i in [0, 1) of it, counted to
            // the 1 / Q below: e^-x is convex, so with d the bin's octaves
            //   n 2^-(d mean f) <= sum 2^-(d f_i) <= n - (1 - 2^-d) sum f_i.
            // (A bin that top-k cuts: all at its near or its far edge.)  The margins
            // cover the rounding of the bins, of exp2f and of these fp32 sums.
            const float oct = c / bn.scale, inv_q = 1.0f / (float)(1 << q_bits), slope = 1.0f - exp2f(-oct);
            float lo4[4], hi4[4], lo_b = 0.0f, hi_b = 0.0f, lo_all, hi_all;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int bin = 4 * tid + q;
                const bool whole = left[q] == n4[q] && bin < kBins - 1;
                const float n = (float)left[q], unit = 1.0f / (1 << kPosBits);
                const float f = whole ? (float)bins4[q].pos * unit : 0.0f;
                const float f_top = whole ? ((float)bins4[q].pos + 1.02f) * unit + inv_q : 1.0f;
                hi4[q] = left[q] ? n * (1.0f - slope * f) * exp2f(-(float)bin * oct) * (1.0f + 3e-5f) : 0.0f;
                lo4[q] = left[q] && bin < kBins - 1 ? n * exp2f(-((float)bin + f_top) * oct) * (1.0f - 3e-5f) : 0.0f;
                lo_b += lo4[q];
                hi_b += hi4[q];
            }
            // the cut lies behind the bins whose mass is surely too small, and
            // in or before the first whose mass surely suffices
            scan_pair(sh, lo_b, hi_b, lo_all, hi_all);
            const float need_lo = top_p * lo_all * (1.0f - 1e-5f), need_hi = top_p * hi_all * (1.0f + 1e-5f);
            int from = kBins, to = kBins - 1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                hi_b += hi4[q];
                lo_b += lo4[q];
                if (from == kBins && left[q] && hi_b * (1.0f + 1e-5f) >= need_lo) from = 4 * tid + q;
                if (to == kBins - 1 && left[q] && lo_b * (1.0f - 1e-5f) >= need_hi) to = 4 * tid + q;
            }
            if (from < kBins) atomicMin(&sh.cut[1], from);
            if (to < kBins - 1) atomicMin(&sh.cut[2], to);
            __syncthreads();
        }
        const int p_from = bounds ? min(sh.cut[1], b_k) : 0, p_to = min(sh.cut[2], b_k);
        int b_end = cut_p && !cut_k ? p_to : b_k;
        if (!(cut_p && cut_k)) b_end = cut_min_p(b_end);
        if (!few) {
            uint32_t before = n_before;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                before += n4[q];
                if (4 * tid + q == b_end) sh.cum[2] = before;
            }
            __syncthreads();
            few = sh.cum[2] <= (uint32_t)kList;
        }
        if (few) {
            if (compact(b_end, cut_p && !cut_k, cut_k, bn)) return;
            // (too many in one CTA's part: as if they were many)
            if (CS > 1) cluster_sync_all();
        }
        // ---- many candidates: the cuts by key.  A bin's keys lie within one
        // bin of its edges.
        auto key_below = [&](int bin) {
            return bin == kBins - 1 ? kKeyNegInf + 1 : max(key_of(mx - (float)(bin + 2) / bn.scale), kKeyNegInf + 1);
        };
        auto key_above = [&](int bin) { return key_of(bin < 1 ? mx : fminf(mx, mx - (float)(bin - 1) / bn.scale)); };
        // The tokens of bins [b0, b1] that are kept so far go, as values, to their
        // warp's part of a list if they fit there (the usual case); else every later
        // pass goes over the warp's tokens again.
        float* near = reinterpret_cast<float*>(sh.list);
        // (the list's end takes the last few tokens of all CTAs, kTok of each)
        constexpr int kTok = kSampThreads / kSampMaxCluster;
        constexpr int kNear = (sizeof(sh.list) / 4 + sizeof(sh.mass) / 4 - kTok * kSampMaxCluster) / kSampWarps;
        float* tok = near + kNear * kSampWarps;
        near += warp * kNear;
        int n_near = 0;
        u64 before = 0;  // mass of this lane's kept tokens before bin b0
        static_assert(offsetof(Shared, mass) == offsetof(Shared, list) + sizeof(sh.list), "one array");
        auto collect = [&](int b0, int b1, u64 (&m)[2], auto masses) {
            // masses: also sum what is kept, and its part before bin b0
            constexpr bool kMasses = decltype(masses)::value;
            __syncthreads();  // (the list has been read)
            n_near = 0;
            u64 rk = keep.base;
            MassSum all = no_mass(), first_part = no_mass();
            uint32_t tops = 0;
            const bool all_kept = keep.key == kKeyNegInf + 1 && keep.ties == ~0ull, inf = isinf(mx);
            // as bin_of: bin < b0 where (mx - x) scale < b0 (a distance that overflows
            // has no mass)
            const float lim0 = (float)b0, lim1 = b1 == kBins - 1 ? INFINITY : (float)(b1 + 1);
            for (int j = 0; j < J; ++j) {
                float x[4];
                load4(mine + j * 128, x);
                bool low[4], near4[4];
                if (!all_kept || inf) {
                    bool in[4];
                    kept4(x, keep, rk, in);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        tops += in[e] && x[e] == mx;
                        x[e] = in[e] ? x[e] : -INFINITY;
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float t = (mx - x[e]) * bn.scale;
                    if (inf) t = x[e] == mx ? 0.0f : INFINITY;
                    low[e] = t < lim0;
                    near4[e] = !low[e] && t < lim1;
                }
                if (kMasses && !inf) {
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        Mass2 w = mass_pair2(x[e], x[e + 1], sc, sh.tab);
                        add_mass(all, w);
                        float h0, h1, l0, l1;
                        unpair(w.hi, h0, h1);
                        unpair(w.lo, l0, l1);
                        w.hi = pair(low[e] ? h0 : 0.0f, low[e + 1] ? h1 : 0.0f);
                        w.lo = pair(low[e] ? l0 : 0.0f, low[e + 1] ? l1 : 0.0f);
                        add_mass(first_part, w);
                    }
                }
                // (a lane has one of them as a rule)
                uint32_t mine4 = (near4[0] ? 1u : 0u) | (near4[1] ? 2u : 0u) | (near4[2] ? 4u : 0u) | (near4[3] ? 8u : 0u);
                for (uint32_t who = __ballot_sync(0xffffffffu, mine4); who; who = __ballot_sync(0xffffffffu, mine4)) {
                    const int to = n_near + __popc(who & ((1u << lane) - 1));
                    const float y = mine4 & 1 ? x[0] : mine4 & 2 ? x[1] : mine4 & 4 ? x[2] : x[3];
                    if (mine4 && to < kNear) near[to] = y;
                    mine4 &= mine4 - 1;
                    n_near += __popc(who);
                }
            }
            if (kMasses) {
                // (with an infinite maximum only its tokens, in bin 0, have a mass)
                const u64 t44 = (u64)tops << kMassBits;
                before = inf ? (b0 > 0 ? t44 : 0ull) : to_units(first_part);
                m[0] = inf ? t44 : to_units(all);
                m[1] = before;
            }
            __syncthreads();
        };
        // f(x) for the tokens of bins [b0, b1] kept so far
        auto each_near = [&](int b0, int b1, auto f) {
            if (n_near <= kNear) {
                for (int i = lane; i < n_near; i += 32) f(near[i]);
            } else {
                u64 rk = keep.base;
                for (int j = 0; j < J; ++j) {
                    float x[4];
                    bool in[4];
                    load4(mine + j * 128, x);
                    kept4(x, keep, rk, in);
#pragma unroll 1
                    for (int e = 0; e < 4; ++e) {
                        const int bin = bin_of(x[e], bn);
                        if (in[e] && bin >= b0 && bin <= b1) f(x[e]);
                    }
                }
            }
        };
        // The last kept token's key among those tokens: `above` (all before
        // their bins) becomes the sum over the keys strictly above it.
        auto find_cut = [&](auto mass, int b0, int b1, uint32_t lo, u64 target, u64& above) -> uint32_t {
            constexpr bool kMass = decltype(mass)::value;
            const uint32_t hi = key_above(b0);
            auto each = [&](auto f) { each_near(b0, b1, f); };
            // A second, finer count of these tokens alone.
            const float top = float_of(hi), width = top - float_of(lo);
            if (width > 0.0f && width < INFINITY) {
                constexpr int kFine = kSampThreads;
                const float scale = fminf((kFine - 1) / width, 3e38f);
                auto fine_of = [&](float x) {
                    const float t = (top - x) * scale;
                    return t < (float)(kFine - 1) ? (int)t : kFine - 1;
                };
                sh.hist[tid] = 0;
                if (tid == 0) sh.cut[1] = sh.cut[2] = kFine - 1;
                __syncthreads();
                each([&](float x) { atomicAdd(&sh.hist[fine_of(x)], 1u); });
                const uint32_t count = read_counts(sh, CS);
                // bounds of the sums up to each bin; a count is exact
                const float n = (float)count, t = (float)tid / scale, t1 = (float)(tid + 1) / scale;
                float hi_1 = !count ? 0.0f : kMass ? n * exp2f(((top - mx) - t) * sc.ch) * (1.0f + 3e-5f) : n;
                float lo_1 = !count ? 0.0f : kMass ? n * exp2f(((top - mx) - t1) * sc.ch) * (1.0f - 3e-5f) : n;
                if (kMass && tid == kFine - 1) lo_1 = 0.0f;
                float lo_b = lo_1, hi_b = hi_1, lo_all, hi_all;
                scan_pair(sh, lo_b, hi_b, lo_all, hi_all);
                const float need = (float)(target - above) * (kMass ? 1.0f / (float)(1ull << kMassBits) : 1.0f);
                const float need_lo = need * (1.0f - 1e-5f), need_hi = need * (1.0f + 1e-5f);
                if (count && (hi_b + hi_1) * (1.0f + 1e-5f) >= need_lo) atomicMin(&sh.cut[1], tid);
                if (count && (lo_b + lo_1) * (1.0f - 1e-5f) >= need_hi) atomicMin(&sh.cut[2], tid);
                __syncthreads();
                const int f0 = sh.cut[1], f1 = sh.cut[2];
                // the sum before these bins, and their tokens to every CTA
                if (tid == 0) {
                    sh.n_tok = 0;
                    sh.pick_key = 0;
                }
                __syncthreads();
                u64 v[1] = {0};
                uint32_t k_min = 0xffffffffu, k_max = 0;
                each([&](float x) {
                    const int bin = fine_of(x);
                    if (bin < f0) v[0] += kMass ? mass_of(x, sc, sh.tab) : 1ull;
                    else if (bin <= f1) {
                        k_min = min(k_min, key_of(x));
                        k_max = max(k_max, key_of(x));
                        const uint32_t at = atomicAdd(&sh.n_tok, 1u);
                        if (at < (uint32_t)kTok) {
                            float* to = tok + rank * kTok + at;
                            if (CS == 1) *to = x;
                            else
                                for (int q = 0; q < CS; ++q) st_dsmem_f32(map_to_rank(smem_u32(to), q), x);
                        }
                    }
                });
                block_sums(sh, v);
                k_min = __reduce_min_sync(0xffffffffu, k_min);
                k_max = __reduce_max_sync(0xffffffffu, k_max);
                if (lane == 0) {
                    sh.least[warp] = k_min;
                    sh.best[warp] = k_max;
                }
                __syncthreads();
                u64 x4[4] = {v[0], sh.n_tok, ~0ull, 0ull};
#pragma unroll
                for (int w = 0; w < kSampWarps; ++w) {
                    x4[2] = sh.least[w] < x4[2] ? sh.least[w] : x4[2];
                    x4[3] = sh.best[w] > x4[3] ? sh.best[w] : x4[3];
                }
                exchange(sh, par, x4, CS, rank);
                u64 sum = 0, most = 0;
                k_min = 0xffffffffu;
                k_max = 0;
                for (int q = 0; q < CS; ++q) {
                    sum += sh.xchg[par][q][0];
                    most = sh.xchg[par][q][1] > most ? sh.xchg[par][q][1] : most;
                    k_min = min(k_min, (uint32_t)sh.xchg[par][q][2]);
                    k_max = max(k_max, (uint32_t)sh.xchg[par][q][3]);
                }
                if (k_min == k_max && above + sum < target) {  // copies of one logit
                    above += sum;
                    return k_min;
                }
                if (k_min < k_max && above + sum < target) {
                    above += sum;
                    if (most <= (u64)kTok) {
                        // each token against the others: a thread a token (the
                        // masses take the place of the bins, read by all)
                        u64* w_s = reinterpret_cast<u64*>(sh.hist);
                        const int from_r = tid / kTok, i = tid % kTok;
                        const bool live = from_r < CS && i < (int)sh.xchg[par][from_r][1];
                        const uint32_t key = live ? key_of(tok[tid]) : 0;
                        w_s[tid] = live ? (kMass ? mass_of(tok[tid], sc, sh.tab) : 1ull) : 0ull;
                        __syncthreads();
                        u64 gt = above, ge = above;
                        for (int r2 = 0; r2 < CS; ++r2) {
                            const int n2 = (int)sh.xchg[par][r2][1];
                            for (int q = r2 * kTok; q < r2 * kTok + n2; ++q) {
                                const uint32_t other = key_of(tok[q]);
                                if (other > key) gt += w_s[q];
                                if (other >= key) ge += w_s[q];
                            }
                        }
                        if (live && gt < target && target <= ge) {  // one key's threads
                            sh.pick_key = key;
                            sh.pick = gt;
                        }
                        __syncthreads();
                        if (sh.pick_key) {
                            above = sh.pick;
                            return sh.pick_key;
                        }
                    }
                    return find_key<kMass>(sh, par, sc, k_min, k_max, target, above, CS, rank, [&](auto f) {
                        each([&](float x) {
                            const int bin = fine_of(x);
                            if (bin >= f0 && bin <= f1) f(x);
                        });
                    });
                }
            }
            return find_key<kMass>(sh, par, sc, lo, hi, target, above, CS, rank, each);
        };
        u64 m[2] = {0, 0};
        if (cut_k) {
            u64 above = sh.cum[0];
            collect(b_k, b_k, m, std::false_type());
            const uint32_t key = find_cut(std::false_type(), b_k, b_k, key_below(b_k), (u64)top_k, above);
            set_keep(key, (u64)top_k - above);
        }
        if (cut_p) {
            collect(p_from, p_to, m, std::true_type());
            cluster_sums(sh, par, m, CS, rank);
            // kept: tokens with less than top_p * m before them
            u64 target = part_up(m[0], pr.p64);
            if (target < 1) target = 1;
            u64 above = m[1];
            const uint32_t key = find_cut(std::true_type(), p_from, p_to, max(keep.key, key_below(p_to)), target, above);
            const u64 w = mass_of(float_of(key), sc, sh.tab);
            u64 ties = w ? (target - above + w - 1) / w : ~0ull;
            if (key == keep.key && keep.ties < ties) ties = keep.ties;
            // The tokens around the cut say what each warp keeps: its mass above the
            // last key, and how many tokens of that key.
            u64 v[2] = {before, 0}, all[2];
            each_near(p_from, p_to, [&](float x) {
                const uint32_t k = key_of(x);
                if (k > key) v[0] += mass_of(x, sc, sh.tab);
                v[1] += k == key;
            });
            v[0] = warp_sum(v[0]);
            v[1] = __reduce_add_sync(0xffffffffu, (uint32_t)v[1]);
            const u64 mass_w = v[0], ties_w = v[1];
            cluster_exclusive(sh, par, v, all, CS, rank);
            keep = {key, ties, v[1]};
            found = w_min == 0;
            at = v[0] + w * min(v[1], ties);
            own = mass_w + w * (min(v[1] + ties_w, ties) - min(v[1], ties));
            total = all[0] + w * min(all[1], ties);
        }
    }

    // ---- the draw: each warp's kept mass
    if (!found) {
        const bool all_kept = keep.key == kKeyNegInf + 1 && keep.ties == ~0ull;
        own = 0;
        if (all_kept && w_min == 0) {
            own = row_mass(mine, J, sc, sh.tab);
        } else {
            u64 rk = keep.base;
            MassSum s = no_mass();
            for (int j = 0; j < J; ++j) {
                float x[4];
                bool in[4];
                load4(mine + j * 128, x);
                kept4(x, keep, rk, in);
                if (isinf(mx)) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) own += in[e] && x[e] == mx ? 1ull << kMassBits : 0ull;
                    continue;
                }
                if (!(in[0] || in[1] || in[2] || in[3])) continue;
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    Mass2 w = mass_pair2(in[e] ? x[e] : -INFINITY, in[e + 1] ? x[e + 1] : -INFINITY, sc, sh.tab);
                    if (w_min) {
                        Mass a, b;
                        unpair(w.hi, a.hi, b.hi);
                        unpair(w.lo, a.lo, b.lo);
                        if (to_units(a) < w_min) a = {0.0f, 0.0f};
                        if (to_units(b) < w_min) b = {0.0f, 0.0f};
                        w = {pair(a.hi, b.hi), pair(a.lo, b.lo)};
                    }
                    add_mass(s, w);
                }
            }
            own += to_units(s);
        }
        own = warp_sum(own);
        u64 v[1] = {own}, all[1];
        cluster_exclusive(sh, par, v, all, CS, rank);
        at = v[0];
        total = all[0];
    }
    const u64 draw = part_down(total, pr.u64_);  // the running mass has to exceed this
    const bool hit = own && at <= draw && draw < at + own;  // one warp of the cluster
    if (tid == 0) sh.n_tok = ~0u;
    __syncthreads();
    if (hit && lane == 0) {
        sh.n_tok = warp;
        sh.pick = at;
        sh.xchg[par ^ 1][0][0] = keep.base;  // (no CTA writes this half any more)
    }
    __syncthreads();
    const uint32_t w_hit = sh.n_tok;
    if (w_hit == ~0u) return;
    // its tokens spread over the CTA's threads, in order
    const float* xw = row_s + (int)w_hit * w_len;
    const int per = (w_len + kSampThreads - 1) / kSampThreads, i0 = min(tid * per, w_len), i1 = min(i0 + per, w_len);
    u64 ties = keep.base;
    if (keep.ties != ~0ull) {
        uint32_t n = 0, sum;
        for (int i = i0; i < i1; ++i) n += key_of(xw[i]) == keep.key;
        ties = sh.xchg[par ^ 1][0][0] + block_exclusive32(sh, n, sum);
    }
    auto token_mass = [&](int i, u64& rk, bool& kept) -> u64 {
        const uint32_t key = key_of(xw[i]);
        kept = key > keep.key || (key == keep.key && rk++ < keep.ties);
        const u64 w = kept ? mass_of(xw[i], sc, sh.tab) : 0;
        return w >= w_min ? w : 0;
    };
    // A kept token may have a mass (above 2^-46, as mass_pair2 has it) and still less
    // than half a unit, and all that its warp holds may be such.
    auto has_mass = [&](float x) { return x == sc.mx || (x - sc.mx) * sc.ch > -46.0f; };
    u64 mine_sum = 0, rk = ties, all_sum;
    int last = -1;
    bool kept;
    for (int i = i0; i < i1; ++i) {
        const u64 w = token_mass(i, rk, kept);
        mine_sum += w;
        if (w || (kept && w_min == 0 && has_mass(xw[i]))) last = i;
    }
    u64 run = sh.pick + block_exclusive(sh, mine_sum, all_sum);
    const int first_hit = c0 + (int)w_hit * w_len;
    if (run <= draw && draw < run + mine_sum) {
        rk = ties;
        int i = i0;
        for (; i < i1 - 1; ++i) {
            run += token_mass(i, rk, kept);
            if (run > draw) break;
        }
        store(first_hit + i, xw[i], total);
    }
    // The warp's sum was rounded per lane, these per token: a draw within those
    // few units of its end belongs to its last token that has a mass (there is one:
    // the warp's sum is not zero).
    if (sh.pick + all_sum <= draw) {
        const int t = __reduce_max_sync(0xffffffffu, last);
        if (lane == 0) sh.least[warp] = (uint32_t)(t + 1);
        __syncthreads();
        if (tid == 0) {
            uint32_t m = 1;
            for (int w = 0; w < kSampWarps; ++w) m = max(m, sh.least[w]);
            store(first_hit + (int)m - 1, xw[m - 1], total);
        }
    }
}

template <typename T>
cudaError_t launch_typed(const SampleArgs& a, cudaStream_t stream) {
    // The fewest CTAs whose shares of a row leave room for two of them on an
    // SM (80 KB each beside the bins and lists); more, up to 8, while the whole
    // call has less than a CTA per SM and the shares stay above 4096 tokens.
    const long long rows = (long long)a.B * a.N_max;
    const int sms = sm_count_cached();
    constexpr int kStep = kSampWarps * 128;
    auto steps = [&](int cs) { return (a.V + cs * kStep - 1) / (cs * kStep); };
    int cs = 1;
    while (cs < 8 && (steps(cs) * kStep * 4 > 80 * 1024 || (rows * cs < sms && a.V / (cs * 2) >= 4096))) cs *= 2;
    const int J = steps(cs);
    const size_t smem = (size_t)J * kStep * 4;
    // rows held by the clusters that run at a time: two CTAs an SM
    int ahead = 2 * sms / cs;
    if (ahead >= rows) ahead = 0;
    cudaError_t e = ensure_smem(sample_kernel<T>, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(sample_kernel<T>, dim3((unsigned)(rows * cs)), dim3(kSampThreads), smem, stream, cs, a, cs, J,
                      ahead);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream) {
    switch (a.type) {
        case DFLV_LOGITS_F32: return launch_typed<float>(a, stream);
        case DFLV_LOGITS_BF16: return launch_typed<__nv_bfloat16>(a, stream);
        case DFLV_LOGITS_F16: return launch_typed<__half>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace dflv
