// given.h -- the sampler's chain drawn from random numbers the caller brings:
// temperature -> min-p -> top-k -> top-p -> renormalise, then the inverse CDF
// in index order ("Top-p (Nucleus) Sampling, in depth", "Batched top-p with a
// different p per request", sample_top_p; "Implement batched top-p sampling
// with temperature", sample), N draws per row from one distribution.
//
//   token = lowest kept i with  sum_{j <= i, j kept} w_j  >  u sum_{j kept} w_j
//
// A draw is decided by where u S falls among up to V running sums, so masses
// are carried to about 1e-13 (doubles and 45-bit integers), not to the 1e-7
// that the race needs.
//
// Weights.  y = x s + b with s = 32 log2(e) / T and b the integer that puts
// the max of the first tokens loaded, the anchor, near y = 2048: a cell
// a = rint(y) spans a thirty-second of an octave of weight, and a token of
// cell a weighs
//
//     2^(a/32) * 2^(h/32),   h = y - a in [-1/2, 1/2],
//
// the second factor by a polynomial of degree 4 (off by less than 8e-14).
// Adding 1.5 2^52 in the fused product rounds x s + b to a and leaves it in
// the low word of the double; h comes from a second fused product, so a cell
// and its h cost three operations.
//
// Cells do not move with the row max, so one pass finds the max and
// histograms the row.  A histogram slot sums the second factors as integers of
// `bits` fractional bits (62 - ceil(log2 V), at most 50): exact in any order.
// The window holds 2048 cells (64 octaves) below the anchor and 2048 above
// it; what is further down weighs less than 2^-64 of the max each, less than
// the sums resolve: it is counted, and has no mass.  A row whose max lies above
// the window takes the pass again.
//
// The cuts.  With the cells ranked down from the max's (rank 0), top-k or
// min-p cut through one bottom cell rb.  The survivors' mass S lies between
// that of the cells above rb and that with rb, so the top-p cut lies in a
// cell of a range [r_lo, r_hi], one cell unless rb holds much mass.  One more
// pass sums the tokens above r_lo per index segment and lists those of the
// cells [r_lo, r_hi] and rb; the list then gives rb's exact survivors, S, the
// crossing cell and by radix select (select.h) the exact cut level.  A row
// with more than kCap such tokens reads them from memory again wherever
// the list would have been read.
//
// The draw finds its segment from the segments' sums, then reads that segment
// alone.  Short rows and large batches run on one workgroup per row; long rows
// are split over workgroups (below) where that is faster.
//
// What bounds it: double-precision arithmetic of about 20 operations a kept
// token and 5 a token of the first pass, on one CU for a row; the second read
// comes from cache.  A row of 128256 float32 logits, all 256 CUs at work: first
// pass 26 us (131 MB at 5 TB/s), cells of the cuts 3, second pass 5 to 57 by the
// size of the nucleus, exact level 5, a round of eight draws 4.  Rows of 1024:
// 3, 3, 2, 2 and 3 us, all of them waits on one another.
#pragma once

#include <type_traits>

#include "common.h"
#include "params.h"
#include "select.h"

namespace nucleus {

constexpr int kOctave = 32;       // cells per octave of weight
constexpr int kSlots = 4096;      // histogram window
constexpr int kSlotsBelow = 2048; // of it, below the anchor: 64 octaves
constexpr int kCopy = kSlots + kWave + 16;  // words between the two copies
static_assert(kCopy * 8 % 256 == 128, "copies half the banks apart");
constexpr int kSubSteps = 4;      // steps of a segment, at least
constexpr int kRankNone = 0x7FFFFFFF;
constexpr double kLn2 = 0.69314718055994530942;
constexpr uint32_t kEmpty = 0x7FC00000u;  // (NaN) an empty place of the list

struct GivenParams {
    const void* logits;        // [B, stride]
    int64_t B, V, stride;
    const float* temperature;  // [B]
    const float* top_p;        // [B]
    const int32_t* top_k;      // [B] or null
    const float* min_p;        // [B] or null
    const void* uniforms;      // [B, N]
    int64_t N;
    int u_f64;
    int32_t* out_token;        // [B, N]
    int32_t* out_count;        // [B]
    float* out_logprob;        // [B, N] or null
    float* out_probs;          // [B, V] or null
    int bits;                  // fractional bits of in-cell weights
};

// 2^(i/32), i = 0 .. 31, correctly rounded.
__device__ constexpr double kRoot[kOctave] = {
    1.0, 1.0218971486541166, 1.0442737824274138, 1.0671404006768237, 1.0905077326652577, 1.1143867425958924,
    1.1387886347566916, 1.1637248587775775, 1.189207115002721, 1.215247359980469, 1.241857812073484,
    1.2690509571917332, 1.2968395546510096, 1.3252366431597413, 1.3542555469368927, 1.383909881963832,
    1.4142135623730951, 1.4451808069770467, 1.4768261459394993, 1.5091644275934228, 1.5422108254079407,
    1.5759808451078865, 1.6104903319492543, 1.645755478153965, 1.681792830507429, 1.718619298122478,
    1.7562521603732995, 1.7947090750031072, 1.8340080864093424, 1.8741676341103, 1.9152065613971474,
    1.9571441241754002};

// The row's lattice.
constexpr double kMagic = 0x1.8p52;  // adding it rounds to an integer
struct Cells {
    double s;    // cells per logit unit
    double bm;   // b + kMagic
    float lo;    // fast rows: a logit just below the window
    bool fast;   // such a logit exists, and lies less than 2^30 cells down
};

// The lattice of a row with anchor x0 (finite) and temperature T > 0.
__device__ __forceinline__ Cells make_cells(float x0, float T)
{
    Cells c;
    // T = +inf: cells wider than any logit, so that every weight is 1.
    c.s = T == INFINITY ? 0x1p-1000 : (kOctave * 1.4426950408889634074) / (double)T;
    // Past |x0| s = 2^44 neighbouring logits are 2^20 cells apart and more,
    // that is of weight 0 beside each other, whatever s is; b stays an exact
    // integer.
    const double ax = fabs((double)x0);
    if (ax * c.s > 0x1p44) c.s = 0x1p44 / ax;
    c.s = uniform(c.s);
    c.bm = uniform(rint((double)kSlotsBelow - (double)x0 * c.s) + kMagic);
    const double lo = (double)x0 - (double)(kSlotsBelow + 16) / c.s;
    float f = (float)lo;
    if ((double)f > lo) f = nextafterf(f, -INFINITY);
    c.lo = uniform(f);
    c.fast = c.lo > -INFINITY;
    return c;
}

// Slot of a logit (far below the window, and for -inf: negative; above:
// >= kSlots; saturated to int32) and its place h in its cell (no number for
// -inf, and without meaning far outside the window).  Monotone in x.
__device__ __forceinline__ int slot_of(const Cells& c, float x, double& h)
{
    const double t = fma((double)x, c.s, c.bm);
    h = fma((double)x, c.s, c.bm - t);
    return cvt_i32_sat(t - kMagic);
}

// Keeps the instructions before it before it.  The per-token arithmetic below
// is a chain of dependent double operations, each of which waits about ten
// cycles for the one before; written one operation for all the tokens of a
// group at a time, the tokens fill each other's waits (left to itself the
// compiler finishes one token before it starts the next).
__device__ __forceinline__ void in_step() { __builtin_amdgcn_sched_barrier(0); }

// The same for N tokens with c.lo <= x of a fast row (FAST: the slot is the
// low word of the rounded sum; above the window's reach, 2^31 cells, it is
// without meaning).
template <int N, bool FAST>
__device__ __forceinline__ void slots_of(const Cells& c, const float (&x)[N], int (&sl)[N], double (&h)[N])
{
    double xd[N], t[N];
#pragma unroll
    for (int j = 0; j < N; ++j) xd[j] = (double)x[j];
    in_step();
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = fma(xd[j], c.s, c.bm);
    in_step();
#pragma unroll
    for (int j = 0; j < N; ++j) h[j] = c.bm - t[j];
    in_step();
#pragma unroll
    for (int j = 0; j < N; ++j) h[j] = fma(xd[j], c.s, h[j]);
    in_step();
#pragma unroll
    for (int j = 0; j < N; ++j)
        sl[j] = FAST ? (int)(uint32_t)__double_as_longlong(t[j]) : cvt_i32_sat(t[j] - kMagic);
}

// 2^(h/32) for |h| <= 1/2: Taylor's polynomial of degree 5 with its last term
// replaced by the cubic nearest to it there (h^5 ~ (20 r^2 h^3 - 5 r^4 h)/16,
// r = 1/2, by the fifth Chebyshev polynomial): degree 4, off by less than
// 8e-14.
constexpr double kL = kLn2 / kOctave, kL5 = kL * kL * kL * kL * kL / 120;
constexpr double kP1 = kL - kL5 * 5 / 256, kP2 = kL * kL / 2, kP3 = kL * kL * kL / 6 + kL5 * 20 / 64,
                 kP4 = kL * kL * kL * kL / 24;

__device__ __forceinline__ double in_cell(double h)
{
    return fma(fma(fma(fma(kP4, h, kP3), h, kP2), h, kP1), h, 1.0);
}

template <int N>
__device__ __forceinline__ void in_cells(const double (&h)[N], double (&q)[N])
{
#pragma unroll
    for (int j = 0; j < N; ++j) q[j] = fma(kP4, h[j], kP3);
    in_step();
#pragma unroll
    for (int j = 0; j < N; ++j) q[j] = fma(q[j], h[j], kP2);
    in_step();
#pragma unroll
    for (int j = 0; j < N; ++j) q[j] = fma(q[j], h[j], kP1);
    in_step();
#pragma unroll
    for (int j = 0; j < N; ++j) q[j] = fma(q[j], h[j], 1.0);
    in_step();
}

// The same times 2^bits, rounded to an integer (below 2^52: added to 2^52, it
// is in the low bits of the double).
struct Fixed {
    double c1, c2, c3, c4, c0;
    __device__ explicit Fixed(double scale)
        : c1(uniform(kP1 * scale)), c2(uniform(kP2 * scale)), c3(uniform(kP3 * scale)), c4(uniform(kP4 * scale)),
          c0(uniform(scale + 0x1p52))
    {
    }
    __device__ __forceinline__ uint64_t operator()(double h) const
    {
        return (uint64_t)__double_as_longlong(fma(fma(fma(fma(c4, h, c3), h, c2), h, c1), h, c0)) -
               0x4330000000000000ull;
    }
    template <int N>
    __device__ __forceinline__ void operator()(const double (&h)[N], uint64_t (&n)[N]) const
    {
        double q[N];
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = fma(c4, h[j], c3);
        in_step();
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = fma(q[j], h[j], c2);
        in_step();
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = fma(q[j], h[j], c1);
        in_step();
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = fma(q[j], h[j], c0);
        in_step();
#pragma unroll
        for (int j = 0; j < N; ++j) n[j] = (uint64_t)__double_as_longlong(q[j]) - 0x4330000000000000ull;
    }
};

// The integer nearest to v < 2^52.
__device__ __forceinline__ uint64_t fixed_point(double v)
{
    return (uint64_t)__double_as_longlong(v + 0x1p52) - 0x4330000000000000ull;
}

// 2^(-rank/32); root: kRoot in LDS.  0 past about 34000 cells down.
__device__ __forceinline__ double rank_weight(const double* root, int rank)
{
    return ldexp(root[-rank & (kOctave - 1)], -rank >> 5);
}

// The lanes for which `v` holds, as a mask in scalar registers.
__device__ __forceinline__ uint64_t lanes(bool v) { return __builtin_amdgcn_ballot_w64(v); }

// A group: the 16 bytes of a row that a lane loads at a time.
template <int DT> struct Group { static constexpr int N = DT == kF32 ? 4 : 8; };

template <int DT>
__device__ __forceinline__ float logit_at(const void* row, int64_t i)
{
    if constexpr (DT == kF32) return ((const float*)row)[i];
    if constexpr (DT == kBF16) return bf16_to_float(((const uint16_t*)row)[i]);
    if constexpr (DT == kF16) return (float)((const _Float16*)row)[i];
}

template <int DT>
__device__ __forceinline__ void unpack(u32x4 v, float (&x)[Group<DT>::N])
{
    if constexpr (DT == kF32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(v[j]);
    } else if constexpr (DT == kBF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(v[j] << 16);
            x[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
        }
    } else {
        typedef _Float16 h8 __attribute__((ext_vector_type(8)));
        const h8 h = __builtin_bit_cast(h8, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (float)h[j];
    }
}

// The 16 bytes of group g.  VEC: rows start on 16-byte boundaries and hold
// whole groups; a group past the end reads the last one.  Otherwise element
// by element, the last element past the end.  The caller masks both.
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 load_raw(const void* row, uint32_t g, uint32_t groups, int64_t V)
{
    if constexpr (VEC) {
        return *((const u32x4*)row + min(g, groups - 1));
    } else {
        constexpr int N = Group<DT>::N;
        u32x4 v;
        if constexpr (DT == kF32) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = ((const uint32_t*)row)[min((int64_t)g * N + j, V - 1)];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = ((const uint16_t*)row)[min((int64_t)g * N + 2 * j, V - 1)];
                const uint32_t hi = ((const uint16_t*)row)[min((int64_t)g * N + 2 * j + 1, V - 1)];
                v[j] = lo | hi << 16;
            }
        }
        return v;
    }
}

// Group g's tokens widened to fp32; -inf past the row's end (checked only
// where `edge` says that the row may end here).
template <int DT>
__device__ __forceinline__ void tokens_of(u32x4 raw, uint32_t g, bool edge, int64_t V, float (&x)[Group<DT>::N])
{
    constexpr int N = Group<DT>::N;
    unpack<DT>(raw, x);
    if (edge) {  // uniform
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = (int64_t)g * N + j < V ? x[j] : -INFINITY;
    }
}

// How a row's groups are dealt out: wave w owns the `steps` * 64 groups from
// w * steps * 64, and its segments are runs of `sps` steps.
struct Deal {
    uint32_t groups;  // of the row
    uint32_t steps;   // of 64 groups, per wave
    uint32_t sps;     // steps per segment
    uint32_t spw;     // segments per wave
};

template <int DT, int NT>
__device__ __forceinline__ Deal deal_out(int64_t V)
{
    Deal d;
    d.groups = (uint32_t)((V + Group<DT>::N - 1) / Group<DT>::N);
    d.steps = (d.groups + NT - 1) / NT;
    d.sps = max((uint32_t)kSubSteps, (d.steps + kWave - 1) / kWave);  // at most 64 segments per wave
    d.spw = (d.steps + d.sps - 1) / d.sps;
    return d;
}

// fn(step, group, tokens) over the wave's steps, in order, with the loads of
// the next steps (128 bytes of a lane) in flight.  Every lane takes every step
// (past the row's end with tokens of -inf).
template <int DT, bool VEC, class Fn>
__device__ __forceinline__ void stream_row(const void* row, const Deal& d, int64_t V, Fn fn)
{
    constexpr int GN = Group<DT>::N, AT = VEC ? (DT == kF32 ? 8 : 4) : 2;
    const uint32_t lane = threadIdx.x & (kWave - 1), g0 = uniform(threadIdx.x / kWave) * d.steps * kWave;
    const uint32_t whole = (uint32_t)(V / GN);  // groups without the row's end
    u32x4 a[AT], b[AT];
    auto fetch = [&](u32x4 (&to)[AT], uint32_t i) {
#pragma unroll
        for (int k = 0; k < AT; ++k)
            to[k] = load_raw<DT, VEC>(row, g0 + min(i + k, d.steps - 1) * kWave + lane, d.groups, V);
    };
    fetch(a, 0);
#pragma unroll 1
    for (uint32_t i = 0; i < d.steps; i += AT) {
        fetch(b, i + AT);
#pragma unroll
        for (int k = 0; k < AT; ++k) {
            if (k > 0 && i + k >= d.steps) break;  // uniform
            const uint32_t g = g0 + (i + k) * kWave;
            float x[GN];
            tokens_of<DT>(a[k], g + lane, g + kWave > whole, V, x);
            fn(i + k, g + lane, x);
        }
#pragma unroll
        for (int k = 0; k < AT; ++k) a[k] = b[k];
    }
}

template <int NT>
struct GivenShared {
    static constexpr int kCap = NT < 512 ? NT * 12 : 6144;  // listed tokens of undecided cells
    static constexpr int kWaves = NT / kWave;
    // Integer masses of the cells (and a slot per lane for the tokens outside).
    // Odd lanes add into a second copy, half a row of banks away, which halves
    // the tokens of one cell that meet at one address (cells that hold
    // a few percent of the row are common).  In the second pass the second
    // copy's place holds the weights 2^(-rank/32) of the surely kept cells, as
    // doubles, and 0 elsewhere.
    alignas(16) uint64_t hist[2 * kCopy];
    alignas(16) uint32_t cnt[kSlots + kWave];
    uint2 list[kCap];          // logit, index
    double sub[NT];            // mass of each segment's surely kept tokens; then of the segments up to it (-1: empty)
    uint64_t subc[NT];         // mass of its kept listed tokens, at 2^-bits
    double pre[NT];            // number of its undecided tokens; then mass of the segments before it
    double root[kOctave];
    SelectShared sel;
    uint64_t red64[kWaves];
    double redf[kWaves];
    int first[2][kWaves];
    uint32_t list_n;
    // decided by one thread, read by all
    double s_above, a_lo, w_bottom;
    uint32_t n_above, n_window;
    int cross;
    uint64_t tc;
    // a few undecided tokens, on one wave
    uint2 few[kWave];
    uint32_t few_n, few_cut;
};

struct SumF64 { __device__ double operator()(double a, double b) const { return a + b; } };
struct MinI { __device__ int operator()(int a, int b) const { return a < b ? a : b; } };
struct MaxF32 { __device__ float operator()(float a, float b) const { return fmaxf(a, b); } };

// Exclusive prefix sum over the workgroup's threads in one fixed order;
// `total` is the whole sum.
template <int NT>
__device__ __forceinline__ double block_exclusive_sum_f64(double v, double* scratch, double& total)
{
    const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
    double wt;
    const double inc = wave_inclusive_sum(v, wt);
    const double prev = wave_shift_up1(inc);
    __syncthreads();
    if (lane == 0) scratch[w] = wt;
    __syncthreads();
    double off = 0.0, all = 0.0;
#pragma unroll
    for (int i = 0; i < NT / kWave; ++i) {
        if (i == w) off = all;
        all += scratch[i];
    }
    total = all;
    return lane == 0 ? off : off + prev;
}

// Mode of a row once its max is known.
enum : int {
    kGivenError = 0,   // token -1
    kGivenGreedy = 1,
    kGivenLevel = 2,   // kept: x >= a level known at once
    kGivenCells = 3,   // kept: by cells and the listed tokens
    kGivenAlone = 4,   // (split rows) left to one workgroup
};

// What the first pass finds (each thread its own).
struct FirstPass {
    float m;           // max; NaN or +inf if one was seen
    uint32_t at;       // without a histogram: the step that first held it
    uint32_t finite;   // with counts: tokens above -inf in this wave
};

enum : int { kPassMax = 0, kPassHist = 1, kPassCount = 2 };

// Straight-line over a group's tokens: a token outside the window goes to its
// lane's own slot past it.
template <int DT, bool VEC, int PASS, bool FAST, class Shared>
__device__ __forceinline__ FirstPass first_pass(const void* row, const Deal& d, int64_t V, const Cells& c,
                                                const Fixed& fx, Shared& sh)
{
    constexpr int GN = Group<DT>::N;
    FirstPass r = {-INFINITY, 0, 0};
    const uint32_t outside = kSlots + (threadIdx.x & (kWave - 1));
    uint64_t* hist = sh.hist + (threadIdx.x & 1) * kCopy;
    stream_row<DT, VEC>(row, d, V, [&](uint32_t i, uint32_t, const float (&x)[GN]) {
        float most = x[0];  // IEEE maximum: NaN stays
#pragma unroll
        for (int j = 1; j < GN; ++j) most = __builtin_elementwise_maximum(most, x[j]);
        if constexpr (PASS == kPassMax) {
            if (!(most <= r.m)) r.at = i;
        }
        r.m = __builtin_elementwise_maximum(r.m, most);
        if constexpr (PASS != kPassMax) {
            float xc[GN];
            int sl[GN];
            double h[GN];
            uint64_t q[GN];
#pragma unroll
            for (int j = 0; j < GN; ++j) {
                xc[j] = FAST ? fmaxf(x[j], c.lo) : x[j];
                if constexpr (PASS == kPassCount) r.finite += (uint32_t)__builtin_popcountll(lanes(x[j] > -INFINITY));
            }
            slots_of<GN, FAST>(c, xc, sl, h);
            fx(h, q);
#pragma unroll
            for (int j = 0; j < GN; ++j) {
                const uint32_t at = min((uint32_t)sl[j], outside);
                atomicAdd((unsigned long long*)&hist[at], (unsigned long long)q[j]);
                if constexpr (PASS == kPassCount) atomicAdd(&sh.cnt[at], 1u);
            }
        }
    });
    return r;
}

// One row's parameters.
struct RowIn {
    float T, P, MP;
    int K;
    bool greedy, use_k, want_hist;
};

__device__ __forceinline__ RowIn row_in(const GivenParams& p, int64_t b)
{
    RowIn r;
    r.T = uniform(p.temperature[b]);
    r.P = uniform(p.top_p[b]);
    r.K = p.top_k ? uniform(p.top_k[b]) : 0;
    r.MP = p.min_p ? uniform(p.min_p[b]) : 0.0f;
    r.greedy = r.T <= 0.0f;
    r.use_k = r.K > 0 && (int64_t)r.K < p.V;
    // A histogram is needed where a cut has to be searched for.
    r.want_hist = !r.greedy && r.P > 0.0f && (r.P < 1.0f || r.use_k);
    return r;
}

__device__ __forceinline__ bool row_error(const RowIn& r, float m)
{
    return !(m > -INFINITY && m < INFINITY) || isnan(r.T) || isnan(r.P) || isnan(r.MP);
}

template <int DT>
__device__ __forceinline__ const void* row_of(const GivenParams& p, int64_t b)
{
    return (const char*)p.logits + (size_t)b * (size_t)p.stride * (DT == kF32 ? 4 : 2);
}

// How a row's tokens are kept, up to the undecided ones.  Ranks count cells
// down from the max's; kRankNone stands for none.
struct RowPlan {
    Cells c;
    double hm;        // place of the max in its cell
    float m;          // max
    float tmp;        // min-p's threshold (-inf: off)
    float level;      // kGivenLevel: kept iff x >= level and finite
    float floor_x;    // finite; every token that may be kept is at or above it
    int mode;
    int top;          // slot of rank 0
    int rb;           // bottom cell; top + 1: the tokens below the window
    int r_lo, r_hi;   // kept: ranks below r_lo; undecided: r_lo .. r_hi and rb
};

constexpr float kLowest = -3.402823466e38f;

// From the max (of a row without error, T > 0) and, where the row wants one,
// the histogram in LDS (`copies`: in two copies) over lattice c; `finite`:
// tokens above -inf (top-k rows).  s_above, a_lo, w_bottom and n_above are left
// in LDS.
template <int NT, class Shared>
__device__ __forceinline__ RowPlan plan_row(Shared& sh, const RowIn& in, Cells c, float m, uint32_t finite, bool copies,
                                            int bits)
{
    const int t = threadIdx.x, lane = t & (kWave - 1), w = t / kWave;
    const float T = in.T, P = in.P, MP = in.MP;
    const int K = in.K;
    const bool use_k = in.use_k, cut_p = P < 1.0f;
    int mode = kGivenCells;
    float level = -INFINITY;
    // min-p: w_i >= min_p w_max  <=>  x_i >= m + T ln(min_p), rounded up.
    float tmp = -INFINITY;
    if (MP > 0.0f && T != INFINITY) {
        const double td = (double)m + (double)T * log((double)fminf(MP, 1.0f));
        float tf = (float)td;
        if ((double)tf < td) tf = nextafterf(tf, INFINITY);
        tmp = uniform(tf);
    }
    if (P <= 0.0f) {
        mode = kGivenLevel;
        level = m;
    } else if (!in.want_hist) {
        mode = kGivenLevel;
        level = tmp;
    }

    double hm;
    if (mode == kGivenLevel) c = make_cells(m, T);
    const int top = uniform(slot_of(c, m, hm));
    int rb = kRankNone;
    int r_lo = 0, r_hi = -1;
    if (mode == kGivenCells) {
        // Thread t looks at ranks PER t .. PER t + PER - 1.
        constexpr int PER = kSlots / NT;
        double wt[PER], run = 0.0;
        uint32_t ct[PER], crun = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = PER * t + i, sl = top - r;
            uint64_t hv = 0;
            if (sl >= 0) sh.hist[sl] = hv = sh.hist[sl] + (copies ? sh.hist[kCopy + sl] : 0);  // joined
            wt[i] = ldexp((double)hv * sh.root[-r & (kOctave - 1)], (-r >> 5) - bits);
            run += wt[i];
        }
        double total;
        const double before = block_exclusive_sum_f64<NT>(run, sh.redf, total);
        uint32_t cbefore = 0;
        int rk = kRankNone;
        if (use_k) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int sl = top - (PER * t + i);
                ct[i] = sl >= 0 ? sh.cnt[sl] : 0u;
                crun += ct[i];
            }
            cbefore = (uint32_t)block_exclusive_sum<NT>(crun, sh.red64);
            uint32_t cc = cbefore;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                cc += ct[i];
                if (rk == kRankNone && cc >= (uint32_t)K && ct[i]) rk = PER * t + i;
            }
            rk = block_reduce<NT>(rk, MinI(), (int*)sh.redf);
            if (t == NT - 1) sh.n_window = cbefore + crun;
        }
        double ht;
        // min-p's threshold is at or below the max, and may lie below the window
        const int rt = tmp > -INFINITY ? top - max(slot_of(c, tmp, ht), -1) : kRankNone;
        rb = min(rk, rt);
        if (cut_p && rb > top) rb = kRankNone;  // below the window: the top-p cut is above it
        if (rb <= top) {
            const int o = rb - PER * t;
            if (o >= 0 && o < PER) {
                double ab = before, wb = 0.0;
                uint32_t ca = cbefore;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    if (i < o) {
                        ab += wt[i];
                        if (use_k) ca += ct[i];
                    }
                    if (i == o) wb = wt[i];
                }
                sh.s_above = ab;
                sh.n_above = ca;
                sh.w_bottom = wb;
            }
        } else if (t == NT - 1) {
            sh.n_above = cbefore + crun;
            sh.s_above = total;
            sh.w_bottom = 0.0;
        }
        if (rb != kRankNone || use_k) __syncthreads();
        if (rb == kRankNone && use_k && !cut_p && finite > (uint32_t)K && sh.n_window < (uint32_t)K)
            rb = top + 1;  // top-k cuts among the tokens below the window: they are listed as one cell
        if (rb == kRankNone && !cut_p) {  // neither cuts: all that min-p leaves
            mode = kGivenLevel;
            level = tmp;
        }
        if (cut_p) {
            // The first cells whose running mass reaches p S for the least and
            // the most S may be: in each wave by ballot, then over the waves.
            const double lo = (double)P * (rb == kRankNone ? total : sh.s_above);
            const double hi = rb == kRankNone ? lo : (double)P * (sh.s_above + sh.w_bottom);
            int mine_lo = kRankNone, mine_hi = kRankNone;
            double ab = before, a_lo = 0.0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int r = PER * t + i;
                const bool cell = wt[i] > 0.0 && r < rb;
                if (cell && mine_lo == kRankNone && ab + wt[i] >= lo) {
                    mine_lo = r;
                    a_lo = ab;
                }
                if (cell && mine_hi == kRankNone && ab + wt[i] >= hi) mine_hi = r;
                ab += wt[i];
            }
            const auto first_of = [&](int v) {
                const uint64_t any = lanes(v != kRankNone);
                return any ? __builtin_amdgcn_readlane(v, (int)__builtin_ctzll(any)) : kRankNone;
            };
            const int w_lo = first_of(mine_lo), w_hi = first_of(mine_hi);
            if (lane == 0) {
                sh.first[0][w] = w_lo;
                sh.first[1][w] = w_hi;
            }
            __syncthreads();
            r_lo = r_hi = kRankNone;
#pragma unroll
            for (int i = 0; i < NT / kWave; ++i) {
                r_lo = min(r_lo, sh.first[0][i]);
                r_hi = min(r_hi, sh.first[1][i]);
            }
            if (rb == kRankNone && r_lo == kRankNone) {
                // Rounding leaves none: the last cell with mass.
                int last = -1;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (wt[i] > 0.0) last = PER * t + i;
                r_lo = r_hi = block_reduce<NT>(last, MaxI32(), (int*)sh.redf);
                const int o = r_lo - PER * t;
                if (o >= 0 && o < PER) {
                    double a = before;
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        if (i < o) a += wt[i];
                    sh.a_lo = a;
                }
            } else {
                r_lo = min(r_lo, rb);
                r_hi = min(r_hi, rb);
                if (mine_lo == r_lo && r_lo != kRankNone) sh.a_lo = a_lo;
                if (r_lo == rb && t == 0) sh.a_lo = sh.s_above;
            }
        } else {
            r_lo = rb;  // every cell above the bottom one is kept
            r_hi = rb;
        }
        r_lo = uniform(r_lo);
        r_hi = uniform(r_hi);
        rb = uniform(rb);
    }

    float floor_x = fmaxf(level, kLowest);
    if (mode == kGivenCells) {
        const int r_end = rb == kRankNone ? r_hi : max(r_hi, rb);  // the last rank that may be kept
        // (a cell and a half of slack covers the roundings)
        if (r_end <= top)
            floor_x = fmaxf((float)(((double)(top - r_end) - 1.5 - (c.bm - kMagic)) / c.s), kLowest);
        if (floor_x > kLowest) floor_x = nextafterf(floor_x, -INFINITY);
    }
    RowPlan o;
    o.c = c;
    o.hm = uniform(hm);
    o.m = m;
    o.tmp = tmp;
    o.level = level;
    o.floor_x = uniform(floor_x);
    o.mode = mode;
    o.top = top;
    o.rb = rb;
    o.r_lo = r_lo;
    o.r_hi = r_hi;
    return o;
}

// Rank of a finite token's cell; all cells below the window are one.
__device__ __forceinline__ int rank_of(const RowPlan& o, float x, double& h)
{
    const int sl = slot_of(o.c, x, h);
    return sl >= 0 ? o.top - sl : o.top + 1;
}

// The mass of a finite token: 0 below the window.
__device__ __forceinline__ double mass_of(const RowPlan& o, const double* root, float x)
{
    double h;
    const int sl = slot_of(o.c, x, h);
    return sl >= 0 ? rank_weight(root, o.top - sl) * in_cell(h) : 0.0;
}

// Its weight beside that of rank 0, however far down.
__device__ __forceinline__ double weight_of(const RowPlan& o, const double* root, float x)
{
    const double y = fma((double)x, o.c.s, o.c.bm - kMagic), a = rint(y);
    return rank_weight(root, -max(cvt_i32_sat(a - (double)o.top), -(1 << 17))) * in_cell(y - a);
}

// A greedy row, or (token -1) one in error.  Every thread of the workgroup.
template <int NT>
__device__ __forceinline__ void store_single(const GivenParams& p, int64_t b, int token)
{
    const int t = threadIdx.x;
    if (t == 0) p.out_count[b] = token >= 0 ? 1 : 0;
    for (int64_t n = t; n < p.N; n += NT) {
        p.out_token[b * p.N + n] = token;
        if (p.out_logprob) p.out_logprob[b * p.N + n] = token >= 0 ? 0.0f : __uint_as_float(0x7FC00000u);
    }
}

// Is x one of the undecided?  (NaN, an empty place's, is not.)
__device__ __forceinline__ bool is_undecided(const RowPlan& o, float x, int& r, double& h)
{
    if (!(x >= o.floor_x)) return false;
    r = rank_of(o, x, h);
    return r >= o.r_lo && (r <= o.r_hi || r == o.rb);
}

// Copies the undecided of a list of ln <= NT places to sh.few, as many as it
// holds, and counts them in sh.few_n.
template <class Shared>
__device__ __forceinline__ void gather_few(Shared& sh, const RowPlan& o, uint32_t ln)
{
    const uint32_t t = threadIdx.x;
    const uint2 e = sh.list[t < ln ? t : 0];
    int r;
    double h;
    const bool mine = t < ln && is_undecided(o, __uint_as_float(e.x), r, h);
    const uint64_t all = lanes(mine);
    if (all) {  // uniform
        uint32_t at = 0;
        if ((t & (kWave - 1)) == 0) at = atomicAdd(&sh.few_n, (uint32_t)__builtin_popcountll(all));
        at = uniform(at) + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
        if (mine && at < kWave) sh.few[at] = e;
    }
}

// The exact cut: the logit at and above which a row's finite tokens are kept.
// The undecided tokens are in sh.list (`listed`: `ln` places) or read from the
// row again; kmin, kmax: this thread's least and largest key of those that
// are in no list.  Adds the kept ones to sh.subc (or gives the one weight of
// all, for sh.pre of each segment) and to `count`.
template <int DT, int NT, class Shared>
__device__ __forceinline__ float resolve_row(Shared& sh, const GivenParams& p, const void* row, const Deal& d,
                                             const RowIn& in, const RowPlan& o, const Fixed& fx, bool listed, uint32_t ln,
                                             uint32_t kmin, uint32_t kmax, uint32_t& count, double& one_weight)
{
    constexpr int GN = Group<DT>::N;
    const int t = threadIdx.x;
    const double scale = ldexp(1.0, p.bits), inv_scale = ldexp(1.0, -p.bits);
    const bool cut_p = in.P < 1.0f;
    uint32_t cut = order_key(fmaxf(o.level, kLowest));
    one_weight = 0.0;
    if (o.mode == kGivenCells) {
        // Every undecided token (key, index), from the list or from memory.
        auto undecided = [&](auto fn) {
            const uint32_t n = listed ? ln : (uint32_t)p.V;
#pragma unroll 1
            for (uint32_t i = t; i < n; i += NT) {
                float x;
                uint32_t idx = i;
                if (listed) {
                    x = __uint_as_float(sh.list[i].x);  // (kEmpty is NaN)
                    idx = sh.list[i].y;
                } else {
                    x = logit_at<DT>(row, i);
                }
                int r;
                double h;
                if (is_undecided(o, x, r, h)) fn(x, idx, r, h);
            }
        };
        // Keys that bound those of rank r's cell (a tenth of a cell to spare).
        auto key_at = [&](int r, double off) {
            if (r > o.top) return off < 0.0 ? 0u : 0xFFFFFFFFu;
            return order_key((float)(((double)(o.top - r) + off - (o.c.bm - kMagic)) / o.c.s));
        };
        // Long runs of one value (more undecided tokens than the list holds,
        // all of one key): they share a fate, which needs no search.
        uint32_t one_key = 0;
        if (!listed) {
            for (uint32_t i = t; i < Shared::kCap; i += NT) {
                const float x = __uint_as_float(sh.list[i].x);
                if (!(x >= o.floor_x)) continue;
                kmin = min(kmin, order_key(x));
                kmax = max(kmax, order_key(x));
            }
            const uint64_t both = block_reduce<NT>(
                (uint64_t)kmax << 32 | (uint32_t)~kmin,
                [](uint64_t a, uint64_t e) {
                    const uint64_t hi = 0xFFFFFFFF00000000ull;
                    return ((a & hi) > (e & hi) ? a & hi : e & hi) | ((uint32_t)a > (uint32_t)e ? (uint32_t)a : (uint32_t)e);
                },
                sh.red64);
            if ((uint32_t)(both >> 32) == ~(uint32_t)both) one_key = (uint32_t)(both >> 32);
        }
        // The crossing cell, the first whose running mass reaches p S, and the
        // mass that it is crossed at.
        auto crossing = [&](double s_bottom, int& cell, uint64_t& thr) {
            const double want = (double)in.P * (sh.s_above + s_bottom);
            double a = sh.a_lo, at = sh.a_lo;
            cell = o.r_lo;
#pragma unroll 1
            for (int r = o.r_lo; r <= o.r_hi; ++r) {
                const double wr =
                    r == o.rb ? s_bottom : rank_weight(sh.root, r) * ((double)sh.hist[o.top - r] * inv_scale);
                if (wr > 0.0) {
                    cell = r;
                    at = a;
                    if (a + wr >= want) break;
                }
                a += wr;
            }
            const double q = (want - at) / (rank_weight(sh.root, cell) * inv_scale);
            thr = !(q > 1.0) ? 1 : (q < 1.8e19 ? (uint64_t)ceil(q) : ~0ull);
        };
        // A kept one: to its segment.
        auto keep = [&](float x, uint32_t idx) {
            const uint32_t step = idx / (GN * kWave), own = step / d.steps;
            atomicAdd((unsigned long long*)&sh.subc[own * d.spw + (step - own * d.steps) / d.sps],
                      (unsigned long long)fixed_point(mass_of(o, sh.root, x) * scale));
            ++count;
        };
        const uint32_t from_minp = order_key(fmaxf(o.tmp, kLowest));
        uint32_t bottom = from_minp;  // lowest key that survives min-p and top-k
        double s_bottom = 0.0;        // mass of the bottom cell's survivors
        const uint64_t thr_k = in.use_k && sh.n_above < (uint32_t)in.K ? (uint64_t)in.K - sh.n_above : 0;
        if (listed && ln <= NT) {
            // At most 64 of them, as in short rows: the first wave has one in
            // every lane, and compares them all (15 rows of 1024: 18.6 -> 15.6 us).
            const int lane = t & (kWave - 1);
            gather_few(sh, o, ln);
            __syncthreads();
            const uint32_t n = uniform(sh.few_n);
            if (n <= kWave) {
                if (t < kWave) {
                    const bool have = (uint32_t)lane < n;
                    const float x = have ? __uint_as_float(sh.few[lane].x) : 0.0f;
                    double h;
                    const int rank = rank_of(o, have ? x : o.m, h);
                    const uint32_t key = order_key(x);
                    const uint64_t w = fx(h);
                    // The lowest level above which the cell's tokens weigh less than thr.
                    auto level_in = [&](int cell, uint64_t weight, uint64_t thr) {
                        const bool here = have && rank == cell && key >= bottom && weight;
                        const uint64_t all = lanes(here);
                        uint64_t above = 0;
#pragma unroll 1
                        for (uint64_t m = all; m; m &= m - 1) {
                            const int j = (int)__builtin_ctzll(m);
                            const uint64_t wj = lane_read64(weight, j);
                            if ((uint32_t)__builtin_amdgcn_readlane((int)key, j) > key) above += wj;
                        }
                        const uint32_t level = wave_reduce(here && above < thr ? key : 0xFFFFFFFFu, MinU32());
                        return all ? level : 0u;
                    };
                    if (o.rb != kRankNone) {
                        if (thr_k) bottom = max(bottom, level_in(o.rb, 1, thr_k));
                        if (o.rb <= o.top && cut_p) {
                            const uint64_t sum =
                                wave_reduce(have && rank == o.rb && key >= bottom ? w : (uint64_t)0, SumU64());
                            s_bottom = rank_weight(sh.root, o.rb) * ((double)sum * inv_scale);
                        }
                    }
                    if (cut_p) {
                        int cell;
                        uint64_t thr;
                        crossing(s_bottom, cell, thr);
                        bottom = max(bottom, level_in(cell, w, thr));
                    }
                    if (have && key >= bottom) keep(x, sh.few[lane].y);
                    if (t == 0) sh.few_cut = bottom;
                }
                __syncthreads();
                return key_value(uniform(sh.few_cut));
            }
        }
        // First the bottom cell by top-k (each token counts 1), then the
        // crossing cell by top-p (each token counts its weight).
#pragma unroll 1
        for (int step = 0; step < 2; ++step) {
            int cell;
            uint64_t thr;
            if (step == 0) {
                if (o.rb == kRankNone) continue;
                cell = o.rb;
                thr = thr_k;
            } else {
                if (!cut_p) break;
                if (t == 0) crossing(s_bottom, sh.cross, sh.tc);
                __syncthreads();
                cell = uniform(sh.cross);
                thr = sh.tc;
            }
            if (thr) {
                uint32_t found = one_key;
                if (!one_key) {
                    const SelectResult r = select_level<NT>(
                        [&](auto fn) {
                            undecided([&](float x, uint32_t, int rank, double h) {
                                const uint32_t key = order_key(x);
                                if (rank == cell && key >= bottom) fn(key, step ? fx(h) : (uint64_t)1);
                            });
                        },
                        [&](uint64_t) { return thr; }, sh.sel, key_at(cell, -0.6), key_at(cell, 0.6));
                    found = r.total ? r.level : 0u;
                }
                bottom = max(bottom, found);
            }
            if (step == 0 && o.rb <= o.top && cut_p) {
                uint64_t sum = 0;
                if (one_key) {
                    sum = t == 0 && one_key >= bottom ? sh.hist[o.top - o.rb] : 0;
                } else {
                    undecided([&](float x, uint32_t, int rank, double h) {
                        if (rank == o.rb && order_key(x) >= bottom) sum += fx(h);
                    });
                }
                sum = block_reduce<NT>(sum, SumU64(), sh.red64);
                s_bottom = rank_weight(sh.root, o.rb) * ((double)sum * inv_scale);
            }
        }
        cut = bottom;
        if (one_key) {
            one_weight = one_key >= cut ? mass_of(o, sh.root, key_value(one_key)) : 0.0;
            if (one_key >= cut) count += (uint32_t)sh.pre[t];
        } else {
            // The kept among them, added to their segments.
            undecided([&](float x, uint32_t idx, int, double) {
                if (order_key(x) >= cut) keep(x, idx);
            });
        }
        __syncthreads();
    }
    return key_value(cut);
}

// The draws, from sh.sub, sh.subc and sh.pre of the row's `subs` segments (no
// more than NT) and the kept tokens' count (of each thread).  Returns the kept
// mass.
template <int DT, bool VEC, int NT, class Shared>
__device__ __forceinline__ double draw_row(Shared& sh, const GivenParams& p, int64_t b, const void* row, const Deal& d,
                                           uint32_t subs, const RowIn& in, const RowPlan& o, float low, uint32_t count,
                                           double one_weight)
{
    constexpr int GN = Group<DT>::N;
    const int t = threadIdx.x, lane = t & (kWave - 1), w = t / kWave;
    const double inv_scale = ldexp(1.0, -p.bits);
    count = (uint32_t)block_reduce<NT>((uint64_t)count, SumU64(), sh.red64);
    const double mine = sh.sub[t] + one_weight * sh.pre[t] + (double)sh.subc[t] * inv_scale;
    double S;
    const double prefix = block_exclusive_sum_f64<NT>(mine, sh.redf, S);
    sh.sub[t] = mine > 0.0 ? prefix + mine : -1.0;
    sh.pre[t] = prefix;
    __syncthreads();
    if (t == 0) p.out_count[b] = (int32_t)count;
    for (int64_t n = w; n < p.N; n += (NT / kWave)) {
        const double u = p.u_f64 ? ((const double*)p.uniforms)[b * p.N + n] : (double)((const float*)p.uniforms)[b * p.N + n];
        int token = -1;
        float xt = 0.0f;  // its logit
        if (u == u) {
            const double at = (u < 0.0 ? 0.0 : u) * S;
            // The first segment whose running sum exceeds `at`.
            uint32_t lo = 0xFFFFFFFFu;
#pragma unroll 1
            for (uint32_t i = 0; i < subs && lo == 0xFFFFFFFFu && u < 1.0; i += kWave) {
                const uint64_t over = lanes(sh.sub[i + lane] > at);
                if (over) lo = i + (uint32_t)__builtin_ctzll(over);
            }
            if (lo != 0xFFFFFFFFu) {
                double run = sh.pre[lo];
                const uint32_t own = lo / d.spw, s0 = own * d.steps + (lo - own * d.spw) * d.sps;
                const uint32_t s1 = min(s0 + d.sps, (own + 1) * d.steps);
                u32x4 raw[kSubSteps];
#pragma unroll
                for (int k = 0; k < kSubSteps; ++k)
                    raw[k] = load_raw<DT, VEC>(row, min(s0 + k, s1 - 1) * kWave + lane, d.groups, p.V);
                bool open = true;
#pragma unroll 1
                for (uint32_t i = s0; i < s1 && open; ++i) {
                    const uint32_t g = i * kWave + lane;
                    float x[GN];
                    tokens_of<DT>(raw[0], g, true, p.V, x);
#pragma unroll
                    for (int k = 0; k + 1 < kSubSteps; ++k) raw[k] = raw[k + 1];
                    raw[kSubSteps - 1] =
                        load_raw<DT, VEC>(row, min(i + kSubSteps, s1 - 1) * kWave + lane, d.groups, p.V);
                    double wg[GN], sum = 0.0;
                    int mine_at = -1;  // this lane's last token with mass
                    float x_at = 0.0f;
#pragma unroll
                    for (int j = 0; j < GN; ++j) {
                        wg[j] = x[j] >= low ? mass_of(o, sh.root, x[j]) : 0.0;
                        sum += wg[j];
                        if (wg[j] > 0.0) {
                            mine_at = (int)(g * GN + j);
                            x_at = x[j];
                        }
                    }
                    double all;
                    const double inc = wave_inclusive_sum(sum, all);
                    const double prev = wave_shift_up1(inc);
                    const uint64_t hit = lanes(run + inc > at && mine_at >= 0), any = lanes(mine_at >= 0);
                    if (hit) {
                        // The first of the lane's tokens past `at`.
                        double a = run + (lane ? prev : 0.0);
                        bool here = true;
#pragma unroll
                        for (int j = 0; j < GN; ++j) {
                            a += wg[j];
                            if (here && a > at && wg[j] > 0.0) {
                                mine_at = (int)(g * GN + j);
                                x_at = x[j];
                                here = false;
                            }
                        }
                    }
                    if (any) {  // the lane that holds it, or so far the last with mass
                        const int L = hit ? (int)__builtin_ctzll(hit) : 63 - (int)__builtin_clzll(any);
                        token = __builtin_amdgcn_readlane(mine_at, L);
                        xt = lane_value(x_at, L);
                    }
                    open = !hit;
                    run += all;
                }
            } else {
                // At or past the end: the row's last kept token of positive weight.
#pragma unroll 1
                for (int64_t i = (int64_t)((d.groups + kWave - 1) / kWave) - 1; i >= 0 && token < 0; --i) {
                    const uint32_t g = (uint32_t)i * kWave + lane;
                    float x[GN], x_at = 0.0f;
                    tokens_of<DT>(load_raw<DT, VEC>(row, g, d.groups, p.V), g, true, p.V, x);
                    int mine_at = -1;
#pragma unroll
                    for (int j = 0; j < GN; ++j)
                        if (x[j] >= low && weight_of(o, sh.root, x[j]) > 0.0) {
                            mine_at = (int)(g * GN + j);
                            x_at = x[j];
                        }
                    const uint64_t any = lanes(mine_at >= 0);
                    if (any) {
                        const int L = 63 - (int)__builtin_clzll(any);
                        token = __builtin_amdgcn_readlane(mine_at, L);
                        xt = lane_value(x_at, L);
                    }
                }
            }
        }
        if (lane == 0) {
            p.out_token[b * p.N + n] = token;
            if (p.out_logprob) {
                float lp = __uint_as_float(0x7FC00000u);
                if (token >= 0)
                    // (the mass is measured from the max's cell, not from the max itself)
                    lp = (float)(((double)xt - (double)o.m) / (double)in.T - (log(S) - o.hm * (kLn2 / kOctave)));
                p.out_logprob[b * p.N + n] = lp;
            }
        }
    }
    return S;
}

// The first pass over a row by one workgroup: its max, and where it wants
// one the histogram in LDS (two copies) over lattice c.
template <int DT, bool VEC, int NT, class Shared>
__device__ __forceinline__ void row_first_pass(Shared& sh, const GivenParams& p, const void* row, const Deal& d,
                                               const RowIn& in, const Fixed& fx, Cells& c, FirstPass& f, float& m)
{
    constexpr int GN = Group<DT>::N;
    const int t = threadIdx.x, lane = t & (kWave - 1), w = t / kWave;
    c = Cells{};
    float anchor = -INFINITY;
    if (in.want_hist) {
        // The anchor: the max of every thread's first group.
        float x[GN];
        const uint32_t g = (uint32_t)w * d.steps * kWave + lane;
        tokens_of<DT>(load_raw<DT, VEC>(row, g, d.groups, p.V), g, true, p.V, x);
#pragma unroll
        for (int j = 0; j < GN; ++j) anchor = fmaxf(anchor, x[j]);
        for (int i = t; i < kSlots; i += NT) {
            sh.hist[i] = sh.hist[kCopy + i] = 0;
            sh.cnt[i] = 0;
        }
        anchor = uniform(block_reduce<NT>(anchor, MaxF32(), (float*)sh.redf));
    }
    m = -INFINITY;
    bool hist = in.want_hist && anchor > -INFINITY && anchor < INFINITY;
    // At most three turns: for the max alone where the first tokens were all
    // masked, with a histogram, and once more where the max lay above its window.
#pragma unroll 1
    for (int turn = 0; turn < 3; ++turn) {
        if (hist) c = make_cells(anchor, in.T);
        if (!hist)
            f = first_pass<DT, VEC, kPassMax, false>(row, d, p.V, c, fx, sh);
        else if (in.use_k && c.fast)
            f = first_pass<DT, VEC, kPassCount, true>(row, d, p.V, c, fx, sh);
        else if (in.use_k)
            f = first_pass<DT, VEC, kPassCount, false>(row, d, p.V, c, fx, sh);
        else if (c.fast)
            f = first_pass<DT, VEC, kPassHist, true>(row, d, p.V, c, fx, sh);
        else
            f = first_pass<DT, VEC, kPassHist, false>(row, d, p.V, c, fx, sh);
        m = uniform(block_reduce<NT>(
            f.m, [](float a, float e) { return __builtin_elementwise_maximum(a, e); }, (float*)sh.redf));
        if (!in.want_hist || !(m > -INFINITY && m < INFINITY)) break;
        double h;
        if (hist && uniform(slot_of(c, m, h)) < kSlots) break;
        // Anchored at the row's own max, no token lies above the window.
        anchor = m;
        if (hist) {
            for (int i = t; i < kSlots; i += NT) {
                sh.hist[i] = sh.hist[kCopy + i] = 0;
                sh.cnt[i] = 0;
            }
            __syncthreads();
        }
        hist = true;
    }
}

// The token of a greedy row: the lowest index that holds the max.  Every
// thread knows the step that first held its own.
template <int DT, bool VEC, int NT, class Shared>
__device__ __forceinline__ int greedy_token(Shared& sh, const GivenParams& p, const void* row, const Deal& d,
                                            const FirstPass& f, float m)
{
    constexpr int GN = Group<DT>::N;
    const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
    uint32_t first = 0xFFFFFFFFu;
    if (f.m == m) {
        const uint32_t g = ((uint32_t)w * d.steps + f.at) * kWave + lane;
        float x[GN];
        tokens_of<DT>(load_raw<DT, VEC>(row, g, d.groups, p.V), g, true, p.V, x);
#pragma unroll
        for (int j = GN - 1; j >= 0; --j)
            if (x[j] == m) first = g * GN + j;
    }
    return (int)block_reduce<NT>(first, MinU32(), (uint32_t*)sh.red64);
}

// One row on one workgroup.
template <int DT, bool VEC, int NT, class Shared>
__device__ __forceinline__ void whole_row(Shared& sh, const GivenParams& p, int64_t b)
{
    constexpr int GN = Group<DT>::N;
    constexpr uint32_t kCap = Shared::kCap;
    const int t = threadIdx.x, lane = t & (kWave - 1), w = t / kWave;
    const void* row = row_of<DT>(p, b);
    const Deal d = deal_out<DT, NT>(p.V);
    const Fixed fx(ldexp(1.0, p.bits));
    const RowIn in = row_in(p, b);

    if (t < kOctave) sh.root[t] = kRoot[t];
    sh.sub[t] = 0.0;
    sh.pre[t] = 0.0;
    sh.subc[t] = 0;
    if (t == 0) sh.list_n = sh.few_n = 0;

    Cells c;
    FirstPass f;
    float m;
    row_first_pass<DT, VEC, NT>(sh, p, row, d, in, fx, c, f, m);
    if (row_error(in, m) || in.greedy) {
        const int token = row_error(in, m) ? -1 : greedy_token<DT, VEC, NT>(sh, p, row, d, f, m);
        store_single<NT>(p, b, token);
        if (p.out_probs)
            for (int64_t i = t; i < p.V; i += NT) p.out_probs[b * p.V + i] = i == token ? 1.0f : 0.0f;
        return;
    }
    uint32_t finite = 0;
    if (in.use_k) finite = (uint32_t)block_reduce<NT>((uint64_t)(lane == 0 ? f.finite : 0), SumU64(), sh.red64);

    // ---- the cells of the cuts -------------------------------------------
    const RowPlan o = plan_row<NT>(sh, in, c, m, finite, true, p.bits);

    // ---- pass 2: masses of the surely kept, list of the undecided -----------
    // Slots above s_sure (kGivenLevel: tokens from o.floor_x up) are surely kept;
    // those from s_und to it, and s_bot where it is apart from them, undecided.
    const int s_sure = o.mode == kGivenLevel || o.r_lo > o.top ? -1 : o.top - o.r_lo;
    const int s_und = o.r_hi > o.top ? 0 : o.top - o.r_hi, s_bot = o.top - o.rb;
    const bool apart = o.mode == kGivenCells && o.rb <= o.top && o.rb > o.r_hi;
    const bool below = o.mode == kGivenCells && o.rb == o.top + 1;  // the undecided are those below the window
    double* const cell_mass = (double*)(sh.hist + kCopy);
    for (int i = t; i <= kSlots; i += NT)
        cell_mass[i] = i > s_sure && i <= o.top ? rank_weight(sh.root, o.top - i) : 0.0;
    __syncthreads();
    uint32_t count = 0;                     // kept tokens, of each lane and of lane 0's wave
    uint32_t kmin = 0xFFFFFFFFu, kmax = 0;  // keys of the undecided that are not listed
    {
        double acc[2] = {0.0, 0.0};
        uint32_t seg_left = d.sps, seg = (uint32_t)w * d.spw, sure_n = 0, und_n = 0;
        uint32_t next = 0, left = 0;  // this wave's next place in the list, and how many it has
        // Lists the tokens whose lanes are in some[j], n in all.
        auto put = [&](const float (&x)[GN], const uint64_t (&some)[GN], uint32_t n, uint32_t g) {
            und_n += n;
            if (n > left) {
                // The next places of the list, in 64s (one LDS atomic): what is
                // left of the last ones stays empty.
                if (lane < left && next + lane < kCap) sh.list[next + lane].x = kEmpty;
                left = (n + kWave - 1) / kWave * kWave;
                uint32_t at = 0;
                if (lane == 0) at = atomicAdd(&sh.list_n, left);
                next = uniform(at);
            }
            left -= n;
#pragma unroll
            for (int j = 0; j < GN; ++j) {
                if (some[j] >> lane & 1) {
                    const uint32_t mine = next + __builtin_amdgcn_mbcnt_hi(
                        (uint32_t)(some[j] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)some[j], 0));
                    if (mine < kCap) {
                        sh.list[mine] = make_uint2(__float_as_uint(x[j]), g * GN + j);
                    } else {
                        const uint32_t key = order_key(x[j]);
                        kmin = min(kmin, key);
                        kmax = max(kmax, key);
                    }
                }
                next += (uint32_t)__builtin_popcountll(some[j]);
            }
        };
        auto end_step = [&](uint32_t i) {
            if (--seg_left == 0 || i + 1 == d.steps) {
                const double sum = wave_reduce(acc[0] + acc[1], SumF64());
                if (lane == 0) {
                    sh.sub[seg] = sum;
                    sh.pre[seg] = (double)und_n;
                }
                acc[0] = acc[1] = 0.0;
                und_n = 0;
                ++seg;
                seg_left = d.sps;
            }
        };
        if (o.mode == kGivenLevel && o.c.fast) {
            stream_row<DT, VEC>(row, d, p.V, [&](uint32_t i, uint32_t, const float (&x)[GN]) {
                double e[GN], q[GN], h[GN];
                float xc[GN];
                int sl[GN];
#pragma unroll
                for (int j = 0; j < GN; ++j) {
                    const bool in = x[j] >= o.floor_x;
                    xc[j] = fmaxf(in ? x[j] : o.c.lo, o.c.lo);
                    sure_n += (uint32_t)__builtin_popcountll(lanes(in));
                }
                slots_of<GN, true>(o.c, xc, sl, h);
#pragma unroll
                for (int j = 0; j < GN; ++j) e[j] = cell_mass[min((uint32_t)sl[j], (uint32_t)kSlots)];
                in_cells(h, q);
#pragma unroll
                for (int j = 0; j < GN; ++j) acc[j & 1] = fma(e[j], q[j], acc[j & 1]);
                end_step(i);
            });
        } else if (o.c.fast && !below) {
            // (a token below o.floor_x falls into a slot of no mass below s_und)
            const float from = fmaxf(o.floor_x, o.c.lo);
            stream_row<DT, VEC>(row, d, p.V, [&](uint32_t i, uint32_t g, const float (&x)[GN]) {
                float most = x[0];
#pragma unroll
                for (int j = 1; j < GN; ++j) most = fmaxf(most, x[j]);
                if (lanes(most >= o.floor_x)) {  // uniform: most steps of many rows hold no such token
                    uint64_t some[GN];
                    uint32_t n = 0;
                    double e[GN], q[GN], h[GN];
                    float xc[GN];
                    int sl[GN];
#pragma unroll
                    for (int j = 0; j < GN; ++j) xc[j] = fmaxf(x[j], from);
                    slots_of<GN, true>(o.c, xc, sl, h);
#pragma unroll
                    for (int j = 0; j < GN; ++j) e[j] = cell_mass[min((uint32_t)sl[j], (uint32_t)kSlots)];
                    in_cells(h, q);
#pragma unroll
                    for (int j = 0; j < GN; ++j) {
                        // (one comparison to a mask: masks are combined in scalar registers)
                        const uint64_t up = lanes(sl[j] > s_sure);
                        sure_n += (uint32_t)__builtin_popcountll(up);
                        some[j] = lanes(sl[j] >= s_und) & ~up;
                        if (apart) some[j] |= lanes(sl[j] == s_bot);
                        n += (uint32_t)__builtin_popcountll(some[j]);
                    }
#pragma unroll
                    for (int j = 0; j < GN; ++j) acc[j & 1] = fma(e[j], q[j], acc[j & 1]);
                    if (n) put(x, some, n, g);  // uniform
                }
                end_step(i);
            });
        } else {
            // Rows whose window reaches past the finite logits, and top-k cuts
            // below the window.
            stream_row<DT, VEC>(row, d, p.V, [&](uint32_t i, uint32_t g, const float (&x)[GN]) {
                uint64_t some[GN];
                uint32_t n = 0;
#pragma unroll
                for (int j = 0; j < GN; ++j) {
                    double h;  // (finite tokens only: a -inf here would make the sum NaN)
                    const bool in = x[j] >= o.floor_x;
                    const int sl = slot_of(o.c, fmaxf(x[j], o.floor_x), h);
                    const bool sure = o.mode == kGivenLevel ? in : in & (sl > s_sure);
                    if (sure & (sl >= 0)) acc[0] = fma(cell_mass[min(sl, kSlots)], in_cell(h), acc[0]);
                    sure_n += (uint32_t)__builtin_popcountll(lanes(sure));
                    const bool und = below ? sl < 0 : (sl >= s_und) | (apart & (sl == s_bot));
                    some[j] = o.mode == kGivenLevel ? 0 : lanes(in & !sure & und);
                    n += (uint32_t)__builtin_popcountll(some[j]);
                }
                if (n) put(x, some, n, g);  // uniform
                end_step(i);
            });
        }
        if (lane == 0) count += sure_n;
        if (lane < left && next + lane < kCap) sh.list[next + lane].x = kEmpty;
    }
    __syncthreads();

    // ---- the exact cut level ---------------------------------------------
    double one_weight;
    const float low =
        resolve_row<DT, NT>(sh, p, row, d, in, o, fx, sh.list_n <= kCap, sh.list_n, kmin, kmax, count, one_weight);

    // ---- the draws ---------------------------------------------------------
    const double S =
        draw_row<DT, VEC, NT>(sh, p, b, row, d, d.spw * Shared::kWaves, in, o, low, count, one_weight);

    // ---- the distribution ---------------------------------------------------
    if (p.out_probs) {
        const double inv = 1.0 / S;
        float* out = p.out_probs + b * p.V;
        const bool vec = p.V % 4 == 0 && (uintptr_t)p.out_probs % 16 == 0;
        stream_row<DT, VEC>(row, d, p.V, [&](uint32_t, uint32_t g, const float (&x)[GN]) {
            float q[GN];
            bool any = false;
#pragma unroll
            for (int j = 0; j < GN; ++j) {
                q[j] = 0.0f;
                any |= x[j] >= low;
            }
            if (lanes(any)) {
#pragma unroll
                for (int j = 0; j < GN; ++j)
                    if (x[j] >= low) q[j] = (float)(weight_of(o, sh.root, x[j]) * inv);
            }
            const int64_t i0 = (int64_t)g * GN;
            if (vec && i0 + GN <= p.V) {
#pragma unroll
                for (int j = 0; j < GN; j += 4) *(f32x4*)(out + i0 + j) = f32x4{q[j], q[j + 1], q[j + 2], q[j + 3]};
            } else {
#pragma unroll
                for (int j = 0; j < GN; ++j)
                    if (i0 + j < p.V) out[i0 + j] = q[j];
            }
        });
    }
}

template <int DT, bool VEC, int NT>
__global__ __launch_bounds__(NT) void given_row_kernel(GivenParams p)
{
    __shared__ GivenShared<NT> sh;
    whole_row<DT, VEC, NT>(sh, p, blockIdx.x);
}

// ---------------------------------------------------------------------------
// Rows split over workgroups.  A part is 32 KB of a row, held in the registers
// of one 256-thread workgroup; three or four launches (one more with the
// distribution):
//
//   given_first_kernel  per row: first pass and cells of the cuts, where there
//                       are rows enough to fill the device; else
//   given_hist_kernel   per part: max and histogram, over a lattice anchored
//                       at the max of 256 groups spread over the whole row
//                       (every part of a row reads the same ones)
//   given_plan_kernel   per row: joins the histograms, finds the cells of the cuts
//   given_mass_kernel   per part: masses of the surely kept tokens per segment,
//                       list of the undecided
//   given_draw_kernel   per row: exact cut, draws
//   given_probs_kernel  per part: probabilities
//
// Parts of 32 KB put a row of 128256 float32 logits on 16 workgroups and keep
// LDS small enough for 7 waves a SIMD (64 KB parts of 512 threads: 36 us for
// the masses of 256 rows, 32 KB 33).  One such row: 6.5, 11, 8, 15 and with
// probabilities 5.5 us; 256 rows: first pass 32, masses 33, draws 19 us.
//
// Launch boundaries are the only joins, so nothing waits inside a kernel and
// the workspace needs no initial value.  What a part cannot do for itself
// (a max above the window, a window that reaches past the finite logits, a
// top-k cut below the window) is left to one workgroup, which runs the
// unsplit row in given_draw_kernel.
// ---------------------------------------------------------------------------
constexpr int kPartThreads = 256;
constexpr int kPartWaves = kPartThreads / kWave;
constexpr int kPartSteps = 8;                                        // groups of a lane
constexpr int kPartSegs = kPartWaves * kPartSteps / kSubSteps;       // segments
constexpr int kPartCap = 1024;                                       // listed tokens
constexpr int kMaxParts = 64;                                        // of a row: its segments fit one per thread
constexpr int kDrawThreads = 512;
constexpr int kMassCells = 2304;                                     // kept cells of a split row, at most
static_assert(kMaxParts * kPartSegs <= kDrawThreads, "one segment per thread of given_draw_kernel");

template <int DT>
constexpr int part_tokens() { return kPartThreads * kPartSteps * Group<DT>::N; }

struct PartHead {  // given_hist_kernel
    float anchor, m;
    uint32_t finite, first;  // top-k rows: tokens above -inf; greedy rows: lowest index of m
    int lo, hi;              // its slots of the histogram are lo .. hi
    int ok;                  // the lattice is a fast one
    int pad;
};
struct PartTail {  // given_mass_kernel
    uint32_t listed, sure, kmin, kmax;
};
struct RowState {
    RowPlan o;
    double s_above, a_lo, S;
    float low;
    uint32_t n_above;
    int token;  // kGivenGreedy, kGivenError
};

struct GivenWork {
    RowState* state;   // [B]
    PartHead* head;    // [B][C]
    PartTail* tail;    // [B][C]
    uint64_t* joined;  // [B][kSlots]: the histogram at the cells of the cuts
    uint64_t* hist;    // [B][C][kSlots] (given_hist_kernel)
    uint32_t* cnt;     // [B][C][kSlots] (given_hist_kernel)
    double* sub;       // [B][C][kPartSegs]
    uint32_t* und;     // [B][C][kPartSegs]
    uint2* list;       // [B][C][kPartCap]
    int C;
};

// The groups of this part in registers: step i of wave w is group
// (part 32 + w 8 + i) 64 + lane of the row.
template <int DT, bool VEC>
__device__ __forceinline__ uint32_t load_part(const void* row, int part, uint32_t groups, int64_t V,
                                              u32x4 (&raw)[kPartSteps])
{
    const uint32_t g0 = ((uint32_t)part * kPartWaves + uniform(threadIdx.x / kWave)) * kPartSteps * kWave;
#pragma unroll
    for (int i = 0; i < kPartSteps; ++i)
        raw[i] = load_raw<DT, VEC>(row, g0 + i * kWave + (threadIdx.x & (kWave - 1)), groups, V);
    return g0;
}

template <int DT, bool VEC>
__global__ __launch_bounds__(kPartThreads) void given_hist_kernel(GivenParams p, GivenWork wk)
{
    constexpr int GN = Group<DT>::N;
    __shared__ uint64_t hist[kSlots + kWave];
    __shared__ uint32_t cnt[kSlots + kWave];
    __shared__ uint64_t red[kPartWaves];
    const int t = threadIdx.x, lane = t & (kWave - 1);
    const int64_t b = blockIdx.x / (uint32_t)wk.C;
    const int part = (int)(blockIdx.x % (uint32_t)wk.C);
    const void* row = row_of<DT>(p, b);
    const uint32_t groups = (uint32_t)((p.V + GN - 1) / GN), whole = (uint32_t)(p.V / GN);
    const RowIn in = row_in(p, b);
    u32x4 raw[kPartSteps];
    const uint32_t g0 = load_part<DT, VEC>(row, part, groups, p.V, raw);
    float anchor = -INFINITY;
    if (in.want_hist) {
        float x[GN];
        const uint32_t g = (uint32_t)((uint64_t)groups * t / kPartThreads);
        tokens_of<DT>(load_raw<DT, VEC>(row, g, groups, p.V), g, true, p.V, x);
#pragma unroll
        for (int j = 0; j < GN; ++j) anchor = fmaxf(anchor, x[j]);
        for (int i = t; i < kSlots; i += kPartThreads) hist[i] = 0;
        if (in.use_k)
            for (int i = t; i < kSlots; i += kPartThreads) cnt[i] = 0;
        anchor = uniform(block_reduce<kPartThreads>(anchor, MaxF32(), (float*)red));
    }
    Cells c = {};
    if (anchor > -INFINITY && anchor < INFINITY) c = make_cells(anchor, in.T);
    const Fixed fx(ldexp(1.0, p.bits));
    float m = -INFINITY;
    uint32_t finite = 0;
    const uint32_t outside = kSlots + lane;
    // fn(step, group, tokens)
    auto each = [&](auto fn) {
#pragma unroll
        for (int i = 0; i < kPartSteps; ++i) {
            const uint32_t g = g0 + i * kWave;
            if (g >= groups) break;  // uniform
            float x[GN];
            tokens_of<DT>(raw[i], g + lane, g + kWave > whole, p.V, x);
            fn(g + lane, x);
        }
    };
    auto bin = [&](const float (&x)[GN], auto count) {
        float xc[GN];
        int sl[GN];
        double h[GN];
        uint64_t q[GN];
#pragma unroll
        for (int j = 0; j < GN; ++j) xc[j] = fmaxf(x[j], c.lo);
        slots_of<GN, true>(c, xc, sl, h);
        fx(h, q);
#pragma unroll
        for (int j = 0; j < GN; ++j) {
            const uint32_t at = min((uint32_t)sl[j], outside);
            atomicAdd((unsigned long long*)&hist[at], (unsigned long long)q[j]);
            if constexpr (count.value) {
                atomicAdd(&cnt[at], 1u);
                finite += (uint32_t)__builtin_popcountll(lanes(x[j] > -INFINITY));
            }
        }
    };
    auto most = [&](const float (&x)[GN]) {
#pragma unroll
        for (int j = 0; j < GN; ++j) m = __builtin_elementwise_maximum(m, x[j]);
    };
    if (c.fast && in.use_k)
        each([&](uint32_t, const float (&x)[GN]) {
            most(x);
            bin(x, std::true_type());
        });
    else if (c.fast)
        each([&](uint32_t, const float (&x)[GN]) {
            most(x);
            bin(x, std::false_type());
        });
    else
        each([&](uint32_t, const float (&x)[GN]) { most(x); });
    m = uniform(block_reduce<kPartThreads>(
        m, [](float a, float e) { return __builtin_elementwise_maximum(a, e); }, (float*)red));
    PartHead o = {anchor, m, 0, 0xFFFFFFFFu, 1, 0, c.fast, 0};
    if (in.greedy) {
        uint32_t first = 0xFFFFFFFFu;
        each([&](uint32_t g, const float (&x)[GN]) {
#pragma unroll
            for (int j = GN - 1; j >= 0; --j)
                if (x[j] == m) first = min(first, g * GN + j);
        });
        o.first = block_reduce<kPartThreads>(first, MinU32(), (uint32_t*)red);
    } else if (c.fast) {
        if (in.use_k) o.finite = (uint32_t)block_reduce<kPartThreads>((uint64_t)(lane == 0 ? finite : 0), SumU64(), red);
        // Its slots: from the lowest in use to the max's.
        double h;
        const int hi = min(uniform(slot_of(c, m, h)), kSlots - 1);
        int lo = kSlots;
        for (int i = t; i <= hi; i += kPartThreads)
            if (lo == kSlots && hist[i]) lo = i;
        lo = block_reduce<kPartThreads>(lo, MinI(), (int*)red);
        const size_t at = ((size_t)b * wk.C + part) * kSlots;
        for (int i = lo + t; i <= hi; i += kPartThreads) wk.hist[at + i] = hist[i];
        if (in.use_k)
            for (int i = lo + t; i <= hi; i += kPartThreads) wk.cnt[at + i] = cnt[i];
        o.lo = lo;
        o.hi = hi;
    }
    if (t == 0) wk.head[b * wk.C + part] = o;
}

// A planned row's state for the kernels that follow.
template <int NT, class Shared>
__device__ __forceinline__ void hand_on(Shared& sh, const GivenWork& wk, int64_t b, RowPlan o)
{
    const int t = threadIdx.x;
    const int kept = o.mode == kGivenLevel || o.r_lo > o.top ? o.top + 1 : o.r_lo;  // cells
    if (!o.c.fast || (o.mode == kGivenCells && o.rb == o.top + 1) || kept > kMassCells) o.mode = kGivenAlone;
    __syncthreads();
    if (o.mode == kGivenCells) {
        uint64_t* joined = wk.joined + (size_t)b * kSlots;
        for (int r = o.r_lo + t; r <= o.r_hi; r += NT) joined[o.top - r] = sh.hist[o.top - r];
        if (t == 0 && o.rb <= o.top) joined[o.top - o.rb] = sh.hist[o.top - o.rb];
    }
    if (t == 0) {
        RowState& st = wk.state[b];
        st.o = o;
        st.s_above = sh.s_above;
        st.a_lo = sh.a_lo;
        st.n_above = sh.n_above;
    }
}

typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The sums over the parts of their slots lo[i] .. hi[i], to LDS.
template <int NT, class Pair, class Word>
__device__ __forceinline__ void merge_parts(const Word* parts, const int* lo, const int* hi, int C, Word* out)
{
    constexpr int PER = kSlots / (2 * NT), AT_ONCE = 8;
    const int t = threadIdx.x;
    Pair sum[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) sum[k] = Pair{0, 0};
#pragma unroll 1
    for (int i0 = 0; i0 < C; i0 += AT_ONCE) {
        Pair v[AT_ONCE][PER];
        int a[AT_ONCE], e[AT_ONCE];
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            const int i = min(i0 + j, C - 1);
            a[j] = uniform(lo[i]);
            e[j] = uniform(hi[i]);
            const Pair* from = (const Pair*)(parts + (size_t)i * kSlots);
#pragma unroll
            for (int k = 0; k < PER; ++k) v[j][k] = from[min(max(t + k * NT, min(a[j], e[j]) >> 1), max(e[j], 0) >> 1)];
            if (i0 + j >= C) e[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int sl = 2 * (t + k * NT);
                sum[k].x += sl >= a[j] && sl <= e[j] ? v[j][k].x : 0;
                sum[k].y += sl + 1 >= a[j] && sl + 1 <= e[j] ? v[j][k].y : 0;
            }
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) ((Pair*)out)[t + k * NT] = sum[k];
}

template <int NT>
__global__ __launch_bounds__(NT) void given_plan_kernel(GivenParams p, GivenWork wk)
{
    typedef GivenShared<NT> Shared;
    __shared__ Shared sh;
    __shared__ int s_lo[kMaxParts], s_hi[kMaxParts];
    const int t = threadIdx.x;
    const int64_t b = blockIdx.x;
    const RowIn in = row_in(p, b);
    const PartHead* head = wk.head + b * wk.C;
    PartHead mine = {-INFINITY, -INFINITY, 0, 0xFFFFFFFFu, 1, 0, 1, 0};
    if (t < wk.C) {
        mine = head[t];
        s_lo[t] = mine.lo;
        s_hi[t] = mine.hi;
    }
    if (t < kOctave) sh.root[t] = kRoot[t];
    const float m = uniform(block_reduce<NT>(
        mine.m, [](float a, float e) { return __builtin_elementwise_maximum(a, e); }, (float*)sh.redf));
    RowState& st = wk.state[b];
    if (row_error(in, m) || in.greedy) {
        const uint32_t first = block_reduce<NT>(mine.m == m ? mine.first : 0xFFFFFFFFu, MinU32(), (uint32_t*)sh.red64);
        if (t == 0) {
            st.o.mode = row_error(in, m) ? kGivenError : kGivenGreedy;
            st.token = row_error(in, m) ? -1 : (int)first;
        }
        return;
    }
    Cells c = {};
    uint32_t finite = 0;
    bool alone = false;
    if (in.want_hist) {
        alone = !head[0].ok;
        if (!alone) {
            c = make_cells(uniform(head[0].anchor), in.T);
            double h;
            alone = uniform(slot_of(c, m, h)) >= kSlots;
        }
        if (!alone) {
            if (in.use_k) finite = (uint32_t)block_reduce<NT>((uint64_t)mine.finite, SumU64(), sh.red64);
            // Four pairs of slots a thread, eight parts' words of them in flight
            // together: what other workgroups wrote takes 1 to 2 us to arrive,
            // however many loads wait for it (16 parts: two at a time 8 us, eight 5).  A
            // pair outside a part's range reads the range's end and drops it.
            merge_parts<NT, u64x2>(wk.hist + (size_t)b * wk.C * kSlots, s_lo, s_hi, wk.C, sh.hist);
            if (in.use_k) merge_parts<NT, u32x2>(wk.cnt + (size_t)b * wk.C * kSlots, s_lo, s_hi, wk.C, sh.cnt);
        }
    }
    __syncthreads();
    if (alone) {
        if (t == 0) st.o.mode = kGivenAlone;
        return;
    }
    hand_on<NT>(sh, wk, b, plan_row<NT>(sh, in, c, m, finite, false, p.bits));
}

template <int DT, bool VEC, int NT>
__global__ __launch_bounds__(NT) void given_first_kernel(GivenParams p, GivenWork wk)
{
    __shared__ GivenShared<NT> sh;
    const int t = threadIdx.x, lane = t & (kWave - 1);
    const int64_t b = blockIdx.x;
    const void* row = row_of<DT>(p, b);
    const Deal d = deal_out<DT, NT>(p.V);
    const Fixed fx(ldexp(1.0, p.bits));
    const RowIn in = row_in(p, b);
    if (t < kOctave) sh.root[t] = kRoot[t];
    Cells c;
    FirstPass f;
    float m;
    row_first_pass<DT, VEC, NT>(sh, p, row, d, in, fx, c, f, m);
    if (row_error(in, m) || in.greedy) {
        const int token = row_error(in, m) ? -1 : greedy_token<DT, VEC, NT>(sh, p, row, d, f, m);
        if (t == 0) {
            wk.state[b].o.mode = token < 0 ? kGivenError : kGivenGreedy;
            wk.state[b].token = token;
        }
        return;
    }
    uint32_t finite = 0;
    if (in.use_k) finite = (uint32_t)block_reduce<NT>((uint64_t)(lane == 0 ? f.finite : 0), SumU64(), sh.red64);
    hand_on<NT>(sh, wk, b, plan_row<NT>(sh, in, c, m, finite, true, p.bits));
}

template <int DT, bool VEC>
__global__ __launch_bounds__(kPartThreads) void given_mass_kernel(GivenParams p, GivenWork wk)
{
    constexpr int GN = Group<DT>::N;
    __shared__ double cell_mass[kMassCells + 1];
    __shared__ double root[kOctave];
    __shared__ uint32_t list_n, sure_all, kmin_all, kmax_all;
    const int t = threadIdx.x, lane = t & (kWave - 1), w = t / kWave;
    const int64_t b = blockIdx.x / (uint32_t)wk.C;
    const int part = (int)(blockIdx.x % (uint32_t)wk.C);
    const RowPlan o = wk.state[b].o;
    if (o.mode != kGivenLevel && o.mode != kGivenCells) return;  // uniform
    const void* row = row_of<DT>(p, b);
    const uint32_t groups = (uint32_t)((p.V + GN - 1) / GN), whole = (uint32_t)(p.V / GN);
    u32x4 raw[kPartSteps];
    const uint32_t g0 = load_part<DT, VEC>(row, part, groups, p.V, raw);
    if (t < kOctave) root[t] = kRoot[t];
    if (t == 0) {
        list_n = sure_all = kmax_all = 0;
        kmin_all = 0xFFFFFFFFu;
    }
    __syncthreads();
    const int s_sure = o.mode == kGivenLevel || o.r_lo > o.top ? -1 : o.top - o.r_lo;
    const int s_und = o.r_hi > o.top ? 0 : o.top - o.r_hi, s_bot = o.top - o.rb;
    const bool apart = o.mode == kGivenCells && o.rb <= o.top && o.rb > o.r_hi;
    // Masses of the surely kept cells from slot s_sure + 1 up, and 0 for every other.
    const uint32_t cells = (uint32_t)(o.top - s_sure);
    for (uint32_t i = t; i < cells; i += kPartThreads) cell_mass[i] = rank_weight(root, o.top - s_sure - 1 - (int)i);
    if (t == 0) cell_mass[cells] = 0.0;
    __syncthreads();
    const size_t at = (size_t)b * wk.C + part;
    uint2* list = wk.list + at * kPartCap;
    uint32_t sure_n = 0, und_n = 0, kmin = 0xFFFFFFFFu, kmax = 0;
    double acc[2] = {0.0, 0.0};
    const bool by_level = o.mode == kGivenLevel;
    const float from = by_level ? o.c.lo : fmaxf(o.floor_x, o.c.lo);
#pragma unroll
    for (int i = 0; i < kPartSteps; ++i) {
        const uint32_t g = g0 + i * kWave;
        if (g < groups) {  // uniform
            float x[GN], xc[GN];
            tokens_of<DT>(raw[i], g + lane, g + kWave > whole, p.V, x);
            float most = x[0];
#pragma unroll
            for (int j = 1; j < GN; ++j) most = fmaxf(most, x[j]);
            if (lanes(most >= o.floor_x)) {  // uniform
                uint64_t some[GN];
                uint32_t n = 0;
                double e[GN], q[GN], h[GN];
                int sl[GN];
                // (a token below floor_x falls into a slot of no mass below s_und,
                // or by a level out of the window)
#pragma unroll
                for (int j = 0; j < GN; ++j)
                    xc[j] = fmaxf(by_level ? (x[j] >= o.floor_x ? x[j] : from) : x[j], from);
                slots_of<GN, true>(o.c, xc, sl, h);
#pragma unroll
                for (int j = 0; j < GN; ++j) e[j] = cell_mass[min((uint32_t)(sl[j] - s_sure - 1), cells)];
                in_cells(h, q);
#pragma unroll
                for (int j = 0; j < GN; ++j) {
                    const uint64_t up = by_level ? lanes(x[j] >= o.floor_x) : lanes(sl[j] > s_sure);
                    sure_n += (uint32_t)__builtin_popcountll(up);
                    some[j] = by_level ? 0 : lanes(sl[j] >= s_und) & ~up;
                    if (apart) some[j] |= lanes(sl[j] == s_bot);
                    n += (uint32_t)__builtin_popcountll(some[j]);
                }
#pragma unroll
                for (int j = 0; j < GN; ++j) acc[j & 1] = fma(e[j], q[j], acc[j & 1]);
                if (n) {  // uniform
                    und_n += n;
                    uint32_t next = 0;
                    if (lane == 0) next = atomicAdd(&list_n, n);
                    next = uniform(next);
#pragma unroll
                    for (int j = 0; j < GN; ++j) {
                        if (some[j] >> lane & 1) {
                            const uint32_t mine = next + __builtin_amdgcn_mbcnt_hi(
                                (uint32_t)(some[j] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)some[j], 0));
                            const uint32_t key = order_key(x[j]);
                            if (mine < kPartCap) list[mine] = make_uint2(__float_as_uint(x[j]), (g + lane) * GN + j);
                            kmin = min(kmin, key);
                            kmax = max(kmax, key);
                        }
                        next += (uint32_t)__builtin_popcountll(some[j]);
                    }
                }
            }
        }
        if (i % kSubSteps == kSubSteps - 1) {
            const double sum = wave_reduce(acc[0] + acc[1], SumF64());
            const size_t seg = at * kPartSegs + w * (kPartSteps / kSubSteps) + i / kSubSteps;
            if (lane == 0) {
                wk.sub[seg] = sum;
                wk.und[seg] = und_n;
            }
            acc[0] = acc[1] = 0.0;
            und_n = 0;
        }
    }
    if (lane == 0) atomicAdd(&sure_all, sure_n);
    if (lanes(kmax != 0)) {  // uniform
        kmin = wave_reduce(kmin, MinU32());
        kmax = ~wave_reduce(~kmax, MinU32());
        if (lane == 0) {
            atomicMin(&kmin_all, kmin);
            atomicMax(&kmax_all, kmax);
        }
    }
    __syncthreads();
    if (t == 0) wk.tail[at] = PartTail{list_n, sure_all, kmin_all, kmax_all};
}

template <int DT, bool VEC, int NT>
__global__ __launch_bounds__(NT) void given_draw_kernel(GivenParams p, GivenWork wk)
{
    typedef GivenShared<NT> Shared;
    constexpr int GN = Group<DT>::N;
    __shared__ Shared sh;
    __shared__ uint32_t s_at[kMaxParts], s_n[kMaxParts];
    const int t = threadIdx.x, lane = t & (kWave - 1), w = t / kWave;
    const int64_t b = blockIdx.x;
    RowState& st = wk.state[b];
    const uint32_t segs = (uint32_t)wk.C * kPartSegs;
    // Everything that does not depend on the row's mode is asked for at once
    // (each wait for memory that other workgroups wrote costs about 1 us).
    const RowState s0 = st;
    double sub = 0.0;
    uint32_t und = 0;
    PartTail tail = {0, 0, 0xFFFFFFFFu, 0};
    if (t < (int)segs) {
        sub = wk.sub[(size_t)b * segs + t];
        und = wk.und[(size_t)b * segs + t];
    }
    if (t < wk.C) tail = wk.tail[(size_t)b * wk.C + t];
    const RowIn in = row_in(p, b);
    const int mode = uniform(s0.o.mode);
    if (mode == kGivenAlone) {
        whole_row<DT, VEC, NT>(sh, p, b);
        return;
    }
    if (mode != kGivenLevel && mode != kGivenCells) {
        store_single<NT>(p, b, uniform(s0.token));
        return;
    }
    const RowPlan o = s0.o;
    const void* row = row_of<DT>(p, b);
    Deal d;
    d.groups = (uint32_t)((p.V + GN - 1) / GN);
    d.steps = segs * kSubSteps;
    d.sps = kSubSteps;
    d.spw = segs;
    if (t < kOctave) sh.root[t] = kRoot[t];
    sh.sub[t] = sub;
    sh.pre[t] = (double)und;
    sh.subc[t] = 0;
    uint32_t count = tail.sure, kmin = tail.kmin, kmax = tail.kmax;
    const uint32_t n = tail.listed;
    uint32_t ln = 0;
    bool listed = true;
    if (o.mode == kGivenCells) {
        // The parts' lists one after another; none where one does not fit.
        const uint64_t before = block_exclusive_sum<NT>((uint64_t)n | (uint64_t)(n > kPartCap) << 40, sh.red64);
        if (t < wk.C) {
            s_at[t] = (uint32_t)before;
            s_n[t] = n;
        }
        if (t == wk.C - 1) {
            sh.n_window = (uint32_t)before + n;
            sh.cross = (before >> 40) || n > kPartCap;
        }
        if (t == 0) {
            sh.s_above = s0.s_above;
            sh.a_lo = s0.a_lo;
            sh.n_above = s0.n_above;
        }
        const uint64_t* joined = wk.joined + (size_t)b * kSlots;
        for (int r = o.r_lo + t; r <= o.r_hi; r += NT) sh.hist[o.top - r] = joined[o.top - r];
        if (t == 0 && o.rb <= o.top) sh.hist[o.top - o.rb] = joined[o.top - o.rb];
        __syncthreads();
        ln = uniform(sh.n_window);
        listed = !uniform(sh.cross) && ln <= Shared::kCap;
        if (listed) {
            for (int i = w; i < wk.C; i += Shared::kWaves) {
                const uint2* from = wk.list + ((size_t)b * wk.C + i) * kPartCap;
                for (uint32_t k = lane; k < s_n[i]; k += 4 * kWave) {
                    uint2 e[4];  // (places past the part's last are read, and left)
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[j] = from[min(k + j * kWave, (uint32_t)kPartCap - 1)];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (k + j * kWave < s_n[i]) sh.list[s_at[i] + k + j * kWave] = e[j];
                }
            }
        } else {
            for (uint32_t i = t; i < Shared::kCap; i += NT) sh.list[i].x = kEmpty;
        }
    }
    if (t == 0) sh.few_n = 0;
    __syncthreads();
    double one_weight;
    const Fixed fx(ldexp(1.0, p.bits));
    const float low = resolve_row<DT, NT>(sh, p, row, d, in, o, fx, listed, ln, kmin, kmax, count, one_weight);
    const double S = draw_row<DT, VEC, NT>(sh, p, b, row, d, segs, in, o, low, count, one_weight);
    if (t == 0) {
        st.S = S;
        st.low = low;
    }
}

template <int DT, bool VEC>
__global__ __launch_bounds__(kPartThreads) void given_probs_kernel(GivenParams p, GivenWork wk)
{
    constexpr int GN = Group<DT>::N;
    __shared__ double root[kOctave];
    const int t = threadIdx.x, lane = t & (kWave - 1);
    const int64_t b = blockIdx.x / (uint32_t)wk.C;
    const int part = (int)(blockIdx.x % (uint32_t)wk.C);
    const RowState& st = wk.state[b];
    const int mode = uniform(st.o.mode);
    if (mode == kGivenAlone) return;  // written already
    float* out = p.out_probs + b * p.V;
    const bool vec = p.V % 4 == 0 && (uintptr_t)p.out_probs % 16 == 0;
    const bool dist = mode == kGivenLevel || mode == kGivenCells;
    const int token = dist ? -1 : uniform(st.token);
    const uint32_t groups = (uint32_t)((p.V + GN - 1) / GN);
    u32x4 raw[kPartSteps];
    const uint32_t g0 = load_part<DT, VEC>(row_of<DT>(p, b), part, groups, p.V, raw);
    if (t < kOctave) root[t] = kRoot[t];
    __syncthreads();
    const RowPlan o = st.o;
    const float low = dist ? st.low : NAN;  // (no logit is at or above it, +inf neither)
    const double inv = dist ? 1.0 / st.S : 0.0;
#pragma unroll
    for (int i = 0; i < kPartSteps; ++i) {
        const uint32_t g = g0 + i * kWave + lane;
        float x[GN], q[GN];
        tokens_of<DT>(raw[i], g, true, p.V, x);
        bool any = false;
#pragma unroll
        for (int j = 0; j < GN; ++j) {
            q[j] = (int)(g * GN + j) == token ? 1.0f : 0.0f;
            any |= x[j] >= low;
        }
        if (lanes(any)) {
#pragma unroll
            for (int j = 0; j < GN; ++j)
                if (x[j] >= low) q[j] = (float)(weight_of(o, root, x[j]) * inv);
        }
        const int64_t i0 = (int64_t)g * GN;
        if (vec && i0 + GN <= p.V) {
#pragma unroll
            for (int j = 0; j < GN; j += 4) *(f32x4*)(out + i0 + j) = f32x4{q[j], q[j + 1], q[j + 2], q[j + 3]};
        } else {
#pragma unroll
            for (int j = 0; j < GN; ++j)
                if (i0 + j < p.V) out[i0 + j] = q[j];
        }
    }
}

// ---------------------------------------------------------------------------
// Speculative acceptance from given uniforms: accept d iff u0 q(d) < p(d),
// else the inverse CDF with u1 over r_i = max(p_i - q_i, 0) in index order.
//
// A short row is one workgroup's.  Longer ones take two launches, as in
// spec.h: a workgroup per 8192-token chunk of every row sums r over the chunks
// of rejected rows in doubles (in a fixed order); then a workgroup per row
// finds the chunk and reads that chunk again.  Bound by latency: a token, its
// two probabilities, the row, one after the other (5 rows of 32000: 8 us in one
// kernel; 256 rows of 128256, a twentieth rejected: 15 us from cache).
// ---------------------------------------------------------------------------
constexpr int kPickThreads = 256;
constexpr int kPickWaves = kPickThreads / kWave;
constexpr int kPickSteps = 8;                              // of 64 groups of 4 tokens, per wave
constexpr int kPickRun = kPickSteps * kWave * 4;           // 2048 tokens
constexpr int kPickChunk = kPickWaves * kPickRun;          // 8192 tokens
constexpr int kPickWide = 1024;                            // threads of pick_row_kernel
constexpr int kPickShort = kPickWide / kWave * kPickRun;   // 32768 tokens: its rows, at most

struct PickParams {
    const float* target;         // [B, V]: p
    const float* draft;          // [B, V]: q
    const int32_t* draft_token;  // [B]
    const void* uniforms;        // [B, 2]
    int u_f64;
    int64_t B, V;
    int32_t* out_token;     // [B]
    int32_t* out_accepted;  // [B] or null
    double* part;           // [B, C] chunk sums (workspace)
    int C;
    int vec;                // rows 16-byte aligned
};

// 1 accepted, 0 rejected, -1 a draft token out of range or u0 not a number.
__device__ __forceinline__ int pick_verdict(const PickParams& p, int64_t b)
{
    const int32_t d = p.draft_token[b];
    const double u = p.u_f64 ? ((const double*)p.uniforms)[2 * b] : (double)((const float*)p.uniforms)[2 * b];
    if (d < 0 || d >= p.V || !(u == u)) return -1;
    return u * (double)p.draft[b * p.V + d] < (double)p.target[b * p.V + d] ? 1 : 0;
}

// max(p - q, 0) of this lane's group in step k of the run of tokens that starts
// at i (0 for NaN and past the row's end).
__device__ __forceinline__ void pick_load(const PickParams& p, int64_t b, int64_t i, int k, double (&r)[4])
{
    const int64_t i0 = i + (k * kWave + (int)(threadIdx.x & (kWave - 1))) * 4;
    const float *P = p.target + b * p.V, *Q = p.draft + b * p.V;
    float a[4], e[4];
    if (p.vec && i0 + 4 <= p.V) {
        const f32x4 va = *(const f32x4*)(P + i0), ve = *(const f32x4*)(Q + i0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = va[j];
            e[j] = ve[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = i0 + j < p.V ? P[i0 + j] : 0.0f;
            e[j] = i0 + j < p.V ? Q[i0 + j] : 0.0f;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const double v = (double)a[j] - (double)e[j];
        r[j] = v > 0.0 ? v : 0.0;
    }
}

__global__ __launch_bounds__(kPickThreads) void pick_chunk_kernel(PickParams p)
{
    __shared__ double red[kPickWaves];
    const int64_t b = blockIdx.x % (uint32_t)p.B;
    const int c = (int)(blockIdx.x / (uint32_t)p.B);
    if (pick_verdict(p, b) != 0) return;  // uniform; nothing reads the slot
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < kPickSteps; ++k) {
        double r[4];
        pick_load(p, b, (int64_t)c * kPickChunk + threadIdx.x / kWave * kPickRun, k, r);
        sum += (r[0] + r[1]) + (r[2] + r[3]);
    }
    sum = block_reduce<kPickThreads>(sum, SumF64(), red);
    if (threadIdx.x == 0) p.part[b * p.C + c] = sum;
}

__global__ __launch_bounds__(kPickThreads) void pick_finish_kernel(PickParams p)
{
    __shared__ double wsum[kPickWaves];
    __shared__ int wlast[kPickWaves], found[kPickWaves];
    const int64_t b = blockIdx.x;
    const int t = threadIdx.x, lane = t & (kWave - 1), w = t / kWave;
    const int verdict = pick_verdict(p, b);
    if (verdict != 0) {
        if (t == 0) {
            p.out_token[b] = verdict > 0 ? p.draft_token[b] : -1;
            if (p.out_accepted) p.out_accepted[b] = verdict > 0 ? 1 : 0;
        }
        return;
    }
    // Every wave finds the chunk for itself, in the same way.
    const double* part = p.part + b * p.C;
    double S = 0.0;
    for (int i = 0; i < p.C; i += kWave) {
        double all;
        wave_inclusive_sum(i + lane < p.C ? part[i + lane] : 0.0, all);
        S += all;
    }
    const double u = p.u_f64 ? ((const double*)p.uniforms)[2 * b + 1] : (double)((const float*)p.uniforms)[2 * b + 1];
    int token = -1;
    if (S > 0.0 && S < (double)INFINITY && u == u) {
        const double at = (u < 0.0 ? 0.0 : (u > 1.0 ? 1.0 : u)) * S;
        int chunk = 0;
        double run = 0.0, before = 0.0;
        for (int i = 0; i < p.C; i += kWave) {
            const double v = i + lane < p.C ? part[i + lane] : 0.0;
            double all;
            const double inc = wave_inclusive_sum(v, all);
            const double prev = wave_shift_up1(inc);
            const uint64_t mass = __ballot(v > 0.0), over = __ballot(v > 0.0 && run + inc > at);
            if (over | mass) {  // the first that exceeds `at`, or so far the last with mass
                const int L = over ? (int)__builtin_ctzll(over) : 63 - (int)__builtin_clzll(mass);
                chunk = i + L;
                before = run + lane_value(prev, L);
            }
            if (over) break;
            run += all;
        }
        double r[kPickSteps][4], sum = 0.0;
#pragma unroll
        for (int k = 0; k < kPickSteps; ++k) pick_load(p, b, (int64_t)chunk * kPickChunk + w * kPickRun, k, r[k]);
#pragma unroll
        for (int k = 0; k < kPickSteps; ++k) sum += (r[k][0] + r[k][1]) + (r[k][2] + r[k][3]);
        sum = wave_reduce(sum, SumF64());
        if (lane == 0) wsum[w] = sum;
        __syncthreads();
        double a0 = before;
        for (int i = 0; i < w; ++i) a0 += wsum[i];
        int hit = -1, last = -1;
#pragma unroll
        for (int k = 0; k < kPickSteps; ++k) {
            const int i0 = (int)((uint32_t)chunk * kPickChunk + (uint32_t)((w * kPickSteps + k) * kWave + lane) * 4u);
            double all;
            const double own = (r[k][0] + r[k][1]) + (r[k][2] + r[k][3]);
            const double inc = wave_inclusive_sum(own, all);
            const double prev = wave_shift_up1(inc);
            double a = a0 + (lane ? prev : 0.0);
            int tok = -1, end = -1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a += r[k][j];
                if (r[k][j] > 0.0) {
                    end = i0 + j;
                    if (tok < 0 && a > at) tok = i0 + j;
                }
            }
            const uint64_t hits = __ballot(tok >= 0), ends = __ballot(end >= 0);
            if (hit < 0 && hits) hit = __builtin_amdgcn_readlane(tok, (int)__builtin_ctzll(hits));
            if (ends) last = __builtin_amdgcn_readlane(end, 63 - (int)__builtin_clzll(ends));
            a0 += all;
        }
        if (lane == 0) {
            found[w] = hit;
            wlast[w] = last;
        }
        __syncthreads();
        for (int i = kPickWaves - 1; i >= 0; --i)
            if (wlast[i] >= 0 && token < 0) token = wlast[i];
        for (int i = kPickWaves - 1; i >= 0; --i)
            if (found[i] >= 0) token = found[i];
    }
    if (t == 0) {
        p.out_token[b] = token;
        if (p.out_accepted) p.out_accepted[b] = 0;
    }
}

// A row of up to kPickShort tokens on one workgroup, a run a wave: the wave
// that holds the draw finds it among what it has in registers.
__global__ __launch_bounds__(kPickWide) void pick_row_kernel(PickParams p)
{
    constexpr int WAVES = kPickWide / kWave;
    __shared__ double wsum[WAVES];
    const int64_t b = blockIdx.x;
    const int t = threadIdx.x, lane = t & (kWave - 1), w = t / kWave;
    const double u = p.u_f64 ? ((const double*)p.uniforms)[2 * b + 1] : (double)((const float*)p.uniforms)[2 * b + 1];
    const int verdict = pick_verdict(p, b);
    if (verdict != 0) {
        if (t == 0) {
            p.out_token[b] = verdict > 0 ? p.draft_token[b] : -1;
            if (p.out_accepted) p.out_accepted[b] = verdict > 0 ? 1 : 0;
        }
        return;
    }
    double r[kPickSteps][4], sum = 0.0;
#pragma unroll
    for (int k = 0; k < kPickSteps; ++k) pick_load(p, b, (int64_t)w * kPickRun, k, r[k]);
#pragma unroll
    for (int k = 0; k < kPickSteps; ++k) sum += (r[k][0] + r[k][1]) + (r[k][2] + r[k][3]);
    sum = wave_reduce(sum, SumF64());
    if (lane == 0) wsum[w] = sum;
    __syncthreads();
    // Every wave looks at all sums in the same way.
    double S;
    const double v = lane < WAVES ? wsum[lane] : 0.0;
    const double run = wave_inclusive_sum(v, S);
    const double at = (u < 0.0 ? 0.0 : (u > 1.0 ? 1.0 : u)) * S;
    const uint64_t mass = __ballot(v > 0.0), over = __ballot(v > 0.0 && run > at);
    if (!(S > 0.0 && S < (double)INFINITY && u == u)) {
        if (t == 0) {
            p.out_token[b] = -1;
            if (p.out_accepted) p.out_accepted[b] = 0;
        }
        return;
    }
    // The first run that exceeds `at`, or the last with mass.
    const int found = over ? (int)__builtin_ctzll(over) : 63 - (int)__builtin_clzll(mass);
    if (w != found) return;
    double before = found ? lane_value(run, found - 1) : 0.0;
    int token = -1;
    bool open = true;
#pragma unroll
    for (int k = 0; k < kPickSteps; ++k) {
        const int i0 = w * kPickRun + (k * kWave + lane) * 4;
        double all;
        const double inc = wave_inclusive_sum((r[k][0] + r[k][1]) + (r[k][2] + r[k][3]), all);
        const double prev = wave_shift_up1(inc);
        double a = before + (lane ? prev : 0.0);
        int tok = -1, end = -1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a += r[k][j];
            if (r[k][j] > 0.0) {
                end = i0 + j;
                if (tok < 0 && a > at) tok = i0 + j;
            }
        }
        const uint64_t hits = __ballot(tok >= 0), ends = __ballot(end >= 0);
        if (open && ends)
            token = hits ? __builtin_amdgcn_readlane(tok, (int)__builtin_ctzll(hits))
                         : __builtin_amdgcn_readlane(end, 63 - (int)__builtin_clzll(ends));
        if (hits) open = false;
        before += all;
    }
    if (lane == 0) {
        p.out_token[b] = token;
        if (p.out_accepted) p.out_accepted[b] = 0;
    }
}

}  // namespace nucleus
