// project.h -- out = act(hidden weight^T + bias) + residual: the product that
// makes logits (a vocabulary projection) and the block of a draft head.
//
// hidden [M, K] and weight [N, K] both run along k in memory, so a 16-byte
// load holds consecutive k of one row of either: 8 16-bit or 4 32-bit
// elements, called a chunk here.  A matrix instruction takes one chunk per
// lane from both sides: lane l holds row l % 16, chunk l / 16 of a group of
// four (16x16x32 on 16-bit elements; four 16x16x4 on fp32, whose k order
// within the group of four chunks is permuted the same way on both sides,
// which a sum over k does not see).  weight is the first operand, so lane l of a result tile
// holds column m = l % 16 and four consecutive n = 4 (l / 16) + r: results
// leave in 16-byte (fp32) or 8-byte (16-bit) stores along n.
//
// Sums are held in fp32; bias, activation and residual are applied in fp32
// and the result is rounded once, to the output type.
#pragma once

#include <type_traits>

#include "common.h"
#include "params.h"

namespace nucleus {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum Activation { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSoftcap = 4 };

struct ProjectParams {
    const char* h;       // hidden, rows hs bytes apart
    const char* w;       // weight, rows ws bytes apart
    char* out;           // rows os elements apart
    const void* bias;    // [N] or null
    const void* res;     // residual, rows rs elements apart, or null
    int64_t M, N, K;
    int64_t hs, ws;      // bytes
    int64_t os, rs;      // elements
    float cap, per_cap;  // softcap; 1 / cap, or 0 where that is no good number
    int act;
    int out_f32, bias_f32, res_f32;
    int vec;             // groups of four n are whole and aligned in out, bias and residual
};

// Element types: DT is kF32, kBF16 or kF16.
template <int DT> struct Elem;
template <> struct Elem<kF32> { typedef float T; };
template <> struct Elem<kBF16> { typedef __bf16 T; };
template <> struct Elem<kF16> { typedef _Float16 T; };

// acc += the 16x16 product over one group of four chunks.
template <int DT>
__device__ __forceinline__ f32x4 mfma_group(u32x4 w, u32x4 h, f32x4 acc)
{
    if constexpr (DT == kBF16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, h), acc,
                                                       0, 0, 0);
    } else if constexpr (DT == kF16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, h), acc, 0,
                                                      0, 0);
    } else {
        const f32x4 a = __builtin_bit_cast(f32x4, w), b = __builtin_bit_cast(f32x4, h);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], acc, 0, 0, 0);
        return acc;
    }
}

// fp32 products are summed in two levels, 32 of k by the matrix instructions
// from 0 and those sums in turn: a quarter-K chain of additions would leave
// about three times the rounding error.  16-bit products, whose instructions
// take 32 of k at once, go on from the running sum.
template <int DT>
__device__ __forceinline__ f32x4 start_of(f32x4 acc)
{
    return DT == kF32 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc;
}
template <int DT>
__device__ __forceinline__ f32x4 joined(f32x4 acc, f32x4 sum)
{
    return DT == kF32 ? acc + sum : sum;
}

// tanh to five units: (1 - e) / (1 + e) with e = e^(-2|x|), and up to 1/4,
// where that cancels, the series to x^9 (the next term is 9e-9 of x).
__device__ __forceinline__ float tanh_of(float x)
{
    const float e = __builtin_amdgcn_exp2f(fabsf(x) * -2.88539008f), x2 = x * x;
    const float far = (1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e);
    float near = fmaf(x2, 62.0f / 2835.0f, -17.0f / 315.0f);
    near = fmaf(x2, near, 2.0f / 15.0f);
    near = fmaf(x2, near, -1.0f / 3.0f);
    near = fmaf(x2 * x, near, x);
    return fabsf(x) < 0.25f ? near : copysignf(far, x);
}

__device__ __forceinline__ float activate(int act, float cap, float per_cap, float z)
{
    switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;  // NaN stays
    case kActGelu: return 0.5f * z * erfcf(z * -0.70710678f);
    case kActSilu: {
        // z / (1 + e^-z), with e^-|z| so that nothing overflows and the
        // reciprocal (off by one unit at most) is of 1 to 2.
        const float e = expf(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + e);
        return (z < 0.0f ? z * e : z) * r;
    }
    // (a product with the reciprocal moves the argument by one unit at most)
    case kActSoftcap: return cap * tanh_of(per_cap != 0.0f ? z * per_cap : z / cap);
    default: return z;
    }
}

// Four elements of bias or residual as they lie in memory, from element n of
// the row at `row`; values4 makes numbers of them, so that the load can be far
// ahead of its use.  VEC: groups of four are whole and aligned; else every
// element is loaded by itself, past the row's end the last again.
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 fetch4(const void* row, int64_t n, int64_t N, int f32)
{
    u32x4 r = {0, 0, 0, 0};
    if (DT == kF32 || f32) {
        const uint32_t* at = (const uint32_t*)row;
        if constexpr (VEC) return *(const u32x4*)(at + n);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = at[min(n + j, N - 1)];
    } else {
        const uint16_t* at = (const uint16_t*)row;
        if constexpr (VEC) {
            const uint2 v = *(const uint2*)(at + n);
            return u32x4{v.x, v.y, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = at[min(n + j, N - 1)];
    }
    return r;
}
template <int DT, bool VEC>
__device__ __forceinline__ f32x4 values4(u32x4 r, int f32)
{
    if (DT == kF32 || f32) return __builtin_bit_cast(f32x4, r);
    if constexpr (VEC) r = u32x4{r[0] & 0xFFFFu, r[0] >> 16, r[1] & 0xFFFFu, r[1] >> 16};
    if constexpr (DT == kBF16) return __builtin_bit_cast(f32x4, r << 16);
    f32x4 z;
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)r[j]);
    return z;
}

// The raw bias of n .. n + 3 and residual of row m there; any n and m (those
// past the end read the last, and are not stored).
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 fetch_bias(const ProjectParams& p, int64_t n)
{
    if (!p.bias) return u32x4{0, 0, 0, 0};
    return fetch4<DT, VEC>(p.bias, n < p.N ? n : 0, p.N, p.bias_f32);
}
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 fetch_residual(const ProjectParams& p, int64_t m, int64_t n)
{
    const int64_t at = min(m, p.M - 1) * p.rs;
    return fetch4<DT, VEC>((const char*)p.res + at * (DT == kF32 || p.res_f32 ? 4 : 2), n < p.N ? n : 0, p.N, p.res_f32);
}

// Finish and store out[m, n .. n + 3] from their sums; elements past N (and
// rows past M) are left alone.  A residual that is `out` itself is fine: each
// element is read by the thread that writes it, before it does.  ACT is the
// activation, or -1 to look at p.act for every element.
template <int DT, bool VEC, int ACT>
__device__ __forceinline__ void project_store(const ProjectParams& p, int64_t m, int64_t n, f32x4 z, u32x4 bias,
                                              u32x4 residual)
{
    typedef typename Elem<DT>::T T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    if (p.bias) z += values4<DT, VEC>(bias, p.bias_f32);
    const int act = ACT < 0 ? p.act : ACT;
    if (act != kActNone) {
#pragma unroll
        for (int r = 0; r < 4; ++r) z[r] = activate(act, p.cap, p.per_cap, z[r]);
    }
    if (p.res) z += values4<DT, VEC>(residual, p.res_f32);
    if (m >= p.M || n >= p.N) return;
    const int64_t o = m * p.os + n;
    const bool f32 = DT == kF32 || p.out_f32;
    if constexpr (VEC) {
        if (f32)
            *(f32x4*)((float*)p.out + o) = z;
        else
            *(T4*)((T*)p.out + o) = __builtin_convertvector(z, T4);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (n + r >= p.N) break;
            if (f32)
                ((float*)p.out)[o + r] = z[r];
            else
                ((T*)p.out)[o + r] = (T)z[r];
        }
    }
}

// The same with the bias and residual asked for here.
template <int DT>
__device__ __forceinline__ void finish_group(const ProjectParams& p, int64_t m, int64_t n, f32x4 z)
{
    u32x4 residual = {0, 0, 0, 0};
    if (p.vec) {
        if (p.res) residual = fetch_residual<DT, true>(p, m, n);
        project_store<DT, true, -1>(p, m, n, z, fetch_bias<DT, true>(p, n), residual);
    } else {
        if (p.res) residual = fetch_residual<DT, false>(p, m, n);
        project_store<DT, false, -1>(p, m, n, z, fetch_bias<DT, false>(p, n), residual);
    }
}

// ---------------------------------------------------------------------------
// Any layout: rows that start anywhere, any K.  A 256-thread workgroup takes
// 64 n x 64 m, 128 bytes of k at a time; every element of a tile is loaded by
// itself (zero past the row's end), packed into LDS chunks and multiplied from
// there, wave w taking 16 n of the 64.  The loads of the next tile are in
// flight while the current one is multiplied.  The element loads bound it:
// N = 4096, K = 4095 takes 82 us with one row and 117 with 48 (bf16), where
// the kernels below take 8.3 and 9.9 at K = 4096; a caller whose rows start off
// 16-byte boundaries does better to pad them.
// ---------------------------------------------------------------------------
constexpr int kAnyTile = 64;   // rows of either side
constexpr int kAnyThreads = 256;

template <int DT>
__global__ __launch_bounds__(kAnyThreads) void project_any_kernel(ProjectParams p)
{
    typedef typename Elem<DT>::T T;
    constexpr int E = 16 / (int)sizeof(T);      // elements of a chunk
    constexpr int KT = 8 * E;                   // elements of k per tile: 128 bytes
    constexpr int ROWB = 128 + 16;              // row pitch in LDS: the 16 spread rows over the banks
    __shared__ __align__(16) char lds[2 * kAnyTile * ROWB];
    const int t = threadIdx.x, lane = t & 63, w = t >> 6;
    const uint32_t nt = (uint32_t)((p.N + kAnyTile - 1) / kAnyTile);
    const int64_t n0 = (int64_t)(blockIdx.x % nt) * kAnyTile, m0 = (int64_t)(blockIdx.x / nt) * kAnyTile;
    // Thread t stages chunk t % 8 of rows t / 8 and t / 8 + 32 of both sides.
    const int cr = t >> 3, cc = t & 7;
    const T* src[4];
    bool in[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t n = n0 + cr + 32 * i, m = m0 + cr + 32 * i;
        in[i] = n < p.N;
        in[2 + i] = m < p.M;
        src[i] = (const T*)(p.w + (in[i] ? n : 0) * p.ws);
        src[2 + i] = (const T*)(p.h + (in[2 + i] ? m : 0) * p.hs);
    }
    T next[4][E];
    auto fetch = [&](int64_t k0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int64_t k = k0 + cc * E + j;
                next[i][j] = (in[i] && k < p.K) ? src[i][k] : (T)0.0f;
            }
    };
    f32x4 acc[4] = {};
    fetch(0);
    for (int64_t k0 = 0; k0 < p.K; k0 += KT) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            typedef T TE __attribute__((ext_vector_type(E)));
            TE v;
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = next[i][j];
            *(TE*)(lds + ((i >> 1) * kAnyTile + cr + 32 * (i & 1)) * ROWB + cc * 16) = v;
        }
        __syncthreads();
        if (k0 + KT < p.K) fetch(k0 + KT);
        f32x4 sum[4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int off = (g * 4 + (lane >> 4)) * 16;
            const u32x4 a = *(const u32x4*)(lds + (16 * w + (lane & 15)) * ROWB + off);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const u32x4 b = *(const u32x4*)(lds + (kAnyTile + 16 * u + (lane & 15)) * ROWB + off);
                sum[u] = mfma_group<DT>(a, b, g == 0 ? start_of<DT>(acc[u]) : sum[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[u] = joined<DT>(acc[u], sum[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t m = m0 + 16 * u + (lane & 15), n = n0 + 16 * w + 4 * (lane >> 4);
        finish_group<DT>(p, m, n, acc[u]);
    }
}

// ---------------------------------------------------------------------------
// Many rows of hidden: a workgroup of WN x WM waves makes a BN (n) x BM (m)
// tile, 128 bytes of k at a step.  Both sides' pieces go from memory straight
// into LDS (16 bytes a lane, no registers), STAGES deep: while step s is
// multiplied the loads of steps s + 1 .. s + STAGES - 1 are in flight, and a
// step costs one barrier.
//
// LDS holds 128-byte rows (eight chunks); chunk x of row r lies at place
// x ^ ((r / 2) % 8), so that the sixteen rows that a quarter wave reads at
// one x fall on sixteen different 16-byte banks groups.  The loads write LDS
// in lane order, so the permutation is made on the address a lane reads from.
//
// Workgroups go to the eight XCDs in turn; each XCD is given a run of
// neighbouring tiles, so that its L2 holds the rows they share.
//
// With few rows the read of weight bounds it (bf16, N = 128256, K = 4096: 1
// row 169 us, 6.2 TB/s; 64 rows 186; 128 rows 210), with many the LDS: eight
// waves of a 256 x 256 tile read 192 KB of it a step and the loads write 64,
// while the matrix cores need 2048 cycles.  256 rows of the above 270 us (298
// with float32 logits, 131 MB of stores); 4096^3 106 us, 1300 TF (a library
// product 101), of it 12 before and after the steps, and 126 with bias, silu
// and a residual; 8192^3 1330 TF.  Two wave groups half a step apart, 64-byte
// steps three to five deep and 128 x 128 pieces for four waves, their reads
// half a step ahead, were each 5 to 20 % slower.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) char lds_char;

// 64 lanes x 16 bytes from rsrc + soff + voff (0 where voff is out of range)
// to LDS bytes `to` .. `to` + 1023, in lane order.  Not tracked by the
// compiler: wait_loads() below waits for it.
__device__ __forceinline__ void load_to_lds(uint32_t to, u32x4 rsrc, uint32_t voff, uint32_t soff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(to), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory");
}

// All but the wave's last N loads have arrived, its LDS reads have returned,
// and every wave of the workgroup has come here.
template <int N>
__device__ __forceinline__ void wait_loads_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// Buffer descriptor of `bytes` bytes at p (wave-uniform).
__device__ __forceinline__ u32x4 buffer_of(const void* p, uint32_t bytes)
{
    const uint64_t a = (uint64_t)p;
    return u32x4{uniform((uint32_t)a), uniform((uint32_t)(a >> 32)) & 0xFFFFu, uniform(bytes), 0x00020000u};
}

constexpr int kXcds = 8;

// The tile of workgroup `id`: an XCD's workgroups (id mod 8 equal) take a run
// of consecutive tiles; tiles run down m within bands of `band` tiles of m,
// then along n.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t nt, uint32_t mt, uint32_t& tn, uint32_t& tm)
{
    const uint32_t T = nt * mt, x = id % kXcds, q = T / kXcds, r = T % kXcds;
    const uint32_t tile = x * q + min(x, r) + id / kXcds;
    constexpr uint32_t band = 4;
    const uint32_t g = tile / (band * nt), rest = tile - g * band * nt;
    const uint32_t rows = min(band, mt - g * band);
    tn = rest / rows;
    tm = g * band + rest % rows;
}

// Sums in LDS: `rows` rows `pitch` bytes apart; row i is the output's row
// m0 + (i / run) apart + i % run.
struct Staged {
    const char* lds;
    int pitch, rows, run, apart;
    int64_t m0;
};

// Finishes them, BN columns from n0, with NW waves.  A thread's columns are the
// same in every row it takes, and so is its bias; rows go four at a time with
// the residuals of the next four on their way.
template <int DT, bool VEC, int ACT, int BN, int NW, int UP>
__device__ __forceinline__ void finish_rows(const ProjectParams& p, const Staged& st, int64_t n0)
{
    constexpr int COLS = BN / 4, STEP = NW * 64 / COLS;
    static_assert(NW * 64 % COLS == 0, "a thread keeps its columns");
    const int col = (int)(threadIdx.x % COLS);
    const int64_t n = n0 + 4 * col;
    const auto row_of = [&](int i) { return i < st.rows ? st.m0 + (i / st.run) * st.apart + i % st.run : p.M; };
    const u32x4 bias = fetch_bias<DT, VEC>(p, n);
    u32x4 next[UP] = {};
    const auto fetch = [&](int i) {
        if (p.res) {  // uniform
#pragma unroll
            for (int k = 0; k < UP; ++k) next[k] = fetch_residual<DT, VEC>(p, row_of(i + k * STEP), n);
        }
    };
    int i = threadIdx.x / COLS;
    fetch(i);
#pragma unroll 1
    for (; i < st.rows; i += UP * STEP) {
        u32x4 residual[UP];
        f32x4 z[UP];
#pragma unroll
        for (int k = 0; k < UP; ++k) {
            residual[k] = next[k];
            z[k] = *(const f32x4*)(st.lds + min(i + k * STEP, st.rows - 1) * st.pitch + col * 16);
        }
        fetch(i + UP * STEP);
#pragma unroll
        for (int k = 0; k < UP; ++k) project_store<DT, VEC, ACT>(p, row_of(i + k * STEP), n, z[k], bias, residual[k]);
    }
}

template <int DT, int BN, int BM, int WN, int WM, int STAGES>
__global__ __launch_bounds__(WN* WM * 64, 1) void project_tile_kernel(ProjectParams p)
{
    constexpr int NW = WN * WM;
    constexpr int STAGE = (BN + BM) * 128;
    constexpr int LN = BN / 8 / NW, LM = BM / 8 / NW;  // loads of a wave per step and side
    constexpr int TN = BN / WN / 16, TM = BM / WM / 16;
    static_assert(LN * 8 * NW == BN && LM * 8 * NW == BM && NW % 2 == 0, "loads divide evenly");
    __shared__ __align__(1024) char lds[STAGES * STAGE];
    const int lane = threadIdx.x & 63, v = uniform((int)(threadIdx.x >> 6));
    const uint32_t nt = (uint32_t)((p.N + BN - 1) / BN), mt = (uint32_t)((p.M + BM - 1) / BM);
    uint32_t tn, tm;
    tile_of(blockIdx.x, nt, mt, tn, tm);
    const int64_t n0 = (int64_t)tn * BN, m0 = (int64_t)tm * BM;
    const int chunks = (int)(p.K * (DT == kF32 ? 4 : 2) / 16);
    const int steps = (chunks + 7) / 8;
    const int nrows = (int)min((int64_t)BN, p.N - n0), mrows = (int)min((int64_t)BM, p.M - m0);
    const u32x4 rw = buffer_of(p.w + n0 * p.ws, (uint32_t)((nrows - 1) * p.ws) + (uint32_t)chunks * 16);
    const u32x4 rh = buffer_of(p.h + m0 * p.hs, (uint32_t)((mrows - 1) * p.hs) + (uint32_t)chunks * 16);

    // Load i of this wave: rows (i NW + v) 8 + lane / 8 of the side, at place
    // lane % 8; rows past the end repeat the last (their results are not
    // stored).  The row's parity pair (r / 2) % 8 does not depend on i.
    const int place = lane & 7, x = place ^ (((v & 1) * 4 + (lane >> 4)) & 7);
    uint32_t ow[LN], oh[LM];
#pragma unroll
    for (int i = 0; i < LN; ++i)
        ow[i] = (uint32_t)min((i * NW + v) * 8 + (lane >> 3), nrows - 1) * (uint32_t)p.ws + (uint32_t)x * 16;
#pragma unroll
    for (int i = 0; i < LM; ++i)
        oh[i] = (uint32_t)min((i * NW + v) * 8 + (lane >> 3), mrows - 1) * (uint32_t)p.hs + (uint32_t)x * 16;
    const uint32_t base = (uint32_t)(uintptr_t)(lds_char*)lds;
    auto issue = [&](int step) {
        const uint32_t to = base + (uint32_t)(step % STAGES) * STAGE + (uint32_t)v * 1024;
        const uint32_t soff = (uint32_t)step * 128;
        const bool in = step * 8 + x < chunks;  // past K: zeros on both sides
#pragma unroll
        for (int i = 0; i < LN; ++i) load_to_lds(to + i * NW * 1024, rw, in ? ow[i] : 0x80000000u, soff);
#pragma unroll
        for (int i = 0; i < LM; ++i) load_to_lds(to + BN * 128 + i * NW * 1024, rh, in ? oh[i] : 0x80000000u, soff);
    };
    // Fragments: row l % 16 of a 16-row tile, chunk 4 g + l / 16.
    const int wn = v % WN, wm = v / WN;
    const int r16 = lane & 15, sw = r16 >> 1;
    const int fw = (wn * TN * 16 + r16) * 128 + (((lane >> 4) ^ sw) * 16);
    const int fh = BN * 128 + (wm * TM * 16 + r16) * 128 + (((lane >> 4) ^ sw) * 16);

    f32x4 acc[TN][TM] = {};
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < steps) issue(s);
    for (int s = 0; s < steps; ++s) {
        if (STAGES > 2 && s + STAGES - 2 < steps)
            wait_loads_and_meet<(STAGES - 2) * (LN + LM)>();
        else
            wait_loads_and_meet<0>();
        if (s + STAGES - 1 < steps) issue(s + STAGES - 1);
        const char* st = lds + (s % STAGES) * STAGE;
        f32x4 sum[TN][TM];
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) sum[i][j] = start_of<DT>(acc[i][j]);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            u32x4 a[TN], b[TM];
#pragma unroll
            for (int i = 0; i < TN; ++i) a[i] = *(const u32x4*)(st + ((fw + i * 2048) ^ (g * 64)));
#pragma unroll
            for (int j = 0; j < TM; ++j) b[j] = *(const u32x4*)(st + ((fh + j * 2048) ^ (g * 64)));
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j) sum[i][j] = mfma_group<DT>(a[i], b[j], sum[i][j]);
        }
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = joined<DT>(acc[i][j], sum[i][j]);
    }
    // Results pass through LDS, JG of the TM tile rows of every wave at a
    // time, so that whole rows of n are finished and stored together (and the
    // epilogue's code is there once).
    constexpr int PITCH = BN * 4 + 16;  // the 16 spread the 16 rows of a tile over the banks
    constexpr int FIT = STAGES * STAGE / (WM * 16 * PITCH);
    constexpr int JG = FIT >= TM ? TM : (FIT >= 4 && TM % 4 == 0 ? 4 : (FIT >= 2 && TM % 2 == 0 ? 2 : 1));
    static_assert(FIT >= 1, "a tile row of every wave fits");
    constexpr int UP = TN * TM > 16 ? 2 : 4;  // (registers hold the other turns' sums)
#pragma unroll 1
    for (int j0 = 0; j0 < TM; j0 += JG) {
        __syncthreads();
#pragma unroll
        for (int now = 0; now < TM; now += JG)
            if (now == j0) {  // uniform
#pragma unroll
                for (int j = 0; j < JG; ++j)
#pragma unroll
                    for (int i = 0; i < TN; ++i)
                        *(f32x4*)(lds + ((wm * JG + j) * 16 + r16) * PITCH + ((wn * TN + i) * 16 + 4 * (lane >> 4)) * 4) =
                            acc[i][now + j];
            }
        __syncthreads();
        const Staged st = {lds, PITCH, WM * JG * 16, JG * 16, TM * 16, m0 + j0 * 16};
        if (!p.vec) {
            finish_rows<DT, false, -1, BN, NW, UP>(p, st, n0);
        } else {
            switch (p.act) {
            case kActRelu: finish_rows<DT, true, kActRelu, BN, NW, UP>(p, st, n0); break;
            case kActGelu: finish_rows<DT, true, kActGelu, BN, NW, UP>(p, st, n0); break;
            case kActSilu: finish_rows<DT, true, kActSilu, BN, NW, UP>(p, st, n0); break;
            case kActSoftcap: finish_rows<DT, true, kActSoftcap, BN, NW, UP>(p, st, n0); break;
            default: finish_rows<DT, true, kActNone, BN, NW, UP>(p, st, n0);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Too few tiles to fill the device: eight waves split k among them.  A
// workgroup makes a 16 (n) x BM (m) tile; wave v takes the 128-byte pieces
// v, v + 8, ... of k through an LDS ring of its own (STAGES pieces, no
// barriers), and the partial tiles meet in LDS at the end.  Bound by how fast
// a workgroup's few rows of weight arrive: 48 x 4096 x 4096 in bf16 9.9 us, 7
// of them the 34 MB at the rate of a large copy (a library product 20.8).
// ---------------------------------------------------------------------------
constexpr int kSplitWaves = 8;

// The wave's own loads but the last N have arrived, and its LDS reads have
// returned.
template <int N>
__device__ __forceinline__ void wait_own_loads()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
}

template <int DT, int BM, int STAGES>
__global__ __launch_bounds__(kSplitWaves * 64, 1) void project_split_kernel(ProjectParams p)
{
    constexpr int STAGE = (16 + BM) * 128;
    constexpr int LM = BM / 8, L = 2 + LM, TM = BM / 16;
    __shared__ __align__(1024) char lds[kSplitWaves * STAGES * STAGE];
    static_assert(kSplitWaves * TM * 1024 <= (int)sizeof(lds), "partial tiles fit");
    const int lane = threadIdx.x & 63, v = uniform((int)(threadIdx.x >> 6));
    const uint32_t nt = (uint32_t)((p.N + 15) / 16);
    const int64_t n0 = (int64_t)(blockIdx.x % nt) * 16, m0 = (int64_t)(blockIdx.x / nt) * BM;
    const int chunks = (int)(p.K * (DT == kF32 ? 4 : 2) / 16);
    const int pieces = (chunks + 7) / 8;
    const int mine = pieces > v ? (pieces - v + kSplitWaves - 1) / kSplitWaves : 0;
    const int nrows = (int)min((int64_t)16, p.N - n0), mrows = (int)min((int64_t)BM, p.M - m0);
    const u32x4 rw = buffer_of(p.w + n0 * p.ws, (uint32_t)((nrows - 1) * p.ws) + (uint32_t)chunks * 16);
    const u32x4 rh = buffer_of(p.h + m0 * p.hs, (uint32_t)((mrows - 1) * p.hs) + (uint32_t)chunks * 16);
    // As in the tile kernel, with eight rows per load: r / 2 mod 8 is
    // (4 i + lane / 16) mod 8 for load i.
    uint32_t ow[2], oh[LM];
    int x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = (lane & 7) ^ ((4 * i + (lane >> 4)) & 7);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        ow[i] = (uint32_t)min(i * 8 + (lane >> 3), nrows - 1) * (uint32_t)p.ws + (uint32_t)x[i] * 16;
#pragma unroll
    for (int i = 0; i < LM; ++i)
        oh[i] = (uint32_t)min(i * 8 + (lane >> 3), mrows - 1) * (uint32_t)p.hs + (uint32_t)x[i & 1] * 16;
    const uint32_t ring = (uint32_t)(uintptr_t)(lds_char*)lds + (uint32_t)(v * STAGES) * STAGE;
    auto issue = [&](int s) {
        const uint32_t to = ring + (uint32_t)(s % STAGES) * STAGE;
        const int piece = v + s * kSplitWaves;
        const uint32_t soff = (uint32_t)piece * 128;
        const bool in[2] = {piece * 8 + x[0] < chunks, piece * 8 + x[1] < chunks};
#pragma unroll
        for (int i = 0; i < 2; ++i) load_to_lds(to + i * 1024, rw, in[i] ? ow[i] : 0x80000000u, soff);
#pragma unroll
        for (int i = 0; i < LM; ++i) load_to_lds(to + 2048 + i * 1024, rh, in[i & 1] ? oh[i] : 0x80000000u, soff);
    };
    const int r16 = lane & 15;
    const int f = r16 * 128 + (((lane >> 4) ^ (r16 >> 1)) * 16);
    // What this thread finishes; its bias and residual arrive under the loop.
    static_assert(TM * 64 <= kSplitWaves * 64, "one group a thread");
    const int64_t m = m0 + 16 * (threadIdx.x >> 6) + r16, n = n0 + 4 * (lane >> 4);
    const bool finishes = (int)threadIdx.x < TM * 64;
    u32x4 bias = {0, 0, 0, 0}, residual = {0, 0, 0, 0};
    if (finishes) {
        bias = p.vec ? fetch_bias<DT, true>(p, n) : fetch_bias<DT, false>(p, n);
        if (p.res) residual = p.vec ? fetch_residual<DT, true>(p, m, n) : fetch_residual<DT, false>(p, m, n);
    }
    f32x4 acc[TM] = {};
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < mine) issue(s);
    for (int s = 0; s < mine; ++s) {
        if (s + STAGES - 1 < mine) {
            wait_own_loads<63>();  // the reads of the stage about to be overwritten
            issue(s + STAGES - 1);
            wait_own_loads<(STAGES - 1) * L>();
        } else {
            wait_own_loads<0>();
        }
        const char* st = lds + (v * STAGES + s % STAGES) * STAGE;
        f32x4 sum[TM];
#pragma unroll
        for (int j = 0; j < TM; ++j) sum[j] = start_of<DT>(acc[j]);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const u32x4 a = *(const u32x4*)(st + (f ^ (g * 64)));
#pragma unroll
            for (int j = 0; j < TM; ++j)
                sum[j] = mfma_group<DT>(a, *(const u32x4*)(st + 2048 + j * 2048 + (f ^ (g * 64))), sum[j]);
        }
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[j] = joined<DT>(acc[j], sum[j]);
    }
    __syncthreads();  // every wave has read its last stage
    f32x4* part = (f32x4*)lds;
#pragma unroll
    for (int j = 0; j < TM; ++j) part[(v * TM + j) * 64 + lane] = acc[j];
    __syncthreads();
    if (finishes) {
        const int e = threadIdx.x;
        f32x4 z = part[e];
#pragma unroll
        for (int w = 1; w < kSplitWaves; ++w) z += part[w * TM * 64 + e];
        if (p.vec)
            project_store<DT, true, -1>(p, m, n, z, bias, residual);
        else
            project_store<DT, false, -1>(p, m, n, z, bias, residual);
    }
}

}  // namespace nucleus
