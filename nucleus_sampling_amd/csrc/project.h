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
    float cap;           // softcap
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

__device__ __forceinline__ float activate(int act, float cap, float z)
{
    switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;  // NaN stays
    case kActGelu: return 0.5f * z * erfcf(z * -0.70710678f);
    case kActSilu: return z / (1.0f + expf(-z));
    case kActSoftcap: return cap * tanhf(z / cap);
    default: return z;
    }
}

template <int DT>
__device__ __forceinline__ float load_elem(const void* p, int64_t i, int f32)
{
    if (DT == kF32 || f32) return ((const float*)p)[i];
    return (float)((const typename Elem<DT>::T*)p)[i];
}

template <int DT>
__device__ __forceinline__ f32x4 load_elem4(const void* p, int64_t i, int f32)
{
    typedef typename Elem<DT>::T T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    if (DT == kF32 || f32) return *(const f32x4*)((const float*)p + i);
    return __builtin_convertvector(*(const T4*)((const T*)p + i), f32x4);
}

// Finish and store out[m, n .. n + 3] from their sums; elements past N (and
// rows past M) are left alone.  A residual that is `out` itself is fine: each
// element is read by the thread that writes it, before it does.
template <int DT>
__device__ __forceinline__ void project_store(const ProjectParams& p, int64_t m, int64_t n, f32x4 z)
{
    typedef typename Elem<DT>::T T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    if (m >= p.M || n >= p.N) return;
    if (p.vec) {
        if (p.bias) z += load_elem4<DT>(p.bias, n, p.bias_f32);
        if (p.act != kActNone) {
#pragma unroll
            for (int r = 0; r < 4; ++r) z[r] = activate(p.act, p.cap, z[r]);
        }
        if (p.res) z += load_elem4<DT>(p.res, m * p.rs + n, p.res_f32);
        const int64_t o = m * p.os + n;
        if (DT == kF32 || p.out_f32)
            *(f32x4*)((float*)p.out + o) = z;
        else
            *(T4*)((T*)p.out + o) = __builtin_convertvector(z, T4);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (n + r >= p.N) break;
            float v = z[r];
            if (p.bias) v += load_elem<DT>(p.bias, n + r, p.bias_f32);
            v = activate(p.act, p.cap, v);
            if (p.res) v += load_elem<DT>(p.res, m * p.rs + n + r, p.res_f32);
            const int64_t o = m * p.os + n + r;
            if (DT == kF32 || p.out_f32)
                ((float*)p.out)[o] = v;
            else
                ((T*)p.out)[o] = (T)v;
        }
    }
}

// ---------------------------------------------------------------------------
// Any layout: rows that start anywhere, any K.  A 256-thread workgroup takes
// 64 n x 64 m, 128 bytes of k at a time; every element of a tile is loaded by
// itself (zero past the row's end), packed into LDS chunks and multiplied from
// there, wave w taking 16 n of the 64.  The loads of the next tile are in
// flight while the current one is multiplied.
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
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int off = (g * 4 + (lane >> 4)) * 16;
            const u32x4 a = *(const u32x4*)(lds + (16 * w + (lane & 15)) * ROWB + off);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const u32x4 b = *(const u32x4*)(lds + (kAnyTile + 16 * u + (lane & 15)) * ROWB + off);
                acc[u] = mfma_group<DT>(a, b, acc[u]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
        project_store<DT>(p, m0 + 16 * u + (lane & 15), n0 + 16 * w + 4 * (lane >> 4), acc[u]);
}

}  // namespace nucleus
