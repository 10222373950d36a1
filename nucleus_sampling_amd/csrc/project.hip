// project.hip -- nucleus_project (declared in include/nucleus.h): argument
// validation, the choice of kernel and its launch on the caller's stream.
#include <hip/hip_runtime.h>

#include <math.h>

#include "nucleus.h"
#include "host.h"
#include "project.h"

using namespace nucleus;

namespace {

size_t elem_bytes(int32_t dtype) { return dtype == NUCLEUS_F32 ? 4 : 2; }

bool known_dtype(int32_t dtype) { return dtype == NUCLEUS_F32 || dtype == NUCLEUS_BF16 || dtype == NUCLEUS_F16; }

// The bytes a [rows, cols] matrix spans.
struct Span {
    uintptr_t lo, hi;
    Span(const void* p, int64_t rows, int64_t cols, int64_t stride, size_t esz)
        : lo((uintptr_t)p), hi(lo + ((size_t)(rows - 1) * (size_t)stride + (size_t)cols) * esz)
    {
    }
    bool meets(const Span& o) const { return lo < o.hi && o.lo < hi; }
};

// A kernel for rows of whole 16-byte chunks on 16-byte boundaries.
struct Shape {
    int kind;         // 0 tile kernel, 1 split kernel
    int bn, bm;       // tile
    float first;      // us for up to one workgroup per CU, K = 4096 16-bit elements
    float next;       // us for each further workgroup per CU
};

// Measured on MI355X with 16-bit elements and K = 4096 (every shape scales
// with K alike), M = 16 .. 2048, N = 1024 .. 32000.  A large tile moves the
// fewest bytes through LDS per product (256 x 256: 112 us a tile and CU, the
// same area in 128 x 128 tiles 148, in 64 x 64 tiles 272) but needs many tiles
// to fill 256 CUs: M = 512, N = 4096 takes 34 us in 64 x 64 tiles, 54 in
// 128 x 128 and 95 in 256 x 256; M = 2048, N = 16384 takes 530, 316 and 235.
// With fewer tiles than that the split kernel fills the device: M = 48,
// N = 4096 takes 11.3 us with it and 20 in 64 x 64 tiles, while M = 64,
// N = 32000 takes 92 and 56.
constexpr Shape kShapes[] = {
    {1, 16, 16, 8.5f, 7.5f},   {1, 16, 32, 10.4f, 9.0f},  {1, 16, 48, 11.3f, 10.5f}, {1, 16, 64, 13.5f, 12.0f},
    {0, 64, 32, 16.8f, 13.0f}, {0, 64, 64, 21.0f, 17.0f}, {0, 128, 64, 31.0f, 28.0f}, {0, 128, 128, 50.0f, 37.0f},
    {0, 256, 256, 95.0f, 112.0f},
};
constexpr int kCus = 256;

int64_t tiles_of(const ProjectParams& p, int bn, int bm) { return ((p.N + bn - 1) / bn) * ((p.M + bm - 1) / bm); }

// The shape with the least estimated time.  fp32 products take eight times
// the matrix-core time, so the largest tile's saving in LDS traffic is not
// seen there: it is left out.
int choose(const ProjectParams& p, bool f32)
{
    int best = 0;
    float least = INFINITY;
    for (int i = 0; i < (int)(sizeof(kShapes) / sizeof(kShapes[0])); ++i) {
        const Shape& s = kShapes[i];
        if (f32 && s.bm == 256) continue;
        const int64_t turns = (tiles_of(p, s.bn, s.bm) + kCus - 1) / kCus;
        const float us = s.first + (float)(turns - 1) * s.next;
        if (us < least) {
            least = us;
            best = i;
        }
    }
    return best;
}

int launched() { return hipGetLastError() == hipSuccess ? NUCLEUS_OK : NUCLEUS_ELAUNCH; }

template <int DT, int BM, int STAGES>
int launch_split(const ProjectParams& p, hipStream_t s)
{
    const int64_t blocks = tiles_of(p, 16, BM);
    if (blocks >= int64_t(1) << 31) return NUCLEUS_EINVAL;
    hipLaunchKernelGGL((project_split_kernel<DT, BM, STAGES>), dim3((unsigned)blocks), dim3(kSplitWaves * 64), 0, s, p);
    return launched();
}

template <int DT, int BN, int BM, int WN, int WM, int STAGES>
int launch_tile(const ProjectParams& p, hipStream_t s)
{
    const int64_t blocks = tiles_of(p, BN, BM);
    if (blocks >= int64_t(1) << 31) return NUCLEUS_EINVAL;
    hipLaunchKernelGGL((project_tile_kernel<DT, BN, BM, WN, WM, STAGES>), dim3((unsigned)blocks), dim3(WN * WM * 64), 0, s,
                       p);
    return launched();
}

template <int DT>
int launch(const ProjectParams& p, hipStream_t s)
{
    const int64_t kbytes = p.K * (DT == kF32 ? 4 : 2);
    // Offsets inside a tile are 32-bit, and 2^31 stands for "past the end".
    const bool fits = 255 * p.ws + kbytes < (int64_t(1) << 31) && 255 * p.hs + kbytes < (int64_t(1) << 31);
    const bool chunked = (uintptr_t)p.h % 16 == 0 && (uintptr_t)p.w % 16 == 0 && p.hs % 16 == 0 && p.ws % 16 == 0 &&
                         kbytes % 16 == 0;
    if (!fits || !chunked) {
        const int64_t blocks = tiles_of(p, kAnyTile, kAnyTile);
        if (blocks >= int64_t(1) << 31) return NUCLEUS_EINVAL;
        hipLaunchKernelGGL(project_any_kernel<DT>, dim3((unsigned)blocks), dim3(kAnyThreads), 0, s, p);
        return launched();
    }
    switch (choose(p, DT == kF32)) {
    case 0: return launch_split<DT, 16, 4>(p, s);
    case 1: return launch_split<DT, 32, 3>(p, s);
    case 2: return launch_split<DT, 48, 2>(p, s);
    case 3: return launch_split<DT, 64, 2>(p, s);
    case 4: return launch_tile<DT, 64, 32, 4, 1, 6>(p, s);
    case 5: return launch_tile<DT, 64, 64, 2, 2, 4>(p, s);
    case 6: return launch_tile<DT, 128, 64, 4, 1, 3>(p, s);
    case 7: return launch_tile<DT, 128, 128, 2, 2, 2>(p, s);
    default:
        if constexpr (DT != kF32) return launch_tile<DT, 256, 256, 4, 2, 2>(p, s);
        return NUCLEUS_EINVAL;  // not chosen for fp32
    }
}

}  // namespace

extern "C" int nucleus_project(const void* hidden, const void* weight, int64_t M, int64_t N, int64_t K, void* out,
                               const nucleus_project_options* opt)
{
    const nucleus_project_options none = {};
    const nucleus_project_options& o = opt ? *opt : none;
    // Products of sizes and strides below stay far inside 64 bits.
    const int64_t most = int64_t(1) << 31;
    if (M < 0 || N < 0 || K < 1 || M >= most || N >= most || K >= most) return NUCLEUS_EINVAL;
    if (!known_dtype(o.dtype) || (o.out_dtype != NUCLEUS_F32 && o.out_dtype != o.dtype)) return NUCLEUS_EINVAL;
    if (o.activation < NUCLEUS_ACT_NONE || o.activation > NUCLEUS_ACT_SOFTCAP) return NUCLEUS_EINVAL;
    if (o.activation == NUCLEUS_ACT_SOFTCAP && !(o.softcap > 0.0f && o.softcap < INFINITY)) return NUCLEUS_EINVAL;
    if (o.bias && o.bias_dtype != NUCLEUS_F32 && o.bias_dtype != o.dtype) return NUCLEUS_EINVAL;
    if (o.residual && o.residual_dtype != NUCLEUS_F32 && o.residual_dtype != o.dtype) return NUCLEUS_EINVAL;
    const int64_t hs = o.hidden_stride ? o.hidden_stride : K, ws = o.weight_stride ? o.weight_stride : K;
    const int64_t os = o.out_stride ? o.out_stride : N, rs = o.residual_stride ? o.residual_stride : N;
    if (hs < K || ws < K || os < N || rs < N || hs >= most || ws >= most || os >= most || rs >= most)
        return NUCLEUS_EINVAL;
    if (M == 0 || N == 0) return NUCLEUS_OK;
    if (!hidden || !weight || !out) return NUCLEUS_EINVAL;
    const size_t esz = elem_bytes(o.dtype), osz = elem_bytes(o.out_dtype);
    const size_t bsz = elem_bytes(o.bias_dtype), rsz = elem_bytes(o.residual_dtype);
    if ((uintptr_t)hidden % esz || (uintptr_t)weight % esz || (uintptr_t)out % osz || (uintptr_t)o.bias % bsz ||
        (uintptr_t)o.residual % rsz)
        return NUCLEUS_EINVAL;
    // Other workgroups read what this one would overwrite; only the residual
    // may be the output itself (each element is read before it is written).
    const Span to(out, M, N, os, osz);
    if (to.meets(Span(hidden, M, K, hs, esz)) || to.meets(Span(weight, N, K, ws, esz)) ||
        (o.bias && to.meets(Span(o.bias, 1, N, N, bsz))))
        return NUCLEUS_EINVAL;
    if (o.residual && to.meets(Span(o.residual, M, N, rs, rsz)) &&
        !(o.residual == out && rs == os && o.residual_dtype == o.out_dtype))
        return NUCLEUS_EINVAL;
    const int dev_rc = check_device();
    if (dev_rc != NUCLEUS_OK) return dev_rc;

    ProjectParams p = {};
    p.h = (const char*)hidden;
    p.w = (const char*)weight;
    p.out = (char*)out;
    p.bias = o.bias;
    p.res = o.residual;
    p.M = M;
    p.N = N;
    p.K = K;
    p.hs = hs * (int64_t)esz;
    p.ws = ws * (int64_t)esz;
    p.os = os;
    p.rs = rs;
    p.cap = o.softcap;
    p.per_cap = o.softcap > 0x1p-100f && o.softcap < 0x1p100f ? 1.0f / o.softcap : 0.0f;
    p.act = o.activation;
    p.out_f32 = o.out_dtype == NUCLEUS_F32;
    p.bias_f32 = o.bias_dtype == NUCLEUS_F32;
    p.res_f32 = o.residual_dtype == NUCLEUS_F32;
    p.vec = N % 4 == 0 && os % 4 == 0 && (uintptr_t)out % (4 * osz) == 0 && (!o.bias || (uintptr_t)o.bias % (4 * bsz) == 0) &&
            (!o.residual || (rs % 4 == 0 && (uintptr_t)o.residual % (4 * rsz) == 0));
    hipStream_t s = (hipStream_t)o.stream;
    if (o.dtype == NUCLEUS_F32) return launch<kF32>(p, s);
    if (o.dtype == NUCLEUS_BF16) return launch<kBF16>(p, s);
    return launch<kF16>(p, s);
}
