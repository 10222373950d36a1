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

template <int DT>
int launch(const ProjectParams& p, hipStream_t s)
{
    const int64_t tiles = ((p.N + kAnyTile - 1) / kAnyTile) * ((p.M + kAnyTile - 1) / kAnyTile);
    if (tiles >= int64_t(1) << 31) return NUCLEUS_EINVAL;
    hipLaunchKernelGGL(project_any_kernel<DT>, dim3((unsigned)tiles), dim3(kAnyThreads), 0, s, p);
    return hipGetLastError() == hipSuccess ? NUCLEUS_OK : NUCLEUS_ELAUNCH;
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
