// given.hip -- the entry points that draw from random numbers the caller
// brings: nucleus_sample_given and nucleus_spec_verify_given (declared in
// include/nucleus.h).
#include <hip/hip_runtime.h>

#include "nucleus.h"
#include "given.h"
#include "host.h"

using namespace nucleus;

namespace {

// Options that only other entry points take.
bool other_options(const nucleus_options* o)
{
    return o->flags || o->seeds || o->out_logprobs || o->out_min_kept_logit || o->history || o->history_len ||
           o->repetition_penalty || o->frequency_penalty || o->presence_penalty || o->allowed_mask ||
           o->split_give_up_row;
}

int64_t parts_of(int64_t V, int32_t dtype)
{
    const int64_t tokens = dtype == NUCLEUS_F32 ? part_tokens<kF32>() : part_tokens<kBF16>();
    const int64_t C = (V + tokens - 1) / tokens;
    return C <= kMaxParts ? C : 0;
}

// Rows are split where that is faster.  Up to 128 rows leave CUs idle at one
// workgroup a row, but the split's launches cost 10 to 20 us whatever the row:
// it pays from 40960 float32 and 49152 16-bit logits a row (us split / on one
// workgroup, float32: 1 row of 32768 35 / 31, of 65536 38 / 46, of 128256
// 42 / 73; 128 rows of 65536 49 / 51, of 128256 66 / 80; bf16: 8 rows of 32768
// 42 / 35, of 65536 46 / 48, of 128256 50 / 76; 128 rows of 128256 68 / 80).
// With more rows one workgroup a row fills the device (256 rows of 65536
// float32 61 / 57, of 128256 bf16 87 / 81).  Float32 rows of 12 parts and more
// are split up to 1024 rows: 256 alike rows of 128256 84 / 85 and 1024 302 / 321,
// and where the rows' kept sets differ in size one workgroup waits for the
// largest (84 / 97).  The workspace, a third of the logits' size there, is why
// larger batches are not.
bool split_pays(int64_t B, int64_t V, int32_t dtype)
{
    const int64_t C = parts_of(V, dtype);
    return (C >= (dtype == NUCLEUS_F32 ? 6 : 4) && B <= 128) || (C >= 12 && dtype == NUCLEUS_F32 && B <= 1024);
}

// Up to this many rows the first pass is split too; from there one workgroup
// a row is faster (rows of 128256 float32: 1 row 42 / 45 us, 32 rows 52 / 52,
// 64 rows 62 / 57).
constexpr int64_t kSplitFirst = 32;

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// The workspace of a split batch, and its regions when `base` is given.
size_t lay_out(int64_t B, int64_t C, char* base, GivenWork* wk)
{
    size_t at = 0;
    const auto region = [&](size_t bytes) {
        char* r = base + at;
        at += align256(bytes);
        return r;
    };
    const size_t parts = (size_t)B * (size_t)C;
    GivenWork o;
    o.state = (RowState*)region((size_t)B * sizeof(RowState));
    o.head = (PartHead*)region(parts * sizeof(PartHead));
    o.tail = (PartTail*)region(parts * sizeof(PartTail));
    o.sub = (double*)region(parts * kPartSegs * 8);
    o.und = (uint32_t*)region(parts * kPartSegs * 4);
    o.list = (uint2*)region(parts * kPartCap * 8);
    o.joined = (uint64_t*)region((size_t)B * kSlots * 8);
    o.hist = nullptr;
    o.cnt = nullptr;
    if (B <= kSplitFirst) {
        o.hist = (uint64_t*)region(parts * kSlots * 8);
        o.cnt = (uint32_t*)region(parts * kSlots * 4);
    }
    o.C = (int)C;
    if (wk) *wk = o;
    return at;
}

template <int DT, bool VEC>
void launch_rows(const GivenParams& p, const GivenWork* wk, hipStream_t s)
{
    const dim3 rows((unsigned)p.B), wide(kDrawThreads);
    if (!wk) {
        hipLaunchKernelGGL((given_row_kernel<DT, VEC, kDrawThreads>), rows, wide, 0, s, p);
        return;
    }
    const dim3 parts((unsigned)(p.B * wk->C)), narrow(kPartThreads);
    if (wk->hist) {
        hipLaunchKernelGGL((given_hist_kernel<DT, VEC>), parts, narrow, 0, s, p, *wk);
        hipLaunchKernelGGL((given_plan_kernel<kDrawThreads>), rows, wide, 0, s, p, *wk);
    } else {
        hipLaunchKernelGGL((given_first_kernel<DT, VEC, kDrawThreads>), rows, wide, 0, s, p, *wk);
    }
    hipLaunchKernelGGL((given_mass_kernel<DT, VEC>), parts, narrow, 0, s, p, *wk);
    hipLaunchKernelGGL((given_draw_kernel<DT, VEC, kDrawThreads>), rows, wide, 0, s, p, *wk);
    if (p.out_probs) hipLaunchKernelGGL((given_probs_kernel<DT, VEC>), parts, narrow, 0, s, p, *wk);
}

template <int DT>
int launch_sample(const GivenParams& p, bool vec, const GivenWork* wk, hipStream_t s)
{
    if (vec)
        launch_rows<DT, true>(p, wk, s);
    else
        launch_rows<DT, false>(p, wk, s);
    return hipGetLastError() == hipSuccess ? NUCLEUS_OK : NUCLEUS_ELAUNCH;
}

size_t uniform_bytes(int32_t dtype) { return dtype == NUCLEUS_F64 ? 8 : 4; }

}  // namespace

extern "C" size_t nucleus_given_workspace_bytes(int64_t B, int64_t V, int32_t dtype)
{
    if (B < 1 || B >= (int64_t(1) << 31) || V < 1 || V >= (int64_t(1) << 31)) return 0;
    if (dtype != NUCLEUS_F32 && dtype != NUCLEUS_BF16 && dtype != NUCLEUS_F16) return 0;
    return split_pays(B, V, dtype) ? lay_out(B, parts_of(V, dtype), nullptr, nullptr) : 0;
}

extern "C" int nucleus_sample_given(const void* logits, int64_t B, int64_t V, const float* temperature,
                                    const float* top_p, const int32_t* top_k, const float* min_p, const void* uniforms,
                                    int32_t uniform_dtype, int64_t N, int32_t* out_token, int32_t* out_keep_count,
                                    float* out_token_logprob, float* out_probs, const nucleus_options* opt)
{
    const nucleus_options none = {};
    const nucleus_options& o = opt ? *opt : none;
    const int64_t most = int64_t(1) << 31;
    const int64_t stride = o.row_stride ? o.row_stride : V;
    if (B < 0 || B >= most || V < 1 || V >= most || N < 1 || N >= most || stride < V) return NUCLEUS_EINVAL;
    if (o.dtype != NUCLEUS_F32 && o.dtype != NUCLEUS_BF16 && o.dtype != NUCLEUS_F16) return NUCLEUS_EINVAL;
    if (uniform_dtype != NUCLEUS_F32 && uniform_dtype != NUCLEUS_F64) return NUCLEUS_EINVAL;
    if (other_options(&o)) return NUCLEUS_EINVAL;
    if (B == 0) return NUCLEUS_OK;
    if (!logits || !temperature || !top_p || !uniforms || !out_token || !out_keep_count) return NUCLEUS_EINVAL;
    const size_t esz = o.dtype == NUCLEUS_F32 ? 4 : 2;
    if ((uintptr_t)logits % esz || !aligned(temperature) || !aligned(top_p) || !aligned(top_k) || !aligned(min_p) ||
        (uintptr_t)uniforms % uniform_bytes(uniform_dtype) || !aligned(out_token) || !aligned(out_keep_count) ||
        !aligned(out_token_logprob) || !aligned(out_probs))
        return NUCLEUS_EINVAL;
    // Without a workspace every row runs on one workgroup.
    const size_t need = o.workspace ? nucleus_given_workspace_bytes(B, V, o.dtype) : 0;
    if (need && (o.workspace_bytes < need || (uintptr_t)o.workspace % 256)) return NUCLEUS_EWORKSPACE;
    const int dev_rc = check_device();
    if (dev_rc != NUCLEUS_OK) return dev_rc;

    GivenParams p = {};
    p.logits = logits;
    p.B = B;
    p.V = V;
    p.stride = stride;
    p.temperature = temperature;
    p.top_p = top_p;
    p.top_k = top_k;
    p.min_p = min_p;
    p.uniforms = uniforms;
    p.N = N;
    p.u_f64 = uniform_dtype == NUCLEUS_F64;
    p.out_token = out_token;
    p.out_count = out_keep_count;
    p.out_logprob = out_token_logprob;
    p.out_probs = out_probs;
    // 16-byte loads: rows start on 16-byte boundaries and are whole groups.
    const bool vec = (uintptr_t)logits % 16 == 0 && ((size_t)stride * esz) % 16 == 0 && ((size_t)V * esz) % 16 == 0;
    int log2v = 0;
    while ((int64_t(1) << log2v) < V) ++log2v;
    p.bits = 62 - log2v < 50 ? 62 - log2v : 50;
    hipStream_t s = (hipStream_t)o.stream;
    GivenWork wk;
    if (need) lay_out(B, parts_of(V, o.dtype), (char*)o.workspace, &wk);
    const GivenWork* split = need ? &wk : nullptr;
    if (o.dtype == NUCLEUS_F32) return launch_sample<kF32>(p, vec, split, s);
    if (o.dtype == NUCLEUS_BF16) return launch_sample<kBF16>(p, vec, split, s);
    return launch_sample<kF16>(p, vec, split, s);
}

extern "C" size_t nucleus_spec_given_workspace_bytes(int64_t B, int64_t V)
{
    if (B < 0 || B >= (int64_t(1) << 31) || V < 1 || V >= (int64_t(1) << 31)) return 0;
    if (V <= kPickShort) return 0;
    return ((size_t)B * (size_t)((V + kPickChunk - 1) / kPickChunk) * 8 + 255) / 256 * 256;
}

extern "C" int nucleus_spec_verify_given(const float* target_probs, const float* draft_probs,
                                         const int32_t* draft_token, int64_t B, int64_t V, const void* uniforms,
                                         int32_t uniform_dtype, int32_t* out_token, int32_t* out_accepted,
                                         const nucleus_options* opt)
{
    const int64_t most = int64_t(1) << 31;
    if (B < 0 || B >= most || V < 1 || V >= most) return NUCLEUS_EINVAL;
    if (uniform_dtype != NUCLEUS_F32 && uniform_dtype != NUCLEUS_F64) return NUCLEUS_EINVAL;
    if (opt && (other_options(opt) || opt->dtype != NUCLEUS_F32 || (opt->row_stride && opt->row_stride != V)))
        return NUCLEUS_EINVAL;
    if (B == 0) return NUCLEUS_OK;
    if (!target_probs || !draft_probs || !draft_token || !uniforms || !out_token) return NUCLEUS_EINVAL;
    if (!aligned(target_probs) || !aligned(draft_probs) || !aligned(draft_token) ||
        (uintptr_t)uniforms % uniform_bytes(uniform_dtype) || !aligned(out_token) || !aligned(out_accepted))
        return NUCLEUS_EINVAL;
    const int64_t C = (V + kPickChunk - 1) / kPickChunk;
    if (B * C >= most) return NUCLEUS_EINVAL;
    const size_t need = nucleus_spec_given_workspace_bytes(B, V);
    if (need && (!opt || !opt->workspace || opt->workspace_bytes < need || (uintptr_t)opt->workspace % 256))
        return NUCLEUS_EWORKSPACE;
    const int dev_rc = check_device();
    if (dev_rc != NUCLEUS_OK) return dev_rc;

    PickParams p = {};
    p.target = target_probs;
    p.draft = draft_probs;
    p.draft_token = draft_token;
    p.uniforms = uniforms;
    p.u_f64 = uniform_dtype == NUCLEUS_F64;
    p.B = B;
    p.V = V;
    p.out_token = out_token;
    p.out_accepted = out_accepted;
    p.part = need ? (double*)opt->workspace : nullptr;
    p.C = (int)C;
    p.vec = V % 4 == 0 && (uintptr_t)target_probs % 16 == 0 && (uintptr_t)draft_probs % 16 == 0;
    hipStream_t s = opt ? (hipStream_t)opt->stream : nullptr;
    // (us a call, one launch / two: 5 rows of 8192 7.8 / 9.7, of 32000 9.9 / 10.4,
    // of 65536 11.8 / 10.2, of 128256 16.9 / 11.9; 256 rows of 32000, half of them
    // rejected, 13.7 / 16.6, of 128256 30 / 32 and with a twentieth rejected 19 / 15)
    if (V <= kPickShort) {
        hipLaunchKernelGGL(pick_row_kernel, dim3((unsigned)B), dim3(kPickWide), 0, s, p);
    } else {
        hipLaunchKernelGGL(pick_chunk_kernel, dim3((unsigned)(B * C)), dim3(kPickThreads), 0, s, p);
        hipLaunchKernelGGL(pick_finish_kernel, dim3((unsigned)B), dim3(kPickThreads), 0, s, p);
    }
    return hipGetLastError() == hipSuccess ? NUCLEUS_OK : NUCLEUS_ELAUNCH;
}
