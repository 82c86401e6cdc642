// Verification of drafted tokens (df11_verify_drafts) by rejection sampling:
// draft d_i is taken while u_i q_i(d_i) < p_i(d_i); at the first one refused
// a token is drawn from max(p - q, 0), behind the last one from p.
//
// The draw inverts the running sum.  Probabilities are taken as whole
// multiples of 2^-40 and summed as 64-bit integers, so the sum of a range,
// and with it the drawn token, is the same however the vocabulary is split;
// u has 24 bits, and the product u * (whole sum) is cut to a whole number.
#include <algorithm>

#include "df11_internal.h"
#include "serve_device.h"

namespace {

using namespace df11serve;

typedef unsigned long long u64;

struct Args {
    const void *draft_tokens;
    const int32_t *counts;
    const uint8_t *target, *draft;
    const float *uniforms;
    void *tokens;
    int32_t *accepted;
    int32_t token_bytes, batch, drafts, vocab;
    int64_t target_batch, target_row, draft_batch, draft_row;
};

constexpr int kThreads = 1024;

struct F32 {
    typedef float type;
    static __device__ __forceinline__ float value(float x) { return x; }
};
struct BF {
    typedef uint16_t type;
    static __device__ __forceinline__ float value(uint16_t x)
    {
        return __builtin_bit_cast(float, (uint32_t)x << 16);
    }
};
struct HF {
    typedef uint16_t type;
    static __device__ __forceinline__ float value(uint16_t x) { return (float)__builtin_bit_cast(_Float16, x); }
};

// p in whole multiples of 2^-40, of p clamped to [0, 1]; NaN is 0
__device__ __forceinline__ u64 whole(float p)
{
    p = p > 0.0f ? fminf(p, 1.0f) : 0.0f;
    return (u64)(p * 1099511627776.0f);
}

__device__ __forceinline__ int64_t token(const void *t, int bytes, int64_t i)
{
    return bytes == 8 ? ((const int64_t *)t)[i] : ((const int32_t *)t)[i];
}

__device__ __forceinline__ void put(void *t, int bytes, int64_t i, int64_t v)
{
    if (bytes == 8) ((int64_t *)t)[i] = v;
    else ((int32_t *)t)[i] = (int32_t)v;
}

// Sum over the workgroup of the values before this thread's, and of all.
__device__ __forceinline__ void scan(u64 x, u64 *part, u64 &before, u64 &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    u64 s = x;
    for (int d = 1; d < 64; d <<= 1) {
        const u64 y = __shfl_up(s, d);
        if (lane >= d) s += y;
    }
    __syncthreads();
    if (lane == 63) part[wave] = s;
    __syncthreads();
    before = s - x;
    total = 0;
    for (int w = 0; w < kThreads / 64; w++) {
        if (w < wave) before += part[w];
        total += part[w];
    }
}

// The weight of token i where the row of p is `p` and that of q is `q`
// (null: certain of token `sure`, -1 none).
template <class T>
__device__ __forceinline__ u64 weight(const typename T::type *p, const typename T::type *q, int64_t sure, int i, bool rest)
{
    const u64 x = whole(T::value(p[i]));
    if (!rest) return x;
    const u64 y = q ? whole(T::value(q[i])) : i == sure ? 1ull << 40 : 0;
    return x > y ? x - y : 0;
}

// One workgroup for each sequence; each thread has a run of the vocabulary.
template <class T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const Args a)
{
    typedef typename T::type type;
    __shared__ u64 part[kThreads / 64];
    __shared__ int first_refused, drawn;
    const int b = blockIdx.x;
    const int count = a.counts ? max(0, min(a.counts[b], a.drafts)) : a.drafts;
    if (threadIdx.x == 0) first_refused = count, drawn = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const int64_t d = token(a.draft_tokens, a.token_bytes, (int64_t)b * a.drafts + i);
        double p = 0.0, q = 0.0;
        if (d >= 0 && d < a.vocab) {
            p = T::value(((const type *)a.target)[b * a.target_batch + i * a.target_row + d]);
            q = a.draft ? (double)T::value(((const type *)a.draft)[b * a.draft_batch + i * a.draft_row + d]) : 1.0;
        }
        const double u = a.uniforms[(int64_t)b * (a.drafts + 1) + i];
        if (!(u * q < p)) atomicMin(&first_refused, i);
    }
    __syncthreads();
    const int n = first_refused;
    const type *p = (const type *)a.target + b * a.target_batch + n * a.target_row;
    const type *q = a.draft && n < count ? (const type *)a.draft + b * a.draft_batch + n * a.draft_row : nullptr;
    const int64_t sure = n < count ? token(a.draft_tokens, a.token_bytes, (int64_t)b * a.drafts + n) : -1;
    const int run = (a.vocab + kThreads - 1) / kThreads;
    const int i0 = min(a.vocab, (int)threadIdx.x * run), i1 = min(a.vocab, i0 + run);
    bool rest = n < count;
    u64 before, total, mine;
    for (;;) {
        mine = 0;
        for (int i = i0; i < i1; i++) mine += weight<T>(p, q, sure, i, rest);
        scan(mine, part, before, total);
        if (total || !rest) break;
        rest = false;
    }
    // the token whose share of the sum holds u * total
    const u64 u = (u64)(fminf(fmaxf(a.uniforms[(int64_t)b * (a.drafts + 1) + a.drafts], 0.0f), 0.99999994f) * 16777216.0f);
    const u64 goal = __umul64hi(u << 40, total);
    if (total && before <= goal && goal < before + mine) {
        u64 s = before;
        for (int i = i0; i < i1; i++) {
            s += weight<T>(p, q, sure, i, rest);
            if (goal < s) {
                drawn = i;
                break;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= a.drafts; i += kThreads) {
        const int64_t at = (int64_t)b * (a.drafts + 1) + i;
        put(a.tokens, a.token_bytes, at,
            i < n ? token(a.draft_tokens, a.token_bytes, (int64_t)b * a.drafts + i) : i == n ? drawn : -1);
    }
    if (threadIdx.x == 0) a.accepted[b] = n;
}

int check(const df11_verify_args *p, Args &a)
{
    const char *who = "df11_verify_drafts";
    if (!p) return df11::fail(DF11_E_ARG, "%s: null arguments", who);
    if (p->dtype != DF11_BF16 && p->dtype != DF11_FP16 && p->dtype != DF11_FP32)
        return df11::fail(DF11_E_ARG, "%s: dtype must be bf16, fp16 or fp32", who);
    if (p->token_bytes != 4 && p->token_bytes != 8)
        return df11::fail(DF11_E_ARG, "%s: tokens must be int32 or int64", who);
    if (p->batch < 0 || p->batch > (1 << 20) || p->drafts < 0 || p->drafts > 1024 || p->vocab < 1 ||
        p->vocab > (1 << 22))
        return df11::fail(DF11_E_ARG, "%s: batch, drafts or vocab out of range", who);
    if (p->target_batch < 0 || p->target_row < 0 || p->draft_batch < 0 || p->draft_row < 0)
        return df11::fail(DF11_E_ARG, "%s: negative stride", who);
    a = Args{p->draft_tokens, p->counts, (const uint8_t *)p->target_probs, (const uint8_t *)p->draft_probs, p->uniforms,
             p->tokens, p->accepted, (int32_t)p->token_bytes, (int32_t)p->batch, (int32_t)p->drafts, (int32_t)p->vocab,
             p->target_batch, p->target_row, p->draft_batch, p->draft_row};
    return DF11_OK;
}

}  // namespace

extern "C" uint64_t df11_verify_drafts_workspace_bytes(const df11_verify_args *p)
{
    (void)p;
    return 0;
}

extern "C" int df11_verify_drafts(const df11_verify_args *p, void *workspace, uint64_t workspace_bytes, void *stream)
{
    const char *who = "df11_verify_drafts";
    Args a;
    const int rc = check(p, a);
    if (rc) return rc;
    if (!a.batch) return DF11_OK;
    const uintptr_t mask = p->dtype == DF11_FP32 ? 3 : 1;
    if (!a.target || ((uintptr_t)a.target & mask) || ((uintptr_t)a.draft & mask) || !a.uniforms || !a.tokens ||
        !a.accepted || (a.drafts && !a.draft_tokens))
        return df11::fail(DF11_E_ARG, "%s: null or misaligned pointer", who);
    hipStream_t st = (hipStream_t)stream;
    if (p->dtype == DF11_FP32) hipLaunchKernelGGL(verify_kernel<F32>, dim3(a.batch), dim3(kThreads), 0, st, a);
    else if (p->dtype == DF11_BF16) hipLaunchKernelGGL(verify_kernel<BF>, dim3(a.batch), dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL(verify_kernel<HF>, dim3(a.batch), dim3(kThreads), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return df11::fail(DF11_E_DEVICE, "%s launch: %s", who, hipGetErrorString(e));
    return DF11_OK;
}
