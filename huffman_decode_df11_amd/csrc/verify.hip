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
    int32_t parts;
    u64 *sums;       // [batch][parts][2]
    int32_t *taken;  // [batch]
};

constexpr int kPiece = 8192;            // tokens of a part: a thread's sum of up to 2^40 each is below 2^53
constexpr int kPartThreads = 256;       // of a part's sums: 32 tokens a thread
constexpr int kDrawThreads = 1024;      // of a sequence's draw, which is all latency: 8 tokens a thread
constexpr int kRun = kPiece / kDrawThreads;

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

// p in whole multiples of 2^-40, of p clamped to [0, 1]; NaN is 0.  A
// double holds such numbers, and their sums below 2^53, exactly.
__device__ __forceinline__ double whole(float p) { return __builtin_trunc((double)fminf(fmaxf(p, 0.0f), 1.0f) * 0x1p40); }

__device__ __forceinline__ int64_t token(const void *t, int bytes, int64_t i)
{
    return bytes == 8 ? ((const int64_t *)t)[i] : ((const int32_t *)t)[i];
}

__device__ __forceinline__ void put(void *t, int bytes, int64_t i, int64_t v)
{
    if (bytes == 8) ((int64_t *)t)[i] = v;
    else ((int32_t *)t)[i] = (int32_t)v;
}

__device__ __forceinline__ u64 wave_sum(u64 x)
{
    for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

// Sums over the wave of the values up to this lane's.
__device__ __forceinline__ u64 wave_scan(u64 s)
{
    const int lane = threadIdx.x & 63;
    for (int d = 1; d < 64; d <<= 1) {
        const u64 y = __shfl_up(s, d);
        if (lane >= d) s += y;
    }
    return s;
}

// The rows that a sequence's drawn token comes from: p's and, if a draft was
// refused, q's (null for a certain drafter, whose token is `sure`).
template <class T>
struct Rows {
    const typename T::type *p, *q;
    int64_t sure;
    bool rest;
    // what token i adds to the sum of max(p - q, 0), x its share of p
    __device__ __forceinline__ double left(double x, double y) const { return fmax(x - y, 0.0); }
    __device__ __forceinline__ double refused(int64_t i) const { return i == sure ? 0x1p40 : 0.0; }
};

// The number of drafts taken: where the first is refused.
template <class T, int kThreads>
__device__ __forceinline__ int drafts_taken(const Args &a, int b, int count, int *lds)
{
    typedef typename T::type type;
    if (threadIdx.x == 0) *lds = count;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const int64_t d = token(a.draft_tokens, a.token_bytes, (int64_t)b * a.drafts + i);
        double p = 0.0, q = 0.0;
        if (d >= 0 && d < a.vocab) {
            p = T::value(((const type *)a.target)[b * a.target_batch + i * a.target_row + d]);
            q = a.draft ? (double)T::value(((const type *)a.draft)[b * a.draft_batch + i * a.draft_row + d]) : 1.0;
        }
        const double u = a.uniforms[(int64_t)b * (a.drafts + 1) + i];
        if (!(u * q < p)) atomicMin(lds, i);   // u has 24 bits and q at most 24: the product is exact
    }
    __syncthreads();
    return *lds;
}

template <class T>
__device__ __forceinline__ Rows<T> rows_of(const Args &a, int b, int count, int n)
{
    typedef typename T::type type;
    return Rows<T>{(const type *)a.target + b * a.target_batch + n * a.target_row,
                   a.draft && n < count ? (const type *)a.draft + b * a.draft_batch + n * a.draft_row : nullptr,
                   n < count && !a.draft ? token(a.draft_tokens, a.token_bytes, (int64_t)b * a.drafts + n) : -1,
                   n < count};
}

// The sums over tokens [i0, i1) of max(p - q, 0) (of p behind the last
// draft) and of p, complete in thread 0.  16 bytes of a row a thread at a
// time, at any alignment.
template <class T, int kThreads>
__device__ __forceinline__ void part_sums(const Rows<T> &r, int i0, int i1, u64 *lds, u64 &rest, u64 &all)
{
    typedef typename T::type type;
    constexpr int V = 16 / sizeof(type);
    struct Vec { type x[V]; };
    double sr = 0.0, sp = 0.0;
    const int whole_vecs = (i1 - i0) / V;
#pragma unroll 4
    for (int k = threadIdx.x; k < whole_vecs; k += kThreads) {
        const int i = i0 + k * V;
        Vec p, q;
        __builtin_memcpy(&p, r.p + i, 16);
        if (r.q) __builtin_memcpy(&q, r.q + i, 16);
#pragma unroll
        for (int j = 0; j < V; j++) {
            const double x = whole(T::value(p.x[j]));
            sp += x;
            if (r.rest) sr += r.left(x, r.q ? whole(T::value(q.x[j])) : r.refused(i + j));
        }
    }
    const int i = i0 + whole_vecs * V + threadIdx.x;
    if (i < i1) {
        const double x = whole(T::value(r.p[i]));
        sp += x;
        if (r.rest) sr += r.left(x, r.q ? whole(T::value(r.q[i])) : r.refused(i));
    }
    const u64 wr = wave_sum((u64)sr), wp = wave_sum((u64)sp);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();
    if (lane == 0) lds[wave] = wr, lds[kThreads / 64 + wave] = wp;
    __syncthreads();
    rest = all = 0;
    for (int w = 0; w < kThreads / 64; w++) rest += lds[w], all += lds[kThreads / 64 + w];
    if (!r.rest) rest = all;
}

// Parts of the vocabulary: each writes its two sums.  128 sequences of
// 128256 bfloat16 tokens: 17 to 20 us for about 50 MB.  The vector ALU is busy
// 10 of 17 us (19 instructions a token of p, that of q among them); the waves
// wait the rest, first for the draft, its probabilities and then the rows.
template <class T>
__global__ void __launch_bounds__(kPartThreads) part_kernel(const Args a)
{
    __shared__ u64 lds[2 * kPartThreads / 64];
    __shared__ int first_refused;
    const int part = blockIdx.x, b = blockIdx.y;
    const int count = a.counts ? max(0, min(a.counts[b], a.drafts)) : a.drafts;
    const int n = drafts_taken<T, kPartThreads>(a, b, count, &first_refused);
    if (part == 0 && threadIdx.x == 0) a.taken[b] = n;
    u64 rest, all;
    part_sums<T, kPartThreads>(rows_of<T>(a, b, count, n), part * kPiece, min(a.vocab, (part + 1) * kPiece), lds, rest, all);
    if (threadIdx.x == 0) {
        u64 *to = a.sums + ((int64_t)b * a.parts + part) * 2;
        to[0] = rest, to[1] = all;
    }
}

// One workgroup for each sequence finds the part that holds u times the
// whole sum, in it the thread's run, and in that the token.  A vocabulary of
// one part is summed here too.  All latency: 5.6 us for one sequence (7.4
// with 256 threads), 8 for 128.
template <class T>
__global__ void __launch_bounds__(kDrawThreads) draw_kernel(const Args a)
{
    constexpr int kWaves = kDrawThreads / 64;
    __shared__ u64 lds[2 * kWaves];
    __shared__ int first_refused, drawn;
    const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int count = a.counts ? max(0, min(a.counts[b], a.drafts)) : a.drafts;
    if (threadIdx.x == 0) drawn = -1;
    const int n = a.parts > 1 ? a.taken[b] : drafts_taken<T, kDrawThreads>(a, b, count, &first_refused);
    Rows<T> r = rows_of<T>(a, b, count, n);
    const float last = a.uniforms[(int64_t)b * (a.drafts + 1) + a.drafts];
    const u64 u = (u64)(fminf(fmaxf(last, 0.0f), 0.99999994f) * 16777216.0f);
    u64 rest = 0, all = 0;
    const u64 *sums = a.sums + (int64_t)b * a.parts * 2;
    if (a.parts == 1) {
        part_sums<T, kDrawThreads>(r, 0, a.vocab, lds, rest, all);
    } else {
        // every wave for itself: no wave waits for another
        for (int i = lane; i < a.parts; i += 64) rest += sums[2 * i], all += sums[2 * i + 1];
        rest = wave_sum(rest), all = wave_sum(all);
    }
    if (!rest) r.rest = false;   // nothing is left of p - q: p itself
    const u64 total = rest ? rest : all;
    const u64 goal = __umul64hi(u << 40, total);   // floor(u * total / 2^24), below total
    int part = 0;
    u64 before = 0;
    if (a.parts > 1) {
        for (int i0 = 0; i0 < a.parts; i0 += 64) {
            const u64 x = i0 + lane < a.parts ? sums[2 * (i0 + lane) + (rest ? 0 : 1)] : 0;
            const u64 s = before + wave_scan(x);
            const u64 past = __ballot(goal < s);
            if (past) {
                const int l = __builtin_ctzll(past);
                part = i0 + l, before = __shfl(s - x, l);
                break;
            }
            before = __shfl(s, 63);
        }
    }
    // the part, kRun tokens in a row to a thread
    const int first = part * kPiece + threadIdx.x * kRun;
    typedef typename T::type type;
    constexpr int V = 16 / sizeof(type) < kRun ? 16 / sizeof(type) : kRun;
    type p[kRun], q[kRun];
#pragma unroll
    for (int v = 0; v < kRun; v += V) {
        if (first + v + V <= a.vocab) {
            __builtin_memcpy(p + v, r.p + first + v, V * sizeof(type));
            if (r.q) __builtin_memcpy(q + v, r.q + first + v, V * sizeof(type));
        } else {
#pragma unroll
            for (int j = 0; j < V; j++) {
                const int i = first + v + j;
                p[v + j] = i < a.vocab ? r.p[i] : 0;
                if (r.q) q[v + j] = i < a.vocab ? r.q[i] : 0;
            }
        }
    }
    double x[kRun], sum = 0.0;
#pragma unroll
    for (int j = 0; j < kRun; j++) {
        x[j] = whole(T::value(p[j]));
        if (r.rest) x[j] = r.left(x[j], r.q ? whole(T::value(q[j])) : r.refused(first + j));
        sum += x[j];
    }
    const u64 mine = (u64)sum;
    u64 s = wave_scan(mine);
    __syncthreads();
    if (lane == 63) lds[wave] = s;
    __syncthreads();
    s += before - mine;
    for (int w = 0; w < wave; w++) s += lds[w];
    if (s <= goal && goal < s + mine) {
#pragma unroll
        for (int j = 0; j < kRun; j++) {
            if (s <= goal && goal < s + (u64)x[j]) drawn = first + j;
            s += (u64)x[j];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= a.drafts; i += kDrawThreads) {
        const int64_t at = (int64_t)b * (a.drafts + 1) + i;
        put(a.tokens, a.token_bytes, at,
            i < n ? token(a.draft_tokens, a.token_bytes, (int64_t)b * a.drafts + i) : i == n ? drawn : -1);
    }
    if (threadIdx.x == 0) a.accepted[b] = n;
}

template <class T>
int launch(const Args &a, hipStream_t st)
{
    if (a.parts > 1) hipLaunchKernelGGL(part_kernel<T>, dim3(a.parts, a.batch), dim3(kPartThreads), 0, st, a);
    hipLaunchKernelGGL(draw_kernel<T>, dim3(a.batch), dim3(kDrawThreads), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return df11::fail(DF11_E_DEVICE, "df11_verify_drafts launch: %s", hipGetErrorString(e));
    return DF11_OK;
}

int check(const df11_verify_args *p, Args &a)
{
    const char *who = "df11_verify_drafts";
    if (!p) return df11::fail(DF11_E_ARG, "%s: null arguments", who);
    if (p->dtype != DF11_BF16 && p->dtype != DF11_FP16 && p->dtype != DF11_FP32)
        return df11::fail(DF11_E_ARG, "%s: dtype must be bf16, fp16 or fp32", who);
    if (p->token_bytes != 4 && p->token_bytes != 8)
        return df11::fail(DF11_E_ARG, "%s: tokens must be int32 or int64", who);
    if (p->batch < 0 || p->batch > 65535 || p->drafts < 0 || p->drafts > 1024 || p->vocab < 1 ||
        p->vocab > (1 << 22))
        return df11::fail(DF11_E_ARG, "%s: batch, drafts or vocab out of range", who);
    if (p->target_batch < 0 || p->target_row < 0 || p->draft_batch < 0 || p->draft_row < 0)
        return df11::fail(DF11_E_ARG, "%s: negative stride", who);
    a = Args{p->draft_tokens, p->counts, (const uint8_t *)p->target_probs, (const uint8_t *)p->draft_probs, p->uniforms,
             p->tokens, p->accepted, (int32_t)p->token_bytes, (int32_t)p->batch, (int32_t)p->drafts, (int32_t)p->vocab,
             p->target_batch, p->target_row, p->draft_batch, p->draft_row,
             (int32_t)((p->vocab + kPiece - 1) / kPiece), nullptr, nullptr};
    return DF11_OK;
}

// A vocabulary of one part needs none.
uint64_t workspace_of(const Args &a) { return a.parts > 1 ? 16ull * a.batch * a.parts + 4ull * a.batch : 0; }

}  // namespace

extern "C" uint64_t df11_verify_drafts_workspace_bytes(const df11_verify_args *p)
{
    Args a;
    return check(p, a) ? 0 : workspace_of(a);
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
    const uint64_t need = workspace_of(a);
    if (workspace_bytes < need || (need && !aligned16(workspace)))
        return df11::fail(DF11_E_ARG, "%s: the workspace must be 16-byte aligned and hold %llu bytes", who,
                          (unsigned long long)need);
    a.sums = (u64 *)workspace;
    a.taken = (int32_t *)(a.sums + 2ll * a.batch * a.parts);
    hipStream_t st = (hipStream_t)stream;
    return p->dtype == DF11_FP32 ? launch<F32>(a, st) : p->dtype == DF11_BF16 ? launch<BF>(a, st) : launch<HF>(a, st);
}
