// What stands between a model's logits and the choice of a token
// (df11_adjust_logits): penalties for tokens that a request has seen, biases,
// and the tokens that its grammar allows.
//
// A workgroup takes a part of the vocabulary of one sequence.  It counts the
// part's tokens in the sequence's history in LDS (whole numbers, so no order
// of the additions shows) and lists them, copies the part of each of its rows
// under the grammar's mask, and goes over the listed tokens once more, in 64
// bits: with several rows that is faster than changing them before they are written,
// where each wave waits for the lane that holds the most of them (32 x 5 rows:
// 24 and 35 us).  Bound by memory: 128 rows of 128256 tokens in float32 with
// histories of 8192, 137 MB in 38 us, 3.6 TB/s (the words are cleared and the
// history is read before the copy begins); one row: 5.8 us, latency.
#include <algorithm>

#include "df11_internal.h"
#include "overlap.h"
#include "serve_device.h"

namespace {

using namespace df11serve;

struct Args {
    const uint8_t *logits;
    uint8_t *out;
    const void *history, *drafts, *bias_tokens;
    const int32_t *lengths, *prompt_lengths;
    const float *repetition, *presence, *frequency, *bias_values;
    const uint8_t *mask;
    int32_t batch, tokens, vocab, history_tokens, biases, rows;   // rows: of a workgroup
    int64_t logits_batch, logits_token, out_batch, out_token, history_batch, draft_batch, bias_batch, mask_batch, mask_token;
    bool counts, penalties;
};

constexpr int kPart = 8192;      // tokens of a workgroup
constexpr int kThreads = 512;

// A token's word in LDS: how often it was said, whether it has a bias, and
// whether the prompt held it.
constexpr uint32_t kCount = 0x3fffffffu, kBiased = 0x40000000u, kPrompt = 0x80000000u;

struct F32 {
    typedef float type;
    static __device__ __forceinline__ float value(float x) { return x; }
    static __device__ __forceinline__ float round(float x) { return x; }
};
template <class E>
struct Half {
    typedef uint16_t type;
    static __device__ __forceinline__ float value(uint16_t x) { return E::value(x); }
    static __device__ __forceinline__ uint16_t round(float x) { return (uint16_t)E::pack(x, 0.0f); }
};

struct Bias {
    int32_t token;   // within the part
    float value;
};

// What a part's tokens are known by: their words, and the list of those whose
// word is not zero.
struct Seen {
    uint32_t *words;
    uint16_t *list;
    int *listed;
    __device__ __forceinline__ void add(uint32_t at, uint32_t old) const
    {
        if (!old) list[atomicAdd(listed, 1)] = (uint16_t)at;   // the first to touch it
    }
};

// A thread's share of a history, and the count of all of it: V tokens at a
// time, the first kAhead of them loaded ahead of the lengths.
template <class I>
struct History {
    static constexpr int V = 16 / sizeof(I), kAhead = 2;
    struct Vec { I x[V]; };
    Vec ahead[kAhead];
    __device__ __forceinline__ void load(const I *tokens, int room)
    {
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            const int k = threadIdx.x + j * kThreads;
            if ((k + 1) * V <= room) __builtin_memcpy(&ahead[j], tokens + (int64_t)k * V, 16);
        }
    }
    __device__ __forceinline__ void count(const Seen &seen, const I *tokens, int n, int prompt, int64_t part, int size) const
    {
        const auto one = [&](int i, int64_t token) {
            const uint64_t at = (uint64_t)(token - part);
            if (at >= (uint64_t)size) return;
            seen.add((uint32_t)at, i < prompt ? atomicOr(seen.words + at, kPrompt) : atomicAdd(seen.words + at, 1u));
        };
        const int vecs = n / V;
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            const int k = threadIdx.x + j * kThreads;
            if (k < vecs)
#pragma unroll
                for (int i = 0; i < V; i++) one(k * V + i, ahead[j].x[i]);
        }
        for (int k = threadIdx.x + kAhead * kThreads; k < vecs; k += kThreads) {
            Vec v;
            __builtin_memcpy(&v, tokens + (int64_t)k * V, 16);
#pragma unroll
            for (int i = 0; i < V; i++) one(k * V + i, v.x[i]);
        }
        const int i = vecs * V + threadIdx.x;
        if (i < n) one(i, tokens[i]);
    }
};

template <class T, class I>
__global__ void __launch_bounds__(kThreads, 6) adjust_kernel(const Args a)
{
    typedef typename T::type type;
    constexpr int V = 16 / sizeof(type), kVecs = kPart / V / kThreads;
    struct Vec { type x[V]; };
    extern __shared__ __align__(16) uint32_t words[];   // [kPart], the list, then the part's biases in their order
    __shared__ int listed, wave_biases[kThreads / 64];
    uint16_t *const list = (uint16_t *)(words + kPart);
    Bias *const biases = (Bias *)(list + kPart);
    const Seen seen{words, list, &listed};
    const int b = blockIdx.x, part = blockIdx.y * kPart, size = min(kPart, a.vocab - part);
    const int t0 = blockIdx.z * a.rows, t1 = min(a.tokens, t0 + a.rows);
    const I *drafts = a.drafts ? (const I *)a.drafts + b * a.draft_batch : nullptr;
    const I *history = (const I *)a.history + b * a.history_batch;
    const int vecs = size / V, behind = vecs * V + threadIdx.x;   // whole vectors, and this thread's token behind them
    const type minus = T::round(-INFINITY);
    const auto row_of = [&](int t) { return (const type *)a.logits + b * a.logits_batch + t * a.logits_token + part; };
    const auto mask_of = [&](int t) { return a.mask ? a.mask + 4 * (b * a.mask_batch + t * a.mask_token) + part / 8 : nullptr; };
    // All that comes from memory is on its way before anything is waited for;
    // a row's logits also while the row before is finished.
    History<I> ahead;
    if (a.penalties) ahead.load(history, a.history_tokens);
    I bias_token = -1;
    float bias_value = 0.0f;
    const auto load_bias = [&](int j) {
        if (j < a.biases) {
            bias_token = ((const I *)a.bias_tokens)[b * a.bias_batch + j];
            bias_value = a.bias_values[(int64_t)b * a.biases + j];
        }
    };
    if (a.biases) load_bias(threadIdx.x);
    Vec v[kVecs];
    uint8_t allowed[kVecs];   // the mask's byte that holds their bits
    const auto load = [&](int t) {
        const type *from = row_of(t);
        const uint8_t *mask = mask_of(t);
#pragma unroll
        for (int j = 0; j < kVecs; j++) {
            const int k = threadIdx.x + j * kThreads;
            if (k >= vecs) continue;
            __builtin_memcpy(&v[j], from + k * V, 16);
            if (mask) allowed[j] = mask[k * V / 8];
        }
    };
    load(t0);
    int bias_count = 0;
    if (a.counts) {
        for (int i = threadIdx.x; i < kPart / 4; i += kThreads) ((u32x4 *)words)[i] = u32x4{0, 0, 0, 0};
        if (threadIdx.x == 0) listed = 0;
        lds_barrier();
        if (a.penalties) {
            const int n = a.history_tokens ? max(0, min(a.lengths[b], a.history_tokens)) : 0;
            const int prompt = a.prompt_lengths ? max(0, min(a.prompt_lengths[b], n)) : 0;
            ahead.count(seen, history, n, prompt, part, size);
            for (int i = threadIdx.x; drafts && i < t0; i += kThreads) {
                const uint64_t at = (uint64_t)((int64_t)drafts[i] - part);
                if (at < (uint64_t)size) seen.add((uint32_t)at, atomicAdd(words + at, 1u));
            }
        }
        // the part's biases, in their order: each wave's behind those of the waves before it
        for (int j0 = 0; j0 < a.biases; j0 += kThreads) {
            const int j = j0 + threadIdx.x;
            if (j0) load_bias(j);
            const uint64_t place = (uint64_t)((int64_t)bias_token - part);
            const bool in = j < a.biases && place < (uint64_t)size;
            const uint64_t all = __ballot(in);
            if ((threadIdx.x & 63) == 0) wave_biases[threadIdx.x >> 6] = __popcll(all);
            lds_barrier();
            int at = bias_count;
            for (int w = 0; w < kThreads / 64; w++) {
                at += w < (int)(threadIdx.x >> 6) ? wave_biases[w] : 0;
                bias_count += wave_biases[w];
            }
            if (in) {
                biases[at + __popcll(all & ((1ull << (threadIdx.x & 63)) - 1))] = Bias{(int32_t)place, bias_value};
                seen.add((uint32_t)place, atomicOr(words + place, kBiased));
            }
            if (j0 + kThreads < a.biases) lds_barrier();
        }
    }
    const double repetition = a.repetition ? a.repetition[b] : 1.0, presence = a.presence ? a.presence[b] : 0.0;
    const double frequency = a.frequency ? a.frequency[b] : 0.0;
    const auto adjust = [&](float raw, uint32_t word, int at) {
        double x = raw;
        if (a.repetition && (word & ~kBiased)) x = x > 0.0 ? x / repetition : x * repetition;
        if (word & kCount) x -= frequency * (word & kCount) + presence;
        if (word & kBiased) {
            double sum = 0.0;
            for (int j = 0; j < bias_count; j++) sum += biases[j].token == at ? (double)biases[j].value : 0.0;
            x += sum;
        }
        return T::round((float)x);
    };
    for (int t = t0; t < t1; t++) {
        if (t > t0 && a.counts && a.penalties && drafts && threadIdx.x == 0) {
            const uint64_t at = (uint64_t)((int64_t)drafts[t - 1] - part);
            if (at < (uint64_t)size) seen.add((uint32_t)at, words[at]++);
        }
        const type *from = row_of(t);
        const uint8_t *mask = mask_of(t);
        type *to = (type *)a.out + b * a.out_batch + t * a.out_token + part;
        // all of the part as if nothing of it was seen
#pragma unroll
        for (int j = 0; j < kVecs; j++) {
            const int k = threadIdx.x + j * kThreads;
            if (k >= vecs) continue;
#pragma unroll
            for (int i = 0; i < V; i++) v[j].x[i] = !mask || (allowed[j] >> (k * V % 8 + i) & 1) ? v[j].x[i] : minus;
            __builtin_memcpy(to + k * V, &v[j], 16);
        }
        if (behind < size) to[behind] = !mask || (mask[behind / 8] >> (behind % 8) & 1) ? from[behind] : minus;
        if (t + 1 < t1) load(t + 1);
        if (!a.counts) continue;
        // the listed ones once more, behind all those stores; where out is
        // logits itself they hold what they held, or the grammar refuses them
        __syncthreads();
        const int n = listed;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int at = list[i];
            if (!mask || (mask[at / 8] >> (at % 8) & 1)) to[at] = adjust(T::value(from[at]), words[at], at);
        }
        if (t + 1 < t1) __syncthreads();
    }
}

// Whether out lies on some of the logits otherwise than as the logits
// themselves.  Rows of the same strides are compared place by place, of others by
// where all of them lie.
bool out_on_logits(const df11_adjust_logits_args *p)
{
    const bool one_batch = p->batch <= 1, one_row = p->tokens <= 1;
    const Axis batch{p->batch, one_batch ? 0 : p->out_batch}, row{p->tokens, one_row ? 0 : p->out_token};
    const Axis other_batch{p->batch, one_batch ? 0 : p->logits_batch}, other_row{p->tokens, one_row ? 0 : p->logits_token};
    const int bytes = p->dtype == DF11_FP32 ? 4 : 2;
    const __int128 out = (uintptr_t)p->out / bytes, logits = (uintptr_t)p->logits / bytes;
    if (batch.stride == other_batch.stride && row.stride == other_row.stride)
        return out != logits && sets_meet(out - logits, batch, row, p->vocab);
    const auto end = [&](const Axis &x, const Axis &y) {
        return (__int128)(x.size - 1) * x.stride + (__int128)(y.size - 1) * y.stride + p->vocab;
    };
    return out < logits + end(other_batch, other_row) && logits < out + end(batch, row);
}

int check(const df11_adjust_logits_args *p, Args &a)
{
    const char *who = "df11_adjust_logits";
    if (!p) return df11::fail(DF11_E_ARG, "%s: null arguments", who);
    if (p->dtype != DF11_BF16 && p->dtype != DF11_FP16 && p->dtype != DF11_FP32)
        return df11::fail(DF11_E_ARG, "%s: dtype must be bf16, fp16 or fp32", who);
    if (p->token_bytes != 4 && p->token_bytes != 8) return df11::fail(DF11_E_ARG, "%s: tokens must be int32 or int64", who);
    if (p->batch < 0 || p->batch > 65535 || p->tokens < 1 || p->tokens > 65535 || p->vocab < 1 || p->vocab > (1 << 22) ||
        p->history_tokens < 0 || p->history_tokens > (1 << 28) || p->biases < 0 || p->biases > 4096)
        return df11::fail(DF11_E_ARG, "%s: batch, tokens, vocab, history or biases out of range", who);
    if (p->logits_batch < 0 || p->logits_token < 0 || p->out_batch < 0 || p->out_token < 0 || p->history_batch < 0 ||
        p->draft_batch < 0 || p->bias_batch < 0 || p->mask_batch < 0 || p->mask_token < 0)
        return df11::fail(DF11_E_ARG, "%s: negative stride", who);
    // rows of out must not share memory: two workgroups would write them
    const bool rows_apart = p->tokens == 1 || p->out_token >= p->vocab;
    const bool batches_apart = p->batch <= 1 || p->out_batch >= (p->tokens - 1) * p->out_token + p->vocab ||
                               (p->out_batch >= p->vocab && p->tokens > 1 && p->out_token >= (p->batch - 1) * p->out_batch + p->vocab);
    if (!rows_apart || !batches_apart) return df11::fail(DF11_E_ARG, "%s: rows of out share memory", who);
    a = Args{(const uint8_t *)p->logits, (uint8_t *)p->out, p->history, p->draft_tokens, p->bias_tokens, p->lengths,
             p->prompt_lengths, p->repetition, p->presence, p->frequency, p->bias_values, (const uint8_t *)p->mask,
             (int32_t)p->batch, (int32_t)p->tokens, (int32_t)p->vocab, (int32_t)p->history_tokens, (int32_t)p->biases, 1,
             p->logits_batch, p->logits_token, p->out_batch, p->out_token, p->history_batch, p->draft_batch, p->bias_batch,
             p->mask_batch, p->mask_token, false, false};
    a.penalties = (p->repetition || p->presence || p->frequency) && (p->history_tokens || (p->draft_tokens && p->tokens > 1));
    a.counts = a.penalties || p->biases;
    return DF11_OK;
}

}  // namespace

extern "C" int df11_adjust_logits(const df11_adjust_logits_args *p, void *stream)
{
    const char *who = "df11_adjust_logits";
    Args a;
    const int rc = check(p, a);
    if (rc) return rc;
    if (!a.batch) return DF11_OK;
    if (out_on_logits(p)) return df11::fail(DF11_E_ARG, "%s: out shares memory with the logits, and is not the logits", who);
    const uintptr_t mask = p->dtype == DF11_FP32 ? 3 : 1, wide = p->token_bytes - 1;
    if (!a.logits || !a.out || (((uintptr_t)a.logits | (uintptr_t)a.out) & mask) || ((uintptr_t)a.mask & 3) ||
        (a.history_tokens && (!a.history || !a.lengths)) || (a.biases && (!a.bias_tokens || !a.bias_values)) ||
        (((uintptr_t)a.history | (uintptr_t)a.drafts | (uintptr_t)a.bias_tokens) & wide))
        return df11::fail(DF11_E_ARG, "%s: null or misaligned pointer", who);
    const int64_t parts = (a.vocab + kPart - 1) / kPart, cus = df11::cu_count();
    // a sequence's rows share one counting, or are split where that leaves CUs idle
    const int64_t groups = std::min<int64_t>(a.tokens, std::max<int64_t>(1, 2 * cus / (parts * a.batch)));
    a.rows = (int32_t)((a.tokens + groups - 1) / groups);
    const dim3 grid(a.batch, (uint32_t)parts, (a.tokens + a.rows - 1) / a.rows);
    if ((double)grid.x * grid.y * grid.z * kThreads > 4294967295.0)
        return df11::fail(DF11_E_ARG, "%s: too many rows for one launch", who);
    const size_t lds = a.counts ? kPart * 6 + a.biases * sizeof(Bias) : 0;
    const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), lds, (hipStream_t)stream, a); };
    const auto by_tokens = [&](auto t) {
        typedef decltype(t) T;
        if (p->token_bytes == 8) launch(adjust_kernel<T, int64_t>);
        else launch(adjust_kernel<T, int32_t>);
    };
    if (p->dtype == DF11_FP32) by_tokens(F32{});
    else if (p->dtype == DF11_BF16) by_tokens(Half<Bf16>{});
    else by_tokens(Half<Fp16>{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return df11::fail(DF11_E_DEVICE, "%s launch: %s", who, hipGetErrorString(e));
    return DF11_OK;
}
