// Eviction from a bounded cache by accumulated attention weight:
// df11_cache_insert puts one token into each head's cache, in the place of
// the slot of least weight when the cache is full; df11_cache_compact cuts a
// long cache down to its latest and heaviest slots.
//
// Both compare whole numbers only (order_of turns a weight into one), and
// equals go to the lowest slot, so what they choose does not depend on the
// order in which the slots are looked at.
#include <algorithm>

#include "df11_internal.h"
#include "serve_device.h"

namespace {

using namespace df11serve;

struct Cache {
    uint16_t *k, *v;
    float *weights;
    int32_t *positions;
    const int32_t *lengths;
    int32_t batch, kv_heads, slots, dim;
    int64_t stride_batch, stride_head, stride_slot;
};

constexpr int kInsertThreads = 512;
constexpr int kInsertEach = 8;   // slots a thread reads at a time

// One workgroup for each sequence and key head.  A slot's rank is one 64-bit
// number, its kind (0 stale, 1 outside the recent window, 2 neither) above
// its order among its kind above its index; the least rank is replaced.
// All latency: 8 slots of a thread are read at once, the new row beside them
// (128 x 8 heads of 4096 slots 9.4 us, 3.6 TB/s; 14.5 with 4 to 16 slots one
// batch behind another and the row behind the search).
__global__ void __launch_bounds__(kInsertThreads) insert_kernel(const Cache c, const uint16_t *k_new,
                                                                const uint16_t *v_new, int64_t new_batch,
                                                                int64_t new_head, const int32_t *pos, int64_t recent,
                                                                int32_t *out_slots, int32_t *out_lengths)
{
    __shared__ uint64_t least[kInsertThreads / 64];
    const int bh = blockIdx.x, b = bh / c.kv_heads, head = bh % c.kv_heads;
    const int n = max(0, min(c.lengths[b], c.slots)), p = pos[b];
    if (threadIdx.x == 0 && head == 0) out_lengths[b] = p < 0 ? n : min(n + 1, c.slots);
    if (p < 0 || c.slots == 0) {
        if (threadIdx.x == 0) out_slots[bh] = -1;
        return;
    }
    const int64_t row = (int64_t)bh * c.slots;
    // the new row, on its way while its slot is looked for (dim / 8 threads, at most 32)
    const int64_t from = b * new_batch + head * new_head;
    const int d = 8 * threadIdx.x;
    u32x4 key{0, 0, 0, 0}, value{0, 0, 0, 0};
    if (d < c.dim) key = *(const u32x4 *)(k_new + from + d), value = *(const u32x4 *)(v_new + from + d);
    int slot = n;
    if (n == c.slots) {
        uint64_t best = ~0ull;
        for (int i0 = threadIdx.x; i0 < n; i0 += kInsertEach * kInsertThreads) {
            int32_t places[kInsertEach];
            float weights[kInsertEach];
#pragma unroll
            for (int j = 0; j < kInsertEach; j++) {
                const int64_t i = row + min(i0 + j * kInsertThreads, n - 1);
                places[j] = c.positions[i], weights[j] = c.weights[i];
            }
#pragma unroll
            for (int j = 0; j < kInsertEach; j++) {
                const int i = min(i0 + j * kInsertThreads, n - 1);   // the last slot again does not change the least
                const int32_t at = places[j];
                const uint64_t kind = at >= p || at < 0 ? 0 : (int64_t)at <= (int64_t)p - recent ? 1 : 2;
                const uint32_t order = kind == 0 ? 0 : kind == 1 ? order_of(weights[j]) : (uint32_t)at ^ 0x80000000u;
                best = min(best, kind << 62 | (uint64_t)order << 30 | (uint32_t)i);
            }
        }
        for (int d = 32; d; d >>= 1) best = min(best, (uint64_t)__shfl_xor((unsigned long long)best, d));
        if ((threadIdx.x & 63) == 0) least[threadIdx.x >> 6] = best;
        __syncthreads();
        for (int w = 0; w < kInsertThreads / 64; w++) best = min(best, least[w]);
        slot = (int)(best & 0x3fffffff);
    }
    const int64_t to = b * c.stride_batch + head * c.stride_head + slot * c.stride_slot;
    if (d < c.dim) *(u32x4 *)(c.k + to + d) = key, *(u32x4 *)(c.v + to + d) = value;
    if (threadIdx.x == 0) {
        c.weights[row + slot] = 0.0f;
        c.positions[row + slot] = p;
        out_slots[bh] = slot;
    }
}

constexpr int kSelectThreads = 1024;
constexpr int kSelectWaves = kSelectThreads / 64;

// What a slot is worth keeping: 0 not at all (stale, or without a token),
// then its weight's order, the recent window above all.
__device__ __forceinline__ uint32_t worth(int32_t at, float w, int32_t pos, int64_t recent)
{
    const uint32_t late = (int64_t)at >= (int64_t)pos - recent ? 0xffffffffu : 0;
    return at >= pos || at < 0 ? 0 : max(late, max(1u, order_of(w)));
}

constexpr int kBins = 4096;

// From the greatest bin down: the one in which `left` is reached, and what is
// in those above it (every thread gets both; there is one).
__device__ __forceinline__ void pick(const uint32_t *bins, int each, uint32_t left, uint32_t *part, uint32_t *picked,
                                     uint32_t &bin, uint32_t &above)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, top = each * kSelectThreads - 1 - each * (int)threadIdx.x;
    uint32_t sum = 0;
    for (int i = 0; i < each; i++) sum += bins[top - i];
    uint32_t s = sum;
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_up(s, d);
        if (lane >= d) s += y;
    }
    if (lane == 63) part[wave] = s;
    __syncthreads();
    s -= sum;
    for (int w = 0; w < kSelectWaves; w++) s += w < wave ? part[w] : 0;
    if (s < left && left <= s + sum) {
        int i = 0;
        while (s + bins[top - i] < left) s += bins[top - i++];
        picked[0] = top - i, picked[1] = s;
    }
    __syncthreads();
    bin = picked[0], above = picked[1];
}

// One workgroup for each sequence and key head.  A wave holds the worths of
// 64 * N slots in a row, N to a lane, in registers.  The worth of the last
// slot that stays is found from its 12 top bits down to its 10 lowest by
// counting the slots that share the bits found so far in bins (the recent
// window and slots worth nothing, each of one worth, are not counted there);
// then each wave writes its kept slots' indexes behind those of the waves
// before it.  What the slots hold is moved by move_kernel: here that would
// wait for memory once for each of a lane's N.  A cache of more than 1024 N
// slots is taken in rounds, whose worths are computed again for each pass.
// 3001 slots 10.8 us (2 to read them), 128 heads of 32768 slots 34 us (9 to
// read, 7 to write the indexes): latency of the passes' barriers and of the
// bins' LDS atomics.
template <int N>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const Cache c, const int32_t *pos, int32_t budget,
                                                                int64_t recent, int32_t out_slots, int32_t *kept,
                                                                int32_t *out_lengths)
{
    constexpr int kRound = kSelectThreads * N;
    __shared__ uint32_t bins[kBins], part[kSelectWaves], picked[2], total[2];
    __shared__ uint32_t waves[2][kSelectWaves][2];
    const int bh = blockIdx.x, b = bh / c.kv_heads, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = max(0, min(c.lengths[b], c.slots)), p = pos[b];
    const int64_t row = (int64_t)bh * c.slots, out_row = (int64_t)bh * out_slots;
    const int rounds = (n + kRound - 1) / kRound;
    if (threadIdx.x == 0 && bh % c.kv_heads == 0) out_lengths[b] = min(n, budget);

    uint32_t w[N];
    const auto load = [&](int round) {
        const int first = round * kRound + wave * 64 * N + lane;
        int32_t at[N];
        float x[N];
#pragma unroll
        for (int j = 0; j < N; j++) {
            const int i = min(first + 64 * j, n - 1);
            at[j] = c.positions[row + i], x[j] = c.weights[row + i];
        }
#pragma unroll
        for (int j = 0; j < N; j++) w[j] = first + 64 * j < n ? worth(at[j], x[j], p, recent) : 0;
    };
    if (rounds == 1) load(0);

    uint32_t limit = 0, above = 0, left = budget;   // slots worth more than `limit`, and what is left to take of the others
    bool sought = true;
    for (int pass = 0; pass < 3 && sought; pass++) {
        const int low = pass == 0 ? 20 : pass == 1 ? 10 : 0, high = pass == 0 ? 32 : low + 10;
        for (int i = threadIdx.x; i < 1 << (high - low); i += kSelectThreads) bins[i] = 0;
        if (pass == 0 && threadIdx.x < 2) total[threadIdx.x] = 0;
        __syncthreads();
        uint32_t late = 0, others = 0;
        for (int round = 0; round < rounds; round++) {
            if (rounds > 1) load(round);
#pragma unroll
            for (int j = 0; j < N; j++) {
                const bool counts = w[j] - 1u < 0xfffffffeu;
                if (pass == 0) {
                    late += __popcll(__ballot(w[j] == 0xffffffffu));
                    others += __popcll(__ballot(counts));
                }
                if (counts && (pass == 0 || w[j] >> high == limit >> high)) atomicAdd(&bins[w[j] >> low & ((1u << (high - low)) - 1)], 1u);
            }
        }
        if (pass == 0 && lane == 0) atomicAdd(&total[0], late), atomicAdd(&total[1], others);
        __syncthreads();
        if (pass == 0) {
            late = total[0], others = total[1];
            if (late >= left) limit = 0xffffffffu, sought = false;       // the window alone
            else if (others <= left - late) above = late + others, left = 0, sought = false;   // all that is worth anything
            else above = late, left -= late;
            if (!sought) break;
        }
        uint32_t bin, over;
        pick(bins, pass == 0 ? kBins / kSelectThreads : 1, left, part, picked, bin, over);
        limit |= bin << low, above += over, left -= over;
        __syncthreads();
    }
    // of the slots worth just `limit` the first `want` stay, but none that is worth nothing
    const uint32_t want = limit ? budget - above : 0;
    const uint64_t before = (1ull << lane) - 1;
    uint32_t more = 0, equal = 0;   // slots worth more and just `limit` in the rounds so far
    for (int round = 0; round < rounds; round++) {
        if (rounds > 1) load(round);
        uint32_t mine[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < N; j++) {
            mine[0] += __popcll(__ballot(w[j] > limit));
            mine[1] += __popcll(__ballot(w[j] == limit));
        }
        if (lane < 2) waves[round & 1][wave][lane] = mine[lane];
        __syncthreads();
        uint32_t m = more, e = equal;
#pragma unroll
        for (int v = 0; v < kSelectWaves; v++) {
            const uint32_t vm = waves[round & 1][v][0], ve = waves[round & 1][v][1];
            m += v < wave ? vm : 0, e += v < wave ? ve : 0;
            more += vm, equal += ve;
        }
#pragma unroll
        for (int j = 0; j < N; j++) {
            const uint64_t over = __ballot(w[j] > limit), same = __ballot(w[j] == limit);
            const uint32_t rank = e + __popcll(same & before);
            if (w[j] > limit || (w[j] == limit && rank < want)) {
                const int i = round * kRound + (wave * N + j) * 64 + lane;
                kept[out_row + m + __popcll(over & before) + min(rank, want)] = i;
            }
            m += __popcll(over), e += __popcll(same);
        }
    }
    const int done = more + min(equal, want);
    for (int i = done + threadIdx.x; i < out_slots; i += kSelectThreads) kept[out_row + i] = -1;
}

// A quarter of a wave moves (or clears) one slot.  Bound by HBM: 16 x 8 x
// 4096 slots of 128 dims, 543 MB in 105 us, the rate of a device copy.
__global__ void __launch_bounds__(256) move_kernel(const Cache c, const Cache out, const int32_t *kept)
{
    const int bh = blockIdx.y, b = bh / c.kv_heads, head = bh % c.kv_heads;
    const int i = blockIdx.x * 16 + threadIdx.x / 16;
    if (i >= out.slots) return;
    const int64_t to = (int64_t)bh * out.slots + i;
    const int from = kept[to];
    const int64_t src = b * c.stride_batch + head * c.stride_head + (int64_t)max(from, 0) * c.stride_slot;
    const int64_t dst = b * out.stride_batch + head * out.stride_head + (int64_t)i * out.stride_slot;
    if ((threadIdx.x & 15) == 0) {
        const int64_t at = (int64_t)bh * c.slots + max(from, 0);
        out.weights[to] = from < 0 ? 0.0f : c.weights[at];
        out.positions[to] = from < 0 ? DF11_NO_TOKEN : c.positions[at];
    }
    for (int d = 8 * (threadIdx.x & 15); d < c.dim; d += 128) {
        const u32x4 zero{0, 0, 0, 0};
        const u32x4 k = from < 0 ? zero : *(const u32x4 *)(c.k + src + d);
        const u32x4 v = from < 0 ? zero : *(const u32x4 *)(c.v + src + d);
        *(u32x4 *)(out.k + dst + d) = k;
        *(u32x4 *)(out.v + dst + d) = v;
    }
}

int make_cache(const char *who, const df11_cache *c, bool lengths, Cache &a)
{
    if (!c) return df11::fail(DF11_E_ARG, "%s: null cache", who);
    if (c->dtype != DF11_BF16 && c->dtype != DF11_FP16)
        return df11::fail(DF11_E_ARG, "%s: dtype must be bf16 or fp16", who);
    if (c->dim < 8 || c->dim > DF11_MAX_DIM || c->dim % 8)
        return df11::fail(DF11_E_ARG, "%s: dim %lld is not a multiple of 8 up to %d", who, (long long)c->dim, DF11_MAX_DIM);
    if (c->batch < 0 || c->kv_heads < 1 || (double)c->batch * c->kv_heads > 65535 || c->slots < 0 ||
        c->slots > (1ll << 30))
        return df11::fail(DF11_E_ARG, "%s: batch, kv_heads or slots out of range", who);
    if (c->stride_batch < 0 || c->stride_head < 0 || c->stride_slot < 0 ||
        (c->stride_batch | c->stride_head | c->stride_slot) % 8)
        return df11::fail(DF11_E_ARG, "%s: cache strides must be multiples of 8", who);
    if (c->batch && ((lengths && !c->lengths) ||
                     (c->slots && (!aligned16(c->k) || !aligned16(c->v) || !c->weights || !c->positions))))
        return df11::fail(DF11_E_ARG, "%s: null or misaligned cache pointer", who);
    a = Cache{(uint16_t *)c->k, (uint16_t *)c->v, c->weights, c->positions, c->lengths, (int32_t)c->batch,
              (int32_t)c->kv_heads, (int32_t)c->slots, (int32_t)c->dim, c->stride_batch, c->stride_head, c->stride_slot};
    return DF11_OK;
}

// Whether no two slots' rows share memory, as those of a cache that is
// written must not (workgroups of different heads would race): each axis has
// to step over all that the axes of smaller strides span.
bool rows_apart(const df11_cache *c)
{
    struct Axis {
        int64_t stride, size;
    } axes[3] = {{c->stride_batch, c->batch}, {c->stride_head, c->kv_heads}, {c->stride_slot, c->slots}};
    std::sort(axes, axes + 3, [](const Axis &x, const Axis &y) { return x.stride < y.stride; });
    __int128 span = c->dim;
    for (const Axis &axis : axes) {
        if (axis.size <= 1) continue;
        if (axis.stride < span) return false;
        span += (__int128)axis.stride * (axis.size - 1);
    }
    return true;
}

bool meet(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes)
{
    return (uintptr_t)a < (uintptr_t)b + b_bytes && (uintptr_t)b < (uintptr_t)a + a_bytes;
}

// Whether the new cache lies on the one it is cut out of: in weights or
// positions, or in keys or values without gaps.  (Two caches may take turns
// in one allocation: rows with gaps are the caller's to keep apart.)
bool caches_meet(const df11_cache *c, const df11_cache *out)
{
    const auto slots = [](const df11_cache *x) { return x->batch * x->kv_heads * x->slots; };
    if (!slots(c) || !slots(out)) return false;
    if (meet(c->weights, 4 * slots(c), out->weights, 4 * slots(out)) ||
        meet(c->positions, 4 * slots(c), out->positions, 4 * slots(out)))
        return true;
    const auto dense = [&](const df11_cache *x) {
        return (x->batch - 1) * x->stride_batch + (x->kv_heads - 1) * x->stride_head + (x->slots - 1) * x->stride_slot +
                   x->dim == slots(x) * x->dim;
    };
    const int64_t bytes = 2 * slots(c) * c->dim, out_bytes = 2 * slots(out) * out->dim;
    return dense(c) && dense(out) &&
           (meet(c->k, bytes, out->k, out_bytes) || meet(c->k, bytes, out->v, out_bytes) ||
            meet(c->v, bytes, out->k, out_bytes) || meet(c->v, bytes, out->v, out_bytes));
}

int launched(const char *who)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return df11::fail(DF11_E_DEVICE, "%s launch: %s", who, hipGetErrorString(e));
    return DF11_OK;
}

}  // namespace

extern "C" int df11_cache_insert(const df11_cache *cache, const void *k_new, const void *v_new, int64_t new_batch,
                                 int64_t new_head, const int32_t *pos, int64_t recent, int32_t *out_slots,
                                 int32_t *out_lengths, void *stream)
{
    const char *who = "df11_cache_insert";
    Cache c;
    const int rc = make_cache(who, cache, true, c);
    if (rc) return rc;
    if (!c.batch) return DF11_OK;
    if (!aligned16(k_new) || !aligned16(v_new) || !pos || !out_slots || !out_lengths || out_lengths == c.lengths)
        return df11::fail(DF11_E_ARG, "%s: null, misaligned or shared pointer", who);
    if (new_batch < 0 || new_head < 0 || (new_batch | new_head) % 8)
        return df11::fail(DF11_E_ARG, "%s: strides must be multiples of 8", who);
    if (recent < 0) return df11::fail(DF11_E_ARG, "%s: recent is negative", who);
    if (!rows_apart(cache)) return df11::fail(DF11_E_ARG, "%s: slots of the cache share memory", who);
    hipLaunchKernelGGL(insert_kernel, dim3(c.batch * c.kv_heads), dim3(kInsertThreads), 0, (hipStream_t)stream, c,
                       (const uint16_t *)k_new, (const uint16_t *)v_new, new_batch, new_head, pos,
                       std::min<int64_t>(recent, 1ll << 32), out_slots, out_lengths);
    return launched(who);
}

extern "C" int df11_cache_compact(const df11_cache *cache, const int32_t *pos, int64_t budget, int64_t recent,
                                  const df11_cache *out_cache, int32_t *kept, int32_t *out_lengths, void *stream)
{
    const char *who = "df11_cache_compact";
    Cache c, out;
    int rc = make_cache(who, cache, true, c);
    if (rc) return rc;
    rc = make_cache(who, out_cache, false, out);
    if (rc) return rc;
    if (out.batch != c.batch || out.kv_heads != c.kv_heads || out.dim != c.dim || out_cache->dtype != cache->dtype)
        return df11::fail(DF11_E_ARG, "%s: the caches differ in batch, heads, dim or type", who);
    if (budget < 1 || recent < 0 || recent > budget || budget > out.slots)
        return df11::fail(DF11_E_ARG, "%s: needs 0 <= recent <= budget <= out slots and a budget of 1", who);
    if (!c.batch) return DF11_OK;
    if (!pos || !kept || !out_lengths || out_lengths == c.lengths)
        return df11::fail(DF11_E_ARG, "%s: null or shared pointer", who);
    if (!rows_apart(out_cache)) return df11::fail(DF11_E_ARG, "%s: slots of the new cache share memory", who);
    if (c.slots && (out.k == c.k || out.v == c.v || caches_meet(cache, out_cache)))
        return df11::fail(DF11_E_ARG, "%s: a cache is not cut down in place", who);
    hipStream_t st = (hipStream_t)stream;
    const auto select = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(c.batch * c.kv_heads), dim3(kSelectThreads), 0, st, c, pos, (int32_t)budget, recent,
                           out.slots, kept, out_lengths);
    };
    // as few slots of a lane as hold the cache in one round (3001 slots 10.8 us
    // with 4, 12 with 8; 14054 slots 16.8 us with 16, 23 with 32)
    if (c.slots <= 4 * kSelectThreads) select(select_kernel<4>);
    else if (c.slots <= 8 * kSelectThreads) select(select_kernel<8>);
    else if (c.slots <= 16 * kSelectThreads) select(select_kernel<16>);
    else select(select_kernel<32>);
    hipLaunchKernelGGL(move_kernel, dim3((out.slots + 15) / 16, c.batch * c.kv_heads), dim3(256), 0, st, c, out, kept);
    return launched(who);
}
