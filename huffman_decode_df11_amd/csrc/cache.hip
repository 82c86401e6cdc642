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

constexpr int kInsertThreads = 256;

// One workgroup for each sequence and key head.  A slot's rank is one 64-bit
// number, its kind (0 stale, 1 outside the recent window, 2 neither) above
// its order among its kind above its index; the least rank is replaced.
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
    int slot = n;
    if (n == c.slots) {
        uint64_t best = ~0ull;
        for (int i = threadIdx.x; i < n; i += kInsertThreads) {
            const int32_t at = c.positions[row + i];
            const uint64_t kind = at >= p || at < 0 ? 0 : (int64_t)at <= (int64_t)p - recent ? 1 : 2;
            const uint32_t value = kind == 0 ? 0 : kind == 1 ? order_of(c.weights[row + i]) : (uint32_t)at ^ 0x80000000u;
            best = min(best, kind << 62 | (uint64_t)value << 30 | (uint32_t)i);
        }
        for (int d = 32; d; d >>= 1) best = min(best, (uint64_t)__shfl_xor((unsigned long long)best, d));
        if ((threadIdx.x & 63) == 0) least[threadIdx.x >> 6] = best;
        __syncthreads();
        for (int w = 0; w < kInsertThreads / 64; w++) best = min(best, least[w]);
        slot = (int)(best & 0x3fffffff);
    }
    const int64_t to = b * c.stride_batch + head * c.stride_head + slot * c.stride_slot;
    const int64_t from = b * new_batch + head * new_head;
    for (int d = 8 * threadIdx.x; d < c.dim; d += 8 * kInsertThreads) {
        *(u32x4 *)(c.k + to + d) = *(const u32x4 *)(k_new + from + d);
        *(u32x4 *)(c.v + to + d) = *(const u32x4 *)(v_new + from + d);
    }
    if (threadIdx.x == 0) {
        c.weights[row + slot] = 0.0f;
        c.positions[row + slot] = p;
        out_slots[bh] = slot;
    }
}

constexpr int kSelectThreads = 1024;

// What a slot is worth keeping: 0 not at all (stale, or without a token), then its
// weight's order, the recent window above all.
__device__ __forceinline__ uint32_t worth(const Cache &c, int64_t row, int i, int32_t pos, int64_t recent)
{
    const int32_t at = c.positions[row + i];
    if (at >= pos || at < 0) return 0;
    if ((int64_t)at >= (int64_t)pos - recent) return 0xffffffffu;
    return max(1u, order_of(c.weights[row + i]));
}

// Sum over a workgroup of the counts before this thread's, and of all.
__device__ __forceinline__ void scan2(uint32_t x, uint32_t *part, uint32_t &before, uint32_t &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t s = x;
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_up(s, d);
        if (lane >= d) s += y;
    }
    __syncthreads();
    if (lane == 63) part[wave] = s;
    __syncthreads();
    before = s - x;
    total = 0;
    for (int w = 0; w < kSelectThreads / 64; w++) {
        if (w < wave) before += part[w];
        total += part[w];
    }
}

// One workgroup for each sequence and key head: the worth of the last slot
// that stays, by four passes over its bytes, then the kept slots in order.
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const Cache c, const int32_t *pos, int32_t budget,
                                                                int64_t recent, const Cache out, int32_t *kept,
                                                                int32_t *out_lengths)
{
    __shared__ uint32_t hist[256];
    __shared__ uint32_t part[kSelectThreads / 64];
    __shared__ uint32_t chosen[2];
    const int bh = blockIdx.x, b = bh / c.kv_heads;
    const int n = max(0, min(c.lengths[b], c.slots)), p = pos[b];
    const int64_t row = (int64_t)bh * c.slots, out_row = (int64_t)bh * out.slots;
    if (threadIdx.x == 0 && bh % c.kv_heads == 0) out_lengths[b] = min(n, budget);

    // the least worth that stays, and how many of just that worth stay
    uint32_t limit = 0, want = budget;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256) hist[threadIdx.x] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kSelectThreads) {
            const uint32_t w = worth(c, row, i, p, recent);
            if (shift == 24 || w >> (shift + 8) == limit >> (shift + 8)) atomicAdd(&hist[w >> shift & 255], 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            // from the top: the byte at which `want` slots are reached (0, if they are not)
            uint32_t left = want, byte = 255;
            while (byte && hist[byte] < left) left -= hist[byte--];
            chosen[0] = limit | byte << shift;
            chosen[1] = left;
        }
        __syncthreads();
        limit = chosen[0], want = chosen[1];
    }
    // slots worth nothing never stay
    if (limit == 0) limit = 1, want = n;
    uint32_t done = 0, equal = 0;
    for (int i0 = 0; i0 < n; i0 += kSelectThreads) {
        const int i = i0 + threadIdx.x;
        const uint32_t w = i < n ? worth(c, row, i, p, recent) : 0;
        uint32_t before, total;
        scan2(w == limit, part, before, total);
        const bool stays = w > limit || (w == limit && equal + before < want);
        equal += total;
        scan2(stays, part, before, total);
        if (stays) {
            const int64_t to = out_row + done + before;
            kept[to] = i;
            out.weights[to] = c.weights[row + i];
            out.positions[to] = c.positions[row + i];
        }
        done += total;
    }
    for (int i = done + threadIdx.x; i < out.slots; i += kSelectThreads) {
        kept[out_row + i] = -1;
        out.weights[out_row + i] = 0.0f;
        out.positions[out_row + i] = DF11_NO_TOKEN;
    }
}

// A quarter of a wave copies (or clears) one slot's key and value.
__global__ void __launch_bounds__(256) move_kernel(const Cache c, const Cache out, const int32_t *kept)
{
    const int bh = blockIdx.y, b = bh / c.kv_heads, head = bh % c.kv_heads;
    const int i = blockIdx.x * 16 + threadIdx.x / 16;
    if (i >= out.slots) return;
    const int from = kept[(int64_t)bh * out.slots + i];
    const int64_t src = b * c.stride_batch + head * c.stride_head + (int64_t)max(from, 0) * c.stride_slot;
    const int64_t dst = b * out.stride_batch + head * out.stride_head + (int64_t)i * out.stride_slot;
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
    if (c.slots && (out.k == c.k || out.v == c.v || out.weights == c.weights || out.positions == c.positions))
        return df11::fail(DF11_E_ARG, "%s: a cache is not cut down in place", who);
    hipStream_t st = (hipStream_t)stream;
    hipLaunchKernelGGL(select_kernel, dim3(c.batch * c.kv_heads), dim3(kSelectThreads), 0, st, c, pos, (int32_t)budget,
                       recent, out, kept, out_lengths);
    hipLaunchKernelGGL(move_kernel, dim3((out.slots + 15) / 16, c.batch * c.kv_heads), dim3(256), 0, st, c, out, kept);
    return launched(who);
}
