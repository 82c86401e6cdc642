// A cache held in 4 bits: keys and values quantised as they are written into
// pages (df11_quantized_write), read back (df11_quantized_read), and attention
// over them (df11_quantized_attention).
//
// A row x of D values (a token's key or value of one head) lies in G groups,
// dim d in group d mod G (G = 2 up to 64 dims, else 4).  With a group's least
// and greatest value: step = (greatest - least) / 15 in the row's own 16-bit
// type, code = floor((x - least) / step + 1/2) in 0 .. 15, and what the code
// stands for is code * step + least.  Groups of every G-th dim rather than of
// neighbours: the eight codes of a 32-bit word then hold whole groups' shares
// in the same places, and both the matrix products below find one group's
// codes of several words side by side without moving any between lanes.
#include <algorithm>
#include <cmath>
#include <type_traits>
#include <utility>

#include "df11_internal.h"
#include "overlap.h"
#include "serve_device.h"

namespace {

using namespace df11serve;

struct Cache {
    uint8_t *k_codes, *v_codes;
    uint32_t *k_scales, *v_scales;   // pairs of (step, least)
    int32_t pages, page, kv_heads, dim, groups;
    int64_t code_page, code_head;    // bytes
    int64_t scale_page, scale_head;  // pairs
    double per_page;                 // 1 / (page / 16)
    const int32_t *table;
    int64_t table_batch;
    int32_t table_pages;
};

// The page of a sequence that holds the 16 positions from 16 u on, as its
// place in the table: floor(u / (page / 16)); (u + 1/2) * per_page is half a
// 1 / (page / 16) away from any whole number, which no rounding of doubles spans.
__device__ __forceinline__ int page_of(const Cache &c, int u) { return (int)(((double)u + 0.5) * c.per_page); }

// The page id in that place, or -1.
__device__ __forceinline__ int page_id(const Cache &c, int b, int at)
{
    if (at >= c.table_pages) return -1;
    const int id = c.table ? c.table[b * c.table_batch + at] : b;
    return id >= 0 && id < c.pages ? id : -1;
}

template <class F, int... I>
__device__ __forceinline__ void each(F &&f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unroll(F &&f)
{
    each(f, std::make_integer_sequence<int, N>{});
}

// ------------------------------------------------------------ write and read

// Sixteen dims of a row to a lane, so a row of DP dims has DP / 16 lanes: 16
// bytes twice from the row, 8 bytes of codes.
template <int DP>
struct RowLanes {
    static constexpr int kLanes = DP / 16;
    static constexpr int G = DP == 64 ? 2 : 4;
};
constexpr int kMoveThreads = 256;

struct WriteArgs {
    Cache c;
    const uint16_t *k, *v;
    const int32_t *positions, *counts;
    int32_t *lengths;
    int32_t batch, tokens, run;
    int64_t k_batch, k_token, k_head, v_batch, v_token, v_head;
};

// Two 16-bit floats as whole numbers of the same order (and back): a NaN is
// beyond the infinity of its sign.
typedef short i16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ i16x2 ordered(uint32_t x)
{
    const i16x2 y = __builtin_bit_cast(i16x2, x);
    return y ^ (__builtin_bit_cast(i16x2, 0x7fff7fffu) & (y >> 15));
}

// The least or greatest pairs over the L lanes of a row.
template <int L, class F>
__device__ __forceinline__ i16x2 over_lanes(i16x2 x, F &&join)
{
    const auto step = [&](auto control) {
        const int y = __builtin_bit_cast(int, x);
        x = join(x, __builtin_bit_cast(i16x2, __builtin_amdgcn_update_dpp(0, y, decltype(control)::value, 0xf, 0xf, true)));
    };
    step(std::integral_constant<int, 0xb1>{});                          // neighbours
    step(std::integral_constant<int, 0x4e>{});                          // pairs of four
    if constexpr (L >= 8) step(std::integral_constant<int, 0x141>{});   // the mirrored lane of eight
    if constexpr (L >= 16) step(std::integral_constant<int, 0x140>{});  // the mirrored lane of sixteen
    return x;
}

// raw: the lane's 16 dims.  Gives its codes and its row's pairs.
//
// A code is floor((x - least) / step + 1/2): the quotient by the inverse, with
// 2^-18 more than 1/2 (x - least and the inverse err by 2^-23 of at most 16),
// has the code or one more as its floor, and (code - 1/2) * step, 13 bits, says
// which.  64 bits are taken where the difference d = x - least is not exact, which
// is seldom, or the step so small that its inverse may not be a number.  Of a least
// value as great in size as x or greater d is exact if d + least is x again.  Of a smaller
// one it is if that is 0, or not below 2^-8 of the step: both are multiples of
// 2^(e - 10), 2^e its power of two, and d is at most 22.5 steps (a subnormal step's
// rounding; else 15.1), so below 2^(e + 14): 24 bits.  (One that is
// smaller still vanishes in d and in d + least alike, and a value on a border
// would have the code above the formula's: all of such a row is taken in 64 bits.)
template <class E, int DP>
__device__ __forceinline__ void quantise(const u32x4 (&raw)[2], u32x2 &codes, uint32_t (&pairs)[RowLanes<DP>::G])
{
    constexpr int G = RowLanes<DP>::G, L = RowLanes<DP>::kLanes;
    i16x2 lo[G / 2], hi[G / 2];   // dims 2 j and 2 j + 1 are of the groups 2 j and 2 j + 1 mod G
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const i16x2 y = ordered(raw[j / 4][j % 4]);
        lo[j % (G / 2)] = j < G / 2 ? y : __builtin_elementwise_min(lo[j % (G / 2)], y);
        hi[j % (G / 2)] = j < G / 2 ? y : __builtin_elementwise_max(hi[j % (G / 2)], y);
    }
#pragma unroll
    for (int g = 0; g < G / 2; g++) {
        lo[g] = over_lanes<L>(lo[g], [](i16x2 u, i16x2 v) { return __builtin_elementwise_min(u, v); });
        hi[g] = over_lanes<L>(hi[g], [](i16x2 u, i16x2 v) { return __builtin_elementwise_max(u, v); });
    }
    // each lane one group's step, in 64 bits, rounded to float32 and to the type
    const int lane = threadIdx.x & (L - 1), mine = lane % G;
    int least = lo[0][0], most = hi[0][0];
#pragma unroll
    for (int g = 1; g < G; g++) least = mine == g ? lo[g / 2][g % 2] : least, most = mine == g ? hi[g / 2][g % 2] : most;
    const bool number = most < (int)E::kExpMask && least > ~(int)E::kExpMask;   // neither infinities nor beyond
    const float from = E::value((uint32_t)(least ^ (least >> 31 & 0x7fff)) & 0xffffu);
    const float to = E::value((uint32_t)(most ^ (most >> 31 & 0x7fff)) & 0xffffu);
    const float wide = number ? (float)(((double)to - (double)from) / 15.0) : NAN;
    const uint32_t pair = E::pack(wide, number ? from : NAN);
    float step[G], half[G], inverse[G], low[G];
    bool exact = true;
    unroll<G>([&](auto k) {
        constexpr int g = decltype(k)::value;
        // from the lane g of four: of two groups the lanes 0 and 2, 1 and 3 hold the same
        pairs[g] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)pair, g * 0x55, 0xf, 0xf, true);
        step[g] = E::value(pairs[g] & 0xffffu);
        low[g] = E::value(pairs[g] >> 16);
        half[g] = -0.5f * step[g];
        inverse[g] = step[g] > 0.0f ? __builtin_amdgcn_rcpf(step[g]) : 0.0f;   // errs by 2^-23
        exact = exact && !(step[g] < 0x1p-100f) && !(__builtin_fabsf(low[g]) < 0x1p-8f * step[g] && low[g] != 0.0f);
    });
    float c[16];
    bool differs[16];
    const auto value = [&](int i) { return E::value(raw[i / 8][i % 8 / 2] >> (i & 1 ? 16 : 0) & 0xffffu); };
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const float x = value(i), d = x - low[i % G];
        differs[i] = d + low[i % G] != x;
        c[i] = __builtin_floorf(__builtin_fmaf(d, inverse[i % G], 0.5f + 0x1p-18f));
        c[i] -= d < __builtin_fmaf(c[i], step[i % G], half[i % G]) ? 1.0f : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 16; i++)
        if (differs[i] || !exact)
            c[i] = step[i % G] > 0.0f
                       ? (float)__builtin_floor(((double)value(i) - (double)low[i % G]) / (double)step[i % G] + 0.5)
                       : 0.0f;
#pragma unroll
    for (int w = 0; w < 2; w++) {
        uint32_t even = 0, odd = 0;   // the codes, a byte each
#pragma unroll
        for (int i = 0; i < 4; i++) {
            even = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_amdgcn_fmed3f(c[8 * w + 2 * i], 0.0f, 15.0f), i, even);   // NaN: 0
            odd = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_amdgcn_fmed3f(c[8 * w + 2 * i + 1], 0.0f, 15.0f), i, odd);
        }
        codes[w] = even | odd << 4;
    }
}

// A row's lanes, then 2^run tokens of one head, whose rows in a page are one
// piece of memory, then heads; keys and values of a token by the same lanes.
// Bound by issue once the rows are many (a code is some eight vector
// instructions): 2 prompts of up to 8191 tokens, 8 heads of 128, 74 MB in 26 us,
// 2.8 TB/s (with the least and greatest values taken in float32 41 us).  48
// single tokens: 5.5 us, latency.
template <class E, int DP>
__global__ void __launch_bounds__(kMoveThreads) write_kernel(const WriteArgs a)
{
    constexpr int L = RowLanes<DP>::kLanes, G = RowLanes<DP>::G;
    const int b = blockIdx.y;
    const int count = a.counts ? max(0, min(a.counts[b], a.tokens)) : a.tokens;
    const int first = a.positions[b];
    if (blockIdx.x == 0 && threadIdx.x == 0) a.lengths[b] = (int)min((int64_t)first + count, (int64_t)0x7fffffff);
    const uint32_t item = (uint32_t)blockIdx.x * (kMoveThreads / L) + threadIdx.x / L;
    const int lane = threadIdx.x % L;
    const uint32_t run = item >> a.run, head = run % a.c.kv_heads;
    const uint32_t t = (run / a.c.kv_heads << a.run) + (item & ((1u << a.run) - 1));
    const int64_t at = (int64_t)first + t;
    const bool there = (int64_t)t < count && at >= 0 && at < (int64_t)a.c.table_pages * a.c.page;
    if (!there) return;   // a row's lanes stay or go together
    // dims past the last one: the row's last eight once more, which change neither least nor greatest values
    const int d0 = min(16 * lane, a.c.dim - 8), d1 = min(16 * lane + 8, a.c.dim - 8);
    u32x4 raw[2][2];
#pragma unroll
    for (int which = 0; which < 2; which++) {
        const uint16_t *from = which ? a.v + b * a.v_batch + t * a.v_token + head * a.v_head
                                     : a.k + b * a.k_batch + t * a.k_token + head * a.k_head;
        raw[which][0] = *(const u32x4 *)(from + d0), raw[which][1] = *(const u32x4 *)(from + d1);
    }
    const int p = page_of(a.c, (int)(at >> 4)), id = page_id(a.c, b, p);
    if (id < 0) return;
    const int row = (int)(at - (int64_t)p * a.c.page), have = a.c.dim - 16 * lane;
    const int64_t code = id * a.c.code_page + head * a.c.code_head + (int64_t)row * (a.c.dim / 2) + 8 * lane;
    const int64_t scale = id * a.c.scale_page + head * a.c.scale_head + (int64_t)row * G;
#pragma unroll
    for (int which = 0; which < 2; which++) {
        u32x2 codes;
        uint32_t pairs[G];
        quantise<E, DP>(raw[which], codes, pairs);
        uint8_t *to = (which ? a.c.v_codes : a.c.k_codes) + code;
        if (have > 8 && a.c.dim % 16 == 0) {
            *(u32x2 *)to = codes;
        } else {
            if (have > 0) *(uint32_t *)to = codes[0];
            if (have > 8) *(uint32_t *)(to + 4) = codes[1];
        }
        if (lane == 0) __builtin_memcpy(__builtin_assume_aligned((which ? a.c.v_scales : a.c.k_scales) + scale, 4 * G), pairs, 4 * G);
    }
}

struct ReadArgs {
    Cache c;
    uint16_t *k, *v;
    const int32_t *first, *lengths;
    int32_t batch, count;
};

// A word of eight codes to a lane, so that a wave's stores are one piece: the
// lanes of a row, then the heads.  Four positions to a thread, whose rows of
// one head lie behind each other in a page.  Bound by the stores: 16 times 8192
// positions of 8 heads of 128, 646 MB in 133 us, 4.8 TB/s (a row a thread 182 us;
// four, through the caches 141; stores that pass them, as here, 133).
constexpr int kReadRows = 4;
template <class E, int DP>
__global__ void __launch_bounds__(kMoveThreads) read_kernel(const ReadArgs a)
{
    constexpr int L = DP / 8, G = RowLanes<DP>::G;
    const int b = blockIdx.y, lane = threadIdx.x % L;
    const uint32_t item = (uint32_t)blockIdx.x * (kMoveThreads / L) + threadIdx.x / L;   // runs of positions by heads
    const int head = (int)(item % a.c.kv_heads);
    const int64_t t0 = (int64_t)(item / a.c.kv_heads) * kReadRows;
    if (t0 >= a.count || 8 * lane >= a.c.dim) return;
    const int64_t first = a.first ? a.first[b] : 0, length = a.lengths[b];
    const int64_t out = (((int64_t)b * a.count + t0) * a.c.kv_heads + head) * a.c.dim + 8 * lane;
    uint32_t w[2][kReadRows], pairs[2][kReadRows][G];
    bool there[kReadRows];
#pragma unroll
    for (int r = 0; r < kReadRows; r++) {
        const int64_t at = first + t0 + r;
        int id = -1, row = 0;
        if (at >= 0 && at < length && at < (int64_t)a.c.table_pages * a.c.page) {
            const int p = page_of(a.c, (int)(at >> 4));
            id = page_id(a.c, b, p);
            row = (int)(at - (int64_t)p * a.c.page);
        }
        there[r] = id >= 0;
        if (!there[r]) continue;
        const int64_t code = id * a.c.code_page + head * a.c.code_head + (int64_t)row * (a.c.dim / 2) + 4 * lane;
        const int64_t scale = id * a.c.scale_page + head * a.c.scale_head + (int64_t)row * G;
#pragma unroll
        for (int which = 0; which < 2; which++) {
            w[which][r] = *(const uint32_t *)((which ? a.c.v_codes : a.c.k_codes) + code);
            __builtin_memcpy(pairs[which][r], __builtin_assume_aligned((which ? a.c.v_scales : a.c.k_scales) + scale, 4 * G), 4 * G);
        }
    }
#pragma unroll
    for (int which = 0; which < 2; which++)
#pragma unroll
        for (int r = 0; r < kReadRows; r++) {
            if (t0 + r >= a.count) break;
            u32x4 y = {};
            if (there[r]) {
                const uint32_t low = w[which][r] & 0x0f0f0f0fu, high = w[which][r] >> 4 & 0x0f0f0f0fu;
                float step[G], least[G], x[8];
                float most = 0.0f;   // a code may stand for more than the type's greatest number, since the step is rounded
#pragma unroll
                for (int i = 0; i < G; i++) {
                    step[i] = E::value(pairs[which][r][i] & 0xffffu), least[i] = E::value(pairs[which][r][i] >> 16);
                    most = __builtin_fmaxf(most, __builtin_fabsf(__builtin_fmaf(15.0f, step[i], least[i])));
                }
#pragma unroll
                for (int i = 0; i < 8; i++)
                    x[i] = __builtin_fmaf((float)((i % 2 ? high : low) >> (8 * (i / 2)) & 255u), step[i % G], least[i % G]);
                if (most > E::kMost)
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        if (__builtin_fabsf(step[i % G]) <= E::kMost && __builtin_fabsf(least[i % G]) <= E::kMost)
                            x[i] = __builtin_amdgcn_fmed3f(x[i], -E::kMost, E::kMost);
#pragma unroll
                for (int i = 0; i < 4; i++) y[i] = E::pack(x[2 * i], x[2 * i + 1]);
            }
            __builtin_nontemporal_store(y, (u32x4 *)((which ? a.v : a.k) + out + (int64_t)r * a.c.kv_heads * a.c.dim));
        }
}

// ------------------------------------------------------------------ attention
//
// For a row q (one query token of one head) over keys j, groups g:
//   s_j = scale * (sum_g step_jg (q_g . c_jg) + sum_g least_jg sum(q_g))
//   o   = sum_j p_j V_j,  o_d = sum_j (p_j step_jg) c_jd + sum_j p_j least_jg
// so the matrix cores multiply the codes themselves, and steps and least
// values meet sums of a whole group: no value is ever made from its code.  A
// code becomes a 16-bit number by one mask-and-or: the bits of 128 + c (bf16)
// or 16 + c (fp16); what the 128 or 16 adds is taken off again through the
// terms of the least values.
//
// A wave has 16 rows and takes 32 keys at a time:
//   S^T: v_mfma_f32_16x16x32, A = codes of key l % 16, dims of group i from
//     the DP / 4 dims that lane l holds of it (place l / 16); the sums of
//     group i times the keys' steps, which the lanes of a row of 16 share, are
//     added up with the lane broadcast of the vector instructions.  One more
//     product takes the keys' (step, least) pairs as they lie in memory
//     against (-128 sum(q_i), sum(q_i)) in three 16-bit parts, one part for
//     each of three lane rows: 24 bits, so nothing is lost.
//   O^T: A = V's codes, product j taking dims W (l % 16) + j (W = DP / 16;
//     all in group j mod G), B = p step_g of 32 keys, rounded to the type.
// Probabilities times steps are the only rounding to 16 bits in between.
//
// Nothing goes through LDS but the joining of the four waves: a lane loads the
// words that it multiplies, for one step ahead, and the pages of 32 steps are
// looked up at once (219 us instead of 317 for 64 requests).  Bound by vector
// instructions, 400 a wave and step, half of them for the steps of K: 24 x 5
// drafts over 2222 to 8891 positions (two tiles of 16 for 20 rows, 173 MB)
// 79 us, the vector ALU busy for 74% of it, the matrix cores for 15%.
constexpr int kWaves = 4;
constexpr int kStep = 32;
constexpr int kMostParts = 64;
__host__ __device__ constexpr int tile_waves(int dim) { return dim <= 128 ? 8 : 4; }   // of 32 rows; at 256 dims a wave needs more than 256 registers
constexpr int kMany = 112;   // rows up to which tiles of 16 are the faster (1 request of 8192 keys, heads of 128:
                             // 96 rows 28 us and 34 us in tiles of 256, 128 rows 32 and 33, 256 rows 46 and 38)

struct Args {
    Cache c;
    const uint16_t *q;
    const int32_t *lengths;
    uint16_t *out;
    float *lse;
    float *part_o;     // [split][row][dim]: a range's own result, which no number of keys makes greater than its values
    float2 *part_ml;   // [split][row]: the power of two that its sum of probabilities is held below, and that sum
    int32_t batch, tokens, heads, group, tiles, splits, granule;
    int64_t q_batch, q_token, q_head, rows;
    float scale2;      // scale * log2(e)
    bool taper;        // kTaper ranges, each shorter than the one before
    bool few;          // at most four rows share a key head's keys
    bool many;         // tiles of 32 rows a wave
    bool wide;         // a workgroup joins a row, not a wave
};

// Where range i of a sequence's n keys begins, in whole granules: even ranges,
// or kTaper ones of 9, 7, .. 1 parts of 25, of which the short ones come last.
constexpr int kTaper = 5;
__device__ __forceinline__ int edge(const Args &a, int n, int i)
{
    const int granules = (n + a.granule - 1) / a.granule;
    const int64_t at = a.taper ? ((int64_t)granules * (kTaper * kTaper - (kTaper - i) * (kTaper - i)) + kTaper * kTaper - 1) / (kTaper * kTaper)
                               : (int64_t)((granules + a.splits - 1) / a.splits) * i;
    return (int)min((int64_t)n, at * a.granule);
}

template <class E> struct Code;
template <> struct Code<Bf16> {
    static constexpr float kOff = 128.0f;
    static constexpr uint32_t kOffBits = 0x43004300u, kMidBits = 0xc308c308u;   // 128, -136
    static constexpr uint32_t kMask = 0x000f000fu;
    // where the codes at bits 4 i of each half of w have to be
    static __device__ __forceinline__ uint32_t shifted(uint32_t w, int i) { return w >> (4 * i); }
};
template <> struct Code<Fp16> {
    static constexpr float kOff = 16.0f;
    static constexpr uint32_t kOffBits = 0x4c004c00u, kMidBits = 0xce00ce00u;   // 16, -24
    static constexpr uint32_t kMask = 0x03c003c0u;
    static __device__ __forceinline__ uint32_t shifted(uint32_t w, int i)
    {
        return i == 0 ? w << 6 : i == 1 ? w << 2 : i == 2 ? w >> 2 : w >> 6;
    }
};

// The value that lane N of each row of 16 lanes holds.
template <int N>
__device__ __forceinline__ float row_lane(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x150 + N, 0xf, 0xf, true));
}

// sum[r] += (what lane r G + i of the row of 16 lanes holds of w) * x[i][r],
// i < G, r < 4.  The multiply-add with a lane broadcast is one instruction,
// which the compiler makes two of.  x comes from the matrix cores: 16 wait
// states cover their latency (8 passes: 12), and w's for a lane broadcast (2).
#define DF11_FMAC(acc, from, w, x) "v_fmac_f32_dpp %" acc ", %" w ", %" x " row_newbcast:" from " row_mask:0xf bank_mask:0xf\n\t"
template <int G>
__device__ __forceinline__ void add_scaled(f32x4 &sum, float w, const f32x4 (&x)[G])
{
    float a = sum[0], b = sum[1], c = sum[2], d = sum[3];
    if constexpr (G == 4) {
        asm volatile("s_nop 15\n\t"
            DF11_FMAC("0", "0", "4", "5") DF11_FMAC("1", "4", "4", "6") DF11_FMAC("2", "8", "4", "7") DF11_FMAC("3", "12", "4", "8")
            DF11_FMAC("0", "1", "4", "9") DF11_FMAC("1", "5", "4", "10") DF11_FMAC("2", "9", "4", "11") DF11_FMAC("3", "13", "4", "12")
            DF11_FMAC("0", "2", "4", "13") DF11_FMAC("1", "6", "4", "14") DF11_FMAC("2", "10", "4", "15") DF11_FMAC("3", "14", "4", "16")
            DF11_FMAC("0", "3", "4", "17") DF11_FMAC("1", "7", "4", "18") DF11_FMAC("2", "11", "4", "19") DF11_FMAC("3", "15", "4", "20")
            : "+v"(a), "+v"(b), "+v"(c), "+v"(d)
            : "v"(w), "v"(x[0][0]), "v"(x[0][1]), "v"(x[0][2]), "v"(x[0][3]), "v"(x[1][0]), "v"(x[1][1]), "v"(x[1][2]),
              "v"(x[1][3]), "v"(x[2][0]), "v"(x[2][1]), "v"(x[2][2]), "v"(x[2][3]), "v"(x[3][0]), "v"(x[3][1]), "v"(x[3][2]),
              "v"(x[3][3]));
    } else {
        asm volatile("s_nop 15\n\t"
            DF11_FMAC("0", "0", "4", "5") DF11_FMAC("1", "2", "4", "6") DF11_FMAC("2", "4", "4", "7") DF11_FMAC("3", "6", "4", "8")
            DF11_FMAC("0", "1", "4", "9") DF11_FMAC("1", "3", "4", "10") DF11_FMAC("2", "5", "4", "11") DF11_FMAC("3", "7", "4", "12")
            : "+v"(a), "+v"(b), "+v"(c), "+v"(d)
            : "v"(w), "v"(x[0][0]), "v"(x[0][1]), "v"(x[0][2]), "v"(x[0][3]), "v"(x[1][0]), "v"(x[1][1]), "v"(x[1][2]),
              "v"(x[1][3]));
    }
    sum = f32x4{a, b, c, d};
}

// sum[i] += (what lane r G + i of the row holds of w) * p[r].  No matrix
// product is on its way to these registers: add_scaled has waited for all.
template <int G>
__device__ __forceinline__ void add_weighted(float (&sum)[G], float w, const float (&p)[4])
{
    if constexpr (G == 4) {
        asm volatile("s_nop 1\n\t"
            DF11_FMAC("0", "0", "4", "5") DF11_FMAC("1", "1", "4", "5") DF11_FMAC("2", "2", "4", "5") DF11_FMAC("3", "3", "4", "5")
            DF11_FMAC("0", "4", "4", "6") DF11_FMAC("1", "5", "4", "6") DF11_FMAC("2", "6", "4", "6") DF11_FMAC("3", "7", "4", "6")
            DF11_FMAC("0", "8", "4", "7") DF11_FMAC("1", "9", "4", "7") DF11_FMAC("2", "10", "4", "7") DF11_FMAC("3", "11", "4", "7")
            DF11_FMAC("0", "12", "4", "8") DF11_FMAC("1", "13", "4", "8") DF11_FMAC("2", "14", "4", "8") DF11_FMAC("3", "15", "4", "8")
            : "+v"(sum[0]), "+v"(sum[1]), "+v"(sum[2]), "+v"(sum[3])
            : "v"(w), "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]));
    } else {
        asm volatile("s_nop 1\n\t"
            DF11_FMAC("0", "0", "2", "3") DF11_FMAC("1", "1", "2", "3") DF11_FMAC("0", "2", "2", "4") DF11_FMAC("1", "3", "2", "4")
            DF11_FMAC("0", "4", "2", "5") DF11_FMAC("1", "5", "2", "5") DF11_FMAC("0", "6", "2", "6") DF11_FMAC("1", "7", "2", "6")
            : "+v"(sum[0]), "+v"(sum[1])
            : "v"(w), "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]));
    }
}
#undef DF11_FMAC

// The greatest of a column's four lanes, one in each row of 16.
__device__ __forceinline__ float over_rows(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    x = fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
    const uint32_t v = __builtin_bit_cast(uint32_t, x);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}

// Where the two halves (16 keys each) of a step lie.
struct Halves {
    int64_t code[2], scale[2];   // bytes; pairs
    uint32_t any;                // keys that some row sees
};

template <class E, int DP>
struct Wave {
    static constexpr int W = DP / 16, G = DP == 64 ? 2 : 4, KW = DP / 32, S = DP / 32;
    f32x4 o[W];
    float least[G];   // sums of p times what code 8 stands for, over this lane's keys
    float m, l;
    // In float16 V's steps go into the products times a power of two that leaves
    // the greatest so far (its bits at most `most`) below 1: as they are, 2^15
    // times a step of 2 would pass its range.  o holds sums of those.  bfloat16
    // has float32's range and does without (24 x 5 drafts 84 us, with it 90).
    static constexpr bool kScaled = std::is_same_v<E, Fp16>;
    float scale;
    uint32_t most;

    __device__ __forceinline__ void begin()
    {
        m = -INFINITY, l = 0.0f, scale = 1.0f, most = 0;
#pragma unroll
        for (int j = 0; j < W; j++) o[j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < G; i++) least[i] = 0.0f;
    }
    // bits: steps of this lane, NaN and infinities left out
    __device__ __forceinline__ void raise_scale(uint32_t bits)
    {
#pragma unroll
        for (int d = 32; d; d >>= 1) bits = max(bits, (uint32_t)__shfl_xor((int)bits, d));
        most = bits | 0x3ffu;   // float16's mantissa
        const float power = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, E::value(most)) & 0x7f800000u);
        const float next = 0.5f / power, by = next / scale;
#pragma unroll
        for (int j = 0; j < W; j++) o[j] *= by;
        scale = next;
    }
    static __device__ __forceinline__ uint32_t step_bits(uint32_t pair)
    {
        const uint32_t u = pair & 0x7fffu;
        return u < E::kExpMask ? u : 0;
    }
};

// One wave over the keys [key0, key1) of a head's pages, every step-th run of 32.
// EVEN: each quarter of DP dims is there as a whole or not at all, so that a
// lane's codes of K are one load.
template <class E, int DP, bool EVEN>
__device__ __forceinline__ void attend_wave(const Args &a, int b, int head, int n, const u32x4 (&q)[DP / 32], const u32x4 &qb,
                                            float qf, int limit, int key0, int key1, int step, Wave<E, DP> &x)
{
    typedef Wave<E, DP> X;
    typedef Code<E> C;
    constexpr int W = X::W, G = X::G, KW = X::KW;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    x.begin();
    if (key0 >= key1) return;
    const int dim = a.c.dim, row_bytes = dim / 2, words = dim / 8;
    // Held in registers: as constants they would make two instructions of the mask-and-or.
    uint32_t mask_bits = C::kMask, off_bits = C::kOffBits;
    asm("" : "+s"(mask_bits));
    asm("" : "+v"(off_bits));
    const auto number = [&](uint32_t w, int i) { return (C::shifted(w, i) & mask_bits) | off_bits; };
    const int all = n - a.tokens + 1;   // keys below this are seen by every row
    const uint8_t *const kc = a.c.k_codes + head * a.c.code_head, *const vc = a.c.v_codes + head * a.c.code_head;
    const uint32_t *const ks = a.c.k_scales + head * a.c.scale_head, *const vs = a.c.v_scales + head * a.c.scale_head;

    // Where the halves of the next 32 steps lie: lane 2 i + k speaks for half k
    // of step i, so that page ids are read once in 32 steps, all at once.
    uint32_t code_lo, code_hi, scale_lo, scale_hi;
    uint64_t there;
    const auto look = [&](int base) {
        const int at = base + (lane >> 1) * step + 16 * (lane & 1);
        int id = -1, row = 0;
        if (at < key1) {
            const int p = page_of(a.c, at >> 4);
            id = page_id(a.c, b, p);
            row = at - p * a.c.page;
        }
        there = __ballot(id >= 0);
        id = max(id, 0);   // no page: what lies in the first one is not seen
        const int64_t code = id * a.c.code_page + (int64_t)row * row_bytes, scale = id * a.c.scale_page + (int64_t)row * G;
        code_lo = (uint32_t)code, code_hi = (uint32_t)(code >> 32), scale_lo = (uint32_t)scale, scale_hi = (uint32_t)(scale >> 32);
    };
    const auto halves = [&](int base, int i) {
        Halves h;
        const int left = n - base;
        h.any = left >= 32 ? 0xffffffffu : (1u << left) - 1;
#pragma unroll
        for (int k = 0; k < 2; k++) {
            if (!(there >> (2 * i + k) & 1)) h.any &= k ? 0x0000ffffu : 0xffff0000u;
            const auto both = [&](uint32_t lo, uint32_t hi) {
                return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, 2 * i + k) << 32 |
                                 (uint32_t)__builtin_amdgcn_readlane(lo, 2 * i + k));
            };
            h.code[k] = both(code_lo, code_hi), h.scale[k] = both(scale_lo, scale_hi);
        }
        return h;
    };
    uint32_t kx[2][KW], kp[2][G], kw[2], vw[2];
    uint32_t vx[8][W / 8 ? W / 8 : 1];
    const int pair_at = G == 4 ? lane : 8 * g + (c & 7);   // the lane's pair: key 4 g + c / G, group c % G
    const auto load_k = [&](const Halves &h) {
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const uint8_t *from = kc + h.code[k];
            if constexpr (EVEN) {
                const int at = c * row_bytes + min(4 * KW * g, row_bytes - 4 * KW);   // dims that are not there: any codes
                __builtin_memcpy(kx[k], __builtin_assume_aligned(from + (uint32_t)at, KW >= 4 ? 16 : 8), 4 * KW);
            } else {
#pragma unroll
                for (int w = 0; w < KW; w++) kx[k][w] = *(const uint32_t *)(from + (uint32_t)(c * row_bytes + 4 * min(KW * g + w, words - 1)));
            }
            const uint32_t *pairs = ks + h.scale[k];
            __builtin_memcpy(kp[k], __builtin_assume_aligned(pairs + (uint32_t)(c * G), 4 * G), 4 * G);
            kw[k] = pairs[(uint32_t)pair_at];
        }
    };
    // a lane past the last dim reads any: its sums go nowhere
    const int v_at = min(c * W, dim - (W < 8 ? W : 8)) / 2, v_more = min(c * W + 8, dim - 8) / 2;
    const auto load_v = [&](const Halves &h) {
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const uint8_t *from = vc + h.code[k];
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const uint32_t row = (4 * g + r) * row_bytes;
                if constexpr (W == 4) vx[4 * k + r][0] = *(const uint16_t *)(from + row + v_at);
                else vx[4 * k + r][0] = *(const uint32_t *)(from + row + v_at);
                if constexpr (W == 16) vx[4 * k + r][1] = *(const uint32_t *)(from + row + v_more);
            }
            vw[k] = (vs + h.scale[k])[(uint32_t)pair_at];
        }
    };

    look(key0);
    int place_of = 0;
    Halves now = halves(key0, 0);
    load_k(now);
    load_v(now);
    for (int base = key0; base < key1; base += step) {
        const int next = base + step;
        f32x4 s[2], sum[2][G];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const u32x4 pairs{kp[k][0], kp[k][1], G == 4 ? kp[k][G - 2] : 0, G == 4 ? kp[k][G - 1] : 0};
            s[k] = E::mfma16(pairs, qb, f32x4{0, 0, 0, 0});
#pragma unroll
            for (int i = 0; i < G; i++) {
                sum[k][i] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int f = 0; f < KW / G; f++) {
                    u32x4 codes;
#pragma unroll
                    for (int w = 0; w < 4; w++)
                        codes[w] = G == 4 ? number(kx[k][4 * f + w], i) : number(kx[k][w / 2], i + 2 * (w & 1));
                    sum[k][i] = E::mfma16(codes, q[i * (KW / G) + f], sum[k][i]);
                }
            }
        }
        const float kstep[2] = {E::value(kw[0] & 0xffffu), E::value(kw[1] & 0xffffu)};
        // The last step's are loaded once more instead: a branch around the
        // loads would make every later wait one for all of them.
        const bool more = next < key1;
        place_of += more;
        if (place_of == 32) look(next), place_of = 0;
        const Halves then = halves(more ? next : base, place_of);
        load_k(then);
        __builtin_amdgcn_sched_barrier(0);   // add_scaled waits for the products above
#pragma unroll
        for (int k = 0; k < 2; k++) {
            s[k] *= qf;
            add_scaled<G>(s[k], kstep[k], sum[k]);
        }
        const bool plain = base + 32 <= all && now.any == 0xffffffffu;   // uniform: every row sees every key
        float vstep[2], vleast[2];
        bool odd = false;
#pragma unroll
        for (int k = 0; k < 2; k++) {
            // what no row sees takes part with weight 0: it must be a number
            if (!plain && !(now.any >> (16 * k + 4 * g + (G == 4 ? c >> 2 : (c & 7) >> 1)) & 1)) vw[k] = 0;
            vstep[k] = E::value(vw[k] & 0xffffu), vleast[k] = __builtin_fmaf(8.0f, vstep[k], E::value(vw[k] >> 16));
            if (!plain) odd = odd || (vw[k] & E::kExpMask) == E::kExpMask || (vw[k] >> 16 & E::kExpMask) == E::kExpMask;
        }
        if constexpr (X::kScaled) {
            const uint32_t bits = max(X::step_bits(vw[0]), X::step_bits(vw[1]));
            if (__any(bits > x.most)) x.raise_scale(bits);
            vstep[0] *= x.scale, vstep[1] *= x.scale;
        }
        if (!plain) {
#pragma unroll
            for (int k = 0; k < 2; k++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int i = 16 * k + 4 * g + r;
                    if (!(now.any >> i & 1) || base + i >= limit) s[k][r] = -INFINITY;
                }
        }
        float mx = s[0][0];
#pragma unroll
        for (int k = 0; k < 2; k++)
#pragma unroll
            for (int r = 0; r < 4; r++) mx = fmaxf(mx, s[k][r]);
        mx = over_rows(mx) * a.scale2;
        // m is kLift below the running maximum, which is raised only past
        // 2^8 times itself: the sums are seldom scaled
        const float low = mx - E::kLift;
        const bool raise = low > x.m + 8.0f;
        if (__any(raise)) {
            const float f = raise ? exp2_fast(x.m - low) : 1.0f;
            x.m = raise ? low : x.m;
            x.l *= f;
#pragma unroll
            for (int j = 0; j < W; j++) x.o[j] *= f;
#pragma unroll
            for (int i = 0; i < G; i++) x.least[i] *= f;
        }
        const float safe = x.m == -INFINITY ? 0.0f : x.m;
        float p[2][4];
#pragma unroll
        for (int k = 0; k < 2; k++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                p[k][r] = exp2_fast(__builtin_fmaf(s[k][r], a.scale2, -safe));
                x.l += p[k][r];
            }
        // Weight 0 times a step that is a number is 0.  Only where steps that
        // some rows must not see are no numbers, the query tokens take turns,
        // each with its unseen keys cleared and the sums of its own rows.
        const int turns = __any(odd) ? a.tokens : 1;
        for (int turn = 0; turn < turns; turn++) {
            // the numbers of V are made here in every turn, not held in registers over all of them
#pragma unroll
            for (int j = 0; j < 8; j++)
#pragma unroll
                for (int w = 0; w < (W / 8 ? W / 8 : 1); w++) asm("" : "+v"(vx[j][w]));
            float step_now[2] = {vstep[0], vstep[1]}, least_now[2] = {vleast[0], vleast[1]};
            if (turns > 1) {
#pragma unroll
                for (int k = 0; k < 2; k++)
                    if (base + 16 * k + 4 * g + (G == 4 ? c >> 2 : (c & 7) >> 1) >= all + turn) step_now[k] = least_now[k] = 0.0f;
            }
            u32x4 pb[G];
            float before[G];
#pragma unroll
            for (int i = 0; i < G; i++) before[i] = x.least[i];
#pragma unroll
            for (int k = 0; k < 2; k++) add_weighted<G>(x.least, least_now[k], p[k]);
            const bool others = turns > 1 && limit != all + turn;   // this lane's row has another turn
            if (turns > 1)
#pragma unroll
                for (int i = 0; i < G; i++) x.least[i] = others ? before[i] : x.least[i];
            unroll<G>([&](auto i) {
                float y[2][4];
#pragma unroll
                for (int k = 0; k < 2; k++)
                    unroll<4>([&](auto r) {
                        y[k][r] = p[k][r] * row_lane<decltype(r)::value * G + decltype(i)::value>(step_now[k]);
                    });
#pragma unroll
                for (int w = 0; w < 4; w++) pb[i][w] = E::pack(y[w >> 1][2 * (w & 1)], y[w >> 1][2 * (w & 1) + 1]);
                if (turns > 1)
#pragma unroll
                    for (int w = 0; w < 4; w++) pb[i][w] = others ? 0 : pb[i][w];
            });
            // byte v of two keys' words, in the low bytes of the halves; the
            // second product of each takes the codes' offset and 8 off
            const u32x4 mid{C::kMidBits, C::kMidBits, C::kMidBits, C::kMidBits};
#pragma unroll
            for (int v = 0; v < W / 2; v++) {
                u32x4 low, high;
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    const uint32_t sel = 0x0c000c00u | (4 + v % 4) << 16 | v % 4;   // 0x0c: a byte of zeros
                    const uint32_t y = __builtin_amdgcn_perm(vx[2 * w + 1][v / 4], vx[2 * w][v / 4], sel);
                    low[w] = number(y, 0), high[w] = number(y, 1);
                }
                x.o[2 * v] = E::mfma16(mid, pb[2 * v % G], E::mfma16(low, pb[2 * v % G], x.o[2 * v]));
                x.o[2 * v + 1] = E::mfma16(mid, pb[(2 * v + 1) % G], E::mfma16(high, pb[(2 * v + 1) % G], x.o[2 * v + 1]));
            }
        }
        load_v(then);
        now = then;
    }
}

// Few rows: a wave with the (at most four) rows of one key head and 64 keys at
// a time, lane l holding key l.
//   S^T: v_mfma_f32_4x4x4, 16 blocks of four keys, each lane's own codes as A;
//     a lane gets the logits of the four keys of its block (lanes 4 b .. 4 b + 3)
//     for row l % 4.  16-row tiles would spend four times the softmax and the
//     scaling on rows that are not there.
//   O^T: as above: B of the products over 32 keys takes its eight keys from
//     the first two or last two blocks of a row of 16 lanes, which are moved to the
//     row's first lanes; the other columns hold other keys' weights and are
//     left out at the end.
// Bound by memory once the keys are many: 64 requests of 4096 to 16384
// positions, 840 MB in 172 to 186 us, 4.5 to 4.9 TB/s, the vector ALU busy for
// half of it (16-row tiles 202 us).  33 requests of 64 dims: 29 us, 3.6 TB/s;
// one request of 1000 positions: 6.4 us, three round trips to memory.
constexpr int kFew = 4, kFewStep = 64;

template <class E>
__device__ __forceinline__ f32x4 mfma4(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mfma4<Bf16>(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, f32x4 c)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, u32x2{a0, a1}), __builtin_bit_cast(s16x4, u32x2{b0, b1}), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mfma4<Fp16>(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, f32x4 c)
{
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    return __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, u32x2{a0, a1}), __builtin_bit_cast(f16x4, u32x2{b0, b1}), c, 0, 0, 0);
}

// The value that lane N of each four lanes holds.
template <int N>
__device__ __forceinline__ float quad_lane(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), N * 0x55, 0xf, 0xf, true));
}
// The value that the lane 4 N places on in the row of 16 holds, N = 1 .. 3.
template <int N>
__device__ __forceinline__ uint32_t blocks_on(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + 16 - 4 * N, 0xf, 0xf, true);
}
// The greatest, or the sum, over the 16 lanes l % 4 apart.
template <class F>
__device__ __forceinline__ float over_blocks(float x, F &&join)
{
    x = join(x, __builtin_bit_cast(float, blocks_on<1>(__builtin_bit_cast(uint32_t, x))));
    x = join(x, __builtin_bit_cast(float, blocks_on<2>(__builtin_bit_cast(uint32_t, x))));
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    x = join(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
    const uint32_t v = __builtin_bit_cast(uint32_t, x);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return join(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}

// FULL: rows of DP dims, so their layout is known here.  prepare() brings the
// queries to LDS, while the first codes are on their way, and gives the power of two
// taken out of their sums; every wave calls it.  q: this lane's row there, in
// the order of the products, its sums' parts first.
template <class E, int DP, bool FULL, class F>
__device__ __forceinline__ void attend_few(const Args &a, int b, int head, int n, const uint32_t *q, F &&prepare, int limit,
                                           int key0, int key1, int step, Wave<E, DP> &x)
{
    typedef Wave<E, DP> X;
    typedef Code<E> C;
    constexpr int W = X::W, G = X::G, kWords = DP / 8;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    float &m = x.m, &l = x.l;
    x.begin();
    const int dim = FULL ? DP : a.c.dim, row_bytes = dim / 2, words = dim / 8;
    uint32_t mask_bits = C::kMask, off_bits = C::kOffBits;
    asm("" : "+s"(mask_bits));
    asm("" : "+v"(off_bits));
    const auto number = [&](uint32_t w, int i) { return (C::shifted(w, i) & mask_bits) | off_bits; };
    const int all = n - a.tokens + 1;   // keys below this are seen by every row
    const uint8_t *const kc = a.c.k_codes + head * a.c.code_head, *const vc = a.c.v_codes + head * a.c.code_head;
    const uint32_t *const ks = a.c.k_scales + head * a.c.scale_head, *const vs = a.c.v_scales + head * a.c.scale_head;

    // Where the quarters of the next 16 steps lie: lane 4 i + k speaks for quarter k of step i.
    uint32_t code_lo, code_hi, scale_lo, scale_hi;
    uint64_t there;
    const auto look = [&](int base) {
        const int at = base + (lane >> 2) * step + 16 * (lane & 3);
        int id = -1, row = 0;
        if (at < key1) {
            const int p = page_of(a.c, at >> 4);
            id = page_id(a.c, b, p);
            row = at - p * a.c.page;
        }
        there = __ballot(id >= 0);
        id = max(id, 0);   // no page: what lies in the first one is not seen
        const int64_t code = id * a.c.code_page + (int64_t)row * row_bytes, scale = id * a.c.scale_page + (int64_t)row * G;
        code_lo = (uint32_t)code, code_hi = (uint32_t)(code >> 32), scale_lo = (uint32_t)scale, scale_hi = (uint32_t)(scale >> 32);
    };
    // This lane's quarter of a step, and which of its quarters there are.
    struct At {
        int64_t code, scale;
        uint32_t quarters;
    };
    const auto find = [&](int i) {
        const int from = 4 * i + g;
        const auto both = [&](uint32_t lo, uint32_t hi) {
            return (int64_t)((uint64_t)(uint32_t)__shfl((int)hi, from) << 32 | (uint32_t)__shfl((int)lo, from));
        };
        return At{both(code_lo, code_hi), both(scale_lo, scale_hi), (uint32_t)(there >> (4 * i)) & 15u};
    };
    uint32_t kx[kWords], kp[G], vp[G], vx[16][W / 8 ? W / 8 : 1];
    const auto load_k = [&](const At &at) {
        const uint8_t *from = kc + at.code + c * row_bytes;
        if constexpr (FULL) {
            __builtin_memcpy(kx, __builtin_assume_aligned(from, 16), 4 * kWords);
        } else {
#pragma unroll
            for (int w = 0; w < kWords; w++) kx[w] = *(const uint32_t *)(from + 4 * min(w, words - 1));   // dims that are not there: any codes
        }
        __builtin_memcpy(kp, __builtin_assume_aligned(ks + at.scale + c * G, 4 * G), 4 * G);
    };
    const int v_at = min(c * W, dim - (W < 8 ? W : 8)) / 2, v_more = min(c * W + 8, dim - 8) / 2;
    const auto load_v = [&](const At &at) {
        const uint8_t *from = vc + at.code;
#pragma unroll
        for (int e = 0; e < 16; e++) {
            if constexpr (W == 4) vx[e][0] = *(const uint16_t *)(from + v_at + e * row_bytes);
            else vx[e][0] = *(const uint32_t *)(from + v_at + e * row_bytes);
            if constexpr (W == 16) vx[e][1] = *(const uint32_t *)(from + v_more + e * row_bytes);
        }
        __builtin_memcpy(vp, __builtin_assume_aligned(vs + at.scale + c * G, 4 * G), 4 * G);
    };

    int place_of = 0;
    At now{};
    const bool some = key0 < key1;
    if (some) {
        look(key0);
        now = find(0);
        load_k(now);
        load_v(now);
    }
    const float qf = prepare();
    if (!some) return;
    for (int base = key0; base < key1; base += step) {
        const int next = base + step;
        f32x4 s{0, 0, 0, 0}, sum[G];
#pragma unroll
        for (int i = 0; i < G; i++) sum[i] = f32x4{0, 0, 0, 0};
        const u32x4 *rows = (const u32x4 *)q;
        asm("" : "+v"(rows));   // read in every step: held in registers they would be DP / 2
#pragma unroll
        for (int w = 0; w < kWords; w += G / 2) {
            if (w % 4 == 0) __builtin_amdgcn_sched_barrier(0);   // numbers of later products would only hold registers
            u32x4 y[G / 2];
#pragma unroll
            for (int k = 0; k < G / 2; k++) y[k] = rows[3 + w + k];
#pragma unroll
            for (int i = 0; i < G; i++)
                sum[i] = mfma4<E>(number(kx[w], i), G == 4 ? number(kx[w + G / 2 - 1], i) : number(kx[w], i + 2), y[i / 2][i % 2 * 2],
                                  y[i / 2][i % 2 * 2 + 1], sum[i]);
        }
#pragma unroll
        for (int part = 0; part < 3; part++) {
            const u32x4 y = rows[part];
#pragma unroll
            for (int i = 0; i < G; i += 2) s = mfma4<E>(kp[i], kp[i + 1], y[i], y[i + 1], s);
        }
        float kstep[G];
#pragma unroll
        for (int i = 0; i < G; i++) kstep[i] = E::value(kp[i] & 0xffffu);
        const bool more = next < key1;   // the last step's are loaded once more instead: no branch around the loads
        place_of += more;
        if (place_of == 16) look(next), place_of = 0;
        const At then = find(place_of);
        load_k(then);
        s *= qf;
        unroll<G>([&](auto i) {
            unroll<4>([&](auto r) {
                constexpr int at = decltype(r)::value;
                s[at] = __builtin_fmaf(quad_lane<at>(kstep[decltype(i)::value]), sum[decltype(i)::value][at], s[at]);
            });
        });
        const bool plain = base + kFewStep <= all && now.quarters == 15u;   // uniform: every row sees every key
        bool odd = false;
        if (!plain) {
            // what no row sees takes part with weight 0: it must be a number
            const bool some = base + lane < n && (now.quarters >> g & 1);
#pragma unroll
            for (int i = 0; i < G; i++) {
                vp[i] = some ? vp[i] : 0;
                odd = odd || (vp[i] & E::kExpMask) == E::kExpMask || (vp[i] >> 16 & E::kExpMask) == E::kExpMask;
            }
#pragma unroll
            for (int r = 0; r < 4; r++)
                if (base + 4 * (lane >> 2) + r >= limit || !(now.quarters >> g & 1)) s[r] = -INFINITY;
        }
        if constexpr (X::kScaled) {
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < G; i++) bits = max(bits, X::step_bits(vp[i]));
            if (__any(bits > x.most)) x.raise_scale(bits);
        }
        float mx = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
        mx = over_blocks(mx, [](float u, float v) { return fmaxf(u, v); }) * a.scale2;
        const float low = mx - E::kLift;   // as in attend_wave
        const bool raise = low > m + 8.0f;
        if (__any(raise)) {
            const float f = raise ? exp2_fast(m - low) : 1.0f;
            m = raise ? low : m;
            l *= f;
#pragma unroll
            for (int j = 0; j < W; j++) x.o[j] *= f;
#pragma unroll
            for (int i = 0; i < G; i++) x.least[i] *= f;
        }
        const float safe = m == -INFINITY ? 0.0f : m;
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; r++) {
            p[r] = exp2_fast(__builtin_fmaf(s[r], a.scale2, -safe));
            l += p[r];
        }
        const int turns = __any(odd) ? a.tokens : 1;   // as in attend_wave
        for (int turn = 0; turn < turns; turn++) {
            // the numbers of V are made here in every turn, not held in registers over all of them
#pragma unroll
            for (int e = 0; e < 16; e++)
#pragma unroll
                for (int w = 0; w < (W / 8 ? W / 8 : 1); w++) asm("" : "+v"(vx[e][w]));
            const bool hidden = turns > 1 && base + lane >= all + turn, others = turns > 1 && limit != all + turn;
            uint32_t y[G][2];
            unroll<G>([&](auto i) {
                constexpr int k = decltype(i)::value;
                const float wide = hidden ? 0.0f : E::value(vp[k] & 0xffffu);
                const float least = hidden ? 0.0f : __builtin_fmaf(8.0f, wide, E::value(vp[k] >> 16));
                const float before = x.least[k], narrow = X::kScaled ? wide * x.scale : wide;
                float z[4];
                unroll<4>([&](auto r) {
                    constexpr int at = decltype(r)::value;
                    z[at] = p[at] * quad_lane<at>(narrow);
                    x.least[k] = __builtin_fmaf(quad_lane<at>(least), p[at], x.least[k]);
                });
                y[k][0] = E::pack(z[0], z[1]), y[k][1] = E::pack(z[2], z[3]);
                if (turns > 1)
                    y[k][0] = others ? 0 : y[k][0], y[k][1] = others ? 0 : y[k][1], x.least[k] = others ? before : x.least[k];
            });
            const u32x4 mid{C::kMidBits, C::kMidBits, C::kMidBits, C::kMidBits};
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int i = 0; i < G; i += 2) {
                    __builtin_amdgcn_sched_barrier(0);   // numbers of later products would only hold registers
                    // two of a row's four blocks, of four keys each
                    u32x4 pb[2];
#pragma unroll
                    for (int k = 0; k < 2; k++)
                        pb[k] = u == 0 ? u32x4{y[i + k][0], y[i + k][1], blocks_on<1>(y[i + k][0]), blocks_on<1>(y[i + k][1])}
                                       : u32x4{blocks_on<2>(y[i + k][0]), blocks_on<2>(y[i + k][1]), blocks_on<3>(y[i + k][0]),
                                               blocks_on<3>(y[i + k][1])};
#pragma unroll
                    for (int v = i / 2; v < W / 2; v += G / 2) {
                        u32x4 lower, upper;
#pragma unroll
                        for (int w = 0; w < 4; w++) {
                            const uint32_t sel = 0x0c000c00u | (4 + v % 4) << 16 | v % 4;
                            const uint32_t both = __builtin_amdgcn_perm(vx[8 * u + 2 * w + 1][v / 4], vx[8 * u + 2 * w][v / 4], sel);
                            lower[w] = number(both, 0), upper[w] = number(both, 1);
                        }
                        x.o[2 * v] = E::mfma16(mid, pb[0], E::mfma16(lower, pb[0], x.o[2 * v]));
                        x.o[2 * v + 1] = E::mfma16(mid, pb[1], E::mfma16(upper, pb[1], x.o[2 * v + 1]));
                    }
                }
        }
        load_v(then);
        now = then;
    }
}

__device__ __forceinline__ bool place(int i, int tiles, int pairs, int &tile, int &pair)
{
    // workgroups i and i + 8 run on one of the eight dies: the row tiles that
    // read the same pages follow each other there
    tile = i / 8 % tiles;
    pair = i % 8 + i / 8 / tiles * 8;
    return pair < pairs;
}
int64_t places(int64_t tiles, int64_t pairs) { return (pairs + 7) / 8 * 8 * tiles; }

__device__ __forceinline__ void put_lse(const Args &a, int64_t row, float m, float l)
{
    if (a.lse) a.lse[row] = l == 0.0f ? -INFINITY : kLn2 * (m + __log2f(l));
}

// The sums of a row's workgroup: each wave's in LDS, joined and written out.
template <class E, int DP>
__device__ __forceinline__ void join_waves(const Args &a, Wave<E, DP> &x, int b, int head, int split, int row0, int row_count)
{
    typedef Wave<E, DP> X;
    constexpr int W = X::W, G = X::G;
    __shared__ float join_o[kWaves][16][DP + 4];
    __shared__ float2 join_ml[kWaves][16];
    const float unscale = X::kScaled ? 1.0f / x.scale : 1.0f;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
    if (g == 0) join_ml[wave][c] = make_float2(x.m, x.l);
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
        for (int j = 0; j < W; j++) join_o[wave][c][(4 * g + r) * W + j] = __builtin_fmaf(x.o[j][r], unscale, x.least[j % G]);
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * (DP / 2); i += 64 * kWaves) {
        const int r = i / (DP / 2), d = 2 * (i % (DP / 2)), at = row0 + r;
        if (at >= row_count || d >= a.c.dim) continue;
        float mm = -INFINITY, ll = 0.0f, u = 0.0f, v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; w++) mm = fmaxf(mm, join_ml[w][r].x);
        const float safe = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
        for (int w = 0; w < kWaves; w++) {
            const float f = exp2_fast(join_ml[w][r].x - safe);
            ll += f * join_ml[w][r].y;
            u += f * join_o[w][r][d], v += f * join_o[w][r][d + 1];
        }
        const int64_t row = ((int64_t)b * a.tokens + at / a.group) * a.heads + head * a.group + at % a.group;
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        if (a.splits == 1) {
            *(uint32_t *)(a.out + row * a.c.dim + d) = E::pack(u * inv, v * inv);
            if (d == 0) put_lse(a, row, mm, ll);
        } else {
            *(float2 *)(a.part_o + (split * a.rows + row) * a.c.dim + d) = make_float2(u * inv, v * inv);
            if (d == 0) a.part_ml[split * a.rows + row] = make_float2(mm, ll);
        }
    }
}

// A power of two that leaves x / it below 16, and its inverse: float16 has bits
// down to 2^-24 for three parts of that.  bfloat16 has them for any number, and steps
// near float32's end, which are multiplied by kOff times that: below 2^-8 there.
template <class E>
__device__ __forceinline__ float power_below(float x, float &inverse)
{
    const uint32_t e = __builtin_bit_cast(uint32_t, x) >> 23;
    const uint32_t power = std::is_same_v<E, Bf16> ? min(e + 9, 253u) : e < 8 ? 127 : e - 3;
    inverse = __builtin_bit_cast(float, (254 - power) << 23);
    return __builtin_bit_cast(float, power << 23);
}

// Part k of x in 16-bit numbers that add up to it, with what the codes' offset
// makes of it: (-kOff, 1) times the part.
template <class E>
__device__ __forceinline__ uint32_t part_pair(float x, int k)
{
#pragma unroll
    for (int i = 0; i < 2; i++)
        if (k > i) x -= E::value(E::pack(x, 0.0f) & 0xffffu);
    x = E::value(E::pack(x, 0.0f) & 0xffffu);
    return E::pack(-Code<E>::kOff * x, x);
}

// A workgroup: a tile of one sequence's rows of one key head over a range of its keys.
struct Item {
    int tile, head, b, split, n, key0, key1;
    bool some;
};
__device__ __forceinline__ Item item_of(const Args &a)
{
    Item x{};
    int pair;
    if (!place(blockIdx.x, a.tiles, a.batch * a.c.kv_heads * a.splits, x.tile, pair)) return x;
    x.head = pair % a.c.kv_heads, x.b = pair / a.c.kv_heads % a.batch, x.split = pair / a.c.kv_heads / a.batch;
    x.n = (int)max((int64_t)0, min((int64_t)a.lengths[x.b], (int64_t)a.c.table_pages * a.c.page));
    x.key0 = edge(a, x.n, x.split), x.key1 = edge(a, x.n, x.split + 1);
    x.some = x.key0 < x.key1 || a.splits == 1;   // the join knows from n that there is no such range
    return x;
}

template <class E, int DP, bool EVEN>
__global__ void __launch_bounds__(64 * kWaves, DP == 256 ? 1 : 2) attend_kernel(const Args a)
{
    typedef Wave<E, DP> X;
    constexpr int G = X::G, KW = X::KW, kRows = 16;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
    const Item it = item_of(a);
    if (!it.some) return;
    const int row_count = a.tokens * a.group;
    const int row = it.tile * kRows + c;
    const int token = row / a.group, h = it.head * a.group + row % a.group;
    const uint16_t *from = a.q + it.b * a.q_batch + min(token, a.tokens - 1) * a.q_token + h * a.q_head;
    u32x4 q[DP / 32], qb;
    float sum[G];
#pragma unroll
    for (int i = 0; i < G; i++) sum[i] = 0.0f;
    // word w of this lane's dims: eight dims, i and i + 4 in group i mod G
#pragma unroll
    for (int w = 0; w < KW; w++) {
        const int d = 8 * (KW * g + w);
        const u32x4 y = *(const u32x4 *)(from + min(d, a.c.dim - 8));   // no branch around the loads
        const bool some = row < row_count && d < a.c.dim;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            uint32_t both = __builtin_amdgcn_perm(y[2 + i / 2], y[i / 2], i & 1 ? 0x07060302u : 0x05040100u);
            both = some ? both : 0;
            sum[i % G] += E::value(both & 0xffffu) + E::value(both >> 16);
            if (G == 4) q[i * (KW / G) + w / 4][w % 4] = both;
            else q[i % 2][2 * w + i / 2] = both;
        }
    }
    float most = 0.0f, inverse;
#pragma unroll
    for (int i = 0; i < G; i++) {
        sum[i] += __shfl_xor(sum[i], 16);
        sum[i] += __shfl_xor(sum[i], 32);
        most = fmaxf(most, fabsf(sum[i]));
    }
    const float qf = power_below<E>(most, inverse);
#pragma unroll
    for (int i = 0; i < 4; i++) qb[i] = i < G && g < 3 ? part_pair<E>(sum[i % G] * inverse, g) : 0;
    X x;
    attend_wave<E, DP, EVEN>(a, it.b, it.head, it.n, q, qb, qf, it.n - a.tokens + 1 + token, it.key0 + kStep * wave, it.key1,
                             kStep * kWaves, x);
    x.l += __shfl_xor(x.l, 16);
    x.l += __shfl_xor(x.l, 32);
#pragma unroll
    for (int i = 0; i < G; i++) {
        x.least[i] += __shfl_xor(x.least[i], 16);
        x.least[i] += __shfl_xor(x.least[i], 32);
    }
    join_waves<E, DP>(a, x, it.b, it.head, it.split, it.tile * kRows, row_count);
}

template <class E, int DP, bool FULL>
__global__ void __launch_bounds__(64 * kWaves, DP == 256 ? 2 : DP == 128 ? 3 : 4) few_kernel(const Args a)
{
    typedef Wave<E, DP> X;
    constexpr int G = X::G;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Item it = item_of(a);
    if (!it.some) return;
    const int row_count = a.tokens * a.group, row = lane & 3;
    const int token = row / a.group, h = it.head * a.group + row % a.group;
    const uint16_t *from = a.q + it.b * a.q_batch + min(token, a.tokens - 1) * a.q_token + h * a.q_head;
    __shared__ alignas(16) uint32_t q[kFew][DP / 2 + 20];   // rows in different banks
    __shared__ float powers[kFew];
    // The first wave brings the queries: a lane the words l / 4 (of eight dims)
    // of its row, on their way before any codes.
    constexpr int kEach = DP > 128 ? 2 : 1;
    u32x4 y[kEach];
#pragma unroll
    for (int k = 0; k < kEach; k++)
        y[k] = *(const u32x4 *)(from + 8 * min((lane >> 2) + 16 * k, a.c.dim / 8 - 1));
    const auto prepare = [&] {
        if (wave == 0) {
            float sum[G];
#pragma unroll
            for (int i = 0; i < G; i++) sum[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < kEach; k++) {
                const int w = (lane >> 2) + 16 * k;
                const bool some = row < row_count && 8 * w < a.c.dim;
#pragma unroll
                for (int i = 0; i < 4; i++) {   // the dims i and i + 4
                    uint32_t both = __builtin_amdgcn_perm(y[k][2 + i / 2], y[k][i / 2], i & 1 ? 0x07060302u : 0x05040100u);
                    both = some ? both : 0;
                    sum[i % G] += E::value(both & 0xffffu) + E::value(both >> 16);
                    if (w < DP / 8) q[row][12 + (G == 4 ? w / 2 * 8 + 2 * i + w % 2 : 4 * w + i % 2 * 2 + i / 2)] = both;
                }
            }
            float most = 0.0f, inverse;
#pragma unroll
            for (int i = 0; i < G; i++) {
                sum[i] = over_blocks(sum[i], [](float u, float v) { return u + v; });
                most = fmaxf(most, fabsf(sum[i]));
            }
            const float power = power_below<E>(most, inverse);
            if (lane < kFew) {
#pragma unroll
                for (int k = 0; k < 3; k++)
#pragma unroll
                    for (int i = 0; i < 4; i++) q[row][4 * k + i] = i < G ? part_pair<E>(sum[i % G] * inverse, k) : 0;
                powers[row] = power;
            }
        }
        __syncthreads();
        return powers[row];
    };
    X x;
    attend_few<E, DP, FULL>(a, it.b, it.head, it.n, q[row], prepare, it.n - a.tokens + 1 + token, it.key0 + kFewStep * wave,
                            it.key1, kFewStep * kWaves, x);
    const auto add = [](float u, float v) { return u + v; };
    x.l = over_blocks(x.l, add);
#pragma unroll
    for (int i = 0; i < G; i++) x.least[i] = over_blocks(x.least[i], add);
    join_waves<E, DP>(a, x, it.b, it.head, it.split, 0, row_count);
}

// Many rows: a workgroup of NW waves has 32 rows a wave, and all share the
// keys and values of a step in LDS, made of their codes there: that costs all
// rows together what scaling sums would cost each wave.  Roundings: a value of
// K is held in two numbers of the type, which leave 2^-16 (bfloat16) of it: the
// logits, and lse, would show one.  A value of V and its weight are rounded to
// float16 for either type, V times the power of two that brings the greatest
// of the range to 2^14, if no bound of a group (but 0) is 2^20 times another:
// 2^-11 of each, and 2^-18 of its bound where that is small.  Else both are
// rounded to the type, so that a value without weight costs others nothing.
// For float16 results V is held in two numbers as well: one and the weight would
// come to half as much again as the result's own rounding.
// (bfloat16 for both, 2^-8, took 4 us of 196 less, and made the error of a
// bfloat16 result half as large again as its own rounding does; V in two numbers of bfloat16, 26 us more.)
// The next step's codes are on their way meanwhile.
//   S^T = K Q^T    v_mfma_f32_32x32x16: the A operand of lane l is key l % 32,
//                  dims 16 i + 8 (l / 32) .. + 7 of step i, the B operand the
//                  same dims of row l % 32.
//   O^T = V^T P^T  lane l's logits belong to row l % 32 and the keys
//                  8 (r / 4) + 4 (l / 32) + r % 4: eight of them are the B
//                  operand of a step of 16 keys, so V is laid out in LDS with
//                  those eight keys of a dim side by side.
// A code becomes a number by one mask-and-or for two (float16: 16 + c for K, and
// for V 1024 + c or 64 + c, as its place in the word has it, which costs float32's
// sum 2^-14 of a step) and one mixed-precision multiply-add.
// Bound by issue: a step of 64 keys (128 dims, 8 waves) has 96 matrix
// instructions a SIMD, 3070 cycles, and 3800 cycles of vector instructions, half
// of them for the values, and takes 6700, 3.4 us at the 1.97 GHz that the card
// holds: the two hardly overlap.  Turns of half of the waves (with three
// buffers of V), fragments further ahead and values made between the products
// took as long, two tiles a wave spilled.  A chunk of 512 tokens over 2048 and
// 8192 positions, 32 heads on 8: 161 us, and 20 us for the joining.
template <class E, int DP, int NW, bool EVEN>
__global__ void __launch_bounds__(64 * NW, DP == 256 ? 1 : 2) tile_kernel(const Args a)
{
    typedef TileShape<DP> S;
    constexpr int kKeys = S::kKeys, G = DP == 64 ? 2 : 4, kWords = DP / 8, kThreads = 64 * NW;
    constexpr int kEach = kKeys * kWords / kThreads;        // words of K of a thread, of one key
    constexpr int kPair = kKeys * kWords / kThreads;        // keys of a thread's word of V
    static_assert(kEach == 4 || kEach == 2, "");
    constexpr int kNumbers = std::is_same_v<E, Fp16> ? 2 : 1;   // float16 to a value of V
    // K is made times a power of two: the greatest code may stand for more than
    // the type's greatest number, since the step is rounded, and bfloat16's 16 steps for
    // more than float32's.
    constexpr float kKeyPower = std::is_same_v<E, Fp16> ? 0.5f : 0.25f;
    constexpr int kHalf = kKeys * DP * 2, kBuffer = (2 + kNumbers) * kHalf;   // a step's K, V^T, and what is left of K (and V)
    __shared__ alignas(1024) char lds[2 * kBuffer];
    __shared__ uint64_t pages[2];   // a byte for each 16 keys of a step: whether there is a page
    __shared__ int odd;             // whether some of V is no number for some rows
    __shared__ uint32_t top, bottom;   // bits of a 32nd of the greatest and the least bound of a group of V
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 31, g = lane >> 5;
    const float scale2 = a.scale2 / kKeyPower;
    Item it = item_of(a);
    if (!it.some) return;
    const int row_count = a.tokens * a.group, n = it.n, all = n - a.tokens + 1;
    const int tile_row = it.tile * 32 * NW;
    // no row of the tile sees more than its last one
    const int key0 = it.key0, key1 = min(it.key1, all + min(row_count - 1, tile_row + 32 * NW - 1) / a.group);
    const int dim = a.c.dim, row_bytes = dim / 2;
    const int row = tile_row + wave * 32 + c;
    const int token = min(row / a.group, a.tokens - 1), h = it.head * a.group + row % a.group;
    const int limit = row < row_count ? all + token : 0;
    if (threadIdx.x == 0) odd = 0, top = 0, bottom = 0x7f800000u;
    if (threadIdx.x < 2) pages[threadIdx.x] = ~0ull;
    __syncthreads();
    u32x4 q[DP / 16];
    const uint16_t *from = a.q + it.b * a.q_batch + token * a.q_token + h * a.q_head;
#pragma unroll
    for (int i = 0; i < DP / 16; i++) {
        const int d = 16 * i + 8 * g;
        const u32x4 x = *(const u32x4 *)(from + min(d, dim - 8));
#pragma unroll
        for (int w = 0; w < 4; w++) q[i][w] = row < row_count && d < dim ? x[w] : 0;
    }

    // What a thread brings: kEach words of a key's K, and a word of kPair keys' V.
    const uint8_t *const kc = a.c.k_codes + it.head * a.c.code_head, *const vc = a.c.v_codes + it.head * a.c.code_head;
    const uint32_t *const ks = a.c.k_scales + it.head * a.c.scale_head, *const vs = a.c.v_scales + it.head * a.c.scale_head;
    const int k_key = threadIdx.x / (kWords / kEach), k_word = threadIdx.x % (kWords / kEach) * kEach;
    const int v_unit = threadIdx.x / kWords, v_word = threadIdx.x % kWords, v_key = v_unit * kPair;
    const int words = dim / 8;
    uint32_t kx[kEach], vx[kPair], kp[G], vp[kPair][G];
    // Where the runs of 16 keys of the next 64 / kRuns steps lie: lane kRuns i + r
    // speaks for run r of step i.
    constexpr int kRuns = kKeys / 16, kSteps = 64 / kRuns;
    uint32_t code_lo, code_hi, scale_lo, scale_hi;
    uint64_t runs_there;
    const auto id_of = [&](int key, int &in) {
        const int at = page_of(a.c, key >> 4);
        in = key - at * a.c.page;
        return page_id(a.c, it.b, at);
    };
    const auto look = [&](int base) {
        int in = 0, id = -1;
        if (base + 16 * lane < n) id = id_of(base + 16 * lane, in);
        runs_there = __ballot(id >= 0);
        id = max(id, 0);   // no page: what lies in the first one is not seen
        const int64_t code = id * a.c.code_page + (int64_t)in * row_bytes, scale = id * a.c.scale_page + (int64_t)in * G;
        code_lo = (uint32_t)code, code_hi = (uint32_t)(code >> 32), scale_lo = (uint32_t)scale, scale_hi = (uint32_t)(scale >> 32);
    };
    bool v_there;
    const int k_in = k_key % 16 * row_bytes + min(4 * k_word, row_bytes - 4 * kEach);
    const int v_in = v_key % 16 * row_bytes + 4 * min(v_word, words - 1);
    // The codes of step i of those.
    const auto load = [&](int i) {
        const auto place = [&](int key, int64_t &code, int64_t &scale) {   // a wave's keys are of one run
            const int from = kRuns * i + __builtin_amdgcn_readfirstlane(key / 16);
            const auto both = [&](uint32_t lo, uint32_t hi) {
                return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi, from) << 32 |
                                 (uint32_t)__builtin_amdgcn_readlane((int)lo, from));
            };
            code = both(code_lo, code_hi), scale = both(scale_lo, scale_hi);
            return from;
        };
        int64_t code, scale;
        place(k_key, code, scale);
        const uint8_t *const kc_run = kc + code;
        const uint32_t *const ks_run = ks + scale;
        v_there = runs_there >> place(v_key, code, scale) & 1;
        const uint8_t *const vc_run = vc + code;
        const uint32_t *const vs_run = vs + scale;
        if constexpr (EVEN) {
            __builtin_memcpy(kx, __builtin_assume_aligned(kc_run + k_in, 4 * kEach), 4 * kEach);
        } else {
#pragma unroll
            for (int w = 0; w < kEach; w++) kx[w] = *(const uint32_t *)(kc_run + k_key % 16 * row_bytes + 4 * min(k_word + w, words - 1));
        }
        __builtin_memcpy(kp, __builtin_assume_aligned(ks_run + k_key % 16 * G, 4 * G), 4 * G);
#pragma unroll
        for (int j = 0; j < kPair; j++) {
            vx[j] = *(const uint32_t *)(vc_run + v_in + j * row_bytes);   // the kPair keys lie behind each other
            __builtin_memcpy(vp[j], __builtin_assume_aligned(vs_run + (v_key % 16 + j) * G, 4 * G), 4 * G);
        }
    };
    float v_scale = 1.0f;
    // A power of two that brings V's values below 2^15 (infinities aside), and
    // whether they are held so.
    const auto find_scale = [&] {
        float most = 0.0f, least = INFINITY;
        for (int key = key0 + threadIdx.x; key < key1; key += 4 * kThreads) {
            uint32_t pairs[4][G];
            bool there[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {   // keys behind the last: that one's once more
                int in, id = id_of(min(key + j * kThreads, key1 - 1), in);
                there[j] = id >= 0;
                id = max(id, 0);
                __builtin_memcpy(pairs[j], __builtin_assume_aligned(vs + id * a.c.scale_page + (int64_t)in * G, 4 * G), 4 * G);
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int i = 0; i < G; i++) {
                    // a 32nd of the bound, which no number of the type brings past float32's range
                    const float x = __builtin_fmaf(15.0f / 32, fabsf(E::value(pairs[j][i] & 0xffffu)), fabsf(E::value(pairs[j][i] >> 16)) / 32);
                    most = there[j] && x < INFINITY ? fmaxf(most, x) : most;
                    least = there[j] && x > 0.0f ? fminf(least, x) : least;
                }
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) most = fmaxf(most, __shfl_xor(most, d)), least = fminf(least, __shfl_xor(least, d));
        if (lane == 0) atomicMax(&top, __builtin_bit_cast(uint32_t, most)), atomicMin(&bottom, __builtin_bit_cast(uint32_t, least));
        lds_barrier();
        const bool apart = __builtin_bit_cast(float, top) > 0x1p20f * __builtin_bit_cast(float, bottom);
        const int power = (int)(top >> 23) - 127 + 5;   // a range without values: -122
        // Far apart: as they are, for the small ones' sake, but for what float16 would
        // not hold, or float32's sum of 2^30 of them, each held up to 2^8 high
        constexpr int kApart = std::is_same_v<E, Fp16> ? 14 : 88;
        v_scale = __builtin_ldexpf(1.0f, apart ? min(kApart - power, 0) : min(14 - power, 126));
        return !apart;
    };
    // The values of a word's eight codes.
    const auto values = [&](uint32_t w, const uint32_t (&pairs)[G], auto exact, float by, float (&y)[8]) {
        constexpr bool kExact = decltype(exact)::value;
        float step[G], least[G];
#pragma unroll
        for (int i = 0; i < G; i++) {
            step[i] = E::value(pairs[i] & 0xffffu) * by;
            least[i] = __builtin_fmaf(kExact ? -16.0f : i % 2 ? -64.0f : -1024.0f, step[i], E::value(pairs[i] >> 16) * by);
        }
        uint32_t x[4];   // dims i and i + 4
#pragma unroll
        for (int i = 0; i < 4; i++)
            x[i] = kExact ? (Code<Fp16>::shifted(w, i) & Code<Fp16>::kMask) | Code<Fp16>::kOffBits
                          : ((i < 2 ? w : w >> 8) & (i % 2 ? 0x00f000f0u : 0x000f000fu)) | (i % 2 ? 0x54005400u : 0x64006400u);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const f16x2 z = __builtin_bit_cast(f16x2, x[i]);
            y[i] = __builtin_fmaf((float)z[0], step[i % G], least[i % G]);
            y[i + 4] = __builtin_fmaf((float)z[1], step[i % G], least[i % G]);
        }
    };
    const int v_to = S::v_at(v_word * 8, v_key / 16 * 2 + (v_key / 4 & 1)) + (v_key / 8 & 1) * 8 + v_key % 4 * 2;
    // A value that a row does not see has weight 0 there, so it must be a
    // number: of keys that no row of the tile sees it is 0 (as a finite one it
    // might pass float16: find_scale looks at the keys below key1); of those that some
    // see it is too, if it is none, and comes last (below).
    const auto clear = [&](int to, int base) {
        const bool whole = __all(v_there);
        if (!whole || base + kKeys > all) {
            const int key = base + v_key;
#pragma unroll
            for (int j = 0; j < kPair; j++)
#pragma unroll
                for (int i = 0; i < G; i++) {
                    const uint32_t x = vp[j][i];
                    const bool number = (x & E::kExpMask) != E::kExpMask && (x >> 16 & E::kExpMask) != E::kExpMask;
                    const bool seen = v_there && key + j < key1;
                    if (seen && key + j >= all && !number) odd = 1;
                    if (!seen || (key + j >= all && !number)) vp[j][i] = 0;
                }
        }
        if (v_word == 0 && v_key % 16 == 0) ((uint8_t *)(pages + to))[v_key / 16] = v_there ? 255 : 0;
    };
    const auto make = [&](auto number, int to) {   // number: the type of weights and V
        typedef decltype(number) N;
        const int k_first = S::k_at(k_key, k_word);   // k_word is a multiple of kEach
#pragma unroll
        for (int w = 0; w < kEach; w++) {
            float y[8];
            values(kx[w], kp, std::true_type{}, kKeyPower, y);
            u32x4 x, left;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                x[i] = E::pack(y[2 * i], y[2 * i + 1]);
                left[i] = E::pack(y[2 * i] - E::value(x[i] & 0xffffu), y[2 * i + 1] - E::value(x[i] >> 16));
            }
            *(u32x4 *)(lds + to * kBuffer + (k_first ^ w * 16)) = x;
            *(u32x4 *)(lds + to * kBuffer + 2 * kHalf + (k_first ^ w * 16)) = left;
        }
        float y[kPair][8];
#pragma unroll
        for (int j = 0; j < kPair; j++) values(vx[j], vp[j], std::false_type{}, v_scale, y[j]);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            char *at = lds + to * kBuffer + S::v_next_dim(v_to, i);
            uint32_t x[kPair / 2];
#pragma unroll
            for (int n = 0; n < kNumbers; n++) {
#pragma unroll
                for (int j = 0; j < kPair / 2; j++) {
                    float &y0 = y[2 * j][i], &y1 = y[2 * j + 1][i];
                    x[j] = N::pack(y0, y1);
                    if (n + 1 < kNumbers) y0 -= N::value(x[j] & 0xffffu), y1 -= N::value(x[j] >> 16);
                }
                __builtin_memcpy(__builtin_assume_aligned(at + n * 2 * kHalf, 2 * kPair), x, 2 * kPair);
            }
        }
    };

    f32x16 o[DP / 32];
#pragma unroll
    for (int i = 0; i < DP / 32; i++)
#pragma unroll
        for (int r = 0; r < 16; r++) o[i][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    constexpr int kK = 2 * (DP / 16), kParts = kKeys / 32, kV = 2 * kNumbers * (DP / 32), kAhead = 4;
    const int k_from = S::k_at(c, g), v_from = S::v_at(c, g);
    f32x16 s[kParts];
    // A step's first products.
    const auto logits = [&](int buffer) {
        u32x4 f[kParts * kK];
        const auto frag = [&](int i) {
            const int j = i / kParts;   // both numbers of each 16 dims in turn
            return *(const u32x4 *)(lds + buffer * kBuffer + S::k_next(k_from, j / 2) + 32 * (i % kParts) * DP * 2 + j % 2 * 2 * kHalf);
        };
#pragma unroll
        for (int i = 0; i < kAhead; i++) f[i] = frag(i);
#pragma unroll
        for (int k = 0; k < kParts; k++)
#pragma unroll
            for (int r = 0; r < 16; r++) s[k][r] = 0.0f;
#pragma unroll
        for (int i = 0; i < kParts * kK; i++) {
            if (i + kAhead < kParts * kK) f[i + kAhead] = frag(i + kAhead);
            s[i % kParts] = E::mfma32(f[i], q[i / kParts / 2], s[i % kParts]);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int i = 0; i < kParts * kK; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (i + kAhead < kParts * kK) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // Its softmax and second products.
    const auto sums = [&](auto number, int buffer, int base, uint64_t there) {
        typedef decltype(number) N;
        u32x4 f[kParts * kV];
        const auto frag = [&](int i) { 
            const int part = i / (DP / 32);   // both numbers of each 16 keys in turn
            return *(const u32x4 *)(lds + buffer * kBuffer + S::v_next(v_from, i % (DP / 32), part / kNumbers) + part % kNumbers * 2 * kHalf);
        };
#pragma unroll
        for (int i = 0; i < kAhead; i++) f[i] = frag(i);
        if (base + kKeys > min(all, key1) || there != ~0ull) {
            __builtin_amdgcn_sched_barrier(0);   // a branch of its own: no other step pays for it
#pragma unroll
            for (int k = 0; k < kParts; k++)
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    const int at = 32 * k + 8 * (r / 4) + 4 * g + r % 4;
                    if (base + at >= min(limit, key1) || !(there >> (8 * (2 * k + r / 8)) & 1)) s[k][r] = -INFINITY;
                }
        }
        float mx = s[0][0];
#pragma unroll
        for (int k = 0; k < kParts; k++)
#pragma unroll
            for (int r = 0; r < 16; r++) mx = fmaxf(mx, s[k][r]);
        mx = fmaxf(mx, __shfl_xor(mx, 32)) * scale2;
        const float low = mx - N::kLift;   // as in attend_wave
        const bool raise = low > m + 8.0f;
        if (__any(raise)) {
            const float by = raise ? exp2_fast(m - low) : 1.0f;
            m = raise ? low : m;
            l *= by;
#pragma unroll
            for (int i = 0; i < DP / 32; i++) o[i] *= by;
        }
        const float safe = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int k = 0; k < kParts; k++)
#pragma unroll
            for (int half = 0; half < 2; half++) {
                u32x4 pb;
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    const float x = exp2_fast(__builtin_fmaf(s[k][8 * half + 2 * w], scale2, -safe));
                    const float y = exp2_fast(__builtin_fmaf(s[k][8 * half + 2 * w + 1], scale2, -safe));
                    l += x + y;
                    pb[w] = N::pack(x, y);
                }
#pragma unroll
                for (int i = 0; i < kNumbers * (DP / 32); i++) {
                    const int at = (2 * k + half) * kNumbers * (DP / 32) + i;
                    if (at + kAhead < kParts * kV) f[at + kAhead] = frag(at + kAhead);
                    o[i % (DP / 32)] = N::mfma32(f[at], pb, o[i % (DP / 32)]);
                }
            }
        __builtin_amdgcn_sched_group_barrier(0x402, 8 * 2 + 4, 0);
#pragma unroll
        for (int i = 0; i < kParts * kV; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (i < kParts * kV - kAhead) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x402, 7, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    const auto run = [&](auto number) {
        clear(0, key0);
        make(number, 0);
        int ahead = 0;   // the step loaded last, of those that look() found
        const auto advance = [&](int base) {
            if (base < key1) ahead++;   // behind the last step: that one's once more
            if (ahead == kSteps) look(base), ahead = 0;
            load(ahead);
        };
        advance(key0 + kKeys);
        lds_barrier();
        for (int base = key0; base < key1; base += 2 * kKeys) {
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const int at = base + half * kKeys;
                if (at >= key1) break;
                const uint64_t there = pages[half];
                clear(1 - half, at + kKeys);
                logits(half);
                make(number, 1 - half);
                advance(at + 2 * kKeys);
                sums(number, half, at, there);
                lds_barrier();
            }
        }
    };
    if (key0 < key1) {
        look(key0);
        load(0);
        if (find_scale() || std::is_same_v<E, Fp16>) run(Fp16{});
        else run(E{});
    }
    if (odd) {
        // what was left out: values that are no numbers, for the rows that see them
        uint32_t bad = 0;
        for (int key = max(key0, all); key < key1; key++) {
            int in;
            const int id = id_of(key, in);
            if (id < 0) continue;
            const uint32_t *pairs = vs + id * a.c.scale_page + (int64_t)in * G;
#pragma unroll
            for (int i = 0; i < G; i++) {
                const bool number = (pairs[i] & E::kExpMask) != E::kExpMask && (pairs[i] >> 16 & E::kExpMask) != E::kExpMask;
                if (!number && key < limit) bad |= 1u << i;
            }
        }
#pragma unroll
        for (int i = 0; i < DP / 32; i++)
#pragma unroll
            for (int r = 0; r < 16; r++) o[i][r] = bad >> (r % G) & 1 ? NAN : o[i][r];   // dim 32 i + 8 (r / 4) + 4 g + r % 4
    }
    const float unscale = 1.0f / v_scale;
    l += __shfl_xor(l, 32);
    if (row >= row_count) return;
    const int64_t out_row = ((int64_t)it.b * a.tokens + token) * a.heads + h;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (a.splits == 1) {
#pragma unroll
        for (int i = 0; i < DP / 32; i++)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int d = 32 * i + 2 * r + 4 * g;
                const f32x4 x = f32x4{o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]} * inv * unscale;
                if (d < dim)
                    *(u32x2 *)(a.out + out_row * dim + d) = u32x2{E::pack(x[0], x[1]), E::pack(x[2], x[3])};
            }
        if (g == 0) put_lse(a, out_row, m, l);
    } else {
        float *to = a.part_o + (it.split * a.rows + out_row) * dim;
#pragma unroll
        for (int i = 0; i < DP / 32; i++)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int d = 32 * i + 2 * r + 4 * g;
                if (d < dim) *(f32x4 *)(to + d) = f32x4{o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]} * inv * unscale;
            }
        if (g == 0) a.part_ml[it.split * a.rows + out_row] = make_float2(m, l);
    }
}

// Joins the ranges (at most 64) of output rows: a wave a row, or (WIDE) a
// workgroup a row whose waves take every fourth range.  Bound by latency where
// the rows are few (4 to 5 us up to 4096 rows, of 128 dims); 32768 rows of 2 to 5
// ranges 21 us, 4 TB/s.
template <class E, bool WIDE>
__global__ void __launch_bounds__(64 * kWaves) join_kernel(const Args a)
{
    __shared__ float2 sums[kWaves][DF11_MAX_DIM / 2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = WIDE ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kWaves + wave;
    if (row >= a.rows) return;
    const int b = (int)(row / ((int64_t)a.tokens * a.heads));
    const int n = (int)max((int64_t)0, min((int64_t)a.lengths[b], (int64_t)a.c.table_pages * a.c.page));
    const bool there = lane < a.splits && edge(a, n, lane) < edge(a, n, lane + 1);
    const uint64_t ranges = __ballot(there);
    const int last = ranges ? 63 - __builtin_clzll(ranges) : 0;
    const float2 mine = there ? a.part_ml[lane * a.rows + row] : make_float2(-INFINITY, 0.0f);
    float m = mine.x;
#pragma unroll
    for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float safe = m == -INFINITY ? 0.0f : m;
    const float part = exp2_fast(mine.x - safe) * mine.y;
    float l = part;
#pragma unroll
    for (int d = 32; d; d >>= 1) l += __shfl_xor(l, d);
    const float factor = part * (l == 0.0f ? 0.0f : 1.0f / l);
    constexpr int kBy = WIDE ? kWaves : 1;
    // every lane goes through the sums, those behind the last dim with that one once
    // more: each holds the factor of a range, which the others read
    for (int d0 = 0; d0 < a.c.dim; d0 += 128) {
        const int d = min(d0 + 2 * lane, a.c.dim - 2);
        float x = 0.0f, y = 0.0f;
        for (int s0 = WIDE ? wave : 0; s0 < a.splits; s0 += 8 * kBy) {
            float2 o[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {   // where there is no range the last one's once more, which is near by now
                const int s = s0 + j * kBy;
                o[j] = *(const float2 *)(a.part_o + ((s < a.splits && ranges >> s & 1 ? s : last) * a.rows + row) * a.c.dim + d);
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int s = s0 + j * kBy;
                if (s >= a.splits || !(ranges >> s & 1)) continue;   // what an empty range left there may be anything
                const float f = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, factor), s));
                x += f * o[j].x, y += f * o[j].y;
            }
        }
        if (WIDE) sums[wave][d / 2] = make_float2(x, y);
        else *(uint32_t *)(a.out + row * a.c.dim + d) = E::pack(x, y);
    }
    if (WIDE) {
        __syncthreads();
        if (2 * threadIdx.x < a.c.dim) {
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; w++) x += sums[w][threadIdx.x].x, y += sums[w][threadIdx.x].y;
            *(uint32_t *)(a.out + row * a.c.dim + 2 * threadIdx.x) = E::pack(x, y);
        }
    }
    if (lane == 0 && (!WIDE || wave == 0)) put_lse(a, row, m, l);
}

// ----------------------------------------------------------------- host side

// Whether out lies on some of q otherwise than as q itself: a workgroup would
// write rows that another has yet to read.
bool out_on_q(const Args &a)
{
    const Axis q[3] = {{a.batch, a.q_batch}, {a.tokens, a.q_token}, {a.heads, a.q_head}};
    int64_t stride = a.c.dim;
    bool same = a.q == a.out;
    for (int i = 2; i >= 0; i--) {
        same = same && (q[i].size == 1 || q[i].stride == stride);
        stride *= q[i].size;
    }
    const uintptr_t from = (uintptr_t)a.out / 2;   // in values, whose addresses are even
    return !same && rows_meet(from, (__int128)from + stride, (uintptr_t)a.q / 2, q, 3, a.c.dim);
}

int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
bool within(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
constexpr int64_t kMost = 1ll << 30;
constexpr int64_t kMostThreads = 0xffffffffll;   // a launch has fewer than 2^32 threads

int make_cache(const char *who, const df11_quantized_cache *p, const int32_t *table, int64_t table_pages,
               int64_t table_batch, int64_t batch, Cache &c)
{
    if (!p) return df11::fail(DF11_E_ARG, "%s: null cache", who);
    if (p->dtype != DF11_BF16 && p->dtype != DF11_FP16) return df11::fail(DF11_E_ARG, "%s: dtype must be bf16 or fp16", who);
    if (!within(p->dim, 8, DF11_MAX_DIM) || p->dim % 8)
        return df11::fail(DF11_E_ARG, "%s: dim %lld is not a multiple of 8 up to %d", who, (long long)p->dim, DF11_MAX_DIM);
    if (!within(p->pages, 0, kMost) || !within(p->page, 16, kMost) || p->page % 16 || !within(p->kv_heads, 1, 65535))
        return df11::fail(DF11_E_ARG, "%s: pages, page (a multiple of 16) or kv_heads out of range", who);
    if (p->code_page < 0 || p->code_head < 0 || p->scale_page < 0 || p->scale_head < 0 ||
        (p->code_page | p->code_head) % 16 || (p->scale_page | p->scale_head) % 8)
        return df11::fail(DF11_E_ARG, "%s: strides of codes must be multiples of 16, of scales multiples of 8", who);
    if (!within(batch, 0, 65535)) return df11::fail(DF11_E_ARG, "%s: batch out of range", who);
    if (table && (!within(table_pages, 0, kMost) || table_batch < 0 || (double)table_pages * p->page > kMost))
        return df11::fail(DF11_E_ARG, "%s: a sequence's pages out of range", who);
    if (p->pages && batch && (!aligned16(p->k_codes) || !aligned16(p->v_codes) || !aligned16(p->k_scales) || !aligned16(p->v_scales)))
        return df11::fail(DF11_E_ARG, "%s: null or misaligned cache pointer", who);
    c.k_codes = (uint8_t *)p->k_codes, c.v_codes = (uint8_t *)p->v_codes;
    c.k_scales = (uint32_t *)p->k_scales, c.v_scales = (uint32_t *)p->v_scales;
    c.pages = p->pages, c.page = p->page, c.kv_heads = p->kv_heads, c.dim = p->dim, c.groups = p->dim <= 64 ? 2 : 4;
    c.code_page = p->code_page, c.code_head = p->code_head, c.scale_page = p->scale_page / 2, c.scale_head = p->scale_head / 2;
    c.per_page = 1.0 / (double)(p->page / 16);
    c.table = table, c.table_batch = table_batch;
    c.table_pages = !p->pages ? 0 : table ? table_pages : 1;
    return DF11_OK;
}

// Whether no two heads' pages share memory, as those of a cache that is
// written must not.
bool pages_apart(const df11_quantized_cache *p, int64_t stride_page, int64_t stride_head, int64_t own)
{
    int64_t small = stride_head, few = p->kv_heads, great = stride_page, many = p->pages;
    if (great < small) std::swap(small, great), std::swap(few, many);
    __int128 span = own;
    if (few > 1) {
        if (small < span) return false;
        span += (__int128)small * (few - 1);
    }
    return many <= 1 || great >= span;
}

bool strides_ok(std::initializer_list<int64_t> strides)
{
    for (int64_t s : strides)
        if (s < 0 || s % 8) return false;
    return true;
}

int launched(const char *who)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return df11::fail(DF11_E_DEVICE, "%s launch: %s", who, hipGetErrorString(e));
    return DF11_OK;
}

template <class F>
void by_shape(int64_t dtype, int dim, F &&f)
{
    const auto shape = [&](auto e) {
        if (dim <= 64) f(e, std::integral_constant<int, 64>{});
        else if (dim <= 128) f(e, std::integral_constant<int, 128>{});
        else f(e, std::integral_constant<int, 256>{});
    };
    if (dtype == DF11_FP16) shape(Fp16{});
    else shape(Bf16{});
}

void plan(Args &a)
{
    const int64_t cus = df11::cu_count();
    a.rows = (int64_t)a.batch * a.tokens * a.heads;
    if (!a.rows) return;
    a.few = a.tokens * a.group <= kFew;
    const int64_t rows = (int64_t)a.tokens * a.group;
    a.many = rows > kMany;
    a.tiles = ceil_div(rows, a.many ? 32 * tile_waves(a.c.dim) : 16);
    const int64_t keys = std::max<int64_t>(1, (int64_t)a.c.table_pages * a.c.page);
    // Ranges of each sequence's own length, which only the GPU knows.  Where
    // the items are many, tapering ones, so that the last workgroups are short
    // (64 requests of 4096 to 16384 keys: 189 us, 193 us in five even ranges;
    // the chunk of tile_kernel 181 us, with 3, 4, 6 and 8 tapering ranges 235,
    // 199, 208 and 197, which is how its two lengths pack: over random lengths a
    // model of the packing gives 1.43 times the even share for five, 1.39 for six,
    // 1.38 for eight); else even ones that fill the device once and a half.
    const int64_t items = (int64_t)a.tiles * a.c.kv_heads * a.batch, step = a.many ? 128 : (a.few ? kFewStep : kStep) * kWaves;
    const int64_t slots = a.many ? cus : cus * (a.few ? (a.c.dim <= 64 ? 4 : a.c.dim <= 128 ? 3 : 2) : a.c.dim <= 64 ? 3 : a.c.dim <= 128 ? 2 : 1);
    a.taper = 3 * items >= slots && items < 4 * slots && keys > 512;
    a.granule = a.taper ? std::max<int64_t>(512, step) : step;
    a.splits = a.taper ? kTaper : std::min({ceil_div(3 * slots, 2 * items), ceil_div(keys, step), (int64_t)kMostParts});
    a.wide = a.rows < 4 * cus;
}

uint64_t part_bytes(const Args &a) { return a.rows && a.splits > 1 ? (uint64_t)a.splits * a.rows * (8 + 4ull * a.c.dim) : 0; }

int make_attention(const df11_quantized_cache *c, const df11_quantized_attention_args *p, Args &a)
{
    const char *who = "df11_quantized_attention";
    if (!p) return df11::fail(DF11_E_ARG, "%s: null arguments", who);
    int rc = make_cache(who, c, p->block_table, p->table_pages, p->table_batch, p->batch, a.c);
    if (rc) return rc;
    if (!within(p->heads, 1, kMost) || p->heads % c->kv_heads)
        return df11::fail(DF11_E_ARG, "%s: %lld heads are no multiple of %lld key heads", who, (long long)p->heads,
                          (long long)c->kv_heads);
    if (!within(p->tokens, 1, 65536) || (double)p->batch * p->tokens * p->heads > kMost)
        return df11::fail(DF11_E_ARG, "%s: batch %lld of %lld tokens out of range", who, (long long)p->batch, (long long)p->tokens);
    if (!strides_ok({p->q_batch, p->q_token, p->q_head}))
        return df11::fail(DF11_E_ARG, "%s: strides must be multiples of 8", who);
    a.q = (const uint16_t *)p->q, a.lengths = p->lengths, a.out = (uint16_t *)p->out, a.lse = p->lse;
    a.batch = p->batch, a.tokens = p->tokens, a.heads = p->heads, a.group = p->heads / c->kv_heads;
    a.q_batch = p->q_batch, a.q_token = p->q_token, a.q_head = p->q_head;
    a.scale2 = (float)(p->scale * 1.44269504088896340736);
    if (!(a.scale2 > 0.0f && a.scale2 < 0x1p126f))   // tile_kernel takes four times that
        return df11::fail(DF11_E_ARG, "%s: scale must be positive and below 2^125", who);
    plan(a);
    return DF11_OK;
}

}  // namespace

extern "C" int df11_quantized_write(const df11_quantized_cache *cache, const df11_quantized_write_args *p, void *stream)
{
    const char *who = "df11_quantized_write";
    if (!p) return df11::fail(DF11_E_ARG, "%s: null arguments", who);
    WriteArgs a{};
    const int rc = make_cache(who, cache, p->block_table, p->table_pages, p->table_batch, p->batch, a.c);
    if (rc) return rc;
    if (!within(p->tokens, 0, kMost)) return df11::fail(DF11_E_ARG, "%s: tokens out of range", who);
    if (!strides_ok({p->k_batch, p->k_token, p->k_head, p->v_batch, p->v_token, p->v_head}))
        return df11::fail(DF11_E_ARG, "%s: strides must be multiples of 8", who);
    if (!p->batch) return DF11_OK;
    const auto on_lengths = [&](const int32_t *x) {
        return x && (uintptr_t)x < (uintptr_t)(p->lengths + p->batch) && (uintptr_t)p->lengths < (uintptr_t)(x + p->batch);
    };
    if ((p->tokens && (!aligned16(p->k) || !aligned16(p->v))) || !p->positions || !p->lengths || on_lengths(p->positions) ||
        on_lengths(p->counts))
        return df11::fail(DF11_E_ARG, "%s: null, misaligned or shared pointer", who);
    const int64_t slots = cache->page;
    if (!pages_apart(cache, cache->code_page, cache->code_head, slots * (a.c.dim / 2)) ||
        !pages_apart(cache, cache->scale_page, cache->scale_head, slots * a.c.groups * 2))
        return df11::fail(DF11_E_ARG, "%s: pages of the cache share memory", who);
    const int64_t pages = cache->pages, heads = cache->kv_heads;
    if (pages && (sets_meet((__int128)(uintptr_t)a.c.v_codes - (uintptr_t)a.c.k_codes, {pages, cache->code_page},
                            {heads, cache->code_head}, slots * (a.c.dim / 2)) ||
                  sets_meet(((__int128)(uintptr_t)a.c.v_scales - (uintptr_t)a.c.k_scales) / 2, {pages, cache->scale_page},
                            {heads, cache->scale_head}, slots * a.c.groups * 2)))
        return df11::fail(DF11_E_ARG, "%s: keys and values of the cache share memory", who);
    a.k = (const uint16_t *)p->k, a.v = (const uint16_t *)p->v;
    a.positions = p->positions, a.counts = p->counts, a.lengths = p->lengths;
    a.batch = p->batch, a.tokens = p->tokens;
    while (a.run < 4 && 2ll << a.run <= p->tokens) a.run++;
    a.k_batch = p->k_batch, a.k_token = p->k_token, a.k_head = p->k_head;
    a.v_batch = p->v_batch, a.v_token = p->v_token, a.v_head = p->v_head;
    int status = DF11_OK;
    by_shape(cache->dtype, a.c.dim, [&](auto e, auto dp) {
        constexpr int DP = decltype(dp)::value;
        const int64_t groups = std::max<int64_t>(1, ceil_div((ceil_div(p->tokens, 1 << a.run) << a.run) * a.c.kv_heads,
                                                                  kMoveThreads / RowLanes<DP>::kLanes));
        if ((double)groups * p->batch > kMostThreads / kMoveThreads) {
            status = df11::fail(DF11_E_ARG, "%s: too many tokens for one launch", who);
            return;
        }
        hipLaunchKernelGGL((write_kernel<decltype(e), DP>), dim3((uint32_t)groups, (uint32_t)p->batch), dim3(kMoveThreads), 0,
                           (hipStream_t)stream, a);
        status = launched(who);
    });
    return status;
}

extern "C" int df11_quantized_read(const df11_quantized_cache *cache, const df11_quantized_read_args *p, void *stream)
{
    const char *who = "df11_quantized_read";
    if (!p) return df11::fail(DF11_E_ARG, "%s: null arguments", who);
    ReadArgs a{};
    const int rc = make_cache(who, cache, p->block_table, p->table_pages, p->table_batch, p->batch, a.c);
    if (rc) return rc;
    if (!within(p->count, 0, kMost)) return df11::fail(DF11_E_ARG, "%s: count out of range", who);
    if (!p->batch || !p->count) return DF11_OK;
    if (!aligned16(p->k) || !aligned16(p->v) || !p->lengths)
        return df11::fail(DF11_E_ARG, "%s: null or misaligned pointer", who);
    const __int128 own = (__int128)p->batch * p->count * a.c.kv_heads * a.c.dim * 2, apart = (__int128)(uintptr_t)p->v - (uintptr_t)p->k;
    if (apart < own && -apart < own) return df11::fail(DF11_E_ARG, "%s: k and v share memory", who);
    a.k = (uint16_t *)p->k, a.v = (uint16_t *)p->v, a.first = p->first, a.lengths = p->lengths;
    a.batch = p->batch, a.count = p->count;
    int status = DF11_OK;
    by_shape(cache->dtype, a.c.dim, [&](auto e, auto dp) {
        constexpr int DP = decltype(dp)::value;
        const int64_t groups = ceil_div(ceil_div(p->count, kReadRows) * a.c.kv_heads, kMoveThreads / (DP / 8));
        if ((double)groups * p->batch > kMostThreads / kMoveThreads) {
            status = df11::fail(DF11_E_ARG, "%s: too many positions for one launch", who);
            return;
        }
        hipLaunchKernelGGL((read_kernel<decltype(e), DP>), dim3((uint32_t)groups, (uint32_t)p->batch), dim3(kMoveThreads), 0,
                           (hipStream_t)stream, a);
        status = launched(who);
    });
    return status;
}

extern "C" uint64_t df11_quantized_attention_workspace_bytes(const df11_quantized_cache *c, const df11_quantized_attention_args *p)
{
    Args a{};
    return make_attention(c, p, a) ? 0 : part_bytes(a);
}

extern "C" int df11_quantized_attention(const df11_quantized_cache *c, const df11_quantized_attention_args *p, void *workspace,
                                        uint64_t workspace_bytes, void *stream)
{
    const char *who = "df11_quantized_attention";
    Args a{};
    const int rc = make_attention(c, p, a);
    if (rc) return rc;
    if (!a.rows) return DF11_OK;
    if (!aligned16(a.q) || !aligned16(a.out) || !a.lengths)
        return df11::fail(DF11_E_ARG, "%s: null or misaligned pointer", who);
    if (out_on_q(a)) return df11::fail(DF11_E_ARG, "%s: out shares memory with q, and is not q itself", who);
    const uint64_t need = part_bytes(a);
    if (workspace_bytes < need || (need && !aligned16(workspace)))
        return df11::fail(DF11_E_ARG, "%s: the workspace must be 16-byte aligned and hold %llu bytes", who,
                          (unsigned long long)need);
    a.part_o = (float *)workspace;
    a.part_ml = (float2 *)(a.part_o + (a.splits > 1 ? (int64_t)a.splits * a.rows * a.c.dim : 0));
    const int64_t items = places(a.tiles, (int64_t)a.batch * a.c.kv_heads * a.splits);
    const int64_t joins = a.splits == 1 ? 0 : a.wide ? a.rows : ceil_div(a.rows, kWaves);
    const int64_t threads = 64 * std::max(kWaves, tile_waves(a.c.dim));   // of a workgroup of any kernel, at most
    if (std::max(items, joins) > kMostThreads / threads)
        return df11::fail(DF11_E_ARG, "%s: too many rows and keys for one launch", who);
    hipStream_t st = (hipStream_t)stream;
    const dim3 block(64 * kWaves);
    by_shape(c->dtype, a.c.dim, [&](auto e, auto dp) {
        typedef decltype(e) E;
        constexpr int DP = decltype(dp)::value;
        const bool even = a.c.dim % (DP / 4) == 0;
        if (a.many && even) hipLaunchKernelGGL((tile_kernel<E, DP, tile_waves(DP), true>), dim3((uint32_t)items), dim3(64 * tile_waves(DP)), 0, st, a);
        else if (a.many) hipLaunchKernelGGL((tile_kernel<E, DP, tile_waves(DP), false>), dim3((uint32_t)items), dim3(64 * tile_waves(DP)), 0, st, a);
        else if (a.few && a.c.dim == DP) hipLaunchKernelGGL((few_kernel<E, DP, true>), dim3((uint32_t)items), block, 0, st, a);
        else if (a.few) hipLaunchKernelGGL((few_kernel<E, DP, false>), dim3((uint32_t)items), block, 0, st, a);
        else if (even) hipLaunchKernelGGL((attend_kernel<E, DP, true>), dim3((uint32_t)items), block, 0, st, a);
        else hipLaunchKernelGGL((attend_kernel<E, DP, false>), dim3((uint32_t)items), block, 0, st, a);
        if (!joins) return;
        if (a.wide) hipLaunchKernelGGL((join_kernel<E, true>), dim3((uint32_t)joins), block, 0, st, a);
        else hipLaunchKernelGGL((join_kernel<E, false>), dim3((uint32_t)joins), block, 0, st, a);
    });
    return launched(who);
}
