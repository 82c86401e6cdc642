// Attention of a generation step: over a prefix that a batch of sequences
// shares (df11_prefix_attention) and over a bounded cache whose slots add up
// the attention they get (df11_cache_attention).
//
// For a row q (one query token of one head) and its keys K_j, values V_j:
//   s_j = scale * q . K_j,   o = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m),
// taken in one pass with the running maximum m and the running sum l: a new
// maximum m' scales the sums so far by exp(m - m').  A range of keys thus
// gives (m, l, o) on its own, and ranges are joined the same way, so the
// keys are split over workgroups and over a workgroup's waves.  Logarithms
// are to base 2: exp(x) = 2^(x log2 e) is one instruction.
//
// Logits, maxima, sums and outputs are float32.  The probabilities are
// rounded to the operands' type (to nearest) for the product with V, since
// the matrix cores take both operands in one type; their sum is taken before
// that, so lse and weights keep float32 accuracy, and the outputs' error is
// 1.1 to 1.4 times that of their own rounding.  A float16 probability keeps
// its 11 bits down to 2^-21 of the row's greatest so far and is gone below 2^-32
// (kLift; without it 2^-14 and 2^-25: 31 keys of 2^-24.6 beside one of 1 gave
// half as much again as they should); a bfloat16 one keeps its 8 throughout.
//
// attend_wave: one wave, 16 rows, 32 keys at a time, no LDS.
//   S^T = K Q^T  v_mfma_f32_16x16x32: the A operand of lane l is key l % 16,
//                dims 8 * (4 i + l / 16) .. + 7 of step i, as they lie in
//                memory; the B operand the same dims of row l % 16.
//   P^T          lane l holds row l % 16 and the keys 4 (l / 16) + 0..3 of
//                each of two 16-key tiles: 8 keys, just the B operand of one
//                32-key step of
//   O^T = V^T P^T  whose A operand wants, for one dim, those 8 keys side by
//                side.  Each lane loads its 8 keys' dims (l % 16) W .. + W - 1
//                (W = dims / 16; a wave reads whole rows of V) and turns the
//                8 x W block in registers (v_perm_b32); product j of the W
//                takes the dims j, W + j, 2 W + j, ...
// Bound by HBM: at 16 rows a step of 32 keys is 16 KB (128 dims) for 32
// products of 16 cycles.  Registers instead of LDS leave no barrier between a
// load and its product; eight waves a CU keep 64 to 128 KB on their way.  33
// requests of 4099 slots of 64 dims: 92 us, 4.7 TB/s (a device copy: 5.2).
#include <algorithm>
#include <cmath>

#include "df11_internal.h"
#include "serve_device.h"

namespace {

using namespace df11serve;

constexpr int kWaves = 4;      // waves of a workgroup, each on every fourth run of 32 keys
constexpr int kRows = 16;      // rows of a tile
constexpr int kStep = 32;      // keys of a step

// What a launch's workgroups do: a prefix in 16-row tiles, or in 128-row
// tiles (both with the sequences' own positions), or bounded caches in tiles
// of 16 or of 128 rows.
enum { kRowTiles, kTiles, kCache, kCacheTiles };

struct Args {
    const uint16_t *q, *prefix_k, *prefix_v, *k, *v;
    const int32_t *lengths, *table, *pos, *positions;
    uint16_t *out;             // NULL: only the rows' logarithms are wanted
    float *lse, *weights;
    float *part_o;             // [slot][row][dim]
    float2 *part_ml;           // [slot][row]
    float *tops;               // many rows of a cache: a row's logarithm (base 2) of its sum, +infinity if it is empty
    float *logits;             // few rows: [batch * kv_heads][rows of a head][logit_stride]
    int32_t batch, tokens, heads, kv_heads, group, dim, prefix, suffix, page, n_pages;
    int64_t q_batch, q_token, q_head, prefix_token, prefix_head, k_batch, k_token, k_head, table_batch;
    int64_t logit_stride;
    float scale2;              // scale * log2(e)
    int32_t prefix_splits, prefix_span, prefix_tiles, suffix_splits, suffix_span, suffix_tiles;
    int64_t prefix_places;     // workgroups of the prefix
    int64_t rows;              // batch * tokens * heads
    int32_t weigh_run;         // many rows: slots of a workgroup that weighs
    bool big;                  // tiles of 128 rows
    bool four;                 // four output rows to a joining workgroup
    bool out_on_q;             // out shares memory with q
};

// Workgroups i and i + 8 run on one of the eight dies, which has an L2 of its
// own: the row tiles that read the same keys and values follow each other
// there, and the dies get the ranges of all lengths alike (with neighbouring
// workgroups on neighbouring ranges of one sequence, two or four ranges left
// dies idle: 528 items of 2050 to 4099 keys 121 and 113 us, 100 so).
__device__ __forceinline__ bool place(int i, int tiles, int pairs, int &tile, int &pair)
{
    tile = i / 8 % tiles;
    pair = i % 8 + i / 8 / tiles * 8;
    return pair < pairs;
}
int64_t places(int64_t tiles, int64_t pairs) { return (pairs + 7) / 8 * 8 * tiles; }

// The 32 keys from `base` on: rows in memory, and which of them which query
// tokens see.  Lane l speaks for key base + l % 32: rel is the key's place
// relative to the first query token (token t sees it when rel <= t).
struct Keys {
    uint32_t any, all;   // keys that some / every query token sees
    int32_t rel;
    int64_t half[2];     // element offset of the first key of each half, if the halves' rows are evenly spaced
    int64_t row;         // of lane l % 32's key, if they are not
};

// What has to come from memory before the keys of a step are known: a
// source's fetch() starts it two steps ahead, its keys() uses it.
struct Ahead {
    int32_t x, y;
};

struct PrefixSource {
    const uint16_t *k, *v;
    int64_t token;
    int32_t n;
    static constexpr bool kEven = true;
    __device__ __forceinline__ Ahead fetch(int, int) const { return Ahead{0, 0}; }
    __device__ __forceinline__ Keys keys(Ahead, int base, int) const
    {
        const int left = n - base;
        const uint32_t m = left >= 32 ? 0xffffffffu : (1u << left) - 1;
        return Keys{m, m, 0, {base * token, (base + 16) * token}, 0};
    }
    __device__ __forceinline__ void logits(int, int, int, f32x4) const {}
};

// EVEN: rows in place, or pages of a multiple of 16 positions.
template <bool EVEN>
struct SuffixSource {
    const uint16_t *k, *v;
    const int32_t *table;
    int64_t batch, token;
    int32_t n, tokens, page, n_pages;
    static constexpr bool kEven = EVEN;
    __device__ __forceinline__ Ahead fetch(int base, int lane) const
    {
        if (EVEN) {
            if (!table) return Ahead{0, 0};
            const int last = (n - 1) / page;
            return Ahead{table[min(base / page, last)], table[min((base + 16) / page, last)]};
        }
        return Ahead{table[min(base + (lane & 31), n - 1) / page], 0};
    }
    __device__ __forceinline__ Keys keys(Ahead id, int base, int lane) const
    {
        const int key = base + (lane & 31);
        const int32_t rel = key - (n - tokens);
        bool there = key < n;
        Keys m;
        m.row = 0;
        if (EVEN) {
            m.half[0] = base * token, m.half[1] = (base + 16) * token;
            if (table) {
                const bool in0 = id.x >= 0 && id.x < n_pages, in1 = id.y >= 0 && id.y < n_pages;
                there = there && (lane & 16 ? in1 : in0);
                m.half[0] = (in0 ? id.x : 0) * batch + (base % page) * token;
                m.half[1] = (in1 ? id.y : 0) * batch + ((base + 16) % page) * token;
            }
        } else {
            there = there && id.x >= 0 && id.x < n_pages;
            m.half[0] = m.half[1] = 0;
            m.row = (there ? id.x : 0) * batch + (min(key, n - 1) % page) * token;
        }
        m.any = (uint32_t)__ballot(there), m.all = (uint32_t)__ballot(there && rel <= 0);
        m.rel = rel;
        return m;
    }
    __device__ __forceinline__ void logits(int, int, int, f32x4) const {}
};

struct CacheSource {
    const uint16_t *k, *v;
    const int32_t *positions;
    float *out;          // this row tile's logits
    int64_t token, stride;
    int32_t n, tokens, pos, row_count;
    static constexpr bool kEven = true;
    __device__ __forceinline__ Ahead fetch(int base, int lane) const
    {
        return Ahead{positions[min(base + (lane & 31), n - 1)], 0};
    }
    __device__ __forceinline__ Keys keys(Ahead at, int base, int lane) const
    {
        const bool some = base + (lane & 31) < n && at.x >= 0 && (int64_t)at.x <= (int64_t)pos + tokens - 1;
        const int32_t rel = some ? at.x - pos : 0x7fffffff;
        return Keys{(uint32_t)__ballot(some), (uint32_t)__ballot(some && rel <= 0), rel,
                    {base * token, (base + 16) * token}, 0};
    }
    // the logits of row `row`, keys key .. key + 3
    __device__ __forceinline__ void logits(int base, int row, int key, f32x4 s) const
    {
        if (row < row_count) *(f32x4 *)(out + row * stride + base + key) = s;
    }
};

// One wave over the keys [key0, key1) of `src`, every `step`-th run of 32.
// q: this lane's row as B operands; t: its query token.  o[j][r] is, for row
// lane % 16, dim (4 (lane / 16) + r) * W + j of the sum; m and l its maximum
// and its sum over this lane's keys.  The next step's keys are on their way
// while a step's softmax and second product run, its values from behind that
// product on.
template <class E, int DP, class Src>
__device__ __forceinline__ void attend_wave(const Src &src, const u32x4 (&q)[DP / 32], int t, int tokens, int dim,
                                            int key0, int key1, int step, float scale2, f32x4 (&o)[DP / 16], float &m,
                                            float &l)
{
    constexpr int W = DP / 16;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int j = 0; j < W; j++) o[j] = f32x4{0, 0, 0, 0};
    if (key0 >= key1) return;

    u32x4 kx[2][DP / 32];
    uint32_t vx[8][W / 2];
    // Rows are at a uniform address plus a lane's 32-bit distance: row i of a
    // half, held back to the last row there is.
    const auto load_k = [&](const Keys &keys, int base) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint16_t *from;
            if (Src::kEven) {
                const int most = src.n - 1 - (base + 16 * h);
                from = src.k + (most < 0 ? keys.half[0] : keys.half[h]) +
                       (uint32_t)(max(0, min(c, most)) * (int32_t)src.token);
            } else {
                from = src.k + __shfl(keys.row, 16 * h + c);
            }
#pragma unroll
            for (int i = 0; i < DP / 32; i++) {
                const int d = 8 * (4 * i + g);
                kx[h][i] = DP == dim || d < dim ? *(const u32x4 *)(from + d) : u32x4{0, 0, 0, 0};
            }
        }
    };
    const int vd = min(c * W, dim - (W < 8 ? W : 8));   // a lane past the last dim reads any: its sums go nowhere
    const auto load_v = [&](const Keys &keys, int base) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int h = j >> 2, i = 4 * g + (j & 3);
            const uint16_t *from;
            if (Src::kEven) {
                const int most = src.n - 1 - (base + 16 * h);
                from = src.v + (most < 0 ? keys.half[0] : keys.half[h]) +
                       (uint32_t)(max(0, min(i, most)) * (int32_t)src.token);
            } else {
                from = src.v + __shfl(keys.row, 16 * h + i);
            }
            if constexpr (W == 4) {
                const u32x2 x = *(const u32x2 *)(from + vd);
                vx[j][0] = x[0], vx[j][1] = x[1];
            } else {
#pragma unroll
                for (int w = 0; w < W / 8; w++) {
                    const u32x4 x = *(const u32x4 *)(from + min(vd + 8 * w, dim - 8));
#pragma unroll
                    for (int y = 0; y < 4; y++) vx[j][4 * w + y] = x[y];
                }
            }
        }
    };

    Keys keys = src.keys(src.fetch(key0, lane), key0, lane);
    Ahead ahead = src.fetch(min(key0 + step, key1 - 1) & ~31, lane);
    load_k(keys, key0);
    load_v(keys, key0);
    for (int base = key0; base < key1; base += step) {
        const int next = base + step;
        f32x4 s[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            s[h] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < DP / 32; i++) s[h] = E::mfma16(kx[h][i], q[i], s[h]);
        }
        Keys then = keys;
        if (next < key1) {
            then = src.keys(ahead, next, lane);
            ahead = src.fetch(min(next + step, key1 - 1) & ~31, lane);
            load_k(then, next);
        }
        const bool plain = keys.any == keys.all;   // uniform
        float mx = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int i = 16 * h + 4 * g + r;
                bool sees = (keys.any >> i) & 1;
                if (!plain) {
                    const int32_t rel = __shfl(keys.rel, i);   // of every lane's key, seen or not
                    sees = sees && rel <= t;
                }
                s[h][r] = sees ? s[h][r] * scale2 : -INFINITY;
                mx = fmaxf(mx, s[h][r]);
            }
            src.logits(base, c, 16 * h + 4 * g, s[h]);
        }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        // m is kLift below the running maximum, which is raised only past 2^8
        // times itself: a probability of up to 2^(8 + kLift) is no less exact,
        // and the sums are seldom scaled.
        const float low = mx - E::kLift;
        const bool raise = low > m + 8.0f;
        if (__any(raise)) {
            const float f = raise ? exp2_fast(m - low) : 1.0f;
            m = raise ? low : m;
            l *= f;
#pragma unroll
            for (int j = 0; j < W; j++) o[j] *= f;
        }
        const float safe = m == -INFINITY ? 0.0f : m;
        u32x4 pb;
#pragma unroll
        for (int w = 0; w < 4; w++) {
            const float x = exp2_fast(s[w / 2][2 * (w & 1)] - safe), y = exp2_fast(s[w / 2][2 * (w & 1) + 1] - safe);
            l += x + y;
            pb[w] = E::pack(x, y);
        }
        // a key that no row of the tile sees takes part with weight 0: its
        // value must be a number
        if (keys.any != 0xffffffffu) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const bool sees = (keys.any >> (16 * (j >> 2) + 4 * g + (j & 3))) & 1;
#pragma unroll
                for (int w = 0; w < W / 2; w++) vx[j][w] = sees ? vx[j][w] : 0;
            }
        }
        // The rows of different query tokens may see different keys.  A
        // number times weight 0 is 0; only where a value that some rows must
        // not see is not a number, the tokens take turns, each with its
        // unseen keys cleared and the sums of its own rows kept.
        bool odd = false;
        if (!plain) {
#pragma unroll
            for (int j = 0; j < 8; j++)
#pragma unroll
                for (int w = 0; w < W / 2; w++)
                    odd = odd || (vx[j][w] & E::kExpMask) == E::kExpMask ||
                          ((vx[j][w] >> 16) & E::kExpMask) == E::kExpMask;
        }
        if (!plain && __any(odd)) {
            for (int turn = 0; turn < tokens; turn++) {
#pragma unroll
                for (int j = 0; j < W; j++) {
                    u32x4 va;
#pragma unroll
                    for (int w = 0; w < 4; w++) {
                        const int i = 16 * (w >> 1) + 4 * g + 2 * (w & 1);
                        const int32_t rel_lo = __shfl(keys.rel, i), rel_hi = __shfl(keys.rel, i + 1);
                        const uint32_t lo = rel_lo <= turn ? vx[2 * w][j / 2] : 0;
                        const uint32_t hi = rel_hi <= turn ? vx[2 * w + 1][j / 2] : 0;
                        va[w] = __builtin_amdgcn_perm(hi, lo, j & 1 ? 0x07060302u : 0x05040100u);
                    }
                    const f32x4 sum = E::mfma16(va, pb, o[j]);
#pragma unroll
                    for (int r = 0; r < 4; r++) o[j][r] = t == turn ? sum[r] : o[j][r];
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; j++) {
                u32x4 va;
#pragma unroll
                for (int w = 0; w < 4; w++)
                    va[w] = __builtin_amdgcn_perm(vx[2 * w + 1][j / 2], vx[2 * w][j / 2], j & 1 ? 0x07060302u : 0x05040100u);
                o[j] = E::mfma16(va, pb, o[j]);
            }
        }
        if (next < key1) load_v(then, next);
        keys = then;
    }
}

// A tile of 128 rows over a range of keys, by a workgroup: each wave has 32
// rows, all share the keys and values in LDS, kKeys of them at a time while
// the next ones are on their way from memory.
//   S^T = K Q^T    v_mfma_f32_32x32x16: the A operand of lane l is key l % 32,
//                  dims 16 i + 8 (l / 32) .. + 7 of step i, the B operand the
//                  same dims of row l % 32.
//   O^T = V^T P^T  lane l's logits belong to row l % 32 and the keys
//                  8 (r / 4) + 4 (l / 32) + r % 4: eight of them are the B
//                  operand of a step of 16 keys, so V is laid out in LDS with
//                  those eight keys of a dim side by side (turned in registers
//                  on its way there).
// LDS: K rows of DP dims and V^T rows of kKeys keys, in 16-byte chunks whose
// place in the row is exchanged by row so that neighbouring rows lie in
// different banks (k_at, v_at).
// 32 rows a wave: a wave's operands from LDS are as many cycles as its
// products, and 64 rows would leave one wave a SIMD (its sums alone 128
// registers).  128 requests behind 32768 positions, 70 GFLOP: 90 us, 785
// TFLOP/s; matrix cores are busy 40% of the time, the vector ALU 45% and LDS
// 37%, one phase of a step mostly behind the other.
constexpr int kTileRows = 32 * kWaves;

// Rows up to this many elements apart go into 128-row tiles: a lane's distance
// spans up to 124 of them (dims to 64) in a 32-bit number.  16-row tiles, whose
// lanes span 15, take the others.
constexpr int64_t kTileStride = 1ll << 25;

template <int DP>
struct TileShape {
    static constexpr int kKeys = 8192 / DP;          // keys of a step: 16 KB of K and of V
    static constexpr int kChunks = DP / 8;           // 16-byte chunks of a K row
    static constexpr int kKeyChunks = kKeys / 8;     // of a V^T row
    static constexpr int kBuffer = 2 * kKeys * DP * 2;
    static __device__ __forceinline__ int k_at(int key, int chunk)
    {
        const int x = DP == 64 ? (key >> 1) & 7 : key & 15;
        return key * DP * 2 + (chunk ^ x) * 16;
    }
    static __device__ __forceinline__ int v_at(int d, int chunk)
    {
        const int x = DP == 64 ? (d ^ (d >> 4)) & 15 : DP == 128 ? ((d >> 1) ^ (d >> 4)) & 7 : ((d >> 2) ^ (d >> 4)) & 3;
        return kKeys * DP * 2 + d * kKeys * 2 + (chunk ^ x) * 16;
    }
    // The same places by exclusive or with one lane's first one: chunk + 2 i
    // of a K row (chunk < 2); dim d + i, i < 8, of V^T (d a multiple of 8);
    // dim d + 32 i and chunk + 2 j of V^T (d < 32, chunk < 2).
    static __device__ __forceinline__ int k_next(int first, int i) { return first ^ (2 * i * 16); }
    static __device__ __forceinline__ int v_next_dim(int first, int i)
    {
        return (first ^ ((DP == 64 ? i : DP == 128 ? i / 2 : i / 4) * 16)) + i * kKeys * 2;
    }
    static __device__ __forceinline__ int v_next(int first, int i, int j)
    {
        return (first ^ (((i ^ j) & (kKeyChunks / 2 - 1)) * 32)) + 32 * i * kKeys * 2;
    }
};

//
// CACHE: the rows are one sequence's and the keys its cache's slots, each
// with its place relative to the first query token (rel, as in Keys) in LDS
// beside its key.
template <class E, int DP, bool CACHE>
__device__ __forceinline__ void tile_block(const Args &a, char *lds, int seq, int head, int tile, int split)
{
    typedef TileShape<DP> S;
    constexpr int kKeys = S::kKeys;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 31, g = lane >> 5;
    const int row_count = (CACHE ? 1 : a.batch) * a.tokens * a.group;
    const int n = CACHE ? max(0, min(a.lengths[seq], a.suffix)) : a.prefix;
    const int span = CACHE ? a.suffix_span : a.prefix_span;
    const int key0 = split * span, key1 = min(n, key0 + span);
    if (key0 >= key1) return;
    const int64_t kv_token = CACHE ? a.k_token : a.prefix_token;
    const int64_t kv_from = CACHE ? seq * a.k_batch + head * a.k_head : head * a.prefix_head;
    const uint16_t *kp = (CACHE ? a.k : a.prefix_k) + kv_from, *vp = (CACHE ? a.v : a.prefix_v) + kv_from;
    const int32_t *places = CACHE ? a.positions + ((int64_t)seq * a.kv_heads + head) * a.suffix : nullptr;
    const int pos = CACHE ? a.pos[seq] : 0;
    // behind the two buffers: rel of each buffer's keys; whether a step has
    // keys that not all tokens see (for three steps in turn); whether any of
    // those had values that are no numbers
    int32_t *const rels = (int32_t *)(lds + 2 * S::kBuffer);
    int32_t *const mixed = rels + 2 * kKeys, *const odd = mixed + 3;
    if (CACHE) {
        if (threadIdx.x < 4) mixed[threadIdx.x] = 0;
        __syncthreads();
    }

    const int row = tile * kTileRows + wave * 32 + c;
    const int t = row / a.group % a.tokens, h = head * a.group + row % a.group;
    const int b = CACHE ? seq : row / (a.group * a.tokens);
    u32x4 q[DP / 16];
#pragma unroll
    for (int i = 0; i < DP / 16; i++) {
        const int d = 16 * i + 8 * g;
        q[i] = row < row_count && d < a.dim
                   ? *(const u32x4 *)(a.q + b * a.q_batch + t * a.q_token + h * a.q_head + d)
                   : u32x4{0, 0, 0, 0};
    }
    // What a thread brings: four chunks of K, and four keys by 8 dims of V,
    // at a uniform address plus its own 32-bit distance.
    u32x4 kx[4], vx[4];
    const int v_quad = threadIdx.x / S::kChunks, v_chunk = threadIdx.x % S::kChunks;
    const uint32_t token = (uint32_t)kv_token;
    int32_t place[4];
    const int my_d = v_chunk * 8 < a.dim ? v_chunk * 8 : 0;
    const bool pad = v_chunk * 8 >= a.dim;   // dims that K does not have take part as 0
    const uint32_t k_far = v_quad * token + my_d, v_far = 4 * v_quad * token + my_d;   // below 2^32: kTileStride
    constexpr int kRowsEach = 256 / S::kChunks;   // keys between a thread's chunks of K
    const auto load = [&](int base) {
        if (base + kKeys <= key1) {
            const uint16_t *k = kp + base * kv_token, *v = vp + base * kv_token;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                kx[j] = *(const u32x4 *)(k + (int64_t)(kRowsEach * j) * kv_token + k_far);
                vx[j] = *(const u32x4 *)(v + j * kv_token + v_far);
                if (CACHE) place[j] = places[base + 4 * v_quad + j];
            }
        } else {
            // the last step: keys past the end are 0
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int kk = base + kRowsEach * j + v_quad, kv = base + 4 * v_quad + j;
                const u32x4 x = *(const u32x4 *)(kp + min(kk, n - 1) * kv_token + my_d);
                const u32x4 y = *(const u32x4 *)(vp + min(kv, n - 1) * kv_token + my_d);
#pragma unroll
                for (int w = 0; w < 4; w++) kx[j][w] = kk < key1 ? x[w] : 0, vx[j][w] = kv < key1 ? y[w] : 0;
                if (CACHE) place[j] = kv < key1 ? places[kv] : -1;
            }
        }
    };
    const int k_to = S::k_at(v_quad, v_chunk);
    // keys 4 w .. 4 w + 3 of a group of 16: half w / 2 of the chunk of lanes l / 32 = w % 2
    const int v_to = S::v_at(v_chunk * 8, v_quad / 4 * 2 + (v_quad & 1)) + (v_quad >> 1 & 1) * 8;
    const auto store = [&](int buffer, int turn) {
        if (CACHE) {
            int32_t rel[4];
            bool some_not = false, no_number = false;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const bool some = place[j] >= 0 && (int64_t)place[j] <= (int64_t)pos + a.tokens - 1;
                rel[j] = some ? place[j] - pos : 0x7fffffff;
                some_not = some_not || rel[j] > 0;
            }
            // A value that a row does not see has weight 0 there, so it must
            // be a number: those that no token sees are 0; those that some
            // see are too, if they are no numbers, and come last (below).
            if (some_not) {
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int w = 0; w < 4; w++) {
                        const uint32_t x = vx[j][w];
                        const bool low = (x & E::kExpMask) == E::kExpMask, high = (x >> 16 & E::kExpMask) == E::kExpMask;
                        no_number = no_number || (rel[j] > 0 && rel[j] < a.tokens && (low || high));
                        vx[j][w] = rel[j] >= a.tokens ? 0
                                   : rel[j] <= 0      ? x
                                                      : (low ? 0 : x & 0xffffu) | (high ? 0 : x & 0xffff0000u);
                    }
                mixed[turn] = 1;
                if (no_number) *odd = 1;
            }
            if (v_chunk == 0)
#pragma unroll
                for (int j = 0; j < 4; j++) rels[(buffer ? kKeys : 0) + 4 * v_quad + j] = rel[j];
            const int then = turn == 2 ? 0 : turn + 1;
            if (threadIdx.x == 0) mixed[then] = 0;
        }
        if (a.dim < DP) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int w = 0; w < 4; w++) kx[j][w] = pad ? 0 : kx[j][w];
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            // rows a multiple of 16 apart exchange their chunks alike
            if (DP < 256) *(u32x4 *)(lds + k_to + buffer + j * kRowsEach * DP * 2) = kx[j];
            else *(u32x4 *)(lds + buffer + S::k_at(v_quad + kRowsEach * j, v_chunk)) = kx[j];
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t sel = i & 1 ? 0x07060302u : 0x05040100u;
            const u32x2 x{__builtin_amdgcn_perm(vx[1][i / 2], vx[0][i / 2], sel),
                          __builtin_amdgcn_perm(vx[3][i / 2], vx[2][i / 2], sel)};
            *(u32x2 *)(lds + buffer + S::v_next_dim(v_to, i)) = x;
        }
    };

    f32x16 o[DP / 32];
#pragma unroll
    for (int i = 0; i < DP / 32; i++)
#pragma unroll
        for (int r = 0; r < 16; r++) o[i][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    // A step's operands in the order of its products: the K rows, each 32 keys
    // in turn, then the V^T rows of each 16 keys; kAhead of them are on their way.
    constexpr int kK = DP / 16, kParts = kKeys / 32, kV = 2 * (DP / 32), kFrags = kParts * (kK + kV), kAhead = 4;
    const int k_from = S::k_at(c, g), v_from = S::v_at(c, g);
    const auto frag = [&](int buffer, int i) {
        int at;
        if (i < kParts * kK) {
            at = S::k_next(k_from, i / kParts) + 32 * (i % kParts) * DP * 2;
        } else {
            i -= kParts * kK;
            at = S::v_next(v_from, i % (DP / 32), i / (DP / 32));
        }
        return *(const u32x4 *)(lds + buffer + at);
    };
    const auto step = [&](int buffer, int left, int turn) {
        const bool some_not = CACHE && __builtin_amdgcn_readfirstlane(mixed[turn]);
        const int32_t *const rel = rels + (buffer ? kKeys : 0);
        f32x16 s[kParts];
        u32x4 f[kFrags];
#pragma unroll
        for (int i = 0; i < kAhead; i++) f[i] = frag(buffer, i);
#pragma unroll
        for (int k = 0; k < kParts; k++)
#pragma unroll
            for (int r = 0; r < 16; r++) s[k][r] = 0.0f;
#pragma unroll
        for (int i = 0; i < kParts * kK; i++) {
            f[i + kAhead] = frag(buffer, i + kAhead);
            s[i % kParts] = E::mfma32(f[i], q[i / kParts], s[i % kParts]);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int i = 0; i < kParts * kK; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        if (some_not) {
#pragma unroll
            for (int k = 0; k < kParts; k++)
#pragma unroll
                for (int r = 0; r < 16; r++)
                    if (rel[32 * k + 8 * (r / 4) + 4 * g + r % 4] > t) s[k][r] = -INFINITY;
        }
        if (!CACHE && left < kKeys) {
            __builtin_amdgcn_sched_barrier(0);   // a branch of its own: no step but the last pays for it
#pragma unroll
            for (int k = 0; k < kParts; k++)
#pragma unroll
                for (int r = 0; r < 16; r++)
                    if (32 * k + 8 * (r / 4) + 4 * g + r % 4 >= left) s[k][r] = -INFINITY;
        }
        float mx = s[0][0];
#pragma unroll
        for (int k = 0; k < kParts; k++)
#pragma unroll
            for (int r = 0; r < 16; r++) mx = fmaxf(mx, s[k][r]);
        mx = fmaxf(mx, __shfl_xor(mx, 32)) * a.scale2;
        const float low = mx - E::kLift;   // as in attend_wave
        const bool raise = low > m + 8.0f;
        if (__any(raise)) {
            const float by = raise ? exp2_fast(m - low) : 1.0f;
            m = raise ? low : m;
            l *= by;
#pragma unroll
            for (int i = 0; i < DP / 32; i++) o[i] *= by;
        }
        const float safe = m == -INFINITY ? 0.0f : m;
        const auto weigh = [&](int k, int half) {
            u32x4 pb;
#pragma unroll
            for (int w = 0; w < 4; w++) {
                const float x = exp2_fast(__builtin_fmaf(s[k][8 * half + 2 * w], a.scale2, -safe));
                const float y = exp2_fast(__builtin_fmaf(s[k][8 * half + 2 * w + 1], a.scale2, -safe));
                l += x + y;
                pb[w] = E::pack(x, y);
            }
            return pb;
        };
#pragma unroll
        for (int k = 0; k < kParts; k++)
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const u32x4 pb = weigh(k, half);
#pragma unroll
                for (int i = 0; i < DP / 32; i++) {
                    const int at = kParts * kK + (2 * k + half) * (DP / 32) + i;
                    if (at + kAhead < kFrags) f[at + kAhead] = frag(buffer, at + kAhead);
                    o[i] = E::mfma32(f[at], pb, o[i]);
                }
            }
        __builtin_amdgcn_sched_group_barrier(0x402, 8 * 2 + 4, 0);
#pragma unroll
        for (int i = 0; i < kFrags - kParts * kK; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (i < kFrags - kParts * kK - kAhead) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x402, 7, 0);
        }
    };

    load(key0);
    store(0, 0);
    __syncthreads();
    int turn = 0;
    for (int base = key0; base < key1; base += 2 * kKeys) {
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int at = base + half * kKeys;
            if (at >= key1) break;
            const bool more = at + kKeys < key1;
            if (more) load(at + kKeys);
            step(half * S::kBuffer, key1 - at, turn);
            turn = turn == 2 ? 0 : turn + 1;
            if (more) store((1 - half) * S::kBuffer, turn);
            __syncthreads();
        }
    }
    if (CACHE && *odd) {
        // What was left out: each value that is no number and that only some
        // tokens see, times its weight for the rows that do.
        for (int base = key0; base < key1; base += 64) {
            const int32_t at = base + lane < key1 ? places[base + lane] : -1;
            // only where some tokens see it: at - pos of any other need not fit 32 bits
            const int32_t rel = at > pos && (int64_t)at < (int64_t)pos + a.tokens && at >= 0 ? at - pos : 0;
            for (uint64_t left = __ballot(rel > 0); left; left &= left - 1) {
                const int i = __builtin_ctzll(left);
                const uint16_t *kr = kp + (base + i) * kv_token, *vr = vp + (base + i) * kv_token;
                float x = 0.0f;
#pragma unroll
                for (int j = 0; j < DP / 16; j++)
#pragma unroll
                    for (int w = 0; w < 8; w++) {
                        const int d = 16 * j + 8 * g + w;
                        const uint32_t y = q[j][w / 2];
                        if (d < a.dim) x += E::value(w & 1 ? y >> 16 : y & 0xffffu) * E::value(kr[d]);
                    }
                x += __shfl_xor(x, 32);
                const bool sees = __shfl(rel, i) <= t;
                const float p = exp2_fast(x * a.scale2 - (m == -INFINITY ? 0.0f : m));
#pragma unroll
                for (int j = 0; j < DP / 32; j++)
#pragma unroll
                    for (int r = 0; r < 16; r++) {
                        const int d = 32 * j + 8 * (r / 4) + 4 * g + r % 4;
                        const uint32_t y = d < a.dim ? vr[d] : 0;
                        if (sees && (y & E::kExpMask) == E::kExpMask) o[j][r] += p * E::value(y);
                    }
            }
        }
    }
    l += __shfl_xor(l, 32);
    if (row < row_count) {
        const int64_t out_row = ((int64_t)b * a.tokens + t) * a.heads + h;   // (caches have no prefix ranges before theirs)
        float *to = a.part_o + (split * a.rows + out_row) * a.dim;
#pragma unroll
        for (int i = 0; i < DP / 32; i++)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int d = 32 * i + 2 * r + 4 * g;
                if (d < a.dim) *(f32x4 *)(to + d) = f32x4{o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]};
            }
        if (g == 0) a.part_ml[split * a.rows + out_row] = make_float2(m, l);
    }
}

// One workgroup: a tile of 16 rows over one range of keys.  Workgroups below
// the prefix count take a tile of all sequences' rows of one key head over a
// range of the prefix, the others a tile of one sequence's rows of one key
// head over a range of its own positions (or of its cache).
template <class E, int DP, int KIND>
__global__ void __launch_bounds__(64 * kWaves, DP == 256 ? 1 : 2) attend_kernel(const Args a)
{
    constexpr bool CACHE = KIND == kCache;
    constexpr int W = DP / 16;
    typedef float JoinO[kRows][DP + 4];
    typedef float2 JoinMl[kRows];
    constexpr int kJoin = kWaves * (sizeof(JoinO) + sizeof(JoinMl));
    constexpr int kTile = 2 * TileShape<DP>::kBuffer + (KIND == kCacheTiles ? 8 * TileShape<DP>::kKeys + 16 : 0);
    constexpr int kLds = KIND == kTiles ? (kTile > kJoin ? kTile : kJoin) : KIND == kCacheTiles ? kTile : kJoin;
    __shared__ alignas(1024) char lds[kLds];
    if constexpr (KIND == kCacheTiles) {
        int tile, pair;
        const int own = a.batch * a.kv_heads;
        if (!place(blockIdx.x, a.suffix_tiles, own * a.suffix_splits, tile, pair)) return;
        tile_block<E, DP, true>(a, lds, pair % own / a.kv_heads, pair % a.kv_heads, tile, pair / own);
        return;
    }
    JoinO *const join_o = (JoinO *)lds;
    JoinMl *const join_ml = (JoinMl *)(lds + kWaves * sizeof(JoinO));
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    int tile, pair, b = 0;
    const bool in_prefix = !CACHE && blockIdx.x < a.prefix_places;
    if (in_prefix) {
        if (!place(blockIdx.x, a.prefix_tiles, a.kv_heads * a.prefix_splits, tile, pair)) return;
    } else {
        if (!place(blockIdx.x - (int)a.prefix_places, a.suffix_tiles, a.batch * a.kv_heads * a.suffix_splits, tile, pair)) return;
    }
    const int head = pair % a.kv_heads;
    int split = pair / a.kv_heads;
    if (!in_prefix) b = split % a.batch, split /= a.batch;
    if constexpr (KIND == kTiles) {
        if (in_prefix) {
            tile_block<E, DP, false>(a, lds, 0, head, tile, split);
            return;
        }
    }
    const int row_count = (in_prefix ? a.batch : 1) * a.tokens * a.group;
    const int span = in_prefix ? a.prefix_span : a.suffix_span;
    const int n = in_prefix ? a.prefix : max(0, min(a.lengths[b], a.suffix));
    const int key0 = split * span, key1 = min(n, key0 + span);
    if (key0 >= key1) return;   // the join knows from n that there is no such range

    // row r of a tile: sequence, query token, head of the group
    const int row = tile * kRows + c;
    const int t = row / a.group % a.tokens;
    const int rb = in_prefix ? row / (a.group * a.tokens) : b;
    const int h = head * a.group + row % a.group;
    u32x4 q[DP / 32];
#pragma unroll
    for (int i = 0; i < DP / 32; i++) {
        const int d = 8 * (4 * i + g);
        q[i] = row < row_count && d < a.dim
                   ? *(const u32x4 *)(a.q + rb * a.q_batch + t * a.q_token + h * a.q_head + d)
                   : u32x4{0, 0, 0, 0};
    }
    f32x4 o[W];
    float m, l;
    const int first = key0 + kStep * wave;
    if constexpr (CACHE) {
        const int64_t bh = (int64_t)b * a.kv_heads + head;
        const int64_t at = b * a.k_batch + head * a.k_head;
        const CacheSource src{a.k + at, a.v + at, a.positions + bh * a.suffix,
                              a.logits + (bh * row_count + tile * kRows) * a.logit_stride, a.k_token, a.logit_stride, n,
                              a.tokens, a.pos[b], row_count - tile * kRows};
        attend_wave<E, DP>(src, q, t, a.tokens, a.dim, first, key1, kStep * kWaves, a.scale2, o, m, l);
    } else if (in_prefix) {
        const PrefixSource src{a.prefix_k + head * a.prefix_head, a.prefix_v + head * a.prefix_head, a.prefix_token, n};
        attend_wave<E, DP>(src, q, t, a.tokens, a.dim, first, key1, kStep * kWaves, a.scale2, o, m, l);
    } else {
        const int64_t at = (a.table ? 0 : b * a.k_batch) + head * a.k_head;
        const int32_t *table = a.table ? a.table + b * a.table_batch : nullptr;
        if (!a.table || a.page % 16 == 0) {
            const SuffixSource<true> src{a.k + at, a.v + at, table, a.k_batch, a.k_token, n, a.tokens, a.page, a.n_pages};
            attend_wave<E, DP>(src, q, t, a.tokens, a.dim, first, key1, kStep * kWaves, a.scale2, o, m, l);
        } else {
            const SuffixSource<false> src{a.k + at, a.v + at, table, a.k_batch, a.k_token, n, a.tokens, a.page, a.n_pages};
            attend_wave<E, DP>(src, q, t, a.tokens, a.dim, first, key1, kStep * kWaves, a.scale2, o, m, l);
        }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) join_ml[wave][c] = make_float2(m, l);
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
        for (int j = 0; j < W; j++) join_o[wave][c][(4 * g + r) * W + j] = o[j][r];
    __syncthreads();
    const int slot = in_prefix ? split : a.prefix_splits + split;
    for (int i = threadIdx.x; i < kRows * DP; i += 64 * kWaves) {
        const int r = i / DP, d = i % DP, at = tile * kRows + r;
        if (at >= row_count || d >= a.dim) continue;
        float mm = -INFINITY, ll = 0.0f, oo = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; w++) mm = fmaxf(mm, join_ml[w][r].x);
        const float safe = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
        for (int w = 0; w < kWaves; w++) {
            const float f = exp2_fast(join_ml[w][r].x - safe);
            ll += f * join_ml[w][r].y;
            oo += f * join_o[w][r][d];
        }
        const int tt = at / a.group % a.tokens, bb = in_prefix ? at / (a.group * a.tokens) : b;
        const int64_t out_row = ((int64_t)bb * a.tokens + tt) * a.heads + head * a.group + at % a.group;
        a.part_o[(slot * a.rows + out_row) * a.dim + d] = oo;
        if (d == 0) a.part_ml[slot * a.rows + out_row] = make_float2(mm, ll);
    }
}

// Ranges of a row's own positions that hold any.
__device__ __forceinline__ int own_splits(const Args &a, int b)
{
    const int n = max(0, min(a.lengths[b], a.suffix));
    return (n + a.suffix_span - 1) / a.suffix_span;
}

constexpr int kMostParts = 256;   // ranges of keys that a row's sums are joined from

// One wave: the maximum and the sum of a row's ranges, of which lane l has
// every 64th.
__device__ __forceinline__ float2 join_row(const Args &a, int64_t row, int parts)
{
    const int lane = threadIdx.x & 63;
    float m = -INFINITY, l = 0.0f;
    for (int s = lane; s < parts; s += 64) {
        const float2 x = a.part_ml[s * a.rows + row];
        const float top = fmaxf(m, x.x), safe = top == -INFINITY ? 0.0f : top;
        l = exp2_fast(m - safe) * l + exp2_fast(x.x - safe) * x.y;
        m = top;
    }
    for (int d = 32; d; d >>= 1) {
        const float om = __shfl_xor(m, d), ol = __shfl_xor(l, d);
        const float top = fmaxf(m, om), safe = top == -INFINITY ? 0.0f : top;
        const float x = exp2_fast(m - safe) * l, y = exp2_fast(om - safe) * ol;
        l = x + y;
        m = top;
    }
    return make_float2(m, l);
}

// A row's logarithm of its sum, for the caller and for the weights.
__device__ __forceinline__ void put_top(const Args &a, int64_t row, float m, float l)
{
    const float top = m + __log2f(l);
    if (a.lse) a.lse[row] = l == 0.0f ? -INFINITY : kLn2 * top;
    if (a.tops) a.tops[row] = l == 0.0f ? INFINITY : top;   // an empty row gives no slot anything
}

// One workgroup joins the ranges of one output row: each wave takes every
// fourth range, each lane two dims.
template <class E>
__device__ __forceinline__ void join_block(const Args &a, int64_t row)
{
    __shared__ float factor[kMostParts];
    __shared__ float2 sums[kWaves][DF11_MAX_DIM / 2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int parts = a.prefix_splits + own_splits(a, (int)(row / ((int64_t)a.tokens * a.heads)));
    const float2 ml = join_row(a, row, parts);
    const float safe = ml.x == -INFINITY ? 0.0f : ml.x;
    if (threadIdx.x < parts) factor[threadIdx.x] = exp2_fast(a.part_ml[threadIdx.x * a.rows + row].x - safe);
    __syncthreads();
    for (int d = 2 * lane; d < a.dim; d += 128) {
        float x = 0.0f, y = 0.0f;
#pragma unroll 4
        for (int s = wave; s < parts; s += kWaves) {
            const float2 o = *(const float2 *)(a.part_o + (s * a.rows + row) * a.dim + d);
            x += factor[s] * o.x, y += factor[s] * o.y;
        }
        sums[wave][d / 2] = make_float2(x, y);
    }
    __syncthreads();
    const float inv = ml.y == 0.0f ? 0.0f : 1.0f / ml.y;
    if (a.out && 2 * threadIdx.x < a.dim) {
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; w++) x += sums[w][threadIdx.x].x, y += sums[w][threadIdx.x].y;
        *(uint32_t *)(a.out + row * a.dim + 2 * threadIdx.x) = E::pack(x * inv, y * inv);
    }
    if (threadIdx.x == 0) put_top(a, row, ml.x, ml.y);
}

// One wave joins the ranges (at most 64) of one output row, lane l the
// factor of range l.  For many rows: their workgroups of four rows are
// resident at once, where those of one row each took two rounds (4096 rows of
// 9 ranges: 11 us).
template <class E>
__device__ __forceinline__ void join_wave(const Args &a, int64_t row)
{
    const int lane = threadIdx.x & 63;
    const int parts = a.prefix_splits + own_splits(a, (int)(row / ((int64_t)a.tokens * a.heads)));
    const float2 mine = lane < parts ? a.part_ml[lane * a.rows + row] : make_float2(-INFINITY, 0.0f);
    float m = mine.x;
#pragma unroll
    for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float safe = m == -INFINITY ? 0.0f : m;
    const float factor = exp2_fast(mine.x - safe);
    float l = factor * mine.y;
#pragma unroll
    for (int d = 32; d; d >>= 1) l += __shfl_xor(l, d);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int d = 2 * lane; a.out && d < a.dim; d += 128) {
        float x = 0.0f, y = 0.0f;
        for (int s0 = 0; s0 < parts; s0 += 8) {
            float2 o[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                o[j] = *(const float2 *)(a.part_o + (min(s0 + j, parts - 1) * a.rows + row) * a.dim + d);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (s0 + j >= parts) break;
                const float f = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, factor), s0 + j));
                x += f * o[j].x, y += f * o[j].y;
            }
        }
        *(uint32_t *)(a.out + row * a.dim + d) = E::pack(x * inv, y * inv);
    }
    if (lane == 0) put_top(a, row, m, l);
}

constexpr int kWeighKeys = 1024;   // slots of a workgroup, four to a thread

// The weights of a run of a head's slots: the probabilities that the rows of
// the head gave them.
__device__ __forceinline__ void weigh_block(const Args &a, int bh, int first)
{
    __shared__ float top[64];
    const int b = bh / a.kv_heads, head = bh % a.kv_heads;
    const int n = max(0, min(a.lengths[b], a.suffix));
    if (first >= n) return;
    const int key = first + 4 * threadIdx.x;
    const int row_count = a.tokens * a.group, parts = own_splits(a, b), wave = threadIdx.x >> 6;
    const auto row_of = [&](int r) {
        return ((int64_t)b * a.tokens + r / a.group) * a.heads + head * a.group + r % a.group;
    };
    float w[4] = {0, 0, 0, 0};
    for (int r0 = 0; r0 < row_count; r0 += 64) {
        const int some = min(64, row_count - r0);
        __syncthreads();
        // many ranges: a wave a row; few: four lanes a row, all rows at once
        // (28 rows of one range: 13.7 us for the launch with a wave a row)
        if (parts > 16) {
            for (int r = wave; r < some; r += kWaves) {
                const float2 ml = join_row(a, row_of(r0 + r), parts);
                if ((threadIdx.x & 63) == 0) top[r] = ml.y == 0.0f ? INFINITY : ml.x + __log2f(ml.y);
            }
        } else {
            const int r = threadIdx.x / 4;
            const int64_t row = row_of(r0 + min(r, some - 1));
            float m = -INFINITY, l = 0.0f;
            float2 x[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int s = (threadIdx.x & 3) + 4 * j;
                x[j] = s < parts ? a.part_ml[s * a.rows + row] : make_float2(-INFINITY, 0.0f);
                m = fmaxf(m, x[j].x);
            }
            m = fmaxf(m, __shfl_xor(m, 1));
            m = fmaxf(m, __shfl_xor(m, 2));
            const float safe = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int j = 0; j < 4; j++) l += exp2_fast(x[j].x - safe) * x[j].y;
            l += __shfl_xor(l, 1);
            l += __shfl_xor(l, 2);
            if (r < some && (threadIdx.x & 3) == 0) top[r] = l == 0.0f ? INFINITY : m + __log2f(l);   // an empty row gives nothing
        }
        __syncthreads();
        if (key < n) {
            const float *from = a.logits + ((int64_t)bh * row_count + r0) * a.logit_stride + key;
#pragma unroll 4
            for (int i = 0; i < some; i++) {
                const f32x4 s = *(const f32x4 *)(from + i * a.logit_stride);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float p = exp2_fast(s[j] - top[i]);
                    w[j] += s[j] == -INFINITY ? 0.0f : p;   // an unseen slot's is 0 also where the row's sum is NaN
                }
            }
        }
    }
    float *to = a.weights + (int64_t)bh * a.suffix + key;
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (key + j < n) to[j] += w[j];
}

// As weigh_block, from the logits taken again, where rows are many and their
// logits would be more bytes than the keys: S = Q K^T with 32 rows of Q from
// LDS against 32 keys of a wave, whose lanes l and l + 32 hold key l % 32's
// logits with 32 rows between them.  128 rows, 4 x 8 heads of 16384 slots: 46
// us, 17 GFLOP and 134 MB (kept logits would be 268 MB to write and to read).
constexpr int kWeighRows = 128;

template <class E, int DP>
__global__ void __launch_bounds__(64 * kWaves, 2) weigh_kernel(const Args a)
{
    typedef TileShape<DP> S;
    __shared__ alignas(1024) char lds[kWeighRows * (DP * 2 + 8)];
    const int bh = blockIdx.y, first = blockIdx.x * a.weigh_run;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 31, g = lane >> 5;
    const int b = bh / a.kv_heads, head = bh % a.kv_heads;
    const int n = max(0, min(a.lengths[b], a.suffix));
    if (first >= n) return;
    float *const top = (float *)(lds + kWeighRows * DP * 2);
    int32_t *const token = (int32_t *)(top + kWeighRows);
    const int row_count = a.tokens * a.group, pos = a.pos[b];
    const uint16_t *kp = a.k + b * a.k_batch + head * a.k_head;
    const int32_t *places = a.positions + (int64_t)bh * a.suffix;
    float *weights = a.weights + (int64_t)bh * a.suffix;
    for (int r0 = 0; r0 < row_count; r0 += kWeighRows) {
        __syncthreads();
        for (int i = threadIdx.x; i < kWeighRows * S::kChunks; i += 64 * kWaves) {
            const int r = i / S::kChunks, d = i % S::kChunks * 8, row = r0 + r;
            const u32x4 x = row < row_count && d < a.dim
                                ? *(const u32x4 *)(a.q + b * a.q_batch + row / a.group * a.q_token +
                                                   (head * a.group + row % a.group) * a.q_head + d)
                                : u32x4{0, 0, 0, 0};
            *(u32x4 *)(lds + S::k_at(r, d / 8)) = x;
        }
        if (threadIdx.x < kWeighRows) {
            const int row = r0 + threadIdx.x, at = row / a.group;
            const bool there = row < row_count;
            top[threadIdx.x] =
                there ? a.tops[((int64_t)b * a.tokens + at) * a.heads + head * a.group + row % a.group] : INFINITY;
            token[threadIdx.x] = there ? at : -0x7fffffff;
        }
        __syncthreads();
        const int q_from = S::k_at(c, g);
        u32x4 kx[DP / 16], next[DP / 16];
        int32_t place, next_place;
        const auto load = [&](int base) {
            const int key = min(base + c, n - 1);
#pragma unroll
            for (int i = 0; i < DP / 16; i++) {
                const int d = 16 * i + 8 * g;
                next[i] = d < a.dim ? *(const u32x4 *)(kp + key * a.k_token + d) : u32x4{0, 0, 0, 0};
            }
            next_place = base + c < n ? places[key] : -1;
        };
        const int end = min(n, first + a.weigh_run);
        load(first + 32 * wave);
        for (int base = first + 32 * wave; base < end; base += 32 * kWaves) {
            const int key = base + c;
#pragma unroll
            for (int i = 0; i < DP / 16; i++) kx[i] = next[i];
            place = next_place;
            if (base + 32 * kWaves < end) load(base + 32 * kWaves);
            const bool some = place >= 0 && (int64_t)place <= (int64_t)pos + a.tokens - 1;
            const int32_t rel = some ? place - pos : 0x7fffffff;
            const bool mixed = __any(rel > 0);
            float w = 0.0f;
            // two tiles of 32 rows at a time, whose products do not wait for each other
            for (int r = 0; r < min(kWeighRows, row_count - r0); r += 64) {
                f32x16 s[2];
#pragma unroll
                for (int k = 0; k < 2; k++)
#pragma unroll
                    for (int i = 0; i < 16; i++) s[k][i] = 0.0f;
#pragma unroll
                for (int i = 0; i < DP / 16; i++)
#pragma unroll
                    for (int k = 0; k < 2; k++)
                        s[k] = E::mfma32(*(const u32x4 *)(lds + S::k_next(q_from, i) + (r + 32 * k) * DP * 2), kx[i], s[k]);
                f32x4 x[2][4];
#pragma unroll
                for (int k = 0; k < 2; k++)
#pragma unroll
                    for (int i = 0; i < 4; i++) x[k][i] = *(const f32x4 *)(top + r + 32 * k + 8 * i + 4 * g);
                if (!mixed && r0 + r + 64 <= row_count) {
#pragma unroll
                    for (int k = 0; k < 2; k++)
#pragma unroll
                        for (int i = 0; i < 16; i++) w += exp2_fast(__builtin_fmaf(s[k][i], a.scale2, -x[k][i / 4][i % 4]));
                } else {
                    for (int k = 0; k < 2; k++)
#pragma unroll
                        for (int i = 0; i < 16; i++) {
                            const float p = exp2_fast(__builtin_fmaf(s[k][i], a.scale2, -x[k][i / 4][i % 4]));
                            const int32_t last = token[r + 32 * k + 8 * (i / 4) + 4 * g + i % 4];
                            w += rel <= last ? p : 0.0f;
                        }
                }
            }
            w += __shfl_xor(w, 32);
            if (g == 0 && some) weights[key] += w;
        }
    }
}

// Workgroups below the number of those that join join a row each (a.four:
// four rows); behind them those of bounded caches add up the slots' weights.
template <class E, bool WEIGH>
__global__ void __launch_bounds__(64 * kWaves) finish_kernel(const Args a)
{
    const int64_t joins = a.four ? (a.rows + kWaves - 1) / kWaves : a.rows;
    if (WEIGH && blockIdx.x >= joins) {
        const int runs = (a.suffix + kWeighKeys - 1) / kWeighKeys, item = blockIdx.x - (int)joins;
        weigh_block(a, item / runs, item % runs * kWeighKeys);
    } else if (a.four) {
        const int64_t row = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
        if (row < a.rows) join_wave<E>(a, row);
    } else {
        join_block<E>(a, blockIdx.x);
    }
}

int ceil_div(int64_t x, int64_t y) { return (int)((x + y - 1) / y); }

// The keys of an item in n ranges, of at least a step of every wave.
void set_ranges(int64_t keys, int64_t n, int32_t *splits, int32_t *span)
{
    constexpr int64_t kLeast = kStep * kWaves;
    n = std::max<int64_t>(1, std::min<int64_t>(kMostParts / 2, n));
    *span = ceil_div(ceil_div(std::max<int64_t>(keys, 1), n), kLeast) * kLeast;
    *splits = keys ? ceil_div(keys, *span) : 0;
}

// The fewest ranges with which all items' workgroups nearly fill the `slots`
// that are resident at a time, once or several times over; one range, which
// has the fewest sums to join, also where it fills three quarters.  528 items
// of 2050 to 4099 keys on 768 slots: 111 us in 1 range, 108 in 2, 100 in 4;
// 512 items of 2048 keys on 512 slots 99 us in 1 range, 102 in 2 or 4; 384
// items of up to 700 keys on 512 slots 29 us in 1 range, 31 in 2, 32 in 4.
int64_t ranges_that_fill(int64_t keys, int64_t items, int64_t slots)
{
    const int64_t most = std::min<int64_t>(ceil_div(keys, kStep * kWaves), ceil_div(8 * slots, items));
    int64_t best = 1;
    double full = 0.0;
    for (int64_t n = 1; n <= most && full < (n == 2 ? 0.75 : 0.9); n++) {
        const double rounds = (double)items * n / slots, x = rounds / std::ceil(rounds);
        if (x > full) full = x, best = n;
    }
    return best;
}

void plan(Args &a, bool cache)
{
    const int64_t cus = df11::cu_count();
    const int64_t resident = a.dim <= 64 ? 3 : a.dim <= 128 ? 2 : 1;   // workgroups of a CU, by the kernels' registers
    a.rows = (int64_t)a.batch * a.tokens * a.heads;
    if (!a.rows) return;
    const int64_t own_rows = (int64_t)a.tokens * a.group, shared_rows = a.batch * own_rows;
    // 128-row tiles from where their time, nearly the same for any number of
    // rows, is the less (us in 16- / 128-row tiles: 8191 shared positions 15.4
    // / 17.8 at 16 rows, 19.1 / 17.3 at 24, 23.4 / 18.7 at 64; caches of 16384
    // slots 99 / 117 at 32 rows, 135 / 120 at 48, 167 / 121 at 64).
    a.big = cache ? own_rows > 32 && a.k_token <= kTileStride : shared_rows > 16 && a.prefix_token <= kTileStride;
    a.prefix_tiles = ceil_div(shared_rows, a.big ? kTileRows : kRows);
    a.suffix_tiles = ceil_div(own_rows, cache && a.big ? kTileRows : kRows);
    // 128-row tiles: one workgroup on each CU, whose partial sums are few and
    // which leaves room for those of the sequences' own positions; two where
    // a long prefix is nearly all there is (attention and join of 128 requests
    // behind 32768 positions with 1024 / 1 of their own: 136 / 106 us with one,
    // 157 / 100 with two; of 64 behind 8191 with 700 / 1: 45 / 29 us with one,
    // 51 / 37 with two).
    const int64_t prefix_items = (int64_t)a.prefix_tiles * a.kv_heads;
    const bool alone = 4ll * a.batch * a.suffix <= a.prefix && a.prefix * prefix_items >= 2048 * cus;
    set_ranges(a.prefix, a.big ? (alone ? 2 : 1) * cus / prefix_items : ranges_that_fill(a.prefix, prefix_items, resident * cus),
               &a.prefix_splits, &a.prefix_span);
    const int64_t suffix_items = (int64_t)a.suffix_tiles * a.kv_heads * a.batch;
    a.prefix_places = a.prefix_splits ? places(a.prefix_tiles, (int64_t)a.kv_heads * a.prefix_splits) : 0;
    set_ranges(a.suffix, ranges_that_fill(a.suffix, suffix_items, resident * cus), &a.suffix_splits, &a.suffix_span);
    // the slots of a workgroup that weighs many rows: 512, whose rows' queries
    // are brought to LDS once, or fewer where that leaves most CUs idle (28
    // tokens over 872 slots of 3 prompts: 15.8 us in runs of 512, 8.4 of 128)
    a.weigh_run = 512;
    while (a.weigh_run > 128 && (int64_t)a.batch * a.kv_heads * ceil_div(a.suffix, a.weigh_run) < 2 * cus) a.weigh_run /= 2;
    // a wave a row where the rows' waves fill the device and their ranges are
    // few, else a workgroup a row (4096 rows of up to 11 ranges 8.6 / 11.3 us,
    // 3840 of 9 6.2 / 9.2; 1024 rows of 36 ranges 15 / 8)
    const int64_t parts = a.prefix_splits + a.suffix_splits;
    a.four = (a.rows >= 4 * cus && parts <= 12) || (a.rows >= 16 * cus && parts <= 64);
}

int64_t part_bytes(const Args &a)
{
    const int64_t slots = a.prefix_splits + a.suffix_splits;
    return slots * a.rows * (8 + 4ll * a.dim);
}

bool small(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

constexpr int64_t kMost = 1ll << 30;

int check_heads(const char *who, int64_t dtype, int64_t batch, int64_t tokens, int64_t heads, int64_t kv_heads,
                int64_t dim)
{
    if (dtype != DF11_BF16 && dtype != DF11_FP16) return df11::fail(DF11_E_ARG, "%s: dtype must be bf16 or fp16", who);
    if (!small(dim, 8, DF11_MAX_DIM) || dim % 8)
        return df11::fail(DF11_E_ARG, "%s: dim %lld is not a multiple of 8 up to %d", who, (long long)dim, DF11_MAX_DIM);
    if (!small(kv_heads, 1, 65535) || !small(heads, 1, kMost) || heads % kv_heads)
        return df11::fail(DF11_E_ARG, "%s: %lld heads are no multiple of %lld key heads", who, (long long)heads,
                          (long long)kv_heads);
    if (!small(batch, 0, kMost) || !small(tokens, 1, 65536) || (double)batch * tokens * heads > kMost)
        return df11::fail(DF11_E_ARG, "%s: batch %lld of %lld tokens out of range", who, (long long)batch,
                          (long long)tokens);
    return DF11_OK;
}

int strides_ok(const char *who, std::initializer_list<int64_t> strides, std::initializer_list<int64_t> rows)
{
    for (int64_t s : strides)
        if (s < 0 || s % 8) return df11::fail(DF11_E_ARG, "%s: stride %lld is not a multiple of 8", who, (long long)s);
    // the distance of a 16-row tile's lane, within 15 rows, is a 32-bit number
    for (int64_t s : rows)
        if (s >= 1ll << 27) return df11::fail(DF11_E_ARG, "%s: rows %lld elements apart", who, (long long)s);
    return DF11_OK;
}

template <class E, int DP, int KIND>
int launch(const Args &a, hipStream_t st)
{
    const int64_t items =
        a.prefix_places + places(a.suffix_tiles, (int64_t)a.batch * a.kv_heads * a.suffix_splits);
    const int64_t finish =
        (a.four ? ceil_div(a.rows, kWaves) : a.rows) + (KIND == kCache ? (int64_t)a.batch * a.kv_heads * ceil_div(a.suffix, kWeighKeys) : 0);
    // a launch has fewer than 2^32 threads; refused here, none of a call's launches has begun
    constexpr int64_t kMostGroups = 0xffffffffll / (64 * kWaves);
    if (items > kMostGroups || finish > kMostGroups)
        return df11::fail(DF11_E_ARG, "attention: too many rows and keys for one launch");
    const dim3 block(64 * kWaves);
    if (items) hipLaunchKernelGGL((attend_kernel<E, DP, KIND>), dim3((uint32_t)items), block, 0, st, a);
    const auto join = [&](const Args &x) {
        hipLaunchKernelGGL((finish_kernel<E, KIND == kCache>), dim3((uint32_t)finish), block, 0, st, x);
    };
    if constexpr (KIND == kCacheTiles) {
        // the weights' logits are taken from q again: where out lies on it, the outputs are joined last
        Args x = a;
        if (a.out_on_q) x.out = nullptr;
        join(x);
        const dim3 grid(ceil_div(a.suffix, a.weigh_run), a.batch * a.kv_heads);
        if (a.suffix) hipLaunchKernelGGL((weigh_kernel<E, DP>), grid, block, 0, st, a);
    }
    if (KIND != kCacheTiles || a.out_on_q) join(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return df11::fail(DF11_E_DEVICE, "attention launch: %s", hipGetErrorString(e));
    return DF11_OK;
}

template <int KIND>
int launch_kind(const Args &a, int64_t dtype, hipStream_t st)
{
    if (dtype == DF11_FP16)
        return a.dim <= 64 ? launch<Fp16, 64, KIND>(a, st) : a.dim <= 128 ? launch<Fp16, 128, KIND>(a, st)
                                                                         : launch<Fp16, 256, KIND>(a, st);
    return a.dim <= 64 ? launch<Bf16, 64, KIND>(a, st) : a.dim <= 128 ? launch<Bf16, 128, KIND>(a, st)
                                                                     : launch<Bf16, 256, KIND>(a, st);
}

int check_workspace(const char *who, void *ws, uint64_t bytes, uint64_t need)
{
    if (bytes < need || (need && !aligned16(ws)))
        return df11::fail(DF11_E_ARG, "%s: the workspace must be 16-byte aligned and hold %llu bytes", who,
                          (unsigned long long)need);
    return DF11_OK;
}

void place(Args &a, void *ws)
{
    const int64_t slots = a.prefix_splits + a.suffix_splits;
    a.part_o = (float *)ws;
    a.part_ml = (float2 *)(a.part_o + slots * a.rows * a.dim);
    float *more = (float *)((char *)ws + (part_bytes(a) + 15) / 16 * 16);
    if (a.positions && a.big) a.tops = more;
    else if (a.positions) a.logits = more;
}

int make_prefix(const df11_prefix_attention_args *p, Args &a)
{
    const char *who = "df11_prefix_attention";
    if (!p) return df11::fail(DF11_E_ARG, "%s: null arguments", who);
    int rc = check_heads(who, p->dtype, p->batch, p->tokens, p->heads, p->kv_heads, p->dim);
    if (rc) return rc;
    if (!small(p->prefix, 0, kMost) || !small(p->suffix, 0, kMost) ||
        (p->block_table && (!small(p->page, 1, kMost) || !small(p->n_pages, 0, kMost) || p->suffix % p->page)))
        return df11::fail(DF11_E_ARG, "%s: prefix, suffix or page sizes out of range", who);
    rc = strides_ok(who, {p->q_batch, p->q_token, p->q_head, p->prefix_token, p->prefix_head, p->k_batch, p->k_token,
                          p->k_head}, {p->prefix_token, p->k_token});
    if (rc) return rc;
    if (p->table_batch < 0) return df11::fail(DF11_E_ARG, "%s: negative table stride", who);
    a.q = (const uint16_t *)p->q;
    a.prefix_k = (const uint16_t *)p->prefix_k, a.prefix_v = (const uint16_t *)p->prefix_v;
    a.k = (const uint16_t *)p->k, a.v = (const uint16_t *)p->v;
    a.lengths = p->lengths, a.table = p->block_table;
    a.out = (uint16_t *)p->out, a.lse = p->lse;
    a.batch = p->batch, a.tokens = p->tokens, a.heads = p->heads, a.kv_heads = p->kv_heads;
    a.group = p->heads / p->kv_heads, a.dim = p->dim, a.prefix = p->prefix;
    a.suffix = p->block_table && !p->n_pages ? 0 : p->suffix;
    a.page = p->block_table ? p->page : 1, a.n_pages = p->n_pages;
    a.q_batch = p->q_batch, a.q_token = p->q_token, a.q_head = p->q_head;
    a.prefix_token = p->prefix_token, a.prefix_head = p->prefix_head;
    a.k_batch = p->k_batch, a.k_token = p->k_token, a.k_head = p->k_head, a.table_batch = p->table_batch;
    a.scale2 = (float)(p->scale * 1.44269504088896340736);
    if (!(a.scale2 > 0.0f && a.scale2 < INFINITY)) return df11::fail(DF11_E_ARG, "%s: scale must be positive", who);
    plan(a, false);
    return DF11_OK;
}

int make_cache(const df11_cache *c, const df11_cache_attention_args *p, Args &a)
{
    const char *who = "df11_cache_attention";
    if (!c || !p) return df11::fail(DF11_E_ARG, "%s: null arguments", who);
    int rc = check_heads(who, c->dtype, c->batch, p->tokens, p->heads, c->kv_heads, c->dim);
    if (rc) return rc;
    if (!small(c->slots, 0, kMost) || (double)c->batch * c->kv_heads > 65535)
        return df11::fail(DF11_E_ARG, "%s: slots or batch * kv_heads out of range", who);
    rc = strides_ok(who, {p->q_batch, p->q_token, p->q_head, c->stride_batch, c->stride_head, c->stride_slot},
                    {c->stride_slot});
    if (rc) return rc;
    a.q = (const uint16_t *)p->q;
    a.k = (const uint16_t *)c->k, a.v = (const uint16_t *)c->v;
    a.lengths = c->lengths, a.pos = p->pos, a.positions = c->positions, a.weights = c->weights;
    a.out = (uint16_t *)p->out;
    a.batch = c->batch, a.tokens = p->tokens, a.heads = p->heads, a.kv_heads = c->kv_heads;
    a.group = p->heads / c->kv_heads, a.dim = c->dim, a.suffix = c->slots, a.page = 1;
    a.q_batch = p->q_batch, a.q_token = p->q_token, a.q_head = p->q_head;
    a.k_batch = c->stride_batch, a.k_token = c->stride_slot, a.k_head = c->stride_head;
    a.scale2 = (float)(p->scale * 1.44269504088896340736);
    if (!(a.scale2 > 0.0f && a.scale2 < INFINITY)) return df11::fail(DF11_E_ARG, "%s: scale must be positive", who);
    plan(a, true);
    if (a.rows) {
        const uintptr_t q = (uintptr_t)p->q, out = (uintptr_t)p->out;
        const uintptr_t q_bytes = 2 * ((a.batch - 1) * a.q_batch + (a.tokens - 1) * a.q_token + (a.heads - 1) * a.q_head + a.dim);
        a.out_on_q = out < q + q_bytes && q < out + 2 * (uintptr_t)(a.rows * a.dim);
    }
    a.logit_stride = a.big ? 0 : (c->slots + 31) / 32 * 32;   // many rows: taken again, not kept
    return DF11_OK;
}

uint64_t cache_bytes(const Args &a)
{
    return (part_bytes(a) + 15) / 16 * 16 + 4ull * a.rows * (a.big ? 1 : a.logit_stride);
}

}  // namespace

extern "C" uint64_t df11_prefix_attention_workspace_bytes(const df11_prefix_attention_args *p)
{
    Args a{};
    return make_prefix(p, a) ? 0 : (uint64_t)part_bytes(a);
}

extern "C" int df11_prefix_attention(const df11_prefix_attention_args *p, void *workspace, uint64_t workspace_bytes,
                                     void *stream)
{
    const char *who = "df11_prefix_attention";
    Args a{};
    int rc = make_prefix(p, a);
    if (rc) return rc;
    if (!a.rows) return DF11_OK;
    if (!aligned16(a.q) || !aligned16(a.out) || !a.lengths || (a.prefix && (!aligned16(a.prefix_k) || !aligned16(a.prefix_v))) ||
        (a.suffix && (!aligned16(a.k) || !aligned16(a.v))))
        return df11::fail(DF11_E_ARG, "%s: null or misaligned pointer", who);
    rc = check_workspace(who, workspace, workspace_bytes, part_bytes(a));
    if (rc) return rc;
    place(a, workspace);
    return a.big ? launch_kind<kTiles>(a, p->dtype, (hipStream_t)stream)
                 : launch_kind<kRowTiles>(a, p->dtype, (hipStream_t)stream);
}

extern "C" uint64_t df11_cache_attention_workspace_bytes(const df11_cache *c, const df11_cache_attention_args *p)
{
    Args a{};
    return make_cache(c, p, a) ? 0 : cache_bytes(a);
}

extern "C" int df11_cache_attention(const df11_cache *c, const df11_cache_attention_args *p, void *workspace,
                                    uint64_t workspace_bytes, void *stream)
{
    const char *who = "df11_cache_attention";
    Args a{};
    int rc = make_cache(c, p, a);
    if (rc) return rc;
    if (!a.rows) return DF11_OK;
    if (!aligned16(a.q) || !aligned16(a.out) || !a.lengths || !a.pos ||
        (a.suffix && (!aligned16(a.k) || !aligned16(a.v) || !a.weights || !a.positions)))
        return df11::fail(DF11_E_ARG, "%s: null or misaligned pointer", who);
    rc = check_workspace(who, workspace, workspace_bytes, cache_bytes(a));
    if (rc) return rc;
    place(a, workspace);
    return a.big ? launch_kind<kCacheTiles>(a, c->dtype, (hipStream_t)stream)
                 : launch_kind<kCache>(a, c->dtype, (hipStream_t)stream);
}
