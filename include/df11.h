/*
 * df11.h -- C ABI of libdf11.so, an MI355X (gfx950) implementation of the
 * DFloat11 (Dynamic-length Float) codec for BF16 weights.
 *
 * What the codec computes (sources cited by page title and section):
 *   [P1] "DFloat11无损压缩技术：基于哈夫曼编码的BFloat16大模型显存优化方案"
 *        (jsqmd.com) 2.1: a BF16 word is 1 sign bit, 8 exponent bits and
 *        7 mantissa bits.  2.2 item 1: the exponents' frequencies are counted
 *        and a Huffman code gives frequent exponents short codes.  2.2 item 2:
 *        sign and mantissa are kept unchanged next to the variable-length
 *        exponent code, packed into aligned blocks (about 11 bits per weight).
 *        2.2 item 3: the compressed weights stay in GPU memory and a GPU
 *        kernel restores BF16 right before the matmul that uses them.
 *   [P2] "DFloat11：用于高效 GPU 推理的 LLM 和扩散模型无损压缩"
 *        (gittoolsai.com), "工作原理": Huffman-coded BF16 exponents, decoded
 *        on the GPU before each matrix product, output bit-for-bit identical.
 *   [P3] "DFloat11重新定义LLM无损压缩的技术边界" (ocdem.com) 2.2: compact
 *        hierarchical lookup tables, a locate phase and a reconstruct phase,
 *        and a parallel prefix sum for output positions; 4.2: each thread
 *        takes a fixed run of encoded bytes; 5.2: 256-byte aligned data.
 *
 * Conventions
 *   - Every function returns DF11_OK (0) or a negative DF11_E_* status, and
 *     never throws.  df11_last_error() gives the calling thread's detail text
 *     for the most recent failure.
 *   - BF16 tensors are passed as their uint16 bit patterns.
 *   - "host" pointers are CPU memory; "device" pointers are GPU memory of the
 *     current HIP device.  Device work is asynchronous on `stream` (a
 *     hipStream_t passed as void*, NULL = the null stream).  The decode,
 *     row-gather and fused-product calls allocate no device memory and keep
 *     no per-call state; only df11_encode_device allocates, the device arrays
 *     it returns (freed with df11_device_encoded_free).
 *
 * Stream format (what df11_encode writes and the kernels read)
 *   exp_words  The exponent codes of all elements in stream order, each code
 *              most significant bit first, laid end to end.  Stream bit j is
 *              bit (31 - j % 32) of 32-bit word j / 32.  Zero bits pad the
 *              stream; when layout.align_elems > 0 zero bits also pad each
 *              block of align_elems elements up to a segment boundary.
 *   sm         One byte per element: sign in bit 7, mantissa in bits 6..0.
 *   segments   The stream is cut into segments of seg_lanes * chunk_bytes
 *              bytes; a segment is decoded by one 64-lane wavefront, each lane
 *              taking one chunk of chunk_bytes bytes.
 *   gaps       One byte per chunk: the distance in bits from the chunk start
 *              to the first code that starts at or after it (0..31), or 0 for
 *              a chunk at or past its segment's last code.
 *   counts     One byte per chunk: the number of codes whose first bit lies
 *              in the chunk (0 for chunks past the segment's last code).  The
 *              decoder's output positions are a prefix sum of these counts.
 *              Optional in a view (n_counts = 0): the decoder then finds each
 *              lane's count itself by walking its chunk (the locate pass).
 *              Encoders always write them; a layout whose chunk could hold
 *              more than 255 codes (chunk bits / shortest code) is refused.
 *   segs       n_segments + 1 records: elem_off = number of codes that start
 *              before the segment (the last record's elem_off = n); nbits =
 *              bits from the segment start to the end of the last code that
 *              starts in it, at most the segment size.
 *   chain      The hierarchical lookup tables: n_tables tables of 256 uint16
 *              entries.  Table 0 is indexed by the next 8 stream bits, each
 *              later table by the 8 bits after its parent's.  Entry bit 15
 *              clear: a code ends here -- exponent in bits 0..7, total code
 *              length in bits 8..13.  Bit 15 set: bits 0..14 name the next
 *              table.
 *   fast       2^fast_bits pairs of uint32 {syms, meta} indexed by the next
 *              fast_bits stream bits: the up to 4 whole codes that fit, first
 *              code in the lowest byte, each byte the exponent rotated right
 *              by one bit; meta = (count << 16) - bits consumed, modulo 2^32;
 *              meta = 0 when the first code is longer than fast_bits.
 *   block_seg  When align_elems > 0: for every block of align_elems elements the
 *              index of the segment its first code starts in, followed by
 *              n_segments (ceil(n / align_elems) + 1 entries); else empty.
 *   Element order is row-major, or, when tile_rows > 0, tile order: the
 *   [rows, cols] matrix is cut into tile_rows x tile_cols tiles taken row
 *   block by row block, row-major inside each tile, or, when tile_kchunk > 0,
 *   in column groups of tile_kchunk columns: group after group, each group
 *   row after row (the order matrix-core operands read).
 */
#ifndef DF11_H
#define DF11_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DF11_OK 0
#define DF11_E_ARG (-1)       /* null/misaligned pointer, size or layout out of range */
#define DF11_E_UNCODED (-2)   /* an input exponent has no code in the codebook */
#define DF11_E_CODE_LEN (-3)  /* max_len outside 1..32, or more than DF11_MAX_TABLES tables */
#define DF11_E_FORMAT (-4)    /* df11_validate found an inconsistent stream or codebook */
#define DF11_E_DEVICE (-5)    /* a HIP call failed; detail in df11_last_error() */
#define DF11_E_ALLOC (-6)     /* an allocation failed */
#define DF11_E_UNSUPPORTED (-7) /* a valid request this build does not handle */

#define DF11_MAX_LEN 32
#define DF11_MAX_TABLES 64
#define DF11_FAST_BITS_MIN 8
#define DF11_FAST_BITS_MAX 12
#define DF11_FAST_BITS_DEFAULT 11
#define DF11_SEG_LANES 64

/* A codebook: code lengths, canonical codes and the lookup tables derived
 * from them.  Plain data; the caller owns the struct. */
typedef struct df11_codebook {
    uint32_t max_len;     /* longest code length (0 when no symbol occurs) */
    uint32_t min_len;     /* shortest code length */
    uint32_t n_symbols;   /* exponents with a code */
    uint32_t n_tables;    /* hierarchical 256-entry tables used in chain[] */
    uint32_t fast_bits;   /* index width of fast[] */
    uint32_t reserved[3];
    uint8_t len[256];     /* code length per exponent, 0 = no code */
    uint32_t code[256];   /* canonical code per exponent, right-aligned */
    uint16_t chain[DF11_MAX_TABLES * 256];
    uint32_t fast[2u << DF11_FAST_BITS_MAX];
} df11_codebook;

/* How the stream is laid out.  Zero-initialise and set what you need:
 * chunk_bytes 0 means 16; seg_lanes 0 means 64. */
typedef struct df11_layout {
    uint32_t chunk_bytes;   /* stream bytes per lane: 16, or 8 (twice the segments, for
                               small tensors that would leave most of the GPU idle) */
    uint32_t seg_lanes;     /* lanes per segment: must be 64 */
    uint64_t align_elems;   /* 0, or begin a new segment every align_elems elements */
    uint64_t rows, cols;    /* matrix shape; cols = 0 means a flat tensor of rows = n */
    uint32_t tile_rows, tile_cols;  /* 0, 0: row-major; else tile order (see above) */
    uint32_t tile_kchunk;           /* 0: row-major inside a tile; else column groups (see above) */
    uint32_t reserved;
} df11_layout;

typedef struct df11_segment {
    uint64_t elem_off;
    uint32_t nbits;
    uint32_t reserved;
} df11_segment;

/* Pointers and sizes of one encoded tensor.  The pointers are all host or all
 * device memory; the caller fills a device view by copying every array of a
 * host view to the GPU and keeping the scalars. */
typedef struct df11_view {
    uint64_t n;             /* elements */
    uint64_t total_bits;    /* end of the last code in the stream */
    uint64_t n_segments;
    uint32_t chunk_bytes, seg_lanes;
    uint64_t rows, cols;
    uint32_t tile_rows, tile_cols;
    uint32_t tile_kchunk;
    int32_t row_win_lo;         /* row window (see below) */
    uint64_t align_elems;
    uint32_t min_len, max_len, n_tables, fast_bits;
    uint32_t max_seg_elems;     /* most codes starting in any one segment */
    uint32_t row_win_span;      /* row window: 0 = none.  For a row-major view with rows and
                                   cols set, both encoders record the window that holds every
                                   segment overlapping any row r: with g(r) = floor(r * cols *
                                   (n_segments / n)), the segment indices in IEEE double
                                   arithmetic (the quotient first), row r's segments lie in
                                   [g(r) + row_win_lo, g(r) + row_win_lo + row_win_span).
                                   df11_decode_rows relies on it as written by the encoder. */
    const uint32_t *exp_words;  uint64_t n_exp_words;  /* n_segments*seg_words + 2 */
    const uint8_t *sm;          uint64_t n_sm;         /* n rounded up to 16 */
    const uint8_t *gaps;        uint64_t n_gaps;       /* n_segments * seg_lanes */
    const df11_segment *segs;   uint64_t n_segs;       /* n_segments + 1 */
    const uint16_t *chain;      uint64_t n_chain;      /* n_tables * 256 */
    const uint32_t *fast;       uint64_t n_fast;       /* 2 << fast_bits */
    const uint64_t *block_seg;  uint64_t n_block_seg;  /* align_elems > 0: first segment of
                                                          every aligned block, then n_segments */
    const uint8_t *counts;      uint64_t n_counts;     /* n_segments * seg_lanes, or 0 */
} df11_view;

typedef struct df11_encoded df11_encoded;   /* opaque, library-owned host arrays */

/* ---------------------------------------------------------------- host side */

/* hist[e] += number of elements of bf16_bits[0..n) whose exponent is e
 * ([P1] 2.2 item 1).  Accumulates, so several tensors can share one codebook.
 * bf16_bits and hist are host pointers; n = 0 is a no-op.  Errors: E_ARG for
 * a null pointer with n > 0. */
int df11_hist_accumulate(const uint16_t *bf16_bits, uint64_t n, uint64_t hist[256]);

/* Build a codebook from an exponent histogram ([P1] 2.2 item 1; [P2]
 * "工作原理"): Huffman code lengths, replaced by the optimal code limited to
 * max_len bits (package-merge) when Huffman is longer; canonical codes in
 * (length, exponent) order; the hierarchical tables ([P3] 2.2) and the
 * fast_bits-wide multi-code table.  max_len in 1..32, fast_bits in 8..12.
 * Errors: E_ARG (null), E_CODE_LEN (max_len out of range or too small for
 * the number of symbols, or more than DF11_MAX_TABLES tables). */
int df11_codebook_build(const uint64_t hist[256], uint32_t max_len, uint32_t fast_bits,
                        df11_codebook *cb);

/* Encode n BF16 words (host) with codebook cb into a new library-owned
 * encoding ([P1] 2.2 item 2; [P3] 4.2): exponent stream, sign+mantissa
 * bytes, per-lane gaps and per-segment records, laid out by `layout` (NULL
 * = defaults).  *out receives the encoding; free it with df11_encoded_free.
 * Every layout it accepts is one the decode calls read.
 * Errors: E_ARG (null pointers, chunk_bytes other than 8 or 16, layout out
 * of range, rows*cols != n, tile shape not dividing the matrix or tile_cols
 * not a multiple of 16), E_UNCODED (an exponent without a code), E_ALLOC. */
int df11_encode(const uint16_t *bf16_bits, uint64_t n, const df11_codebook *cb,
                const df11_layout *layout, df11_encoded **out);

void df11_encoded_free(df11_encoded *enc);

/* Fill *v with host pointers into enc (valid until df11_encoded_free). */
int df11_encoded_view(const df11_encoded *enc, df11_view *v);

/* The layout df11_decode_gemm needs for an [rows, cols] weight: tile order
 * with tiles of df11_gemm_tile_rows() x df11_gemm_tile_cols() elements in
 * 8-column groups, each tile beginning a segment.  Errors: E_ARG when the
 * shape does not divide. */
int df11_gemm_layout(uint64_t rows, uint64_t cols, df11_layout *layout);
uint32_t df11_gemm_tile_rows(void);
uint32_t df11_gemm_tile_cols(void);

/* O(n) CPU check of a host view against its codebook: array sizes, table
 * consistency, gaps and segment records recomputed by walking the stream.
 * Returns DF11_OK or E_FORMAT / E_ARG with the first problem in
 * df11_last_error().  Detection path for corrupt data; the kernels do not
 * check streams. */
int df11_validate(const df11_view *host_view, const df11_codebook *cb);

/* ---------------------------------------------------------- device encoder */

/* A tensor encoded on the GPU: every array in device memory owned by the
 * library (including a copy of the codebook's tables). */
typedef struct df11_device_encoded df11_device_encoded;

/* Exponent histogram of n BF16 words in device memory, added into hist
 * (host) ([P1] 2.2 item 1).  Synchronises `stream`.  Errors: E_ARG (null),
 * E_DEVICE. */
int df11_hist_device(const uint16_t *device_bits, uint64_t n, uint64_t hist[256], void *stream);

/* Encode n BF16 words in device memory on the GPU ([P1] 2.2 items 1-2;
 * [P3] 4.1 on the cost of offline compression): the same stream, sign and
 * mantissa bytes, gaps, segment records and block index, byte for byte, as
 * df11_encode with the same codebook and layout.  The library allocates the
 * device arrays; free them with df11_device_encoded_free.  Synchronises
 * `stream` (twice: the stream length decides the output sizes).  Errors:
 * E_ARG (null, layout), E_UNCODED (an exponent without a code), E_ALLOC,
 * E_DEVICE. */
int df11_encode_device(const uint16_t *device_bits, uint64_t n, const df11_codebook *cb,
                       const df11_layout *layout, void *stream, df11_device_encoded **out);
void df11_device_encoded_free(df11_device_encoded *enc);

/* Fill *v with the device pointers of enc (valid until
 * df11_device_encoded_free): a device view for df11_decode and friends. */
int df11_device_encoded_view(const df11_device_encoded *enc, df11_view *v);

/* Copy a device encoding into a new host encoding (free with
 * df11_encoded_free), e.g. to store it or to check it with df11_validate.
 * Errors: E_ARG, E_ALLOC, E_DEVICE. */
int df11_device_encoded_to_host(const df11_device_encoded *enc, df11_encoded **out);

/* -------------------------------------------------------------- device side */

/* Decode a device view into out[0..n) BF16 bits in row-major order
 * ([P1] 2.2 item 3; [P3] 2.2 locate/reconstruct with a prefix sum).
 * out: device, 16-byte aligned, n elements.  Bit-exact: every input pattern,
 * including zeros, subnormals, Inf and NaN payloads, comes back unchanged.
 * Writes stay inside out[0..n) even for a corrupt stream (the exponent
 * words, gaps or counts; then the values are unspecified): every write
 * address comes from the segment records, which are checked against n.
 * The view's max_seg_elems (set by the encoders) sizes the staging: a
 * hand-built view that understates it leaves the larger segments' outputs
 * unwritten.  n = 0 is a no-op.  Errors: E_ARG (null, misaligned, view
 * inconsistent, max_seg_elems 0 or above segment bits / shortest code),
 * E_UNSUPPORTED (tables too large for the kernel), E_DEVICE. */
int df11_decode(const df11_view *device_view, uint16_t *out, void *stream);

/* Decode several device views in one launch: view i into outs[i] (device,
 * 16-byte aligned, views[i].n elements), for example the seven matrices of a
 * decoder layer.  views is a host array of `count` device views that share
 * their device tables (the same chain and fast pointers, i.e. one codebook
 * uploaded once).  Same guarantees and errors as df11_decode, plus E_ARG when
 * the views do not share their tables.  More than 16 views are decoded in
 * launches of 16. */
int df11_decode_batch(const df11_view *device_views, uint16_t *const *outs, uint32_t count,
                      void *stream);

/* Explicit launch choices of a decode, for measurements and tests.  A zeroed
 * struct, or NULL, is the library's own choice. */
#define DF11_STORES_AUTO 0       /* streaming when the launch writes more than the 256 MB last-level cache */
#define DF11_STORES_CACHED 1     /* normal loads and stores: the output stays cache-resident for its consumer */
#define DF11_STORES_STREAMING 2  /* nontemporal BF16 stores */
typedef struct df11_decode_tuning {
    uint32_t waves;        /* waves per workgroup: 0 = from occupancy and size, else 4, 6, ..., 16 */
    uint32_t stores;       /* DF11_STORES_* */
    uint32_t groups;       /* workgroups per launch: 0 = as many as are resident at once (each wave
                              then walks several segments), else that many, at most 2^31 - 1 */
    uint32_t reserved[5];  /* zero */
} df11_decode_tuning;

/* df11_decode_batch with explicit launch choices ([P3] 5.2: occupancy is
 * the tuning lever).  The output is the same for every choice.  Errors: as
 * df11_decode_batch, and E_ARG for a choice out of range or a wave count
 * whose staging and tables do not fit in LDS. */
int df11_decode_batch_tuned(const df11_view *device_views, uint16_t *const *outs, uint32_t count,
                            const df11_decode_tuning *tuning, void *stream);

/* Row gather: decode rows rows[0..n_rows) of a row-major [rows, cols] view
 * into out[i][0..cols) (device, 16-byte aligned, n_rows x cols BF16), for
 * an embedding lookup that restores only the rows a batch uses ([P1] 2.2
 * item 3: weights are restored right before use).  rows: device int64 ids,
 * 8-byte aligned.  For a few rows whose view records a row window of at
 * most 16 segments (row_win_span), each row gets a workgroup in which every
 * segment of the window has its own wave, so no search precedes the segment
 * loads, and the row's sign+mantissa bytes are copied into LDS beside them;
 * otherwise the segments that
 * overlap each requested row are found from an interpolated guess, checked
 * against the 64 segment records around it, else by a 64-way search (up to
 * eight waves per row, one segment each).  Segments are decoded whole
 * (8-byte chunks halve the segments and with them the latency of a lookup);
 * only the row's elements are written.  An id outside
 * [0, rows) leaves its output row unwritten.  Bit-exact like df11_decode.  Errors: E_ARG (null, misaligned,
 * tile-ordered view, cols not a multiple of 8), E_UNSUPPORTED, E_DEVICE. */
int df11_decode_rows(const df11_view *device_view, const int64_t *rows, uint64_t n_rows, uint16_t *out,
                     void *stream);

/* Fused decode + matrix product ([P1] 2.2 item 3: decoded weights feed the
 * matmul and are discarded): y[b][j] = sum_k x[b][k] * W[j][k] for W the
 * [rows = N, cols = K] weight of `w` (encoded with df11_gemm_layout), x a
 * device [B, K] BF16 row-major matrix, y a device [B, N] float32 matrix.
 * Products of BF16 values are exact in float32 and accumulate in float32.
 * w_debug: NULL, or a device [N, K] buffer that also receives the decoded
 * BF16 weights.  B in 1..256.  x, y and w_debug 16-byte aligned.  y is
 * overwritten.  When the weight has too few 32-row blocks to fill the
 * device, a row block's work is split across workgroups (along K, or into
 * runs of its segments) and the partial sums are added into y (cleared
 * first, on the same stream) with float atomics, so the order of those few
 * additions, and with it the last bits of y, can differ from run to run.
 * The kernel is chosen by B: up to 64 rows (128 with the workspace of
 * df11_decode_gemm_ex) one whose decoder waves hand tiles of exponents to
 * matrix-core waves through a ring in LDS, above that (with the workspace)
 * one whose ring holds whole BF16 tiles, else one that merges each decoded
 * tile once into a BF16 tile in LDS shared by all batch tiles (two row
 * blocks per workgroup above 112 rows); w_debug calls take a
 * tile-synchronous kernel up to 32 rows and the shared-tile one above.  A
 * kernel that forms the products on the vector ALU (one or two rows) and a
 * segment-parallel one (up to 64 rows) are explicit choices
 * (df11_decode_gemm_ex makes every choice explicit).
 * Non-finite x: a row of x holding Inf or NaN gives a non-finite row of y;
 * where a plain product would give +-Inf, the segment-parallel and vector
 * kernels may give NaN instead (they multiply the weights of a
 * neighbouring segment, masked to +0, by the same x).  Rows of x without
 * them are unaffected.
 * Errors: E_ARG (null, misaligned, layout not from df11_gemm_layout, B out
 * of range), E_UNSUPPORTED, E_DEVICE. */
int df11_decode_gemm(const df11_view *device_view, const uint16_t *x, uint32_t B,
                     float *y, uint16_t *w_debug, void *stream);

/* Output types of df11_decode_gemm_out. */
#define DF11_Y_F32 0
#define DF11_Y_BF16 1

/* df11_decode_gemm with the type of y chosen by y_dtype: DF11_Y_F32 is
 * df11_decode_gemm itself; DF11_Y_BF16 makes y a device [B, N] BF16 matrix,
 * each element the float32 sum rounded once to the nearest BF16 (ties to
 * even; NaN stays NaN).  A BF16 y is written by exactly one workgroup per
 * element (the K range is not split), so it is the same on every run.
 * Errors: as df11_decode_gemm, and E_ARG for an unknown y_dtype. */
int df11_decode_gemm_out(const df11_view *device_view, const uint16_t *x, uint32_t B,
                         void *y, int y_dtype, uint16_t *w_debug, void *stream);

/* Explicit kernel choices of a fused product, for measurements and tests.
 * A zeroed struct, or NULL, is the library's own choice. */
#define DF11_GEMM_AUTO 0
#define DF11_GEMM_SEGMENT 1   /* segment-parallel: up to 64 rows of x, no w_debug */
#define DF11_GEMM_WIDE 2      /* one BF16 tile in LDS shared by the batch tiles: 33 rows of x or more */
#define DF11_GEMM_TILED 3     /* tile-synchronous, any rows of x */
#define DF11_GEMM_VECTOR 4    /* dot products on the vector ALU: one or two rows of x, no w_debug */
#define DF11_GEMM_PIPE 5      /* decoder and matrix-core waves on a ring of BF16 tiles in LDS: any rows of x */
#define DF11_GEMM_RING 6      /* as DF11_GEMM_PIPE with exponent-only planes, two workgroups per CU: up to 128 rows of x
                                 (two matrix-core waves per batch tile, k_slices, up to 64) */
typedef struct df11_gemm_tuning {
    uint32_t kernel;       /* DF11_GEMM_* */
    uint32_t row_blocks;   /* wide kernel: 0 = by B, else 1 or 2 row blocks per workgroup */
    uint32_t parts;        /* segment-parallel and vector kernels: 0 = enough runs of a row block's
                              segments to fill the device, else that many (float32 y) */
    uint32_t split;        /* wide, tile-synchronous, pipelined and exponent-ring kernels (named in
                              `kernel`): 0 = by occupancy, else that many K ranges per row block
                              (float32 y) */
    uint32_t one_writer;   /* nonzero: every element of y is summed by one workgroup in a fixed
                              order (no K ranges, no segment runs: parts and split 1), so a
                              float32 y is the same on every run; slower for weights with too few
                              row blocks to fill the device */
    uint32_t tiles_per_wave; /* pipelined kernel: 0 = by B, else 1 or 2 batch tiles of 32 rows of x
                              per matrix-core wave */
    uint32_t k_slices;     /* exponent-ring kernel: 0 = by B, else 1 or 2 matrix-core waves per batch
                              tile of x, each taking that share of a tile's k-steps (2: up to 64 rows) */
    uint32_t reserved[1];  /* zero */
} df11_gemm_tuning;

/* Bytes of the workspace df11_decode_gemm_ex can use for B rows of x with
 * this weight: x repacked in the matrix cores' operand order (16 bytes per
 * lane and k-step, one contiguous kilobyte per wavefront load, rows past B
 * zero): 32 T rows of x, (K / 16) * T * 1024 bytes, for T = 2, 4 or 8
 * batch tiles of 32 rows (B up to 64, 128, 256).  0 when B <= 32, where x
 * is read in place, and for a view not in the fused layout. */
uint64_t df11_decode_gemm_workspace_bytes(const df11_view *device_view, uint32_t B);

/* df11_decode_gemm_out with explicit kernel choices and a workspace
 * ([P1] 2.2 item 3: decoded weights feed the matmul; [P3] 5.2: the kernel
 * shape is tuned to the hardware).  tuning: NULL or zeroed = the library's
 * choice.  workspace: NULL, or device memory of workspace_bytes >=
 * df11_decode_gemm_workspace_bytes(w, B), 256-byte aligned, owned by the
 * caller and not used by any other work on the GPU until this call's work on
 * `stream` has finished: above 32 rows of x a packing kernel first writes x
 * into it in operand order (overwriting all of the bytes it needs, so its
 * contents need no clearing), and the product reads x from there (up_proj at
 * 64 / 128 / 256 rows: 63 / 103 / 97 us with x read in place, 47 / 63 / 85
 * us with x packed, the packing included).
 * y agrees with every choice within the float32 summation order.  Errors:
 * as df11_decode_gemm_out, E_ARG for a choice that does not apply (w_debug
 * or more than 64 rows of x on the segment-parallel kernel, w_debug or more
 * than 2 rows on the vector one, 32 rows or fewer on the wide one, split
 * without a kernel that takes it, parts or split above 1 with a BF16 y or
 * with one_writer) or a workspace too
 * small or misaligned, E_UNSUPPORTED when the chosen kernel's LDS does not
 * fit this weight. */
int df11_decode_gemm_ex(const df11_view *device_view, const uint16_t *x, uint32_t B, void *y, int y_dtype,
                        uint16_t *w_debug, const df11_gemm_tuning *tuning, void *workspace,
                        uint64_t workspace_bytes, void *stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation):
 * df11_decode_gemm_ex with the packed x kept in the library's own scratch,
 * a 16 MiB array in device memory that every device the library runs on
 * holds until the process ends; no allocation happens in the call.  The
 * scratch covers df11_decode_gemm_workspace_bytes(w, B) <= 16 MiB, that is
 * K * T <= 262144 (T = 2, 4, 8 batch tiles for B up to 64, 128, 256; K up to
 * 32768 at 256 rows of x).  All such calls on one GPU share its scratch:
 * calls that overlap in time on one GPU (other streams, other threads) race
 * on it; calls ordered on one stream do not (each packs x afresh, nothing
 * has to start at zero).  Errors: as df11_decode_gemm_ex, and E_UNSUPPORTED
 * when the packed x would not fit the scratch. */
int df11_decode_gemm_noalloc(const df11_view *device_view, const uint16_t *x, uint32_t B, void *y,
                             int y_dtype, uint16_t *w_debug, const df11_gemm_tuning *tuning, void *stream);

/* ------------------------------------------------------- token generation */

/* The operators of one generation step around the compressed weights ([P2]
 * "工作原理": compressed weights serve token generation; [P1] 2.2 item 3):
 * attention for sequences that share a prefix, attention over a bounded
 * cache that evicts by accumulated attention weight, and the verification
 * of drafted tokens.  All pointers are device memory of the current device;
 * the work is asynchronous on `stream`; nothing is allocated.  Every field
 * of the argument structs is 8 bytes wide, strides are in elements, and
 * the last axis (dim, vocabulary) is contiguous.  A call that has nothing
 * to compute (batch 0) launches nothing. */

/* Element types of the operands below. */
#define DF11_BF16 0
#define DF11_FP16 1
#define DF11_FP32 2   /* probabilities only */

#define DF11_MAX_DIM 256
#define DF11_NO_TOKEN 0x7fffffff   /* position of a cache slot that holds no token */

/* Attention of `batch` sequences, `tokens` query tokens each, over a prefix
 * that all of them share followed by each sequence's own positions:
 *
 *   o[b,t,h] = sum_j softmax_j(scale * q[b,t,h] . K_j) V_j,   h' = h / (heads / kv_heads)
 *
 * over the keys K_j of prefix_k[0..prefix)[h'] and of the sequence's own
 * first lengths[b] - (tokens - 1) + t positions [h'] (the `tokens` query tokens are
 * the last of those lengths[b] positions and see each other causally; a
 * length outside [0, suffix] is taken as the nearer end).  A row without a
 * visible key is zero, its lse -infinity.  The prefix is read once for all
 * sequences, not once for each.  Own positions are [batch, suffix] rows
 * (block_table NULL: k_batch, k_token, k_head strides) or lie in pages:
 * position s of sequence b is row s % page of page
 * block_table[b * table_batch + s / page] (k_batch is then the stride
 * between pages, suffix = pages per sequence * page); a page id outside
 * [0, n_pages) holds no visible position.  K and V share their strides.
 * What masked or unused positions hold, NaN and infinities included, does not reach the output.
 * Statistics and sums are float32; the probabilities are rounded to the
 * operands' type for the product with V. */
typedef struct df11_prefix_attention_args {
    const void *q, *prefix_k, *prefix_v, *k, *v;
    const int32_t *lengths;       /* [batch] */
    const int32_t *block_table;   /* [batch, suffix / page], or NULL */
    void *out;                    /* [batch, tokens, heads, dim], contiguous, the type of q; may be q itself */
    float *lse;                   /* [batch, tokens, heads] natural log of the sum, or NULL */
    int64_t dtype, batch, tokens, heads, kv_heads, dim, prefix, suffix, page, n_pages;
    int64_t q_batch, q_token, q_head, prefix_token, prefix_head, k_batch, k_token, k_head, table_batch;
    double scale;
} df11_prefix_attention_args;

/* Device bytes df11_prefix_attention needs as workspace (partial sums of
 * key ranges); 0 for arguments it refuses. */
uint64_t df11_prefix_attention_workspace_bytes(const df11_prefix_attention_args *a);

/* workspace: 16-byte aligned, at least that many bytes, not used by other
 * work until this call's work has finished; its contents need no clearing.
 * The result does not depend on the run.  Errors: E_ARG (null or misaligned
 * pointer -- 16 bytes for q, k, v and out, strides multiples of 8, those between
 * a head's keys below 2^27 -- sizes out of range, dim not a multiple of 8 or above DF11_MAX_DIM, heads not a
 * multiple of kv_heads, scale not positive, workspace too small), E_DEVICE. */
int df11_prefix_attention(const df11_prefix_attention_args *a, void *workspace, uint64_t workspace_bytes,
                          void *stream);

/* A bounded cache: for each sequence and key head `slots` slots of a key, a
 * value, the attention weight the slot has gathered and the position of its
 * token.  Sequence b uses the slots [0, lengths[b]).  A slot whose position
 * is DF11_NO_TOKEN (or negative) holds none: it is not seen, and is the first
 * to be replaced.  So is one whose position is at or past the sequence's next
 * position, but only until the sequence has passed that position: then it
 * counts as seen, beside any other slot of the same position.  A caller that
 * takes tokens back (refused drafts) sets the positions of their slots to
 * DF11_NO_TOKEN before the next token is inserted.  Weights that the queries
 * of such tokens gave to other slots stay. */
typedef struct df11_cache {
    void *k, *v;                  /* [batch, kv_heads, slots, dim] */
    float *weights;               /* [batch, kv_heads, slots], contiguous */
    int32_t *positions;           /* [batch, kv_heads, slots], contiguous */
    const int32_t *lengths;       /* [batch] */
    int64_t dtype, batch, kv_heads, slots, dim, stride_batch, stride_head, stride_slot;
} df11_cache;

/* Attention over a bounded cache: query token t of sequence b, at position
 * pos[b] + t, sees the used slots whose position is at most its own; o as
 * in df11_prefix_attention.  weights[b, h', s] += the sum of the
 * probabilities that the query tokens and the heads / kv_heads heads of h'
 * gave slot s.  Every weight is added by one thread in a fixed order. */
typedef struct df11_cache_attention_args {
    const void *q;
    const int32_t *pos;           /* [batch] */
    void *out;                    /* [batch, tokens, heads, dim], contiguous; may be q itself */
    int64_t tokens, heads, q_batch, q_token, q_head;
    double scale;
} df11_cache_attention_args;

uint64_t df11_cache_attention_workspace_bytes(const df11_cache *c, const df11_cache_attention_args *a);
/* Workspace and errors as df11_prefix_attention. */
int df11_cache_attention(const df11_cache *c, const df11_cache_attention_args *a, void *workspace,
                         uint64_t workspace_bytes, void *stream);

/* One token into every sequence's cache: k_new, v_new [batch, kv_heads, dim]
 * (strides new_batch, new_head) at position pos[b], with weight 0.  Each key
 * head takes the slot lengths[b] while that is below `slots`; then the first
 * stale slot; then, of the slots whose position is at most pos[b] - recent
 * (the `recent` latest positions, the new one among them, are kept), the
 * one of least weight, the lowest of equals (a NaN weight counts as less
 * than any); and if there is none, the slot of the lowest position.  A
 * sequence with pos[b] < 0 takes no token.  No other slot is written: stale
 * ones that are left keep their positions (df11_cache above).  out_slots [batch, kv_heads]: the slot taken, or
 * -1.  out_lengths [batch]: min(lengths[b] + 1, slots), lengths[b] for a
 * sequence that takes none (lengths itself is not written; out_lengths must
 * be another array).  Errors: as df11_prefix_attention, and E_ARG for a cache
 * whose slots share memory (a stride smaller than what lies inside it). */
int df11_cache_insert(const df11_cache *c, const void *k_new, const void *v_new, int64_t new_batch,
                      int64_t new_head, const int32_t *pos, int64_t recent, int32_t *out_slots,
                      int32_t *out_lengths, void *stream);

/* A cache cut down to `budget` slots for each sequence and key head, into
 * another cache `out` (of out->slots >= budget slots, same batch, heads,
 * dim and type; out->lengths is not used; no memory shared with `c`).  With pos[b] the sequence's next
 * position: stale slots are dropped; of the others the `recent` latest
 * positions are kept, then the greatest weights, the lowest slot of equals
 * (NaN as above), `budget` in all; they keep their slot order.  kept [batch, kv_heads, out->slots]: the
 * slots of `c` that were kept, -1 behind them.  Slots of `out` behind the
 * kept ones are zero with weight 0 and position DF11_NO_TOKEN.  out_lengths[b] =
 * min(lengths[b], budget).  Errors: as df11_prefix_attention, and E_ARG for
 * recent > budget, budget > out->slots or an `out` whose slots share memory. */
int df11_cache_compact(const df11_cache *c, const int32_t *pos, int64_t budget, int64_t recent,
                       const df11_cache *out, int32_t *kept, int32_t *out_lengths, void *stream);

/* Verification of drafted tokens by rejection sampling, which leaves the
 * emitted tokens distributed as the target model's.  For each sequence the
 * drafts i = 0, 1, ... are taken in order while u_i * q_i(d_i) < p_i(d_i)
 * (p the target's probabilities, q the drafter's; the product exact).  At
 * the first one refused a token is drawn from max(p_i - q_i, 0), or from p
 * behind the last draft when all are taken, by the last uniform u: the
 * first token whose running sum exceeds u times the whole sum.  The sums are
 * taken over whole multiples of 2^-40 (each probability clamped to [0, 1],
 * NaN as 0, and cut to such a multiple), so no order of summation changes
 * them.  Where max(p - q, 0) is zero everywhere p is used; where that is zero
 * too the drawn token is -1. */
typedef struct df11_verify_args {
    const void *draft_tokens;     /* [batch, drafts], int32 or int64 (token_bytes 4 or 8), contiguous */
    const int32_t *counts;        /* [batch] drafts of each sequence (clamped to [0, drafts]), or NULL: all */
    const void *target_probs;     /* [batch, drafts + 1, vocab]; sequence b's row behind its last draft is counts[b] */
    const void *draft_probs;      /* [batch, drafts, vocab], or NULL: the drafter is certain, q(d) = 1 */
    const float *uniforms;        /* [batch, drafts + 1] in [0, 1), contiguous; the last one draws */
    void *tokens;                 /* [batch, drafts + 1]: the drafts taken, the drawn token, then -1 */
    int32_t *accepted;            /* [batch] drafts taken */
    int64_t dtype, token_bytes, batch, drafts, vocab;
    int64_t target_batch, target_row, draft_batch, draft_row;
} df11_verify_args;

uint64_t df11_verify_drafts_workspace_bytes(const df11_verify_args *a);
/* A drafted token outside [0, vocab) is refused (p = q = 0 there).  batch at most 65535, vocab at
 * most 2^22, drafts at most 1024.  Workspace as df11_prefix_attention.  Errors: E_ARG, E_DEVICE. */
int df11_verify_drafts(const df11_verify_args *a, void *workspace, uint64_t workspace_bytes, void *stream);

/* A cache held in 4 bits, in pages.  A row of `dim` values (a token's key or
 * value of one key head) lies in G groups, G = 2 for dims up to 64 and 4
 * above, dim d in group d mod G.  With a group's least and greatest value:
 *
 *   step   = (greatest - least) / 15, rounded to float32, then to `dtype`
 *   code_d = floor((x_d - least) / step + 1/2) in 64 bits, from 0 to 15 (0 where step is 0)
 *
 * and the code stands for code_d * step + least.  A group that holds a NaN
 * or an infinity gets a step and a least value of NaN; what comes of a group
 * with a step or least value that is no number is NaN or infinite.  codes: dim 2 i in the
 * low half of byte i; scales: (step, least) of each group.  A page holds
 * `page` positions (a multiple of 16) of every key head, a head's positions
 * one behind the other.  Strides between pages and heads are in bytes for
 * codes (multiples of 16), in elements for scales (multiples of 8); K and V share them. */
typedef struct df11_quantized_cache {
    void *k_codes, *v_codes;      /* [pages, kv_heads, page, dim / 2] bytes */
    void *k_scales, *v_scales;    /* [pages, kv_heads, page, G, 2] of dtype */
    int64_t dtype, pages, page, kv_heads, dim, code_page, code_head, scale_page, scale_head;
} df11_quantized_cache;

/* Position s of sequence b is row s % page of page
 * block_table[b * table_batch + s / page]; without a table sequence b has
 * page b alone.  A page id outside [0, pages) and a position outside the
 * sequence's pages hold nothing: nothing is written there, nothing seen. */

/* Token t < counts[b] (all `tokens` where counts is NULL; clamped to [0,
 * tokens]) of sequence b to position positions[b] + t.  k, v [batch, tokens,
 * kv_heads, dim] of the cache's type, any strides that are multiples of 8.
 * lengths[b] = positions[b] + the sequence's count.  Rows of other positions
 * stay as they are.  No two tokens of a call may go to the same row: what it
 * holds afterwards would be a mixture.  Errors: E_ARG (null or misaligned
 * pointer -- 16 bytes for k, v and the cache -- sizes or strides out of
 * range, pages, or keys and values, that share memory, lengths on positions or
 * counts), E_DEVICE. */
typedef struct df11_quantized_write_args {
    const void *k, *v;
    const int32_t *positions;     /* [batch] */
    const int32_t *counts;        /* [batch], or NULL */
    const int32_t *block_table;   /* [batch, table_pages], or NULL */
    int32_t *lengths;             /* [batch] */
    int64_t batch, tokens, table_pages, table_batch, k_batch, k_token, k_head, v_batch, v_token, v_head;
} df11_quantized_write_args;
int df11_quantized_write(const df11_quantized_cache *c, const df11_quantized_write_args *a, void *stream);

/* k, v [batch, count, kv_heads, dim], contiguous: the positions first[b] ..
 * first[b] + count - 1 (from 0 where first is NULL) of sequence b as the
 * values they stand for, taken in float32 and rounded to the cache's type, those
 * of numbers past its greatest one to that (the step of a group is rounded, so
 * that code 15 may stand for more than what was written); zeros from
 * lengths[b] on and where nothing is held.  Errors as df11_quantized_write, and
 * E_ARG for k and v that share memory. */
typedef struct df11_quantized_read_args {
    void *k, *v;
    const int32_t *first;         /* [batch], or NULL */
    const int32_t *lengths;       /* [batch] */
    const int32_t *block_table;   /* [batch, table_pages], or NULL */
    int64_t batch, count, table_pages, table_batch;
} df11_quantized_read_args;
int df11_quantized_read(const df11_quantized_cache *c, const df11_quantized_read_args *a, void *stream);

/* Attention over a quantised cache: the `tokens` query tokens of sequence b
 * are the last of its lengths[b] positions (a length outside what its pages
 * hold is taken as the nearer end), token t sees lengths[b] - (tokens - 1) +
 * t of them; o and lse as in df11_prefix_attention, over the values that the
 * codes stand for.  Rows that see nothing are zero, their lse -infinity.  What
 * unseen positions hold does not reach the output.  Statistics and sums are
 * float32; probabilities times steps are rounded to the operands' type, and
 * where more than 112 rows (tokens times heads of a key head) share their keys,
 * the probabilities and the values of V: to float16, those times a power of two
 * for their greatest, where no group of a range reaches 2^20 times as far as
 * another, else to the type (K's values, and V's of a float16 cache, are held to
 * twice as many bits); there a value of V is also off by up to 2^-13 of its step
 * where it is made.
 * Up to 112 rows values of V past 2^115 / n over n positions may come out infinite
 * or NaN (sums of n probabilities, held up to 2^8 high, times a step and 128 + a
 * code), and float16 holds a probability times a step to 2^-31 of
 * the greatest step among a sequence's positions, seen or not.
 * K may be what any finite row is written as; scale is positive and below
 * 2^125; logits past float32's range are no numbers.
 * Workspace and errors as df11_prefix_attention; the result does not depend
 * on the run. */
typedef struct df11_quantized_attention_args {
    const void *q;                /* [batch, tokens, heads, dim] */
    const int32_t *lengths;       /* [batch] */
    const int32_t *block_table;   /* [batch, table_pages], or NULL */
    void *out;                    /* [batch, tokens, heads, dim], contiguous; may be q itself, no other of its memory */
    float *lse;                   /* [batch, tokens, heads], or NULL */
    int64_t batch, tokens, heads, table_pages, table_batch, q_batch, q_token, q_head;
    double scale;
} df11_quantized_attention_args;
uint64_t df11_quantized_attention_workspace_bytes(const df11_quantized_cache *c, const df11_quantized_attention_args *a);
int df11_quantized_attention(const df11_quantized_cache *c, const df11_quantized_attention_args *a, void *workspace,
                             uint64_t workspace_bytes, void *stream);

/* A request's wishes on its next tokens' logits.  Row t of sequence b, token i:
 *
 *   x = logits[b, t, i]
 *   x = x > 0 ? x / repetition[b] : x * repetition[b]   if i was seen
 *   x = x - (frequency[b] * n + presence[b])            if n > 0
 *   x = x + the sum of the bias_values[b, j] with bias_tokens[b, j] = i
 *   x = -infinity                                       if bit i of mask[b, t] is 0
 *
 * Seen are the tokens history[b, 0 .. lengths[b]) and the drafts before the
 * row, draft_tokens[b, 0 .. t); n counts those of them behind the first
 * prompt_lengths[b] (clamped to [0, lengths[b]]; NULL: 0).  lengths are clamped to
 * [0, history_tokens].  Tokens outside [0, vocab) are passed over.  The terms
 * of a token are taken in 64 bits, then rounded to float32 and to
 * the type; the sum of a token's biases is taken in their order.  NULL: no such
 * term (logits without any are copied).  mask: words of 32 bits, bit i % 32
 * of word i / 32.  out may be logits itself (the same strides), or share no
 * memory with it; with other strides neither may lie between the other's rows. */
typedef struct df11_adjust_logits_args {
    const void *logits;           /* [batch, tokens, vocab], last axis contiguous */
    void *out;                    /* the same type; strides out_batch, out_token */
    const void *history;          /* [batch, history_tokens], int32 or int64 (token_bytes 4 or 8) */
    const int32_t *lengths;       /* [batch] */
    const int32_t *prompt_lengths;/* [batch], or NULL */
    const void *draft_tokens;     /* [batch, tokens - 1] of the same width, or NULL */
    const float *repetition, *presence, *frequency;   /* [batch] each, or NULL */
    const void *bias_tokens;      /* [batch, biases] of the same width, or NULL */
    const float *bias_values;     /* [batch, biases] */
    const int32_t *mask;          /* [batch, tokens, (vocab + 31) / 32], or NULL; strides mask_batch, mask_token */
    int64_t dtype, token_bytes, batch, tokens, vocab, history_tokens, biases;
    int64_t logits_batch, logits_token, out_batch, out_token, history_batch, draft_batch, bias_batch, mask_batch, mask_token;
} df11_adjust_logits_args;

/* batch and tokens at most 65535, vocab at most 2^22, biases at most 4096.
 * Errors: E_ARG (null or misaligned pointer, sizes or strides out of range,
 * rows of out that share memory, out on some of logits), E_DEVICE. */
int df11_adjust_logits(const df11_adjust_logits_args *a, void *stream);

/* ---------------------------------------------------------------- utilities */
const char *df11_status_string(int status);
const char *df11_last_error(void);
const char *df11_version(void);

#ifdef __cplusplus
}
#endif
#endif /* DF11_H */
