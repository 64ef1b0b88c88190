/*
 * df11.h -- C ABI of the DF11 (DFloat11) codec for one AMD Instinct MI355X (gfx950).
 *
 * The method: "DFloat11: Kompresi inferensi GPU lossless yang mengecilkan LLM
 * menjadi 70% ukurannya" (GeekNews, id.news.hada.io topic 20542).  Section
 * names below are that page's headings.
 *
 * A BF16 weight keeps its sign and 7-bit mantissa verbatim in one
 * PackedSignMantissa byte, while its 8-bit exponent is Huffman-coded into the
 * bit-packed EncodedExponent stream ("Format DFloat11").  Decoding walks a
 * hierarchy of 256-entry LUTs cut from height-8 subtrees of the code tree, the
 * unused exponent values 240..255 acting as pointers to lower LUTs, plus a
 * 256-byte CodeLengths table ("Decoding berbasis LUT hierarkis").  Each GPU
 * thread decodes the codes that start in its own n-byte segment, from a start
 * bit stored in Gaps; each thread block's first output index is stored once
 * ("Kernel GPU 2 tahap dan metadata bantu").
 *
 * Conventions for every function:
 *  - Return value: DF11_OK (0) or a negative df11_status.  Nothing throws across
 *    this ABI.  Validation runs before any write or launch; on failure no output
 *    buffer is written and no work is enqueued.
 *  - The caller owns every buffer, host and device.  The library never
 *    allocates, frees or synchronises device memory, and keeps no global state;
 *    host functions are reentrant.
 *  - Integers in buffers are little-endian; bit streams are MSB-first (bit p of a
 *    stream is bit 7 - p%8 of byte p/8).
 *  - "host" arguments are host pointers, "device" arguments are device pointers
 *    (hipMalloc'd or equivalent) on the current HIP device.
 */
#ifndef DF11_H
#define DF11_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Most elements one stream may hold: 2^32 - 2^16.  The decoders index
 * elements with 32-bit integers; the margin below 2^32 keeps every index
 * they form (a group's rounded chunk end, a wave's run of rounds ahead)
 * below 2^32 as well. */
#define DF11_MAX_ELEMENTS 4294901760ull

typedef enum df11_status {
    DF11_OK = 0,
    DF11_E_INVALID_ARG = -1,        /* null pointer, unsupported layout, bad size argument */
    DF11_E_RESERVED_EXPONENT = -2,  /* input has exponent >= 240 (Inf/NaN or |x| >= 2^113) */
    DF11_E_CODE_TOO_LONG = -3,      /* a Huffman code would exceed 32 bits */
    DF11_E_TOO_MANY_LUTS = -4,      /* the code tree needs more than 16 lower LUTs */
    DF11_E_BUFFER_TOO_SMALL = -5,   /* a caller buffer is smaller than required */
    DF11_E_BAD_STREAM = -6,         /* header fields or codebook are inconsistent */
    DF11_E_TOO_LARGE = -7,          /* N > DF11_MAX_ELEMENTS elements in one stream */
    DF11_E_HIP = -8                 /* a HIP launch or query failed */
} df11_status;

/* Exponent values 240..255 are pointers inside the LUTs, never symbols. */
#define DF11_FIRST_POINTER 240
/* The root LUT plus one lower LUT per pointer value. */
#define DF11_MAX_LUTS 17
/* Longest code; Gaps hold 5-bit offsets in [0, 31]. */
#define DF11_MAX_CODE_LEN 32
/* Size, in uint32 words, of the dynamic-schedule work counters
 * (df11_device_stream.schedule). */
#define DF11_SCHEDULE_WORDS 144
/* Most streams one df11_decompress_batch call decodes. */
#define DF11_MAX_BATCH 16
/* Token rows and smallest row length of df11_linear. */
#define DF11_LINEAR_MAX_TOKENS 8
#define DF11_LINEAR_MIN_IN_FEATURES 512

/* Element types of the operators around the products. */
#define DF11_BF16 0
#define DF11_FP16 1
#define DF11_FP32 2
/* Most tokens of a product with an epilogue whose decode is fused in. */
#define DF11_EPILOGUE_FUSED_TOKENS 32
/* Activations of the products' epilogues: none, max(z, 0), z / (1 + exp(-z)),
 * z Phi(z), and the tanh approximation of the last. */
#define DF11_ACT_NONE 0
#define DF11_ACT_RELU 1
#define DF11_ACT_SILU 2
#define DF11_ACT_GELU 3
#define DF11_ACT_GELU_TANH 4

/* The codebook shared by all tensors of one stream (host, plain data).
 *   code_lengths[e]: Huffman code length of exponent e, 0 if unused
 *                    (the page's CodeLengths table).
 *   codes[e]:        canonical code of e, right-aligned in code_lengths[e] bits.
 *   luts[i][x]:      LUT i indexed by the next 8 bits x.  A value v < 240 is an
 *                    exponent whose code ends within those 8 bits; v >= 240
 *                    points to LUT 256 - v for the following 8 bits.  LUT 0 is
 *                    the root; lower LUTs are numbered by depth, then prefix.
 *   n_luts:          number of LUTs in use (1..17).
 *   max_len:         longest code length (1..32). */
typedef struct df11_codebook {
    uint8_t code_lengths[256];
    uint32_t codes[256];
    uint8_t luts[DF11_MAX_LUTS][256];
    uint32_t n_luts;
    uint32_t max_len;
} df11_codebook;

/* Launch-shape parameters stored in the stream.
 *   bytes_per_thread (n):  EncodedExponent bytes per decoding thread; the
 *                          page's experiments use 8.  The encoder accepts n >= 4;
 *                          the GPU decoder supports n == 8.
 *   threads_per_group (G): threads per output-position block, a multiple of 64;
 *                          the GPU decoder supports G == 256. */
typedef struct df11_layout {
    uint32_t bytes_per_thread;
    uint32_t threads_per_group;
} df11_layout;

/* Stream header (host).  Buffer sizes include zero padding:
 *   enc_bytes     = round_up(n_threads * n, 16) + 16
 *   sm_bytes      = round_up(n_elements, 64)
 *   gaps_bytes    = 4 * (ceil(5 * n_threads / 32) + 1)
 *   out_pos_bytes = 4 * (n_groups + 1)
 * n_threads = ceil(total_bits / (8 n)), n_groups = ceil(n_threads / G).
 * max_group_elems is the largest out_pos[g+1] - out_pos[g]; df11_plan leaves it
 * at its upper bound G * 8n, df11_encode sets the exact value. */
typedef struct df11_header {
    uint64_t n_elements;
    uint64_t total_bits;
    uint32_t bytes_per_thread;
    uint32_t threads_per_group;
    uint64_t n_threads;
    uint64_t n_groups;
    uint32_t n_luts;
    uint32_t max_len;
    uint64_t enc_bytes;
    uint64_t sm_bytes;
    uint64_t gaps_bytes;
    uint64_t out_pos_bytes;
    uint32_t max_group_elems;
    uint32_t reserved;
} df11_header;

/* A stream resident in device memory (the struct itself is host memory).
 *   enc          device, h.enc_bytes     EncodedExponent, zero-padded
 *   sm           device, h.sm_bytes      PackedSignMantissa: sign in bit 7, mantissa in bits 0..6
 *   gaps         device, h.gaps_bytes    5-bit MSB-first start offsets, one per thread
 *   out_pos      device, n_groups + 1    first output index of each group; last entry N
 *   luts         device, n_luts * 256    df11_codebook.luts rows 0..n_luts-1
 *   code_lengths device, 256             df11_codebook.code_lengths
 *   decode_table device, df11_decode_table_bytes(decode_table_bits)
 *                                        built by df11_build_decode_table, or
 *                                        NULL: a caller holding only the page's
 *                                        arrays passes NULL, and every
 *                                        workgroup then derives the same table
 *                                        in LDS from luts and code_lengths
 *                                        (about a microsecond per launch)
 *   decode_table_bits                    index width of decode_table (10..12);
 *                                        0 with a NULL decode_table selects 11
 *   groups_per_workgroup                 launch shape: groups decoded together by one
 *                                        workgroup (1, 2 or 4); 0 picks the default
 *   schedule     device, DF11_SCHEDULE_WORDS uint32, or NULL
 *                                        work counters for dynamic load balancing:
 *                                        zero-filled by the caller once; every
 *                                        launch leaves them zero again.  Launches
 *                                        that share one must not overlap in time
 *                                        (use one per stream of work); within one
 *                                        batched launch, a stream whose counters
 *                                        an earlier stream of the batch also uses
 *                                        runs the static schedule.  NULL
 *                                        selects a static schedule, which is
 *                                        also used for streams too short to
 *                                        gain from balancing.
 *   max_workgroups                       launch at most this many workgroups (0: as
 *                                        many as fit on the GPU at once); a smaller
 *                                        grid leaves CUs to kernels running
 *                                        concurrently on other streams.  A
 *                                        batched launch takes the smallest cap
 *                                        of its streams and still gives every
 *                                        non-empty stream one workgroup, so it
 *                                        launches at most max(cap, streams).
 *   tile_cols                            0: the stream holds its elements in their
 *                                        own order.  Else the stream holds a
 *                                        (N / tile_cols) x tile_cols matrix in
 *                                        MFMA tile order (df11_tile_order;
 *                                        tile_cols a multiple of 32, N a
 *                                        multiple of 64 * tile_cols): the
 *                                        decompress entry points write it back
 *                                        row-major, and df11_matmul takes only
 *                                        such streams. */
typedef struct df11_device_stream {
    df11_header h;
    const uint8_t *enc;
    const uint8_t *sm;
    const uint8_t *gaps;
    const uint32_t *out_pos;
    const uint8_t *luts;
    const uint8_t *code_lengths;
    const void *decode_table;
    uint32_t decode_table_bits;
    uint32_t groups_per_workgroup;
    uint32_t *schedule;
    uint32_t max_workgroups;
    uint32_t tile_cols;
} df11_device_stream;

/* Accumulate the 256-bin exponent histogram of n BF16 words (host).
 * "Format DFloat11": the Huffman tree is built from the exponent distribution;
 * call once per tensor to share one codebook across tensors.
 * bf16: host, n uint16 BF16 bit patterns.  hist: host, 256 counters, accumulated
 * (not cleared).  DF11_E_RESERVED_EXPONENT if any exponent is >= 240
 * ("Decoding berbasis LUT hierarkis": those values are reused as pointers);
 * hist is then left unchanged. */
int df11_histogram(const uint16_t *bf16, uint64_t n, uint64_t hist[256]);

/* Build the codebook from a histogram (host): Huffman code lengths (ties broken
 * by (weight, id) with leaf id = exponent, merged node id = 256 + merge index),
 * canonical codes, CodeLengths and the hierarchical LUTs ("Format DFloat11",
 * "Decoding berbasis LUT hierarkis").  With fewer than two used exponents the
 * smallest unused exponents below 240 are added with weight 0.
 * Errors: DF11_E_RESERVED_EXPONENT (hist[e] > 0 for e >= 240),
 * DF11_E_CODE_TOO_LONG, DF11_E_TOO_MANY_LUTS.  cb is written only on success. */
int df11_build_codebook(const uint64_t hist[256], df11_codebook *cb);

/* Exact buffer sizes for n elements whose exponent histogram is hist (host).
 * Not on the page: the page fixes what the arrays hold, not how a caller
 * sizes them; this lets the caller allocate every buffer of df11_encode
 * before encoding.  hist must be the histogram of exactly the data that
 * df11_encode will see.  Fills every header field; max_group_elems is an
 * upper bound until encode. */
int df11_plan(const df11_codebook *cb, const uint64_t hist[256], uint64_t n, const df11_layout *lay,
              df11_header *h);

/* Encode n BF16 words (host) into caller buffers sized by df11_plan:
 * enc (h->enc_bytes), sm (h->sm_bytes), gaps (h->gaps_bytes), out_pos
 * (h->n_groups + 1 entries).  h must come from df11_plan for this data; on
 * success it is completed (total_bits, max_group_elems).  Every byte of the
 * buffers is written, padding included.
 * "Kernel GPU 2 tahap dan metadata bantu": gap_t is the bit offset of the first
 * code starting at or after bit 8 n t (the end of the stream counts as a code
 * start); out_pos[g] counts the codes that start before thread g G's segment.
 * Errors: DF11_E_RESERVED_EXPONENT, DF11_E_INVALID_ARG (an exponent without a
 * code, or h does not match the data), DF11_E_TOO_LARGE. */
int df11_encode(const df11_codebook *cb, const uint16_t *bf16, uint64_t n, const df11_layout *lay,
                df11_header *h, uint8_t *enc, uint8_t *sm, uint8_t *gaps, uint32_t *out_pos);

/* Reorder a rows x cols row-major BF16 matrix (host) into MFMA tile order,
 * the element order df11_matmul consumes.  Not on the page (the page fixes no
 * element order); the order of this library's matrix-core product.  Position
 * s of the ordered sequence holds W[r][c] with
 *   panel p = s / (64 cols), q = s mod (64 cols)
 *   k-step ks = q / 2048, u = q mod 2048
 *   n-tile nt = u / 512, v = u mod 512, lane l = v / 8, j = v mod 8
 *   r = 64 p + 16 nt + (l mod 16),  c = 32 ks + 8 (l / 16) + j
 * so every 8 consecutive elements are 8 consecutive columns of one row, and
 * each 512-element block is the B operand that the 64 lanes of a gfx950
 * v_mfma_f32_16x16x32_bf16 read for 16 rows x 32 columns of W.
 * w, out: host, rows * cols uint16, not overlapping.  rows a multiple of 64,
 * cols a multiple of 32, else DF11_E_INVALID_ARG. */
int df11_tile_order(const uint16_t *w, uint64_t rows, uint64_t cols, uint16_t *out);

/* Size in bytes of the decode table for index width bits (10..12), 0 if
 * unsupported.  Not on the page: the decode table is this decoder's own
 * derived data (see df11_build_decode_table). */
uint64_t df11_decode_table_bytes(uint32_t bits);

/* Build the GPU decoder's first-level table from the codebook (host).
 * The table is derived data, not part of the compressed format: for every
 * bits-wide window it lists the complete codes at the start of the window
 * (up to five exponents, their start offsets and their total length) so one LDS
 * lookup resolves several short codes; windows whose first code is longer than
 * the index width fall back to the page's LUT hierarchy.  Layout: for each
 * window x, uint32 words 2x (up to four rotated exponents, one per byte) and
 * 2x + 1 (codes << 11 | bits, the fifth exponent in bits 16..23), then one
 * uint16 start mask per window.
 * table: host, df11_decode_table_bytes(bits) bytes. */
int df11_build_decode_table(const df11_codebook *cb, uint32_t bits, void *table, uint64_t table_bytes);

/* Decompress a device-resident stream into out (device, h.n_elements uint16,
 * not aliasing any input), enqueued on hip_stream (a hipStream_t; NULL is the
 * null stream).  Returns after the launch; buffers must stay alive until the
 * stream's work completes.  Every element of out is overwritten with the
 * original BF16 bits ("Kernel GPU 2 tahap dan metadata bantu": per-thread
 * count, block prefix sum, re-decode into an LDS write buffer, coalesced
 * write).  A stream whose header is valid but whose payload is corrupt cannot
 * make the kernel access memory out of bounds; its output is unspecified.
 * Errors: DF11_E_INVALID_ARG (null pointers, unsupported n, G or
 * decode_table_bits), DF11_E_BAD_STREAM (header sizes inconsistent),
 * DF11_E_HIP (launch failed). */
int df11_decompress(const df11_device_stream *s, uint16_t *out, void *hip_stream);

/* Decompress the stream of a whole transformer block -- every linear weight of
 * the block encoded as one stream with a shared codebook -- into one scratch
 * buffer just before the block's forward pass ("Dekompresi per transformer
 * block").  scratch: device, scratch_elems uint16; views into it (element
 * offset, shape) are kept by the caller.  Same kernel and errors as
 * df11_decompress, plus DF11_E_BUFFER_TOO_SMALL if scratch_elems < N. */
int df11_decompress_block(const df11_device_stream *s, uint16_t *scratch, uint64_t scratch_elems,
                          void *hip_stream);

/* Decompress several independent streams -- each with its own codebook,
 * decode table and output -- in one launch, for instance every linear weight
 * of a transformer block encoded with a codebook of its own ("Dekompresi per
 * transformer block" batches a block's matrices into one launch because a
 * single matrix is too small to fill the GPU).  The grid is divided between
 * the streams in proportion to their work.
 *   streams  host array of n_streams device streams (as for df11_decompress);
 *            all non-empty ones must use the same decode_table_bits and
 *            groups_per_workgroup
 *   outs     host array of n_streams device pointers; outs[i] receives
 *            streams[i].h.n_elements uint16, 16-byte aligned, and may not
 *            overlap any other output or any stream's buffers
 * Streams with N = 0 are skipped.  Errors: DF11_E_TOO_LARGE (n_streams >
 * DF11_MAX_BATCH), DF11_E_INVALID_ARG (mismatched table widths or launch
 * shapes, overlapping buffers, or as for df11_decompress), DF11_E_BAD_STREAM,
 * DF11_E_HIP.  Nothing is launched unless every stream is valid. */
int df11_decompress_batch(const df11_device_stream *streams, uint32_t n_streams, uint16_t *const *outs,
                          void *hip_stream);

/* df11_decompress_batch for callers that cannot allocate device memory or
 * own work-counter buffers (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc): the same decode, with each
 * stream's dynamic-schedule counters taken from a fixed device array inside
 * the library (DF11_MAX_BATCH sets of DF11_SCHEDULE_WORDS uint32, 9 KB per
 * GPU, held until the process ends) instead of streams[i].schedule, which is
 * ignored.  The call allocates nothing: it launches a small kernel that zeroes
 * the counters of this call's streams, then the decode, both on hip_stream.
 * Every call on one GPU shares that array, so calls that overlap in time on
 * one GPU race (serialize them, e.g. on one stream).  Arguments, output and
 * errors as for df11_decompress_batch; DF11_E_TOO_LARGE for more than
 * DF11_MAX_BATCH streams, DF11_E_HIP if the array's device address cannot
 * be found. */
int df11_decompress_batch_noalloc(const df11_device_stream *streams, uint32_t n_streams, uint16_t *const *outs,
                                  void *hip_stream);

/* df11_decompress with the decode kernel timed by the GPU: start_event and
 * stop_event (hipEvent_t created by the caller, either may be NULL) are
 * recorded when the kernel itself starts and ends, so hipEventElapsedTime of
 * the pair is the kernel's duration without the launch gap.  Used to measure
 * the decoder; same arguments, output and errors as df11_decompress.  With a
 * stream of N = 0 nothing is launched and the events are not recorded. */
int df11_decompress_timed(const df11_device_stream *s, uint16_t *out, void *hip_stream, void *start_event,
                          void *stop_event);

/* df11_decompress_batch with the batched kernel timed like
 * df11_decompress_timed: start_event and stop_event (either may be NULL) are
 * recorded when the kernel itself starts and ends.  Same arguments, output
 * and errors as df11_decompress_batch; when every stream is empty nothing is
 * launched and the events are not recorded. */
int df11_decompress_batch_timed(const df11_device_stream *streams, uint32_t n_streams, uint16_t *const *outs,
                                void *hip_stream, void *start_event, void *stop_event);

/* y = x W^T with the decompression fused into the matrix product: W is the
 * stream decoded and viewed as an out_features x in_features row-major BF16
 * matrix, and its BF16 values never reach HBM.  The page's section
 * "Dekompresi yang disesuaikan untuk inferensi GPU" decompresses each weight
 * matrix right before its matrix multiplication; the section "Opini Hacker
 * News" suggests a GEMM that decompresses each tile before the arithmetic,
 * which this is for small token counts (token-by-token generation), where the
 * product is bound by reading W.
 *   w             device stream, h.n_elements == out_features * in_features,
 *                 elements in their own (row-major) order: tile_cols == 0
 *   x             device, n_tokens x in_features BF16 (uint16 bit patterns),
 *                 row-major, 16-byte aligned; read only
 *   n_tokens      1 .. DF11_LINEAR_MAX_TOKENS
 *   in_features   a multiple of 8, at least DF11_LINEAR_MIN_IN_FEATURES
 *   y             device, n_tokens x out_features float, row-major, 4-byte
 *                 aligned, overlapping neither x nor the stream's buffers;
 *                 every element is overwritten
 * y[t][r] is the sum over c of x[t][c] * W[r][c], each product exact in float
 * and the sums taken in float in an unspecified order (atomic adds), so the
 * low bits can differ between calls.  Enqueued on hip_stream (a zeroing kernel
 * for y, then the decode kernel); uses w's schedule counters like
 * df11_decompress, so calls sharing a stream descriptor must not overlap in
 * time.  Errors: DF11_E_INVALID_ARG (sizes, alignment, overlap, or as for
 * df11_decompress), DF11_E_BAD_STREAM, DF11_E_TOO_LARGE (n_tokens *
 * out_features >= 2^32), DF11_E_HIP.  With N = 0 (out_features = 0) nothing
 * is launched. */
int df11_linear(const df11_device_stream *w, const uint16_t *x, uint32_t n_tokens, uint32_t in_features,
                uint32_t out_features, float *y, void *hip_stream);

/* df11_linear accumulating into y: y += x W^T, with the same arguments,
 * sums and errors, and no zeroing kernel; y must hold the values to add to
 * (zeros, say, set once for several products that share one buffer). */
int df11_linear_acc(const df11_device_stream *w, const uint16_t *x, uint32_t n_tokens, uint32_t in_features,
                    uint32_t out_features, float *y, void *hip_stream);

/* df11_linear with start_event and stop_event (hipEvent_t, either may be
 * NULL) recorded when the fused kernel itself starts and ends (the zeroing
 * kernel before it is not included), to measure the fused product.  Same
 * arguments, output and errors. */
int df11_linear_timed(const df11_device_stream *w, const uint16_t *x, uint32_t n_tokens, uint32_t in_features,
                      uint32_t out_features, float *y, void *hip_stream, void *start_event, void *stop_event);

/* df11_linear for several weight matrices that multiply the same x -- a
 * transformer block's q, k and v projections, or its gate and up projections
 * -- in one launch, the grid split between them in proportion to their work
 * (small matrices alone cannot fill the GPU).
 *   ws            host array of n_streams device streams (as for df11_linear);
 *                 the non-empty ones must share decode_table_bits
 *   x, n_tokens, in_features   shared by all, as for df11_linear
 *   out_features  host array: rows of each matrix
 *   ys            host array of device outputs, n_tokens x out_features[i]
 *                 floats each, overlapping neither each other, x nor any
 *                 stream's buffers; overwritten
 *   start_event, stop_event   hipEvent_t or NULL, recorded at the fused
 *                 kernel's own start and end
 * One kernel zeroes every output, then one fused kernel runs.  Errors:
 * DF11_E_TOO_LARGE (n_streams > DF11_MAX_BATCH, or the outputs' total
 * >= 2^32 floats), DF11_E_INVALID_ARG (as for df11_linear, mismatched table
 * widths, overlaps), DF11_E_BAD_STREAM, DF11_E_HIP.  Nothing is launched
 * unless every stream is valid. */
int df11_linear_batch(const df11_device_stream *ws, uint32_t n_streams, const uint16_t *x, uint32_t n_tokens,
                      uint32_t in_features, const uint32_t *out_features, float *const *ys, void *hip_stream,
                      void *start_event, void *stop_event);

/* df11_linear_batch accumulating into every output: ys[i] += x W_i^T, with
 * the same arguments and errors and no zeroing kernel. */
int df11_linear_batch_acc(const df11_device_stream *ws, uint32_t n_streams, const uint16_t *x, uint32_t n_tokens,
                          uint32_t in_features, const uint32_t *out_features, float *const *ys, void *hip_stream,
                          void *start_event, void *stop_event);

/* y = x W^T on the matrix cores with the decompression fused in, for any
 * number of tokens: the page's section "Dekompresi yang disesuaikan untuk
 * inferensi GPU" decompresses each weight matrix right before its matrix
 * multiplication and discards the BF16 copy; the section "Opini Hacker News"
 * suggests a GEMM that decompresses each tile before the arithmetic.  Here
 * every decoded 16 x 32 tile of W goes from the decoder's registers straight
 * into v_mfma_f32_16x16x32_bf16 with the matching tile of x; W's BF16 never
 * reaches HBM.
 *   w             device stream in MFMA tile order: tile_cols == in_features
 *                 (df11_tile_order), h.n_elements == out_features * in_features
 *   x             device, n_tokens x in_features BF16, row-major, 16-byte
 *                 aligned, finite values; read only
 *   n_tokens      >= 1; the stream is swept once per 64 tokens (once up to 16,
 *                 32 or 64)
 *   in_features   a multiple of 32;  out_features a multiple of 64
 *   y             device, n_tokens x out_features float, row-major, 4-byte
 *                 aligned, overlapping neither x nor the stream's buffers;
 *                 every element is overwritten
 * y[t][r] is the sum over c of x[t][c] * W[r][c]: products exact in float,
 * sums in float in an unspecified order (partial sums of a row from several
 * workgroups meet in float atomics), so the low bits can differ between
 * calls.  Enqueued on hip_stream: a zeroing kernel for y, then the fused
 * kernel.  Up to 8 tokens, a stream with schedule counters and at least 12
 * super-groups (2 groups) per workgroup sweeps fixed ranges over 95% of them
 * and hands the rest out with its counters (which launches sharing them
 * must not overlap in time, as for df11_decompress); otherwise the counters
 * are not used.  Not on the page (a load-balancing choice).  Errors:
 * DF11_E_INVALID_ARG (sizes, alignment, overlap, a stream not in tile order,
 * or as for df11_decompress), DF11_E_BAD_STREAM, DF11_E_TOO_LARGE
 * (n_tokens * out_features >= 2^32), DF11_E_HIP. */
int df11_matmul(const df11_device_stream *w, const uint16_t *x, uint32_t n_tokens, uint32_t in_features,
                uint32_t out_features, float *y, void *hip_stream);

/* df11_matmul accumulating into y (y += x W^T): no zeroing kernel. */
int df11_matmul_acc(const df11_device_stream *w, const uint16_t *x, uint32_t n_tokens, uint32_t in_features,
                    uint32_t out_features, float *y, void *hip_stream);

/* df11_matmul with start_event and stop_event (hipEvent_t, either may be
 * NULL) recorded when the fused kernel itself starts and ends. */
int df11_matmul_timed(const df11_device_stream *w, const uint16_t *x, uint32_t n_tokens, uint32_t in_features,
                      uint32_t out_features, float *y, void *hip_stream, void *start_event, void *stop_event);

/* df11_matmul for several weight matrices in one launch, each with its own
 * x and y (a transformer block's q, k and v on one x, or gate and up; or
 * every product of a step), the grid split between them in proportion to
 * their work: small matrices alone cannot fill the GPU, and one launch pays
 * one start and one tail.
 *   ws            host array of n_streams device streams, as for df11_matmul;
 *                 the non-empty ones must share decode_table_bits
 *   xs            host array of device x pointers (xs[i]: n_tokens x
 *                 in_features[i] BF16), may repeat
 *   in_features, out_features   host arrays, as for df11_matmul
 *   ys            host array of device outputs, n_tokens x out_features[i]
 *                 floats, overlapping neither each other, any x nor any
 *                 stream's buffers
 *   accumulate    0: every output is overwritten (one zeroing kernel runs
 *                 first); else ys[i] += xs[i] W_i^T
 *   start_event, stop_event   hipEvent_t or NULL, recorded at the fused
 *                 kernel's own start and end
 * The schedule counters serve as for df11_matmul when every non-empty stream
 * qualifies and none shares its counters with an earlier stream of the
 * batch; otherwise the whole launch sweeps fixed ranges.  Errors:
 * DF11_E_TOO_LARGE (n_streams > DF11_MAX_BATCH, the outputs' total >= 2^32
 * floats), as for df11_matmul otherwise.  Nothing is launched unless every
 * stream is valid. */
int df11_matmul_batch(const df11_device_stream *ws, uint32_t n_streams, const uint16_t *const *xs, uint32_t n_tokens,
                      const uint32_t *in_features, const uint32_t *out_features, float *const *ys, int accumulate,
                      void *hip_stream, void *start_event, void *stop_event);

/* ---------------------------------------------------------------------------
 * Operators around the products of a transformer block.  Not on the page,
 * which leaves everything but the weights to the framework that runs the
 * model: what a forward through compressed weights computes between one
 * product and the next.  Strides are in elements.  A buffer of elements is
 * aligned to one element unless stated otherwise; 16-byte aligned rows are
 * read and written fastest.  Every sum is taken in float in an
 * order that the shapes alone fix, so that a call's results do not change
 * from run to run, and every result is rounded once.  None of these calls
 * uses memory of the library's own: calls that share no output and no
 * workspace may overlap in time, unless stated otherwise.
 * ------------------------------------------------------------------------- */

/* RMS norm with the residual's addition:
 *   s = round(x + residual), or x without a residual
 *   y = s * rstd * weight, rstd = 1 / sqrt(mean(s^2) + eps)
 * with s rounded to the rows' type first, so that y is the norm of the very
 * values that the residual stream carries on.
 *   x          device, rows x cols of dtype (DF11_BF16, DF11_FP16, DF11_FP32),
 *              x_stride from row to row
 *   residual   device, rows x cols of dtype, or NULL
 *   weight     device, cols of weight_dtype (dtype or DF11_FP32), or NULL (ones)
 *   rows       0 .. 2^30; with 0 nothing is launched
 *   cols       1 .. 2^30
 *   sum        device, rows x cols, receives s; or NULL.  Only with a residual
 *   y          device, rows x cols
 *   rstd       device, rows floats, or NULL; kept for df11_rms_norm_grad
 * sum and y may each lie exactly on x or on residual (same address and
 * stride), but not on each other.  A row with a NaN is NaN throughout; one with
 * an infinity is NaN there and zero elsewhere, and one whose squares pass
 * float's range (magnitudes of 1e19) is zero; other rows are not touched by
 * either.  Errors: DF11_E_INVALID_ARG (types, sizes, alignment,
 * output rows that overlap, other overlaps), DF11_E_HIP. */
int df11_rms_norm(const void *x, uint64_t x_stride, const void *residual, uint64_t residual_stride,
                  const void *weight, uint32_t weight_dtype, uint32_t rows, uint32_t cols, uint32_t dtype, float eps,
                  void *sum, uint64_t sum_stride, void *y, uint64_t y_stride, float *rstd, void *hip_stream);

/* Bytes of df11_rms_norm_grad's workspace when it computes dweight. */
uint64_t df11_rms_norm_grad_workspace(uint32_t rows, uint32_t cols);

/* Gradients of df11_rms_norm, with h = s * rstd:
 *   dx = rstd * (dy * weight - h * mean(dy * weight * h)) + dsum
 *   dweight = sum over the rows of dy * h
 * dx is the gradient of x and of residual alike.
 *   s, rstd      the forward call's sum (x itself without a residual) and rstd
 *   dy, dsum     device, rows x cols of dtype: the gradients of y and, or
 *                NULL, of sum
 *   dx           device, rows x cols of dtype; may lie exactly on s, dy or dsum
 *   dweight      device, cols of weight_dtype, or NULL; needs weight.  With no
 *                rows it is zero
 *   workspace    device, 16-byte aligned, df11_rms_norm_grad_workspace bytes
 *                (with dweight; else it may be NULL)
 * Errors: as for df11_rms_norm, DF11_E_BUFFER_TOO_SMALL. */
int df11_rms_norm_grad(const void *s, uint64_t s_stride, const void *weight, uint32_t weight_dtype, const float *rstd,
                       const void *dy, uint64_t dy_stride, const void *dsum, uint64_t dsum_stride, uint32_t rows,
                       uint32_t cols, uint32_t dtype, void *dx, uint64_t dx_stride, void *dweight, void *workspace,
                       uint64_t workspace_bytes, void *hip_stream);

/* What a product does with its sums z before it writes them (host struct of
 * device pointers):
 *   df11_matmul_epilogue   out = act(z + bias[0]) + residual
 *   df11_gated_matmul      out = act(z0 + bias[0]) * (z1 + bias[1]) + residual
 *   bias             device, out_features of bias_dtype, or NULL; bias[1] only
 *                    for a gated product
 *   residual         device, n_tokens x out_features of residual_dtype,
 *                    residual_stride elements from row to row, or NULL
 *   out              device, n_tokens x out_features of out_dtype; may lie
 *                    exactly on residual (same address, stride and type)
 *   pre              device, n_tokens x out_features floats each, row-major,
 *                    16-byte aligned: receive z + bias (both or neither for a gated product),
 *                    for df11_matmul_epilogue_grad; or NULL
 *   activation       one of DF11_ACT_*
 * Types are DF11_BF16 or DF11_FP32.  Everything up to out is float; out is
 * rounded once. */
typedef struct df11_epilogue {
    const void *bias[2];
    const void *residual;
    void *out;
    float *pre[2];
    uint64_t residual_stride;
    uint64_t out_stride;
    uint32_t bias_dtype;
    uint32_t residual_dtype;
    uint32_t out_dtype;
    uint32_t activation;
} df11_epilogue;

/* Bytes of the workspace of df11_matmul_epilogue (up NULL) or
 * df11_gated_matmul for n_tokens tokens on the current device; 0 for streams
 * that those calls refuse, or where nothing needs computing. */
uint64_t df11_epilogue_workspace(const df11_device_stream *w, const df11_device_stream *up, uint32_t n_tokens);

/* y = act(x W^T + bias) + residual with W compressed, for any number of
 * tokens: df11_matmul with its epilogue.
 *   w             device stream in MFMA tile order, as for df11_matmul
 *   x             device, n_tokens x in_features BF16, 16-byte aligned, x_stride
 *                 elements (a multiple of 8) from row to row
 *   in_features   a multiple of 32, with x_stride at most 2^22;  out_features a
 *                 multiple of 64
 *   workspace     device, 256-byte aligned, df11_epilogue_workspace bytes; holds
 *                 nothing between calls, but calls that overlap in time need
 *                 one each
 * Sums are taken in float in an order fixed by the stream, the shapes and the
 * device, not by timing.  A token whose x holds an infinity or a NaN gives
 * infinities or NaN in its own sums alone (0 * inf included: a weight of zero
 * does not hide it, and where two ranges of the stream meet, up to
 * DF11_EPILOGUE_FUSED_TOKENS tokens, a sum may be NaN for an infinity).  Up to DF11_EPILOGUE_FUSED_TOKENS tokens the decode
 * is fused into the product; beyond, the stream is decoded into the workspace.
 * A stream's schedule counters are not used: calls of one stream may overlap in
 * time, on any streams and from any threads, and so may a captured call's
 * replays (but not two replays of one graph, which have the same outputs).
 * With no tokens or no outputs nothing is launched.  Errors: DF11_E_INVALID_ARG,
 * DF11_E_BAD_STREAM, DF11_E_TOO_LARGE (n_tokens * features >= 2^32),
 * DF11_E_BUFFER_TOO_SMALL, DF11_E_HIP. */
int df11_matmul_epilogue(const df11_device_stream *w, const uint16_t *x, uint64_t x_stride, uint32_t n_tokens,
                         uint32_t in_features, uint32_t out_features, const df11_epilogue *e, void *workspace,
                         uint64_t workspace_bytes, void *hip_stream);

/* The gated product of a feed-forward block, both projections in one launch:
 *   out = act(x Wg^T + bias[0]) * (x Wu^T + bias[1]) + residual
 * gate and up have the same shape and decode_table_bits and may be the same
 * stream.  Otherwise as df11_matmul_epilogue. */
int df11_gated_matmul(const df11_device_stream *gate, const df11_device_stream *up, const uint16_t *x,
                      uint64_t x_stride, uint32_t n_tokens, uint32_t in_features, uint32_t out_features,
                      const df11_epilogue *e, void *workspace, uint64_t workspace_bytes, void *hip_stream);

/* What a product's backward pass reads and writes (host struct of device
 * pointers).  With z the sums after the bias that the forward call kept in
 * df11_epilogue.pre, dy the gradient of its output:
 *   one weight   dz = dy * act'(z);  dx = dz W
 *   gated        dz0 = dy * z1 * act'(z0), dz1 = dy * act(z0);
 *                dx = dz0 Wg + dz1 Wu
 *   dbias[i] = sum over the tokens of dz_i
 * (the residual's gradient is dy itself; the weights are frozen.)
 *   dy           device, n_tokens x out_features of dy_dtype, dy_stride
 *                elements from row to row
 *   pre          16-byte aligned; unused (may be NULL) for one weight without
 *                an activation
 *   dx           device, n_tokens x in_features of dx_dtype, or NULL
 *   dbias        device, out_features of bias_dtype each, or NULL
 * Types are DF11_BF16 or DF11_FP32.  dz is rounded to BF16 for dx, the matrix
 * cores' operand type (at most 2^-8 of each dz), and stays float for dbias. */
typedef struct df11_product_grad {
    const void *dy;
    const float *pre[2];
    void *dx;
    void *dbias[2];
    uint64_t dy_stride;
    uint64_t dx_stride;
    uint32_t dy_dtype;
    uint32_t dx_dtype;
    uint32_t bias_dtype;
    uint32_t activation;
} df11_product_grad;

/* Bytes of df11_matmul_epilogue_grad's workspace on the current device; 0 for
 * streams that the call refuses, or where nothing needs computing. */
uint64_t df11_epilogue_grad_workspace(const df11_device_stream *w, const df11_device_stream *up, uint32_t n_tokens,
                                      const df11_product_grad *g);

/* The backward pass of df11_matmul_epilogue (up NULL) or df11_gated_matmul,
 * through the frozen compressed weights: the streams are decoded into the
 * workspace.  Sizes, streams, workspace, sums and errors as for the forward
 * calls, and out_features at most 2^22; no output may overlap anything else.
 * With no tokens dbias is zero; with no out_features nothing is launched, dx
 * stays as it is. */
int df11_matmul_epilogue_grad(const df11_device_stream *w, const df11_device_stream *up, uint32_t n_tokens,
                              uint32_t in_features, uint32_t out_features, const df11_product_grad *g,
                              void *workspace, uint64_t workspace_bytes, void *hip_stream);

/* The softmax cross entropy through a compressed output head, without keeping
 * the logits (host struct of device pointers).  With z = x W^T over the classes
 * 0 .. vocab - 1,
 *   loss = log(sum over v of exp(z_v)) - z_target
 *   grad = d loss / dx = sum over v of p_v W_v - W_target,  p = softmax(z)
 *   targets        n_tokens int64.  A token whose target is ignore_index has a
 *                  loss of zero and a gradient of minus zero; one whose target is
 *                  no class otherwise, NaN
 *   loss           n_tokens floats
 *   total          a float, or NULL: the sum of loss over the tokens, divided by
 *                  their number if mean
 *   count          a float, or NULL: that number (tokens not ignored)
 *   grad           n_tokens x in_features floats, 16-byte aligned, or NULL; kept
 *                  for df11_cross_entropy_grad
 *   vocab          1 .. out_features; W's rows from there on are padding
 *   mean           0 or 1 */
typedef struct df11_loss {
    const int64_t *targets;
    float *loss;
    float *total;
    float *count;
    float *grad;
    int64_t ignore_index;
    uint32_t vocab;
    uint32_t mean;
} df11_loss;

/* Bytes of df11_cross_entropy's workspace on the current device (with_grad: with
 * l->grad); 0 for streams that the call refuses, or where nothing needs
 * computing. */
uint64_t df11_cross_entropy_workspace(const df11_device_stream *w, uint32_t n_tokens, int with_grad);

/* The loss, and with l->grad its gradient with respect to x in the same call, W
 * frozen.  Logits are float and never stored; a token's sum of exponentials is
 * taken without the target's own, so that the loss and p_target - 1 keep their
 * relative accuracy where the target is all but certain.  For grad the other
 * exponentials are rounded to BF16, the matrix cores' operand type (at most 2^-8
 * of each), piece by piece of the vocabulary, and its sums are float.
 *   w, x, in_features, out_features   as for df11_matmul_epilogue, out_features
 *                and in_features up to 2^22, n_tokens * in_features below 2^32
 *                and with l->grad n_tokens below 2^24
 *   workspace    device, 256-byte aligned, df11_cross_entropy_workspace bytes;
 *                holds nothing between calls, but calls that overlap in time need
 *                one each
 * A token whose x holds an infinity or a NaN, or whose target's logit overflows, or
 * another's to plus infinity, gets NaN (one at minus infinity has p = 0); other
 * tokens are not touched by it.  Results do not change from run to run; calls of
 * one stream may overlap in time.  With no tokens only total and count are
 * written.
 * Errors: DF11_E_INVALID_ARG, DF11_E_BAD_STREAM, DF11_E_TOO_LARGE,
 * DF11_E_BUFFER_TOO_SMALL, DF11_E_HIP. */
int df11_cross_entropy(const df11_device_stream *w, const uint16_t *x, uint64_t x_stride, uint32_t n_tokens,
                       uint32_t in_features, uint32_t out_features, const df11_loss *l, void *workspace,
                       uint64_t workspace_bytes, void *hip_stream);

/* x's gradient from the one that df11_cross_entropy kept: dx = g grad, rounded
 * once, where a token's g is dy[token * dy_stride], or with count (the call's, of a
 * mean) that over count (zero if it is zero).  An element of grad that is minus zero
 * (ignored tokens' are, no other's) gives zero whatever g is.  dy_stride 0: one
 * dy for all tokens.  dx: n_tokens x in_features of dx_dtype (DF11_BF16 or
 * DF11_FP32), dx_stride elements from row to row, overlapping nothing else.
 * n_tokens below 2^24.
 * Errors: DF11_E_INVALID_ARG, DF11_E_TOO_LARGE, DF11_E_HIP. */
int df11_cross_entropy_grad(const float *grad, const float *dy, uint64_t dy_stride, const float *count,
                            uint32_t n_tokens, uint32_t in_features, void *dx, uint64_t dx_stride, uint32_t dx_dtype,
                            void *hip_stream);

/* ---------------------------------------------------------------------------
 * A paged cache of keys and values, and attention over it.  Not on the page.
 * Sequence s of a batch holds lengths[s] tokens in the cache and brings the
 * new tokens starts[s] .. starts[s + 1] - 1 of the batch: its i-th new token
 * belongs at place lengths[s] + i, which lies in page
 * page_table[s][place / page_size] at place % page_size.  What the arrays on
 * the device hold is not known to the host; the kernels check it: a token
 * before starts[0] or behind starts[n_seqs] belongs to no sequence, and a place
 * beyond table_pages pages, or in a page outside 0 .. n_pages - 1, is neither
 * read nor written.  A stride along a dimension of one element is not used.
 * (Starts that decrease give unspecified results, in
 * bounds.)  All types are DF11_BF16, DF11_FP16 or, where stated, DF11_FP32.
 * ------------------------------------------------------------------------- */

/* Largest head_dim. */
#define DF11_MAX_HEAD_DIM 256

/* The cache (host struct of device pointers).  Element (page, place, head, d) of
 * k is at page * k_page_stride + place * k_place_stride + head * k_head_stride +
 * d, so that (pages, page_size, heads, head_dim) and (pages, heads, page_size,
 * head_dim) both fit; likewise v.
 *   k, v       16-byte aligned, strides multiples of 8, below 2^40
 *   n_pages    1 .. 2^31 - 1;  page_size 1 .. 2^20;  heads 1 .. 4096
 *   head_dim   a multiple of 8, 8 .. DF11_MAX_HEAD_DIM
 *   dtype      DF11_BF16 or DF11_FP16 */
typedef struct df11_kv_cache {
    void *k;
    void *v;
    uint64_t k_page_stride, k_place_stride, k_head_stride;
    uint64_t v_page_stride, v_place_stride, v_head_stride;
    uint32_t n_pages;
    uint32_t page_size;
    uint32_t heads;
    uint32_t head_dim;
    uint32_t dtype;
    uint32_t reserved;
} df11_kv_cache;

/* The batch (host struct of device pointers).
 *   starts       n_seqs + 1, not decreasing
 *   lengths      n_seqs
 *   page_table   n_seqs x table_pages, table_stride from sequence to sequence;
 *                table_pages * page_size at most 2^30
 *   n_tokens     rows of the call's per-token arrays, 0 .. 2^24 */
typedef struct df11_kv_batch {
    const int32_t *starts;
    const int32_t *lengths;
    const int32_t *page_table;
    uint64_t table_stride;
    uint32_t n_seqs;
    uint32_t table_pages;
    uint32_t n_tokens;
    uint32_t reserved;
} df11_kv_batch;

/* What df11_append_kv takes beside them (host struct of device pointers).
 *   k, v          n_tokens x heads x head_dim of dtype: element (token, head, d)
 *                 at token * stride + head * head_stride + d
 *   q             n_tokens x q_heads x head_dim of dtype, q_heads 1 .. 4096; or
 *                 NULL, with q_heads 0
 *   q_out         n_tokens x q_heads x head_dim of the cache's dtype; with q only.
 *                 May lie exactly on q (same address, strides and type).  q, k and
 *                 v may be parts of the rows of one tensor
 *   rotary        rotary_rows x rotary_dims floats: row p holds the cosines of
 *                 position p's angles, then their sines; or NULL (no rotation)
 *   rotary_dims   even, 2 .. head_dim: the dimensions of a head that are rotated,
 *                 in pairs (d, d + rotary_dims / 2), or (2 d, 2 d + 1) if
 *                 interleaved; the others are copied
 *   positions     n_tokens, or NULL (every token's place)
 *   dtype         DF11_BF16, DF11_FP16 or DF11_FP32
 * Strides below 2^40, of heads below 2^32. */
typedef struct df11_append {
    const void *k;
    const void *v;
    const void *q;
    void *q_out;
    const float *rotary;
    const int32_t *positions;
    uint64_t k_stride, k_head_stride;
    uint64_t v_stride, v_head_stride;
    uint64_t q_stride, q_head_stride;
    uint64_t q_out_stride, q_out_head_stride;
    uint64_t rotary_rows;
    uint32_t rotary_dims;
    uint32_t interleaved;
    uint32_t q_heads;
    uint32_t dtype;
} df11_append;

/* Appends the new tokens' keys and values to the cache, rotated on the way, and
 * rotates their queries: a pair (a, b) becomes (a cos - b sin, b cos + a sin),
 * in float and rounded once to the cache's type; v is copied.  A position
 * outside the table gives NaN.  Rows of q_out that belong to no sequence are
 * left as they were, and so is the rest of the cache.  Places that two tokens
 * share receive either one's elements.  One launch; with no tokens none.
 * Places, heads and pages lie apart: of each half every stride steps over all that
 * the smaller ones reach, and so do the halves of each other, which may be parts of
 * one tensor.  Errors: DF11_E_INVALID_ARG (types, sizes, alignment, overlaps, also of
 * the cache's places), DF11_E_HIP. */
int df11_append_kv(const df11_kv_cache *cache, const df11_kv_batch *batch, const df11_append *a, void *hip_stream);

/* What df11_tree_attention takes beside the cache and the batch (host struct of
 * device pointers).
 *   q, out       n_tokens x q_heads x head_dim of the cache's dtype: element
 *                (token, head, d) at token * stride + head * head_stride + d;
 *                16-byte aligned, strides multiples of 8.  Query head h reads
 *                key head h / (q_heads / heads).  out may lie exactly on q
 *   lse          n_tokens x q_heads floats, or NULL: the natural logarithm of the
 *                sum of exp(scale q . k) over what the query sees
 *   mask         n_tokens x mask_cols bytes, mask_stride from token to token, or
 *                NULL.  Every query sees the lengths[s] cached places of its
 *                sequence; of the sequence's new tokens it sees the j-th if byte
 *                j of its row is not zero (none from mask_cols on), or without a
 *                mask those up to itself.  (With mask_cols 0 a mask is any address
 *                but NULL, of which nothing is read)
 *   scale        positive, finite
 *   q_heads      a multiple of the cache's heads, at most 4096 */
typedef struct df11_attention {
    const void *q;
    void *out;
    float *lse;
    const uint8_t *mask;
    uint64_t q_stride, q_head_stride;
    uint64_t out_stride, out_head_stride;
    uint64_t mask_stride;
    uint32_t mask_cols;
    uint32_t q_heads;
    float scale;
    uint32_t reserved;
} df11_attention;

/* Bytes of df11_tree_attention's workspace on the current device, the same for
 * every content of the batch's arrays; 0 for arguments that the call refuses, or
 * where nothing needs computing. */
uint64_t df11_tree_attention_workspace(const df11_kv_cache *cache, const df11_kv_batch *batch,
                                       const df11_attention *a);

/* Attention of a batch's new tokens (one each when decoding, a tree of drafted
 * ones, a piece of a prompt) over a paged cache that already holds their keys
 * and values:
 *   out = sum over the visible places j of p_j v_j,  p = softmax(scale q . k_j)
 * Scores, the softmax's maximum and sums, and out's sums are float; p is rounded
 * to the cache's type for its product with v (the matrix cores' operand type), and
 * out is divided by the sum of p as rounded (lse has it unrounded) and rounded
 * once.  (That rounding is 2^-8 of p at most in DF11_BF16 and 2^-11 in DF11_FP16,
 * there also up to 2^-32 of the largest score's p: over 2^21 places as much as the
 * result's own.)  A query that sees nothing gets zeros and an lse of minus infinity.  What a place holds reaches only the
 * queries that see it: an infinity or a NaN elsewhere in the cache does not.
 * Rows that belong to no sequence are left as they were.
 *   workspace    device, 256-byte aligned, df11_tree_attention_workspace bytes;
 *                holds nothing between calls, but calls that overlap in time need
 *                one each
 * Results do not change from run to run.  Errors: DF11_E_INVALID_ARG,
 * DF11_E_TOO_LARGE (more tiles of queries and places than 2^31),
 * DF11_E_BUFFER_TOO_SMALL, DF11_E_HIP. */
int df11_tree_attention(const df11_kv_cache *cache, const df11_kv_batch *batch, const df11_attention *a,
                        void *workspace, uint64_t workspace_bytes, void *hip_stream);

/* ---------------------------------------------------------------------------
 * rANS exponent coder.  The discussion on the page ("Opini Hacker News")
 * names rANS as an entropy coder that suits SIMD-style instruction sets better
 * than Huffman; the page gives no format, so this one is this library's own:
 * the plain static rANS of asymmetric numeral systems (Duda) with 16-bit
 * renormalisation, laid out for 64-lane waves.
 *   - Frequencies f[s] of the exponents sum to M = 2^DF11_RANS_PROB_BITS;
 *     c[s] = f[0] + ... + f[s - 1].  A state x lies in [2^16, 2^32).
 *   - Encoding s: while x >= f[s] * 2^(32 - prob_bits), emit x mod 2^16 and
 *     shift it out; then x = floor(x / f[s]) * M + x mod f[s] + c[s].
 *     Decoding: slot = x mod M, s with c[s] <= slot < c[s] + f[s],
 *     x = f[s] * floor(x / M) + slot - c[s], and if x < 2^16,
 *     x = x * 2^16 + the next word.
 *   - Segments of DF11_RANS_LANES x DF11_RANS_STEPS exponents: lane l of a
 *     segment codes its positions step * lanes + l with a state of its own
 *     (2^16 when encoding starts).  The decoder takes a segment's words step
 *     by step, and within a step in lane order, one per lane whose state fell
 *     below 2^16.  Per segment the stream stores the lanes' start states and
 *     the offset of its words.
 * Sign/mantissa bytes are stored as for DF11 (PackedSignMantissa).
 * ------------------------------------------------------------------------- */
#define DF11_RANS_PROB_BITS 12
#define DF11_RANS_LANES 64
#define DF11_RANS_STEPS 512
/* Entries of the decoder's slot table (M). */
#define DF11_RANS_TABLE_ENTRIES 4096

typedef struct df11_rans_header {
    uint64_t n_elements;  /* N */
    uint64_t n_segments;  /* ceil(N / (lanes * steps)) */
    uint64_t n_words;     /* 16-bit words in the stream */
    uint32_t prob_bits;   /* DF11_RANS_PROB_BITS */
    uint32_t lanes;       /* DF11_RANS_LANES */
    uint32_t steps;       /* DF11_RANS_STEPS */
    uint32_t reserved;
} df11_rans_header;

/* Quantize an exponent histogram to rANS frequencies summing to 2^12 (host):
 * every used exponent gets max(1, floor(hist * M / N)); a sum below M gives
 * the difference to the most frequent exponent (lowest value on ties); while
 * the sum is above M the largest frequency above 1 (lowest value on ties)
 * drops by one.  An empty histogram gives all zeros.  Errors:
 * DF11_E_INVALID_ARG (null pointer), DF11_E_RESERVED_EXPONENT (hist[e] > 0 for
 * e >= 240). */
int df11_rans_quantize(const uint64_t hist[256], uint32_t freq[256]);

/* rANS-encode n BF16 words (host).  freq: from df11_rans_quantize (or any
 * table summing to M that covers every exponent present).  Outputs (host,
 * caller-allocated): states ceil(n / 32768) * 64 uint32; word_offsets
 * ceil(n / 32768) + 1 uint32 (segment g's words are [word_offsets[g],
 * word_offsets[g + 1])); words room for words_cap uint16 (n always suffices);
 * sm n bytes.  h is filled in.  Errors: DF11_E_INVALID_ARG (null pointer, a
 * table not summing to M, an exponent with frequency 0),
 * DF11_E_RESERVED_EXPONENT, DF11_E_BUFFER_TOO_SMALL (words_cap), DF11_E_TOO_LARGE
 * (n > DF11_MAX_ELEMENTS). */
int df11_rans_encode(const uint32_t freq[256], const uint16_t *w, uint64_t n, uint32_t *states,
                     uint32_t *word_offsets, uint16_t *words, uint64_t words_cap, uint8_t *sm, df11_rans_header *h);

/* The decoder's slot table (host): entry k (0 <= k < 4096) is the rotated
 * exponent s of slot k (s >> 1 | (s & 1) << 7) in bits 0-7, f[s] - 1 in bits
 * 8-19 and k - c[s] in bits 20-31.  table: DF11_RANS_TABLE_ENTRIES uint32.
 * Errors: DF11_E_INVALID_ARG (null pointer, a table not summing to M). */
int df11_rans_build_table(const uint32_t freq[256], uint32_t *table);

/* A device-resident rANS stream (buffers are device pointers, owned by the
 * caller).  words holds h.n_words words followed by padding up to a multiple
 * of 8 words plus 8 more (the decoder reads words 8 at a time), 16-byte
 * aligned; sm holds the N sign/mantissa bytes padded to a multiple of 64,
 * 16-byte aligned. */
typedef struct df11_rans_device_stream {
    df11_rans_header h;
    const uint32_t *table;         /* DF11_RANS_TABLE_ENTRIES entries (df11_rans_build_table) */
    const uint32_t *states;        /* h.n_segments * 64 */
    const uint32_t *word_offsets;  /* h.n_segments + 1 */
    const uint16_t *words;
    const uint8_t *sm;
} df11_rans_device_stream;

/* Decode a device-resident rANS stream into out (device, N uint16, 16-byte
 * aligned, not overlapping the stream), enqueued on hip_stream.  Every
 * element of out is overwritten with the original BF16 bits.  A corrupt
 * payload cannot make the kernel access memory out of bounds; its output is
 * unspecified.  Errors: DF11_E_INVALID_ARG (null pointers, alignment, layout
 * fields other than 12 / 64 / 512, overlap), DF11_E_BAD_STREAM (sizes
 * inconsistent), DF11_E_TOO_LARGE, DF11_E_HIP. */
int df11_rans_decompress(const df11_rans_device_stream *s, uint16_t *out, void *hip_stream);

/* df11_rans_decompress with start_event / stop_event (hipEvent_t, either may
 * be NULL) recorded at the decode kernel's own start and end. */
int df11_rans_decompress_timed(const df11_rans_device_stream *s, uint16_t *out, void *hip_stream,
                               void *start_event, void *stop_event);

/* Static, human-readable name of a status code.  Not on the page (the page
 * describes no API); the names are those of enum df11_status. */
const char *df11_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* DF11_H */
