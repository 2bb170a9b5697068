/*
 * kvc.h -- C ABI of libkvc, a lossless KV-cache entropy coder for MI355X (gfx950).
 *
 * The method ("speculative KV coding"): both ends of a KV transfer rebuild a
 * predictor mean mu and a frozen, calibrated per-(kv, head, channel) sigma;
 * every KV scalar is arithmetic-coded under the mixture
 *     q = 0.95 N(mu, sigma^2) + 0.03 N(mu, (3 sigma)^2) + 0.02 p_hat,
 * p_hat being the empirical marginal over the BF16 (or e4m3) alphabet, and
 * the decoder rebuilds KV exactly from the bits and (mu, sigma).
 * Sources: wiki page "Speculative KV Coding" (aisparkup.com), sections
 * "pipeline", "predictor choice" and "mixture distribution"; blog post
 * "推测性KV编码：用预测模型实现缓存无损压缩4倍" (blog.hotdry.top), sections
 * "engineering choice of predictor" and "application scenarios and
 * deployment parameters".
 *
 * The byte stream is format KVC-1: integer mixture CDF with total 2^31 and
 * every frequency >= 1, 64-bit-state rANS with 16-bit words, 64 interleaved
 * lanes (one per channel) per chunk of up to chunk_tokens tokens, a chunk
 * directory for random access, and a checksum of the side information.
 *
 * Conventions for every call:
 *   - Pointers named d_* are DEVICE pointers owned by the caller; pointers
 *     named h_* are HOST pointers.  The library never allocates memory and
 *     never frees caller memory; scratch comes from a caller workspace.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     All work is queued on it; calls that return a host value synchronise
 *     that stream once before returning; the *_async calls queue the work
 *     and return at once, their outcome read later by the *_result call
 *     (one synchronisation), so that many calls can be queued, on one stream
 *     or several, with no host round trip between them.
 *   - Layouts are row-major: KV and mu are [planes][tokens][channels] with
 *     channels fastest; sigma is [planes][channels] float32; the marginal
 *     prefix is uint32[N + 1] (N = 65536 for bf16, 256 for e4m3).
 *   - Every call returns a kvc_status; no exception crosses the ABI.  On an
 *     error, outputs are undefined (but never written out of bounds).
 *   - Concurrent calls on different streams are safe (each with its own
 *     workspace).  The state the library keeps, per device, lives in static
 *     device arrays (no allocation): the base CDF tables, copied on first
 *     use, and the mixture and decoder tables of every (weights, narrow
 *     part) a process uses (up to 8), built on first use by a kernel on the
 *     calling stream, which that first call synchronises; all of them are
 *     only read afterwards.  kvc_decode_noalloc's scratch is the one
 *     exception, see there.
 *   - Graph capture: once a call with the same weights and narrow part has
 *     run on the device (so its tables exist), kvc_encode without a size
 *     pointer and kvc_decode_async only launch kernels (the control block is
 *     cleared by a kernel, not a memset) and may be captured in a HIP graph
 *     and replayed; their *_result calls synchronise and stay outside it.
 */
#ifndef KVC_H
#define KVC_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kvc_status {
    KVC_OK = 0,
    KVC_ERR_INVALID = -1,   /* bad argument, shape, dtype, weights or sigma   */
    KVC_ERR_CAPACITY = -2,  /* output buffer or workspace too small           */
    KVC_ERR_CORRUPT = -3,   /* stream malformed or damaged                    */
    KVC_ERR_MISMATCH = -4,  /* sigma / prefix differ from the encoder's       */
    KVC_ERR_DEVICE = -5     /* a HIP call failed                              */
} kvc_status;

enum { KVC_BF16 = 0, KVC_E4M3 = 1, KVC_F32 = 2 };   /* E4M3 = OCP float8 e4m3fn */

#define KVC_HEADER_BYTES 128
#define KVC_DECODE_WORKSPACE_BYTES 917504   /* control block, escape tables, coder tables */
#define KVC_ESTIMATE_WORKSPACE_BYTES 256
#define KVC_ENCODE_STAGES 2
#define KVC_DECODE_STAGES 2

/* Optional per-call measurements (pass NULL to skip; costs a few events). */
typedef struct kvc_encode_info {
    float stage_ms[KVC_ENCODE_STAGES];  /* GPU time of: side-information checksum
                                           and per-call tables, coding kernel
                                           (which also places every chunk at its
                                           final offset)                          */
} kvc_encode_info;

typedef struct kvc_decode_info {
    float stage_ms[KVC_DECODE_STAGES];  /* GPU time of: side-information checksum
                                           and per-call tables, decoding kernel   */
    uint32_t reserved;
    uint64_t fallback_symbols;          /* symbols not found by the aim: slots in
                                           the floor-and-escape range (looked up
                                           through the bucket table) plus
                                           Gaussian slots whose aimed cell did not
                                           hold the target                        */
} kvc_decode_info;

typedef struct kvc_params {
    int32_t kv_dtype;        /* KVC_BF16 or KVC_E4M3                               */
    int32_t mu_dtype;        /* KVC_BF16 or KVC_F32                                */
    uint32_t w_narrow_bp;    /* weight of N(mu, sigma^2), basis points: 9500        */
    uint32_t w_wide_bp;      /* weight of N(mu, (3 sigma)^2), basis points: 300     */
                             /* the escape part p_hat gets 10000 - both; (10000, 0)
                                is a single Gaussian and needs no prefix table     */
    uint32_t chunk_tokens;   /* tokens per chunk; 0 = the library's default:
                                of the lengths ceil(tokens / k) between 1024
                                and 256 (or tokens, if fewer), the one with
                                the least rounds x (length + 9), a round being
                                8,192 chunks (one wave each) at once (with
                                sigma blocks: of the divisors of the block
                                length in that range, else the largest
                                divisor below it); chunk_tokens * channels
                                < 2^29                                           */
    uint32_t sigma_block_tokens; /* position-aware sigma ([blog] "limitations and
                                future directions"): 0 = one sigma per (plane,
                                channel), d_sigma [planes][channels]; B > 0 =
                                one sigma per (plane, block of B tokens,
                                channel), d_sigma [planes][ceil(tokens / B)]
                                [channels], token t using block t / B.  B must
                                be a multiple of chunk_tokens unless B >=
                                tokens (KVC_ERR_INVALID).  Recorded in the
                                stream header.                                 */
    uint32_t narrow_dof;     /* the narrow part's shape ([wiki] "future directions",
                                [blog] "limitations and future directions": a
                                better residual model): 0 = the pages'
                                N(mu, sigma^2); nu = 1..16 = Student's t with nu
                                degrees of freedom, location mu, scale sigma,
                                truncated to +-24 sigma and renormalised there.
                                The wide part and p_hat are unchanged.
                                Recorded in the stream header.                 */
    uint32_t channel_split;  /* per-channel mixture weights ([wiki] "future directions",
                                [blog] "limitations and future directions": a
                                better residual model): 0 = the call's weights on
                                every channel; 1 = each (plane, channel) has its
                                own narrow weight w_c in basis points, 0 ..
                                w_narrow_bp + w_wide_bp, its wide weight
                                w_narrow_bp + w_wide_bp - w_c (the escape weight
                                stays the call's).  The weights are side
                                information: the sigma buffer (d_sigma) holds
                                the sigma words followed by planes x channels
                                uint32 weights, [planes][channels], and every
                                call that takes it (encode, decode, reload,
                                estimate) reads both; sigma_bytes / strides
                                count both.  The coder's budgets are T_n(c) =
                                min(floor(T w_c / 10^4), T_n + T_w), T_w(c) =
                                T_n + T_w - T_n(c) with T = 2^31 - N.  A weight
                                above w_narrow_bp + w_wide_bp: KVC_ERR_INVALID.
                                Recorded in the stream header; covered by the
                                side-information checksum.                     */
    int64_t planes;          /* G = layers * 2 * batch * kv_heads                  */
    int64_t tokens;          /* T                                                  */
    int64_t channels;        /* D, a positive multiple of 64                       */
} kvc_params;

/* Stream format version written and accepted: 4 (Gaussian and floor-and-escape
   slots in separate ranges of the coder; the CDF argument q = floor(z * 2^24);
   the header's bytes [92, 96) hold the CRC-32 of its bytes [0, 92)). */
int kvc_version(void);

/* Human-readable name of a status code (static string). */
const char* kvc_status_string(int status);

/*
 * The format's two standard-normal CDF tables on the grid z_k = -24 + k/256,
 * k = 0..12288, computed on the host: h_narrow[k] = round(2^31 Phi(z_k)) and
 * h_wide[k] = round(2^31 Phi(z_k / 3)).  The mixture table the coder uses is
 * floor(T_n h_narrow[k] / 2^31) + floor(T_w h_wide[k] / 2^31).  Needs no GPU.
 * Returns KVC_ERR_INVALID for a NULL pointer.
 */
int kvc_phi_tables(uint32_t* h_narrow /* [12289] */, uint32_t* h_wide /* [12289] */);

/*
 * The narrow part's table for narrow_dof (kvc_params): narrow_dof = 0 gives
 * h_narrow of kvc_phi_tables; nu = 1..16 gives round(2^31 (F(z_k) - F(-24))
 * / (F(24) - F(-24))) for Student's t with nu degrees of freedom.  Needs no
 * GPU.  KVC_ERR_INVALID for a NULL pointer or nu > 16.
 */
int kvc_narrow_table(uint32_t narrow_dof, uint32_t* h_out /* [12289] */);

/*
 * Sizes for kvc_encode: the largest stream the call can produce (every
 * scalar at two 16-bit words, the worst case of the coder) and the workspace
 * it needs.  Host only; returns KVC_ERR_INVALID for bad parameters.
 */
int kvc_encode_sizes(const kvc_params* p, uint64_t* h_max_stream_bytes,
                     uint64_t* h_workspace_bytes);

/*
 * Encoder ([wiki] "pipeline": KV_full and (mu, sigma) go into the arithmetic
 * coder, which emits the bits).  Codes d_kv (bf16 or e4m3 bit patterns,
 * p->planes x p->tokens x p->channels of them) under the mixture around d_mu
 * with d_sigma and the marginal prefix d_prefix (NULL allowed when
 * w_narrow_bp + w_wide_bp == 10000); the buffers must hold what *p
 * describes.  Writes the stream to d_out, its length to *h_out_bytes and,
 * when h_header_out is not NULL, a host copy of its 128-byte header (what
 * kvc_decode takes) to h_header_out.  Every sigma must lie in [2^-96, 2^96],
 * else KVC_ERR_INVALID.  If the stream does not fit out_capacity the call
 * returns KVC_ERR_CAPACITY and sets *h_out_bytes to the size it needed.
 * Synchronises `stream` once.
 * h_out_bytes == NULL makes the call asynchronous: it queues the work and
 * returns KVC_OK (h_header_out and h_info must then be NULL);
 * kvc_encode_result on the same workspace gives the outcome later.
 * h_info: NULL, or receives the GPU time of each stage, measured with HIP
 * events on `stream`.
 */
int kvc_encode(const kvc_params* p, const void* d_kv, const void* d_mu,
               const float* d_sigma, const uint32_t* d_prefix, void* d_out,
               uint64_t out_capacity, uint64_t* h_out_bytes, void* h_header_out,
               void* d_workspace, uint64_t workspace_bytes, void* stream,
               kvc_encode_info* h_info);

/*
 * Outcome of the last encode queued with this workspace: synchronises
 * `stream` once, then returns the status kvc_encode would have returned and
 * fills *h_out_bytes (and, if not NULL, the 128-byte h_header_out) as it
 * would have.
 */
int kvc_encode_result(const void* d_workspace, void* stream, uint64_t* h_out_bytes,
                      void* h_header_out);

/*
 * Parse the 128-byte stream header held in HOST memory into *h_params and
 * the total stream length *h_stream_bytes.  Host only; KVC_ERR_CORRUPT if
 * the header is not a valid KVC-1 header.
 */
int kvc_stream_info(const void* h_header, uint64_t header_bytes, kvc_params* h_params,
                    uint64_t* h_stream_bytes);

/*
 * Decoder ([wiki] "pipeline": the bitstream plus (mu, sigma) give back
 * KV_full exactly).  h_header is a HOST copy of the stream's first 128
 * bytes (kvc_encode's h_header_out, or the head of a host-resident stream);
 * shape and parameters come from it, and the call checks, before anything
 * runs, that the header is a valid KVC-1 header (CRC included:
 * KVC_ERR_CORRUPT), that in_bytes is the length it gives (KVC_ERR_CORRUPT),
 * and that the caller's buffers hold what it describes (KVC_ERR_INVALID):
 * mu_bytes >= scalars x mu element size, sigma_bytes >= 4 x sigma words
 * (with per-channel weights, channel_split in the header: 4 x (sigma words
 * + planes x channels), the weights following sigma in d_sigma),
 * prefix_bytes >= 4 x (N + 1) when the mixture has an escape part,
 * kv_out_bytes >= scalars x KV element size.  On the device the stream's
 * own header must equal h_header (KVC_ERR_CORRUPT, nothing decoded).
 * d_in holds in_bytes of a KVC-1 stream; d_mu, d_sigma, d_prefix must be
 * the encoder's (checked through the stream's checksum: KVC_ERR_MISMATCH,
 * nothing decoded).  Writes KV bit patterns to d_kv_out
 * ([planes][tokens][channels]).  Returns KVC_ERR_CORRUPT if the stream is
 * malformed, truncated or damaged (every lane must start from a state in
 * [2^47, 2^63), end in the initial state and consume exactly its chunk).
 * Workspace: KVC_DECODE_WORKSPACE_BYTES, 256-byte aligned.  Synchronises
 * `stream` once (the status read).  h_info: NULL, or receives the stage
 * times and the number of symbols the aim did not find.
 */
int kvc_decode(const void* h_header, const void* d_in, uint64_t in_bytes,
               const void* d_mu, uint64_t mu_bytes, const float* d_sigma,
               uint64_t sigma_bytes, const uint32_t* d_prefix, uint64_t prefix_bytes,
               void* d_kv_out, uint64_t kv_out_bytes, void* d_workspace,
               uint64_t workspace_bytes, void* stream, kvc_decode_info* h_info);

/*
 * kvc_decode without its synchronisation: the host-side checks run and
 * return their status at once; the work is queued on `stream` and its
 * outcome is read later by kvc_decode_result on the same workspace (which
 * must not be reused before that).
 */
int kvc_decode_async(const void* h_header, const void* d_in, uint64_t in_bytes,
                     const void* d_mu, uint64_t mu_bytes, const float* d_sigma,
                     uint64_t sigma_bytes, const uint32_t* d_prefix, uint64_t prefix_bytes,
                     void* d_kv_out, uint64_t kv_out_bytes, void* d_workspace,
                     uint64_t workspace_bytes, void* stream);

/*
 * kvc_decode for callers that cannot allocate device memory (code under
 * graph capture, tight serving loops, harnesses that forbid allocation):
 * no workspace argument and no allocation of any kind.  Its scratch is a
 * fixed array of KVC_NOALLOC_SCRATCH_BYTES in device memory that the
 * library holds on every device it runs on until the process ends; the
 * decoder's scratch does not grow with the stream, so every stream
 * kvc_decode accepts fits (a layout needing more would be refused with
 * KVC_ERR_CAPACITY).  Arguments, checks, output and statuses as
 * kvc_decode; synchronises `stream` once.  Every call on one device
 * shares that device's scratch (cleared by the call where it must start at
 * zero): calls that overlap on one device, from several threads or on
 * several streams, race, and the caller must serialise them.
 */
#define KVC_NOALLOC_SCRATCH_BYTES 917504
int kvc_decode_noalloc(const void* h_header, const void* d_in, uint64_t in_bytes,
                       const void* d_mu, uint64_t mu_bytes, const float* d_sigma,
                       uint64_t sigma_bytes, const uint32_t* d_prefix, uint64_t prefix_bytes,
                       void* d_kv_out, uint64_t kv_out_bytes, void* stream);

/*
 * Host-offload reload ([wiki] "use scenarios": KV offloaded from DRAM to
 * VRAM; [blog] "application scenarios and deployment parameters": KV moved
 * over PCIe in compressed form, decoding fast enough to keep up with the
 * transfer).  Decodes n KVC-1 streams held in HOST memory (h_streams[l],
 * h_stream_bytes[l] bytes; pinned memory, e.g. from hipHostMalloc, lets the
 * copies run asynchronously) into device memory, one stream per layer: the
 * copy of stream l + 1 to the device runs on copy_stream while stream l is
 * decoded on `stream`, through two halves of d_staging (each 256-byte
 * aligned, staging_bytes / 2 rounded down to 256: every stream must fit one,
 * else KVC_ERR_CAPACITY).  Stream l decodes with the mu at d_mu + l x
 * mu_stride, the sigma at d_sigma + l x sigma_stride bytes and the shared
 * d_prefix, into d_kv_out + l x kv_stride; each stride is also the bytes
 * available there, checked against the stream's header as kvc_decode checks
 * its buffers.  Every layer's header (read in host memory) and buffers
 * pass these checks before anything is copied or launched.  Workspace: n x
 * KVC_DECODE_WORKSPACE_BYTES, 256-byte aligned (one decode workspace per
 * layer).  Synchronises `stream` and `copy_stream` once at the end and
 * returns the first failing layer's status (KVC_OK when all decode), its
 * index in *h_failed (-1 if none; may be NULL).
 */
int kvc_reload(int64_t n, const void* const* h_streams, const uint64_t* h_stream_bytes,
               const void* d_mu, uint64_t mu_stride, const float* d_sigma, uint64_t sigma_stride,
               const uint32_t* d_prefix, uint64_t prefix_bytes, void* d_kv_out, uint64_t kv_stride,
               void* d_staging, uint64_t staging_bytes, void* d_workspace, uint64_t workspace_bytes,
               void* stream, void* copy_stream, int64_t* h_failed);

/*
 * Outcome of the last decode queued with this workspace: synchronises
 * `stream` once and returns the status kvc_decode would have returned;
 * h_info (may be NULL) receives the fallback count (stage times are -1).
 */
int kvc_decode_result(const void* d_workspace, void* stream, kvc_decode_info* h_info);

/*
 * Paged output for kvc_decode_paged: the serving engine's KV cache as page
 * pools.  Pool p = 2 * layer + kv (K then V of each layer) is laid out
 * [num_pages][page_tokens][heads][channels] in the stream's KV dtype; the
 * stream's planes are ordered (layer, kv, batch, head), so planes = layers *
 * 2 * batch * heads; token t of sequence b lives in page
 * block_table[b * max_pages + t / page_tokens], row t % page_tokens.
 */
typedef struct kvc_paged_kv {
    void* const* d_pools;          /* device array of n_pools pool base pointers      */
    const int32_t* d_block_table;  /* device [batch][max_pages] physical page numbers */
    int64_t n_pools;               /* entries of d_pools: layers * 2                  */
    uint64_t pool_bytes;           /* bytes of every pool, >= num_pages x page_tokens
                                      x heads x channels x KV element size           */
    int64_t batch;                 /* sequences                                       */
    int64_t heads;                 /* KV heads per pool row                           */
    int64_t max_pages;             /* row stride of the table, >= ceil(tokens /
                                      page_tokens)                                    */
    int64_t num_pages;             /* pages in every pool, < 2^31                    */
    uint32_t page_tokens;          /* tokens per page                                 */
    uint32_t reserved;             /* 0                                               */
} kvc_paged_kv;

/*
 * Decoder fused into the consumer's layout ([blog] "application scenarios
 * and deployment parameters": a compressed prefix-cache entry is
 * decompressed when it is hit, and decoding has to keep up with the rate
 * at which the cache is consumed).  As kvc_decode, but every decoded row
 * goes straight to its page of the paged KV cache described by *h_paged
 * (host struct; its pointers are device pointers) instead of a contiguous
 * [planes][tokens][channels] array: no second pass over the KV.  Rows of
 * pages the table does not name are left untouched.  KVC_ERR_INVALID if the
 * planes are not n_pools x batch x heads with n_pools even, the table is
 * too narrow, a page holds 2^32 bytes or more, pool_bytes is short of
 * num_pages pages, or (checked on the device before the decode) an entry of
 * the columns the tokens use lies outside [0, num_pages): then nothing is
 * written.  Header and buffer checks as kvc_decode.
 */
int kvc_decode_paged(const void* h_header, const void* d_in, uint64_t in_bytes,
                     const void* d_mu, uint64_t mu_bytes, const float* d_sigma,
                     uint64_t sigma_bytes, const uint32_t* d_prefix, uint64_t prefix_bytes,
                     const kvc_paged_kv* h_paged, void* d_workspace, uint64_t workspace_bytes,
                     void* stream, kvc_decode_info* h_info);

/*
 * The paged cache around a decode: the calls below build the block table
 * that kvc_decode_paged and the attention read, append a step's new K/V rows
 * to its pages, and attend to them.  None of them synchronises unless its
 * declaration says so, and each launches kernels only (no memset, no copy),
 * so that all of them may be captured in a HIP graph and replayed; calls
 * that may run at the same time need workspaces of their own.
 */

/*
 * Block tables and slot maps from request lengths.  Request b holds
 * d_held_in[b] pages (the first entries of its row of d_block_table) and
 * d_cached_lens[b] tokens, and gets d_new_lens[b] more this step; free pages
 * are a stack, d_free_pages[0 .. *d_free_in), the last entry on top.  With
 * P = page_tokens and need_b = ceil((cached_b + new_b) / P):
 *   - request b takes max(0, need_b - held_b) pages from the top of the stack,
 *     requests in order, each request's pages in order; they are appended to
 *     its row of the table;
 *   - with trim = 1 a request that holds more than need_b pages first gives
 *     the surplus back (a finished request, cached = new = 0, gives all), in
 *     such an order that trimming what a call just took restores the stack;
 *     without it (0) surplus pages stay with the request.  A page that stands
 *     in several requests' rows must not be trimmed;
 *   - d_held_out[b] = need_b with trim, else max(held_b, need_b), *d_free_out
 *     the stack's new height.  d_held_out / d_free_out may be d_held_in /
 *     d_free_in (the state is updated in place) or other arrays (the old state
 *     stays readable; the pages given back are written above the old top);
 *   - the step's new tokens are rows, request after request: d_row_starts[b]
 *     is the first of request b, d_row_starts[batch] their number.  Row r, the
 *     i-th new token of request b, has d_positions[r] = cached_b + i and
 *     d_slots[r] = page x P + position % P, the page being the table's for
 *     position / P.  Rows behind the last, up to max_rows, get -1 in both.
 * Entries of the table behind a request's pages are left as they were.
 * On an error (kvc_block_table_result): KVC_ERR_INVALID for a negative length,
 * a held count outside [0, max_pages], a *d_free_in outside [0,
 * free_capacity] or 2^31 free and surplus pages together; KVC_ERR_CAPACITY where a request needs more than max_pages
 * pages or 2^31 tokens, the step more pages than are free, more than max_rows
 * rows, or a trim more than free_capacity entries.  The table, the stack, the
 * held counts and the height are then what they were, every row start is 0
 * and every slot and position -1, so that what is queued behind it appends
 * and attends to nothing.  A page number outside [0, num_pages), in the stack
 * or the table, is KVC_ERR_INVALID too: rows on such a page get slot -1, the
 * rest is written.
 * h_rows == NULL makes the call asynchronous; otherwise it synchronises
 * `stream` once, sets *h_rows to the number of rows and returns the outcome.
 * Workspace: KVC_BLOCK_TABLE_WORKSPACE_BYTES(batch), 256-byte aligned.
 */
#define KVC_BLOCK_TABLE_WORKSPACE_BYTES(batch) (256u + 12u * ((uint64_t)(batch) + 64u))
typedef struct kvc_block_table {
    int64_t batch;                  /* requests                                       */
    int64_t max_pages;              /* row stride of the table; batch x max_pages < 2^31 */
    int64_t num_pages;              /* pages in every pool, < 2^31                    */
    int64_t free_capacity;          /* entries of d_free_pages, < 2^31                */
    int64_t max_rows;               /* entries of d_slots and d_positions, < 2^31     */
    uint32_t page_tokens;           /* tokens per page                                */
    uint32_t trim;                  /* 0 or 1                                         */
    const int32_t* d_cached_lens;   /* [batch]; NULL: no request has any              */
    const int32_t* d_new_lens;      /* [batch]; NULL: no request gets any             */
    const int32_t* d_held_in;       /* [batch]                                        */
    int32_t* d_held_out;            /* [batch]                                        */
    int32_t* d_block_table;         /* [batch][max_pages]                             */
    int32_t* d_free_pages;          /* [free_capacity]                                */
    const int32_t* d_free_in;       /* [1]                                            */
    int32_t* d_free_out;            /* [1]                                            */
    int32_t* d_row_starts;          /* [batch + 1]                                    */
    int64_t* d_slots;               /* [max_rows] (NULL allowed)                      */
    int32_t* d_positions;           /* [max_rows] (NULL allowed)                      */
} kvc_block_table;
int kvc_build_block_table(const kvc_block_table* p, void* d_workspace, uint64_t workspace_bytes,
                          void* stream, int64_t* h_rows);

/*
 * Outcome of the last kvc_build_block_table queued with this workspace:
 * synchronises `stream` once, returns its status and sets *h_rows (may be
 * NULL) to the number of rows.
 */
int kvc_block_table_result(const void* d_workspace, void* stream, int64_t* h_rows);

/*
 * New K/V rows into the pages of one layer: row r of d_k ([rows] rows of
 * heads x channels values of src_dtype, row_stride values apart) goes to slot
 * d_slots[r] of pool 2 x layer, row r of d_v to the same slot of pool 2 x
 * layer + 1, a slot being page x page_tokens + row as kvc_build_block_table
 * gives it.  Rows whose slot is negative or past the pool are skipped; two
 * rows of one slot leave a mix of both.  kv_dtype is the pools' type:
 * values of the same type are copied bit for bit; bf16 into e4m3 is the
 * float32 quotient x / k_scale (x / v_scale) rounded to nearest even, what lies beyond +-448
 * saturated, NaN kept.  Scales are finite and positive, and 1 when the types
 * are the same.  h_paged as for kvc_decode_paged (its table is not read and
 * may be NULL), its pools 16-byte aligned.  d_k and d_v 16-byte aligned, row strides (in values, at
 * least heads x channels; not looked at for one row) such that every row is.  Does not
 * synchronise; KVC_ERR_INVALID for bad arguments, nothing launched.
 */
int kvc_paged_append(const kvc_paged_kv* h_paged, int64_t layer, int32_t kv_dtype, int64_t channels,
                     const void* d_k, const void* d_v, int32_t src_dtype, int64_t rows,
                     int64_t k_row_stride, int64_t v_row_stride, const int64_t* d_slots,
                     float k_scale, float v_scale, void* stream);

/*
 * Attention of drafted tokens over a paged cache.  Sequence b of h_paged's
 * batch has d_context_lens[b] tokens in its pages that every row of it sees,
 * and behind them its n_b = d_row_starts[b + 1] - d_row_starts[b] drafted
 * tokens (already appended, at positions context_b + 0 .. n_b - 1); row
 * d_row_starts[b] + i of d_q is drafted token i.  It sees drafted token j
 * where bit j % 64 of word j / 64 of its row of d_tree_mask ([rows]
 * [mask_words]) is set, j < n_b (bits behind n_b are ignored); without a
 * mask (NULL) it sees j <= i: a chain, a piece of a prompt or, n_b = 1, the
 * next token.  With query head a reading KV head a / (q_heads / heads):
 *     s_t = softmax_scale x k_scale x <q, K_t>,
 *     o = v_scale x sum_t e^(s_t) V_t / sum_t e^(s_t)  over the tokens seen,
 *     lse = log sum_t e^(s_t);
 * a row that sees nothing has o = 0 and lse = -infinity.  What K or V hold
 * (NaN, infinity) at tokens that a row does not see has no part in it; an
 * infinity in V of a drafted token that it sees is one in the output, however
 * small its weight (of a context token whose weight is 0 in float32 it may be
 * NaN).  Sums, maxima and the output's accumulation are float32; the weights
 * are rounded to bf16 for the matrix instructions, the output to bf16.  V is
 * summed with weights of up to 2^8 before the division: what passes 3.4e38
 * then is infinite.  Rows behind d_row_starts[batch] are left as they were.
 * q and out bf16, the cache bf16 or e4m3, its pools 16-byte aligned;
 * channels 64, 128, 192 or 256;
 * q_heads a multiple of heads, at most 1024 per KV head, rows x q_heads <
 * 2^31; at most 16384 sequences; heads x (rows x (q_heads / heads) / 16 +
 * min(rows, batch)) < 2^30; num_pages x page_tokens < 2^31;
 * softmax_scale x k_scale / log 2 a finite float32.
 * rows_per_sequence and max_tokens shape the launch only; results do not
 * depend on them: the usual n_b (0: rows / batch) and the longest context +
 * n_b (0: max_pages x page_tokens).
 * Does not synchronise.  kvc_paged_attention_result gives KVC_ERR_INVALID
 * where a sequence's row starts fall or pass `rows`, its context is negative
 * or it passes max_pages x page_tokens tokens (that sequence's rows are not
 * written; where row starts fall, others' may not be either), or where a page number read lies outside [0, num_pages) (page 0 is
 * read in its place: its rows are undefined).
 * Workspace: kvc_paged_attention_sizes, 256-byte aligned.
 */
typedef struct kvc_attention {
    const void* d_q;                /* [rows][q_heads][channels] bf16                 */
    int64_t q_row_stride;           /* in values, multiples of 8 (a stride between one
                                       row or one head is not looked at)              */
    int64_t q_head_stride;
    void* d_out;                    /* [rows][q_heads][channels] bf16                 */
    int64_t out_row_stride;         /* in values, multiples of 8; heads are channels apart */
    float* d_lse;                   /* [rows][q_heads] or NULL                        */
    const int32_t* d_row_starts;    /* [batch + 1]                                    */
    const int32_t* d_context_lens;  /* [batch]; NULL: none has any                    */
    const uint64_t* d_tree_mask;    /* [rows][mask_words] or NULL                     */
    int64_t mask_words;             /* 0 without a mask                               */
    int64_t rows;                   /* rows of q and out, < 2^24                      */
    int64_t rows_per_sequence;
    int64_t max_tokens;
    int64_t q_heads;
    int64_t channels;
    int32_t kv_dtype;               /* KVC_BF16 or KVC_E4M3                           */
    float softmax_scale;
    float k_scale, v_scale;         /* finite, positive                               */
} kvc_attention;
int kvc_paged_attention_sizes(const kvc_paged_kv* h_paged, const kvc_attention* p,
                              uint64_t* h_workspace_bytes);
int kvc_paged_attention(const kvc_paged_kv* h_paged, int64_t layer, const kvc_attention* p,
                        void* d_workspace, uint64_t workspace_bytes, void* stream);

/*
 * Outcome of the last kvc_paged_attention queued with this workspace:
 * synchronises `stream` and returns its status.
 */
int kvc_paged_attention_result(const void* d_workspace, void* stream);

/*
 * Queries, keys and values of a layer's new tokens on their way from the
 * projection: norms, rotation by position, and the append, in one pass.  Row
 * r of d_q, d_k and d_v is one token; q_heads heads of queries and h_paged's
 * heads of keys and values, of `channels` bf16 values each.  For a head x of
 * the queries (d_q_norm given) or keys (d_k_norm)
 *     y = x / sqrt(mean(x^2) + eps) * norm,
 * with one weight a channel, the same for all heads; without it (NULL) y = x.
 * Then, with t = d_positions[r] x d_frequencies[i] (radians) for the pair i of
 * the first `rotary` channels, channels i and rotary / 2 + i, or with
 * neighbours = 1 channels 2 i and 2 i + 1:
 *     (a, b) -> (a cos t - b sin t, a sin t + b cos t).
 * Queries are rounded to bf16 into d_q_out (which may be d_q, with the same
 * strides).  Keys and values go to slot d_slots[r] of pools 2 x layer and 2 x
 * layer + 1: keys rounded to the pools' type once, values as kvc_paged_append
 * writes them (bf16 bit for bit; e4m3 of the float32 quotients x / k_scale and
 * x / v_scale, to nearest even, saturated at +-448, NaN kept; scales finite
 * and positive, 1 for bf16 pools).  Of a row whose position is negative
 * nothing is written; of one whose slot is negative or past the pools no key
 * and value.  Two rows of one slot leave a mix of both.  A sum of squares is
 * float32, and float64 where that would overflow; t is formed in float64, off
 * by at most 2^-51 of itself, and whole turns are taken off there, so that far
 * positions are as exact as near ones; all else is float32.
 * channels 64, 128, 192 or 256; rotary a multiple of 16 from 0 (no rotation:
 * d_frequencies and d_positions may be NULL) to channels; eps at least 1e-30
 * where there is a norm; q_heads 0 (d_q and d_q_out not looked at) to 65536.
 * d_q, d_k, d_v, d_q_out, the norms and the pools 16-byte aligned.  h_paged's
 * table is not read and may be NULL.  Does not synchronise; KVC_ERR_INVALID
 * for bad arguments, nothing launched.
 */
typedef struct kvc_qkv {
    const void* d_q;                /* [rows][q_heads][channels] bf16                 */
    int64_t q_row_stride;           /* strides in values, multiples of 8 (one between
                                       one row or one head is not looked at)          */
    int64_t q_head_stride;
    const void* d_k;                /* [rows][heads][channels] bf16                   */
    int64_t k_row_stride;
    int64_t k_head_stride;
    const void* d_v;                /* [rows][heads][channels] bf16                   */
    int64_t v_row_stride;
    int64_t v_head_stride;
    void* d_q_out;                  /* [rows][q_heads][channels] bf16                 */
    int64_t q_out_row_stride;       /* in values, a multiple of 8; heads are channels apart */
    const void* d_q_norm;           /* [channels] of norm_dtype, or NULL              */
    const void* d_k_norm;           /* [channels] of norm_dtype, or NULL              */
    const double* d_frequencies;    /* [rotary / 2] radians a position                */
    const int32_t* d_positions;     /* [rows]                                         */
    const int64_t* d_slots;         /* [rows]                                         */
    int64_t rows;                   /* < 2^31                                         */
    int64_t q_heads;
    int64_t channels;
    int64_t rotary;
    int32_t kv_dtype;               /* of the pools: KVC_BF16 or KVC_E4M3             */
    int32_t norm_dtype;             /* KVC_BF16 or KVC_F32                            */
    uint32_t neighbours;            /* 0 or 1                                         */
    float eps;
    float k_scale, v_scale;
} kvc_qkv;
int kvc_paged_qkv(const kvc_paged_kv* h_paged, int64_t layer, const kvc_qkv* p, void* stream);

/*
 * Verification of drafted tokens against the target's probabilities, with
 * given random numbers: what is kept is distributed as if the target had been
 * sampled token by token.  Sequence b's n_b = d_row_starts[b + 1] -
 * d_row_starts[b] rows (at most KVC_MAX_DRAFT_NODES) are the nodes of a tree:
 * node 0 the last token that the sequence has (its d_tokens entry is not
 * looked at), node i > 0 a drafted token behind node d_parents[row] < i (a
 * place in the sequence, not a row; d_parents NULL: i - 1, a chain).  Row r of
 * d_target holds the target's probabilities of the token behind node r, row r
 * of d_draft (where given) those that the children of node r were drawn from,
 * each child by itself.  Beginning with node 0, the children of the current
 * node are tested in the order of their rows; with y the target's row at
 * first, t a child's token and u its d_accept entry:
 *   - with d_draft (q its row), after a rejection y is first scaled by the
 *     float32 of 1 / sum(y); the child is accepted where u q[t] < y[t]; else y
 *     becomes max(y - q, 0);
 *   - without (tokens picked, not drawn) it is accepted where u m < y[t], m
 *     being 1 less the y[t] of the children rejected before; else y[t]
 *     becomes 0.
 * An accepted child becomes the current node, with a new y.  Where no child is
 * accepted the walk stops and the last token is drawn from y (from the
 * target's row where sum(y) is 0): the first x whose sum(y[0 .. x]) is greater
 * than floor(u S), u being d_sample[b] and S the whole sum.
 * Out come d_kept_lens[b], the nodes kept, node 0 among them (1 to n_b; 0
 * where n_b is 0); d_kept[row starts + j], the j-th of them; and d_out_tokens
 * [row starts + j], the sequence's new tokens, one a kept node, the drawn one
 * last; both -1 behind.  Rows behind d_row_starts[batch] are left as they
 * were.
 * Probabilities are float32 and compared in float64 (u m of large m rounded
 * to it); y is float32, each step rounded once; sums count whole units of
 * 2^-42, rounded down, and are exact: nothing depends on an order of
 * summation.  What is no number from 0 to 1 counts as the nearer of them, NaN
 * as 0; rows of probabilities are taken to sum to 1.  Random numbers lie in
 * [0, 1).
 * vocab and batch at most 2^20, batch x ceil(vocab / 4096) < 2^24; a row
 * stride (in values, at least vocab) between one row is not looked at.  With
 * d_draft and d_parents the time grows with the square of the siblings that
 * are rejected at one node (64 of them over 131072 tokens take 4.4 ms, so a
 * thousand about a second).  Does not synchronise.
 * kvc_verify_drafts_result gives KVC_ERR_INVALID where a sequence's row starts
 * fall or pass `rows` or it has too many nodes (its kept length is then 0 and
 * nothing else of it written), where a parent does not come before its node
 * (which is then not reached), a token lies outside the vocabulary (it is
 * never accepted), or the probabilities that a token is drawn from are all 0
 * (the token is then -1).
 * Workspace: kvc_verify_drafts_sizes (of batch and vocab), 256-byte
 * aligned, all zero before its first call and again before a call of another
 * batch than the last (its parts lie elsewhere then).
 */
#define KVC_MAX_DRAFT_NODES 1024
typedef struct kvc_drafts {
    int64_t batch;
    int64_t rows;                   /* < 2^31                                         */
    int64_t vocab;
    const int32_t* d_row_starts;    /* [batch + 1]                                    */
    const int32_t* d_tokens;        /* [rows]                                         */
    const int32_t* d_parents;       /* [rows] or NULL                                 */
    const float* d_target;          /* [rows][vocab]                                  */
    int64_t target_row_stride;
    const float* d_draft;           /* [rows][vocab] or NULL                          */
    int64_t draft_row_stride;
    const float* d_accept;          /* [rows]                                         */
    const float* d_sample;          /* [batch]                                        */
    int32_t* d_kept;                /* [rows]                                         */
    int32_t* d_kept_lens;           /* [batch]                                        */
    int32_t* d_out_tokens;          /* [rows]                                         */
} kvc_drafts;
int kvc_verify_drafts_sizes(const kvc_drafts* p, uint64_t* h_workspace_bytes);
int kvc_verify_drafts(const kvc_drafts* p, void* d_workspace, uint64_t workspace_bytes, void* stream);

/*
 * Outcome of the last kvc_verify_drafts queued with this workspace:
 * synchronises `stream` and returns its status.
 */
int kvc_verify_drafts_result(const void* d_workspace, void* stream);

/*
 * Kept tokens moved together.  Of sequence b's drafted tokens (as
 * kvc_paged_attention sees them: n_b rows, token i at position
 * d_context_lens[b] + i) the d_kept_lens[b] tokens d_kept[d_row_starts[b] + j],
 * places that rise with j, stay: in every pool of h_paged, the row of the
 * j-th goes to position d_context_lens[b] + j.  What kvc_verify_drafts gives
 * is taken as it is; the sequence's context is then d_context_lens[b] +
 * d_kept_lens[b], and kvc_build_block_table with trim gives the rest back.
 * Rows of other positions are left as they were (those behind the last kept
 * one hold what they held, or a kept row's copy).  A drafted token's page must
 * not stand in another request's row of the table.
 * d_context_lens NULL: none has any.  batch at most 2^20, at most 2^20 pools,
 * which are 16-byte aligned.  Does not synchronise.  kvc_paged_compact_result
 * gives KVC_ERR_INVALID where a sequence's row starts fall or pass `rows`, its
 * lengths are negative or pass its row of the table or 2^31 tokens, more is
 * kept than there is, or places do not rise or lie outside its rows (nothing
 * of it is moved), or where a page number lies outside [0, num_pages) (the
 * rows that it concerns are not moved).
 * Workspace: KVC_COMPACT_WORKSPACE_BYTES(batch), 256-byte aligned.
 */
#define KVC_COMPACT_WORKSPACE_BYTES(batch) (256u + 4u * (uint64_t)(batch))
int kvc_paged_compact(const kvc_paged_kv* h_paged, int32_t kv_dtype, int64_t channels, int64_t rows,
                      const int32_t* d_row_starts, const int32_t* d_context_lens, const int32_t* d_kept,
                      const int32_t* d_kept_lens, void* d_workspace, uint64_t workspace_bytes,
                      void* stream);

/*
 * Outcome of the last kvc_paged_compact queued with this workspace:
 * synchronises `stream` and returns its status.
 */
int kvc_paged_compact_result(const void* d_workspace, void* stream);

/*
 * Requests that start from another's tokens: pages held by several requests,
 * with a count of the further holders of every page (d_extra[page], 0 where
 * one request holds it or none; pages that kvc_build_block_table hands out
 * have 0).  The state is that of kvc_build_block_table: the table, the pages
 * each request holds, the stack of free pages.  With P = page_tokens:
 *
 * kvc_fork_pages: for k < count, request c = d_children[k], which holds
 * no page, gets the T = d_context_lens[p] tokens of request p =
 * d_parents[k] (NULL: none has any):
 *   - the first T / P pages of p's row of the table are entered in c's, and
 *     d_extra of each goes up by one;
 *   - where P does not divide T, a page is popped from the stack (children in
 *     their order) and entered behind them, and the T % P tokens of p's
 *     next page are copied to it in every pool of h_paged;
 *   - c holds ceil(T / P) pages.
 * A child of -1 is none (padding); no request may be a child twice.  The child
 * can then be extended like any request: its new tokens' pages are its own.
 * All or nothing: on KVC_ERR_INVALID (a request outside the batch, a child
 * that holds pages, is its parent or stands twice, a parent that holds fewer
 * pages than its tokens need or more than max_pages, a negative length,
 * *d_free_in outside [0, free_capacity], a page to be popped or copied from
 * outside [0, num_pages)) and KVC_ERR_CAPACITY (fewer pages free than wanted)
 * the held counts and the height of the stack are what they were and nothing
 * else is written.  A page number outside the pools among those entered in a
 * child's row is KVC_ERR_INVALID too: it is entered, not counted.
 *
 * kvc_release_pages: the requests d_requests[k], k < count (-1: none), are
 * finished: each page that they hold loses a holder (d_extra goes down by
 * one); pages that no request holds any more go to the stack, in ascending
 * order, the highest on top; their d_extra is 0; the requests hold none.
 * KVC_ERR_INVALID for a request outside the batch, a held count outside [0,
 * max_pages] (both left alone), a request that stands twice (released once),
 * a page number outside the pools (passed over), a page that loses more
 * holders than it has (given back once), or a *d_free_in outside [0,
 * free_capacity] (nothing is done); KVC_ERR_CAPACITY where the stack would
 * pass free_capacity, as one that holds a page twice may (what fits is pushed).
 * It looks through a mark of every page of the pools, so that large pools take
 * longer however few pages are released (32768 pages 4 us, a million 110).
 *
 * A request whose pages were shared is finished with kvc_release_pages, not
 * with a trim, and not trimmed below the tokens that it was forked from or
 * with: kvc_build_block_table does not know d_extra, and would put pages that
 * others hold on the stack without an error.  d_held_out / d_free_out may be
 * d_held_in / d_free_in, or other arrays.  count at most 1024, at most 2^20
 * pools, which are 16-byte aligned; free_capacity at least num_pages.  Neither
 * call synchronises;
 * kvc_shared_pages_result gives the outcome of the last one of either kind
 * queued with the workspace.
 * Workspace: KVC_SHARED_PAGES_WORKSPACE_BYTES(num_pages), 256-byte aligned,
 * all zero before the first call that uses it.
 */
#define KVC_MAX_SHARED_REQUESTS 1024
#define KVC_SHARED_PAGES_WORKSPACE_BYTES(num_pages) \
    (256u + 4096u + 64u * (((uint64_t)(num_pages) + 31u) / 32u))
typedef struct kvc_shared_pages {
    int64_t free_capacity;          /* entries of d_free_pages, < 2^31                */
    int32_t* d_block_table;         /* [batch][max_pages] of h_paged                  */
    const int32_t* d_held_in;       /* [batch]                                        */
    int32_t* d_held_out;            /* [batch]                                        */
    int32_t* d_free_pages;          /* [free_capacity]                                */
    const int32_t* d_free_in;       /* [1]                                            */
    int32_t* d_free_out;            /* [1]                                            */
    int32_t* d_extra;               /* [num_pages]                                    */
} kvc_shared_pages;
int kvc_fork_pages(const kvc_paged_kv* h_paged, int32_t kv_dtype, int64_t channels,
                   const kvc_shared_pages* p, int64_t count, const int32_t* d_parents,
                   const int32_t* d_children, const int32_t* d_context_lens, void* d_workspace,
                   uint64_t workspace_bytes, void* stream);
int kvc_release_pages(const kvc_paged_kv* h_paged, int32_t kv_dtype, int64_t channels,
                      const kvc_shared_pages* p, int64_t count, const int32_t* d_requests,
                      void* d_workspace, uint64_t workspace_bytes, void* stream);
int kvc_shared_pages_result(const void* d_workspace, void* stream);

/*
 * Sigma calibration ([wiki] "predictor choice": per-(kv, head, channel)
 * variance calibrated on data, then frozen; [blog] "deployment parameters":
 * 128 sequences of 1024 tokens).  d_kv and d_mu are [reps][planes][tokens]
 * [channels]; writes d_sigma_out[planes][channels] = max(sigma_floor,
 * sqrt(mean over reps and tokens of (kv - mu)^2)), accumulated in float64
 * in a fixed order (deterministic); residuals that are not finite are left
 * out, and a channel with none left gets the floor.  d_workspace (256-byte
 * aligned) holds the float64 partial sums: at least
 * KVC_CALIBRATE_WORKSPACE_BYTES(planes, channels) bytes.  Returns
 * KVC_ERR_INVALID for bad shapes, a non-positive floor or a short
 * workspace.  Does not synchronise.
 */
#define KVC_CALIBRATE_WORKSPACE_BYTES(planes, channels) \
    ((uint64_t)(planes) * (uint64_t)(channels) * 1024u)
int kvc_calibrate_sigma(const void* d_kv, const void* d_mu, int32_t kv_dtype,
                        int32_t mu_dtype, int64_t reps, int64_t planes, int64_t tokens,
                        int64_t channels, float sigma_floor, float* d_sigma_out,
                        void* d_workspace, uint64_t workspace_bytes, void* stream);

/*
 * Position-aware sigma calibration ([blog] "limitations and future
 * directions": a static per-channel sigma ignores how the residual changes
 * with position).  As kvc_calibrate_sigma, per block of block_tokens
 * tokens: d_sigma_out[planes][n_blocks][channels] with n_blocks =
 * ceil(tokens / block_tokens), block j taking the mean over reps and the
 * tokens [j * block_tokens, min((j + 1) * block_tokens, tokens)).
 * block_tokens = 0 or >= tokens gives one block (the per-plane sigma).
 * Workspace: KVC_CALIBRATE_WORKSPACE_BYTES(planes * n_blocks, channels).
 */
int kvc_calibrate_sigma_blocks(const void* d_kv, const void* d_mu, int32_t kv_dtype,
                               int32_t mu_dtype, int64_t reps, int64_t planes, int64_t tokens,
                               int64_t channels, int64_t block_tokens, float sigma_floor,
                               float* d_sigma_out, void* d_workspace, uint64_t workspace_bytes,
                               void* stream);

/*
 * Rate-fitted sigma ([blog] "limitations and future directions": better
 * residual models; [blog] "engineering choice of predictor": sigma measured
 * once on held-out data).  The RMS of kvc_calibrate_sigma_blocks is the base;
 * one outlier in a few hundred inflates it.  For each (plane, block, channel)
 * this call keeps, of the candidates max(sigma_floor, base * (1 - j/32)),
 * j = 0..24 (float32 products), the one under which the held-out data cost
 * the fewest bits in the coder's own integer model: the sum over the data
 * of 2^16 (31 - e) - L[m] for each frequency f = C(s+1) - C(s), with e the
 * top bit of f, m the 8 bits below it and L[m] = round(2^16 log2(1 + m/256));
 * the first j on a tie (an integer sum: deterministic).  The mixture
 * weights, the narrow part (narrow_dof, as in kvc_params) and d_prefix
 * (NULL allowed for a single Gaussian) are the ones the data will be coded
 * with.  sigma_floor in [2^-96, 2^96].  Output and
 * block_tokens as kvc_calibrate_sigma_blocks.  Workspace (256-byte aligned):
 * KVC_CALIBRATE_RATE_WORKSPACE_BYTES(planes * n_blocks, channels).  Does
 * not synchronise.
 */
#define KVC_CALIBRATE_RATE_WORKSPACE_BYTES(rows, channels) \
    ((uint64_t)(rows) * (uint64_t)(channels) * (1024u + 12800u) + 65536u)
int kvc_calibrate_sigma_rate(const void* d_kv, const void* d_mu, int32_t kv_dtype,
                             int32_t mu_dtype, int64_t reps, int64_t planes, int64_t tokens,
                             int64_t channels, int64_t block_tokens, float sigma_floor,
                             uint32_t w_narrow_bp, uint32_t w_wide_bp, uint32_t narrow_dof,
                             const uint32_t* d_prefix, float* d_sigma_out, void* d_workspace,
                             uint64_t workspace_bytes, void* stream);

/*
 * Per-channel mixture weights ([wiki] "future directions" and [blog]
 * "limitations and future directions": a better residual model; the pages'
 * 0.95 / 0.03 split is one choice for every channel, [wiki] "mixture
 * distribution").  For each (plane, channel), of the narrow weights
 * w_j = max(w_narrow_bp + w_wide_bp - 200 j, 0), j = 0..15, writes to
 * d_split_out[planes][channels] (uint32) the one under which the held-out
 * data d_kv / d_mu ([reps][planes][tokens][channels]) cost the fewest bits
 * in the coder's own integer model with that channel's budgets (the sum of
 * kvc_calibrate_sigma_rate; the first j on a tie: deterministic).  d_sigma
 * is the sigma the data will be coded with: [planes][channels], or per
 * block of block_tokens tokens [planes][ceil(tokens / block_tokens)]
 * [channels] (block_tokens = 0 or >= tokens: one block); the weights,
 * narrow_dof and d_prefix (NULL allowed for a single Gaussian) as the
 * stream will use them.  Workspace (256-byte aligned):
 * KVC_CALIBRATE_SPLIT_WORKSPACE_BYTES(planes, channels).  KVC_ERR_INVALID
 * for bad shapes or arguments.  Does not synchronise.
 */
#define KVC_CALIBRATE_SPLIT_WORKSPACE_BYTES(planes, channels) \
    ((uint64_t)(planes) * (uint64_t)(channels) * 8192u)
int kvc_calibrate_split(const void* d_kv, const void* d_mu, int32_t kv_dtype, int32_t mu_dtype,
                        int64_t reps, int64_t planes, int64_t tokens, int64_t channels,
                        int64_t block_tokens, const float* d_sigma, uint32_t w_narrow_bp,
                        uint32_t w_wide_bp, uint32_t narrow_dof, const uint32_t* d_prefix,
                        uint32_t* d_split_out, void* d_workspace, uint64_t workspace_bytes,
                        void* stream);

/*
 * Empirical marginal ([wiki] "mixture distribution": an empirical BF16
 * distribution catches extreme outliers).  d_samples holds n bit patterns
 * (bf16 or e4m3); writes the integer prefix d_prefix_out[b] =
 * floor(T_e * cum[b] / cum[N]) of the +1-smoothed histogram in value order,
 * with T_e the escape budget of the weights.  n < 2^32 - 2^16.  Does not
 * synchronise.
 */
int kvc_build_marginal(const void* d_samples, int32_t dtype, uint64_t n,
                       uint32_t w_narrow_bp, uint32_t w_wide_bp,
                       uint32_t* d_prefix_out, void* stream);

/*
 * Bits per scalar ([wiki] "core idea": the rate is the cross-entropy of the
 * model).  h_bits_out[0] = mean of -log2(f/2^31) under the integer model the
 * coder uses; h_bits_out[1] = mean -log2 q under the continuous mixture over
 * the same cells (float64, per-scalar cost capped at 64 bits).  With
 * p->channel_split = 1, d_sigma carries the per-channel weights after sigma
 * (as for kvc_encode) and each channel's weights are used.  Workspace:
 * KVC_ESTIMATE_WORKSPACE_BYTES.  Synchronises `stream` once.
 */
int kvc_estimate_bits(const kvc_params* p, const void* d_kv, const void* d_mu,
                      const float* d_sigma, const uint32_t* d_prefix, double* h_bits_out,
                      void* d_workspace, uint64_t workspace_bytes, void* stream);

/*
 * The shared CDF itself ([blog] "deployment parameters": encoder and decoder
 * must agree on it bit for bit), with the narrow part narrow_dof (as in
 * kvc_params).  For each of `pairs` (mu, sigma) pairs,
 * writes C(b) for b = 0..N to d_out[pair][N + 1].  d_mu holds `pairs`
 * values of mu_dtype, d_sigma `pairs` floats.  Synchronises `stream` once
 * (to report an invalid sigma).
 */
int kvc_cdf_table(int32_t kv_dtype, int32_t mu_dtype, uint32_t w_narrow_bp,
                  uint32_t w_wide_bp, uint32_t narrow_dof, const void* d_mu, const float* d_sigma,
                  int64_t pairs, const uint32_t* d_prefix, uint32_t* d_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVC_H */
