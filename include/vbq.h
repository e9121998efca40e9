/*
 * vbq.h -- C ABI of the packed mixed-bit weight library for MI355X (gfx950).
 *
 * The library computes y = x . W^T for a frozen weight matrix W (N x K) that
 * is stored group-quantised: every contiguous group of 64 weights along K has
 * its own bit-width b in {1, 2, 4, 8}, an fp16 scale s and an fp16 offset o,
 * and dequantises as w = s*q + o with integer code q in [0, 2^b - 1].
 *   - Per-group widths from {1,2,4,8} on 64-weight groups, packed low-bit
 *     storage and a fused dequantise-and-multiply for bandwidth-bound decode:
 *     VBQ abstract, page "In-Cell Learning: Language Models That Update Their
 *     Own Weights in Sequence Without Changing the File They Ship".
 *   - Asymmetric (scale + offset) quantisation: SLQ abstract, page
 *     thelatestinai.com/papers/2512.18934.
 *   - Per-weight residual inside each quantisation cell, bit-identical
 *     re-quantisation, revocation by dropping the residual, bounded drift:
 *     page "Nothing Changed but the Model: CellFill -- Bounded In-Cell
 *     Learning for Bit-Identical, Revocable Updates to Quantized LLMs",
 *     section Abstract.
 *
 * Conventions for every call:
 *   - Ownership: the caller allocates and frees every buffer it passes. The
 *     library allocates nothing, keeps no state between calls (apart from
 *     cached device attributes) and needs no workspace: partial sums stay
 *     on-chip inside a workgroup. (vbq_gemv_batched_static keeps a scratch
 *     array; kv4_attention, kv4_attention_shared, kv4_fork and token_logprobs
 *     take a workspace from the caller.) The calls can therefore be captured into a HIP graph as they are. Buffers marked "device" live in GPU memory of
 *     the current HIP device; "host" buffers are ordinary CPU memory.
 *   - Asynchrony: compute calls enqueue work on `stream` and return without
 *     waiting. Argument errors are found before anything is enqueued: the
 *     call returns a non-zero vbq_status and enqueues nothing. A failed kernel
 *     launch returns VBQ_ERR_HIP. No C++ exception crosses this boundary.
 *   - fp16 and bf16 values are passed as their 16-bit patterns (uint16_t).
 *   - Calls that share output buffers must not overlap in time.
 *   - Results of the GEMV calls are identical from run to run for the same
 *     inputs and shapes (fixed summation order; nothing depends on timing).
 *
 * Execution layout of a packed matrix (see vbq_matrix). The pages give no
 * layout; this one fills every block of 64 records of one width and makes
 * the byte position of every record a closed form of its tile's header, so
 * a kernel can issue all of a tile's loads at once and give each lane one
 * record of any column.
 *   Tiles. The matrix is cut into tiles of VBQ_TILE_ROWS = 32 rows by
 *   VBQ_TILE_GROUPS = 64 k-groups (4096 columns), stored k-tile major: tile
 *   t = kt * RT + rt covers rows 32 rt .. 32 rt + R - 1 and k-groups
 *   64 kt .. 64 kt + G_t - 1, with RT = ceil(N / 32), KT = ceil(K / 4096),
 *   R = min(32, N - 32 rt), G_t = min(64, K/64 - 64 kt). Column l < G_t of a
 *   tile is its k-group 64 kt + l; r < R is its row 32 rt + r.
 *   Width class c = 0, 1, 2, 3 for b = 1, 2, 4, 8.
 *   Records. The groups of class c of a tile are numbered e = 0 .. N_c - 1
 *   in column-major order: column l ascending and, within a column, its
 *   rows of class c ascending. Record e of class c is entry e % 64 of block
 *   e / 64 of the class; block k holds m_k = min(64, N_c - 64 k) records.
 *   A tile's bytes are, in order (every area starts 16-byte aligned and is
 *   zero-padded to a multiple of 16 bytes):
 *     map   : for l < G_t, 8 bytes at 8 l: u32 plane0 then u32 plane1, where
 *             bit r of plane0 is (class of group (r, l)) & 1 and bit r of
 *             plane1 is (class of group (r, l)) >> 1, for r < R (higher bits
 *             zero). These are the 2 bits of width per group.
 *     blocks: for c = 0, 1, 2, 3 and k = 0 .. ceil(N_c / 64) - 1, block
 *             (c, k):
 *               codes area: entry j's 2b u32 words at byte 8 b j;
 *               so area   : entry j's u32 at byte 4 j, fp16 scale in bits
 *                           0-15 and fp16 offset in bits 16-31.
 *   A full block takes 512 b + 256 bytes, so with C_c the byte (from the
 *   tile's start) where class c's first block begins, record e of class c
 *   has its codes at C_c + (e / 64)(512 b + 256) + 8 b (e % 64) and its
 *   scale/offset word at C_c + (e / 64)(512 b + 256) + up16(8 b m) +
 *   4 (e % 64), m being its block's record count; C_0 is the map's size and
 *   C_(c+1) = C_c + (bytes of class c's blocks).
 *   Record words: with h = 16/b, the pair p = (code 2p, code 2p+1), p < 32,
 *   sits in word p/h: code 2p at bit (p%h)*b (LSB first) and code 2p+1 at
 *   bit 16 + (p%h)*b.
 *   The tiles follow each other in storage order in one byte stream.
 *   tiles[4t..4t+3] = { first 16-byte unit of tile t, its size in 16-byte
 *   units, N_0 | N_1 << 16, N_2 | N_3 << 16 }. Entry t = n_tiles holds
 *   { total 16-byte units, invalid-width count, error flags, 0 }.
 */
#ifndef VBQ_H
#define VBQ_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define VBQ_ABI_VERSION 4
#define VBQ_GROUP 64          /* weights per quantisation group (along K) */
#define VBQ_TILE_ROWS 32      /* rows per layout tile */
#define VBQ_TILE_GROUPS 64    /* k-groups (of 64 weights) per layout tile */
#define VBQ_MAX_GROUPS 4095   /* K / 64 must not exceed this */
#define VBQ_MAX_BATCH 8       /* largest batch of the GEMV calls */
#define VBQ_MAX_LAUNCH_MATS 32 /* matrices per batched call */

typedef enum vbq_status {
  VBQ_OK = 0,
  VBQ_ERR_INVALID_ARG = 1,   /* null pointer or bad count */
  VBQ_ERR_SHAPE = 2,         /* N < 1, K < 64, K % 64 != 0, K/64 > VBQ_MAX_GROUPS, M < 1, mismatched shapes */
  VBQ_ERR_BITWIDTH = 3,      /* a width not in {1,2,4,8} */
  VBQ_ERR_ALIGNMENT = 4,     /* a buffer not aligned as documented */
  VBQ_ERR_UNSUPPORTED = 5,   /* batch out of range, or a size the kernels do not take */
  VBQ_ERR_CAPACITY = 6,      /* the layout does not match the buffers it was given */
  VBQ_ERR_HIP = 7            /* a HIP runtime call or kernel launch failed */
} vbq_status;

/* Descriptor of caller-owned device buffers holding one packed matrix.
 * Sizes come from vbq_pack_query; vbq_pack fills the buffers. */
typedef struct vbq_matrix {
  int32_t n_rows;      /* N, output features */
  int32_t n_cols;      /* K, input features, multiple of 64 */
  int64_t n_tiles;     /* ceil(N / 32) * ceil(K / 4096) */
  int64_t n_bytes16;   /* size of `stream` in 16-byte units, at most 2^27 - 1 (2 GiB - 16 bytes) */
  uint32_t* tiles;     /* device, (n_tiles + 1) * 4 words, 16-byte aligned */
  uint32_t* stream;    /* device, n_bytes16 * 4 words, 16-byte aligned */
} vbq_matrix;

/* Sizes of the buffers of a packed matrix, plus accounting figures. */
typedef struct vbq_layout_sizes {
  int64_t n_tiles;
  int64_t n_records;         /* N * K / 64 (one record per group) */
  int64_t n_bytes16;
  int64_t max_tile_bytes16;
  int64_t code_bits;         /* sum over groups of 64 * width: bits of codes proper */
  int64_t groups_by_width[4]; /* number of groups of width 1, 2, 4, 8 */
} vbq_layout_sizes;

/* ABI version (VBQ_ABI_VERSION of the built library). */
int vbq_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char* vbq_status_string(int status);

/* Host-only sizing of the execution layout (VBQ abstract: one width per
 * 64-weight group). widths_host: host, N x K/64 uint8 in natural (row,
 * k-group) order. out: host. Returns VBQ_ERR_SHAPE or VBQ_ERR_BITWIDTH on bad
 * input, VBQ_ERR_UNSUPPORTED for a stream above 2 GiB - 16 bytes. Touches no
 * GPU. */
vbq_status vbq_pack_query(const uint8_t* widths_host, int32_t N, int32_t K, vbq_layout_sizes* out);

/* Quantise W and write the execution layout (offline step).
 * Quantiser, per group of 64 (VBQ abstract for the groups and widths; SLQ
 * abstract for scale + offset), in binary32 without contraction:
 *   lo = min, hi = max; scale16 = fp16(f32(hi - lo) / (2^b - 1));
 *   offset16 = fp16(lo); s, o = those fp16 values;
 *   q = s == 0 ? 0 : clamp(rint(f32(w - o) / s), 0, 2^b - 1)   (ties to even).
 * W: device, N x K float32, row-major, 16-byte aligned.
 * widths: device, N x K/64 uint8 in natural order (the same values given to
 *   vbq_pack_query for the sizes in m).
 * m: host descriptor; every field must be set from vbq_pack_query and the
 *   two device pointers. Invalid widths, or a layout that does not match the
 *   descriptor, are detected on the device: nothing is then written beyond the
 *   tile table, and vbq_matrix_check reports the error. */
vbq_status vbq_pack(const float* W, const uint8_t* widths, const vbq_matrix* m, hipStream_t stream);

/* Waits for `stream` and reads the totals entry written by vbq_pack.
 * Returns VBQ_OK, VBQ_ERR_BITWIDTH (invalid widths on the device) or
 * VBQ_ERR_CAPACITY (layout larger than the descriptor's sizes). */
vbq_status vbq_matrix_check(const vbq_matrix* m, hipStream_t stream);

/* Fused dequantise-and-multiply (VBQ abstract: a kernel that dequantises and
 * multiplies in one pass, for memory-bandwidth-bound decode):
 *   y[b][n] = sum_k x[b][k] * (s*q + o + r[n][k])     (r only if residual != NULL)
 * accumulated in fp32; codes are never expanded in memory. The sum over a
 * tile's 4096 columns is formed first; several k-tiles (and the residual's
 * part) are then added in a fixed order inside one workgroup.
 * x: device, B x K fp16, 16-byte aligned. B in [1, VBQ_MAX_BATCH].
 * residual: device, N x K fp16 row-major (natural order), 16-byte aligned, or
 *   NULL. NULL serves the released artifact; the in-cell update (CellFill
 *   abstract) is revoked simply by passing NULL.
 * y: device, B x N float32, 4-byte aligned; fully overwritten.
 * Batches run as passes of at most 4 rows (2 with a residual); each code is
 * decoded once per pass and multiplied with every row of the pass. */
vbq_status vbq_gemv(const vbq_matrix* m, const uint16_t* x, int32_t B, const uint16_t* residual, float* y,
                    hipStream_t stream);

/* Compact in-cell residual (CellFill abstract, page "Nothing Changed but the
 * Model: CellFill -- Bounded In-Cell Learning for Bit-Identical, Revocable
 * Updates to Quantized LLMs": the update is a residual inside each weight's
 * rounding cell, served beside the frozen artifact and revoked by dropping
 * it). The page fixes no storage for the residual; this library's compact
 * form is one signed byte f per weight in [-127, 127], standing for
 *   r[n][k] = s[n][g] * f[n][k] / 256        (g = k / 64, s the fp16 scale)
 * so |r| <= 127/256 s < s/2: every encodable residual is inside its cell.
 *
 * vbq_gemv_cell8: y[b][n] = sum_k x[b][k] * (s*q + o + s*f/256), fp32
 *   accumulation, the residual term of each (row, group) added to the
 *   group's record term before the tile's row sums. Arguments as vbq_gemv;
 *   cell: device, N x K int8 row-major (natural order), 16-byte aligned,
 *   not NULL (the base weights are vbq_gemv with residual NULL).
 * cell8_encode: f = clamp(rint(f32(r / s) * 256), -127, 127) per weight in
 *   binary32 (IEEE division, ties to even), f = 0 where s = 0; residuals
 *   beyond the cell clamp to its edge. residual: device, N x K fp16 (finite
 *   values), 16-byte aligned; cell: device, N x K int8, 16-byte aligned,
 *   fully overwritten.
 * cell8_decode: r = fp16(s * f / 256) (exact before the one rounding), the
 *   fp16 residual that vbq_gemv and cell_requant_verify take. cell and
 *   residual as above; residual fully overwritten.
 * Scales come from the packed matrix m, so the residual follows the scales
 * that are served. */
vbq_status vbq_gemv_cell8(const vbq_matrix* m, const uint16_t* x, int32_t B, const int8_t* cell, float* y,
                          hipStream_t stream);
vbq_status cell8_encode(const vbq_matrix* m, const uint16_t* residual, int8_t* cell, hipStream_t stream);
vbq_status cell8_decode(const vbq_matrix* m, const int8_t* cell, uint16_t* residual, hipStream_t stream);

/* Several independent GEMVs in one launch (same batch B, no residual; VBQ
 * abstract, fused dequantise-and-multiply): y_i = x_i . dequant(W_i)^T for
 * i < count <= VBQ_MAX_LAUNCH_MATS. ms, xs, ys: host arrays of `count`
 * entries (descriptors and device pointers as for vbq_gemv). Used to run all
 * projections of a decoder layer as one launch. */
vbq_status vbq_gemv_batched(int32_t count, const vbq_matrix* ms, const uint16_t* const* xs, float* const* ys,
                            int32_t B, hipStream_t stream);

/* vbq_gemv_batched for callers that cannot allocate (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation), spread
 * over more workgroups: every k-tile of a matrix with K > 4096 gets a
 * workgroup of its own, and the row sums of a row-tile's k-tiles meet in a
 * scratch area the library keeps in static device memory (one copy per
 * device, 1 MiB of partial sums and 16384 row-tile counters, held until the
 * process ends; nothing is allocated per call). The workgroup that finishes
 * a row-tile's last k-tile adds the partial sums in k-tile order, the order
 * vbq_gemv_batched uses, so both calls give the same bits, and sets the
 * row-tile's counter back to zero. Arguments and results as for
 * vbq_gemv_batched. A launch needing more than the scratch holds (more than
 * 8192 tiles of such matrices at one batch row, 8192 / min(B, 4) at B rows) returns
 * VBQ_ERR_UNSUPPORTED before anything is enqueued. Calls that overlap in
 * time on one device race on the scratch and must not be made; a call whose
 * kernels do not complete can leave counters behind for the next call. */
vbq_status vbq_gemv_batched_static(int32_t count, const vbq_matrix* ms, const uint16_t* const* xs,
                                   float* const* ys, int32_t B, hipStream_t stream);

/* GEMV over several levels of one weight matrix (RRQ abstract on page
 * thelatestinai.com/papers/2512.18934: a 2-bit base plus 2-bit residual
 * levels served from one checkpoint), in one launch:
 *   y[b][n] = sum over levels i of x[b] . dequant(W_i)[n]
 * (the levels' k-tiles are summed in a fixed order, fp32)
 * ms: host array of `count` <= VBQ_MAX_LAUNCH_MATS descriptors of equal N
 * and K (else VBQ_ERR_SHAPE). x: device, B x K fp16 (B = 1..8), 16-byte
 * aligned. y: device, B x N float32, 4-byte aligned, fully overwritten. */
vbq_status vbq_gemv_levels(int32_t count, const vbq_matrix* ms, const uint16_t* x, int32_t B, float* y,
                           hipStream_t stream);

/* Batched dequantise-and-multiply for M >= 64 tokens (VBQ abstract: the fused
 * dequantise-and-multiply, here for many tokens at once): tiles of W are
 * decoded to bf16 in LDS and contracted on MFMA with fp32 accumulation.
 *   y[m][n] = sum_k x[m][k] * bf16(fma(s, q, o))
 * where fma is the binary32 fused multiply-add (one rounding of s*q + o) and
 * bf16 rounds to nearest even. Any M >= 1 is accepted; the path pays off from
 * about 64 tokens. x_bf16: device, M x K bfloat16, 16-byte aligned, with
 * M * K * 2 < 2^32 (else VBQ_ERR_UNSUPPORTED). y: device, M x N float32,
 * 16-byte aligned, fully overwritten. */
vbq_status vbq_gemm(const vbq_matrix* m, const uint16_t* x_bf16, int32_t M, float* y, hipStream_t stream);

/* Re-quantisation check of an in-cell update (CellFill abstract: the
 * release's codes and scales stay frozen, the residual stays inside each
 * weight's cell, and re-quantising gives back the released codes exactly).
 * For every weight, in binary32 without contraction, with s, o, r the fp16
 * values and L = 2^b - 1 of the weight's group:
 *   deq = f32(s*q) + o;  v = deq + r;
 *   q'  = s == 0 ? 0 : clamp(rint((v - o) / s), 0, L)
 *   mismatch    when q' != q
 *   out of cell when s > 0 ? |r| >= 0.5*s : r != 0
 * Scales and offsets are frozen (carried through unchanged).
 * residual: device, N x K fp16 natural order, 16-byte aligned.
 * result: device, 3 x uint64, 8-byte aligned: { mismatches, out-of-cell
 *   count, smallest linear index n*K + k with either, or UINT64_MAX }.
 * requant_codes: device, same size as m->stream (16-byte aligned), receives a
 *   copy of the stream with every code replaced by its re-quantised value
 *   (map, scales, offsets and padding copied), so the artifact can be
 *   compared bit-for-bit; may be NULL. */
vbq_status cell_requant_verify(const vbq_matrix* m, const uint16_t* residual, uint64_t* result,
                               uint32_t* requant_codes, hipStream_t stream);

/* The error a packed level leaves (RRQ abstract on page
 * thelatestinai.com/papers/2512.18934: each residual level quantises what the
 * levels before it leave):
 *   E_out[n][k] = E_in[n][k] - (f32(s*q) + o)
 * in binary32, one rounding per operation; the next level is vbq_pack of
 * E_out. E_in, E_out: device, N x K float32 natural order, 8-byte aligned;
 * E_out may be E_in. Every width is accepted. */
vbq_status vbq_residual_error(const vbq_matrix* m, const float* E_in, float* E_out, hipStream_t stream);

/* Drift bound of an in-cell update (CellFill abstract: bounded drift). For
 * every residual with each |r[n][k]| below half its group's scale,
 *   |y_r[b][n] - y[b][n]| = |sum_k x[b][k] r[n][k]| <= bound[b][n], where
 *   bound[b][n] = 0.5 * sum_g s[n][g] * sum_{k in g} |x[b][k]|
 * with s the stored fp16 scales. It is computed in binary32 (each group's
 * |x| sum in k order; groups added in a fixed order), so repeated calls agree
 * bit for bit. It is the supremum: r = sign(x) s/2 attains it.
 * x: device, B x K fp16 (B = 1..8, else VBQ_ERR_UNSUPPORTED), 16-byte aligned.
 * bound: device, B x N float32, 4-byte aligned, fully overwritten. */
vbq_status cell_drift_bound(const vbq_matrix* m, const uint16_t* x, int32_t B, float* bound, hipStream_t stream);

/* ---- 4-bit key/value cache ------------------------------------------------------
 *
 * Keys and values of decoder attention, held in 4 bits in this library's
 * group format (VBQ abstract for groups of 64 and packed low-bit storage, SLQ
 * abstract for scale + offset): 64 consecutive channels of one token of one
 * key/value head are a group with 4-bit codes, an fp16 scale and an fp16
 * offset, 36 bytes per 64 values.
 *
 * Quantiser, in binary32 without contraction:
 *   w' = w is NaN ? 0 : clamp(w, -61440, 61440); lo = min, hi = max of the group;
 *   scale16 = fp16(f32(hi - lo) * f32(1/15)); offset16 = fp16(lo); s, o = those values;
 *   q = s == 0 ? 0 : clamp(rint(f32(w' - o) / s), 0, 15)       (ties to even)
 * and the value held is f32(s*q) + o. With the clamp s <= 8192, so every value
 * held is a finite number that fp16 can round to: a cache written by kv4_append
 * holds no infinity and no NaN, and a token that a mask hides cannot reach an
 * output. A NaN that was stored as 0 is reported in the flag word.
 *
 * Pages. The cache is n_pages pages of page_tokens tokens (a power of two,
 * 32 .. 65536). Position p of a sequence is token p % page_tokens of the page
 * that entry p / page_tokens of the sequence's row of the block table names.
 * A page holds, for each key/value head in turn, page_tokens / 32 blocks of 32
 * tokens; a block takes 2304 bytes per 64 channels (G = head_dim / 64 groups):
 *   1024 G bytes of key codes, 1024 G bytes of value codes (group by group),
 *   128 G bytes of key scales and offsets, 128 G bytes of value scales and
 *   offsets (per group 32 fp16 scales, then 32 fp16 offsets).
 * With t < 32 the token in its block and c < 64 the channel in its group:
 *   key codes:   u32 word 4*(16*(c%32/8) + 4*(t/8) + t%4) + 2*(t%8/4) + c/32 of
 *                the group, bits 4*(c%8) .. 4*(c%8)+3;
 *   value codes: u32 word 64*(t/8) + c of the group, bits 4*(t%8) .. 4*(t%8)+3;
 *   key scale and offset:   entry t;
 *   value scale and offset: entry 8*(t/8) + 2*(t%4) + t%8/4.
 * The words are the operands of the matrix instructions that read them, so a
 * wavefront's loads are contiguous and no code moves between lanes.
 *
 * Ownership and streams as everywhere in this header. Several sequences may
 * read a page; a page that is written belongs to one sequence. Calls that
 * write tokens another call reads must be ordered by the caller.
 *
 * Device-side errors. Lengths, starts and block tables live on the device, so
 * the kernels check them: a page outside 0 .. n_pages-1 is never touched, a
 * sequence whose numbers do not fit is left out. What was found is OR-ed into
 * the flag word. */
#define VBQ_KV4_BLOCK_TOKENS 32
#define VBQ_KV4_MAX_GROUPS 4      /* head_dim = 64, 128, 192 or 256 */
#define VBQ_KV4_FLAG_PAGE 1u      /* a block-table entry outside the cache */
#define VBQ_KV4_FLAG_LENGTH 2u    /* lengths or starts that are negative, beyond the table or the stated maxima */
#define VBQ_KV4_FLAG_NAN 4u       /* kv4_append stored a NaN as 0 */
#define VBQ_KV4_FLAG_FULL 8u      /* kv4_fork found fewer free pages than it needed */

typedef enum vbq_dtype { VBQ_F16 = 0, VBQ_BF16 = 1, VBQ_F32 = 2 } vbq_dtype;

/* Descriptor of a cache (caller-owned device buffers). */
typedef struct vbq_kv4 {
  int64_t n_pages;        /* >= 1, at most 2^31 - 1 */
  int32_t page_tokens;    /* power of two, 32 .. 65536 */
  int32_t n_kv_heads;     /* 1 .. 4096 */
  int32_t head_dim;       /* 64, 128, 192 or 256 */
  int32_t reserved;       /* 0 */
  uint8_t* data;          /* device, n_pages * kv4_page_bytes(...), 16-byte aligned */
  uint32_t* flags;        /* device, one word, or NULL */
} vbq_kv4;

/* A range of tokens of every sequence of a batch: sequence b's tokens
 * start[b] .. start[b] + cu[b+1] - cu[b] - 1 are rows cu[b] .. cu[b+1] - 1 of
 * the tensors that hold them. */
typedef struct vbq_kv4_range {
  int32_t batch;          /* 1 .. 65535 */
  int32_t table_width;    /* entries per row of the block table, >= 1 */
  int32_t total_tokens;   /* rows of the tensors, >= 0 */
  int32_t max_tokens;     /* no sequence has more rows than this; >= 0. With m the lesser of this and
                             total_tokens, (m + 62) / 32 * n_kv_heads is below 2^24 (a read: 2^26) */
  const int32_t* table;   /* device, [batch][table_width] */
  const int32_t* start;   /* device, [batch], first position */
  const int32_t* cu;      /* device, [batch + 1], cumulative row counts from 0 */
} vbq_kv4_range;

/* Bytes of one page, 0 if the sizes are not supported. Host only. */
int64_t kv4_page_bytes(int32_t page_tokens, int32_t n_kv_heads, int32_t head_dim);

/* Quantises keys and values as they are written. k, v: device, rows [token]
 * [head][channel] of type `dtype` (a vbq_dtype) with the given strides in
 * elements between tokens and heads (channels are contiguous); base pointers
 * and strides are multiples of 16 bytes. A token's place is overwritten; the
 * other tokens of its block keep theirs. */
vbq_status kv4_append(const vbq_kv4* cache, const vbq_kv4_range* r, const void* k, const void* v, int32_t dtype,
                      int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                      hipStream_t stream);

/* Reads tokens back: f32(s*q) + o rounded once to `dtype`. k, v: device,
 * [total_tokens][n_kv_heads][head_dim], contiguous, 16-byte aligned; either
 * may be NULL. Rows of tokens whose page is not in the cache are zeroed; rows of
 * a sequence that is left out, and of none, keep what they held. */
vbq_status kv4_read(const vbq_kv4* cache, const vbq_kv4_range* r, void* k, void* v, int32_t dtype,
                    hipStream_t stream);

/* Attention of new query tokens over a cache:
 *   out[t][h] = sum_j softmax_j(scale * q[t][h] . K_j) V_j
 * over the positions j that the row sees, with K, V the values held for head
 * h / (n_heads / n_kv_heads). Sequence b holds kv_lens[b] tokens; its queries
 * are rows cu_q[b] .. cu_q[b+1] - 1 and stand at its last positions, so query
 * i of n is at p = kv_lens[b] - n + i. It sees j < kv_lens[b] with
 *   causal:  j <= p
 *   window:  j > p - window or j < sinks     (window > 0, causal only)
 * A row that sees nothing gives zeros (and lse = -infinity); rows of a sequence
 * that is left out, and of none, keep what they held. A NaN or infinity
 * in q reaches the outputs of its own row only, and so does a number so large
 * that scale * log2(e) * |q| reaches 2^121. Scores have to be numbers that fp32
 * holds.
 * Scores are sums in fp32 of products of q with the exact codes; scale, offset
 * and softmax are fp32. A row of q is scaled by a power of two that brings its
 * largest number to [2^13, 2^14) and held in fp16: numbers down to 2^-27 (fp16)
 * or 2^-30 (bf16) of that largest one keep every bit, smaller ones lose their
 * low bits. The matrix unit adds eight products at a time and cuts off what lies
 * 24 bits below the largest. Where up to 32 rows (16) share a head's tokens, see
 * below, codes are subnormal numbers and cost it 6 of these bits: of a product of
 * a query and a code, what is below 2^-18 of the largest |q| of the eight.
 * The product with the values depends on the rows that share a head's tokens,
 * max_q * n_heads / n_kv_heads:
 *   up to 32 (16 for head_dim 256): exact codes times p s (p the probability, s the token's scale in
 *     the group), p s as the sum of two fp16 numbers, offsets in fp32;
 *   more: values rounded once to fp16, p rounded to fp16; for fp16 outputs what
 *     that rounding leaves of p is multiplied too.
 * All sums are fp32. Results repeat bit for bit for the same sizes (max_q and
 * max_kv among them: they decide how the work is cut). */
typedef struct vbq_kv4_attn {
  int32_t batch;          /* 1 .. 65535 */
  int32_t table_width;
  int32_t total_q;        /* rows of q, >= 0 */
  int32_t max_q;          /* no sequence has more queries than this. batch * n_kv_heads, times the tiles of 128
                             that the rows of a head take (see above), is below 2^24 (2^23 with 9 .. 32 rows) */
  int32_t max_kv;         /* no sequence holds more tokens than this */
  int32_t n_heads;        /* a multiple of the cache's n_kv_heads */
  int32_t dtype;          /* VBQ_F16 or VBQ_BF16: q and out */
  int32_t causal;         /* 0 or 1 */
  int32_t window;         /* 0: none */
  int32_t sinks;          /* first tokens that a window leaves visible */
  float scale;            /* > 0, and scale * log2(e) is a finite fp32 number */
  int32_t reserved;       /* 0 */
  const int32_t* table;   /* device, [batch][table_width] */
  const int32_t* kv_lens; /* device, [batch] */
  const int32_t* cu_q;    /* device, [batch + 1] */
  const void* q;          /* device, [total_q][n_heads][head_dim] with the strides below, 16-byte aligned */
  int64_t q_token_stride; /* in elements, multiples of 8 */
  int64_t q_head_stride;
  void* out;              /* device, [total_q][n_heads][head_dim], contiguous, 16-byte aligned */
  float* lse;             /* device, [total_q][n_heads], natural log of the sum of exponentials, or NULL */
  void* workspace;        /* device, kv4_attention_workspace() bytes, 16-byte aligned (NULL if 0). Its first
                             4 * VBQ_KV4_COUNTERS bytes are zero before the first call that uses it; every
                             call leaves them zero. Calls that overlap in time need workspaces of their own. */
  int64_t workspace_bytes;
} vbq_kv4_attn;

#define VBQ_KV4_COUNTERS 2048

/* Bytes of workspace that kv4_attention needs for these sizes (pointers are
 * not looked at), or -1 if the sizes are refused. Host only. */
int64_t kv4_attention_workspace(const vbq_kv4* cache, const vbq_kv4_attn* a);
vbq_status kv4_attention(const vbq_kv4* cache, const vbq_kv4_attn* a, hipStream_t stream);

/* ---- several continuations of one prompt ---------------------------------------------
 *
 * Parallel sampling, beam search and the scoring of candidates decode sequences
 * that begin alike. kv4_fork makes sequences of a cache go on from others,
 * kv4_attention_shared reads what a group of them has in common once for all,
 * head_norm_rotary makes the queries and keys that enter, and token_logprobs says how
 * likely the next tokens are.
 *
 * Queries and keys: norms for each head, and the rotation by position, in one pass.
 * With x a head's D channels of one token and R = rotary_dim <= D:
 *   n = x * w / sqrt(mean(x^2) + eps)          (n = x where the tensor has no weight)
 *   pair i < R/2 is channels (i, i + R/2), or (2i, 2i + 1) where `interleaved`;
 *   a' = a cos(phi_i) - b sin(phi_i), b' = b cos(phi_i) + a sin(phi_i) for a pair (a, b),
 *   phi_i = positions[axis[i]][token] * inv_freq[i] radians; channels from R on stay n.
 * Sums and products are fp32, angles binary64; one rounding to the output's type. The
 * sum of x^2 has to be a number that fp32 holds. Several axes (time, height and width of
 * an image's patches) are pairs that go by different rows of the positions. */
typedef struct vbq_head_rotary {
  int32_t head_dim;       /* D: 64, 128, 192 or 256 */
  int32_t rotary_dim;     /* R: a multiple of 16, 0 .. D */
  int32_t axes;           /* rows of the positions, 1 .. 255 */
  int32_t interleaved;    /* 0 or 1 */
  float eps;              /* >= 0, finite */
  int32_t reserved;       /* 0 */
  const float* inv_freq;  /* device, [R/2] */
  const uint8_t* axis;    /* device, [R/2], each below `axes` (larger ones count as the last), or NULL: row 0 for all */
  const float* q_weight;  /* device, [D], 16-byte aligned, or NULL: queries are not normed */
  const float* k_weight;  /* the same for keys */
} vbq_head_rotary;

/* Rows [token][head][channel] of a vbq_dtype; strides in elements. Channels are
 * contiguous; base pointers and strides are multiples of 16 bytes. An output may be its
 * own input (same pointer, type and strides) and overlaps nothing else. */
typedef struct vbq_head_rows {
  const void* in;
  void* out;
  int64_t in_token_stride, in_head_stride, out_token_stride, out_head_stride;
  int32_t heads;          /* 0 .. 65536; 0: no such tensor, nothing else is looked at */
  int32_t in_dtype;       /* the same for queries and keys */
  int32_t out_dtype;
  int32_t reserved;       /* 0 */
} vbq_head_rows;

/* positions: device, int32, row a of axis a is at positions + a * position_stride
 * (NULL if R is 0); any number, negative ones too. n_tokens >= 0; times the heads of q and k
 * together, up to 2^40 are taken. */
vbq_status head_norm_rotary(const vbq_head_rotary* plan, const vbq_head_rows* q, const vbq_head_rows* k,
                            const int32_t* positions, int64_t position_stride, int32_t n_tokens, hipStream_t stream);

/* Sequences become continuations of others. refs[page] counts the entries of block
 * tables that name a page, 0 for a free one (counts of entries in other tables, or of
 * anything else that holds a page, stay in it). Entries of a row that name no page are
 * -1. With P = page_tokens, new sequence b goes on from old sequence p = parents[b]
 * (-1: from none, it is empty), L = lens_in[p]:
 *   lens_out[b] = L;
 *   entries j < L / P (whole pages): those of p, shared;
 *   entries from there on, j < ceil((L + reserve[b]) / P): the first b with this parent
 *     keeps those of p that name a page with refs_in 1; every other entry is a free page,
 *     and the L % P tokens of a part page are copied into it (whole blocks of 32);
 *   the other entries: -1.
 * refs_out: refs_in less the entries of table_in, plus those of table_out. So an old
 * sequence that nothing goes on from is dropped, and its pages are free. The i-th page
 * taken, in the order of b, then j, is the i-th lowest with refs_in 0; pages that this
 * call frees are not taken by it. Outputs overlap no input. Entries outside 0 ..
 * n_pages-1 are left out (not -1: FLAG_PAGE; also -1 below ceil(L / P)); a parent outside
 * -1 .. batch_in-1 or with a length that does not fit counts as none, entries beyond the
 * table and negative reserves as 0 (FLAG_LENGTH); where free pages run out, entries are
 * -1 and nothing is copied (FLAG_FULL).
 * Pages are 16 GiB at most.
 * Layers of a model that share one table each have a cache of their own, of as many pages of
 * as many tokens: a call for each, with the same inputs, copies its pages and writes the same
 * tables, lengths and counts, on one stream into the same outputs.
 * kv4_fork_workspace: bytes for calls of these sizes (or less), -1 if they are refused.
 * Calls that overlap in time need workspaces of their own; nothing in it has to be set. */
typedef struct vbq_kv4_fork {
  int32_t batch_in, batch_out;  /* 1 .. 65535 */
  int32_t table_width;          /* 1 .. 2^20 */
  int32_t reserved;             /* 0 */
  const int32_t* table_in;      /* device, [batch_in][table_width] */
  const int32_t* lens_in;       /* device, [batch_in] */
  const int32_t* refs_in;       /* device, [n_pages], 16-byte aligned */
  const int32_t* parents;       /* device, [batch_out] */
  const int32_t* reserve;       /* device, [batch_out] tokens, or NULL: 0 */
  int32_t* table_out;           /* device, [batch_out][table_width] */
  int32_t* lens_out;            /* device, [batch_out] */
  int32_t* refs_out;            /* device, [n_pages], 16-byte aligned */
  void* workspace;              /* device, 16-byte aligned */
  int64_t workspace_bytes;
} vbq_kv4_fork;
int64_t kv4_fork_workspace(const vbq_kv4* cache, int32_t batch_in, int32_t batch_out, int32_t table_width);
vbq_status kv4_fork(const vbq_kv4* cache, const vbq_kv4_fork* f, hipStream_t stream);

/* Attention of sequences that have their first tokens in common: kv4_attention's results,
 * with what a group of sequences shares read once for the rows of all of them.
 * Group g is sequences cu_groups[g] .. cu_groups[g+1] - 1; its first shared[g] tokens lie
 * in the pages that the table's row of its first sequence names (the other rows' entries
 * of whole blocks of 32 among them are not read). Sequences of no group have nothing in
 * common. Queries stand behind the shared tokens: kv_lens[b] less the sequence's queries
 * is shared[g] at least. Windows are not offered (window and sinks are 0). max_kv is not
 * looked at; max_own is: no sequence holds more tokens beyond its group's shared ones.
 * A sequence for whose group or itself numbers do not fit is left out (FLAG_LENGTH).
 * The arithmetic is kv4_attention's, with the rows of a group together in place of a
 * sequence's for the shared tokens: max_group_q * n_heads / n_kv_heads decides how their values
 * are multiplied (above 32, or 16 for head_dim 256: rounded once to fp16), max_q * n_heads /
 * n_kv_heads for the own ones. Sums of both kinds are joined in fp32. Where the stated sizes are so
 * small that it takes less time (by max_shared, max_own, batch and heads at most 20000 blocks of 32
 * tokens in all, and at most 32 rows of a sequence, or 16), sequences read the shared tokens one
 * by one, with the products of their own rows: a wider bound can change the last bits.
 * Where a sequence has 128 rows of a key/value head or more by itself, kv4_attention over a
 * table whose rows all name the shared pages takes as long or less.
 * workspace: as for kv4_attention, of kv4_attention_shared_workspace() bytes, the first
 * 8 * VBQ_KV4_COUNTERS of them zero before the first call that uses it; every call, and every
 * kv4_attention on the same workspace, leaves them zero. */
typedef struct vbq_kv4_groups {
  int32_t n_groups;       /* 1 .. 65535 */
  int32_t max_shared;     /* no group shares more tokens than this */
  int32_t max_own;
  int32_t max_group_q;    /* no group's sequences have more queries in all */
  const int32_t* cu_groups; /* device, [n_groups + 1], not falling, at most batch */
  const int32_t* shared;  /* device, [n_groups] */
  int64_t reserved;       /* 0 */
} vbq_kv4_groups;
int64_t kv4_attention_shared_workspace(const vbq_kv4* cache, const vbq_kv4_attn* a, const vbq_kv4_groups* g);
vbq_status kv4_attention_shared(const vbq_kv4* cache, const vbq_kv4_attn* a, const vbq_kv4_groups* g,
                                hipStream_t stream);

/* Log probabilities of rows of logits x[0 .. vocab-1] (those of an LM head, say), in one
 * pass over them; sums are fp32:
 *   lse = log sum_i exp(x_i); logprob_i = x_i - lse; entropy = -sum_i exp(logprob_i) logprob_i
 * Tokens stand in the order of their logits, largest first, equal ones by their number:
 * rank is the given token's place in it, from 0, and the `top` first are listed. Logits may
 * be -infinity (masked). A row of nothing else has lse and log probabilities -infinity and
 * entropy 0. A row that holds a NaN or +infinity gives NaN, and -1 for rank and numbers. A
 * given token outside 0 .. vocab-1 gives NaN and -1.
 * Results repeat bit for bit for the same sizes and alignment of the rows. */
#define VBQ_LOGPROBS_MAX_TOP 32
#define VBQ_LOGPROBS_COUNTERS 512
typedef struct vbq_logprobs {
  int32_t rows;           /* >= 0; times the workgroups of a row (up to 32), below 2^24 */
  int32_t vocab;          /* 1 .. 2^30 */
  int32_t dtype;          /* a vbq_dtype */
  int32_t top;            /* 0 .. VBQ_LOGPROBS_MAX_TOP, at most vocab */
  int64_t row_stride;     /* in elements */
  const void* logits;     /* device, aligned to its type */
  const void* tokens;     /* device, [rows], int32 or int64, or NULL: none */
  int32_t token_bytes;    /* 4 or 8 */
  int32_t reserved;       /* 0 */
  float* logprob;         /* device, [rows] (with tokens) */
  int32_t* rank;          /* device, [rows] (with tokens) */
  float* entropy;         /* device, [rows], or NULL */
  float* lse;             /* device, [rows], or NULL */
  float* top_logprob;     /* device, [rows][top] (with top > 0) */
  int32_t* top_index;     /* device, [rows][top] (with top > 0) */
  void* workspace;        /* device, 16-byte aligned (NULL if 0 bytes). Its first 4 * VBQ_LOGPROBS_COUNTERS
                             bytes are zero before the first call that uses it; every call leaves them zero. Calls that overlap in time
                             need workspaces of their own. */
  int64_t workspace_bytes;
} vbq_logprobs;
int64_t token_logprobs_workspace(int32_t rows, int32_t vocab, int32_t top);
vbq_status token_logprobs(const vbq_logprobs* a, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* VBQ_H */
