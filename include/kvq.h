/*
 * kvq.h -- C ABI of the GB300 KV-cache quantisation codec (libkvq.so).
 *
 * The library turns bf16 K/V rows into compact KV-cache formats and back, with
 * hand-written sm_103a CUDA kernels:
 *   - NVFP4 row codec: per (token, KV head) row of head_dim values, packed E2M1
 *     nibbles (low nibble = even element), an E4M3 scale for each block of 16 and
 *     an FP32 scale for the row: head_dim/2 + head_dim/16 + 4 bytes (76 B at head_dim 128).
 *     Source: "feat(kvcache): add nvfp4 kv quantization (FreeToken PR #408)",
 *     Summary and the codec-delta port note.
 *   - INT4 affine codec with group size G (G64 by default), FP32 arithmetic and
 *     FP16 min/scale metadata; K grouped over token rows per (head, channel), V
 *     over channels per (token, head).  Source: "vllm-rlt PR #166: INT4 KV
 *     packing/unpacking and cross-loop residual reconstruction", Purpose.
 *   - Residual encode/decode against the reconstructed predecessor with a compact
 *     int32 position map (same page, Purpose).
 *   - FP8 E4M3 row codec: one E4M3 byte per element and a single FP32 scale for
 *     each (token, KV head) row, in a code buffer with the geometry of the bf16 one.
 *     Source: FreeToken PR #408, the fp8 store notes.
 *   - FP8 E4M3 pages: E4M3 bytes with one power-of-two FP32 scale per (block of tokens,
 *     head), raised as tokens are appended.
 * Attention reads the pool as it is: kvq_decode_attention (one query a sequence) and
 * kvq_attention (several, with score options); kvq_plan_pages makes a step's block tables
 * and slot ids on the GPU.  Over long contexts: kvq_append stores turned keys and keeps
 * their bounds, kvq_select_blocks lists the blocks that a query wants, and
 * kvq_sparse_attention reads those alone.
 *
 * Conventions shared by every entry point
 *   Memory   every pointer argument that a kernel touches is DEVICE memory
 *            (cudaMalloc / the torch caching allocator) owned by the caller.  The
 *            library allocates nothing, frees nothing and never synchronises, so
 *            every entry point but kvq_decode_attention_noalloc (see there) may be
 *            captured in a CUDA graph.  Host or unregistered
 *            pointers are rejected with KVQ_ERR_NOT_DEVICE_PTR before any launch
 *            (the FreeToken page records a host tensor handed to a kernel).
 *   bf16     K/V tensors are bf16 [rows][heads][dim] views with inner stride 1 and
 *            their OWN row and head pitches, in elements.  K and V never share a
 *            pitch argument: the FreeToken page records a store kernel that read V
 *            at K's row pitch and corrupted it.
 *   Streams  work is enqueued on `stream` (a cudaStream_t; NULL = legacy default).
 *   Errors   argument errors are returned as kvq_status before anything is
 *            launched; kvq_last_error() gives a one-line reason (thread-local).
 *            Data-dependent errors (a slot id past the pool, a block-table entry
 *            outside the pool, a bad position) can only be seen on the device: the
 *            kernel skips the offending row and ORs a KVQ_DEV_* bit into
 *            *dev_status (a caller-owned device uint32, may be NULL).  No kernel
 *            traps or asserts, so a bad id never poisons the CUDA context (the
 *            FreeToken page records a device-side assert that did).
 *   Floats   every result is bit-exact against the plain CPU definition of the
 *            codec: one IEEE binary32 operation at a time, round to nearest even,
 *            no FMA contraction, no flush to zero, in this order.  NVFP4 encode:
 *            rs = amax / 2688; per 16-block t = min((vb / 6) / rs, 448) (0 if rs is
 *            0), bs = E4M3(t), s = bs * rs, q = x * (1 / s) (x / s when 1 / s
 *            overflows, signed zeros when s is 0), code = E2M1(min(|q|, 6)) with
 *            x's sign.  NVFP4 decode: bf16((e2m1 * bs) * rs).  FP8: rs = amax / 448,
 *            q = x * (1 / rs), decode bf16(e4m3 * rs).  INT4: sc = (mx - mn) / 15,
 *            code = clamp(rint((x - mn) / sc), 0, 15) from the FP32 mn and sc (codes
 *            0 when sc is 0), then FP16 metadata; decode bf16(code * sc16 + mn16).
 *            Residuals: r = bf16(cur - prev), out = bf16(prev + decoded r).
 *   Inputs   finite values only; INT4 also needs |x| < 65504 (FP16 metadata).
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define KVQ_API __attribute__((visibility("default")))
#else
#define KVQ_API
#endif

typedef struct CUstream_st* kvq_stream_t; /* identical to cudaStream_t */

typedef enum {
  KVQ_OK = 0,
  KVQ_ERR_INVALID_ARG = 1,    /* null/negative/inconsistent sizes or pointers */
  KVQ_ERR_UNSUPPORTED = 2,    /* a valid request this build does not implement */
  KVQ_ERR_MISALIGNED = 3,     /* a base or pitch breaks the 16-byte rule below */
  KVQ_ERR_NOT_DEVICE_PTR = 4, /* a pointer is host, unregistered or managed memory */
  KVQ_ERR_CUDA = 5            /* the CUDA runtime reported an error at launch */
} kvq_status;

typedef enum {
  KVQ_FMT_NVFP4 = 1,        /* row codec: E2M1 + E4M3 per 16 + one FP32 scale per row */
  KVQ_FMT_INT4 = 2,         /* affine INT4, FP16 minimum and scale per group of G */
  KVQ_FMT_FP8 = 3,          /* E4M3 + one FP32 scale per row */
  KVQ_FMT_NVFP4_TENSOR = 4, /* E2M1 + E4M3 per 16 along the kind's axis + one FP32 scale per tensor */
  KVQ_FMT_FP8_PAGE = 5      /* pools: E4M3 + one power-of-two FP32 scale per (block of tokens, head) */
} kvq_format;
typedef enum { KVQ_KIND_KEY = 0, KVQ_KIND_VALUE = 1 } kvq_kind;

/* Bits ORed into *dev_status by the kernels. */
#define KVQ_DEV_BAD_SLOT 1u   /* slot id >= num_slots (row skipped) */
#define KVQ_DEV_BAD_BLOCK 2u  /* block-table entry < 0 or past the pool (row skipped) */
#define KVQ_DEV_BAD_POS 4u    /* position outside [0, rows) or not strictly increasing; append: past the angles */
#define KVQ_DEV_BAD_SEQLEN 8u /* seq_lens[s] outside [0, min(max_seq_len, blocks*block_size)] */
#define KVQ_DEV_NO_SPACE 32u  /* page plan: the free list or the token arrays ran out (request refused) */
#define KVQ_DEV_TIMEOUT 16u   /* attention, block choice: a bounded wait for a copy ran out (results unspecified) */

/* A bf16 view: element (r, h, d) is ptr[r*row_pitch + h*head_pitch + d].
 * ptr must be 16-byte aligned and both pitches multiples of 8 elements. */
typedef struct {
  const void* ptr;
  int64_t row_pitch;
  int64_t head_pitch;
} kvq_bf16_in;

typedef struct {
  void* ptr;
  int64_t row_pitch;
  int64_t head_pitch;
} kvq_bf16_out;

/* One tensor's planes in a paged pool, slot-major.  Format NVFP4:
 *   codes  [num_slots][num_heads][head_dim/2]   E2M1 nibbles, low nibble = even element
 *   bscale [num_slots][num_heads][head_dim/16]  E4M3 block scales
 *   rscale [num_slots][num_heads]               FP32 row scales
 * Format FP8: codes [num_slots][num_heads][head_dim] E4M3 bytes, rscale as above,
 * bscale unused (may be NULL).
 * Format FP8_PAGE: codes as FP8; rscale [num_slots / block_size][num_heads], one scale for
 * the block_size tokens of a (block, head): value = e4m3 * rscale[slot / block_size][head].
 * The library writes powers of two; kvq_restore takes any scale, attention any that is finite
 * and not negative.
 * Slot = block * block_size + offset.  Every plane used must be 16-byte aligned. */
typedef struct {
  uint8_t* codes;
  uint8_t* bscale;
  float* rscale;
} kvq_plane;

typedef struct {
  kvq_plane k;
  kvq_plane v;
  int64_t num_slots;  /* a multiple of block_size */
  int32_t block_size; /* tokens per page (16 in the pages' pools) */
  int32_t num_heads;
  int32_t head_dim;   /* a multiple of 16, at most 512 */
  int32_t fmt;        /* format of the K plane: KVQ_FMT_NVFP4, KVQ_FMT_FP8 or KVQ_FMT_FP8_PAGE */
  int32_t v_fmt;      /* format of the V plane; 0 = the same as fmt.  FP8 K with NVFP4 V
                         is the k8v4 split of the FreeToken page (fp8 store notes) */
} kvq_pool;

/* A logical (non-paged) packed tensor [rows][heads][dim], caller-allocated.
 *   fmt NVFP4: codes [rows][heads][dim/2], meta0 = bscale uint8 [rows][heads][dim/16],
 *              rscale float [rows][heads], meta1 unused; group_size must be 16.
 *   fmt FP8  : codes [rows][heads][dim] E4M3, rscale float [rows][heads]; meta0 and
 *              meta1 unused; group_size ignored.
 *   fmt NVFP4_TENSOR: the logical NVFP4 layout of vllm-rlt PR #166 (Purpose): codes
 *              [rows][heads][dim/2], meta0 = bscale uint8, [ceil(rows/16)][heads][dim]
 *              for kind KEY (16 token rows per head and channel) or [rows][heads][dim/16]
 *              for kind VALUE (16 channels), rscale float [1] = tensor amax / 2688;
 *              group_size 16.  Logical pack / unpack only.
 *   fmt INT4 : codes [rows][heads][dim/2], meta0 = FP16 minimum, meta1 = FP16 scale,
 *              each [ceil(rows/G)][heads][dim] for kind KEY (groups of G token rows
 *              per head and channel) or [rows][heads][ceil(dim/G)] for kind VALUE
 *              (groups of G channels per token and head); rscale unused.
 *              G is one of 16, 32, 64, 128, 256, 512; the last group may be partial.
 * dim must be a multiple of 16 (at most 512); pointers 16-byte aligned. */
typedef struct {
  int32_t fmt;
  int32_t kind;
  int32_t group_size;
  int32_t rows;
  int32_t heads;
  int32_t dim;
  uint8_t* codes;
  void* meta0;
  void* meta1;
  float* rscale;
} kvq_packed;

/* Fused quantise + scatter of K and V into a paged pool (the encode hot path), each
 * in its plane's format (NVFP4, FP8 E4M3 with one FP32 scale per row, or FP8 E4M3 with one
 * scale per (block, head)).
 * Source: FreeToken PR #408, Summary ("CUDA Graph-safe KV writes") and the fp8 store
 * notes (the destination slots are read from a device tensor; one launch under graph capture).
 *   k, v       bf16 [num_tokens][num_heads][head_dim] views; either may be NULL
 *              (that tensor is not stored); not both.
 *   slot_ids   device int64 [num_tokens]; token t goes to slot slot_ids[t]; a
 *              negative id skips the token (padding); an id >= num_slots skips it
 *              and sets KVQ_DEV_BAD_SLOT.  Duplicate ids: undefined last writer.
 *   pool       planes written in place (only the rows of the given slots).
 * Format FP8_PAGE appends to pages: rows of one page that stand next to each other in
 * slot_ids raise the page's scale together.  With s0 the stored scale (none where it is
 * not a positive finite number, or where these rows hold the page's first slot, which
 * starts the page over):
 *   s = max(s0, the smallest power of two p >= 2^-126 with |x| <= 448 p for every finite x)
 *   codes E4M3(x * (1 / s)), an infinity as the largest code of its sign; where s > s0 > 0
 *   the page's other rows become E4M3(code * (s0 / s)), whatever they hold.
 * All rows of a (page, head) in one call must stand next to each other (a skipped token
 * ends a run): two runs on one page, like duplicate ids, leave that page's codes and
 * scale unspecified.
 * One kernel launch (two when K and V planes have different formats); num_tokens ==
 * 0 launches nothing. */
KVQ_API kvq_status kvq_quant_scatter(const kvq_bf16_in* k, const kvq_bf16_in* v, int32_t num_tokens,
                             const int64_t* slot_ids, const kvq_pool* pool,
                             uint32_t* dev_status, kvq_stream_t stream);

/* Rotation of kvq_append: position p turns each pair (a, b) of the first rot_dim channels to
 * (a c - b s, b c + a s), c and s being the cosine and sine of the pair's angle at p. */
typedef struct {
  const float* cos_sin;     /* device f32 [num_positions][rot_dim], 16-byte aligned: the rot_dim / 2 cosines of a
                               position, then its sines (scaled frequencies and factors are the caller's
                               matter); NULL, with the other fields 0: nothing is turned */
  int32_t num_positions;
  int32_t rot_dim;          /* a multiple of 16, at most head_dim; channels behind it pass */
  int32_t interleaved;      /* 0: pairs (i, i + rot_dim / 2); else (2i, 2i + 1) */
  const int32_t* positions; /* device int32 [num_tokens] */
} kvq_rotation;

/* Append to a paged pool with the position rotation on the way: K turned, then K and V
 * quantised and scattered as kvq_quant_scatter does, Q turned beside them, and the bounds of each
 * block's keys kept for kvq_select_blocks.  One kernel launch; may be captured in a CUDA graph.
 *   k, v, slot_ids, pool  as kvq_quant_scatter (each plane in its own format; k or v may be NULL).
 *              K is turned in binary32 (every product and sum rounded once, no FMA) and goes
 *              through the codec from there, without a rounding to bf16.
 *   rotation   host struct, read during the call; NULL: K goes in as it is.
 *   q, q_out   bf16 [num_tokens][num_q_heads][head_dim]: q_out = bf16(turned q); both NULL or
 *              neither; needs a rotation.  q_out may be exactly q (same pointer and pitches);
 *              otherwise it overlaps no element of q, k or v (KVQ_ERR_INVALID_ARG; views of unlike row
 *              pitches are refused where their spans meet).
 *   key_bounds NULL, or device bf16 [num_slots / block_size][num_heads][2][head_dim], 16-byte
 *              aligned: [0] and [1] become the least and the largest bf16(turned k) of the block's rows, channel
 *              by channel: of this call's rows alone where they hold the block's first slot, else
 *              of them and what was there.  A NaN does not count.  Needs k.
 * A token whose position is negative is skipped whole (kvq_plan_pages marks those behind the last
 * with -1), as is one at num_positions or beyond (KVQ_DEV_BAD_POS); one whose slot is negative or
 * past the pool (KVQ_DEV_BAD_SLOT) has its q turned only.
 * Where the pool's format is FP8_PAGE or key_bounds is given, all rows of a block in one call must stand
 * next to each other: from the first to the last of them slot_ids holds slots of that block only
 * (tokens skipped for their position among them count for nothing; a token without a slot ends the
 * rows).  Else what the block holds of scale, codes or bounds is unspecified, as after duplicate
 * ids.  The inputs overlap no output but q_out. */
KVQ_API kvq_status kvq_append(const kvq_bf16_in* k, const kvq_bf16_in* v, int32_t num_tokens, const int64_t* slot_ids,
                              const kvq_pool* pool, const kvq_rotation* rotation, const kvq_bf16_in* q,
                              const kvq_bf16_out* q_out, int32_t num_q_heads, void* key_bounds, uint32_t* dev_status,
                              kvq_stream_t stream);

/* Paged restore: gather and dequantise pool rows back to bf16 (the decode side).  Source: FreeToken PR #408, Summary ("Triton restore paths"); vllm-rlt
 * PR #166 review (pack_paged / unpack_paged over [pages, page_size, heads, dim]).
 *   block_table  device int32 [num_seqs][max_blocks]; token t of sequence s lives in
 *                slot block_table[s][t / block_size] * block_size + t % block_size.
 *   seq_lens     device int32 [num_seqs]; tokens t >= seq_lens[s] are not written.
 *   k_out/v_out  bf16 views of [num_seqs * max_seq_len][num_heads][head_dim]: row
 *                s * max_seq_len + t receives token t of sequence s.  Either may be
 *                NULL (that tensor is not restored); not both.
 * NVFP4: y = bf16(e2m1 * block_scale * row_scale), the product rounded once in fp32;
 * FP8: y = bf16(e4m3 * row_scale); FP8_PAGE: the same with the page's scale.  One launch (two when K and V planes have
 * different formats).
 * Rows with a bad block id are skipped (KVQ_DEV_BAD_BLOCK); a sequence with a bad
 * length is skipped whole (KVQ_DEV_BAD_SEQLEN). */
KVQ_API kvq_status kvq_restore(const kvq_pool* pool, const int32_t* block_table, int32_t num_seqs,
                       int32_t max_blocks, const int32_t* seq_lens, int32_t max_seq_len,
                       const kvq_bf16_out* k_out, const kvq_bf16_out* v_out,
                       uint32_t* dev_status, kvq_stream_t stream);

/* Logical pack: x [out->rows][out->heads][out->dim] -> *out in out->fmt / kind / G.
 * Source: vllm-rlt PR #166, Purpose (pack_kv(values, kind, format)). */
KVQ_API kvq_status kvq_pack(const kvq_bf16_in* x, const kvq_packed* out, kvq_stream_t stream);

/* Logical unpack: *in -> y [in->rows][in->heads][in->dim] bf16.
 * Source: vllm-rlt PR #166, Purpose (unpack_kv(packed)).
 * INT4: y = bf16(code * scale16 + min16), a mul then an add in fp32. */
KVQ_API kvq_status kvq_unpack(const kvq_packed* in, const kvq_bf16_out* y, kvq_stream_t stream);

/* Residual encode against the reconstructed predecessor.
 * Source: vllm-rlt PR #166, Purpose (encode_residual(current, previous, kind,
 * format); the kept rows are packed together, each call owning its int32 position list).
 *   cur, prev   bf16 [num_rows][heads][dim] (heads/dim from payload).
 *   pos         device int32 [num_pos], strictly increasing in [0, num_rows), or
 *               NULL for the dense case (then num_pos must equal num_rows).
 *   payload     packed [num_pos][heads][dim]: r[p] = bf16(cur[pos[p]] - prev[pos[p]])
 *               encoded in payload->fmt / kind / G (INT4 KEY groups follow the
 *               compact row order).  payload->rows must equal num_pos.
 *   pos_out     device int32 [num_pos] receiving the owned copy of pos (NULL: none).
 * A position outside [0, num_rows) contributes a zero residual row and sets
 * KVQ_DEV_BAD_POS; an unsorted map sets KVQ_DEV_BAD_POS (results then unspecified,
 * never out of bounds). */
KVQ_API kvq_status kvq_encode_residual(const kvq_bf16_in* cur, const kvq_bf16_in* prev,
                               int32_t num_rows, const int32_t* pos, int32_t num_pos,
                               const kvq_packed* payload, int32_t* pos_out,
                               uint32_t* dev_status, kvq_stream_t stream);

/* Residual decode: out = prev, and for every kept row p,
 * out[pos[p]] = bf16(prev[pos[p]] + unpack(payload)[p]).  Absent rows inherit prev.
 * Source: vllm-rlt PR #166, Purpose (decode_residual(residual, previous)).
 *   out  may be exactly prev (same pointer and pitches: in-place, only the kept rows
 *        are touched) or must not overlap it (every row is written).
 * Bad positions: as kvq_encode_residual (rows outside [0, num_rows) are skipped). */
KVQ_API kvq_status kvq_decode_residual(const kvq_packed* payload, const int32_t* pos, int32_t num_pos,
                               const kvq_bf16_in* prev, int32_t num_rows,
                               const kvq_bf16_out* out, uint32_t* dev_status,
                               kvq_stream_t stream);

/* Paged decode attention over a quantised pool: the step downstream of the
 * restore, with K and V dequantised in registers instead of restored to bf16.
 * Source: FreeToken PR #408, Summary (restore paths) and fp8 store notes (the row
 * scale multiplies the score and the output); vllm-rlt PR #166, review by 0z5a
 * (dequantise to 16 bits in registers and keep the 16-bit MMA).
 * One query token per sequence.  For query head qh (KV head qh / (num_q_heads /
 * pool->num_heads)):
 *   out[s][qh] = softmax_t(scale * q[s][qh] . k_t) . v_t   over t < seq_lens[s],
 * with k_t, v_t the decoded pool rows (each plane in its own format: NVFP4, FP8 or
 * FP8_PAGE).  What the pool holds behind a sequence's last token is never used.
 *   q    bf16 [num_seqs][num_q_heads][head_dim] through q->row_pitch (per sequence)
 *        and q->head_pitch (per head), inner stride 1; 16-byte aligned.
 *   out  bf16, indexed the same way through its own pitches.
 *   head_dim 64, 128 or 256; num_q_heads a multiple of num_heads, at most 16 query
 *   heads per KV head.  seq_lens[s] <= min(max_seq_len, max_blocks * block_size), which may
 *   be up to 2^31 - 65536 tokens (KVQ_ERR_UNSUPPORTED above).
 *   scale  positive and finite (KVQ_ERR_INVALID_ARG otherwise).
 *   workspace  device memory of kvq_decode_attention_workspace(...) bytes, 16-byte
 *              aligned (may be NULL when that is 0); caller-owned, reused by the next
 *              call on the same stream.
 * Accuracy: K, V and Q enter the f16 MMA exactly (Q through a power-of-two
 * prescale); products and sums are fp32; P is rounded once to f16 (relative 2^-11,
 * relative to a reference of V's row scales) and the output once to bf16, so
 * |out - exact| <= 2^-9 |exact| + (2^-11 + 2^-24 n) max|v| plus fp32 rounding, where exact is
 * the attention of the decoded rows and n counts the keys of less than 2^-14 of the largest
 * weight (P in f16 ends at 2^-25; only many thousands of such keys in one split show).
 * A NaN in a row of q, or in a K row that it sees, makes its output NaN.
 * An empty sequence writes zeros.  A bad length (KVQ_DEV_BAD_SEQLEN) or a block
 * entry outside the pool (KVQ_DEV_BAD_BLOCK) leaves that sequence's output untouched.
 * Every wait of the kernel on a copy into shared memory is bounded (about 0.1 s); one
 * that runs out sets KVQ_DEV_TIMEOUT, and the call's results are then unspecified.
 * One or two kernel launches. */
KVQ_API kvq_status kvq_decode_attention(const kvq_pool* pool, const int32_t* block_table,
                                        int32_t num_seqs, int32_t max_blocks, const int32_t* seq_lens,
                                        int32_t max_seq_len, const kvq_bf16_in* q, int32_t num_q_heads,
                                        float scale, const kvq_bf16_out* out, void* workspace,
                                        size_t workspace_bytes, uint32_t* dev_status,
                                        kvq_stream_t stream);

/* kvq_decode_attention for callers that cannot allocate device memory.  Some callers
 * have no way to hand the library a workspace: an engine whose memory planner has
 * already given all free HBM to the KV pool, or a host runtime that passes in only
 * the tensors it owns and offers no allocator hook.  A cudaMalloc can also
 * synchronise the device, which a decode step cannot afford.  This entry point
 * allocates nothing (no cudaMalloc, cudaFree or allocating library routine): the
 * split partials go to a scratch array that is part of the library image, 48 MiB of
 * device memory that every GPU which loads the library holds until the process exits.
 * The pages have no counterpart to this entry point; it exists for such callers.
 *   Limit    the partials need kvq_decode_attention_workspace(...) bytes; a call
 *            that needs more than 48 MiB returns KVQ_ERR_UNSUPPORTED.  The split
 *            policy keeps every supported shape under 40.5 MB on a 152-SM GPU.
 *   Set-up   the first call on a device looks up the scratch array's device address
 *            (with that device current) and keeps it; make that first call before
 *            any stream capture.  A failed lookup returns KVQ_ERR_CUDA.
 *   Sharing  there is one scratch array per device, shared by every call of this
 *            entry point on it, and it keeps the last call's contents (each call
 *            writes every partial it later reads, so nothing needs clearing).  Calls
 *            that overlap on the GPU race on it; kvq_decode_attention with a caller
 *            workspace has no such limit.
 * Arguments, argument checks, results and device status are those of
 * kvq_decode_attention without the workspace pair. */
KVQ_API kvq_status kvq_decode_attention_noalloc(const kvq_pool* pool, const int32_t* block_table,
                                                int32_t num_seqs, int32_t max_blocks,
                                                const int32_t* seq_lens, int32_t max_seq_len,
                                                const kvq_bf16_in* q, int32_t num_q_heads, float scale,
                                                const kvq_bf16_out* out, uint32_t* dev_status,
                                                kvq_stream_t stream);

/* Workspace bytes kvq_decode_attention needs for these sizes on the current device
 * (0 when the call runs without one).  Host-only query. */
KVQ_API size_t kvq_decode_attention_workspace(int32_t num_seqs, int32_t num_heads, int32_t num_q_heads,
                                              int32_t head_dim, int32_t max_seq_len);

/* Options of kvq_attention; a zero field is off. */
typedef struct {
  float softcap;               /* logits become softcap * tanh(logit / softcap); 0, or 2^-10 to 2^10 */
  const float* alibi_slopes;   /* device f32 [num_q_heads]: slope * (key position - query position) is added
                                  to the (capped) logit; finite */
  int32_t window;              /* a query at position p sees keys t > p - window only; >= 0 */
  const int32_t* prefix_lens;  /* device int32 [num_seqs]: every query of sequence s also sees the keys behind
                                  it up to t < min(prefix_lens[s], seq_lens[s]) */
  const int32_t* key_starts;   /* device int32 [num_tokens]: a query sees keys t >= key_starts[token] only
                                  (the first token of its document, or the end of left padding) */
} kvq_attn_options;

/* Paged attention of several query tokens per sequence over a quantised pool: prompt
 * chunks behind a cached prefix, draft tokens, single tokens with score options, any mix of
 * them in one call.  Beside kvq_decode_attention, whose one query sees its whole sequence.
 * (max_query_len picks the kernel for all sequences of a call: many single tokens beside a long
 * chunk are faster as two calls.)
 *   query_starts  device int32 [num_seqs + 1]: sequence s owns rows query_starts[s] ..
 *                 query_starts[s + 1] - 1 of q and out, its LAST n tokens: row i of them sits
 *                 at position p = seq_lens[s] - n + i.  Their K and V rows are in the pool
 *                 already (kvq_plan_pages, kvq_quant_scatter).  n = 0 is fine.
 *                 The starts do not decrease.
 * With lo = max(0, p + 1 - window, key_starts[row]) and hi = max(p + 1, prefix), row and
 * query head qh (KV head qh / (num_q_heads / pool->num_heads)) get
 *   softmax over t in [lo, hi) of  cap(scale * q . k_t) + slope * (t - p),  times v_t;
 * a row that sees no key gets zeros.  The options combine as written: with prefix_lens a
 * query also sees keys of later documents below the prefix, since key_starts bounds its document
 * on the left only, and alibi_slopes favours the keys ahead of it (t > p) over those behind;
 * neither happens without a prefix.  Cache rows outside the span of the keys that a
 * sequence's rows see (unwritten rows behind it, left padding before it) are never used,
 * whatever they hold.
 *   q, out        bf16 [num_tokens][num_q_heads][head_dim] through their own pitches.
 *   max_query_len at least the largest n (at most max_seq_len is used).
 *   min(max_seq_len, max_blocks * block_size) up to 2^31 - 65536 tokens (KVQ_ERR_UNSUPPORTED above).
 *   head_dim 64, 128 or 256; at most 16 query heads per KV head; scale positive, finite.
 *   options       host struct, read during the call; NULL: plain causal attention.
 *   workspace     device memory of kvq_attention_workspace(...) bytes, 16-byte aligned (may be
 *                 NULL when that is 0); caller-owned.  Calls that may overlap on the GPU, and
 *                 graphs that may replay at the same time, need one each.
 * Accuracy as kvq_decode_attention (one f16 rounding of P, one bf16 rounding of out; products,
 * maxima and sums in fp32), max|v| being that of the keys that the row sees, with 2^-30 n in place
 * of 2^-24 n (2^-25 n for a row whose mask hides keys of larger V from it), for V scales between
 * 2^-48 and 2^48, 0 and the 2^-126 that a store gives a page of zeros, and K scales up to 2^64;
 * the cap is within 2^-20 of
 * softcap absolutely.  Waits are bounded as there (KVQ_DEV_TIMEOUT).
 * A NaN in a row of q, or in a K row that a query sees, makes NaN of that query's output and of
 * no other's; one in a V row may reach every query of its sequence.
 * A sequence whose length is outside [0, min(max_seq_len, max_blocks * block_size)], or whose
 * query rows are outside [0, num_tokens], more than max_query_len or more than its length,
 * keeps its rows of out (KVQ_DEV_BAD_SEQLEN); rows that need a block entry outside the pool
 * keep theirs (KVQ_DEV_BAD_BLOCK); rows of no sequence keep theirs.
 * One or two kernel launches; may be captured in a CUDA graph. */
KVQ_API kvq_status kvq_attention(const kvq_pool* pool, const int32_t* block_table, int32_t num_seqs,
                                 int32_t max_blocks, const int32_t* seq_lens, int32_t max_seq_len,
                                 const kvq_bf16_in* q, const int32_t* query_starts, int32_t num_tokens,
                                 int32_t max_query_len, int32_t num_q_heads, float scale,
                                 const kvq_attn_options* options, const kvq_bf16_out* out, void* workspace,
                                 size_t workspace_bytes, uint32_t* dev_status, kvq_stream_t stream);

/* Workspace bytes kvq_attention needs for these sizes on the current device (0 when the
 * call runs without one).  Host-only query. */
KVQ_API size_t kvq_attention_workspace(int32_t num_seqs, int32_t num_tokens, int32_t num_heads,
                                       int32_t num_q_heads, int32_t head_dim, int32_t max_query_len,
                                       int32_t max_seq_len);

/* Blocks of the cache that a query token wants, for each KV head: those with the highest bound on a
 * score.  With the g = num_q_heads / num_heads query heads of KV head h and the bounds lo, hi of a
 * block's keys (kvq_append),
 *   score(block) = sum_d [ (sum_g max(q_gd, 0)) hi_d + (sum_g min(q_gd, 0)) lo_d ]  >=  sum_g q_g . k_t
 * for every key t of the block as kvq_append turned it (up to the rounding of the bounds; the key that
 * attention reads is that one rounded to the pool's format, and may lie outside them by as much).  A query
 * at position p chooses among blocks 0 to p / block_size: the first_blocks first and the last_blocks last of them in any case, then the
 * highest scores until topk are listed (all of them where there are no more than topk); equal scores
 * go by the lower index.
 *   key_bounds     device bf16 [num_blocks][num_heads][2][head_dim], 16-byte aligned.
 *   block_table, seq_lens, max_seq_len, q, query_starts, num_tokens, max_query_len  as kvq_attention.
 *   selected       device int32 [num_tokens][num_heads][topk]: block numbers within the sequence
 *                  (indexes of its block_table row), ascending, -1 behind the last.  Rows of no
 *                  sequence, and of a refused one (KVQ_DEV_BAD_SEQLEN), keep theirs.
 *   head_dim 64, 128 or 256; at most 16 query heads per KV head; first_blocks + last_blocks <=
 *   topk; sequences of up to 32768 blocks (any number where topk reaches for all of them).
 *   workspace      device memory of kvq_select_blocks_workspace(...) bytes, 16-byte aligned;
 *                  caller-owned; one for each call that may run at the same time.  It holds every score:
 *                  about 4 bytes for each (query token, KV head, block of max_seq_len), 2.3 GB for 8192 tokens
 *                  over 131,072 in 16-token blocks and 8 heads.  A long chunk may come in pieces, each with
 *                  the sequence's length up to its own last token: the lists are the same.
 * max_query_len picks the kernels and the grid for all sequences of a call: many single tokens beside a long
 * chunk are faster as two calls (512 tokens at the end of 32768 and 63 single tokens over 8192 each, 16-token
 * blocks, 8 heads, head_dim 128, 64 listed: 547 us as one call, 157 as two).
 * The list is that of the exact scores: what binary32 cannot tell apart is scored again, in pairs of
 * binary32 numbers or in binary64 (scores of unlike blocks that agree to 2^-38 of their terms' size may go
 * either way).  A NaN score ranks below all numbers, and a
 * block whose table entry lies outside the pool below that (KVQ_DEV_BAD_BLOCK, where scores are needed).
 * Two kernel launches (one where topk reaches for all blocks of max_seq_len); may be captured in
 * a CUDA graph. */
KVQ_API kvq_status kvq_select_blocks(const void* key_bounds, int64_t num_blocks, int32_t block_size, int32_t num_heads,
                                     int32_t head_dim, const int32_t* block_table, int32_t num_seqs, int32_t max_blocks,
                                     const int32_t* seq_lens, int32_t max_seq_len, const kvq_bf16_in* q,
                                     const int32_t* query_starts, int32_t num_tokens, int32_t max_query_len,
                                     int32_t num_q_heads, int32_t first_blocks, int32_t last_blocks, int32_t topk,
                                     int32_t* selected, void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                     kvq_stream_t stream);

/* Workspace bytes kvq_select_blocks needs for these sizes.  Host-only query. */
KVQ_API size_t kvq_select_blocks_workspace(int32_t num_tokens, int32_t num_heads, int32_t max_seq_len, int32_t block_size);

/* Attention over listed blocks of the cache: kvq_attention's causal form (no window, prefix, key
 * starts or ALiBi bias) with, for each query token and KV head, only the keys of its listed blocks.
 *   selected   device int32 [num_tokens][num_heads][topk], as kvq_select_blocks writes it or from
 *              elsewhere: block numbers within the sequence, in any order; an entry that is negative
 *              or behind the query's own block counts for nothing, one that stands there twice
 *              counts twice.  topk at most 4096.
 * A query at position p sees the keys t <= p of its blocks; a row that sees none gets zeros.  Keys
 * of other blocks are not read.  The grid goes by max_query_len: many single tokens beside a long chunk are faster
 * as two calls (the step above: 365 us as one call, 190 as two).
 *   softcap    0, or 2^-10 to 2^10: logits become softcap * tanh(logit / softcap).
 *   workspace  device memory of kvq_sparse_attention_workspace(...) bytes, 16-byte aligned (may be
 *              NULL when that is 0); caller-owned; one for each call that may run at the same time.
 * All else (pool formats, head_dim, heads, accuracy, refused sequences, NaN) as kvq_attention;
 * rows (token, KV head) whose list needs a block entry outside the pool keep what they held
 * (KVQ_DEV_BAD_BLOCK).  One or two kernel launches; may be captured in a CUDA graph. */
KVQ_API kvq_status kvq_sparse_attention(const kvq_pool* pool, const int32_t* block_table, int32_t num_seqs,
                                        int32_t max_blocks, const int32_t* seq_lens, int32_t max_seq_len,
                                        const kvq_bf16_in* q, const int32_t* query_starts, int32_t num_tokens,
                                        int32_t max_query_len, int32_t num_q_heads, const int32_t* selected,
                                        int32_t topk, float scale, float softcap, const kvq_bf16_out* out,
                                        void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                        kvq_stream_t stream);

/* Workspace bytes that are enough for kvq_sparse_attention at these sizes, and at any smaller
 * num_tokens and topk, on the current device (0 when all those calls run without one): one buffer sized for the
 * largest step serves every step.  A call refuses only less than it uses itself, which
 * kvq_sparse_attention_workspace_exact tells.  Host-only query. */
KVQ_API size_t kvq_sparse_attention_workspace(int32_t num_tokens, int32_t num_heads, int32_t num_q_heads, int32_t head_dim,
                                              int32_t block_size, int32_t topk);

/* Workspace bytes that a call at exactly these sizes uses, on the current device: for a caller that allocates for
 * each call (most calls use none, and fewer tokens may use more).  Host-only query. */
KVQ_API size_t kvq_sparse_attention_workspace_exact(int32_t num_tokens, int32_t num_heads, int32_t num_q_heads,
                                                    int32_t head_dim, int32_t block_size, int32_t topk);

/* Page plan of a step: block tables, slot maps and lengths from request lengths, on the
 * GPU, ready for kvq_quant_scatter, kvq_decode_attention and kvq_attention.
 * Request s holds cached_lens[s] tokens (c) and gets new_lens[s] more (n).  It takes
 * ceil((c + n) / block_size) - ceil(c / block_size) blocks off free_blocks, requests in order:
 *   block_table  [num_seqs][max_blocks]: the entries of the new blocks are written, no other.
 *   seq_lens     [num_seqs]: c + n.
 *   query_starts [num_seqs + 1]: prefix sums of n (at most max_tokens).
 *   slot_ids     [max_tokens]: token query_starts[s] + i goes to the slot of position c + i;
 *                -1 behind the last token (kvq_quant_scatter skips those).
 *   positions    [max_tokens]: c + i; -1 behind the last token.  May be NULL.
 *   num_used     [1]: how many blocks of the free list are taken.
 * All int32 (slot_ids int64) device memory; no output may overlap another of the arrays
 * (KVQ_ERR_INVALID_ARG).
 * A request is refused when a length is negative or c + n exceeds max_blocks * block_size
 * (KVQ_DEV_BAD_SEQLEN), or when the free list or max_tokens does not reach for it
 * (KVQ_DEV_NO_SPACE): its seq_lens entry and slots become -1, so that the calls after this
 * one leave it alone, and its table row stays; later requests that need blocks are refused
 * with it once the free list has run out.  A token whose block entry is negative gets
 * slot -1 (KVQ_DEV_BAD_BLOCK).
 * One kernel launch; may be captured in a CUDA graph. */
KVQ_API kvq_status kvq_plan_pages(const int32_t* cached_lens, const int32_t* new_lens, int32_t num_seqs,
                                  const int32_t* free_blocks, int32_t num_free, int32_t block_size,
                                  int32_t* block_table, int32_t max_blocks, int32_t* seq_lens,
                                  int32_t* query_starts, int64_t* slot_ids, int32_t* positions,
                                  int32_t max_tokens, int32_t* num_used, uint32_t* dev_status,
                                  kvq_stream_t stream);

/* Bytes held by codes plus scale sidecars for rows x heads x dim in a format,
 * excluding allocator overhead (vllm-rlt PR #166 review: storage_bytes).  76 per
 * NVFP4 row at dim 128; INT4 G64: 4 + 32/64 bits per element for full groups; FP8_PAGE:
 * group_size is the block size.
 * Returns 0 for an invalid request.  Host-only; needs no GPU. */
KVQ_API size_t kvq_storage_bytes(kvq_format fmt, kvq_kind kind, int32_t group_size, int64_t rows,
                         int32_t heads, int32_t dim);

/* Static name of a status code.  Host-only. */
KVQ_API const char* kvq_status_string(kvq_status status);

/* One-line reason for the last non-OK status returned on this thread. */
KVQ_API const char* kvq_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* KVQ_H */
