/*
 * fa.h -- C ABI of the B200 (sm_100a) exact-attention library (libfa_b200.so).
 *
 * The library computes exact scaled-dot-product attention
 *
 *     O = softmax(scale * Q K^T + mask) V,      L_i = ln sum_j exp(scale * q_i . k_j + mask_ij)
 *
 * block by block with an online softmax, so the N x N score matrix never reaches
 * device memory.  The formula is the one the FlashAttention pages print
 * (FlashAttention (NL), "Problemen met standaard attention", with 1/sqrt(d_k) as the
 * usual scale); the tiling, the online softmax (running row maximum and running sum of
 * exponentials) and the single fused kernel are that page's "Tiling en blokgewijze
 * verwerking", "Online berekening van Softmax" and "Samensmelting van bewerkingen in een
 * CUDA-kernel"; the backward recomputes the probabilities from L instead of storing them
 * (memory-optimized flash attention page, "How it works").
 *
 * Conventions shared by every entry point
 *   Layout     Q, K, V, O, dO, dQ, dK, dV are contiguous bf16 arrays [B, H, N, d] (d fastest,
 *              row stride d elements, head stride N*d); L is contiguous fp32 [B, H, N].
 *              Self-attention: queries and keys have the same length N.
 *   Pointers   every array argument is a DEVICE pointer of the current CUDA device; the
 *              caller allocates, owns and frees all of them.  The library allocates no
 *              device memory and keeps no pointer after a call returns.
 *   Streams    `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *              Every call only enqueues work on that stream and returns; it never
 *              synchronises (fa_check_status excepted).
 *   Masks      causal = 1 keeps key j for query i iff j <= i.  window = W > 0 with
 *              causal = 1 also requires j >= i - W + 1 (one-sided band); with causal = 0
 *              it keeps |i - j| <= W - 1 (the local window on both sides).  Either band
 *              counts the diagonal, so W = 1 keeps only key i; window = 0 means no band.
 *              (The sparse-attention glossary, "Abgrenzung & Vergleiche", names sliding-
 *              window attention as a purely local window and fixes no convention.)  Keys
 *              j >= N never exist.  Every query keeps its diagonal, so no row is empty
 *              (the paged forwards, whose sequences may hold no key, excepted).
 *   Scale      applied inside: S = scale * Q K^T.  Must be finite and > 0.
 *   Errors     arguments are validated before anything is enqueued; a rejected call
 *              returns its FA_ERR_* code and touches no memory.  A failed launch returns
 *              FA_ERR_CUDA.  Kernel-side waits are bounded: one that runs out records a
 *              timeout in a device status word that fa_check_status() reports.
 *   Device     a compute-capability 10.0 GPU (B200, sm_100a); others give FA_ERR_DEVICE.
 */
#ifndef FA_B200_H
#define FA_B200_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FA_EXPORT __attribute__((visibility("default")))
#else
#define FA_EXPORT
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_NULL = 1,       /* a required pointer is NULL */
  FA_ERR_SHAPE = 2,      /* a size < 1, H not a multiple of H_kv, N_q > N_k, or beyond the launch limits */
  FA_ERR_HEADDIM = 3,    /* d is not 64, 128 or 256 */
  FA_ERR_ALIGN = 4,      /* a bf16 array is not 16-byte aligned, or L not 4-byte aligned */
  FA_ERR_MASK = 5,       /* causal not 0/1, or window < 0 */
  FA_ERR_WORKSPACE = 6,  /* workspace missing or smaller than fa_bwd_ / fa_decode_workspace_size */
  FA_ERR_CUDA = 7,       /* a CUDA runtime call or kernel launch failed */
  FA_ERR_DEVICE = 8,     /* the current device is not compute capability 10.0 */
  FA_ERR_TIMEOUT = 9,    /* a kernel-side wait ran out of time (reported by fa_check_status) */
  FA_ERR_SCALE = 10,     /* scale is not finite and > 0 */
  FA_ERR_NOALLOC_LIMIT = 11, /* fa_bwd_noalloc: fa_bwd_workspace_size(...) exceeds its 64 MiB scratch */
  FA_ERR_INTERNAL = 12,  /* a kernel found it could not run as built (reported by fa_check_status) */
  FA_ERR_PHASES = 13,    /* fa_bwd_phases: phase mask outside 1..7 */
  FA_ERR_CACHE = 14,     /* fa_paged_kv: a count < 1, page_size not a multiple of 16 or > 32768, table_stride < max_pages */
  FA_ERR_INDEX = 15,     /* a page number, length, count or position was out of range (reported by fa_check_status) */
  FA_ERR_ROTATION = 16   /* fa_rotation: rot, axes or sections out of range */
} fa_status;

/*
 * Forward pass.  Writes O (bf16 [B,H,N,d]) and L (fp32 [B,H,N], natural-log logsumexp of
 * the masked, scaled scores of each query row).  Reads q, k, v (bf16 [B,H,N,d]).
 * d must be 64, 128 or 256.  Extra device memory: none beyond O and L.  d = 256 runs a kernel of
 * its own (one 128-row query tile per CTA, 64-key K/V tiles).
 */
FA_EXPORT int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
           float scale, int causal, int window, void* stream);

/*
 * Bytes of device workspace fa_bwd needs: 4 * B*H * Np * (d + 2) with Np = N rounded up to
 * a multiple of 128 (per row: D, L in log2 units, and a d-wide fp32 dQ accumulator).
 * Returns 0 when the shape itself is invalid.  O(N * d): no N x N buffer.
 */
FA_EXPORT size_t fa_bwd_workspace_size(int B, int H, int N, int d);

/*
 * Backward pass with recomputation.  From q, k, v, the forward's o and lse, and the output
 * gradient dO (bf16 [B,H,N,d]) it writes dQ, dK, dV (bf16 [B,H,N,d]): the gradients of
 * sum(O o dO).  Same mask, scale and shape arguments as the forward that produced o and lse.
 * `workspace` (device, caller-owned, 16-byte aligned, at least fa_bwd_workspace_size bytes)
 * is scratch: it is overwritten and may be reused once the call's work has completed on
 * `stream`.  Three kernels are enqueued: D = rowsum(dO o O) with a cleared accumulator, the
 * fused recompute kernel, and the dQ scaling.  d must be 64, 128 or 256; d = 256 runs a kernel of
 * its own (one CTA per 64-key tile and head-dim half).
 */
FA_EXPORT int fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                     void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal, int window,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * The backward pass split into its three phases, so that a caller can time or interleave
 * them.  `phases` is a mask of
 *   1  preprocess: D = rowsum(dO o O), L in log2 units and a cleared fp32 dQ accumulator,
 *      all in `workspace`;
 *   2  the recompute kernel: dK and dV written, dQ accumulated in `workspace`;
 *   4  finalise: dQ = scale * accumulator, written as bf16.
 * Calling it with 1, then 2, then 4 on one stream with the same arguments and workspace
 * does exactly what one fa_bwd call (mask 7) does.  Arguments, validation and errors are
 * fa_bwd's; a mask outside 1..7 gives FA_ERR_PHASES.
 */
FA_EXPORT int fa_bwd_phases(const void* q, const void* k, const void* v, const void* o, const float* lse,
                            const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale,
                            int causal, int window, void* workspace, size_t workspace_bytes, int phases,
                            void* stream);

/*
 * Element strides of one bf16 array of logical shape [B, heads, N, d] whose d elements are
 * contiguous: element (b, h, n, c) is at b * b_stride + h * h_stride + n * n_stride + c.  The
 * packed layout [B, heads, N, d] is {heads*N*d, N*d, d}; [B, N, heads, d] (sequence-major) is
 * {N*heads*d, d, heads*d}.
 */
typedef struct fa_strides {
  long long b, h, n;
} fa_strides;

/*
 * Shared K/V heads (multi-query and grouped-query attention).  The FlashAttention (NL) page
 * lists Multi-Query Attention among what FlashAttention-2 supports ("Evolutie en verdere
 * ontwikkelingen"); here H query heads read H_kv K/V heads (H a multiple of H_kv; H_kv = 1 is
 * multi-query, H_kv = H is fa_fwd / fa_bwd), in contiguous groups: query head h reads K/V
 * head h / (H / H_kv).  q, o, dO, dq: bf16 [B,H,N,d]; k, v, dk, dv: bf16 [B,H_kv,N,d]; lse:
 * fp32 [B,H,N].  dk and dv are the sums over each K/V head's query heads.  Everything else
 * (masks, scale, ownership, errors, streams) is as for fa_fwd / fa_bwd; the workspace is
 * fa_bwd_workspace_size(B, H, N, d) bytes (it scales with the query heads), and `phases` is
 * as for fa_bwd_phases (7 = the whole backward).  FA_ERR_SHAPE also when H_kv < 1 or H is not
 * a multiple of H_kv.
 */
FA_EXPORT int fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv,
                         int N, int d, float scale, int causal, int window, void* stream);
FA_EXPORT int fa_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const float* lse,
                         const void* dO, void* dq, void* dk, void* dv, int B, int H, int H_kv, int N, int d,
                         float scale, int causal, int window, void* workspace, size_t workspace_bytes,
                         int phases, void* stream);

/*
 * fa_fwd_gqa / fa_bwd_gqa on arrays with arbitrary strides (for instance the sequence-major
 * [B, N, H, d] layout of many frameworks) instead of packed ones.  `strides` (host memory)
 * holds one fa_strides per array: q, k, v, o for the forward (4 entries, or NULL for packed
 * arrays); q, k, v, o, dO, dq, dk, dv for the backward (8 entries, not NULL).  Every stride must
 * be a positive multiple of 8 elements (FA_ERR_ALIGN otherwise); strides that make an output
 * overlap itself are the caller's error.  lse stays packed fp32 [B, H, N].  The pages print no
 * layout: the strides only say where the same [B, heads, N, d] elements live.
 */
FA_EXPORT int fa_fwd_strided(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                             int H_kv, int N, int d, const fa_strides* strides, float scale, int causal, int window,
                             void* stream);
FA_EXPORT int fa_bwd_strided(const void* q, const void* k, const void* v, const void* o, const float* lse,
                             const void* dO, void* dq, void* dk, void* dv, int B, int H, int H_kv, int N, int d,
                             const fa_strides* strides, float scale, int causal, int window, void* workspace,
                             size_t workspace_bytes, int phases, void* stream);

/*
 * Forward of a few new query rows over a longer key sequence: a generation step over a
 * key/value cache.  The FlashAttention (NL) page names engines for LLM inference that work on
 * the key/value cache during streaming generation ("Gespecialiseerde oplossingen": FlashInfer;
 * its references add FlashDecoding++); it prints no interface.  Reading: the N_q query rows are
 * the last N_q of the N_k key positions, so query row i stands at position N_k - N_q + i and
 * the masks of fa_fwd apply there (causal: keys j <= N_k - N_q + i; with a window W also
 * j >= N_k - N_q + i - W + 1; a window without causal keeps |j - (N_k - N_q + i)| <= W - 1).
 * N_q = N_k is the self-attention of fa_fwd_gqa.
 *
 *   q, o   bf16 [B, H, N_q, d];  k, v  bf16 [B, H_kv, N_k, d]  (H a multiple of H_kv; query
 *          head h reads K/V head h / (H / H_kv));  lse  fp32 [B, H, N_q], packed.
 *   strides  NULL for packed arrays, else 4 fa_strides (q, k, v, o) as for fa_fwd_strided.
 *   d      64, 128 or 256.
 *   workspace  device memory of at least fa_decode_workspace_size(...) bytes, 16-byte aligned,
 *          owned by the caller; it holds the per-split partial results (fp32).  When that size
 *          is 0 (the keys fit one split) workspace may be NULL.
 *
 * The keys are cut into splits that run on separate CTAs; a second kernel merges the splits'
 * partial outputs by their logsumexps.  How the problem is cut depends only on the arguments
 * of fa_decode_workspace_size, which returns 0 for an invalid problem.  Errors, scale, streams
 * and ownership are as for fa_fwd; FA_ERR_SHAPE also when N_q > N_k, FA_ERR_WORKSPACE when the
 * workspace is missing or short.
 */
FA_EXPORT size_t fa_decode_workspace_size(int B, int H, int H_kv, int N_q, int N_k, int d, int causal, int window);
FA_EXPORT int fa_fwd_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv,
                            int N_q, int N_k, int d, const fa_strides* strides, float scale, int causal, int window,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_fwd_decode over an FP8 key/value cache.  The FlashAttention (NL) page says FlashAttention-3
 * supports FP8 ("Evolutie en verdere ontwikkelingen"), without a format; the reading is that
 * paper's E4M3 with one scale per tensor: K = k_scale * E4M3(k8), V = v_scale * E4M3(v8), where
 * E4M3 has 1 sign, 4 exponent (bias 7) and 3 mantissa bits, subnormals, no infinities, and
 * S.1111.111 as NaN (NaN codes give NaN results).
 *
 *   k8, v8   E4M3 codes, one byte each, [B, H_kv, N_k, d]; with `strides`, their strides count
 *            bytes and must be multiples of 16.
 *   k_scale, v_scale  finite and > 0 (FA_ERR_SCALE otherwise).
 *   everything else as for fa_fwd_decode (q, o bf16; lse fp32; the same workspace size,
 *   fa_decode_workspace_size).
 *
 * The kernels convert the codes to f16, which is exact, and run the products with f16 operands:
 * Q is rounded to f16 after clamping to +-65504, and P enters P V as f16.  k_scale multiplies
 * the softmax scale; v_scale multiplies O before it is rounded to bf16.
 */
FA_EXPORT int fa_fwd_decode_fp8kv(const void* q, const void* k8, const void* v8, float k_scale, float v_scale,
                                  void* o, float* lse, int B, int H, int H_kv, int N_q, int N_k, int d,
                                  const fa_strides* strides, float scale, int causal, int window, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * Forward on FP8 (E4M3) Q, K and V with one scale per tensor: Q = q_scale * E4M3(q8),
 * K = k_scale * E4M3(k8), V = v_scale * E4M3(vt8)^T; the FP8 forward the FlashAttention (NL)
 * page attributes to FlashAttention-3 ("Evolutie en verdere ontwikkelingen").  E4M3 as for
 * fa_fwd_decode_fp8kv.  Both products run on the tensor cores' 8-bit path (E4M3 x E4M3 -> fp32);
 * P is rounded to E4M3 before P V (O carries that rounding: relative 2^-4 per weight).
 *
 *   q8     E4M3 codes [B, H, N, d], packed;  k8  [B, H_kv, N, d], packed.
 *   vt8    V transposed: E4M3 codes [B, H_kv, d, N], packed (N contiguous), so that both operands
 *          of the 8-bit P V product are K-major.
 *   o, lse bf16 [B, H, N, d] and fp32 [B, H, N], packed.
 *   d must be 128 (FA_ERR_HEADDIM otherwise); N a multiple of 16 (FA_ERR_SHAPE); the scales
 *   finite and > 0 (FA_ERR_SCALE).  Masks, scale, errors and streams as for fa_fwd_gqa.
 *
 */
FA_EXPORT int fa_fwd_fp8(const void* q8, const void* k8, const void* vt8, float q_scale, float k_scale, float v_scale,
                         void* o, float* lse, int B, int H, int H_kv, int N, int d, float scale, int causal, int window,
                         void* stream);

/*
 * Paged key/value cache.  Keys and values of many sequences live in pages of page_size rows that
 * are handed out as sequences grow: row j of sequence b is row j % page_size of page
 * table[b * table_stride + j / page_size].
 *
 *   k, v        bf16 pages [n_pages, H_kv, page_size, d], or (fp8 = 1) E4M3 codes of the same
 *               shape, one byte each, with K = k_scale * E4M3(k), V = v_scale * E4M3(v).
 *   *_strides   element strides; b steps from page to page, h from head to head, n from row to row.
 *               Positive multiples of 8 (fp8: 16) elements; the packed layout is
 *               {H_kv*page_size*d, page_size*d, d}.
 *   table       device int32 [B, max_pages], rows table_stride >= max_pages apart.  Only the
 *               entries that the lengths reach are read.
 *   page_size   a multiple of 16, at most 32768.
 *   k_scale, v_scale   finite and > 0, and so must be what the kernels form of them in fp32 (FA_ERR_SCALE):
 *               1 / k_scale and 1 / v_scale in the append, scale * k_scale * log2(e) in the forwards.
 *               Not read with fp8 = 0.
 *
 * Page numbers, lengths, counts and positions live on the device, so that a captured graph follows a
 * growing cache.  One that is out of range is never used as an address, and fa_check_status reports
 * FA_ERR_INDEX:
 *   a position     its row is not stored, neither q nor k and v;
 *   a page number  the append leaves its rows' k and v out (their q needs no page); the forwards read
 *                  zeros;
 *   a length past the table's reach   the append leaves k and v out of the rows past it; the forwards
 *                  read it as the table's reach;
 *   a count        is read as 0 or N, the nearer of the two.
 * A negative length is read as 0, an idle slot, and is no error.
 */
typedef struct fa_paged_kv {
  void* k;
  void* v;
  const int* table;
  fa_strides k_strides, v_strides;
  long long table_stride;
  int n_pages, page_size, max_pages, fp8;
  float k_scale, v_scale;
} fa_paged_kv;

/*
 * Position rotation.  Pair p of a head, standing at position t, turns by the angle whose cosine and
 * sine are cos_t[t][p] and sin_t[t][p]: (a, b) -> (a cos - b sin, b cos + a sin).
 *
 *   cos_t, sin_t  device fp32 [n_angles, rot / 2], packed, 16-byte aligned.
 *   rot           rotated elements of a head, its first ones: a multiple of 16, at most d.
 *   interleaved   0: pair p is elements (p, p + rot / 2); 1: elements (2p, 2p + 1).
 *   axes          1 to 4.  sections[a] >= 1 pairs, in order, turn by axis a's position (for
 *                 instance time, height and width of a film's rows); they add up to rot / 2.
 *   positions     device int32 [axes, B, N], packed; NULL (one axis only): the row's place in
 *                 its sequence.
 */
typedef struct fa_rotation {
  const float* cos_t;
  const float* sin_t;
  const int* positions;
  int rot, n_angles, axes, interleaved;
  int sections[4];
} fa_rotation;

/*
 * Appends N new rows per sequence to a paged cache, rotating q and k on the way.
 *
 *   q, q_out   bf16 [B, H, N, d]: rotated q; q_out may be q.  H = 0: none (both NULL).
 *   k, v       bf16 [B, H_kv, N, d].
 *   lengths    device int32 [B]: keys of each sequence AFTER the append.
 *   counts     device int32 [B], 0 to N: rows of each sequence that are new, its first ones
 *              (NULL: all N; the attention after it then takes the same counts, see
 *              fa_fwd_paged_ragged).  Row i < counts[b] becomes row lengths[b] - counts[b] + i of its
 *              sequence.  Rows past counts[b], and rows whose place would be negative (an idle
 *              slot with length 0), are padding: nothing of them is written, q_out neither.
 *   rotation   NULL: none; q is then copied to q_out.
 *   strides    NULL for packed arrays, else 4 fa_strides (q, k, v, q_out).
 *   d          64, 128 or 256.
 *
 * The rotation runs in fp32; its result is rounded once, to bf16, or to the nearest E4M3 code of
 * value * (1 / scale), values past 448 to 448.  Pages that are not written keep their contents.  Where two
 * rows name the same place of a page (a page that stands in the tables twice), each run of 8 elements there
 * may come from either.
 */
FA_EXPORT int fa_kv_append(const void* q, const void* k, const void* v, void* q_out, const fa_paged_kv* cache,
                           const int* lengths, const int* counts, const fa_rotation* rotation, int B, int H, int H_kv,
                           int N, int d, const fa_strides* strides, void* stream);

/*
 * Forward of N_q new query rows per sequence over a paged cache: fa_fwd_decode with a length of
 * its own for each sequence.  Query row i of sequence b stands at position lengths[b] - N_q + i,
 * where the causal and window masks apply; a row that no key is allowed for (an idle slot with
 * length 0, a causal row before its sequence's first key) gives O = 0 and L = -inf.
 *
 * The ragged form follows an append with the same counts: of sequence b's N_q rows the first
 * counts[b] are new ones, row i at position lengths[b] - counts[b] + i, as fa_kv_append placed it; the
 * others are padding, whatever they hold, and give O = 0 and L = -inf.
 *
 *   q, o       bf16 [B, H, N_q, d]; o may be q; lse fp32 [B, H, N_q], packed; lengths device int32 [B].
 *   counts     device int32 [B], 0 to N_q (NULL: all N_q).
 *   strides    NULL for packed arrays, else 2 fa_strides (q, o).
 *   workspace  device memory of at least fa_paged_workspace_size(...) bytes, 16-byte aligned,
 *              owned by the caller; overwritten, and free again once the call's work is done.
 *              Calls that may run at the same time need one each.
 *
 * Two kernels are enqueued.  Meant for few rows: every 16 rows of a K/V head (its query heads
 * times N_q) pass over the keys once.  FA_ERR_SHAPE also when B * H_kv * ceil(rows / 16) *
 * (ceil(table's keys / step) + 2) comes to 2^31 or more, whatever the lengths are (step: 16 keys, or 32 at
 * d = 64 and 64 at d = 64 over E4M3 pages, 32 at d = 128 over E4M3 pages; 4096 sequences with 8 heads and a
 * table of a million keys each do at d = 128), for tables of more than 2^29 keys a sequence, and for
 * N_q > 2^28.
 *
 * Over bf16 pages P enters P V as bf16; over E4M3 pages the products run on f16 operands: K and V
 * exactly, Q rounded to f16 after clamping to +-65504, P as f16 (weights below 2^-29 of a row's largest, or
 * 2^-25 in a shared prefix, with fewer bits, and lost below 2^-40, or 2^-36).  NaN stays NaN.  Infinities and NaN
 * in rows of a page that no query row may attend do not reach the result.
 */
FA_EXPORT size_t fa_paged_workspace_size(int B, int H, int H_kv, int N_q, int d);
FA_EXPORT int fa_fwd_paged(const void* q, const fa_paged_kv* cache, const int* lengths, void* o, float* lse, int B,
                           int H, int H_kv, int N_q, int d, const fa_strides* strides, float scale, int causal,
                           int window, void* workspace, size_t workspace_bytes, void* stream);
FA_EXPORT int fa_fwd_paged_ragged(const void* q, const fa_paged_kv* cache, const int* lengths, const int* counts,
                                  void* o, float* lse, int B, int H, int H_kv, int N_q, int d,
                                  const fa_strides* strides, float scale, int causal, int window, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * fa_fwd_paged for a batch whose sequences all begin with the same prefix_len keys: their part is
 * computed once for the whole batch, each K/V head's rows of all sequences together on the tensor
 * cores, and joined with each sequence's own part by the logsumexps.
 *
 *   prefix_len    0 to 2^29.
 *   prefix_pages  device int32, ceil(prefix_len / page_size) page numbers of `cache`.  prefix_len = 0
 *                 (prefix_pages may be NULL) is fa_fwd_paged.
 *   lengths, cache->table   each sequence's OWN keys, those after the prefix.  Row i of sequence b
 *                 stands at position prefix_len + lengths[b] - N_q + i (ragged: - counts[b] + i); it
 *                 attends the whole prefix, and its own keys as in fa_fwd_paged (causal or all; there is
 *                 no window).
 *   workspace     at least fa_shared_workspace_size(...) bytes.
 *
 * Everything else as for fa_fwd_paged.  Three kernels are enqueued.
 */
FA_EXPORT size_t fa_shared_workspace_size(int B, int H, int H_kv, int N_q, int d, int prefix_len);
FA_EXPORT int fa_fwd_shared(const void* q, const fa_paged_kv* cache, const int* prefix_pages, int prefix_len,
                            const int* lengths, void* o, float* lse, int B, int H, int H_kv, int N_q, int d,
                            const fa_strides* strides, float scale, int causal, void* workspace, size_t workspace_bytes,
                            void* stream);
FA_EXPORT int fa_fwd_shared_ragged(const void* q, const fa_paged_kv* cache, const int* prefix_pages, int prefix_len,
                                   const int* lengths, const int* counts, void* o, float* lse, int B, int H, int H_kv,
                                   int N_q, int d, const fa_strides* strides, float scale, int causal, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Human-readable name of a status code (static string, never NULL). */
FA_EXPORT const char* fa_status_string(int status);

/*
 * Synchronises `stream`, then reads and clears the device status word of the current
 * device.  Returns FA_ERR_INTERNAL if a kernel since the last check refused to run (its
 * dynamic shared memory was not 1 KB aligned), else FA_ERR_TIMEOUT if one gave up on a
 * bounded wait, else FA_ERR_INDEX if a page number, length, count or position was out of range,
 * FA_ERR_CUDA if the synchronisation failed, FA_OK otherwise.
 */
FA_EXPORT int fa_check_status(void* stream);

/*
 * Time limit, in nanoseconds, of every kernel-side wait launched after this call
 * (process-wide; default 4e9 = 4 s).  0 restores the default.
 */
FA_EXPORT void fa_set_wait_limit_ns(unsigned long long limit_ns);

/*
 * Failure-detection self-test: enqueues one small kernel that waits on a barrier nothing
 * ever completes, under a limit of `limit_ns` nanoseconds (clamped to [1 us, 1 s]).  The
 * wait runs out, the kernel records a timeout and exits, and the next fa_check_status()
 * returns FA_ERR_TIMEOUT.  No memory is touched besides the status word.
 */
FA_EXPORT int fa_selftest_timeout(unsigned long long limit_ns, void* stream);

/*
 * Backward pass for callers that cannot allocate device memory.  The FlashAttention pages
 * have no counterpart of this entry point; it exists for code that may not call cudaMalloc
 * and has no allocator to ask: for example an operator running as a plugin inside a host
 * framework that owns all device memory, or a latency-critical service that forbids
 * allocation (which can synchronise the device) once it has started.
 *
 * Same arguments and results as fa_bwd, without the workspace: the scratch (D, L and the
 * fp32 dQ accumulator) lives in one 64 MiB array inside the library, which every GPU that
 * loads the library holds until the process exits.  Problems whose
 * fa_bwd_workspace_size(B, H, N, d) exceeds 64 MiB (67108864 bytes) are rejected with
 * FA_ERR_NOALLOC_LIMIT before anything is enqueued; for d = 128 that allows
 * B*H*ceil(N/128)*128 <= 129055 rows, e.g. 31 heads of N = 4096.
 *
 * The first call on a device looks up the array's device address (cudaGetSymbolAddress,
 * with that device current), so make that first call before any stream capture begins.
 * The call itself allocates nothing (no cudaMalloc, cudaFree or allocating library call);
 * every scratch byte the kernels read is rewritten at the start of each call.  All calls
 * share the one array: two calls whose work overlaps on the GPU (different streams, or
 * several host threads) race on it and give wrong results -- serialise them.
 */
FA_EXPORT int fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const float* lse,
                             const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                             float scale, int causal, int window, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_B200_H */
