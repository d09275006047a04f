/*
 * moe_w8a8 -- fused W8A8 MoE expert block for AMD MI355X (gfx950).
 *
 * One call runs the expert block of a DeepSeek-style decode step on one GPU:
 *   1. dispatch grouping: per-local-expert token counts (expert_token_nums),
 *      their exclusive prefix sum and the stable (expert, token, k) row order;
 *   2. per-row dynamic INT8 quantisation of x (optionally times smooth scales);
 *   3. grouped INT8 GEMM1 (gate and up halves) with exact int32 accumulation;
 *   4. dequantisation by per-output-channel weight scale x per-row scale,
 *      SwiGLU, and per-row INT8 requantisation;
 *   5. grouped INT8 GEMM2 (down) and dequantisation to bf16;
 *   6. routing-weighted top-k combine into `output`, and the optional shared
 *      expert on every active token into `share_output`.
 * Options of the same call (moe_w8a8_dims_t): the routing weight folded into
 * GEMM2's row scale (fuse_route_scale), group-wise activation scales
 * (quant_mode 2), and FP4 weights with FP8 activations (weight_format).
 * Around it (at the end of this file): the pre-norm with 8-bit output, the
 * router, and dense products with 4-bit weights; dense products in 8-bit
 * integers, the quantiser of an activation, the norm that joins the block's
 * outputs to the residual stream, and tokens sorted by expert and back.
 *
 * Passages that define the operation (pages, by title):
 *   "FusedDeepMoE Kernel 深度分析报告": sec. 1.2 (inputs, outputs, attributes),
 *     sec. 2.1 (tiling info: ep size/rank, experts per rank, bs, k, h, 2*inter),
 *     sec. 4.1 (dispatch: counts, prefix sum, quantisation fused in dispatch),
 *     sec. 4.2 (combine: fp32 sum over k of row x routing weight, one bf16 cast),
 *     sec. 6.1 (int32 -> fp32, x weight scale per column, x per-token scale,
 *               left half x/(1+exp(-x))), sec. 6.2 (same dequant, cast to bf16),
 *     sec. 7.2 (BlockQuant: scale = max|h|/127, q = rint(h*127/max)),
 *     sec. 9.4 (supported ranges).
 *   "DeepSeek V4 Decode Optimization" sec. 0: INT8 weights with FP32
 *     per-output-channel scales; activations quantised per token, amax
 *     floored by an eps and rescaled to 127; scales stay FP32.
 *
 * Conventions shared by every entry point:
 *   - Tensor pointers are DEVICE pointers, row-major, owned by the caller; the
 *     library never frees or retains them. 16-byte alignment is required for
 *     x, output, share_output and every weight; the workspace must be 256-byte
 *     aligned.
 *   - Calls are stream-ordered and asynchronous: no host synchronisation, no
 *     allocation. The library keeps no state between calls, so calls are
 *     reentrant when each uses its own workspace; two calls in flight that
 *     share one workspace race.
 *   - Host-detectable errors (bad sizes, NULL required pointers, misaligned
 *     pointers, short workspace) return a negative status and launch nothing.
 *     A pair whose expert id lies outside [0, moe_expert_num) is dropped and
 *     counted in a diagnostics word (readable through moe_w8a8_debug_t).
 *     HIP launch failures return MOE_ERR_HIP; faults inside kernels surface at
 *     the caller's next synchronisation.
 */
#ifndef MOE_W8A8_H
#define MOE_W8A8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__) || defined(__clang__)
#define MOE_W8A8_API __attribute__((visibility("default")))
#else
#define MOE_W8A8_API
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1, /* NULL / misaligned pointer, inconsistent sizes */
    MOE_ERR_UNSUPPORTED = -2, /* legal for the operator, outside what this library runs */
    MOE_ERR_WORKSPACE = -3,   /* workspace pointer NULL or workspace_bytes too small */
    MOE_ERR_HIP = -4,         /* a HIP runtime call or kernel launch failed */
    MOE_ERR_SCRATCH_LIMIT = -5 /* moe_w8a8_forward_noalloc: the call needs more
                                  than MOE_W8A8_NOALLOC_SCRATCH_BYTES of workspace */
} moe_status_t;

/* Sizes and attributes of one call (FusedDeepMoE sec. 1.2 attributes and the
 * sec. 2.1 tiling struct, minus the communication-only group_ep / global_bs). */
typedef struct {
    int32_t num_tokens;     /* T >= 0 rows of x; T == 0 is legal (all counts 0)     */
    int32_t hidden;         /* H > 0, multiple of 256                                */
    int32_t inter;          /* I > 0, multiple of 256; GEMM1 has 2*I outputs:        */
                            /*   gate = rows [0, I), up = rows [I, 2I) of gmm1_weight */
    int32_t share_inter;    /* I_s: shared-expert intermediate, multiple of 256;     */
                            /*   0 = no shared expert                                */
    int32_t topk;           /* K in [1, 16]                                          */
    int32_t moe_expert_num; /* E_g >= 1 global routed experts                        */
    int32_t ep_rank_size;   /* >= 1, divides E_g; E_loc = E_g / ep_rank_size <= 512  */
    int32_t ep_rank_id;     /* in [0, ep_rank_size): local experts are global ids    */
                            /*   [ep_rank_id*E_loc, (ep_rank_id+1)*E_loc)            */
    int32_t quant_mode;     /* 1 = per-token dynamic INT8; 2 = per token and group:  */
                            /*   one amax / scale per row and group of quant_group   */
                            /*   consecutive elements along the contraction, each    */
                            /*   group's int32 partial dequantised by its own scale  */
                            /*   and the groups summed in fp32 ("DeepSeek V4 Decode  */
                            /*   Optimization" sec. 3.1); see quant_group            */
    float amax_eps;         /* > 0: row amax floor (e.g. 1e-6)                       */
    int32_t weight_layout;  /* MOE_WEIGHT_ROW_MAJOR: the layouts listed at           */
                            /*   moe_w8a8_forward; MOE_WEIGHT_PACKED: all four       */
                            /*   weight tensors come from moe_w8a8_pack_weights      */
    int32_t fuse_route_scale; /* 0: combine multiplies each routed bf16 row by its   */
                            /*   routing weight (FusedDeepMoE sec. 4.2); 1: the     */
                            /*   weight is folded into the row's GEMM2 dequant scale */
                            /*   (fl(hs * w), "DeepSeek V4 Decode Optimization" sec. */
                            /*   2.3) and combine only sums; z rows then carry it    */
    int32_t weight_format;  /* MOE_WEIGHT_INT8: the W8A8 block above.               */
                            /*   MOE_WEIGHT_MXFP4: the FP8/FP4 variant of the expert */
                            /*   GEMMs ("FIFO Pipeline Analysis ... Mega MoE": FP8   */
                            /*   GEMMs, FP8 cast after SwiGLU, FP4 weights): x and h */
                            /*   are quantised per row to FP8 E4M3 (scale = a'/448, */
                            /*   q = e4m3((v*448)/a'), round to nearest even,        */
                            /*   saturating), the weights are OCP E2M1 with one E8M0 */
                            /*   scale per 32 k elements and keep their fp32         */
                            /*   per-channel scales, the GEMMs accumulate in fp32.   */
                            /*   Requires weight_layout == MOE_WEIGHT_PACKED (else   */
                            /*   MOE_ERR_UNSUPPORTED) with every weight tensor       */
                            /*   written by moe_w8a8_pack_weights_mx; the debug      */
                            /*   acc1 / acc2 dumps then hold fp32 bit patterns       */
    int32_t quant_group;    /* quant_mode 2: elements per group, 64, 128 or 256      */
                            /*   (so it divides H, I and I_s); INT8 weights only,    */
                            /*   not with fuse_route_scale (MOE_ERR_UNSUPPORTED      */
                            /*   otherwise). The debug                               */
                            /*   xs / hs dumps then hold H/G and max(I, I_s)/G       */
                            /*   scales per row, acc1 / acc2 the fp32 bits of the    */
                            /*   dequantised group sums. Ignored for quant_mode 1    */
    int32_t requant_in_epilogue; /* 0: h is requantised by a launch of its own.     */
                            /*   1: inside GEMM1's epilogue where the batch runs the */
                            /*   decode GEMM (T <= 16, INT8 weights, quant_mode 1):  */
                            /*   the last of a chunk's GEMM1 workgroups to finish    */
                            /*   quantises the chunk's rows, found by an arrival     */
                            /*   count per chunk that the same call's routing resets */
                            /*   ("FIFO Pipeline Analysis ... Mega MoE": the first   */
                            /*   GEMM's epilogue ends in the cast after SwiGLU, with */
                            /*   arrival counts; "FusedDeepMoE Kernel 深度分析报告"  */
                            /*   sec. 7: SwiGLU and quantisation fused). Results are */
                            /*   identical either way; other batches ignore it       */
} moe_w8a8_dims_t;

enum { MOE_WEIGHT_ROW_MAJOR = 0, MOE_WEIGHT_PACKED = 1 };
enum { MOE_WEIGHT_INT8 = 0, MOE_WEIGHT_MXFP4 = 1 };

/* Optional intermediates for testing (every field may be NULL; all are device
 * buffers written in stream order). Rows are "grouped rows": rows [0, P) are
 * the kept routed pairs in (local expert, token, k) order, rows [P, P+T_act)
 * the shared expert's rows, one per active token in token order. With
 * R = T*K + T rows of capacity and Imax = max(I, I_s):                       */
typedef struct {
    int32_t *sorted_pair;   /* [T*K]   pair id t*K+k of routed row r           */
    int32_t *row_of_pair;   /* [T*K]   routed row of pair t*K+k, -1 if dropped */
    int32_t *group_offset;  /* [E_loc+1] exclusive prefix sum of the counts    */
    int32_t *shared_token;  /* [T]     token of shared row P+i                 */
    int32_t *num_rows;      /* [4]     P, T_act, #ids out of range, #chunks    */
    int8_t  *q_x;           /* [R, H]  GEMM1 input codes                       */
    float   *xs;            /* [R]     their per-row dequant scale             */
    int32_t *acc1;          /* [R, 2*Imax] GEMM1 int32 accumulators            */
    float   *h;             /* [R, Imax] SwiGLU output (fp32)                  */
    int8_t  *q_h;           /* [R, Imax] GEMM2 input codes                     */
    float   *hs;            /* [R]     their per-row dequant scale             */
    int32_t *acc2;          /* [R, H]  GEMM2 int32 accumulators                */
    uint16_t *z;            /* [R, H]  bf16 GEMM2 output rows                  */
    void   **stage_events;  /* [6] caller-created hipEvent_t (NULL entries are
                               skipped), recorded on the stream before routing
                               and after each stage: routing with the
                               quantisation of x, GEMM1, requant, GEMM2,
                               combine                                        */
    void   **kernel_events; /* [4] caller-created hipEvent_t (NULL entries are
                               skipped) bound to the GEMM kernels themselves
                               (hipExtLaunchKernel): start and end of the GEMM1
                               launch, start of the first and end of the last
                               GEMM2 launch. Unlike stage_events they add no
                               marker between kernels, so their elapsed times
                               are the kernels' own durations.               */
} moe_w8a8_debug_t;

/* Workspace bytes that moe_w8a8_forward needs for these dims. The size depends
 * only on T, H, I, I_s, K, E_loc and the options. The workspace holds every
 * intermediate the launches of one call hand to each other, as FusedDeepMoE
 * sec. 2.2 (workspace layout) does: the grouped rows' quantised GEMM1 input and
 * its scales, the SwiGLU output, the quantised GEMM2 input and its scales, the
 * GEMM2 output rows before combine, and the per-expert counts, prefix sum and
 * row order; here also the GEMM work-item list and per-call counters. Returns
 * MOE_ERR_INVALID_ARG for NULL arguments and the same size errors as
 * moe_w8a8_forward. */
MOE_W8A8_API moe_status_t moe_w8a8_workspace_size(const moe_w8a8_dims_t *dims, size_t *bytes);

/*
 * The fused expert block (FusedDeepMoE sec. 1.2 signature; EP communication
 * left out: non-local pairs are dropped, so `output` holds this rank's
 * partial sum, exactly as one expert-parallel rank computes before combine).
 *
 *  x                  bf16 [T, H]   (x, expert_ids, expert_scales and output
 *                     may be NULL when T == 0)
 *  expert_ids         int32 [T, K] global expert ids
 *  expert_scales      fp32 [T, K] routing weights
 *  gmm1_weight        int8 [E_loc, 2I, H]  (output channel major, H contiguous)
 *  gmm1_weight_scale  fp32 [E_loc, 2I]
 *  gmm2_weight        int8 [E_loc, H, I]   (I contiguous)
 *  gmm2_weight_scale  fp32 [E_loc, H]
 *  share_gmm1_weight  int8 [2I_s, H], share_gmm1_weight_scale fp32 [2I_s]  } all four NULL
 *  share_gmm2_weight  int8 [H, I_s],  share_gmm2_weight_scale fp32 [H]     } iff I_s == 0
 *  expert_smooth_scales fp32 [E_loc, H] or NULL: x is multiplied by the row of
 *                     the pair's expert before quantisation
 *  share_smooth_scales  fp32 [H] or NULL (requires I_s > 0)
 *  x_active_mask      uint8 [T] (0 / non-0) or NULL = every token active
 *  output             bf16 [T, H]  sum over kept pairs (k ascending, fp32) of
 *                     expert row x routing weight, one bf16 rounding; rows of
 *                     inactive tokens or tokens with no kept pair are 0
 *  share_output       bf16 [T, H]  shared-expert output (unweighted), 0 on
 *                     inactive tokens; required iff I_s > 0, else ignored
 *  expert_token_nums  int32 [E_loc] kept pairs per local expert
 *  workspace          device scratch of >= moe_w8a8_workspace_size() bytes;
 *                     need not be zeroed; contents are undefined afterwards
 *  dbg                NULL in production; else intermediates (above)
 *  stream             hipStream_t to launch on (NULL = the default stream)
 *
 * Values: x, the routing weights, the weight scales and the smooth scales are
 * taken to be finite (the block the pages describe defines nothing else). A
 * NaN or infinity in a token's inputs makes that token's rows and outputs
 * unspecified; every row of the block is computed independently of the other
 * tokens, so the rest of the result is unaffected. Expert ids outside
 * [0, moe_expert_num) drop their pair (the routing diagnostics word counts
 * them); duplicated ids in one token's top-k are kept as separate pairs.
 */
MOE_W8A8_API moe_status_t moe_w8a8_forward(const moe_w8a8_dims_t *dims,
                              const void *x,
                              const int32_t *expert_ids,
                              const float *expert_scales,
                              const int8_t *gmm1_weight,
                              const float *gmm1_weight_scale,
                              const int8_t *gmm2_weight,
                              const float *gmm2_weight_scale,
                              const int8_t *share_gmm1_weight,
                              const float *share_gmm1_weight_scale,
                              const int8_t *share_gmm2_weight,
                              const float *share_gmm2_weight_scale,
                              const float *expert_smooth_scales,
                              const float *share_smooth_scales,
                              const uint8_t *x_active_mask,
                              void *output,
                              void *share_output,
                              int32_t *expert_token_nums,
                              void *workspace,
                              size_t workspace_bytes,
                              const moe_w8a8_debug_t *dbg,
                              void *stream);

/*
 * moe_w8a8_forward without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc). Every other argument, the result and the
 * errors are those of moe_w8a8_forward; the call allocates nothing (no
 * hipMalloc, no hipFree, no allocating library routine).
 *
 * The workspace is a device array built into the library,
 * MOE_W8A8_NOALLOC_SCRATCH_BYTES bytes on each GPU the library runs on, held
 * from module load until the process ends. Its device address is looked up
 * on the first call on each device (the device that is current at the call,
 * which must be the stream's device). Calls whose workspace (see
 * moe_w8a8_workspace_size) would exceed it return MOE_ERR_SCRATCH_LIMIT and
 * launch nothing: at hidden 4096, intermediate 2048, top-8 with a shared
 * expert, batches of up to about 128 tokens fit.
 *
 * All calls on one GPU share that GPU's array, so two calls that may overlap
 * on one GPU (different streams, or different host threads without ordering)
 * race: order them on one stream, or use moe_w8a8_forward with a workspace
 * each. The array keeps the last call's contents; nothing needs to start at
 * zero (every index and counter the block uses is rebuilt by each call).
 */
#define MOE_W8A8_NOALLOC_SCRATCH_BYTES (32u << 20)
MOE_W8A8_API moe_status_t moe_w8a8_forward_noalloc(const moe_w8a8_dims_t *dims,
                              const void *x,
                              const int32_t *expert_ids,
                              const float *expert_scales,
                              const int8_t *gmm1_weight,
                              const float *gmm1_weight_scale,
                              const int8_t *gmm2_weight,
                              const float *gmm2_weight_scale,
                              const int8_t *share_gmm1_weight,
                              const float *share_gmm1_weight_scale,
                              const int8_t *share_gmm2_weight,
                              const float *share_gmm2_weight_scale,
                              const float *expert_smooth_scales,
                              const float *share_smooth_scales,
                              const uint8_t *x_active_mask,
                              void *output,
                              void *share_output,
                              int32_t *expert_token_nums,
                              const moe_w8a8_debug_t *dbg,
                              void *stream);

/*
 * Re-lay int8 weights once, at load time, into the order the GEMM kernels
 * stream (the MI355X counterpart of the NZ weight format that FusedDeepMoE
 * sec. 5.3 / 8.1 feeds its cube unit). Nothing is computed; bytes move.
 *
 *  src    int8 [groups, n, k], k contiguous (a gmm*_weight tensor: n = 2I, k = H
 *         for GEMM1; n = H, k = I for GEMM2; groups = E_loc, or 1 for a shared
 *         expert)
 *  which  MOE_PACK_GMM1 for a gmm1 tensor, MOE_PACK_GMM2 for a gmm2 tensor
 *  dst    int8, same size; for group g, tile position p and 64-byte k step s,
 *         the 1024 bytes at ((g*(n/16) + p)*(k/64) + s)*1024 hold, at byte
 *         16*l + b (l in [0,64), b in [0,16)), src[g][16j + l%16][64s +
 *         16*(l/16) + b], where j = p for GEMM2 and, for GEMM1 (gate tiles
 *         j < n/32, up tiles after them), j = p/2 for even p and n/32 + p/2
 *         for odd p: gate tile j and up tile j follow each other
 *  n % 32 == 0, k % 64 == 0; src and dst 16-byte aligned and not overlapping.
 *  Stream-ordered; returns MOE_ERR_INVALID_ARG for bad sizes, pointers or
 *  `which`.
 */
enum { MOE_PACK_GMM1 = 1, MOE_PACK_GMM2 = 2 };
MOE_W8A8_API moe_status_t moe_w8a8_pack_weights(const int8_t *src, int8_t *dst, int64_t groups, int32_t n,
                                                int32_t k, int32_t which, void *stream);

/*
 * FP4 weights for weight_format == MOE_WEIGHT_MXFP4, re-laid once at load time
 * (OCP microscaling formats: E2M1 elements, E8M0 scale 2^(e-127) per block of
 * 32 consecutive k elements of a weight row).
 *
 *  data         uint8 [groups, n, k/2]: element k' of row r in the low nibble
 *               of byte k'/2 when k' is even, the high nibble when odd
 *  block_scale  uint8 [groups, n, k/32] E8M0 exponents (255 = NaN: not allowed)
 *  which        MOE_PACK_GMM1 / MOE_PACK_GMM2 as for moe_w8a8_pack_weights
 *  dst          moe_w8a8_packed_mx_bytes(groups, n, k) bytes, 16-byte aligned:
 *               first the element blocks, exactly as moe_w8a8_pack_weights lays
 *               out a [groups, n, k/2] int8 tensor (one 1024-byte block per
 *               16-row tile and 128-element k step), then the scales: for group
 *               g, tile position p and k step s, the 64 bytes at
 *               D + ((g*(n/16) + p)*(k/128) + s)*64, D = groups*n*k/2, hold at
 *               byte l (l in [0,64)) block_scale[g][16j + l%16][4s + l/16], with
 *               j the tile of position p as in moe_w8a8_pack_weights
 *  n % 32 == 0, k % 128 == 0; no buffer may overlap dst. Stream-ordered.
 */
MOE_W8A8_API moe_status_t moe_w8a8_packed_mx_bytes(int64_t groups, int32_t n, int32_t k, size_t *bytes);
MOE_W8A8_API moe_status_t moe_w8a8_pack_weights_mx(const uint8_t *data, const uint8_t *block_scale, uint8_t *dst,
                                                   int64_t groups, int32_t n, int32_t k, int32_t which,
                                                   void *stream);

/*
 * Cache warm ("DeepSeek V4 Decode Optimization" sec. 4.5, inter-layer
 * eviction): read the device range [ptr, ptr + bytes) once on `stream` and
 * discard it, so that its lines sit in the 256 MB memory-side cache (and an
 * XCD's L2) when a later kernel reads them. A hint with no destination: no
 * value anywhere changes, and dropping the call changes no result. Meant for
 * the next layer's weights that every call touches (the shared expert's),
 * issued on a second stream while the current layer runs its latency-bound
 * launches; a range larger than the cache evicts itself. ptr 16-byte aligned,
 * bytes a multiple of 16 (MOE_ERR_INVALID_ARG otherwise); bytes == 0 is a
 * no-op. Stream-ordered, no allocation.
 */
MOE_W8A8_API moe_status_t moe_w8a8_warm(const void *ptr, size_t bytes, void *stream);

/*
 * Read-bandwidth probe, for measurement only: read the device range
 * [ptr, ptr + bytes) once on `stream` over the whole chip, with the access
 * pattern of the GEMMs' weight stream (each wave loads 1 KB contiguous per
 * instruction, non-temporal, eight loads in flight), and discard the data.
 * Timing it over a range larger than the 256 MB memory-side cache gives the
 * HBM read rate this device reaches, the measured counterpart of the
 * published peak that a memory-bound kernel's roofline fraction is set
 * against. No value anywhere changes. ptr 16-byte aligned, bytes a multiple
 * of 16 (MOE_ERR_INVALID_ARG otherwise); bytes == 0 is a no-op.
 * Stream-ordered, no allocation.
 */
MOE_W8A8_API moe_status_t moe_w8a8_read_probe(const void *ptr, size_t bytes, void *stream);

/*
 * Read-and-write probe, for measurement only: the larger-batch GEMMs' weight
 * stream together with their output writes. [src, src + src_bytes) is read in
 * work items of 256 KB (one two-wave workgroup each, six resident per CU;
 * each wave reads two 64 KB tiles in 1 KB steps through a ring of eight
 * non-temporal loads per tile), and every item then writes its equal share
 * of [dst, dst + dst_bytes) with 16-byte stores, as a GEMM workgroup writes
 * its output rows after its contraction. Timing it with a GEMM's own read and
 * write byte counts gives the rate that mix reaches on the device: writes to
 * HBM while the read stream saturates it cost several times their bytes.
 * src is not changed; dst receives arbitrary values. src 16-byte aligned,
 * src_bytes a multiple of 262144 (0 is a no-op); dst_bytes a multiple of 16
 * and at most src_bytes; dst 16-byte aligned and not overlapping src when
 * dst_bytes > 0 (MOE_ERR_INVALID_ARG otherwise). Stream-ordered, no
 * allocation.
 */
MOE_W8A8_API moe_status_t moe_w8a8_read_write_probe(const void *src, size_t src_bytes, void *dst, size_t dst_bytes,
                                                    void *stream);

/*
 * moe_w8a8_forward on activations that are quantised already (by
 * moe_w8a8_norm_quant, or by a program of the caller's own): the block then
 * skips its own quantisation of x. Results are bit for bit those of
 * moe_w8a8_forward on any x whose codes and scales these are.
 *
 *  q_x      [T, H] codes: int8 (MOE_WEIGHT_INT8) or FP8 E4M3 (MOE_WEIGHT_MXFP4;
 *           moe_w8a8_norm_quant makes them with MOE_QUANT_E4M3). Bytes do not
 *           tell which they are: that is not checked
 *  x_scale  fp32 [T] (quant_mode 1) or [T, H / quant_group] (quant_mode 2);
 *           element i of token t stands for q_x[t][i] * its scale
 *
 * Both 16-byte aligned, and required unless T == 0. There are no smooth
 * scales: they multiply x before its quantisation, by expert, which codes
 * cannot express. Every other argument, and the errors, are those of
 * moe_w8a8_forward.
 */
MOE_W8A8_API moe_status_t moe_w8a8_forward_quantized(const moe_w8a8_dims_t *dims,
                              const void *q_x,
                              const float *x_scale,
                              const int32_t *expert_ids,
                              const float *expert_scales,
                              const int8_t *gmm1_weight,
                              const float *gmm1_weight_scale,
                              const int8_t *gmm2_weight,
                              const float *gmm2_weight_scale,
                              const int8_t *share_gmm1_weight,
                              const float *share_gmm1_weight_scale,
                              const int8_t *share_gmm2_weight,
                              const float *share_gmm2_weight_scale,
                              const uint8_t *x_active_mask,
                              void *output,
                              void *share_output,
                              int32_t *expert_token_nums,
                              void *workspace,
                              size_t workspace_bytes,
                              const moe_w8a8_debug_t *dbg,
                              void *stream);

/* ------------------------------------------------------------------------
 * Around the expert block: the pre-norm, the router, and the dense products
 * of the same model with 4-bit weights. The conventions at the top of this
 * file hold for them too; with num_tokens == 0 a call does nothing, whatever
 * its pointers.
 * ------------------------------------------------------------------------ */

/* Element types of the operators below. */
enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_FP16 = 1, MOE_DTYPE_FP32 = 2, MOE_DTYPE_INT8 = 3 };
/* 8-bit outputs of moe_w8a8_norm_quant. */
enum { MOE_QUANT_NONE = 0, MOE_QUANT_INT8 = 1, MOE_QUANT_E4M3 = 2 };

typedef struct {
    int32_t num_tokens;   /* T in [0, 65536]                                          */
    int32_t hidden;       /* H in [1, 16384], any size                                */
    int32_t dtype;        /* of x, residual, residual_out and y: BF16, FP16 or FP32   */
    int32_t weight_dtype; /* of weight: the same as dtype, or FP32                    */
    int32_t quant;        /* MOE_QUANT_*: what q holds                                */
    int32_t quant_group;  /* 0: one scale per row; 64, 128 or 256 (dividing H): one   */
                          /*   per row and group of that many consecutive elements    */
    float rms_eps;        /* >= 1e-30: added to the mean square                       */
    float amax_eps;       /* >= 1e-20: floor of an amax, as in moe_w8a8_dims_t        */
} moe_w8a8_norm_dims_t;

/*
 * Residual addition, root-mean-square norm and 8-bit quantisation in one pass:
 *
 *   r = x + residual                         (fp32; residual_out = r rounded)
 *   y = r * weight / sqrt(mean(r^2) + rms_eps)  (fp32; y rounded once)
 *   codes of y before its rounding, by the block's own rule: a' = max(max|y|,
 *   amax_eps), scale = a' / 127 (int8) or a' / 448 (E4M3), q = y / scale
 *   rounded to nearest even
 *
 * q and q_scale are what moe_w8a8_forward_quantized (and, one scale per row,
 * moe_w8a8_linear_w4) take. With p = r * weight, y / max|y| = p / max|p|: the
 * codes are computed from p, so they do not depend on the order in which the
 * squares are summed (rows under the amax floor apart).
 *
 *  x             [T, H]
 *  residual      [T, H] or NULL (then r = x, and residual_out must be NULL)
 *  weight        [H] or NULL (all ones)
 *  residual_out  [T, H] or NULL
 *  y             [T, H] or NULL
 *  q, q_scale    [T, H] bytes, and fp32 [T] or [T, H / quant_group]; both NULL
 *                iff quant == MOE_QUANT_NONE
 *
 * Every pointer is 16-byte aligned (q_scale: 4, but 16 where
 * moe_w8a8_forward_quantized is to take it). residual_out and y may be x
 * or residual themselves (not both the same one); any other overlap of an
 * output with anything is refused. At least one of y and q is given. A row
 * whose values are not finite, or whose squares' sum or r * weight * 448 leaves
 * fp32, is unspecified; the other rows are not affected by it.
 */
MOE_W8A8_API moe_status_t moe_w8a8_norm_quant(const moe_w8a8_norm_dims_t *dims, const void *x, const void *residual,
                                              const void *weight, void *residual_out, void *y, void *q,
                                              float *q_scale, void *stream);

/* Scores of the router. */
enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1, MOE_SCORE_SQRT_SOFTPLUS = 2 };

typedef struct {
    int32_t num_tokens;     /* T in [0, 65536]                                        */
    int32_t hidden;         /* H in [1, 16384], any size                              */
    int32_t moe_expert_num; /* E in [1, 1024]                                         */
    int32_t topk;           /* K in [1, min(16, E)]                                   */
    int32_t score;          /* MOE_SCORE_*: softmax over the experts, 1/(1+exp(-l)),  */
                            /*   or sqrt(log(1 + exp(l)))                             */
    int32_t normalize;      /* 1: a token's weights are divided by their sum          */
    int32_t dtype;          /* of x: BF16, FP16 or FP32                               */
    int32_t weight_dtype;   /* of weight: the same as dtype, or BF16 or FP32          */
    float route_scale;      /* finite: every weight is multiplied by it at the end    */
} moe_w8a8_gate_dims_t;

/*
 * The router: logits, scores and top-k choice of experts, whose results are
 * moe_w8a8_forward's expert_ids and expert_scales.
 *
 *   l[t,e] = sum_h x[t,h] * weight[e,h];  s = score(l)
 *   the K experts with the largest s + bias (of l where bias is NULL: every
 *   score rises with l), in falling order, ties to the lowest id
 *   weight of a chosen expert: s (without bias), over the chosen ones' sum if
 *   `normalize`, times route_scale; rounded once, to fp32
 *
 * The choice is that of 64-bit sums, whatever the types: it changes with the
 * order of a sum (with the batch, that is) only where two values are within
 * the last bits of such sums. The weights come from 64-bit logits too, or, in
 * large products of x and weight both BF16, both FP16, or x BF16 and weight
 * FP32 (softmax with a bias apart), from logits whose sums of 64 products are
 * in fp32.
 *
 *  x              [T, H]
 *  weight         [E, H]
 *  bias           fp32 [E] or NULL. -infinity takes an expert out
 *  expert_ids     int32 [T, K]
 *  expert_scales  fp32 [T, K]
 *  workspace      >= moe_w8a8_gate_workspace_size() bytes, 256-byte aligned
 *
 * An expert whose logit is NaN is taken as not there, by the softmax too, and
 * so is one whose logit is -infinity where bias is NULL. Where fewer than K
 * experts are left, by the bias or so, the places that remain get id -1, which
 * the block drops, and weight 0.
 * x and weight are 16-byte aligned, the others 4. The outputs overlap nothing.
 * The workspace's size does not fall as T or E grows: one that is made for the
 * largest batch serves every smaller one.
 */
MOE_W8A8_API moe_status_t moe_w8a8_gate_workspace_size(const moe_w8a8_gate_dims_t *dims, size_t *bytes);
MOE_W8A8_API moe_status_t moe_w8a8_gate(const moe_w8a8_gate_dims_t *dims, const void *x, const void *weight,
                                        const float *bias, int32_t *expert_ids, float *expert_scales,
                                        void *workspace, size_t workspace_bytes, void *stream);

typedef struct {
    int32_t num_tokens;   /* T in [0, 65536]                                          */
    int32_t out_features; /* N in [1, 2^20]; even when gated                          */
    int32_t in_features;  /* K in [1, 2^17], a multiple of group; N * K <= about 2^34 */
    int32_t group;        /* 32, 64 or 128 consecutive k share a scale                */
    int32_t act_dtype;    /* of x: BF16, FP16 or INT8                                 */
    int32_t gated;        /* 0: out [T, N]; 1: rows [0, N/2) are the gate, [N/2, N)   */
                          /*   the up projection, out [T, N/2] = silu(gate) * up      */
    int32_t has_zeros;    /* 1: zero points per row and group; 0: all of them 8       */
} moe_w8a8_linear_w4_dims_t;

/*
 * Dense product with 4-bit weights:
 *
 *   o[t,n] = x_scale[t] * sum_k x[t,k] * (code[n,k] - zero[n,k/group]) * scale[n,k/group] + bias[n]
 *
 * and out = o, or SwiGLU of its halves (gated), rounded once. A group's sum is
 * exact for INT8 x and in fp32 otherwise; groups are summed in fp32.
 *
 * The weights are re-laid once, at load time, for one (N, K, group, act_dtype
 * kind, gated, has_zeros); num_tokens may differ from call to call, and BF16
 * and FP16 share one layout.
 *
 *  codes    uint8 [N, K/2]: element k in the low nibble of byte k/2 when k is
 *           even, the high nibble when odd
 *  scale    fp32 [N, K/group]
 *  zero     uint8 [N, K/group], values 0..15; NULL iff has_zeros == 0
 *  dst      moe_w8a8_packed_w4_bytes() bytes, 16-byte aligned: 1024 bytes of
 *           codes per 16 rows and 128 k (both padded with zeros), then the
 *           scales and the zero points of those tiles in the same order. Gated:
 *           a tile holds 8 gate rows and their 8 up rows in turn
 */
MOE_W8A8_API moe_status_t moe_w8a8_packed_w4_bytes(const moe_w8a8_linear_w4_dims_t *dims, size_t *bytes);
MOE_W8A8_API moe_status_t moe_w8a8_pack_weights_w4(const moe_w8a8_linear_w4_dims_t *dims, const uint8_t *codes,
                                                   const float *scale, const uint8_t *zero, void *dst,
                                                   void *stream);
/*
 *  x        [T, K], 16-byte aligned
 *  x_scale  fp32 [T] for INT8 x, else NULL
 *  weight   from moe_w8a8_pack_weights_w4 with the same dims
 *  bias     fp32 [N] or NULL
 *  out      bf16 (BF16 and INT8 x) or fp16 (FP16 x) [T, N] or [T, N/2],
 *           16-byte aligned, overlapping nothing
 *
 * x is taken to be finite, and below 2^100 in magnitude; a token's outputs
 * depend on no other token's row. No workspace.
 */
MOE_W8A8_API moe_status_t moe_w8a8_linear_w4(const moe_w8a8_linear_w4_dims_t *dims, const void *x,
                                             const float *x_scale, const void *weight, const float *bias, void *out,
                                             void *stream);

/* ------------------------------------------------------------------------
 * Between the block and the rest of a W8A8 program: dense products of the
 * same model in 8-bit integers, the quantiser of an activation that comes
 * from no norm, the norm that joins the block's outputs to the residual
 * stream, and tokens sorted by expert (for other ranks' experts, or for a
 * program's own) and back. The conventions at the top of this file hold; with
 * num_tokens == 0 a call does nothing, whatever its pointers, but that
 * moe_w8a8_dispatch writes its counts and offsets, and moe_w8a8_combine_grad
 * zeros to drows.
 * ------------------------------------------------------------------------ */

typedef struct {
    int32_t num_tokens;   /* T in [0, 65536]                                          */
    int32_t out_features; /* N in [1, 2^20]; even when gated                          */
    int32_t in_features;  /* K in [1, 65536], any size; N * K <= about 2^34           */
    int32_t out_dtype;    /* of out: BF16, FP16 or FP32                               */
    int32_t gated;        /* 0: out [T, N]; 1: rows [0, N/2) are the gate, [N/2, N)   */
                          /*   the up projection, out [T, N/2] = silu(gate) * up      */
} moe_w8a8_linear_w8_dims_t;

/*
 * Dense product in 8-bit integers, the block's GEMM rule for one weight:
 *
 *   acc[t,n] = sum_k x[t,k] * codes[n,k]          (exact, int32)
 *   o[t,n]   = (float(acc) * scale[n]) * x_scale[t] + bias[n]   (fp32)
 *
 * and out = o, or SwiGLU of its halves (gated), rounded once. x and x_scale
 * are what moe_w8a8_norm_quant, moe_w8a8_join_norm and moe_w8a8_quant write
 * with one scale per row. A token's outputs are the same bits in every batch.
 *
 * The weights are re-laid once, at load time, for one (N, K, gated);
 * num_tokens and out_dtype may differ from call to call.
 *
 *  codes    int8 [N, K]
 *  scale    fp32 [N]
 *  dst      moe_w8a8_packed_w8_bytes() bytes, 16-byte aligned: for each 16
 *           rows and 64 k (rows padded to a multiple of 16, k to one of 128,
 *           with zeros) 1024 bytes, byte 16*l + b (l in [0,64), b in [0,16))
 *           holding row l % 16, k 16*(l/16) + b; then the rows' scales in the
 *           same order. Gated: a tile holds 8 gate rows and their 8 up rows
 *           in turn
 */
MOE_W8A8_API moe_status_t moe_w8a8_packed_w8_bytes(const moe_w8a8_linear_w8_dims_t *dims, size_t *bytes);
MOE_W8A8_API moe_status_t moe_w8a8_pack_weights_w8(const moe_w8a8_linear_w8_dims_t *dims, const int8_t *codes,
                                                   const float *scale, void *dst, void *stream);
/*
 *  x        int8 [T, K], 16-byte aligned
 *  x_scale  fp32 [T]
 *  weight   from moe_w8a8_pack_weights_w8 with the same dims
 *  bias     fp32 [N] or NULL
 *  out      [T, N] or [T, N/2], 16-byte aligned, overlapping nothing
 */
MOE_W8A8_API moe_status_t moe_w8a8_linear_w8(const moe_w8a8_linear_w8_dims_t *dims, const int8_t *x,
                                             const float *x_scale, const void *weight, const float *bias, void *out,
                                             void *stream);

typedef struct {
    int32_t num_tokens;   /* T in [0, 65536]                                          */
    int32_t hidden;       /* H in [1, 16384], any size                                */
    int32_t dtype;        /* of x: BF16, FP16 or FP32                                 */
    int32_t quant;        /* MOE_QUANT_INT8 or MOE_QUANT_E4M3                         */
    int32_t quant_group;  /* 0: one scale per row; 64, 128 or 256 (dividing H): one   */
                          /*   per row and group of that many consecutive elements    */
    float amax_eps;       /* >= 1e-20: floor of an amax, as in moe_w8a8_dims_t        */
} moe_w8a8_quant_dims_t;

/*
 * The block's quantiser for any activation: v = x * smooth (fp32), a' =
 * max(max|v|, amax_eps) over the row or group, scale = a' / 127 (int8) or
 * a' / 448 (E4M3), q = v / scale rounded to nearest even.
 *
 *  x        [T, H]
 *  smooth   fp32 [H] or NULL (all ones)
 *  q        [T, H] bytes
 *  q_scale  fp32 [T] or [T, H / quant_group]
 *
 * x, smooth and q are 16-byte aligned, q_scale 4; the outputs overlap nothing.
 * A row whose values are not finite, or leave fp32 when multiplied by 448, is
 * unspecified; the other rows are not affected by it.
 */
MOE_W8A8_API moe_status_t moe_w8a8_quant(const moe_w8a8_quant_dims_t *dims, const void *x, const float *smooth, void *q,
                                         float *q_scale, void *stream);

typedef struct {
    int32_t num_tokens;   /* T in [0, 65536]                                          */
    int32_t hidden;       /* H in [1, 16384], any size                                */
    int32_t dtype;        /* of block, share, residual, residual_out and y: BF16,     */
                          /*   FP16 or FP32                                           */
    int32_t weight_dtype; /* of post_weight, gate and weight: the same as dtype, or   */
                          /*   FP32                                                   */
    int32_t post_norm;    /* 1: the block's output is normed before it is added       */
    int32_t gate_rows;    /* rows of gate: 0 (none), 1, or T                          */
    int32_t quant;        /* MOE_QUANT_*: what q holds                                */
    int32_t quant_group;  /* as in moe_w8a8_norm_dims_t                               */
    float residual_scale; /* finite                                                   */
    float branch_scale;   /* finite                                                   */
    float post_eps;       /* >= 1e-30: added to the block's mean square               */
    float rms_eps;        /* >= 1e-30: added to the stream's mean square              */
    float amax_eps;       /* >= 1e-20                                                 */
} moe_w8a8_join_norm_dims_t;

/*
 * What stands between the block's outputs and the next layer, in one pass:
 *
 *   b = block + share * share_scale[t]
 *   n = (b * post_weight) / sqrt(mean(b^2) + post_eps)     (post_norm; else b)
 *   r = residual * residual_scale + n * (gate * branch_scale)
 *   residual_out = r rounded
 *   y and the codes: those of moe_w8a8_norm_quant's norm of r (before its
 *   rounding) by weight
 *
 * fp32 operations in this order, each rounded by itself; mean(b^2), and
 * mean(r^2) here, are summed in fp64 and 1 / sqrt(...) is rounded once. So no
 * output depends on the order of a sum: a token's are the same bits in every
 * batch.
 *
 *  block         [T, H]
 *  share         [T, H] or NULL; share_scale fp32 [T] or NULL (all ones; NULL
 *                without share)
 *  residual      [T, H] or NULL (zeros)
 *  post_weight   [H] or NULL (all ones; NULL without post_norm)
 *  gate          [H] or [T, H] as gate_rows says; NULL iff gate_rows == 0 (ones)
 *  weight        [H] or NULL (all ones)
 *  residual_out  [T, H] or NULL
 *  y             [T, H] or NULL
 *  q, q_scale    as in moe_w8a8_norm_quant
 *
 * Every pointer is 16-byte aligned (share_scale 4; q_scale 4, but 16 where
 * moe_w8a8_forward_quantized is to take it). residual_out and y may be block,
 * share or residual themselves (not both the same one); any other overlap of
 * an output with anything is refused. At least one of residual_out, y and q is
 * given. A row whose values are not finite, or leave fp32 in their squares'
 * sum or multiplied by 448, is unspecified; the other rows are not affected.
 */
MOE_W8A8_API moe_status_t moe_w8a8_join_norm(const moe_w8a8_join_norm_dims_t *dims, const void *block,
                                             const void *share, const float *share_scale, const void *residual,
                                             const void *post_weight, const void *gate, const void *weight,
                                             void *residual_out, void *y, void *q, float *q_scale, void *stream);

typedef struct {
    int32_t num_tokens;     /* T in [0, 65536]                                        */
    int32_t topk;           /* K in [1, 16]                                           */
    int32_t moe_expert_num; /* E in [1, 1024]                                         */
    int32_t hidden;         /* H in [1, 16384], any size                              */
    int32_t dtype;          /* of x and rows: BF16, FP16, FP32, or INT8 (any 8-bit    */
                            /*   codes: bytes are moved)                              */
    int32_t scale_groups;   /* fp32 scales of a row of x, in [0, 256]                 */
    int32_t row_align;      /* 1, 2, 4, ... 256: an expert's rows begin at a multiple */
} moe_w8a8_dispatch_dims_t;

/*
 * Tokens sorted by expert. Pair (t, k) is kept where expert_ids[t,k] lies in
 * [0, E) and token t is active; an expert's pairs get consecutive rows in the
 * order of (t, k), beginning at the next multiple of row_align:
 *
 *   expert_token_nums[e] = kept pairs of expert e
 *   expert_offset[e] = its first row; expert_offset[E]: behind the last one,
 *                rounded up to row_align too
 *   row_of_pair[t,k] = the pair's row, -1 if it is dropped
 *   pair_of_row[r] = the row's pair t*K + k, -1 where a row has none
 *   rows[r] = x[t], row_scale[r] = x_scale[t]: zeros in the rows that fill an
 *                expert's last row_align, left as they were behind
 *                expert_offset[E]
 *
 * Ids follow moe_w8a8_gate (-1: none). Rows of one expert can be sent to its
 * rank as they are, and a rank's rows run through moe_w8a8_forward_quantized
 * with topk 1.
 *
 *  expert_ids         int32 [T, K]
 *  x, rows            [T, H] and [R, H] with R from moe_w8a8_dispatch_rows (the
 *                     most that T*K pairs can need); both NULL: maps only
 *  x_scale, row_scale fp32 [T, scale_groups], [R, scale_groups]; NULL iff
 *                     scale_groups == 0 or rows is NULL
 *  x_active_mask      uint8 [T] (0 / non-0) or NULL = every token active
 *  expert_token_nums  int32 [E];  expert_offset  int32 [E + 1]
 *  row_of_pair        int32 [T, K];  pair_of_row  int32 [R]
 *  workspace          >= moe_w8a8_dispatch_workspace_size() bytes (0 for small
 *                     batches: then NULL will do), 256-byte aligned. The size
 *                     does not fall as T or E grows
 *
 * x and rows are 16-byte aligned, the others 4. The outputs overlap nothing.
 */
MOE_W8A8_API moe_status_t moe_w8a8_dispatch_rows(const moe_w8a8_dispatch_dims_t *dims, int64_t *rows);
MOE_W8A8_API moe_status_t moe_w8a8_dispatch_workspace_size(const moe_w8a8_dispatch_dims_t *dims, size_t *bytes);
MOE_W8A8_API moe_status_t moe_w8a8_dispatch(const moe_w8a8_dispatch_dims_t *dims, const int32_t *expert_ids,
                                            const void *x, const float *x_scale, const uint8_t *x_active_mask,
                                            void *rows, float *row_scale, int32_t *expert_token_nums,
                                            int32_t *expert_offset, int32_t *row_of_pair, int32_t *pair_of_row,
                                            void *workspace, size_t workspace_bytes, void *stream);

typedef struct {
    int32_t num_tokens;   /* T in [0, 65536]                                          */
    int32_t topk;         /* K in [1, 16]                                             */
    int32_t hidden;       /* H in [1, 16384], any size                                */
    int32_t num_rows;     /* R in [0, 2^22] rows                                      */
    int32_t dtype;        /* of rows and drows: BF16, FP16 or FP32                    */
    int32_t out_dtype;    /* of out, addend and dout: the same as dtype, or FP32      */
} moe_w8a8_combine_dims_t;

/*
 * Sorted rows back to their tokens:
 *
 *   out[t] = sum over k (ascending, fp32, from +0) of rows[row_of_pair[t,k]] *
 *            expert_scales[t,k], + addend[t]; rounded once
 *
 * Pairs whose row lies outside [0, R) add nothing. With bf16 rows this is the
 * block's own combine, bit for bit. Without expert_scales it is the gradient
 * of moe_w8a8_dispatch: rows = the gradient of its rows, out = that of x.
 *
 *  rows           [R, H]
 *  row_of_pair    int32 [T, K]
 *  expert_scales  fp32 [T, K] or NULL (all ones: no product is formed)
 *  addend         [T, H] or NULL; may be out itself
 *  out            [T, H], overlapping nothing else
 *
 * rows, addend and out are 16-byte aligned, the others 4.
 */
MOE_W8A8_API moe_status_t moe_w8a8_combine(const moe_w8a8_combine_dims_t *dims, const void *rows,
                                           const int32_t *row_of_pair, const float *expert_scales, const void *addend,
                                           void *out, void *stream);
/*
 * Its gradient, given that of out (which is that of addend, too):
 *
 *   drows[r] = dout[t] * expert_scales[t,k] (fp32, then rounded to dtype) for
 *              the pair (t, k) of row r; zeros in rows without one
 *   dscales[t,k] = sum over h (fp32) of rows[row_of_pair[t,k]][h] * dout[t][h],
 *              0 for a dropped pair
 *
 * The two maps are those that moe_w8a8_dispatch wrote, each the other's
 * inverse; a pair whose row is not the pair's by pair_of_row is taken as
 * dropped, so that no row is written twice.
 *
 *  dout           [T, H]
 *  row_of_pair    int32 [T, K];  pair_of_row  int32 [R]
 *  rows           [R, H]; NULL iff dscales is
 *  expert_scales  fp32 [T, K] or NULL (all ones)
 *  drows          [R, H] or NULL, overlapping nothing
 *  dscales        fp32 [T, K] or NULL, overlapping nothing; one of the two is
 *                 given
 */
MOE_W8A8_API moe_status_t moe_w8a8_combine_grad(const moe_w8a8_combine_dims_t *dims, const void *dout,
                                                const int32_t *row_of_pair, const int32_t *pair_of_row,
                                                const void *rows, const float *expert_scales, void *drows,
                                                float *dscales, void *stream);

/* Static description of a status code. Never NULL. */
MOE_W8A8_API const char *moe_w8a8_status_string(moe_status_t status);

#ifdef __cplusplus
}
#endif
#endif /* MOE_W8A8_H */
