/*
 * pq2.h -- C ABI of the GB300 (sm_103a) PQ2_0 ternary-weight matmul library.
 *
 * The operation, as the pages define it:
 *   [P1] "Making a ternary reasoning model fast in vLLM", page "From CUDA to
 *        Triton and Gluon";
 *   [P2] the same series, page "Chasing llama.cpp at batch one".
 *
 *   y[m,n] = sum_g (dot(codes[n,g], q[m,g]) - sum(q[m,g])) * S[m,g] * WS[n,g]
 *
 * Weights are 2-bit codes 0,1,2 standing for -1,0,+1, four to a byte, with
 * one fp16 scale per 128 weights ([P1] "One token at a time": the PQ2_0 code
 * and the per-group scale).  Activations are quantised to int8 per 128 values
 * and stored in plane order, so the activation of weight 4*byte+s sits at
 * position s*32+byte of its group; plane s of a 32-bit code word,
 * (w >> 2s) & 0x03030303, then lines up with four consecutive activation
 * bytes, and the -1 offset is one subtraction of sum(q) per group (same
 * section).
 *
 * Notation and layouts (all row-major, all buffers owned by the caller):
 *   M tokens, K inputs (K % 128 == 0), N outputs, G = K / 128.
 *   x      fp16  [M, K]      activations
 *   qp     int8  [M, K]      quantised activations, plane order: the value of
 *                            natural index k is at g*128 + (k&3)*32 + ((k&127)>>2)
 *   S      fp32  [M, G]      activation scale per group
 *   T      int32 [M, G]      sum of the group's int8 values
 *   codes  uint8 [N, K/4]    weight k of row n in byte n*K/4 + (k>>2), bits 2*(k&3)
 *   WS     fp16  [N, G]      weight scale per group
 *   y      fp32  [M, N]      output (fully overwritten, never accumulated into)
 *
 * Conventions shared by every entry point:
 *   - Pointers are device pointers unless stated, 16-byte aligned
 *     (PQ2_ERR_MISALIGNED otherwise); sizes are element counts.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Work is enqueued asynchronously on it; nothing here
 *     synchronises, except pq2_last_device_error.
 *   - The library allocates and frees no memory.  Scratch space, where an
 *     operation needs it, is passed in as `workspace` / `workspace_bytes`
 *     (size from pq2_workspace_bytes).
 *   - Arguments are checked on the host before any launch; on error nothing
 *     is enqueued and the status says why.  A failed launch returns
 *     PQ2_ERR_CUDA.  Device faults surface at the caller's next
 *     synchronisation, as for any CUDA call.
 *   - Results are deterministic: the same inputs give bit-identical outputs
 *     (fixed-order reductions, no atomics on data).
 *   - NaN or Inf in x is not checked; the result is then undefined.
 *   - Kernels wait on on-chip barriers with a bounded spin; a wait that runs
 *     out sets a device error word that pq2_last_device_error reports as
 *     PQ2_ERR_TIMEOUT.
 */
#ifndef PQ2_H
#define PQ2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pq2_status {
    PQ2_OK = 0,
    PQ2_ERR_INVALID_ARG = 1,       /* null pointer, negative size, bad op  */
    PQ2_ERR_UNSUPPORTED_SHAPE = 2, /* K % 128 != 0, M out of range, ...    */
    PQ2_ERR_MISALIGNED = 3,        /* a pointer is not 16-byte aligned      */
    PQ2_ERR_CUDA = 4,              /* a CUDA runtime call or launch failed  */
    PQ2_ERR_TIMEOUT = 5,           /* a kernel's bounded wait ran out       */
    PQ2_ERR_WORKSPACE = 6,         /* workspace missing or too small        */
    PQ2_ERR_BOUNDS = 7             /* bounds-checked build: a kernel skipped
                                      a store outside its buffer            */
} pq2_status;

/* Operation selectors for pq2_workspace_bytes and pq2_group_dots. */
enum {
    PQ2_OP_GEMV = 0,     /* pq2_gemv            (M == 1)            */
    PQ2_OP_SMALL = 1,    /* pq2_gemm_small      (2 <= M <= 16)      */
    PQ2_OP_PREFILL = 2,  /* pq2_gemm_prefill    (M >= 1)            */
    PQ2_OP_MATMUL = 3,   /* pq2_matmul          (M >= 1, from fp16) */
    PQ2_OP_SWIGLU_DOWN = 4 /* pq2_mlp_down_swiglu (M >= 1; K = I)     */
};

/* Largest K any entry point accepts (G <= 2048 groups). */
#define PQ2_MAX_K 262144

/* Static text for a status code; never NULL. */
const char* pq2_status_string(int status);

/* Library version string, e.g. "pq2-gb300 0.1 sm_103a". */
const char* pq2_version(void);

/*
 * pq2_quantize_act -- fused activation quantisation and plane reorder.
 *   [P1] "Prompt processing": the quantize kernel writes q [m,k] int8,
 *   s [m,G] fp32 and t [m,G] int32 per 128-value group; [P1] "One token at
 *   a time": q is stored in plane order.
 * Per (m, g): amax = max |x|; d = amax / 127 (fp32, round to nearest even);
 * q = round-half-even(x / d) clamped to [-127, 127]; S = d; T = sum q.  A
 * group of zeros gives d = 0, q = 0, T = 0.  (The pages fix the outputs but
 * not the scale formula; this is the plain symmetric reading.)
 *   x_f16  in   fp16 [M, K]
 *   qp     out  int8 [M, K] plane order
 *   S, T   out  fp32 / int32 [M, G]
 * M >= 0 (M == 0 enqueues nothing), 1 <= K <= PQ2_MAX_K, K % 128 == 0.
 */
pq2_status pq2_quantize_act(const void* x_f16, int64_t M, int64_t K,
                            int8_t* qp, float* S, int32_t* T, void* stream);

/*
 * pq2_quantize_swiglu -- the activation between the two projections of a
 * decode MLP, fused with the quantisation of pq2_quantize_act.  The pages
 * link the MLP's gate/up and down projections ([P1] "Choose the
 * configuration with the proxy": replayed gate -> down pairs) but do not
 * define the activation; this is the plain SwiGLU reading:
 *   gate = gu[m, 0..I), up = gu[m, I..2I);  h = silu(gate) * up,
 *   silu(g) = g / (1 + exp(-g)),
 * every step one fp32 operation with round-to-nearest, exp computed by Cody
 * and Waite's argument reduction and a degree-7 Taylor polynomial (a fixed
 * sequence of fused multiply-adds, so a CPU restatement gets the same bits);
 * h is rounded to fp16, saturating at +-65504, then quantised exactly as
 * pq2_quantize_act quantises x.
 *   gu     in   fp32 [M, 2I]  (typically the y of the gate/up projection)
 *   qp     out  int8 [M, I] plane order
 *   S, T   out  fp32 / int32 [M, I/128]
 * M >= 0 (M == 0 enqueues nothing), 1 <= I <= PQ2_MAX_K, I % 128 == 0.
 * NaN or Inf in gu: the result is undefined.
 */
pq2_status pq2_quantize_swiglu(const float* gu, int64_t M, int64_t I,
                               int8_t* qp, float* S, int32_t* T, void* stream);

/*
 * pq2_pack_weights -- the "prepared" weight planes: ternary values to codes.
 *   [P1] "One token at a time": codes 0,1,2 for -1,0,+1, four to a byte,
 *   weight 4*byte+s in bits 2s; [P1] "A power proxy for the rest of the
 *   model": prepared weights carry the scales as a separate plane.
 *   tern    in   int8 [N, K], every value in {-1, 0, +1}
 *   ws_f16  in   fp16 [N, G]  (may be NULL together with ws_out)
 *   codes   out  uint8 [N, K/4]
 *   ws_out  out  fp16 [N, G]  copy of ws_f16 (may alias ws_f16)
 * A value outside {-1,0,1} is stored as code 3 (read as +2 by the matmul
 * kernels) and sets the device error word; the host cannot see it without a
 * synchronisation, so validate ternary inputs before packing.
 */
pq2_status pq2_pack_weights(const int8_t* tern, const void* ws_f16, int64_t N, int64_t K,
                            uint8_t* codes, void* ws_out, void* stream);

/*
 * pq2_gemv -- the M = 1 decode matmul y[n] for all n.
 *   [P1] "One token at a time: plain Triton is enough" (plane extraction
 *   with (w >> 2s) & 0x03030303 feeding DP4A, the per-group sum(q)
 *   subtraction, fp32 accumulation of dot * s * ws); [P2] "The win: a program
 *   just for one token" (no token dimension, separate scale plane).
 *   qp [1,K], S [1,G], T [1,G], codes [N,K/4], ws_f16 [N,G] in; y [1,N] out.
 * N >= 1, 128 <= K <= PQ2_MAX_K, K % 128 == 0.
 */
pq2_status pq2_gemv(const int8_t* qp, const float* S, const int32_t* T,
                    const uint8_t* codes, const void* ws_f16, float* y,
                    int64_t N, int64_t K, void* stream);

/*
 * pq2_gemm_small -- small batches, 2 <= M <= 16 token rows.
 *   [P1] "Small batches: make the register layout explicit", "Use a ring
 *   buffer for longer rows", "Extend the kernels to sixteen token rows";
 *   split-K partial sums, where used, are reduced in the fixed order
 *   0,1,2,... ([P1] "Choose the configuration with the proxy").
 *   Same operands as pq2_gemv with M rows; y [M,N].
 *   workspace: device scratch of pq2_workspace_bytes(PQ2_OP_SMALL, M, N, K)
 *   bytes (may be NULL when that is 0).
 *   2 to 4 token rows run on DP4A, each code word shared by the rows, where
 *   a CTA's group terms fit its shared memory (the workspace is then not
 *   touched; each row's y equals pq2_gemv on that row, bit for bit); larger
 *   M on the tensor cores.
 */
pq2_status pq2_gemm_small(const int8_t* qp, const float* S, const int32_t* T,
                          const uint8_t* codes, const void* ws_f16, float* y,
                          int64_t M, int64_t N, int64_t K,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * pq2_gemm_small_ex -- pq2_gemm_small with a flags word: 0, or
 *   PQ2_WEIGHTS_STATIC (defined below, as for pq2_matmul_ex): the caller
 *   promises that codes and ws_f16 are not written by any operation enqueued
 *   on `stream` before this call that may still be running when it starts.
 *   The DP4A kernel for 2 to 4 token rows then requests its weights (an L2
 *   prefetch of its slice and its first rows) before the preceding kernel
 *   has finished; qp, S and T are still read only after it.  y is
 *   bit-identical to pq2_gemm_small.  Other bits give PQ2_ERR_INVALID_ARG;
 *   the tensor-core path ignores the flag.
 */
pq2_status pq2_gemm_small_ex(const int8_t* qp, const float* S, const int32_t* T,
                             const uint8_t* codes, const void* ws_f16, float* y, int64_t M,
                             int64_t N, int64_t K, uint32_t flags, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * pq2_gemm_prefill -- prompt processing, any M >= 1 (built for M > 16).
 *   [P1] "Prompt processing: check configuration and launch costs" (2-D
 *   output tiles, per-group integer products and the same per-group
 *   dequantise-accumulate order as the M = 1 path).
 *   Same operands as pq2_gemm_small; y [M,N].
 *   workspace: pq2_workspace_bytes(PQ2_OP_PREFILL, M, N, K) bytes; for
 *   shapes the 128 x 256 tile kernel may take (at least 8 tiles of 128
 *   tokens, M > 896, and at least 128 tiles of 128 x 256) it includes the
 *   weights expanded to one byte per weight (N*K bytes), written once per
 *   call.
 */
pq2_status pq2_gemm_prefill(const int8_t* qp, const float* S, const int32_t* T,
                            const uint8_t* codes, const void* ws_f16, float* y,
                            int64_t M, int64_t N, int64_t K,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * pq2_matmul -- the whole path from fp16 activations: pq2_quantize_act, then
 * pq2_gemv (M == 1), pq2_gemm_small (M <= 16) or pq2_gemm_prefill.  The
 * pages' routing by token count ([P1] "Defaults and switches").
 *   x_f16 [M,K] fp16, codes, ws_f16 in; y [M,N] fp32 out.
 *   workspace: pq2_workspace_bytes(PQ2_OP_MATMUL, M, N, K) bytes (holds the
 *   quantised activations plus the chosen kernel's own scratch).  For M == 1
 *   and K <= 32768 the GEMV kernel quantises x itself (one launch) and no
 *   workspace is needed (size 0, workspace may be NULL).
 */
pq2_status pq2_matmul(const void* x_f16, const uint8_t* codes, const void* ws_f16, float* y,
                      int64_t M, int64_t N, int64_t K,
                      void* workspace, size_t workspace_bytes, void* stream);

/* Flags of pq2_matmul_ex. */
#define PQ2_WEIGHTS_STATIC 1u

/*
 * pq2_matmul_ex -- pq2_matmul with flags.  (The pages have no counterpart to
 * the flag; it lets a decode loop overlap one call's weight stream with the
 * preceding call's arithmetic.)
 *   flags: 0 or PQ2_WEIGHTS_STATIC; other bits give PQ2_ERR_INVALID_ARG.
 *   PQ2_WEIGHTS_STATIC: the caller promises that codes and ws_f16 are not
 *     written by any operation enqueued on `stream` before this call that may
 *     still be running when it starts (typically: weights packed or copied
 *     once, then many calls).  The M == 1 fused kernel and the DP4A kernel
 *     for a few tokens (2 <= M <= 4 where the shape allows) may then read
 *     them before the preceding kernel on the stream has finished
 *     (programmatic dependent launch).  x_f16 is still read only after that
 *     kernel is done.  If the promise is broken, y is undefined.  Results
 *     are bit-identical to pq2_matmul.  The other paths ignore the flag.
 *   Other arguments, workspace and errors as pq2_matmul.
 */
pq2_status pq2_matmul_ex(const void* x_f16, const uint8_t* codes, const void* ws_f16, float* y,
                         int64_t M, int64_t N, int64_t K, uint32_t flags,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * pq2_mlp_down_swiglu -- the down projection of a decode MLP from its gate/up
 * output: pq2_quantize_swiglu, then pq2_gemv (M == 1), pq2_gemm_small
 * (M <= 16) or pq2_gemm_prefill, as pq2_matmul routes.
 *   gu [M, 2I] fp32 in; codes [N, I/4], ws_f16 [N, I/128] in; y [M, N] fp32 out.
 *   workspace: pq2_workspace_bytes(PQ2_OP_SWIGLU_DOWN, M, N, I) bytes (the
 *   quantised h plus the matmul's own scratch); never 0.
 * Errors as pq2_matmul.
 */
pq2_status pq2_mlp_down_swiglu(const float* gu, const uint8_t* codes, const void* ws_f16, float* y,
                               int64_t M, int64_t N, int64_t I,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * pq2_gemm_bf16_splitk -- the small unquantised projection of a decode step
 * ([P1] "Speed up a small unquantised projection": in_proj_ba, N = 96,
 * K = 5120, a few tokens at a time): y = bf16(x . w^T), computed as a
 * split-K GEMM whose fp32 partial sums are added in a fixed order, so the
 * same inputs give the same bits on every call.
 *   x [M, K] bf16 in, w [N, K] bf16 in, y [M, N] bf16 out; bf16 values are
 *   passed as their 16-bit patterns, rows contiguous.  Products and sums in
 *   fp32, one rounding of each output to bf16 (nearest, ties to even).
 *   M >= 0 and N >= 0 (either 0 enqueues nothing), 0 <= K <= PQ2_MAX_K
 *   (K == 0 writes zeros; x and w may then be null), K % 8 == 0, M <= PQ2_MAX_M_BF16,
 *   N <= PQ2_MAX_N_BF16: PQ2_ERR_UNSUPPORTED_SHAPE otherwise.  x and w
 *   16-byte aligned, y 2-byte aligned: PQ2_ERR_MISALIGNED otherwise.
 *   flags: 0 or PQ2_WEIGHTS_STATIC (w may be read before the preceding
 *   kernel on the stream has finished); other bits: PQ2_ERR_INVALID_ARG.
 *   One launch, no workspace.  Built for M <= 16; a larger M runs as
 *   independent 16-token tiles that each read w again.
 */
#define PQ2_MAX_M_BF16 1048560
#define PQ2_MAX_N_BF16 1073741824
pq2_status pq2_gemm_bf16_splitk(const uint16_t* x, const uint16_t* w, uint16_t* y, int64_t M,
                                int64_t N, int64_t K, uint32_t flags, void* stream);

/*
 * The steps around a projection (the pages time the projections alone; these
 * are what a serving step over several requests runs between them).
 */

/* Element types of the arrays below. */
#define PQ2_F32 0
#define PQ2_F16 1
#define PQ2_BF16 2

/* Flags of pq2_rmsnorm and pq2_norm_residual (PQ2_WEIGHTS_STATIC, the norm
 * weights w, w_post and w_next and never the gate, may be added). */
#define PQ2_NORM_UNIT_OFFSET 2u /* weights are stored as w - 1                  */
#define PQ2_NORM_NO_POST 4u     /* the block's output is not normed             */
#define PQ2_GATE_SIGMOID 8u     /* the gate enters as sigmoid(gate)             */
#define PQ2_GATE_SILU 16u       /* the gate enters as gate * sigmoid(gate)      */

/* Widest row of the two norms. */
#define PQ2_NORM_MAX_H 49152

/*
 * pq2_rmsnorm -- the norm before a block:
 *   x[m] = r[m] / sqrt(mean(r[m]^2) + eps) * w
 * in fp32, rounded once (nearest even; values past fp16's range become inf)
 * to x's type -- fp16 is what pq2_matmul takes, bf16 what
 * pq2_gemm_bf16_splitk takes.
 *   r in [M, H] (r_type, row stride ld_r >= H elements), w in [H] (w_type) or
 *   NULL (1), x out [M, H] (x_type, ld_x >= H).  x may be r where their types
 *   and strides are the same (PQ2_ERR_INVALID_ARG otherwise).
 * M >= 0 (M == 0 enqueues nothing), 1 <= H <= PQ2_NORM_MAX_H, eps >= 0.
 * Pointers need their element's alignment only (PQ2_ERR_MISALIGNED
 * otherwise); rows on 16-byte boundaries with H % 8 == 0 take the vector path.
 */
pq2_status pq2_rmsnorm(const void* r, int r_type, int64_t ld_r, const void* w, int w_type, void* x,
                       int x_type, int64_t ld_x, int64_t M, int64_t H, float eps, uint32_t flags,
                       void* stream);

/*
 * pq2_norm_residual -- the end of a block, and the norm before the next one,
 * in one pass:
 *   n    = y / sqrt(mean(y^2) + eps) * w_post      (n = y * w_post with NO_POST)
 *   r'   = r + alpha * act(gate) * n               (gate absent: 1)
 *   x    = r' / sqrt(mean(r'^2) + eps) * w_next    (from r' before rounding)
 * per row, in fp32; r' and x are rounded once.  A struct, for its many
 * optional parts; every pointer is a device pointer.
 *   y       in   [M, H] the block's output (fp32 from pq2_matmul)
 *   r       in   [M, H] residual stream
 *   r_out   out  [M, H] of r's type; may be r, with the same row stride
 *   w_post  in   [H] or NULL (1)
 *   gate    in   [M, H] with row stride ld_gate >= H, or one vector [H] for
 *                all rows (ld_gate == 0), or NULL
 *   w_next  in   [H] or NULL (1)
 *   x       out  [M, H] the next block's input, or NULL (not computed)
 * Other rules as pq2_rmsnorm.  Nothing but r_out and r may overlap.
 */
typedef struct pq2_norm_residual_args {
    const void* y;
    const void* r;
    void* r_out;
    const void* w_post;
    const void* gate;
    const void* w_next;
    void* x;
    int64_t ld_y, ld_r, ld_r_out, ld_gate, ld_x; /* row strides, elements */
    int32_t y_type, r_type, w_type, gate_type, x_type;
    float eps, alpha;
    uint32_t flags;
} pq2_norm_residual_args;
pq2_status pq2_norm_residual(const pq2_norm_residual_args* args, int64_t M, int64_t H,
                             void* stream);

/*
 * pq2_lora_add -- low-rank adapters of many requests beside a shared
 * projection: for every token m with adapter l = ids[m] >= 0
 *   y_out[m] = y_in[m] + scales[l] * B[l] (A[l] x[m])
 * and y_out[m] = y_in[m] for ids[m] < 0.  Products and sums in fp32 or
 * better; the rank-sized intermediate is never rounded to fewer than 22 bits
 * of its largest value.
 *   x       in   [M, K] (type: PQ2_F16 or PQ2_BF16; row stride ld_x >= K)
 *   A       in   [L, R, K], B in [L, N, R], both of x's type
 *   ids     in   int32 [M].  A value >= L counts as no adapter and sets the
 *                device error word (PQ2_ERR_INVALID_ARG from
 *                pq2_last_device_error).
 *   ranks   in   int32 [L] or NULL (all R): rows of A (columns of B) in use,
 *                0 <= rank <= R; the others may hold anything
 *   scales  in   fp32 [L] or NULL (1)
 *   y_in, y_out  [M, N] (y_type: PQ2_F32 or PQ2_BF16; row strides ld_in,
 *                ld_out >= N); the same array, or arrays that do not overlap
 *   workspace    pq2_lora_workspace_bytes(M, N, K, L, R) bytes; enough for any
 *                smaller M too
 * M >= 0 and N >= 0 (either 0 enqueues nothing), 8 <= K <= PQ2_MAX_K with
 * K % 8 == 0, 8 <= R <= PQ2_LORA_MAX_R with R % 8 == 0,
 * 1 <= L <= PQ2_LORA_MAX_L, M <= PQ2_LORA_MAX_M.  x, A, B and workspace
 * 16-byte aligned and ld_x % 8 == 0; y_in and y_out aligned to their element.
 * NaN or Inf in x, or in the ranks in use: that token's y is undefined.
 */
#define PQ2_LORA_MAX_R 256
#define PQ2_LORA_MAX_L 16384
#define PQ2_LORA_MAX_M 1048576
size_t pq2_lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R);
pq2_status pq2_lora_add(const void* x, int64_t ld_x, const void* A, const void* B, int type,
                        const int32_t* ids, const int32_t* ranks, const float* scales,
                        const void* y_in, int64_t ld_in, void* y_out, int64_t ld_out, int y_type,
                        int64_t M, int64_t N, int64_t K, int64_t L, int64_t R, void* workspace,
                        size_t workspace_bytes, void* stream);
/* The same with the arguments in one struct, for bindings that convert them
 * one by one. */
typedef struct {
    const void *x, *A, *B;
    const int32_t *ids, *ranks;
    const float* scales;
    const void* y_in;
    void *y_out, *workspace;
    int64_t ld_x, ld_in, ld_out, M, N, K, L, R;
    size_t workspace_bytes;
    int32_t type, y_type;
} pq2_lora_add_args;
pq2_status pq2_lora_add_packed(const pq2_lora_add_args* args, void* stream);

/*
 * pq2_verify_drafts -- which drafted tokens the target model keeps, and the
 * token after them, from given random numbers.  Sequence b's token rows are
 * row_start[b] .. row_start[b+1]-1: one per draft and one more.  With
 * p = softmax(logits[row] / temperature[b]) and q the drafter's probabilities
 * at the row (q NULL: it proposed its draft with certainty), row after row:
 *   draft d = drafts[row] is kept while u[row] * q(d) < p(d);
 *   at the first draft that is not: token = argmax_v max(p(v) - q(v), 0) / e[b][v]
 *   (argmax_v p(v) / e[b][v] where that is 0 everywhere);
 *   after the last draft: token = argmax_v p(v) / e[b][v].
 * With e drawn from Exp(1) and u from U[0, 1), kept drafts and token follow
 * the target's distribution.  temperature[b] <= 0: greedy -- a draft is kept
 * while it is the row's argmax, and token is the argmax of the row after.
 * temperature[b] may be infinite (every value that is not masked alike).
 * Ties go to the lowest index.  Values of -inf are masked (never drawn); a
 * row with nothing else keeps no draft and gives token -1.  A draft outside
 * [0, V) ends the sequence's drafts (padding): its row is the row after.
 *   logits      in   fp32 [rows, V], row stride ld_logits >= V (no NaN, no +inf)
 *   row_start   in   int32 [B + 1], 0 <= row_start[b] <= row_start[b+1] <= rows;
 *                    a sequence that breaks this keeps 0 and sets the device
 *                    error word; the others are not affected (two that share
 *                    rows, possible only around a broken one, are undefined).
 *                    A sequence without rows keeps 0.
 *   drafts      in   int32 [rows] (a sequence's last one is not read as a draft)
 *   q           in   fp32 [rows, V], row stride ld_q >= V, or NULL
 *   u           in   fp32 [rows]
 *   e           in   fp32 [B, V], row stride ld_e >= V, > 0
 *   temperature in   fp32 [B]
 *   accepted    out  int32 [B]   drafts kept
 *   tokens      out  int32 [rows] kept drafts, then token, then -1
 *   workspace   pq2_verify_workspace_bytes(B, rows, V) bytes, 16-byte aligned
 * B >= 0 (0 enqueues nothing), rows >= 0, 1 <= V <= 2^30.  logits, q, u and e:
 * 4-byte aligned (PQ2_ERR_MISALIGNED otherwise).
 */
size_t pq2_verify_workspace_bytes(int64_t B, int64_t rows, int64_t V);
pq2_status pq2_verify_drafts(const float* logits, int64_t ld_logits, const int32_t* row_start,
                             const int32_t* drafts, const float* q, int64_t ld_q, const float* u,
                             const float* e, int64_t ld_e, const float* temperature,
                             int32_t* accepted, int32_t* tokens, int64_t B, int64_t rows, int64_t V,
                             void* workspace, size_t workspace_bytes, void* stream);
/* The same with the arguments in one struct, for bindings that convert them
 * one by one. */
typedef struct {
    const float* logits;
    const int32_t *row_start, *drafts;
    const float *q, *u, *e, *temperature;
    int32_t *accepted, *tokens;
    void* workspace;
    int64_t ld_logits, ld_q, ld_e, B, rows, V;
    size_t workspace_bytes;
} pq2_verify_drafts_args;
pq2_status pq2_verify_drafts_packed(const pq2_verify_drafts_args* args, void* stream);

/*
 * Rotary positions.  A table holds, for positions first .. first + count - 1,
 * the cosine and sine of each pair's angle: fp32 [count, rot / 2, 2].
 */

/* How a table's frequencies f_i = base^(-2 i / rot), i = 0 .. rot/2 - 1, are
 * scaled for contexts longer than the trained one. */
#define PQ2_ROPE_PLAIN 0  /* as they are                                        */
#define PQ2_ROPE_LINEAR 1 /* f_i / factor                                       */
#define PQ2_ROPE_BASE 2   /* base * factor^(rot / (rot - 2)) for base (rot > 2) */
#define PQ2_ROPE_RAMP 3   /* by the index: f_i where it turns at least `high`
                             times over `old_len` positions, f_i / factor where
                             at most `low` times, and linear in i between the
                             two indexes (rounded outwards, kept within 0 .. rot - 1,
                             at least 0.001 apart)                              */
#define PQ2_ROPE_BANDS 4  /* by the wavelength w = 2 pi / f_i: f_i where
                             w < old_len / high, f_i / factor where w > old_len / low,
                             between them (1 - t) f_i / factor + t f_i with
                             t = (old_len / w - low) / (high - low)             */
typedef struct pq2_rope_scaling {
    int32_t kind;
    float magnitude;  /* cosines and sines are multiplied by this (0: 1)        */
    double factor;    /* >= 1 (kinds 1 to 4)                                    */
    double old_len;   /* > 0 (kinds 3 and 4)                                    */
    double low, high; /* 0 < low < high (kinds 3 and 4)                         */
} pq2_rope_scaling;

/* Largest rotated part, and largest head, of the entry points below. */
#define PQ2_ROPE_MAX_DIM 512

/*
 * pq2_rope_table -- table out: fp32 [count, rot / 2, 2].  Frequencies and
 * angles in 64 bits, cosines and sines rounded once to fp32.
 *   scaling: NULL (PQ2_ROPE_PLAIN) or a host struct, read before the call returns.
 * 2 <= rot <= PQ2_ROPE_MAX_DIM, rot % 2 == 0; base > 1; first >= 0, count >= 0 (0
 * enqueues nothing), first + count <= 2^31.  table 16-byte aligned.
 */
pq2_status pq2_rope_table(float* table, int64_t first, int64_t count, int64_t rot, double base,
                          const pq2_rope_scaling* scaling, void* stream);

/* Flags of pq2_rope and pq2_cache4_append. */
#define PQ2_ROPE_NEIGHBOURS 1u /* pairs (2i, 2i + 1); without it (i, i + rot/2) */
#define PQ2_ROPE_INVERSE 2u    /* by the negative angle (pq2_rope only)         */

/*
 * pq2_rope -- turns the first `rot` values of every head by its token's angles:
 *   a' = a cos - b sin,  b' = b cos + a sin
 * for every pair (a, b), each product and sum one fp32 operation, rounded once
 * to the output's type; the values behind `rot` are copied.
 * One call takes up to two arrays (queries and keys) of the same tokens.
 *   x, x2         in   [M, heads, dim] and [M, heads2, dim] (x_type; x2 and out2
 *                      may be NULL with heads2 == 0)
 *   out, out2     out  the same shapes (out_type); out may be x and out2 may be x2
 *                      where types and strides are the same; else nothing overlaps
 *   table         in   fp32 [table_rows, rot / 2, 2] (pq2_rope_table, or one's own)
 *   positions     in   int32 [M], rows of the table; a token with one outside
 *                      [0, table_rows) is left as it was in the outputs and sets the device
 *                      error word (PQ2_ERR_INVALID_ARG from pq2_last_device_error).  With
 *                      rot == 0 neither it nor the table is read
 * ld_*: strides from token to token, hs_*: from head to head (both >= dim), in
 * elements.  A head's values are adjacent.  The gradient of x is the same call with
 * PQ2_ROPE_INVERSE on the gradient of out.
 * M >= 0 (0 enqueues nothing), 1 <= dim <= PQ2_ROPE_MAX_DIM, 0 <= rot <= dim,
 * rot % 2 == 0, heads + heads2 <= 65536, M <= 2^24.  Pointers aligned to their elements, the table to
 * 16 bytes.  The vector path takes dims of 64, 128 and 256 whose pairs fall on
 * 16-byte boundaries (rot / 2, or rot with NEIGHBOURS, a multiple of dim / 32).
 */
typedef struct pq2_rope_args {
    const void *x, *x2;
    void *out, *out2;
    const float* table;
    const int32_t* positions;
    int64_t ld_x, hs_x, ld_x2, hs_x2, ld_out, hs_out, ld_out2, hs_out2;
    int64_t M, table_rows;
    int32_t heads, heads2, dim, rot, x_type, out_type;
    uint32_t flags;
    int32_t reserved; /* 0 */
} pq2_rope_args;
pq2_status pq2_rope(const pq2_rope_args* args, void* stream);

/*
 * A cache of keys and values in 4 bits, in pages of T tokens (T % 16 == 0).
 * A page of one key/value head is T / 16 tiles of 16 tokens, each
 *     16 rows of D/2 bytes   key codes (value 2i in the low half of byte i)
 *     16 rows of D/2 bytes   value codes
 *     16 pairs of fp16       scale and offset of each key row
 *     16 pairs of fp16       scale and offset of each value row
 * (16 (D + 8) bytes), the heads of a page one behind the other.  Every row of
 * D values has one scale and one offset; a code c stands for c * scale + offset.
 * From values x of a row, in fp32, each step rounded to nearest even:
 *     scale  = fp16(min((max - min) * (1/15), 65504)),  offset = fp16(min clamped to +-65504)
 *     c      = rint((x - offset) * (1 / scale)) clamped to 0 .. 15     (0 where scale is 0)
 * with 1/15 the nearest fp32.  NaN or Inf in a row: its contents are undefined.
 *
 * The sequences of a call:
 *   row_start  int32 [B + 1]  token rows row_start[b] .. row_start[b+1] - 1 are
 *                             sequence b's newest; rows from row_start[B] on
 *                             belong to none (padding): outputs there are left as they were
 *   lens       int32 [B]      tokens of the sequence with the new ones: row i of
 *                             its n rows has position lens[b] - n + i
 *   pages      int32 [B, W]   page of positions T j .. T j + T - 1 (row stride ld_pages >= W);
 *                             entries behind the last token's are not read
 */
#define PQ2_CACHE4_MAX_HEADS 1024

/* The arguments that the calls on such a cache share. */
typedef struct pq2_cache4 {
    void* pool;             /* 16-byte aligned                                   */
    const int32_t* pages;
    const int32_t* row_start;
    const int32_t* lens;
    int64_t page_stride;    /* bytes from page to page (>= pq2_cache4_page_bytes, % 16 == 0) */
    int64_t num_pages;      /* in the pool                                       */
    int64_t ld_pages;
    int64_t B, W;
    int32_t heads, dim;     /* key/value heads; 64, 128 or 256 values            */
    int32_t page_tokens;    /* T: a multiple of 16, at most 1024                 */
    int32_t reserved;       /* 0                                                 */
} pq2_cache4;

/* Bytes of a page (all its heads); 0 for sizes that are not supported. */
size_t pq2_cache4_page_bytes(int64_t heads, int64_t dim, int64_t page_tokens);

/*
 * pq2_cache4_append -- new tokens into the cache: keys turned by their
 * positions (pq2_rope's arithmetic), keys and values quantised and stored; with q, the
 * queries turned in the same launch.
 *   k, v       in   [M, heads, dim] (x_type), token and head strides in elements
 *   q, q_out   q in [M, q_heads, dim] (x_type), q_out out (out_type), or both NULL with
 *                   q_heads == 0.  q_out may be q where type and strides are the same.
 *   table      in   fp32 [table_rows, rot / 2, 2], or NULL with rot == 0 (nothing is turned)
 *   positions  in   int32 [M] rows of the table, or NULL: the tokens' positions
 * A token whose position, page or row of the table lies outside its range is
 * skipped and sets the device error word (PQ2_ERR_INVALID_ARG from
 * pq2_last_device_error); a page past the pool leaves q alone to be written.
 * Two tokens of one call must not have the same place in the cache.
 * flags: 0 or PQ2_ROPE_NEIGHBOURS.  M: rows of the arrays, 0 <= M <= 2^24.
 */
typedef struct pq2_cache4_append_args {
    pq2_cache4 cache;
    const void *k, *v, *q;
    void* q_out;
    const float* table;
    const int32_t* positions;
    int64_t ld_k, hs_k, ld_v, hs_v, ld_q, hs_q, ld_q_out, hs_q_out;
    int64_t M, table_rows;
    int32_t q_heads, rot, x_type, out_type;
    uint32_t flags;
    int32_t reserved; /* 0 */
} pq2_cache4_append_args;
pq2_status pq2_cache4_append(const pq2_cache4_append_args* args, void* stream);

/*
 * pq2_cache4_read -- the values that the cache holds for the call's token rows
 * (code * scale + offset in fp32, rounded once): k_out, v_out [M, heads, dim]
 * (out_type; either may be NULL).  Rows without a place in the cache are
 * skipped as in pq2_cache4_append.
 */
typedef struct pq2_cache4_read_args {
    pq2_cache4 cache;
    void *k_out, *v_out;
    int64_t ld_k, hs_k, ld_v, hs_v;
    int64_t M;
    int32_t out_type, reserved; /* 0 */
} pq2_cache4_read_args;
pq2_status pq2_cache4_read(const pq2_cache4_read_args* args, void* stream);

/*
 * pq2_cache4_attend -- attention of the call's token rows over the cache:
 *   out[m, h] = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale * q[m, h] . k_j)
 * over the positions j <= p(m) of its sequence, p(m) - window < j where window > 0; k and
 * v of key/value head h / (q_heads / heads).  The new tokens' keys and values
 * have to be in the cache (pq2_cache4_append).  A row that sees nothing (its position
 * below 0) gives zeros.  Scores, maxima, sums and accumulated outputs are
 * fp32.  What enters the products with fewer bits, for a sequence with up to 48 rows per
 * key/value head (n q_heads / heads; 32 with dim 256) and, in brackets, with more:
 *   q           times a power of two of its row's own, as fp16: a value is off by at most 2^-28
 *               [2^-35] of the row's largest, and those within 2^17 [2^24] of that
 *               (bf16: 2^20 [2^27]) are exact.  [The row's sum is kept to 2^-22 of itself or 2^-31
 *               of the row's largest, a key's offset to 2^-21 of itself or 2^-17 of its scale, and a
 *               scale below 2^-25 of its offset counts as that.]
 *   weights w   times the values' scales over a power of two, as fp16: 11 bits of itself,
 *               or a key's part of an output to 2^-24 of the largest values' scale that the row
 *               sees (beside rows of the sequence with scores past 2^22: that those see)
 * (B == 1: max_rows, or M, stands for the sequence's rows.)
 *   q, out     [M, q_heads, dim] (type: PQ2_F16 or PQ2_BF16), token and head
 *              strides in elements, a head's values adjacent
 *   max_rows   an upper bound of the sequences' rows that the host knows
 *              (1 in a decode step), or 0 (M); it chooses the kernels and is
 *              part of the contract: a sequence with more rows gets none of
 *              them (and sets the device error word)
 *   workspace  pq2_cache4_attend_workspace_bytes(M, q_heads, heads, dim) bytes, 16-byte aligned;
 *              enough for fewer rows too
 * Pages outside the pool among those that a sequence needs: its rows are
 * undefined and the device error word is set; lens past W T likewise (nothing behind the
 * table is read).  NaN or Inf in q: that row and head undefined; the same where scale times a
 * value, or that times a value or a scale of a key, is 2^108 or more in size, or scale
 * itself 2^80.  out and q do not overlap.
 * Results do not depend on other sequences' contents, but the order in which a
 * row's partial sums are joined depends on the sequences' lengths.
 * M >= 0, B >= 0 (0 enqueues nothing), q_heads % heads == 0, q_heads / heads <= 64,
 * window >= 0, scale finite; M <= 2^20, M * q_heads <= 2^30.  q and out 16-byte aligned with strides
 * % 8 == 0.
 */
typedef struct pq2_cache4_attend_args {
    pq2_cache4 cache;
    const void* q;
    void *out, *workspace;
    int64_t ld_q, hs_q, ld_out, hs_out;
    int64_t M, max_rows, window;
    size_t workspace_bytes;
    float scale;
    int32_t q_heads, type, reserved; /* 0 */
} pq2_cache4_attend_args;
size_t pq2_cache4_attend_workspace_bytes(int64_t M, int64_t q_heads, int64_t heads, int64_t dim);
pq2_status pq2_cache4_attend(const pq2_cache4_attend_args* args, void* stream);

/*
 * The pages of a cache between two steps.  refs [P] counts each page's
 * holders: the sequences of the table, and whoever else keeps it (a stored prefix).
 *
 * pq2_pages_update -- slot b goes on from slot source[b] (itself, another:
 * a fork, or < 0: none, the slot is emptied) with the first keep[b] of that
 * slot's lens[source[b]] tokens, and gets pages for new_lens[b] tokens in all.
 * With k = min(keep, lens[source], new_lens) (0 without a source), the k / T whole pages are
 * shared.  A page of which only the first k % T tokens are kept goes on to
 * the lowest slot that keeps such a part if nobody else holds it (whole, or
 * from outside the table); every other such slot gets a page and a pair
 * (old, new) in copies, to be copied before the slot's next append.  Pages
 * that are wanted are taken in the order of slots and positions, lowest free page first.
 *   pages       in   int32 [B, W] (row stride ld_pages); lens int32 [B]
 *   refs        in   int32 [P]
 *   source, keep, new_lens  in int32 [B]; new_lens <= W T
 *   pages_out   out  int32 [B, W] (row stride ld_out), -1 behind the last page; not `pages`
 *   refs_out    out  int32 [P]; may be refs
 *   copies      out  int32 [B, 2]: slot b's pair, or (-1, -1)
 *   info        out  int32 [2]: free pages left, pages that were wanted and not there
 *                    (their entries are -1)
 * Values out of range (source >= B, keep or lens or new_lens outside [0, W T],
 * a page outside [0, P) in use) count as the nearest in range (a source past B as none, such a page as
 * -1, held by nobody) and set the device error word.
 *   workspace   pq2_pages_workspace_bytes(B, P) bytes, 16-byte aligned
 * 0 <= B <= 2^20, 1 <= W <= 2^20, B W <= 2^30, 0 <= P <= 2^28, 1 <= T <= 2^20,
 * W T <= 2^30 (PQ2_ERR_UNSUPPORTED_SHAPE otherwise).
 */
typedef struct pq2_pages_update_args {
    const int32_t *pages, *lens, *refs, *source, *keep, *new_lens;
    int32_t *pages_out, *refs_out, *copies, *info;
    void* workspace;
    int64_t ld_pages, ld_out, B, W, P, T;
    size_t workspace_bytes;
} pq2_pages_update_args;
size_t pq2_pages_workspace_bytes(int64_t B, int64_t P);
pq2_status pq2_pages_update(const pq2_pages_update_args* args, void* stream);

/*
 * pq2_pages_compact -- which pages to move so that the n in use (refs > 0) are
 * pages 0 .. n - 1: the i-th page in use from n on goes to the i-th free one
 * below n.
 *   pages, lens, refs  in   as above
 *   pages_out          out  [B, W]: the same places, moved; -1 behind the last page
 *   refs_out           out  [P]; may be refs
 *   copies             out  int32 [P / 2, 2]: the moves (old, new), then (-1, -1)
 *   info               out  int32 [2]: pages in use, moves
 * Sizes, workspace and out-of-range values as pq2_pages_update.
 */
typedef struct pq2_pages_compact_args {
    const int32_t *pages, *lens, *refs;
    int32_t *pages_out, *refs_out, *copies, *info;
    void* workspace;
    int64_t ld_pages, ld_out, B, W, P, T;
    size_t workspace_bytes;
} pq2_pages_compact_args;
pq2_status pq2_pages_compact(const pq2_pages_compact_args* args, void* stream);

/*
 * pq2_pages_copy -- copies pages of a pool within it: for each of the n pairs
 * (old, new) whose two pages are in [0, P), in each of `layers` pools that lie
 * layer_stride bytes apart.  Pairs with a negative page are skipped; a page >= P is
 * skipped too and sets the device error word.  No new page may be another pair's old or new one.
 *   pool  16-byte aligned; page_bytes, page_stride (>= page_bytes), layer_stride % 16 == 0
 *   pairs int32 [n, 2], 8-byte aligned
 * n >= 0 (0 enqueues nothing), n <= 2^28, 0 <= layers <= 65536, 0 <= P <= 2^31,
 * page_bytes <= 2^32.
 */
pq2_status pq2_pages_copy(void* pool, int64_t page_bytes, int64_t page_stride, int64_t P,
                          int64_t layers, int64_t layer_stride, const int32_t* pairs, int64_t n,
                          void* stream);

/*
 * pq2_workspace_bytes -- scratch bytes `op` needs for this shape (0 if none,
 * SIZE_MAX if the shape is not supported).
 */
size_t pq2_workspace_bytes(int op, int64_t M, int64_t N, int64_t K);

/*
 * pq2_group_dots -- debug view of the integer part of a kernel: the same
 * kernel as `op` (PQ2_OP_GEMV, PQ2_OP_SMALL or PQ2_OP_PREFILL), writing the
 * per-group ternary dots dot(codes,q) - sum(q) instead of y
 * ([P1] "One token at a time": the -1 offset as one subtraction per group).
 *   dots out int32 [M, N, G].  Other operands as for `op`; workspace as for
 *   `op`.  For PQ2_OP_GEMV, M must be 1.
 */
pq2_status pq2_group_dots(int op, const int8_t* qp, const int32_t* T, const uint8_t* codes,
                          int64_t M, int64_t N, int64_t K, int32_t* dots,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * pq2_last_device_error -- synchronises `stream`, then reads and clears the
 * current device's error word: PQ2_ERR_TIMEOUT if a kernel's bounded wait ran
 * out, PQ2_ERR_BOUNDS (bounds-checked build only) if a kernel skipped a store
 * outside its buffer, PQ2_ERR_INVALID_ARG if pq2_pack_weights met a
 * non-ternary value or an index array of pq2_lora_add, pq2_verify_drafts, the
 * rotary positions, the cache or its pages a value outside its range,
 * PQ2_OK otherwise (PQ2_ERR_CUDA if the synchronisation itself failed).
 */
pq2_status pq2_last_device_error(void* stream);

/*
 * pq2_gemm_small_noalloc -- pq2_gemm_small for callers that cannot allocate
 * device memory (no allocator of their own, or allocation not allowed where
 * they run): the same kernel, with its split-K scratch in a fixed 4 MiB
 * device array that the library holds on every device it is loaded on until
 * the process exits.  (The pages have no counterpart to this entry point;
 * it exists for callers of this library.)
 *   Same operands as pq2_gemm_small, no workspace.  Returns
 *   PQ2_ERR_WORKSPACE if the shape needs more than
 *   pq2_gemm_small_noalloc_max_scratch() bytes of scratch on this device.
 *   For the tensor-core kernel (5 or more tokens) the scratch is about
 *   (min(SMs, 256) + ceil(N/128)) * M * 512 bytes of partial sums plus
 *   ceil(K/512) * 16 KB of token tiles: on a 152-SM GPU, 16 tokens fit up
 *   to about N = 40,000 at K = 5120, and an lm_head-scale N = 248,320 gets
 *   PQ2_ERR_WORKSPACE.  2 to 4 tokens, where the DP4A kernel takes them,
 *   need no scratch.
 *   The first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress) and should come before any stream capture.
 *   All calls share the array: calls that may run at the same time on the
 *   GPU (unordered streams) race on it.  No cudaMalloc, cudaFree or other
 *   allocating call is made.
 */
pq2_status pq2_gemm_small_noalloc(const int8_t* qp, const float* S, const int32_t* T,
                                  const uint8_t* codes, const void* ws_f16, float* y,
                                  int64_t M, int64_t N, int64_t K, void* stream);

/* Size in bytes of the fixed scratch array behind pq2_gemm_small_noalloc. */
size_t pq2_gemm_small_noalloc_max_scratch(void);

/* Kernel variants for pq2_debug_force_kernel. */
#define PQ2_VARIANT_DEFAULT 0        /* the library's own routing                  */
#define PQ2_VARIANT_GEMV_DIRECT 1    /* M = 1: look-ahead loads into registers      */
#define PQ2_VARIANT_GEMV_RING 2      /* M = 1: bulk-copy ring in shared memory      */
#define PQ2_VARIANT_GEMV_STAGED 3    /* M = 1 fused: whole slice staged before wait */
#define PQ2_VARIANT_SMALL_DP4A 1     /* 2..8 tokens: DP4A, code words shared        */
#define PQ2_VARIANT_SMALL_TC 2       /* tcgen05, weights in tensor memory, 16-token
                                        tile (5..16 tokens by default)              */
#define PQ2_VARIANT_SMALL_TILE 3     /* tcgen05 token-tile kernel (16 tokens)       */
#define PQ2_VARIANT_SMALL_WTILE 4    /* tcgen05, 128 weight rows per MMA, tokens as
                                        the 128-row operand (16 tokens)             */
#define PQ2_VARIANT_PREFILL_128 1    /* tcgen05 128 x 128 tiles, in-kernel expansion */
#define PQ2_VARIANT_PREFILL_WIDE 2   /* tcgen05 128 x 256 tiles, pre-expanded weights */
#define PQ2_VARIANT_PREFILL_TILE 3   /* tcgen05 token-tile kernel, M <= 64 (by
                                        default 17-32 tokens)                       */
#define PQ2_VARIANT_PREFILL_WTILE 4  /* tcgen05, 128 weight rows per MMA, tokens as
                                        the 128-row operand, M <= 64 (by default
                                        33-64 tokens when a CTA gets at most 4
                                        items of 128 rows x 4 groups)               */

/*
 * pq2_debug_force_kernel -- test hook: from now on, calls of `op`
 * (PQ2_OP_GEMV, PQ2_OP_SMALL or PQ2_OP_PREFILL; pq2_matmul, pq2_group_dots
 * and pq2_mlp_down_swiglu route through them) run kernel `variant` of that op
 * (PQ2_VARIANT_*), or follow the library's own routing again with
 * PQ2_VARIANT_DEFAULT.  Every variant computes the same integer group dots
 * and the same y, bit for bit; the hook exists so that tests can check each
 * kernel on shapes the routing would give to another.  A call whose shape
 * the forced variant cannot take returns PQ2_ERR_UNSUPPORTED_SHAPE.
 * pq2_workspace_bytes accounts for the forced variant, so set it before
 * sizing a workspace.  Process-wide; not for use while other threads call
 * the library.  PQ2_ERR_INVALID_ARG for an unknown op or variant.
 */
pq2_status pq2_debug_force_kernel(int op, int variant);

/*
 * pq2_debug_gemv_floor -- measurement hook: enqueues one launch of an empty
 * kernel (it waits for the preceding kernel on the stream and lets the next
 * one start launching, nothing else) with the grid, block and shared memory
 * that pq2_matmul_ex(M = 1, N, K, flags) gets.  A chain of these times the
 * launch and dependency latency a chain of real calls pays before any byte
 * moves: the floor of a dependent sequence of M = 1 calls.  No pointer is
 * passed and nothing is written.  Errors as pq2_matmul_ex (shape, flags).
 */
pq2_status pq2_debug_gemv_floor(int64_t N, int64_t K, uint32_t flags, void* stream);

/*
 * pq2_debug_mma_rate -- measurement hook: the rate at which one thread per SM
 * can issue tcgen05 MMAs of the kind the tensor-core kernels use
 * (kind::f8f6f4, e4m3 operands, M = 128, N = n, K = 32; A in tensor memory,
 * B in shared memory), back to back into one accumulator.  Enqueues one
 * launch of one CTA per SM; on completion cycles[sm] holds the SM clock
 * cycles from the first issue to the completion of `iters` MMAs (0 if the
 * bounded wait ran out).  n in {32, 64, 128, 256}, 1 <= iters <= 2^24.
 *   cycles  device uint64 array of at least (number of SMs) entries.
 * Multiply-adds per cycle per SM: 128 * n * 32 * iters / cycles.
 */
pq2_status pq2_debug_mma_rate(int n, int iters, uint64_t* cycles, void* stream);

/*
 * pq2_debug_set_wait_limit_ns -- bound on every on-chip barrier wait, in
 * nanoseconds (default 2e9).  For tests of the timeout path only.
 */
pq2_status pq2_debug_set_wait_limit_ns(uint64_t ns);

/*
 * pq2_debug_skip_stage -- test hook: from now on, the producer of every
 * bulk-copy pipeline withholds its stage number `stage` (never issues it), so
 * the consumers' bounded wait runs out and the call reports PQ2_ERR_TIMEOUT
 * through pq2_last_device_error.  -1 turns it off (the default).  Attention with
 * many rows withholds a piece of expanded keys, or piece stage - 65536 of values.
 */
pq2_status pq2_debug_skip_stage(int stage);

/*
 * pq2_bounds_checked -- 1 in the bounds-checked build of the library
 * (libpq2_debug.so, compiled with PQ2_DEBUG=1), 0 in the normal one.  In the
 * bounds-checked build every kernel store to an output (y, the integer dots,
 * residual, x, accepted, tokens) and to the split-K and statistics scratch
 * first checks that it lies inside its buffer; a store
 * that does not is skipped and pq2_last_device_error reports PQ2_ERR_BOUNDS.
 * Results are otherwise bit-identical to the normal build's.  It stands in
 * for a memory checker on GPUs where none can be run.
 */
int pq2_bounds_checked(void);

/*
 * pq2_debug_shrink_bounds -- test hook of the bounds-checked build: from now
 * on the checks treat the last `elements` elements of every checked buffer as
 * outside it, so that the stores a call makes there are reported
 * (PQ2_ERR_BOUNDS) and skipped (no memory outside the buffers is touched).
 * 0 turns it off (the default); no effect in the normal build.
 * PQ2_ERR_INVALID_ARG for a negative count.
 */
pq2_status pq2_debug_shrink_bounds(int elements);

#ifdef __cplusplus
}
#endif

#endif /* PQ2_H */
