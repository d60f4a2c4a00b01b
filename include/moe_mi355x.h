/*
 * moe_mi355x.h - C ABI of the DeepSeekMoE layer on AMD MI355X (gfx950), and of
 * what a decoder block has around it: norm, 4-bit products, latent attention.
 *
 * The layer (sources: the "DeepSeek-V3 Technical Report" reading guide on
 * xyznot.com, Turkish edition "Okuma rehberi" and French edition "Guide de
 * lecture", Method section 2 "DeepSeekMoE with auxiliary-loss-free
 * balancing", cited below as [RG-MoE]; its "Key ideas" section, FP8 bullet,
 * cited as [RG-FP8]):
 *
 *   s_{i,t}  = Sigmoid(u_t . e_i)                       affinity sentence
 *   g'_{i,t} = s_{i,t} if s_{i,t}+b_i is in the Top-K   gate equation
 *              of {s_{j,t}+b_j}, else 0; g = g' normalised
 *   h'_t     = u_t + sum_j FFN^(s)_j(u_t)                combine equation
 *              + sum_i g_{i,t} FFN^(r)_i(u_t)
 *   b_i     <- b_i - gamma if expert i is overloaded,    bias rule
 *              b_i + gamma if underloaded (gamma = 0.001)
 *
 * One forward is: moe_route -> moe_permute -> [fp8_quantize_tiles] ->
 * moe_expert_gemm -> moe_combine, then moe_bias_update at the end of a step.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Pointers named as device pointers must point to device memory (HBM) of
 *    the current HIP device; the caller owns every buffer.  The library
 *    allocates and frees no memory, keeps no pointer after a call returns
 *    and holds no state between calls (no stream, event, lock or cache of
 *    its own), except moe_permute_noalloc's device array and its address
 *    per GPU.
 *  - `stream` is a hipStream_t (NULL = the null stream).  Every call
 *    enqueues its kernels on it and returns without synchronising; calls on
 *    distinct streams may run concurrently from different threads.
 *  - Tensors are row-major and contiguous, element offsets are 64-bit.
 *    Data tensors (u, centroids, x, weights, y, out, q and the workspaces)
 *    must be 16-byte aligned (hipMalloc and torch allocations are 256-byte
 *    aligned); index, gate, load, bias and scale arrays need only the
 *    alignment of their element type.  A misaligned data tensor is
 *    MOE_EINVAL.
 *    bf16 is stored as raw 16-bit patterns, E4M3 as one byte per value (OCP
 *    E4M3FN: exponent bias 7, largest finite 448, no infinities).
 *  - Arguments are checked on the host before any launch.  A bad argument
 *    returns MOE_EINVAL (or MOE_EUNSUPPORTED / MOE_EWORKSPACE) and launches
 *    nothing; a launch failure returns MOE_EHIP.  With valid arguments the
 *    device code cannot fail.  moe_last_error() gives a message for the last
 *    failing call of the calling thread.  Device data (indices, counts) is
 *    not validated: it must come from the producing entry point.
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 5

/* Limits of this implementation. */
#define MOE_MAX_EXPERTS 1024   /* routed + shared experts */
#define MOE_MAX_K 16           /* routed experts per token */
#define MOE_TILE_ROWS 256      /* rows per entry of the GEMM tile map */
#define MOE_NORM_MAX_D 32768   /* columns of moe_rmsnorm */
#define MOE_FEW_TOKENS 32      /* tokens of moe_layer_few */
#define MLA_MAX_REQUESTS 8192  /* requests or packed sequences of the mla_* calls */

typedef enum {
  MOE_OK = 0,
  MOE_EINVAL = 1,        /* NULL pointer, size out of range, bad enum */
  MOE_EUNSUPPORTED = 2,  /* a valid combination the library does not run */
  MOE_EWORKSPACE = 3,    /* workspace smaller than the size helper returns */
  MOE_EHIP = 4           /* the HIP runtime reported an error at launch */
} moe_status;

typedef enum {
  MOE_F32 = 0,
  MOE_BF16 = 1,
  MOE_E4M3 = 2,
  MOE_E2M1 = 3 /* two codes per byte, an exponent byte per 32 columns (fp4_*) */
} moe_dtype;

/* Flags of moe_combine: drop a term of the combine equation (component checks). */
#define MOE_COMBINE_NO_RESIDUAL 1u
#define MOE_COMBINE_NO_SHARED 2u
#define MOE_COMBINE_NO_ROUTED 4u

int moe_abi_version(void);
const char* moe_status_str(int status);
/* Message of the last failing call made by this thread ("" if none). */
const char* moe_last_error(void);

/* ------------------------------------------------------------------------
 * moe_route: sigmoid affinities, bias-steered top-K, normalised gates, loads.
 * [RG-MoE] affinity sentence and gate equation.
 *
 *   u          device [T, d], dtype u_t (MOE_F32 or MOE_BF16): token states
 *   centroids  device [Nr, d] fp32: expert centroids e_i
 *   bias       device [Nr] fp32: routing bias b_i (read only here)
 *   topk_idx   device [T, K] int32 out: selected experts of each token,
 *              ordered by s+b descending; an exact tie goes to the lower index
 *   topk_gate  device [T, K] fp32 out: g = s / (sum of the selected s) -
 *              the gate keeps s, the bias only steers the selection
 *   topk_score device [T, K] fp32 out, may be NULL: s of the selected experts
 *   expert_load device [Nr] int32 out: number of tokens that selected each
 *              expert (overwritten, not accumulated)
 *   ws         device workspace of at least moe_route_workspace_bytes(T, d, Nr)
 *   Affinities are computed in fp32 (products exact, fp32 accumulation in
 *   blocks) and the sigmoid in fp32.
 *   Errors: MOE_EINVAL for NULL required pointers, T < 0, d < 1,
 *   Nr outside [1, MOE_MAX_EXPERTS], K outside [1, min(Nr, MOE_MAX_K)],
 *   d not a multiple of 8; MOE_EWORKSPACE when ws_bytes is too small.
 *   T == 0 is valid: expert_load is zeroed and nothing else is written.
 * ---------------------------------------------------------------------- */
size_t moe_route_workspace_bytes(int T, int d, int Nr);
moe_status moe_route(const void* u, moe_dtype u_t, const float* centroids, const float* bias,
                     int T, int d, int Nr, int K,
                     int32_t* topk_idx, float* topk_gate, float* topk_score, int32_t* expert_load,
                     void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * moe_permute: expert-contiguous, padded row layout (stable counting sort).
 * Realises the per-expert token sets that the combine equation sums over;
 * no token is dropped (blog "DeepSeek 알고 아는 척 좀 해보자 – 단편: 671B
 * 파라미터의 괴물, DeepSeek-V3", section "DeepSeekMoE & load balancing").
 *
 * Segment i < Nr holds the rows (t, k) with topk_idx[t, k] == i in increasing
 * t; segment Nr + j (j < Ns) holds every token 0..T-1 in order (shared expert
 * j, gate 1).  Each segment is padded with rows of token -1 to a multiple of
 * tile_m (a power of two in [1, MOE_TILE_ROWS]).
 *
 *   topk_idx   device [T, K] int32 in (from moe_route)
 *   seg_offset device [Nr+Ns+1] int32 out: first row of each segment;
 *              seg_offset[Nr+Ns] = padded rows in use
 *   row_token  device [P_max] int32 out: token of every row, -1 = padding
 *              (rows from seg_offset[Nr+Ns] to P_max are -1 as well)
 *   inv_row    device [T, K] int32 out: row that holds (t, k)
 *   tile_map   device [tiles_max, 4] int32 out: in segment order, each
 *              segment cut into tiles of MOE_TILE_ROWS rows (the last one
 *              shorter): {segment, first row, rows, token rows}; the token
 *              rows of a tile come first, its padding rows after them
 *   n_tiles    device [1] int32 out: entries of tile_map in use
 *   P_max = moe_permute_rows(...), tiles_max = moe_permute_tiles_max(...)
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes or tile_m;
 *   MOE_EWORKSPACE when ws_bytes < moe_permute_workspace_bytes(...).
 * ---------------------------------------------------------------------- */
size_t moe_permute_rows(int T, int K, int Nr, int Ns, int tile_m);
size_t moe_permute_tiles_max(int T, int K, int Nr, int Ns, int tile_m);
size_t moe_permute_workspace_bytes(int T, int K, int Nr, int Ns);
moe_status moe_permute(const int32_t* topk_idx, int T, int K, int Nr, int Ns, int tile_m,
                       int32_t* seg_offset, int32_t* row_token, int32_t* inv_row,
                       int32_t* tile_map, int32_t* n_tiles,
                       void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * moe_permute_noalloc: moe_permute without a workspace argument, for callers
 * that cannot allocate device memory (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc).  It allocates nothing:
 * the same kernels use a 4 MiB device array of the library's own (one copy
 * per GPU, held until the process ends; its address is looked up once per
 * device on the first call made with that device current).  Results are
 * those of moe_permute, bit for bit.
 *   Arguments, layouts and errors as moe_permute, without ws / ws_bytes;
 *   MOE_EWORKSPACE when the sizes need more than the array holds:
 *   moe_permute_workspace_bytes(T, K, Nr, Ns) must not exceed
 *   moe_permute_noalloc_scratch_bytes() (4 MiB: e.g. T up to 1048576 tokens
 *   with Nr = 256, T up to 262144 with Nr = 1024).
 *   Every call on one GPU uses that GPU's array: calls that overlap in time
 *   on one GPU (different streams or threads) race and must be serialised
 *   by the caller.
 * ---------------------------------------------------------------------- */
size_t moe_permute_noalloc_scratch_bytes(void);
moe_status moe_permute_noalloc(const int32_t* topk_idx, int T, int K, int Nr, int Ns, int tile_m,
                               int32_t* seg_offset, int32_t* row_token, int32_t* inv_row,
                               int32_t* tile_map, int32_t* n_tiles, void* stream);

/* ------------------------------------------------------------------------
 * moe_expert_gemm: every expert's SwiGLU FFN on its rows of the layout.
 * FFN^(s)_j and FFN^(r)_i of the [RG-MoE] combine equation; the pages do not
 * print the FFN form, this library uses SwiGLU:
 *   FFN(x) = W2 (SiLU(W_gate x) * (W_up x)),  SiLU(a) = a * sigmoid(a).
 * y[row] = FFN_{segment(row)}(x[row_token[row]]) for every token row of
 * every tile; padding rows of y (and of h in ws) may be left unwritten.
 *
 *   x, x_t      device [T, d]: MOE_F32, MOE_BF16, or MOE_E4M3 codes
 *   x_scale     device [T, d/128] fp32 for x_t == MOE_E4M3 (1x128 tiles,
 *               from fp8_quantize_tiles), else NULL
 *   w_t         MOE_F32, MOE_BF16 or MOE_E4M3 (128x128 blocks, [RG-FP8])
 *   w13         device [Nr+Ns, 2I, d]: rows 0..I-1 W_gate, rows I..2I-1 W_up
 *   w13_scale   device [Nr+Ns, 2I/128, d/128] fp32 for MOE_E4M3, else NULL
 *   w2          device [Nr+Ns, d, I]: W_down
 *   w2_scale    device [Nr+Ns, d/128, I/128] fp32 for MOE_E4M3, else NULL
 *   seg_offset, row_token, tile_map, n_tiles: from moe_permute
 *   ws          device workspace, moe_gemm_workspace_bytes(...) bytes: holds
 *               the hidden state h of every row
 *   y, y_t      device [P_max, d] out, MOE_F32 or MOE_BF16
 * Supported (x_t, w_t, y_t): (F32, F32, F32); (BF16, BF16, BF16|F32);
 * (BF16, E4M3, BF16) - fp8 weights, bf16 activations, h kept in bf16;
 * (E4M3, E4M3, BF16|F32) - fp8 activations and weights; h is re-quantised
 * to E4M3 in 1x128 tiles (scale rule of fp8_quantize_tiles) before the down
 * projection.
 * E4M3 scales must be powers of two, as fp8_quantize_tiles writes them: the
 * matrix instructions apply them as exponents per 128-wide K block, which is
 * exact; only the exponent field of a scale is read.  Accumulation is fp32
 * throughout.
 *   T == 0 is valid (x and x_scale may then be NULL): nothing is written.
 *   Errors: MOE_EINVAL for NULL pointers or bad sizes; MOE_EUNSUPPORTED for
 *   other dtype combinations; bf16 with d % 128 or I % 64 nonzero; E4M3 x E4M3
 *   with d or I not a multiple of 256 or above 8192; an operand of 2 GiB or
 *   more on the MFMA paths; MOE_EWORKSPACE for a small ws.
 * ---------------------------------------------------------------------- */
size_t moe_gemm_workspace_bytes(int T, int K, int Nr, int Ns, int d, int I, int tile_m,
                                moe_dtype x_t, moe_dtype w_t);
moe_status moe_expert_gemm(const void* x, moe_dtype x_t, const float* x_scale,
                           moe_dtype w_t, const void* w13, const float* w13_scale,
                           const void* w2, const float* w2_scale,
                           int T, int K, int Nr, int Ns, int d, int I, int tile_m,
                           const int32_t* seg_offset, const int32_t* row_token,
                           const int32_t* tile_map, const int32_t* n_tiles,
                           void* ws, size_t ws_bytes,
                           void* y, moe_dtype y_t, void* stream);

/* ------------------------------------------------------------------------
 * moe_combine: h'_t = u_t + sum_j y[shared_j(t)] + sum_k g[t,k] y[inv_row[t,k]]
 * ([RG-MoE] combine equation).  Accumulates in fp32 in a fixed order
 * (residual, shared experts ascending, routed k ascending), so results are
 * bitwise reproducible.
 *
 *   u, u_t       device [T, d], MOE_F32 or MOE_BF16
 *   y, y_t       device [P_max, d] from moe_expert_gemm
 *   inv_row      device [T, K] int32, topk_gate device [T, K] fp32
 *   seg_offset   device [Nr+Ns+1] int32 (shared rows: seg_offset[Nr+j] + t)
 *   flags        MOE_COMBINE_* bits to drop terms
 *   out, out_t   device [T, d] out, MOE_F32 or MOE_BF16 (may not alias y)
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes, d not a multiple of 8.
 * ---------------------------------------------------------------------- */
moe_status moe_combine(const void* u, moe_dtype u_t, const void* y, moe_dtype y_t,
                       const int32_t* inv_row, const float* topk_gate, const int32_t* seg_offset,
                       int T, int d, int K, int Nr, int Ns, unsigned flags,
                       void* out, moe_dtype out_t, void* stream);

/* ------------------------------------------------------------------------
 * moe_expert_gemm_combine: moe_expert_gemm and moe_combine in one call, the
 * combine fused into the down projection ([RG-MoE] combine equation):
 *   out[t] = u_t + sum_j y[shared_j(t)] + sum_k g[t,k] y[inv_row[t,k]]
 * with every y row added to its token's row of out by fp32 atomic adds in
 * the down projection's epilogue, so y is never written to memory (about
 * 2 GB less traffic per 8192-token V3 prefill step than moe_expert_gemm +
 * moe_combine).  The order of the adds is not fixed: results agree with
 * moe_combine's to fp32 rounding of the sum and are not bitwise
 * reproducible (use moe_combine for that).  y rows are summed unrounded
 * (moe_combine reads them rounded to y_t).
 *   Arguments as moe_expert_gemm (x, weights, layout, tile_m), plus
 *   inv_row, topk_gate device [T, K] from moe_permute / moe_route
 *   u, u_t       device [T, d] tokens, MOE_F32 or MOE_BF16 (the residual)
 *   flags        MOE_COMBINE_* bits, as moe_combine
 *   ws           device, moe_gemm_combine_workspace_bytes(...) bytes
 *   out          device [T, d] fp32 out (overwritten; may not alias u)
 *   Supported (x_t, w_t): (BF16, BF16) with d % 256 == 0 and I % 128 == 0;
 *   (E4M3, E4M3) with d, I multiples of 256 up to 8192; else
 *   MOE_EUNSUPPORTED.  Other errors as moe_expert_gemm and moe_combine.
 * ---------------------------------------------------------------------- */
size_t moe_gemm_combine_workspace_bytes(int T, int K, int Nr, int Ns, int d, int I, int tile_m,
                                        moe_dtype x_t, moe_dtype w_t);
moe_status moe_expert_gemm_combine(const void* x, moe_dtype x_t, const float* x_scale,
                                   moe_dtype w_t, const void* w13, const float* w13_scale,
                                   const void* w2, const float* w2_scale,
                                   int T, int K, int Nr, int Ns, int d, int I, int tile_m,
                                   const int32_t* seg_offset, const int32_t* row_token,
                                   const int32_t* tile_map, const int32_t* n_tiles,
                                   const int32_t* inv_row, const float* topk_gate,
                                   const void* u, moe_dtype u_t, unsigned flags,
                                   void* ws, size_t ws_bytes, float* out, void* stream);

/* ------------------------------------------------------------------------
 * moe_bias_update: end-of-step bias rule ([RG-MoE] bias rule).  The pages do
 * not define "overloaded"; this library compares the load with the mean
 * load T*K/Nr exactly in integers: Nr*c_i > T*K -> b_i -= gamma,
 * Nr*c_i < T*K -> b_i += gamma, equal -> unchanged; one fp32 add.
 *
 *   expert_load  device [Nr] int32 (from moe_route of this step)
 *   total_assign T*K, the number of (token, expert) assignments of the step
 *   gamma        bias step (0.001 on the pages)
 *   bias         device [Nr] fp32, updated in place
 *   Errors: MOE_EINVAL for NULL pointers, Nr out of range, total_assign < 0,
 *   non-finite or negative gamma.
 * ---------------------------------------------------------------------- */
moe_status moe_bias_update(const int32_t* expert_load, int Nr, long long total_assign,
                           float gamma, float* bias, void* stream);

/* ------------------------------------------------------------------------
 * fp8_quantize_tiles: tile-wise E4M3 quantisation ([RG-FP8]: 1x128 tiles for
 * activations, 128x128 blocks for weights).  The pages give no scale rule;
 * this library uses, per tile, the power of two sc = 2^k with the smallest
 * k >= -126 such that amax <= 448 * sc (sc = 1 for an all-zero tile), and
 * code = round-to-nearest-even(x / sc) (exact division).  A power-of-two
 * scale is the E8M0 block scale the gfx950 scaled MFMA applies in hardware;
 * code * sc is exact in fp32 and in bf16.  NaN is never produced for finite
 * input.  Scales are stored as fp32 values.
 *
 *   x, x_t     device [rows, cols], MOE_F32 or MOE_BF16
 *   tile_rows  1 or 128 (rows must be a multiple of it); tile_cols 128
 *              (cols must be a multiple of it)
 *   q          device [rows, cols] uint8 out (E4M3 codes)
 *   scale      device [rows/tile_rows, cols/tile_cols] fp32 out
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes or tile shapes.
 * ---------------------------------------------------------------------- */
moe_status fp8_quantize_tiles(const void* x, moe_dtype x_t, long long rows, long long cols,
                              int tile_rows, int tile_cols, uint8_t* q, float* scale, void* stream);

/* ------------------------------------------------------------------------
 * fp8_dequantize_tiles: the values that E4M3 tiles stand for ([RG-FP8]
 * tiles), out[r, c] = decode(q[r, c]) * scale[r / tile_rows, c / 128]: the
 * operand an E4M3 product multiplies.  With power-of-two scales (as
 * fp8_quantize_tiles writes them) every value is exact in fp32, and in bf16
 * for scales >= 2^-124.  The E4M3 training step uses it for Q(u), the input
 * its gate/up weight gradient takes (straight-through quantisers).
 *
 *   q          device [rows, cols] uint8 E4M3 codes
 *   scale      device [rows/tile_rows, cols/128] fp32
 *   tile_rows  1 or 128; tile_cols 128 (as fp8_quantize_tiles)
 *   out, out_t device [rows, cols] out, MOE_F32 or MOE_BF16
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes or tile shapes, out_t.
 * ---------------------------------------------------------------------- */
moe_status fp8_dequantize_tiles(const uint8_t* q, const float* scale, long long rows, long long cols,
                                int tile_rows, int tile_cols, void* out, moe_dtype out_t, void* stream);

/* ------------------------------------------------------------------------
 * fp8_quantize_runs: E4M3 along the rows of the permuted layout, the token
 * axis along which a weight gradient sums ([RG-FP8] gives E4M3 for all
 * tensors but no tile along the tokens; the reading kept here is its 1x128
 * activation tile turned along that axis).  Segment e, rows
 * seg_offset[e] .. seg_offset[e+1]-1 (bounds clamped to [0, P]), is cut
 * into runs of 128 rows from its first row, the last run shorter; each
 * column of each run gets its own power-of-two scale by the rule of
 * fp8_quantize_tiles.  Run r of segment e is scale row run_offset[e] + r.
 *
 *   x, x_t     device, MOE_F32 or MOE_BF16: gather == 0: [P, cols], row r
 *              of the layout is x row r; gather != 0: [x_rows, cols], row r
 *              is x row row_token[r] (the token rows of moe_permute)
 *   row_token  device [P]: a row with row_token < 0 (padding), or whose
 *              token is not a row of x, counts as zeros
 *   seg_offset device [n_seg + 1] (moe_permute's, n_seg = Nr + Ns)
 *   run_offset device [n_seg + 1] int32 out: run_offset[e] = sum over
 *              e' < e of ceil(rows of e' / 128), run_offset[n_seg] = runs
 *   q          device [P, cols] uint8 out: codes of the rows of every
 *              segment (0 on padding rows); other rows untouched
 *   scale      device [fp8_quantize_runs_max(P, n_seg), cols] fp32 out:
 *              rows 0 .. runs-1 written
 *   Errors: MOE_EINVAL for NULL pointers (x may be NULL when it has no
 *   rows to read: P == 0, or gather with x_rows == 0), bad sizes
 *   (cols % 128 != 0, P < 0, n_seg < 1, gather == 0 with x_rows < P), x_t;
 *   MOE_EUNSUPPORTED for an operand of 2 GiB or more.
 * ---------------------------------------------------------------------- */
long long fp8_quantize_runs_max(long long P, int n_seg);  /* (P + 127 n_seg) / 128 */
moe_status fp8_quantize_runs(const void* x, moe_dtype x_t, long long x_rows, int cols,
                             const int32_t* row_token, int gather, const int32_t* seg_offset,
                             int n_seg, long long P, int32_t* run_offset, uint8_t* q,
                             float* scale, void* stream);

/* ========================================================================
 * Backward pass (bf16 activations and weights).  The pages print no
 * backward pass; these calls compute the chain rule through the forward
 * above.  The top-K selection and the bias b are piecewise constant in the
 * inputs, so no gradient flows through them and b receives none; the
 * gradient reaches the affinities only through the gates of the selected
 * experts.  With G = dL/dh' (the gradient of the layer output), one step is
 *   moe_expert_gemm_train (forward, keeping h and [a | b])
 *   moe_combine_backward  -> dy (gradient of every expert row), dgate, dz
 *   moe_expert_gemm_backward -> dx (gradient of every expert row's input),
 *                               dW13, dW2
 *   moe_route_backward    -> du, de
 * after moe_route / moe_permute of the forward (same buffers).
 * ====================================================================== */

/* ------------------------------------------------------------------------
 * moe_expert_gemm_train: moe_expert_gemm for (x_t, w_t) = (BF16, BF16) that
 * also keeps what the backward needs: h [P_max, I] (bf16, SiLU(a) * b) and
 * ab [P_max, 2I] (bf16: columns 0..I-1 a = W_gate x, I..2I-1 b = W_up x) of
 * every token row (padding rows unwritten).  y as in moe_expert_gemm.
 *   ws  device, moe_gemm_train_workspace_bytes(...) bytes (work schedule)
 *   Errors: as moe_expert_gemm; MOE_EUNSUPPORTED unless d % 256 == 0,
 *   I % 128 == 0 (d <= 65280, I <= 32640) and every operand < 2 GiB.
 * ---------------------------------------------------------------------- */
size_t moe_gemm_train_workspace_bytes(int T, int K, int Nr, int Ns, int d, int I, int tile_m);
moe_status moe_expert_gemm_train(const void* x, const void* w13, const void* w2,
                                 int T, int K, int Nr, int Ns, int d, int I, int tile_m,
                                 const int32_t* seg_offset, const int32_t* row_token,
                                 const int32_t* tile_map, const int32_t* n_tiles,
                                 void* ws, size_t ws_bytes, void* h, void* ab,
                                 void* y, moe_dtype y_t, void* stream);

/* ------------------------------------------------------------------------
 * moe_expert_gemm_train_w8: moe_expert_gemm for (x_t, w_t) = (E4M3, E4M3)
 * ([RG-FP8]: x in 1x128 tiles, weights in 128x128 blocks, h re-quantised in
 * 1x128 tiles before the down projection) that also keeps, for
 * moe_expert_gemm_backward_w8, ab [P_max, 2I] (bf16 pre-activations from
 * the fp32 accumulators) and h [P_max, I] (bf16: the E4M3 h that the down
 * projection multiplies, code x scale, exact).  y as in moe_expert_gemm.
 *   x, x_scale     device [T, d] E4M3 codes, [T, d/128] fp32 scales
 *   w13 .. w2_scale as moe_expert_gemm_backward_w8
 *   ws  device, moe_gemm_train_w8_workspace_bytes(...) bytes (work schedule
 *       and the E4M3 h)
 *   Errors: as moe_expert_gemm_train; MOE_EUNSUPPORTED unless d % 256 == 0,
 *   I % 256 == 0, d <= 8192 and I <= 8192.
 * ---------------------------------------------------------------------- */
size_t moe_gemm_train_w8_workspace_bytes(int T, int K, int Nr, int Ns, int d, int I, int tile_m);
moe_status moe_expert_gemm_train_w8(const uint8_t* x, const float* x_scale,
                                    const uint8_t* w13, const float* w13_scale,
                                    const uint8_t* w2, const float* w2_scale,
                                    int T, int K, int Nr, int Ns, int d, int I, int tile_m,
                                    const int32_t* seg_offset, const int32_t* row_token,
                                    const int32_t* tile_map, const int32_t* n_tiles,
                                    void* ws, size_t ws_bytes, void* h, void* ab,
                                    void* y, moe_dtype y_t, void* stream);

/* ------------------------------------------------------------------------
 * moe_combine_backward: gradients of the [RG-MoE] combine equation and of
 * the gate equation (g = s / sum of the selected s) for one step.
 *   grad_out, g_t  device [T, d] G = dL/dh', MOE_F32 or MOE_BF16
 *   y, y_t         device [P_max, d] expert outputs of the forward
 *   inv_row, topk_gate, topk_score: device [T, K] from moe_permute/moe_route
 *   seg_offset     device [Nr+Ns+1]
 *   dy             device [P_max, d] bf16 out: g[t,k] * G_t on row (t, k),
 *                  G_t on the shared rows of t (padding rows unwritten)
 *   dgate          device [T, K] fp32 out: <G_t, y[row(t, k)]>
 *   dz             device [T, K] fp32 out: dL/d(u_t . e_i) of the selected
 *                  experts, (dgate_k - sum_j g_j dgate_j) / S_t * s (1 - s)
 *   dz_row         device [P_max] fp32 out: dz of row (t, k) at that row
 * The dot products are summed in fp32 in a fixed order (deterministic).
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes, d % 8 != 0.
 * ---------------------------------------------------------------------- */
moe_status moe_combine_backward(const void* grad_out, moe_dtype g_t, const void* y, moe_dtype y_t,
                                const int32_t* inv_row, const float* topk_gate, const float* topk_score,
                                const int32_t* seg_offset, int T, int d, int K, int Nr, int Ns,
                                void* dy, float* dgate, float* dz, float* dz_row, void* stream);

/* ------------------------------------------------------------------------
 * moe_expert_gemm_backward: gradients of every expert's SwiGLU FFN on its
 * rows (bf16 operands, fp32 accumulation on the matrix cores):
 *   dh = dy W2,  da = dh * b * SiLU'(a),  db = dh * SiLU(a)
 *   dx = [da | db] W13 (per row),  dW2_e = sum_rows dy^T h,
 *   dW13_e = sum_rows [da | db]^T x
 *   x              device [T, d] bf16 tokens of the forward
 *   w13, w2        device bf16 weights as in moe_expert_gemm
 *   h, ab          device, from moe_expert_gemm_train
 *   dy             device [P_max, d] bf16 from moe_combine_backward
 *   ws             device, moe_gemm_backward_workspace_bytes(...) bytes
 *                  (holds [da | db] of every row and the weight-gradient
 *                  kernels' list of experts per XCD)
 *   dx             device [P_max, d] bf16 out (padding rows unwritten)
 *   dw13, dw2      device [Nr+Ns, 2I, d] and [Nr+Ns, d, I] out (overwritten;
 *                  experts with no rows get zeros), dw_t MOE_F32 or MOE_BF16
 * Every output element is summed by one thread in a fixed order.
 *   Errors: MOE_EINVAL for NULL pointers or bad sizes; MOE_EUNSUPPORTED
 *   unless d % 256 == 0, I % 128 == 0 and every operand < 2 GiB;
 *   MOE_EWORKSPACE for a small ws.
 * ---------------------------------------------------------------------- */
size_t moe_gemm_backward_workspace_bytes(int T, int K, int Nr, int Ns, int d, int I, int tile_m);
moe_status moe_expert_gemm_backward(const void* x, const void* w13, const void* w2,
                                    const void* h, const void* ab, const void* dy,
                                    int T, int K, int Nr, int Ns, int d, int I, int tile_m,
                                    const int32_t* seg_offset, const int32_t* row_token,
                                    const int32_t* tile_map, const int32_t* n_tiles,
                                    void* ws, size_t ws_bytes, void* dx,
                                    void* dw13, void* dw2, moe_dtype dw_t, void* stream);

/* ------------------------------------------------------------------------
 * moe_expert_gemm_backward_w8: moe_expert_gemm_backward with the two
 * input-gradient products on E4M3 operands, after [RG-FP8] (E4M3
 * everywhere, 1x128 tiles for activations, 128x128 blocks for weights):
 * dy and then [da | db] are quantised in 1x128
 * tiles along their K axis (d, 2I) with power-of-two scales, and multiply
 * the E4M3 weights of the forward, block-scaled E8M0 on the matrix cores:
 *   dh = Q(dy) Q(W2),  dx = Q([da | db]) Q(W13)
 * The weight gradients are those of moe_expert_gemm_backward (bf16 dy,
 * [da | db], h, x): their K axis is the token axis, for which the pages give
 * no tiling.  x is the expert input as the forward multiplied it: the bf16
 * u after a bf16 forward; after the E4M3 forward (moe_expert_gemm_train_w8)
 * Q(u) decoded by fp8_dequantize_tiles, so that dW13 = [da | db]^T Q(u) is
 * the gradient through a straight-through quantiser.  Codes of dy and
 * [da | db] are decided from their bf16 values.
 *   w13, w13_scale device E4M3 [Nr+Ns, 2I, d] with fp32 [Nr+Ns, 2I/128,
 *                  d/128] block scales, w2, w2_scale [Nr+Ns, d, I] with
 *                  [Nr+Ns, d/128, I/128] (as fp8_quantize_tiles writes them
 *                  with 128x128 tiles; powers of two)
 *   ws             device, moe_gemm_backward_w8_workspace_bytes(...) bytes
 *   every other argument as moe_expert_gemm_backward
 *   Errors: as moe_expert_gemm_backward; MOE_EUNSUPPORTED also for
 *   d > 16384 or I > 8192.
 * ---------------------------------------------------------------------- */
size_t moe_gemm_backward_w8_workspace_bytes(int T, int K, int Nr, int Ns, int d, int I, int tile_m);
moe_status moe_expert_gemm_backward_w8(const void* x, const uint8_t* w13, const float* w13_scale,
                                       const uint8_t* w2, const float* w2_scale,
                                       const void* h, const void* ab, const void* dy,
                                       int T, int K, int Nr, int Ns, int d, int I, int tile_m,
                                       const int32_t* seg_offset, const int32_t* row_token,
                                       const int32_t* tile_map, const int32_t* n_tiles,
                                       void* ws, size_t ws_bytes, void* dx,
                                       void* dw13, void* dw2, moe_dtype dw_t, void* stream);

/* ------------------------------------------------------------------------
 * moe_expert_gemm_backward_f8: moe_expert_gemm_backward_w8 with the two
 * weight-gradient products on E4M3 operands too, so that every product of
 * the backward is E4M3 ([RG-FP8]: E4M3 for all tensors).  Their K axis is
 * the token axis: both operands are quantised in runs of 128 rows of one
 * expert per column (fp8_quantize_runs), each run and column with its
 * power-of-two scale, and multiply on the block-scaled matrix cores:
 *   dW2_e  = R(dy_e)^T R(h_e),  dW13_e = R([da | db]_e)^T R(x_e)
 * (fp32 accumulation).  dy and [da | db] are quantised from their bf16
 * values; h and x are the bf16 operands of the forward (after the E4M3
 * forward: the decoded E4M3 h and Q(u), exact in bf16), quantised again
 * along the tokens.  dx as in moe_expert_gemm_backward_w8.  dy and
 * [da | db] are each read once for both of their E4M3 layouts (the 1x128
 * tiles of the input-gradient products and the token runs).
 *   ws  device, moe_gemm_backward_f8_workspace_bytes(...) bytes
 *   every other argument as moe_expert_gemm_backward_w8
 *   Errors: as moe_expert_gemm_backward_w8.
 * ---------------------------------------------------------------------- */
size_t moe_gemm_backward_f8_workspace_bytes(int T, int K, int Nr, int Ns, int d, int I, int tile_m);
moe_status moe_expert_gemm_backward_f8(const void* x, const uint8_t* w13, const float* w13_scale,
                                       const uint8_t* w2, const float* w2_scale,
                                       const void* h, const void* ab, const void* dy,
                                       int T, int K, int Nr, int Ns, int d, int I, int tile_m,
                                       const int32_t* seg_offset, const int32_t* row_token,
                                       const int32_t* tile_map, const int32_t* n_tiles,
                                       void* ws, size_t ws_bytes, void* dx,
                                       void* dw13, void* dw2, moe_dtype dw_t, void* stream);

/* ------------------------------------------------------------------------
 * moe_route_backward: the layer's input and centroid gradients.
 *   du_t = G_t + sum of dx over the token's shared and routed rows
 *          + sum_k dz[t,k] e_{topk_idx[t,k]}           (fp32, that order)
 *   de_i = sum over the rows of segment i, in row order, of dz_row * u_t
 *   grad_out, g_t  device [T, d] G, MOE_F32 or MOE_BF16
 *   dx             device [P_max, d] bf16 from moe_expert_gemm_backward
 *   u, u_t         device [T, d] tokens, MOE_F32 or MOE_BF16
 *   centroids      device [Nr, d] fp32
 *   topk_idx, inv_row, dz: device [T, K]; dz_row device [P_max]
 *   seg_offset, row_token: from moe_permute
 *   du, du_t       device [T, d] out, MOE_F32 or MOE_BF16
 *   de             device [Nr, d] fp32 out (overwritten)
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes, d % 8 != 0.
 * ---------------------------------------------------------------------- */
moe_status moe_route_backward(const void* grad_out, moe_dtype g_t, const void* dx,
                              const void* u, moe_dtype u_t, const float* centroids,
                              const int32_t* topk_idx, const int32_t* inv_row,
                              const float* dz, const float* dz_row,
                              const int32_t* seg_offset, const int32_t* row_token,
                              int T, int d, int K, int Nr, int Ns,
                              void* du, moe_dtype du_t, float* de, void* stream);

/* ========================================================================
 * Entering the layer: the root-mean-square norm of a pre-norm block.
 * ====================================================================== */

/* ------------------------------------------------------------------------
 * moe_rmsnorm: residual addition, root-mean-square norm and E4M3 tiles in
 * one pass over the rows:
 *   r = x + resid,  c = (mean_j r_j^2 + eps)^(-1/2),  u_j = r_j c w_j
 * in fp32 (sum of squares included); each output is rounded once, from the
 * fp32 value (u and the codes from the unrounded r).
 *   x, x_t       device [T, d], MOE_F32 or MOE_BF16
 *   resid, r_t   device [T, d] or NULL (r = x), MOE_F32 or MOE_BF16
 *   weight, w_t  device [d], MOE_F32 or MOE_BF16
 *   eps          finite, >= 0
 *   r_out        device [T, d] out of type r_t, or NULL; may be resid, or x
 *                where x_t == r_t (r_t is not read when resid and r_out are
 *                NULL)
 *   u, u_t       device [T, d] out, MOE_F32 or MOE_BF16, or NULL when q is
 *                given; may be x where x_t == u_t
 *   q, q_scale   device [T, d] uint8 and [T, d/128] fp32 out: u in 1x128
 *                E4M3 tiles by the rule of fp8_quantize_tiles, or both NULL
 *   rstd         device [T] fp32 out: c, for moe_rmsnorm_backward; or NULL
 * A row of zeros with eps == 0 gives NaN, as the formula does.  A row whose
 * sum of squares passes the fp32 range (values of about 2^64 / sqrt(d) and
 * more) gives c = 0 and u = 0; with eps == 0 one whose squares all fall below
 * it (values under 2^-75) gives c = infinity.  A NaN or an infinity stays in
 * its own row.
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes or types, d % 8 != 0 (d %
 *   128 != 0 with q), a misaligned tensor; MOE_EUNSUPPORTED for d >
 *   MOE_NORM_MAX_D.  T == 0 is valid: nothing is written.
 * ---------------------------------------------------------------------- */
moe_status moe_rmsnorm(const void* x, moe_dtype x_t, const void* resid, moe_dtype r_t,
                       const void* weight, moe_dtype w_t, float eps, long long T, int d,
                       void* r_out, void* u, moe_dtype u_t, uint8_t* q, float* q_scale,
                       float* rstd, void* stream);

/* ------------------------------------------------------------------------
 * moe_rmsnorm_backward: gradients of moe_rmsnorm, with xhat = r c and
 * g = du w:
 *   dx_j = dr_j + c (g_j - xhat_j mean_i(g_i xhat_i))   (of x and of resid)
 *   dw_j = sum_t du_tj xhat_tj
 * in fp32.  Codes q carry no gradient of their own: du is the gradient of u
 * (straight through the quantiser).
 *   du, du_t     device [T, d], MOE_F32 or MOE_BF16
 *   r, r_t       device [T, d], MOE_F32 or MOE_BF16: r_out of the forward (x
 *                when it had no residual)
 *   weight, w_t  device [d]; rstd device [T] fp32 from the forward
 *   dr           device [T, d] of type r_t: gradient that reaches r along the
 *                residual stream, or NULL (zero)
 *   dx           device [T, d] of type r_t out; may be dr, or du where
 *                du_t == r_t
 *   dw           device [d] fp32 out (overwritten), summed in a fixed order
 *   ws           device, moe_rmsnorm_backward_workspace_bytes(T, d) bytes
 *   Errors: as moe_rmsnorm; MOE_EWORKSPACE for a small ws.  T == 0 is valid:
 *   dw is zeroed.
 * ---------------------------------------------------------------------- */
size_t moe_rmsnorm_backward_workspace_bytes(long long T, int d);
moe_status moe_rmsnorm_backward(const void* du, moe_dtype du_t, const void* r, moe_dtype r_t,
                                const void* weight, moe_dtype w_t, const float* rstd,
                                const void* dr, long long T, int d, void* dx, float* dw,
                                void* ws, size_t ws_bytes, void* stream);

/* ========================================================================
 * 4-bit weights.  A value is an E2M1 code (sign, two exponent bits with bias
 * 1, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) times
 * 2^(b - 127), b a byte that 32 consecutive columns of a row share (b = 255:
 * NaN).  Two codes to a byte, the even column in the low half; rows of q are
 * cols / 2 bytes, rows of scale cols / 32 bytes.
 * ====================================================================== */

/* ------------------------------------------------------------------------
 * fp4_quantize_groups: per group of 32 the smallest 2^k (k >= -126) with
 * amax <= 6 * 2^k (k = 0 for a group of zeros), b = k + 127, and code =
 * round-to-nearest-even(x / 2^k): the rule of fp8_quantize_tiles for this
 * format; finite input never saturates.  A group that holds an infinity or a
 * NaN, which the codes cannot hold, gets b = 255 and codes 0: it reads as NaN.
 *   x, x_t   device [rows, cols], MOE_F32 or MOE_BF16
 *   q        device [rows, cols / 2] uint8 out; scale device [rows, cols / 32]
 *            uint8 out
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes (cols % 32 != 0), x_t.
 * fp4_dequantize_groups: the values, exact in fp32 and in bf16 (for b <= 252).
 * ---------------------------------------------------------------------- */
moe_status fp4_quantize_groups(const void* x, moe_dtype x_t, long long rows, long long cols,
                               uint8_t* q, uint8_t* scale, void* stream);
moe_status fp4_dequantize_groups(const uint8_t* q, const uint8_t* scale, long long rows,
                                 long long cols, void* out, moe_dtype out_t, void* stream);

/* ------------------------------------------------------------------------
 * fp4_matvec: products of a 4-bit weight matrix with a few token rows,
 *   y[t, n] = sum_k x[t, k] W[n, k],  W the values of (q, scale)
 * (fp32 sums in a fixed order, one rounding to y_t).  Made for few tokens,
 * where reading W bounds it; any T is computed, W being read again for every
 * 32 tokens.
 *   x, x_t   device [T, K], MOE_BF16
 *   q, scale device [N, K / 2], [N, K / 32] uint8
 *   y, y_t   device [T, N] out, MOE_F32 or MOE_BF16 (element alignment)
 *   ws       not used, may be NULL: fp4_matvec_workspace_bytes(T, N, K) is 0
 *            for all sizes
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes (K < 32, K % 32 != 0) or
 *   types; MOE_EUNSUPPORTED for fp32 x, K above 2^20, T above 1048560, N
 *   above 2^27.  T == 0 or N == 0 is valid.
 * ---------------------------------------------------------------------- */
size_t fp4_matvec_workspace_bytes(int T, long long N, int K);
moe_status fp4_matvec(const void* x, moe_dtype x_t, const uint8_t* q, const uint8_t* scale, int T,
                      long long N, int K, void* y, moe_dtype y_t, void* ws, size_t ws_bytes,
                      void* stream);

/* ------------------------------------------------------------------------
 * moe_layer_few: the whole layer forward for at most MOE_FEW_TOKENS tokens
 * in one call (a decode step of a few sequences, or a few drafted tokens):
 * the routing of moe_route, the FFNs of moe_expert_gemm and the sum of
 * moe_combine, reading each touched expert's weights once.
 *   u, u_t       device [T, d], MOE_F32 or MOE_BF16
 *   centroids, bias: as moe_route
 *   w_t, w13, w13_scale, w2, w2_scale: as moe_expert_gemm for MOE_F32,
 *                MOE_BF16 and MOE_E4M3 (fp32 block scales); MOE_E2M1: codes
 *                [Nr+Ns, 2I, d/2] and [Nr+Ns, d, I/2] with exponent bytes
 *                [Nr+Ns, 2I, d/32] and [Nr+Ns, d, I/32] (fp4_quantize_groups)
 *   resid, r_t   device [T, d], MOE_F32 or MOE_BF16, added to the output: u
 *                for the combine equation, the stream r of moe_rmsnorm for a
 *                pre-norm block; NULL adds nothing
 *   topk_idx, topk_gate, topk_score (may be NULL), expert_load (may be NULL):
 *                out, as moe_route
 *   ws           device, moe_layer_few_workspace_bytes(...) bytes
 *   out, out_t   device [T, d] out, MOE_F32 or MOE_BF16; may be u or resid of
 *                the same type
 * Supported (u_t, w_t): (F32, F32), and BF16 with BF16, E4M3 or E2M1.  Every
 * sum is fp32 in a fixed order, so results are bitwise reproducible; with
 * bf16 tokens h is rounded to bf16 (the operand of the down projection), y is
 * not rounded.
 *   Errors: MOE_EINVAL for NULL pointers, bad types or sizes (d or I not a
 *   multiple of 8, K, Nr, Ns as moe_route and moe_permute); MOE_EUNSUPPORTED
 *   for T > MOE_FEW_TOKENS, other type pairs, E4M3 with d or I not a multiple
 *   of 128, E2M1 with d or I not a multiple of 32, an expert's matrix, the
 *   centroids or h of 2 GiB or more, min(T K, Nr) + Ns times I / 16 or d / 32
 *   of 2^22 or more; MOE_EWORKSPACE for a small ws.  T == 0 is
 *   valid: expert_load is zeroed.
 * ---------------------------------------------------------------------- */
size_t moe_layer_few_workspace_bytes(int T, int d, int Nr, int Ns, int I, int K, moe_dtype u_t);
moe_status moe_layer_few(const void* u, moe_dtype u_t, const float* centroids, const float* bias,
                         moe_dtype w_t, const void* w13, const void* w13_scale,
                         const void* w2, const void* w2_scale,
                         int T, int d, int Nr, int Ns, int I, int K,
                         const void* resid, moe_dtype r_t,
                         int32_t* topk_idx, float* topk_gate, float* topk_score, int32_t* expert_load,
                         void* ws, size_t ws_bytes, void* out, moe_dtype out_t, void* stream);

/* ========================================================================
 * Latent attention ("DeepSeek-V3 Technical Report" reading guide, Method
 * section 1): the keys and values of a token's heads come from one latent c
 * (dc values) and one rotary key r (dr values) that all heads share,
 *   k_{j,h} = [W^K_h c_j ; r_j],  v_{j,h} = W^V_h c_j
 * with dn values in the first part of a key and dv in a value.  A cache keeps
 * c and r only.  dn, dr, dv and dc are multiples of 8, dn and dv <= 128,
 * dr <= 64, dc <= 512; the rotations are the caller's.  scale is positive and
 * at most 2^127.
 * ====================================================================== */

/* ------------------------------------------------------------------------
 * mla_pages_extend: pages and slots of the tokens that a step adds to the
 * requests of a paged cache, from their lengths.  Request b has seq_len[b]
 * tokens and gets new_len[b] more; its token j lies in page
 * block_table[b, j / page_size], at slot page * page_size + j % page_size.
 * Requests take pages in their order, from the top of the stack of free pages:
 * the i-th page that the step takes is free_pages[n_free - 1 - i].  A request
 * whose tokens need more than table_width pages, more free pages than those
 * before it left (it is counted with them all the same), or rows past N is not
 * served: it gets no page, its length stays and its tokens get slot -1.  A
 * request without new tokens needs none of these and is always served.
 *   seq_len, new_len  device [B] int32 (values below 0 count as 0)
 *   block_table       device [B, table_width] int32, in and out: the first
 *                     ceil(seq_len / page_size) entries of a row are read, the
 *                     entries of new pages are written
 *   free_pages        device [n_list] int32; n_free device [1] int32
 *   seq_len_out, n_free_out  device [B], [1] int32 out; may be seq_len, n_free
 *   n_failed          device [1] int32 out: requests that were not served
 *   cu_new            device [B + 1] int32 out: new tokens before each request
 *   slot, position    device [N] int32 out: of the new tokens, request by
 *                     request; position is the token's place j in its request.
 *                     -1 in both for rows past the last new token
 *   ws                device, mla_pages_workspace_bytes(B) bytes (may be NULL
 *                     for N and B up to 4096)
 * The free list and the tables must hold pages p with 0 <= p and
 * (p + 1) * page_size < 2^31.
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes; MOE_EUNSUPPORTED for B >
 *   MLA_MAX_REQUESTS; MOE_EWORKSPACE for a small ws.  B == 0 and N == 0 are
 *   valid.
 * mla_pages_release: the pages of the requests marked in `done` (device [B]
 * int32, not 0) go back on the stack, request by request, and their lengths
 * become 0; seq_len, free_pages and n_free are updated in place.  Pages past
 * the list's end (n_list entries) are dropped.  Nobody counts a page's owners: a
 * page that the caller has put into several tables (mla_decode reads such) is to
 * be released with one of them.
 * ---------------------------------------------------------------------- */
size_t mla_pages_workspace_bytes(int B);
moe_status mla_pages_extend(const int32_t* seq_len, const int32_t* new_len, int B, int page_size,
                            int32_t* block_table, int table_width, const int32_t* free_pages,
                            int n_list, const int32_t* n_free, int32_t* seq_len_out,
                            int32_t* n_free_out, int32_t* n_failed, int32_t* cu_new,
                            int32_t* slot, int32_t* position, int N, void* ws, size_t ws_bytes,
                            void* stream);
moe_status mla_pages_release(const int32_t* done, int32_t* seq_len, int B, int page_size,
                             const int32_t* block_table, int table_width, int32_t* free_pages,
                             int n_list, int32_t* n_free, void* stream);

/* ------------------------------------------------------------------------
 * mla_cache_write: row slot[t] of the cache becomes [c_t ; r_t].
 *   latent, ld_latent device bf16, T rows of dc values, ld_latent apart
 *   k_rope, ld_rope   device bf16, T rows of dr values, ld_rope apart
 *   slot              device [T] int32; a token whose slot is not in
 *                     [0, n_slots) is not written; slots must be distinct
 *   cache             device [n_slots, dc + dr] bf16 out
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes, strides that are not
 *   multiples of 8; MOE_EUNSUPPORTED for dc > 512 or dr > 64.  T == 0 is valid.
 * ---------------------------------------------------------------------- */
moe_status mla_cache_write(const void* latent, long long ld_latent, const void* k_rope,
                           long long ld_rope, const int32_t* slot, long long T, int dc, int dr,
                           void* cache, long long n_slots, void* stream);

/* ------------------------------------------------------------------------
 * mla_decode: attention of the newest S tokens of each request over its
 * cached tokens (theirs among them), in absorbed form:
 *   q~ = (W^K_h)^T q^n,  s_j = scale (q~ . c_j + q^r . r_j),
 *   o = W^V_h sum_j softmax(s)_j c_j
 * Token i (0 .. S - 1) of request b sees the cached tokens
 * j < seq_len[b] - (S - 1 - i); one that sees none gets zeros.  q~ and, where
 * the work is divided into blocks of 64 rows, the softmax weights are rounded to
 * bf16 as operands (in blocks of 32 they are two bf16 halves); sums, maxima and the join of
 * the parts that one request is split into are fp32, in a fixed order for given
 * lengths, so results are bitwise reproducible.
 *   q            device [B, S, H, dn + dr] bf16, q^n then the rotated q^r
 *   w_kv         device [H, dn + dv, dc] bf16: W^K_h, then W^V_h (the rows of
 *                the projection that gives mla_attention's kv)
 *   cache        device [n_pages, page_size, dc + dr] bf16
 *   block_table  device [B, table_width] int32; seq_len device [B] int32, on
 *                the device: a captured call follows both
 *   max_len      an upper bound on seq_len, by which the work is divided (a
 *                longer request is computed right all the same)
 *   out, out_t   device [B, S, H, dv] out, MOE_F32 or MOE_BF16
 *   ws           device, mla_decode_workspace_bytes(...) bytes
 * A page outside [0, n_pages) among those of a request's tokens, or a length
 * past table_width * page_size or 2^31 - 256, makes the request's outputs NaN; no
 * memory outside the cache is read.  A NaN or an infinity in a cached row reaches the
 * tokens that see it and, with S > 1, may reach those of the same request that
 * do not; it stays in its request.  Memory behind a request's last token does
 * not matter.
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes or types; MOE_EUNSUPPORTED
 *   for sizes above the limits, B > MLA_MAX_REQUESTS, S > 64, H > 1024,
 *   B S H > 2^26 or 2^31 slots; MOE_EWORKSPACE for a small ws.  B == 0 is valid.
 * ---------------------------------------------------------------------- */
size_t mla_decode_workspace_bytes(int B, int S, int H, int dn, int dr, int dv, int dc,
                                  long long max_len);
moe_status mla_decode(const void* q, const void* w_kv, const void* cache, long long n_pages,
                      int page_size, const int32_t* block_table, int table_width,
                      const int32_t* seq_len, int B, int S, int H, int dn, int dr, int dv, int dc,
                      long long max_len, float scale, void* out, moe_dtype out_t, void* ws,
                      size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * mla_attention: attention over B packed sequences in expanded form; rows
 * cu_q[b] .. cu_q[b+1] - 1 of q meet rows cu_k[b] .. cu_k[b+1] - 1 of kv:
 *   s_ij = scale (q^n_i . k_j + q^r_i . r_j),  out_i = sum_j softmax(s_i)_j v_j
 * causal: query i of lq sees keys j <= i + lk - lq (the last query sees all
 * keys).  A query that sees no key gets zeros and lse = -infinity.  The softmax
 * weights are rounded to bf16 for the product with v; sums are fp32 in a fixed
 * order.
 *   q            device [Tq, H, dn + dr] bf16
 *   kv           device [Tk, H, dn + dv] bf16: k, then v of each head
 *   k_rope, ld_rope  device bf16, Tk rows of dr values, ld_rope apart
 *   cu_q, cu_k   device [B + 1] int32, not falling, within [0, Tq] and [0, Tk]
 *   out, out_t   device [Tq, H, dv] out, MOE_F32 or MOE_BF16
 *   lse          device [Tq, H] fp32 out: log sum_j exp(s_ij); or NULL
 * Rows of no sequence are left as they were, and hold anything.  A NaN or an
 * infinity in a key or value reaches the queries that see it, and may reach
 * others of the same sequence and head.
 *   Errors: MOE_EINVAL for NULL pointers, bad sizes or types; MOE_EUNSUPPORTED
 *   for sizes above the limits, B > MLA_MAX_REQUESTS, H > 1024,
 *   (max(Tq, Tk) / 128 + B) H > 2^22 or Tk dr > 2^33.  Tq == 0 and B == 0 are
 *   valid.
 * ---------------------------------------------------------------------- */
moe_status mla_attention(const void* q, const void* kv, const void* k_rope, long long ld_rope,
                         const int32_t* cu_q, const int32_t* cu_k, int B, long long Tq,
                         long long Tk, int H, int dn, int dr, int dv, int causal, float scale,
                         void* out, moe_dtype out_t, float* lse, void* stream);

/* ------------------------------------------------------------------------
 * mla_attention_backward: gradients of mla_attention's out (none flows
 * through lse): with P = exp(s - lse) and D_i = sum_d dout_id out_id,
 *   dv = P^T dout,  dS = P (dout v^T - D),  dq = scale dS k,  dk = scale dS^T q
 * and dk_rope the sum of the rotary columns of dk over the heads.  P and dS are
 * rounded to bf16 as operands; sums are fp32 in a fixed order, so results are
 * bitwise reproducible.
 *   dout         device [Tq, H, dv] bf16
 *   out, out_t, lse: as mla_attention left them
 *   dq, dkv, dk_rope, g_t  device [Tq, H, dn + dr], [Tk, H, dn + dv], [Tk, dr]
 *                out, MOE_F32 or MOE_BF16 (all three); rows of no sequence are
 *                left as they were
 *   ws           device, mla_attention_backward_workspace_bytes(...) bytes: 8 Tq H
 *                for two statistics of a row, 4 H Tk dr for the heads' parts of
 *                dk_rope (dr 64 and 128 heads: 134 MB at 4096 keys, 2.1 GB at 65536)
 *   every other argument as mla_attention
 *   Errors: as mla_attention; MOE_EWORKSPACE for a small ws.  Tq == 0 gives
 *   zeros in dkv and dk_rope.
 * ---------------------------------------------------------------------- */
size_t mla_attention_backward_workspace_bytes(long long Tq, long long Tk, int H, int dr);
moe_status mla_attention_backward(const void* dout, const void* q, const void* kv,
                                  const void* k_rope, long long ld_rope, const void* out,
                                  moe_dtype out_t, const float* lse, const int32_t* cu_q,
                                  const int32_t* cu_k, int B, long long Tq, long long Tk, int H,
                                  int dn, int dr, int dv, int causal, float scale, void* dq,
                                  void* dkv, void* dk_rope, moe_dtype g_t, void* ws,
                                  size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_H */
