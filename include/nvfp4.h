/*
 * nvfp4.h -- C ABI of the B200 (sm_100a) NVFP4 quantizer and block-scaled GEMM.
 *
 * Format, as the pages state it:
 *  - Elements are E2M1 (1 sign, 2 exponent, 1 mantissa bit), 16 values in
 *    [-6, 6] (asector.ru, "Nvidia dobivaetsya uspekha s 4-bitnym formatom
 *    NVFP4", section "NVFP4 and Blackwell"; iitak.ru, "Thinking Machines
 *    uskorila obuchenie Inkling 2 Small 4-bitnymi chislami", section "Details").
 *  - Two-level scaling: one local scale per 16-element block and one global
 *    scale per tensor (asector, "NVFP4 and Blackwell").  The block scale is an
 *    E4M3 byte (this library's choice: the worked multiplier 9 of iitak,
 *    "Details", is not a power of two); the global scale is FP32.
 *  - Optional 16x16 2D block scales for weights, invariant under transpose,
 *    and a random Hadamard transform for outlier gradients (asector,
 *    "Experiments and comparison with FP8"; iitak, "How it works").
 *  - Round-to-nearest-even or unbiased stochastic rounding (asector, "NVFP4
 *    and Blackwell"; iitak, "How it works": 2.25 -> 2 w.p. 3/4, 3 w.p. 1/4).
 *  - MXFP8 requantisation for backward operands: E4M3 elements with one E8M0
 *    scale per 32 (iitak, "How it works" and "But": 8.25 bits per number).
 *
 * Conventions shared by every call:
 *  - Every tensor pointer is a DEVICE pointer owned by the caller.  The
 *    library allocates no device memory; scratch comes from a caller-provided
 *    workspace whose size the *_workspace_size helpers return.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Calls only enqueue work and return; they never synchronise.
 *  - The returned status reports argument and launch errors.  Errors the
 *    device detects (a bounded wait that ran out, a gather index out of range)
 *    are written to a status word in the workspace, which every call that is
 *    given a workspace clears first; nvfp4_workspace_status() synchronises the
 *    stream and returns the word of the last call that used that workspace.
 *  - A workspace serves one call at a time: calls that may overlap on the GPU
 *    (other streams, other captured graphs) take one each.
 *  - Matrices are row-major.  "Rowwise" quantisation blocks 16 consecutive
 *    elements along a row; "columnwise" quantises the transpose, so its codes
 *    are [cols, rows/2] and its 16-blocks run down a column of the input.
 *  - Codes: two E2M1 nibbles per byte, the even element in the low nibble.
 *  - Inputs must be finite; non-finite input gives unspecified codes.
 */
#ifndef NVFP4_H
#define NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NVFP4_OK = 0,
    NVFP4_ERR_INVALID_ARG = 1, /* null pointer, bad enum, inconsistent flags     */
    NVFP4_ERR_SHAPE = 2,       /* size not a multiple of the block or tile       */
    NVFP4_ERR_ALIGN = 3,       /* pointer or leading dimension not 16-byte aligned */
    NVFP4_ERR_UNSUPPORTED = 4, /* no sm_100 device, or an unsupported combination */
    NVFP4_ERR_CUDA = 5,        /* a CUDA runtime call failed                     */
    NVFP4_ERR_TIMEOUT = 6,     /* device side: a bounded wait ran out            */
    NVFP4_ERR_WORKSPACE = 7,   /* workspace missing or too small                 */
    NVFP4_ERR_INDEX = 8        /* device side: a gather index was out of range   */
} nvfp4_status;

enum { NVFP4_RNE = 0, NVFP4_SR = 1 };                 /* rounding          */
enum { NVFP4_1D16 = 0, NVFP4_2D16x16 = 1 };           /* block scaling     */
enum { NVFP4_ROWWISE = 1, NVFP4_COLWISE = 2 };        /* output bitmask    */
enum { NVFP4_SF_ROWMAJOR = 0, NVFP4_SF_MMA = 1 };     /* scale-byte layout */
enum { NVFP4_OUT_F32 = 0, NVFP4_OUT_BF16 = 1 };       /* GEMM / dequant output */
enum { NVFP4_SOFTMAX = 0, NVFP4_SIGMOID = 1 };        /* routing scores    */

/*
 * Scale-byte layouts.
 *  NVFP4_SF_ROWMAJOR: scale of 16-block b of row r at sf[r * (K/16) + b],
 *    where K is the length of the quantised rows (cols rowwise, rows
 *    columnwise).  In 2D mode the byte of each 16x16 tile is stored in all 16
 *    rows' entries, so the shapes stay those of 1D.
 *  NVFP4_SF_MMA: the tiled layout the tensor cores read.  Rows are grouped in
 *    blocks of 128 and 16-blocks in groups of 4 (64 elements); each group is a
 *    512-byte atom, atoms ordered with the K group fastest:
 *      offset = ((r/128) * (K/64) + b/4) * 512 + (r%32)*16 + ((r%128)/32)*4 + b%4.
 *    Buffers must hold ceil(rows/128)*128 rows (bytes = nvfp4_sf_mma_bytes);
 *    bytes of padding rows are not written.  K must be a multiple of 64.
 *  With group_offsets (MoE layout), each group e's rows start a fresh
 *    128-row block: row r of group e uses padded row
 *    r - off[e] + sum_{e'<e} ceil((off[e'+1]-off[e'])/128)*128.
 */

/* Stochastic-rounding bits come from Philox4x32-10 (Salmon et al., SC'11),
 * key = seed (low word, high word).  idx is the element's position in the
 * OUTPUT's row-major order (for columnwise outputs, the transpose's order).
 *
 * NVFP4 codes (stream 0 = rowwise, 1 = columnwise).  The pages say stochastic
 * rounding is built into Blackwell (asector, "NVFP4 and Blackwell"); the
 * library feeds that built-in conversion, which consumes one 32-bit random word
 * per 4 consecutive elements.  Element idx uses word (idx/4) % 4 of
 * Philox(counter = (idx/16 low word, idx/16 high word, stream, offset)), and
 * element k = idx % 4 of that 4-group draws the 16-bit value
 *     u = 65535 - v,  v (high byte : low byte) =
 *         k = 0: B2 : B0          k = 1: rev(B0) : rev(B2)
 *         k = 2: B3 : B1          k = 3: rev(B1) : rev(B3)
 * where B0..B3 are the word's bytes (B0 least significant) and rev reverses
 * the bit order of a byte.  The element rounds up iff u < floor(f * 2^16), f
 * its position between its two grid neighbours, so each element rounds up
 * with probability exactly floor(f * 2^16) / 2^16.  Elements 4g, 4g+1 (and
 * 4g+2, 4g+3) read the same two bytes: their decisions are not independent,
 * though the covariance of any two of them is at most 5.5 / 2^16.
 *
 * MXFP8 codes (stream 2): 16 bits per element, element idx taking the
 * 16-bit half (idx % 2) of word (idx % 8) / 2 of Philox(counter = (idx/8 low
 * word, idx/8 high word, 2, offset)); up iff that value is below
 * floor(f * 2^16) on the E4M3 grid.
 *
 * The Hadamard signs are bits 0..15 of word 0 of Philox(counter (0,0,3,0),
 * key = seed): they depend on the seed only, so two tensors quantised with one
 * seed share the transform and it cancels in their product. */
typedef struct {
    int rounding;          /* NVFP4_RNE | NVFP4_SR (NVFP4 codes, both directions) */
    int scaling;           /* NVFP4_1D16 | NVFP4_2D16x16                        */
    int outputs;           /* NVFP4_ROWWISE | NVFP4_COLWISE bitmask (may be 0)  */
    int rht_colwise;       /* 1: 16-point random Hadamard on columnwise vectors  */
    int sf_layout;         /* NVFP4_SF_ROWMAJOR | NVFP4_SF_MMA                   */
    uint64_t seed;         /* Philox key                                         */
    uint32_t offset;       /* Philox counter word 3: selects a sub-stream        */
    const float* amax_in;  /* optional device [2] = {amax rowwise, amax columnwise
                              (after the Hadamard when rht_colwise)}; NULL = compute */
    /* Gather (MoE): output row i reads input row row_index[i]; the input has
     * src_rows rows.  NULL = identity (src_rows ignored). */
    const int32_t* row_index;
    int64_t src_rows;
    /* MoE scale layout: device offsets [num_groups+1] of output rows; only with
     * NVFP4_SF_MMA and the rowwise output; 1 <= num_groups <= 256.  NULL = dense. */
    const int32_t* group_offsets;
    int num_groups;
    /* Optional MXFP8 copy produced in the same pass (E4M3 codes [rows, cols] /
     * [cols, rows] with E8M0 scales per 32 along the block axis, row-major). */
    int mx_outputs;        /* NVFP4_ROWWISE | NVFP4_COLWISE bitmask, 0 = none    */
    int mx_rounding;       /* NVFP4_RNE | NVFP4_SR (stream 2)                    */
    uint8_t* mx_q_row;
    uint8_t* mx_sf_row;
    uint8_t* mx_q_col;
    uint8_t* mx_sf_col;
    /* Layout of the MXFP8 scale bytes: NVFP4_SF_ROWMAJOR ([rows, K/32]) or
     * NVFP4_SF_MMA, the 128x4 atoms of the NVFP4 tiled layout with 32-element
     * blocks (byte of block b of row r at ((r/128)*(K/128) + b/4)*512 +
     * (r%32)*16 + ((r%128)/32)*4 + b%4; bytes = mxfp8_sf_mma_bytes), which
     * mxfp8_gemm reads.  NVFP4_SF_MMA needs the block axis a multiple of 128. */
    int mx_sf_layout;
} nvfp4_quant_params;

/* Bytes of scale storage in NVFP4_SF_MMA layout for a [rows, k] operand. */
size_t nvfp4_sf_mma_bytes(int64_t rows, int64_t k);

/* Bytes of MXFP8 scale storage in NVFP4_SF_MMA layout for a [rows, k] operand
 * (one E8M0 byte per 32 elements; ceil(rows/128)*128 rows). */
size_t mxfp8_sf_mma_bytes(int64_t rows, int64_t k);

/* Bytes of scale storage in NVFP4_SF_MMA layout for the grouped (MoE) layout:
 * sum over groups of ceil(rows_e/128)*128 rows; bounded by
 * (total_rows + 128*num_groups) rows, which this returns. */
size_t nvfp4_sf_mma_grouped_bytes(int64_t total_rows, int num_groups, int64_t k);

/* Workspace bytes nvfp4_quantize needs (global amax and the status word). */
size_t nvfp4_quantize_workspace_size(int64_t rows, int64_t cols, const nvfp4_quant_params* p);

/*
 * nvfp4_quantize -- NVFP4 quantisation of a bf16 matrix x [rows, ld] (row-major,
 * cols <= ld), rowwise and/or columnwise in one pass over the data, plus an
 * optional MXFP8 copy.
 *
 * Steps (asector "NVFP4 and Blackwell" / "Experiments and comparison with
 * FP8"; iitak "Details" / "How it works"):
 *   amax (per direction; over the transformed values when rht_colwise),
 *   S = 2688/amax and g = amax/2688 (FP32 divisions; amax 0 -> 1, 1; S capped
 *   at 2^118 with g = 2^-118), block amax over 16 (1D) or 16x16 (2D),
 *   scale byte = E4M3_RNE_satfinite((amax_b / 6) * S), d = its value,
 *   y = x * (S / d), code = RNE or SR of y onto E2M1 (saturating at 6;
 *   d = 0 gives +-0 codes).
 *
 * Outputs (NULL when that direction is not requested):
 *   q_row  [rows, cols/2] codes,  sf_row scales,  g_row [1] FP32 decode scale;
 *   q_col  [cols, rows/2] codes,  sf_col scales,  g_col [1].
 * Shapes: rows, cols multiples of 16; MXFP8 needs its block axis a multiple
 * of 32; NVFP4_SF_MMA needs the quantised length a multiple of 64.
 * Alignment: x and ld*2 bytes 16-byte aligned; outputs 16-byte aligned.
 * Returns NVFP4_ERR_SHAPE / _ALIGN / _INVALID_ARG / _WORKSPACE before any
 * launch, NVFP4_ERR_CUDA if a launch fails.
 */
nvfp4_status nvfp4_quantize(const void* x_bf16, int64_t rows, int64_t cols, int64_t ld,
                            const nvfp4_quant_params* p, uint8_t* q_row, uint8_t* sf_row,
                            float* g_row, uint8_t* q_col, uint8_t* sf_col, float* g_col,
                            void* workspace, size_t ws_bytes, void* stream);

/*
 * nvfp4_quantize_noalloc -- nvfp4_quantize for callers that cannot supply a
 * workspace.  (The pages have no counterpart: this is an interface
 * convenience, not part of the method.)
 *
 * Who needs it: code that may not allocate device memory at the point of the
 * call -- for example a host framework whose GPU memory is entirely reserved
 * by its own caching allocator, or a latency-critical path that must never
 * reach cudaMalloc, which can synchronise the whole device.
 *
 * Behaviour: identical results to nvfp4_quantize.  The quantiser's scratch
 * (the two amax words and the device status word, 12 bytes for any tensor
 * size) lives in a 256-byte array compiled into the library; every GPU that
 * loads the library keeps that array until the process exits.  The call
 * allocates nothing and calls no allocating routine.
 *  - Maximum: the scratch a call needs (nvfp4_quantize_workspace_size) must fit
 *    in the 256-byte array, otherwise NVFP4_ERR_WORKSPACE and nothing is
 *    launched.  Today's quantiser needs 256 bytes for every accepted shape.
 *  - The first call on each device looks up the array's device address (with
 *    that device current); make that first call before any stream capture.
 *  - All calls share the one array, and each clears it before use: calls that
 *    may overlap on the GPU (different streams, or concurrent host threads)
 *    race on it and must be serialised by the caller.  Device-side errors (a
 *    gather index out of range, a bounded wait that ran out) land in the
 *    array's status word; nvfp4_quantize_noalloc_status reads it.
 *  - If the address lookup fails (NVFP4_ERR_CUDA), nothing is launched and the
 *    next call tries the lookup again.
 */
nvfp4_status nvfp4_quantize_noalloc(const void* x_bf16, int64_t rows, int64_t cols, int64_t ld,
                                    const nvfp4_quant_params* p, uint8_t* q_row, uint8_t* sf_row,
                                    float* g_row, uint8_t* q_col, uint8_t* sf_col, float* g_col,
                                    void* stream);

/*
 * nvfp4_quantize_noalloc_status -- the device status word of the most recent
 * nvfp4_quantize_noalloc call on the current device (NVFP4_OK,
 * NVFP4_ERR_TIMEOUT or NVFP4_ERR_INDEX), read after synchronising `stream`,
 * then cleared; the same contract as nvfp4_workspace_status, for the array
 * compiled into the library.  It allocates nothing.  (No counterpart in the
 * pages either.)
 */
nvfp4_status nvfp4_quantize_noalloc_status(void* stream);

/*
 * mxfp8_quantize -- MXFP8 (iitak, "How it works" and "But"): per 32-element
 * block e = clamp(floor(log2 amax) - 8, -127, 127) (OCP MX v1.0 rule),
 * E8M0 byte e + 127 (amax 0 -> byte 0), element = E4M3 of x * 2^-e, RNE
 * satfinite or SR (Philox stream 2).
 * directions: NVFP4_ROWWISE (codes [rows, cols], scales [rows, cols/32]) and/or
 * NVFP4_COLWISE (codes [cols, rows], scales [cols, rows/32]).  The block axis
 * must be a multiple of 32, the other a multiple of 16 (any row count for
 * NVFP4_ROWWISE alone).
 */
nvfp4_status mxfp8_quantize(const void* x_bf16, int64_t rows, int64_t cols, int64_t ld,
                            int directions, int rounding, uint64_t seed, uint32_t offset,
                            uint8_t* q_row, uint8_t* e8_row, uint8_t* q_col, uint8_t* e8_col,
                            void* stream);

/*
 * mxfp4_quantize -- MXFP4, the Open Compute Project 4-bit format the pages
 * compare NVFP4 against (hightech; asector, "NVFP4 and Blackwell" and the
 * comparison with MXFP4).  The pages do not restate it; the OCP MX v1.0 rule
 * is used: per 32-element block e = clamp(floor(log2 amax) - 2, -127, 127)
 * (2 = largest E2M1 exponent), E8M0 byte e + 127 (amax 0 -> byte 0), element =
 * E2M1 of x * 2^-e, round-to-nearest-even saturating at +-6.  No tensor scale.
 * Codes two per byte, even index in the low nibble.
 * directions: NVFP4_ROWWISE (codes [rows, cols/2], scales [rows, cols/32])
 * and/or NVFP4_COLWISE (codes [cols, rows/2], scales [cols, rows/32]); both
 * come from one read of x.  sf_layout: NVFP4_SF_ROWMAJOR, or NVFP4_SF_MMA (the
 * 128x4 atoms of 32-blocks that mxfp4_gemm reads; bytes = mxfp8_sf_mma_bytes
 * of the same shape; the block axis a multiple of 128).  rows and cols
 * multiples of 32 (NVFP4_ERR_SHAPE);
 * x, q_row, q_col 16-byte aligned and ld a multiple of 8 (NVFP4_ERR_ALIGN);
 * a requested direction with a NULL output -> NVFP4_ERR_INVALID_ARG.  All
 * buffers are device memory owned by the caller; asynchronous on `stream`.
 */
nvfp4_status mxfp4_quantize(const void* x_bf16, int64_t rows, int64_t cols, int64_t ld,
                            int directions, int sf_layout, uint8_t* q_row, uint8_t* e8_row,
                            uint8_t* q_col, uint8_t* e8_col, void* stream);

/*
 * nvfp4_gather_rows -- MoE dispatch of quantised rows (iitak, "Details" and
 * "But": tokens travel to the expert layers, where NVFP4 is used).  Output row
 * i is source row row_index[i]: its codes [k/2 bytes] and its scale bytes,
 * moved from the dense NVFP4_SF_MMA layout of a [src_rows, k] operand into the
 * grouped NVFP4_SF_MMA layout of group_offsets (device [num_groups+1],
 * 1 <= num_groups <= 256), or into the dense layout when group_offsets is NULL.
 * Quantising the tokens once and gathering gives the same bytes as quantising
 * the gathered rows whenever every token is routed at least once (the global
 * scale then comes from the same amax).  k a multiple of 64, at most 2^28; q_src, q_dst
 * 16-byte aligned, scale pointers 4-byte aligned.  Out-of-range indices are
 * reported in the workspace status word (optional workspace).
 */
nvfp4_status nvfp4_gather_rows(const uint8_t* q_src, const uint8_t* sf_src, int64_t src_rows,
                               int64_t k, const int32_t* row_index, int64_t rows,
                               const int32_t* group_offsets, int num_groups, uint8_t* q_dst,
                               uint8_t* sf_dst, void* workspace, size_t ws_bytes, void* stream);

/*
 * nvfp4_dequantize -- the value an NVFP4 tensor stands for: each 4-bit element
 * times its block's scale times the tensor's global scale (asector, "NVFP4 and
 * Blackwell": a local scale per 16-element block on top of one scale per
 * tensor; iitak, "Details": -6 times the multiplier 9 gives back -54).
 * Computed as x_hat = (e2m1(code) * d) * g, the first product exact, one FP32
 * rounding, then (for NVFP4_OUT_BF16) RNE to bf16.
 * q [rows, cols/2], sf in sf_layout, g device [1]; out [rows, cols].
 */
nvfp4_status nvfp4_dequantize(const uint8_t* q, const uint8_t* sf, const float* g, int64_t rows,
                              int64_t cols, int sf_layout, int out_dtype, void* out,
                              void* stream);

/* Workspace bytes nvfp4_gemm / nvfp4_grouped_gemm / mxfp8_gemm / mxfp4_gemm
 * need: the status word (bytes 8..11) and the call's SM cycle count (bytes
 * 16..23), both cleared by every call. */
size_t nvfp4_gemm_workspace_size(int64_t M, int64_t N, int64_t K);

/*
 * nvfp4_gemm_cycles -- measurement aid (no counterpart in the pages): the SM
 * clock cycles, kernel entry to exit, of the longest-running CTA of the last
 * GEMM call that used `workspace`.  Divided by that call's CUDA-event time it
 * gives the SM clock the call actually ran at (the power limit lowers it under
 * dense FP4 work, which the driver's clock readout does not show).
 * Synchronises `stream`; *cycles is host memory.  NVFP4_ERR_INVALID_ARG for a
 * null workspace or output pointer.
 */
nvfp4_status nvfp4_gemm_cycles(void* workspace, void* stream, uint64_t* cycles);

/*
 * nvfp4_gemm -- block-scaled NVFP4 GEMM on the tcgen05 tensor cores
 * (asector, "NVFP4 and Blackwell": scaled computation with high-precision
 * accumulation):
 *   D[i][j] = ga * gb * sum_k (e2m1(a_ik) * sa(i, k/16)) * (e2m1(b_jk) * sb(j, k/16))
 * with FP32 accumulation.  "TN": A [M, K] and B [N, K] are both K-contiguous
 * codes (qa [M, K/2], qb [N, K/2]); scales sfa / sfb in NVFP4_SF_MMA layout;
 * ga, gb device FP32 [1].  D [M, ldd] FP32 or bf16 (RNE), row-major.
 * amax_out: optional device FP32 [1]; the call sets it to max |D| over the
 * stored values (after rounding to the output type), so the next NVFP4
 * quantisation of D can take it as amax_in and skip its amax pass.
 * Shapes: K a multiple of 256 (one pipeline stage), M and N multiples of 16;
 * ldd >= N with ldd * element size a multiple of 16 bytes.
 */
nvfp4_status nvfp4_gemm(const uint8_t* qa, const uint8_t* sfa, const float* ga,
                        const uint8_t* qb, const uint8_t* sfb, const float* gb, int64_t M,
                        int64_t N, int64_t K, int out_dtype, void* D, int64_t ldd,
                        float* amax_out, void* workspace, size_t ws_bytes, void* stream);

/*
 * mxfp8_gemm -- block-scaled MXFP8 GEMM on the tcgen05 tensor cores, for the
 * backward pass of the recipe on the iitak page ("How it works": the backward
 * pass runs in 8-bit MXFP8; "But": 8 bits per element plus one 8-bit scale per
 * 32, 8.25 bits per number):
 *   D[i][j] = sum_k (e4m3(a_ik) * 2^(ea(i, k/32) - 127)) * (e4m3(b_jk) * 2^(eb(j, k/32) - 127))
 * with FP32 accumulation, no tensor scale.  "TN": qa [M, K] and qb [N, K] E4M3
 * codes (one byte each, K-contiguous); sfa / sfb E8M0 bytes in the
 * NVFP4_SF_MMA layout with 32-element blocks (mx_sf_layout of
 * nvfp4_quant_params).  D [M, ldd] FP32 or bf16 (RNE); amax_out as for
 * nvfp4_gemm.  Shapes: K a multiple of 128 (one pipeline stage), M and N
 * multiples of 16; ldd >= N with ldd * element size a multiple of 16 bytes;
 * every pointer 16-byte aligned (amax_out 4).  Errors as for nvfp4_gemm.
 */
nvfp4_status mxfp8_gemm(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb,
                        const uint8_t* sfb, int64_t M, int64_t N, int64_t K, int out_dtype,
                        void* D, int64_t ldd, float* amax_out, void* workspace, size_t ws_bytes,
                        void* stream);

/*
 * mxfp4_gemm -- block-scaled MXFP4 GEMM on the tcgen05 tensor cores
 * (kind::mxf4), the OCP format the pages compare NVFP4 against (hightech;
 * asector, "NVFP4 and Blackwell"):
 *   D[i][j] = sum_k (e2m1(a_ik) * 2^(ea(i, k/32) - 127)) * (e2m1(b_jk) * 2^(eb(j, k/32) - 127))
 * with FP32 accumulation, no tensor scale.  "TN": qa [M, K/2], qb [N, K/2]
 * E2M1 codes (even element in the low nibble); sfa / sfb E8M0 bytes in the
 * tiled layout of mxfp4_quantize(..., NVFP4_SF_MMA, ...).  D [M, ldd] FP32 or
 * bf16 (RNE); amax_out as for nvfp4_gemm.  Shapes: K a multiple of 256, M and
 * N multiples of 16, ldd >= N with ldd * element size a multiple of 16 bytes;
 * pointers 16-byte aligned (amax_out 4).  Errors as for nvfp4_gemm.
 */
nvfp4_status mxfp4_gemm(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb,
                        const uint8_t* sfb, int64_t M, int64_t N, int64_t K, int out_dtype,
                        void* D, int64_t ldd, float* amax_out, void* workspace, size_t ws_bytes,
                        void* stream);

/*
 * nvfp4_grouped_gemm -- MoE grouped form (iitak, "Details": NVFP4 in the
 * expert layers): rows [off[e], off[e+1]) of the stacked A [total_rows, K]
 * are multiplied by expert e's B_e [N, K]:
 *   D[i][j] = ga * gb[e] * sum_k a_hat_ik b_hat_e,jk.
 * 1 <= G <= 256.  group_offsets: device int32 [G+1], non-decreasing, off[0] = 0,
 * off[G] = total_rows.  sfa in the grouped NVFP4_SF_MMA layout (see above);
 * qb [G, N, K/2], sfb [G] consecutive NVFP4_SF_MMA blocks of N rows each,
 * gb device [G].  D [total_rows, N] row-major; amax_out as for nvfp4_gemm.
 * The tile schedule is computed on the device from group_offsets: the host
 * never reads the offsets.
 */
nvfp4_status nvfp4_grouped_gemm(int G, const int32_t* group_offsets, int64_t total_rows,
                                const uint8_t* qa, const uint8_t* sfa, const float* ga,
                                const uint8_t* qb, const uint8_t* sfb, const float* gb,
                                int64_t N, int64_t K, int out_dtype, void* D, float* amax_out,
                                void* workspace, size_t ws_bytes, void* stream);

/*
 * mxfp8_combine -- the receiving end of the MXFP8-compressed expert combine
 * (iitak, "But": expert outputs travel at 8.25 bits per number instead of 16).
 * q [rows, cols] E4M3 codes and e8 [rows, cols/32] row-major E8M0 scales are the
 * expert-output rows this rank received (mxfp8_quantize rowwise on the sender);
 * token t's k rows are slot_row[t*k + j] (device int32, -1 = no row) with
 * routing weights weight[t*k + j] (device FP32).  Computes, in FP32 with one
 * rounding per product and per sum, j in order,
 *   out[t][c] = sum_j weight[t][j] * (e4m3(q[r][c]) * 2^(e8[r][c/32] - 127)),
 * then RNE to bf16 into out_bf16 [tokens, cols].  cols a multiple of 32;
 * 1 <= k <= 64; q and out 16-byte aligned.  A row index >= rows is
 * skipped and reported in the optional workspace's status word
 * (NVFP4_ERR_INDEX).  Asynchronous on `stream`; allocates nothing.
 */
nvfp4_status mxfp8_combine(const uint8_t* q, const uint8_t* e8, int64_t rows, int64_t cols,
                           const int32_t* slot_row, const float* weight, int64_t tokens, int k,
                           void* out_bf16, void* workspace, size_t ws_bytes, void* stream);

/*
 * nvfp4_rmsnorm -- root-mean-square norm with the residual's addition, in bf16
 * or as the MXFP8 operand of mxfp8_gemm, in one pass over the data.  (The pages
 * name no norm; it is the step before the layers they quantise.)
 *   h = bf16(x + residual)    (h = x without a residual)
 *   rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * weight   (FP32)
 * x, residual [rows, ld] bf16; weight [cols] of weight_dtype (NVFP4_OUT_F32 or
 * NVFP4_OUT_BF16).  Outputs, each only where its pointer is given:
 *   h [rows, ldh] bf16 (with a residual only, and then required; may be x or
 *     residual itself, at the same stride);
 *   y [rows, ldy] bf16;  rstd [rows] FP32 (nvfp4_rmsnorm_backward reads it);
 *   amax_out [1] FP32: max |y| as stored, for nvfp4_quant_params.amax_in;
 *   mx_q [rows, cols] E4M3 codes and mx_sf E8M0 bytes of y, unrounded before, by
 *     mxfp8_quantize's rule; mx_sf in mx_sf_layout.  In the NVFP4_SF_MMA layout
 *     (mxfp8_sf_mma_bytes) the bytes of the padding rows are zeroed.
 * At least one of y and mx_q.  rows >= 0; cols a multiple of 8 (with mx_q: of
 * 32, tiled: of 128), at most 32768; pointers 16-byte aligned, strides
 * multiples of 8.  eps >= 0; with eps = 0 a row of zeros gives NaN.
 */
nvfp4_status nvfp4_rmsnorm(const void* x_bf16, int64_t ldx, const void* residual_bf16, int64_t ldr,
                           const void* weight, int weight_dtype, float eps, int64_t rows,
                           int64_t cols, void* h_bf16, int64_t ldh, void* y_bf16, int64_t ldy,
                           float* rstd, float* amax_out, uint8_t* mx_q, uint8_t* mx_sf,
                           int mx_sf_layout, void* stream);

/* Workspace bytes nvfp4_rmsnorm_backward needs for dweight. */
size_t nvfp4_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols);

/*
 * nvfp4_rmsnorm_backward -- gradients of nvfp4_rmsnorm from those of y (dy) and
 * of h (dh, NULL = none): with n = h * rstd,
 *   dx = dh + rstd * (weight * dy - n * mean(weight * dy * n)),
 *   dweight = sum over rows of dy * n        (NULL = not wanted).
 * dx is the gradient of x and of residual.  It may be dy or dh itself.  dweight
 * has weight_dtype; its sum is FP32 in a fixed order.  Shapes and alignment as
 * for nvfp4_rmsnorm.  The workspace is needed for dweight; without it one may be
 * given (16 bytes, 16-byte aligned), whose status word is then cleared.
 */
nvfp4_status nvfp4_rmsnorm_backward(const void* dy_bf16, int64_t lddy, const void* h_bf16,
                                    int64_t ldh, const void* dh_bf16, int64_t lddh,
                                    const void* weight, int weight_dtype, const float* rstd,
                                    int64_t rows, int64_t cols, void* dx_bf16, int64_t lddx,
                                    void* dweight, void* workspace, size_t ws_bytes, void* stream);

typedef struct {
    int top_k;        /* experts per token, 1..32                                   */
    int score;        /* NVFP4_SOFTMAX | NVFP4_SIGMOID                              */
    int groups;       /* expert groups of equal size, 1..32 (1 = no limit)          */
    int topk_groups;  /* groups a token may choose from                             */
    int group_top;    /* 1 | 2: a group's rank is the sum of that many best scores  */
    int renormalize;  /* 1: weights divided by the chosen scores' sum               */
    float scale;      /* factor on the weights                                      */
} nvfp4_route_params;

/* Workspace bytes nvfp4_route needs; up to 256 means that it may be left out. */
size_t nvfp4_route_workspace_size(int64_t tokens, int experts);

/*
 * nvfp4_route -- MoE routing (iitak, "Details": tokens travel to their experts):
 * the experts of each token, the combine's weights, and the order of the routed
 * rows that nvfp4_gather_rows, the grouped products and the combines read.
 *   logits [tokens, ld] of logits_dtype; s = softmax or sigmoid of a token's
 *   logits.  The top_k experts are chosen by s + bias (bias [experts] FP32 or
 *   NULL, it steers the choice only) among the topk_groups groups whose
 *   group_top best s + bias sum highest; ties go to the lower index.  Without
 *   bias and groups the logits themselves are compared; otherwise scores are
 *   told apart as far as FP64 does.  weight = scale * s, divided by the sum of
 *   the chosen s with renormalize.
 * A logit at or below bf16's lowest finite value (-3.3895e38; FP32's lowest and
 * -inf among them) masks its expert.  Where fewer than top_k experts are left,
 * the remaining slots have expert -1, weight 0 and row -1.  A NaN ranks last: the
 * logit where logits are compared, the score otherwise (a NaN logit makes all of
 * a token's softmax scores NaN).
 * Outputs: expert, weight [tokens, top_k], by falling rank; group_offsets
 * [experts + 1]; row_index [tokens * top_k]: the token of each routed row, rows
 * in expert order and by (token, slot) within an expert, -1 behind the last row
 * (group_offsets[experts]); slot_row [tokens, top_k]: each slot's row.
 * tokens >= 0; 1 <= top_k <= experts / groups * topk_groups; experts <= 512 (the
 * calls that take group_offsets accept up to 256 groups; nvfp4_combine and
 * mxfp8_combine read slot_row alone).
 */
nvfp4_status nvfp4_route(const void* logits, int logits_dtype, int64_t ld, const float* bias,
                         int64_t tokens, int experts, const nvfp4_route_params* p, int32_t* expert,
                         float* weight, int32_t* group_offsets, int32_t* row_index,
                         int32_t* slot_row, void* workspace, size_t ws_bytes, void* stream);

/*
 * nvfp4_route_backward -- the logits' gradient from that of nvfp4_route's
 * weights (dweight [tokens, top_k] FP32), for the experts it chose: dlogits
 * [tokens, ldd] of logits_dtype, every entry written (the choice itself has no
 * gradient, bias neither).  Slots with expert -1 give nothing.  Of p, top_k,
 * score, renormalize and scale count.
 */
nvfp4_status nvfp4_route_backward(const float* dweight, const void* logits, int logits_dtype,
                                  int64_t ld, const int32_t* expert, int64_t tokens, int experts,
                                  const nvfp4_route_params* p, void* dlogits, int64_t ldd,
                                  void* stream);

/*
 * nvfp4_combine -- weighted sum of each token's expert rows, where they are on
 * this GPU in bf16 or FP32 (mxfp8_combine is the form for rows that travelled):
 *   out[t] = base[t] + sum_j weight[t][j] * rows[slot_row[t][j]]
 * in FP32 in slot order, rounded once to bf16.  rows [n_rows, cols] of
 * rows_dtype; slot_row, weight [tokens, k]; base, out [tokens, cols] bf16 (base
 * NULL = 0; out may be base).  Slots with a negative row are left out; a row
 * index >= n_rows is left out and reported in the optional workspace's status
 * word.  cols a multiple of 8, 1 <= k <= 64, row pointers 16-byte aligned.
 */
nvfp4_status nvfp4_combine(const void* rows, int rows_dtype, int64_t n_rows, int64_t cols,
                           const int32_t* slot_row, const float* weight, int64_t tokens, int k,
                           const void* base_bf16, void* out_bf16, void* workspace, size_t ws_bytes,
                           void* stream);

/* Workspace bytes of nvfp4_combine_backward (the status word, a bit a row). */
size_t nvfp4_combine_backward_workspace_size(int64_t n_rows);

/*
 * nvfp4_combine_backward -- gradients of nvfp4_combine:
 *   drows[slot_row[t][j]] = weight[t][j] * dout[t]      (rows_dtype)
 *   dweight[t][j] = <dout[t], rows[slot_row[t][j]]>     (FP32; 0 for left-out slots)
 * Each row belongs to one slot at most, as nvfp4_route's do.  With a workspace
 * that is checked: a slot whose row another has named (which of the two is not
 * determined), or past n_rows, is left out and reported (NVFP4_ERR_INDEX); without
 * one the gradient of a row that two slots name is unspecified.  used_rows (device
 * int32, group_offsets + experts of nvfp4_route): rows that no slot names are
 * zeroed, those from *used_rows on without a look at the slots; tokens * k is then
 * below 2^31.  NULL: rows that no slot names are left as they were.  drows may be
 * rows and dweight weight; with used_rows not both, nor drows rows where n_rows
 * exceeds tokens * k (NVFP4_ERR_INVALID_ARG).
 */
nvfp4_status nvfp4_combine_backward(const void* dout_bf16, const void* rows, int rows_dtype,
                                    int64_t n_rows, int64_t cols, const int32_t* slot_row,
                                    const float* weight, int64_t tokens, int k,
                                    const int32_t* used_rows, void* drows, float* dweight,
                                    void* workspace, size_t ws_bytes, void* stream);

/*
 * nvfp4_gemv -- a few bf16 rows times an NVFP4 matrix (asector, "NVFP4 and
 * Blackwell"), the form of nvfp4_gemm for single tokens:
 *   D[i][j] = g * sum_k x[i][k] * (e2m1(q_jk) * e4m3(sf(j, k/16)))
 * x [rows, ldx] bf16, not quantised; q [N, K/2], sf and g as nvfp4_gemm's B
 * (NVFP4_SF_MMA layout).  Sums are FP32, in a fixed order.  D [rows, ldd] FP32 or
 * bf16 (RNE).  Any number of rows; meant for up to about 32: the matrix is read
 * again for every 8 or 16 rows, and for fewer where K is long and that costs less
 * than going over x in parts.  N a multiple of 16, K of 64 and at most 45056, ldx >= K of 8;
 * rows * N * K below about 2^43 (NVFP4_ERR_SHAPE); x, q, sf 16-byte aligned.
 */
nvfp4_status nvfp4_gemv(const void* x_bf16, int64_t ldx, int64_t rows, const uint8_t* q,
                        const uint8_t* sf, const float* g, int64_t N, int64_t K, int out_dtype,
                        void* D, int64_t ldd, void* stream);

/*
 * nvfp4_grouped_gemv -- nvfp4_gemv with one matrix per group, the form of
 * nvfp4_grouped_gemm for a few tokens: row i of D, in group e by group_offsets
 * (device int32 [G + 1], non-decreasing from 0, 1 <= G <= 256), is row row_index[i]
 * of x [src_rows, ldx] (NULL: row i) times matrix e.  q [G, N, K/2], sf [G]
 * consecutive NVFP4_SF_MMA blocks, g [G].  Rows behind group_offsets[G] are left as they were; an index
 * outside x gives a row of zeros and is reported in the optional workspace's
 * status word.  N a multiple of 128; otherwise as nvfp4_gemv.
 */
nvfp4_status nvfp4_grouped_gemv(int G, const int32_t* group_offsets, int64_t total_rows,
                                const void* x_bf16, int64_t ldx, int64_t src_rows,
                                const int32_t* row_index, const uint8_t* q, const uint8_t* sf,
                                const float* g, int64_t N, int64_t K, int out_dtype, void* D,
                                int64_t ldd, void* workspace, size_t ws_bytes, void* stream);

/* Workspace bytes of nvfp4_expert_mlp. */
size_t nvfp4_expert_mlp_workspace_size(int64_t total_rows, int64_t hidden, int64_t ffn);

/*
 * nvfp4_expert_mlp -- the experts of a MoE layer for a few tokens (iitak,
 * "Details": NVFP4 in the expert layers), their products as nvfp4_grouped_gemv's:
 *   h_i = silu(x_r gate_e^T) * (x_r up_e^T), or max(x_r up_e^T, 0)^2 without a gate,
 *   out[t] = base[t] + sum_j weight[t][j] * (h_i down_e^T),  i = slot_row[t][j]
 * for routed row i of expert e, r = row_index[i] (all as nvfp4_route gives them).
 * x [tokens, ldx] bf16; gate (all three pointers NULL: none) and up [G, ffn, hidden / 2],
 * down [G, hidden, ffn / 2] with consecutive NVFP4_SF_MMA blocks and g [G]; base, out
 * [tokens, hidden] bf16 (base NULL = 0; out may be base).  The products and what
 * becomes of them are FP32; h enters the last product as FP16 at a power of two a
 * row, off by at most 2^-11 of itself and 2^-38 of its row's largest.
 * Slots with a negative row are left out; a row_index outside x gives a row of
 * zeros, a slot_row at or behind group_offsets[G] or total_rows is left out, and
 * both are reported in the workspace's status word.  hidden and ffn multiples of 128
 * and at most 45056, 1 <= G <= 256, 1 <= k <= 64; otherwise as nvfp4_grouped_gemv
 * and nvfp4_combine.
 */
nvfp4_status nvfp4_expert_mlp(int G, const int32_t* group_offsets, int64_t total_rows,
                              const void* x_bf16, int64_t ldx, int64_t tokens,
                              const int32_t* row_index, const uint8_t* gate_q,
                              const uint8_t* gate_sf, const float* gate_g, const uint8_t* up_q,
                              const uint8_t* up_sf, const float* up_g, const uint8_t* down_q,
                              const uint8_t* down_sf, const float* down_g, int64_t hidden,
                              int64_t ffn, const int32_t* slot_row, const float* weight, int k,
                              const void* base_bf16, void* out_bf16, void* workspace,
                              size_t ws_bytes, void* stream);

/*
 * A paged cache of keys and values held in NVFP4 (asector, "NVFP4 and
 * Blackwell": a local scale per 16-element block on top of one scale per
 * tensor), blocks along the head dimension: codes q [2][pages][kv_heads]
 * [page_size][dim / 2] and E4M3 bytes sf [2][pages][kv_heads][page_size]
 * [dim / 16], the keys before the values.  amax [2] (device FP32): the largest
 * magnitudes of keys and of values, which fix the two FP32 scales as in
 * nvfp4_quantize with amax_in (g = amax / 2688; larger values saturate).  Token n
 * of sequence s is token n % page_size of page table[s][n / page_size].
 * dim 64, 128 or 256; page_size a power of two from 16 to 1024; q and sf 16-byte
 * aligned.  nvfp4_dequantize reads keys or values as a row-major tensor of
 * pages * kv_heads * page_size rows.
 */
typedef struct {
    uint8_t* q;
    uint8_t* sf;
    const float* amax;
    int64_t pages;
    int kv_heads;
    int page_size;
    int dim;
} nvfp4_kv_cache;

/*
 * nvfp4_kv_append -- keys and values of new tokens into a cache, keys and queries
 * turned by their positions on the way.  (The pages name no attention; it is the
 * step between the products that they quantise.)
 *   k, v [tokens][kv_heads][dim] bf16 (ld: elements from token to token, hs: from
 *   head to head; both multiples of 8), token t at place position[t] of sequence
 *   sequence[t] (NULL: sequence t), device int32.  table [sequences][ldt >=
 *   table_pages] device int32.
 * With cos and sin (FP32 [angles][rot / 2], rows by position) the first rot
 * elements of a head are turned: (a, b) -> (a cos - b sin, b cos + a sin) for the
 * pairs (x[i], x[i + rot / 2]), or with neighbours = 1 (x[2 i], x[2 i + 1]), exact
 * up to one rounding to bf16 (where each product is finite in FP32); the keys are
 * then quantised as nvfp4_quantize does it.  q [tokens][heads][dim] is turned likewise
 * into q_out (which may be q, at the same strides), whose heads do not overlap;
 * heads = 0 and NULL without queries.  Without cos, rot = 0.
 * A token with a negative position or sequence is left out, its row of q_out as it
 * was.  One whose sequence, place or page does not exist, or whose position is not
 * below angles, is left out and reported in the optional workspace's status word
 * (NVFP4_ERR_INDEX).  Of two tokens at one place, each block of 8 codes and each
 * scale byte is one of theirs.  rot a multiple of 32; pointers 16-byte aligned
 * (table, position and sequence 4).
 */
nvfp4_status nvfp4_kv_append(const nvfp4_kv_cache* cache, const void* k_bf16, int64_t ldk, int64_t hsk,
                             const void* v_bf16, int64_t ldv, int64_t hsv, int64_t tokens,
                             const int32_t* table, int64_t ldt, int64_t sequences,
                             int64_t table_pages, const int32_t* position, const int32_t* sequence,
                             const float* cos, const float* sin, int64_t angles, int rot,
                             int neighbours, const void* q_bf16, int64_t ldq, int64_t hsq, int heads,
                             void* q_out, int64_t ldo, int64_t hso, void* workspace, size_t ws_bytes,
                             void* stream);

/* Workspace bytes of nvfp4_kv_attention; capacity = table_pages * page_size (those of the
 * status word alone for sizes that the call refuses). */
size_t nvfp4_kv_attention_workspace_size(int64_t sequences, int queries, int heads, int kv_heads,
                                         int dim, int64_t capacity);

/*
 * nvfp4_kv_attention -- attention of a few query tokens per sequence over a cache,
 * the queries in bf16 (not quantised; a head's elements below 2^-31 of its largest
 * are taken to 2^-39 of that), the cached keys and values as they stand:
 *   out[s][i][h] = sum_n p_n v_n,  p = softmax(scale <q[s][i][h], k_n>)
 * over the tokens n that query i sees: those up to its own place lengths[s] -
 * queries + i, of the window (0: all) last ones.  Query heads h belong to key head h
 * / (heads / kv_heads).  q [sequences][queries][heads][dim] bf16 (strides in
 * elements, multiples of 8); lengths device int32 [sequences], the queries' own
 * tokens included; out contiguous bf16; lse (NULL: not wanted) FP32 [sequences]
 * [queries][heads]: log sum_n exp(scale <q, k_n>).  A query that sees no token (as
 * in a sequence of length 0) has out 0 and lse -inf.  Softmax and sums are FP32;
 * each exponential goes into the product with v (not into its own sum) rounded to
 * FP16, off by at most 2^-11 of itself and 2^-34 of its row's largest.
 * The table is read up to a sequence's length; with a window the pages before the
 * first query's may be gone (any entry).  Another page outside the cache counts as
 * zeros, a length outside 0..table_pages * page_size as the nearer end; both are
 * reported in the workspace's status word (NVFP4_ERR_INDEX).  Meant for few rows
 * (queries * heads / kv_heads): the cache is decoded again for every eight.
 * Results do not depend on timing.  Their last bits may depend on the other
 * sequences of a call and on the table's width: by these go the places where a long
 * sequence is cut and the tokens (32 or 64) that a running maximum is taken of.
 */
nvfp4_status nvfp4_kv_attention(const void* q_bf16, int64_t ldb, int64_t ldi, int64_t ldh,
                                int64_t sequences, int queries, int heads,
                                const nvfp4_kv_cache* cache, const int32_t* table, int64_t ldt,
                                int64_t table_pages, const int32_t* lengths, float scale,
                                int64_t window, void* out_bf16, float* lse, void* workspace,
                                size_t ws_bytes, void* stream);

/* Synchronise `stream` and return the device status word of a workspace
 * (NVFP4_OK, NVFP4_ERR_TIMEOUT or NVFP4_ERR_INDEX); clears it. */
nvfp4_status nvfp4_workspace_status(void* workspace, void* stream);

/* Text of a status code (static storage). */
const char* nvfp4_status_string(nvfp4_status s);

/* Library version: major * 10000 + minor * 100 + patch (200: adds mx_sf_layout
 * to nvfp4_quant_params, the sf_layout argument of mxfp4_quantize, mxfp8_gemm,
 * mxfp4_gemm and mxfp8_sf_mma_bytes; 300: adds the norm, routing, combine and
 * gemv calls; 400: adds the paged cache, attention over it and nvfp4_expert_mlp). */
int nvfp4_version(void);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_H */
