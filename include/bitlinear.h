/*
 * bitlinear.h -- C ABI of the B200 (sm_100a) BitLinear W1.58A8 library.
 *
 * The operation is the BitLinear forward of BitNet b1.58: ternary weights from
 * absmean quantisation packed four per byte, activations quantised per token to
 * int8 by absmax, an exact integer contraction, and a dequantisation to bf16.
 * Sources: "BitNet b1.58 2B4T Technical Report" paper card (ai-papers.xuzou.cn),
 * sections "Method Adaptation" (absmean ternary weights, per-token absmax int8
 * activations, subln, ReLU^2, no bias, four ternary weights per int8 value in
 * HBM, pack-store-load-unpack-compute kernel), "Compute Setup" (packed 1.58-bit
 * weights for inference, a custom W1.58A8 CUDA kernel) and "Bottleneck" (no
 * library kernel serves W1.58A8); the fishai news digest of the same report
 * (news.fishai.com.cn/news/3455510), list of the BitLinear layer's parts.
 *
 * Conventions shared by every call:
 *   - All tensor pointers are DEVICE pointers, allocated and owned by the caller.
 *     The library allocates no device memory in any call.
 *   - bf16 tensors are passed as their 16-bit patterns (uint16_t).
 *   - Matrices are row-major. W is [N, K] (out x in, as nn.Linear); x is [M, K];
 *     y and acc are [M, N].
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream). Arguments are validated on the host before anything is
 *     launched; on an error nothing is launched and the status says why.
 *   - No call synchronises the stream, except bitlinear_validate_packed and
 *     bitlinear_get_device_error, which say so.
 *   - No C++ exception crosses this boundary. A failed launch returns BL_ERR_CUDA.
 *   - Calls on different streams may overlap only if their workspaces differ.
 *   - The output y of a linear layer or FFN may be its x or its residual (an update
 *     in place; bitlinear_forward_noalloc too). Other arguments must not overlap
 *     what a call writes, unless the call says so.
 *   - Kernels launch with programmatic dependent launch: a call's kernel may start
 *     while the previous kernel in the stream finishes, and waits for it before
 *     reading its inputs x / h or writing anything. The packed weights (Wp, Wg,
 *     Wu, Wd, Wq) are the exception: the streamed GEMVs start copying them before that
 *     wait. So packed weights must not be written by the kernel just before the
 *     call in the same stream if that kernel triggers programmatic dependent launch
 *     early (the library's own kernels that do never write weights; the packing
 *     calls, host copies and ordinary kernels complete before a call starts).
 *
 * Packed weight format (this library's reading; the paper card, "Method
 * Adaptation", only fixes four ternary weights per 8-bit value): Wp is [N, K/4]
 * uint8, row-major. Byte j of row n holds weights k = 4j .. 4j+3; weight 4j+i
 * is stored in bits 2i..2i+1 as the code q+1 in {0, 1, 2} (q in {-1, 0, +1}).
 * Code 3 is invalid.
 *
 * Arithmetic (every step is one IEEE fp32 operation, round to nearest even, with
 * no fused multiply-add, unless noted):
 *   gamma = fp32( sum_{n,k} |W[n,k]| / (N*K) )      sum and division in fp64
 *   Wq    = clip(rint(W / (gamma + 1e-5)), -1, 1)
 *   s_m   = 127 / max(max_k |x[m,k]|, 1e-5)
 *   xq    = clip(rint(x * s_m), -128, 127)
 *   acc   = sum_k Wq[n,k] * xq[m,k]                 exact int32
 *   y     = bf16( float(acc) * (gamma / s_m) )      [+ float(residual) before bf16]
 */
#ifndef BITLINEAR_H
#define BITLINEAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, declared here so this header needs no CUDA headers. */
typedef struct CUstream_st* bl_stream_t;

typedef enum {
    BL_OK = 0,
    BL_ERR_NULL = 1,        /* a required pointer is NULL */
    BL_ERR_SHAPE = 2,       /* a size is negative, zero where it may not be, K % 4 != 0, or too large */
    BL_ERR_ALIGN = 3,       /* a pointer is not aligned as the call requires */
    BL_ERR_DTYPE = 4,       /* unknown bl_dtype */
    BL_ERR_WORKSPACE = 5,   /* workspace smaller than bitlinear_workspace_bytes() */
    BL_ERR_UNSUPPORTED = 6, /* valid arguments this build does not handle (e.g. no sm_100 device) */
    BL_ERR_CUDA = 7,        /* a CUDA call or launch failed */
    BL_ERR_TIMEOUT = 8,     /* a bounded wait inside a kernel gave up (see bitlinear_get_device_error) */
    BL_ERR_BAD_CODE = 9,    /* packed weights hold the invalid code 3 */
    BL_ERR_BAD_BATCH = 10   /* a kernel met a page, length or position out of range (see bitlinear_get_device_error) */
} bl_status;

typedef enum { BL_BF16 = 0, BL_FP32 = 1 } bl_dtype;

/* Operation ids for bitlinear_workspace_bytes. */
typedef enum {
    BL_OP_PACK = 0,     /* sizes: N, K of the weight */
    BL_OP_FORWARD = 1,  /* sizes: M, N, K */
    BL_OP_FFN = 2,      /* sizes: M, N = f (hidden), K = d (model width) */
    BL_OP_VALIDATE = 3, /* sizes ignored */
    BL_OP_FFN_TP_UP = 4,    /* sizes: M, N = f_local (the rank's hidden columns), K = d */
    BL_OP_FFN_TP_DOWN = 5,  /* sizes: M, N = d, K = f_local */
    BL_OP_KV4_ATTENTION = 6, /* sizes: M = max_q, N = Hq / Hkv, K = D */
    BL_OP_FORWARD_INT8 = 7  /* sizes: M, N, K */
} bl_op;

/* Kernels for M <= 16 tokens (bitlinear_set_gemv_kernel). */
typedef enum {
    BL_GEMV_AUTO = 0,   /* the library picks per call (default) */
    BL_GEMV_STREAM = 1, /* streamed GEMV: dp4a (one token) / mma.sync (2..16 tokens) on registers */
    BL_GEMV_TENSOR = 2, /* tcgen05 GEMV: weights unpacked into tensor memory, tokens as the MMA's N */
    BL_GEMV_LUT = 3     /* lookup tables of activation partial sums indexed by packed weight nibbles
                           (the T-MAC method of the bitnet.cpp CPU kernels); four tokens per pass */
} bl_gemv_kernel;

/* Human-readable name of a status. Never NULL; host only. */
const char* bitlinear_status_string(bl_status status);

/* Bytes of workspace `op` needs for the given sizes (0 for an invalid op).
 * Host only, no CUDA call. The workspace must be 256-byte aligned. */
size_t bitlinear_workspace_bytes(int op, int64_t M, int64_t N, int64_t K);

/*
 * Absmean ternary quantisation and packing of one weight tensor (one-time work).
 * Paper card, "Method Adaptation": weights quantised with absmean onto {-1, 0, +1}
 * in the forward pass, four ternary weights packed into one 8-bit value in HBM.
 *
 *   W      [N, K] device, bf16 bits (wdt = BL_BF16) or fp32 (BL_FP32); 16-byte aligned
 *   N, K   N >= 1, K >= 4, K % 4 == 0, N*K < 2^40
 *   Wp     [N, K/4] device uint8 output (format above); 16-byte aligned
 *   gamma  [1] device fp32 output: mean |W| (the per-tensor absmean scale)
 *   ws     device workspace of bitlinear_workspace_bytes(BL_OP_PACK, 0, N, K) bytes
 * Deterministic: the fp64 sum runs in a fixed order for given N, K.
 */
bl_status bitlinear_pack_weights(const void* W, int wdt, int64_t N, int64_t K,
                                 uint8_t* Wp, float* gamma,
                                 void* ws, size_t ws_bytes, bl_stream_t stream);

/*
 * Per-token absmax quantisation of activations to int8.
 * Paper card, "Method Adaptation": activations quantised per token with absmax
 * to 8-bit integers.
 *
 *   x      [M, K] device bf16 bits; 16-byte aligned
 *   M, K   M >= 0 (M == 0 is a no-op), K >= 4, K % 4 == 0
 *   xq     [M, K] device int8 output, row-major; 16-byte aligned
 *   scale  [M] device fp32 output: s_m = 127 / max(absmax_m, 1e-5)
 *   xsum   [M] device int32 output: sum_k xq[m,k]; may be NULL
 */
bl_status bitlinear_quant_act(const uint16_t* x, int64_t M, int64_t K,
                              int8_t* xq, float* scale, int32_t* xsum, bl_stream_t stream);

/*
 * One BitLinear forward: quantise x per token, contract with the packed ternary
 * weights, dequantise to bf16. Dig news article on the release, section 2:
 * nn.Linear replaced by BitLinear; paper card, "Method Adaptation": packed int8
 * weights loaded to on-chip memory, unpacked right before the matmul, multiplied
 * with int8 activations. No bias.
 *
 *   Wp        [N, K/4] device packed weights; 16-byte aligned
 *   gamma     [1] device fp32 (as written by bitlinear_pack_weights)
 *   N, K      N >= 0, K >= 4, K % 4 == 0
 *   x         [M, K] device bf16 bits; 2-byte aligned (16-byte for the fast kernels)
 *   M         M >= 0; M == 0 or N == 0 launches nothing
 *   residual  [M, N] device bf16 bits added before the final rounding; may be NULL
 *   y         [M, N] device bf16 bits output; 4-byte aligned
 *   acc       [M, N] device int32 output of the exact accumulator; may be NULL
 *   ws        device workspace of bitlinear_workspace_bytes(BL_OP_FORWARD, M, N, K) bytes
 * Kernel choice: M <= 16 streams the packed weights once through a
 * bandwidth-bound GEMV (K % 256 == 0, Wp and x 16-byte aligned), quantising x
 * inside the same kernel for M <= 4 (not for four tokens with K > 4096 on small
 * N, where the separate quantisation is faster) when the codes of all M tokens
 * fit in 48 KiB (M * (K + 64) bytes); larger M runs the tensor-core GEMM (K % 64 == 0, same
 * alignment, any N), which for shapes whose tiles would leave most of the
 * last wave idle splits tiles across CTAs and keeps their partial sums in the
 * workspace (bitlinear_workspace_bytes includes that scratch only for such
 * shapes); other shapes take a generic kernel. Every path gives the same bits.
 */
bl_status bitlinear_forward(const uint8_t* Wp, const float* gamma, int64_t N, int64_t K,
                            const uint16_t* x, int64_t M, const uint16_t* residual,
                            uint16_t* y, int32_t* acc,
                            void* ws, size_t ws_bytes, bl_stream_t stream);

/*
 * Per-row absmean variant of bitlinear_pack_weights: one gamma per output row
 * instead of one per tensor (the paper card "BitNet b1.58 2B4T Technical
 * Report", "Method Adaptation", gives one absmean per weight tensor; this is the
 * finer-grained variant of that reading):
 *   gammas[n] = fp32( sum_k |W[n, k]| / K )     sum and division in fp64
 *   q[n, k]   = clip(rint(W[n, k] / (gammas[n] + 1e-5)), -1, 1)
 * and the same packed layout. Arguments as bitlinear_pack_weights, with
 * gammas [N] device fp32 (4-byte aligned) in place of gamma; no workspace.
 */
bl_status bitlinear_pack_weights_rowwise(const void* W, int wdt, int64_t N, int64_t K,
                                         uint8_t* Wp, float* gammas, bl_stream_t stream);

/*
 * bitlinear_forward with the per-row gammas of bitlinear_pack_weights_rowwise:
 *   y[m, n] = bf16([residual[m, n] +] float(acc[m, n]) * (gammas[n] / s_m))
 * Arguments, kernel choice and errors as bitlinear_forward, with gammas [N]
 * device fp32 in place of gamma; the same workspace.
 */
bl_status bitlinear_forward_rowwise(const uint8_t* Wp, const float* gammas, int64_t N, int64_t K,
                                    const uint16_t* x, int64_t M, const uint16_t* residual,
                                    uint16_t* y, int32_t* acc,
                                    void* ws, size_t ws_bytes, bl_stream_t stream);

/*
 * Several BitLinear projections of one input in one call, optionally after a
 * unit-weight RMSNorm of the input: the attention side of a BitNet b1.58 block
 * (paper card "BitNet b1.58 2B4T Technical Report", "Method Adaptation":
 * BitLinear replaces the linear layers, subln sub-layer normalisation; fishai
 * digest, BitLinear list). The query, key and value projections read the same
 * normalised x; the output projection reads the subln-normalised attention
 * output and adds the residual.
 *   y[m, n] = bf16([residual[m, n] +] float(acc[m, n]) * (gammas[seg(n)] / s_m))
 *   xq, s   = quant(rmsnorm ? x * r : x),  r = 1 / sqrtf(float(sum_k x^2 / K) + 1e-5)
 *             per token (sum in fp64; x * r kept in fp32 and quantised as in
 *             bitlinear_forward)
 * Arguments:
 *   Wp        [N, K/4] device: the packed rows of nseg weight matrices stacked
 *             row-wise (each packed by bitlinear_pack_weights; packed rows are
 *             independent, so stacking is a byte copy); N = sum of seg_rows
 *   gammas    [nseg] device fp32: gamma of each matrix, in the same order
 *   seg_rows  [nseg] host: rows of each matrix, each >= 1; 1 <= nseg <= 4
 *   K, x, M   as bitlinear_forward
 *   rmsnorm   0: quantise x; 1: quantise the unit-weight RMSNorm of x
 *   residual, y, acc   [M, N], as bitlinear_forward
 *   ws        device workspace of bitlinear_workspace_bytes(BL_OP_FORWARD, M, N, K)
 * Kernel choice as bitlinear_forward. Segment boundaries on multiples of 16 rows
 * keep the streamed GEMV (M <= 16) and on multiples of 32 the tensor-core GEMM;
 * other boundaries run the generic kernel. Errors: BL_ERR_SHAPE for nseg outside
 * 1..4, rmsnorm not 0 or 1, a segment without rows, or the bitlinear_forward
 * shape rules on N = sum of seg_rows; otherwise as bitlinear_forward.
 */
bl_status bitlinear_forward_ex(const uint8_t* Wp, const float* gammas, const int64_t* seg_rows,
                               int32_t nseg, int64_t K, const uint16_t* x, int64_t M,
                               int32_t rmsnorm, const uint16_t* residual, uint16_t* y,
                               int32_t* acc, void* ws, size_t ws_bytes, bl_stream_t stream);

/*
 * One FFN sub-layer of BitNet b1.58 (fishai digest: ReLU^2 in the FFN, subln;
 * paper card, "Method Adaptation": subln, ReLU^2 feed-forward, no bias):
 *   xq, s   = quant(x)                       x [M, d]
 *   g, u    = deq(Wg . xq), deq(Wu . xq)     fp32, [M, f]
 *   h       = max(g, 0)^2 * u
 *   hn      = h / sqrt(mean_j h^2 + 1e-5)    unit-weight RMSNorm; sum in fp64
 *   q2, s2  = quant(hn)
 *   y       = bf16(residual + deq(Wd . q2))  y [M, d]; residual may be NULL
 *   Wg, Wu  [f, d/4] packed; gg, gu [1] device fp32
 *   Wd      [d, f/4] packed; gd [1] device fp32
 *   d, f    multiples of 4
 *   ws      bitlinear_workspace_bytes(BL_OP_FFN, M, f, d) bytes
 * Alignment as bitlinear_forward.
 */
bl_status bitlinear_ffn(const uint8_t* Wg, const float* gg, const uint8_t* Wu, const float* gu,
                        const uint8_t* Wd, const float* gd, int64_t d, int64_t f,
                        const uint16_t* x, int64_t M, const uint16_t* residual, uint16_t* y,
                        void* ws, size_t ws_bytes, bl_stream_t stream);

/*
 * bitlinear_forward without a workspace, for callers that cannot allocate.
 * The pages have no counterpart of this call; it exists for deployment.
 *
 * Some callers cannot call cudaMalloc where they run a layer: a plugin inside an
 * engine that reserved all device memory at start-up and allows no allocation
 * afterwards, or a latency-critical loop in which an allocation would implicitly
 * synchronise the device. They may also have no workspace buffer to pass. This
 * call computes what bitlinear_forward computes, to the same integers and bf16
 * bits, but keeps its scratch in a fixed 1 MiB array inside the library's own
 * device memory, which every GPU that loads the library holds until the process
 * exits. It always runs the separate act-quant kernel and then the GEMV (the
 * streamed one when K % 256 == 0 and Wp and x are 16-byte aligned, else the
 * generic one), also for M > 16, where bitlinear_forward uses the tensor cores:
 * large M is correct but slow here.
 *
 *   Arguments as bitlinear_forward, minus ws / ws_bytes.
 *   Limit: the scratch must hold the activation codes plus two per-token words:
 *          round256(M*K) + 2*round256(4*M) <= 1048576 bytes (for example M <= 16 at
 *          K <= 28672). Larger sizes return BL_ERR_WORKSPACE and launch nothing.
 *   No call allocates device memory or calls an allocating library routine.
 *   The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress). After a cudaDeviceReset the next call on that
 *   device looks it up again.
 *   Every call on a device shares the one array, which keeps the last call's
 *   contents (nothing in it needs to start at zero). Calls that can overlap on
 *   the GPU (other streams, unordered host threads) race on it: order them.
 */
bl_status bitlinear_forward_noalloc(const uint8_t* Wp, const float* gamma, int64_t N, int64_t K,
                                    const uint16_t* x, int64_t M, const uint16_t* residual,
                                    uint16_t* y, int32_t* acc, bl_stream_t stream);

/*
 * Selects, for the whole process, which kernel the forward calls
 * (bitlinear_forward, _ex, _rowwise and the projections inside bitlinear_ffn)
 * use for M <= 16 tokens; the choice is read when a call launches its kernels.
 * It exists to compare the kernels and to pin one in deployment; every kernel
 * computes the same integers and bf16 bits. A kernel that cannot take a call's
 * shape or alignment (all need K % 256 == 0 and 16-byte aligned Wp and x)
 * leaves that call to the automatic choice. The paper card "BitNet b1.58 2B4T
 * Technical Report", "Method Adaptation", describes one GPU kernel, the
 * streamed and tensor-core GEMVs are this library's designs for B200, and the
 * lookup-table GEMV follows the bitnet.cpp CPU kernels (dignews article on the
 * release, section 3: lookup tables after T-MAC, lossless).
 *   kind   a bl_gemv_kernel value
 * Returns the previous selection, or -1 (and changes nothing) for an unknown kind.
 * Host only, no CUDA call.
 */
int bitlinear_set_gemv_kernel(int kind);

/*
 * Tensor-parallel pieces of the FFN sub-layer. The pages give no distributed
 * detail (paper card "BitNet b1.58 2B4T Technical Report", "Limits"); this is
 * the library's split of bitlinear_ffn over P ranks (one GPU each): rank r owns
 * f_local of the f hidden columns, i.e. those rows of the gate and up weights
 * and those columns of the down weight, packed with the gammas of the whole
 * tensors. Per layer, between the calls, the caller exchanges (NCCL over
 * NVLink, or any transport): the per-token sums ss (fp64, sum) and maxima hmax
 * (fp32, max) after bitlinear_ffn_tp_up, and the int32 accumulators (sum, exact
 * in any order) after bitlinear_ffn_tp_down. The result equals bitlinear_ffn on
 * the whole weights bit for bit, up to the order of the fp64 sum of the ranks'
 * ss (a different fp32 subln factor needs those sums to straddle an fp32
 * rounding boundary).
 *
 * Packing a shard: the per-tensor gamma of the paper card's absmean ("Method
 * Adaptation") is over the whole tensor, so each rank adds its fp64 sum of |W|
 * (bitlinear_absmean_sum, into a device double) to the others' and packs its
 * shard with that total (bitlinear_pack_weights_global).
 */

/* fp64 sum of |W| over one shard [N, K] of a weight tensor (bf16 or fp32, as
 * bitlinear_pack_weights), written to *sum (device, 8-byte aligned), in a fixed
 * order. ws: bitlinear_workspace_bytes(BL_OP_PACK, 0, N, K) bytes. */
bl_status bitlinear_absmean_sum(const void* W, int wdt, int64_t N, int64_t K, double* sum,
                                void* ws, size_t ws_bytes, bl_stream_t stream);

/* Pack one shard [N, K] with the gamma of the whole tensor:
 *   gamma = fp32(*total_sum / total_count)   (device double, fp64 division)
 * total_sum: the fp64 sum of |W| over every shard; total_count: the element count
 * of the whole tensor (>= N * K). Wp [N, K/4] and gamma [1] as bitlinear_pack_weights. */
bl_status bitlinear_pack_weights_global(const void* W, int wdt, int64_t N, int64_t K, const double* total_sum,
                                        int64_t total_count, uint8_t* Wp, float* gamma, bl_stream_t stream);

/* Rank-local first half of the FFN: xq, s = quant(x) (x [M, d] whole on every
 * rank); g, u = deq(Wg . xq), deq(Wu . xq) on the rank's f_local rows (fp32);
 * h = max(g, 0)^2 * u -> h [M, f_local] fp32 (device); per token the rank's share of
 * the subln statistics: ss[m] = sum_j h[m, j]^2 (fp64) and hmax[m] = max_j |h[m, j]|.
 *   Wg, Wu  [f_local, d/4] packed shard rows; gg, gu [1] device fp32 (whole-tensor gammas)
 *   ws      bitlinear_workspace_bytes(BL_OP_FFN_TP_UP, M, f_local, d) bytes */
bl_status bitlinear_ffn_tp_up(const uint8_t* Wg, const float* gg, const uint8_t* Wu, const float* gu,
                              int64_t d, int64_t f_local, const uint16_t* x, int64_t M, float* h, double* ss,
                              float* hmax, void* ws, size_t ws_bytes, bl_stream_t stream);

/* Rank-local second half, after ss and hmax are reduced over the ranks
 * (ss_all = sum, hmax_all = max; device, [M]):
 *   r  = 1 / sqrtf(float(ss_all / f_total) + 1e-5)
 *   s2 = 127 / max(fl(hmax_all * r), 1e-5)          -> s2 [M] device fp32
 *   q2 = clip(rint(fl(h * r) * s2))                  the rank's columns
 *   acc[m, n] = sum_{j in the rank's columns} Wd[n, j] q2[m, j]  -> acc [M, d] int32
 *   Wd  [d, f_local/4] packed shard columns (packed with the whole tensor's gamma)
 *   ws  bitlinear_workspace_bytes(BL_OP_FFN_TP_DOWN, M, d, f_local) bytes */
bl_status bitlinear_ffn_tp_down(const uint8_t* Wd, int64_t d, int64_t f_local, int64_t f_total, const float* h,
                                int64_t M, const double* ss_all, const float* hmax_all, int32_t* acc, float* s2,
                                void* ws, size_t ws_bytes, bl_stream_t stream);

/* After acc is summed over the ranks: y = bf16([residual +] float(acc) * (gd / s2)).
 *   acc [M, d] int32, s2 [M] fp32, gd [1] (whole-tensor gamma), residual [M, d] bf16
 *   (may be NULL), y [M, d] bf16; all device. No workspace. */
bl_status bitlinear_ffn_tp_finish(const int32_t* acc, const float* gd, const float* s2, const uint16_t* residual,
                                  uint16_t* y, int64_t M, int64_t d, bl_stream_t stream);

/*
 * Attention with keys and values held in 4 bits in a paged cache: the part of a
 * decoder block between its Q/K/V projections (bitlinear_forward_ex) and its
 * output projection. The pages name the block's linear layers and norms only
 * (paper card "BitNet b1.58 2B4T Technical Report", "Method Adaptation"); the
 * cache format is this library's.
 *
 * Quantisation. A vector (one token, one key/value head, D dims; keys after their
 * rotation) is cut into groups of 32 consecutive dims. With A = max |x| of a group:
 *   step = fl(A / 7) rounded to five significant bits (nearest, ties to even);
 *          0 where A < 2^-100
 *   c    = rint(fl(x / step))  in [-7, 7];  0 where step = 0
 * The value held is c * step, a bf16 number exactly. A key or value vector with
 * a NaN, an infinity or a magnitude of 2^120 or more marks its token in that
 * head: the key steps become NaN, the value steps and all codes 0, so every
 * query that sees the token is NaN in the heads that share it, and no other is.
 *
 * Cache. Pages of P tokens, four arrays:
 *   kc, vc  [num_pages, Hkv, P, D/2] uint8   codes n = c + 8, two per byte
 *   ks, vs  [num_pages, Hkv, P, D/32] bf16   steps
 * The D/2 bytes of a vector are D/8 little-endian 32-bit words; word
 * t * (D/32) + g holds dims 32 g + 8 t .. + 7, the j-th in bits 4j .. 4j+3.
 * Steps of values in tokens that are attended to must be finite (those that
 * bitlinear_kv4_append writes are).
 *
 * Batch. S sequences, their new tokens stacked in M rows:
 *   q_start     [S + 1] device int32: rows q_start[s] .. q_start[s+1] - 1 belong to
 *               sequence s; not decreasing, q_start[0] = 0, q_start[S] <= M. Rows at or after
 *               q_start[S] are padding: nothing is written to them.
 *   kv_len      [S] device int32: tokens of the sequence in the cache, the new
 *               ones included. New token i of n has position kv_len - n + i; one
 *               whose position is negative (an idle sequence, kv_len 0) is not
 *               stored, its row is left as it was, and its attention output is zero.
 *   page_table  [S, W] device int32, rows table_stride elements apart: page of the
 *               tokens w P .. w P + P - 1. Entries past the last token are not read.
 * A page may stand in several rows (a shared prefix) where it is only read; the
 * tokens that a call appends must not share a slot.
 * The arrays live on the device and must not change while a call that was given
 * them runs (its blocks read them at different times). The kernels check their
 * contents: a page id outside 0 .. num_pages - 1, a kv_len below 0 or above W P (of
 * a sequence with new tokens), a q_start that leaves 0 .. M or decreases, or a
 * position past the rotation table sets the device error word
 * (bitlinear_get_device_error: BL_ERR_BAD_BATCH); no
 * access leaves the buffers, and the rows concerned (all rows of a batch whose
 * q_start decreases) are unspecified.
 *
 * Sizes for all calls: D 64 or 128; P 16, 32, 64, 128 or 256; 1 <= S <= 4096;
 * Hq % Hkv == 0, Hq <= 1024; M <= 65535; W >= 1, W P < 2^30, S Hkv W P < 2^36;
 * 1 <= num_pages < 2^31.
 */
typedef struct {
    uint8_t* kc;        /* 16-byte aligned, as the other three */
    uint16_t* ks;
    uint8_t* vc;
    uint16_t* vs;
    int64_t num_pages;
    int32_t page_size;  /* P */
    int32_t kv_heads;   /* Hkv */
    int32_t head_dim;   /* D */
} bl_kv4_cache;

typedef struct {
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* page_table;
    int64_t table_stride;
    int32_t S;
    int32_t W;
} bl_kv4_batch;

/*
 * Rotate the queries and keys of the batch's new tokens and store keys and
 * values in the cache. With position p and the pair (a, b) of dims:
 *   a' = fl(fl(a cos) - fl(b sin)),  b' = fl(fl(b cos) + fl(a sin))
 * Keys are quantised from the fp32 a', b'; values from their bf16.
 *   q, k, v     [M, Hq | Hkv | Hkv, D] device bf16; row m of x at x + m * x_stride
 *               elements, heads side by side (the column blocks of a stacked
 *               projection fit as they are); 16-byte aligned, strides multiples of 8
 *   q_out       rotated queries, bf16, rows q_out_stride apart; may be q itself
 *               (with the same stride)
 *   cos_sin     [max_pos, D] device fp32: row p holds D/2 cosines, then D/2 sines;
 *               16-byte aligned
 *   interleaved 0: pairs (i, i + D/2); 1: pairs (2i, 2i + 1); pair i uses entry i
 * M == 0 launches nothing.
 */
bl_status bitlinear_kv4_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                               const uint16_t* v, int64_t v_stride, int64_t M, int32_t Hq, const float* cos_sin,
                               int64_t max_pos, int32_t interleaved, const bl_kv4_cache* cache,
                               const bl_kv4_batch* batch, uint16_t* q_out, int64_t q_out_stride,
                               bl_stream_t stream);

/*
 * Read the cached values of the batch's tokens back: k, v [M, Hkv, D] device
 * bf16, 16-byte aligned, contiguous. (With q_start cumulating whole lengths this
 * reads whole sequences.)
 */
bl_status bitlinear_kv4_read(const bl_kv4_cache* cache, const bl_kv4_batch* batch, int64_t M, uint16_t* k,
                             uint16_t* v, bl_stream_t stream);

/*
 * Causal attention of the batch's new tokens over the cache (their own keys
 * included, so after bitlinear_kv4_append). Query head h reads key/value head
 * h / (Hq / Hkv):
 *   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale (q . k_j - max)),  j <= position
 * on the values that the cache holds; products and sums in fp32, p_j rounded to
 * bf16 for the product with v_j (not in the denominator). The exponentials are good
 * to 2^-20; where max_q Hq / Hkv > 16, a quarter of them to 7.5e-5. A row that sees
 * no key is zero. A query with a NaN or an infinity makes its row NaN in that head,
 * and so does a visible key with scale q . k log2(e) above fp32's range; one with
 * q . k above it, and queries of magnitude 2^100 / max(1, scale) or more, may. A key
 * whose score lies below that range weighs nothing beside others.
 * (M Hq / 256 + S Hkv) (W P / 128 + 8) < 2^31.
 *   q, out      [M, Hq, D] device bf16, rows q_stride / out_stride elements apart;
 *               16-byte aligned, strides multiples of 8; must not overlap
 *   max_q       the largest number of new tokens of a sequence (host): a sequence
 *               with more is reported as BL_ERR_BAD_BATCH and left out. It chooses the
 *               kernel for the whole batch: up to max_q Hq / Hkv = 16 one for few rows,
 *               beyond it one that works on 256 rows at a time, whatever a sequence
 *               brings. So give it as it is, and send single tokens and prompts in
 *               calls of their own where time matters (64 tokens on 4096 keys each and
 *               a prompt of 512: 173 us in one call, 56 and 23 in two)
 *   scale       2^-100 .. 2^100 (commonly 1 / sqrt(D))
 *   ws          bitlinear_workspace_bytes(BL_OP_KV4_ATTENTION, max_q, Hq / Hkv, D) bytes
 * Deterministic: the same inputs give the same bits.
 */
bl_status bitlinear_kv4_attention(const uint16_t* q, int64_t q_stride, int64_t M, int32_t Hq, int64_t max_q,
                                  float scale, const bl_kv4_cache* cache, const bl_kv4_batch* batch, uint16_t* out,
                                  int64_t out_stride, void* ws, size_t ws_bytes, bl_stream_t stream);

/*
 * 8-bit weights, for the layers that BitNet b1.58 does not ternarise (the
 * vocabulary head): one step per output row, activations quantised per token as
 * in bitlinear_quant_act (paper card "BitNet b1.58 2B4T Technical Report",
 * "Method Adaptation": per-token absmax to 8-bit integers).
 *   wstep[n]   = fl(max(max_k |W[n, k]|, 1e-30) / 127)
 *   Wq[n, k]   = clip(rint(fl(W[n, k] / wstep[n])), -127, 127)
 * A row with a NaN or an infinity has it as its step and zeros as its codes, so its
 * outputs are NaN.
 * W [N, K] bf16 or fp32 as bitlinear_pack_weights (16-byte aligned), but K % 16 == 0;
 * Wq [N, K] int8, 16-byte aligned; wstep [N] fp32.
 */
bl_status bitlinear_pack_weights_int8(const void* W, int wdt, int64_t N, int64_t K, int8_t* Wq, float* wstep,
                                      bl_stream_t stream);

/*
 * One 8-bit linear layer:
 *   xq, s  = quant(rmsnorm ? x * r : x)           as bitlinear_forward_ex
 *   acc    = sum_k Wq[n, k] * xq[m, k]            exact int32 (K <= 131072)
 *   y      = [residual +] fl(fl(float(acc) * wstep[n]) * fl(1 / s_m))
 * rounded to bf16 (ydt = BL_BF16) or kept fp32 (BL_FP32: y is float).
 *   Wq        [N, K] device int8, 16-byte aligned; N >= 0, K >= 16, K % 16 == 0
 *   x         [M, K] device bf16, 16-byte aligned; 0 <= M <= 65535
 *   residual  [M, N] device bf16, may be NULL; acc [M, N] device int32, may be NULL
 *   y         [M, N], contiguous
 *   ws        bitlinear_workspace_bytes(BL_OP_FORWARD_INT8, M, N, K) bytes
 */
bl_status bitlinear_forward_int8(const int8_t* Wq, const float* wstep, int64_t N, int64_t K, const uint16_t* x,
                                 int64_t M, int32_t rmsnorm, const uint16_t* residual, void* y, int ydt,
                                 int32_t* acc, void* ws, size_t ws_bytes, bl_stream_t stream);

/*
 * Check packed weights for the invalid code 3. SYNCHRONISES `stream`.
 * Returns BL_OK when every code is valid, BL_ERR_BAD_CODE otherwise; the number
 * of invalid codes is written to *bad_count (host pointer, may be NULL).
 *   ws  bitlinear_workspace_bytes(BL_OP_VALIDATE, 0, 0, 0) bytes of device memory
 */
bl_status bitlinear_validate_packed(const uint8_t* Wp, int64_t N, int64_t K, int64_t* bad_count,
                                    void* ws, size_t ws_bytes, bl_stream_t stream);

/*
 * SYNCHRONISES `stream`, then reports BL_ERR_CUDA for a pending CUDA error,
 * BL_ERR_TIMEOUT when a bounded wait inside one of this library's kernels gave up
 * since the last call on this device (the kernel that gave up wrote no output it
 * could not finish and returned), or BL_ERR_BAD_BATCH when an attention-side
 * kernel met a page, length or position out of range; the flags are cleared by
 * this call.
 */
bl_status bitlinear_get_device_error(bl_stream_t stream);

/*
 * Self-test of the failure path (no counterpart in the method; it exists to
 * test this library's error reporting). Launches, on `stream`, one thread that
 * waits with the library's bounded mbarrier wait on a barrier nothing arrives
 * on; after limit_us microseconds (1 .. 2,000,000) the wait gives up, records a
 * timeout in the device error word and the kernel returns normally. The next
 * bitlinear_get_device_error on this device then reports BL_ERR_TIMEOUT (and
 * clears it). The GPU context stays usable. Returns the launch status.
 */
bl_status bitlinear_selftest_timeout(int64_t limit_us, bl_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_H */
