/*
 * hk_gemm — dense BF16 GEMM  C = A · Bᵀ  for NVIDIA GB300 (sm_103a).
 *
 * The operation is the one the HipKittens pages measure most ("L2" detail
 * page, §3 "Target operation" table, row "BF16 GEMM": bf16 inputs, FP32
 * accumulation, bf16 output; §7 and §9.2 describe its hot loop as the
 * "ABt" product, so the second operand is stored N×K and used transposed;
 * §3 "Launch config" fixes the 256×256 output tile and 64-wide K step).
 *
 * Semantics of every entry point that computes:
 *
 *     C[i*ldc + j] = bf16_rne( Σ_{k<K}  A[i*lda + k] · B[j*ldb + k] )
 *
 * for 0 ≤ i < M, 0 ≤ j < N, with products and sums in FP32 on the tensor
 * cores (the order of the FP32 additions is unspecified), rounded once to
 * bf16 with round-to-nearest-even. There is no alpha/beta and no
 * accumulation into C; entries of C outside the M×N window (the padding
 * between N and ldc) are never written.
 *
 * Layout: A is M×K row-major, B is N×K row-major ("TN"), C is M×N row-major,
 * all bf16 (2 bytes per element, passed as raw device pointers). Leading
 * dimensions are in ELEMENTS.
 *
 * Ownership: A, B, C and any workspace are caller-owned DEVICE memory on the
 * device the call runs on. The library never frees them. C must not overlap
 * A or B.
 *
 * Alignment (a requirement of the Tensor Memory Accelerator): A, B and C
 * must be 16-byte aligned and lda, ldb, ldc multiples of 8, else
 * HK_ERR_MISALIGNED.
 *
 * Edge values: M == 0 or N == 0 -> HK_OK, nothing launched (pointers may be
 * NULL). K == 0 -> C (M×N) is filled with +0. Negative sizes, lda < K,
 * ldb < K, ldc < N or sizes ≥ 2^31 -> HK_ERR_INVALID_ARG.
 *
 * Device: the library runs on compute capability 10.3 (GB300) only; any
 * other device -> HK_ERR_UNSUPPORTED_DEVICE. There is no CPU fallback.
 *
 * Asynchrony: computing calls enqueue work on `stream` (a cudaStream_t; NULL
 * is the legacy default stream) and return without synchronising. Launch
 * failures are returned as HK_ERR_LAUNCH. Every wait inside the kernel is
 * bounded; a wait that runs out sets a device status word, the kernel drains
 * and returns, and the status is read with hk_gemm_plan_device_status or
 * hk_gemm_last_device_status after the stream has been synchronised.
 *
 * Thread safety: plans are immutable after creation and may be run from
 * several host threads at once; hk_gemm_bf16 is thread safe.
 */
#ifndef HK_GEMM_H
#define HK_GEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum hk_status {
    HK_OK = 0,
    HK_ERR_INVALID_ARG = 1,        /* a size, leading dimension or pointer is invalid */
    HK_ERR_MISALIGNED = 2,         /* pointer not 16-byte aligned or ld not a multiple of 8 */
    HK_ERR_UNSUPPORTED_DEVICE = 3, /* not a compute capability 10.3 device */
    HK_ERR_LAUNCH = 4,             /* the CUDA launch (or a CUDA runtime call) failed */
    HK_ERR_TIMEOUT = 5,            /* a bounded wait inside the kernel ran out */
    HK_ERR_WORKSPACE = 6,          /* workspace missing, too small or misaligned */
    HK_ERR_CUDA = 7                /* another CUDA runtime error (see hk_gemm_last_error_string) */
} hk_status;

/* Plan flags (hk_gemm_config.flags). */
#define HK_FLAG_NONE 0u
/* Test only: the producer withholds its arrival on the first shared-memory
 * stage, so a bounded wait on that stage runs out (the MMA issuer's) and
 * the call reports HK_ERR_TIMEOUT through the device status word. No GPU
 * fault is caused. */
#define HK_FLAG_FAULT_DROP_ARRIVE 0x1u
/* Keep the tiles of the last partial round whole (by default, when they fill
 * at most half of the CTA pairs, each runs as two halves of half the tile's
 * width: 256x128 for the 256x256 pair, 256x64 for the 256x128 pair). */
#define HK_FLAG_NO_TAIL_SPLIT 0x2u

/* Fused epilogue activations: C = bf16(act(A·Bᵀ + bias) [+ R]). */
#define HK_ACT_NONE 0
#define HK_ACT_RELU 1               /* max(x, 0) */
#define HK_ACT_GELU 2               /* x·Φ(x) = 0.5·x·(1 + erf(x/√2)) */
#define HK_ACT_SILU 3               /* x·σ(x) = x / (1 + e^(−x)) */

/* Kernel variants (hk_gemm_config.kernel). A "pair" kernel runs on clusters
 * of two CTAs (tcgen05 cta_group::2) with 256-row output tiles; a "single"
 * kernel runs one CTA per output tile of 128 rows and suits M <= 128. The
 * 256x128 and 256x112 pairs (bf16 only) stream a narrower slice of B per
 * pair: for 128 < M <= 256 with few output tiles they fill the GPU without a
 * K split (N = 8192 makes 74 tiles of 112 for the 76 pairs of a GB300, 64 of
 * 128), and its 23 KB stages leave room for a ninth in the ring (the
 * streaming rate of these shapes grows with the bytes in flight). The 256x112
 * pair never runs the last round's tiles as half-width units
 * (HK_FLAG_NO_TAIL_SPLIT is implied). */
#define HK_KERNEL_AUTO 0            /* chosen by the plan's time model: single-CTA kernels for M <= 128, pairs above 384 (E4M3: 128), either between */
#define HK_KERNEL_PAIR_256x256 1
#define HK_KERNEL_SINGLE_128x256 2
#define HK_KERNEL_SINGLE_128x192 3
#define HK_KERNEL_SINGLE_128x128 4
#define HK_KERNEL_SINGLE_128x64 5
#define HK_KERNEL_PAIR_256x128 6
#define HK_KERNEL_PAIR_256x112 7

/* Tuning knobs of a plan. Zero in any field selects the default. */
typedef struct hk_gemm_config {
    int32_t group_m;        /* grouped rasterisation: height of a group in output-tile rows (default 8) */
    int32_t max_clusters;   /* cap on the persistent grid, in work units (CTA pairs or CTAs; default: all that fit) */
    int32_t split_k;        /* K splits per output tile (0: chosen by the plan, which splits only when
                               the tiles do not fill one wave; 1: never; > 1: forced) */
    int32_t kernel;         /* HK_KERNEL_* (default HK_KERNEL_AUTO) */
    uint64_t timeout_ns;    /* limit of each bounded wait in the kernel (default 1 s) */
    uint32_t flags;         /* HK_FLAG_* */
    uint32_t activation;    /* fused epilogue activation, HK_ACT_* (used by hk_gemm_plan_run_epilogue) */
    int32_t input_type;     /* HK_INPUT_BF16 (default) or HK_INPUT_E4M3 (1-byte operands, ld multiples of 16) */
    float alpha;            /* scale applied to the fp32 accumulator before rounding (0: 1.0) */
} hk_gemm_config;

#define HK_INPUT_BF16 0
#define HK_INPUT_E4M3 1

/* What a plan chose (for logging and benchmarks). */
typedef struct hk_gemm_plan_info {
    int64_t M, N, K;
    int32_t kernel;                   /* HK_KERNEL_* actually used */
    int32_t ctas_per_unit;            /* 2 for a pair kernel, 1 for a single-CTA kernel */
    int32_t tile_m, tile_n, tile_k;   /* output tile of one work unit and K step */
    int32_t stages;                   /* depth of the shared-memory ring */
    int32_t num_tiles;                /* output tiles */
    int32_t grid_ctas;                /* CTAs launched */
    int32_t group_m;
    int32_t split_k;
    int32_t kernels_per_run;          /* kernel launches one run enqueues */
    int32_t smem_bytes;               /* dynamic shared memory per CTA */
    size_t workspace_bytes;
    int32_t tail_split_tiles;         /* tiles of the last round run as two half-width units */
    int32_t reserved;
} hk_gemm_plan_info;

typedef struct hk_gemm_plan hk_gemm_plan;

/* One-shot GEMM on the current device: C = bf16(A · Bᵀ).
 * Equivalent to a plan with the default config run with no workspace (the
 * default plan never needs one). The first call on a device creates a small
 * per-device context (a 16-byte device status word) and is therefore not
 * capturable in a CUDA graph; later calls allocate nothing. The plans of
 * recent shapes are kept (a small per-process cache, also used by
 * hk_gemm_bf16_epilogue, hk_gemm_bf16_fused and hk_gemm_fp8_e4m3), and each
 * keeps the tensor maps of its last A, B and C, so a repeated call does no
 * planning and, with the same pointers, no tensor-map encoding. */
hk_status hk_gemm_bf16(const void* A, const void* B, void* C,
                       int64_t M, int64_t N, int64_t K,
                       int64_t lda, int64_t ldb, int64_t ldc, void* stream);

/* Create a plan for one problem shape on `device`. `config` may be NULL.
 * Does all host-side work once: argument checks, device check, tile and
 * schedule choice, and allocates the plan's 16-byte device status word.
 * On success *out owns the plan; free it with hk_gemm_plan_destroy. */
hk_status hk_gemm_plan_create(hk_gemm_plan** out, int64_t M, int64_t N, int64_t K,
                              int64_t lda, int64_t ldb, int64_t ldc, int device,
                              const hk_gemm_config* config);

/* Bytes of device workspace a run needs (0 when no K split is used). With
 * S > 1 splits it holds S fp32 partial matrices (S × M × N', N' = N rounded
 * up to the tile width); a second kernel sums them in split order
 * (deterministic) and writes C. */
size_t hk_gemm_plan_workspace_size(const hk_gemm_plan* plan);

/* Fill *info with what the plan chose. */
hk_status hk_gemm_plan_get_info(const hk_gemm_plan* plan, hk_gemm_plan_info* info);

/* Enqueue one GEMM with the plan's shape on `stream`. `workspace` must hold
 * hk_gemm_plan_workspace_size(plan) bytes, 256-byte aligned (may be NULL when
 * that size is 0); it is scratch, owned by the caller, and must not be used by
 * another run that can overlap this one. The call allocates nothing. */
hk_status hk_gemm_plan_run(const hk_gemm_plan* plan, const void* A, const void* B, void* C,
                           void* workspace, size_t workspace_bytes, void* stream);

/* GEMM with a fused epilogue (the HipKittens pages fuse nothing into their
 * GEMM; this is the cheapest extension once the epilogue stage exists):
 *     C[i,j] = bf16_rne( act( Σ_k A[i,k]·B[j,k] + bias[j] ) )
 * computed in fp32 (accumulator + bias, then the activation) before the one
 * rounding. `bias` is a device vector of N bf16 values, 16-byte aligned, or
 * NULL (no bias); `activation` is an HK_ACT_* code (HK_ERR_INVALID_ARG
 * otherwise). Everything else as hk_gemm_bf16. */
hk_status hk_gemm_bf16_epilogue(const void* A, const void* B, void* C, const void* bias,
                                int64_t M, int64_t N, int64_t K,
                                int64_t lda, int64_t ldb, int64_t ldc,
                                int32_t activation, void* stream);

/* Plan form: the activation is hk_gemm_config.activation of the plan; the
 * bias (or NULL) is given per run. Otherwise as hk_gemm_plan_run. */
hk_status hk_gemm_plan_run_epilogue(const hk_gemm_plan* plan, const void* A, const void* B, void* C,
                                    const void* bias, void* workspace, size_t workspace_bytes,
                                    void* stream);

/* GEMM with a fused epilogue that also adds a residual:
 *     C[i,j] = bf16_rne( act( Σ_k A[i,k]·B[j,k] + bias[j] ) + R[i,j] )
 * in fp32 before the one rounding. The HipKittens "L2" detail page (§8
 * "Deployment context", Fusion scope) keeps the residual add in a separate
 * memory-bound kernel; here it rides in the GEMM's epilogue, which reads R
 * once while the tensor cores work on the next tile. `R` is a device matrix
 * of M×N bf16 values, row-major with leading dimension `ldr` (elements, a
 * multiple of 8 and ≥ N), 16-byte aligned (else HK_ERR_MISALIGNED), or NULL
 * (no residual). R may be C itself (same pointer, ldr == ldc): an in-place
 * update C ← act(A·Bᵀ + bias) + C; any other overlap of R and C is rejected
 * with HK_ERR_INVALID_ARG. `bias` and `activation` as hk_gemm_bf16_epilogue;
 * everything else as hk_gemm_bf16. */
hk_status hk_gemm_bf16_fused(const void* A, const void* B, void* C, const void* bias, const void* R,
                             int64_t M, int64_t N, int64_t K,
                             int64_t lda, int64_t ldb, int64_t ldc, int64_t ldr,
                             int32_t activation, void* stream);

/* Plan form of hk_gemm_bf16_fused: the activation is the plan's
 * hk_gemm_config.activation; bias, R and ldr are given per run (a K split
 * adds bias, activation and R in its reduction kernel). Also for E4M3 plans:
 * alpha, then bias, activation and R. Otherwise as hk_gemm_plan_run. */
hk_status hk_gemm_plan_run_fused(const hk_gemm_plan* plan, const void* A, const void* B, void* C,
                                 const void* bias, const void* R, int64_t ldr,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* FP8 GEMM (the pages' second GEMM: 8-bit floating-point inputs, FP32
 * accumulation, bf16 output), with one scale per operand tensor:
 *     C[i,j] = bf16_rne( (scale_a·scale_b) · Σ_k e4m3(A[i,k])·e4m3(B[j,k]) )
 * A (M×K) and B (N×K) hold E4M3 codes (1 sign, 4 exponent bits with bias 7,
 * 3 fraction bits; no infinities; largest magnitude 448), row-major,
 * K-contiguous; C is bf16 as in hk_gemm_bf16. lda and ldb are in elements
 * (= bytes) and must be multiples of 16, ldc a multiple of 8 (else
 * HK_ERR_MISALIGNED); scale_a·scale_b is formed in double and rounded once
 * to float. The products accumulate in fp32 on the tensor cores
 * (tcgen05.mma kind::f8f6f4). Block-scaled MXFP8 is not provided. */
hk_status hk_gemm_fp8_e4m3(const void* A, const void* B, void* C,
                           int64_t M, int64_t N, int64_t K,
                           int64_t lda, int64_t ldb, int64_t ldc,
                           float scale_a, float scale_b, void* stream);

/* MXFP8 GEMM (the pages' FP8 GEMM row: MXFP8 inputs, FP32 accumulation; a
 * bf16 output here): E4M3 operands whose K dimension is cut into blocks of 32
 * elements, each block of each row scaled by one UE8M0 byte E (value
 * 2^(E-127); 255 is NaN, as in the OCP MX format):
 *     C[i,j] = bf16_rne( Σ_b 2^(SFA[i,b]-127)·2^(SFB[j,b]-127)·Σ_{k in block b} A[i,k]·B[j,k] )
 * A (M×K) and B (N×K) hold E4M3 codes as in hk_gemm_fp8_e4m3 (lda, ldb
 * multiples of 16); SFA (M × K/32) and SFB (N × K/32) hold the scale bytes,
 * row-major with row strides ldsfa, ldsfb ≥ K/32 (bytes, any alignment); C is
 * bf16 as in hk_gemm_bf16. K must be a multiple of 32 (else
 * HK_ERR_INVALID_ARG). The products accumulate in fp32 on the tensor cores
 * (tcgen05.mma kind::mxf8f6f4 with block scales: 256×256 tiles on CTA pairs
 * when M > 128, else 128×192 tiles on one CTA).
 * `workspace` (device memory, 256-byte aligned, caller-owned, at least
 * hk_gemm_mxfp8_workspace_size(M, N, K) bytes, else HK_ERR_WORKSPACE)
 * receives the scales rearranged per tile and K stage by a small kernel
 * that runs first on `stream`; calls that overlap on the GPU must not share
 * it. Errors and asynchrony as hk_gemm_bf16. */
hk_status hk_gemm_mxfp8(const void* A, const void* B, const void* SFA, const void* SFB, void* C,
                        int64_t M, int64_t N, int64_t K,
                        int64_t lda, int64_t ldb, int64_t ldsfa, int64_t ldsfb, int64_t ldc,
                        void* workspace, size_t workspace_bytes, void* stream);

/* The same with test and tuning controls: `flags` takes
 * HK_FLAG_FAULT_DROP_ARRIVE (the producer withholds one arrival on the
 * first stage, so a bounded wait runs out and the status word reports
 * HK_ERR_TIMEOUT; other bits are rejected with HK_ERR_INVALID_ARG),
 * `timeout_ns` bounds each wait (0: 1 s). */
hk_status hk_gemm_mxfp8_ex(const void* A, const void* B, const void* SFA, const void* SFB, void* C,
                           int64_t M, int64_t N, int64_t K,
                           int64_t lda, int64_t ldb, int64_t ldsfa, int64_t ldsfb, int64_t ldc,
                           void* workspace, size_t workspace_bytes, uint32_t flags, uint64_t timeout_ns,
                           void* stream);

/* Bytes of workspace hk_gemm_mxfp8 needs for this shape (0 when M, N or K is 0). */
size_t hk_gemm_mxfp8_workspace_size(int64_t M, int64_t N, int64_t K);

/* Synchronise the plan's device and read-and-clear its status word:
 * HK_OK, or HK_ERR_TIMEOUT if a bounded wait ran out in any run since the
 * last read. */
hk_status hk_gemm_plan_device_status(hk_gemm_plan* plan);

/* The same for the calls of the one-shot entry points (hk_gemm_bf16,
 * hk_gemm_bf16_epilogue, hk_gemm_bf16_fused, hk_gemm_fp8_e4m3, hk_gemm_mxfp8(_ex),
 * hk_attention_fwd(_ex), hk_gemm_bf16_noalloc, hk_gemm_fp4(_ex), hk_kv8_append,
 * hk_attention_kv8(_ex), hk_attention_kv8_shared(_ex), hk_kv8_arrange, hk_kv8_compact,
 * hk_kv8_copy_pages) on `device`; HK_ERR_INVALID_ARG if a page index or a length
 * of a paged cache was out of range (and no wait ran out). */
hk_status hk_gemm_last_device_status(int device);

void hk_gemm_plan_destroy(hk_gemm_plan* plan);

/* GEMM that allocates nothing, for callers that cannot call cudaMalloc when
 * they run a GEMM (code inside a memory pool or arena that owns all device
 * memory, allocator or runtime hooks that must not re-enter the allocator,
 * services that fix their memory at start-up). This entry point has no
 * counterpart on the HipKittens pages; it exists for those callers.
 *
 * Same operation, arguments and errors as hk_gemm_bf16, plus `split_k`
 * (0: chosen automatically, 1: never split K, > 1: forced). Its K-split
 * scratch and its status word live in one fixed array inside the library's
 * device image: 32 MiB of scratch, resident on every device that loads the
 * library until the process exits. A forced split_k whose fp32 partials
 * (split_k × M × N rounded up to the tile width × 4 bytes) exceed 32 MiB is
 * rejected with HK_ERR_WORKSPACE; an automatic split that would not fit is
 * not taken. The caller provides A, B and C; nothing is allocated, freed or
 * set up through an allocating library routine.
 *
 * The first call on a device looks up the array's device address (once, with
 * that device current); make that first call before any stream capture (a
 * first call whose stream is capturing is refused with HK_ERR_INVALID_ARG).
 * All calls on a device share the array and it keeps the last call's
 * contents (nothing in it needs to start at zero). Calls that overlap on the
 * GPU race on it: order them on one stream or serialise them. A bounded wait
 * that runs out in this variant is reported by hk_gemm_last_device_status(),
 * which reads and clears the status word in the array without allocating. */
hk_status hk_gemm_bf16_noalloc(const void* A, const void* B, void* C,
                               int64_t M, int64_t N, int64_t K,
                               int64_t lda, int64_t ldb, int64_t ldc,
                               int32_t split_k, void* stream);

/* Attention forward, MHA or GQA (the pages' second workload: HipKittens "L2"
 * detail page, §3 "Target operation" table, rows "MHA fwd" / "GQA fwd";
 * §5 "Numerical considerations" and §9.3 for the online softmax with
 * temperature sqrt(1/D)):
 *
 *     O[b,h,i,:] = bf16_rne( Σ_j P[i,j] · V[b,g,j,:] ),
 *     P[i,:]     = softmax_j( Q[b,h,i,:]·K[b,g,j,:] / sqrt(D) ),
 *     g = h / (Hq / Hkv)  (consecutive query heads share a KV head),
 *
 * over the keys j < S, or j ≤ i when `causal` is non-zero. Q·Kᵀ and P·V run
 * on the tensor cores (bf16 operands, fp32 accumulation); P is rounded to
 * bf16 before P·V and the row sums use the unrounded fp32 P; exp is the
 * hardware base-2 exponential. `lse`, when not NULL, receives per row the
 * natural-log sum ln Σ_j exp(Q·K/sqrt(D)) in fp32, [B, Hq, S].
 *
 * Layout: Q and O are [B, Hq, S, D], K and V are [B, Hkv, S, D], contiguous
 * row-major bf16 device arrays (16-byte aligned, else HK_ERR_MISALIGNED);
 * lse is a 4-byte-aligned fp32 device array or NULL. O must not overlap the
 * inputs. D must be 64 or 128, Hkv ≥ 1 must divide Hq, and B·Hq·S must stay
 * below 2^31 (else HK_ERR_INVALID_ARG). B, Hq or S equal to 0: HK_OK,
 * nothing launched. Asynchronous on `stream`; a bounded wait that runs out
 * is reported by hk_gemm_last_device_status(device). */
hk_status hk_attention_fwd(const void* Q, const void* K, const void* V, void* O, float* lse,
                           int64_t B, int64_t Hq, int64_t Hkv, int64_t S, int64_t D,
                           int32_t causal, void* stream);

/* The same with test and tuning controls: `flags` takes
 * HK_FLAG_FAULT_DROP_ARRIVE (the producer never fills the first K/V slot,
 * so a bounded wait runs out and the status word reports HK_ERR_TIMEOUT),
 * `timeout_ns` bounds each wait (0: 1 s). */
hk_status hk_attention_fwd_ex(const void* Q, const void* K, const void* V, void* O, float* lse,
                              int64_t B, int64_t Hq, int64_t Hkv, int64_t S, int64_t D,
                              int32_t causal, uint32_t flags, uint64_t timeout_ns, void* stream);

/* ---------------------------------------------------------------------------
 * Microscaled 4-bit floating point (MXFP4, NVFP4): quantisation and product.
 *
 * Values are E2M1 codes (1 sign, 2 exponent, 1 fraction bit; magnitudes 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6), with one scale per block of a row's columns:
 *
 *   HK_FP4_MXFP4  blocks of 32; scale 2^E, kept as the UE8M0 byte E + 127 (255:
 *                 NaN), E = floor(log2 amax) - 2 of the block's largest magnitude
 *                 (at least -127; 0 for a block of zeros: byte 0);
 *                 code = e2m1(x / 2^E).
 *   HK_FP4_NVFP4  blocks of 16; scale s in E4M3, s = e4m3(amax / (6·g)) with a
 *                 global scale g > 0 of the whole matrix (one float in DEVICE
 *                 memory, NULL: 1); code = e2m1(x · (1 / (s·g))); a value is
 *                 code · s · g. g = amax of the matrix / 2688 uses the whole range.
 *
 * e2m1 and e4m3 round to nearest, halves to even; magnitudes above the
 * largest become the largest (6 and 448). A block with a NaN or an infinity
 * gets a NaN scale (255, 0x7F) and codes 0: its values are NaN.
 *
 * A quantised matrix of rows × cols is two device arrays, 16-byte aligned:
 *   codes   two per byte, the even column in the low half; rows of `ld` BYTES, a
 *           multiple of 16 and at least ceil(cols / 32) · 16; columns past the
 *           matrix up to the next multiple of 32 hold code 0;
 *   scales  hk_fp4_scales_size bytes in tiles of 128 rows × 4 blocks (512
 *           bytes), row groups outermost: the scale of row r, block b is at
 *             ((r / 128) · (nb / 4) + b / 4) · 512 + (r % 32) · 16 + (r % 128 / 32) · 4 + b % 4
 *           with nb the blocks of a row padded to whole 256-column chunks
 *           (nb = ceil(cols / 256) · 8 or · 16). Blocks past the matrix hold 0.
 * hk_fp4_quantize writes both, padding included; the product reads them as
 * they are (nothing is rearranged at call time). */
#define HK_FP4_MXFP4 0
#define HK_FP4_NVFP4 1

/* Element types of the arrays that quantisation reads and writes. */
#define HK_TYPE_BF16 0
#define HK_TYPE_FP16 1
#define HK_TYPE_FP32 2

/* Bytes of the scales of a rows × cols matrix (0 for an empty one or an unknown format). */
size_t hk_fp4_scales_size(int64_t rows, int64_t cols, int32_t format);

/* Quantise X (rows × cols, row-major, element type x_type, leading dimension
 * ldx in elements, any alignment of its element type; 16-byte aligned rows are
 * read in 16-byte pieces). `global_scale` is NULL for MXFP4. rows or cols 0:
 * HK_OK, nothing written. Asynchronous on `stream`, allocates nothing. */
hk_status hk_fp4_quantize(const void* X, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx,
                          void* codes, int64_t ld_codes, void* scales, int32_t format,
                          const float* global_scale, void* stream);

/* The values of a quantised matrix, code · (scale · g), rounded once to y_type. */
hk_status hk_fp4_dequantize(const void* codes, int64_t ld_codes, const void* scales, int32_t format,
                            const float* global_scale, int64_t rows, int64_t cols,
                            void* Y, int32_t y_type, int64_t ldy, void* stream);

/* Product of two quantised matrices of one format:
 *     C[i,j] = bf16_rne( ga·gb · Σ_b SA[i,b]·SB[j,b] · Σ_{k in block b} A[i,k]·B[j,k] )
 * A (M × K) and B (N × K) as above, lda and ldb in BYTES; C is M × N bf16,
 * row-major, ldc ≥ N in elements, any 2-byte alignment. global_a and global_b
 * are the operands' global scales (device memory, NULL: 1; NULL for MXFP4).
 * The products run on the tensor cores with fp32 sums (tcgen05.mma kind::mxf4
 * and kind::mxf4nvf4); a NaN scale gives NaN in its row or column of C. K = 0
 * fills C with +0. Asynchronous on `stream`, needs no workspace; a bounded
 * wait that runs out is reported by hk_gemm_last_device_status. */
hk_status hk_gemm_fp4(const void* A, const void* SFA, const void* B, const void* SFB, void* C,
                      int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc,
                      int32_t format, const float* global_a, const float* global_b, void* stream);

/* The same with tuning and test controls: `kernel` is HK_KERNEL_AUTO (chosen by
 * shape), HK_KERNEL_PAIR_256x256 (CTA pairs) or HK_KERNEL_SINGLE_128x128 (one
 * CTA, tiles of 128 rows of B × 16 to 128 rows of A, K cut into `split_k` parts
 * of a cluster: 0 chosen, 1, 2, 4 or 8); `flags` takes
 * HK_FLAG_FAULT_DROP_ARRIVE (the first stage is never filled, so a bounded wait
 * runs out), `timeout_ns` bounds each wait (0: 1 s). */
hk_status hk_gemm_fp4_ex(const void* A, const void* SFA, const void* B, const void* SFB, void* C,
                         int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc,
                         int32_t format, const float* global_a, const float* global_b,
                         int32_t kernel, int32_t split_k, uint32_t flags, uint64_t timeout_ns, void* stream);

/* ---------------------------------------------------------------------------
 * A paged key/value cache held in 8 bits, the append to it and attention over it.
 *
 * Pages of `page_size` tokens (16, 32, 64 or 128) hold E4M3 codes of every KV
 * head, with one fp32 scale per page and head, always a power of two: a cached
 * value is code · scale. All four arrays are caller-owned device memory,
 * contiguous:
 *   k_codes, v_codes   [num_pages, heads, page_size, head_dim] bytes, 16-byte aligned
 *   k_scale, v_scale   [num_pages, heads]
 * head_dim is 64 or 128, heads at most 65535, a sequence's room (max_pages ·
 * page_size) below 2^31 - 127 tokens. A fresh cache needs no initialisation: the append
 * that puts the first token into a page sets its scale.
 *
 * Which pages a sequence owns is said by a block table of int32, [B, max_pages]
 * with `table_stride` elements between rows: token j of sequence b lies in page
 * block_table[b][j / page_size] at place j % page_size. Entries past a
 * sequence's tokens are not read. A page index outside [0, num_pages) or a
 * length outside the table is never followed: such tokens are not written, the
 * output of such a sequence is unspecified (the others' is not), and
 * hk_gemm_last_device_status reports HK_ERR_INVALID_ARG. */
typedef struct hk_kv8_cache {
    void* k_codes;
    void* v_codes;
    float* k_scale;
    float* v_scale;
    int64_t num_pages;
    int32_t heads;
    int32_t page_size;
    int32_t head_dim;
    int32_t reserved;
} hk_kv8_cache;

/* Append T tokens (or counts[b] <= T of them, its first) to each of B
 * sequences, which hold starts[b] tokens before: token t goes to position
 * starts[b] + t. K and V are [B, T, heads, head_dim] arrays of `type` (bf16,
 * fp16 or fp32) with strides (b, t, head) in elements and contiguous rows of
 * head_dim (16-byte aligned rows are read in 16-byte pieces).
 * The new tokens of a page need the scale 2^e, e >= -126 the smallest with
 * amax <= 448 · 2^e over their finite values. A page that already holds tokens
 * of the sequence keeps its scale where that is larger; else its codes are
 * rounded again to the new scale. Rounding is to nearest, halves to even;
 * infinities become ±448 · scale, NaN stays NaN. Calling it again with the
 * same arguments changes nothing. Pages must not be shared between sequences
 * that are appended to. Asynchronous on `stream`, allocates nothing (but the
 * status word, once). */
hk_status hk_kv8_append(const hk_kv8_cache* cache, const void* K, const void* V, int32_t type,
                        int64_t B, int64_t T, const int64_t k_strides[3], const int64_t v_strides[3],
                        const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                        const int32_t* starts, const int32_t* counts, void* stream);

/* Attention of T query tokens per sequence over its lengths[b] cached tokens:
 *     O[b,t,h,:] = Σ_j P_j · V_j,  P = softmax_j( scale · Q[b,t,h,:]·K_j ),
 * K_j and V_j the cached values of head h / (Hq / heads). With `causal` query t
 * stands at position lengths[b] - n + t, n = counts[b] (NULL: T), and sees the
 * tokens up to it (the queries' own keys are in the cache); else it sees all
 * lengths[b]. A query that sees no token, and queries t >= counts[b], give a row
 * of zeros and a log-sum-exp of -inf. A NaN among a token's values makes its
 * dimension NaN in the queries that see the token and in no others. `scale` must not
 * be negative; 0: 1/sqrt(head_dim).
 * Q and O are [B, T, Hq, head_dim] of `type` (bf16 or fp16), strides (b, t, head)
 * in elements, contiguous rows (O's must not overlap). lse, when not NULL: fp32
 * [B, T, Hq], natural log of the sum of exp(scale · q·k).
 * Many query rows per KV head (a prompt) run on the attention-forward kernel when Q
 * is bf16 with rows that are 16-byte aligned; fp16 and other rows run on the
 * few-row kernels whatever their number (2048 tokens x 64 heads of 128 against 16384: 806
 * us and 4311 us).
 * Scores, softmax sums and outputs are summed in fp32. Besides the rounding of O, the
 * weights are rounded before they meet V: to f16 on the few-row kernels (2^-11 of a
 * weight, down to 2^-29 of the row's largest), to bf16 on the many-row form (2^-8).
 * `workspace`: device memory of hk_attention_kv8_workspace_size(_ex) bytes, 256-byte
 * aligned, scratch of this call (calls that overlap on the GPU must not share
 * it). Asynchronous on `stream`; a bounded wait that runs out is reported by
 * hk_gemm_last_device_status. */
hk_status hk_attention_kv8(const void* Q, int32_t type, const int64_t q_strides[3], const hk_kv8_cache* cache,
                           const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                           const int32_t* lengths, const int32_t* counts,
                           void* O, const int64_t o_strides[3], float* lse,
                           int64_t B, int64_t T, int64_t Hq, int32_t causal, float scale,
                           void* workspace, size_t workspace_bytes, void* stream);

/* The same with test controls. `flags`: which kernels run, HK_KV8_FEW_ROWS (whatever
 * the rows are) or HK_KV8_MANY_ROWS (refused for rows that they cannot take), 0: chosen by
 * shape; HK_KV8_FAULT_DROP_ARRIVE: an arrival is withheld, so that a bounded wait runs
 * out. `timeout_ns` bounds each wait (0: 1 s). */
#define HK_KV8_FEW_ROWS 0x10u
#define HK_KV8_MANY_ROWS 0x20u
#define HK_KV8_FAULT_DROP_ARRIVE 0x40u
hk_status hk_attention_kv8_ex(const void* Q, int32_t type, const int64_t q_strides[3], const hk_kv8_cache* cache,
                              const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                              const int32_t* lengths, const int32_t* counts,
                              void* O, const int64_t o_strides[3], float* lse,
                              int64_t B, int64_t T, int64_t Hq, int32_t causal, float scale,
                              void* workspace, size_t workspace_bytes, uint32_t flags, uint64_t timeout_ns,
                              void* stream);

/* Bytes of workspace that are enough for hk_attention_kv8 whatever the type and the
 * strides are: 0 for an empty problem and for few query rows over short block
 * tables; else 10 to 37 MB, or (many query rows) the bf16 keys and values of as many
 * sequences as fit 512 MB, of one at least. */
size_t hk_attention_kv8_workspace_size(const hk_kv8_cache* cache, int64_t B, int64_t T, int64_t Hq, int64_t max_pages);

/* Bytes that the call with these arguments needs, and asks for: those of the kernels
 * that it runs on (fp16 queries and rows that TMA cannot read need no bf16 keys and
 * values). Q and O are looked at for their alignment only. */
size_t hk_attention_kv8_workspace_size_ex(const void* Q, int32_t type, const int64_t q_strides[3],
                                          const hk_kv8_cache* cache, int64_t max_pages, const void* O,
                                          const int64_t o_strides[3], int64_t B, int64_t T, int64_t Hq,
                                          uint32_t flags);

/* ---------------------------------------------------------------------------
 * Which pages of the cache a sequence holds: growing, cutting back, ending, forking and
 * reordering sequences, and moving pages together. All of it runs on the device (nothing is
 * read back, so that it may be captured in a graph).
 *
 * A pool goes with one or several caches of the same pages (a model's layers):
 *   refs    int32 [num_pages]: how many table entries name each page; 0: it is free
 *   table   int32 [rows, max_pages], table_stride elements between rows: the block table that
 *           hk_kv8_append and hk_attention_kv8 read
 *   held    int32 [rows]: tokens whose pages a row has, ceil(held / page_size) entries; entries
 *           past them mean nothing
 * An empty pool is refs and held of zeros. num_pages at most 2^30, rows · max_pages below 2^31. */
typedef struct hk_kv8_pool {
    int32_t* refs;
    int32_t* table;
    int32_t* held;
    int64_t num_pages;
    int64_t table_stride;
    int32_t rows;
    int32_t max_pages;
    int32_t page_size;
    int32_t reserved;
} hk_kv8_pool;

/* Arrange the pool's rows anew, all at once: row i becomes the first keep[i] tokens of what row
 * parents[i] was before the call (NULL: of its own), with pages for room[i] >= keep[i] tokens.
 * keep, room, parents: int32 [rows] on the device (keep and room may be held itself). So
 *   room[i] above what row i holds      takes pages (for tokens to come),
 *   keep[i] below it                    cuts the row back; keep = room = 0 ends it,
 *   parents[i] = j                      forks row j, or (for several rows) reorders them.
 * Pages that are whole within keep[i] are shared with the parent. The pages above, into which
 * tokens will be appended, belong to row i alone: it goes on in its parent's where it is the parent's
 * heir (i itself where parents[i] = i; else, where the parent becomes another row's, the lowest
 * row with that parent), no other entry names the page and no other row keeps it whole; else in free pages, the
 * lowest ones first, in order of row and slot. Of a page that holds tokens of keep[i] the contents are copied
 * in every one of the n_caches caches. keep[i] counts tokens that were appended, not
 * only held: a page that counts as whole is not written again.
 * Free are pages with refs = 0 before the call; what the call frees is free for the next one.
 * *missing (device): 0, or the pages that lacked, or -1: a row's parent, tokens or page
 * index is out of range (hk_gemm_last_device_status then reports HK_ERR_INVALID_ARG). Unless it is 0 nothing
 * was changed. `copies` (device, or NULL): int32 [2, rows], each row's page that was copied and
 * its copy, -1 where there is none (for other caches: hk_kv8_copy_pages).
 * `workspace`: device memory of hk_kv8_arrange_workspace_size bytes, 256-byte aligned, scratch of
 * this call. Asynchronous on `stream`, allocates nothing (but the status word, once). */
hk_status hk_kv8_arrange(const hk_kv8_pool* pool, const int32_t* keep, const int32_t* room, const int32_t* parents,
                         const hk_kv8_cache* caches, int32_t n_caches, int32_t* copies, int32_t* missing,
                         void* workspace, size_t workspace_bytes, void* stream);
size_t hk_kv8_arrange_workspace_size(const hk_kv8_pool* pool);

/* Move the U pages in use to the places [0, U): the k-th used page at U or above goes to the k-th free page
 * below U, in every cache, in the table and in refs. moved: int32 [num_pages] on the device, where
 * each page is now, -1 where it was free. A page index out of range in a row's entries stays as it is and
 * hk_gemm_last_device_status reports HK_ERR_INVALID_ARG. Workspace and asynchrony as above. */
hk_status hk_kv8_compact(const hk_kv8_pool* pool, const hk_kv8_cache* caches, int32_t n_caches, int32_t* moved,
                         void* workspace, size_t workspace_bytes, void* stream);
size_t hk_kv8_compact_workspace_size(const hk_kv8_pool* pool);

/* Copy page src_pages[i] of each src[j] to page dst_pages[i] of dst[j] (codes and scales), i < n, j <
 * n_caches; entries of -1 in both lists are left out. dst[j] may be src[j] or another cache of the same heads,
 * page size and head dimension (a larger pool); no page may be written twice or be read and written
 * in one call. An index out of range is not followed and hk_gemm_last_device_status
 * reports HK_ERR_INVALID_ARG. Asynchronous on `stream`. */
hk_status hk_kv8_copy_pages(const hk_kv8_cache* dst, const hk_kv8_cache* src, int32_t n_caches,
                            const int32_t* dst_pages, const int32_t* src_pages, int64_t n, void* stream);

/* Attention as hk_attention_kv8 for a batch whose sequences begin with the same tokens in the
 * same pages (hk_kv8_arrange forks them so): the shared pages are read once per group.
 * Group g < G is the sequences [groups[g], groups[g + 1]) of the batch (int32 [G + 1] on the device, from 0
 * to B, strictly increasing); the first shared[g] tokens (int32 [G] on the device) of each of them lie in the same pages,
 * which every sequence's own table row names too. They are read once, by the first sequence's row, as far as they fill whole
 * blocks of 128 tokens. shared[g] = 0, and groups of one sequence, are fine. The result is hk_attention_kv8's, but for the
 * order of its fp32 sums and, on the tensor-core kernel, the rounding of weights: in f16 they are 2^-11 of a weight down to 2^-21
 * of the row's largest so far, and 2^-32 of that below (2^-29 and 2^-40 in hk_attention_kv8); where pages' scales of values
 * differ by more than 2^7 they are bf16, 2^-8, for fp16 queries too. Not shared in
 * fact, and read by a sequence itself, are tokens past the first sequence's length, and those of a
 * sequence that has queries which do not see all of them. Where groups are out of order or range, sequences
 * read all their tokens themselves (but, in a batch of several launches, those of few-row launches whose own groups
 * are in order) and hk_gemm_last_device_status reports HK_ERR_INVALID_ARG.
 * By the sizes that the host knows the call runs on a tensor-core kernel for what is shared (rows of Q that are
 * 16-byte aligned, up to 64 groups), on few-row kernels, or, where
 * reading everything for each sequence costs less (few sequences, short tables, 1024 query rows of a sequence and KV head or
 * more), as hk_attention_kv8, which does not look at the groups. The table's width stands for the lengths there: a table much wider than
 * the sequences can make a small call take the form of a large one. A launch of up to 512 sequences counts its tiles of 32 tokens
 * (sequences · KV heads · what the table has room for) in 31 bits; a wider table is HK_ERR_INVALID_ARG.
 * `workspace`: device memory of hk_attention_kv8_shared_workspace_size bytes (up to 44 MB and 8 · head_dim bytes for
 * each of up to 2^17 query rows, or what hk_attention_kv8 needs), 256-byte aligned. Everything else as hk_attention_kv8. */
hk_status hk_attention_kv8_shared(const void* Q, int32_t type, const int64_t q_strides[3], const hk_kv8_cache* cache,
                                  const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                                  const int32_t* lengths, const int32_t* counts, const int32_t* groups,
                                  const int32_t* shared, int64_t G, void* O, const int64_t o_strides[3], float* lse,
                                  int64_t B, int64_t T, int64_t Hq, int32_t causal, float scale, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* The same with test controls. `flags`: HK_KV8_FEW_ROWS (units of 16 query rows) or HK_KV8_MANY_ROWS (what is shared
 * in units of 128 rows on the tensor-core kernel); each is refused for what it does not take. 0: chosen by shape;
 * HK_KV8_FAULT_DROP_ARRIVE. `timeout_ns` bounds each wait (0: 1 s). */
hk_status hk_attention_kv8_shared_ex(const void* Q, int32_t type, const int64_t q_strides[3], const hk_kv8_cache* cache,
                                     const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                                     const int32_t* lengths, const int32_t* counts, const int32_t* groups,
                                     const int32_t* shared, int64_t G, void* O, const int64_t o_strides[3], float* lse,
                                     int64_t B, int64_t T, int64_t Hq, int32_t causal, float scale, void* workspace,
                                     size_t workspace_bytes, uint32_t flags, uint64_t timeout_ns, void* stream);
size_t hk_attention_kv8_shared_workspace_size(const hk_kv8_cache* cache, int64_t B, int64_t T, int64_t Hq, int64_t max_pages,
                                              int64_t G);
/* Bytes that the call with these arguments needs, and asks for (as hk_attention_kv8_workspace_size_ex). */
size_t hk_attention_kv8_shared_workspace_size_ex(const void* Q, int32_t type, const int64_t q_strides[3],
                                                 const hk_kv8_cache* cache, int64_t max_pages, const void* O,
                                                 const int64_t o_strides[3], int64_t B, int64_t T, int64_t Hq, int64_t G,
                                                 uint32_t flags);

/* The norm of each head's query and key and the rotation by its token's position, in one pass:
 *     y = x / sqrt(mean(x^2) + eps) · w;   (a, b) -> (a cos t - b sin t, a sin t + b cos t)
 * over pairs i < `pairs` of y: (y[i], y[i + pairs]), or with `interleaved` (y[2i], y[2i + 1]); the
 * elements from 2·pairs on are not turned. t = positions[axis(i)] · inv_freq[i]: pairs [0, sections[0]) turn by
 * the first axis, the next sections[1] by the second, and so on (time, height, width; `sections` is a HOST
 * array of `axes` numbers, 1 to 4, that add up to `pairs`; NULL with one axis).
 * Q [B, T, Hq, D] and K [B, T, Hk, D] of `type` (bf16, fp16 or fp32), their outputs QO and KO, each with strides (b, t,
 * head) in elements and contiguous rows; an output may be its input (then with its strides), else it must
 * not overlap one, and its rows must not overlap. Hq or Hk 0 leaves that operand out. D a multiple of 8 up to
 * 256, pairs a multiple of 8. q_weight, k_weight [D] of `type` or fp32 (weight_type), NULL: 1. eps < 0: no
 * norm and no weights (they are not read). positions: int32 on the device with strides (axis, b, t) in elements;
 * inv_freq: fp32 [pairs] on the device, of magnitude below 2^10 (above, bits of the angle are lost; not
 * finite: NaN).
 * The norm is summed in fp32 (elements whose squares pass its range, above 10^19, make a row of zeros), t is
 * reduced to 2^-31 of a turn and then rounded to fp32, at most 2^-25.9 of a turn off whatever the position (for
 * frequencies up to 1), and the result is rounded once.
 * Asynchronous on `stream`, allocates nothing. */
hk_status hk_qk_norm_rope(const void* Q, const int64_t q_strides[3], const void* K, const int64_t k_strides[3],
                          void* QO, const int64_t qo_strides[3], void* KO, const int64_t ko_strides[3], int32_t type,
                          int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D, const void* q_weight,
                          const void* k_weight, int32_t weight_type, float eps, const int32_t* positions,
                          const int64_t pos_strides[3], const int32_t* sections, int32_t axes, const float* inv_freq,
                          int64_t pairs, int32_t interleaved, void* stream);

/* Static description of a status code. */
const char* hk_status_string(hk_status status);

/* Detail of the last error on the calling host thread (never NULL). */
const char* hk_gemm_last_error_string(void);

#ifdef __cplusplus
}
#endif

#endif /* HK_GEMM_H */
