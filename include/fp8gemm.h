/*
 * fp8gemm.h -- C ABI of the MI355X (gfx950) FP8 e4m3 fine-grained-scaled GEMM library.
 *
 * Operation.  The NT GEMM D = A . B^T (DeepGEMM digest, GeekNews topic 19459,
 * section "GEMM arayuzu ve yerlesim kisitlari": the naming is D = C + A @ B
 * with NT meaning A row-major and B stored [N,K]; this library has no C
 * addend) with DeepSeek-V3 fine-grained scaling (GeekNews topic 19444,
 * opening bullets; 7minutos.es, "Detalles y beneficios tecnicos"):
 *
 *     D[m,n] = bf16( sum_kb  P_kb[m,n] * sa[kb][m] * sb[n/128][kb] )
 *     P_kb[m,n] = sum_{k in slice kb} e4m3(A[m,k]) * e4m3(B[n,k])
 *
 * Each 128-wide K slice is computed by the matrix cores into a fresh fp32
 * partial P_kb and then scaled and added ("promoted") into an fp32
 * accumulator; the accumulator is rounded once to BF16 (nearest-even).
 *
 * Types.  FP8 operands are e4m3fn bytes (OCP: bias 7, max 448, NaN 0x7F/0xFF)
 * passed as uint8_t.  Scales are IEEE fp32.  BF16 results are uint16_t bit
 * patterns.  Kb = ceil(K/128), Nb = ceil(N/128).
 *
 * K tails.  The digest leaves K % 128 != 0 open.  Reading taken here: K must
 * be a multiple of 16 (the 16-byte row granularity of the operand loads); the
 * last K group is then partial and holds the K % 128 remaining columns, with
 * its own factors (the casts take its amax over those columns alone).  This
 * holds for the power-of-two (UE8M0) calls too; the K-grouped GEMM keeps
 * K % 128 == 0.
 *
 * Scale layouts.  Activation scales are per (row, 128-wide K group) and are
 * stored K-group-major ("transposed", as the digest requires for the LHS
 * factors): sa[kb * ld_sa + m], ld_sa >= rows.  Weight scales
 * are per 128x128 block, row-major: sb[nb * Kb + kb].
 *
 * Ownership.  Every pointer named "device" is device memory owned by the
 * caller; the library never frees or retains caller pointers.  Each GEMM or
 * cast call only enqueues kernels on `stream` (a hipStream_t; NULL is the
 * default stream) and returns: no call allocates device memory or
 * synchronises, so every call can be captured into a HIP graph (the masked
 * form, whose counts the host never learns, is made for that).  Scratch
 * memory, where a plan needs it, comes from the caller as a `workspace`
 * argument (gemm_fp8_nt_ws, the NN/TN/TT layouts, the K-grouped GEMM, the gated
 * backward pass, gemm_int4_nt, the expert layers).  The
 * one exception is the opt-in debug check FG_CHECK_DEVICE (see the grouped
 * calls), which reads a result back.
 *
 * Errors.  Preconditions that the host can check are checked before anything
 * is launched; on failure the call returns the status, launches nothing, and
 * fg_last_error() describes the failure (thread-local, valid until the next
 * call on the same thread).  A call with no output elements (M == 0 or
 * N == 0, M_total == 0, M_cap == 0) returns FG_OK without launching.  A
 * launch failure returns FG_EHIP with the HIP error string.  Preconditions on
 * device-resident metadata (expert indices, masks) are documented per call
 * and are not checked by default (checking needs a host synchronisation);
 * the debug mode FG_CHECK_DEVICE=1 checks them (see the grouped calls).
 */
#ifndef FP8GEMM_H
#define FP8GEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FG_OK = 0,
  FG_EINVAL = 1,      /* null pointer, negative size, G <= 0, leading dimension too small */
  FG_EALIGN = 2,      /* K % 16 != 0 (K % 128 != 0 where stated), M_total % 128 != 0, misaligned pointer or row stride */
  FG_EUNSUPPORTED = 3,/* sizes beyond what the kernels index (see per call) */
  FG_EHIP = 4         /* a HIP launch failed; see fg_last_error() */
} fg_status;

/*
 * Dense NT GEMM (the digest's fp8_gemm_nt without C).
 *   A   device [M, K] e4m3, row stride lda bytes   (lda >= K, lda % 16 == 0, A 16-byte aligned)
 *   sa  device fp32 [Kb][ld_sa]                    (ld_sa >= M, 4-byte aligned)
 *   B   device [N, K] e4m3, row stride ldb bytes   (ldb >= K, ldb % 16 == 0, B 16-byte aligned)
 *   sb  device fp32 [Nb][Kb]                       (4-byte aligned)
 *   D   device [M, N] bf16, row stride ldd elems   (ldd >= N, 2-byte aligned; rows that are 8- or
 *       16-byte aligned get vector stores); written
 * M, N >= 0 arbitrary; K % 16 == 0 (a partial last K group when K % 128 != 0).
 * K == 0 writes D = 0 (sa, sb may then be NULL).
 * Only D[0:M, 0:N] is written.  lda, ldb <= 4 MiB (FG_EUNSUPPORTED beyond).
 * Few rows (M <= 128) run a weight-streaming kernel; this call never splits
 * its K range over workgroups (gemm_fp8_nt_ws does, with a workspace).  The
 * kernel and plan depend only on the arguments and the device (not on the CU
 * cap, earlier calls or graph capture), so results are bit-for-bit
 * reproducible.  Allocates nothing.
 */
fg_status gemm_fp8_nt(const uint8_t* A, int64_t lda, const float* sa, int64_t ld_sa,
                      const uint8_t* B, int64_t ldb, const float* sb,
                      uint16_t* D, int64_t ldd, int M, int N, int K, void* stream);

/*
 * gemm_fp8_nt with a caller's workspace, which lets the few-row plan
 * (M <= 128) split the K range over several workgroups when the column tiles
 * alone cannot occupy the device (decode shapes); the fp32 partials of the
 * splits meet in the workspace and are added in a fixed split order, so the
 * result is reproducible and does not depend on the workspace's history.
 *   workspace        device, 256-byte aligned, or NULL (then the plan of gemm_fp8_nt)
 *   workspace_bytes  >= fg_nt_workspace_bytes(M, N, K) (FG_EINVAL otherwise); any
 *                    size works for a shape whose plan does not split (need 0)
 * Workspace contract: its first 64 KiB are arrival counters and must be zero
 * before the workspace is first used (e.g. allocate it zero-filled); every
 * call leaves them zero.  The rest holds partials and needs no
 * initialisation.  A workspace is in use until the call's work on `stream`
 * has finished; calls that may run at the same time (other streams, a graph
 * replayed on another stream) must use different workspaces.  Everything
 * else as gemm_fp8_nt; the output equals gemm_fp8_nt's within the stated
 * tolerance (bit for bit when the plan does not split).  Allocates nothing.
 */
fg_status gemm_fp8_nt_ws(const uint8_t* A, int64_t lda, const float* sa, int64_t ld_sa,
                         const uint8_t* B, int64_t ldb, const float* sb,
                         uint16_t* D, int64_t ldd, int M, int N, int K,
                         void* workspace, int64_t workspace_bytes, void* stream);

/*
 * gemm_fp8_nt_ws for callers that cannot allocate device memory at all (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation): the same plan and the same results, bit for bit, as
 * gemm_fp8_nt_ws with a large enough workspace, with the split-K buffers in
 * a scratch array of the library instead: 8 MiB + 64 KiB per GPU, a static
 * device array that each GPU the library runs on holds until the process
 * ends.  Each split call clears the arrival counters it uses (a small fill
 * kernel, no memset) before its GEMM.  Every call on one GPU shares that
 * GPU's scratch, so calls that overlap in time on one GPU (other streams,
 * graphs replayed concurrently) race; serialise them.  The plan never needs
 * more scratch than the array holds (the split is bounded by it); a plan that
 * did would return FG_EUNSUPPORTED.  Nothing is allocated; everything else as
 * gemm_fp8_nt.
 */
fg_status gemm_fp8_nt_noalloc(const uint8_t* A, int64_t lda, const float* sa, int64_t ld_sa,
                              const uint8_t* B, int64_t ldb, const float* sb,
                              uint16_t* D, int64_t ldd, int M, int N, int K, void* stream);

/* Workspace bytes gemm_fp8_nt_ws needs for (M, N, K) on the current device:
 * 0 when its plan does not split K, else 64 KiB of counters plus the
 * partials.  -1 for a negative size or when the device cannot be queried. */
int64_t fg_nt_workspace_bytes(int M, int N, int K);

/* Upper bound of fg_nt_workspace_bytes over every shape (8 MiB + 64 KiB):
 * a workspace of this size serves every call. */
int64_t fg_nt_workspace_max_bytes(void);

/*
 * Dense NT GEMM with an addend, D = C + A . B^T (the digest, "GEMM arayuzu ve
 * yerlesim kisitlari": every GEMM kernel is named after D = C + A @ B, and
 * fp8_gemm_nt computes D = C + A @ B.T).
 *   C   device fp32 [M, N], row stride ldc elems   (ldc >= N, 4-byte aligned; rows that are
 *       16-byte aligned get vector loads); read only, may not overlap D
 *   every other argument as in gemm_fp8_nt.
 * C is added to the fp32 accumulator once, after the last K slice, and the sum
 * is rounded to BF16 once.  K == 0 writes D = bf16(C).  Same kernels and
 * plans as gemm_fp8_nt (no K split).  C == NULL is FG_EINVAL when M, N > 0.
 */
fg_status gemm_fp8_nt_c(const uint8_t* A, int64_t lda, const float* sa, int64_t ld_sa,
                        const uint8_t* B, int64_t ldb, const float* sb, const float* C, int64_t ldc,
                        uint16_t* D, int64_t ldd, int M, int N, int K, void* stream);

/*
 * The other storage layouts (the digest's fp8_gemm_{nn, tn, tt}, section
 * "Dense ve Grouped GEMM"; the same D = C + A @ B naming).  The first letter
 * says whether the stored A is used as is (n: A [M, K]) or transposed (t: A
 * stored [K, M]); the second the same for B, where t is the NT form's
 * B [N, K] and n stores B as [K, N]:
 *   gemm_fp8_nn   D = C + A . B      A [M, K] (lda bytes, as in gemm_fp8_nt), B [K, N] (ldb >= N bytes)
 *   gemm_fp8_tn   D = C + A^T . B    A [K, M] (lda >= M bytes),                B [K, N] (ldb >= N bytes)
 *   gemm_fp8_tt   D = C + A^T . B^T  A [K, M] (lda >= M bytes),                B [N, K] (as in gemm_fp8_nt)
 * The scale factors belong to the logical operands, in the NT layouts: sa
 * fp32 [Kb][ld_sa] (1x128 along K for each of the M rows), sb fp32 [Nb][Kb]
 * (128x128 blocks of the [N, K] operand).  C: fp32 [M, N] addend (row stride
 * ldc >= N) or NULL for none.  D: as in gemm_fp8_nt.  An operand stored MN-major
 * has no alignment requirement on the copying path.
 * Two paths serve the MN-major operands:
 *  - copies: each MN-major operand is first transposed, K-major, into the
 *    caller's device workspace (a byte copy bound by HBM), then the NT
 *    kernels run on the copy.  The stored [K, .] operands have at most
 *    65535*128 rows (FG_EUNSUPPORTED).
 *  - copy-free: the large-tile kernel stages each MN-major operand as
 *    stored.  Each such operand must be 16-byte aligned with a row stride
 *    and a column count (M for A, N for B) that are multiples of 16.
 * workspace_bytes > 0: workspace must be 16-byte aligned and hold at least
 *    fg_layout_workspace_bytes(layout, M, N, K) bytes (FG_EINVAL otherwise);
 *    it is in use until the call's work on `stream` has finished.  The call
 *    takes the copy-free path where the operands allow it and the large
 *    kernel's 256 x 256 tiles keep the device's CUs at least three quarters
 *    busy over their rounds (measured on MI355X at M = 4096: level with or
 *    2-9 % faster than the copies there, 2-7 % slower than them at
 *    N = 2112), and the copies otherwise.  Both paths give the same bits.
 * workspace_bytes == 0 (workspace ignored): the copy-free path; operands it
 *    cannot take give FG_EALIGN.  For callers without device memory to spare.
 * K <= 2^22 (FG_EUNSUPPORTED).  K % 16 == 0.  Nothing is allocated.
 */
fg_status gemm_fp8_nn(const uint8_t* A, int64_t lda, const float* sa, int64_t ld_sa,
                      const uint8_t* B, int64_t ldb, const float* sb, const float* C, int64_t ldc,
                      uint16_t* D, int64_t ldd, int M, int N, int K,
                      void* workspace, int64_t workspace_bytes, void* stream);
fg_status gemm_fp8_tn(const uint8_t* A, int64_t lda, const float* sa, int64_t ld_sa,
                      const uint8_t* B, int64_t ldb, const float* sb, const float* C, int64_t ldc,
                      uint16_t* D, int64_t ldd, int M, int N, int K,
                      void* workspace, int64_t workspace_bytes, void* stream);
fg_status gemm_fp8_tt(const uint8_t* A, int64_t lda, const float* sa, int64_t ld_sa,
                      const uint8_t* B, int64_t ldb, const float* sb, const float* C, int64_t ldc,
                      uint16_t* D, int64_t ldd, int M, int N, int K,
                      void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes the copying path of gemm_fp8_<layout> needs for (M, N, K)
 * (a workspace of 0 bytes selects the copy-free path instead); layout is one
 * of "nt" (0), "nn", "tn", "tt".  -1 for an unknown layout, a negative size
 * or sizes the call rejects. */
int64_t fg_layout_workspace_bytes(const char* layout, int M, int N, int K);

/*
 * K-grouped TN GEMM for MoE weight gradients (the digest's
 * k_grouped_fp8_gemm_tn_contiguous, section "Dense ve Grouped GEMM": grouped
 * along K, M and N fixed).  Group g owns the ks[g] consecutive K rows that
 * start at k_g = ks[0] + .. + ks[g-1] and computes
 *     D[g] = C[g] + A_g^T . B_g          (A_g = A[k_g : k_g + ks[g], :], B_g likewise)
 *   A   device [K_total, M] e4m3, row stride lda >= M bytes (K_total = sum of ks)
 *   sa  device fp32 [K_total/128][ld_sa], ld_sa >= M: 1x128 factors along K per column m of A
 *   B   device [K_total, N] e4m3, row stride ldb >= N bytes
 *   sb  device fp32 [Nb][K_total/128]: 128x128 blocks of the logical [N, K] operand
 *   ks  HOST int [G]; each a multiple of 128 (FG_EALIGN otherwise); 0 allowed (D[g] = C[g], or 0)
 *   C   device fp32 [G, M, N] addend, contiguous, or NULL
 *   D   device bf16 [G, M, N], contiguous; written
 * Group g uses the factors of its own K groups (columns k_g/128 .. of sa
 * and sb).  Groups with ks[g] = 0 get D[g] = C[g] (or 0) from a fill
 * kernel; the groups with K rows run as one persistent launch (one per run
 * of 256 such groups), all on `stream`.  The workspace selects how the
 * operands are read:
 *  - workspace_bytes > 0: both are transposed K-major into the caller's
 *    device workspace (16-byte aligned, at least
 *    fg_k_grouped_workspace_bytes(M, N, K_total) bytes; FG_EINVAL
 *    otherwise), which is in use until the call's work on `stream` has
 *    finished.  The faster path.
 *  - workspace_bytes == 0 (workspace ignored): no copy; the kernel stages A
 *    and B as stored.  They must be 16-byte aligned, with lda, ldb, M and N
 *    multiples of 16 (FG_EALIGN otherwise).
 * K_total <= 2^22 (FG_EUNSUPPORTED).  Nothing is allocated.
 */
fg_status gemm_fp8_k_grouped_tn_contiguous(const uint8_t* A, int64_t lda, const float* sa, int64_t ld_sa,
                                           const uint8_t* B, int64_t ldb, const float* sb,
                                           const int* ks, int G, const float* C, uint16_t* D, int M, int N,
                                           void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes the copying path of gemm_fp8_k_grouped_tn_contiguous needs
 * (0 bytes selects the copy-free path); -1 for a negative size or sizes the
 * call rejects. */
int64_t fg_k_grouped_workspace_bytes(int M, int N, int64_t K_total);

/*
 * M-grouped "contiguous" GEMM (digest, section "Dense ve Grouped GEMM": the
 * experts share N and K; every expert's rows are concatenated along M and each
 * expert segment is aligned to the GEMM M block, here 128 rows).
 *   A         device [M_total, K] e4m3, packed rows (row stride K)
 *   sa        device fp32 [Kb][ld_sa], ld_sa >= M_total
 *   B         device [G, N, K] e4m3, packed
 *   sb        device fp32 [G][Nb][Kb]
 *   m_indices device int32 [M_total]: expert of each row, or -1 for a padding row
 *   D         device [M_total, N] bf16, packed (row stride N)
 * M_total % 128 == 0, K % 16 == 0, G >= 1.
 * Device-side precondition (not checked): within each aligned 128-row block
 * every non-negative index is the same value e < G.  The block is computed
 * against B[e], where e is the largest index in the block below G; rows whose
 * index is not e (padding) are left untouched; a block of padding only is
 * skipped.  An index >= G counts as padding, so no weight outside B is ever
 * addressed.
 * Debug mode: with the environment variable FG_CHECK_DEVICE=1 a check kernel
 * validates m_indices first and the host reads its result back (this
 * synchronises the stream, and the call returns FG_EINVAL while the stream
 * is being captured); an index outside [-1, G), or one that differs from the
 * other non-negative indices of its 128-row block, returns FG_EINVAL naming
 * the row, and the GEMM is not launched.
 */
fg_status gemm_fp8_grouped_contiguous(const uint8_t* A, const float* sa, int64_t ld_sa,
                                      const uint8_t* B, const float* sb,
                                      const int32_t* m_indices,
                                      uint16_t* D, int M_total, int N, int K, int G, void* stream);

/*
 * M-grouped "masked" GEMM for decoding (digest, "Dense ve Grouped GEMM": the
 * per-expert token count lives on the device, the CPU does not know it, and
 * only the valid region is computed).
 *   A        device [G, M_cap, K] e4m3, packed
 *   sa       device fp32 [G][Kb][ld_sa], ld_sa >= M_cap
 *   B        device [G, N, K] e4m3, packed
 *   sb       device fp32 [G][Nb][Kb]
 *   masked_m device int32 [G]: valid rows of each group
 *   D        device [G, M_cap, N] bf16, packed
 *   expected_m  host hint of the typical count (0 = unknown); accepted for interface compatibility,
 *               the plan does not use it (measured: the tile width chosen from G, M_cap and N is best)
 * Group g computes rows [0, clamp(masked_m[g], 0, M_cap)); every other row of
 * D[g] is left untouched (bit for bit).  K % 16 == 0, G >= 1.
 * Debug mode (FG_CHECK_DEVICE=1, as for the contiguous form): a count
 * outside [0, M_cap], which the unchecked call clamps, returns FG_EINVAL
 * naming the group, and the GEMM is not launched.
 */
fg_status gemm_fp8_grouped_masked(const uint8_t* A, const float* sa, int64_t ld_sa,
                                  const uint8_t* B, const float* sb,
                                  const int32_t* masked_m,
                                  uint16_t* D, int G, int M_cap, int N, int K,
                                  int expected_m, void* stream);

/*
 * Per-token (1 x 128) FP8 cast of activations (the digest leaves casting to
 * the user, "GEMM arayuzu ve yerlesim kisitlari"; this is the library's own
 * helper).  For each row m and group kb:
 *     amax = max |x[m, 128kb : min(128kb+128, K)]|
 *     s    = max(amax, 1e-4f) / 448          (fp32, correctly rounded)
 *     q    = e4m3_RNE(x / s)                 (fp32 division, nearest-even)
 *   x   device fp32 [M, K], row stride ldx elements (ldx >= K, ldx % 4 == 0, 16-byte aligned)
 *   q   device [M, K] e4m3, packed (row stride K), 8-byte aligned
 *   sa  device fp32 [Kb][ld_sa], ld_sa >= M (written; the GEMM's activation-scale layout)
 * K % 16 == 0 (the last group holds K % 128 columns when K % 128 != 0).
 * Input values must be finite.
 */
fg_status fp8_cast_per_token(const float* x, int64_t ldx, uint8_t* q, float* sa, int64_t ld_sa,
                             int M, int K, void* stream);

/*
 * Per-block (128 x 128) FP8 cast of a weight matrix, same formula with amax
 * taken over each 128x128 block (the last row block covers N % 128 rows, the
 * last column block K % 128 columns).
 *   w   device fp32 [N, K], row stride ldw elements (ldw >= K, ldw % 4 == 0, 16-byte aligned)
 *   q   device [N, K] e4m3, packed, 4-byte aligned
 *   sb  device fp32 [Nb][Kb] (written; the GEMM's weight-scale layout)
 * K % 16 == 0.  For expert weights [G, N, K] with N % 128 == 0 one call on
 * [G*N, K] yields the [G][Nb][Kb] layout; otherwise call once per expert.
 */
fg_status fp8_cast_per_block(const float* w, int64_t ldw, uint8_t* q, float* sb,
                             int N, int K, void* stream);

/*
 * The same two casts from BF16 inputs (raw bf16 bit patterns).  Each input
 * is widened to fp32 exactly and then quantised as fp8_cast_per_token /
 * fp8_cast_per_block quantise that fp32 value (same formula, same outputs).
 *   x   device bf16 [M, K], row stride ldx elements (ldx >= K, ldx % 8 == 0), 16-byte aligned
 *   w   device bf16 [N, K], row stride ldw elements (ldw >= K, ldw % 4 == 0), 16-byte aligned
 * Other arguments, outputs and errors as for the fp32-input casts.
 */
fg_status fp8_cast_per_token_bf16(const uint16_t* x, int64_t ldx, uint8_t* q, float* sa, int64_t ld_sa,
                                  int M, int K, void* stream);
fg_status fp8_cast_per_block_bf16(const uint16_t* w, int64_t ldw, uint8_t* q, float* sb,
                                  int N, int K, void* stream);

/*
 * Power-of-two (UE8M0) scale factors.  The digest's layout section
 * ("GEMM arayuzu ve yerlesim kisitlari") gives the newer architecture's
 * factors as UE8M0 -- an unsigned exponent byte e, value 2^(e - 127) -- packed
 * four to a 32-bit integer.  Same granularity as the fp32 factors; four
 * consecutive K groups share an int32, K group 4i + j in byte j (least
 * significant first).  Kb4 = ceil(Kb / 4).
 *
 * Dense GEMM  D = bf16( sum_kb 2^(sa - 127) 2^(sb - 127) (A_kb . B_kb^T) )
 *   A   device [M, K] e4m3, row stride lda bytes (lda >= K, lda % 16 == 0), 16-byte aligned
 *   sa  device int32 [Kb4][ld_sa], ld_sa >= M: byte kb % 4 of sa[kb / 4][m] is row m's factor
 *       of K group kb
 *   B   device [N, K] e4m3, row stride ldb bytes (ldb >= K, ldb % 16 == 0), 16-byte aligned
 *   sb  device int32 [Nb][Kb4]: byte kb % 4 of sb[nb][kb / 4] is block (nb, kb)'s factor
 *   D   device [M, N] bf16, row stride ldd elements
 * The matrix cores apply the factors (gfx950's scaled FP8 MFMA) and add each
 * 128-deep slice into fp32 accumulators; the output is the same definition
 * as gemm_fp8_nt with factors 2^(e - 127).  Factor bytes 0 and 255 are not
 * meaningful inputs (the casts below never write them).  K % 16 == 0 (a
 * partial last K group when K % 128 != 0), lda, ldb <= 4 MiB.  Allocates
 * nothing; errors as for gemm_fp8_nt.
 */
fg_status gemm_fp8_nt_ue8m0(const uint8_t* A, int64_t lda, const int32_t* sa, int64_t ld_sa,
                            const uint8_t* B, int64_t ldb, const int32_t* sb,
                            uint16_t* D, int64_t ldd, int M, int N, int K, void* stream);

/*
 * Contiguous M-grouped GEMM (digest, "Dense ve Grouped GEMM") with
 * power-of-two factors: gemm_fp8_grouped_contiguous's layout and row mapping,
 * with the factors of gemm_fp8_nt_ue8m0.
 *   A          device [M_total, K] e4m3, packed
 *   sa         device int32 [Kb4][ld_sa], ld_sa >= M_total (packed as for gemm_fp8_nt_ue8m0)
 *   B          device [G, N, K] e4m3, packed
 *   sb         device int32 [G][Nb][Kb4]
 *   m_indices  device int32 [M_total]: expert of each row, -1 = padding row
 *   D          device [M_total, N] bf16, packed
 * Row m with m_indices[m] = e in [0, G) is computed with expert e's weights
 * as gemm_fp8_nt_ue8m0 computes it; padding rows of D are left untouched.
 * Each 128-row block holds one expert (or padding).  K % 16 == 0,
 * M_total % 128 == 0, G >= 1.  Allocates nothing; errors as for
 * gemm_fp8_grouped_contiguous.
 */
fg_status gemm_fp8_grouped_contiguous_ue8m0(const uint8_t* A, const int32_t* sa, int64_t ld_sa,
                                            const uint8_t* B, const int32_t* sb,
                                            const int32_t* m_indices,
                                            uint16_t* D, int M_total, int N, int K, int G, void* stream);

/*
 * Masked grouped GEMM (decode; digest, "Dense ve Grouped GEMM") with
 * power-of-two factors: gemm_fp8_grouped_masked's layout and row masking,
 * with the factors of gemm_fp8_nt_ue8m0 packed per group.
 *   A        device [G, M_cap, K] e4m3, packed
 *   sa       device int32 [G][Kb4][ld_sa], ld_sa >= M_cap (packed as for gemm_fp8_nt_ue8m0)
 *   B        device [G, N, K] e4m3, packed
 *   sb       device int32 [G][Nb][Kb4]
 *   masked_m device int32 [G]: valid rows of each group
 *   D        device [G, M_cap, N] bf16, packed
 *   expected_m  accepted for interface compatibility; not used
 * Group g computes rows [0, clamp(masked_m[g], 0, M_cap)) as gemm_fp8_nt_ue8m0
 * computes them; every other row of D[g] is left untouched (bit for bit).
 * K % 16 == 0, G >= 1.  Allocates nothing; errors as for
 * gemm_fp8_grouped_masked.
 */
fg_status gemm_fp8_grouped_masked_ue8m0(const uint8_t* A, const int32_t* sa, int64_t ld_sa,
                                        const uint8_t* B, const int32_t* sb,
                                        const int32_t* masked_m,
                                        uint16_t* D, int G, int M_cap, int N, int K,
                                        int expected_m, void* stream);

/*
 * Per-token (1 x 128) cast with power-of-two factors: as fp8_cast_per_token,
 * but the fp32 factor max(amax, 1e-4f) / 448 is rounded up to the next power
 * of two 2^(e - 127) (so no code saturates) and e is written as a byte:
 *   sa  device int32 [Kb4][ld_sa], ld_sa >= M; byte kb % 4 of sa[kb / 4][m] is
 *       written for every kb < Kb (bytes for K groups >= Kb are not written)
 */
fg_status fp8_cast_per_token_ue8m0(const float* x, int64_t ldx, uint8_t* q, int32_t* sa, int64_t ld_sa,
                                   int M, int K, void* stream);

/*
 * Per-block (128 x 128) cast with power-of-two factors (rounding as above):
 *   sb  device int32 [Nb][Kb4]; byte kb % 4 of sb[nb][kb / 4] is written for every kb < Kb
 */
fg_status fp8_cast_per_block_ue8m0(const float* w, int64_t ldw, uint8_t* q, int32_t* sb,
                                   int N, int K, void* stream);

/*
 * The two power-of-two-factor casts from BF16 inputs (raw bf16 bit patterns),
 * widened to fp32 exactly first, as fp8_cast_per_token_bf16 /
 * fp8_cast_per_block_bf16 do:
 *   x   device bf16 [M, K], row stride ldx elements (ldx >= K, ldx % 8 == 0), 16-byte aligned
 *   w   device bf16 [N, K], row stride ldw elements (ldw >= K, ldw % 4 == 0), 16-byte aligned
 * Other arguments, outputs and errors as for fp8_cast_per_token_ue8m0 /
 * fp8_cast_per_block_ue8m0.
 */
fg_status fp8_cast_per_token_ue8m0_bf16(const uint16_t* x, int64_t ldx, uint8_t* q, int32_t* sa, int64_t ld_sa,
                                        int M, int K, void* stream);
fg_status fp8_cast_per_block_ue8m0_bf16(const uint16_t* w, int64_t ldw, uint8_t* q, int32_t* sb,
                                        int N, int K, void* stream);

/*
 * 8-bit-integer products and the gated feed-forward block.  Operands are
 * signed bytes with an fp32 scale per row (a token of the activations, an
 * output channel of the weights), or BF16.  All matrices are row-major with
 * their last dimension contiguous.
 * Rows that lie a multiple of 128 bytes apart load fastest (others cost up to
 * 30 % of a product's time).
 * Only the backward pass needs a workspace.  Their plans depend only on the
 * arguments, the device, the CU cap and the environment variable
 * FG_LINEAR_PLAN (read in every call, for tuning and tests: it forces a plan,
 * and with it the order of bf16 sums).  Sums have a fixed order in every plan,
 * so results are reproducible.
 */

/*
 * Cast of each row to signed bytes, for either operand of gemm_int8_nt:
 *     s[m] = max(max_k |x[m, k]|, 1e-4f) * (1.0f / 127.0f)    (fp32)
 *     q    = rint(x / s[m])                                   (fp32 division, nearest-even; |q| <= 127)
 *   x   device fp32 (or bf16) [M, K], row stride ldx elements (ldx >= K, 16-byte aligned rows)
 *   q   device [M, K], packed, 16-byte aligned
 *   s   device fp32 [M]
 * K % 16 == 0.  Input values must be finite.  K == 0 (the largest of no
 * values is 0) writes s alone and reads neither x nor q.
 */
fg_status int8_cast_per_row(const float* x, int64_t ldx, int8_t* q, float* s, int M, int K, void* stream);
fg_status int8_cast_per_row_bf16(const uint16_t* x, int64_t ldx, int8_t* q, float* s, int M, int K, void* stream);

/*
 * D[m,n] = bf16( sa[m] * sb[n] * sum_k A[m,k] * B[n,k] ), the sum exact in int32.
 *   A   device [M, K] int8, row stride lda bytes (lda >= K, lda % 16 == 0, A 16-byte aligned)
 *   sa  device fp32 [M]
 *   B   device [N, K] int8, row stride ldb bytes (ldb >= K, ldb % 16 == 0, B 16-byte aligned)
 *   sb  device fp32 [N]
 *   D   device [M, N] bf16, row stride ldd elements (ldd >= N); only D[0:M, 0:N] is written
 * 0 <= M <= 2^30, 0 <= N <= 2^29, K % 16 == 0, K <= 131056 (the sum of more
 * products may leave int32), rows of at most 4 MiB (FG_EUNSUPPORTED past these
 * limits).  K == 0 writes D = sa * sb * 0.  The product is scaled as (sum * sa[m]) * sb[n] in fp32 and
 * rounded once.  D may not overlap an input.  Allocates nothing.
 */
fg_status gemm_int8_nt(const int8_t* A, int64_t lda, const float* sa, const int8_t* B, int64_t ldb, const float* sb,
                       uint16_t* D, int64_t ldd, int M, int N, int K, void* stream);

/* Activations of the gated block: act(x) = x / (1 + exp(-y)), y = x (SiLU) or
 * y = 2 sqrt(2/pi) (x + 0.044715 x^3) (the tanh form of GELU). */
typedef enum { FG_ACT_SILU = 0, FG_ACT_GELU_TANH = 1 } fg_activation;

/*
 * Gated feed-forward block: both projections, the activation and the product
 * in one kernel,
 *     g = X . W[0:F]^T,  u = X . W[F:2F]^T,  H = bf16( act(g) * u ).
 *   X   device [M, K] bf16, row stride ldx elements (ldx >= K, ldx % 8 == 0, X 16-byte aligned)
 *   W   device [2F, K] bf16, gate rows then up rows, row stride ldw elements (as ldx)
 *   H   device [M, F] bf16, row stride ldh elements (ldh >= F); written
 *   P   NULL, or device fp32 [M, 2F] (row stride ldp >= 2F): receives [g u] for the backward pass
 * 0 <= M <= 2^30, 0 <= F <= 2^29, K % 8 == 0 (K == 0: g = u = 0), rows of X
 * and W of at most 4 MiB.
 * g and u are accumulated in fp32 and not rounded before the activation.  H
 * and P may not overlap each other or an input.  Allocates nothing.
 */
fg_status gated_ffn_bf16(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, uint16_t* H, int64_t ldh,
                         float* P, int64_t ldp, int M, int F, int K, int activation, void* stream);

/*
 * Its gradients, given dH:
 *     dg = dH * u * act'(g),  du = dH * act(g),
 *     dX = bf16( [dg du] . W ),  dW = bf16( [dg du]^T . X ).
 *   dH  device [M, F] bf16, row stride lddh
 *   X, W as in the forward call
 *   P   the forward call's pre-activations [g u], or NULL: they are recomputed from X and W
 *   dX  device [M, K] bf16, row stride lddx, or NULL (not wanted)
 *   dW  device [2F, K] bf16, row stride lddw, or NULL (not wanted)
 *   workspace  device, 256-byte aligned, fg_gated_ffn_backward_workspace_bytes(M, F, K) bytes; holds
 *       [dg du] in bf16 and, where dX or the pair is small, fp32 partials of their sums (at most
 *       32 MiB); needs no initialisation; in use until the call's work has finished
 * dX and dW accumulate in fp32 over the bf16 pair [dg du].  M == 0 writes
 * dW = 0, F == 0 writes dX = 0.  M <= 2^30; F <= 2^20 (a row of [dg du] is at
 * most 4 MiB; with M == 0, F <= 2^28); K and rows of X and W as in the forward
 * call.  Outputs may not overlap inputs.
 */
fg_status gated_ffn_bf16_backward(const uint16_t* dH, int64_t lddh, const uint16_t* X, int64_t ldx,
                                  const uint16_t* W, int64_t ldw, const float* P, int64_t ldp, uint16_t* dX,
                                  int64_t lddx, uint16_t* dW, int64_t lddw, int M, int F, int K, int activation,
                                  void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes of gated_ffn_bf16_backward; -1 for negative sizes, M or K
 * above 2^30 and F above 2^28.  The call's other limits (F <= 2^20 with M > 0,
 * K % 8 == 0, rows of 4 MiB) are not looked at here. */
int64_t fg_gated_ffn_backward_workspace_bytes(int M, int F, int K);

/*
 * The gated block on 8-bit integers (serving):
 *     g = sx * sw[0:F] * (X . W[0:F]^T),  u likewise with rows F..2F-1,  H = bf16( act(g) * u ).
 *   X, sx, W, sw  as A, sa, B, sb of gemm_int8_nt, W and sw of 2F rows
 *   H             device [M, F] bf16, row stride ldh (ldh >= F); written
 * M, F, K as M, N, K in gemm_int8_nt.  H may not overlap an input.
 * Allocates nothing.
 */
fg_status gated_ffn_int8(const int8_t* X, int64_t ldx, const float* sx, const int8_t* W, int64_t ldw,
                         const float* sw, uint16_t* H, int64_t ldh, int M, int F, int K, int activation,
                         void* stream);

/*
 * 4-bit weights with a scale for each group of a row, and their product with a
 * few rows of bf16 activations.
 *
 * Packing.  Columns 8 i .. 8 i + 7 of a row are one little-endian 32-bit word:
 * column 8 i + j in bits 8 j .. 8 j + 3 and column 8 i + 4 + j in bits 8 j + 4 ..
 * 8 j + 7 (j < 4).  A row is padded to whole chunks of 128 columns (64 bytes);
 * columns 32 m + 8 q .. 32 m + 8 q + 7 of a chunk (m, q < 4) are its word 4 q + m.
 * What padding words hold does not matter to the products.
 *
 * Groups.  `group` is 32, 64 or a multiple of 128; group g of a row is its
 * columns g group .. (g + 1) group - 1, the last one may be partial.  K % 32 == 0.
 * With Kg = ceil(K / group), Kp = ceil(K / 128):
 *   q  device [N][64 Kp] bytes, packed, 16-byte aligned
 *   s  device bf16 [N][Kg]
 *   z  NULL (every zero point is 8), or device uint8 [N][Kg], 0 <= z <= 255
 * stand for w[n,k] = s[n, k / group] * (q[n,k] - z[n, k / group]).
 */

/*
 * Cast of weights to this form (x: fp32, or bf16 widened exactly), in fp32 steps:
 *   z == NULL:  s = bf16(max(max |x|, 1e-20f) / 7),                q = clamp(rint(x / s) + 8, 0, 15)
 *   else:       lo = min(min x, 0), hi = max(max x, 0),
 *               s = bf16(max(hi - lo, 1e-20f) / 15), z = clamp(rint(-lo / s), 0, 15),
 *               q = clamp(rint(x / s) + z, 0, 15)
 * over each group.  w: device [N, K], row stride ldw elements (ldw >= K,
 * 16-byte aligned rows).  Padding words are written as zeros.  Input values must
 * be finite; hi - lo may pass the largest fp32 (it is taken of halves).
 * K <= 2^20.  N == 0 or K == 0 writes nothing.
 */
fg_status int4_cast_per_group(const float* w, int64_t ldw, uint8_t* q, uint16_t* s, uint8_t* z, int N, int K, int group,
                              void* stream);
fg_status int4_cast_per_group_bf16(const uint16_t* w, int64_t ldw, uint8_t* q, uint16_t* s, uint8_t* z, int N, int K,
                                   int group, void* stream);

/*
 * D[m,n] = bf16( sum_k A[m,k] * sb[n, k / group] * (B[n,k] - zb[n, k / group]) )
 *   A   device [M, K] bf16, row stride lda elements (lda >= K, lda % 8 == 0, 16-byte aligned, rows of at most 4 MiB)
 *   B, sb, zb  4-bit weights [N, K] as above (zb may be NULL)
 *   D   device [M, N] bf16, row stride ldd elements (ldd >= N); only D[0:M, 0:N] is written
 *   workspace  NULL, or device, 256-byte aligned, fg_int4_workspace_bytes(M, N, K) bytes (0 for
 *       most sizes); needs no initialisation; in use until the call's work has finished
 * Made for M <= 64, where HBM is read for the weights once; more rows are taken
 * 16 to 64 at a time.  M <= 2^20, N <= 2^26, K % 32 == 0, K <= 2^20.  K == 0
 * writes zeros.  Sums are in fp32, the zero point is taken out of a group's sum
 * once (so that sum |A| B and zb sum |A| of a group must stay below fp32's largest
 * number), and the result is rounded once.  A row of A with an infinity or a NaN
 * gives a row of D that holds infinities or NaN.  Sums have a fixed order, which
 * depends on the sizes only.  The workspace and D may not overlap anything else.
 * Allocates nothing.  Runs as one kernel, or two where the reduction is split.
 */
fg_status gemm_int4_nt(const uint16_t* A, int64_t lda, const uint8_t* B, const uint16_t* sb, const uint8_t* zb,
                       uint16_t* D, int64_t ldd, int M, int N, int K, int group, void* workspace,
                       int64_t workspace_bytes, void* stream);

/* Workspace bytes of gemm_int4_nt; -1 for sizes that it refuses. */
int64_t fg_int4_workspace_bytes(int M, int N, int K);

/* Scores of the expert router: a softmax over the experts, or a sigmoid of each logit. */
typedef enum { FG_SCORE_SOFTMAX = 0, FG_SCORE_SIGMOID = 1 } fg_scoring;

/*
 * Expert router.  For each token, s = softmax(l) or sigmoid(l), and the k experts
 * with the largest s + bias (without a bias and with one group: with the largest
 * logits); equal ones in the order of their indices.  With groups > 1 the E /
 * groups consecutive experts of a group stand together: a group's value is the
 * sum of its two largest s + bias, and only experts of the top_groups groups
 * with the largest values are candidates.
 *   logits   device fp32 (or bf16) [T, E], row stride ld elements
 *   bias     NULL, or device fp32 [E]
 *   ids      device int32 [T, k]: the chosen experts, best first
 *   weights  device fp32 [T, k]: scale * s of the chosen, with `normalize` over
 *            the sum of the chosen s (0 where that is 0)
 * An expert whose logit (or bias) is -infinity is no candidate; places that no
 * candidate is left for hold id -1 and weight 0.  A NaN is chosen after all
 * numbers and gives NaN weights: under softmax all of its row's, and so does
 * +infinity.
 * T <= 2^25, 1 <= k <= min(E, 64), E <= 1024, groups <= 64 divides E.  Scores and
 * what they are compared by are computed in 64 bits, weights are rounded once.
 * One kernel, no workspace.
 */
fg_status moe_route(const float* logits, int64_t ld, const float* bias, int32_t* ids, float* weights, int T, int E, int k,
                    int scoring, int groups, int top_groups, int normalize, float scale, void* stream);
fg_status moe_route_bf16(const uint16_t* logits, int64_t ld, const float* bias, int32_t* ids, float* weights, int T, int E,
                         int k, int scoring, int groups, int top_groups, int normalize, float scale, void* stream);

/*
 * Its gradient: dlogits (device, the logits' type, [T, E], row stride ld_dl;
 * every element is written) from dweights (device fp32 [T, k]), the logits and
 * the forward call's ids, scoring, normalize and scale.  Places whose id is not
 * in [0, E) have no gradient, and their dweights are not read; the choice itself
 * and the bias have none.  With an id in two places of a row both add up.  Under
 * softmax a NaN or +infinity among a row's logits gives NaN for all of the row.
 */
fg_status moe_route_backward(const float* dweights, const float* logits, int64_t ld, const int32_t* ids, float* dlogits,
                             int64_t ld_dl, int T, int E, int k, int scoring, int normalize, float scale, void* stream);
fg_status moe_route_backward_bf16(const float* dweights, const uint16_t* logits, int64_t ld, const int32_t* ids,
                                  uint16_t* dlogits, int64_t ld_dl, int T, int E, int k, int scoring, int normalize,
                                  float scale, void* stream);

/*
 * A whole expert layer for a few tokens, in two kernels (for more of them a third
 * adds partial sums):
 *     D[t] = bf16( sum_j weights[t,j] * W2[e] . h ),  e = ids[t,j],
 *     h = act(g) * u,  g = W1[e][0:F] . X[t],  u = W1[e][F:2F] . X[t].
 *   X    device [T, K] bf16, row stride ldx elements (ldx >= K, ldx % 8 == 0, 16-byte aligned, rows of at most 4 MiB)
 *   W1   device [E, 2F, K] e4m3, packed, gate rows then up rows, 16-byte aligned
 *   s1   device fp32 [E][ceil(2F/128)][ceil(K/128)]   (fp8_cast_per_block of each expert's W1)
 *   W2   device [E, K, F] e4m3, packed, 16-byte aligned
 *   s2   device fp32 [E][ceil(K/128)][ceil(F/128)]
 *   ids  device int32 [T, k]; a place whose id is not in [0, E) is left out
 *        (moe_route's -1, or an expert of another device), and its weight is not read
 *   weights  device fp32 [T, k]
 *   D    device [T, K] bf16, row stride ldd elements (ldd >= K); a token with no place left gets zeros
 *   workspace  device, 256-byte aligned, fg_moe_ffn_workspace_bytes(T, k, F) bytes; needs no
 *        initialisation; in use until the call's work has finished
 * Activations are not quantised: products are of bf16 X (or of h, kept in fp32)
 * with the exact values of the codes, summed in fp32; D is rounded once.  A token
 * that names an expert twice has the sum of both weights.  For each 64 tokens the
 * weights of every named expert are read from HBM once.  A kernel takes 1 to 32
 * tokens of an expert at a time, by the average over the experts (1 or 2 where most
 * have a token or none), and streams the expert's weights again for each further so
 * many, from cache where they fit: ids that crowd on few experts take longer than
 * ids that are spread over the same ones.  With hundreds of tokens the grouped GEMMs
 * are faster (e4m3; there are none on 4-bit weights).  Sums have a fixed order, which
 * depends on the sizes and ids only.
 * T <= 2^20, 1 <= k <= 32, 1 <= E <= 1024, K and F multiples of 16 up to 2^16.
 * F == 0 writes zeros.  The workspace and D may not overlap anything else; calls
 * that may run at the same time (two streams, two graphs) need a workspace each.
 * Allocates nothing.
 */
fg_status moe_ffn_fp8(const uint16_t* X, int64_t ldx, const uint8_t* W1, const float* s1, const uint8_t* W2,
                      const float* s2, const int32_t* ids, const float* weights, uint16_t* D, int64_t ldd, int T, int k,
                      int E, int F, int K, int activation, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * The same on 4-bit weights (see int4_cast_per_group):
 *   W1, s1, z1  E matrices of [2F, K], one after the other; W2, s2, z2  E of [K, F]
 *   (z1 and z2 are both given, or both NULL: FG_EINVAL otherwise)
 * K and F multiples of 32 up to 2^16.  Everything else as moe_ffn_fp8.
 */
fg_status moe_ffn_int4(const uint16_t* X, int64_t ldx, const uint8_t* W1, const uint16_t* s1, const uint8_t* z1,
                       const uint8_t* W2, const uint16_t* s2, const uint8_t* z2, const int32_t* ids, const float* weights,
                       uint16_t* D, int64_t ldd, int T, int k, int E, int F, int K, int group, int activation,
                       void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes of moe_ffn_fp8 and moe_ffn_int4; -1 for sizes that both refuse. */
int64_t fg_moe_ffn_workspace_bytes(int T, int k, int F);

/* Row alignment of each expert segment in the contiguous layout: 128. */
int fg_get_mk_alignment_for_contiguous_layout(void);

/* Cap on the compute units the GEMM kernels spread their persistent workgroups
 * over (the digest's set_num_sms); 0 (the default) means all of them.  Kernels
 * without persistent workgroups do not follow it: the few-row (decode) kernels,
 * the casts and copies, the router, the 4-bit product and the few-token expert
 * layers, and the gated backward pass's gradient pair (from kept pre-activations or
 * partial sums) and addition of partial sums.
 * Results do not depend on the cap (every tile is computed whole by one
 * workgroup), but for the bf16 gated block and its gradients, whose plan,
 * and so the order of their fp32 sums, follows it.  Process-wide, not thread-safe against concurrent launches. */
void fg_set_num_cus(int n);
int fg_get_num_cus(void);

/* Description of the last failure on this thread ("" after success). */
const char* fg_last_error(void);

/* Library version string. */
const char* fg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8GEMM_H */
