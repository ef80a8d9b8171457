/* Tokens drawn from logits by temperature, top-k, top-p and min-p from given random numbers,
 * and the probabilities that these settings leave (what draft_verify takes as target and draft).
 *
 * Row t has logits l_v, v < vocab, a temperature T, a count k, a mass p, a share m and a uniform
 * u in [0, 1). With L the largest logit and z_v = (L - l_v) * min(log2(e) / T, FLT_MAX) in fp32
 * (every operation rounded to nearest, log2(e) = 0x1.715476p0; z_v = 0 where l_v = L), n = floor(z)
 * and f = z - n, the weight of a token is a whole number,
 *   w_v = floor(P(f) * 2^(40 - n)), 0 where z_v >= 41,
 *   P(f) = 1 + f (c1 + f (c2 + f (c3 + f (c4 + f (c5 + f c6))))) in fp32, every product and sum
 *   rounded to nearest: 2^-f for f in [0, 1) within 2^-22.3 of its value
 *   (c1 .. c6 = -0x1.62e42cp-1, 0x1.ebfacp-3, -0x1.c6948ep-5, 0x1.39e3fcp-7, -0x1.4e2aeap-10,
 *   0x1.c946d2p-14: the minimax polynomial of that form, rounded to fp32).
 * So 2^40 stands for the largest token, and a token below 2^-40 of it (27.7 in l / T) weighs 0. The
 * order of the tokens is by logit, larger first, then by index, smaller first. Kept are
 *   - of all tokens, the first k (top-k; k <= 0: all),
 *   - of these, the shortest beginning whose weights sum to at least p times the sum of them
 *     (top-p; p >= 1: all; p <= 0: the first token),
 *   - of these, the tokens with w_v >= m * 2^40 (min-p; m <= 0: all).
 * With S the sum of the kept weights, the token drawn is the least v with w_0 + .. + w_v >
 * floor(u * S), the sum over kept tokens; the probability of a kept token is w_v / S, of another 0.
 * T = 0 keeps the first token alone. Sums are 64-bit integers and every comparison is exact, so a
 * result does not depend on the order of the sums: it is the same on every run and for every
 * split of the vocabulary.
 */
#ifndef TOKEN_SAMPLE_H
#define TOKEN_SAMPLE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* sample_stream_t; /* identical to cudaStream_t */

/* Types of the logits. */
enum { SAMPLE_BF16 = 0, SAMPLE_FP16 = 1, SAMPLE_FP32 = 2 };

/* Host-side return codes (negative: nothing was enqueued). */
enum {
  SAMPLE_OK = 0,
  SAMPLE_ERR_NULL = -1,   /* logits NULL (with rows > 0), tokens without uniforms, or neither
                             tokens nor probs */
  SAMPLE_ERR_SHAPE = -2,  /* rows < 0 or > 2^27, vocab < 1 or > 2^20, a row stride below vocab,
                             param_rows < 1, dtype unknown */
  SAMPLE_ERR_ALIGN = -3,  /* an array not aligned to its elements */
  SAMPLE_ERR_CUDA = -4    /* the launch or a device query failed */
};

/* Device status bits, OR-ed into *status. */
enum {
  SAMPLE_STATUS_NAN = 1,     /* a logit is NaN: taken as -infinity */
  SAMPLE_STATUS_EMPTY = 2,   /* every logit of a row is -infinity: its token is -1, its
                                probabilities are 0 */
  SAMPLE_STATUS_PARAM = 4,   /* a setting is NaN, a temperature negative or infinite, a min-p
                                above 1: T is taken as 1, top-p and min-p as off */
  SAMPLE_STATUS_UNIFORM = 8  /* a uniform outside [0, 1) or NaN: clamped (NaN to 0) */
};

/* One launch.
 *   logits       device [rows, ld], bf16, fp16 or fp32; -infinity excludes a token
 *   temperature  device float32 [ceil(rows / param_rows)] or NULL (1)
 *   top_k        device int32 of the same length or NULL (off)
 *   top_p        device float32 of the same length or NULL (off)
 *   min_p        device float32 of the same length or NULL (off)
 *   param_rows   rows t of one t / param_rows share their settings (a verify step's rows)
 *   uniforms     device float32 [rows]; may be NULL where tokens is
 *   tokens       device int32 [rows] or NULL
 *   probs        device float32 [rows, probs_ld] or NULL; may not overlap the logits
 *   status       device int32 [1] or NULL: SAMPLE_STATUS_* bits OR-ed in */
int token_sample(const void* logits, int64_t ld, int dtype, int rows, int vocab,
                 const float* temperature, const int32_t* top_k, const float* top_p,
                 const float* min_p, int param_rows, const float* uniforms, int32_t* tokens,
                 float* probs, int64_t probs_ld, int32_t* status, sample_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TOKEN_SAMPLE_H */
