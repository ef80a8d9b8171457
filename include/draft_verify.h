/* Verification of drafted tokens against the target's probabilities from given random
 * numbers (speculative decoding: the tokens come out distributed as the target's own).
 *
 * Request j has n drafted tokens d_0 .. d_{n-1}, target rows p_0 .. p_n, draft rows
 * q_0 .. q_{n-1}, and uniforms in [0, 1): u_0 .. u_{n-1} test the drafts, r draws.
 *   - the first a drafts are kept, a the least i with not (u_i * q_i(d_i) < p_i(d_i))
 *     (decided exactly), or n if there is none;
 *   - one more token is drawn from the weights w = max(p_a - q_a, 0) if a < n, and p_n
 *     if a = n (p_a where max(p_a - q_a, 0) is 0 everywhere): the least v with
 *     w(0) + .. + w(v) > floor(r * (w(0) + .. + w(V - 1))).
 * Without draft probabilities the draft is a point mass: q_i is 1 at d_i, 0 elsewhere.
 * For the draw, probabilities are whole multiples of 2^-60 (rounded to nearest even),
 * subtracted and summed as 64-bit integers, so the result does not depend on the order
 * of the sums: it is the same on every run and for every split of the vocabulary.
 */
#ifndef DRAFT_VERIFY_H
#define DRAFT_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* verify_stream_t; /* identical to cudaStream_t */

/* Host-side return codes (negative: nothing was enqueued). */
enum {
  VERIFY_OK = 0,
  VERIFY_ERR_NULL = -1,   /* a required pointer is NULL (with reqs > 0) */
  VERIFY_ERR_SHAPE = -2,  /* reqs < 0, drafts outside [0, VERIFY_MAX_DRAFTS], vocab < 1 or
                             > 2^30, a row stride below vocab, a request stride below 0 */
  VERIFY_ERR_ALIGN = -3,  /* an array not 4-byte aligned */
  VERIFY_ERR_CUDA = -4    /* the launch or a device query failed */
};

/* Device status bits, OR-ed into *status. */
enum {
  VERIFY_STATUS_COUNT = 1,  /* n_drafts[j] outside [0, drafts]: its outputs are -1, kept 0 */
  VERIFY_STATUS_TOKEN = 2,  /* a tested draft token outside [0, vocab): refused */
  VERIFY_STATUS_PROB = 4,   /* a probability that was read is NaN, negative or > 1: taken as
                               0, 0 and 1; or the weights sum to more than 8 (the token is -1
                             where they sum to 15 or more) */
  VERIFY_STATUS_EMPTY = 8,  /* the row to draw from is 0 everywhere: the token is -1 */
  VERIFY_STATUS_UNIFORM = 16 /* a uniform that was read outside [0, 1) or NaN: clamped (NaN
                               to 0) */
};

#define VERIFY_MAX_DRAFTS 31

/* One launch.
 *   target      device float32: row i of request j at target + j * target_req +
 *               i * target_row, vocab probabilities, drafts + 1 rows per request
 *   draft       device float32, the same with drafts rows per request, or NULL (point
 *               masses)
 *   tokens      device int32 [reqs, drafts]: the drafted tokens
 *   n_drafts    device int32 [reqs] or NULL (all have `drafts`)
 *   uniforms    device float32 [reqs, drafts + 1]: column i tests draft i, the last
 *               column draws
 *   out_tokens  device int32 [reqs, drafts + 1]: the kept drafts, the drawn token, then -1
 *   kept        device int32 [reqs]: drafts kept
 *   status      device int32 [1] or NULL: VERIFY_STATUS_* bits OR-ed in */
int draft_verify(const float* target, int64_t target_req, int64_t target_row, const float* draft,
                 int64_t draft_req, int64_t draft_row, const int32_t* tokens,
                 const int32_t* n_drafts, const float* uniforms, int reqs, int drafts, int vocab,
                 int32_t* out_tokens, int32_t* kept, int32_t* status, verify_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DRAFT_VERIFY_H */
