/*
 * dspark.h -- C ABI of the DSpark drafter hot path on AMD Instinct MI355X (gfx950).
 *
 * The path: a gamma-step Markov-head refinement of a parallel backbone's base
 * logits, the confidence head with per-position temperature calibration, the
 * prefix survival products, and the hardware-aware prefix scheduler that picks
 * per-request verification lengths maximising tau * SPS(B).
 *
 * Sources (the DSpark pages):
 *   [P1] DSpark explainer (zhichai.net/topic/178208222): section 二 "design 1"
 *        (Markov-head equation), section 二 "design 2" (confidence head, STS,
 *        hardware-aware prefix scheduler), section 三 challenges 1-2 (asynchronous
 *        top-K scheduling, global search without early stop).
 *   [P3] DSpark news summary (10100.com/article/149061879), part 01 and Figure 1
 *        (anchor as first predicted position, Markov rank 256, survival products).
 *   [P4] DeepSeek-V4-Pro DSpark integration note (demingchina.com/news/12928)
 *        (markov_w1/markov_w2 logits bias, rank 512, block size 5, fp32
 *        confidences, greedy draft sampling).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers into caller-owned memory on the
 *     current HIP device, row-major, densely packed.  bf16 tensors are passed
 *     as raw 16-bit patterns (uint16_t).  The library keeps no pointer after
 *     the call returns and allocates no device memory: scratch comes from a
 *     caller-provided workspace whose size the *_workspace() queries return.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = the default stream)
 *     and the call returns without synchronising the host, so calls can be
 *     captured in HIP graphs.  Calls on different streams with distinct
 *     outputs and workspaces may run concurrently.
 *   - Host-visible argument checks run before anything is enqueued; a failing
 *     check returns a status other than DSPARK_OK and enqueues nothing.  Token
 *     ids inside device buffers (anchors, tokens) are checked on the device:
 *     the draft turns a request whose anchor lies outside [0, V) into tokens
 *     of -1, and the confidence head gives NaN for a position whose previous
 *     token lies outside [0, V), so a bad id is detectable rather than
 *     silently clamped.
 *   - dspark_last_error() returns a thread-local description of the last
 *     failure on the calling thread.
 *
 * Notation: R requests, gamma draft positions per request, V vocabulary size,
 * r Markov rank, d backbone hidden size.
 */
#ifndef DSPARK_H
#define DSPARK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DSPARK_OK = 0,
  DSPARK_EINVAL = 1,       /* NULL required pointer, non-positive size, bad mode or temperature */
  DSPARK_EWORKSPACE = 2,   /* workspace NULL or smaller than the query says */
  DSPARK_EUNSUPPORTED = 3, /* valid but outside what the kernels are built for (see each call) */
  DSPARK_EDEVICE = 4       /* a HIP launch or runtime call failed; see dspark_last_error() */
} dspark_status;

typedef enum {
  DSPARK_GREEDY = 0, /* x_k = argmax_v z_v */
  DSPARK_SAMPLE = 1  /* x_k = argmax_v (z_v / T - ln(-ln u_v))  (Gumbel-max) */
} dspark_mode;

/* Storage order of the [R, gamma, V] fp32 arrays of dspark_markov_draft (base,
 * uniforms, bias_out).  Element (m, k, v) -- request m, position k (0-based),
 * vocabulary entry v -- sits at
 *   DSPARK_LAYOUT_RGV:   (m * gamma + k) * V + v                     (row-major [R][gamma][V])
 *   DSPARK_LAYOUT_TILED: ((k * C + v / 32) * 32 + v % 32) * R + m,  C = ceil(V / 32)
 * The tiled order ([gamma][C][32][R], the tail entries of the last chunk
 * padding) is column-major inside each 32-entry chunk: for one vocabulary
 * entry the requests are contiguous, so every load of a 32-request tile reads
 * whole 128-byte lines and a chunk of all requests is one contiguous block
 * (the logits-transposed output of a backbone LM-head GEMM, or a random-number
 * fill, produces it at no extra cost).  Row-major arrays are read with the
 * vocabulary entries on the lanes instead, so there a load reads 128
 * contiguous bytes of one request row. */
typedef enum {
  DSPARK_LAYOUT_RGV = 0,
  DSPARK_LAYOUT_TILED = 1
} dspark_layout;

/* Limits of this build. */
#define DSPARK_MAX_RANK 512          /* r <= 512 and r % 16 == 0 */
#define DSPARK_MAX_CANDIDATES (1 << 23) /* R * gamma; also R * (1 + gamma) < 2^24, which keeps
                                           the fixed-point tau sum exact (below 2^64) */

/* Optional per-step timing hooks for dspark_markov_draft.  When non-NULL,
 * begin[k] and end[k] (k = 0..gamma-1) receive the start and stop time of the
 * fused step kernel of position k+1: they are attached to that kernel's
 * dispatch (hipExtLaunchKernel), so hipEventElapsedTime(begin[k], end[k]) is
 * the kernel's own duration.  Each entry is a hipEvent_t created by the caller
 * (NULL entries are skipped); count must be >= gamma. */
typedef struct {
  void* const* begin;
  void* const* end;
  int count;
} dspark_step_events;

/* Result summary of dspark_schedule, written to DEVICE memory (32 bytes). */
typedef struct {
  int32_t B_star;   /* chosen verification budget B* = R + m* */
  int32_t m_star;   /* number of draft tokens admitted, summed over requests */
  uint64_t tau_fx;  /* tau* in fixed point, units of 2^-40 */
  double tau;       /* tau* = tau_fx * 2^-40 (double rounding of tau_fx, then exact scale) */
  double theta;     /* Theta* = tau * SPS(B*) */
} dspark_schedule_info;

/* Bytes of workspace dspark_markov_draft needs for these sizes (0 if invalid). */
size_t dspark_markov_draft_workspace(int R, int gamma, int V, int r);

/*
 * Markov-head draft: the gamma sequential refinement steps of [P1] section 二
 * design 1 (Markov-head equation B(x_{k-1}, .) = W1[x_{k-1}] W2), with x_0 the
 * anchor ([P3] part 01) and the logits bias added to the backbone's base
 * logits ([P4]).  For k = 1..gamma and every request m:
 *     e      = W1[x_{k-1}, :]                         (r values)
 *     z_v    = base[m, k-1, v] + sum_i e_i * W2(i, v)  (fp32, bf16 products, fp32 accumulation)
 *     x_k    = argmax_v z_v                            (GREEDY)
 *            = argmax_v z_v / T - ln(-ln u[m,k-1,v])   (SAMPLE)
 * Equal maxima resolve to the smallest token id.
 *
 *   W1        [V, r] bf16   Markov embedding table (row t = W1[t]).
 *   W2        [V, r] bf16   the r x V projection stored column by column:
 *                           element (i, v) at W2[v * r + i].
 *   layout    DSPARK_LAYOUT_RGV or DSPARK_LAYOUT_TILED: storage order of base,
 *             uniforms and bias_out (see dspark_layout).
 *   base      [R, gamma, V] fp32 backbone base logits (in `layout` order; the
 *             tiled order holds gamma * C * 32 * R floats).  NULL in GREEDY mode
 *             drafts from the Markov bias alone (base taken as zero; no logits
 *             are read, so a call costs the gather + bias GEMM + argmax only).
 *   anchors   [R] int32     anchor token of each request (x_0); a request whose
 *                           anchor is outside [0, V) gets tokens -1 throughout.
 *   mode      DSPARK_GREEDY or DSPARK_SAMPLE.
 *   temperature  > 0 and finite when mode == DSPARK_SAMPLE; ignored for GREEDY.
 *   uniforms  [R, gamma, V] fp32 in (0, 1) in `layout` order, required iff SAMPLE
 *             (NULL for GREEDY).
 *   tokens    [R, gamma] int32 output, tokens[m * gamma + k - 1] = x_k (-1 after a
 *             bad anchor, or where every score of a row is -inf or NaN).
 *   bias_out  optional [R, gamma, V] fp32 output (in `layout` order) of the
 *             Markov bias of every step (a debugging aid; NULL on the hot path).
 *   workspace device scratch of ws_bytes >= dspark_markov_draft_workspace(...),
 *             16-byte aligned: up to 16 packed 64-bit partial results per
 *             request and step.  Its contents on entry do not matter (the call clears what
 *             it uses in its first launch).
 *   events    optional timing hooks (NULL on the hot path).
 * Errors: EINVAL for NULL required pointers (base is optional only in GREEDY
 * mode), W1 or W2 not 16-byte aligned, R/gamma/V/r <= 0, V < 2, a bad layout
 * or mode, a non-positive or non-finite temperature in SAMPLE mode, or
 * uniforms given in GREEDY mode; EUNSUPPORTED for r > DSPARK_MAX_RANK or
 * r % 16 != 0, and where the 32-bit byte offsets of one step would overflow:
 * ceil(V/32)*32*r > 2^30, gamma*V >= 2^22 (DSPARK_LAYOUT_RGV, per block of
 * requests) or ceil(V/32)*R >= 2^24 (DSPARK_LAYOUT_TILED, all requests); EWORKSPACE if the workspace
 * is NULL or too small, EINVAL if it is not 16-byte aligned; EDEVICE on a
 * launch failure.
 */
dspark_status dspark_markov_draft(const uint16_t* W1, const uint16_t* W2, const float* base,
                                  const int32_t* anchors, int R, int gamma, int V, int r,
                                  int layout, int mode, float temperature, const float* uniforms,
                                  int32_t* tokens, float* bias_out, void* workspace,
                                  size_t ws_bytes, const dspark_step_events* events,
                                  void* stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * draft as dspark_markov_draft with no bias output, no timing hooks and no
 * workspace argument.  Its scratch (the packed per-step results) lives in a
 * static device array of DSPARK_NOALLOC_SCRATCH_BYTES that each GPU holds
 * until the process ends; the call allocates nothing.
 * Limit: dspark_markov_draft_workspace(R, gamma, V, r) <= DSPARK_NOALLOC_SCRATCH_BYTES,
 * i.e. R * gamma <= 32768; larger sizes return DSPARK_EUNSUPPORTED.
 * Concurrency: every call on one GPU uses that GPU's one array, so calls that
 * overlap in time on the same device (other streams, other host threads) race
 * and must be serialised by the caller.  Each call clears what it uses first.
 * Errors: as dspark_markov_draft (without the workspace errors), plus
 * EUNSUPPORTED above the limit and EDEVICE if the array's address cannot be
 * found on the current device.
 */
#define DSPARK_NOALLOC_SCRATCH_BYTES (4u << 20)
dspark_status dspark_markov_draft_noalloc(const uint16_t* W1, const uint16_t* W2,
                                          const float* base, const int32_t* anchors, int R,
                                          int gamma, int V, int r, int layout, int mode,
                                          float temperature, const float* uniforms,
                                          int32_t* tokens, void* stream);

/* Bytes of workspace dspark_rnn_draft needs (0 if invalid). */
size_t dspark_rnn_draft_workspace(int R, int gamma, int V, int r, int d);

/*
 * RNN-head draft: the alternative sequential stage of [P3] part 01 (a
 * recurrent in-block state updated by a gate over the concatenated history
 * state, previous-token embedding and backbone hidden state; [P1] section 二
 * design 1, the RNN head that remembers the whole prefix).  The pages give no
 * equations; this build reads them as, for k = 1..gamma and every request m,
 *     u_k = [s_{k-1}; e_k; h_k],  e_k = W1[x_{k-1}, :] (x_0 = anchor),  s_0 = 0
 *     g_k = sigmoid(G u_k + b_g)             (update gate, r units)
 *     c_k = e_k + tanh(C u_k + b_c)          (candidate: embedding row + correction)
 *     s_k = g_k * c_k + (1 - g_k) * s_{k-1}  (fp32 state)
 *     z_v = base[m, k-1, v] + sum_i bf16(s_k)_i W2(i, v),  x_k selected as in
 *           dspark_markov_draft (GREEDY or SAMPLE)
 * Products take bf16 operands with fp32 accumulation: the state enters them
 * rounded to bf16.  A gate saturated at 1 with C = 0, b_c = 0 is the Markov head.
 *   U         [2r, 2r + d] bf16, 16-byte aligned: rows 0..r-1 are G, rows
 *             r..2r-1 are C; columns [0, r) act on s_{k-1}, [r, 2r) on e_k,
 *             [2r, 2r + d) on h_k.
 *   b_rnn     [2r] fp32 = [b_g; b_c].
 *   h         [R, gamma, d] bf16 backbone hidden states (16-byte aligned), d % 8 == 0.
 *   W1, W2, base, anchors, layout, mode, temperature, uniforms, tokens, events
 *             as for dspark_markov_draft (no bias output).
 *   state_out optional [R, r] fp32 output: the state s_gamma after the last step
 *             (a debugging aid; NULL on the hot path).
 *   workspace >= dspark_rnn_draft_workspace(R, gamma, V, r, d) bytes, 256-byte
 *             aligned: packed words, the token-independent pre-activations and
 *             two copies of the state.
 * A call is 2 gamma + 2 launches.  Errors: as dspark_markov_draft, plus EINVAL
 * for NULL U / b_rnn / h or d <= 0, EUNSUPPORTED for d % 8 != 0, a misaligned U
 * or h, R * gamma * 2r >= 2^31, or 2r + d > 2^22.
 */
dspark_status dspark_rnn_draft(const uint16_t* W1, const uint16_t* W2, const uint16_t* U,
                               const float* b_rnn, const float* base, const uint16_t* h,
                               const int32_t* anchors, int R, int gamma, int V, int r, int d,
                               int layout, int mode, float temperature, const float* uniforms,
                               int32_t* tokens, float* state_out, void* workspace, size_t ws_bytes,
                               const dspark_step_events* events, void* stream);

/*
 * Confidence head with STS calibration, [P1] section 二 design 2 (confidence
 * head equation, sequential temperature scaling) and [P4] (fp32 scores):
 *     s_{m,k} = sum_{i<d} w[i] h[m,k-1,i] + sum_{i<r} w[d+i] W1[x_{k-1}, i]
 *     c_{m,k} = 1 / (1 + exp(-s_{m,k} / T_k))
 * with x_0 = anchors[m] and x_k = tokens[m, k-1].  Optionally also the prefix
 * survival a_{m,j} = c_{m,1} * ... * c_{m,j}, multiplied left to right in fp32.
 *
 *   h         [R, gamma, d] bf16 backbone hidden states.
 *   W1        [V, r] bf16 (as in dspark_markov_draft).
 *   anchors   [R] int32; tokens [R, gamma] int32 (the draft).
 *   w_conf    [d + r] fp32, ordered [w_h; w_e].
 *   sts_temp  optional [gamma] fp32 positive temperatures T_k (NULL => 1).
 *   conf      [R, gamma] fp32 output c.
 *   surv      optional [R, gamma] fp32 output a (NULL to skip).
 * Errors: EINVAL for NULL required pointers or non-positive sizes; EDEVICE on a
 * launch failure.  Temperatures are device data: they must be positive.  A
 * position whose x_{k-1} lies outside [0, V) gets c = NaN (and so do its
 * survival and the later ones of that request).
 */
dspark_status dspark_confidence(const uint16_t* h, const uint16_t* W1, const int32_t* anchors,
                                const int32_t* tokens, const float* w_conf,
                                const float* sts_temp, int R, int gamma, int d, int V, int r,
                                float* conf, float* surv, void* stream);

/*
 * Prefix survival alone ([P1] section 二 design 2, scheduler definitions):
 * surv[m, j] = conf[m, 0] * ... * conf[m, j], sequential fp32 products.
 * conf and surv are [R, gamma] fp32 device arrays (they may not alias).
 */
dspark_status dspark_survival(const float* conf, int R, int gamma, float* surv, void* stream);

/*
 * W2 storage conversion.  The draft entry points take the r x V projection of
 * [P1] section 二 design 1 (Markov-head equation) stored column by column
 * (element (i, v) at W2[v * r + i]); this converts a row-by-row copy (element
 * (i, v) at w2_rv[i * V + v]) into that storage, once, when the weights are
 * loaded.  Off the drafting path.
 *   w2_rv     [r, V] bf16 device array (read).
 *   w2_store  [V, r] bf16 device array (written); must not overlap w2_rv.
 * Enqueued on `stream`; no host sync.  Errors: EINVAL for NULL pointers,
 * sizes <= 0 or overlapping arrays; EUNSUPPORTED for r above 4194240 or V
 * above 2^30 - 1; EDEVICE on a launch failure.
 */
dspark_status dspark_w2_store_from_rv(const uint16_t* w2_rv, int r, int V, uint16_t* w2_store,
                                     void* stream);

/* Bytes of workspace dspark_schedule needs (0 if invalid). */
size_t dspark_schedule_workspace(int R, int gamma);

/*
 * Hardware-aware prefix scheduler, [P1] section 二 design 2 (objective
 * Theta = tau * SPS(B), B = sum_r (1 + l_r), tau = sum_r (1 + sum_{j<=l_r} a_{r,j}),
 * global sort of candidates by survival) and section 三 challenge 2 (no early
 * stop: every budget is evaluated).  Candidates (r, j) carry id r*gamma + j-1
 * and key a_{r,j}; they are ordered by key descending, equal keys by id
 * ascending.  With q = rint(a * 2^40) and S_m the exact integer sum of the
 * first m ordered q's, Theta_m = double(R*2^40 + S_m) * 2^-40 * double(sps[R+m-1])
 * for m = 0..R*gamma; m* is the smallest m attaining the maximum, and l_r is
 * the number of request r's candidates among the first m* ordered ones.
 *
 *   surv      [R, gamma] fp32 survival probabilities (device data); values outside
 *             [0, 1] are clamped into it and NaN is taken as 0 (for the order,
 *             q and tau alike).
 *   sps       [B_max] fp32, sps[B-1] = SPS(B) >= 0, the engine's profiled steps/s.
 *   B_max     >= R * (1 + gamma).
 *   lengths   [R] int32 output l_r.
 *   order     optional [R * gamma] int32 output, the sorted candidate ids.
 *   info      optional dspark_schedule_info output (device memory).
 *   workspace >= dspark_schedule_workspace(R, gamma) bytes.
 * Errors: EINVAL for NULL required pointers, non-positive sizes or
 * B_max < R*(1+gamma); EUNSUPPORTED if R*gamma > DSPARK_MAX_CANDIDATES or
 * R*(1+gamma) >= 2^24; EWORKSPACE; EDEVICE.
 */
dspark_status dspark_schedule(const float* surv, const float* sps, int R, int gamma, int B_max,
                              int32_t* lengths, int32_t* order, dspark_schedule_info* info,
                              void* workspace, size_t ws_bytes, void* stream);

/* Admission rules of dspark_schedule_ex. */
typedef enum {
  DSPARK_SCHED_GLOBAL = 0,      /* global search over every budget (= dspark_schedule) */
  DSPARK_SCHED_EARLY_STOP = 1,  /* the greedy scan with its break */
  DSPARK_SCHED_CAPACITY = 2     /* a predicted batch capacity, top candidates */
} dspark_sched_mode;

/*
 * The scheduler with a choice of admission rule.  Candidates, their order,
 * q, S_m, Theta_m, l_r and the info fields are those of dspark_schedule.
 *   DSPARK_SCHED_GLOBAL: identical to dspark_schedule.
 *   DSPARK_SCHED_EARLY_STOP ([P1] section 二 design 2, greedy steps 3-5, the
 *     theoretical version that [P3] part 01 describes as non-anticipating):
 *     candidates are admitted in order while Theta keeps rising; m* is the
 *     smallest m with Theta_{m+1} <= Theta_m, or R*gamma if there is none.
 *   DSPARK_SCHED_CAPACITY ([P1] section 三 challenge 1, [P3] part 01: the
 *     asynchronous production form): `capacity` K is the predicted size of the
 *     next verification batch in tokens, anchors included; m* = clamp(K - R,
 *     0, R*gamma) (the dynamic top-K).  sps and B_max are not used (sps may be
 *     NULL); info->theta reports tau*.
 *   capacity  >= 0, used by DSPARK_SCHED_CAPACITY only.
 * Other arguments as for dspark_schedule; the workspace size is the same.
 * Errors: as dspark_schedule, plus EINVAL for an unknown mode or a negative
 * capacity (sps and B_max are checked only when the mode uses them).
 */
dspark_status dspark_schedule_ex(const float* surv, const float* sps, int R, int gamma, int B_max,
                                 int mode, int capacity, int32_t* lengths, int32_t* order,
                                 dspark_schedule_info* info, void* workspace, size_t ws_bytes,
                                 void* stream);

/* Bytes of workspace dspark_draft_step needs (0 if invalid). */
size_t dspark_draft_step_workspace(int R, int gamma, int V, int r);

/*
 * Number of kernel launches one dspark_draft_step call makes for these sizes,
 * layout, mode and temperature, with W1 and w_conf + d 16-byte aligned (a
 * misaligned one can add the separate finishing launch).  Host-side planning
 * only (it reads the current device's properties); nothing is launched.
 * Errors: EINVAL for NULL count, bad sizes, unknown layout or mode, or a
 * non-positive sampling temperature.
 */
dspark_status dspark_draft_step_launches(int R, int gamma, int V, int r, int layout, int mode,
                                         float temperature, int* count);

/*
 * One whole drafting step of the head in one call: the gamma-step Markov-head
 * draft ([P1] section 二 design 1, as dspark_markov_draft), the confidence head
 * with STS and the prefix survivals ([P1] section 二 design 2, as
 * dspark_confidence), and the global-search schedule ([P1] section 二 design 2
 * and section 三 challenge 2, as dspark_schedule).  The results are those of
 * the three calls in sequence (up to the rounding order of the confidence
 * dot products).  It runs as a prologue that clears the draft's packed words
 * and computes the token-independent part w_h . h of every confidence logit,
 * then the gamma step kernels (whose first V group also computes
 * w_e . W1[x_{k-1}] from the rows it gathered), then the finishing work: the
 * sigmoid with STS, the survival products and the schedule.  That work needs
 * x_0 .. x_{gamma-2} only; where the last step's launch has a workgroup with
 * no step work (the rank-512 sampling kernel, whose V groups rarely fill the
 * launch), that workgroup does it beside the step, and the step workgroup
 * that finishes last unpacks the last tokens: gamma + 1 launches.  Otherwise
 * it is one launch after the last step (up to 8192 candidates; beyond that the
 * schedule's global path follows it): gamma + 2 or more.
 * dspark_draft_step_launches gives the count for given sizes.
 *   W1 ... uniforms   as for dspark_markov_draft (no bias output).
 *   h, w_conf, sts_temp, d   as for dspark_confidence; w_conf must be 16-byte
 *                            aligned and d a multiple of 4.
 *   sps, B_max               as for dspark_schedule.
 *   tokens, conf, surv       [R, gamma] outputs; lengths [R]; order [R*gamma]
 *                            and info optional, as for dspark_schedule.
 *   workspace  >= dspark_draft_step_workspace(R, gamma, V, r) bytes, 256-byte
 *              aligned; its contents on entry do not matter.
 *   events     optional per-step timing hooks of the gamma step kernels.
 * Errors: the union of the three calls' errors, plus EUNSUPPORTED for a
 * misaligned w_conf or d % 4 != 0 and EINVAL for a misaligned workspace.
 */
dspark_status dspark_draft_step(const uint16_t* W1, const uint16_t* W2, const float* base,
                                const int32_t* anchors, int R, int gamma, int V, int r,
                                int layout, int mode, float temperature, const float* uniforms,
                                const uint16_t* h, const float* w_conf, const float* sts_temp,
                                int d, const float* sps, int B_max, int32_t* tokens, float* conf,
                                float* surv, int32_t* lengths, int32_t* order,
                                dspark_schedule_info* info, void* workspace, size_t ws_bytes,
                                const dspark_step_events* events, void* stream);

/*
 * Verification side, [P1] section 三 challenge 3 (every verified token is one
 * flattened element; a marker tensor carries the within-sequence
 * dependencies) and [P3] Figure 1 (the target verifies anchor + kept prefix
 * in parallel).  Request r contributes 1 + l_r elements: its anchor, then its
 * first l_r drafts, at positions pos0[r] + j, each marked with r.
 *   anchors      [R] int32;  tokens [R, gamma] int32 drafts (row r, draft j at
 *                r*gamma + j - 1);  lengths [R] int32 l_r (values outside
 *                [0, gamma] are clamped into it).
 *   pos0         optional [R] int32 position of each anchor (0 if NULL).
 *   flat_tokens  [R*(1+gamma)] int32 output (the first B entries are written).
 *   flat_pos, flat_req  optional outputs of the same size: positions, request ids.
 *   cu_seqlens   [R+1] int32 output: segment starts, cu_seqlens[R] = B.
 * Errors: EINVAL for NULL required pointers or non-positive sizes;
 * EUNSUPPORTED if R*(1+gamma) exceeds 2^31 - 1; EDEVICE.
 */
dspark_status dspark_verify_pack(const int32_t* anchors, const int32_t* tokens,
                                 const int32_t* lengths, const int32_t* pos0, int R, int gamma,
                                 int32_t* flat_tokens, int32_t* flat_pos, int32_t* flat_req,
                                 int32_t* cu_seqlens, void* stream);

/*
 * Greedy verification of a flattened batch ([P3] Figure 1): t_e = argmax_v of
 * target_logits row e (the target's next token after element e; ties resolve to
 * the smallest id; rows must be free of NaN).  For request r with segment
 * start s = cu_seqlens[r] and l_r = cu_seqlens[r+1] - s - 1 drafts, drafts are
 * accepted while tokens[r, j] == t_{s+j}; accepted[r] = their number and
 * next_token[r] = t_{s + accepted[r]} (the correction of the first rejected
 * draft, or the bonus token when all are accepted).
 *   target_logits  [rows, V] fp32, row e for flattened element e (rows >= B;
 *                  rows from B on are not read).
 *   cu_seqlens     [R+1] as written by dspark_verify_pack.
 *   target_argmax  [R*(1+gamma)] int32 output (the first B entries are written).
 *   accepted, next_token  [R] int32 outputs.
 * Errors: EINVAL for NULL pointers or non-positive sizes; EUNSUPPORTED if
 * R*(1+gamma) exceeds 2^31 - 1; EDEVICE.
 */
dspark_status dspark_verify_greedy(const float* target_logits, const int32_t* cu_seqlens,
                                   const int32_t* tokens, int R, int gamma, int V,
                                   int32_t* target_argmax, int32_t* accepted,
                                   int32_t* next_token, void* stream);

/*
 * Acceptance probability of paired rows ([P1] section 二 design 2, the
 * confidence head's label 1 - TV(p_draft, p_target)):
 *   out[i] = sum_v min(softmax(draft_logits[i] / T)_v, softmax(target_logits[i] / T)_v).
 *   draft_logits, target_logits  [n, V] fp32 (each row needs a finite value;
 *                                -inf entries are allowed).
 *   temperature  T > 0 and finite.
 *   out          [n] fp32 output.
 * Errors: EINVAL for NULL pointers, non-positive sizes or a bad temperature;
 * EDEVICE.
 */
dspark_status dspark_accept_prob(const float* draft_logits, const float* target_logits, int n,
                                 int V, float temperature, float* out, void* stream);

/* ------------------------------------------------------------------------
 * Verification over a paged key/value cache: the target engine's side of the
 * step between the flattened batch and its logits.  [P1] section 三 challenge
 * 3: every verified token is one flattened element, and the attention takes
 * the dependencies inside a sequence from a marker tensor.  The pages give no
 * kernels or layouts for it; these are this library's own.
 *
 * Request r has ctx_len[r] tokens in the cache and brings the elements
 * cu_seqlens[r] .. cu_seqlens[r+1] - 1 of the flattened batch (n_r of them: an
 * anchor and its drafts), as a chain or as a tree.  Element j of the segment
 * (0-based) is kept at cache position ctx_len[r] + j.
 *
 * Pages.  Position p of request r lies in page block_table[r, p / P] at offset
 * p % P, P = page_size a power of two in [16, 1024]; a slot is
 * page * P + offset (int64).  block_table is [R, max_pages] int32; entries
 * behind a request's last page are neither read nor written.
 *
 * Cache.  For Hk heads of D values and c = 16 / (bytes per element):
 *     k_cache [num_pages][Hk][D / c][P][c]     element (page, h, d, o) at
 *             (((page * Hk + h) * (D / c) + d / c) * P + o) * c + d % c
 *     v_cache [num_pages][Hk][D][P]            ((page * Hk + h) * D + d) * P + o
 * Both are the operand order of the matrix instructions, so a 16-byte load of
 * either feeds them without a transpose.  DSPARK_E4M3 caches hold x / scale in
 * OCP e4m3 (finite values up to 448) with one scale per head for the keys and
 * one for the values.
 *
 * A pool that runs short.  dspark_page_map turns a request down on the device,
 * and the calls behind it have already been enqueued.  They learn of it from
 * mapped_len, its new_len (dspark_tree_attention_ex, dspark_verify_tree_ex,
 * dspark_kv_commit_ex): the request's rows are NaN, nothing is accepted, no page
 * is written, and it keeps its context for another step.  Without mapped_len they
 * go by block_table, which names pages of others behind a request's last page.
 * For chains, which need no commit, the length to keep is
 * min(ctx_len + 1 + accepted, mapped_len); where that is ctx_len the request was
 * turned down and its next token is not one.
 *
 * Outputs share no memory with inputs or with each other unless an entry says
 * that they may.
 * ------------------------------------------------------------------------ */

/* Element types of the cache calls. */
typedef enum {
  DSPARK_BF16 = 0,
  DSPARK_FP16 = 1,
  DSPARK_E4M3 = 2 /* caches only */
} dspark_dtype;

#define DSPARK_MAX_PAGE_REQUESTS 16384 /* R of dspark_page_map / dspark_page_trim */
#define DSPARK_MAX_MASK_WORDS 32       /* 32-bit words of a tree mask row: 1024 nodes */

/* State of a ring of free pages, in DEVICE memory (16 bytes).  The free pages
 * are ring[(head + i) mod num_pages] for 0 <= i < count.  A new pool of n pages
 * is ring = 0, 1, ..., n - 1 with head = 0 and count = n. */
typedef struct {
  int32_t head;
  int32_t count;
  int32_t refused;  /* output: requests that the call turned down */
  int32_t reserved; /* written as 0 */
} dspark_page_pool;

/*
 * Pages and slots for the new elements of every request, from lengths that
 * only the device knows.  With n_r = cu_seqlens[r+1] - cu_seqlens[r],
 *     need_r = ceil((cur_len[r] + n_r) / P) - ceil(cur_len[r] / P),
 *     S_r    = need_0 + ... + need_{r-1}
 * request r is served if S_r + need_r <= count: its new pages are
 *     block_table[r, ceil(cur_len[r] / P) + i] = ring[(head + S_r + i) mod num_pages]
 * slots[cu_seqlens[r] + j] is the slot of position cur_len[r] + j and
 * new_len[r] = cur_len[r] + n_r.  A request that is not served (the pool is
 * short, cur_len[r] or n_r negative, more than max_pages pages or 2^31 - 1 tokens)
 * leaves its block_table row as it was, gets slots of -1 and new_len[r] = cur_len[r], and
 * counts in pool_out->refused; one that asks for no page is served whatever
 * the pool holds, and one with too many pages takes none from the others.  A
 * slot whose page id lies outside [0, num_pages) is -1.
 *   cur_len     [R] int32 tokens that each request holds.
 *   cu_seqlens  [R+1] int32 segment starts.
 *   block_table [R, max_pages] int32, new entries written.
 *   ring        [num_pages] int32 (read).
 *   pool        device dspark_page_pool before the call (read).
 *   pool_out    device dspark_page_pool after it; apart from pool, so that a call
 *               can be repeated.
 *   slots       [max_tokens] int64 output; entries from cu_seqlens[R] on are left
 *               as they were, elements from max_tokens on get no slot.
 *   new_len     [R] int32 output, apart from cur_len.
 * One launch.  Errors: EINVAL for NULL pointers, sizes <= 0, a page size that
 * is no power of two in [16, 1024], pool_out on pool or new_len on cur_len;
 * EUNSUPPORTED for R > DSPARK_MAX_PAGE_REQUESTS; EDEVICE on a launch failure.
 */
dspark_status dspark_page_map(const int32_t* cur_len, const int32_t* cu_seqlens, int R,
                              int max_tokens, int page_size, int max_pages, int num_pages,
                              int32_t* block_table, const int32_t* ring,
                              const dspark_page_pool* pool, dspark_page_pool* pool_out,
                              int64_t* slots, int32_t* new_len, void* stream);

/*
 * Pages back to the pool: request r keeps keep_len[r] of its cur_len[r] tokens
 * (keep_len is clamped into [0, cur_len]; 0 ends a request).  With
 * give_r = ceil(cur_len[r] / P) - ceil(keep_len[r] / P) and S its running sum,
 *     ring[(head + count + S_r + i) mod num_pages] = block_table[r, ceil(keep_len[r] / P) + i]
 * and the pool's count grows by the sum.  block_table is not changed: the
 * entries behind the last kept page are not read by page calls any more (other
 * calls learn from mapped_len where a request ends).  Page ids go back as the
 * row names them.  A keep_len of -1, as dspark_kv_commit gives it for a path
 * that it refuses, is 0 and ends the request; with dspark_kv_commit_ex the
 * request keeps its context.
 * A request with cur_len[r] < 0 or more than max_pages pages gives nothing and
 * counts in pool_out->refused; if the ring would hold more than num_pages
 * pages (pages given back twice) nothing is written to it and refused = R.
 * One launch.  Errors: as dspark_page_map.
 */
dspark_status dspark_page_trim(const int32_t* cur_len, const int32_t* keep_len, int R,
                               int page_size, int max_pages, int num_pages,
                               const int32_t* block_table, int32_t* ring,
                               const dspark_page_pool* pool, dspark_page_pool* pool_out,
                               void* stream);

/*
 * Keys and values of new elements into their slots.
 *   k, v        rows of [Hk, D] elements of `dtype` (BF16 or FP16), row e at
 *               k + e * k_stride (strides in elements, multiples of 8, at least
 *               Hk * D; bases 16-byte aligned).
 *   slots       [max_tokens] int64 as dspark_page_map writes them; an element
 *               whose slot lies outside [0, num_pages * P) is skipped.  The slots
 *               of one call are distinct (of two elements with one slot, either
 *               may be kept, value by value).
 *   count       optional device int32: the number of elements (cu_seqlens + R);
 *               NULL stands for max_tokens.
 *   cache_dtype `dtype` itself, or DSPARK_E4M3.
 *   k_scale, v_scale  [Hk] fp32 positive, required with DSPARK_E4M3 (NULL
 *               otherwise): x / scale (fp32) is clamped to +-448 and rounded to
 *               nearest even; NaN stays NaN.
 * Errors: EINVAL for NULL pointers, sizes <= 0, bad types, page sizes, strides
 * or alignment, scales missing or given without DSPARK_E4M3; EUNSUPPORTED for
 * D outside {64, 96, 128, 192, 256} or Hk > 65535; EDEVICE.
 */
dspark_status dspark_kv_store(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                              int dtype, const int64_t* slots, const int32_t* count,
                              int max_tokens, int Hk, int D, int page_size, int num_pages,
                              int cache_dtype, const float* k_scale, const float* v_scale,
                              void* k_cache, void* v_cache, void* stream);

/*
 * The accepted path to the front: for i = 1 .. accepted[r] the keys and values
 * at position ctx_len[r] + path[r, i] move to position ctx_len[r] + i, and
 * new_len[r] = ctx_len[r] + 1 + accepted[r].  accepted[r] = -1 (a request
 * without elements) moves nothing and gives new_len[r] = ctx_len[r].
 *   k_cache, v_cache  caches of `layers` layers, layer l at l * k_layer_stride
 *               (v_layer_stride) elements (multiples of 16 / element size; a
 *               layer apart at least).
 *   path        [R, max_nodes] int32: 0, then strictly increasing node numbers (as
 *               dspark_verify_tree writes them).
 * A request whose path is not such a sequence, whose accepted count lies
 * outside [-1, max_nodes), or that touches a page id outside [0, num_pages) or
 * a position past its table or 2^31 - 1 moves nothing and gets new_len[r] = -1.
 *   new_len     [R] int32 output, apart from ctx_len and accepted.
 * Behind the pages that a request holds its block_table row may name pages of
 * others: where a pool can run short, dspark_kv_commit_ex is the call to use.
 * Errors: EINVAL for NULL pointers, sizes <= 0, a bad page size or type,
 * misaligned caches or strides, layers that overlap, new_len on ctx_len or
 * accepted; EUNSUPPORTED for D as above, layers > 65535 or R > 65535; EDEVICE.
 */
dspark_status dspark_kv_commit(void* k_cache, void* v_cache, int64_t k_layer_stride,
                               int64_t v_layer_stride, int layers, int cache_dtype,
                               const int32_t* block_table, const int32_t* ctx_len,
                               const int32_t* path, const int32_t* accepted, int R, int max_nodes,
                               int Hk, int D, int page_size, int max_pages, int num_pages,
                               int32_t* new_len, void* stream);

/*
 * dspark_kv_commit for requests whose elements dspark_page_map may have turned
 * down.
 *   mapped_len  [R] int32 (dspark_page_map's new_len) or NULL, which is
 *               dspark_kv_commit: no position from mapped_len[r] on is read or
 *               written.
 * With mapped_len a request that dspark_kv_commit would refuse, or whose path
 * leads to mapped_len[r] or behind it, moves nothing and keeps its context:
 * new_len[r] = ctx_len[r].  dspark_page_trim from mapped_len to new_len then
 * gives back the pages of what was not accepted, and no others.
 * Errors: as dspark_kv_commit, plus EINVAL for new_len on mapped_len.
 */
dspark_status dspark_kv_commit_ex(void* k_cache, void* v_cache, int64_t k_layer_stride,
                                  int64_t v_layer_stride, int layers, int cache_dtype,
                                  const int32_t* block_table, const int32_t* ctx_len,
                                  const int32_t* mapped_len, const int32_t* path,
                                  const int32_t* accepted, int R, int max_nodes, int Hk, int D,
                                  int page_size, int max_pages, int num_pages, int32_t* new_len,
                                  void* stream);

/* Bytes of workspace dspark_tree_attention needs (0 if invalid).  It depends on
 * the current device's number of compute units. */
size_t dspark_tree_attention_workspace(int R, int max_tokens, int Hq, int Hk, int D);

/*
 * Attention of every element over its request's context and over the elements
 * of its own segment that its mask names.  For element i of request r and
 * query head y (key/value head h = y / (Hq / Hk)):
 *     s_t  = scale * k_scale[h] * sum_d q[e, y, d] k[t, h, d]
 *     out  = sum_t softmax(s)_t * v_scale[h] v[t, h, :]
 *     lse  = ln sum_t exp(s_t)
 * over the positions t < ctx_len[r] and t = ctx_len[r] + j with j visible to i:
 * j <= i where tree_mask is NULL (a chain), else bit j % 32 of
 * tree_mask[e, j / 32] (bits past the segment or past mask_words are not set).
 * A row that sees nothing gives out = 0 and lse = -inf; positions that a row
 * does not see do not reach it, whatever their keys and values hold.
 * Products take the element type with fp32 accumulation (e4m3 keys and values
 * are widened first, exactly); scores, maxima and sums are fp32; each
 * probability is rounded to the element type before it meets the values.
 *   q           rows of [Hq, D] elements of `dtype`, row e at q + e * q_stride
 *               (elements; a multiple of 8, base 16-byte aligned).
 *   ctx_len     [R] int32; cu_seqlens [R+1] int32.  Rows from
 *               min(cu_seqlens[R], max_tokens) on are neither read nor written.
 *   tree_mask   [max_tokens, mask_words] uint32 or NULL (mask_words is then 0).
 *   k_scale, v_scale  [Hk] fp32 with a DSPARK_E4M3 cache, NULL otherwise.
 *   scale       finite, also times log2(e).
 *   out         rows of [Hq, D] elements of `dtype`, row e at out + e * out_stride;
 *               may be q itself, with its stride, and no other part of its rows.
 *   lse         optional [max_tokens, Hq] fp32.
 *   workspace   >= dspark_tree_attention_workspace(...) bytes, 256-byte aligned;
 *               its contents on entry do not matter, and calls that may run at
 *               the same time need one each.
 * A request's rows are NaN where ctx_len[r] < 0 or it has more positions than its
 * table (or 2^31 - 2^16).  A page id outside [0, num_pages) is not touched: rows
 * that see a position of it are NaN, and other rows of the request may be.
 * Where a row's sums are split depends on the lengths of the whole batch: the
 * same call gives the same bits, a request in another batch the same values up
 * to the rounding of fp32 sums.
 * Errors: EINVAL for NULL pointers, sizes <= 0, Hq not a multiple of Hk, bad
 * types, page sizes, strides, alignment or scale, scales missing or given
 * without DSPARK_E4M3, out on a part of q; EUNSUPPORTED for D outside
 * {64, 96, 128, 192, 256}, mask_words > DSPARK_MAX_MASK_WORDS, R > 2^20 or
 * max_tokens * Hq above 2^31 - 1; EWORKSPACE; EDEVICE.
 */
dspark_status dspark_tree_attention(const void* q, int64_t q_stride, int dtype,
                                    const void* k_cache, const void* v_cache, int cache_dtype,
                                    const float* k_scale, const float* v_scale,
                                    const int32_t* block_table, const int32_t* ctx_len,
                                    const int32_t* cu_seqlens, const uint32_t* tree_mask,
                                    int mask_words, int R, int max_tokens, int Hq, int Hk, int D,
                                    int page_size, int max_pages, int num_pages, float scale,
                                    void* out, int64_t out_stride, float* lse, void* workspace,
                                    size_t ws_bytes, void* stream);

/*
 * dspark_tree_attention for requests whose elements dspark_page_map may have
 * turned down.
 *   mapped_len  [R] int32 (dspark_page_map's new_len) or NULL, which is
 *               dspark_tree_attention.  A request with more positions than
 *               mapped_len[r] (ctx_len[r] and its elements) does not hold them,
 *               whatever its block_table row names behind its last page: its
 *               rows are NaN and no page of it is read.
 * Errors: as dspark_tree_attention.
 */
dspark_status dspark_tree_attention_ex(const void* q, int64_t q_stride, int dtype,
                                       const void* k_cache, const void* v_cache, int cache_dtype,
                                       const float* k_scale, const float* v_scale,
                                       const int32_t* block_table, const int32_t* ctx_len,
                                       const int32_t* mapped_len, const int32_t* cu_seqlens,
                                       const uint32_t* tree_mask, int mask_words, int R,
                                       int max_tokens, int Hq, int Hk, int D, int page_size,
                                       int max_pages, int num_pages, float scale, void* out,
                                       int64_t out_stride, float* lse, void* workspace,
                                       size_t ws_bytes, void* stream);

/*
 * A forest of drafted nodes in the form that the attention reads.  parents[e]
 * is the segment-local number of element e's parent, smaller than its own, or
 * -1 for a root.
 *   mask      [max_tokens, mask_words] uint32 output: bits of the element itself
 *             and of its ancestors.
 *   flat_pos  optional [max_tokens] int32 output: pos0[r] + depth (pos0 [R] int32,
 *             0 if NULL).
 *   flat_req  optional [max_tokens] int32 output: the request.
 * An element with a parent outside [-1, own number) on its way to the root, or
 * with a number of 32 * mask_words or more, gets an empty mask row and
 * position -1.  Rows from cu_seqlens[R] on are left as they were.
 * Errors: EINVAL for NULL pointers or sizes <= 0; EUNSUPPORTED for mask_words >
 * DSPARK_MAX_MASK_WORDS; EDEVICE.
 */
dspark_status dspark_tree_pack(const int32_t* parents, const int32_t* cu_seqlens,
                               const int32_t* pos0, int R, int max_tokens, int mask_words,
                               uint32_t* mask, int32_t* flat_pos, int32_t* flat_req, void* stream);

/*
 * Greedy verification of trees: dspark_verify_greedy where every segment is a
 * tree whose node 0 is the anchor.  t_e = argmax_v of target_logits row e (ties
 * to the smallest id; rows free of NaN).  The walk starts at node 0 and goes
 * from a node to its lowest-numbered child whose token is the node's t, as long
 * as there is one.
 *   target_logits  [max_tokens, V] fp32; rows from cu_seqlens[R] on are not read.
 *   tokens, parents  [max_tokens] int32 flattened (the anchor's token is not read).
 *   max_nodes      nodes of a segment that are looked at, and columns of path.
 *   target_argmax  [max_tokens] int32 output (the first cu_seqlens[R] are written).
 *   accepted       [R] int32 output: drafts accepted (-1 for an empty segment).
 *   path           [R, max_nodes] int32 output: 0, the accepted nodes, then -1.
 *   next_token     [R] int32 output: t of the last node on the path (-1 if empty).
 * Errors: EINVAL for NULL pointers or sizes <= 0; EDEVICE.
 */
dspark_status dspark_verify_tree(const float* target_logits, const int32_t* cu_seqlens,
                                 const int32_t* tokens, const int32_t* parents, int R,
                                 int max_tokens, int max_nodes, int V, int32_t* target_argmax,
                                 int32_t* accepted, int32_t* path, int32_t* next_token,
                                 void* stream);

/*
 * dspark_verify_tree for requests whose elements dspark_page_map may have turned
 * down.
 *   ctx_len, mapped_len  [R] int32 (cur_len and new_len of dspark_page_map), or
 *               both NULL, which is dspark_verify_tree.  A request with more
 *               positions than mapped_len[r] (ctx_len[r] and its elements) counts as
 *               an empty segment: accepted -1, a path of -1, next_token -1.  Its rows'
 *               argmaxes are written; its logits may be NaN.
 * Errors: as dspark_verify_tree, plus EINVAL for one of the two without the
 * other.
 */
dspark_status dspark_verify_tree_ex(const float* target_logits, const int32_t* cu_seqlens,
                                    const int32_t* tokens, const int32_t* parents,
                                    const int32_t* ctx_len, const int32_t* mapped_len, int R,
                                    int max_tokens, int max_nodes, int V, int32_t* target_argmax,
                                    int32_t* accepted, int32_t* path, int32_t* next_token,
                                    void* stream);

/* Static description of a status code. */
const char* dspark_status_string(int status);

/* Thread-local description of the last failure on this thread ("" if none). */
const char* dspark_last_error(void);

/* Hash of the source files and compile flags this library was built from (32 hex
 * digits; "unknown" for a build outside the package's build script).  Loaders
 * compare it with the sources they ship to detect a stale library. */
const char* dspark_source_hash(void);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_H */
