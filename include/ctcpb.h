/*
 * ctcpb.h -- C ABI of the GB300-native batched CTC prefix beam search decoder.
 *
 * What it computes ("GPU CTC Prefix Beam Search Decoder", OASR docs):
 *   log_prob[B, T, V] (float32 log-probabilities, label 'blank_id' is the CTC
 *   blank) -> per row the N best collapsed label sequences and their CTC
 *   posterior log-scores, by prefix beam search (section 3): each hypothesis
 *   keeps a blank-ending and a non-blank-ending log-probability (3.1), extends
 *   by every non-blank label through the two paths of 3.2 / 3.4.1, keeps its
 *   blank/stay slot (3.4.2), merges a shorter hypothesis' extension into the
 *   longer hypothesis it equals (3.4.3) and keeps the best `beam` candidates
 *   (3.4.4-3.4.5).  Offline decoding may skip blank-dominant frames (3.5);
 *   streaming decoding carries the beam state across chunks (section 8).
 *
 * Conventions (all calls):
 *   - Every buffer pointer is a DEVICE pointer, allocated and owned by the
 *     caller; the library never allocates or frees memory (section 5).
 *   - log_prob rows are float32 with V contiguous; stride_b / stride_t are in
 *     elements (64-bit, so offsets past 2^31 elements are fine, section 13).
 *   - Calls are asynchronous on `stream` and never synchronise with the host.
 *   - Return value: CTCPB_OK (0) or a negative status for argument errors
 *     found on the host (nothing is launched then).  Conditions found on the
 *     device set bits in a status word inside the workspace / state, read with
 *     ctcpb_read_status().
 *   - Workspace and state buffers must be 256-byte aligned.
 *
 * Arithmetic: float32 with a fixed operation order and the library's own
 * logsumexp, max(a, b) + F(|a - b|) with F(d) = log(1 + e^-d) evaluated from a
 * table of degree-5 Taylor polynomials (96 segments of width 1/4; F = 0 from
 * d = 24 on), so results are reproducible bit for bit on any launch shape.
 */
#ifndef CTCPB_H
#define CTCPB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without including the CUDA headers. */
typedef struct CUstream_st* ctcpb_stream_t;

/* Host-side status codes. */
#define CTCPB_OK 0
#define CTCPB_EINVAL (-1)   /* a dimension or configuration value is out of range */
#define CTCPB_ENULL (-2)    /* a required pointer is NULL */
#define CTCPB_EALIGN (-3)   /* workspace/state pointer not 256-byte aligned */
#define CTCPB_ESIZE (-4)    /* workspace/state buffer smaller than the size query */
#define CTCPB_ECUDA (-5)    /* a CUDA launch failed (the runtime error is pending) */

/*
 * The coefficient table of the library's logsumexp ("GPU CTC Prefix Beam
 * Search Decoder", section 3: logsumexp(a, b) = max + log(1 + exp(-|a - b|))).
 * log(1 + e^-d) is evaluated on 96 segments [k/4, (k+1)/4) by the degree-5
 * Taylor polynomial about the segment midpoint k/4 + 1/8 (zero for d >= 24);
 * entry 6k + n is the n-th coefficient of segment k, the float32 rounding of
 * the n-th derivative over n!.  Writes the first min(n, 576) entries to the
 * HOST buffer `out` and returns 576 (the table's size), so callers and tests
 * can check the arithmetic the kernels use; negative on a bad argument.
 */
int ctcpb_lse_table(float* out, int n);

/* Device-side status bits (ctcpb_read_status). */
#define CTCPB_DEV_HEADER 0x1u   /* state header does not match the call's dims/config: call skipped */
#define CTCPB_DEV_PAGES 0x2u    /* paged token pool exhausted: the beam kept its prefix (section 13) */
#define CTCPB_DEV_TIMEOUT 0x4u  /* a bounded inter-block wait gave up: results of the call are invalid */
#define CTCPB_DEV_OVERFLOW 0x8u /* an internal candidate buffer overflowed: results are invalid */
#define CTCPB_DEV_BOOST 0x10u   /* a label-boost entry was rejected and ignored (see ctcpb_boost) */
#define CTCPB_DEV_TARGET 0x20u  /* a target outside [0, V) was ignored (ctcpb_cross_entropy), or a pair's index of N
                                   or more (ctcpb_preference_loss) */

/*
 * Decoder configuration (section 11).
 *   beam             beam width, 1..128 (MAX_BEAM_SIZE of section 11).
 *   nbest            hypotheses returned per row, 1..beam.
 *   blank_id         CTC blank label, 0..V-1.
 *   max_seq_len      cap on labels per hypothesis; a hypothesis at the cap has
 *                    no non-blank extension (section 11).  <= 0 selects the
 *                    default: T offline (never binds), 4096 when streaming.
 *   blank_threshold  offline frame skip (section 3.5): frame t is decoded iff
 *                    log_prob[b,t,blank] < log(blank_threshold); >= 1 keeps all
 *                    frames, <= 0 keeps none (section 13).  Ignored when
 *                    streaming.  Must not be NaN.
 *   paged            0: flat double-buffered token rows (section 7, "Flat");
 *                    1: paged, prefix-shared, reference-counted pages (4.2, 7).
 *   page_size        labels per page in paged mode, 1..1024 (section 11: 16).
 *   list_len         labels ranked per frame by the vocabulary pre-pass; 0
 *                    selects min(2*beam+2, V-1) (section 3.4.7).  Any value in
 *                    1..V-1 gives the same decode: when a frame's list cannot
 *                    prove the selection, that step re-ranks the whole frame.
 *   word_boundary    0: no word-boundary label (a zero-initialised config);
 *                    1: space_id is the model's word-boundary ("space") label
 *                    (sections 3.4.1/3.4.2): its extension always takes
 *                    lp[space] + lse(pb, pnb), so every space frame is a token
 *                    of its own, and a space-ending beam has no stay path.
 *   space_id         the word-boundary label, 0..V-1 (no effect when it equals
 *                    blank_id); ignored when word_boundary is 0.
 *   max_boost        0: no label boosting.  1..4096: every row (utterance or
 *                    stream) may boost up to max_boost labels (ctcpb_boost);
 *                    the workspace / state then holds a label-boost hash table
 *                    per row, and the decode runs kernel instantiations that
 *                    read it (the plain ones carry no boosting code).
 */
typedef struct ctcpb_config {
  int32_t beam;
  int32_t nbest;
  int32_t blank_id;
  int32_t max_seq_len;
  float blank_threshold;
  int32_t paged;
  int32_t page_size;
  int32_t list_len;
  int32_t word_boundary;
  int32_t space_id;
  int32_t max_boost;
} ctcpb_config;

/*
 * Label boosting: the per-utterance word-boosting table of "GPU-Accelerated
 * WFST Beam Search Decoder for CTC-based Speech Recognition" (one hash table
 * per utterance, consulted whenever an output label is emitted), applied to
 * CTC labels at the extension point the decoder page names in section 15
 * (scores added to the extension table before the top-K).  A label c that an
 * extension emits -- including the repeat after a blank -- scores
 * lp'[c] = lp[c] + bonus[c] (float32, clamped at -FLT_MAX) in place of
 * lp[c]: in the per-frame label ranking (so step 0 seeds by lp'), in the
 * section 3.4.1 extensions and in the 3.4.3 merge folds.  The blank and the
 * stay path emit no label and keep lp.  Without pruning a prefix scores its
 * CTC log-posterior plus the sum of its labels' bonuses; a positive bonus
 * favours the label, a negative one penalises it.
 *
 * The table of every row is given in compressed-row form, all DEVICE arrays:
 *   row_ptr  [B + 1] int32: row b's entries are [row_ptr[b], row_ptr[b+1])
 *   tokens   [row_ptr[B]] int32: the boosted labels
 *   bonus    [row_ptr[B]] float32: their bonuses
 * Entries are taken in order.  One is rejected -- ignored, with
 * CTCPB_DEV_BOOST set in the device status -- when its label is outside
 * [0, V) or is the blank, repeats an earlier label of the row, its bonus is
 * not finite or exceeds 1e6 in magnitude, or the row already holds max_boost
 * labels; a row whose offsets decrease is ignored whole.
 */
typedef struct ctcpb_boost {
  const int32_t* row_ptr;
  const int32_t* tokens;
  const float* bonus;
} ctcpb_boost;

/*
 * Diagnostic counters of the last call on a workspace or state (synchronises
 * the device): [0] decode steps, [1] steps whose first candidate set could not
 * prove the selection, [2] steps that fell back to an exhaustive selection
 * (warp kernel: over the frame's list; block kernel: the chunked sort of every
 * candidate), [3] steps that also scored every unlisted label of the frame,
 * [4] merges proposed by prefix hashes and confirmed on stored tokens, [5]
 * launches that ran the pre-pass and the steps of a tile as one cooperative
 * kernel (CTCPB_NO_FUSE=1 in the environment makes every call use two kernels
 * instead).
 */
int ctcpb_read_counters(const void* ws_or_state, uint32_t counters[6]);

/* Human-readable text for a host status code. */
const char* ctcpb_status_string(int status);

/*
 * Workspace bytes for ctcpb_decode_offline on [B, T, V] (section 5,
 * calculate_[paged_]workspace_size).  Writes *bytes; returns a status.
 */
int ctcpb_workspace_size(const ctcpb_config* cfg, int B, int T, int V, size_t* bytes);

/*
 * Offline decode (section 3.7 / 12.1, ctc_beam_search_decode[_paged]).
 *   log_prob      [B, T, V] float32, element strides stride_b, stride_t (>= V).
 *   seq_lengths   [B] int32 valid frames per row (values clamped to [0, T]);
 *                 NULL means T for every row.  Frames t >= len_b are never read.
 *   ws, ws_bytes  workspace of at least ctcpb_workspace_size() bytes; its
 *                 contents need no initialisation and are overwritten.
 *   out_tokens    [B, nbest, out_len] int32: labels of each hypothesis, padded
 *                 with -1; a hypothesis longer than out_len is cut (its length
 *                 still reports the full count, section 13).
 *   out_lengths   [B, nbest] int32;  out_scores [B, nbest] float32.
 *   Hypotheses are ordered by score (descending); a row with fewer live
 *   hypotheses than nbest has dead slots (length 0, score -FLT_MAX, tokens -1);
 *   a row with no decoded frame returns the empty hypothesis with score 0 in
 *   slot 0 (section 13).  B == 0 is a no-op.
 */
int ctcpb_decode_offline(const ctcpb_config* cfg, const float* log_prob, int64_t stride_b, int64_t stride_t,
                         const int32_t* seq_lengths, int B, int T, int V, void* ws, size_t ws_bytes,
                         int32_t* out_tokens, int32_t* out_lengths, float* out_scores, int out_len,
                         ctcpb_stream_t stream);

/*
 * ctcpb_decode_offline with label boosting (ctcpb_boost): row b of the batch
 * boosts the labels of boost's row b.  Requires cfg->max_boost >= 1.  A NULL
 * boost is ctcpb_decode_offline.  Errors: CTCPB_EINVAL when max_boost is 0,
 * CTCPB_ENULL for a NULL row_ptr, tokens or bonus, otherwise as
 * ctcpb_decode_offline.
 */
int ctcpb_decode_offline_boosted(const ctcpb_config* cfg, const ctcpb_boost* boost, const float* log_prob,
                                 int64_t stride_b, int64_t stride_t, const int32_t* seq_lengths, int B, int T,
                                 int V, void* ws, size_t ws_bytes, int32_t* out_tokens, int32_t* out_lengths,
                                 float* out_scores, int out_len, ctcpb_stream_t stream);

/*
 * Offline decode of a batch that lives in HOST memory, results written to
 * host memory: the only call of this header whose data pointers are host
 * pointers (the workspace is device memory, as everywhere).  The frames go
 * to the device in chunks (whole 64-frame tiles, at least 1 MB of each row)
 * on the library's own copy stream (valid frames only: row b's first
 * seq_lengths[b]), while `stream` decodes every chunk already there; the
 * results come back on `stream`.  The output
 * is exactly ctcpb_decode_offline's on the same frames.
 *   log_prob      host [B, T, V] float32, element strides stride_b, stride_t.
 *   seq_lengths   host [B] int32, or NULL (T for every row).
 *   ws, ws_bytes  DEVICE workspace of ctcpb_host_workspace_size() bytes
 *                 (its size depends on out_len).
 *   out_tokens / out_lengths / out_scores   host, the layout of
 *                 ctcpb_decode_offline.
 * Asynchrony: with page-locked log_prob, seq_lengths and outputs the call
 * returns once everything is enqueued and completes on `stream` (synchronise
 * it before reading the outputs); pageable buffers make CUDA stage the copies
 * and the call may block.  The host buffers must stay valid until `stream`
 * completes.  Calls are serialised on each device (a lock guards the copy
 * stream and its events).
 */
int ctcpb_host_workspace_size(const ctcpb_config* cfg, int B, int T, int V, int out_len, size_t* bytes);
int ctcpb_decode_offline_host(const ctcpb_config* cfg, const float* log_prob, int64_t stride_b, int64_t stride_t,
                              const int32_t* seq_lengths, int B, int T, int V, void* ws, size_t ws_bytes,
                              int32_t* out_tokens, int32_t* out_lengths, float* out_scores, int out_len,
                              ctcpb_stream_t stream);

/* The same with label boosting (ctcpb_boost: DEVICE arrays, as in
 * ctcpb_decode_offline_boosted; requires cfg->max_boost >= 1). */
int ctcpb_decode_offline_host_boosted(const ctcpb_config* cfg, const ctcpb_boost* boost, const float* log_prob,
                                      int64_t stride_b, int64_t stride_t, const int32_t* seq_lengths, int B, int T,
                                      int V, void* ws, size_t ws_bytes, int32_t* out_tokens, int32_t* out_lengths,
                                      float* out_scores, int out_len, ctcpb_stream_t stream);

/*
 * Offline decode for callers that cannot allocate device memory.  The pages
 * have no counterpart.  It is for code that may not call cudaMalloc: a plugin
 * of an engine that owns the device heap and forbids allocations from outside
 * it, or a real-time path that must not block in the allocator.  Same
 * arguments and results as ctcpb_decode_offline without the workspace: the
 * workspace is a fixed device array of CTCPB_NOALLOC_SCRATCH_BYTES inside this
 * library, held by every device that loads the library until the process
 * exits.
 *   - Returns CTCPB_ESIZE when the problem's workspace (ctcpb_workspace_size)
 *     exceeds CTCPB_NOALLOC_SCRATCH_BYTES; nothing is launched then.
 *   - Calls no allocator.  The first call on each device looks up the array's
 *     device address (cudaGetSymbolAddress) with that device current, and
 *     keeps it for the process.  The kept address does not survive
 *     cudaDeviceReset: do not use this call on a device after resetting it.
 *   - All calls on a device share the one array, which keeps the last call's
 *     contents (each call resets what it reads before reading it).  Calls
 *     whose work overlaps on the GPU (different streams, or several host
 *     threads) race and corrupt each other's results.  Serialise them, e.g. on
 *     one stream.
 *   - ctcpb_noalloc_read_status reads the array's device status word (the
 *     CTCPB_DEV_* bits of the last call on the current device, as
 *     ctcpb_read_status does for a workspace).  It synchronises the device.
 */
#define CTCPB_NOALLOC_SCRATCH_BYTES (32u << 20)
int ctcpb_decode_offline_noalloc(const ctcpb_config* cfg, const float* log_prob, int64_t stride_b, int64_t stride_t,
                                 const int32_t* seq_lengths, int B, int T, int V, int32_t* out_tokens,
                                 int32_t* out_lengths, float* out_scores, int out_len, ctcpb_stream_t stream);
int ctcpb_noalloc_read_status(uint32_t* device_status);

/*
 * Streaming state bytes for B independent streams of vocabulary V (section 5,
 * calculate_[paged_]state_buffer_size).  The state holds each stream's beam,
 * its label storage and its step/frame counters (section 4.3).
 */
int ctcpb_state_size(const ctcpb_config* cfg, int B, int V, size_t* bytes);

/*
 * Reset a streaming state (section 8, init_streaming_state[_paged]): every
 * stream starts before its first frame.  The state is position independent
 * (offsets, not pointers), so it may be copied with cudaMemcpy and resumed.
 */
int ctcpb_stream_init(const ctcpb_config* cfg, void* state, size_t state_bytes, int B, int V,
                      ctcpb_stream_t stream);

/*
 * Set the label boosts of every stream of a state (ctcpb_boost; requires
 * cfg->max_boost >= 1): they replace the streams' previous boosts and apply
 * from the next decoded frame on (ctcpb_stream_init clears them).  Errors:
 * CTCPB_EINVAL when max_boost is 0, CTCPB_ENULL for a NULL boost, row_ptr,
 * tokens or bonus, otherwise as ctcpb_stream_step_chunk.
 */
int ctcpb_stream_set_boost(const ctcpb_config* cfg, void* state, size_t state_bytes, int B, int V,
                           const ctcpb_boost* boost, ctcpb_stream_t stream);

/*
 * Decode one chunk of frames for every stream (section 8, ctc_beam_search_chunk).
 *   lp_chunk   [B, chunk_T, V] float32 with element strides stride_b, stride_t.
 *   n_frames   [B] int32 device array: stream b decodes its first n_frames[b]
 *              rows of the chunk (values clamped to [0, chunk_T]); NULL means
 *              chunk_T for every stream.
 * Streaming never skips frames (section 3.5).  The step and frame counters
 * live in the state on the device.  Decoding a stream in any chunking gives
 * the same result as decoding its frames offline without skipping.
 */
int ctcpb_stream_step_chunk(const ctcpb_config* cfg, void* state, size_t state_bytes, int B, int V,
                            const float* lp_chunk, int64_t stride_b, int64_t stride_t, const int32_t* n_frames,
                            int chunk_T, ctcpb_stream_t stream);

/*
 * ctcpb_stream_step_chunk with a speech mask (section 8's is_speech_mask of
 * ctc_beam_search_chunk; sections 14 and 15: frames marked as non-speech
 * bypass the decoder).
 *   is_speech    [B, chunk_T] uint8 device array, row stride mask_stride
 *                (>= chunk_T): frame j of stream b is decoded iff
 *                is_speech[b * mask_stride + j] != 0.
 * A masked frame still advances the stream's frame counter; the decoder
 * treats it like a frame skipped by the blank threshold (section 3.5): the
 * next decoded frame collapses the beam's blank-ending residue (section 3.4).
 * Decoding a stream in any chunking gives the same result as decoding its
 * frames offline with the same mask.  Errors: CTCPB_ENULL for a null mask,
 * CTCPB_EINVAL for mask_stride < chunk_T, otherwise as ctcpb_stream_step_chunk.
 */
int ctcpb_stream_step_chunk_masked(const ctcpb_config* cfg, void* state, size_t state_bytes, int B, int V,
                                   const float* lp_chunk, int64_t stride_b, int64_t stride_t,
                                   const int32_t* n_frames, const uint8_t* is_speech, int64_t mask_stride,
                                   int chunk_T, ctcpb_stream_t stream);

/*
 * Decode one frame for every stream (section 9, ctc_beam_search_step: one
 * streaming frame).
 *   lp_frame   [B, V] float32, row stride stride_b (>= V) elements.
 *   is_speech  [B] uint8 device array or NULL: stream b decodes the frame iff
 *              is_speech[b] != 0; NULL decodes it for every stream.  A stream
 *              whose flag is 0 still advances its frame counter, like a masked
 *              frame of ctcpb_stream_step_chunk_masked: this is how a caller
 *              that drops frames marks the gap that the pages' step call takes
 *              as actual_frame_index.
 * The same as ctcpb_stream_step_chunk (ctcpb_stream_step_chunk_masked when
 * is_speech is given) with chunk_T = 1, and with the same errors.
 */
int ctcpb_stream_step(const ctcpb_config* cfg, void* state, size_t state_bytes, int B, int V,
                      const float* lp_frame, int64_t stride_b, const uint8_t* is_speech, ctcpb_stream_t stream);

/*
 * Write the current N best of every stream (section 8, read_streaming_results)
 * in the output layout of ctcpb_decode_offline.  Does not modify the state.
 */
int ctcpb_read_state(const ctcpb_config* cfg, const void* state, size_t state_bytes, int B, int V,
                     int32_t* out_tokens, int32_t* out_lengths, float* out_scores, int out_len,
                     ctcpb_stream_t stream);

/*
 * Self-test of the bounded waits (failure detection without a GPU fault).
 * One warp runs the two forms of wait the kernels use against conditions
 * that never complete, and gives up as the kernels do:
 *   flags      [nflags] uint32 device array: ready flags acquired up to 32 at
 *              a time, as the fused launch waits for ranked records; the wait
 *              stops at the first flag still 0 after max_spins tries
 *              (1 <= max_spins <= 2^20, about 100 ns a try);
 *   then an mbarrier phase that expects two arrivals and gets one, waited on
 *   with the pre-pass's bounded barrier wait (under a second).
 *   out        [3] uint32 device array: out[0] = flags found set in order,
 *              out[1] = CTCPB_DEV_TIMEOUT if the flag wait gave up, out[2] =
 *              CTCPB_DEV_TIMEOUT if the barrier wait gave up (it always does).
 * Asynchronous on `stream`; the context stays usable.  Errors: CTCPB_EINVAL
 * for nflags < 0 or max_spins out of range, CTCPB_ENULL for a NULL out (or
 * NULL flags with nflags > 0), CTCPB_ECUDA for a failed launch.
 */
int ctcpb_selftest_waits(const uint32_t* flags, int nflags, long long max_spins, uint32_t* out,
                         ctcpb_stream_t stream);

/*
 * Copy the device status word of a workspace or state to *device_status.
 * Synchronises the device (for tests and error reporting, not the hot path).
 */
int ctcpb_read_status(const void* ws_or_state, uint32_t* device_status);

/* ---- Stage entry points (the steps of the hot path, exposed for testing
 * and per-kernel timing). */

/* Stages of ctcpb_decode_offline, in launch order. */
#define CTCPB_STAGE_INIT 0x1u    /* reset the workspace's per-row state (section 3.7) */
#define CTCPB_STAGE_SELECT 0x2u  /* frame selection (section 3.5) */
#define CTCPB_STAGE_RANK 0x4u    /* vocabulary pre-pass of every kept frame (section 3.4.7) */
#define CTCPB_STAGE_STEPS 0x8u   /* all decode steps of every row (sections 3.3-3.4) */
#define CTCPB_STAGE_OUTPUT 0x10u /* N-best gather (section 3.6) */
#define CTCPB_STAGE_ALL 0x1fu

/*
 * ctcpb_decode_offline restricted to the stages in stage_mask, on the same
 * workspace and with the same arguments.  Running the five stages in order,
 * in one call or several, is exactly ctcpb_decode_offline; a stage reads what
 * the earlier stages left in the workspace.
 */
int ctcpb_decode_offline_staged(const ctcpb_config* cfg, const float* log_prob, int64_t stride_b, int64_t stride_t,
                                const int32_t* seq_lengths, int B, int T, int V, void* ws, size_t ws_bytes,
                                int32_t* out_tokens, int32_t* out_lengths, float* out_scores, int out_len,
                                uint32_t stage_mask, ctcpb_stream_t stream);

/* Number of labels the pre-pass ranks per frame for this config and V (>= 1),
 * or a negative status for an invalid config. */
int ctcpb_list_len(const ctcpb_config* cfg, int V);

/*
 * Frame selection (section 3.5): sel [B, T] int32 receives the kept frames of
 * each row in order (the rest of the row is -1), nsel [B] their count.  The
 * frames, lengths and threshold are read as in ctcpb_decode_offline.  Errors:
 * CTCPB_EINVAL for B or T < 0 or a stride below V, CTCPB_ENULL for a NULL
 * nsel (or log_prob or sel with T > 0); B == 0 is a no-op.
 */
int ctcpb_select_frames(const ctcpb_config* cfg, const float* log_prob, int64_t stride_b, int64_t stride_t,
                        const int32_t* seq_lengths, int B, int T, int V, int32_t* sel, int32_t* nsel,
                        ctcpb_stream_t stream);

/*
 * Vocabulary pre-pass (section 3.4.7) over R frame rows (row r at
 * log_prob + r * stride_r): the first L = list_len non-blank live labels by
 * (log-prob desc, label asc) -> ids [R, L] int32 / lps [R, L] float32 (padded
 * with -1 / -FLT_MAX), cnt [R], the blank log-prob lpb [R], and the next
 * ranked label after the list (front_id [R], front_lp [R]; -1 / -FLT_MAX when
 * none).  A label is live iff its log-prob is > -FLT_MAX (NaN and -inf are
 * read as -FLT_MAX).  Errors: CTCPB_EINVAL for R < 0 or stride_r < V,
 * CTCPB_ENULL for any NULL array; R == 0 is a no-op.
 */
int ctcpb_topk_prepass(const ctcpb_config* cfg, const float* log_prob, int64_t stride_r, int R, int V,
                       int32_t* ids, float* lps, int32_t* cnt, float* lpb, float* front_lp, int32_t* front_id,
                       ctcpb_stream_t stream);

/* ---- The label head: what produces log_prob and what trains it.
 *
 * An acoustic model ends in a layer norm and a linear head; the head's
 * log-softmax is the decoder's log_prob.  Rows are frames (or tokens): x is
 * [N, H], row r at x + r * ldx elements, its features contiguous.  The
 * conventions above hold: device pointers, caller-owned memory, asynchronous
 * calls, statuses.  Element types: */
#define CTCPB_F32 0
#define CTCPB_BF16 1
#define CTCPB_F16 2
/* Limits: N <= 2^24 rows, H <= 8192 features, V <= 2^20 labels. */

/*
 * Layer norm: y = (x - mean) * rstd * weight + bias, with the mean and
 * rstd = 1 / sqrt(variance + eps) of each row (variance over H, not H - 1).
 *   type         of x and y: CTCPB_F32, CTCPB_BF16 or CTCPB_F16.
 *   param_type   of weight and bias: `type` or CTCPB_F32.
 *   weight, bias [H], each may be NULL (1 and 0).
 *   mean, rstd   [N] float32, for the backward pass; both NULL: not written.
 * Sums and statistics are float32; y is rounded once.  N == 0 is a no-op.
 */
int ctcpb_layer_norm(int type, int param_type, const void* x, int64_t ldx, const void* weight, const void* bias,
                     float eps, int64_t N, int H, void* y, int64_t ldy, float* mean, float* rstd,
                     ctcpb_stream_t stream);

/*
 * Its backward pass: with xh = (x - mean) * rstd and t = dy * weight,
 *   dx = rstd * (t - mean_H(t) - xh * mean_H(t * xh)),
 *   dweight = sum over rows of dy * xh,  dbias = sum over rows of dy.
 * x, mean, rstd as given to and written by ctcpb_layer_norm.  dx, dweight and
 * dbias may each be NULL (not computed); with N == 0 the sums are 0.  The row
 * sums are made in a fixed order, so results are reproducible bit for bit.
 * The workspace is needed for dweight and dbias.
 */
int ctcpb_layer_norm_workspace_size(int64_t N, int H, size_t* bytes);
int ctcpb_layer_norm_backward(int type, int param_type, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                              const void* weight, const float* mean, const float* rstd, int64_t N, int H, void* dx,
                              int64_t lddx, void* dweight, void* dbias, void* ws, size_t ws_bytes,
                              ctcpb_stream_t stream);

/*
 * The decoder's input: out[r, :] = log_softmax(x[r] weight^T + bias), float32.
 *   type       of x and weight: CTCPB_BF16 or CTCPB_F16 (products on the
 *              tensor cores, accumulated in float32).
 *   weight     [V, H], row stride ldw elements.
 *   bias       [V] of bias_type (`type` or CTCPB_F32), or NULL.  A bias of
 *              -inf takes its label out (log-probability -inf); a row whose
 *              labels are all out is NaN.
 *   out        row stride ldo (>= V) elements.  Rows that start on 16-byte
 *              boundaries (ldo % 4 == 0) are written, and decoded, fastest.
 *   ws         ctcpb_log_probs_workspace_size() bytes.
 * A value is (z - max z) - log sum exp(z - max z), the difference exact where it
 * is small: never above 0, and 0 for a certain label, however large its z.
 * The tensor cores cut their accumulator off at every 16 features.  The mean of
 * that for dense features of either sign, 0.26 * 2^-24 of z for each 16, is put
 * back in all three calls.  Such z are then right to 0.13 * 2^-24 for each 16 on
 * average (2.5e-7 of z at H = 512); sums that are exact (one-hot features, small
 * integers) are 0.26 too large (5e-7 of z at H = 512, 8e-6 at 8192), and products
 * of one sign up to 1.5 too small.
 * Any strides >= H and any alignment of the element type are taken; x or
 * weight whose rows do not start on 16-byte boundaries, or whose H is no multiple
 * of 8, are laid out again in the workspace first (every workspace of these calls
 * has the room, 2 N H and 2 V H bytes, used or not).  N == 0 is a no-op.
 */
int ctcpb_log_probs_workspace_size(int type, int64_t N, int V, int H, size_t* bytes);
int ctcpb_log_probs(int type, int bias_type, const void* x, int64_t ldx, const void* weight, int64_t ldw,
                    const void* bias, int64_t N, int V, int H, float* out, int64_t ldo, void* ws, size_t ws_bytes,
                    ctcpb_stream_t stream);

/*
 * Softmax cross entropy of the head's logits z = x weight^T + bias, which are
 * never stored: loss_r = lse_r - z[r, target_r], lse_r = log sum_c exp z[r, c].
 * (loss_r from the distances to the row's largest z: never below 0.)
 *   targets       [N] int32.  A row whose target is ignore_index takes no part:
 *                 its x is not read into any sum, its loss and lse are 0.  Any
 *                 other target outside [0, V) is ignored as well and sets
 *                 CTCPB_DEV_TARGET in the status word.
 *   reduction     CTCPB_REDUCE_NONE: loss is [N]; _MEAN: one value, the mean over
 *                 the rows that take part (NaN if none does); _SUM: one value.
 *   lse           [N] float32, for the backward pass.
 * Types as in ctcpb_log_probs; the losses are float32.
 */
#define CTCPB_REDUCE_NONE 0
#define CTCPB_REDUCE_MEAN 1
#define CTCPB_REDUCE_SUM 2
int ctcpb_cross_entropy_workspace_size(int type, int64_t N, int V, int H, int backward, size_t* bytes);
int ctcpb_cross_entropy(int type, int bias_type, const void* x, int64_t ldx, const void* weight, int64_t ldw,
                        const void* bias, const int32_t* targets, int64_t N, int V, int H, int32_t ignore_index,
                        int reduction, float* loss, float* lse, void* ws, size_t ws_bytes, ctcpb_stream_t stream);

/*
 * Its gradients: with d[r, c] = (exp(z[r, c] - lse_r) - [c = target_r]) * g_r,
 *   dx = d weight  [N, H],  dweight = d^T x  [V, H],  dbias = sum_r d[r]  [V],
 * where g_r is grad[r] (REDUCE_NONE), grad[0] (REDUCE_SUM) or grad[0] over the
 * number of rows that take part (REDUCE_MEAN); ignored rows get exact zeros.
 * z is made again with the forward call's roundings: the target of a row that is
 * certain of it (lse_r is z[r, target_r] in float32) has d = 0.
 *   grad          device float32: [N] or one value.
 *   lse           of the forward call, on the same x, weight, bias and targets.
 *   dx, dweight   of `type`, row strides lddx, lddw;  dbias of bias_type.  Each
 *                 may be NULL (not computed).
 * The logits are made again, in pieces of the vocabulary whose d takes at most
 * 256 MB of the workspace, or 512 bytes a row where that is more (a piece is at
 * least 256 labels; above 524,288 rows).  d is held in `type` (16 bits), in small
 * calls as two such terms, the rounded value and what that took off; every sum is float32 and in
 * a fixed order, so results are reproducible bit for bit.  An ignored row's
 * grad[r] is of no account, whatever it holds; one of a kept row that is not
 * finite shows in that row of dx and in the sums over rows.  CTCPB_F16 with
 * REDUCE_NONE holds d relative to the largest finite |grad[r]| of the kept rows:
 * what is below 2^-39 of it (2^-29: with fewer bits) is lost.
 */
int ctcpb_cross_entropy_backward(int type, int bias_type, const float* grad, const void* x, int64_t ldx,
                                 const void* weight, int64_t ldw, const void* bias, const int32_t* targets,
                                 const float* lse, int64_t N, int V, int H, int32_t ignore_index, int reduction,
                                 void* dx, int64_t lddx, void* dweight, int64_t lddw, void* dbias, void* ws,
                                 size_t ws_bytes, ctcpb_stream_t stream);

/* ---- Around the label head: a norm for convolutional blocks, dropout, and the
 * losses that train the model from the decoder's own N-best lists. */

/*
 * Group norm with an activation, over frames with their channels last:
 *   y[b, t, c] = act((x[b, t, c] - mean[b, g]) * rstd[b, g] * weight[c] + bias[c]),
 * g = c / (C / G), the mean and rstd = 1 / sqrt(variance + eps) taken over the
 * frames t < lengths[b] and the C / G channels of the group.
 *   type          of x and y: CTCPB_F32, CTCPB_BF16 or CTCPB_F16.
 *   param_type    of weight and bias: `type` or CTCPB_F32.
 *   x, y          [B, T, C]: utterance b, frame t at b * stride_b + t * stride_t
 *                 elements, C contiguous; stride_t >= C, stride_b any but negative.
 *   weight, bias  [C], each may be NULL (1 and 0).
 *   lengths       [B] int32 frames of each utterance (clamped to [0, T]); NULL: T.
 *                 Frames from there on are not read, and y is 0 there.
 *   activation    CTCPB_ACT_NONE, CTCPB_ACT_RELU max(h, 0) or CTCPB_ACT_SILU
 *                 h / (1 + exp(-h)).
 *   mean, rstd    [B, G] float32, for the backward pass; both NULL: not written.
 *                 An utterance without frames has mean 0 and rstd 0.
 * Limits: B * T <= 2^24 frames, C <= 8192 channels, G divides C.  The variance is
 * the mean squared distance from the mean (no difference of large sums); sums
 * and statistics are float32 in a fixed order, y is rounded once.  y may not
 * overlap x.  B * T == 0 is a no-op, but for mean and rstd.
 *   ws            ctcpb_group_norm_workspace_size() bytes; NULL where that is 0 (a
 *                 forward call whose utterances' groups fit in shared memory).
 */
#define CTCPB_ACT_NONE 0
#define CTCPB_ACT_RELU 1
#define CTCPB_ACT_SILU 2
int ctcpb_group_norm_workspace_size(int type, int B, int T, int C, int G, int backward, size_t* bytes);
int ctcpb_group_norm(int type, int param_type, const void* x, int64_t x_stride_b, int64_t x_stride_t,
                     const void* weight, const void* bias, const int32_t* lengths, float eps, int activation, int B,
                     int T, int C, int G, void* y, int64_t y_stride_b, int64_t y_stride_t, float* mean, float* rstd,
                     void* ws, size_t ws_bytes, ctcpb_stream_t stream);

/*
 * Its backward pass: with xh = (x - mean) * rstd, h = xh * weight + bias,
 * dh = dy * act'(h) (relu'(0) = 0) and t = dh * weight,
 *   dx = rstd * (t - mean_g(t) - xh * mean_g(t * xh)),  0 from lengths[b] on,
 *   dweight = sum over b, t of dh * xh,  dbias = sum over b, t of dh.
 * x, weight, bias, lengths, mean, rstd and activation as in the forward call.
 * dx, dweight and dbias may each be NULL (not computed); no frames: sums of 0.
 * Results are reproducible bit for bit.  dx may not overlap x or dy.
 */
int ctcpb_group_norm_backward(int type, int param_type, const void* dy, int64_t dy_stride_b, int64_t dy_stride_t,
                              const void* x, int64_t x_stride_b, int64_t x_stride_t, const void* weight,
                              const void* bias, const int32_t* lengths, const float* mean, const float* rstd,
                              int activation, int B, int T, int C, int G, void* dx, int64_t dx_stride_b,
                              int64_t dx_stride_t, void* dweight, void* dbias, void* ws, size_t ws_bytes,
                              ctcpb_stream_t stream);

/*
 * Dropout from a counter-based generator; its mask is never stored.
 *   y[r, c] = residual[r, c] + (kept ? x[r, c] * 65536 / (65536 - k) : 0)
 * Element i = r * H + c, whatever the strides, is kept iff its 16-bit number is at
 * least k = 65536 p, rounded to the nearest integer (half to even): p is held to
 * 2^-16, the factor is exact for the p that is.  The number is half i % 8 (low
 * half of a word first) of the four words of Philox4x32 with 10 rounds (Salmon,
 * Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), key =
 * the seed's low and high word, counter = (i / 8 low, high, offset low, high).
 *   rng        [2] int64, on the device: seed and offset.  Another offset gives
 *              other numbers; the caller changes it between steps (a replayed
 *              graph reads what it holds then).
 *   p          in [0, 1]; k = 65536 drops all.  A dropped element is 0 whatever x
 *              holds.
 *   residual   of x's type, or NULL.
 *   x, y       [N, H] of `type`, rows ldx, ldr, ldy elements apart; y may be x or
 *              residual itself, with its stride.
 * Limits: N <= 2^24 rows, H <= 8192.  The sum is float32, rounded once.
 * The backward pass is the same call on dy without a residual (the residual's
 * gradient is dy itself).
 */
int ctcpb_dropout(int type, const void* x, int64_t ldx, const void* residual, int64_t ldr, double p,
                  const int64_t* rng, int64_t N, int H, void* y, int64_t ldy, ctcpb_stream_t stream);

/*
 * The clipped policy loss of sequences (hypotheses of N-best lists) with a KL term.
 * A sequence's tokens have negative log-probabilities, as ctcpb_cross_entropy gives
 * them without a reduction (CTCPB_REDUCE_NONE), and an advantage A.  With
 *   ratio = exp(old_nll - nll),  u = nll - ref_nll,
 *   token loss = -min(ratio * A, clamp(ratio, 1 - clip_low, 1 + clip_high) * A)
 *                + kl_weight * (exp(u) - 1 - u).
 *   nll, old_nll, ref_nll   [S, L] float32, rows ld_* elements apart; ref_nll NULL:
 *                 no KL term (kl_weight is of no account).
 *   advantages    [S] float32 (ld_advantages == 0), or [S, L] with rows that far apart.
 *                 Where A is 0 the first term is 0, whatever the ratio.
 *   lengths       [S] int32 tokens of each sequence (clamped to [0, L]); NULL: L.
 *                 What a row holds behind them is of no account.
 *   clip_low      in [0, inf), clip_high in [0, inf]; whether a ratio is past the
 *                 border is decided without rounding it.
 *   reduction     CTCPB_REDUCE_NONE: loss is [S, L], 0 behind the lengths; _MEAN: one
 *                 value, the mean over all tokens; _SUM; or CTCPB_REDUCE_SEQUENCE_MEAN:
 *                 the mean, over the sequences that have tokens, of each one's mean.
 *                 Means over nothing are NaN, their gradients 0.
 *   grad          the loss's gradient, device float32: one value, or [S, L] (NONE),
 *                 dense; NULL with dnll NULL.
 *   loss          NULL: not written.
 *   stats         [2] float32 or NULL: the mean over all tokens of exp(u) - 1 - u
 *                 (0 without ref_nll), and the share of tokens held at the border.
 *   dnll          [S, L] float32, dense, or NULL: the gradient with respect to nll,
 *                 0 behind the lengths; in the same pass, as ctcpb_cross_entropy_backward
 *                 takes it.
 *   ws            ctcpb_policy_loss_workspace_size() bytes; may be NULL where that is
 *                 256 (small calls, which have only the status in it).
 * Sums over tokens are pairs of float32 (value and error), made in a fixed order.
 * Limits: S, L <= 2^24, S * L < 2^32.
 */
#define CTCPB_REDUCE_SEQUENCE_MEAN 3
int ctcpb_policy_loss_workspace_size(int64_t S, int64_t L, size_t* bytes);
int ctcpb_policy_loss(const float* nll, int64_t ld_nll, const float* old_nll, int64_t ld_old, const float* ref_nll,
                      int64_t ld_ref, const float* advantages, int64_t ld_advantages, const int32_t* lengths,
                      int64_t S, int64_t L, double clip_low, double clip_high, float kl_weight, int reduction,
                      const float* grad, float* loss, float* stats, float* dnll, void* ws, size_t ws_bytes,
                      ctcpb_stream_t stream);

/*
 * The preference loss of a pair of hypotheses of each N-best list.  With
 *   R[b, n] = sum over the hypothesis' tokens of (ref_nll - nll)   (its log-probability,
 *             over the reference model's; `average`: over its length too),
 *   z[b] = beta * (R[b, chosen[b]] - R[b, rejected[b]]) - margin,
 *   loss[b] = (1 - s) * log(1 + exp(-z)) + s * log(1 + exp(z)),  s = label_smoothing.
 *   nll, ref_nll       [B, N, L] float32: hypothesis n of list b is row b * N + n, rows
 *                      ld_* apart; ref_nll NULL: 0.
 *   chosen, rejected   [B] int32 in [0, N).  A list with a negative index takes no part:
 *                      its loss, margin and gradients are 0.  One with an index of N or
 *                      more is ignored as well and sets CTCPB_DEV_TARGET in the
 *                      workspace's status.  Both the same: z = -margin, no gradient.
 *   lengths            [B, N] int32 (clamped to [0, L]); NULL: L.  R of none is 0.
 *   reduction          CTCPB_REDUCE_NONE: loss is [B]; _MEAN: over the lists that take
 *                      part (NaN if none does; gradients 0); _SUM.
 *   grad               device float32: one value, or [B] (NONE); NULL with dnll NULL.
 *   loss, margins      margins [B]: z.  Each may be NULL.
 *   dnll               [B, N, L] float32, dense, or NULL: the gradient with respect to
 *                      nll, 0 for the other hypotheses and behind the lengths.
 *   ws                 as in ctcpb_policy_loss; without one there is no status.
 * R is summed in pairs of float32 (value and error), in a fixed order.
 * Limits: B * N, L <= 2^24; 0 <= s <= 1; beta and margin finite.
 */
int ctcpb_preference_loss_workspace_size(int64_t B, int N, int64_t L, size_t* bytes);
int ctcpb_preference_loss(const float* nll, int64_t ld_nll, const float* ref_nll, int64_t ld_ref,
                          const int32_t* chosen, const int32_t* rejected, const int32_t* lengths, int64_t B, int N,
                          int64_t L, float beta, float margin, float label_smoothing, int average, int reduction,
                          const float* grad, float* loss, float* margins, float* dnll, void* ws, size_t ws_bytes,
                          ctcpb_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CTCPB_H */
