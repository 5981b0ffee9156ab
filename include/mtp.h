/*
 * mtp.h — C ABI of the GB300 multi-token-prediction (MTP) speculative
 * decoding step: the MTP drafter head, the batched flush of completed pairs
 * into the draft KV cache, the sampling transforms, the rejection-sampling
 * verify and the KV rollback.
 *
 * Conventions for every entry point
 *  - Pointers named d_* are CUDA device pointers; h_* are host pointers.
 *    No torch or CUDA C++ types appear; `mtp_stream` is a cudaStream_t.
 *  - Every call is asynchronous on the given stream, allocates nothing, never
 *    reads device memory on the host and never synchronises, so a caller can
 *    capture a whole round into a CUDA graph. Only mtp_load / mtp_free
 *    allocate and free (the handle's scratch and norm copies) and may block.
 *  - Arguments are validated on the host before any launch; a bad argument
 *    returns a status and launches nothing. Faults seen on the device (a
 *    non-finite logit, a bounded wait that ran out) are OR-ed, as
 *    1 << MTP_ERR_*, into a device status word that the caller reads at its
 *    one per-round synchronisation: the handle's word (mtp_device_status) for
 *    the head calls, the caller's d_status for spec_verify, which takes no
 *    handle. The outputs of a call whose status word gained a bit carry no
 *    meaning; spec_verify's still stay in range (token ids in [0, V), counts
 *    in [0, depth]).
 *  - The caller owns every buffer it passes. Large weights, the borrowed
 *    embedding / lm_head and the KV buffers are borrowed by mtp_load and must
 *    outlive the handle.
 *
 * Notation: H hidden, nq / nkv query / key-value heads, dh head_dim, I SwiGLU
 * intermediate, V vocabulary, R rows (independent sequences), d draft depth.
 */
#ifndef MTP_H
#define MTP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* mtp_stream; /* cudaStream_t */
typedef struct mtp_handle* mtp_t;

typedef enum {
  MTP_OK = 0,
  MTP_ERR_UNSUPPORTED_ARCH = 1, /* architecture is not "qwen3_5_mtp" */
  MTP_ERR_MISSING_TENSOR = 2,   /* one of the 15 head tensors is absent */
  MTP_ERR_DUP_TENSOR = 3,       /* a tensor name appears twice */
  MTP_ERR_UNKNOWN_TENSOR = 4,   /* a name outside the 15-tensor inventory */
  MTP_ERR_SHAPE = 5,            /* a tensor's shape or dtype disagrees with the config */
  MTP_ERR_CONFIG_BOUNDS = 6,    /* a config scalar is out of range */
  MTP_ERR_NOT_BOUND = 7,        /* no borrowed embedding was given (bind skipped) */
  MTP_ERR_KV_CAPACITY = 8,      /* a write would pass the KV capacity */
  MTP_ERR_BAD_ARG = 9,          /* null pointer, bad count, bad sampling parameter */
  MTP_ERR_NONFINITE = 10,       /* device status bit: a non-finite logit was seen */
  MTP_ERR_TIMEOUT = 11,         /* device status bit: a bounded wait on an asynchronous copy ran out */
  MTP_ERR_CUDA = 12,            /* a CUDA runtime call failed */
  MTP_ERR_LAYOUT = 13           /* tensor names mix the raw-HF "mtp." and split layouts */
} mtp_status;

enum { MTP_DTYPE_F32 = 0, MTP_DTYPE_BF16 = 1 };

/* Head configuration. Mirrors the text_config scalars of a qwen3_5_mtp
 * drafter ("support the qwen3_5_mtp drafter" issue, "Where the MTP weights
 * actually live": hidden_size, head_dim, mtp_num_hidden_layers). Bounds are
 * checked at load ("bound the qwen3_5_mtp drafter config scalars at load"). */
typedef struct {
  const char* architecture; /* must equal "qwen3_5_mtp" */
  int32_t hidden;           /* H, multiple of 256, <= 16384 */
  int32_t n_q, n_kv;        /* query / kv heads; n_q % n_kv == 0 */
  int32_t head_dim;         /* dh in {64, 128, 256} */
  int32_t inter;            /* I, multiple of 256 */
  int32_t vocab;            /* V, <= 1 << 20 */
  int32_t mtp_layers;       /* must be 1 (the published head has one layer) */
  int32_t max_rows;         /* R, 1..64 */
  int32_t kv_capacity;      /* slots per row, multiple of 64 */
  int32_t max_depth;        /* drafts per round, 1..16 */
  float eps;                /* RMSNorm epsilon */
  float rope_theta;         /* RoPE base */
  int32_t dtype;            /* MTP_DTYPE_F32 or MTP_DTYPE_BF16: weights, embedding, KV */
} mtp_config;

/* One named head tensor (device memory, row-major). Names follow either the
 * raw-HF layout ("mtp.fc.weight", ...) or the split drafter layout
 * ("fc.weight", ...). In the raw-HF layout the loader adds 1.0 to the seven
 * RMSNorm weights (suffixes .input_layernorm.weight,
 * .post_attention_layernorm.weight, .q_norm.weight, .k_norm.weight,
 * norm.weight, pre_fc_norm_embedding.weight, pre_fc_norm_hidden.weight) exactly
 * once ("Upstream contract to port", sanitize paragraph). */
typedef struct {
  const char* name;
  const void* data;
  int32_t dtype;
  int32_t ndim;     /* 1 or 2 */
  int64_t shape[2];
} mtp_tensor;

/* Per-row sampling parameters. temperature 0 (or top_k 1) is greedy: the
 * point mass at the argmax ("greedy is a special case of sampled decoding",
 * Ollama MLX-runner commit log). rep_penalty 1, top_k 0, top_p 1, min_p 0
 * disable their transforms.
 *
 * flags: 0, or MTP_SAMPLE_ARGMAX_DRAFT on a sampled row: the drafter proposes
 * the argmax of its (penalised) logits instead of a sample, and spec_verify
 * treats that draft as a point mass q (q(x) = 1): x is accepted with
 * probability p(x) and a rejection draws from p with x removed, so the
 * committed tokens still follow p. This is the drafter flag
 * supports_greedy_draft_argmax ("feat(inference): support the qwen3_5_mtp
 * drafter" issue, Upstream contract to port); mtp_draft then needs neither
 * d_q nor d_u for the row, and spec_verify reads no q for it. */
#define MTP_SAMPLE_ARGMAX_DRAFT 1
typedef struct {
  float temperature;  /* >= 0 */
  float rep_penalty;  /* > 0 */
  float top_p;        /* (0, 1] */
  float min_p;        /* [0, 1) */
  int32_t top_k;      /* 0 = off, else 1..1024 */
  int32_t flags;      /* 0 or MTP_SAMPLE_ARGMAX_DRAFT; other bits are rejected
                         (frequency penalty is not implemented) */
} mtp_sampling;

/* Draft KV cache buffers, caller-owned device memory, borrowed by mtp_load.
 * k, v: [max_rows][n_kv][kv_capacity][head_dim] in the config dtype.
 * len:  [max_rows] int32, the number of valid slots per row; the library
 *       keeps it equal to its host-side lengths after every call. */
typedef struct {
  void* k;
  void* v;
  int32_t* len;
} mtp_kv;

/* Default round budget including the bonus token: mtp_layers + 2 (the
 * drafter's block_size, "Upstream contract to port"). Drafts per round are
 * block_size - 1. */
int32_t mtp_default_block_size(const mtp_config* cfg);

const char* mtp_status_str(mtp_status s);

/* Validate the config and the tensor table, copy the seven norm vectors into
 * library memory as fp32 (with the raw-HF +1.0 applied once), borrow every
 * matrix, the embedding and the lm_head (NULL = tied to embed, the drafter's
 * bind fallback), borrow the KV buffers, set every row length to h_len[r]
 * (or 0 if h_len is NULL) and allocate the scratch. Blocks until the copies
 * finish. Errors: UNSUPPORTED_ARCH, MISSING/DUP/UNKNOWN_TENSOR, LAYOUT, SHAPE,
 * CONFIG_BOUNDS, NOT_BOUND (embed NULL), BAD_ARG, CUDA. On error *out is NULL
 * and nothing stays allocated. */
mtp_status mtp_load(const mtp_config* cfg, const mtp_tensor* tensors, int32_t n_tensors,
                    const void* d_embed, const void* d_lm_head, mtp_kv kv,
                    const int32_t* h_len, mtp_stream stream, mtp_t* out);

mtp_status mtp_free(mtp_t h);

/* Host view of the per-row draft KV lengths (the library's source of truth;
 * mirrored into kv.len on the device). h_len: [max_rows]. */
mtp_status mtp_get_lengths(mtp_t h, int32_t* h_len);

/* Set row lengths (e.g. after the caller pre-filled or restored the cache). */
mtp_status mtp_set_lengths(mtp_t h, mtp_stream stream, const int32_t* h_len);

/* Device pointer of the handle's status word (int32, OR of 1 << status). */
int32_t* mtp_device_status(mtp_t h);

/*
 * mtp_flush — write completed pairs into the draft KV.
 * Slot S pairs the token at S+1 with the target hidden at S ("Ollama qwen3_5
 * MTP loader and SelfDraft path", Facts: pairing and the 256-token flush cap).
 * Row r's pairs j = 0..h_pairs[r]-1 go to slots len[r] + j, and len[r]
 * advances by h_pairs[r]. For a one-layer head a slot's K and V depend only on
 * its own pair (fc, input norm, k/v projections, k_norm, RoPE), so the flush
 * computes exactly those; no attention is needed.
 *   d_tok [rows][pmax] int32, d_hid [rows][pmax][H] in hid_dtype.
 * Errors: BAD_ARG (rows > max_rows, a count < 0 or > pmax), KV_CAPACITY.
 */
mtp_status mtp_flush(mtp_t h, mtp_stream stream, int32_t rows, const int32_t* h_pairs,
                     int32_t pmax, const int32_t* d_tok, const void* d_hid, int32_t hid_dtype);

/*
 * mtp_draft — propose `depth` tokens per row with one head call per token.
 * The first call consumes h_pairs[r] >= 1 pairs of row r at slots len[r]..:
 * the first h_pairs[r]-1 are pending completed pairs (flushed in the same
 * pass), the last is the newest pair (token c_T, target hidden at T-1) and
 * yields the step-1 logits. Step k >= 2 consumes the step-(k-1) draft token
 * and the head's own pre-norm hidden h2 at the next slot.
 * Token selection per row: greedy rows take the argmax of the (penalised)
 * logits; sampled rows apply the transform chain (repetition penalty over the
 * window "last hist_w of d_hist[r] ++ drafts so far", temperature, top-k,
 * top-p, min-p) and draw by inverse CDF with d_u[r][k-1].
 *   d_tok [rows][pmax] int32, d_hid [rows][pmax][H] (hid_dtype)
 *   h_params [rows] (host), d_hist [rows][hist_w] int32 (oldest first, -1 empty)
 *   d_u [rows][depth] float in [0,1) (may be NULL if every row is greedy)
 *   d_draft [rows][depth] int32 out
 *   d_q [rows][depth][V] float out: the distribution each sampled draft was
 *       drawn from (rows that are greedy are left untouched); may be NULL if
 *       every row is greedy
 *   d_logits [rows][depth][V] float out (optional, NULL to skip)
 *   d_hidden [rows][depth][H] float out: h2 per step (optional)
 * After the call len[r] has advanced by h_pairs[r] + depth - 1; kv_rollback
 * keeps only the slots of the first call (len before + h_pairs[r]).
 * Errors: BAD_ARG, KV_CAPACITY.
 */
mtp_status mtp_draft(mtp_t h, mtp_stream stream, int32_t rows, int32_t depth,
                     const int32_t* h_pairs, int32_t pmax, const int32_t* d_tok,
                     const void* d_hid, int32_t hid_dtype, const mtp_sampling* h_params,
                     const int32_t* d_hist, int32_t hist_w, const float* d_u,
                     int32_t* d_draft, float* d_q, float* d_logits, float* d_hidden);

/*
 * spec_verify — rejection-sampling verify of a block of target logits
 * (Leviathan et al., Chen et al.; "greedy is a special case of sampled
 * decoding", Ollama MLX-runner commit log).
 * For each row r, with p_i the transformed target distribution of row i
 * (window "last hist_w of d_hist[r] ++ x_1..x_i"):
 *   for i = 1..d: accept x_i iff q_i(x_i) > 0 and u[i-1] < p_{i-1}(x_i)/q_i(x_i)
 *   first reject at i: y ~ norm(max(p_{i-1} - q_i, 0)) with u[d]
 *   all accepted:      y ~ p_d with u[d]          (the bonus token)
 * Greedy rows: accept iff x_i == argmax p_{i-1}; y = argmax of the stopping row.
 *   d_logits [rows][depth+1][vocab] float, d_draft [rows][depth] int32
 *   d_q [rows][depth][vocab] float (ignored for greedy rows; NULL if all greedy)
 *   h_params [rows] (host), d_hist [rows][hist_w], d_u [rows][depth+1]
 *   d_n_acc [rows] out, d_out_tok [rows][depth+1] out (accepted drafts, then y,
 *   then -1), d_stats [rows][depth+2] int32 accumulated (NULL to skip):
 *   [0] rounds, [1] rounds with a rejection (rollbacks), [1+i] accepts at i.
 *   h_out (optional, pinned host, [rows][depth+2]): n_acc then out_tok per row,
 *   the round's one device->host read. Page-locked memory the device can
 *   address (cudaHostAlloc / cudaMallocHost) is written by the verify kernel
 *   itself; other host memory gets a copy enqueued after the kernel. Either
 *   way it is complete once the stream has reached the end of this call. In
 *   device-addressable memory each row's n_acc is stored after its out_tok
 *   with release semantics at system scope: a host that set n_acc negative
 *   beforehand may poll it instead of waiting for the stream.
 *   d_status (optional, device int32): OR-ed with 1 << MTP_ERR_NONFINITE when
 *   a target logit the verify reads is NaN or infinite, and with
 *   1 << MTP_ERR_TIMEOUT when a bounded wait of the streaming path ran out
 *   (fail-closed errors, "Ollama qwen3_5 MTP loader and SelfDraft path",
 *   Facts). The caller clears it; NULL drops these reports.
 *   d_workspace: spec_verify_workspace_bytes(rows, depth, vocab) bytes (the
 *   transform descriptors, then the streaming path's accept flags and kept lists).
 * Calls with more (row, position) tasks than one wave of 8-CTA clusters holds,
 * whose sampled rows all cut to a top-k of at most 256 below the vocabulary,
 * take a streaming path: one CTA per task reads its target row once. Its
 * results are identical.
 * Errors: BAD_ARG.
 */
size_t spec_verify_workspace_bytes(int32_t rows, int32_t depth, int32_t vocab);

mtp_status spec_verify(mtp_stream stream, int32_t rows, int32_t depth, int32_t vocab,
                       const float* d_logits, const int32_t* d_draft, const float* d_q,
                       const mtp_sampling* h_params, const int32_t* d_hist, int32_t hist_w,
                       const float* d_u, int32_t* d_n_acc, int32_t* d_out_tok,
                       int32_t* d_stats, int32_t* h_out, int32_t* d_status, void* d_workspace);

/*
 * mtp_set_draft_head — which copy of the tied output head the drafter reads.
 * MTP_HEAD_BF16 (the default): the borrowed head itself. MTP_HEAD_FP8: an fp8
 * e4m3 copy with one fp32 scale per row (scale = max|row| / 448, codes =
 * e4m3(w / scale), round to nearest even, saturating), made from the borrowed
 * head by this call and owned by the handle (vocab * hidden bytes + vocab
 * floats, allocated on the first request). The draft logits become
 * scale[v] * sum_k e4m3(code[v,k]) * x[k]: half the head's bytes per draft
 * step, a draft-only change ("Ollama qwen3_5 MTP loader and SelfDraft path",
 * Facts: quantizing the draft's tied output head; the format is not stated
 * there). spec_verify is untouched: it reads the target's logits. Call again
 * after the borrowed head's contents change. bf16 heads only; asynchronous on
 * the stream. Errors: BAD_ARG, CONFIG_BOUNDS (fp32 head or hidden % 16),
 * CUDA.
 */
#define MTP_HEAD_BF16 0
#define MTP_HEAD_FP8 1
mtp_status mtp_set_draft_head(mtp_t h, mtp_stream stream, int32_t format);

/*
 * Draft-depth controller (host-side; "Ollama qwen3_5 MTP loader and SelfDraft
 * path", Facts: depth control; Ollama MLX-runner commit "choose the
 * speculative draft length to maximize throughput"). It picks the depth N in
 * [0, max_depth] that maximises committed(N) / cost(N): committed(N) =
 * 1 + sum_{i<=N} prod_{j<=i} a_j from per-position acceptance a_j (Laplace-
 * smoothed counts of rounds that reached position j), cost(N) = the mean
 * measured seconds of a round at depth N (an unmeasured depth extends its
 * measured neighbours linearly). N never exceeds one past the deepest position
 * with data. Every 4th round it returns one past its choice (a probe); while
 * the choice is plain decode each probe doubles that interval, up to 512
 * rounds. Before any other choice it runs one round of plain decode (depth 0)
 * to measure the base cost.
 * State persists for the object's lifetime. No GPU work; not thread-safe.
 *   mtp_depth_ctl_next: depth to draft this round (0 = plain decode).
 *   mtp_depth_ctl_observe: feed back the round actually run (depth, accepted
 *     drafts n_acc <= depth, wall-clock seconds > 0); BAD_ARG otherwise.
 *   mtp_depth_ctl_state: optional host outputs a[max_depth] (acceptance
 *     estimates), cost[max_depth+1] (seconds per round), the probe interval.
 */
typedef struct mtp_depth_ctl* mtp_depth_ctl_t;
mtp_status mtp_depth_ctl_create(int32_t max_depth, mtp_depth_ctl_t* out);
void mtp_depth_ctl_free(mtp_depth_ctl_t c);
int32_t mtp_depth_ctl_next(mtp_depth_ctl_t c);
mtp_status mtp_depth_ctl_observe(mtp_depth_ctl_t c, int32_t depth, int32_t n_acc, double round_seconds);
mtp_status mtp_depth_ctl_state(mtp_depth_ctl_t c, double* h_accept, double* h_cost, int32_t* h_interval);

/*
 * spec_verify_noalloc — spec_verify without a caller-provided workspace, for
 * callers that cannot allocate device memory (a host whose own pool owns all
 * device memory, or code running where a cudaMalloc would stall the device or
 * is forbidden). The pages have no counterpart; it exists for such hosts.
 * Same arguments and results as spec_verify minus d_workspace (d_status
 * included). The scratch
 * (one 32-byte descriptor per verified row and position) is a fixed array
 * inside the library, 1088 descriptors (34,816 bytes) per device, held for
 * the life of the process: rows * (depth + 1) above 1088 returns
 * MTP_ERR_BAD_ARG. The first call on a device, with that device current, looks
 * up the array's address; make it before capturing a stream into a graph.
 * Every call shares the array, so calls that can run at the same time on the
 * GPU (unordered streams) race on it. Allocates nothing.
 */
mtp_status spec_verify_noalloc(mtp_stream stream, int32_t rows, int32_t depth, int32_t vocab,
                               const float* d_logits, const int32_t* d_draft, const float* d_q,
                               const mtp_sampling* h_params, const int32_t* d_hist, int32_t hist_w,
                               const float* d_u, int32_t* d_n_acc, int32_t* d_out_tok,
                               int32_t* d_stats, int32_t* h_out, int32_t* d_status);

/*
 * kv_rollback — drop speculative cache slots after a verify.
 * Draft KV: row r keeps only the slots of the last mtp_draft's first head call
 * (its length becomes the length before that call + h_pairs[r]); with
 * zero_tail the dropped slots are zeroed. Target KV (optional): each
 * d_target_len[r] is trimmed by block - (d_n_acc[r] + 1), block = depth + 1
 * verified positions: the positions past the accepted drafts and the one
 * committed correction or bonus token are dropped ("support the qwen3_5_mtp
 * drafter" issue, comment on qualifying the qwen3_5 path). Rows never drafted
 * are left as they are.
 * Errors: BAD_ARG.
 */
mtp_status kv_rollback(mtp_t h, mtp_stream stream, int32_t rows, const int32_t* d_n_acc,
                       int32_t* d_target_len, int32_t depth, int32_t zero_tail);

/*
 * ------------------------------------------------ paged 4-bit KV cache
 *
 * A cache for the model that verifies the drafts: it appends a block of
 * positions per row and round, is trimmed by the round's device-side counts,
 * and is read by every query of the block. Pages are planned on the GPU from
 * device-side lengths, so a round needs no host read before its next one.
 *
 * Layout. K and V are two arrays [n_pages][n_kv][page][kv_q4_row_bytes(dh)] of
 * bytes, page a multiple of 16 slots, dh in {64, 128, 256}. A row holds one
 * slot of one head: dh/2 bytes of codes (element 2i in the low half of byte i,
 * 2i+1 in the high half), then dh/16 bytes of scales. A code is e2m1 (sign,
 * then 0, .5, 1, 1.5, 2, 3, 4, 6), a scale e4m3 for 16 elements:
 *   element = e2m1(code) * e4m3(scale of its 16) * 2^exp[head]
 * with an optional exponent per head, which puts the head's range into the
 * scales' (2^-9 to 448). Slot s is slot s % page of page s / page.
 */
typedef struct {
  void* k;               /* device, 16-byte aligned */
  void* v;
  const int32_t* k_exp;  /* device [n_kv], in [-64, 64]; NULL = 0 */
  const int32_t* v_exp;
  int32_t n_kv, head_dim, page, n_pages; /* n_pages * page < 2^31 */
} kv_q4_cache;

/* Bytes of one slot of one head, dh/2 + dh/16; 0 if head_dim is not supported. */
size_t kv_q4_row_bytes(int32_t head_dim);

/*
 * kv_page_plan — block tables and slot maps from the rows' lengths.
 * Row r's pages cover d_cover[r] positions; the caller keeps the first
 * d_keep[r] <= d_cover[r] of them (the rest were rejected) and appends
 * d_new[r] >= 0. With held = ceil(cover / page) and
 * want = ceil((keep + new) / page), the row gives held - want pages back or
 * takes want - held more.
 *   d_table [rows][max_pages] in/out: the pages of row r are its first
 *       ceil(cover / page) entries; entries past them carry no meaning.
 *   d_free [n_pages] in/out: the free pages, a stack of
 *       n_free = n_pages - sum_r held entries (every page is a row's or free).
 *   d_cover_out [rows] out: keep + new, the d_cover of the next call and the
 *       cache length that kv_q4_attend takes; d_cover (held to the table's
 *       positions) where the row is refused.
 *   d_start [rows + 1] out: the rows' appended positions are packed, row r's at
 *       [start[r], start[r + 1]).
 *   d_slot, d_pos [max_tokens] out: slot and position of every packed position;
 *       -1 past the last one, and d_slot -1 for a refused row.
 * No output may overlap d_cover, d_keep or d_new, which are read until the end.
 * Order: pages given back go onto the stack from the last row's last page to
 * the first row's first, then pages are taken off it from the first row on, so
 * a plan that undoes another leaves the stack as it was. The lengths are inputs
 * only and no entry that is read is written: a call repeated on the same
 * lengths gives the same result.
 * A row is refused (its pages stay) with 1 << MTP_ERR_KV_CAPACITY in d_status
 * when the stack runs out before it (in row order) or it would need more than
 * max_pages, and with 1 << MTP_ERR_BAD_ARG when its lengths are invalid, its
 * positions pass max_tokens; d_slot is -1 (and BAD_ARG set) also where an entry
 * of the table or of the stack is no page. d_status may be NULL.
 * Errors: BAD_ARG (rows outside 1..4096, page not a multiple of 16,
 * rows * max_pages or n_pages * page of 2^31 and more, a null pointer, an output
 * over a length array).
 */
mtp_status kv_page_plan(mtp_stream stream, int32_t rows, int32_t page, int32_t max_pages, int32_t n_pages,
                        int32_t max_tokens, const int32_t* d_cover, const int32_t* d_keep, const int32_t* d_new,
                        int32_t* d_table, int32_t* d_free, int32_t* d_cover_out, int32_t* d_start, int32_t* d_slot,
                        int32_t* d_pos, int32_t* d_status);

/*
 * kv_q4_append — round K and V rows to 4 bits and write them to their slots.
 *   d_k, d_v: element (t, head, i) at t * tok_stride + head * head_stride + i,
 *       strides in elements (a slice of a fused q/k/v projection will do)
 *   d_slot [tokens]: kv_page_plan's; -1 skips the position, any other value
 *       outside [0, n_pages * page) skips it and sets 1 << MTP_ERR_BAD_ARG in
 *       d_status. Two positions with the same slot leave bytes of both.
 * Rounding, per 16 elements y = x * 2^-exp: scale = e4m3(max|y| / 6) (fp32
 * quotient, to nearest even, at most 448), code = the e2m1 value nearest to
 * |y| / scale (exact, the even code when two are as near, 6 beyond 6); a zero
 * scale gives zero codes. 16 elements with a NaN or an infinity among them are
 * stored as NaN (scale 0x7F) and set 1 << MTP_ERR_NONFINITE.
 * kv_q4_read — the values of slots, [tokens][n_kv][head_dim] contiguous in
 * dtype, d_k and d_v 16-byte aligned; zeros where d_slot skips. Errors of both:
 * BAD_ARG.
 */
mtp_status kv_q4_append(mtp_stream stream, const kv_q4_cache* cache, int32_t tokens, const void* d_k,
                        int64_t k_tok_stride, int64_t k_head_stride, const void* d_v, int64_t v_tok_stride,
                        int64_t v_head_stride, int32_t dtype, const int32_t* d_slot, int32_t* d_status);
mtp_status kv_q4_read(mtp_stream stream, const kv_q4_cache* cache, int32_t tokens, const int32_t* d_slot, void* d_k,
                      void* d_v, int32_t dtype, int32_t* d_status);

/*
 * kv_q4_attend — attention of each row's newest positions over its pages.
 * Row r has queries [start[r], start[r + 1]) of the packed d_q and
 * L = d_len[r] cached positions, its own among them: its i-th query stands at
 * position L - n + i (n its query count) and sees the positions up to its own,
 * with window > 0 only the last `window` of those. Per query head (n_q / n_kv
 * of them share a KV head):
 *   s_j = scale * q . k_j,  out = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j)
 * A query that sees nothing gets zeros and lse = -inf. A NaN in a K row that a
 * query sees makes its outputs on that head NaN, one in V its 16 dimensions;
 * positions out of sight may hold anything. Rows of d_out and d_lse outside
 * [start[0], start[rows]) are not written.
 *   d_q: element (t, head, i) at t * tok_stride + head * head_stride + i
 *   d_out [tokens][n_q][head_dim] contiguous in dtype; d_lse [tokens][n_q] float
 *       (optional)
 *   d_table [rows][max_pages], d_start [rows + 1], d_len [rows]: kv_page_plan's
 *   max_q: the most queries of a row, as the caller knows it; it chooses the
 *       kernel's shape. Rows that have more are still computed.
 *   d_workspace: kv_q4_attend_workspace_bytes(...) bytes, 16-byte aligned.
 * Scores and sums are fp32. q enters as f16 after a power-of-two scaling per
 * query and head (exact for bf16 but for elements 2^-30 below the largest);
 * fp32 q as two f16 parts (22 bits). The softmax weights are f16 (11 bits;
 * fp32 q: two parts, 22 bits) down to 2^-21 of the largest, below that in steps
 * of 2^-31 of it.
 * The tensor core's sums drop the bits past fp32's: over the 1024 (fp32 q) or
 * 16,384 positions at most that it sums up at a time, 4e-6 or 7e-5 of the sum.
 * A page entry outside [0, n_pages) sets 1 << MTP_ERR_BAD_ARG in d_status and
 * its positions are not read; a bounded wait that ran out sets
 * 1 << MTP_ERR_TIMEOUT. Errors: BAD_ARG (rows outside 1..4096, n_q above 1024 or
 * no multiple of n_kv, tokens * n_q or max_pages * page of 2^31 and more, d_q not
 * aligned to its type, d_out or d_workspace not to 16 bytes, a null pointer).
 */
size_t kv_q4_attend_workspace_bytes(const kv_q4_cache* cache, int32_t n_q, int32_t max_q, int32_t dtype);
mtp_status kv_q4_attend(mtp_stream stream, const kv_q4_cache* cache, int32_t rows, int32_t n_q, int32_t tokens,
                        const void* d_q, int64_t tok_stride, int64_t head_stride, int32_t dtype,
                        const int32_t* d_table, int32_t max_pages, const int32_t* d_start, const int32_t* d_len,
                        int32_t max_q, float scale, int32_t window, void* d_out, float* d_lse, int32_t* d_status,
                        void* d_workspace);

/*
 * ------------------------------------------------ trees of drafts, prompts
 *
 * A round that drafts a tree verifies all of its nodes at once: they are
 * appended to the cache like a block of positions (kv_page_plan with
 * d_new = the node counts, kv_q4_append_rope with the nodes' positions), each
 * attends the row's committed prefix and its own ancestors, and of the path
 * that the target confirms the rows are moved together behind the prefix.
 * Node 0 of a row is the last committed token; a node's parent comes before it.
 */
#define MTP_TREE_MAX 128  /* nodes of a row */
#define MTP_MAX_CACHES 64 /* layers of one kv_q4_tree_commit */
#define MTP_ROPE_MAX 128  /* rotated pairs */

/* Frequencies of a rotation by position, in turns per position (units of
 * 2^-64), caller-owned host memory. */
typedef struct {
  int32_t rot_dim; /* the first rot_dim dimensions are rotated: pairs (i, i + rot_dim / 2) */
  uint64_t turn[MTP_ROPE_MAX];
} mtp_rope;

/* Fill *out: pair i turns by theta^(-2i/rot_dim) radians a position, or by
 * h_freq[i] where h_freq is given (rot_dim / 2 of them, finite; scaled
 * rotations). Host only. Errors: BAD_ARG (rot_dim odd or outside 0..256, theta
 * not positive or not finite). */
mtp_status mtp_rope_init(int32_t rot_dim, double theta, const double* h_freq, mtp_rope* out);

/*
 * kv_q4_append_rope — norms, rotation and append of a projection's rows.
 * Queries and keys: y = x / sqrt(mean x^2 + eps) * w over the head (without
 * d_q_norm or d_k_norm: y = x), then the pairs (y_i, y_{i + rot_dim / 2}) turned
 * by d_pos * frequency i, a frequency held to 2^-51 of itself. Queries
 * go to d_q_out, keys to the cache and, unless it is NULL, to d_k_out; values go
 * to the cache as they are. The cache's 4 bits are rounded (as by kv_q4_append)
 * from keys that are good to 2^-30, not from d_k_out.
 *   d_q, d_k, d_v: element (t, head, i) at t * tok_stride + head * head_stride + i,
 *       strides in elements (slices of a fused projection will do), dtype each
 *   d_q_norm, d_k_norm [head_dim] float, 16-byte aligned, applied as they are
 *       (with the +1 of a raw-HF checkpoint added); NULL = no norm
 *   d_pos, d_slot [tokens]: a position below 0 is padding: its rows of the outputs
 *       are zeros and nothing is appended. d_slot -1 appends nothing; any other
 *       slot outside the cache, or a slot beside a position below 0, sets
 *       1 << MTP_ERR_BAD_ARG in d_status and appends nothing. Two positions with
 *       the same slot leave bytes of both.
 *   d_q_out [tokens][n_q][head_dim], d_k_out [tokens][n_kv][head_dim] (optional)
 *       contiguous in dtype, 16-byte aligned. Each may be its own input where that
 *       is contiguous; any other overlap is refused.
 * 16 elements of K or V with a NaN or an infinity are stored as NaN and set
 * 1 << MTP_ERR_NONFINITE. Squares are summed in fp32. Errors: BAD_ARG (n_q
 * outside 1..1024, rot_dim above head_dim, eps negative or not finite,
 * tokens * (n_q + 2 n_kv) near 2^31, an input not aligned to its type, a null
 * pointer, an overlap).
 */
mtp_status kv_q4_append_rope(mtp_stream stream, const kv_q4_cache* cache, int32_t tokens, int32_t n_q,
                             const void* d_q, int64_t q_tok_stride, int64_t q_head_stride, const void* d_k,
                             int64_t k_tok_stride, int64_t k_head_stride, const void* d_v, int64_t v_tok_stride,
                             int64_t v_head_stride, int32_t dtype, const float* d_q_norm, const float* d_k_norm,
                             float eps, const mtp_rope* rope, const int32_t* d_pos, const int32_t* d_slot,
                             void* d_q_out, void* d_k_out, int32_t* d_status);

/*
 * kv_tree_plan — positions and ancestor masks of trees, once for all layers.
 * Row r has n = start[r + 1] - start[r] <= MTP_TREE_MAX nodes, which stand at
 * the cached positions len[r] - n .. len[r] - 1.
 *   d_parent [tokens]: the parent's number within the row, below the node's own;
 *       -1 where the node hangs on the prefix
 *   d_pos [tokens] out: len - n + depth (for the rotation, and for a window)
 *   d_mask [tokens][MTP_TREE_MAX / 32] out, 16-byte aligned: bit a of a node's
 *       mask is node a, its ancestors and itself; with window > 0 only the last
 *       `window` of them
 * A node with an invalid parent and its descendants get position -1, an empty
 * mask and 1 << MTP_ERR_BAD_ARG in d_status, as do all nodes of a row with too
 * many of them or with len < n. Entries outside [start[0], start[rows]) are not
 * written. Errors: BAD_ARG (rows outside 1..4096, a null or unaligned pointer,
 * an output over an input).
 */
mtp_status kv_tree_plan(mtp_stream stream, int32_t rows, int32_t tokens, const int32_t* d_parent,
                        const int32_t* d_start, const int32_t* d_len, int32_t window, int32_t* d_pos, int32_t* d_mask,
                        int32_t* d_status);

/*
 * kv_q4_attend_tree — kv_q4_attend for the nodes of trees: query i of row r sees
 * the prefix [0, len - n), with window > 0 from position d_pos - window + 1 on,
 * and the nodes whose bits its mask has (kv_tree_plan's, or any other set;
 * bits from n on mean nothing). Arguments, arithmetic and workspace
 * (kv_q4_attend_workspace_bytes) as there.
 *   d_mask [tokens][MTP_TREE_MAX / 32], 16-byte aligned
 *   d_pos [tokens]: needed with window > 0 only; held to [len - n, len - 1]
 * A row of more than MTP_TREE_MAX nodes sets 1 << MTP_ERR_BAD_ARG in d_status,
 * and its outputs are not written. Errors: kv_q4_attend's, and BAD_ARG for max_q
 * above MTP_TREE_MAX, d_mask null or unaligned, a window without d_pos.
 */
mtp_status kv_q4_attend_tree(mtp_stream stream, const kv_q4_cache* cache, int32_t rows, int32_t n_q, int32_t tokens,
                             const void* d_q, int64_t tok_stride, int64_t head_stride, int32_t dtype,
                             const int32_t* d_table, int32_t max_pages, const int32_t* d_start, const int32_t* d_len,
                             const int32_t* d_mask, const int32_t* d_pos, int32_t max_q, float scale, int32_t window,
                             void* d_out, float* d_lse, int32_t* d_status, void* d_workspace);

/*
 * kv_q4_tree_commit — the confirmed path of each row's tree, moved together in
 * every layer's cache. The path starts at node 0; behind a node follows its
 * lowest-numbered child whose token is the target's choice after that node, as
 * long as there is one and the path is shorter than max_path. With a choice
 * drawn from the target's distribution at every node the committed tokens
 * follow that distribution; with its argmax the verify is greedy.
 *   caches [n_caches] (host, at most MTP_MAX_CACHES): the layers, which share the
 *       block table and have one shape; two that overlap are refused. 0 = the
 *       path only (d_table may then be NULL)
 *   d_parent, d_tok, d_choice [tokens]: per node its parent (kv_tree_plan), its
 *       token, and the token that the target puts behind it
 *   d_n_acc [rows] out: accepted drafts, path length - 1 (0 for a row without nodes)
 *   d_out_tok [rows][max_path] out: the committed tokens, d_choice along the
 *       path (the accepted drafts, then the target's own), then -1
 *   d_path [rows][max_path] out (optional): the path's nodes, then -1
 *   d_keep [rows] out: len - n + path length, kv_page_plan's d_keep
 * The cached rows of path node k go to place k, position len - n + k; no other
 * row's table may name those pages. Moves whose table entry is no page are
 * left out and set 1 << MTP_ERR_BAD_ARG in d_status, as does a parent that is
 * not below its node (which then is nobody's child); rows with too many nodes,
 * or len outside [n, max_pages * page], also set it, move nothing, have no
 * path and keep len. A second call on the same tree would move rows that have
 * moved. Errors: BAD_ARG (rows outside 1..4096, max_path outside
 * 1..MTP_TREE_MAX, a null pointer, overlapping outputs).
 */
mtp_status kv_q4_tree_commit(mtp_stream stream, const kv_q4_cache* caches, int32_t n_caches, int32_t rows,
                             int32_t tokens, const int32_t* d_table, int32_t max_pages, const int32_t* d_start,
                             const int32_t* d_len, const int32_t* d_parent, const int32_t* d_tok,
                             const int32_t* d_choice, int32_t max_path, int32_t* d_n_acc, int32_t* d_out_tok,
                             int32_t* d_keep, int32_t* d_path, int32_t* d_status);

/*
 * kv_attend_prompt — causal attention of whole prompts over their own keys and
 * values, unrounded (the cache then serves what follows them). Row r holds
 * positions [start[r], start[r + 1]) of the packed tokens; its i-th query sees
 * the positions up to its own, with window > 0 only the last `window` of them:
 *   s_ij = scale * q_i . k_j,  out_i = sum_j softmax(s_i)_j v_j,  lse_i = log sum_j exp(s_ij)
 *   d_q, d_k, d_v: element (t, head, i) at t * tok_stride + head * head_stride + i
 *       (slices of a fused projection will do); bases and strides multiples of
 *       16 bytes, strides above 0 and below 2^40 bytes
 *   d_out [tokens][n_q][head_dim] contiguous in dtype, 16-byte aligned;
 *   d_lse [tokens][n_q] float (optional)
 *   max_len: the most positions of a row, as the caller knows it, at least 1. A hint:
 *       rows that have more are still computed. The launch's shape does not need it now
 *   d_workspace: kv_attend_prompt_workspace_bytes(tokens, rows), 16-byte aligned. The
 *       kernels do not write it now, so calls may share one
 * Positions that a query does not see may hold anything; what it does see and is
 * NaN or infinite shows in its outputs. Rows of d_out and d_lse outside
 * [start[0], start[rows]) are not written. Scores, sums and outputs are
 * accumulated in fp32; with bf16 the softmax weights are rounded to bf16 for the
 * product with V (off by at most 2^-8 of each). A bounded wait that ran out sets
 * 1 << MTP_ERR_TIMEOUT in d_status. Errors: BAD_ARG (rows outside 1..4096, n_q
 * outside 1..1024 or no multiple of n_kv, head_dim not 64, 128 or 256, tokens *
 * n_q of 2^31 and more, a null or unaligned pointer, an output over an input).
 */
size_t kv_attend_prompt_workspace_bytes(int32_t tokens, int32_t rows);
mtp_status kv_attend_prompt(mtp_stream stream, int32_t rows, int32_t n_q, int32_t n_kv, int32_t head_dim, int32_t tokens,
                         const void* d_q, int64_t q_tok_stride, int64_t q_head_stride, const void* d_k,
                         int64_t k_tok_stride, int64_t k_head_stride, const void* d_v, int64_t v_tok_stride,
                         int64_t v_head_stride, int32_t dtype, const int32_t* d_start, int32_t max_len, float scale,
                         int32_t window, void* d_out, float* d_lse, int32_t* d_status, void* d_workspace);

/*
 * spec_logprobs — log probabilities of given tokens under raw logits (no
 * transforms), with their ranks, the entropy and the likeliest alternatives.
 *   d_logits [n] rows of vocab logits (dtype), row_stride elements apart: for
 *       a verified block, spec_verify's d_logits as rows * (depth + 1) rows
 *   d_tok [n]: the given tokens; -1 (d_out_tok past a row's committed tokens)
 *       gives log probability 0 and rank -1, any other id outside [0, vocab)
 *       the same with 1 << MTP_ERR_BAD_ARG in d_status
 *   d_logprob [n] out: x_t - log sum_j exp(x_j)
 *   d_rank [n] out (optional): tokens before t in the order (logit descending,
 *       id ascending)
 *   d_entropy [n] out (optional): -sum_j p_j log p_j, in nats
 *   d_top_id, d_top_lp [n][top] out: the first `top` (0..64) tokens of that
 *       order and their log probabilities; id -1 and -inf past the last token
 *       with p > 0 possible (logit above -inf)
 * Logits of -inf are masked tokens; a row with nothing else gives -inf (0 for
 * entropy). A NaN or +inf sets 1 << MTP_ERR_NONFINITE; the row's outputs then
 * carry no meaning, ids stay in range. d_workspace:
 * spec_logprobs_workspace_bytes(n, vocab, top) bytes, 16-byte aligned. A bounded
 * wait that ran out sets 1 << MTP_ERR_TIMEOUT. Errors: BAD_ARG (n above 65535,
 * vocab outside 1..2^20, top above 64, a row_stride below vocab, d_logits not
 * aligned to its type, a null pointer).
 */
size_t spec_logprobs_workspace_bytes(int32_t n, int32_t vocab, int32_t top);
mtp_status spec_logprobs(mtp_stream stream, int32_t n, int32_t vocab, const void* d_logits, int64_t row_stride,
                         int32_t dtype, const int32_t* d_tok, int32_t top, float* d_logprob, int32_t* d_rank,
                         float* d_entropy, int32_t* d_top_id, float* d_top_lp, int32_t* d_status, void* d_workspace);

/* Test hook of the streaming verify's bounded waits: the next spec_verify
 * call that takes the streaming path leaves ring stage `stage` of every task
 * unfilled (a copy that never lands) and gives each wait `wait_polls` polls,
 * so its waits run out; it then reports MTP_ERR_TIMEOUT in d_status, writes
 * in-range outputs and leaves the context usable. One-shot, process-wide, not
 * for production use. Errors: BAD_ARG (stage < 0 or wait_polls < 1). */
mtp_status mtp_test_verify_stall(int32_t stage, int32_t wait_polls);

/* Number of kernels this library has launched in the process so far. */
int64_t mtp_kernel_launches(void);

/* Timing hook for the benchmark: kernels of the kinds selected by `mask`
 * (bit i = kind i, -1 = all, 0 = off) are bracketed by CUDA events on the
 * launching stream; mtp_profile_read synchronises those events and returns,
 * per kernel kind, the summed milliseconds and the launch count since the
 * last read. Kinds are listed by mtp_profile_kind_name(i) for
 * i < mtp_profile_kinds(). */
mtp_status mtp_profile_enable(mtp_t h, int32_t mask);
int32_t mtp_profile_kinds(void);
const char* mtp_profile_kind_name(int32_t kind);
mtp_status mtp_profile_read(mtp_t h, float* h_ms, int32_t* h_launches);

#ifdef __cplusplus
}
#endif
#endif /* MTP_H */
