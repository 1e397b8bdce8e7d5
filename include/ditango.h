/*
 * ditango.h -- C ABI of the partitioned-attention hot path with selective
 * attention-state reuse, for NVIDIA B200 (sm_100a).
 *
 * What it computes (sources by page title and section):
 *  - "DiTango: Cost-Effective Parallel Diffusion Generation with Selective
 *    Attention State Reuse", technical summary:
 *      Metodologia: the token sequence is split into P context partitions and
 *        attention is computed per (query partition i, KV partition j) pair;
 *        near partitions contribute most (spatial locality).
 *      1. Anchor-Guided Selection Planner: per pair, recompute ("fresh") or
 *        reuse the previous denoising step's attention state, guided by the
 *        partition's importance w; anchor steps recompute everything;
 *        "Strategia per Gruppi": decisions per group of adjacent partitions.
 *      2. State-Centric Parallel Runtime, "Composizione dello Stato": an
 *        attention state is (output, log-sum-exp); states are cached instead
 *        of raw K/V and compose associatively and commutatively;
 *        "Calcolo dello Stato di Gruppo": one state per group;
 *        "Composizione Dinamica dei Gruppi": cached states are merged
 *        recursively into coarser groups to shrink the cache.
 *  - "Efficient-vDiT: Efficient Video Diffusion Transformers With Attention
 *    Tile", abstract: a frame-tile sparse mask whose cost grows linearly
 *    with the number of frames.
 *
 * Conventions shared by every entry point
 *  - Every buffer is allocated by the caller.  "dev" marks device pointers,
 *    "host" host pointers.  The library keeps no pointer after a call
 *    returns and allocates no device memory.
 *  - Every device-side call is asynchronous on `stream` (a cudaStream_t;
 *    NULL is the legacy default stream) and never synchronises the host.
 *  - Arguments are validated before anything is launched: a bad argument
 *    returns DITANGO_ERR_INVALID, a valid but unsupported shape returns
 *    DITANGO_ERR_UNSUPPORTED, a failed launch returns DITANGO_ERR_CUDA.
 *    Device-side failures (a pipeline wait that exceeded its time limit) are
 *    written as a status code into `dev_status` where a call takes one.
 *  - Token order is frame-major; partitions are contiguous token ranges.
 *  - Units: the KV side may be grouped into G runs of adjacent partitions
 *    (ditango_geom.G, group_off).  The unit of planning and of storage is
 *    (query partition i, KV group c); its state is attention of partition
 *    i's rows against every allowed key of the group's partitions.  Without
 *    groups (G = 0) each partition is its own group, G = P and a unit is the
 *    pair (i, j).  A unit is active when some pair (i, j), j in c, is.
 *  - State layout ("state buffer"): O is [n_idx][B*H][Lmax][d], float32 or
 *    (state_bf16 = 1, a compressed cache) bfloat16 bit patterns, and lse is
 *    float32 [n_idx][B*H][Lmax], where Lmax = max partition length
 *    (ditango_state_rows) and the leading index is either the slot of an
 *    active unit (row-major rank of the active units, see ditango_slot_table)
 *    or the position of a unit in the fresh list.  Row r of unit (i, c)
 *    holds query token part_off[i] + r; rows r >= L_i are never written.
 *    O is normalised (sum_k softmax_k v_k) and lse is the natural
 *    log-sum-exp of the scaled logits.
 *  - Plan: int8 [P * G], entry i * G + c; codes 0 skip (masked unit),
 *    1 fresh, 2 reuse.
 */
#ifndef DITANGO_H
#define DITANGO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DITANGO_OK = 0,
  DITANGO_ERR_INVALID = 1,      /* bad argument (null, negative, inconsistent) */
  DITANGO_ERR_UNSUPPORTED = 2,  /* valid but outside what the kernels handle */
  DITANGO_ERR_CUDA = 3,         /* a CUDA runtime/driver call failed */
  DITANGO_ERR_TIMEOUT = 4,      /* device: a pipeline wait exceeded its limit */
  DITANGO_ERR_BOUNDS = 5        /* device, checked builds: a device-resident input (a count,
                                   a fresh list, a plan code) out of range */
} ditango_status;

enum { DITANGO_PLAN_SKIP = 0, DITANGO_PLAN_FRESH = 1, DITANGO_PLAN_REUSE = 2 };

typedef void *ditango_stream; /* cudaStream_t */

/* Geometry of one attention call; host struct, read during the call only.
 *   B, H     batch and heads; N tokens; d head dim in {64, 96, 128}.
 *   P        partitions, 1 <= P <= 64; part_off host int32 [P+1],
 *            part_off[0] = 0 < part_off[1] < ... < part_off[P] = N.
 *   F        frames of the frame-tile mask, 0 = no mask (all pairs active);
 *            else 1 <= F <= 64, frame_off host int32 [F+1] (same rules as
 *            part_off) and frame_mask host uint8 [F*F], row = query frame,
 *            nonzero = the query frame may attend the key frame.  The mask
 *            applies token by token; pair (i, j) is active when some token of
 *            partition i may attend some token of partition j.  Partitions may
 *            straddle frames: single logits are then masked inside the pair,
 *            and a row that may attend none of a unit's keys gets lse = -inf,
 *            O = 0 for that unit.
 *   q/k/v_strides  element strides of the (b, h, n) dimensions of the bf16
 *            Q, K, V tensors; the d dimension is contiguous.  Strides times 2
 *            bytes must be multiples of 16 and the base pointers 16-byte
 *            aligned (TMA).  The stride of a dimension of size 1 is ignored.
 *   G        KV groups; 0 = one group per partition (group_off ignored).
 *            Else 1 <= G <= P and group_off host int32 [G+1] holds partition
 *            indices, group_off[0] = 0 < ... < group_off[G] = P: group c is
 *            partitions group_off[c] .. group_off[c+1]-1. */
typedef struct {
  int32_t B, H, N, d;
  int32_t P, F;
  const int32_t *part_off;
  const int32_t *frame_off;
  const uint8_t *frame_mask;
  int64_t q_strides[3];
  int64_t k_strides[3];
  int64_t v_strides[3];
  int32_t G;
  const int32_t *group_off;
} ditango_geom;

/* Library version (major * 10000 + minor * 100 + patch). */
int32_t ditango_version(void);

/* Static string for a status code. */
const char *ditango_status_string(int32_t status);

/* Validate a geometry without launching anything. */
ditango_status ditango_check_geom(const ditango_geom *g);

/* Number of active units (= slots): units (i, c) with a pair (i, j), j in c,
 * whose tokens the frame mask lets attend each other (all P*G when F = 0).
 * Returns -1 on a bad geometry. */
int64_t ditango_num_active(const ditango_geom *g);

/* Lmax, rows per (index, b*h) block of a state buffer. -1 on a bad geometry. */
int64_t ditango_state_rows(const ditango_geom *g);

/* Host helper: slot_out host int32 [P*G] receives the slot of each unit,
 * -1 for masked units (row-major rank of the active units). */
ditango_status ditango_slot_table(const ditango_geom *g, int32_t *slot_out);

/* Bytes of device scratch ditango_plan needs; also the size of the mass
 * partials ditango_merge can emit (the same layout: float32 block sums
 * [P][B*H][ceil(Lmax / 128)][G + 1], see ditango_merge). */
size_t ditango_plan_workspace_size(const ditango_geom *g);

/* The same value under its shorter name. */
size_t ditango_workspace_size(const ditango_geom *g);

/* Plan: per unit, fresh or reuse (DiTango, 1. Anchor-Guided Selection
 * Planner and its group strategy; spatial locality from Metodologia).
 *   cache_lse    dev float32 state-buffer lse indexed by slot (the previous
 *                step's cached states); may be NULL when anchor != 0.
 *   cache_valid  dev uint8 [slots] (nonzero = slot holds a state) or NULL
 *                (all valid).  An invalid slot is forced fresh and holds no
 *                mass.
 *   band_k       the band: unit (i, c) is always fresh when some active
 *                pair (i, j), j in c, has |i - j| <= band_k.
 *   budget       fraction of active units to recompute: the fresh count is
 *                max(|band|, floor(budget * active + 1e-9)); the units added
 *                beyond the band are those of largest mass w, ties to the
 *                lower linear index i*G + c.
 *   anchor       nonzero: every active unit fresh (an anchor step).
 * w[i][c] = mean over (b, h, rows r of partition i) of
 *           exp(lse_ic[r]) / sum_{c' active, valid} exp(lse_ic'[r]),
 * computed in float32 with a fixed reduction order (deterministic).
 * Outputs (dev): plan int8 [P*G]; fresh_list int32 [slots] = linear indices
 * i*G + c of the fresh units in row-major order; counts int32 [2] = {fresh,
 * reuse}; score_out float32 [P*G] (w, 0 for masked units) or NULL.
 * workspace: dev, >= ditango_plan_workspace_size bytes. */
ditango_status ditango_plan(const ditango_geom *g, const float *cache_lse,
                            const uint8_t *cache_valid, int32_t band_k, double budget,
                            int32_t anchor, int8_t *plan, int32_t *fresh_list,
                            int32_t *counts, float *score_out, void *workspace,
                            size_t workspace_bytes, ditango_stream stream);

/* Plan from mass partials: ditango_plan with its first stage (the mass
 * score read from the cache) replaced by the block sums a ditango_merge
 * call emitted (its mass_partials argument) -- DiTango, "Anchor Steps":
 * the importance w is refreshed from the states just composed, without
 * reading the cache again.  The partials describe the cache as that merge
 * left it (every state it composed counts as valid); after anything else
 * has changed the cache (states invalidated or written by another call, a
 * composition), plan with ditango_plan instead.  The same selection,
 * outputs and determinism as ditango_plan; given the partials of a merge
 * whose composed states are the cache's valid states, the plan and scores
 * are bit-identical to ditango_plan's on that cache.
 *   mass_partials  dev, written by ditango_merge, mass_bytes >=
 *                  ditango_plan_workspace_size (else INVALID); the part of
 *                  the buffer past the block sums serves as scratch (the
 *                  per-unit means), so the block sums themselves are left
 *                  unchanged.
 *   cache_valid    as for ditango_plan (invalid slots are forced fresh). */
ditango_status ditango_plan_from_mass(const ditango_geom *g, float *mass_partials,
                                     size_t mass_bytes, const uint8_t *cache_valid,
                                     int32_t band_k, double budget, int8_t *plan,
                                     int32_t *fresh_list, int32_t *counts, float *score_out,
                                     ditango_stream stream);

/* Partial attention states of the fresh units (tcgen05 tensor cores, TMA).
 * For each fresh unit (i, c) = fresh_list[f], f < counts[0] (read on the
 * device), and each (b, h): S = Q_i K_c^T * scale over the keys K_c of the
 * active pairs of group c, O = softmax(S) V_c (normalised), lse =
 * logsumexp(S) -- the state of DiTango's "Composizione dello Stato" (one
 * pair, or a whole group: "Calcolo dello Stato di Gruppo").  bf16 inputs, fp32 accumulation and softmax;
 * the probabilities are rounded to bf16 for the P V product.
 *   Q, K, V      dev bf16 (uint16 bit patterns) with the geometry's strides.
 *   scale        logit scale; 0 means 1/sqrt(d).
 *   out_O/out_lse  dev state buffer; index = f (out_by_slot = 0) or the
 *                unit's slot (out_by_slot = 1, e.g. writing the cache in
 *                place).  Must hold counts[0] (resp. all slots) indices.
 *   state_bf16   nonzero: O is stored as bf16 (the normalised fp32 O rounded
 *                to nearest even); lse stays float32.  A compressed cache
 *                halves the cache memory and the merge's read traffic
 *                (DiTango, "Significato e Claim": cache memory is the
 *                method's limitation and cache compression its next step).
 *   out_valid    dev uint8 [slots] or NULL; with out_by_slot = 1 the written
 *                slots are set to 1.
 *   drift_rows   dev float32 [P][B*H][Lmax] or NULL (needs out_by_slot = 1):
 *                for each fresh local unit -- the unit of partition i that
 *                holds partition i, always in the band -- row r receives
 *                |lse_new - lse_old|, lse_old being the slot's lse before
 *                this call overwrites it (equal values, -inf included, give
 *                0): the local state's change that ditango_plan_error reads
 *                (DiTango, "Predizione Online").
 *   dev_status   dev int32 or NULL; set to DITANGO_ERR_TIMEOUT if a pipeline
 *                wait exceeded the limit (the kernel then stops cleanly).
 *   work_counter dev int32 [2], 8-byte aligned, or NULL.  With it, each CTA
 *                of the persistent kernel takes the next work item when it is
 *                ready for one (balanced whatever the items' sizes); without
 *                it, items are dealt in a fixed stride.  Zero it once when it
 *                is allocated: every launch leaves it at zero again.  Launches
 *                that may run at the same time (other streams, concurrent
 *                graph branches) must not share one.
 */
ditango_status ditango_attn_partial(const ditango_geom *g, const uint16_t *Q,
                                    const uint16_t *K, const uint16_t *V,
                                    const int32_t *fresh_list, const int32_t *counts,
                                    float scale, void *out_O, float *out_lse,
                                    int32_t out_by_slot, int32_t state_bf16,
                                    uint8_t *out_valid, float *drift_rows,
                                    int32_t *dev_status, int32_t *work_counter,
                                    ditango_stream stream);

/* Merge: the final output of every token is the log-sum-exp composition of
 * the states of its partition's active units (DiTango, "Composizione dello
 * Stato"): L = log sum_c exp(lse_c), O = sum_c exp(lse_c - L) O_c, with
 * fresh states read from part_O/part_lse (indexed by fresh-list position)
 * and reused ones from cache_O/cache_lse (indexed by slot).  part_O = NULL
 * means the fresh states were already written into the cache slots
 * (ditango_attn_partial with out_by_slot = 1).  The weights
 * exp(lse_c - L) of a row are computed in a fixed order (largest lse first
 * subtracted, a fixed summation tree), shared with ditango_plan's mass
 * score.
 *   plan          dev int8 [P*G] from ditango_plan.
 *   writeback     nonzero: also copy each fresh state into its cache slot
 *                 and mark cache_valid (ignored when part_O is NULL).
 *   state_bf16    format of every state buffer passed (see ditango_attn_partial).
 *   out           dev [B, H, N, d] (element strides out_strides for b, h, n;
 *                 NULL = contiguous), bf16 bits (out_is_fp32 = 0) or float32.
 *   out_lse       dev float32 [B, H, N] or NULL.
 *   mass_partials dev float32 of ditango_plan_workspace_size bytes, or NULL:
 *                 receives, per (query partition i, b*h, block of 128 rows),
 *                 every active unit's sum of its weights over the block's
 *                 rows (0 for a unit the plan skipped) -- the next step's
 *                 importance w before averaging (DiTango, "Anchor Steps":
 *                 refreshed from the states just composed); pass it to
 *                 ditango_plan_from_mass.  Column G is not written.
 * A token whose partition has no active pair gets O = 0, lse = -inf. */
ditango_status ditango_merge(const ditango_geom *g, const int8_t *plan,
                             const void *part_O, const float *part_lse,
                             void *cache_O, float *cache_lse, uint8_t *cache_valid,
                             int32_t writeback, int32_t state_bf16, void *out,
                             int32_t out_is_fp32, const int64_t *out_strides,
                             float *out_lse, float *mass_partials, ditango_stream stream);

/* Cache update: copy the fresh states (indexed by fresh position) into their
 * cache slots and mark them valid -- the write half of an anchor step
 * (DiTango, "Anchor Steps": everything is recomputed and the cache
 * refreshed). */
ditango_status ditango_cache_update(const ditango_geom *g, const int8_t *plan,
                                    const void *part_O, const float *part_lse,
                                    void *cache_O, float *cache_lse,
                                    uint8_t *cache_valid, int32_t state_bf16,
                                    ditango_stream stream);

/* Dynamic group composition (DiTango, "Composizione Dinamica dei Gruppi"):
 * merge the cached states of a fine grouping into the states of a coarser
 * one, with no recomputation: the coarse unit (i, C) gets the log-sum-exp
 * composition of the fine units (i, c), c inside C, that are active.
 *   fine, coarse  geometries identical except for G/group_off, and every
 *                 coarse group boundary a fine group boundary (else INVALID);
 *                 applied repeatedly (groups of 1 -> 2 -> 4 ...) the cache
 *                 halves at every level.
 *   fine_O/fine_lse/fine_valid      dev state buffer of the fine slots
 *                 (fine_valid may be NULL: all valid).
 *   coarse_O/coarse_lse/coarse_valid  dev state buffer of the coarse slots
 *                 (coarse_valid may be NULL); must not overlap the fine one.
 * A coarse slot is valid only if every fine slot it covers is; an invalid
 * one is marked 0 and its rows are not written.  Both buffers use the
 * state format state_bf16 (bf16 results are rounded to nearest even). */
ditango_status ditango_cache_compose(const ditango_geom *fine, const ditango_geom *coarse,
                                     const void *fine_O, const float *fine_lse,
                                     const uint8_t *fine_valid, void *coarse_O,
                                     float *coarse_lse, uint8_t *coarse_valid,
                                     int32_t state_bf16, ditango_stream stream);

/* Error-growth planner state (DiTango, 1. Anchor-Guided Selection Planner:
 * "Modellazione dell'Errore", "Anchor Steps", "Predizione Online").  Device
 * buffers owned by the caller, zeroed once before the first (anchor) step and
 * then carried from step to step by ditango_plan_error. */
typedef struct {
  float *w;                 /* dev float32 [P*G]: importance, refreshed after anchors */
  float *age;               /* dev float32 [slots]: local drift accumulated since each
                               cached state was computed */
  float *delta;             /* dev float32 [P]: last measured local drift (output) */
  uint8_t *local_ok;        /* dev uint8 [P]: the local unit held a state before the
                               last step's attention call */
  const float *drift_rows;  /* dev float32 [P][B*H][Lmax]: written by
                               ditango_attn_partial (drift_rows argument) */
} ditango_error_state;

/* Plan by predicted reuse error.  The same contract as ditango_plan (band,
 * invalid slots, budget, fresh list, counts, workspace) with the ranking
 * score replaced:
 *   delta_i = mean over (b, h, rows of partition i) of drift_rows, when
 *             local_ok[i] (else 0) -- the local state's change in the last
 *             step, standing in for the drift of the partition's remote
 *             states;
 *   age     = 0 for units the previous plan made fresh, age + delta_i for
 *             the units it reused;
 *   score   = w * (age + delta_i): the predicted error of reusing the unit
 *             at this step; the non-band units of largest score fill the
 *             budget (ties to the lower index i*G + c).
 *   plan     in: the previous step's plan (zeros before the first step);
 *            out: this step's plan.
 *   anchor   nonzero: every active unit fresh (an anchor step, "Anchor
 *            Steps"); w, age and delta are left alone.
 *   refresh_w  nonzero (the step after an anchor): w is recomputed from the
 *            cache as in ditango_plan and stored in es->w; otherwise es->w
 *            is used as held.
 *   score_out  dev float32 [P*G] or NULL: the score (0 for masked units).
 * Every call also records es->local_ok for the next step (whether the local
 * unit's slot is valid now, before this step's attention call). */
ditango_status ditango_plan_error(const ditango_geom *g, const float *cache_lse,
                                  const uint8_t *cache_valid, int32_t band_k, double budget,
                                  int32_t anchor, int32_t refresh_w,
                                  const ditango_error_state *es, int8_t *plan,
                                  int32_t *fresh_list, int32_t *counts, float *score_out,
                                  void *workspace, size_t workspace_bytes,
                                  ditango_stream stream);

/* Allocation-free variant of ditango_plan (no counterpart in the papers: it
 * exists for callers, not for the method).  For callers that cannot allocate
 * device memory -- code running inside an arena it does not own, a serving
 * process whose allocator is frozen after start-up, or a host that must not
 * call cudaMalloc between steps -- and so cannot provide ditango_plan's
 * workspace.  Same arguments, meaning and results as ditango_plan without
 * workspace/workspace_bytes; the scratch is a fixed 4 MiB device array inside
 * the library (held by every GPU that loads the library until the process
 * exits).  Returns DITANGO_ERR_UNSUPPORTED when ditango_plan_workspace_size
 * exceeds 4 MiB (anchor plans need no scratch and are never rejected).
 * Allocates nothing itself: no cudaMalloc, cudaFree or allocating library
 * call.  But the CUDA runtime loads the library's device code lazily by
 * default, so the first call on a device (in a context) is what makes the
 * driver load the module and reserve the 4 MiB array; that first load can
 * fail under memory pressure.  A caller whose allocator is frozen should
 * make one call per device at start-up (it must anyway come before any
 * stream capture), or run with CUDA_MODULE_LOADING=EAGER.
 * The array's device address is looked up with cudaGetSymbolAddress, with
 * the device current, on the first call in each context and cached with the
 * context's unique ID; after cudaDeviceReset (a new context) the next call
 * looks it up again.  Every call shares the one array per device and
 * overwrites all of the scratch it reads, so nothing carries over between
 * calls; but calls that overlap on the GPU (other streams, concurrent graph
 * branches) race on it -- order them. */
ditango_status ditango_plan_noalloc(const ditango_geom *g, const float *cache_lse,
                                    const uint8_t *cache_valid, int32_t band_k, double budget,
                                    int32_t anchor, int8_t *plan, int32_t *fresh_list,
                                    int32_t *counts, float *score_out, ditango_stream stream);

/* ---------------------------------------------------------------------------
 * A key/value history in 4 bits.  Where states cannot stand in for a history
 * (the queries are new: the next chunk of a streamed video, text tokens), its
 * keys and values are kept instead, in pages of DITANGO_PAGE tokens and 4 bits
 * a value, for a batch of requests of any lengths.  Attention over it gives
 * states (O, lse) like the rest of the library: written into a state buffer's
 * slot (the strides allow it) they merge with the partitions' own.
 *
 * A page of one key head is DITANGO_PAGE * (d + 8) bytes: K codes, V codes
 * (token-major, d/2 bytes a token, channel 2b in the low half of byte b), then
 * for each token K's (scale, least) and for each token V's, all bf16.  A code
 * c in 0..15 stands for c * scale + least.  least is the row's least value
 * (exact: the rows are bf16) and scale the smallest bf16 value whose 15 steps
 * reach its largest, so that every value is at most half a step off.
 *
 * Slots: token place page * DITANGO_PAGE + offset.  Tables: block_table int32
 * [R][max_blocks] holds the pages of each request in order; entries behind a
 * request's last page may hold anything.  Page numbers out of range are never
 * followed: they count as pages without tokens, and DITANGO_ERR_BOUNDS is
 * recorded in dev_status (in every build). */
enum { DITANGO_PAGE = 64, DITANGO_QBLOCK = 128 };

typedef struct {
  int32_t n_pages, Hkv, d; /* pages, key heads, head dim in {64, 96, 128} */
  uint8_t *data;           /* dev [n_pages][Hkv][DITANGO_PAGE * (d + 8)], 16-byte aligned */
} ditango_kv4;

/* Block tables, slot map and offsets of a batch, from request lengths (the
 * device's counterpart of ditango_slot_table; nothing is read on the host).
 * Request r holds ctx_len[r] tokens and receives new_len[r] more; its first
 * ceil(ctx_len / 64) table entries are its pages.  The pages that it lacks are
 * taken from free_pages in request order, and every new token's slot is
 * written in request order.
 *   R            requests, 1 <= R <= 4096 (else UNSUPPORTED).
 *   ctx_len, new_len  dev int32 [R];  free_pages  dev int32 [n_free].
 *   block_table  dev int32 [R][max_blocks], in and out: only new entries are
 *                written.
 *   kv_len       dev int32 [R] out: ctx_len + new_len.  Must not overlap the
 *                inputs (INVALID), like every other output.
 *   q_off        dev int32 [R + 1] out: running sum of new_len.
 *   slot_map     dev int64 [max_tokens] out: slots of the new tokens; -1 from
 *                q_off[R] on.
 *   pages_used   dev int32 [1] out: entries of free_pages taken.
 * A request that does not fit (a negative length, more than max_blocks pages,
 * the free list or max_tokens exhausted) takes nothing: its kv_len stays
 * ctx_len, its tokens' slots are -1, and DITANGO_ERR_BOUNDS is recorded.  What it
 * lacked counts against the requests behind it that need pages or token places
 * themselves, not against those that need none. */
ditango_status ditango_block_tables(int32_t R, int32_t max_blocks, int32_t max_tokens,
                                    int32_t n_pages, const int32_t *ctx_len,
                                    const int32_t *new_len, const int32_t *free_pages,
                                    int32_t n_free, int32_t *block_table, int32_t *kv_len,
                                    int32_t *q_off, int64_t *slot_map, int32_t *pages_used,
                                    int32_t *dev_status, ditango_stream stream);

/* Write T tokens into the slots slot_map dev int64 [T] (-1: the token is left
 * out; slots out of range: left out and recorded; the slots of one call must
 * differ, else what is stored there is undefined).  K, V dev bf16
 * [T][Hkv][d] with (token, head) element strides, multiples of 8, and 16-byte
 * aligned.  Codes are exactly round-to-nearest-even of (x - least) / scale.  A
 * row that holds an infinity or a NaN is stored as NaN.  T * Hkv < 2^27 (else
 * UNSUPPORTED), here and in ditango_kv4_read. */
ditango_status ditango_kv4_write(const ditango_kv4 *c, int64_t T, const uint16_t *K,
                                 const uint16_t *V, const int64_t k_strides[2],
                                 const int64_t v_strides[2], const int64_t *slot_map,
                                 int32_t *dev_status, ditango_stream stream);

/* Read slots back as bf16 rows (each value c * scale + least rounded once);
 * rows of slots -1 or out of range are left as they were.  The result can be
 * the K and V of ditango_attn_partial or ditango_block_attn. */
ditango_status ditango_kv4_read(const ditango_kv4 *c, int64_t T, uint16_t *K, uint16_t *V,
                                const int64_t k_strides[2], const int64_t v_strides[2],
                                const int64_t *slot_map, int32_t *dev_status,
                                ditango_stream stream);

/* Summaries of the pages that hold tokens [ctx_len[r], kv_len[r]) of the
 * requests, for ditango_block_select: sum_codes dev int8 [n_pages][Hkv][d],
 * sum_scale dev float32 [n_pages][Hkv], of the mean of all of the page's keys
 * up to kv_len (see ditango_block_summary).  Call it after ditango_kv4_write. */
ditango_status ditango_kv4_summary(const ditango_kv4 *c, int32_t R, int32_t max_blocks,
                                   const int32_t *ctx_len, const int32_t *kv_len,
                                   const int32_t *block_table, int8_t *sum_codes,
                                   float *sum_scale, int32_t *dev_status,
                                   ditango_stream stream);

/* The pages that one query token a request attends: ditango_block_select
 * (own_blocks 0) over the page summaries, for Q dev bf16 [R][H][d] ((request,
 * head) element strides, multiples of 8, 16-byte aligned), whose codes it forms
 * itself.
 *   max_blocks   width of block_table, <= 51200 (else UNSUPPORTED).
 *   q_codes, q_scale  dev int8 [R][H][d] and float32 [R][H]: scratch, used when
 *                the heads of a key head are more than 16 or max_blocks is too
 *                wide for all their scores in shared memory.
 *   sel, sel_count  dev int32 [R][Hkv][max_sel] and [R][Hkv] out, max_sel >=
 *                max(k, sink + 1 + 2 band) (the band counts with band >= 0). */
ditango_status ditango_kv4_select(const ditango_kv4 *c, int32_t R, int32_t H, int32_t max_blocks,
                                  int32_t k, int32_t band, int32_t sink, int32_t max_sel,
                                  const uint16_t *Q, const int64_t q_strides[2],
                                  const int8_t *sum_codes, const float *sum_scale,
                                  const int32_t *block_table, const int32_t *kv_len,
                                  int8_t *q_codes, float *q_scale, int32_t *sel,
                                  int32_t *sel_count, int32_t *dev_status,
                                  ditango_stream stream);

/* Bytes of device scratch of ditango_kv4_attn (0 for an unsupported d).  Zero
 * it once when it is allocated: every launch leaves its counters at zero
 * again (not one that recorded DITANGO_ERR_TIMEOUT: zero it before the next).
 * Launches that may run at the same time (other streams, concurrent graph
 * branches) must not share one. */
size_t ditango_kv4_attn_workspace_size(int32_t d);

/* Attention of the requests' new tokens over their histories.  Token t of
 * request r (row q_off[r] + t of Q) attends the first kv_len[r] tokens of the
 * request, with causal != 0 those before and at its own place, the new tokens
 * being the last ones: kv_len - (n - 1 - t) tokens, n = q_off[r+1] - q_off[r].
 * Query head h reads key head h / (H / Hkv).
 *   T, max_q     rows of Q, and a bound on the new tokens of one request (it
 *                chooses the kernel; a bound that is too small costs time only).
 *                Nothing is done for T = 0.
 *   Q            dev bf16 [T][H][d], (token, head) element strides, multiples
 *                of 8, 16-byte aligned.
 *   q_off, kv_len, block_table   as ditango_block_tables leaves them.
 *   sel, sel_count  dev int32 [R][Hkv][max_sel] and [R][Hkv], or NULL: only the
 *                listed blocks (indices into the request's table row, distinct)
 *                are attended, for all new tokens of the request alike.  Indices
 *                out of range count as empty, counts as 0 or max_sel, and are
 *                recorded as DITANGO_ERR_BOUNDS.
 *   scale        logit scale; 0 means 1/sqrt(d).
 *   out          dev [T][H][d] bf16 or float32 (out_is_fp32), (token, head)
 *                element strides out_strides, multiples of 4 (NULL: packed);
 *                16-byte (bf16: 8-byte) aligned.  Must not be Q.
 *   out_lse      dev float32 (token, head) strides lse_strides (NULL: [T][H]),
 *                or NULL.
 *   workspace    dev, ditango_kv4_attn_workspace_size bytes, 16-byte aligned.
 * A row that sees no key gets O = 0, lse = -inf.  Rows behind q_off[R] are left
 * as they were.  Keys that a row does not see never touch it, whatever they
 * hold.  For the second product a probability is rounded to fp16, to 2^-30 of the
 * row's largest at worst; lse and the sums are fp32.  Where more than 16 rows of a
 * key head go together, a value is rounded to fp16 too, to 2^-15 of the largest that
 * the row sees at worst (probabilities and values to bf16 where values that not all
 * rows see are 2^10 or more apart).  The result does not depend on the order in which
 * blocks run. */
ditango_status ditango_kv4_attn(const ditango_kv4 *c, int32_t R, int32_t H, int32_t T,
                                int32_t max_q, int32_t max_blocks, const uint16_t *Q,
                                const int64_t q_strides[2], const int32_t *q_off,
                                const int32_t *kv_len, const int32_t *block_table,
                                const int32_t *sel, const int32_t *sel_count, int32_t max_sel,
                                float scale, int32_t causal, void *out, int32_t out_is_fp32,
                                const int64_t *out_strides, float *out_lse,
                                const int64_t *lse_strides, void *workspace,
                                size_t workspace_bytes, int32_t *dev_status,
                                ditango_stream stream);

/* ---------------------------------------------------------------------------
 * Attention over selected key blocks: the plan's idea (near units always, of
 * the others the most important ones under a budget) at the grain of query
 * blocks of DITANGO_QBLOCK rows and key blocks of DITANGO_PAGE rows, per head,
 * with a score that needs no earlier step.
 *
 * Summaries of the blocks of x dev bf16 [B][H][N][d] ((b, h, n) element
 * strides, multiples of 8; 16-byte aligned): of each block of `block` rows
 * (DITANGO_PAGE or DITANGO_QBLOCK; the last one may be shorter) the sum S over
 * its rows (fp64, of sums of up to four rows in fp32, which are exact for values
 * within 2^14 of one another) and, with top = max |S|,
 *   codes int8 [B][H][nb][d] = rint(127 S / top), scale float32 [B][H][nb] =
 *   top / (127 n), mean float32 [B][H][nb][d] (or NULL) = S / n.
 *   len          dev int32 [B] valid rows, or NULL; blocks without a valid row,
 *                and blocks whose sum is not finite, get codes 0 and scale 0. */
ditango_status ditango_block_summary(int32_t B, int32_t H, int32_t N, int32_t d, int32_t block,
                                     const uint16_t *x, const int64_t strides[3],
                                     const int32_t *len, int8_t *codes, float *scale,
                                     float *mean, ditango_stream stream);

/* Both summaries of a call in one launch: Q's blocks of DITANGO_QBLOCK rows and
 * K's of DITANGO_PAGE rows (k_len, k_mean as len and mean above).  H + Hkv <=
 * 65535. */
ditango_status ditango_block_summaries(int32_t B, int32_t H, int32_t Hkv, int32_t Nq, int32_t Nk,
                                       int32_t d, const uint16_t *Q, const int64_t q_strides[3],
                                       const uint16_t *K, const int64_t k_strides[3],
                                       const int32_t *k_len, int8_t *q_codes, float *q_scale,
                                       int8_t *k_codes, float *k_scale, float *k_mean,
                                       ditango_stream stream);

/* Selection.  Per (b, key head g, query block i) the score of key block j is
 *   k_scale_j * sum over query heads h of g, ascending, of q_scale_h (q_h . k_j)
 * in fp32, each operation rounded by itself (the dot product of codes is a
 * whole number), -0 counting as 0 and NaN as the least.  Always taken: j <
 * sink, and with band >= 0 the blocks within band of the query block's own
 * (own_blocks * i ... own_blocks * i + own_blocks - 1; own_blocks = 0: the
 * request's last block).  Then the best others until max(those, k) are taken
 * or none is left, ties to the lower j.
 *   q_codes int8 [B][H][n_q][d], q_scale float32 [B][H][n_q].
 *   k_codes, k_scale  [B][Hkv][n_k][d] and [B][Hkv][n_k], or with block_table
 *                (dev int32 [B][n_k]) the pages' [n_pages][Hkv][d] and
 *                [n_pages][Hkv].
 *   k_len        dev int32 [B] or NULL: only blocks that hold one of the first
 *                k_len[b] tokens can be taken.
 *   sel          dev int32 [B][Hkv][n_q][max_sel] out: ascending, then -1;
 *   sel_count    dev int32 [B][Hkv][n_q] out.  max_sel must hold k and what is
 *                always taken: max(k, sink + max(own_blocks, 1) + 2 band), else
 *                INVALID.
 * n_k <= 51200 (else UNSUPPORTED). */
ditango_status ditango_block_select(int32_t B, int32_t H, int32_t Hkv, int32_t n_q, int32_t n_k,
                                    int32_t d, int32_t k, int32_t band, int32_t sink,
                                    int32_t own_blocks, int32_t max_sel, const int8_t *q_codes,
                                    const float *q_scale, const int8_t *k_codes,
                                    const float *k_scale, const int32_t *block_table,
                                    int32_t n_pages, const int32_t *k_len, int32_t *sel,
                                    int32_t *sel_count, int32_t *dev_status,
                                    ditango_stream stream);

/* Attention of every query block over its listed key blocks (tcgen05, TMA).
 *   Q            dev bf16 [B][H][Nq][d]; K, V [B][Hkv][Nk][d]; (b, h, n) element
 *                strides as in ditango_geom.  Query head h reads key head
 *                h / (H / Hkv).
 *   sel, sel_count  dev int32 [B][Hkv][ceil(Nq / DITANGO_QBLOCK)][max_sel] and
 *                [B][Hkv][ceil(Nq / DITANGO_QBLOCK)]: distinct key blocks, in
 *                any order.  Entries out of range count as empty and are
 *                recorded as DITANGO_ERR_BOUNDS.
 *   k_len        dev int32 [B] valid keys, or NULL; what lies behind them never
 *                touches the result.
 *   out          dev [B][H][Nq][d] bf16 or float32 (out_is_fp32), (b, h, n)
 *                element strides, multiples of 16 bytes (NULL: packed).
 *   out_lse      dev float32 [B][H][Nq] or NULL.
 * bf16 products with fp32 accumulation and softmax; the probabilities are
 * rounded to bf16 for the second product.  A query block without keys gets
 * O = 0, lse = -inf. */
ditango_status ditango_block_attn(int32_t B, int32_t H, int32_t Hkv, int32_t Nq, int32_t Nk,
                                  int32_t d, const uint16_t *Q, const uint16_t *K,
                                  const uint16_t *V, const int64_t q_strides[3],
                                  const int64_t k_strides[3], const int64_t v_strides[3],
                                  const int32_t *sel, const int32_t *sel_count, int32_t max_sel,
                                  const int32_t *k_len, float scale, void *out,
                                  int32_t out_is_fp32, const int64_t *out_strides,
                                  float *out_lse, int32_t *dev_status, ditango_stream stream);

/* The same with (b, h, n) element strides of out_lse (NULL: packed), so that O and
 * lse may be a slot of a state buffer, [B * H][Lmax], and merge with the
 * partitions' states. */
ditango_status ditango_block_attn_strided(int32_t B, int32_t H, int32_t Hkv, int32_t Nq, int32_t Nk,
                                          int32_t d, const uint16_t *Q, const uint16_t *K,
                                          const uint16_t *V, const int64_t q_strides[3],
                                          const int64_t k_strides[3], const int64_t v_strides[3],
                                          const int32_t *sel, const int32_t *sel_count,
                                          int32_t max_sel, const int32_t *k_len, float scale,
                                          void *out, int32_t out_is_fp32,
                                          const int64_t *out_strides, float *out_lse,
                                          const int64_t *lse_strides, int32_t *dev_status,
                                          ditango_stream stream);

/* Time limit, in nanoseconds, of every wait inside the kernels (default
 * 1e9).  Process-wide; read at each launch. */
void ditango_set_wait_limit_ns(int64_t ns);

/* Checked builds.  The library built with -DDITANGO_CHECK
 * (libditango_check.so) validates the device-resident inputs the host cannot
 * see without a synchronisation -- ditango_attn_partial's counts[0] (at most
 * the active units) and fresh list (unit indices in range, active, strictly
 * row-major), and the plan codes ditango_merge reads -- before using them.  A
 * bad attention input makes the kernel compute nothing and record
 * DITANGO_ERR_BOUNDS (also in dev_status when given); a bad plan code is
 * recorded and the unit left out.  The release build skips these checks.
 * ditango_checked_build: 1 in a checked build, 0 otherwise.
 * ditango_check_status: the recorded status (DITANGO_OK if none) into
 * *status_out (host), cleared when reset != 0; synchronises with the device.
 * Always 0 in the release build. */
int32_t ditango_checked_build(void);
ditango_status ditango_check_status(int32_t *status_out, int32_t reset);

/* Failure-detection self-test: launches one block that waits on a barrier
 * nothing will complete, with a limit of limit_ns; the kernel returns and
 * writes DITANGO_ERR_TIMEOUT into dev_status (dev int32).  Exercises the
 * same bounded wait the pipeline kernels use. */
ditango_status ditango_selftest_bounded_wait(int64_t limit_ns, int32_t *dev_status,
                                             ditango_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* DITANGO_H */
