/*
 * emb.h -- C ABI of the GB300 sparse embedding training step.
 *
 * One training step of a multi-table, multi-hot embedding layer on one GPU:
 *   emb_forward          lookup + pooling + concatenation, one fused kernel
 *   emb_backward_update  dedup of the touched rows, per-row gradient reduction
 *                        and the SGD / Adagrad update, in place
 *   emb_unique           the stand-alone dedup primitive
 * and, further down, the dense side's operators: an expert layer (sort,
 * dispatch, products, combine, and their gradients; the whole of it in one call
 * for a few tokens), layer norm and dropout around it, and orthogonalised updates
 * for its weights.
 *
 * The operations are the ones the GTC 2022 "Merlin HugeCTR" slides name
 * (slides "COMMON EMBEDDING PRIMITIVES" and "HUGECTR EMBEDDING LAYER": table
 * lookup, pooling/reduction, concatenation, fused into one kernel; slide
 * "WEIGHT CONVERSION FOR MIXED PRECISION TRAINING": FP32 optimizer math, FP16
 * tables), with the reduction-based (RB) and unique-based (UB) backward
 * flavours named in "NVIDIA EMBark revoluciona la formacion en sistemas de
 * recomendacion a escala", section "Integracion del cluster".
 *
 * Conventions shared by every call
 *  - Pointers are DEVICE pointers unless their name ends in _host.  Device
 *    arrays must be aligned to their element size (int64: 8 bytes, int32 and
 *    fp32: 4, fp16/bf16: 2); the pooled output and grad_out to 16 bytes (the
 *    kernels move 4 columns at a time).  A misaligned pointer returns
 *    EMB_ERR_INVALID_ARG with nothing enqueued.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Every call that takes a stream only enqueues work on it and
 *    returns without waiting, except the *_host copies and emb_sync_status.
 *  - Return value: EMB_OK or a negative emb_status.  Problems the host can see
 *    (null pointers, sizes beyond the limits given at creation, bad enums)
 *    return at once with nothing enqueued.  Problems only the GPU can see (a
 *    key outside [0, rows), a bag whose table id is not j / batch, a full hash
 *    table, a bounded wait that ran out) never trap: the offending lookup or
 *    row is skipped and a sticky error word in the layer records it, returned
 *    and cleared by emb_sync_status.
 *  - Thread safety: a layer may be used from one host thread at a time; calls
 *    on one layer must be issued on one stream (or be ordered by the caller).
 */
#ifndef EMB_H
#define EMB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    EMB_OK = 0,
    EMB_ERR_INVALID_ARG = -1,   /* bad argument, detected on the host (or a bad table id on the GPU) */
    EMB_ERR_OOM = -2,           /* device allocation failed */
    EMB_ERR_CUDA = -3,          /* a CUDA runtime call or launch failed */
    EMB_ERR_KEY_RANGE = -4,     /* GPU saw a key outside [0, rows) */
    EMB_ERR_CAPACITY = -5,      /* GPU hash table full */
    EMB_ERR_TIMEOUT = -6,       /* a bounded GPU wait gave up (see emb_dense_status) */
    EMB_ERR_STATE = -7          /* call out of order (e.g. backward before any forward) */
} emb_status;

typedef enum { EMB_F32 = 0, EMB_F16 = 1, EMB_BF16 = 2 } emb_dtype;
typedef enum { EMB_POOL_SUM = 0, EMB_POOL_MEAN = 1 } emb_pooling;
typedef enum {
    EMB_OPT_SGD = 0,
    EMB_OPT_ADAGRAD = 1,            /* one fp32 accumulator per element */
    EMB_OPT_ROWWISE_ADAGRAD = 2     /* one fp32 accumulator per row */
} emb_opt;
typedef enum {
    EMB_BWD_REDUCTION = 0,      /* RB: sort (row id, bag) pairs, reduce each run of equal ids */
    EMB_BWD_UNIQUE_SORT = 1,    /* UB: sort-based dedup to unique/inverse/counts first, then reduce */
    EMB_BWD_UNIQUE_HASH = 2     /* UB: hash-based dedup first, then reduce by inverse index */
} emb_bwd_variant;

/* One embedding table.  dim must be a multiple of 4 in [4, 128]; rows >= 1.
 * lr / eps / init_acc: SGD uses lr; both Adagrads use all three (init_acc is
 * the initial accumulator value).  The layer stores weights in `dtype` and the
 * accumulators in fp32 (rows*dim of them for Adagrad, rows for row-wise
 * Adagrad); all arithmetic is fp32.
 * master_fp32 (fp16/bf16 tables only; EMB_ERR_INVALID_ARG for fp32): GTC 2022
 * HugeCTR slides, "WEIGHT CONVERSION FOR MIXED PRECISION TRAINING" -- the
 * optimizer keeps FP32 weights and the FP16 copy the forward reads is
 * converted from them.  The layer then holds rows*dim fp32 master values;
 * every update steps the master in fp32 and stores the 16-bit weight as the
 * new master rounded to nearest-even, so steps smaller than half a 16-bit
 * ulp accumulate instead of being rounded away.
 * dynamic (GTC 2022 HugeCTR slides, "HUGECTR EMBEDDING LAYER": embeddings
 * behind a GPU hash table): the table's keys are arbitrary int64 ids, not row
 * indices, and `rows` is the capacity.  emb_forward finds each key's row in an
 * open-addressing map over the rows (linear probing from a hash of table and
 * key) and, for a key it has not seen, takes a free row and gives it initial
 * values: the counter-based values of emb_init_uniform with splitmix64
 * output number (key << 8) ^ (t << 57) ^ c, the table's init_acc and, with
 * master_fp32, the fp32 value as master.  Nothing is evicted: a lookup that
 * finds the table full is skipped and reported as EMB_ERR_CAPACITY.  The key
 * -2^63 is reserved and reported like an out-of-range key.  Everything after
 * the lookup (dedup ids, row I/O) uses the row, which emb_find_keys gives. */
typedef struct {
    int64_t rows;
    int32_t dim;
    int32_t dtype;     /* emb_dtype */
    int32_t pooling;   /* emb_pooling */
    int32_t opt;       /* emb_opt */
    float lr;
    float eps;
    float init_acc;
    int32_t master_fp32; /* 1: keep an fp32 master copy of a 16-bit table (see below); 0: none */
    int32_t dynamic;     /* 1: keys are arbitrary int64 ids mapped to rows by a hash map (see below) */
} emb_table_spec;

typedef struct emb_layer emb_layer;   /* opaque; owns tables, optimizer state and workspace */

/* Create a layer of `num_tables` tables (1..4096).  GTC 2022 HugeCTR slides,
 * "CHALLENGES OF EMBEDDING LAYER": the tables' memory demand is the first
 * challenge the slide names (there answered by spreading tables over GPUs),
 * and lower precision such as FP16 the common answer; here every table (fp32,
 * fp16 or bf16), its optimizer state and the step's workspace are held in this
 * one GPU's memory.  The sum of all rows must be
 * below 2^32 - 1.  `max_batch` (>= 1) and `max_nnz` (>= 0, < 2^31) bound every
 * later forward: the workspace for that many bags and lookups is allocated
 * here, once, so the step itself allocates nothing.  Weights are NOT
 * initialised (call emb_init_uniform or emb_set_rows).  On success *out owns
 * the device memory until emb_destroy.  Allocation failure: EMB_ERR_OOM with
 * nothing leaked and *out untouched.
 * Test hooks, read here from the environment (unset in normal use):
 * EMB_TEST_ALLOC_LIMIT_BYTES caps what this call may allocate (to reach the
 * EMB_ERR_OOM path); EMB_TEST_REDUCE_CHUNK (a power of two in [32, 256])
 * raises the layer's reduction chunk length, so small inputs run the kernels
 * large multi-hot inputs get.  Neither changes any result. */
int emb_create(const emb_table_spec* specs, int32_t num_tables, int32_t max_batch,
               int64_t max_nnz, emb_layer** out);

/* Free everything the layer owns.  Synchronises the device first.  NULL is a
 * no-op.  No passage: library convenience. */
int emb_destroy(emb_layer* layer);

/* Fill every table with the counter-based uniform values
 *   w(t, r, c) = lo + (hi - lo) * ((h >> 40) * 2^-24),  h = splitmix64 output
 *   number n = t*2^44 + r*2^12 + c of the stream started from state `seed`,
 * evaluated in fp32 with one rounding per operation and then rounded to
 * nearest-even into the table dtype; set every Adagrad accumulator to its
 * table's init_acc and every fp32 master to the fp32 value.  A dynamic table
 * is emptied instead (all keys forgotten); its rows get the same kind of
 * values, from this seed/lo/hi, when keys take them.  Asynchronous on
 * `stream`.  No passage: library convenience (the pages give no
 * initialisation; this counter-based one lets tests regenerate any row). */
int emb_init_uniform(emb_layer* layer, uint64_t seed, float lo, float hi, void* stream);

/* Forward: lookup + pooling + concatenation (GTC 2022 HugeCTR slides, "COMMON
 * EMBEDDING PRIMITIVES"; Merlin overview article, section "HugeCTR").
 *   keys       int64[nnz]            local row ids, bags back to back
 *   offsets    int64[T*batch + 1]    CSR boundaries, bag j = t*batch + b
 *                                    (table-major); offsets[0] = 0,
 *                                    non-decreasing, offsets[T*batch] = nnz
 *   table_ids  int32[T*batch]        table of bag j; must equal j / batch
 *   out        fp32[batch, sum(dim)] out[b, doff_t + c] = s_j * sum over the
 *                                    bag of W_t[key][c]; s_j = 1 (sum) or
 *                                    1/L_j (mean); an empty bag gives 0;
 *                                    doff_t = dim_0 + ... + dim_(t-1)
 * All of keys/offsets/table_ids/out are caller-owned; none is kept after the
 * call.  The lookup's global row ids and bag ids are kept in the layer's
 * workspace for the next emb_backward_update.  A key outside [0, rows_t) or a
 * wrong table id is skipped (contributes 0, gets no gradient) and flagged
 * (EMB_ERR_KEY_RANGE / EMB_ERR_INVALID_ARG at emb_sync_status).  Offsets
 * that leave [0, nnz] or decrease are clamped on the GPU (into [0, nnz],
 * then to the bag start) before any key is read, and flagged as
 * EMB_ERR_INVALID_ARG at emb_sync_status; the pooled output and a following
 * backward are then meaningless but every access stays inside the caller's
 * arrays and the layer's workspace. */
int emb_forward(emb_layer* layer, const int64_t* keys, const int64_t* offsets,
                const int32_t* table_ids, int64_t nnz, int32_t batch, float* out,
                void* stream);

/* Backward + update for the most recent emb_forward on this layer: the
 * reduction-based (RB) or unique-based (UB) backward of "NVIDIA EMBark
 * revoluciona la formacion en sistemas de recomendacion a escala", section
 * "Integracion del cluster" (RB reduces the gradients of equal keys; UB
 * dedups the keys first), with the FP32 optimizer of the GTC 2022 HugeCTR
 * slides, "WEIGHT CONVERSION FOR MIXED PRECISION TRAINING":
 *   G_u[c] = sum over lookups i of row u of s_bag(i) * grad_out[b(i), doff_t + c]
 * then one optimizer step per touched row u (untouched rows are not read):
 *   SGD:     W <- W - lr*G
 *   Adagrad: A <- A + G*G ; W <- W - lr*G/(sqrt(A)+eps)     (per element)
 *   row-wise Adagrad: a <- a + (1/dim) * sum_c G[c]^2 (one accumulator a per
 *            row) ; W <- W - lr*G/(sqrt(a)+eps).  The pages name only the
 *            fp32 optimizer; this is the row-wise form of the open DLRM
 *            embedding libraries, which moves 4 bytes of state per row
 *            instead of 4*dim.
 * fp32 math, W stored back rounded to nearest-even into its dtype.
 * grad_out: fp32[batch, sum(dim)], caller-owned, same layout as `out`.
 * variant: emb_bwd_variant.  All variants give the same indices and the same
 * update up to fp32 rounding order; each variant is deterministic.
 * EMB_ERR_STATE if no forward preceded it. */
int emb_backward_update(emb_layer* layer, const float* grad_out, int32_t variant, void* stream);

/* Early dedup.  With variant >= 0 (an emb_bwd_variant), every later
 * emb_forward also enqueues the dedup of that backward variant on an
 * internal stream of the layer: the global ids and bags are extracted and
 * sorted (or hashed) while the pooling kernel runs on the caller's stream --
 * the dedup needs only the batch's keys, not the pooled output.  A following
 * emb_backward_update on the caller's stream waits for it and, if called with
 * the same variant, goes straight to the segmented reduction (with another
 * variant it redoes the dedup).  Results are identical to the default mode.
 * variant = -1 (default) turns it off.  The caller's input buffers must stay
 * valid until that backward is enqueued; no extra memory is used.  Passage:
 * "NVIDIA EMBark ...", section "Integracion del cluster" (the UB dedup needs
 * only the keys), and the fused embedding kernels of the GTC 2022 HugeCTR
 * slides, "HUGECTR EMBEDDING LAYER". */
int emb_set_early_dedup(emb_layer* layer, int32_t variant);

/* Keep (1) or drop (0, default) the dedup by-products of later backwards so
 * emb_dedup_result can return them.  EMB_BWD_REDUCTION then also writes the
 * sorted unique ids, counts and segment offsets it otherwise never forms.
 * No passage: library convenience (tests and callers that want the dedup). */
int emb_set_keep_dedup(emb_layer* layer, int32_t keep);

/* Copy the dedup result of the last emb_backward_update (with keep_dedup on)
 * into caller device buffers, each sized for the forward's nnz (NULL = skip):
 *   unique       int64[U]    global row ids row_base[t] + key, ascending
 *   inverse      int32[nnz]  unique[inverse[i]] = global id of lookup i;
 *                            skipped lookups get U.  Not formed by
 *                            EMB_BWD_REDUCTION (EMB_ERR_STATE if requested)
 *   counts       int32[U]    lookups per unique row
 *   seg_offsets  int32[U+1]  exclusive prefix sum of counts
 *   sorted_bags  int32[nnz]  bag id of each lookup, grouped by unique row,
 *                            ascending lookup order inside a group
 *   num_unique_host          U (the call synchronises `stream` for it)
 * EMB_ERR_STATE if there is no such result.  Passage: "NVIDIA EMBark ...",
 * section "Integracion del cluster" (the unique keys, inverse index and
 * counts of the UB dedup). */
int emb_dedup_result(emb_layer* layer, int64_t* unique, int32_t* inverse, int32_t* counts,
                     int32_t* seg_offsets, int32_t* sorted_bags, int64_t* num_unique_host,
                     void* stream);

/* Stand-alone dedup of arbitrary int64 keys: the dedup step that the
 * unique-based (UB) backward of "NVIDIA EMBark revoluciona la formacion en
 * sistemas de recomendacion a escala", section "Integracion del cluster",
 * runs before reducing gradients:
 *   unique       int64[n]    distinct keys, ascending, in unique[0..U)
 *   inverse      int32[n]    unique[inverse[i]] == keys[i]
 *   counts       int32[n]    counts[k] = #{i : keys[i] == unique[k]}, k < U
 *   seg_offsets  int32[n+1]  nullable; exclusive prefix sum of counts, [0..U]
 *   num_unique   int64[1]    U, written on the device
 * n in [0, 2^31).  `workspace` is caller-owned device memory of at least
 * emb_unique_workspace(n) bytes, 256-byte aligned; the call keeps no pointer
 * after it returns.  Sort-based (own LSD radix sort over the key range), so
 * the result is deterministic. */
int emb_unique_workspace(int64_t n, size_t* bytes);
int emb_unique(const int64_t* keys, int64_t n, int64_t* unique, int32_t* inverse,
               int32_t* counts, int32_t* seg_offsets, int64_t* num_unique,
               void* workspace, size_t workspace_bytes, void* stream);

/* emb_unique without any allocation, for callers that cannot allocate device
 * memory at call time: for instance a plugin whose enqueue path runs inside a
 * host framework that forbids cudaMalloc there (it may synchronise the device,
 * and fails outright under a fixed memory budget), or a serving thread that
 * must not touch the allocator while requests are in flight.  There is no
 * counterpart on the pages: this is a library convenience, not part of the
 * embedding method.
 *
 * Arguments and results are exactly those of emb_unique, minus the workspace:
 * the scratch is one array compiled into the library (12 MB of device
 * memory, held on every GPU that loads the library until the process exits).
 * n must be at most EMB_UNIQUE_NOALLOC_MAX_KEYS; larger n returns
 * EMB_ERR_INVALID_ARG and enqueues nothing.  The first call on a device looks
 * up the array's address on that device (the device current at the call), so
 * make that first call before any stream capture.  All calls share the one
 * array: calls whose GPU work overlaps -- on different streams or from
 * different threads without ordering -- race on it and give wrong results; the
 * contents left by the previous call are never relied on.  The address looked
 * up on a device stays in use for the life of the process: after
 * cudaDeviceReset on that device the function must not be called again. */
#define EMB_UNIQUE_NOALLOC_MAX_KEYS 262144
int emb_unique_noalloc(const int64_t* keys, int64_t n, int64_t* unique, int32_t* inverse,
                       int32_t* counts, int32_t* seg_offsets, int64_t* num_unique, void* stream);

/* Copy rows [row0, row0+n) of table t between the layer and host memory.
 * weights_host holds n*dim values of the table dtype (fp32, or the raw 16-bit
 * patterns of fp16/bf16); state_host (nullable; Adagrad tables only) n*dim
 * fp32, or n fp32 for row-wise Adagrad.  Synchronous: the call waits for
 * `stream`.  No passage: library convenience (checkpoint and resume, tests). */
int emb_get_rows(emb_layer* layer, int32_t t, int64_t row0, int64_t n, void* weights_host,
                 float* state_host, void* stream);
int emb_set_rows(emb_layer* layer, int32_t t, int64_t row0, int64_t n,
                 const void* weights_host, const float* state_host, void* stream);

/* Inference cache of table t (GTC 2022 HugeCTR slides, slide "HUGECTR:
 * SCALABLE, ACCELERATED RECSYS TRAINING": inference served through an
 * embedding cache on the GPU in front of the hierarchical parameter server,
 * HPS): fp16 copies of n chosen
 * rows (device int64 row ids; a dynamic table's rows from emb_find_keys),
 * looked up through a hash map from row to cache slot.  Replaces any earlier
 * cache of the table; n = 0 removes it.  The copies are a snapshot of the
 * rows at this call (16-bit tables are converted from their stored values
 * to fp16): training steps do not refresh them.  Tables of 2^31 rows or more
 * take no cache (EMB_ERR_INVALID_ARG).  Allocates device memory for the cache
 * and synchronises `stream`; EMB_ERR_OOM when it cannot allocate.
 * An id outside [0, rows) is skipped and flagged like a bad key. */
int emb_cache_build(emb_layer* layer, int32_t t, const int64_t* rows, int64_t n, void* stream);

/* Inference-only forward: the pooled, concatenated output of emb_forward
 * (same arguments, layout and error reporting), reading every row held in
 * its table's cache from the fp16 cache and every other row from the table.
 * Dynamic tables look keys up without inserting; an id the table does not
 * hold contributes nothing and is not an error.  Nothing is kept for a
 * backward: a following emb_backward_update still refers to the last
 * emb_forward.  Allocates nothing.  Passage: as for emb_cache_build. */
int emb_forward_infer(emb_layer* layer, const int64_t* keys, const int64_t* offsets,
                      const int32_t* table_ids, int64_t nnz, int32_t batch, float* out,
                      void* stream);

/* Rows of n keys (device int64) of dynamic table t, into rows_out (device
 * int64; -1 for a key the table does not hold).  Inserts nothing.
 * Asynchronous; EMB_ERR_INVALID_ARG for a table that is not dynamic.
 * Passage: GTC 2022 HugeCTR slides, "HUGECTR EMBEDDING LAYER" (the GPU hash
 * table from keys to embedding rows). */
int emb_find_keys(emb_layer* layer, int32_t t, const int64_t* keys, int64_t n, int64_t* rows_out,
                  void* stream);

/* The fp32 master copy of rows [row0, row0+n) of table t (a table created
 * with master_fp32 = 1; EMB_ERR_INVALID_ARG otherwise), n*dim fp32 in host
 * memory, for checkpoints and tests.  Synchronous: the call waits for
 * `stream`.  Setting the master does not touch the 16-bit weights: set both
 * (emb_set_rows) to restore a checkpoint.  Passage: GTC 2022 HugeCTR slides,
 * "WEIGHT CONVERSION FOR MIXED PRECISION TRAINING" (the FP32 weights behind
 * FP16 tables). */
int emb_get_master_rows(emb_layer* layer, int32_t t, int64_t row0, int64_t n, float* master_host,
                        void* stream);
int emb_set_master_rows(emb_layer* layer, int32_t t, int64_t row0, int64_t n,
                        const float* master_host, void* stream);
/* Gather n arbitrary rows' master values (device int64 ids) into a device
 * buffer of n*dim fp32.  Asynchronous; out-of-range ids are skipped and
 * flagged like bad keys.  Passage: as for emb_get_master_rows. */
int emb_gather_master_rows(emb_layer* layer, int32_t t, const int64_t* rows, int64_t n, float* master_out,
                           void* stream);

/* Gather n arbitrary rows (device int64 ids, each in [0, rows_t)) of table t
 * into device buffers: weights_out n*dim of the table dtype, state_out
 * (nullable) n*dim fp32 (row-wise Adagrad: n fp32).  Asynchronous.
 * Out-of-range ids are skipped and flagged like bad keys.  No passage:
 * library convenience (tests and checkpoints). */
int emb_gather_rows(emb_layer* layer, int32_t t, const int64_t* rows, int64_t n,
                    void* weights_out, float* state_out, void* stream);

/* Wait for `stream`, then return and clear the sticky device error word
 * (EMB_OK if the GPU saw nothing wrong).  No passage: library convenience. */
int emb_sync_status(emb_layer* layer, void* stream);

/* Number of kernels the library launched on behalf of this layer since the
 * last reset (reset = 1 clears it after reading).  No passage: library
 * convenience (measurement). */
int emb_launch_count(emb_layer* layer, int64_t* count_host, int32_t reset);

/* Phase timing.  With enable = 1 the layer records CUDA events on the call's
 * stream around each phase of every later step -- EMB_PHASE_FORWARD (the
 * fused lookup/pooling kernel), EMB_PHASE_DEDUP (global-id sort or hash
 * dedup, from the start of emb_backward_update up to the reduction) and
 * EMB_PHASE_REDUCE_UPDATE (segmented reduction + optimizer kernels) -- and
 * adds their elapsed times.  With early dedup the dedup phase runs on the
 * layer's internal stream, overlapping the forward.  A step's events are
 * read back only when a ring of 64 steps comes round to its slot again, so
 * timing adds no host wait to a step.  emb_phase_times waits for the last
 * recorded events, writes the accumulated milliseconds of the n (<= 3)
 * phases and the number of steps they cover, and, with reset = 1, clears
 * them.  No passage: library convenience (measurement). */
enum { EMB_PHASE_FORWARD = 0, EMB_PHASE_DEDUP = 1, EMB_PHASE_REDUCE_UPDATE = 2, EMB_NUM_PHASES = 3 };
int emb_set_timing(emb_layer* layer, int32_t enable);
int emb_phase_times(emb_layer* layer, float* ms_host, int32_t n, int64_t* steps_host, int32_t reset);

/* -------------------------------------------------------------------------
 * Experts.  The dense side of a recommender sends each sample (token) of the
 * pooled embeddings to k of E experts and adds their answers up, weighted.
 * The calls below are the data movement and the products of that layer; the
 * router's scores, the activation between two products and the loss are the
 * caller's.  They keep no state and need no layer: every array is the
 * caller's.  Types named "dtype" are an emb_dtype.  A "stride" is the distance
 * in elements between the starts of two consecutive rows, at least the row's
 * width; the elements of a row are contiguous.  Arrays without a stride are
 * contiguous.  Rows of a multiple of 8 elements, all at 16-byte boundaries, are
 * moved 16 bytes at a time, rows of even widths, strides and addresses two elements
 * at a time, any other one element at a time.
 * What the GPU alone can see (an id outside [-1, E), a bounded wait that ran
 * out) is recorded in a sticky word of the device, see emb_dense_status.
 * ------------------------------------------------------------------------- */

/* Where each assignment of a batch goes.  Assignment a = t * k + j is token t's
 * j-th expert, P = tokens * k (0 <= P < 2^31).  Device arrays:
 *   offsets[E + 1]  first row of each expert's group; offsets[E] rows are kept
 *   src[P]          the assignment in row p, in increasing order within a
 *                   group; -1 for p >= offsets[E]
 *   pos[P]          the row of assignment a, -1 for one without an expert
 * The calls that read a plan skip a pos outside [0, P) and read offsets
 * clamped into [0, P] and made non-decreasing, so no plan sends them outside
 * the arrays.  tokens >= 0, k in [1, 64], experts (E) in [1, 1024]. */
typedef struct {
    int32_t* offsets;
    int32_t* src;
    int32_t* pos;
    int64_t tokens;
    int32_t k;
    int32_t experts;
} emb_expert_plan;

/* Build a plan: a stable sort of the assignments by expert.  ids[P] are int32
 * (id_bytes 4) or int64 (id_bytes 8); id -1 is an assignment without an expert
 * (a dropped one).  Any other id outside [0, E) is treated as -1 and recorded
 * as EMB_ERR_KEY_RANGE.  The arrays of `plan` are written.  The workspace
 * (256-byte aligned, emb_expert_sort_workspace bytes) is free again once the
 * call's work on the stream is done; up to EMB_EXPERT_SORT_ALONE assignments
 * nothing reads or writes it.  No passage: library convenience (the pages stop
 * at the embeddings). */
#define EMB_EXPERT_SORT_ALONE 4096
int emb_expert_sort_workspace(int64_t tokens, int32_t k, int32_t experts, size_t* bytes);
int emb_expert_sort(const void* ids, int32_t id_bytes, const emb_expert_plan* plan, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Gather the tokens' rows in expert order, rows[p] = x[src[p] / k] for
 * p < offsets[E] and 0 for the rows after them, x [tokens, width] and rows
 * [P, width]; and the gradient of x, grad_x[t] = sum_j grad_rows[pos[t, j]],
 * added in fp32 in the order of j and rounded once.  A token without experts
 * gets a zero gradient.  Both types are any emb_dtype.  No passage: library
 * convenience. */
int emb_expert_dispatch(const emb_expert_plan* plan, const void* x, int32_t x_dtype, int64_t x_stride, int64_t width,
                        void* rows, int32_t rows_dtype, void* stream);
int emb_expert_dispatch_grad(const emb_expert_plan* plan, const void* grad_rows, int32_t rows_dtype,
                             int64_t grad_stride, int64_t width, void* grad_x, int32_t x_dtype, void* stream);

/* Back to tokens, weighted: out[t] = sum_j weights[t, j] * rows[pos[t, j]],
 * fp32 weights and sums, in the order of j, rounded once to out_dtype; a token
 * without experts gets zeros.  The gradients:
 *   grad_rows[p]       = weights[src[p]] * grad_out[src[p] / k]   (0 for p >= offsets[E]),  in rows' dtype
 *   grad_weights[t, j] = <grad_out[t], rows[pos[t, j]]>           (0 without an expert),    fp32
 * The weight of an assignment without an expert is not used: it may be
 * anything, NaN included.  No passage: library convenience. */
int emb_expert_combine(const emb_expert_plan* plan, const void* rows, int32_t rows_dtype, int64_t rows_stride,
                       const float* weights, int64_t width, void* out, int32_t out_dtype, void* stream);
int emb_expert_combine_grad(const emb_expert_plan* plan, const void* grad_out, int32_t out_dtype, int64_t grad_stride,
                            const void* rows, int32_t rows_dtype, int64_t rows_stride, const float* weights,
                            int64_t width, void* grad_rows, float* grad_weights, void* stream);

/* Each expert's product over its own rows.  dtype is EMB_F16 or EMB_BF16 for
 * every array; in_width and out_width are multiples of 8; all arrays are
 * 16-byte aligned and strides multiples of 8; weight is
 * [E, out_width, in_width].  For p in group e (offsets[e] <= p < offsets[e+1]):
 *   y[p]           = weight[e] rows[p]                         [P, out_width]
 *   grad_rows[p]   = weight[e]^T grad_y[p]                     [P, in_width]
 *   grad_weight[e] = sum over the group of grad_y[p] rows[p]^T [E, out_width, in_width]
 * with products exact, sums in fp32 and one rounding to dtype.  The tensor cores
 * add 16 products at a time and cut a sum off at fp32's last bit where fp32
 * arithmetic rounds: a sum of n terms of one sign comes out about 6e-9 n of it too
 * small (2.4e-5 for n = 4096, 3.9e-4 for 65536, fp16's own half bit being 4.9e-4);
 * of mixed signs the cuts cancel.  (The forward of up to four rows is fp32
 * arithmetic.)  Rows p >= offsets[E] are written as zeros and not read; an expert
 * without rows has a zero grad_weight.  A group's results do not depend on the
 * rows of the others, whatever they hold.  No passage: library convenience. */
int emb_expert_linear(const emb_expert_plan* plan, const void* rows, int64_t rows_stride, const void* weight,
                      int64_t in_width, int64_t out_width, int32_t dtype, void* y, void* stream);
int emb_expert_linear_grad_rows(const emb_expert_plan* plan, const void* grad_y, int64_t grad_stride,
                                const void* weight, int64_t in_width, int64_t out_width, int32_t dtype,
                                void* grad_rows, void* stream);
int emb_expert_linear_grad_weight(const emb_expert_plan* plan, const void* grad_y, int64_t grad_stride,
                                  const void* rows, int64_t rows_stride, int64_t in_width, int64_t out_width,
                                  int32_t dtype, void* grad_weight, void* stream);

/* The whole expert layer for a few tokens, from their ids to their sums, in two to four
 * kernels:
 *   out[t] = sum_j weights[t, j] down[e] act(up[e] x[t]),  e = ids[t, j]
 * ids [tokens, k] as for emb_expert_sort (-1: none; any other id outside [0, E) is
 * treated as -1 and recorded as EMB_ERR_KEY_RANGE); tokens * k is at most
 * EMB_EXPERT_LAYER_ASSIGNMENTS (more go through a plan).  x [tokens, in_width] is fp32
 * (rounded to dtype first, as by emb_expert_dispatch) or of dtype, EMB_F16 or EMB_BF16;
 * up is [E, hidden, in_width] ([E, 2 hidden, in_width] for EMB_ACT_SWIGLU: the gates' rows,
 * then the rows they let through), down [E, out_width, hidden], both of dtype; weights
 * fp32 [tokens, k]; out [tokens, out_width] of any emb_dtype.  Widths are multiples of 8,
 * x, up, down and out 16-byte aligned, x's rows at multiples of 16 bytes.  A chosen expert's
 * weights are read once for each 64 of its assignments (in tiles, of a call of more than 64
 * tokens, for each 128).  Sums are
 * fp32 as in the experts' products; what the activation gives is rounded to dtype, the
 * type the second product takes, y stays fp32 up to the sum over j, in order.  A token
 * without experts gets zeros; the weight of an assignment without one is not used.
 * Activations: relu, v / (1 + exp(-v)), v (1 + erf(v / sqrt 2)) / 2 (as v erfc(-v / sqrt 2) / 2,
 * so that it keeps its digits where it is small), and gate / (1 + exp(-gate)) times the other half.  The workspace is 256-byte aligned,
 * emb_expert_layer_workspace bytes, and free again once the call's work is done.
 * emb_expert_layer_tiles tells which of its two ways a call takes, by its sizes: 1, tiles of the
 * weights on the tensor cores, 0, warps that read them straight; either gives results
 * within the same bounds.  No passage: library convenience. */
#define EMB_EXPERT_LAYER_ASSIGNMENTS 512
enum { EMB_ACT_RELU = 0, EMB_ACT_SILU = 1, EMB_ACT_GELU = 2, EMB_ACT_SWIGLU = 3 };
int emb_expert_layer_workspace(int64_t tokens, int32_t k, int64_t in_width, int64_t hidden, int64_t out_width,
                               size_t* bytes);
int emb_expert_layer(const void* ids, int32_t id_bytes, int64_t tokens, int32_t k, int32_t experts, const void* x,
                     int32_t x_dtype, int64_t x_stride, int64_t in_width, const void* up, const void* down,
                     int32_t dtype, int64_t hidden, int64_t out_width, int32_t activation, const float* weights,
                     void* out, int32_t out_dtype, void* workspace, size_t workspace_bytes, void* stream);
int emb_expert_layer_tiles(int64_t tokens, int32_t k, int32_t experts, int32_t x_dtype, int64_t in_width,
                           int64_t hidden, int64_t out_width, int32_t activation, int32_t* tiles);

/* Orthogonalise `batch` matrices G [rows, cols] by `steps` (1..32) quintic
 * Newton-Schulz steps, as the Muon optimiser does with a momentum
 * (K. Jordan et al., 2024):
 *   X = G / (|G|_F + eps);  steps times:  A = X X^T,  X <- a X + (b A + c A A) X
 * (on the transpose where rows > cols).  G is any emb_dtype, with
 * batch_stride and row_stride in elements; out is bf16 [batch, rows, cols],
 * contiguous.  Between the steps X is held as the sum of two fp16 numbers
 * (times a power of two of its own, so |G| may be far below eps) and A as one,
 * of the products only the first one's; sums are fp32.  That is about a tenth of
 * the error of bf16 arithmetic, not fp32's.  Of the result's 2-norm (the output's
 * rounding to bf16 alone is 1.7e-3): with coefficients that converge 1.8e-3, up to
 * 32 steps; with Muon's, which do not, it grows with the steps, to 2.1e-3 at 5,
 * 2.5e-3 at 6, 3.4e-3 at 8, 4.8e-3 at 12 and 2e-2 at 32.  A zero matrix stays
 * zero, or with eps 0 gives NaNs (0 / 0); one that holds an infinity or a NaN
 * gives NaNs and leaves the others alone.  rows and cols in [1, 65536].  The
 * workspace is 256-byte aligned, emb_orthogonalize_workspace bytes.  No passage:
 * library convenience. */
int emb_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, size_t* bytes);
int emb_orthogonalize(const void* update, int32_t dtype, int64_t batch_stride, int64_t row_stride, int64_t batch,
                      int64_t rows, int64_t cols, int32_t steps, float a, float b, float c, float eps, void* out,
                      void* workspace, size_t workspace_bytes, void* stream);

/* Layer norm of the rows of x [rows, width], and its gradients, g = grad_y:
 *   h = (x - mean) rstd,  rstd = 1 / sqrt(variance + eps),  y = h weight + bias
 *   grad_x      = rstd (g weight - mean(g weight) - h mean(g weight h))   in x's dtype
 *   grad_weight = sum over the rows of g h,  grad_bias = sum over the rows of g
 * weight, bias, grad_weight and grad_bias are [width] of param_dtype; a null weight
 * stands for ones, a null bias for zeros.  Any dtypes; y and grad_x are contiguous, x and
 * grad_y have a row stride.  Statistics and sums are fp32 in a fixed order, with one
 * rounding at the end; the mean's own rounding is taken off again, and rows of any
 * finite size keep their variance.  A row that holds an infinity or a NaN is NaN, and so
 * are its columns' sums; other rows are not touched.  A null grad_x, grad_weight or
 * grad_bias is not computed; without rows the sums are zero.  width in [1, 2^24], eps
 * in [1e-24, fp32's largest].  Rows are copied from and to 16-byte boundaries: up to 15
 * bytes beside x and grad_y may be read, never used.  The workspace is 256-byte
 * aligned, emb_layer_norm_grad_workspace bytes.  No passage: library convenience. */
int emb_layer_norm(const void* x, int32_t x_dtype, int64_t x_stride, int64_t rows, int64_t width, const void* weight,
                   const void* bias, int32_t param_dtype, float eps, void* y, int32_t y_dtype, void* stream);
int emb_layer_norm_grad_workspace(int64_t rows, int64_t width, size_t* bytes);
int emb_layer_norm_grad(const void* grad_y, int32_t y_dtype, int64_t grad_stride, const void* x, int32_t x_dtype,
                        int64_t x_stride, int64_t rows, int64_t width, const void* weight, int32_t param_dtype,
                        float eps, void* grad_x, void* grad_weight, void* grad_bias, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Dropout: y = residual + x / (1 - rate) where the element is kept, residual where it
 * is dropped, whatever x holds there (a null residual stands for zeros); x and y
 * [rows, width] of any dtypes, residual of y's, y contiguous.  The gradient of x is the
 * same call on grad_y without a residual.  Element i = row * width + column is kept
 * when u >= rate * 2^16 (rounded to a whole number, and 1 - rate with it), u being 16
 * bits of Philox4x32 with 7 rounds (J. Salmon et al., "Parallel random numbers: as easy as
 * 1, 2, 3", 2011): counter words (i / 8, its high word, offset, its high word), key
 * the low and high word of the seed, half i % 2 (0: low) of the result's word
 * i % 8 / 2.  So the mask depends on seed, offset and i alone and is never stored.
 * seed_at (nullable, 8-byte aligned) is the seed in device memory, read when the call
 * runs, in place of `seed`.  rate in [0, 1].  No passage: library convenience. */
int emb_dropout(const void* x, int32_t x_dtype, int64_t x_stride, int64_t rows, int64_t width, double rate,
                uint64_t seed, const uint64_t* seed_at, uint64_t offset, const void* residual,
                int64_t residual_stride, void* y, int32_t y_dtype, void* stream);

/* Wait for the stream; return and clear the device's sticky status of the
 * calls of this section (EMB_OK, EMB_ERR_KEY_RANGE or EMB_ERR_TIMEOUT).  Of
 * several threads that ask at once, one gets what there is.  No passage:
 * library convenience. */
int emb_dense_status(void* stream);

/* Static description of an emb_status value.  No passage: library convenience. */
const char* emb_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* EMB_H */
