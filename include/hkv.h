/*
 * hkv.h -- C ABI of a cache-semantic GPU key-value hash table (GB300, sm_103a).
 *
 * The operations follow "HierarchicalKV: A GPU Hash Table with Cache
 * Semantics for Continuous Online Embedding Storage" (arXiv 2603.17168v1),
 * cited below as HKV.  Keys are uint64, scores uint64, values float32 rows of
 * `dim` elements.  A table of capacity C has B = C / 128 buckets of 128 slots
 * (HKV §3.2).  Every key lives in one bucket b1 = H(k) mod B (single mode) or
 * in one of two buckets b1, b2 (dual mode, HKV §3.4), where H is the 64-bit
 * MurmurHash3 finalizer and b2 = H(k ^ 0x9E3779B97F4A7C15) mod B, moved to
 * (b1 + 1) mod B when it equals b1.
 *
 * Reserved keys: 0xFFFFFFFFFFFFFFF0 .. 0xFFFFFFFFFFFFFFFF are sentinels of
 * the table.  An input key in that range is skipped by every call (find
 * reports it not found) and counted; see hkv_get_error_counts.
 *
 * Ranks: admission and victim choice compare ranks, tuples compared
 * lexicographically as unsigned integers, so equal scores never leave a
 * choice open.  Single mode ranks an entry by (score, new, key), where `new`
 * is 1 for an entry placed by the current call and 0 for one that was
 * resident before it: an incoming key of equal score outranks an older
 * entry (HKV Algorithm 2 admits on score >= the bucket minimum), and the key
 * decides between entries of equal score and age.  Dual mode ranks by
 * (score, key) (HKV Algorithm 3 admits on score > the minimum).
 *
 * Batches: duplicate keys inside one insert_or_assign or assign batch
 * collapse to their last occurrence.  Inside one insert_or_assign call the
 * keys already resident are updated first, then the absent keys are placed;
 * in single mode the result is therefore a pure function of the table and the
 * batch (bucket b ends up with the 128 highest-ranked of its residents and of
 * the absent keys hashed to it).  In dual mode each absent key is routed to
 * one of its buckets by Algorithm 3's rules applied to per-bucket summaries
 * (occupancy and lowest score as of the bucket's last upsert pass), each
 * bucket then keeps the highest-ranked of its entries and its routed keys,
 * and the keys displaced by that pass are routed once more with the updated
 * summaries; which keys win near the margin depends on that processing
 * order, but a key that ends up absent always lost to a full bucket all of
 * whose entries outrank it.
 *
 * Memory: all pointer arguments except the `*_host` ones are device pointers
 * (or pointers the device can dereference: mapped or managed host memory).
 * The caller owns them; they must stay valid until the stream reaches the
 * call.  The table owns its storage.  Row-major value buffers hold n * dim
 * float32; a 16-byte aligned base and dim % 4 == 0 select the vector path.
 *
 * Streams: `stream` is a cudaStream_t passed as void* (NULL = legacy default
 * stream).  Every batched call is asynchronous: it validates its arguments,
 * enqueues kernels and returns.  Argument errors are returned at once and
 * enqueue nothing.
 *
 * Score policies (HKV §3.3 "Scoring policies"; §5 Exp #3c, Table 8 names
 * kLru, kLfu, kEpochLru, kEpochLfu and kCustomized without defining their
 * update rules).  A table is created with one policy (mode bits 4-7), which
 * decides the score a call writes for a key (insert_or_assign,
 * insert_and_evict, find_or_insert, assign):
 *   HKV_POLICY_CUSTOMIZED  the caller's score; scores == NULL: the table's
 *                          step counter, which starts at 1 and grows by 1
 *                          per NULL-score call (assign with NULL keeps the
 *                          scores).
 *   HKV_POLICY_LRU         the table clock: the step counter, which under this
 *                          policy grows by 1 per score-writing call.  scores
 *                          must be NULL (else HKV_ERR_INVALID).
 *   HKV_POLICY_EPOCH_LRU   (epoch << 32) | (clock mod 2^32); scores NULL.
 *   HKV_POLICY_LFU         a frequency: scores are per-occurrence increments
 *                          (NULL: 1 each).  The increments of all occurrences
 *                          of a key in one call add up; a resident key gets
 *                          old score + sum, an absent key competes with sum;
 *                          sums saturate at 2^64 - 1.
 *   HKV_POLICY_EPOCH_LFU   (epoch << 32) | f, where f is the LFU rule applied
 *                          to the low 32 bits of the old score, saturating at
 *                          2^32 - 1 (the count survives epoch changes).
 * The epoch is a 32-bit value of the table (0 at creation, hkv_set_epoch),
 * read when a call is issued.  find_or_insert never changes a resident key.
 *
 * Roles (HKV §3.5, Table 4): find, size and export are readers; assign is an
 * updater; insert_or_assign and erase are inserters.  Calls of conflicting
 * roles issued on different streams are ordered by CUDA events in host issue
 * order: readers overlap readers, updaters overlap updaters, an inserter
 * overlaps nothing.  Calls on one table may come from several host threads.
 */
#ifndef HKV_H_
#define HKV_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct hkv_table hkv_table; /* opaque, owned by the library */
typedef int hkv_status;

enum {
  HKV_MODE_SINGLE = 0, /* one candidate bucket per key (HKV §3.2) */
  HKV_MODE_DUAL = 1,   /* two candidate buckets, score-based choice (HKV §3.4) */
  HKV_MODE_TIERED = 2  /* flag: values above the HBM budget live in mapped host memory (HKV §3.6) */
};

/* Score policy, ORed into hkv_create's mode (see "Score policies"). */
enum {
  HKV_POLICY_CUSTOMIZED = 0x00,
  HKV_POLICY_LRU = 0x10,
  HKV_POLICY_LFU = 0x20,
  HKV_POLICY_EPOCH_LRU = 0x30,
  HKV_POLICY_EPOCH_LFU = 0x40,
  HKV_POLICY_MASK = 0xF0
};

enum {
  HKV_OK = 0,
  HKV_ERR_INVALID = -1,      /* bad argument; nothing was enqueued */
  HKV_ERR_OOM = -2,          /* device or pinned host allocation failed */
  HKV_ERR_CUDA = -3,         /* a CUDA runtime call failed */
  HKV_ERR_RESERVED_KEY = -4, /* hkv_get_error_counts: reserved keys were skipped */
  HKV_ERR_TIMEOUT = -5       /* hkv_get_error_counts: keys were abandoned after a bounded wait */
};

#define HKV_SLOTS_PER_BUCKET 128
#define HKV_RESERVED_KEY_LO 0xFFFFFFFFFFFFFFF0ull
#define HKV_MAX_BATCH 0x7FFFFFFFull /* largest n accepted by a batched call */

/* Create a table.  HKV §3.1-§3.2 (bucketed layout), §3.6/§4.2 (tiered).
 *  capacity        slots; a positive multiple of 128 (B = capacity / 128;
 *                  B >= 2 in dual mode).
 *  dim             float32 elements per value row, >= 1.
 *  mode            HKV_MODE_SINGLE or HKV_MODE_DUAL, optionally | HKV_MODE_TIERED,
 *                  | one HKV_POLICY_* (default HKV_POLICY_CUSTOMIZED).
 *  value_hbm_bytes with TIERED: HBM budget for value rows.  Rows of whole
 *                  buckets 0 .. R-1 (R = floor(budget / (128 * 4 * dim)) * 128)
 *                  live in HBM, the rest in pinned host memory the device
 *                  reads and writes directly (see HKV_HOST_SLAB_MAPPED_MAX).
 *                  Ignored without TIERED (all rows in HBM).
 *  device          CUDA device ordinal the table lives on.
 *  out             receives the table handle.
 * Keys, digests and scores always live in HBM.  The table starts empty.
 * Synchronous.  Errors: INVALID, OOM, CUDA (nothing is leaked). */
hkv_status hkv_create(uint64_t capacity, uint32_t dim, uint32_t mode, uint64_t value_hbm_bytes,
                      int device, hkv_table** out);

/* The host slab of a tiered table (the rows above the HBM budget) is
 * cudaHostAllocMapped memory when it holds at most this many bytes, and
 * pinned memory from a memory pool on the device's nearest host NUMA node
 * when it is larger.  Measured on a GB300 (Grace host, 64 KiB pages, NVLink-
 * C2C), random 256-byte row reads from the GPU: mapped memory reads at 183-208
 * GB/s while the process's mapped footprint is at most 16 GiB and at 7-12
 * GB/s beyond 24 GiB; pool memory reads at 26-28 GB/s from 8 GiB to 32 GiB.
 * Where the system offers no host memory pool, a larger slab is mapped
 * memory too.  Either way a row's device address is fixed for the table's
 * life. */
#define HKV_HOST_SLAB_MAPPED_MAX (16ull << 30)

/* Wait for all work on the table and free it.  NULL is a no-op. */
hkv_status hkv_destroy(hkv_table* table);

/* Reader.  HKV Algorithm 1 (digest-accelerated find; two buckets in dual
 * mode).  For each i < n: if keys[i] is resident, found_out[i] = 1,
 * values_out[i*dim .. +dim) = its value row and, when scores_out != NULL,
 * scores_out[i] = its score; otherwise found_out[i] = 0 and the value and
 * score outputs of row i are left untouched.  The table is not modified. */
hkv_status hkv_find(hkv_table* table, uint64_t n, const uint64_t* keys, float* values_out,
                    uint8_t* found_out, uint64_t* scores_out, void* stream);

/* Inserter.  HKV Algorithm 2 (single mode) / Algorithm 3 (dual mode):
 * upsert with bucket-local admission and eviction.  A resident key gets the
 * new value and score unconditionally.  An absent key takes a free slot of
 * its bucket (dual mode: the less occupied candidate, ties to b1); when the
 * bucket is full (dual: both full) it replaces the lowest-ranked entry of the
 * bucket (dual: of the candidate whose lowest rank is lower) if it ranks
 * higher than that entry, else it is rejected.  Dual mode applies these rules
 * batch-wise as described under "Batches".
 *  scores  per-key scores (LFU policies: increments) or NULL; the score an
 *          entry receives follows the table's policy (see "Score
 *          policies"); under HKV_POLICY_CUSTOMIZED, NULL gives every key of
 *          the call the step counter.
 * Outcome totals accumulate in hkv_get_op_counts. */
hkv_status hkv_insert_or_assign(hkv_table* table, uint64_t n, const uint64_t* keys,
                                const float* values, const uint64_t* scores, void* stream);

/* Inserter, single-bucket tables only (HKV §7: the dual-bucket mode covers
 * insert_or_assign and find).  HKV §4.1 insert_and_evict: the same update as
 * hkv_insert_or_assign, and every entry that was resident before the call
 * and is displaced by it is written to evicted_keys_out / evicted_values_out
 * / evicted_scores_out (values and scores may be NULL) as it was when
 * displaced (a key updated by this call and then displaced carries its new
 * value and score), at consecutive positions in unspecified order;
 * *evicted_count_out (device) receives their number.  Outputs need room for
 * n entries.  Dual-mode tables return HKV_ERR_INVALID. */
hkv_status hkv_insert_and_evict(hkv_table* table, uint64_t n, const uint64_t* keys,
                                const float* values, const uint64_t* scores,
                                uint64_t* evicted_keys_out, float* evicted_values_out,
                                uint64_t* evicted_scores_out, uint64_t* evicted_count_out,
                                void* stream);

/* Inserter, single-bucket tables only.  HKV §4.1 find_or_insert (lookup
 * with insertion for cold start): absent keys are inserted with their row of
 * values_inout and the score the table's policy gives them under
 * HKV Algorithm 2; resident keys are not modified.  Afterwards, for each i:
 * when keys[i] is resident, found_out[i] = 1 and row i of values_inout holds
 * its stored value; otherwise (admission rejected it) found_out[i] = 0 and
 * row i is left unchanged.  Dual-mode tables return HKV_ERR_INVALID. */
hkv_status hkv_find_or_insert(hkv_table* table, uint64_t n, const uint64_t* keys,
                              float* values_inout, const uint64_t* scores, uint8_t* found_out,
                              void* stream);

/* Reader.  HKV §3.5 contains: found_out[i] = 1 iff keys[i] is resident.
 * Reads digests and keys only, no value row. */
hkv_status hkv_contains(hkv_table* table, uint64_t n, const uint64_t* keys, uint8_t* found_out,
                        void* stream);

/* Reader.  HKV §5.2-§5.3 find*: like hkv_find, but instead of copying a
 * resident key's value row, values_ptr_out[i] receives the device address of
 * the row inside the table (HBM, or the mapped host slab in tiered mode);
 * NULL on a miss.  The addresses stay valid until the next inserter call on
 * the table (insert_or_assign, insert_and_evict, find_or_insert, erase). */
hkv_status hkv_find_ptr(hkv_table* table, uint64_t n, const uint64_t* keys, float** values_ptr_out,
                        uint8_t* found_out, uint64_t* scores_out, void* stream);

/* Updater.  HKV §3.5: overwrites the value and the score of resident keys
 * in place; absent keys are ignored; nothing is inserted, evicted or moved.
 * The score follows the table's policy (see "Score policies"); under
 * HKV_POLICY_CUSTOMIZED with scores == NULL the scores are left as they are
 * and the step counter does not move. */
hkv_status hkv_assign(hkv_table* table, uint64_t n, const uint64_t* keys, const float* values,
                      const uint64_t* scores, void* stream);

/* Inserter.  HKV §3.5: removes each resident key; its slot becomes free. */
hkv_status hkv_erase(hkv_table* table, uint64_t n, const uint64_t* keys, void* stream);

/* Reader.  HKV §3.5 (size): number of resident entries, written to the host
 * variable *size_host.  Synchronises with `stream`. */
hkv_status hkv_size(hkv_table* table, uint64_t* size_host, void* stream);

/* Reader.  HKV §4.1 export_batch_if with the predicate score >= min_score
 * (the score-threshold dump of the DynamicEmb API page).  Scans slots
 * [slot_begin, slot_end) (slot = bucket * 128 + position, end clamped to the
 * capacity) and writes each matching entry to keys_out / values_out /
 * scores_out (values_out and scores_out may be NULL) at consecutive
 * positions in unspecified order.  *count_out (device) receives the number
 * written; outputs must have room for slot_end - slot_begin entries. */
hkv_status hkv_export(hkv_table* table, uint64_t slot_begin, uint64_t slot_end, uint64_t min_score,
                      uint64_t* keys_out, float* values_out, uint64_t* scores_out,
                      uint64_t* count_out, void* stream);

/* Cumulative counts since creation, read synchronously (waits for the
 * table's outstanding work).  reserved_keys: input keys skipped because they
 * were reserved sentinels.  timeouts: bounded device-side waits that ran out
 * (none in the default build; the pipelined measurement build counts a bucket
 * copy that did not arrive in time, then loads that bucket directly).
 * Returns HKV_ERR_TIMEOUT when timeouts > 0, else HKV_ERR_RESERVED_KEY when
 * reserved_keys > 0, else HKV_OK; the counts are written in every case. */
hkv_status hkv_get_error_counts(hkv_table* table, uint64_t* reserved_keys_host,
                                uint64_t* timeouts_host);

/* Cumulative outcome totals of insert_or_assign / assign / erase since
 * creation (or the last reset), read synchronously.  For insert_or_assign:
 * updated = resident keys overwritten; admitted = absent keys resident after
 * their call; rejected = absent keys not resident after their call; evicted =
 * keys resident before a call that it displaced.  assign adds to updated,
 * erase to erased. */
typedef struct hkv_op_counts {
  uint64_t updated, admitted, evicted, rejected, erased;
} hkv_op_counts;
hkv_status hkv_get_op_counts(hkv_table* table, hkv_op_counts* out_host);
hkv_status hkv_reset_op_counts(hkv_table* table);

/* Static facts about a table.  Value row r (r = bucket * 128 + slot) lives
 * at device address hbm_values_addr + r * dim * 4 when r < hbm_value_rows,
 * else at host_values_addr + (r - hbm_value_rows) * dim * 4 (the mapped host
 * slab of a tiered table; 0 when there is none), so a row address returned
 * by hkv_find_ptr maps back to its row and bucket. */
typedef struct hkv_info {
  uint64_t capacity, num_buckets, hbm_value_rows;
  uint32_t dim, mode;
  int device;
  uint64_t hbm_values_addr, host_values_addr;
} hkv_info;
hkv_status hkv_get_info(hkv_table* table, hkv_info* out_host);

/* Set the table's 32-bit epoch (HKV §3.3 epoch-aware scoring; see "Score
 * policies").  Calls issued afterwards use it; calls already issued keep the
 * epoch they were issued with.  Any policy accepts it; only the EPOCH
 * policies read it.  Errors: INVALID (NULL table). */
hkv_status hkv_set_epoch(hkv_table* table, uint32_t epoch);

/* insert_or_assign for callers that cannot let the library allocate.
 *
 * The paper has no counterpart: this is a deployment variant of
 * hkv_insert_or_assign with the same arguments and the same results.  That
 * call takes its per-call working memory from a stream-ordered pool; this
 * one uses a fixed array of HKV_NOALLOC_SCRATCH_BYTES compiled into the
 * library, for callers whose device memory is already handed out (e.g. to a
 * framework's caching allocator), who keep a fixed memory budget, or whose
 * serving loop must never enter cudaMalloc/cudaFree (which can synchronise
 * the device).  It calls no allocation routine.
 *  - Limit: the batch's working memory must fit the array, i.e.
 *      a(8M) + a(4M) + 256 + a(B) bytes in single mode and
 *      2 a(8M) + 3 a(4M) + a(M) + 256 + a(4n) + a(B) bytes in dual mode,
 *    plus a(8M) under the LFU policies (2 a(8M) in dual mode), with M the
 *    smallest power of two >= max(64, 2n), B the bucket count and a(x) = x
 *    rounded up to a multiple of 256.  Larger batches return HKV_ERR_INVALID and enqueue
 *    nothing (split them, or use hkv_insert_or_assign).  In single mode that
 *    is up to 2^20 keys per call for tables of at most 2^23 - 256 buckets,
 *    and up to 2^19 keys under the LFU policies for tables of at most
 *    12 * 2^20 - 256 buckets; a call of 2^20 + 1 keys (2^19 + 1 under LFU)
 *    is refused on any table.
 *  - Sharing: every call on every table of a device uses the same array and
 *    clears it before use.  Calls whose kernels overlap on the GPU (on
 *    different streams, from any table) race on it and corrupt each other's
 *    results: keep such calls on one stream, or order them with events.
 *  - Ordering on the table: as for hkv_insert_or_assign (an inserter), using
 *    CUDA events the table created with it, so later calls on other streams,
 *    hkv_get_op_counts and hkv_destroy wait for this one.
 *  - Set-up: the first call on a device (made with any table of that device)
 *    looks up the array's device address with cudaGetSymbolAddress and keeps
 *    it for the life of the process; make that first call before any stream
 *    capture.  cudaDeviceReset on that device destroys its tables and may
 *    move the array; do not call this function on that device afterwards. */
#define HKV_NOALLOC_SCRATCH_BYTES (32ull << 20)
hkv_status hkv_insert_or_assign_noalloc(hkv_table* table, uint64_t n, const uint64_t* keys,
                                        const float* values, const uint64_t* scores, void* stream);

/* ---------------------------------------------------------------------------
 * Operators on looked-up rows.
 *
 * A training step on a table's rows runs find -> 4-bit copies -> products ->
 * loss and gradient -> norm and clipping -> assign; a serving step scores
 * hidden states against 4-bit copies of rows.  With an adapter for each user, a
 * row of the table, the adapters' product goes onto the shared one, and log
 * probabilities of the answers are taken from their logits.  The calls below are
 * the steps between the table's own.  They take no table: they run on the current
 * device, which must be the device of `stream`, are asynchronous, allocate
 * nothing, keep nothing between calls and may be captured into a CUDA graph.
 * Argument errors are found on the host and enqueue nothing.  All matrices
 * are row-major; a stride is the number of elements from one row to the next
 * (at least the row length).  Rows, columns and counts are at most
 * HKV_MAX_BATCH; element offsets are 64 bits wide.  Results do not depend on
 * scheduling: no sum is taken in the order of atomics. */

/* Element types of the operators' buffers. */
enum { HKV_F32 = 0, HKV_BF16 = 1, HKV_F16 = 2 };

/* Microscaled 4-bit matrices (OCP microscaling formats, MXFP4).  A row is cut
 * into blocks of 32 columns.  A block's scale byte s stands for 2^(s - 127),
 * s = max(E - 2, 0) with E the biased exponent of the block's largest
 * magnitude as a float32 (0 for zero and subnormals); an element is the
 * nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (e2m1, with a sign) to x / scale,
 * ties to the even code, 6 above the range.  A block that holds a NaN or an
 * infinity has s = 255 and stands for 32 NaNs (its codes are 0).
 *  codes   rows x ceil(cols / 32) x 16 bytes, two codes a byte, the lower
 *          column in the low half; columns past `cols` are 0.
 *  scales  ceil(rows / 128) x ceil(cols / 128) groups of 512 bytes, one group
 *          for 128 rows by 4 blocks, byte (r % 32) * 16 + (r / 32 % 4) * 4 +
 *          block % 4 of it for row r; bytes of rows and blocks past the
 *          matrix are 0.
 * Both 16-byte aligned. */
#define HKV_MX_BLOCK 32
#define HKV_MX_CODE_BYTES(rows, cols) ((uint64_t)(rows) * (((uint64_t)(cols) + 31) / 32) * 16)
#define HKV_MX_SCALE_BYTES(rows, cols) \
  ((((uint64_t)(rows) + 127) / 128) * (((uint64_t)(cols) + 127) / 128) * 512)

/* The 4-bit copy of x (rows x cols, float32, bfloat16 or float16): of its
 * rows (codes, scales), of its columns (codes_t, scales_t: the copy of the
 * cols x rows transpose, blocks running along x's rows), or both from one
 * read.  Pass NULL for both pointers of a copy that is not wanted; at least
 * one copy is.  The products of a backward pass need the copies along the
 * other axis: dX = dY W takes the rows of dY and the columns of W, and
 * dW = dY^T X the columns of dY and of X. */
hkv_status hkv_mx_quantize(uint64_t rows, uint64_t cols, const void* x, int x_type,
                           uint64_t x_stride, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                           uint8_t* scales_t, void* stream);

/* The values a 4-bit matrix stands for, exact in float32 and bfloat16
 * (float16: rounded, infinite past its range). */
hkv_status hkv_mx_dequantize(uint64_t rows, uint64_t cols, const uint8_t* codes,
                             const uint8_t* scales, void* y, int y_type, uint64_t y_stride,
                             void* stream);

/* y (m x n) = A B^T for 4-bit matrices A (m x k) and B (n x k): products of
 * elements are exact, sums are taken in float32, y is rounded once.  k = 0
 * gives zeros.  A block of NaNs makes its whole row (A) or column (B) of y
 * NaN. */
hkv_status hkv_mx_matmul(uint64_t m, uint64_t n, uint64_t k, const uint8_t* a_codes,
                         const uint8_t* a_scales, const uint8_t* b_codes, const uint8_t* b_scales,
                         void* y, int y_type, uint64_t y_stride, void* stream);

/* Preference loss over pairs of token sequences (the logistic loss of paired
 * log ratios), from logits.  `logits` holds one row of `vocab` logits for
 * each of `rows` tokens.  Sequence s has rows offsets[s] .. offsets[s + 1]
 * (offsets: device, 2 * pairs + 1 ascending values in 0 .. rows); sequence p
 * is the chosen and sequence pairs + p the rejected one of pair p.  A token
 * whose label lies outside 0 .. vocab - 1 is not counted: its logits have no
 * effect, whatever they hold.  Banned entries may hold -inf or any finite
 * number; a counted row that holds a NaN or +inf, or nothing above -inf, gives
 * NaN.  For counted tokens
 *   logps[t]  = logits[t][labels[t]] - lse[t],  lse[t] = log sum exp logits[t]
 *   ratios[s] = sum of logps[t] - ref_logps[t] over the counted tokens of s,
 *               divided by their number when `average` is not 0 (0 for a
 *               sequence without counted tokens; ref_logps NULL: zeros)
 *   h         = beta * (ratios[p] - ratios[pairs + p])
 *   losses[p] = -(1 - label_smoothing) log sigmoid(h)
 *               - label_smoothing log sigmoid(-h)
 * logps is 0 for tokens that are not counted.  Sums are taken in float32, so
 * ratios of logits near that type's range may overflow to infinities.  For the
 * backward call the forward call also writes row_grad[t] = d losses[p] /
 * d logps[t] (0 for tokens that are not counted or lie in no sequence) and
 * row_pair[t] = p (-1 in no sequence).  beta is finite,
 * 0 <= label_smoothing <= 1. */
hkv_status hkv_preference_loss(uint64_t pairs, uint64_t rows, uint64_t vocab, const void* logits,
                               int type, uint64_t stride, const int64_t* labels,
                               const int64_t* offsets, const float* ref_logps, float beta,
                               float label_smoothing, int average, float* losses, float* ratios,
                               float* logps, float* lse, float* row_grad, int32_t* row_pair,
                               void* stream);

/* Gradient of sum_p dlosses[p] * losses[p] with respect to the logits
 * (dlosses NULL: ones), in the logits' type:
 *   dlogits[t][v] = g (1[v = labels[t]] - exp(logits[t][v] - lse[t])),
 *   g = dlosses[row_pair[t]] * row_grad[t]
 * and zeros for a token that is not counted or lies in no sequence.  Where
 * lse[t] is too large for one float to give the exponent (1024 or more in
 * magnitude: a row whose mask leaves nothing), the row's softmax is taken from
 * its maximum.  dlogits may be the logits' own buffer with the same stride, and
 * must not overlap them otherwise. */
hkv_status hkv_preference_loss_backward(uint64_t pairs, uint64_t rows, uint64_t vocab,
                                        const void* logits, int type, uint64_t stride,
                                        const int64_t* labels, const float* lse,
                                        const float* row_grad, const int32_t* row_pair,
                                        const float* dlosses, void* dlogits, uint64_t dstride,
                                        void* stream);

/* Log probabilities of given tokens, with the entropy and the largest entries
 * of their rows of logits.  `logits` holds one row of `vocab` logits for each
 * of `rows` tokens.  A token whose label lies outside 0 .. vocab - 1 is not
 * counted: its logits have no effect, whatever they hold, its logps and
 * entropy are 0, its top_ids -1 and its top_logps -inf.  With labels NULL (and
 * logps NULL) every row is counted.  For counted tokens
 *   logps[t]        = logits[t][labels[t]] - lse[t],  lse[t] = log sum exp logits[t]
 *   entropy[t]      = -sum_v p_v log p_v,  log p_v = logits[t][v] - lse[t]
 *   top_ids[t][j]   = the j-th largest entry's index, of equal ones the lower
 *                     first (-0 equals 0), j < top
 *   top_logps[t][j] = its log p
 * Entries may hold -inf or any finite mask (log p -inf, and 0 to the entropy);
 * a counted row that holds a NaN or +inf, or nothing above -inf, gives NaNs and
 * top_ids of -1.  For the backward call lse (NULL where it is not wanted) gets
 * two floats for each row, lse[t] and what that float leaves out of it.  top is
 * at most HKV_MAX_TOP (the lanes of a warp, whose maxima bound it) and at most
 * vocab. */
#define HKV_MAX_TOP 32
hkv_status hkv_token_logps(uint64_t rows, uint64_t vocab, const void* logits, int type,
                           uint64_t stride, const int64_t* labels, uint32_t top, float* logps,
                           float* entropy, float* top_logps, int64_t* top_ids, float* lse,
                           void* stream);

/* Gradient of sum_t dlogps[t] * logps[t] + dentropy[t] * entropy[t] with
 * respect to the logits (either may be NULL: zeros), in their type:
 *   dlogits[t][v] = dlogps[t] (1[v = labels[t]] - p_v)
 *                   - dentropy[t] p_v (log p_v + entropy[t])
 * and zeros for a token that is not counted.  labels, lse and entropy are the
 * forward call's.  dlogits may be the logits' own buffer with the same stride,
 * and must not overlap them otherwise. */
hkv_status hkv_token_logps_backward(uint64_t rows, uint64_t vocab, const void* logits, int type,
                                    uint64_t stride, const int64_t* labels, const float* lse,
                                    const float* entropy, const float* dlogps, const float* dentropy,
                                    void* dlogits, uint64_t dstride, void* stream);

/* Low-rank adapters: `count` pairs of thin matrices of `type` (the call's),
 * down (rank x k) and up (n x rank).  Adapter a's row r starts a * down_step +
 * r * down_stride (up: up_step, up_stride) elements in, so that an adapter may
 * be a row of a larger buffer, as of a table's rows.  scales (device) has a
 * float32 factor for each adapter, NULL: 1.  1 <= rank <= HKV_MAX_RANK; strides
 * are at most 2^31, steps at most 2^40.  (64 ranks: a tile's sums by all ranks stay
 * in a warp's registers and both factors' stages in shared memory.) */
#define HKV_MAX_RANK 64
typedef struct hkv_adapters {
  uint64_t count;
  const void* down;
  uint64_t down_step, down_stride;
  const void* up;
  uint64_t up_step, up_stride;
  const float* scales;
  uint32_t rank;
} hkv_adapters;

/* Adapters of many requests beside a shared projection.  Request s has the rows
 * offsets[s] .. offsets[s + 1] - 1 of x (tokens x k) and of y (tokens x n), and
 * the adapter which[s] (offsets, which: device, requests + 1 ascending values in
 * 0 .. tokens, and requests values):
 *   h[t] = scale * down x[t]          y[t] = base[t] + up h[t]
 * with sums in float32 and y rounded once.  base (NULL: zeros) may be y itself,
 * with the same stride.  Rows of no request, and of one whose which[s] lies
 * outside 0 .. count - 1, have y[t] = base[t]; where y is base they are left as
 * they are.  y must not overlap base otherwise, nor x, the adapters or the requests
 * (columns of one buffer side by side do not).  hidden (device memory of
 * HKV_ADAPTER_HIDDEN_BYTES, 16-byte aligned, which overlaps nothing else) gets h for
 * the backward call; of h, 16 digits go on for 16-bit matrices, 24 for float32.  A row with an infinity in it may give NaN where the
 * formula gives an infinity.  `adapters` is read before the call returns. */
#define HKV_ADAPTER_HIDDEN_BYTES(tokens, rank, type) \
  ((uint64_t)(tokens) * ((rank) <= 16 ? 16 : (rank) <= 32 ? 32 : 64) * ((type) == HKV_F32 ? 6 : 4))
hkv_status hkv_adapter_matmul(uint64_t tokens, uint64_t k, uint64_t n, int type,
                              const hkv_adapters* adapters, uint64_t requests,
                              const int64_t* offsets, const int64_t* which, const void* x,
                              uint64_t x_stride, const void* base, uint64_t base_stride, void* y,
                              uint64_t y_stride, void* hidden, void* stream);

/* Its gradients, from dy (tokens x n) and the forward call's x and hidden:
 *   dh[t]    = scale * up^T dy[t]     dx[t] = base[t] + down^T dh[t]
 *   ddown[a] = sum over the rows t of a's requests of dh[t] x[t]^T
 *   dup[a]   = sum of dy[t] h[t]^T
 * (base, tokens x k: as above).  ddown (count x rank x k) and dup (count x n x
 * rank) are contiguous, in the matrices' type, rounded once, and zero for an
 * adapter of no request; either may be NULL.  dhidden is scratch like hidden, of its
 * own.  dx must not overlap x or dy, nor base unless it is base; ddown, dup and dhidden
 * must not overlap one another or anything else.  Every adapter's blocks read all of
 * which: beyond some thousands of adapters and requests that is most of the time, and
 * it grows with their product. */
hkv_status hkv_adapter_matmul_backward(uint64_t tokens, uint64_t k, uint64_t n, int type,
                                       const hkv_adapters* adapters, uint64_t requests,
                                       const int64_t* offsets, const int64_t* which, const void* x,
                                       uint64_t x_stride, const void* dy, uint64_t dy_stride,
                                       const void* hidden, const void* base, uint64_t base_stride,
                                       void* dx, uint64_t dx_stride, void* ddown, void* dup,
                                       void* dhidden, void* stream);

/* One gradient: n elements of `type` at `data`.  Where `out` is not NULL the
 * clipped gradient is written there as `out_type`; it may be `data` itself
 * with the same type, and must not overlap it otherwise, nor another gradient
 * of the call or its out (HKV_ERR_INVALID; a gradient is listed once). */
typedef struct hkv_grad {
  const void* data;
  void* out;
  uint64_t n;
  int32_t type, out_type;
} hkv_grad;

/* Global norm of `count` gradients and clipping to it:
 *   *norm_out = sqrt(sum over all gradients and elements of g^2)   (device)
 *   out       = f * g, f = 1 if *norm_out <= max_norm, else max_norm / *norm_out
 * An infinite norm gives f = 0 and a NaN norm f = NaN (and nothing is added to
 * the norm that max_norm is divided by, as some libraries do).  Where f is 1, out
 * is data and the types agree, nothing is written.  `grads` is a host array,
 * read before the call returns.  `work` is device memory of
 * HKV_CLIP_WORK_BYTES (4-byte aligned) that no other call uses meanwhile.
 * Squares are summed in float32: their sum is infinite from 3.4e38 on, and
 * elements below 1e-19 lose digits of theirs, all of them below 1e-23.  The sum's
 * order depends on the sizes, on the tensors' addresses within 32 bytes and on
 * the number of SMs.  max_norm is not negative. */
#define HKV_CLIP_WORK_BYTES 16384
hkv_status hkv_clip_grad_norm(uint64_t count, const hkv_grad* grads, float max_norm,
                              float* norm_out, void* work, void* stream);

/* Bounded device-side waits of the operators that ran out since the library
 * was loaded, on the current device (0 unless the device failed); such a call
 * returned without complete results.  Waits for the device's outstanding
 * work.  Returns HKV_ERR_TIMEOUT when the count is not 0. */
hkv_status hkv_get_wait_timeouts(uint64_t* timeouts_host);

/* Human-readable name of a status code (static storage). */
const char* hkv_status_string(hkv_status status);

#ifdef __cplusplus
}
#endif

#endif /* HKV_H_ */
