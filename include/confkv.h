/*
 * confkv.h -- C ABI of the CONF-KV per-decode-step cache manager for one
 * NVIDIA GB300 (sm_103a).
 *
 * The method: CONF-KV, "Confidence-Aware KV Cache Eviction with
 * Mixed-Precision Storage for Long-Horizon LLM".  Citations name the page and
 * the section they come from:
 *   [rainbus]  paper.rainbus.top/paper/2605.24786 -- sections 核心方法 (core
 *              method), 方法步骤详情 (Algorithm 1, steps 1-13), 前置知识
 *              (prerequisites: EMA, blockwise online softmax), 复现评估
 *              (reproducibility: hyper-parameters).
 *   [gist-de]  gist.science/de/paper/2605.24786 -- Technischer
 *              Zusammenfassung, Methodik: Konfidenzschätzung, Adaptive
 *              Budgetauswahl, Token-Ranking und Eviktion, Systemintegration.
 *
 * Conventions
 *   - Every function returns a status: CONFKV_OK (0) or a negative code below.
 *     Nothing aborts, traps or exits the process.
 *   - All tensor arguments of confkv_prefill / confkv_step are DEVICE
 *     pointers owned by the caller; the library reads inputs and writes
 *     outputs and keeps no reference after the call returns.  The only device
 *     memory the library uses is the caller-allocated workspace (see
 *     confkv_workspace_bytes); it never calls cudaMalloc itself.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Device work is enqueued on it and the call returns without
 *     synchronising, except where a function says it synchronises.
 *   - Device-side anomalies (an INT8 region that would overflow, an
 *     inconsistent eviction count) set bits of a device status word; they are
 *     reported as CONFKV_EDEVICE by the next confkv_get_stats.
 *   - Layouts are row-major, outermost index first.  L layers, B sequences,
 *     Hq query heads, Hkv KV heads, d head dim (64 or 128), V vocabulary.
 */
#ifndef CONFKV_H
#define CONFKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CONFKV_OK 0
#define CONFKV_EINVAL (-1)     /* bad argument or configuration */
#define CONFKV_ECAPACITY (-2)  /* a cache region or output buffer is too small */
#define CONFKV_ECUDA (-3)      /* a CUDA runtime call failed */
#define CONFKV_ETIMEOUT (-4)   /* a bounded device wait gave up */
#define CONFKV_ENOTIMPL (-5)   /* shape not supported by the compiled kernels */
#define CONFKV_EDEVICE (-6)    /* the device status word reports an error */
#define CONFKV_ESTATE (-7)     /* call out of order (e.g. step before prefill) */

#define CONFKV_Q_FP16 0
#define CONFKV_Q_BF16 1

/* Element types of the calls that take a dtype (the first two are the query
 * types above). */
#define CONFKV_FP16 0
#define CONFKV_BF16 1
#define CONFKV_FP32 2

/*
 * Configuration.  Defaults on the pages: w = (0.4, 0.3, 0.3) and tau = 0.7
 * ([gist-de] Konfidenzschätzung; [rainbus] 核心方法), alpha = 0.65
 * ([rainbus] 核心方法), lambda = 0.9 ([rainbus] 前置知识, EMA), P = 32 or 64,
 * W = 128 ([rainbus] 复现评估).
 */
typedef struct confkv_config {
  int32_t L, Hq, Hkv, d, V;   /* layers, query heads, KV heads, head dim, vocab */
  int32_t B;                  /* sequences stepped together */
  int32_t cap;                /* INT8 slots per (layer, sequence): must hold the
                                 prefill older than W and every budget + 1;
                                 rounded up to a multiple of 16 */
  int32_t W;                  /* FP16 window: the newest W tokens stay FP16 */
  int32_t P;                  /* protected window: the newest P tokens are never
                                 evicted ([gist-de] Token-Ranking und Eviktion) */
  int32_t q_dtype;            /* CONFKV_Q_FP16 or CONFKV_Q_BF16 */
  int32_t max_evict;          /* rows of evicted_pos per (layer, sequence);
                                 0 selects cap + W + 16 */
  double tau;                 /* budget threshold: N = n_high if c >= tau */
  double w_H, w_m, w_p;       /* confidence weights */
  float alpha;                /* rank weight of the EMA mass */
  float lam;                  /* EMA decay */
  const int32_t* n_high;      /* host [L]: tight budget per layer (c >= tau) */
  const int32_t* n_low;       /* host [L]: loose budget per layer (c < tau);
                                 per-layer values give the pyramidal variant
                                 ([gist-de] Systemintegration) */
  int32_t compaction;         /* CONFKV_COMPACT_TAIL_FILL (0, default): each
                                 evicted INT8 slot below the new length takes a
                                 survivor from above it (at most k moves);
                                 CONFKV_COMPACT_ORDERED (1): survivors keep
                                 position order (every survivor above the first
                                 hole moves), the contiguous compaction of
                                 [gist-de] Systemintegration, kept as an
                                 ablation of the layout */
} confkv_config;

enum { CONFKV_COMPACT_TAIL_FILL = 0, CONFKV_COMPACT_ORDERED = 1 };

typedef struct confkv_ctx confkv_ctx;

/* Bytes of device workspace the context needs (state + scratch).  Returns
 * CONFKV_EINVAL for an invalid configuration: d not 64/128, Hq % Hkv != 0,
 * Hq / Hkv > 8, V < 2 or V > 4096 * 1024, some budget < P or < 1, cap < 16,
 * W < 1, compaction not 0 or 1. */
int confkv_workspace_bytes(const confkv_config* cfg, size_t* bytes);

/* Create a context over `workspace` (device memory, >= the size above, 256-byte
 * aligned, owned by the caller and kept alive until confkv_destroy).  The
 * context copies the configuration, including n_high / n_low.  Synchronous. */
int confkv_create(const confkv_config* cfg, void* workspace, size_t workspace_bytes,
                  confkv_ctx** out);

/* Free the host-side context (the workspace stays the caller's). */
void confkv_destroy(confkv_ctx* ctx);

/*
 * Ingest the prefill and reset the cache.  k, v: device fp16
 * [L][B][Hkv][t_max][d]; sequence b uses its first prefill_len[b] tokens
 * (prefill_len is a HOST array of B values, 0 <= prefill_len[b] <= t_max).
 * Scales per (layer, sequence, KV head, channel) from the absmax over the
 * prefill: s = absmax / 127 in float32 (1 if the channel is zero).  Positions
 * >= prefill_len - W stay FP16; older positions are stored as INT8 codes
 * clamp(rint(x / s), -127, 127) ([gist-de] Systemintegration; the pages do
 * not describe prefill, this rule follows their per-head per-channel INT8).
 * EMA mass starts at 0.  Returns CONFKV_ECAPACITY if prefill_len - W > cap,
 * CONFKV_EINVAL if k or v is not 2-byte aligned.
 */
int confkv_prefill(confkv_ctx* ctx, const int32_t* prefill_len, const void* k, const void* v,
                   int64_t t_max, void* stream);

/*
 * Prefill by layer: the same cache as confkv_prefill, from what a model has
 * in hand while it runs its prompt -- one layer's K/V of all sequences, rows
 * packed without padding -- so that no layer's K/V has to be kept.
 *   confkv_prefill_begin  resets the cache and fixes the prompt lengths
 *       (HOST array of B).  Until every layer is written the context is not
 *       prefilled: confkv_step, confkv_read_layer, confkv_import_unit,
 *       confkv_set_clock and confkv_export_unit of a layer not yet written
 *       return CONFKV_ESTATE.  CONFKV_ECAPACITY if a length
 *       minus W exceeds cap.
 *   confkv_prefill_layer  writes layer `layer`: k, v device [rows][Hkv][d],
 *       rows = the sum of the lengths, sequence b's rows after those of
 *       b - 1; dtype CONFKV_FP16 or CONFKV_BF16 (converted to fp16 first).
 *       Scales, codes and window are those of confkv_prefill on the same
 *       values.  Layers in any order; one written twice keeps the last.
 *       CONFKV_ESTATE outside confkv_prefill_begin .. last layer.
 * Strides are in elements, row first, then KV head; channels are contiguous;
 * base addresses are multiples of 16 bytes and strides of 8 elements.  With
 * rows = 0, k, v and the strides may be NULL.  Both calls are asynchronous on
 * `stream` and refuse stream capture (CONFKV_ESTATE), like every call that
 * changes the host's bounds.
 */
int confkv_prefill_begin(confkv_ctx* ctx, const int32_t* prefill_len, void* stream);
int confkv_prefill_layer(confkv_ctx* ctx, int32_t layer, const void* k, const void* v, int32_t dtype,
                         const int64_t* k_stride, const int64_t* v_stride, void* stream);

/*
 * The resident entries of one layer as packed K/V, dequantised on the device
 * (confkv_export_unit gives codes and scales to the host): for attention of
 * further prompt tokens over a cache, or for handing a sequence on.  Entries
 * of further tokens go into the cache by confkv_step only: a prefill starts it
 * anew.
 *   k, v       device [rows][Hkv][d], dtype CONFKV_FP16 or CONFKV_BF16:
 *              fp16 window entries converted, INT8 entries code * scale in
 *              fp32, then rounded to dtype
 *   positions  device int32 [rows]: absolute position of each row
 *   cu         device int32 [B + 1], written: sequence b has rows cu[b] ..
 *              cu[b+1]-1, INT8 entries in slot order (by position until the
 *              first eviction), then the window by position
 *   rows       rows the buffers hold; confkv_read_rows gives a bound that
 *              always suffices (exact until the first step).  Entries beyond
 *              `rows` are dropped and set CONFKV_STATUS_CAPACITY; rows behind
 *              the last sequence are not written.
 * Strides as in confkv_prefill_layer.  Needs a prefilled context (else
 * CONFKV_ESTATE); asynchronous on `stream`, may be captured.
 */
int confkv_read_rows(confkv_ctx* ctx, int64_t* rows);
int confkv_read_layer(confkv_ctx* ctx, int32_t layer, int32_t dtype, void* k, void* v, const int64_t* k_stride,
                      const int64_t* v_stride, int32_t* positions, int32_t* cu, int64_t rows, void* stream);

/*
 * One decode step for all B sequences: the token at position
 * t_b = prefill_len[b] + (steps done since prefill) ([rainbus] 方法步骤详情,
 * Algorithm 1):
 *   q      [L][B][Hq][d]  fp16 or bf16 (q_dtype): the decode query
 *   k_new  [L][B][Hkv][d] fp16, v_new likewise: the new token's K/V
 *   logits [B][V] fp32: next-token logits (temperature 1)
 * Outputs (device):
 *   out         [L][B][Hq][d] fp32: attention of q over the cache plus the new
 *               token, before any eviction of this step
 *   budget      [B][L] int32: N chosen for (sequence, layer)
 *   confidence  [B] fp32 or NULL: c of each sequence
 *   evicted_pos [L][B][max_evict] int32: absolute positions evicted by this
 *               step, ascending; only the first n_evicted[l][b] entries of a
 *               row are written
 *   n_evicted   [L][B] int32
 * The step computes c = w_H(1 - H/log V) + w_m sigmoid(log p1 - log p2) +
 * w_p p1, N = n_high if c >= tau else n_low, attention with the per-token
 * attention mass averaged over query heads, the EMA a <- lam a + (1 - lam) A,
 * and, if the cache holds more than N entries (the new token not counted),
 * evicts the n - N lowest s = alpha a_hat + (1 - alpha) r_hat among entries
 * older than the newest P, compacts the INT8 region, requantises the entry
 * that leaves the FP16 window and appends the new token.
 * Alignment: q must be 16-byte aligned (the attention kernel copies query
 * rows with bulk copies), k_new and v_new 4-byte aligned (read as 32-bit
 * words), logits, out, budget, confidence, evicted_pos and n_evicted 4-byte
 * aligned; otherwise CONFKV_EINVAL, before anything is launched.  Tensors
 * from a torch allocation or a contiguous slice at a multiple of 8 elements
 * satisfy all of these.
 * Returns CONFKV_ECAPACITY (before launching anything) if the worst case of
 * this step could overflow cap or max_evict.
 */
int confkv_step(confkv_ctx* ctx, const void* q, const void* k_new, const void* v_new,
                const float* logits, float* out, int32_t* budget, float* confidence,
                int32_t* evicted_pos, int32_t* n_evicted, void* stream);

/*
 * confkv_step with HOST buffers (same shapes); returns once the outputs are
 * in the host buffers.  Two modes, chosen per call, with identical results:
 *  - mapped: when k_new, v_new, logits and every output buffer lie in
 *    page-locked host memory the device can address (cudaHostAlloc,
 *    cudaMallocHost or cudaHostRegister), the kernels read those inputs and
 *    write those outputs in place over the host link.  Only q is copied, to
 *    a staging buffer inside the workspace, on a second library-owned
 *    stream (created on the first call) while the first kernel runs.
 *  - staged: otherwise every input is copied to staging buffers inside the
 *    workspace first, and the outputs are copied back (the attention output
 *    on the second stream while the last kernel runs).  Pinned memory makes
 *    these copies asynchronous DMA.
 * Mapped mode also needs k_new and v_new 4-byte aligned and every other
 * buffer but q 4-byte aligned; misaligned pinned buffers take the staged
 * mode.  q has no alignment requirement here (it is always staged).
 * confidence may be NULL.  Of each row of evicted_pos only the first
 * n_evicted entries are meaningful; in mapped mode only those are written,
 * in staged mode as many as the step's worst-case eviction count are copied
 * back.  The rest of the row is untouched.
 */
int confkv_step_host(confkv_ctx* ctx, const void* q, const void* k_new, const void* v_new,
                     const float* logits, float* out, int32_t* budget, float* confidence,
                     int32_t* evicted_pos, int32_t* n_evicted, void* stream);

/* CUDA graphs.  The step index lives in device memory, so the three kernels
 * of a confkv_step captured into a CUDA graph (stream capture on `stream`)
 * replay correctly step after step.  The host still keeps worst-case bounds
 * (capacity, eviction rows, attention launch shape), so replays go inside a
 * reservation:
 *   confkv_graph_reserve(ctx, n)  checks that n more steps fit under the
 *       worst-case bounds and pins one attention launch shape valid for all
 *       of them.  CONFKV_ECAPACITY if they do not fit, CONFKV_ESTATE before
 *       prefill, CONFKV_EINVAL if n < 1.
 *   confkv_step under capture then records a step without running it and
 *       without advancing the host state; under capture without a
 *       reservation it returns CONFKV_ESTATE.  confkv_step_host is never
 *       captured (CONFKV_ESTATE).
 *   confkv_graph_advance(ctx, k)  accounts for k executed replays (k at most
 *       the steps left in the reservation, else CONFKV_ESTATE).  Plain
 *       confkv_step calls inside a reservation use the pinned shape and
 *       count against it as well.
 *   confkv_graph_release(ctx)  drops the reservation (prefill and
 *       confkv_import_unit drop it too).
 * The pages have no counterpart of these calls: they serve callers that put
 * the cache manager into their own decode graph. */
int confkv_graph_reserve(confkv_ctx* ctx, int64_t steps);
/* Self-test of failure detection: launches one CTA that waits on an mbarrier
 * nothing ever arrives on, with the decode kernels' polling loop but a short
 * limit (4096 polls).  The wait runs out and sets the time-out bit
 * (CONFKV_STATUS_TIMEOUT) of the device status word, which the next
 * confkv_get_stats reports as CONFKV_EDEVICE; nothing faults and the context
 * stays usable (confkv_prefill clears the word).  Asynchronous on `stream`.
 * The pages have no counterpart: it tests this library's own bounded waits. */
int confkv_selftest_timeout(confkv_ctx* ctx, void* stream);
int confkv_graph_advance(confkv_ctx* ctx, int64_t steps);
int confkv_graph_release(confkv_ctx* ctx);

/* Cache of one (sequence b, layer l) in a plain host layout.  Caller-owned
 * buffers sized for cap INT8 entries and W + 16 FP16 entries:
 *   pos8[cap], ema8[cap], k8/v8[cap][Hkv][d] int8 codes,
 *   posR[W+16], emaR[W+16], k16/v16[W+16][Hkv][d] fp16 bit patterns,
 *   sK, sV [Hkv][d] fp32 scales.
 * INT8 entries are listed in slot order, FP16 entries in ring-slot order. */
typedef struct confkv_unit_host {
  int32_t n8, nR;
  int32_t* pos8;
  float* ema8;
  int8_t* k8;
  int8_t* v8;
  int32_t* posR;
  float* emaR;
  uint16_t* k16;
  uint16_t* v16;
  float* sK;
  float* sV;
} confkv_unit_host;

/* Copy the cache of (b, l) to host (synchronises `stream`).  CONFKV_ESTATE
 * before a prefill, and for a layer that a prefill by layer has yet to write. */
int confkv_export_unit(confkv_ctx* ctx, int32_t b, int32_t l, confkv_unit_host* out, void* stream);

/* Overwrite the cache of (b, l) from host buffers in the export layout
 * (synchronises `stream`).  FP16 entries go to ring slot pos mod (W + 16);
 * two entries must not share a slot.  Used to resume from a checkpoint or to
 * load a crafted state.  The first import into a context that was not
 * prefilled empties all other units; its clock is at 0 or where
 * confkv_set_clock put it. */
int confkv_import_unit(confkv_ctx* ctx, int32_t b, int32_t l, const confkv_unit_host* in,
                       void* stream);

/* Position clock: prefill_len[B] (host) and the number of steps done since
 * prefill.  confkv_set_clock restores it with a checkpoint. */
int confkv_get_clock(confkv_ctx* ctx, int32_t* prefill_len, int64_t* steps);
int confkv_set_clock(confkv_ctx* ctx, const int32_t* prefill_len, int64_t steps, void* stream);

/* Bits of the device status word (confkv_stats.device_status). */
enum {
  CONFKV_STATUS_CAPACITY = 1,     /* an INT8 region would have overflowed cap */
  CONFKV_STATUS_EVICT_BOUND = 2,  /* more evictions than evicted_pos rows hold */
  CONFKV_STATUS_BAD_COUNT = 4,    /* eviction count differs from n - N */
  CONFKV_STATUS_TIMEOUT = 8       /* a bounded wait inside a kernel gave up */
};

typedef struct confkv_stats {
  int64_t steps;             /* steps since prefill */
  int64_t evicted;           /* entries evicted since prefill */
  int64_t moved;             /* entries moved by compaction */
  int64_t requantised;       /* entries moved from FP16 to INT8 */
  double attn_bytes;         /* algorithmic bytes of the attention kernel, summed */
  double step_bytes;         /* algorithmic bytes of whole steps, summed */
  int64_t resident;          /* cache entries resident now, all units */
  int64_t resident_bytes;    /* K/V bytes resident now at stored widths */
  int32_t device_status;     /* raw device status bits (0 = ok) */
  int64_t host_h2d_bytes;    /* bytes the last confkv_step_host moved host -> device */
  int64_t host_d2h_bytes;    /* bytes the last confkv_step_host moved device -> host */
  int64_t peak_resident;     /* largest `resident` seen at the end of any step since
                                prefill (exact: summed on the device every step) */
  int64_t peak_resident_bytes; /* largest `resident_bytes` at the end of any step
                                since prefill (the pages' peak KV memory, [rainbus]
                                results table) */
  int64_t workspace_bytes;   /* device bytes the context holds: the caller's
                                workspace (the allocator footprint; fixed at create) */
  int64_t launches;          /* kernels this context has launched for decode steps
                                since it was created (host count) */
} confkv_stats;

/* Read the counters and the device status word (synchronises `stream`).
 * Returns CONFKV_EDEVICE if the status word is non-zero. */
int confkv_get_stats(confkv_ctx* ctx, confkv_stats* out, void* stream);

/* Per-kernel timing with CUDA events on the launching stream.  While enabled,
 * every `every`-th confkv_step (the first one included) records events
 * around its three kernels (confidence and append / attention /
 * select-compact-requant); the others run without events, since each event
 * record between kernels costs the stream about two microseconds.
 * confkv_profile_read synchronises and returns the summed milliseconds of
 * each kernel and the number of steps recorded, then clears them.  At most
 * `max_steps` recorded steps are kept.  CONFKV_EINVAL if max_steps < 1 or
 * every < 1. */
int confkv_profile_enable(confkv_ctx* ctx, int32_t max_steps, int32_t every);
int confkv_profile_disable(confkv_ctx* ctx);
int confkv_profile_read(confkv_ctx* ctx, double* ms_prestep, double* ms_attention,
                        double* ms_select, int32_t* steps);

/* Attention launch shape chosen for the next step: CTAs per (layer, sequence,
 * KV head) unit and dynamic shared memory per CTA.  Units go to the split-K
 * kernel (2-8 CTAs per unit in one cluster) only when there are fewer units
 * than persistent CTAs (two per SM) and every CTA of a cluster still streams
 * at least 64 16-token blocks; otherwise each unit runs whole on the
 * persistent kernel (splits = 1).  confkv_launch_plan does the same planning
 * without a context. */
int confkv_attention_plan(confkv_ctx* ctx, int32_t* splits, int32_t* smem_bytes);

/* How confkv_step runs a step on the device (results do not depend on it):
 *   CONFKV_STEP_AUTO (default)  one kernel launch for the whole step when
 *       every (layer, sequence, KV head) unit can have an SM of its own
 *       (one CTA per unit; the SMs left over reduce the vocabulary, or with
 *       none left the units' epilogue warps take one chunk of at most 4096
 *       logits each), the INT8 region of a unit stays within 8192 tokens,
 *       compaction is tail fill, the selection's working set and the
 *       unit's scores fit the kernel's shared memory and the logits are in
 *       device memory; otherwise three launches;
 *   CONFKV_STEP_SEPARATE  always three launches (confidence reduction and
 *       append; attention; selection).
 * The fused launch removes two kernel launches and their gaps from steps of
 * small shapes (the pages' per-step profile, [rainbus] 复现评估, is
 * dominated by such fixed costs there).  confkv_step_launches gives the
 * launches the next step would take.  CONFKV_EINVAL for a null ctx or an
 * unknown mode.  The pages give no counterpart: these are launch controls of
 * this library. */
enum { CONFKV_STEP_AUTO = 0, CONFKV_STEP_SEPARATE = 1 };
int confkv_set_step_mode(confkv_ctx* ctx, int32_t mode);
int confkv_step_launches(confkv_ctx* ctx, int32_t* launches);

/* Caps the attention grid at `ctas` CTAs; 0 (the default) lets the
 * persistent kernel use two CTAs per SM.  The split-K kernel is chosen only
 * while units x splits stays within the cap, otherwise the persistent kernel
 * runs on at most `ctas` CTAs.  A smaller grid leaves SMs to work on other
 * streams, at a proportional cost in attention time.  Takes effect at the
 * next launch (a captured graph keeps the grid it was captured with; steps
 * inside a graph reservation keep the reserved plan).  Results do not depend
 * on it.  The pages give no counterpart: it is a
 * launch-shape control of this library.  CONFKV_EINVAL for a null ctx or a
 * negative count. */
int confkv_set_attention_ctas(confkv_ctx* ctx, int32_t ctas);

/* Grid of the attention launch chosen for the next step: `ctas` CTAs in
 * clusters of `cluster`.  The persistent kernel (one CTA per unit in
 * confkv_attention_plan) runs unclustered CTAs that each walk whole
 * (layer, sequence, KV head) units; the split-K kernel runs one cluster of
 * `splits` CTAs per unit. */
int confkv_attention_grid(confkv_ctx* ctx, int32_t* ctas, int32_t* cluster);

/* The attention launch a step would take, planned on the host alone (no
 * context; nothing runs on a GPU): for configuration `cfg`, a bound
 * `n8_bound` on the INT8 entries of any (layer, sequence) and a cap
 * `attn_ctas` on the persistent grid (0 = none, as confkv_set_attention_ctas),
 * `splits` CTAs per (layer, sequence, KV head) unit (1 = the persistent
 * kernel) and a grid of `ctas` CTAs in clusters of `cluster`.  A context
 * plans each step the same way with its own host bound on n8 (the largest
 * prefill minus W, then at most the largest budget).  The SM count is the
 * current device's, 152 (GB300) when none can be queried.  CONFKV_EINVAL
 * for a null argument, an invalid configuration, a negative bound or cap,
 * or a bound above cap; CONFKV_ECAPACITY when no launch fits in shared
 * memory.  The pages give no counterpart: it exposes this library's launch
 * planning. */
int confkv_launch_plan(const confkv_config* cfg, int64_t n8_bound, int32_t attn_ctas, int32_t* splits,
                       int32_t* ctas, int32_t* cluster);

/* Byte offset of (token tau in [0,16), channel c) inside one 16-token block of
 * the device layout: kind 0 = INT8 K, 1 = INT8 V, 2 = FP16 K, 3 = FP16 V.
 * Host-only helper for tests of the interleave; -1 for bad arguments. */
int32_t confkv_block_offset(int32_t kind, int32_t d, int32_t tau, int32_t c);

/* Largest number of per-chunk partial results confkv_confidence_noalloc can
 * hold: B * ceil(V / 4096) must not exceed it.  The library reserves this
 * scratch (32 bytes per partial, 128 KiB) on every GPU that loads it, for as
 * long as the process runs. */
#define CONFKV_NOALLOC_MAX_PARTIALS 4096

/*
 * Confidence c of B next-token distributions, computed without allocating
 * any device memory.  The paper has no counterpart of this call: it exists
 * for callers that cannot allocate where they need the score -- a plug-in
 * whose host process owns every device buffer through its own pool, a
 * real-time loop that forbids allocation after start-up, or code that must
 * not risk the implicit synchronisation an allocation can cause.  The caller
 * passes only its input and output:
 *   logits      device fp32 [B][V] (temperature 1)
 *   confidence  device fp32 [B], written: the same c as the `confidence`
 *               output of confkv_step, c = w_H (1 - H / log V) +
 *               w_m sigmoid(log p1 - log p2) + w_p p1
 * The partial results of the vocabulary reduction go to one fixed scratch
 * array owned by the library (CONFKV_NOALLOC_MAX_PARTIALS entries per GPU).
 * Every call uses that same array and leaves its last contents there, so
 * calls whose kernels overlap on the GPU (streams without ordering between
 * them) race and give wrong results; order them on one stream.  The first
 * call on a device looks up the array's device address (once per device,
 * with that device current); make that first call before any stream capture.
 * Returns CONFKV_ECAPACITY, without launching anything, if
 * B * ceil(V / 4096) > CONFKV_NOALLOC_MAX_PARTIALS; CONFKV_EINVAL for null
 * pointers, logits or confidence not 4-byte aligned, B < 1, V < 2 or
 * non-finite weights.  Asynchronous on `stream`.
 */
int confkv_confidence_noalloc(const float* logits, int32_t B, int32_t V, double w_H, double w_m,
                              double w_p, float* confidence, void* stream);

/*
 * Norms and rotary positions of queries and keys, in one pass: the tensors
 * that a model's projections give become the q, k_new of confkv_step, or the
 * q, k of a prompt.  The paper has no counterpart.  Per token and head:
 *   y = x * rsqrt(mean(x^2) + eps) * weight     (without a weight: y = x)
 *   (a, b) -> mscale (a cos t - b sin t, b cos t + a sin t)
 * for the pairs of the first rot channels, (2i, 2i + 1) if `interleaved`,
 * else (i, i + rot / 2), with t = 2 pi * position * turns[i] / 2^64.  Channels
 * from rot on are not rotated.  All arithmetic is fp32 (angles exact modulo
 * one turn, then rounded to fp32), rounded to the output type at the end.
 *   q [n][Hq][d], k [n][Hkv][d] in in_dtype; q_out, k_out the same shapes in
 *   their own types; any of fp16, bf16, fp32.  Strides in elements, token
 *   first, then head; channels contiguous, addresses aligned to the element.
 *   Hkv = 0: no keys (k, k_out ignored).  An output may be its input (same
 *   address, strides and type); otherwise outputs must overlap nothing.
 *   q_weight, k_weight: [d] in w_dtype, or NULL (no norm for that tensor)
 *   positions: device int32 [n]; turns: device [rot / 2], from
 *   confkv_rotary_frequencies; both may be NULL if rot = 0
 * d up to 512 (CONFKV_ENOTIMPL above).  Fast for d = 64, 128, 256 with rot a
 * multiple of 16 and every row on a 16-byte boundary.  Asynchronous on
 * `stream`, may be captured.
 */
typedef struct confkv_rotary_args {
  int32_t n, Hq, Hkv, d, rot;
  int32_t interleaved;
  int32_t in_dtype, w_dtype, q_out_dtype, k_out_dtype;
  float eps, mscale;
  const void *q, *k;
  void *q_out, *k_out;
  int64_t q_stride[2], k_stride[2], q_out_stride[2], k_out_stride[2];
  const void *q_weight, *k_weight;
  const int32_t* positions;
  const uint64_t* turns;
} confkv_rotary_args;
int confkv_qk_rotary(const confkv_rotary_args* args, void* stream);

/* Frequencies of the rot / 2 pairs as turns per position in units of 2^-64
 * (HOST array `turns`), and the factor of the rotated channels.  Pair i turns
 * by f_i = base^(-2i / rot) radians per position (base > 1);
 *   CONFKV_ROTARY_LINEAR  f_i / factor
 *   CONFKV_ROTARY_NTK     base * factor^(rot / (rot - 2)) in place of base
 *   CONFKV_ROTARY_YARN    (arXiv 2309.00071) with r = original_length f_i /
 *       (2 pi) turns in the trained length, g = clamp((r - beta_slow) /
 *       (beta_fast - beta_slow), 0, 1): f_i g + f_i / factor (1 - g), and
 *       mscale = 0.1 ln(factor) + 1 (1 otherwise).  The ramp is linear in the
 *       turns r, as in that paper.  Code that loads such checkpoints commonly
 *       ramps linearly in the pair index i between rounded bounds, which gives
 *       other frequencies within the ramp: for those and other rules,
 *       confkv_qk_rotary takes any table of turns.
 * factor >= 1.  Host only. */
enum { CONFKV_ROTARY_PLAIN = 0, CONFKV_ROTARY_LINEAR = 1, CONFKV_ROTARY_NTK = 2, CONFKV_ROTARY_YARN = 3 };
int confkv_rotary_frequencies(int32_t rot, double base, int32_t scaling, double factor, double original_length,
                              double beta_fast, double beta_slow, uint64_t* turns, float* mscale);

/*
 * Attention of packed prompts.  The paper has no counterpart: its decode step
 * starts from a prefilled cache, and this is the attention that produces the
 * prefill's own hidden states, for a whole prompt, a chunk of one against its
 * history, or single tokens.  Sequence b of B holds query rows
 * cu_q[b] .. cu_q[b+1]-1 of q and key rows cu_k[b] .. cu_k[b+1]-1 of k and v:
 *   out[i][h] = sum_j softmax_j(scale q[i][h] . k[j][h / G]) v[j][h / G],
 *   lse[i][h] = log sum_j exp(scale q[i][h] . k[j][h / G]),   G = Hq / Hkv,
 * over all keys of the sequence, or with `causal` over those up to the
 * query's own position, the queries being the last of the sequence: query i
 * of lq sees keys 0 .. lk - lq + i.  A row that sees no key gets out = 0 and
 * lse = -inf.
 *   q [total_q][Hq][d], k, v [total_k][Hkv][d], out [total_q][Hq][d], all
 *   fp16 or all bf16 (dtype), d = 64 or 128.  Strides are in elements, token
 *   first, then head; channels are contiguous.  Every base address is a
 *   multiple of 16 bytes, every stride of 8 elements and at least d.
 *   lse: fp32 [total_q][Hq], or NULL.
 *   cu_q, cu_k: DEVICE int32 [B + 1], ascending from 0; values outside
 *   [0, total] are clamped to it.  Rows of out and lse that belong to no
 *   sequence are not written.  total_q, total_k < 2^31 - 4096.
 * Scores, maxima, sums and the accumulated output are fp32; the weights are
 * rounded to `dtype` for the product with v (fp16: a weight less than 2^-25 of
 * the row's largest is off by up to 2^-36 of that one instead of 2^-11 of
 * itself), the output once at the end.
 * Values of keys that no query of the call sees do not reach the output,
 * NaN and infinities among them.  Within a sequence a non-finite value of v may
 * also reach rows that do not see it (a weight of zero times infinity): those
 * whose own last key is at most 126 + floor(128 / G) keys before it.  out must
 * not overlap an input.
 * The keys of few rows are split over a cluster of CTAs and joined, by a rule
 * on the sizes above: the same call gives the same bits every time, but a
 * sequence's last bits may depend on the sizes of the call it is part of.
 * The call uses no workspace and may be captured; two calls may run at once.
 * Asynchronous on `stream`.  CONFKV_EINVAL for a bad argument,
 * CONFKV_ENOTIMPL for another d.
 */
typedef struct confkv_prompt_args {
  int32_t B, Hq, Hkv, d;
  int32_t dtype;              /* CONFKV_Q_FP16 or CONFKV_Q_BF16 */
  int32_t causal;
  int32_t total_q, total_k;
  float scale;                /* > 0 */
  int32_t reserved;           /* 0 */
  const void *q, *k, *v;
  void* out;
  float* lse;
  const int32_t *cu_q, *cu_k;
  int64_t q_stride[2], k_stride[2], v_stride[2], out_stride[2];
} confkv_prompt_args;
int confkv_prompt_attention(const confkv_prompt_args* args, void* stream);

/* Whether a bounded wait of a confkv_prompt_attention kernel gave up on the
 * current device since the last call (CONFKV_STATUS_TIMEOUT in `bits`, and
 * CONFKV_EDEVICE): outputs of the calls since then are not valid (rows are
 * unwritten, or NaN where only a part of their keys was lost).  The calls
 * themselves are asynchronous and do not report it.
 * Synchronises `stream` and clears the word. */
int confkv_prompt_status(int32_t* bits, void* stream);

/* Self-test of failure detection: confkv_prompt_attention with one CTA of the
 * first sequence's last rows (which have to see a key) whose softmax warps do
 * nothing, and waits that give up after 2^20 cycles.  The CTA's other warps
 * run into that limit, set the bit above, wait for their copies and products
 * in flight and leave; nothing faults, and the next call works as ever.
 * Asynchronous on `stream`. */
int confkv_selftest_prompt_timeout(const confkv_prompt_args* args, void* stream);

/*
 * Decoding with several candidates per sequence.  The paper has no
 * counterpart: its step takes one token per sequence.  Three operators:
 * attention of drafted tokens over the cache (speculative decoding), the
 * selection of beams, and the exchange of cache states that follows it.
 */

/*
 * Attention of a tree of drafted tokens over the cache of one layer, which it
 * only reads: T tokens per sequence, of which draft t of sequence b sees every
 * resident entry, itself and its ancestors among the drafts:
 *   out[b][t][h] = sum_j softmax_j(scale q[b][t][h] . k_j) v_j,
 *   lse[b][t][h] = log sum_j exp(scale q[b][t][h] . k_j).
 * T = 1 is the attention of a single new token.  What has been accepted goes
 * into the cache by confkv_step, token by token, so that masses and evictions
 * stay those of plain decoding; an entry that a step would evict between two
 * accepted tokens is still seen here.
 *   q [B][T][Hq][d], k, v [B][T][Hkv][d], out as q; all fp16 or all bf16
 *   (dtype).  k and v are rounded to fp16 first, as the cache would store them.
 *   Strides are in elements, sequence, token, head; channels are contiguous.
 *   Base addresses are multiples of 16 bytes and strides of 8 elements; inputs
 *   may be broadcast (stride 0).  out must overlap nothing.
 *   lse: fp32 [B][T][Hq], or NULL
 *   parents: device int32 with strides parents_stride (sequence, token): the
 *   draft before draft t on its path, an index below t; any other value (-1)
 *   says that t follows the cache.  NULL: a chain, each token after the last.
 *   lens: device int32 [B], drafts in use (clamped to 0 .. T), or NULL: all.
 *   Rows of the others are written: out = 0, lse = -inf, and their q, k and v
 *   are not read.
 * T is at most CONFKV_TREE_MAX_DRAFTS.  Scores, maxima, sums and the
 * accumulated output are fp32, the scales of INT8 keys are applied to q in two
 * fp16 parts, the output is rounded once at the end.  The weights are two fp16
 * parts where few rows are taken (always for T Hq / Hkv <= 8 in the default
 * mode): off by 2^-22 of themselves.  Many rows have them in one: off by 2^-11.
 * In both cases by up to 2^-29 of the row's largest where that is more.
 * Non-finite values of drafts reach only the rows that see them.
 *   workspace: confkv_tree_workspace_bytes(ctx, T) of device memory (0 where the
 *   mode or the sizes rule out dealt keys: T Hq / Hkv <= 8 in the default mode,
 *   or more than 304 tiles of 128 rows), 16-byte aligned, for this call alone:
 *   nothing in it has to be set before or is kept after.  CONFKV_ECAPACITY for
 *   less than that.  The default mode asks for it (some 20 MB with 128 channels)
 *   also for calls that then take a kernel without dealt keys: which one depends
 *   on the lengths at the call.
 * Needs a prefilled context (else CONFKV_ESTATE); asynchronous on `stream`;
 * may be captured, and a replay reads the cache as it then is.  Calls on
 * several streams may run at once as long as nothing writes the cache.  The
 * keys of few rows are split over CTAs and joined by a rule on sizes and
 * lengths: the same call gives the same bits, but a sequence's last bits may
 * depend on the sizes of the whole call.
 */
#define CONFKV_TREE_MAX_DRAFTS 128
typedef struct confkv_tree_args {
  int32_t layer, T;
  int32_t dtype;              /* CONFKV_FP16 or CONFKV_BF16 */
  float scale;                /* > 0 */
  const void *q, *k, *v;
  void* out;
  float* lse;
  const int32_t *parents, *lens;
  int64_t q_stride[3], k_stride[3], v_stride[3], out_stride[3];
  int64_t parents_stride[2];
  void* workspace;
  size_t workspace_bytes;
} confkv_tree_args;
int confkv_tree_workspace_bytes(confkv_ctx* ctx, int32_t T, size_t* bytes);
int confkv_tree_attention(confkv_ctx* ctx, const confkv_tree_args* args, void* stream);

/* Which kernel confkv_tree_attention runs (results agree within their
 * rounding):
 *   CONFKV_TREE_AUTO (default)  the one that a model of them expects to be
 *       fastest, from the sizes and the host's bounds on the INT8 entries
 *   CONFKV_TREE_ROWS   16 rows (draft, query head of a KV head) per CTA, read
 *       straight from the stored layout: few rows, short caches
 *   CONFKV_TREE_TILES  128 rows per CTA on converted tiles, keys in equal parts
 *       within a cluster: many rows
 *   CONFKV_TREE_DEALT  the same with the keys of each sequence dealt out by its
 *       own length, through the workspace; as CONFKV_TREE_TILES where the call
 *       has more than 304 tiles of 128 rows
 * CONFKV_EINVAL for a null ctx or an unknown mode. */
enum { CONFKV_TREE_AUTO = 0, CONFKV_TREE_ROWS = 1, CONFKV_TREE_TILES = 2, CONFKV_TREE_DEALT = 3 };
int confkv_set_tree_mode(confkv_ctx* ctx, int32_t mode);

/* Self-test of failure detection: confkv_tree_attention by its many-row
 * kernel, with one CTA whose softmax warps do nothing and waits that give up
 * after 2^20 cycles.  Its other warps run into that limit, set
 * CONFKV_STATUS_TIMEOUT in the context's status word (confkv_get_stats), wait
 * for their products in flight and leave; nothing faults, rows of that CTA's
 * cluster become NaN, and the next call works as ever.  Asynchronous. */
int confkv_selftest_tree_timeout(confkv_ctx* ctx, const confkv_tree_args* args, void* stream);

/*
 * Selection of beams: the n best continuations of each of `groups` groups of
 * `beams` beams, over beams and vocabulary.  A beam k with score s_k offers
 * each token v at
 *   s_k + x_kv - log sum_w exp(x_kw),      x_k = logits[group][k],
 * a finished beam (finished[group][k] != 0) only end_token, at s_k itself.
 * Written per group, best first:
 *   scores_out fp32, parents int32 (the beam k), tokens int32, each [groups][n].
 * Ties go to the lowest k, then the lowest v.  Only continuations above -inf
 * count: NaN counts as -inf, a beam whose score or log-sum-exp is not finite
 * offers nothing, and places for which there is none are (-inf, 0, 0).
 *   logits [groups][beams][V], dtype CONFKV_FP16, BF16 or FP32, with strides
 *   in elements (group, beam), the vocabulary contiguous; aligned to the element
 *   scores fp32 [groups][beams]; finished uint8 [groups][beams] or NULL
 *   workspace: confkv_beam_workspace_bytes of device memory, 16-byte aligned,
 *   for this call alone: nothing in it has to be set before or is kept after.
 * Beams are compared by sums of 48 bits over a log-sum-exp whose exponentials
 * and partial sums are fp32 (off by about 1e-7): continuations of different
 * beams that close together may change places.  A sum that leaves fp32 is -inf.
 * beams and n at most CONFKV_BEAM_MAX, n at most beams * V.  The outputs must
 * not overlap the inputs or each other.  Asynchronous on `stream`, may be
 * captured.  CONFKV_ECAPACITY for too small a workspace.
 */
#define CONFKV_BEAM_MAX 64
typedef struct confkv_beam_args {
  int32_t groups, beams, V, n;
  int32_t dtype, end_token;
  const void* logits;
  int64_t logits_stride[2];
  const float* scores;
  const uint8_t* finished;
  float* scores_out;
  int32_t *parents, *tokens;
  void* workspace;
  size_t workspace_bytes;
} confkv_beam_args;
int confkv_beam_workspace_bytes(int32_t groups, int32_t beams, int32_t V, int32_t n, size_t* bytes);
int confkv_beam_select(const confkv_beam_args* args, void* stream);

/*
 * Exchange of cache states after a selection of beams: in every layer,
 * sequence g * beams + k takes over the state (entries, scales, positions,
 * EMA masses) that sequence g * beams + parents[g * beams + k] had before the
 * call; later steps go on from there.  parents: device int32 [B]; a value
 * outside 0 .. beams - 1 leaves the sequence as it is.  B has to be a multiple
 * of beams (at most CONFKV_BEAM_MAX; at most 65535 groups), and the sequences of a group have to
 * have the same prompt length (CONFKV_EINVAL): states keep their positions.
 * In place and without a workspace; only sequences whose parent is another one
 * are written.  Needs a prefilled context (else CONFKV_ESTATE); asynchronous
 * on `stream`, may be captured (also inside a reservation, between steps).
 */
int confkv_reorder(confkv_ctx* ctx, const int32_t* parents, int32_t beams, void* stream);

/* Human-readable text of a status code. */
const char* confkv_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t confkv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CONFKV_H */
