/*
 * mfsdp.h - C ABI of the owner-local Muon + AdamW optimizer step (gfx950).
 *
 * What it computes.  "MatrixFSDP: Communication-Free Matrix Optimizers Under
 * ZeRO-3 Parameter Sharding" (arXiv 2607.05895), Abstract and §1: with
 * owner-shaped sharding, each 2D weight lives whole on one data-parallel
 * rank, so that rank can run Muon's Newton-Schulz on it with no optimizer
 * collective, while tensors that are not matrices are grouped onto tail
 * owners and use AdamW.  The update has to be the one full-matrix Muon
 * gives on the gathered matrix (Abstract; §1).  This
 * library is that owner-local step for one GPU: a table of whole tensors
 * (offsets, shapes, dtypes, roles; the paper's MatrixShard metadata, Abstract)
 * that live in one flat parameter buffer, and one call that updates all of
 * them.
 *
 * Per Muon matrix W (rows x cols), gradient G, momentum M (fp32, or bf16 by
 * hparams.momentum_dtype):
 *   M <- beta*M + G;  U <- G + beta*M (Nesterov) or U <- M;
 *   X <- U / (||U||_F + eps), taken in the wide orientation (tall -> U^T);
 *   ns_steps times: A = X X^T;  B = b*A + c*A*A;  X <- a*X + B*X;
 *   O = X back in W's orientation;
 *   W <- W*(1 - lr*weight_decay) - lr*scale*O,
 *   scale = sqrt(max(1, rows/cols)) (mode 0) or 0.2*sqrt(max(rows, cols)) (mode 1).
 * Per AdamW tail tensor (1-based step t):
 *   m <- b1*m + (1-b1)*g;  v <- b2*v + (1-b2)*g^2;
 *   W <- W*(1 - lr_a*wd_a) - lr_a*(m/(1-b1^t)) / (sqrt(v/(1-b2^t)) + eps_a).
 * Every stored value is rounded once to its storage type, to nearest-even
 * (moments in 8 bits as described at mfsdp_moments_args).
 *
 * Ownership.  The caller allocates every device buffer (params, grads,
 * state, workspace, ns_out).  The library never allocates device memory.
 * A plan is host memory owned by the library until mfsdp_plan_destroy.
 *
 * Errors.  Every function returns mfsdp_status; no C++ exception crosses the
 * boundary and nothing aborts the process.  mfsdp_last_error_message()
 * returns a thread-local description of the last failure on this thread.
 */
#ifndef MFSDP_H
#define MFSDP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mfsdp_status {
    MFSDP_OK = 0,
    MFSDP_ERR_INVALID_ARGUMENT = 1,   /* null pointer, negative size, bad step, out of range */
    MFSDP_ERR_OVERLAP = 2,            /* two table entries share parameter bytes */
    MFSDP_ERR_MISALIGNED = 3,         /* entry offset not a multiple of 16 bytes */
    MFSDP_ERR_UNSUPPORTED = 4,        /* dtype, role, precision or dimension not supported */
    MFSDP_ERR_WORKSPACE_TOO_SMALL = 5,/* workspace_bytes below mfsdp_plan_workspace_bytes */
    MFSDP_ERR_HIP = 6,                /* a HIP runtime call or kernel launch failed */
    MFSDP_ERR_INTERNAL = 7
} mfsdp_status;

typedef enum mfsdp_dtype {
    MFSDP_F32 = 0,
    MFSDP_BF16 = 1
} mfsdp_dtype;

typedef enum mfsdp_role {
    MFSDP_ROLE_AUTO = 0,   /* Muon iff rows > 1 and cols > 1, else AdamW */
    MFSDP_ROLE_MUON = 1,   /* force Muon (rows >= 1, cols >= 1) */
    MFSDP_ROLE_ADAMW = 2,  /* force AdamW */
    MFSDP_ROLE_ADAMW8 = 3  /* AdamW with its moments in 8 bits: 2.06 state bytes an element in place of 8 */
} mfsdp_role;

/* One whole tensor of the owner buffer (one row of the owner table).
 * offset: byte offset into the params buffer; the grads buffer uses the same
 *         offset.  Must be a multiple of 16.
 * rows, cols: logical shape, row-major.  A 1D tensor of length L is rows=1,
 *         cols=L.  rows*cols == 0 is an empty shard: legal and skipped.
 * dtype:  storage type of both the parameter and its gradient.
 * role:   mfsdp_role. */
typedef struct mfsdp_entry {
    uint64_t offset;
    int64_t rows;
    int64_t cols;
    int32_t dtype;
    int32_t role;
} mfsdp_entry;

/* Hyper-parameters.  Floats are used as the float32 values given. */
typedef struct mfsdp_hparams {
    float lr;                 /* Muon learning rate */
    float weight_decay;       /* Muon decoupled weight decay (multiplied by lr) */
    float momentum;           /* beta */
    int32_t nesterov;         /* 1: U = G + beta*M; 0: U = M */
    int32_t ns_steps;         /* Newton-Schulz iterations, 0..64 */
    float ns_a, ns_b, ns_c;   /* quintic coefficients */
    float ns_eps;             /* added to ||U||_F */
    int32_t lr_scale_mode;    /* 0: sqrt(max(1, rows/cols)); 1: 0.2*sqrt(max(rows, cols)) */
    int32_t ns_precision;     /* 0: bf16 operands, fp32 accumulate; 1: fp32 operands and accumulate */
    float adam_lr;
    float adam_beta1;
    float adam_beta2;
    float adam_eps;
    float adam_weight_decay;
    int32_t momentum_dtype;   /* storage type of the Muon momentum: MFSDP_F32 (0, the default) or
                                 MFSDP_BF16, rounded to nearest-even once per step.  bf16 halves the
                                 momentum's memory, keeping the owner's optimizer state small (the
                                 ZeRO-3-scale memory the MatrixFSDP abstract asks for), and the
                                 momentum pass then moves 8 B per bf16 element instead of 12.  The
                                 AdamW moments stay fp32. */
    int32_t ns_tile_gram;     /* output tile edge of the Newton-Schulz Gram contraction: 0 = chosen by
                                 the planner (256 when the phase has at least 512 tiles of 256, else
                                 128), or 128 or 256 to force it (for tests and tuning; the result
                                 is the same up to fp32 summation order) */
    int32_t ns_tile_poly;     /* the same for the polynomial B = b A + c A A */
    int32_t ns_tile_update;   /* the same for the update X <- a X + B X; a forced edge also turns off
                                 the planner's split of a short last round of 256-tiles into 128-tiles */
    uint32_t guard_bytes;     /* 0 normally.  Otherwise at most 16 MiB: the plan leaves this many
                                 bytes (rounded up to 256) unused after every region it lays out in
                                 the state and in the workspace (mfsdp_plan_regions lists them), so
                                 that a test can fill the gaps with canaries and check after a step
                                 that no kernel wrote outside its regions.  Costs only memory. */
} mfsdp_hparams;

typedef struct mfsdp_plan_s* mfsdp_plan_t;

/* Per-entry layout facts a caller needs to read or seed state. */
typedef struct mfsdp_entry_info {
    int32_t role;             /* resolved: MFSDP_ROLE_MUON, MFSDP_ROLE_ADAMW, MFSDP_ROLE_ADAMW8, or -1 for an
                                 empty entry */
    int32_t transposed;       /* Muon: 1 if rows > cols (Newton-Schulz runs on the transpose) */
    int64_t m, n;             /* Muon: oriented shape, m = min(rows, cols) */
    uint64_t state_offset;    /* Muon: momentum (momentum_dtype); AdamW: fp32 first moment, or its codes and
                                 scales for MFSDP_ROLE_ADAMW8 (bytes into state) */
    uint64_t state_offset2;   /* AdamW: the second moment likewise (bytes into state); 0 otherwise */
    uint64_t ns_out_offset;   /* Muon: element offset of the fp32 O export in ns_out */
    float lr_scale;           /* Muon: the shape scale applied to lr */
} mfsdp_entry_info;

/* Which caller buffer a plan region lies in. */
#define MFSDP_BUFFER_STATE 0
#define MFSDP_BUFFER_WORKSPACE 1

/* One region the plan lays out in the state or the workspace. */
typedef struct mfsdp_region {
    uint64_t offset;          /* bytes into the buffer */
    uint64_t bytes;           /* bytes the step may read or write there */
    int32_t buffer;           /* MFSDP_BUFFER_STATE or MFSDP_BUFFER_WORKSPACE */
    int32_t entry;            /* table entry it belongs to, -1 for a region shared by all entries */
} mfsdp_region;

/* Step flags. */
#define MFSDP_STEP_DESCRIPTORS_RESIDENT 1u  /* the workspace already holds this plan's
                                               descriptors from an earlier step with the
                                               same workspace pointer; skip the upload */

typedef struct mfsdp_step_args {
    void* params;             /* device, updated in place */
    const void* grads;        /* device, read only; same offsets as params */
    void* state;              /* device, mfsdp_plan_state_bytes, zero-filled before step 1 */
    void* workspace;          /* device, mfsdp_plan_workspace_bytes, 256-byte aligned;
                                 library scratch: the caller must not write it between steps */
    uint64_t workspace_bytes;
    int64_t step;             /* 1-based step count (AdamW bias correction) */
    void* stream;             /* hipStream_t; NULL = the null stream */
    float* ns_out;            /* NULL, or device fp32 [mfsdp_plan_ns_out_elems]: O per Muon entry,
                                 row-major in the entry's own shape, at entry_info.ns_out_offset */
    uint32_t flags;           /* MFSDP_STEP_* */
    void** events;            /* NULL, or n_events hipEvent_t created by the caller: the step
                                 records events[0] after the descriptor upload, events[1] after
                                 the AdamW tail, events[2] after momentum + norm, and for
                                 Newton-Schulz iteration k (1-based) events[3k], events[3k+1],
                                 events[3k+2] after its Gram, polynomial and update launches.
                                 Every event is recorded even when its phase is empty. */
    uint32_t n_events;        /* must be >= mfsdp_plan_num_events when events != NULL */
} mfsdp_step_args;

/* Validate an owner table and lower it to a plan (host only; no HIP call).
 * entries: n rows (may be NULL when n == 0).  param_bytes: size of the params
 * buffer, used for bounds checks.  hp: copied into the plan.
 * Errors: INVALID_ARGUMENT (null pointer, n < 0, negative dim, entry past
 * param_bytes, bad hyper-parameter), OVERLAP, MISALIGNED, UNSUPPORTED (dtype,
 * role, ns_precision, momentum_dtype, an ns_tile_* other than 0, 128 and
 * 256, a dimension above 2^22, a Muon matrix whose padded Newton-Schulz
 * buffer reaches 2 GiB).  *out is set only on success.  The plan depends on
 * its arguments only (no environment variable is read). */
mfsdp_status mfsdp_plan_create(const mfsdp_entry* entries, int64_t n, uint64_t param_bytes,
                               const mfsdp_hparams* hp, mfsdp_plan_t* out);

/* Bytes of optimizer state the plan lays out (momentum for Muon entries, fp32
 * or bf16 by hp->momentum_dtype, then fp32 first and second moments for AdamW
 * entries, then those in 8 bits), each region 256-byte aligned. */
mfsdp_status mfsdp_plan_state_bytes(mfsdp_plan_t plan, uint64_t* bytes);

/* Bytes of device workspace one step needs (descriptors, norm partials,
 * Newton-Schulz buffers). */
mfsdp_status mfsdp_plan_workspace_bytes(mfsdp_plan_t plan, uint64_t* bytes);

/* Number of fp32 elements of the optional ns_out export. */
mfsdp_status mfsdp_plan_ns_out_elems(mfsdp_plan_t plan, uint64_t* elems);

/* Number of phase-boundary events a step records when args->events is set
 * (3 + 3*ns_steps). */
mfsdp_status mfsdp_plan_num_events(mfsdp_plan_t plan, uint32_t* n);

/* Number of table entries and the layout facts of entry i. */
mfsdp_status mfsdp_plan_num_entries(mfsdp_plan_t plan, int64_t* n);
mfsdp_status mfsdp_plan_entry_info(mfsdp_plan_t plan, int64_t i, mfsdp_entry_info* info);

/* One owner step: enqueue every kernel on args->stream and return without
 * synchronising.  Launch failures return MFSDP_ERR_HIP; a fault inside a
 * kernel surfaces at the caller's next synchronisation.  One plan serves one
 * stream at a time; two steps that share a workspace must not overlap.
 * Errors: INVALID_ARGUMENT (null plan or args, null buffer needed by the
 * table, step < 1 with an AdamW entry, misaligned workspace, too few
 * events), WORKSPACE_TOO_SMALL, HIP. */
mfsdp_status mfsdp_owner_step(mfsdp_plan_t plan, const mfsdp_step_args* args);

/* Every region the plan lays out, state first, then workspace, each in
 * increasing offset: Muon momentum and AdamW first and second moments in the
 * state; in the workspace the descriptor blob (one region: it is uploaded
 * as one copy), the per-matrix scale factors, the norm partial sums, and per
 * Muon matrix its two X^T buffers and its A and B.  The step reads and
 * writes state and workspace bytes inside these regions only.  Writes
 * min(*count, capacity) entries to regions (which may be NULL when capacity
 * is 0) and the total number to *count.  Host only.
 * Errors: INVALID_ARGUMENT (NULL plan or count, capacity < 0, NULL regions
 * with capacity > 0). */
mfsdp_status mfsdp_plan_regions(mfsdp_plan_t plan, mfsdp_region* regions, int64_t capacity, int64_t* count);

/* ---- A step that allocates nothing ----
 *
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  The same
 * step as mfsdp_owner_step (same kernels, bitwise the same results), except
 * that the workspace is a fixed array inside the library: a file-scope
 * device array of MFSDP_STATIC_WORKSPACE_BYTES, which every GPU the library
 * runs on holds until the process ends.  The caller still passes params,
 * grads, state, ns_out and events as for mfsdp_owner_step, with workspace =
 * NULL and workspace_bytes = 0.  The call allocates nothing (no hipMalloc,
 * hipFree or allocating library routine); on its first call on a device it
 * looks up that device's copy of the array (hipGetSymbolAddress).
 * Every call on one GPU shares that GPU's array, which keeps the last call's
 * contents: calls that overlap on one GPU (two streams, two threads) race
 * and must be serialised by the caller.  The step writes every workspace
 * byte before it reads it, so nothing is cleared between calls.
 * MFSDP_STEP_DESCRIPTORS_RESIDENT skips the descriptor upload only when the
 * previous static call on this device used the same plan.
 * Errors: those of mfsdp_owner_step, plus INVALID_ARGUMENT (workspace not
 * NULL or workspace_bytes not 0), WORKSPACE_TOO_SMALL (the plan needs more
 * than MFSDP_STATIC_WORKSPACE_BYTES: use mfsdp_owner_step), UNSUPPORTED
 * (device index 64 or more), HIP. */
#define MFSDP_STATIC_WORKSPACE_BYTES (64ull << 20)
mfsdp_status mfsdp_owner_step_static(mfsdp_plan_t plan, const mfsdp_step_args* args);

/* Free a plan.  NULL is accepted. */
mfsdp_status mfsdp_plan_destroy(mfsdp_plan_t plan);

/* ---- Gradients of the owner buffer, between the backward pass and the step ----
 *
 * The global L2 norm of every gradient in the buffer, the norm of each
 * tensor, and clipping to a largest norm:
 *
 *   sumsq = sum over entries and elements of g^2;  norm = sqrt(sumsq);
 *   scale = min(1, max_norm / (norm + eps));       g <- scale * g.
 *
 * The owner holds whole tensors, so each of these is local to it; the
 * global norm over several owners needs one 16-byte record from each
 * (mfsdp_grad_total).  The clipped gradient is either written
 * (mfsdp_grad_clip) or formed as the step reads it (mfsdp_owner_step_scaled,
 * which moves no byte more than mfsdp_owner_step).  The scale stays on the
 * device throughout: nothing here synchronises, and every call below can be
 * captured into a graph once its descriptors are resident.  As for
 * mfsdp_owner_step, the current device must be the stream's and the buffers'.
 *
 * Squares and sums are fp64 in a fixed order: results are bitwise the same
 * from run to run, and no finite gradient overflows or vanishes in them.
 * Non-finite gradients propagate by the formulas: a NaN makes norm and scale
 * NaN; an Inf makes norm Inf and scale 0 (so the Inf itself becomes NaN); with
 * max_norm INFINITY the scale is 1 all the same.
 * Bytes of the buffers that belong to no entry are neither read into a
 * result nor written. */

/* What mfsdp_grad_norm and mfsdp_grad_total write (device memory, 16-byte
 * aligned; its scale field is what mfsdp_grad_clip and
 * mfsdp_owner_step_scaled take). */
typedef struct mfsdp_grad_stats {
    double sumsq;             /* sum of squares */
    float norm;               /* sqrt(sumsq), formed in fp64 and rounded once */
    float scale;              /* min(1, max_norm/(norm + eps)), formed in fp64 and rounded once */
} mfsdp_grad_stats;

/* Device workspace of mfsdp_grad_norm and mfsdp_grad_clip on this plan's
 * table (descriptors, partial sums and the norm's counters; separate from the
 * step's).  It may serve any number of calls, one at a time: two calls that
 * overlap (two streams, two graphs) need a workspace each.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED (a table of more than 2^31 - 1 work
 * items). */
mfsdp_status mfsdp_plan_grad_workspace_bytes(mfsdp_plan_t plan, uint64_t* bytes);

typedef struct mfsdp_grad_norm_args {
    const void* grads;        /* device, read only; the plan's offsets; 16-byte aligned */
    void* workspace;          /* device, mfsdp_plan_grad_workspace_bytes, 256-byte aligned; library
                                 scratch: the caller must not write it between calls */
    uint64_t workspace_bytes;
    double max_norm;          /* > 0; INFINITY: scale is 1 whatever the norm */
    double eps;               /* >= 0, finite */
    mfsdp_grad_stats* stats;  /* device, written */
    float* entry_norms;       /* NULL, or device fp32 [mfsdp_plan_num_entries]: the L2 norm of each
                                 entry's gradient (0 for an empty entry), formed in fp64 and rounded once */
    void* stream;             /* hipStream_t; NULL = the null stream */
    uint32_t flags;           /* MFSDP_STEP_DESCRIPTORS_RESIDENT: an earlier mfsdp_grad_norm or
                                 mfsdp_grad_clip of this plan already filled this workspace; skip the
                                 upload.  Other bits must be 0. */
} mfsdp_grad_norm_args;

/* Enqueue the norm pass.  An empty table gives norm 0 and scale 1.
 * Errors: INVALID_ARGUMENT (null pointer, misaligned buffer, max_norm or eps
 * out of range, unknown flag), WORKSPACE_TOO_SMALL, UNSUPPORTED (as above),
 * HIP. */
mfsdp_status mfsdp_grad_norm(mfsdp_plan_t plan, const mfsdp_grad_norm_args* args);

/* Join the records of several owners: stats->sumsq = the sum of parts[0..count)
 * in that order (so every owner that holds the same records computes the same
 * bits), and norm and scale from it.  parts: device, 16-byte aligned, each as
 * mfsdp_grad_norm wrote it; only sumsq is read.  stats may be one of parts.
 * Errors: INVALID_ARGUMENT (null or misaligned pointer, count outside
 * 1..65536, max_norm or eps out of range), HIP. */
mfsdp_status mfsdp_grad_total(const mfsdp_grad_stats* parts, int64_t count, double max_norm, double eps,
                              mfsdp_grad_stats* stats, void* stream);

typedef struct mfsdp_grad_clip_args {
    const void* grads;        /* device, the plan's offsets; 16-byte aligned */
    void* out;                /* device, the same offsets; grads itself (in place), or a buffer that
                                 does not overlap it; 16-byte aligned */
    const float* scale;       /* device, one value, 4-byte aligned */
    void* workspace;          /* as in mfsdp_grad_norm_args */
    uint64_t workspace_bytes;
    void* stream;
    uint32_t flags;           /* as in mfsdp_grad_norm_args */
} mfsdp_grad_clip_args;

/* Enqueue out <- scale * grads over every entry: the fp32 product rounded
 * once to the entry's type.  A scale of exactly 1 leaves every bit: in place
 * nothing is read or written then, else the entries are copied.
 * Errors: INVALID_ARGUMENT (null pointer, misaligned buffer, buffers that
 * overlap in part, unknown flag), WORKSPACE_TOO_SMALL, UNSUPPORTED, HIP. */
mfsdp_status mfsdp_grad_clip(mfsdp_plan_t plan, const mfsdp_grad_clip_args* args);

/* mfsdp_owner_step with every gradient multiplied by *grad_scale (device,
 * fp32, 4-byte aligned) as it is read: g' = scale * g in fp32, unrounded to
 * the storage type, takes the place of g in the Muon momentum and in AdamW.
 * For fp32 gradients the result is bitwise that of mfsdp_grad_clip followed
 * by mfsdp_owner_step; a scale of 1 gives bitwise mfsdp_owner_step.
 * It takes the caller's workspace; the step on the library's own
 * (mfsdp_owner_step_static) has no scaled form: clip the gradients there.
 * Errors: those of mfsdp_owner_step, plus INVALID_ARGUMENT (NULL or
 * misaligned grad_scale). */
mfsdp_status mfsdp_owner_step_scaled(mfsdp_plan_t plan, const mfsdp_step_args* args, const float* grad_scale);

/* ---- AdamW moments in 8 bits ----
 *
 * An entry with the role MFSDP_ROLE_ADAMW8 takes the AdamW step of
 * mfsdp_owner_step (and its scaled and static forms) with both moments held
 * in 8 bits; entries of either kind may share a table, and the small ones
 * are best left in 32.  A group of 128 consecutive elements (the last one of
 * a tensor may be shorter) shares an fp32 scale for each moment, the largest
 * magnitude in it:
 *
 *   m = scale_m * c*|c| / 127^2,  c an int8 in -127..127;
 *   sqrt(v) = scale_r * (d / 255)^2,  d a uint8 in 0..255, at least 1 where v > 0.
 *
 * In the state each moment is a byte an element at state_offset (first) or
 * state_offset2 (second), and from the next multiple of 256 bytes after
 * rows*cols of them on, one scale a group.  A state of zeros is m = v = 0.
 *
 * The step forms m, v and the parameter in fp32 from the values held, the
 * parameter from m and v before they are rounded.  Codes are rounded down
 * after a dither in (0, 1) is added that step count (its low 32 bits), entry
 * index and element index alone fix, so that slow averages (beta2 = 0.999)
 * move by less than a code step on average and results are bitwise the same
 * from run to run:
 *   mix(h): h ^= h>>16; h *= 0x85ebca6b; h ^= h>>13; h *= 0xc2b2ae35; h ^= h>>16;
 *   key = mix(step + 0x9e3779b9 * (entry + 1));
 *   word = mix((index>>1) + 0x9e3779b9 * (index>>33) + key), in 32 bits;
 *   bytes 0 and 1 of it are of an even element's m and sqrt(v), 2 and 3 of
 *   the odd one's; the dither is (byte + 0.5) / 256.
 * Non-finite moments: a group that holds one is NaN from then on (its
 * parameters of that step follow the formulas).  Both moments are kept for
 * gradients down to 1e-37, to fp32 roundings or, where a value is subnormal,
 * half of 2^-149; a squared gradient above the fp32 range counts as non-finite.
 *
 * mfsdp_moments_read and mfsdp_moments_write turn an entry's state into
 * values and back, for a run that goes over to 8 bits or back, or a
 * checkpoint in another form. */
typedef struct mfsdp_moments_args {
    void* state;              /* device, the owner's state; 256-byte aligned; read does not write it */
    void* first;              /* device, rows*cols values of type: the first moment; 16-byte aligned */
    void* second;             /* device, as first: the second moment (v, not its root) */
    int32_t type;             /* mfsdp_dtype of first and second */
    void* stream;
} mfsdp_moments_args;

/* first, second <- the moments of entry `entry` (MFSDP_ROLE_ADAMW or
 * MFSDP_ROLE_ADAMW8), rounded once to type.  Enqueues one launch (more for
 * more than 2^35 elements), so it can be captured; the current device must be
 * the stream's and the buffers'.  An empty entry does nothing.
 * Errors: INVALID_ARGUMENT (null or misaligned pointer, entry out of range),
 * UNSUPPORTED (type, an entry with another role), HIP. */
mfsdp_status mfsdp_moments_read(mfsdp_plan_t plan, int64_t entry, const mfsdp_moments_args* args);

/* The entry's state <- first, second: in 8 bits to the nearest code (no
 * dither), else rounded to fp32.  A negative or NaN second moment makes its
 * group NaN in 8 bits.  What is read must not overlap the state.
 * Errors: as mfsdp_moments_read. */
mfsdp_status mfsdp_moments_write(mfsdp_plan_t plan, int64_t entry, const mfsdp_moments_args* args);

/* ---- An embedding table of the owner buffer ----
 *
 * An embedding is a 2D tensor that trains with AdamW (role
 * MFSDP_ROLE_ADAMW), held whole by its owner like any other entry: rows =
 * vocabulary, cols = width.  These two calls read it where it lies in the
 * owner's params and form its gradient where the step reads it:
 *
 *   lookup:  out[i][:] = scale * W[id_i - first_id][:];
 *   grad:    G[v][:] (+)= scale * sum over i with id_i - first_id = v of dout[i][:].
 *
 * An id outside first_id .. first_id + rows - 1 has a zero row in the
 * lookup and no part in the gradient: a vocabulary cut into several entries
 * is looked up in each with its own first_id and the results added, and a
 * negative id marks padding.  Whatever dout holds at such a position (NaN
 * too) is not read into a result.  Sums are fp32, formed in an order that
 * depends on the ids and sizes alone (bitwise the same from run to run, no
 * atomics on values), multiplied by scale in fp32, and rounded once to the
 * entry's type.  Both calls only enqueue launches on the stream, so they can
 * be captured; the current device must be the stream's and the buffers'.
 * What a call writes (out, or grads and workspace) must not overlap what it
 * reads (params, ids, dout). */
typedef enum mfsdp_id_type {
    MFSDP_I32 = 0,
    MFSDP_I64 = 1
} mfsdp_id_type;

typedef struct mfsdp_embed_lookup_args {
    const void* params;       /* device, the owner's params buffer; 16-byte aligned */
    const void* ids;          /* device, n_ids of id_type, aligned to their size */
    int64_t n_ids;            /* 0 .. 2^30; 0: nothing is done */
    int32_t id_type;          /* mfsdp_id_type */
    int32_t out_type;         /* mfsdp_dtype of out */
    int64_t first_id;         /* id of the table's row 0, 0 .. 2^62 */
    void* out;                /* device, n_ids rows of cols elements, aligned to the element size */
    int64_t out_stride;       /* elements from one row of out to the next, >= cols; 0 = cols */
    float scale;
    void* stream;
} mfsdp_embed_lookup_args;

/* Enqueue the lookup in entry `entry` of the plan (any role).  Elements of
 * out between two rows are not touched.
 * Errors: INVALID_ARGUMENT (null pointer, entry out of range, n_ids,
 * first_id or out_stride out of range, misaligned buffer), UNSUPPORTED
 * (id_type, out_type), HIP. */
mfsdp_status mfsdp_embed_lookup(mfsdp_plan_t plan, int64_t entry, const mfsdp_embed_lookup_args* args);

/* Device workspace of mfsdp_embed_grad for up to n_ids ids: it never falls as
 * n_ids grows, so one for the largest batch serves every smaller one.  Small
 * batches need 0 bytes.  Errors: INVALID_ARGUMENT. */
mfsdp_status mfsdp_plan_embed_workspace_bytes(mfsdp_plan_t plan, int64_t entry, int64_t n_ids, uint64_t* bytes);

typedef struct mfsdp_embed_grad_args {
    void* grads;              /* device, the owner's grads buffer; 16-byte aligned */
    const void* ids;          /* as in mfsdp_embed_lookup_args */
    int64_t n_ids;            /* 0 .. 2^30 */
    int32_t id_type;
    int32_t dout_type;        /* mfsdp_dtype of dout */
    int64_t first_id;
    const void* dout;         /* device, n_ids rows of cols elements, aligned to the element size; may be
                                 NULL when n_ids is 0 */
    int64_t dout_stride;      /* elements from one row of dout to the next, >= cols; 0 = cols */
    float scale;
    int32_t accumulate;       /* 0: every row of the entry's gradient is written, zeros where no id
                                 points, whatever the scale; 1: the sums are added to what is there, and rows without an id
                                 are not touched */
    void* workspace;          /* device, mfsdp_plan_embed_workspace_bytes, 256-byte aligned; written
                                 before it is read, so it needs no clearing and may be shared by calls
                                 that do not overlap; NULL where 0 bytes are needed */
    uint64_t workspace_bytes;
    void* stream;
} mfsdp_embed_grad_args;

/* Enqueue the gradient of entry `entry`.
 * Errors: INVALID_ARGUMENT (null pointer, entry out of range, n_ids,
 * first_id, dout_stride or accumulate out of range, misaligned buffer),
 * UNSUPPORTED (id_type, dout_type), WORKSPACE_TOO_SMALL, HIP. */
mfsdp_status mfsdp_embed_grad(mfsdp_plan_t plan, int64_t entry, const mfsdp_embed_grad_args* args);

/* ---- The output head over a table of the owner buffer ----
 *
 * A table as above read the other way: logits of a row x_i of activations
 * over the table's rows, z_ij = scale * x_i . W_j, and from them
 *
 *   logp_i    = z_it - log sum_j e^z_ij, t = id_i - first_id;
 *   entropy_i = -sum_j p_ij ln p_ij,  p_ij = e^z_ij / sum_k e^z_ik;
 *   the top_k rows with the largest z_ij, largest first, ties to the lower id.
 *
 * The table may be any 2D entry of up to 2^20 columns, bf16 or fp32, tied to
 * the embedding or not.  Logits are sums in fp32 of products of the values
 * given, bf16 or fp32 (exact, but for at most 2^-22 of a product of two fp32
 * values, and bits under 2^-133 of an fp32 value below 2^-109); the sums over
 * them are fp32 in an order that sizes alone fix (bitwise the same from run to
 * run, no atomics).
 *
 * A negative id marks padding: log probability and entropy 0, no
 * alternatives, no gradient, and whatever x holds there (NaN too) is not read
 * into a result.  An id of 0 or more outside the table has no target here:
 * its log probability is 0 and has no gradient, its entropy and alternatives
 * are the table's.  ids may be NULL: every row counts and none has a target.
 * Non-finite logits propagate by the formulas: a NaN or +Inf makes the row's
 * log probability and entropy NaN; a NaN is never among the alternatives.  A
 * logit of -Inf has probability 0, as a target log probability -Inf, and comes
 * last among the alternatives; a row of nothing else has log probability NaN
 * and entropy 0.  dx is NaN in the columns where the table is infinite.  An
 * infinite value of an fp32 x or table may make a logit NaN where the formula
 * has an infinite one.
 *
 * A vocabulary cut into several entries: mfsdp_head_logprob on each with its
 * own first_id, then mfsdp_head_total joins the records (and alternatives),
 * and mfsdp_head_grad of each entry takes the joined ones; dx is then the sum
 * of the entries' dx.
 *
 * The calls only enqueue launches on the stream, so they can be captured; the
 * current device must be the stream's and the buffers'.  What a call writes
 * must not overlap what it reads or anything else it writes, but for
 * mfsdp_head_total's records. */

/* What a row's distribution is known by, in base 2 (y = log2(e) * z). */
typedef struct mfsdp_head_record {
    float max;                /* largest y */
    float sum;                /* sum of 2^(y - max) */
    float wsum;               /* sum of 2^(y - max) * (y - max) */
    float target;             /* y of the target, 0 without one */
    int32_t found;            /* 1: the target is among the rows summed */
    int32_t active;           /* 0: padding (all other fields are 0 then) */
} mfsdp_head_record;

/* Device workspace of mfsdp_head_logprob on up to n rows with up to top_k
 * alternatives, and with grad = 1 of mfsdp_head_grad on as many too: about n *
 * (rows + min(rows, 32768)) bf16 elements and 8 bytes for each of x more, n
 * rounded up to 256; with fp32 among the operands n * rows times 6 bytes.  For
 * more than 64 rows, and with grad = 1, it holds a copy of a table that is fp32
 * or whose cols are no multiple of 64.  It never falls as n grows, so one for the
 * largest batch serves every smaller one.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED (as mfsdp_head_logprob). */
mfsdp_status mfsdp_plan_head_workspace_bytes(mfsdp_plan_t plan, int64_t entry, int64_t n, int32_t x_type,
                                             int32_t top_k, int32_t grad, uint64_t* bytes);

typedef struct mfsdp_head_logprob_args {
    const void* params;       /* device, the owner's params buffer; 16-byte aligned */
    const void* x;            /* device, n rows of cols elements, aligned to the element size */
    int64_t n;                /* 0 .. 2^22; 0: nothing is done */
    int64_t x_stride;         /* elements from one row of x to the next, >= cols; 0 = cols */
    int32_t x_type;           /* mfsdp_dtype of x */
    int32_t id_type;          /* mfsdp_id_type */
    const void* ids;          /* NULL, or device, n of id_type, aligned to their size */
    int64_t first_id;         /* id of the table's row 0, 0 .. 2^62 */
    float scale;              /* finite */
    int32_t top_k;            /* 0 .. 64; the lists below have as many entries a row */
    mfsdp_head_record* records; /* device, n, written; 8-byte aligned */
    float* logp;              /* NULL, or device fp32 [n] */
    float* entropy;           /* NULL, or device fp32 [n] */
    int64_t* top_ids;         /* device [n][top_k] (first_id + row; -1 where the table has no more rows); may be
                                 NULL when top_k is 0 */
    float* top_logp;          /* NULL, or device fp32 [n][top_k]: their log probabilities (-inf with id -1) */
    float* top_logits;        /* NULL, or device fp32 [n][top_k]: their y, for mfsdp_head_total */
    void* workspace;          /* device, mfsdp_plan_head_workspace_bytes, 256-byte aligned; written before it
                                 is read, so it needs no clearing and may be shared by calls that do not
                                 overlap */
    uint64_t workspace_bytes;
    void* stream;
} mfsdp_head_logprob_args;

/* Enqueue the log probabilities over entry `entry` of the plan (any role).
 * An empty entry gives records without sum or target, log probabilities and
 * entropies 0 and no alternatives.
 * Errors: INVALID_ARGUMENT (null pointer, entry out of range, n, first_id,
 * x_stride, scale or top_k out of range, misaligned buffer), UNSUPPORTED
 * (id_type, x_type, more than 2^20 columns, more than 2^24 - 1 tiles of 128 x
 * 128 logits or table elements or a third as many of 64 x 64 elements of x),
 * WORKSPACE_TOO_SMALL, HIP. */
mfsdp_status mfsdp_head_logprob(mfsdp_plan_t plan, int64_t entry, const mfsdp_head_logprob_args* args);

typedef struct mfsdp_head_total_args {
    const mfsdp_head_record* parts; /* device, [count][n]; 8-byte aligned */
    int64_t count;            /* 1 .. 65536 */
    int64_t n;                /* 0 .. 2^22 */
    mfsdp_head_record* records; /* device, [n], written; may be one of parts */
    float* logp;              /* NULL, or device fp32 [n] */
    float* entropy;           /* NULL, or device fp32 [n] */
    const int64_t* part_top_ids;   /* device [count][n][top_k], of the parts' mfsdp_head_logprob */
    const float* part_top_logits;  /* device [count][n][top_k], likewise */
    int64_t* top_ids;         /* as in mfsdp_head_logprob_args */
    float* top_logp;
    float* top_logits;
    int32_t top_k;            /* 0 .. 64; 0: the five arrays above are not used */
    void* stream;
} mfsdp_head_total_args;

/* Join the records of several entries or owners in their order: the same
 * bits wherever the same records are joined.  Parts are the tables in the
 * order of their ids, for ties among alternatives; a target is in at most one
 * of them.
 * Errors: INVALID_ARGUMENT (null or misaligned pointer, count, n or top_k out
 * of range), HIP. */
mfsdp_status mfsdp_head_total(const mfsdp_head_total_args* args);

typedef struct mfsdp_head_grad_args {
    const void* params;       /* as in mfsdp_head_logprob_args, down to scale */
    const void* x;
    int64_t n;
    int64_t x_stride;
    int32_t x_type;
    int32_t id_type;
    const void* ids;
    int64_t first_id;
    float scale;
    int32_t accumulate;       /* 0: the entry's gradient is written; 1: added to what is there */
    const mfsdp_head_record* records; /* device, n: of mfsdp_head_logprob with the same arguments, or joined */
    const float* dlogp;       /* device fp32 [n]: gradient of the log probabilities */
    const float* dentropy;    /* NULL (zeros), or device fp32 [n]: gradient of the entropies */
    void* dx;                 /* NULL, or device, n rows of cols elements of x_type: written, zeros for padding */
    int64_t dx_stride;        /* elements from one row of dx to the next, >= cols; 0 = cols */
    void* grads;              /* NULL, or device, the owner's grads buffer; 16-byte aligned */
    void* workspace;          /* device, mfsdp_plan_head_workspace_bytes with grad = 1; as in
                                 mfsdp_head_logprob_args */
    uint64_t workspace_bytes;
    void* stream;
} mfsdp_head_grad_args;

/* Enqueue the gradients of x and of the table:
 *   dz_ij = scale * (dlogp_i ([j = t] - p_ij) - dentropy_i p_ij (ln p_ij + entropy_i)),
 *   dx = dz W,  G (+)= dz^T x.
 * Logits are formed again.  Where x and the table are bf16, dz is rounded to
 * bf16, but for a row's entries of 1/32 or more of |scale| (|dlogp| 2 (1 - p_t)
 * + |dentropy| 2 entropy), its sum of |dz| or more, which keep 2^-16 of
 * themselves or better (with records of other operands than the call's they may
 * not); else it is fp32.  The
 * sums are fp32, rounded once to x_type and to the entry's type (after what was
 * there is added).  No rows and accumulate = 0 writes zeros.
 * Errors: as mfsdp_head_logprob, and INVALID_ARGUMENT (records or dlogp NULL
 * or misaligned, accumulate or dx_stride out of range). */
mfsdp_status mfsdp_head_grad(mfsdp_plan_t plan, int64_t entry, const mfsdp_head_grad_args* args);

/* ---- Owner planner (host only) ----
 *
 * "MatrixFSDP" (arXiv 2607.05895), Abstract: a balance-aware owner planner
 * decides which data-parallel rank owns each whole 2D weight, and tensors
 * that are not matrices are grouped onto a few tail owners.  The pages name the
 * planner only; this one reads "balance-aware" as: every tensor goes whole
 * to one owner, an owner's step time is the sum of its tensors' costs, and
 * the plan minimises the largest owner time under a per-owner memory cap.
 *
 * Cost of a tensor: Muon (m = min(rows, cols), n = max): ns_steps * (4 m^2 n
 * + 2 m^3) / flop_rate + rows*cols * (3 es + 2 em + es_ns) / byte_rate (grad
 * read, param read and write, momentum read and write, the Newton-Schulz
 * input write; es = param bytes, em = momentum bytes (4, or 2 with
 * momentum_dtype MFSDP_BF16), es_ns = 2 for bf16 Newton-Schulz, 4 for fp32);
 * AdamW: rows*cols * (3 es + 16) / byte_rate; MFSDP_ROLE_ADAMW8: rows*cols *
 * (3 es + 4) / byte_rate and 16 B for each group of 128 elements.
 * Memory of a tensor on its owner: params and grads (2 es per element),
 * state (em B per element for Muon, 8 for AdamW, a byte for each moment and
 * the scales for MFSDP_ROLE_ADAMW8), and for Muon the
 * Newton-Schulz buffers of mfsdp_plan_create (two X^T of n_p x m_p and A, B
 * of m_p x m_p, m_p and n_p padded to 256, es_ns per element), each region
 * rounded up to 256 bytes.  (The plan's descriptor blob and norm partials,
 * a few bytes per tile, are not counted.)
 *
 * Algorithm: tensors in decreasing cost (ties: larger memory, then lower
 * index) each go to the owner with the least cost so far that has room
 * under the cap (ties: lower owner); then moves and swaps of single tensors
 * off the most loaded owner are applied while they lower the largest owner
 * cost.  Deterministic.  Without a binding cap the first pass alone is
 * within 4/3 of the optimal largest cost (longest-processing-time bound).
 */
typedef struct mfsdp_tensor {
    int64_t rows, cols;       /* 1D tensors: rows = 1; rows*cols = 0 is an empty tensor */
    int32_t dtype;            /* mfsdp_dtype of params and grads */
    int32_t role;             /* mfsdp_role, resolved as in mfsdp_entry */
} mfsdp_tensor;

typedef struct mfsdp_partition_params {
    int32_t n_owners;         /* >= 1 */
    int32_t ns_steps;         /* Newton-Schulz iterations in a Muon tensor's cost, >= 0 */
    int32_t ns_precision;     /* 0: bf16 Newton-Schulz buffers, 1: fp32 */
    int32_t momentum_dtype;   /* Muon momentum storage, as in mfsdp_hparams: MFSDP_F32 (0) or MFSDP_BF16 */
    uint64_t mem_cap_bytes;   /* per-owner memory cap; 0 = none */
    double flop_rate;         /* FLOP/s of the Newton-Schulz contractions, > 0 */
    double byte_rate;         /* bytes/s of the elementwise passes, > 0 */
} mfsdp_partition_params;

typedef struct mfsdp_tensor_place {
    int32_t owner;            /* 0 .. n_owners-1 */
    int32_t role;             /* resolved: MFSDP_ROLE_MUON, MFSDP_ROLE_ADAMW or MFSDP_ROLE_ADAMW8 (empty
                                 tensors: ADAMW) */
    uint64_t offset;          /* bytes into the owner's flat parameter buffer: the owner's tensors in
                                 input order, each at a 256-byte aligned offset */
    double cost;              /* seconds, by the model above */
    uint64_t mem_bytes;       /* by the model above */
} mfsdp_tensor_place;

/* Assign n tensors to owners.  place: n entries, written on success.
 * owner_cost, owner_mem_bytes, owner_param_bytes: NULL or n_owners entries
 * each (sum of costs, sum of memory, end of the last tensor in the owner's
 * flat buffer).  Each owner's tensors, in input order at their offsets, form
 * a table mfsdp_plan_create accepts.
 * Errors: INVALID_ARGUMENT (null pointer, n < 0, n_owners < 1, negative
 * dimension, ns_steps < 0, rates not positive and finite), UNSUPPORTED
 * (dtype, role, ns_precision, a tensor larger than the memory cap, or no
 * owner with room left for a tensor). */
mfsdp_status mfsdp_owner_partition(const mfsdp_tensor* tensors, int64_t n, const mfsdp_partition_params* pp,
                                   mfsdp_tensor_place* place, double* owner_cost, uint64_t* owner_mem_bytes,
                                   uint64_t* owner_param_bytes);

/* ---- Owner-shard checkpoint resharding (host only) ----
 *
 * "MatrixFSDP" (arXiv 2607.05895), Abstract: owner-shard checkpoint
 * resharding.  A checkpoint holds whole tensors; these two calls copy one
 * owner's tensors and their optimizer state between the owner's flat
 * buffers (laid out by its plan) and one buffer per tensor, in host memory,
 * byte for byte (no conversion).  Resharding to another owner count is
 * gather from every old owner, mfsdp_owner_partition for the new count,
 * scatter into every new owner; every value comes back bit-exact.
 *
 * For entry i of the plan's table (numel = rows*cols):
 *   tensors[i]  numel parameter elements in the entry's dtype, row-major;
 *   state1[i]   numel elements: Muon momentum (the plan's momentum_dtype), or AdamW first moment (fp32;
 *               MFSDP_ROLE_ADAMW8: the codes and scales as they lie in the state, from state_offset to the
 *               last scale, numel rounded up to 256 and 4 bytes for each group of 128 elements);
 *   state2[i]   numel fp32: AdamW second moment (likewise; unused for Muon).
 * Any array pointer may be NULL (that part is not copied); an element may be
 * NULL where numel is 0 or the part does not apply.  params / state are the
 * owner's buffers (param_bytes >= the end of its last tensor, state_bytes >=
 * mfsdp_plan_state_bytes).  Bytes outside the tensors and state regions are
 * not touched.
 * Errors: INVALID_ARGUMENT (null plan, a needed buffer or element NULL,
 * buffer too small). */
mfsdp_status mfsdp_owner_gather(mfsdp_plan_t plan, const void* params, uint64_t param_bytes, const void* state,
                                uint64_t state_bytes, void* const* tensors, void* const* state1,
                                void* const* state2);
mfsdp_status mfsdp_owner_scatter(mfsdp_plan_t plan, const void* const* tensors, const void* const* state1,
                                 const void* const* state2, void* params, uint64_t param_bytes, void* state,
                                 uint64_t state_bytes);

/* ---- Measurement probes (NOT part of the optimizer step) ----
 *
 * The two calls below compute nothing of the owner step and touch none of
 * a plan's buffers.  They exist so that a benchmark can report, on the
 * same GPU and in the same run, the rates the part sustains for the two
 * kinds of work the step does (bf16 MFMA on Gaussian data; HBM streaming),
 * beside the published peaks.  A caller that only runs the optimizer never
 * needs them. */

/* Measurement support (not part of the step): enqueue on `stream` a
 * register-only loop of bf16 MFMAs (v_mfma_f32_32x32x16_bf16, fp32
 * accumulate) over `blocks` blocks of 4 waves, each wave running `iters`
 * iterations of 32 MFMAs on 16 operand fragments per lane taken from
 * `operands` (device memory, operand_bytes >= 1024, a multiple of 16,
 * 16-byte aligned; read only).  The MFMA clock depends on the operand data,
 * so with the contractions' own kind of data (Gaussian bf16) the elapsed
 * time gives the rate the part sustains for them, as opposed to the
 * published dense peak.  sink: device, blocks * 4 floats, written.  *flops
 * (optional) receives the FLOPs enqueued.  The caller times the launch (for
 * example with events on `stream`).  Errors: INVALID_ARGUMENT, HIP. */
mfsdp_status mfsdp_probe_mfma_bf16(const void* operands, uint64_t operand_bytes, int32_t blocks, int32_t iters,
                                   float* sink, void* stream, double* flops);

/* Measurement support (not part of the step): enqueue on `stream` one pass
 * of 16-byte accesses over `bytes` of device memory: mode 0 reads src, mode
 * 1 writes dst, mode 2 copies src to dst (as many bytes read as written, the
 * mix of the elementwise phases).  2048 blocks of 256 threads, each walking
 * contiguous 32 KB chunks with 8 accesses in flight per thread.  The caller
 * times the launch; the
 * bytes moved are `bytes` (modes 0, 1) or 2 * bytes (mode 2).  sink: device,
 * 8192 floats, written.  Errors: INVALID_ARGUMENT (mode, NULL buffer, bytes
 * not a nonzero multiple of 16, misaligned buffer), HIP. */
mfsdp_status mfsdp_probe_hbm(void* dst, const void* src, uint64_t bytes, int32_t mode, float* sink, void* stream);

/* Static description of a status code. */
const char* mfsdp_status_string(mfsdp_status status);

/* Thread-local description of the last error on this thread ("" if none). */
const char* mfsdp_last_error_message(void);

#ifdef __cplusplus
}
#endif

#endif /* MFSDP_H */
