/*
 * hc.h -- C ABI of the MI355X (gfx950) emulated ring AllReduce data path and
 * the lossless bf16 exponent codecs, HCZ1 (fixed-length codes) and HCE1
 * (Huffman codes), and of the operators around the exchange: gradient norm and
 * clipping, embedding lookup and gradient, the norm of rows, routing to experts,
 * tokens by expert, and the optimizer's step (library: libhc.so).
 *
 * The ring is emulated on ONE GPU: R "ranks" are R device buffers in the same
 * HBM; a hop's link transfer is the receiver reading the sender's buffer.  All
 * calls are asynchronous and stream ordered, like the NCCL-style
 * allreduce(sendbuf, recvbuf, count, dtype, op, comm, stream) interface that
 * "CCCL: In-GPU Compression-Coupled Collective Communication" keeps (section
 * 3, "CCCL Overview"); argument errors are found on the host before anything
 * is enqueued.  The only reduction is sum.
 *
 * Memory and ownership
 *   - Every data pointer below is a DEVICE pointer unless it says HOST.
 *     sendbufs/recvbufs are HOST arrays of nranks DEVICE pointers.
 *   - The caller owns every buffer, workspace and stream.  The library never
 *     allocates or frees device memory and keeps no state between calls
 *     except a thread-local copy of the last error message, and the static
 *     device array (about 1 MiB per GPU) of hc_compress_bf16_noalloc.
 *   - Alignment (else HC_ERR_INVALID_ARGUMENT): rank buffers of the
 *     uncompressed ring calls to their element size (16-byte alignment of
 *     every slice takes the vector path, anything else a per-element path);
 *     every pointer of the codec and compressed calls to 16 bytes.
 *   - Buffers of different ranks must not overlap, except for the in-place
 *     forms stated per call.  Sizes are in elements unless named *_bytes.
 *
 * Errors
 *   - HC_ERR_INVALID_ARGUMENT: NULL pointer, nranks outside 1..HC_MAX_RANKS,
 *     misaligned pointer, count constraints, unknown dtype or option value.
 *   - HC_ERR_INSUFFICIENT_CAPACITY: workspace or output capacity too small.
 *   - HC_ERR_UNSUPPORTED: an option the call cannot honour (the copy engine
 *     for hc_compressed_allreduce, or in a process whose HIP runtime would not
 *     put the copies on the DMA engines).
 *   - HC_ERR_DEVICE: a HIP call failed; hc_last_error() has the text.
 *   - HC_ERR_CORRUPT_STREAM: only ever written by the device into the
 *     caller's status word of hc_decompress_bf16 / hc_decompress_bf16_entropy.
 *   The first three are found on the host before anything is enqueued.  An
 *   HC_ERR_DEVICE return can follow launches of the same call that were
 *   already enqueued; the stream then holds a partial operation.  No call
 *   aborts or throws across the ABI.
 */
#ifndef HC_H
#define HC_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HC_MAX_RANKS 64
#define HC_BLOCK_ELEMS 16384u        /* codec block: 16384 bf16 = 32 KB */
#define HC_HCZ1_MAGIC 0x315A4348u    /* "HCZ1" little-endian */

/* Every enum of this header also names the ends of the int32 range (the
 * *_RANGE_MIN_ / *_RANGE_MAX_ entries, never valid arguments), so that any
 * 32-bit value a C caller passes is a value of the type in C++ as well: the
 * library's checks then reject unknown values instead of reading a value the
 * type cannot hold. */
typedef enum {
    HC_SUCCESS = 0,
    HC_ERR_INVALID_ARGUMENT = 1,
    HC_ERR_UNSUPPORTED = 2,
    HC_ERR_INSUFFICIENT_CAPACITY = 3,
    HC_ERR_CORRUPT_STREAM = 4,
    HC_ERR_DEVICE = 5,
    HC_STATUS_RANGE_MIN_ = INT32_MIN,
    HC_STATUS_RANGE_MAX_ = INT32_MAX
} hc_status_t;

typedef enum {
    HC_F32 = 0,
    HC_BF16 = 1,
    HC_DTYPE_RANGE_MIN_ = INT32_MIN,
    HC_DTYPE_RANGE_MAX_ = INT32_MAX
} hc_dtype_t;

/* Options.  Pass NULL for the defaults (all fields zero mean default).
 *   chunk_fraction: chunk size as a fraction of the per-rank buffer, default
 *     0.01 ("a chunk is about 1% of the data", "ResCCL: Resource-Efficient
 *     Scheduling for Collective Communication", section 1).  The chunk is
 *     rounded up to 1024 elements (uncompressed) or to whole 16384-element
 *     codec blocks (compressed).  It changes scheduling only, never a value.
 *   cu_budget: 0 = size grids for the whole GPU; k > 0 = launch a persistent
 *     grid sized for k compute units (pair it with a stream from
 *     hc_stream_create_cu_budget(k)).
 *   Environment, read at every call (none is required):
 *     HC_CHUNK_FRACTION (a number in (0, 1]) and HC_CU_BUDGET (an integer in
 *       0..4096) replace the two defaults above where opts is NULL or leaves
 *       the field 0; a malformed value makes every call that takes options
 *       return HC_ERR_INVALID_ARGUMENT, naming the variable.  (The compressed
 *       allreduce, which takes no CU budget, ignores HC_CU_BUDGET.)
 *     HC_LOG (anything but empty or "0") prints each call's plan and each
 *       ring-step launch's shape and tile policy to stderr, one line each,
 *       prefixed "hc: ".
 *     HC_STREAM_STORE_MIN_BYTES (a whole number; default 335544320, 320 MiB):
 *       a ring-step launch that writes at least this many bytes on all CUs
 *       moves one 16-byte vector per lane with non-temporal stores, since its
 *       output no longer fits MI355X's 256 MB Infinity Cache for the next
 *       step to read back; smaller launches use two vectors and ordinary
 *       stores, CU-budget launches four.  Values are the same either way.
 *     HC_CHAIN_MAX_BYTES (a whole number; default 268435456, 256 MiB): an
 *       hc_allreduce whose R buffers hold at most this many bytes runs as
 *       one launch in which each workgroup carries one tile through every
 *       hop in ring order (unless step_events or copy_engine ask for per-step
 *       launches); larger ones launch once per ring step.  When set, it is
 *       also hc_compressed_allreduce's threshold (bytes of its R buffers),
 *       which otherwise always runs as one launch.  Values and wire bytes are
 *       the same either way.
 *     HC_LOOKBACK_SPIN_LIMIT (1..2^32-1; default 2^22): polls a compress
 *       block's look-back makes before the call gives up (see
 *       hc_compress_bf16).
 *   step_events / n_step_events: optional timing hook.  When step_events is
 *     not NULL it holds n_step_events caller-created HIP events (created
 *     with timing enabled), used as step_event_mode says, with steps =
 *     hc_step_count(op, nranks).  Too few events is HC_ERR_INVALID_ARGUMENT.
 *     NULL records nothing; so does a call with nothing to do (count 0).
 *   step_event_mode: 0 = boundaries: step_events[k] is recorded on the stream
 *     right before ring step k and step_events[steps] after the last step
 *     (steps + 1 events), so an interval also holds the gap between two
 *     launches.  1 = kernel stamps (2 * steps events): step k's first kernel
 *     stamps step_events[2k] with its start time and its kernels stamp
 *     step_events[2k+1] with their end time (hipExtLaunchKernel), so an
 *     interval is the step's kernel execution as a kernel trace reports it.
 *     A step that runs no kernel (copy-engine copies; the all-gather step
 *     that the last reduce-scatter step already did) records both events on
 *     the stream around what it enqueues.  Other values are
 *     HC_ERR_INVALID_ARGUMENT.
 *   copy_engine: 0 = all-gather copy steps run as copy kernels on the
 *     compute units; 1 = they run on the GPU's DMA copy engines
 *     (hipMemcpyAsync of kind hipMemcpyDeviceToDeviceNoCU, stream ordered,
 *     one copy per receiver and step), holding no compute unit at all.  This
 *     is the offload of "HOCCL: Offloading Collective Communication from GPU
 *     Cores to Accelerate Distributed Training" (section 2): a copy can leave
 *     the cores, a reduction cannot, so reduce-scatter steps always run on
 *     the compute units.  Applies to hc_all_gather, to the all-gather half of
 *     hc_allreduce and to one-rank copies; hc_compressed_allreduce decodes
 *     during its all-gather and rejects it (HC_ERR_UNSUPPORTED).  Other
 *     values are HC_ERR_INVALID_ARGUMENT.  Which engine serves such a copy
 *     is the HIP runtime's choice: measured on MI355X, the ROCm 7.2 runtime
 *     in /opt/rocm uses the DMA engines (about 60 GB/s per copy, one copy at
 *     a time per stream), while the 7.0 runtime bundled with the PyTorch
 *     2.10 wheel runs the same calls as blit kernels on the compute units.
 *     So a call with copy_engine = 1 in a process whose HIP runtime is older
 *     than 7.2 returns HC_ERR_UNSUPPORTED (nothing is enqueued) instead of
 *     silently using the compute units; hc_copy_engine_available() tells in
 *     advance. */
typedef struct {
    double chunk_fraction;
    int32_t cu_budget;
    int32_t n_step_events;
    hipEvent_t *step_events;
    int32_t copy_engine;
    int32_t step_event_mode;
} hc_opts_t;

/*
 * hc_allreduce -- ring AllReduce (sum) over nranks emulated ranks.
 * "Breaking the computation and communication abstraction barrier in
 * distributed machine learning workloads" ("The idea"): AllReduce is a
 * ReduceScatter followed by an AllGather, and every rank ends with the same
 * full result (local -> replicated).  Runs R-1 recvReduceCopy steps then R-1
 * copy steps ("ResCCL ...", section 1).  At reduce-scatter step s receiver q
 * folds slice (q-2-s) mod R received from q-1 into its own data; at
 * all-gather step s it copies slice (q-1-s) mod R from q-1.  Element i of
 * slice j is therefore hop(...hop(x[j+1][i], x[j+2][i])..., x[j][i]).
 *   fp32: hop = one IEEE binary32 add (round to nearest even, subnormals
 *         kept); bf16: both operands widened exactly to fp32, one add, the
 *         sum rounded to bf16 nearest-even.  A NaN sum becomes the canonical
 *         quiet NaN (0x7FC00000 / 0x7FC0).
 *   sendbufs[r], recvbufs[r]: count elements each.  In place is allowed:
 *   sendbufs[r] == recvbufs[r] for every r.  Slices are ceil(count/R) long
 *   (the last ones short or empty when R does not divide count).
 *   Schedule: up to HC_CHAIN_MAX_BYTES of buffers (256 MiB by default) the
 *   hops run in one launch, each workgroup taking one tile of one slice
 *   through all 2(R-1) hops in order ("ResCCL ...", section 3: dependencies
 *   exist only within a chunk); above it, or with step_events or
 *   copy_engine, one launch per ring step.  Both make the same reads and
 *   writes and give the same bits.
 */
hc_status_t hc_allreduce(void *const *sendbufs, void *const *recvbufs, size_t count,
                         hc_dtype_t dtype, int nranks, const hc_opts_t *opts,
                         hipStream_t stream);

/*
 * hc_allreduce_bf16_f32carry -- the bf16 ring AllReduce of hc_allreduce with
 * the other reading of "fp32 accumulation, bf16 round-to-nearest-even
 * output": the reduce-scatter carries fp32 partials and the sum is rounded to
 * bf16 once, by the slice's owner at the last reduce-scatter step.  Same ring,
 * slices, chunks and fold order as hc_allreduce: element i of slice j is
 * bf16(((f(x[j+1][i]) + f(x[j+2][i])) + ...) + f(x[j][i])) with f the exact
 * widening and every + one fp32 add (a NaN sum becomes the canonical NaN);
 * the all-gather copies the bf16 result.  With 2 ranks this equals
 * hc_allreduce; with 1 it is a copy.  Partials cost 4 bytes instead of 2, so
 * a middle reduce-scatter hop moves 10 bytes per element instead of 6.
 *   sendbufs[r], recvbufs[r]: count bf16 elements each; in place is allowed
 *   (sendbufs[r] == recvbufs[r] for every r).
 *   d_ws: >= hc_workspace_bytes(HC_OP_ALLREDUCE_F32_CARRY, count, nranks,
 *   HC_BF16) bytes, 16-byte aligned, overlapping no rank buffer: two fp32
 *   partial slots per rank (ping-pong between steps).  May be NULL when
 *   nranks <= 2 (no partial is stored).  The caller owns it; its contents
 *   after the call are unspecified.
 *   Errors as hc_allreduce, plus HC_ERR_INSUFFICIENT_CAPACITY for a short
 *   workspace; nothing is enqueued on an argument error.
 */
hc_status_t hc_allreduce_bf16_f32carry(void *const *sendbufs, void *const *recvbufs, size_t count,
                                       int nranks, void *d_ws, size_t ws_bytes, const hc_opts_t *opts,
                                       hipStream_t stream);

/*
 * hc_reduce_scatter -- ring ReduceScatter (sum): rank r receives slice r of
 * the elementwise sum ("Breaking the computation and communication
 * abstraction barrier ...", "The idea": each rank keeps its 1/N slice;
 * local -> sliced).  Same hop and fold order as hc_allreduce.
 *   sendbufs[r]: recvcount*nranks elements; recvbufs[r]: recvcount elements.
 *   In place is allowed: recvbufs[r] == sendbufs[r] + r*recvcount elements.
 *   d_ws: device workspace of at least hc_workspace_bytes(HC_OP_REDUCE_SCATTER,
 *   recvcount*nranks, nranks, dtype) bytes; it holds the partials in flight.
 */
hc_status_t hc_reduce_scatter(void *const *sendbufs, void *const *recvbufs, size_t recvcount,
                              hc_dtype_t dtype, int nranks, void *d_ws, size_t ws_bytes,
                              const hc_opts_t *opts, hipStream_t stream);

/*
 * hc_all_gather -- ring AllGather: every rank receives the concatenation of
 * all ranks' sendbufs, slice j = rank j's data (sliced -> replicated, same
 * page).  Step 0 also copies each rank's own data into its own output.
 *   sendbufs[r]: sendcount elements; recvbufs[r]: sendcount*nranks elements.
 *   In place is allowed: sendbufs[r] == recvbufs[r] + r*sendcount elements.
 */
hc_status_t hc_all_gather(void *const *sendbufs, void *const *recvbufs, size_t sendcount,
                          hc_dtype_t dtype, int nranks, const hc_opts_t *opts,
                          hipStream_t stream);

/*
 * hc_allreduce_sgd -- the allreduce of gradients fused with an SGD update of
 * the weights: "Breaking the computation and communication abstraction
 * barrier in distributed machine learning workloads" ("The idea") moves an
 * elementwise optimizer update between the ReduceScatter and the AllGather,
 * so that each rank updates only the slice whose sum it holds and the
 * AllGather spreads updated weights instead of summed gradients.
 *   grads[r], weights[r]: count elements each, dtype HC_F32 or HC_BF16,
 *     element-aligned; all 2*nranks buffers pairwise disjoint.
 *   g = the ring allreduce sum of the grads, exactly as hc_allreduce computes
 *     it (same fold order, same per-hop rounding).  For slice j (the
 *     hc_allreduce slicing) the new weight is weights[j] - lr*g, the product
 *     and the difference rounded once each in fp32 (bf16: operands widened
 *     exactly, result rounded to nearest even; a NaN result is the canonical
 *     quiet NaN).  On return every weights[r] holds the new weights; slice j
 *     comes from rank j's weights before the call (when every rank holds the
 *     same weights, as in data-parallel training, that is simply w - lr*g).
 *   grads are the reduction's scratch: their contents after the call are
 *     partial sums, unspecified.
 *   lr: any finite float (not finite: HC_ERR_INVALID_ARGUMENT).
 *   opts: chunk_fraction, cu_budget, step_events (2*(nranks-1) steps, 1 for
 *     one rank) and copy_engine (the all-gather copies) as for hc_allreduce.
 * Asynchronous on stream; argument errors are detected before anything is
 * enqueued.
 */
hc_status_t hc_allreduce_sgd(void *const *grads, void *const *weights, size_t count, hc_dtype_t dtype,
                             int nranks, float lr, const hc_opts_t *opts, hipStream_t stream);

/* Largest HCZ1 stream for n bf16 elements (every block stored raw):
 * 32 + round_up(8*n_blocks, 16) + sum over blocks of 16 + round_up(2*m, 16). */
size_t hc_compress_bound_bf16(size_t n);

/*
 * hc_compress_bf16 -- lossless bf16 compression into one HCZ1 stream.
 * "CCCL ...", section 4.1: sign and fraction are sent raw, the 8-bit exponent
 * is coded from a frequency table; section 4.3: each block builds its own
 * table and uses fixed-length codes; section 4.4: one pass, each block writes
 * straight into the output; section 5 "Handling data alignment": a partial
 * tail block is stored raw.
 * Format (little-endian, all padding zero): 32-byte header {u32 magic
 * 0x315A4348, u32 block_elems 16384, u64 n, u32 n_blocks, u32 flags 0, u64
 * total_bytes}; u64 rec_off[n_blocks] padded to 16 bytes; the records in
 * block order.  Record: 16-byte header {u8 mode (0 raw, 1 coded), u8 b, u16
 * 0, u32 m, u32 n_esc, u32 rec_bytes}; raw: m words padded to 16; coded
 * (m == 16384 only): dictionary of the K = 2^b-1 most frequent exponents
 * (count descending, exponent ascending) in max(16, 2^b) bytes; b code
 * planes of 2048 bytes (bit i%8 of byte i/8 of plane k = bit k of code[i],
 * code = dictionary index or K for an escape); the sign/fraction plane
 * sm[i] = sign<<7 | fraction (16384 bytes); the escaped exponents in index
 * order, padded to 16.  b is the smallest 1..7 with the fewest bytes; a block
 * is raw when that is not below 16 + 32768 bytes.
 *   d_in: n bf16 words.  d_out: out_cap >= hc_compress_bound_bf16(n) bytes.
 *   d_out_bytes: one device u64, receives the stream size; it receives 0
 *   (and the stream is not valid) only if a block's wait for its
 *   predecessors' sizes ran past its bound (about four million polls).
 *   d_ws: >= hc_workspace_bytes(HC_OP_COMPRESS, n, 1, HC_BF16) bytes (block
 *   offsets in flight).  Calls sharing a workspace must not overlap.
 */
hc_status_t hc_compress_bf16(const uint16_t *d_in, size_t n, void *d_out, size_t out_cap,
                             uint64_t *d_out_bytes, void *d_ws, size_t ws_bytes,
                             hipStream_t stream);

/*
 * hc_compress_bf16_noalloc -- hc_compress_bf16 without a workspace argument,
 * for callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation).  The same
 * kernels, the same stream byte for byte.  The look-back workspace is a
 * static device array inside the library (8320 + 8 * 131072 bytes, about
 * 1 MiB), one copy per GPU, held until the process ends; its address is
 * taken once per device on that device's first call.  The call allocates
 * nothing (no hipMalloc, no allocating library routine) and clears the part
 * of the array it uses with a fill kernel on the stream.
 *   n: at most 131072 * 16384 = 2^31 elements, else
 *   HC_ERR_INSUFFICIENT_CAPACITY (nothing is enqueued).
 *   Every call on one GPU shares that GPU's array: calls that overlap on one
 *   GPU (on different streams, or from several threads) race and may write
 *   wrong streams; order them on one stream.
 *   Other arguments and errors as hc_compress_bf16.
 */
hc_status_t hc_compress_bf16_noalloc(const uint16_t *d_in, size_t n, void *d_out, size_t out_cap,
                                     uint64_t *d_out_bytes, hipStream_t stream);

/*
 * hc_compress_bf16_scoped -- hc_compress_bf16 with code tables shared by
 * groups of blocks.  "CCCL ...", section 4.3 weighs one global table (more
 * work before any block can be coded) against a table per block (the
 * overhead of many small tables) and picks the per-block one; this call
 * makes the choice a parameter so both ends can be measured.
 *   table_blocks: G >= 1 groups the full blocks in order, G at a time (the
 *   last group may be shorter); 0 puts every full block in one group.  A
 *   group's dictionary is its summed exponent histogram ranked count
 *   descending, exponent ascending; its b (1..7) is the one with the fewest
 *   summed coded bytes over its blocks, ties to the smaller b.  Each full
 *   block is coded with its group's dictionary and b unless that record
 *   would not be below 16 + 32768 bytes, then it is raw; the partial tail
 *   block is raw.  Each record still carries its dictionary, so the result
 *   is an ordinary HCZ1 stream for hc_decompress_bf16, and G = 1 writes the
 *   same bytes as hc_compress_bf16.
 *   d_ws: >= hc_workspace_bytes(HC_OP_COMPRESS_SCOPED, n, 1, HC_BF16) bytes
 *   (independent of G).  Other arguments and errors as hc_compress_bf16.
 */
hc_status_t hc_compress_bf16_scoped(const uint16_t *d_in, size_t n, void *d_out, size_t out_cap,
                                    uint64_t *d_out_bytes, size_t table_blocks, void *d_ws,
                                    size_t ws_bytes, hipStream_t stream);

/*
 * hc_compress_bf16_staged -- hc_compress_bf16 in three global rounds, the
 * design "CCCL ...", section 4.4 replaces: every block encodes into a
 * fixed-size temporary slot (16 + 32768 bytes), a prefix over the record
 * sizes places the records, and a coalescing copy writes them into the
 * stream.  The same encoder and format: the stream equals hc_compress_bf16's
 * byte for byte.  For measuring the single-round design against it.
 *   d_ws: >= hc_workspace_bytes(HC_OP_COMPRESS_STAGED, n, 1, HC_BF16) bytes
 *   (the slots, about 2.0 bytes per element).  Other arguments and errors as
 *   hc_compress_bf16.
 */
hc_status_t hc_compress_bf16_staged(const uint16_t *d_in, size_t n, void *d_out, size_t out_cap,
                                    uint64_t *d_out_bytes, void *d_ws, size_t ws_bytes,
                                    hipStream_t stream);

/*
 * hc_compress_bf16_entropy -- lossless bf16 compression with an entropy-coded
 * exponent: one "HCE1" stream.  "CCCL ...", section 4.1 codes the exponent
 * from a frequency table with sign and fraction raw, and section 6.5
 * compares the fixed-length core with an entropy coder whose output is
 * smaller by under 7%; here each full block codes its exponents with its own
 * canonical Huffman code (lengths limited to 12 bits; codes assigned as in
 * RFC 1951, section 3.2.2), the same container and single-pass writer as
 * hc_compress_bf16.
 * Format (little-endian, all padding zero): the HCZ1 container with magic
 * 0x31454348.  Record: 16-byte header {u8 mode (0 raw, 2 coded), u8 lmax (12
 * coded, 0 raw), u16 n_sym (exponents present; 0 raw), u32 m, u32 n_words
 * (0 raw), u32 rec_bytes}; raw: m words padded to 16; coded (m == 16384
 * only): code length of exponent e (0 absent, 1..12) in the low nibble of
 * byte 16 + e/2 for even e, the high nibble for odd e; bytes 144..16527 the
 * sign/fraction plane sm[i] = sign<<7 | fraction; from byte 16528 the
 * n_words 32-bit words, padded to 16: rec_bytes = 16528 +
 * round_up(4*n_words, 16).  A full block is coded when that is below
 * 16 + 32768 bytes, else raw; the partial tail block is raw.
 * Code construction: leaves in increasing count, equal counts by decreasing
 * exponent; the lighter of (next leaf, next merged node) is taken first, a
 * leaf on a tie; a single exponent gets length 1.  Lengths over 12 become 12,
 * then while the Kraft sum exceeds 1 the longest code shorter than 12
 * (ties: smallest count, then largest exponent) grows by one bit.
 * Word layout: 64 lanes, lane j takes elements 64*i + j (step i = 0..255);
 * its codes, most significant bit first, form a bit stream whose bit b is bit
 * b%32 of its word b/32.  Word w of a lane is stored at the first step whose
 * code ends past bit 32*w of that stream, and the words are stored in (that
 * step, lane) order -- the order in which a decoder running the 64 lanes in
 * lockstep needs them.
 *   d_ws: >= hc_workspace_bytes(HC_OP_COMPRESS_ENTROPY, n, 1, HC_BF16)
 *   bytes.  Other arguments and errors as hc_compress_bf16 (the bound is
 *   hc_compress_bound_bf16(n)).
 */
hc_status_t hc_compress_bf16_entropy(const uint16_t *d_in, size_t n, void *d_out, size_t out_cap,
                                     uint64_t *d_out_bytes, void *d_ws, size_t ws_bytes,
                                     hipStream_t stream);

/*
 * hc_decompress_bf16_entropy -- exact inverse of hc_compress_bf16_entropy.
 * Arguments and errors as hc_decompress_bf16; besides the container, a coded
 * record is rejected when its lengths exceed 12 or break the Kraft
 * inequality, n_sym disagrees with them, a code is missing, the words do not
 * run out exactly at the last code, or a padding bit is set.
 */
hc_status_t hc_decompress_bf16_entropy(const void *d_in, size_t in_bytes, uint16_t *d_out, size_t n,
                                       int32_t *d_status, hipStream_t stream);

/*
 * hc_decompress_bf16 -- exact inverse of hc_compress_bf16.
 *   d_in: in_bytes readable bytes holding a stream of n elements (the stream
 *   may be shorter than in_bytes).  d_out: n bf16 words.  d_status: one
 *   device int32, required; set to HC_SUCCESS, or to HC_ERR_CORRUPT_STREAM
 *   when any field fails validation (magic, block size, n, block count,
 *   contiguous in-bounds offsets, record sizes against the format, b in
 *   1..7, escape count, zero padding) -- then d_out is left all zero.  Reads
 *   never go past in_bytes, whatever the stream holds.
 */
hc_status_t hc_decompress_bf16(const void *d_in, size_t in_bytes, uint16_t *d_out, size_t n,
                               int32_t *d_status, hipStream_t stream);

/*
 * hc_compressed_allreduce -- the ring of hc_allreduce on bf16 with every hop
 * payload sent compressed ("CCCL ...", section 5, "Selective compression":
 * the sender compresses what it sends, the receiver decompresses what it
 * receives and reduces it with its own uncompressed data).  Reduce-scatter
 * hop: decompress -> bf16 hop -> compress (the last one also writes the
 * output); all-gather hop: decompress into the output and forward the same
 * bytes.  Chunks are whole codec blocks; a slice's unaligned end travels as a
 * raw block.  Lossless, so the result is bit-identical to hc_allreduce.
 *   sendbufs/recvbufs: as hc_allreduce (bf16 only; in place allowed).
 *   d_ws: >= hc_workspace_bytes(HC_OP_COMPRESSED_ALLREDUCE, count, nranks,
 *   HC_BF16) bytes: two wire buffers per rank, one fixed-size slot per codec
 *   block (the preallocated regions of "CCCL ...", section 4.4).
 *   d_wire_bytes: optional device u64; receives the bytes that would cross
 *   the links: the sum over every (hop, chunk) stream of its HCZ1 size.
 *   Schedule: one launch, one workgroup per codec block and slice, each
 *   carrying its block through every hop in ring order, with the wire slots
 *   indexed by slice; with step_events, or beyond HC_CHAIN_MAX_BYTES when that
 *   is set, one launch per ring step.  Same records, wire bytes and output
 *   either way.
 */
hc_status_t hc_compressed_allreduce(void *const *sendbufs, void *const *recvbufs, size_t count,
                                    int nranks, void *d_ws, size_t ws_bytes,
                                    uint64_t *d_wire_bytes, const hc_opts_t *opts,
                                    hipStream_t stream);

typedef enum {
    HC_OP_REDUCE_SCATTER = 0,
    HC_OP_COMPRESS = 1,
    HC_OP_COMPRESSED_ALLREDUCE = 2,
    HC_OP_ALLREDUCE = 3,
    HC_OP_ALL_GATHER = 4,
    HC_OP_COMPRESS_SCOPED = 5,
    HC_OP_COMPRESS_ENTROPY = 6,
    HC_OP_COMPRESS_STAGED = 7,
    HC_OP_ALLREDUCE_F32_CARRY = 8,
    HC_OP_RANGE_MIN_ = INT32_MIN,
    HC_OP_RANGE_MAX_ = INT32_MAX
} hc_op_t;

/* Workspace bytes for an operation; count = elements per rank buffer
 * (the send buffer for reduce-scatter, the input for compress).  Returns 0
 * on invalid arguments and for operations that need no workspace. */
size_t hc_workspace_bytes(hc_op_t op, size_t count, int nranks, hc_dtype_t dtype);

/* Ring steps of an operation (for hc_opts_t.step_events): allreduce 2(R-1),
 * reduce-scatter R-1, all-gather R-1 (step 0 includes the local copies),
 * compressed allreduce 2R-1 (the first compression is step 0); an operation
 * over one rank counts 1.  Returns -1 for an unknown op or nranks. */
int hc_step_count(hc_op_t op, int nranks);

/*
 * hc_stream_create_cu_budget -- a HIP stream whose kernels may run only on k
 * compute units (hipExtStreamCreateWithCUMask, default priority), for
 * running a collective beside compute on fewer CUs; "HOCCL: Offloading
 * Collective Communication from GPU Cores to Accelerate Distributed Training"
 * (section 2) measures the share of cores such traffic holds while compute
 * runs.  The k CUs are spread evenly over the GPU's XCDs and shader engines
 * (measured with hc_cu_census: k = 8, 16, 32, 64 give exactly k CUs, k/8 on
 * every XCD).  *out receives the stream; the caller destroys it with
 * hc_stream_destroy.  Same as hc_stream_create_cu_range(0, k, out).
 */
hc_status_t hc_stream_create_cu_budget(int k, hipStream_t *out);

/* A stream limited to CU mask bits [first, first + k) (0 <= first, k >= 1,
 * first + k <= the CU count; else HC_ERR_INVALID_ARGUMENT).  Bits are handed
 * out round-robin over the XCDs, so a run is an even spread and
 * hc_stream_create_cu_range(k, ncu - k) holds exactly the CUs that
 * hc_stream_create_cu_budget(k) leaves free: compute on the one beside
 * communication on the other shares no CU. */
hc_status_t hc_stream_create_cu_range(int first, int k, hipStream_t *out);
hc_status_t hc_stream_destroy(hipStream_t stream);

/*
 * hc_cu_census -- where the workgroups of a launch on `stream` run: the
 * evidence that a CU-budget stream holds exactly the compute units it was
 * given ("HOCCL ...", section 2: the share of cores that communication holds
 * while compute runs is the quantity measured).  Launches n_workgroups
 * one-wave workgroups; each holds its CU for hold_us microseconds (a bounded
 * wait, so that the launch spreads over every CU the stream may use), then
 * writes d_ids[2w] = its HW_ID register (bits 8..15 hold the CU, shader
 * array and shader engine numbers) and d_ids[2w + 1] = its XCC_ID register
 * (bits 0..3: the XCD).  A CU is identified by (XCC_ID & 15, HW_ID bits
 * 8..15).
 *   d_ids: 2 * n_workgroups device u32, 4-byte aligned.  n_workgroups:
 *   1..65536; hold_us: 0..100000.  Asynchronous on stream.
 */
hc_status_t hc_cu_census(uint32_t *d_ids, int n_workgroups, int hold_us, hipStream_t stream);

/* Chunk size in elements for a per-rank buffer of count elements
 * (align = 1024 uncompressed, 16384 compressed); 0 on invalid input. */
size_t hc_chunk_elems(size_t count, double chunk_fraction, size_t align);

/* One Transfer(srcRank, dstRank, step, chunkId, opType) task of the ring
 * ("ResCCL ...", section 3), with the element range it moves. */
typedef struct {
    int32_t src, dst, step, chunk;
    int32_t op;        /* 1 = recvReduceCopy (reduce-scatter), 2 = copy (all-gather) */
    int32_t slice;
    uint64_t off, len; /* element range inside the per-rank buffer */
} hc_task_t;

/* Host-only: the allreduce task list the launcher executes (reduce-scatter
 * steps then all-gather steps; receiver-major, then chunk, in each step).
 * Returns the number of tasks; writes at most cap (tasks may be NULL). */
size_t hc_ring_tasks(int nranks, size_t count, size_t chunk, hc_task_t *tasks, size_t cap);

/* 1 when this process's HIP runtime runs copy_engine copies on the DMA
 * engines (runtime 7.2 or later), else 0: then copy_engine = 1 is
 * HC_ERR_UNSUPPORTED. */
int hc_copy_engine_available(void);

/* ------------------------------------------------------------------------
 * The training step around the exchange: what produces the gradients that
 * the ranks sum, and what happens to the sum before the update.
 *
 * All of these are asynchronous on `stream`, may be captured into a graph,
 * and give the same bits when they are called again on the same buffers:
 * every sum has a fixed order, and where more than the sizes fixes it, the
 * call says so.  Elements are fp32 or bf16; bf16 is widened exactly, sums are
 * held in fp32 (the norm in fp64) and each result is rounded once, to nearest
 * even.  Pointers need only their element's alignment, except workspaces (16
 * bytes); rows may be further apart than they are wide (strides in elements,
 * never less than the width).  Offsets are 64-bit.  Outputs must not overlap inputs unless a call
 * says so; that is the caller's to keep, like the sizes of its buffers.
 * A workspace too small is HC_ERR_INSUFFICIENT_CAPACITY; its contents need
 * not be kept between calls, and a call in flight owns it.
 * ------------------------------------------------------------------------ */

typedef enum {
    HC_NORM_L2 = 0,    /* sqrt of the sum of squares */
    HC_NORM_INF = 1,   /* largest absolute value */
    HC_NORM_RANGE_MIN_ = INT32_MIN,
    HC_NORM_RANGE_MAX_ = INT32_MAX
} hc_norm_t;

/*
 * The norm of many gradients taken as one vector, and clipping by it.
 *   grads, outs, counts, dtypes: HOST arrays of ntensors entries.  A tensor
 *     of count 0 is skipped (its pointer may be NULL); ntensors 0 has norm 0.
 *   hc_grad_norm: *d_norm (device fp32) = the norm.  Squares and sums are
 *     fp64, so that no finite fp32 or bf16 gradient overflows or vanishes in
 *     them; the result is rounded once to fp32.  A NaN anywhere gives NaN.
 *     The order of the fp64 sum follows the counts, the types and where the
 *     tensors (and outputs) lie: their places in lines of 128 bytes, and which
 *     of them follow one another in memory.  The same values elsewhere, or
 *     with other outputs, may so give a norm that, in rare cases, differs in
 *     its last bit.
 *   hc_clip_grads: outs[i] = coef * grads[i] with coef = min(1, max_norm /
 *     (*d_norm + 1e-6)) in fp32 (NaN stays NaN, an infinite norm gives 0).
 *     In place where outs[i] == grads[i]; a coefficient of 1 writes nothing
 *     in place.  outs must not overlap one another or, unless equal, a
 *     gradient (HC_ERR_INVALID_ARGUMENT): a gradient listed twice would be
 *     scaled twice.  *d_norm may be a norm summed over more than these
 *     tensors (other ranks' shards).
 *   hc_clip_grad_norm: both, with *d_norm written.  max_norm >= 0.
 *   ws: hc_grad_norm_workspace_bytes(ntensors) bytes (all three).
 */
size_t hc_grad_norm_workspace_bytes(size_t ntensors);
hc_status_t hc_grad_norm(const void *const *grads, const size_t *counts, const hc_dtype_t *dtypes,
                         size_t ntensors, hc_norm_t norm, float *d_norm, void *ws, size_t ws_bytes,
                         hipStream_t stream);
hc_status_t hc_clip_grads(const void *const *grads, void *const *outs, const size_t *counts,
                          const hc_dtype_t *dtypes, size_t ntensors, const float *d_norm, float max_norm,
                          void *ws, size_t ws_bytes, hipStream_t stream);
hc_status_t hc_clip_grad_norm(const void *const *grads, void *const *outs, const size_t *counts,
                              const hc_dtype_t *dtypes, size_t ntensors, hc_norm_t norm, float max_norm,
                              float *d_norm, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * hc_embedding -- rows of a table by token id, scaled:
 *   out[t] = round(scale * weight[ids[t] - vocab_start]).
 * An id outside [vocab_start, vocab_start + vocab) gives a zero row: with the
 * vocabulary split over ranks, each rank looks up its part and hc_allreduce
 * adds the ranks' rows.
 *   ids: ntokens device integers of id_bytes (4 or 8) bytes.
 *   weight: vocab rows of dim elements, weight_stride elements apart; out:
 *   ntokens rows, out_stride apart, of the same dtype.
 *   vocab, ntokens < 2^31; dim < 2^31.
 */
hc_status_t hc_embedding(const void *ids, int id_bytes, size_t ntokens, const void *weight, hc_dtype_t dtype,
                         size_t vocab, size_t dim, size_t weight_stride, int64_t vocab_start, float scale,
                         void *out, size_t out_stride, hipStream_t stream);

/*
 * hc_embedding_grad -- the table's gradient, from tokens sorted by id:
 *   dweight[v] = round(scale * sum over t with ids[t] - vocab_start == v of dout[t])
 * summed in fp32 in an order that the ids, ntokens and dim fix (so a table split
 * by columns may add up in another order than the whole).  Rows that no token has
 * become zero, or with accumulate != 0 stay as they are, while the others get
 * dweight[v] + that sum (added in fp32, rounded once).
 *   padding_id: tokens of this id (counted as in ids, before vocab_start) add
 *     nothing; a negative value names none.
 *   dout: ntokens rows of dout_dtype, dout_stride apart; dweight: vocab rows
 *     of dweight_dtype, dweight_stride apart.
 *   ws: hc_embedding_grad_workspace_bytes(ntokens, vocab, dim) bytes, which are
 *     enough for fewer tokens, rows and columns as well (0 on invalid sizes).
 */
size_t hc_embedding_grad_workspace_bytes(size_t ntokens, size_t vocab, size_t dim);
hc_status_t hc_embedding_grad(const void *ids, int id_bytes, size_t ntokens, const void *dout,
                              hc_dtype_t dout_dtype, size_t dout_stride, size_t vocab, size_t dim,
                              int64_t vocab_start, int64_t padding_id, float scale, void *dweight,
                              hc_dtype_t dweight_dtype, size_t dweight_stride, int accumulate, void *ws,
                              size_t ws_bytes, hipStream_t stream);

/*
 * Tokens sorted by expert, and back: the two sides of an expert-parallel
 * exchange.  Token t chooses k experts; its choice j is slot s = t * k + j.
 * Slots are laid out by expert, in slot order within an expert (stable), each
 * expert's rows beginning at a multiple of row_align (1: packed).
 *
 * hc_expert_plan_t holds the layout.  The caller fills in the sizes and the
 * device buffers; hc_expert_sort writes the buffers, the other calls read
 * them:
 *   row_of_slot[ntokens * k]: the slot's row, or -1 if its expert is not one
 *     of these (another rank's, or a masked token's id).
 *   slot_of_row[rows]: the row's slot, or -1 (padding, and every row past
 *     the last expert's).
 *   expert_offsets[nexperts + 1]: each expert's first row; the last entry is
 *     the end of all rows in use, padding included.
 *   expert_counts[nexperts]: each expert's slots.
 *   rows: the rows the buffers have room for, at least
 *     hc_expert_rows_bound(ntokens, k, nexperts, row_align).
 * The calls that read a plan treat a row number outside [0, rows) as -1.
 * k in 1..HC_MAX_TOPK, nexperts in 1..HC_MAX_EXPERTS, row_align >= 1; slots
 * and rows < 2^31.
 */
#define HC_MAX_TOPK 64
#define HC_MAX_EXPERTS 1024
typedef struct {
    size_t ntokens;
    int32_t k;
    int32_t nexperts;
    int32_t row_align;
    size_t rows;
    int32_t *row_of_slot;
    int32_t *slot_of_row;
    int32_t *expert_offsets;
    int32_t *expert_counts;
} hc_expert_plan_t;

/* ntokens * k + min(nexperts, ntokens * k) * (row_align - 1); 0 on invalid sizes. */
size_t hc_expert_rows_bound(size_t ntokens, int k, int nexperts, int row_align);
/* 0 where no workspace is needed, and on invalid sizes.  Enough for fewer slots
 * and experts as well. */
size_t hc_expert_sort_workspace_bytes(size_t nslots, int nexperts);
/* experts: ntokens * k device integers of id_bytes (4 or 8) bytes; this
 * rank's experts are [expert_start, expert_start + nexperts). */
hc_status_t hc_expert_sort(const void *experts, int id_bytes, int64_t expert_start, const hc_expert_plan_t *plan,
                           void *ws, size_t ws_bytes, hipStream_t stream);
/* rows[row_of_slot[t * k + j]] = x[t]; padding rows of an expert become zero,
 * rows past the last expert's stay as they are. */
hc_status_t hc_expert_dispatch(const void *x, hc_dtype_t dtype, size_t dim, size_t x_stride,
                               const hc_expert_plan_t *plan, void *rows, size_t rows_stride, hipStream_t stream);
/* out[t] = round(sum over j of weights[t * k + j] * rows[row_of_slot[t * k + j]]),
 * in fp32, j ascending; a slot without a row adds nothing, so a token without
 * any gets a zero row.  weights: ntokens * k device fp32, or NULL for ones
 * (which makes it the gradient of hc_expert_dispatch). */
hc_status_t hc_expert_combine(const void *rows, hc_dtype_t dtype, size_t dim, size_t rows_stride,
                              const hc_expert_plan_t *plan, const float *weights, void *out, size_t out_stride,
                              hipStream_t stream);
/* The gradient of hc_expert_combine:
 *   drows[row_of_slot[t * k + j]] = round(weights[t * k + j] * dout[t]), padding rows zero;
 *   dweights[t * k + j] = sum over d of dout[t][d] * rows[row_of_slot[t * k + j]][d] in fp32,
 *   0 for a slot without a row. */
hc_status_t hc_expert_combine_grad(const void *dout, hc_dtype_t dtype, size_t dim, size_t dout_stride,
                                   const void *rows, size_t rows_stride, const hc_expert_plan_t *plan,
                                   const float *weights, void *drows, size_t drows_stride, float *dweights,
                                   hipStream_t stream);

/*
 * The root-mean-square norm of rows, after a residual's addition:
 *   h = round(x + residual)   (x itself where residual is NULL)
 *   out = round(h * r * weight),   r = 1 / sqrt(mean of h^2 + eps)
 * in fp32; h is rounded to the rows' type first, so that the norm and its
 * gradient are of the values that sum_out holds.  No finite row's squares
 * overflow, nor do they vanish beside an eps of 0 or one as small (where r is
 * past fp32, with a mean of squares and an eps below 2^-256 together, the row is
 * infinite; of zeroes alone it is NaN).  A NaN makes its row NaN; an infinity
 * makes the row 0 and itself NaN.
 *   x, residual, sum_out, out: ntokens rows of dtype, each with its stride; dim
 *     in 1..HC_MAX_NORM_DIM.
 *     residual may be NULL, and so may sum_out (h is then not kept); sum_out
 *     without residual is HC_ERR_INVALID_ARGUMENT.  sum_out and out may each
 *     be x or residual, with its stride (not one the other).
 *   weight: dim elements of weight_dtype.  eps >= 0, finite.
 *
 * hc_rms_norm_8bit writes rows of 8 bits (e4m3: 4 bits of exponent, 3 of
 * mantissa, no infinities, largest 448), one byte each, with scales: for each
 * group of `group` columns (32, 64, 128 or 256, the last one shorter; 0: the
 * whole row)
 *   t = h * weight,  a = largest |t| of the group,
 *   out = nearest e4m3 of t * (448 / a),  scales[row][group] = a * r / 448,
 * so that out * scale is the norm's output.  The codes do not depend on r, nor
 * on any order of summation.  A group of zeroes has scale 0; one with a NaN or
 * an infinity has a scale that is NaN.  A row of 8 bits with its scales may go
 * through hc_expert_dispatch, two bytes as one bf16 element and a scale as fp32
 * (the rows are copied as they are).
 *   out: apart from the other rows (HC_ERR_INVALID_ARGUMENT if it begins where
 *     some of them do); sum_out may be x or residual.
 *   scales: ntokens rows of ceil(dim / group) (or 1) fp32, scales_stride apart.
 */
#define HC_MAX_NORM_DIM 32768
hc_status_t hc_rms_norm(const void *x, hc_dtype_t dtype, size_t ntokens, size_t dim, size_t x_stride,
                        const void *residual, size_t residual_stride, const void *weight,
                        hc_dtype_t weight_dtype, float eps, void *sum_out, size_t sum_stride, void *out,
                        size_t out_stride, hipStream_t stream);
hc_status_t hc_rms_norm_8bit(const void *x, hc_dtype_t dtype, size_t ntokens, size_t dim, size_t x_stride,
                             const void *residual, size_t residual_stride, const void *weight,
                             hc_dtype_t weight_dtype, float eps, void *sum_out, size_t sum_stride, void *out,
                             size_t out_stride, int group, float *scales, size_t scales_stride,
                             hipStream_t stream);
/*
 * The gradient of hc_rms_norm, of its h (x there, or sum_out):
 *   dx = round(r * (dout * weight - h * r^2 * mean(dout * weight * h)) + dsum)
 *   dweight = round(sum over tokens of dout * h * r), or with accumulate != 0
 *     round(dweight + that sum)
 * in fp32; the order of the sums follows the sizes.  dout * weight is fp32's, and
 * so is its product with h, summed over a row, unless the row's squares pass
 * fp32 themselves (then of h 2^-80 times as large).  A NaN or an infinity in h
 * makes its row of dx NaN.
 *   dsum: the gradient that arrives at h beside the norm's, or NULL.  dx may
 *     be dout, h or dsum, with its stride.
 *   dweight: dim elements of dweight_dtype, or NULL (not computed).
 *   ws: hc_rms_norm_grad_workspace_bytes(ntokens, dim) bytes, which are enough
 *     for fewer tokens and columns as well (0 on invalid sizes); none is needed
 *     where dweight is NULL.
 */
size_t hc_rms_norm_grad_workspace_bytes(size_t ntokens, size_t dim);
hc_status_t hc_rms_norm_grad(const void *dout, hc_dtype_t dtype, size_t ntokens, size_t dim, size_t dout_stride,
                             const void *h, size_t h_stride, const void *weight, hc_dtype_t weight_dtype,
                             float eps, const void *dsum, size_t dsum_stride, void *dx, size_t dx_stride,
                             void *dweight, hc_dtype_t dweight_dtype, int accumulate, void *ws, size_t ws_bytes,
                             hipStream_t stream);

/*
 * hc_route -- each token's k experts and their weights, from its logits:
 *   s = softmax(logits) or sigmoid(logits), over or for each of nexperts;
 *   c = s + bias (s itself without a bias);
 *   of the ngroups groups of nexperts / ngroups experts in a row, the
 *   top_groups with the largest value stay, the value being the largest c in
 *   the group (group_best 1) or the sum of its two largest (2);
 *   experts = the k largest c in them, the largest first;
 *   weights = scale * s of each, divided by their sum if renormalise.
 * Equal values go to the lowest group and expert.  The order is that of c (or,
 * without a bias, of the logits) as 64 bits hold it; the weights are fp32.
 * An expert whose logit or bias is -inf is never chosen, and adds nothing to
 * its group's value; a slot that is left without one gets expert -1 and weight
 * 0 (hc_expert_sort gives it no row).  A masked token is a row of -inf.  A NaN
 * value comes before all others and makes its weights NaN (with softmax the
 * whole row's).
 *   logits: ntokens rows of nexperts elements of dtype, logits_stride apart.
 *   bias: nexperts device fp32, or NULL: for balance; it moves the choice, not
 *     the weights.
 *   experts, weights: ntokens * k device int32 and fp32.
 *   nexperts in 1..HC_MAX_EXPERTS, a multiple of ngroups; ngroups in
 *   1..HC_MAX_GROUPS; top_groups in 1..ngroups; k in 1..HC_MAX_TOPK, at most
 *   the experts of top_groups groups.
 *
 * hc_route_grad -- the gradient of the weights, the choice held:
 *   dlogits = round(sum over j of dweights[j] * d weights[j] / d logits)
 * for every expert, zero where nothing depends on it.  Slots whose expert is
 * not in [0, nexperts), or has a logit of -inf, add nothing.  An expert that a
 * token lists twice counts twice.  Of opts, k, scores, renormalise and scale
 * are read.  dlogits may be logits, with its stride.
 */
typedef enum {
    HC_SCORES_SOFTMAX = 0,
    HC_SCORES_SIGMOID = 1,
    HC_SCORES_RANGE_MIN_ = INT32_MIN,
    HC_SCORES_RANGE_MAX_ = INT32_MAX
} hc_scores_t;
#define HC_MAX_GROUPS 64
typedef struct {
    int32_t k;
    hc_scores_t scores;
    int32_t ngroups;      /* 1: no groups */
    int32_t top_groups;
    int32_t group_best;   /* 1 or 2 */
    int32_t renormalise;
    float scale;
    const float *bias;
} hc_route_opts_t;
hc_status_t hc_route(const void *logits, hc_dtype_t dtype, size_t ntokens, int nexperts, size_t logits_stride,
                     const hc_route_opts_t *opts, int32_t *experts, float *weights, hipStream_t stream);
hc_status_t hc_route_grad(const void *logits, hc_dtype_t dtype, size_t ntokens, int nexperts, size_t logits_stride,
                          const hc_route_opts_t *opts, const int32_t *experts, const float *dweights,
                          void *dlogits, size_t dlogits_stride, hipStream_t stream);

/*
 * An AdamW step over many tensors in one launch:
 *   g' = c * g,  c = grad_scale * min(1, max_norm / (|grad_scale| * *d_norm + 1e-6))
 *   m = beta1 * m + (1 - beta1) * g',  v = beta2 * v + (1 - beta2) * (g' * g')
 *   p = p * (1 - lr * weight_decay * decay) -
 *       lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * in fp32.  p is fp32 or bf16, g fp32 or bf16, whatever p is.
 *
 * hc_adamw_plan_t holds the tensors.  hc_adamw_plan writes their table into
 * d_table (hc_adamw_table_bytes(ntensors) device bytes, 16-byte aligned) and
 * fills in *plan (HOST); hc_adamw takes the step, as often as the tensors stay
 * where they are.  The table must be written (stream order) before it is used.
 *   params, grads, exp_avgs (m), exp_avg_sqs (v), counts, param_dtypes,
 *     grad_dtypes: HOST arrays of ntensors entries, of which no host memory is
 *     kept.  A tensor of count 0 is skipped.
 *   State of 32 bits (m_scales and v_scales NULL): m and v are fp32.
 *   m, v and what is stored of them are computed by the operations as they
 *     stand here, each rounded once to fp32 (none fused), sqrt(v) and the
 *     quotient by the scale among them: other programs can follow them bit for bit.
 *   State of 8 bits: m holds e4m3 codes of m and v those of sqrt(v), a byte
 *     each; m_scales[i] and v_scales[i] hold ceil(counts[i] / HC_STATE_BLOCK)
 *     fp32, a scale for each block of HC_STATE_BLOCK values in a row:
 *     value = code * scale, scale = largest magnitude of the block * (1 / 448) (0
 *     for a block of zeroes, or of magnitudes below 2^-100).  The step's own p is computed
 *     from m and v before they are rounded; a root that is not 0 is never
 *     stored as 0.  A v past fp32 is NaN, in its p too (in 32 bits it is infinite).  Codes and scales of zero are the state before step 1.
 *   copies: NULL, or an entry per tensor: NULL, or count bf16 values that
 *     receive the updated fp32 parameter, rounded to nearest.
 *   decays: NULL (all 1), or the factor of weight_decay per tensor.
 *   What a plan writes must not overlap anything else in it: parameters, states,
 *     scales and copies of all tensors (HC_ERR_INVALID_ARGUMENT).
 *
 * hc_adamw_opts_t:
 *   step >= 1, or d_step, a device int64 that is read instead (a captured
 *     launch then follows it; one below 1 makes the parameters NaN); lr, or
 *     d_lr, a device fp32.
 *   d_norm: device fp32, the norm of the gradients before grad_scale, to clip
 *     by; NULL: no clipping, c = grad_scale.  max_norm >= 0.
 *   skip_nonfinite: with d_norm, a norm that is infinite or NaN leaves
 *     everything as it is.
 *   seed: 0 rounds to nearest.  Else 8-bit states and bf16 parameters are
 *     rounded up with the probability of what is cut off (to 1 / 65536), by 32
 *     bits that are a function of seed, step, the tensor's place in the plan
 *     and the value's in the tensor; small changes then count in the mean.
 *       mix(x): x ^= x >> 16; x *= 0xB7E15163; x ^= x >> 15; x *= 0x6A09E667; x ^= x >> 16
 *       key = mix(mix(mix(mix(low half of seed) ^ high half) ^ low half of step) ^ tensor)
 *       bits = mix(mix(key ^ high half of i) + low half of i * 0x9E3779B9), mod 2^32
 *     of which m takes the low 16, sqrt(v) the high 16, and p the high 16 of
 *     bits * 0x9E3779B9, as (16 bits + 1/2) / 65536 for m and sqrt(v), and
 *     added to the 16 bits that are cut off for p.
 */
#define HC_STATE_BLOCK 128
typedef struct {
    size_t ntensors;      /* that are not empty */
    uint64_t chunks;
    int32_t state_bits;
    const void *d_table;
} hc_adamw_plan_t;
typedef struct {
    int64_t step;
    double lr, beta1, beta2, eps, weight_decay;
    float grad_scale, max_norm;
    const float *d_norm;
    const float *d_lr;
    const int64_t *d_step;
    uint64_t seed;
    int32_t skip_nonfinite;
} hc_adamw_opts_t;
size_t hc_adamw_table_bytes(size_t ntensors);
hc_status_t hc_adamw_plan(hc_adamw_plan_t *plan, void *const *params, const void *const *grads,
                          void *const *exp_avgs, void *const *exp_avg_sqs, float *const *m_scales,
                          float *const *v_scales, void *const *copies, const float *decays, const size_t *counts,
                          const hc_dtype_t *param_dtypes, const hc_dtype_t *grad_dtypes, size_t ntensors,
                          void *d_table, size_t table_bytes, hipStream_t stream);
hc_status_t hc_adamw(const hc_adamw_plan_t *plan, const hc_adamw_opts_t *opts, hipStream_t stream);

const char *hc_status_string(hc_status_t status);
const char *hc_last_error(void);  /* thread-local, "" when none */
const char *hc_version(void);

#ifdef __cplusplus
}
#endif

#endif /* HC_H */
