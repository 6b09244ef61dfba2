/*
 * nvfp4_moe.h -- C ABI of the routed-expert MoE layer with weight-only NVFP4
 * (W4A16) experts, for one NVIDIA GB300 GPU (sm_103a).
 *
 * The layer (one call of nvfp4_moe_forward):
 *   route   : top-k of each token's router logits, weights = softmax over the
 *             k chosen logits;
 *   permute : group the T*k routed rows by expert (stable);
 *   gate/up : g = gs_g * (Wg x), u = gs_u * (Wu x), h = silu(g) * u;
 *   down    : y = gs_d * (Wd h);
 *   combine : out[t] = sum_j w[t][j] * y[t, j], rounded once to BF16.
 *
 * Sources.  The experts are "weight-only NVFP4": 4-bit values, one scale per
 * 16 weights and a per-tensor global scale ("tenhkspark/GLM-5.3-Flash-NVFP4-
 * Wabi", Config expectations: group_size = 16, weight_scale_2; "GLM-5.3-Flash
 * on Blackwell", The quantization).  Activations are BF16 and there is NO
 * activation scale anywhere in this interface: a weight-only MoE path that
 * consumes an input scale read an uninitialised 0.0 and zeroed every expert
 * ("GLM-5.3-Flash on Blackwell", The model loaded, served an API, and produced
 * garbage).  The 4-bit values are OCP MX E2M1, the group scales OCP E4M3.
 *
 * Beyond that forward the same kernels serve: a shared expert
 * (config.num_shared_experts), the routing variants (nvfp4_moe_set_scoring),
 * the BF16 router linear on the GPU (nvfp4_moe_set_router /
 * nvfp4_moe_forward_routed), the W4A4 comparison variant
 * (nvfp4_moe_set_act_quant), a dense W4A16 NVFP4 linear (nvfp4_linear_*), an
 * allocation-free decode forward (nvfp4_moe_forward_decode_static) and a
 * decode forward on pinned host buffers (nvfp4_moe_forward_host).  The 4-bit
 * products a layer is made of are there on their own too: NVFP4 experts over
 * ragged row groups, with the gradient of their input (nvfp4_grouped_*), and
 * a dense linear with INT4 weights and group scales (nvfp4_int4_*).  So is what
 * a block has around them: routing with its gradient (nvfp4_route_*), SwiGLU
 * with 8-bit checkpoints for its backward pass (nvfp4_swiglu_*), the RMS norm
 * with the residual's addition (nvfp4_norm_*), whose 8-bit output feeds a dense
 * linear with 8-bit integers on both sides (nvfp4_int8_*).
 *
 * Conventions for every call:
 *   - returns a status, never throws, never prints unless NVFP4_MOE_LOG=1;
 *   - device pointers are CUDA global-memory pointers on the handle's device
 *     (nvfp4_moe_forward_host alone takes host pointers);
 *     the caller keeps ownership of every pointer it passes;
 *   - work is enqueued on `stream`; only calls documented as synchronous
 *     wait for the GPU;
 *   - shape and pointer errors are detected on the host, before any launch, and
 *     change nothing; a pack that fails for another reason leaves the handle
 *     unpacked, also where it was packed before.
 */
#ifndef NVFP4_MOE_H_
#define NVFP4_MOE_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum nvfp4_moe_status {
  NVFP4_MOE_OK = 0,
  NVFP4_MOE_ERR_INVALID_ARG = 1,       /* null handle/pointer, bad enum, misaligned pointer */
  NVFP4_MOE_ERR_UNSUPPORTED_SHAPE = 2, /* T, top_k, E, H or I outside the supported range   */
  NVFP4_MOE_ERR_NOT_PACKED = 3,        /* forward before a successful pack                  */
  NVFP4_MOE_ERR_WORKSPACE = 4,         /* device allocation failed in create                */
  NVFP4_MOE_ERR_CUDA = 5,              /* a CUDA runtime call failed (see status string)    */
  NVFP4_MOE_ERR_TIMEOUT = 6,           /* a bounded device-side wait gave up                */
  NVFP4_MOE_ERR_BAD_SCALE = 7,         /* tensor scale <= 0, NaN or Inf                     */
  NVFP4_MOE_ERR_NOT_IMPLEMENTED = 8,
  NVFP4_MOE_ERR_DEVICE_CHECK = 9       /* a device-side bounds check fired                  */
} nvfp4_moe_status;

typedef enum nvfp4_moe_logits_dtype {
  NVFP4_MOE_LOGITS_F32 = 0,
  NVFP4_MOE_LOGITS_BF16 = 1
} nvfp4_moe_logits_dtype;

typedef enum nvfp4_moe_out_dtype {
  NVFP4_MOE_OUT_BF16 = 0,      /* the layer's output rounded once to BF16 */
  NVFP4_MOE_OUT_F32 = 1,       /* the FP32 combine result, unrounded      */
  NVFP4_MOE_OUT_F16 = 2        /* FP16: the INT8 linear alone             */
} nvfp4_moe_out_dtype;

typedef enum nvfp4_moe_score {
  NVFP4_MOE_SCORE_SOFTMAX = 0,
  NVFP4_MOE_SCORE_SIGMOID = 1
} nvfp4_moe_score;

typedef enum nvfp4_moe_path {
  NVFP4_MOE_PATH_AUTO = 0,     /* T <= decode_max_tokens -> decode, else prefill */
  NVFP4_MOE_PATH_DECODE = 1,   /* one streaming kernel, dequantised in registers  */
  NVFP4_MOE_PATH_PREFILL = 2   /* grouped tcgen05 GEMM, dequantised into TMEM     */
} nvfp4_moe_path;

/* Layer shape and limits, fixed at create.
 *   num_experts       E, 1..256
 *   hidden            H, multiple of 128, 128..16384
 *   inter             I (expert intermediate size), multiple of 128, 128..16384
 *   max_tokens        largest T a forward may pass (sizes the workspace), >= 1
 *   max_top_k         largest top_k a forward may pass, 1..min(E, 16)
 *   decode_max_tokens T at or below which AUTO picks the decode path, 0..16
 *   logits_dtype      nvfp4_moe_logits_dtype of router_logits
 *   device            CUDA device ordinal the handle lives on
 *   out_dtype         nvfp4_moe_out_dtype of out (BF16 unless set)
 *   num_shared_experts S, 0 or 1: the layer's single shared expert, used by
 *                     every token with weight 1 on top of its top_k routed
 *                     experts and added after them ("GLM-5.3-Flash on
 *                     Blackwell", The model loaded, served an API, and produced
 *                     garbage: "the single shared expert"; "GLM-5.3-Flash-NVFP4-h
 *                     — W4A16 dense-side quantization": shared experts in W4A16
 *                     NVFP4).  It has the routed experts' H and I, is packed as
 *                     expert E (after the E routed ones) and needs
 *                     E + S <= 256 and max_top_k + S <= 16.                     */
typedef struct nvfp4_moe_config {
  int num_experts;
  int hidden;
  int inter;
  int max_tokens;
  int max_top_k;
  int decode_max_tokens;
  int logits_dtype;
  int device;
  int out_dtype;
  int num_shared_experts;
} nvfp4_moe_config;

typedef struct nvfp4_moe* nvfp4_moe_t;

/* Allocate a handle: the packed-weight blob ((E + S) * 3*H*I * 9/16 bytes) and
 * the forward workspace (sized for max_tokens * (max_top_k + S) routed rows),
 * both on config->device.  Synchronous.  *out is NULL on failure. */
nvfp4_moe_status nvfp4_moe_create(const nvfp4_moe_config* config, nvfp4_moe_t* out);

/* Copy the experts into the handle's device layout: for every 128 weight rows
 * and 64-element K chunk, one 4608-byte tile of 4096 bytes of codes, ordered
 * so that each 16-byte vector holds two rows x 16 elements (one scale group
 * each; a 16-row group's vectors ordered by K group, then row), followed by
 * the matching 512 bytes of scales; a row block's tiles
 * follow one another along K, so any run of its chunks is one contiguous
 * bulk copy; the gate and up rows are interleaved in groups of 8.  Loads of
 * this layout are 16-byte vectorised and fully coalesced on both the decode
 * and the prefill path.
 * All inputs are DEVICE pointers in the canonical layout, per expert e (E
 * below counts the shared expert too when the handle has one: it is the last):
 *   w13_q [E][2I][H/2]  uint8  E2M1 codes, gate rows 0..I-1 then up rows
 *                              I..2I-1, row-major over K = H; element 2j in the
 *                              low nibble of byte j, element 2j+1 in the high
 *   w13_s [E][2I][H/16] uint8  E4M3 scale of elements 16g..16g+15 of the row
 *   w2_q  [E][H][I/2]   uint8  down projection, same rules with K = I
 *   w2_s  [E][H][I/16]  uint8
 *   gscale [E][3]       float  per-tensor scales (gate, up, down)
 * Every gscale must be finite and > 0, else NVFP4_MOE_ERR_BAD_SCALE and the
 * handle stays unpacked (this reads gscale back to the host: synchronous).
 * Inputs may be freed once the call returns. */
nvfp4_moe_status nvfp4_moe_pack(nvfp4_moe_t h, const uint8_t* w13_q, const uint8_t* w13_s,
                                const uint8_t* w2_q, const uint8_t* w2_s, const float* gscale,
                                cudaStream_t stream);

/* One forward of the layer, enqueued on `stream`; no host synchronisation and
 * no allocation, so the call can be captured into a CUDA graph.
 *   router_logits [T][E]  float or BF16 (config.logits_dtype), device
 *   x             [T][H]  BF16 activations, device, 16-byte aligned
 *   out           [T][H]  BF16 (or FP32, config.out_dtype) result, device,
 *                         16-byte aligned
 * 1 <= T <= max_tokens, 1 <= top_k <= max_top_k.  Ties between equal logits
 * go to the lower expert index; a NaN logit ranks below -inf and is counted
 * (see nvfp4_moe_get_status).  Concurrent forwards on one handle race on its
 * workspace: serialise them on one stream. */
nvfp4_moe_status nvfp4_moe_forward(nvfp4_moe_t h, const void* router_logits, int T, int top_k,
                                   const void* x, void* out, cudaStream_t stream);

/* The same forward (the layer above) with router_logits, x and out in HOST
 * memory that CUDA has mapped into the device's address space: page-locked
 * buffers from cudaHostAlloc / cudaMallocHost (mapped, at the same address,
 * whenever addressing is unified, as on every 64-bit system) or from
 * cudaHostRegister with cudaHostRegisterMapped.  Layouts, alignment and
 * ranges as for nvfp4_moe_forward.  The decode kernel reads the logits and x
 * and writes out in place -- on a Grace-Blackwell node over the coherent
 * CPU-GPU link -- so a step moves its inputs and its result without a
 * copy-engine transfer or a staging buffer.
 * Decode only: the W4A16 streaming decode kernel, T <= decode_max_tokens.  A
 * call that would take another path (T above that, a path forced to prefill,
 * W4A4 activation quantisation) returns NVFP4_MOE_ERR_UNSUPPORTED_SHAPE; a
 * pointer that is not mapped page-locked host memory (pageable, managed or
 * device memory) returns NVFP4_MOE_ERR_INVALID_ARG.  Both before anything is
 * enqueued.  Asynchronous like nvfp4_moe_forward: out holds the result once
 * `stream` has completed, and until then the host must neither write the
 * inputs nor read out. */
nvfp4_moe_status nvfp4_moe_forward_host(nvfp4_moe_t h, const void* router_logits, int T, int top_k,
                                        const void* x, void* out, cudaStream_t stream);

/* Synchronous: waits for the device, then reports the device-side status word
 * accumulated since the last call (and clears it).  Returns NVFP4_MOE_OK,
 * NVFP4_MOE_ERR_TIMEOUT or NVFP4_MOE_ERR_DEVICE_CHECK; *nan_logits (may be
 * NULL) receives the number of NaN router logits seen. */
nvfp4_moe_status nvfp4_moe_get_status(nvfp4_moe_t h, uint32_t* nan_logits);

/* Force a path (testing and measurement); AUTO by default.  The environment
 * variable NVFP4_MOE_FORCE_PATH=decode|prefill sets the default at create. */
nvfp4_moe_status nvfp4_moe_set_path(nvfp4_moe_t h, int path);

/* Decode forward that allocates nothing.  The GLM-5.3-Flash pages have no
 * counterpart to this call; it exists for callers that cannot call
 * cudaMalloc and so cannot create a handle: plugins whose host framework owns
 * and budgets every device byte, static-memory runtimes that forbid
 * allocation after start-up, and code that must not allocate while a graph
 * is being captured (no test in tests/ captures it).  It computes what
 * nvfp4_moe_forward computes on the decode path, from caller memory only:
 *   packed_experts  DEVICE, 16-byte aligned, E * 3*H*I*9/16 bytes in the
 *                   layout nvfp4_moe_pack writes (see nvfp4_moe_debug_packed_blob)
 *   gscale [E][3]   DEVICE float tensor scales (finite, > 0: not re-checked)
 *   router_logits [T][E] (logits_dtype), x [T][H] BF16, out [T][H] BF16
 * 1 <= T <= 16, 1 <= top_k <= min(E, 16); H, I as in nvfp4_moe_config.
 * All intermediates live in one static device array of 16 MiB that every GPU
 * loading this library holds until the process exits.  It needs about
 * T*top_k*(4.25*I + 4*H) + 36*H bytes plus small tables -- under 1 MiB for
 * E=128, H=4096, I=1536, T=2, top_k=8.
 * A shape needing more than the array returns
 * NVFP4_MOE_ERR_UNSUPPORTED_SHAPE before anything is enqueued.  The regions
 * that must start at zero are cleared by every call.  The first call on each
 * device looks up the array's device address and sets the decode kernels'
 * shared-memory attribute, with that device current: make it before any
 * stream capture.  Device ordinals 0..63 only (NVFP4_MOE_ERR_INVALID_ARG
 * above).  Calls whose GPU work overlaps (other streams, concurrent graph
 * replays) share the array and race: serialise them.  The call returns once
 * the work is enqueued; device-side errors (a bounded wait that gave up,
 * leaving a partial output; NaN router logits) are collected in a status word
 * inside the array that no call clears: read it with
 * nvfp4_moe_static_get_status. */
nvfp4_moe_status nvfp4_moe_forward_decode_static(const uint8_t* packed_experts, const float* gscale,
                                                 int num_experts, int hidden, int inter,
                                                 const void* router_logits, int logits_dtype, int T, int top_k,
                                                 const void* x, void* out, cudaStream_t stream);

/* Synchronous: waits for the current device, then reports and clears the
 * status word that nvfp4_moe_forward_decode_static calls on this device have
 * accumulated since the last read: NVFP4_MOE_OK, NVFP4_MOE_ERR_TIMEOUT (some
 * call's bounded wait gave up and its output is incomplete) or
 * NVFP4_MOE_ERR_DEVICE_CHECK; *nan_logits (may be NULL) receives the number
 * of NaN router logits those calls saw.  Like the forward it allocates
 * nothing; NVFP4_MOE_ERR_CUDA if a CUDA call fails. */
nvfp4_moe_status nvfp4_moe_static_get_status(uint32_t* nan_logits);

/* Fault injection for the allocation-free path's bounded-wait test, process-
 * wide: fault = 1 makes later nvfp4_moe_forward_decode_static calls issue no
 * weight copies, so their waits expire (after about 2 s) and report
 * NVFP4_MOE_ERR_TIMEOUT through nvfp4_moe_static_get_status; the GPU context
 * stays usable.  fault = 0 restores normal operation. */
nvfp4_moe_status nvfp4_moe_static_debug_set_fault(int fault);

/* Scoring rule of the route step (the router variants).  The pages keep the
 * routers as BF16 linears and do not state how their outputs become choices
 * and weights ("GLM-5.3-Flash on Blackwell", The quantization); the default
 * is softmax over the k chosen logits.  With s_e = softmax over all experts
 * (NVFP4_MOE_SCORE_SOFTMAX) or sigmoid(l_e) (NVFP4_MOE_SCORE_SIGMOID):
 *   choice : the k largest s_e + bias_e (bias NULL: the k largest logits,
 *            the same order), equal values -> lower expert index, NaN last;
 *   weights: the chosen s_e (never the bias); renormalize = 1 divides them
 *            by their sum over the k slots (softmax: the default rule;
 *            sigmoid: 1/k each if the sum is 0); then times scale.
 * bias: DEVICE float [num_experts] or NULL, copied on `stream` (the copy is
 * ordered before later forwards on that stream); scale finite and > 0.  A
 * shared expert keeps weight 1 under every rule.  Applies to later forwards
 * and nvfp4_moe_debug_route; a dense-linear handle returns
 * NVFP4_MOE_ERR_INVALID_ARG. */
nvfp4_moe_status nvfp4_moe_set_scoring(nvfp4_moe_t h, int score_func, int renormalize, float scale,
                                       const float* bias, cudaStream_t stream);

/* The router linear inside the library.  The routers stay BF16 linears
 * ("GLM-5.3-Flash on Blackwell", The quantization; "tenhkspark/GLM-5.3-Flash-
 * NVFP4-Wabi", Config expectations: the mlp.gate routers are excluded from
 * quantisation), so their logits can be computed here instead of passed in:
 *   nvfp4_moe_set_router copies w_router, DEVICE BF16 [num_experts][hidden]
 *   (16-byte aligned), into the handle (allocates once, then reuses; ordered
 *   on `stream`);
 *   nvfp4_moe_forward_routed is nvfp4_moe_forward with
 *   logits[t][e] = sum_h x[t][h] * w_router[e][h], accumulated in FP32 (no
 *   linear bias), computed on the GPU first: a GEMV kernel for T <= 16, the
 *   tcgen05 GEMM for larger T (its TMA descriptor over x is encoded on the
 *   host each call, so a captured graph replays with the x it was captured
 *   with).  Its time counts as route + permute in the stage times.
 *   nvfp4_moe_debug_logits copies the last forward_routed's logits
 *   [T][num_experts] FP32 to a DEVICE buffer.
 * NVFP4_MOE_ERR_INVALID_ARG: forward_routed before set_router, or a dense-
 * linear handle. */
nvfp4_moe_status nvfp4_moe_set_router(nvfp4_moe_t h, const void* w_router, cudaStream_t stream);
nvfp4_moe_status nvfp4_moe_forward_routed(nvfp4_moe_t h, int T, int top_k, const void* x, void* out,
                                          cudaStream_t stream);
nvfp4_moe_status nvfp4_moe_debug_logits(nvfp4_moe_t h, float* logits, cudaStream_t stream);

/* W4A4 comparison variant.  The stock checkpoint's routed experts are W4A4
 * NVFP4: activations are quantised to NVFP4 too, against a per-module FP32
 * input scale ("tenhkspark/GLM-5.3-Flash-NVFP4-Wabi", opening summary).
 * With input_scale set (DEVICE float [num_experts][2]: the gate/up input
 * scale, then the down input scale, of every routed expert; each finite and
 * > 0, else NVFP4_MOE_ERR_BAD_SCALE -- an input scale of 0 zeroes every expert,
 * "GLM-5.3-Flash on Blackwell", The model loaded, served an API, and produced
 * garbage), every routed expert quantises its input x and its hidden h
 * (rounded to BF16 first) per 16 elements: scale = E4M3(amax * fl(1/fl(6 is))),
 * code = E2M1(v * fl(1/fl(scale is))), round-to-nearest-even, saturating,
 * in FP32 in that order; the input scales multiply the tensor scales after
 * the dot products.  The shared
 * expert stays W4A16.  The quantised values are exact in BF16/FP16, so the
 * products run on the same tensor-core paths as W4A16.  NULL turns the
 * variant off.  Synchronous (reads the scales back to check them). */
nvfp4_moe_status nvfp4_moe_set_act_quant(nvfp4_moe_t h, const float* input_scale, cudaStream_t stream);

/* Per-stage timing.  With profiling on, every forward records CUDA events on
 * its stream before and after each stage.  nvfp4_moe_get_stage_times
 * (synchronous) returns in ms[0..3] the summed milliseconds of route+permute,
 * gate/up GEMM, down GEMM and combine over the forwards since profiling was
 * switched on or last read, and their number in *count; then it starts over.
 * Do not switch profiling on while capturing a CUDA graph. */
nvfp4_moe_status nvfp4_moe_set_profiling(nvfp4_moe_t h, int on);
nvfp4_moe_status nvfp4_moe_get_stage_times(nvfp4_moe_t h, float* ms, int* count);

/* Static text for a status code. */
const char* nvfp4_moe_status_string(nvfp4_moe_status s);

/* Text of the last error seen on this handle (CUDA error name, failed check). */
const char* nvfp4_moe_last_error(nvfp4_moe_t h);

/* Free the handle and its device memory (synchronises the device first). */
void nvfp4_moe_destroy(nvfp4_moe_t h);

/* ---- inspection entry points (same ABI; used by the parity tests) ------- */

/* Route and permute exactly as the forward of the chosen path does, into
 * caller DEVICE buffers, with K = top_k + S slots per token (the shared
 * expert, id E, weight 1, in the last): ids [T][K] int32, weights [T][K]
 * float, offsets [E+S+1] int32, perm [T*K] int32 (flattened index t*K+j of
 * the routed row at each expert-major position). */
nvfp4_moe_status nvfp4_moe_debug_route(nvfp4_moe_t h, const void* router_logits, int T, int top_k,
                                       int32_t* ids, float* weights, int32_t* offsets,
                                       int32_t* perm, cudaStream_t stream);

/* Copy the handle's packed expert blob (E * 3*H*I*9/16 bytes, the layout
 * described at nvfp4_moe_pack; per expert: the gate/up matrix's tiles
 * [2I/128][H/64][4608 B], then the down matrix's [H/128][I/64][4608 B]) into
 * a caller DEVICE buffer of at least that many bytes. */
nvfp4_moe_status nvfp4_moe_debug_packed_blob(nvfp4_moe_t h, void* dst, size_t dst_bytes, cudaStream_t stream);

/* Phase timeline of the decode kernel (handles created with the environment
 * variable NVFP4_MOE_TRACE=1 only).  Synchronous.  Copies up to n values into
 * host_dst: for each CTA c and warp w, 16 values at [(c*16 + w)*16]:
 * globaltimer nanosecond stamps 0 kernel start, 1 routed, 2 gate/up done,
 * 3 first down wait over, 4 down done, 5 exit barrier passed; durations (ns)
 * 6 gate/up and 7 down end-of-phase block finishing; stamps 8 inputs loaded,
 * 9 top-k chosen, 10 expert offsets scanned (warp 0 of each CTA only),
 * 11 gate/up stream ended, 12 down stream ended, 13 first gate/up stage
 * landed; 14 and 15: the SM clock counter (clock64) at stamps 0 and 1;
 * unused slots 0.  Clears the buffer. */
nvfp4_moe_status nvfp4_moe_debug_trace(nvfp4_moe_t h, uint64_t* host_dst, size_t n, size_t* n_written);

/* Dequantise one tensor of one expert from the PACKED blob into a caller
 * DEVICE buffer of float [N][K]: value = fp32(e2m1 * e4m3) * gscale, one
 * FP32 rounding.  which: 0 gate [I][H], 1 up [I][H], 2 down [H][I]. */
nvfp4_moe_status nvfp4_moe_debug_dequant(nvfp4_moe_t h, int expert, int which, float* w_out,
                                         cudaStream_t stream);

/* Copy the last forward's intermediates, in expert-major routed-row order
 * (row p = perm position p), into caller DEVICE buffers:
 *   hidden [T*K][I] float: h = silu(g)*u as the down GEMM consumed it, after
 *          its rounding to 16 bits (K = top_k + S),
 *   y      [T*K][H] float (expert output before the routing weight). */
nvfp4_moe_status nvfp4_moe_debug_intermediates(nvfp4_moe_t h, void* hidden, float* y,
                                               cudaStream_t stream);

/* Fault injection for the bounded-wait test: fault = 1 makes the prefill
 * producer and the decode kernel issue no copies, so the consumers' waits
 * expire (after about 2 s), the kernels record NVFP4_MOE_ERR_TIMEOUT in the
 * status word and return; the GPU context stays usable.  fault = 0 restores
 * normal operation. */
nvfp4_moe_status nvfp4_moe_debug_set_fault(nvfp4_moe_t h, int fault);

/* Fill every workspace buffer that each forward rewrites before it reads it
 * (routing tables, gathered and hidden activations, expert outputs, the
 * decode kernels' activation rows) with `byte`, on `stream`; the counters and
 * the status word keep their values.  A forward after it must give
 * bit-identical results: no kernel reads memory it has not written in the
 * same forward (the unused MMA columns that read such rows are never kept).
 * Tests use 0xFF (NaN in FP16, BF16 and FP32). */
nvfp4_moe_status nvfp4_moe_debug_poison_workspace(nvfp4_moe_t h, int byte, cudaStream_t stream);

/* Host only (no GPU needed): the status code a device status word stands for
 * -- bit 0 a bounded wait that gave up (NVFP4_MOE_ERR_TIMEOUT), bit 1 a
 * device-side bounds check that fired (NVFP4_MOE_ERR_DEVICE_CHECK; the checks
 * run when the handle was created with NVFP4_MOE_CHECKS=1), none
 * NVFP4_MOE_OK.  nvfp4_moe_get_status and nvfp4_moe_static_get_status decode
 * the words they read this way. */
nvfp4_moe_status nvfp4_moe_decode_status_word(uint32_t flags);

/* ---------------------------------------------------------------------------
 * Dense W4A16 NVFP4 linear: out[t] = gs * W x[t] for one weight matrix W
 * [N][K] in the same weight-only format as the experts (E2M1 codes, one E4M3
 * scale per 16 elements of a row, one FP32 tensor scale gs; activations
 * BF16, no activation scale).  The dense side of the model -- the attention
 * projections, the shared experts and lm_head -- is quantised this way
 * ("GLM-5.3-Flash-NVFP4-h — W4A16 dense-side quantization", opening summary
 * and Config expectations: W4A16_NVFP4 modules with group_size = 16).  It
 * runs on the same two paths as the MoE layer, as a one-matrix case: T <= 16
 * on the decode GEMV kernel, larger T on the tcgen05 GEMM kernel, both
 * writing out directly (no routing, no combine).
 *
 * A linear handle is an nvfp4_moe_t: nvfp4_moe_destroy, nvfp4_moe_set_path,
 * nvfp4_moe_get_status, nvfp4_moe_set_profiling / get_stage_times,
 * nvfp4_moe_debug_packed_blob and nvfp4_moe_debug_set_fault apply to it;
 * nvfp4_moe_pack, nvfp4_moe_forward, nvfp4_moe_debug_route and
 * nvfp4_moe_debug_intermediates return NVFP4_MOE_ERR_INVALID_ARG and
 * nvfp4_moe_debug_dequant NVFP4_MOE_ERR_NOT_IMPLEMENTED on it; the linear
 * calls below return NVFP4_MOE_ERR_INVALID_ARG on an MoE handle.
 * ------------------------------------------------------------------------- */
typedef struct nvfp4_linear_config {
  int out_features;      /* N: 16..16384, a multiple of 16 */
  int in_features;       /* K: 128..16384, a multiple of 128 */
  int max_tokens;        /* largest T of any forward, 1..2^20 */
  int decode_max_tokens; /* 0..16: T <= this takes the decode (GEMV) path */
  int out_dtype;         /* nvfp4_moe_out_dtype */
  int device;            /* CUDA device ordinal */
} nvfp4_linear_config;

/* Allocate a linear handle: the packed matrix (Np*K*9/16 bytes, Np = N
 * rounded up to a multiple of 128; the padding rows hold zeros and are never
 * written out) and a small workspace (tables for max_tokens rows; no
 * activation copies), on config->device.  Synchronous.  *out is NULL on
 * failure. */
nvfp4_moe_status nvfp4_linear_create(const nvfp4_linear_config* config, nvfp4_moe_t* out);

/* Copy W into the handle's device layout (the per-128-row, per-64-K-chunk
 * layout nvfp4_moe_pack writes for one down matrix).  DEVICE inputs:
 *   w_q [N][K/2]  uint8  E2M1 codes, row-major; element 2j in the low nibble
 *                        of byte j, element 2j+1 in the high (16-byte aligned)
 *   w_s [N][K/16] uint8  E4M3 scale of elements 16g..16g+15 of the row
 *   gscale [1]    float  the tensor scale: finite and > 0, else
 *                        NVFP4_MOE_ERR_BAD_SCALE and the handle stays unpacked
 * Synchronous (reads gscale back to the host).  Inputs may be freed once the
 * call returns. */
nvfp4_moe_status nvfp4_linear_pack(nvfp4_moe_t h, const uint8_t* w_q, const uint8_t* w_s, const float* gscale,
                                   cudaStream_t stream);

/* out [T][N] = gs * x [T][K] W^T, accumulated in FP32 and rounded once to
 * BF16 (or stored as FP32, config.out_dtype); x BF16 and out DEVICE, both
 * 16-byte aligned, 1 <= T <= max_tokens.  Enqueued on `stream`, no host
 * synchronisation and no allocation; the prefill path encodes a TMA
 * descriptor for x on the host each call, so a captured graph replays with
 * the x pointer it was captured with.  Concurrent forwards on one handle
 * race on its workspace: serialise them on one stream. */
nvfp4_moe_status nvfp4_linear_forward(nvfp4_moe_t h, int T, const void* x, void* out, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Grouped W4A16 NVFP4 products: E matrices W_e [N][K] in the experts' format,
 * each multiplied with its own run of rows.  For layers whose steps do not
 * fit nvfp4_moe_forward -- another activation, biases or adapters between the
 * products, rows that arrive already sorted from another rank -- and for
 * tuning what surrounds the frozen experts:
 *   forward : out[r] = gs_e W_e   x[r]    [R][K] -> [R][N]
 *   backward: dx[r]  = gs_e W_e^T dy[r]   [R][N] -> [R][K]
 * for offsets[e] <= r < offsets[e+1].  The 4-bit weights are constants, so dx
 * is the product's only gradient.  E = 1 is a dense linear's gradient.
 *
 * A grouped handle is an nvfp4_moe_t: nvfp4_moe_destroy, nvfp4_moe_last_error,
 * nvfp4_moe_set_path, nvfp4_moe_get_status, nvfp4_moe_set_profiling /
 * get_stage_times (the product counts as the down GEMM),
 * nvfp4_moe_debug_packed_blob and nvfp4_moe_debug_set_fault apply to it; the
 * MoE layer's and the other products' calls return NVFP4_MOE_ERR_INVALID_ARG
 * (nvfp4_moe_debug_dequant NVFP4_MOE_ERR_NOT_IMPLEMENTED).
 * ------------------------------------------------------------------------- */
typedef struct nvfp4_grouped_config {
  int num_experts;  /* E: 1..256 */
  int out_features; /* N: 16..16384, a multiple of 16 */
  int in_features;  /* K: 128..16384, a multiple of 128 */
  int max_rows;     /* largest R of any call, 1..2^24 */
  int out_dtype;    /* nvfp4_moe_out_dtype of out and of dx */
  int device;       /* CUDA device ordinal */
} nvfp4_grouped_config;

/* Allocate a grouped handle: the packed matrices (E*Np*K*9/16 bytes, Np = N
 * rounded up to a multiple of 128) on config->device; no workspace.
 * Synchronous.  *out is NULL on failure. */
nvfp4_moe_status nvfp4_grouped_create(const nvfp4_grouped_config* config, nvfp4_moe_t* out);

/* Copy the matrices into the handle's device layout (per expert that of
 * nvfp4_linear_pack; forward and backward read the same bytes).  DEVICE
 * inputs:
 *   w_q [E][N][K/2]  uint8  E2M1 codes, as in nvfp4_linear_pack (16-byte aligned)
 *   w_s [E][N][K/16] uint8  E4M3 scales
 *   gscale [E]       float  tensor scales: finite and > 0, else
 *                           NVFP4_MOE_ERR_BAD_SCALE and the handle stays unpacked
 * Synchronous.  Inputs may be freed once the call returns. */
nvfp4_moe_status nvfp4_grouped_pack(nvfp4_moe_t h, const uint8_t* w_q, const uint8_t* w_s, const float* gscale,
                                    cudaStream_t stream);

/* The products above, enqueued on `stream`; no host synchronisation, no
 * allocation and no workspace: calls on one handle may overlap and be captured
 * (the tensor descriptor over x is encoded on the host each call, so a captured
 * graph replays with the pointers it was captured with, and with the offsets
 * their memory then holds).
 *   R        rows of x and out, 0..max_rows; 0 does nothing
 *   offsets  [E+1] int32 DEVICE, 0 <= offsets[0] <= .. <= offsets[E] <= R: read
 *            on the device.  An expert may have no row; rows outside
 *            offsets[0]..offsets[E]-1 are read by no product and left as they
 *            are in out.  Offsets that break the rule compute nothing and set
 *            NVFP4_MOE_ERR_DEVICE_CHECK (nvfp4_moe_get_status).
 *   x, dy    BF16 DEVICE, 16-byte aligned, rows ld elements apart
 *   out, dx  BF16 or FP32 (config.out_dtype) DEVICE, 16-byte aligned; must not
 *            overlap the input
 *   ld*      at least the row length, a multiple of 8, at most 2^24
 * Products are exact and accumulated in FP32; one rounding to BF16 at the end.
 * The tensor cores cut off the bits that an addition drops: an FP32 result is off
 * by about 1.2e-9 of its norm per term that one accumulator adds.  The GEMM has two,
 * so 2e-6 at 4096 terms (E4M3 scales over their whole range; FP32 arithmetic 8e-7).
 * The forward takes the streaming kernel for few rows (by default up to 8 per
 * expert on average, fewer where K is above 4096: 5 at 7168, 2 at 16384;
 * nvfp4_moe_set_path forces either; the streaming kernel takes at most 2048
 * rows), the tcgen05 GEMM above; the backward always the GEMM.  The
 * streaming kernel multiplies x as FP16 times a power of two per row: what lies
 * 2^-38 below a row's largest magnitude is rounded away. */
nvfp4_moe_status nvfp4_grouped_forward(nvfp4_moe_t h, int R, const int32_t* offsets, const void* x, int64_t ldx,
                                       void* out, int64_t ldo, cudaStream_t stream);
nvfp4_moe_status nvfp4_grouped_backward(nvfp4_moe_t h, int R, const int32_t* offsets, const void* dy, int64_t ld_dy,
                                        void* dx, int64_t ld_dx, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Dense linear with INT4 weights and group scales, for up to 16 tokens: the
 * other weight-only 4-bit format dense layers come in.
 *   out[t][n] = sum_k s[n][k/g] * (q[n][k] - z[n][k/g]) * x[t][k]
 * q 0..15, one scale and one zero point per g consecutive elements of a row.
 * An INT4 handle is an nvfp4_moe_t with the same calls as a grouped one;
 * nvfp4_moe_set_path has no effect on it.
 * ------------------------------------------------------------------------- */
typedef enum nvfp4_moe_act_dtype {
  NVFP4_MOE_ACT_BF16 = 0,
  NVFP4_MOE_ACT_F16 = 1
} nvfp4_moe_act_dtype;

typedef struct nvfp4_int4_config {
  int out_features; /* N: 16..2^20, a multiple of 16 */
  int in_features;  /* K: 128..16384, a multiple of 128 */
  int group_size;   /* g: 32, 64 or 128 */
  int max_tokens;   /* largest T of any forward, 1..16 */
  int act_dtype;    /* nvfp4_moe_act_dtype of x and of the scales */
  int out_f32;      /* 1: out is FP32, 0: x's type */
  int device;       /* CUDA device ordinal */
} nvfp4_int4_config;

/* Allocate an INT4 handle: the packed matrix (N*K/2 bytes of codes and 3 bytes a
 * group, N rounded up to a multiple of 32) on config->device.  Synchronous.  *out is NULL on failure. */
nvfp4_moe_status nvfp4_int4_create(const nvfp4_int4_config* config, nvfp4_moe_t* out);

/* Copy the matrix into the handle's device layout.  DEVICE inputs:
 *   w_q   [N][K/2] uint8   codes, element 2j in the low nibble of byte j (16-byte aligned)
 *   scale [N][K/g] BF16 or FP16 (config.act_dtype), finite
 *   zero  [N][K/g] uint8   zero points 0..15, or NULL: 8 everywhere
 * NVFP4_MOE_ERR_BAD_SCALE, and the handle is left unpacked, for a scale that is
 * not finite or a zero point above 15.  Synchronous.  Inputs may be freed once
 * the call returns.  Zero points are laid out only where there are any: after a
 * pack that adds or drops them a captured forward has to be captured again. */
nvfp4_moe_status nvfp4_int4_pack(nvfp4_moe_t h, const uint8_t* w_q, const void* scale, const uint8_t* zero,
                                 cudaStream_t stream);

/* out [T][N] as above, 1 <= T <= max_tokens; x [T][K] and out DEVICE, 16-byte
 * aligned, rows ldx / ldo elements apart (at least the row length, a multiple
 * of 8, at most 2^24), not overlapping.  Per group sum q x and z sum x are formed
 * in FP32 (each q x is exact, their sum is the tensor cores', which cut off what an
 * addition drops), their difference times the scale is added in FP32, and the result
 * rounded once: an FP32 result is off by 1 to 3e-7 of its norm, the more the nearer
 * the codes are to their zero points; 1e-7 where x is FP16.  x is multiplied as FP16 times a power of two per token
 * (FP16 x too): what lies 2^-34 below a token's largest magnitude is rounded away.
 * Infinities and NaNs of x count as in the formula (slower: such a token's outputs
 * are added up once more).  Enqueued on `stream`; no host synchronisation, no
 * allocation and no workspace: calls on one handle may overlap and be captured. */
nvfp4_moe_status nvfp4_int4_forward(nvfp4_moe_t h, int T, const void* x, int64_t ldx, void* out, int64_t ldo,
                                    cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Routing on its own: the choice of experts, its weights, the tables that the
 * grouped products and the combination of their rows read, and the gradient of
 * the weights.  Per token, over E experts:
 *   s_e = softmax of the logits, or 1 / (1 + exp(-l_e))    (config.score)
 *   c_e = s_e + bias_e; the logit itself where there is no bias (both scores
 *         increase with it)
 *   groups: E / groups experts that follow one another make a group.  Its value
 *         is its largest c, or with group_top = 2 the sum of its two largest
 *         (of s_e + bias_e, the bias being 0 if there is none); experts of the
 *         top_groups groups of largest value may be chosen.
 *   choice: the top_k largest c, the largest first
 *   weight_j = scale * s_j, divided by the sum of the chosen s if renormalize
 * Among equals the lower index comes first, for groups as for experts.  The
 * order is that of c, and of the groups' values, evaluated in 64 bits; the
 * weights are FP32.
 * A NaN logit has s = 0 and ranks below every number (its group counts it as
 * -inf), and so does an expert whose bias is NaN; a bias of -inf or of the
 * type's lowest value keeps an expert behind all others.  Softmax where no
 * logit is above -inf: s = 1 / E for each -inf; where some are +inf: those share 1.
 * Weights are FP32: a sigmoid below 2^-127 is 0 in them.  Renormalised ones whose
 * sigmoids sum to less than 2^-25 are the softmax of the chosen logits, which they
 * are then to a rounding, however small; those whose scores are all 0 (-inf, NaN)
 * are scale / top_k each.
 *
 * A route handle is an nvfp4_moe_t: nvfp4_moe_destroy, nvfp4_moe_last_error and
 * nvfp4_moe_get_status (which counts NaN logits) apply to it; the other
 * operators' calls return NVFP4_MOE_ERR_INVALID_ARG.
 * ------------------------------------------------------------------------- */
typedef struct nvfp4_route_config {
  int num_experts;  /* E: 1..512 */
  int top_k;        /* 1..16, at most top_groups * E / groups */
  int groups;       /* 1..32, a divisor of E */
  int top_groups;   /* 1..groups; groups: no limit */
  int group_top;    /* 1 or 2; at most E / groups */
  int score;        /* nvfp4_moe_score */
  int renormalize;  /* 0 or 1 */
  float scale;      /* finite */
  int logits_dtype; /* nvfp4_moe_logits_dtype of the logits and of their gradient */
  int device;       /* CUDA device ordinal */
} nvfp4_route_config;

nvfp4_moe_status nvfp4_route_create(const nvfp4_route_config* config, nvfp4_moe_t* out);

/* Enqueued on `stream`; no host synchronisation, no allocation and no
 * workspace: calls on one handle may overlap and be captured.
 *   T       0..2^20 tokens; 0 writes zeros to offsets and nothing else
 *   logits  [T][E] DEVICE, rows ld elements apart (E..2^24)
 *   bias    [E] float DEVICE, or NULL
 *   ids     [T][top_k] int32 out   the choice
 *   weights [T][top_k] float out
 *   offsets [E+1] int32 out        rows offsets[e] .. offsets[e+1]-1 are e's, as
 *                                  nvfp4_grouped_forward takes them
 *   perm    [T*top_k] int32 out    the row at a position: t * top_k + j, ascending
 *                                  within an expert
 *   inv     [T*top_k] int32 out    perm's inverse: the position of row t * top_k + j
 * None of the outputs may overlap another or an input. */
nvfp4_moe_status nvfp4_route_forward(nvfp4_moe_t h, int T, const void* logits, int64_t ld, const float* bias,
                                     int32_t* ids, float* weights, int32_t* offsets, int32_t* perm, int32_t* inv,
                                     cudaStream_t stream);

/* dlogits [T][E] (the logits' type, rows ld_dl apart) from dweights [T][top_k]
 * for the choice ids; the choice itself is constant.  An id outside 0..E-1 counts
 * as none, an expert named twice twice.  Softmax whose largest logit is
 * infinite, NaN logits, and renormalised sigmoids whose logits are all -inf have no
 * gradient (zeros).  dlogits may be logits. */
nvfp4_moe_status nvfp4_route_backward(nvfp4_moe_t h, int T, const void* logits, int64_t ld, const int32_t* ids,
                                      const float* dweights, void* dlogits, int64_t ld_dl, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Root-mean-square norm with the residual's addition:
 *   sum = x + residual, rounded to the 16-bit type (x itself without a residual)
 *   y   = weight * sum * rstd, rstd = 1 / sqrt(mean(sum^2) + eps)
 *   q   = round(127 v / max |v|), v = weight * sum; q_scale = max |y| / 127
 * so that y is about q * q_scale: the input of nvfp4_int8_forward.  q is the
 * exactly rounded quotient, ties to even, in -127..127.  A row of zeros has y, codes
 * and a scale of 0 also where eps is 0 (codes and scale too where its products are
 * all below 2^-149); one that is not finite has codes 0 and a scale of NaN.  Without
 * eps rstd may be beyond FP32 (a row below 2^-128): it is infinite then, y, q and
 * q_scale are right all the same, and the row has no gradient (NaN or infinite).
 * Backward, of sum (which is x's and the residual's):
 *   dx = rstd * (weight * dy) - sum * rstd^3 / H * sum_h(weight * dy * sum) + dsum
 *   dweight = sum over the rows of dy * sum * rstd
 * A norm handle is an nvfp4_moe_t like a route handle.
 * ------------------------------------------------------------------------- */
typedef struct nvfp4_norm_config {
  int hidden;    /* H: 8..16384, a multiple of 8 */
  float eps;     /* >= 0, finite */
  int act_dtype; /* nvfp4_moe_act_dtype of all rows and of the weight */
  int device;    /* CUDA device ordinal */
} nvfp4_norm_config;

/* Synchronous.  The handle holds the workspace of dweight (at most H * 4 KB). */
nvfp4_moe_status nvfp4_norm_create(const nvfp4_norm_config* config, nvfp4_moe_t* out);

/* T 0..2^20 rows of H, DEVICE, 16-byte aligned (q: 8), rows ld elements apart: at
 * least H, a multiple of 8, at most 2^24.
 *   residual NULL: none, and sum has to be NULL; else sum may be x or residual
 *   y, q     either may be NULL, not both; y may be x; q_scale [T] float with q
 *   rstd     [T] float, for the backward pass, or NULL
 * Otherwise outputs must not overlap inputs or one another.  No host
 * synchronisation, no allocation and no workspace: calls may overlap and be
 * captured. */
nvfp4_moe_status nvfp4_norm_forward(nvfp4_moe_t h, int T, const void* x, int64_t ldx, const void* residual,
                                    int64_t ld_res, const void* weight, void* sum, int64_t ld_sum, void* y, int64_t ldy,
                                    int8_t* q, int64_t ldq, float* q_scale, float* rstd, cudaStream_t stream);

/* sum and rstd [T] are the forward's.  dsum: the gradient that reaches sum on its
 * other way, or NULL.  dx may be dy or dsum.  dweight [H] float (16-byte aligned)
 * or NULL; it is written, not added to, in an order of summation that depends on
 * T and H alone.  Calls with a dweight use the handle's workspace: serialise
 * those on one stream, captured ones too. */
nvfp4_moe_status nvfp4_norm_backward(nvfp4_moe_t h, int T, const void* dy, int64_t ld_dy, const void* sum,
                                     int64_t ld_sum, const void* weight, const float* rstd, const void* dsum,
                                     int64_t ld_dsum, void* dx, int64_t ld_dx, float* dweight, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * SwiGLU between the grouped gate/up and down products, with gate and up kept
 * for the backward pass in 8 bits (half of what they take):
 *   h = silu(gate) * up
 *   codes = round(127 v / peak), scales = peak / 127, peak the largest magnitude of
 *           128 elements of a row that follow one another (a row's last ones may be
 *           fewer); exactly rounded, ties to even
 * Backward, with g and u = codes * scales, s = 1 / (1 + exp(-g)):
 *   dgate = dh * u * s * (1 + g * (1 - s)),  dup = dh * g * s
 * A block of 128 that is not finite comes back as NaN.  exp is evaluated to about
 * 2^-21 (|g| 2^-24 where |g| is larger than 16), and s below 2^-126, from g = -87.3
 * down, counts as 0; all arithmetic is FP32, with one rounding at the end.
 * A SwiGLU handle is an nvfp4_moe_t like a route handle.
 * ------------------------------------------------------------------------- */
typedef struct nvfp4_swiglu_config {
  int inter;     /* I: 16..16384, a multiple of 16 */
  int act_dtype; /* nvfp4_moe_act_dtype of all rows */
  int device;    /* CUDA device ordinal */
} nvfp4_swiglu_config;

nvfp4_moe_status nvfp4_swiglu_create(const nvfp4_swiglu_config* config, nvfp4_moe_t* out);

/* R 0..2^24 rows of I, DEVICE, 16-byte aligned, rows ld elements apart: at least I,
 * a multiple of 8, at most 2^24 (gate and up may be halves of one matrix).
 *   codes  [R][2][I] int8 out (gate, up), 16-byte aligned, and
 *   scales [R][2][ceil(I / 128)] float out; or both NULL: nothing is kept
 * h may be gate or up; otherwise outputs must not overlap inputs or one another.
 * No host synchronisation, no allocation and no workspace: calls may overlap and
 * be captured. */
nvfp4_moe_status nvfp4_swiglu_forward(nvfp4_moe_t h, int R, const void* gate, int64_t ld_gate, const void* up,
                                      int64_t ld_up, void* out, int64_t ld_out, int8_t* codes, float* scales,
                                      cudaStream_t stream);
/* The same conditions; dgate or dup may be dh. */
nvfp4_moe_status nvfp4_swiglu_backward(nvfp4_moe_t h, int R, const int8_t* codes, const float* scales, const void* dh,
                                       int64_t ld_dh, void* dgate, int64_t ld_dgate, void* dup, int64_t ld_dup,
                                       cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Dense linear with 8-bit integers on both sides, a scale per token and per output:
 *   out[t][n] = x_scale[t] * w_scale[n] * sum_k x[t][k] w[n][k] + bias[n]
 * The sum is exact; it, and the product of the scales, are rounded to FP32, their
 * product with the bias added is rounded once more, and once to the result's type.
 * An INT8 handle is an nvfp4_moe_t with the same calls as an INT4 one.
 * ------------------------------------------------------------------------- */
typedef struct nvfp4_int8_config {
  int out_features; /* N: 16..2^20, a multiple of 16 */
  int in_features;  /* K: 16..16384, a multiple of 16 */
  int max_tokens;   /* largest T of any forward, 1..2^20 */
  int out_dtype;    /* nvfp4_moe_out_dtype */
  int device;       /* CUDA device ordinal */
} nvfp4_int8_config;

/* Allocate an INT8 handle: the packed matrix (N*K bytes, both rounded up to
 * multiples of 128) and, for max_tokens above 64, a workspace that holds as many
 * tokens in FP16 (256 MB at most) on config->device.  Synchronous.  *out is NULL on
 * failure. */
nvfp4_moe_status nvfp4_int8_create(const nvfp4_int8_config* config, nvfp4_moe_t* out);

/* Copy the matrix into the handle's device layout.  DEVICE inputs:
 *   w       [N][K] int8   (16-byte aligned), -128..127
 *   w_scale [N] float     finite, else NVFP4_MOE_ERR_BAD_SCALE and the handle is
 *                         left unpacked
 *   bias    [N] float, or NULL: none
 * Synchronous.  Inputs may be freed once the call returns.  After a pack that adds
 * or drops the bias a captured forward has to be captured again. */
nvfp4_moe_status nvfp4_int8_pack(nvfp4_moe_t h, const int8_t* w, const float* w_scale, const float* bias,
                                 cudaStream_t stream);

/* Activations for the forward from 16-bit ones: x [T][K] of x_dtype
 * (nvfp4_moe_act_dtype), 16-byte aligned, rows ldx elements apart (at least K, a
 * multiple of 8, at most 2^24); q [T][K] int8, 8-byte aligned, rows ldq apart (the
 * same), q_scale [T] float: round(127 x / max |x|) and max |x| / 127 per row, as in
 * nvfp4_norm_forward.  T 0..2^20.  May overlap other calls and be captured. */
nvfp4_moe_status nvfp4_int8_quantize(nvfp4_moe_t h, int T, const void* x, int x_dtype, int64_t ldx, int8_t* q,
                                     int64_t ldq, float* q_scale, cudaStream_t stream);

/* out [T][N] as above, 0 <= T <= max_tokens; x [T][K] int8 and out DEVICE, 16-byte
 * aligned, rows ldx / ldo elements apart (at least the row length, ldx a multiple
 * of 16 and ldo of 8, at most 2^24), not overlapping; x_scale [T] float, whose NaNs
 * and infinities reach their row.  Enqueued on `stream`; no host synchronisation
 * and no allocation; calls may be captured (above 16 tokens the tensor descriptor
 * over x is encoded on the host, so a captured graph replays with the pointers it
 * was captured with).  Up to 64 tokens calls on one handle may overlap.  Above,
 * they use its workspace: serialise those on one stream, captured ones too (graphs
 * that may run at the same time need a handle each). */
nvfp4_moe_status nvfp4_int8_forward(nvfp4_moe_t h, int T, const int8_t* x, int64_t ldx, const float* x_scale, void* out,
                                    int64_t ldo, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_MOE_H_ */
