/*
 * mpb.h -- C ABI of libmpb, the MI355X (gfx950) mixed-precision MoE layer.
 *
 * The layer is the one PagedWeight runs inside its serving loop ("PagedWeight:
 * Efficient MoE LLM Serving with Dynamic Quality-Aware Weight Quantization",
 * §3.3 "Fused Mixed-Precision MoE Kernel"): top-K routing, expert gate_up with
 * SwiGLU, the down projection and the routing-weighted output accumulation,
 * with every expert weight read straight from Any-Precision bit-planes and
 * per-row lookup tables at the bitwidth q_i committed for its linear-block
 * (§3.1 "Paged Weight Representation").
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Return value: 0 on success, a negative MPB_E_* code on failure. No C++
 *   exception crosses the ABI. mpb_last_error() gives a message for the last
 *   failure of the calling thread.
 * - Pointers named *_dev / device arrays are device (HBM) addresses; *_host are
 *   host addresses. All buffers are owned by the caller and only borrowed: the
 *   caller keeps them alive until the stream has passed the enqueued work. The
 *   library allocates no device memory.
 * - stream is a hipStream_t passed as void* (NULL = the default stream). Work is
 *   enqueued asynchronously; argument validation happens synchronously on the
 *   host before anything is enqueued, so a failed call enqueues nothing. Device
 *   faults surface at the caller's next synchronisation of that stream.
 * - One controlling thread; the library takes no locks.
 *
 * Linear-blocks. For a layer with E routed and S shared experts, block
 * i = 2*e + u, e in [0, E+S) (routed first), u = 0 for gate_up ([N=2I rows,
 * Kd=H]; rows 0..I-1 gate, rows I..2I-1 up) and u = 1 for down ([N=H, Kd=I]).
 * Supported bitwidths B_i = {3,...,8} for every block.
 *
 * Canonical bit-plane format (the interchange format mpb_pack_block reads):
 * planes[p][n][w], uint32, p = 0..7 with plane 0 the code's most significant
 * bit; bit j of word w holds element k = 32*w + j of row n. The b-bit index of
 * an element is formed from planes 0..b-1 (the top b planes, §2.2 and §3.1).
 * Canonical LUT of bitwidth b: [N][2^b] fp16 (one centroid table per row),
 * indexed by that b-bit index.
 */
#ifndef MPB_H
#define MPB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    MPB_OK = 0,
    MPB_E_ARG = -1,          /* null pointer, bad enum, bad count */
    MPB_E_SHAPE = -2,        /* dimension not supported (see each call) */
    MPB_E_RANGE = -3,        /* block index i or bitwidth b out of range */
    MPB_E_NOT_RESIDENT = -4, /* bitwidth above the block's resident planes */
    MPB_E_WS = -5,           /* workspace too small */
    MPB_E_HIP = -6,          /* a HIP launch or API call failed */
    MPB_E_UNINIT = -7,       /* mpb_init has not bound a layer */
    MPB_E_BUSY = -8          /* a page transfer of the block is still in flight */
};

enum { MPB_PAGE_GPU = 0, MPB_PAGE_CPU = 1, MPB_PAGE_IN_TRANSFER = 2 }; /* page states */

enum { MPB_F16 = 0, MPB_BF16 = 1, MPB_F32 = 2 }; /* activation dtypes; MPB_F32 only where a call takes it */

typedef struct {
    int32_t H; /* hidden size, multiple of 64 */
    int32_t I; /* expert intermediate size, multiple of 64 */
    int32_t E; /* routed experts, 1..512 */
    int32_t S; /* shared (always-on) experts, 0..64 */
    int32_t K; /* experts per token, 1..min(E,16) */
} mpb_layer_desc;

/*
 * Bind a layer: its geometry and the weight page table of committed bitwidths
 * q_i (§3.1: one table row per linear-block; q_i is the bitwidth the serving
 * kernels read the block at). q_dev is a caller-owned device int32 array of
 * 2*(E+S) entries that the FFN kernels read; q_init_host (2*(E+S) values in
 * 3..8) is copied into it on `stream` and into the host mirror, and all planes
 * of every block are marked resident. `stream` becomes the stream on which
 * set_committed_bits enqueues its updates. Rebinding replaces the previous
 * layer. Errors: MPB_E_ARG (null pointer), MPB_E_SHAPE (geometry outside the
 * ranges above), MPB_E_RANGE (an initial q outside 3..8), MPB_E_HIP.
 */
int mpb_init(const mpb_layer_desc* d, int32_t* q_dev, const int32_t* q_init_host, void* stream);

/* Bytes of one packed plane page of an [N][Kd] block: N * ceil(Kd/128) * 16
 * (= N*Kd/8 when Kd is a multiple of 128; rows are padded to 128 elements). */
size_t mpb_plane_page_bytes(int N, int Kd);

/*
 * Packer (bit-plane layout for the kernels). Reads one block's canonical planes
 * canon_dev ([8][N][Kd/32] uint32, device) and writes 8 packed plane pages,
 * plane_pages_host[p] (host array of 8 device pointers, each
 * mpb_plane_page_bytes(N, Kd) bytes). Packed pages are plane-major, so a block
 * at bitwidth b is read through its first b pages only (§3.1: a b-bit block
 * consists of b bit-planes and the b-bit table). The packed layout inside a
 * page is private to this library. Needs N % 32 == 0 and Kd % 64 == 0, else
 * MPB_E_SHAPE. Does not need mpb_init.
 */
int mpb_pack_block(const uint32_t* canon_dev, int N, int Kd, uint32_t* const* plane_pages_host,
                   void* stream);

/*
 * Table images (§2.2: a b-bit weight is its b-bit index plus the b-bit lookup
 * table; §3.3: the fused kernel reads the table at the committed bitwidth).
 * moe_ffn reads every block's b-bit LUT from an image laid out the way its
 * kernels hold tables on chip, so that a workgroup loads its part with plain
 * copies. kind 0: a gate_up block (N = 2I rows: 0..I-1 gate, I..2I-1 up;
 * N % 128 == 0); kind 1: a down block (N = H rows; N % 64 == 0); N <= 131072;
 * b in 3..8.
 * mpb_table_image_bytes returns ceil(N/128) * 256 * 2^b, or MPB_E_ARG (bad
 * kind), MPB_E_RANGE (b) or MPB_E_SHAPE (N). mpb_pack_table reads the canonical
 * [N][2^b] fp16 LUT lut_dev and writes the image to image_dev (that many
 * bytes, device), enqueued on stream; same errors plus MPB_E_ARG for a null
 * pointer and MPB_E_HIP. The layout inside an image is private to this
 * library. Neither needs mpb_init.
 */
int64_t mpb_table_image_bytes(int kind, int N, int b);
int mpb_pack_table(int kind, const uint16_t* lut_dev, int N, int b, uint16_t* image_dev, void* stream);

/*
 * Router (§2.1: a learned gate scores all E experts per token; the K best are
 * run and weighted). X_dev: [T][H] activations of x_dtype (MPB_F16 or
 * MPB_BF16); W_router_dev: [E][H] fp32; bias_dev: [E] fp32 added to the
 * logits, or NULL. Logits are accumulated in fp64 (every product of an
 * activation and a router weight is exact in fp64) in a fixed order. Writes
 * topk_idx_dev [T][K] int32: the K largest exact logits in descending order,
 * ties to the lower expert index (the fp64 order is checked against a bound
 * on its rounding error; experts the bound cannot separate are ranked again
 * on their exact sums), and topk_w_dev [T][K] fp32 = softmax over all E
 * experts restricted to the K winners and renormalised (equal to a softmax
 * over the K winning fp64 logits).
 * ws_dev: device workspace of ws_bytes >= moe_route_workspace_bytes(T, E)
 * (fp64 logits, summed in up to 8 hidden-dimension parts for small batches,
 * and the norms that bound their rounding error; unused for batches of up to
 * 128 tokens with E * H <= 16384, whose logits stay on chip; contents not
 * preserved). Needs
 * 1 <= K <= min(E, 16), E <= 512, H a multiple of 64 up to 65536, T <= 2^20;
 * T == 0 is a no-op. Errors: MPB_E_ARG, MPB_E_SHAPE, MPB_E_WS, MPB_E_HIP.
 * Does not need mpb_init.
 */
size_t moe_route_workspace_bytes(int T, int E);
int moe_route(const void* X_dev, int x_dtype, const float* W_router_dev, const float* bias_dev,
              int T, int H, int E, int K, int32_t* topk_idx_dev, float* topk_w_dev, void* ws_dev,
              size_t ws_bytes, void* stream);

/*
 * Routing mass of a batch (§2.1, Eq. 1; the statistic the planner's hot and
 * cold buckets are built from, §3.2): mass_dev[e] = sum of topk_w over the
 * entries routed to expert e / sum of topk_w over all entries, for e < E, in
 * fp64 with a fixed summation order (deterministic). topk_idx_dev/topk_w_dev
 * are [T][K] as written by moe_route; ids outside [0, E) are ignored; an
 * empty batch gives zeros. Needs E <= 512, K <= min(E, 16), T <= 2^20.
 * Errors: MPB_E_ARG, MPB_E_SHAPE, MPB_E_HIP. Does not need mpb_init.
 */
int moe_routing_mass(const int32_t* topk_idx_dev, const float* topk_w_dev, int T, int E, int K,
                     double* mass_dev, void* stream);

/* Workspace bytes moe_ffn needs for T tokens of the bound layer (0 if unbound). */
size_t moe_ffn_workspace_bytes(int T);

/*
 * Fused MoE FFN of the bound layer (§3.3): groups the T tokens by expert,
 * runs gate_up + SwiGLU (h = SiLU(gate) * up) and the down projection of
 * every expert with tokens, and accumulates
 *   out[t] = sum_k topk_w[t][k] * FFN_{topk_idx[t][k]}(x_t) + sum_s FFN_{E+s}(x_t).
 * Each block's weights are dequantised on the fly from its first q_i packed
 * plane pages and its q_i-bit LUT, with q_i read from q_dev on the device.
 *   X_dev       [T][H] x_dtype activations
 *   topk_idx_dev/topk_w_dev  [T][K] as produced by moe_route; expert ids
 *               outside [0, E) contribute nothing
 *   planes_dev  device array of 2*(E+S)*8 device pointers: entry i*8 + p is
 *               plane page p of block i (written by mpb_pack_block). Only pages
 *               p < q_i are dereferenced.
 *   luts_dev    device array of 2*(E+S)*6 device pointers: entry i*6 + (b-3) is
 *               block i's b-bit table image (mpb_pack_table; kind 0 for even
 *               i, kind 1 for odd i). Only b == q_i is read.
 *   q_dev       the page table bound by mpb_init (MPB_E_ARG for any other);
 *               values 3..8
 *   out_dev     [T][H] fp32, overwritten
 *   ws_dev      workspace of ws_bytes >= moe_ffn_workspace_bytes(T)
 *   stream      the stream bound by mpb_init, where set_committed_bits
 *               writes q_i (so every launch is ordered with every commit, and
 *               page offloads wait for the launches that may read the pages),
 *               or a stream under graph capture (its kernels run when the
 *               graph is replayed; ordering replays against commits and page
 *               offloads is then the caller's part). Any other stream:
 *               MPB_E_ARG.
 * The kernels' on-chip table space is sized at enqueue time for the highest
 * bitwidth in the host mirror; a graph captured from this call must be
 * captured again after a block is raised above that bitwidth (its outputs
 * would otherwise be NaN, never silently wrong).
 * Results are deterministic for every T: the grouping counts with integer
 * atomics only, and every floating-point sum runs in a fixed order.
 * Errors: MPB_E_UNINIT, MPB_E_ARG, MPB_E_WS, MPB_E_HIP, and MPB_E_SHAPE when T
 * is too large for the layer (the kernels address the activations, T*H*2
 * bytes, and h, about 4*T*(K+S)*I bytes, with 32-bit offsets: each must stay
 * below 4 GiB; the launch grid must stay below 2^31 workgroups).
 */
int moe_ffn(const void* X_dev, int x_dtype, int T, const int32_t* topk_idx_dev,
            const float* topk_w_dev, const uint32_t* const* planes_dev,
            const uint16_t* const* luts_dev, const int32_t* q_dev, float* out_dev, void* ws_dev,
            size_t ws_bytes, void* stream);

/*
 * moe_ffn for callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * arguments, kernels and results as moe_ffn, with the workspace taken from a
 * device array that the library holds, 32 MiB per GPU, for the life of the
 * process (its address is looked up once per device, at mpb_init or at the
 * first call on that device). Allocates nothing itself; the caller still
 * passes inputs and outputs. Tokens whose workspace (moe_ffn_workspace_bytes
 * for bf16, slightly less for fp16) exceeds 32 MiB are refused with
 * MPB_E_WS: the limit is 292 tokens for a layer of H 2048, I 1408, 60 routed
 * + 4 shared experts, top-4, and 151 tokens for H 4096, I 14336, 8 experts,
 * top-2. Every call on one GPU shares that
 * GPU's array and leaves its contents behind; nothing in it needs to start at
 * zero. Calls that overlap on one GPU (on different streams, or from
 * different threads) race on the array and must be serialised by the caller.
 * Errors: as moe_ffn.
 */
int moe_ffn_static(const void* X_dev, int x_dtype, int T, const int32_t* topk_idx_dev,
                   const float* topk_w_dev, const uint32_t* const* planes_dev,
                   const uint16_t* const* luts_dev, const int32_t* q_dev, float* out_dev, void* stream);

/*
 * The whole layer in one launch (§3.3: routing, expert activation, down
 * projection and output accumulation in one fused kernel): moe_route followed
 * by moe_ffn, as one persistent kernel whose workgroups take units of work in
 * a fixed order (router logits, top-K, grouping, gate_up tiles, down tiles,
 * combine) and wait on device counters for the units they read from; a down
 * tile starts as soon as its own group's gate_up tiles are done. Results are
 * bit-identical to moe_route + moe_ffn on the same inputs (same arithmetic,
 * same order), except that for batches of up to 128 tokens with at most 16384
 * router weights moe_route sums each fp64 logit in another fixed order, which
 * can change the routing only where two logits lie within an fp64 ulp of a
 * tie or a weight within one of an fp32 rounding boundary. Arguments as for
 * those two calls; topk_idx_dev / topk_w_dev
 * receive the routing. ws_dev: at least moe_fused_workspace_bytes(T) bytes,
 * 256-byte aligned; its first moe_fused_counter_bytes() bytes are counters
 * that must be zero before the first call with this workspace (allocate it
 * zero-filled); every call leaves them zero again, so the workspace can be
 * reused, also by graph replays.
 * Calls sharing a workspace must not overlap. Every device-side wait is
 * bounded: a wait that runs out (only possible if the counters were not zero)
 * makes out NaN. Gate_up takes 32-token items (the decode configuration) for
 * every T. The stream rule is moe_ffn's. Errors: as moe_route and moe_ffn, plus MPB_E_ARG for a misaligned
 * workspace.
 */
size_t moe_fused_counter_bytes(void);
size_t moe_fused_workspace_bytes(int T);
int moe_fused(const void* X_dev, int x_dtype, int T, const float* W_router_dev, const float* bias_dev,
              int32_t* topk_idx_dev, float* topk_w_dev, const uint32_t* const* planes_dev,
              const uint16_t* const* luts_dev, const int32_t* q_dev, float* out_dev, void* ws_dev,
              size_t ws_bytes, void* stream);

/*
 * Norms before and after a block, fused with its gate and residual scale: what
 * reads the residual stream before a MoE layer and adds the layer's output to
 * it. With rms(v) = 1 / sqrt(mean(v^2) + eps) over a row of H elements,
 *   u = o rms(o) gamma_post       (u = o where gamma_post_dev is NULL)
 *   y = r + scale * sigmoid(gate) * u     (no factor for MPB_GATE_NONE)
 *   r_out = y,  x_out = y rms(y) gamma_next
 * in fp32, each output rounded once (x_out is formed from the unrounded y).
 *   o_dev       [T][H] fp32, the block's output as moe_ffn writes it, or NULL:
 *               nothing is added (y = r), r_out_dev must be NULL and only x_out
 *               is written (the norm before the first block)
 *   r_dev       [T][H] x_dtype residual stream
 *   gate_dev    MPB_GATE_TOKEN: [T] fp32; MPB_GATE_FULL: [T][H] x_dtype; NULL
 *               for MPB_GATE_NONE. Gate values before the sigmoid.
 *   gamma_post_dev, gamma_next_dev   [H] fp32 multipliers (a model that stores
 *               gamma - 1 passes 1 + its weights), or NULL: no norm of o, no
 *               x_out. gamma_next_dev and x_out_dev go together.
 *   r_out_dev, x_out_dev   [T][H] x_dtype; r_out may be r itself.
 * Row pointers and gammas are 16-byte aligned. scale finite, eps > 0. Needs H a
 * multiple of 64 up to 65536, T <= 2^20; T == 0 is a no-op. Rows beyond T are
 * not touched. Squares are summed in fp32: a row whose sum of squares passes
 * 3.4e38 has rms 0.
 * Errors: MPB_E_ARG, MPB_E_SHAPE, MPB_E_HIP. Does not need mpb_init.
 */
enum { MPB_GATE_NONE = 0, MPB_GATE_TOKEN = 1, MPB_GATE_FULL = 2 };
int moe_block_norm(const float* o_dev, const void* r_dev, int x_dtype, int T, int H, const void* gate_dev,
                   int gate_kind, const float* gamma_post_dev, const float* gamma_next_dev, float scale, float eps,
                   void* r_out_dev, void* x_out_dev, void* stream);

/*
 * Backward pass of moe_block_norm. y_dev is the stream after the block (the
 * r_out it wrote; r itself for a call with o NULL); dr_out_dev and dx_dev are
 * the gradients of r_out and x_out ([T][H] x_dtype; either may be NULL: zeros,
 * and dx NULL means that the forward call had no x_out: gamma_next is NULL too
 * and y_dev may be). Writes
 *   dr_dev      [T][H] x_dtype, the gradient of r
 *   do_dev      [T][H] fp32, the gradient of o, or NULL
 *   dgate_dev   in the gate's form and type, or NULL
 *   dgamma_post_dev, dgamma_next_dev   [H] fp32 sums over the T rows, or NULL
 * o_dev is read only with a gate or gamma_post and may be NULL otherwise.
 * dr may be dr_out or dx itself, and do may be o. Every sum is in fp32 and in
 * a fixed order (deterministic). ws_dev (16-byte aligned): at least
 * moe_block_norm_grad_workspace_bytes(T, H) bytes, needed only for the gamma
 * gradients; contents not preserved, one per call that may overlap another.
 * T == 0 zeroes the gamma gradients.
 * Limits and errors as above, plus MPB_E_WS.
 */
size_t moe_block_norm_grad_workspace_bytes(int T, int H);
int moe_block_norm_grad(const float* o_dev, const void* y_dev, int x_dtype, int T, int H, const void* gate_dev,
                        int gate_kind, const float* gamma_post_dev, const float* gamma_next_dev, float scale,
                        float eps, const void* dr_out_dev, const void* dx_dev, void* dr_dev, float* do_dev,
                        void* dgate_dev, float* dgamma_post_dev, float* dgamma_next_dev, void* ws_dev,
                        size_t ws_bytes, void* stream);

/*
 * Router losses of a batch: the load-balance loss and the z loss that train or
 * watch a router, with the per-expert counts. Over the live tokens (mask_dev[t]
 * != 0, or all where mask_dev is NULL; a token all of whose logits are -inf is
 * not live either),
 *   l = X W_router^T + bias, lse = log sum_e exp(l), p = exp(l - lse)
 *   counts[e] = live (token, slot) pairs with topk_idx = e,  counts[E] = N =
 *               live tokens,  prob[e] = sum_t p_te
 *   balance = E / (K N^2) sum_e counts[e] prob[e]   (1 for a uniform router)
 *   z = 1/N sum_t lse_t^2
 *   loss[0..2] = alpha balance + beta z, balance, z
 *   X_dev, W_router_dev, bias_dev, topk_idx_dev   as for moe_route (16-byte
 *               aligned X and W_router); ids outside [0, E) are not counted
 *   logits_dev  [T][E] fp32, lse_dev [T] fp32: kept for the gradient. Rows of
 *               masked tokens are zeros (what X holds there is not used); a
 *               token that is not live for its logits has lse -inf.
 *   counts_dev  [E + 1] int32, prob_dev [E] fp32, loss_dev [3] fp32
 * Sums over a data-parallel group: counts and prob add up over ranks, and the
 * gradient below takes the added counts (the balance loss of the global batch).
 * The logits are exact products accumulated in fp32, in an order other than
 * moe_route's fp64 one; every sum has a fixed order (deterministic). No live
 * token: losses 0. ws_dev (16-byte aligned): at least
 * moe_router_loss_workspace_bytes(T, H, E) bytes (for this T: a smaller batch
 * may need more), contents not preserved, one per call that may overlap
 * another. Infinite inputs of a live token give its logits, and with them the
 * losses, infinite or NaN values. Limits as for moe_route. Errors: MPB_E_ARG,
 * MPB_E_SHAPE, MPB_E_WS, MPB_E_HIP. Does not need mpb_init.
 */
size_t moe_router_loss_workspace_bytes(int T, int H, int E);
int moe_router_loss(const void* X_dev, int x_dtype, const float* W_router_dev, const float* bias_dev,
                    const int32_t* topk_idx_dev, const uint8_t* mask_dev, int T, int H, int E, int K, float alpha,
                    float beta, float* logits_dev, float* lse_dev, int32_t* counts_dev, float* prob_dev,
                    float* loss_dev, void* ws_dev, size_t ws_bytes, void* stream);

/*
 * Gradients of moe_router_loss's loss[0], and of whatever used the routing
 * weights, with respect to X, W_router and bias. With f_e = counts[e] / (K N)
 * (the counts have no gradient) and w the routing weights (the softmax over the
 * token's K winning logits, as moe_route writes them),
 *   dl_te = gloss p_te (alpha E / N (f_e - sum_j f_j p_tj) + 2 beta / N lse_t)
 *         + sum over slots k with topk_idx = e of w_k (gw_k - sum_j w_j gw_j)
 *   dX = dl W_router, dW_router = dl^T X, dbias = sum_t dl
 * for live tokens; a token that is not live has dl = 0, a zero row of dX, and
 * its X is not used.
 *   logits_dev, lse_dev   as moe_router_loss wrote them
 *   counts_dev  as it wrote them, or their sum over a data-parallel group
 *   gw_dev      [T][K] fp32 gradient of the routing weights, or NULL (zeros);
 *               slots whose id is outside [0, E) are left out of w
 *   gloss_dev   device fp32 scalar, the gradient of loss[0], or NULL (1)
 *   dX_dev [T][H], dW_dev [E][H], dbias_dev [E]   fp32 (the gradients of a
 *               mean over a batch fall below fp16's range), each may be NULL
 * Accumulated in fp32, every sum in a fixed order: dW from dl and X exactly,
 * dX from dl and W_router to 22 bits each, where a value is not below 2^-28 of
 * its token's largest dl or its column's largest W_router (below that to 2^-49
 * of the largest). Workspace (the forward call's may be reused), limits and errors as
 * above.
 */
int moe_router_loss_grad(const void* X_dev, int x_dtype, const float* W_router_dev, const int32_t* topk_idx_dev,
                         const uint8_t* mask_dev, const float* logits_dev, const float* lse_dev,
                         const int32_t* counts_dev, int T, int H, int E, int K, float alpha, float beta,
                         const float* gw_dev, const float* gloss_dev, float* dX_dev, float* dW_dev, float* dbias_dev,
                         void* ws_dev, size_t ws_bytes, void* stream);

/*
 * Low-rank adapters of many requests beside a projection that all of them
 * share: for token t with adapter a = adapter_dev[t],
 *   out_t = base_t + scales[a] * B_a (A_a x_t)
 * and out_t = base_t for a token whose id is outside [0, n) (none).
 *   X_dev       [T][Kd] x_dtype
 *   A_dev       [n][R][Kd] x_dtype, B_dev [n][N][R] x_dtype: n adapters stacked
 *               for rank up to R. Rows of A and columns of B past an adapter's
 *               own rank are not used, whatever they hold.
 *   ranks_dev   [n] int32 or NULL (all R); values are clamped to 0..R, an
 *               adapter of rank 0 adds nothing
 *   scales_dev  [n] fp32 or NULL (1)
 *   adapter_dev [T] int32, in any order
 *   base_dev    [T][N] fp32, e.g. what moe_ffn wrote, or NULL (zeros)
 *   out_dev     [T][N] fp32; may be base_dev (tokens without an adapter are
 *               then not touched)
 * Tokens are gathered by adapter on the device, so ids may change from call to
 * call (also under graph replay). Products are exact, sums fp32 in a fixed
 * order (deterministic), and A_a x_t is not rounded below fp32; a token whose x,
 * A_a or B_a holds infinite values gets infinite or NaN ones. Needs Kd and N
 * multiples of 64 (Kd <= 65536, N <= 131072), R a multiple of 8 in 8..128, n in
 * 1..4096, T <= 2^20, 16-byte aligned rows; T == 0 is a no-op. ws_dev (16-byte
 * aligned): at least moe_adapters_workspace_bytes(T, Kd, n, R) bytes (for this
 * T: a smaller batch may need more), contents not preserved; calls that may
 * overlap need a workspace each. Errors:
 * MPB_E_ARG, MPB_E_SHAPE, MPB_E_WS, MPB_E_HIP. Does not need mpb_init.
 */
size_t moe_adapters_workspace_bytes(int T, int Kd, int n, int R);
int moe_adapters(const void* X_dev, int x_dtype, int T, int Kd, const void* A_dev, const void* B_dev,
                 const int32_t* ranks_dev, const float* scales_dev, int n, int R, int N, const int32_t* adapter_dev,
                 const float* base_dev, float* out_dev, void* ws_dev, size_t ws_bytes, void* stream);

/*
 * Dense projection with bias, activation and residual in its epilogue: the
 * projection that all requests share (moe_adapters' base), the products of a dense
 * layer, a model's output head.
 *   z = X W^T + bias,  y = res + act(z)
 *   X_dev       [T][Kd] x_dtype;  W_dev [N][Kd] x_dtype;  bias_dev [N] fp32 or NULL
 *   act         MPB_ACT_*: none, relu, silu z / (1 + e^-z), gelu z Phi(z), or its
 *               form z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3)))
 *   res_dev     [T][N] of y's type, or NULL; may be y_dev
 *   z_dev       [T][N] x_dtype, what the gradient needs of an activation, or NULL
 *   y_dev       [T][N] of y_dtype: x_dtype or MPB_F32
 * Products are exact, sums fp32 in a fixed order (deterministic), and act is taken
 * of the unrounded z, in fp32: a sigmoid of x within (6 + |x|) 2^-24 of itself (for y of
 * 16 bits 0 below x = -88.7), Phi(-|z|) within (18 + 1.1 z^2) 2^-24 of itself (either
 * may be 0 where it is under 2^-126). Each output is rounded once. Needs Kd a multiple of
 * 64 up to 65536, N a multiple of 8 up to 524288, T <= 2^20, 16-byte aligned rows; T == 0
 * is a no-op. ws_dev (16-byte aligned): at least moe_linear_workspace_bytes(T, Kd, N)
 * bytes (for this T: a smaller batch may need more), contents not preserved; calls
 * that may overlap need a workspace each. Errors: MPB_E_ARG, MPB_E_SHAPE, MPB_E_WS,
 * MPB_E_HIP. Does not need mpb_init.
 */
enum { MPB_ACT_NONE = 0, MPB_ACT_RELU = 1, MPB_ACT_SILU = 2, MPB_ACT_GELU = 3, MPB_ACT_GELU_TANH = 4 };
size_t moe_linear_workspace_bytes(int T, int Kd, int N);
int moe_linear(const void* X_dev, int x_dtype, const void* W_dev, const float* bias_dev, int act, const void* res_dev,
               int T, int Kd, int N, void* z_dev, void* y_dev, int y_dtype, void* ws_dev, size_t ws_bytes,
               void* stream);

/*
 * Gradients of moe_linear (that of res is dy itself). From z as the forward call
 * wrote it (NULL for MPB_ACT_NONE) and the gradient of y,
 *   dz = dy act'(z);  dX = dz W,  dW = dz^T X,  dbias = sum_t dz
 *   dy_dev      [T][N] of dy_dtype: x_dtype or MPB_F32
 *   dX_dev      [T][Kd] x_dtype;  dW_dev [N][Kd] fp32;  dbias_dev [N] fp32; each
 *               may be NULL (W_dev is read for dX, X_dev for dW)
 * relu' is 0 at 0. Sums are fp32 in a fixed order (deterministic). Where dz is not
 * dy itself (an activation, or fp32 dy) the products take it in two fp16 parts, bf16 X
 * and W as fp16 beside them: dX and dW from dz to 22 bits, dbias from dz itself; dz is
 * also off by 2^-38 of the largest |dy|, X and W by 2^-38 of their largest.
 * fp16 parts carry a power of two, so that small gradients keep their bits whatever
 * their range; an infinite or NaN dz gives infinite or NaN sums. T == 0 zeroes dW
 * and dbias. ws_dev: at least moe_linear_grad_workspace_bytes(T, Kd, N, act, dy_dtype)
 * bytes. Limits and errors as above.
 */
size_t moe_linear_grad_workspace_bytes(int T, int Kd, int N, int act, int dy_dtype);
int moe_linear_grad(const void* X_dev, int x_dtype, const void* W_dev, int act, const void* z_dev, const void* dy_dev,
                    int dy_dtype, int T, int Kd, int N, void* dX_dev, float* dW_dev, float* dbias_dev, void* ws_dev,
                    size_t ws_bytes, void* stream);

/*
 * Norms of query and key heads and the rotation by their positions, in one pass:
 * what follows the projection of queries, keys and values. For every head
 *   n = x rms(x) gamma, rms(x) = 1 / sqrt(mean(x^2) + eps)   (n = x without gamma)
 *   out = n with the pairs of its first Dr elements turned: pair i, (a, b), to
 *   (a cos f - b sin f, a sin f + b cos f), f = pos[axis_i][t] freq_i
 *   q_dev, k_dev   [T][Hq][D] and [T][Hk][D] x_dtype, q_stride and k_stride
 *               elements from token to token (slices of one packed projection);
 *               k_dev may be NULL with Hk 0
 *   gamma_q_dev, gamma_k_dev   [D] fp32, or NULL: that side has no norm
 *   pos_dev     [A][T] int32 positions, one row for each of A axes (time, height
 *               and width of image and video tokens; A = 1 for text)
 *   axis_dev    [Dr / 2] int32, the axis of every pair, or NULL (axis 0); a pair
 *               whose axis is outside [0, A) is not turned
 *   freq_dev    [Dr / 2] fp32, radians a position
 *   pairs       MPB_PAIRS_HALVES: pair i is elements i and i + Dr / 2;
 *               MPB_PAIRS_NEIGHBOURS: elements 2 i and 2 i + 1
 *   q_out_dev, k_out_dev   x_dtype, their own strides; may be q_dev and k_dev with
 *               the same strides
 * Dr == 0: no rotation (pos, axis and freq are not used). Angles are formed in fp64
 * and kept as a fraction of a turn: positions of 2^31 keep 2^-24 of a turn. The
 * rest is fp32, each output rounded once. Needs D and Dr multiples of 16, 16 <= D
 * <= 512, Dr <= D, Hq in 1..1024, Hk in 0..1024, A in 1..8, T <= 2^20, strides
 * multiples of 8 that hold the token's heads, 16-byte aligned pointers; T == 0 is a
 * no-op. Errors: MPB_E_ARG, MPB_E_SHAPE, MPB_E_HIP. Does not need mpb_init.
 */
enum { MPB_PAIRS_HALVES = 0, MPB_PAIRS_NEIGHBOURS = 1 };
int moe_head_norm(const void* q_dev, int64_t q_stride, const void* k_dev, int64_t k_stride, int x_dtype, int T, int Hq,
                  int Hk, int D, const float* gamma_q_dev, const float* gamma_k_dev, float eps, const int32_t* pos_dev,
                  int A, const int32_t* axis_dev, const float* freq_dev, int Dr, int pairs, void* q_out_dev,
                  int64_t q_out_stride, void* k_out_dev, int64_t k_out_stride, void* stream);

/*
 * Gradients of moe_head_norm: of q and k from those of q_out and k_out (x_dtype,
 * strides of their own), and of the two gammas, summed over tokens and heads.
 *   q_dev, k_dev   as in the forward call; a side without gamma is not read and may
 *               be NULL
 *   dq_dev, dk_dev   x_dtype; may be dq_out_dev and dk_out_dev, or q_dev and k_dev,
 *               with the same strides
 *   dgamma_q_dev, dgamma_k_dev   [D] fp32, or NULL
 * Sums are fp32 in a fixed order (deterministic). ws_dev (16-byte aligned): at least
 * moe_head_norm_grad_workspace_bytes(T, Hq, Hk, D) bytes, needed only for the gammas'
 * gradients; contents not preserved, one per call that may overlap another. T == 0
 * zeroes them. Limits and errors as above, plus MPB_E_WS.
 */
size_t moe_head_norm_grad_workspace_bytes(int T, int Hq, int Hk, int D);
int moe_head_norm_grad(const void* q_dev, int64_t q_stride, const void* k_dev, int64_t k_stride, int x_dtype, int T,
                       int Hq, int Hk, int D, const float* gamma_q_dev, const float* gamma_k_dev, float eps,
                       const int32_t* pos_dev, int A, const int32_t* axis_dev, const float* freq_dev, int Dr, int pairs,
                       const void* dq_out_dev, int64_t dq_out_stride, const void* dk_out_dev, int64_t dk_out_stride,
                       void* dq_dev, int64_t dq_stride, void* dk_dev, int64_t dk_stride, float* dgamma_q_dev,
                       float* dgamma_k_dev, void* ws_dev, size_t ws_bytes, void* stream);

/*
 * Distillation of a teacher's stored top logits: what a model whose experts run at
 * lower bitwidths loses against the full one, and its gradient, which trains what has a
 * backward pass here: the output head, dense projections and norms (the packed experts
 * and moe_adapters have none: past them it goes by the residual stream alone).
 * For every row, with p = softmax(s / tau) over the V student logits and k stored
 * teacher logits y_j at ids_j,
 *   q_j = exp(y_j / tau - L)
 *   kl  = sum_j q_j (log q_j - log p_j) + q_r (log q_r - log p_r)
 *   loss = tau^2 sum_t weight_t kl_t
 * Where teacher_lse_dev is given, L is the teacher's own logsumexp of y / tau over
 * its whole vocabulary, and what the k entries leave of both distributions is one
 * more outcome: q_r = 1 - sum_j q_j (not below 0), p_r = the student's probability
 * of all other ids. Where it is NULL, L is taken over the k entries and q_r = 0.
 *   S_dev       [T][V] s_dtype (MPB_F16, MPB_BF16 or MPB_F32), s_stride elements from row to
 *               row; rows may begin at any element
 *   ids_dev, teacher_dev   [T][k] int32 and fp32, in any order; an entry whose id is
 *               outside [0, V) does not count, entries of one id add up their q
 *   teacher_lse_dev   [T] fp32 or NULL
 *   weight_dev  [T] fp32, or NULL (1 / T); a row of weight 0 (padding) is not read,
 *               has kl 0 and a gradient of zeros
 *   stats_dev   [T][4] fp32, for moe_distill_loss_grad
 *   kl_dev      [T] fp32;  loss_dev [1] fp32
 *   dS_dev      the gradient of S, s_dtype and s_stride, formed in the same launch,
 *               or NULL; may be S_dev
 *   gloss_dev   device fp32 scalar, the gradient of loss, or NULL (1)
 * The gradient is gloss weight tau (Q p_v - q_v) for an entry and gloss weight tau
 * p_v (Q - q_r / p_r) elsewhere, Q = sum_j q_j + q_r. Student logits may be -inf
 * (masked): p_v = 0, and kl is infinite where the teacher gives such an id (or the
 * rest, if all of it is masked) weight. A row that is -inf throughout, or has no
 * entries, has kl 0 and a gradient of zeros. NaN and +inf logits give NaN. Exponentials
 * are fp32 and summed in fp32 in a fixed order, sums over the entries and rows are fp64;
 * loss and kl have the same bits with and without dS. dS may
 * not overlap S otherwise and lies at the same offset from a 16-byte boundary. Needs
 * V in 1..400000, k in 1..256, tau in 1e-3..1e3, T <= 2^20; T == 0: loss 0. Errors:
 * MPB_E_ARG, MPB_E_SHAPE, MPB_E_HIP. Does not need mpb_init.
 */
int moe_distill_loss(const void* S_dev, int s_dtype, int64_t s_stride, const int32_t* ids_dev, const float* teacher_dev,
                     const float* teacher_lse_dev, const float* weight_dev, int T, int V, int k, float tau,
                     float* stats_dev, float* kl_dev, float* loss_dev, void* dS_dev, const float* gloss_dev,
                     void* stream);

/* The gradient of moe_distill_loss as a call of its own, from its stats: the same
 * arguments, results and errors. */
int moe_distill_loss_grad(const void* S_dev, int s_dtype, int64_t s_stride, const int32_t* ids_dev,
                          const float* teacher_dev, const float* teacher_lse_dev, const float* weight_dev, int T, int V,
                          int k, float tau, const float* stats_dev, void* dS_dev, const float* gloss_dev, void* stream);

/*
 * Commit bitwidth b for linear-block i (§3.1 and §3.3: the planner lowers or
 * raises q_i at a safe boundary; a reload raises q_i only once its pages are
 * GPU-resident). Validates 0 <= i < 2*(E+S), b in 3..8 and that planes 0..b-1
 * of the block are GPU-resident (a reload whose copies have not completed
 * leaves its pages in transfer, and the commit is refused until they have:
 * MPB_E_NOT_RESIDENT). Then updates the host mirror and enqueues the device
 * write of q_dev[i] on the bound stream: FFN launches enqueued before it read
 * the old value, later ones the new value. Errors: MPB_E_UNINIT, MPB_E_RANGE,
 * MPB_E_NOT_RESIDENT, MPB_E_HIP.
 */
int set_committed_bits(int i, int b);

/*
 * Weight bytes the committed bitwidths hold (§3.1, Eq. 3: M_i^b counts the b
 * bit-planes and the b-bit LUT of block i): sum over blocks of
 * N_i*Kd_i*q_i/8 + N_i*2^q_i*2, from the host mirror. touched_host, if not
 * NULL, is a host array of 2*(E+S) flags restricting the sum. Returns the byte
 * count, or MPB_E_UNINIT.
 */
int64_t mpb_committed_bytes(const uint8_t* touched_host);

/* Host mirror of q_i (test and planner use); MPB_E_UNINIT / MPB_E_RANGE. */
int mpb_get_committed_bits(int i);

/*
 * Test export: dequantise one block through the same device index assembly and
 * LUT lookup the FFN kernels use. pages_host: host array of b device pointers
 * (packed plane pages 0..b-1); lut_b_dev: canonical [N][2^b] fp16 LUT; writes
 * out_f16_dev [N][Kd] fp16 in canonical element order. Shapes as for
 * mpb_pack_block; b in 3..8 else MPB_E_RANGE.
 */
int mpb_dequant_block(const uint32_t* const* pages_host, const uint16_t* lut_b_dev, int N, int Kd,
                      int b, uint16_t* out_f16_dev, void* stream);

/*
 * The same dequantisation (§3.1, Eq. 2) read through a table image
 * (mpb_pack_table of kind `kind` for this block, b bits, image_dev on the
 * device) the way the FFN kernels stage and index it: a check that an image
 * holds every table entry where those kernels look it up. Writes out_f16_dev
 * [N][Kd] fp16 in canonical element order. Shapes as for mpb_table_image_bytes
 * (N % 128 == 0 for kind 0, N % 64 == 0 for kind 1) and Kd % 64 == 0;
 * MPB_E_ARG for a bad kind or a null pointer,
 * MPB_E_RANGE (b), MPB_E_SHAPE, MPB_E_HIP.
 */
int mpb_dequant_block_image(const uint32_t* const* pages_host, const uint16_t* image_dev, int kind, int N,
                            int Kd, int b, uint16_t* out_f16_dev, void* stream);

/*
 * Page movement (§3.1 after Eq. 3, §3.3 "Asynchronous Page Movement",
 * Figure 4: an offload first lowers q_i, then moves the pages above it to CPU
 * memory; a reload first moves the pages back and raises q_i only once they
 * are GPU-resident). A weight page is one bit-plane with its table state
 * (§3.1): page p (0..7) of block i is plane page p and, for p >= 2, the table
 * image of bitwidth p + 1 (the table a block reads once it uses p + 1 planes),
 * so a block with r resident pages can run at any q_i <= r. Each page is in
 * one state: MPB_PAGE_GPU (p below the block's resident count),
 * MPB_PAGE_IN_TRANSFER (a copy is enqueued and not known to have completed)
 * or MPB_PAGE_CPU. The library only enqueues copies and tracks states; the
 * caller owns every buffer.
 *
 * mpb_offload_pages(i, r, ...): needs q_i <= r (else MPB_E_NOT_RESIDENT:
 * lower q_i with set_committed_bits first). Enqueues on copy_stream the
 * copies of the resident pages p = r..7 to host memory: plane page p
 * (mpb_plane_page_bytes(N, Kd) bytes) from dev_planes[p] to host_planes[p],
 * table image p + 1 (mpb_table_image_bytes(i % 2, N, p + 1) bytes) from
 * dev_tables[p - 2] to host_tables[p - 2]. The copies start after every
 * launch enqueued on the bound stream before the last lowering of q_i (the
 * only launches that may read those pages). The pages are IN_TRANSFER at once
 * (commits above r are refused from now on) and CPU when the copies have
 * completed; from then on no FFN launch reads them and the caller may reuse
 * their device memory. No-op if no page above r is resident.
 * mpb_reload_pages(i, r, ...): enqueues on copy_stream the copies of the
 * non-resident pages p < r from host memory into the caller's device buffers
 * dev_planes[p] / dev_tables[p - 2] (if these moved, the caller also writes
 * their addresses into the pointer arrays it passes to moe_ffn). They are
 * IN_TRANSFER until the copies have completed, then GPU, and only then may
 * q_i be raised to r. No-op if pages 0..r-1 are already resident.
 * dev_planes / host_planes: host arrays of 8 pointers (entry p: plane page
 * p); dev_tables / host_tables: host arrays of 6 pointers (entry b - 3: the
 * table image of bitwidth b). Only the entries of the pages that move are
 * read and must be non-NULL. Host buffers should be pinned (hipHostMalloc)
 * for the copies to be asynchronous. copy_stream: a hipStream_t other than
 * the bound one, so the copies overlap the layer's kernels. A block has at
 * most one transfer in flight: MPB_E_BUSY otherwise. States are refreshed by
 * polling the transfer's completion (never blocking) in every call that
 * reads them.
 * Errors: MPB_E_UNINIT, MPB_E_RANGE (i, or r outside 3..8), MPB_E_ARG (a
 * needed pointer is NULL), MPB_E_NOT_RESIDENT, MPB_E_BUSY, MPB_E_HIP.
 */
int mpb_offload_pages(int i, int r, void* const* host_planes, const uint32_t* const* dev_planes,
                      void* const* host_tables, const uint16_t* const* dev_tables, void* copy_stream);
int mpb_reload_pages(int i, int r, const void* const* host_planes, uint32_t* const* dev_planes,
                     const void* const* host_tables, uint16_t* const* dev_tables, void* copy_stream);

/* State of page p (0..7) of block i: MPB_PAGE_*, or MPB_E_UNINIT /
 * MPB_E_RANGE / MPB_E_HIP (the transfer's copy stream reported a failure). */
int mpb_page_state(int i, int p);

/* Number of GPU-resident pages of block i (3..8; pages 0..n-1 are resident),
 * or MPB_E_UNINIT / MPB_E_RANGE. */
int mpb_get_resident_planes(int i);

/*
 * Test hook: declare how many of block i's planes are GPU-resident (3..8)
 * without moving anything; set_committed_bits then refuses b > r. Lowering r
 * below the committed q_i is refused with MPB_E_NOT_RESIDENT (offload lowers
 * q_i first), and any change while a transfer is in flight with MPB_E_BUSY.
 * MPB_E_UNINIT / MPB_E_RANGE.
 */
int mpb_set_resident_planes(int i, int r);

/*
 * Planner step (§3.2, Algorithm 1; Eqs. 3-8), host only: turns KV-cache
 * pressure into a byte target D (Eq. 7), scores one-bit reductions of routed
 * linear-blocks by predicted damage (Eq. 4 global damage, Eq. 5-6 prompt
 * residual, Eq. 8 with the routing bucket's multiplier) per released byte
 * (Eq. 3), greedily builds one candidate plan per bitwidth-floor stage, keeps
 * the newest plan of every stage in the queue, and when pressure is triggered
 * selects the page-movement plan {(i, q_i -> d_i, Delta_i)}.
 * Readings of the steps the pages leave open:
 *  - a step lowers one block by one bit; a block's steps are taken in order;
 *    GreedySelect repeatedly takes the available step with the smallest
 *    damage / released bytes (ties to the lower block index) until the
 *    released bytes reach D;
 *  - stage s allows block i down to max(stage_floor[s], floor of i's routing
 *    bucket); relaxing the depth cap is moving to the next stage;
 *  - SelectBestPlan: the first stage whose plan reaches D, else the plan that
 *    releases the most bytes (the largest safe reduction), ties to the earlier
 *    stage;
 *  - pressure is triggered when F_blk <= T_blk; D uses F_blk - P_blk (free
 *    blocks after the pending KV growth);
 *  - routing buckets: experts sorted by routing mass, hottest first (ties to
 *    the lower index); bucket k ends at rank ceil(bucket_frac[k] * E);
 *  - candidates are routed blocks whose pages may move (movable_host[i] != 0,
 *    or every routed block if movable_host is NULL); shared experts' blocks
 *    never change.
 * Floating-point evaluation order is fixed (Eq. 5 summed left to right, eta
 * through the C library's exp, damage sums in step order), so a plan is
 * reproducible bit for bit.
 */
typedef struct {
    int32_t n_buckets;         /* 1..8 */
    double bucket_frac[8];     /* cumulative share of experts per bucket, increasing, last 1.0 */
    double mu[8];              /* damage multiplier per bucket, > 0 */
    int32_t floor[8];          /* bitwidth floor per bucket, 3..8 */
    int32_t n_stages;          /* 1..6 */
    int32_t stage_floor[6];    /* global floor per stage, 3..8, strictly decreasing */
    double eps;                /* damage floor of Eq. 8, > 0 */
    double alpha;              /* strength of Eq. 6 */
    double rho_min, rho_max;   /* clip range of Eq. 6, rho_min <= rho_max */
    /* Eq. 5-6 heads per block type u (0 gate_up, 1 down) and one-bit
     * transition b -> b-1, b = 4..8 at index b - 4 */
    double head_w[2][5][3];
    double head_a[2][5];
    double head_c[2][5];       /* confidence */
    int64_t T_blk;             /* free-block threshold (Eq. 7) */
    int64_t F_blk;             /* current free KV blocks */
    int64_t P_blk;             /* pending KV growth in blocks (0: Eq. 7 as printed) */
    int64_t B_kv;              /* bytes of one KV block */
} mpb_planner_params;

typedef struct {
    int32_t i;                 /* linear-block */
    int32_t from, to;          /* q_i -> d_i */
    int64_t delta;             /* M_i^{from} - M_i^{to} (Eq. 3) */
    double damage;             /* sum of the predicted damage of its steps */
} mpb_plan_entry;

typedef struct {
    int64_t D;                 /* byte target (Eq. 7) */
    int32_t triggered;         /* 1 if pressure is triggered */
    int32_t stage;             /* stage of the selected plan, -1 if not triggered */
    int32_t n_plan;            /* entries written to plan_host */
    int32_t pad;
    int64_t released;          /* sum of delta over the selected plan */
    double damage;             /* sum of damage over the selected plan (entry order) */
    int64_t stage_released[6]; /* per stage plan in the queue */
    double stage_damage[6];
} mpb_plan_summary;

/*
 * mpb_plan_step(d, q_host, movable_host, sens_host, mass_host, phi_host, prm,
 *               queue_host, plan_host, summary):
 *   d            layer geometry (as for mpb_init; no layer needs to be bound)
 *   q_host       [2(E+S)] committed bitwidths (3..8)
 *   movable_host [2(E+S)] flags or NULL
 *   sens_host    [2(E+S)][6] s_i^b for b = 3..8 (Eq. 4)
 *   mass_host    [E] routing mass (Eq. 1, e.g. from moe_routing_mass)
 *   phi_host     [2(E+S)][3] routed-input features (Eq. 5)
 *   queue_host   out: [n_stages][2(E+S)] desired bitwidths of each stage's
 *                plan (the refreshed plan queue); may be NULL
 *   plan_host    out: up to 2(E+S) entries, ascending i, only when triggered
 *   summary      out
 * All pointers are host memory owned by the caller. Does not touch the GPU.
 * Errors: MPB_E_ARG (null pointer, parameter out of its range),
 * MPB_E_SHAPE (geometry), MPB_E_RANGE (a q outside 3..8).
 */
int mpb_plan_step(const mpb_layer_desc* d, const int32_t* q_host, const uint8_t* movable_host,
                  const double* sens_host, const double* mass_host, const double* phi_host,
                  const mpb_planner_params* prm, int32_t* queue_host, mpb_plan_entry* plan_host,
                  mpb_plan_summary* summary);

/*
 * Profiling hook: with n == 5 or 7, every following moe_ffn records
 * events_host[0..n-1] (host array of hipEvent_t handles, caller-created) on
 * its stream: 0 before the grouping kernels, 1 and 2 at the start and end of
 * the gate_up kernel (recorded by its launch, so 1 -> 2 is the kernel alone
 * and 0 -> 1 includes the dispatch of gate_up), 3 before the combine and 4
 * after it, and with n == 7, 5 and 6 at the start and end of the down kernel
 * (recorded by its launch), so the caller can time each phase with
 * hipEventElapsedTime. n == 0 turns recording off. The handles are borrowed
 * until the hook is changed. MPB_E_ARG for any other n or a null handle.
 */
int mpb_set_kernel_events(void* const* events_host, int n);

/* Message of the calling thread's last failure ("" if none). */
const char* mpb_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* MPB_H */
