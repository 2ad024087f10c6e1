// kernels.h -- internal launch functions of libmoe (not part of the C ABI).
#pragma once

#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace moe {

// Counts one kernel launch (process-wide, for moe_launch_count()).
void count_launch();

// The status of an entry point whose CUDA call failed.  The runtime keeps such an error, and
// the next launcher that asks for the last one would report it for a call that was right:
// it is taken here, with the call that it belongs to.
inline moe_status cuda_failed() {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
}

// Launches and counts kern as a dependent of the kernel before it on the stream, in
// clusters of `cluster` blocks: it may be placed while that kernel still runs, and
// waits for it by dependency_wait() -- in every block, since what follows on the
// stream waits for kern alone -- before it touches what that kernel writes or reads.
// The kernel before may let it start early by dependency_release().
template <class... P, class... A>
cudaError_t launch_dependent(void (*kern)(P...), unsigned grid, unsigned threads, size_t smem,
                             unsigned cluster, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, P(args)...);
    count_launch();
    return err != cudaSuccess ? err : cudaGetLastError();
}
__device__ __forceinline__ void dependency_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void dependency_release() {
    asm volatile("griddepcontrol.launch_dependents;");
}

// tmap.cu: bf16 tensor maps, box = box_cols x box_rows (x 1), swizzle of
// swizzle_bytes (64 or 128 = the box's row length in bytes; 0 = none)
bool tensor_maps_available();
bool tensor_map_2d_bf16(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols,
                        uint32_t box_cols, uint32_t box_rows, uint32_t swizzle_bytes = 128);
bool tensor_map_3d_bf16(CUtensorMap *m, const void *base, uint64_t n_mat, uint64_t rows,
                        uint64_t cols, uint32_t box_cols, uint32_t box_rows,
                        uint32_t swizzle_bytes = 128);
// byte tiles (FP8 payload: row-major box without swizzle; int8 operands: 128-byte swizzle)
bool tensor_map_2d_u8(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols,
                      uint32_t box_cols, uint32_t box_rows, uint32_t swizzle_bytes = 0);
bool tensor_map_3d_u8(CUtensorMap *m, const void *base, uint64_t n_mat, uint64_t rows,
                      uint64_t cols, uint32_t box_cols, uint32_t box_rows,
                      uint32_t swizzle_bytes);

// two byte tensors [n_mat, rows, cols], the second `gap` bytes (below 2^40) behind the
// first, as one of five dimensions (column, row in group, first or second, group,
// matrix): a box brings box_groups groups of rows of both, the two in turn, with
// 128-byte swizzle.  The strides keep the encoder's stated limits (multiples of 16,
// below 2^40), but do not nest as in its example of a padded array, where each is the one
// before times an extent: gap stands before the group's stride, as the strides of
// any view with swapped dimensions do.  An address is the base plus coordinate times
// stride, dimension by dimension, and each coordinate is checked against its own extent,
// so every byte that a box brings lies in one of the two tensors.
bool tensor_map_pair_u8(CUtensorMap *m, const void *first, uint64_t gap, uint64_t n_mat,
                        uint64_t rows, uint64_t cols, uint32_t box_cols, uint32_t group,
                        uint32_t box_groups);

// route.cu
cudaError_t launch_route_select(const float *scores, const float *bias, int T, int E, int G,
                                int K, int M, int32_t *topk_idx, float *topk_w, cudaStream_t st);

// dispatch.cu
struct DispatchWs {
    int32_t *hist_t;       // [E, nblk] copies of expert e in token block b
    int32_t *base_t;       // [E, nblk] exclusive prefix of hist_t along b
    int32_t *send_part;    // [nblk, G*G]
    int32_t *sendtok_part; // [nblk, G*G]
};
constexpr int DISPATCH_BLOCK = 256;  // tokens per dispatch block
inline int dispatch_nblk(int T) { return (T + DISPATCH_BLOCK - 1) / DISPATCH_BLOCK; }
cudaError_t launch_dispatch(const void *x, const int32_t *topk_idx, int T, int d, int E, int G,
                            int K, int32_t *counts, int32_t *offsets, int32_t *send,
                            int32_t *send_tok, int32_t *perm_token, int32_t *inv_perm,
                            void *x_perm, const DispatchWs &ws, int32_t *status, cudaStream_t st);

// dispatch.cu: the gather-permute alone, x_perm[inv_perm[t][j]] = x[t]
// (rows of up to 14 KB through the copy engine with bounded waits recording into
// status, which may be null; wider rows by 16-byte thread copies)
cudaError_t launch_permute(const void *x, const int32_t *inv_perm, int T, int d, int K,
                           void *x_perm, cudaStream_t st, int32_t *status = nullptr,
                           int64_t timeout_ns = 2000000000LL);
// dispatch.cu, FP8 payload: x_perm_q[row] = E4M3(x[token] / s) and x_scale[row][b] = s
// (one scale per 128 channels, s = amax / 448); d % 128 == 0
cudaError_t launch_gather_fp8(const void *x, const int32_t *inv_perm, int T, int d, int K,
                              uint8_t *x_perm_q, float *x_scale, cudaStream_t st);

// ep.cu: expert parallelism over `world` ranks (E / world experts each)
cudaError_t launch_ep_plan(const int32_t *counts_all, int world, int E, int me, int32_t *base,
                           int32_t *local_offsets, cudaStream_t st);
cudaError_t launch_ep_dispatch(const void *x, const int32_t *topk_idx, const int32_t *offsets,
                               const int32_t *inv_perm, const int32_t *base, void *const *recv_x,
                               int64_t recv_rows, int T, int d, int E, int K, int world,
                               int32_t *status, cudaStream_t st);
cudaError_t launch_ep_dispatch_fp8(const void *x, const int32_t *topk_idx,
                                   const int32_t *offsets, const int32_t *inv_perm,
                                   const int32_t *base, void *const *recv_q,
                                   void *const *recv_scale, int64_t recv_rows, int T, int d, int E,
                                   int K, int world, int32_t *status, cudaStream_t st);
cudaError_t launch_ep_token_plan(const int32_t *topk_idx, int T, int E, int K, int world,
                                  int32_t *tok_slot, int32_t *tok_counts, cudaStream_t st);
cudaError_t launch_ep_token_base(const int32_t *tok_counts_all, int world, int me,
                                 int32_t *tok_base, cudaStream_t st);
cudaError_t launch_ep_dispatch_dedup(const void *x, const int32_t *topk_idx, const int32_t *offsets,
                                     const int32_t *inv_perm, const int32_t *base,
                                     const int32_t *tok_slot, const int32_t *tok_base,
                                     void *const *recv_tok, int32_t *const *recv_idx,
                                     int64_t tok_rows, int64_t recv_rows, int T, int d, int E, int K,
                                     int world, int32_t *status, cudaStream_t st,
                                     const float *topk_w = nullptr, int32_t *const *list = nullptr,
                                     float *const *lw = nullptr, int32_t *const *lcnt = nullptr);
cudaError_t launch_ep_fanout(const void *recv_tok, const int32_t *recv_idx,
                             const int32_t *local_offsets, int El, int64_t tok_rows,
                             int64_t recv_rows, int d, void *recv_x, int32_t *status,
                             cudaStream_t st);
cudaError_t launch_ep_dispatch_dedup_fp8(const void *x, const int32_t *topk_idx,
                                         const int32_t *offsets, const int32_t *inv_perm,
                                         const int32_t *base, const int32_t *tok_slot,
                                         const int32_t *tok_base, void *const *recv_tq,
                                         void *const *recv_ts, int32_t *const *recv_idx,
                                         int64_t tok_rows, int64_t recv_rows, int T, int d, int E,
                                         int K, int world, int32_t *status, cudaStream_t st);
cudaError_t launch_ep_fanout_fp8(const void *recv_tq, const float *recv_ts,
                                 const int32_t *recv_idx, const int32_t *local_offsets, int El,
                                 int64_t tok_rows, int64_t recv_rows, int d, void *recv_q,
                                 float *recv_scale, int32_t *status, cudaStream_t st);
cudaError_t launch_ep_combine_plan(const int32_t *topk_idx, const float *topk_w,
                                   const int32_t *offsets, const int32_t *inv_perm,
                                   const int32_t *base, const int32_t *tok_slot,
                                   const int32_t *tok_base, int32_t *const *list,
                                   float *const *lw, int32_t *const *lcnt, int64_t tok_rows,
                                   int64_t recv_rows, int T, int E, int K, int world,
                                   int32_t *status, cudaStream_t st);
cudaError_t launch_ep_precombine(const void *recv_y, const int32_t *list, const float *lw,
                                 const int32_t *lcnt, const int32_t *tok_base, int world,
                                 int64_t tok_rows, int64_t recv_rows, int d, int K, void *partial,
                                 int32_t *status, cudaStream_t st);
cudaError_t launch_ep_combine_dedup(const int32_t *topk_idx, const int32_t *tok_slot,
                                    const int32_t *tok_base, const void *const *partial,
                                    const void *y_shared, int64_t tok_rows, int T, int d, int E,
                                    int K, int world, void *out, int32_t *status,
                                    cudaStream_t st);
cudaError_t launch_ep_combine(const int32_t *topk_idx, const float *topk_w, const int32_t *offsets,
                              const int32_t *inv_perm, const int32_t *base,
                              const void *const *recv_y, int64_t recv_rows, const void *y_shared,
                              int T, int d, int E, int K, int world, void *out, int32_t *status,
                              cudaStream_t st);

// pack.cu: expert weights as tile-contiguous, pre-swizzled 32 KB blocks
// (byte offsets of the four regions inside the packed buffer)
struct PackedLayout {
    int nt1, kb1, nt2, kb2, nt1s, kb2s;  // column tiles / k blocks per region
    size_t gu, down, gu_s, down_s, total;
};
PackedLayout packed_layout(int E, int d, int d_ff, int n_shared, int d_ff_shared);
cudaError_t launch_pack_weights(int E, int d, int d_ff, int n_shared, int d_ff_shared,
                                const void *w_gate, const void *w_up, const void *w_down,
                                const void *ws_gate, const void *ws_up, const void *ws_down,
                                void *packed, cudaStream_t st);

// combine.cu
cudaError_t launch_combine(const void *y_perm, const int32_t *inv_perm, const float *topk_w,
                           const void *y_shared, int T, int d, int K, int64_t n_rows, void *out,
                           cudaStream_t st);

// gemm_sm100.cu
struct FfnArgs {
    int T, d, E, K, d_ff, n_shared, d_ff_shared;
    const void *x_perm;        // [T*K, d] bf16, or unused when perm_token / x_perm_q is set
    const int32_t *perm_token; // [T*K] or nullptr: routed row r of GEMM1 is x[perm_token[r]]
    const uint8_t *x_perm_q;   // [T*K, d] FP8 E4M3 payload or nullptr (with x_scale)
    const float *x_scale;      // [T*K, d/128]
    const int32_t *offsets;
    const void *w_gate, *w_up, *w_down;
    void *h;        // [T*K, d_ff] bf16 scratch
    void *y_perm;   // [T*K, d] bf16
    const void *x;  // [T, d]
    const void *ws_gate, *ws_up, *ws_down;
    const void *packed;  // weights from launch_pack_weights, or null: the row-major ones above
    void *h_shared; // [T, n_shared*d_ff_shared] bf16 scratch
    void *y_shared; // [T, d]
    int32_t *status;   // the workspace's 256-byte status block: word 0 the status,
                       // words 16 and 17 the grouped GEMMs' tile counters
    int64_t timeout_ns;
};
cudaError_t launch_expert_ffn(const FfnArgs &a, cudaStream_t st);
// router_tc.cu: router affinities on the tensor cores; e (fp32 [E, d]) is
// split into three bf16 parts in e_split ([3, E, d] bf16 scratch);
// scores = f(x.e + off), f = sigmoid (affinity 0) or sqrt(softplus) (1).
// Work is split over d into router_splits(T, E, d) ranges when the batch has
// too few 128 x 128 tiles to fill the SMs; partial ([splits, T, E] fp32
// scratch, needed when splits > 1) holds their logits.
inline int router_splits(int T, int E, int d) {
    const int tiles = ((T + 127) / 128) * ((E + 127) / 128);
    const int kmax = d / 64 / 4;  // at least four k blocks per range
    int s = tiles > 0 ? 148 / tiles : 1;
    if (s > kmax) s = kmax;
    return s < 1 ? 1 : s;
}
cudaError_t launch_router_logits_tc(const void *x, const float *e, const float *off, int T, int d,
                                    int E, int affinity, void *e_split, float *partial,
                                    float *scores, int32_t *status, int64_t timeout_ns,
                                    cudaStream_t st);

// router_tc.cu: e (fp32 [E, d]) -> its three exact bf16 parts e_split [3, E, d]
cudaError_t launch_router_split(const float *e, int E, int d, void *e_split, cudaStream_t st);

// router_fused.cu: affinities and node-limited top-K in one kernel (E <= 256,
// G <= 32, E/G <= 32), from the bf16 parts written by launch_router_split;
// scores (nullable) receives the affinities.  The reduction over d is split
// over a cluster of router_fused_cluster(T, d) CTAs.
bool router_fused_supported(int E, int G, int K);
int router_fused_cluster(int T, int d);
cudaError_t launch_router_select_fused(const void *x, const void *e_split, const float *off,
                                       const float *bias, int T, int d, int E, int G, int K,
                                       int M, int affinity, float *scores, int32_t *topk_idx,
                                       float *topk_w, int32_t *status, int64_t timeout_ns,
                                       cudaStream_t st);

// route_variants.cu: the hash router (token ids -> K experts in M groups,
// gates 1/K; token_ids NULL = row index) and the per-expert bias update.
cudaError_t launch_hash_route(const int64_t *token_ids, int T, int E, int G, int K, int M,
                              int32_t *topk_idx, float *topk_w, cudaStream_t st);
cudaError_t launch_bias_update(const int32_t *counts, int E, int T, int K, float gamma,
                               float *bias, cudaStream_t st);
// balance.cu: the balance loss and the router's gradient.  Tokens are cut into
// tiles of balance_tile(T, n_seq): two tiles per SM for long batches, and at least 32
// tokens (two or four per lane group of a block) for short ones; up to 1024 tokens
// make BAL_CLUSTER such tiles at most, the blocks of one cluster.  A block takes the
// sequences of its tile one after the other, some 1.5 us each: where they average half
// a tile or less, a tile is one average sequence, down to 8 tokens (1000 x 256 with 32,
// 128 and 512 sequences 13.8, 46 and 184 us without, 9.0, 9.7 and 18.5 with; twice the
// average 11.9, 12.2, 29.7) and to T / 2048, at most 2304 tiles (a long sequence among short
// ones is joined by one block).  part and part_n ([tiles, 2, E] each) hold the tiles'
// shares of the sequences that cross them.
constexpr int BAL_CLUSTER = 8;
inline int balance_tile(int T, int n_seq) {
    const int tiles = T <= 1024 ? BAL_CLUSTER : 2 * 148;
    const int c = std::max(32, (int)(((int64_t)T + tiles - 1) / tiles));
    const int average = std::max({8, T / std::max(1, n_seq), T / 2048});
    return 2 * average <= c ? average : c;
}
cudaError_t launch_balance_loss(const float *scores, const int32_t *topk_idx,
                                const int32_t *offsets, int n_seq, float alpha, int T, int E,
                                int K, int32_t *counts, float *prob, float *loss, float *part,
                                int32_t *part_n, int32_t *status, cudaStream_t st);
cudaError_t launch_route_backward(const float *scores, const int32_t *topk_idx,
                                  const float *d_topk_w, const int32_t *offsets, int n_seq,
                                  const int32_t *counts, const float *d_loss, float alpha, int T,
                                  int E, int K, bool softplus, float *d_logits, int32_t *status,
                                  cudaStream_t st);

// combine.cu: gradients of the combine with respect to y_perm and the gates
cudaError_t launch_combine_backward(const void *d_out, const void *y_perm,
                                    const int32_t *inv_perm, const float *topk_w, int T, int d,
                                    int K, int64_t n_rows, void *d_y_perm, float *d_topk_w,
                                    cudaStream_t st);

// quant_int8.cu: rows to int8 codes and one fp32 scale each (s = amax / 127,
// q = rint(x / s)).  bf16 rows of `cols` values, or those of two fp32 matrices; rows that run over n_mat
// matrices [n_mat, rows, cols] with one scale for all of them; and the dispatch,
// codes and scale of token t into the rows inv_perm[t][.] of x_perm_q (and, with
// x_q, once in token order).
cudaError_t launch_quantize_rows_bf16(const void *x, int64_t rows, int cols, int8_t *q,
                                      float *scale, cudaStream_t st);
cudaError_t launch_quantize_rows_f32(const float *x, int64_t rows, int cols, int8_t *q,
                                     float *scale, const float *x2, int64_t rows2, int cols2,
                                     int8_t *q2, float *scale2, cudaStream_t st);
cudaError_t launch_quantize_joint_bf16(const void *x, int n_mat, int64_t rows, int cols,
                                       int8_t *q, float *scale, cudaStream_t st);
// The dispatch with int8 rows; one kernel for batches of one dispatch block, which then
// writes offsets, else the plan of dispatch.cu and the gather behind it.  (256 tokens of 2048
// over 256 experts, one kernel and three: K = 16 8.7 and 23.9 us, K = 32 17.7 and 45.6.)
inline bool dispatch_int8_in_one(int T) { return T > 0 && T <= DISPATCH_BLOCK; }
cudaError_t launch_dispatch_int8(const void *x, const int32_t *topk_idx, int T, int d, int E, int G,
                                 int K, int32_t *counts, int32_t *offsets, int32_t *send,
                                 int32_t *send_tok, int32_t *perm_token, int32_t *inv_perm,
                                 int8_t *x_perm_q, float *x_scale, int8_t *x_q, float *x_q_scale,
                                 const DispatchWs &ws, int32_t *status, cudaStream_t st);

// gemm_int8.cu: the expert FFN on int8 codes (see moe_expert_ffn_int8)
struct FfnInt8Args {
    int T, d, E, K, d_ff, n_shared, d_ff_shared;
    const int8_t *x_perm_q;  // [T*K, d]
    const float *x_scale;    // [T*K]
    const int32_t *offsets;
    moe_int8_weights w;
    float *h;                // [T*K, d_ff] scratch, fp32
    int8_t *h_q;             // [T*K, d_ff] scratch
    float *h_scale;          // [T*K]
    void *y_perm;            // [T*K, d] bf16
    const int8_t *x_q;       // [T, d] the shared experts' input
    const float *x_q_scale;  // [T]
    float *h_shared;         // [T, n_shared * d_ff_shared] scratch
    int8_t *h_shared_q;
    float *h_shared_scale;
    void *y_shared;          // [T, d] bf16
    // the kernel before this call's first (and all before it) has ended when that kernel's
    // blocks run: offsets and weights may be read before what it writes is there
    bool after_quantize;
    int32_t *status;
    int64_t timeout_ns;
};
cudaError_t launch_expert_ffn_int8(const FfnInt8Args &a, cudaStream_t st);

cudaError_t launch_bounded_wait_selftest(int64_t timeout_ns, int32_t *status, cudaStream_t st);

}  // namespace moe
