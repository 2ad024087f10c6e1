// balance.cu -- the router's training side: the sequence-wise balance loss with
// its per-expert counts, and the gradient of that loss and of the gates with
// respect to the router's logits.
//
// Loss of sequence s, tokens t in [o_s, o_(s+1)), N_s = o_(s+1) - o_s:
//   p_(t,i) = s_(t,i) / S_t,  S_t = sum_i s_(t,i)        (p = 0 where S_t = 0)
//   c_(s,i) = number of copies (t, j) with topk_idx[t][j] = i
//   P_(s,i) = 1/N_s sum_t p_(t,i)
//   L_s     = alpha sum_i (E / (K N_s)) c_(s,i) P_(s,i)
// Gradient (the counts are constants), with g_s = dL/dL_s alpha E / (K N_s^2),
// dw the gradient of the gates w_j = s_j / Z, Z the sum of the chosen s_j:
//   ds_(t,i) = g_s (c_i - sum_k c_k p_(t,k)) / S_t
//              + [i chosen as slot j] (dw_j - sum_k dw_k w_k) / Z
//   dL_(t,i) = ds_(t,i) * s (1 - s)               (sigmoid)
//              ds_(t,i) * (1 - e^(-s^2)) / (2 s)  (sqrt(softplus): sigmoid(L) / 2s)
// computed with s taken out of the slope, s / S = p and s_j / Z = w_j, so that
// affinities near the smallest floats neither overflow nor lose digits:
//   dL_(t,i) = r(s) (g_s (c_i - sum_k c_k p_k) p_i + [chosen] (dw_j - sum_k dw_k w_k) w_j)
//   r(s) = 1 - s, or (1 - e^(-s^2)) / (2 s^2) (1/2 at s = 0)
// Both are one pass over the affinities and bound by HBM for long batches, by
// launch latency for short ones.
//
// A token's row is held by a group of lanes (16, or 32 from 512 experts), four
// consecutive experts per 16-byte load, so that its sums are 4 or 5 shuffles.
// The loss keeps its running sums of p in registers: a block owns a tile of
// consecutive tokens and closes a sequence inside it by a reduction in a fixed
// order; a sequence that crosses tiles leaves one partial row per tile, which a
// second kernel adds in tile order.  No float atomics: equal inputs give equal
// bits.
#include "kernels.h"

namespace moe {
namespace {

constexpr int BAL_THREADS = 512;
constexpr int BAL_WARPS = BAL_THREADS / 32;
constexpr int BAL_CLUSTER = 8;         // blocks that share one crossing sequence
constexpr int BAL_JOIN_THREADS = 256;

// Lanes of a token's group and values a lane loads at once.
template <int GROUP, int VEC, int N>
struct Row {
    static constexpr int kGroup = GROUP, kVec = VEC, kN = N;
    static constexpr int kGroups = BAL_THREADS / GROUP;
    // first of the VEC experts of this lane's q-th load
    static __device__ __forceinline__ int expert(int lane, int q) {
        return (q * GROUP + lane) * VEC;
    }
    static __device__ __forceinline__ void load(const float *row, int lane, int E,
                                                float (&v)[N * VEC]) {
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int i = expert(lane, q);
            if constexpr (VEC == 4) {
                float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < E) w = __ldg(reinterpret_cast<const float4 *>(row + i));
                v[4 * q] = w.x; v[4 * q + 1] = w.y; v[4 * q + 2] = w.z; v[4 * q + 3] = w.w;
            } else {
                v[q] = i < E ? __ldg(row + i) : 0.f;
            }
        }
    }
    // The reciprocal of the group's sum of v, 0 for a sum of 0.  A tiny row is
    // first scaled by a power of two (*down undoes it), or 1 / sum would overflow.
    static __device__ __forceinline__ float inverse_sum(float (&v)[N * VEC], float *down) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < N * VEC; ++q) s += v[q];
        s = sum(s);
        *down = 1.0f;
        if (fabsf(s) < 0x1p-60f) {
            *down = 0x1p-80f;
            s *= 0x1p80f;
#pragma unroll
            for (int q = 0; q < N * VEC; ++q) v[q] *= 0x1p80f;
        }
        return s != 0.f ? 1.0f / s : 0.f;
    }
    static __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int o = GROUP / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return v;
    }
};

// The sequence of token t: the last s with offsets[s] <= t, or -1; n_seq means
// behind the last one.  Whatever the values, offsets[s] <= t < offsets[s + 1].
__device__ __forceinline__ int find_sequence(const int32_t *offsets, int n_seq, int t) {
    int lo = -1, hi = n_seq + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(offsets + mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Offsets of a sequence, kept inside the batch.  offsets == nullptr: one
// sequence of all T tokens.
__device__ __forceinline__ void sequence_range(const int32_t *offsets, int s, int T, int *lo,
                                               int *hi) {
    *lo = offsets ? max(0, min(T, __ldg(offsets + s))) : 0;
    *hi = offsets ? max(0, min(T, __ldg(offsets + s + 1))) : T;
}

// Sum over the block in a fixed order; every thread gets it.
__device__ __forceinline__ double block_sum(double v, double *scratch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    double total = 0.0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) total += scratch[w];
    return total;
}

struct BalanceArgs {
    const float *scores;
    const int32_t *topk_idx;
    const int32_t *offsets;  // or nullptr
    int n_seq, T, E, K, tile;
    float alpha;
    int32_t *counts;
    float *prob, *loss;
    float *part;       // [tiles, 2, E]: sums of p of the sequence that comes in (0), goes out (1)
    int32_t *part_n;   // [tiles, 2, E]: its counts
    int32_t *status;
};

// One tile of tokens per block.
template <class R>
__global__ void __launch_bounds__(BAL_THREADS, R::kN * R::kVec <= 16 ? 2 : 1)
balance_tile_kernel(const BalanceArgs a) {
    extern __shared__ float red[];             // [BAL_WARPS, E]
    int *hist = reinterpret_cast<int *>(red + BAL_WARPS * a.E);  // [E]
    __shared__ double scratch[BAL_WARPS];
    constexpr int NV = R::kN * R::kVec;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int glane = lane % R::kGroup, group = threadIdx.x / R::kGroup;
    const int lo_tile = blockIdx.x * a.tile;
    const int hi_tile = (int)min((int64_t)a.T, (int64_t)lo_tile + a.tile);

    // empty sequences, and offsets that are not monotone or leave the batch
    for (int s = blockIdx.x * BAL_WARPS + warp; s < a.n_seq; s += gridDim.x * BAL_WARPS) {
        int lo = 0, hi = a.T;
        if (a.offsets) {
            lo = __ldg(a.offsets + s), hi = __ldg(a.offsets + s + 1);
            if (lane == 0 && (lo < 0 || hi < lo || hi > a.T))
                record_status(a.status, MOE_ERR_DEVICE_FAULT);
            sequence_range(a.offsets, s, a.T, &lo, &hi);
        }
        if (hi > lo) continue;
        for (int i = lane; i < a.E; i += 32) {
            a.counts[(size_t)s * a.E + i] = 0;
            a.prob[(size_t)s * a.E + i] = 0.f;
        }
        if (lane == 0) a.loss[s] = 0.f;
    }

    for (int t = lo_tile; t < hi_tile;) {
        int s = 0, s_lo = 0, s_hi = a.T;
        if (a.offsets) {
            s = find_sequence(a.offsets, a.n_seq, t);
            if (s >= a.n_seq) break;  // padding behind the last sequence
            if (s < 0) {              // ... or in front of the first
                t = max(t + 1, __ldg(a.offsets));
                continue;
            }
            sequence_range(a.offsets, s, a.T, &s_lo, &s_hi);
        }
        const int end = min(hi_tile, s_hi);
        for (int i = threadIdx.x; i < a.E; i += BAL_THREADS) hist[i] = 0;
        __syncthreads();
        for (int64_t c = (int64_t)t * a.K + threadIdx.x; c < (int64_t)end * a.K;
             c += BAL_THREADS) {
            const int i = __ldg(a.topk_idx + c);
            if (i >= 0 && i < a.E) atomicAdd(hist + i, 1);
            else record_status(a.status, MOE_ERR_DEVICE_FAULT);
        }
        float acc[NV];
#pragma unroll
        for (int q = 0; q < NV; ++q) acc[q] = 0.f;
        // whole warps stay in the loop: the sums are shuffles
        for (uint32_t u = t; u < (uint32_t)end; u += R::kGroups) {
            const uint32_t tok = u + group;
            float v[NV];
            if (tok < (uint32_t)end) {
                R::load(a.scores + (size_t)tok * a.E, glane, a.E, v);
            } else {
#pragma unroll
                for (int q = 0; q < NV; ++q) v[q] = 0.f;
            }
            float down;
            const float inv = R::inverse_sum(v, &down);
#pragma unroll
            for (int q = 0; q < NV; ++q) acc[q] = fmaf(v[q], inv, acc[q]);
        }
        if constexpr (R::kGroup == 16) {
#pragma unroll
            for (int q = 0; q < NV; ++q) acc[q] += __shfl_xor_sync(0xFFFFFFFFu, acc[q], 16);
        }
        if (lane < R::kGroup) {
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int i = R::expert(glane, q / R::kVec) + q % R::kVec;
                if (i < a.E) red[warp * a.E + i] = acc[q];
            }
        }
        __syncthreads();
        const bool whole = s_lo >= lo_tile && s_hi <= hi_tile;
        const size_t row = whole ? (size_t)s * a.E
                                 : ((size_t)blockIdx.x * 2 + (s_lo >= lo_tile)) * a.E;
        float *const out_p = whole ? a.prob : a.part;
        int32_t *const out_n = whole ? a.counts : a.part_n;
        const int len = s_hi - s_lo;
        double dot = 0.0;
        for (int i = threadIdx.x; i < a.E; i += BAL_THREADS) {
            float p = 0.f;
#pragma unroll
            for (int w = 0; w < BAL_WARPS; ++w) p += red[w * a.E + i];
            const int n = hist[i];
            out_n[row + i] = n;
            out_p[row + i] = whole ? p / (float)len : p;
            dot += (double)n * p;
        }
        if (whole) {
            dot = block_sum(dot, scratch);
            if (threadIdx.x == 0)
                a.loss[s] = (float)((double)a.alpha * a.E / ((double)a.K * len * len) * dot);
        }
        __syncthreads();  // red, hist and scratch are free again
        t = end;
    }
}

// The sequences that cross tiles: BAL_CLUSTER blocks for each tile but the
// last take the sequence that starts in it and goes on, if there is one, each
// for a share of the experts.
__global__ void __cluster_dims__(BAL_CLUSTER, 1, 1) __launch_bounds__(BAL_JOIN_THREADS)
balance_join_kernel(const BalanceArgs a) {
    constexpr int COLS = 32, PARTS = BAL_JOIN_THREADS / COLS;
    __shared__ float sp[PARTS][COLS];
    __shared__ int sn[PARTS][COLS];
    __shared__ double scratch[BAL_JOIN_THREADS / 32];
    __shared__ double shared_dot[BAL_CLUSTER];
    const int b = blockIdx.x / BAL_CLUSTER, rank = blockIdx.x % BAL_CLUSTER;
    const int lo_tile = b * a.tile, hi_tile = lo_tile + a.tile;
    int s = 0, s_lo = 0, s_hi = a.T;
    if (a.offsets) {
        s = find_sequence(a.offsets, a.n_seq, hi_tile - 1);
        if (s < 0 || s >= a.n_seq) return;  // the whole cluster leaves
        sequence_range(a.offsets, s, a.T, &s_lo, &s_hi);
    }
    if (s_lo < lo_tile || s_hi <= hi_tile) return;
    cluster_sync_all();  // every block runs before one writes to another's shared memory
    const int last = (s_hi - 1) / a.tile;
    const int len = s_hi - s_lo;
    const int col = threadIdx.x % COLS, part = threadIdx.x / COLS;
    double dot = 0.0;
    for (int i0 = rank * COLS; i0 < a.E; i0 += BAL_CLUSTER * COLS) {
        const int i = i0 + col;
        float p = 0.f;
        int n = 0;
        if (i < a.E) {
#pragma unroll 8
            for (int k = b + part; k <= last; k += PARTS) {
                const size_t at = ((size_t)k * 2 + (k == b)) * a.E + i;
                p += a.part[at];
                n += a.part_n[at];
            }
        }
        sp[part][col] = p;
        sn[part][col] = n;
        __syncthreads();
        if (part == 0 && i < a.E) {
            p = 0.f, n = 0;
#pragma unroll
            for (int k = 0; k < PARTS; ++k) p += sp[k][col], n += sn[k][col];
            a.counts[(size_t)s * a.E + i] = n;
            a.prob[(size_t)s * a.E + i] = p / (float)len;
            dot += (double)n * p;
        }
        __syncthreads();
    }
    dot = block_sum(dot, scratch);
    if (threadIdx.x == 0) {  // rank 0 adds the shares in rank order
        const uint32_t to = mapa_shared(smem_u32(&shared_dot[rank]), 0);
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(dot) : "memory");
    }
    cluster_sync_all();
    if (rank == 0 && threadIdx.x == 0) {
        double total = 0.0;
        for (int r = 0; r < BAL_CLUSTER; ++r) total += shared_dot[r];
        a.loss[s] = (float)((double)a.alpha * a.E / ((double)a.K * len * len) * total);
    }
}

struct RouteGradArgs {
    const float *scores;
    const int32_t *topk_idx;
    const float *d_topk_w;   // or nullptr
    const int32_t *offsets;  // or nullptr
    int n_seq;
    const int32_t *counts;
    const float *d_loss;     // or nullptr: no balance loss
    float alpha;
    int T, E, K, tile, softplus;
    float *d_logits;
    int32_t *status;
};

template <class R>
__global__ void __launch_bounds__(BAL_THREADS, R::kN * R::kVec <= 16 ? 2 : 1)
route_backward_kernel(const RouteGradArgs a) {
    extern __shared__ float gates[];  // [groups, E]: the gates' part of a token's row
    constexpr int NV = R::kN * R::kVec;
    const int lane = threadIdx.x & 31, glane = lane % R::kGroup;
    const int group = threadIdx.x / R::kGroup;
    float *mine = gates + group * a.E;
    const bool gate = a.d_topk_w != nullptr, balance = a.d_loss != nullptr;
    if (gate) {
        for (int i = threadIdx.x; i < R::kGroups * a.E; i += BAL_THREADS) gates[i] = 0.f;
        __syncthreads();
    }
    float pull[NV];  // g_s (c_i - K N_s / E) of the current sequence
#pragma unroll
    for (int q = 0; q < NV; ++q) pull[q] = 0.f;
    int cur_lo = 0, cur_hi = 0;  // tokens for which `pull` holds
    const int lo_tile = blockIdx.x * a.tile;
    const int hi_tile = (int)min((int64_t)a.T, (int64_t)lo_tile + a.tile);
    bool counted = false;        // ... and whether they lie in a sequence
    for (uint32_t u = lo_tile; u < (uint32_t)hi_tile; u += R::kGroups) {
        const bool in = u + group < (uint32_t)hi_tile;
        const int tok = in ? (int)(u + group) : lo_tile;
        float v[NV];
        if (in) {
            R::load(a.scores + (size_t)tok * a.E, glane, a.E, v);
        } else {
#pragma unroll
            for (int q = 0; q < NV; ++q) v[q] = 0.f;
        }
        if (balance && in && (tok < cur_lo || tok >= cur_hi)) {
            int s = 0;
            cur_lo = 0, cur_hi = a.T;
            if (a.offsets) {
                s = find_sequence(a.offsets, a.n_seq, tok);
                cur_lo = s < 0 ? 0 : __ldg(a.offsets + s);
                cur_hi = s >= a.n_seq ? a.T : __ldg(a.offsets + s + 1);
            }
            counted = s >= 0 && s < a.n_seq;
            const int s_lo = max(0, cur_lo), len = min(a.T, cur_hi) - s_lo;
            // sum_i p_i = 1, so any constant taken off the counts leaves the
            // gradient as it is; their mean takes the cancellation out of it
            const double g = counted ? (double)__ldg(a.d_loss + s) * a.alpha /
                                           ((double)a.K * len * len)
                                     : 0.0;
            const int64_t mean = (int64_t)a.K * len;
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int i = R::expert(glane, q / R::kVec) + q % R::kVec;
                pull[q] = 0.f;
                if (counted && i < a.E)
                    pull[q] = (float)(g * (double)((int64_t)__ldg(a.counts + (size_t)s * a.E + i) *
                                                       a.E - mean));
            }
        }
        float down = 1.0f, inv = 0.f, dot = 0.f;
        if (balance) {
            inv = R::inverse_sum(v, &down);
#pragma unroll
            for (int q = 0; q < NV; ++q) dot = fmaf(pull[q], v[q], dot);
            dot = R::sum(dot) * inv;
        }
        if (gate) {
            float z = 0.f, wsum = 0.f;
            float sj[32 / R::kGroup], dw[32 / R::kGroup];
            int idx[32 / R::kGroup];
#pragma unroll
            for (int h = 0; h < 32 / R::kGroup; ++h) {
                const int j = h * R::kGroup + glane;
                idx[h] = -1;
                sj[h] = dw[h] = 0.f;
                if (in && j < a.K) {
                    idx[h] = __ldg(a.topk_idx + (size_t)tok * a.K + j);
                    if (idx[h] < 0 || idx[h] >= a.E) {
                        record_status(a.status, MOE_ERR_DEVICE_FAULT);
                        idx[h] = -1;
                    } else {
                        sj[h] = __ldg(a.scores + (size_t)tok * a.E + idx[h]);
                        dw[h] = __ldg(a.d_topk_w + (size_t)tok * a.K + j);
                    }
                }
                z += sj[h];
            }
            z = R::sum(z);
            float w[32 / R::kGroup];
#pragma unroll
            for (int h = 0; h < 32 / R::kGroup; ++h) {
                w[h] = z != 0.f ? __fdiv_rn(sj[h], z) : 0.f;
                wsum = fmaf(dw[h], w[h], wsum);
            }
            wsum = R::sum(wsum);
            // added, not stored: an expert listed twice has two gates
#pragma unroll
            for (int h = 0; h < 32 / R::kGroup; ++h)
                if (idx[h] >= 0) atomicAdd(mine + idx[h], (dw[h] - wsum) * w[h]);
            __syncwarp();
        }
        float o[NV];
#pragma unroll
        for (int q = 0; q < R::kN; ++q) {
            const int i = R::expert(glane, q);
            float gt[R::kVec];
#pragma unroll
            for (int k = 0; k < R::kVec; ++k) gt[k] = 0.f;
            if (gate && i < a.E) {
                if constexpr (R::kVec == 4) {
                    float4 *at = reinterpret_cast<float4 *>(mine + i);
                    const float4 g4 = *at;
                    gt[0] = g4.x; gt[1] = g4.y; gt[2] = g4.z; gt[3] = g4.w;
                    *at = make_float4(0.f, 0.f, 0.f, 0.f);
                } else {
                    gt[0] = mine[i];
                    mine[i] = 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < R::kVec; ++k) {
                const int n = q * R::kVec + k;
                const float s = v[n] * down, s2 = s * s;
                float d = gt[k];
                if (balance && counted) d = fmaf(pull[n] - dot, v[n] * inv, d);
                const float r = a.softplus ? (s2 > 0x1p-100f ? -expm1f(-s2) / (2.0f * s2) : 0.5f)
                                           : 1.0f - s;
                o[n] = d != 0.f ? d * r : 0.f;  // no pull, no gradient, whatever s holds
            }
            if (in && i < a.E) {
                float *dst = a.d_logits + (size_t)tok * a.E + i;
                if constexpr (R::kVec == 4)
                    *reinterpret_cast<float4 *>(dst) =
                        make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                else
                    *dst = o[q];
            }
        }
        if (gate) __syncwarp();  // the zeroed gates are seen before the next token's
    }
}

// Calls f with the row layout for E experts.
template <class F>
cudaError_t with_row(int E, F f) {
    if (E % 4 == 0) {
        if (E <= 64) return f(Row<16, 4, 1>{});
        if (E <= 128) return f(Row<16, 4, 2>{});
        if (E <= 256) return f(Row<16, 4, 4>{});
        if (E <= 512) return f(Row<32, 4, 4>{});
        return f(Row<32, 4, 8>{});
    }
    if (E <= 64) return f(Row<32, 1, 2>{});
    if (E <= 256) return f(Row<32, 1, 8>{});
    return f(Row<32, 1, 32>{});
}

template <class Kern>
cudaError_t allow_smem(Kern kern, size_t bytes) {
    if (bytes <= 48 * 1024) return cudaSuccess;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace

cudaError_t launch_balance_loss(const float *scores, const int32_t *topk_idx,
                                const int32_t *offsets, int n_seq, float alpha, int T, int E,
                                int K, int32_t *counts, float *prob, float *loss, float *part,
                                int32_t *part_n, int32_t *status, cudaStream_t st) {
    if (n_seq == 0) return cudaSuccess;
    BalanceArgs a{scores, topk_idx, offsets, n_seq, T, E, K, balance_tile(T), alpha,
                  counts, prob, loss, part, part_n, status};
    const int tiles = T > 0 ? (T + a.tile - 1) / a.tile : 1;
    const size_t smem = sizeof(float) * (size_t)E * (BAL_WARPS + 1);
    cudaError_t err = with_row(E, [&](auto row) {
        auto kern = balance_tile_kernel<decltype(row)>;
        const cudaError_t e = allow_smem(kern, smem);
        if (e != cudaSuccess) return e;
        kern<<<tiles, BAL_THREADS, smem, st>>>(a);
        count_launch();
        return cudaGetLastError();
    });
    if (err != cudaSuccess || tiles == 1) return err;
    balance_join_kernel<<<(tiles - 1) * BAL_CLUSTER, BAL_JOIN_THREADS, 0, st>>>(a);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_route_backward(const float *scores, const int32_t *topk_idx,
                                  const float *d_topk_w, const int32_t *offsets, int n_seq,
                                  const int32_t *counts, const float *d_loss, float alpha, int T,
                                  int E, int K, bool softplus, float *d_logits, int32_t *status,
                                  cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    RouteGradArgs a{scores, topk_idx, d_topk_w, offsets, n_seq, counts, d_loss, alpha,
                    T, E, K, 0, softplus, d_logits, status};
    return with_row(E, [&](auto row) {
        using R = decltype(row);
        auto kern = route_backward_kernel<R>;
        const size_t smem = d_topk_w ? sizeof(float) * (size_t)E * R::kGroups : 0;
        const cudaError_t e = allow_smem(kern, smem);
        if (e != cudaSuccess) return e;
        a.tile = balance_tile(T);
        kern<<<(T + a.tile - 1) / a.tile, BAL_THREADS, smem, st>>>(a);
        count_launch();
        return cudaGetLastError();
    });
}

}  // namespace moe
