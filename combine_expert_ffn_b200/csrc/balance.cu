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
// Both are one pass over the affinities.  The loss of 262144 tokens x 256 experts
// takes 49 us and 2 for the sequences that cross tiles, 5.6 TB/s of its 277 MB:
// HBM bounds it.  The gradient of 131072 x 256 takes 51 us, 5.2 TB/s of 268 MB; of
// 196601 x 64 with sqrt(softplus) 36 us, 2.8 TB/s, where the arithmetic of a value
// (some 25 instructions) bounds it.  Short batches are bound by launch latency.
//
// A token's row is held by a group of 8, 16 or 32 lanes (by the number of
// experts), four consecutive experts per 16-byte load, so that a warp works on up
// to four tokens and their sums are 3 to 5 shuffles; the next row is loaded while
// the current one is worked on.
// The loss keeps its running sums of p in registers: a block owns a tile of
// consecutive tokens and closes a sequence inside it by a reduction in a fixed
// order; a sequence that crosses tiles leaves one partial row per tile, which a
// second kernel adds in tile order.  No float atomics: equal inputs give equal
// bits.
#include <climits>

#include "kernels.h"

namespace moe {
namespace {

constexpr int BAL_THREADS = 512;
constexpr int BAL_WARPS = BAL_THREADS / 32;
constexpr int BAL_JOIN_THREADS = 1024;
constexpr int GRAD_THREADS = 256;

// 1 / s within 1 ulp, 0 for 0 (|s| at least 2^-60: no overflow, no denormal).
__device__ __forceinline__ float reciprocal(float s) {
    return s != 0.f ? __fdividef(1.0f, s) : 0.f;
}

// Lanes of a token's group and values a lane loads at once.
template <int GROUP, int VEC, int N>
struct Row {
    static constexpr int kGroup = GROUP, kVec = VEC, kN = N, kValues = N * VEC;
    static constexpr int kMaxE = GROUP * VEC * N;  // experts that fit
    // first of the VEC experts of this lane's q-th load
    static __device__ __forceinline__ int expert(int lane, int q) {
        return (q * GROUP + lane) * VEC;
    }
    // row `tok` of scores, zeros from `end` on
    static __device__ __forceinline__ void load(const float *scores, uint32_t tok, uint32_t end,
                                                int lane, int E, float (&v)[N * VEC]) {
        const float *row = scores + (size_t)tok * E;
        const bool in = tok < end;
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int i = expert(lane, q);
            if constexpr (VEC == 4) {
                float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
                if (in && i < E) w = *reinterpret_cast<const float4 *>(row + i);
                v[4 * q] = w.x; v[4 * q + 1] = w.y; v[4 * q + 2] = w.z; v[4 * q + 3] = w.w;
            } else {
                v[q] = in && i < E ? row[i] : 0.f;
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
        return reciprocal(s);
    }
    static __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int o = GROUP / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return v;
    }
    // (a quarter warp's reduction by redux: 196601 x 64 38.4 us for 36.4 with shuffles; a
    // whole warp's: 16384 x 512 15.2 for 15.7)
    static __device__ __forceinline__ uint32_t largest(uint32_t v) {
        if constexpr (GROUP == 32) {
            return __reduce_max_sync(0xFFFFFFFFu, v);
        } else {
#pragma unroll
            for (int o = GROUP / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
            return v;
        }
    }
};

// The sequence of token t: the last s with offsets[s] <= t, or -1; n_seq means
// behind the last one.  Whatever the values, offsets[s] <= t < offsets[s + 1].
__device__ __forceinline__ int find_sequence(const int32_t *offsets, int n_seq, int t) {
    int lo = -1, hi = n_seq + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (offsets[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}
// The same by a whole warp, 32 probes at a time: the search is a chain of loads.
__device__ __forceinline__ int warp_find_sequence(const int32_t *offsets, int n_seq, int t) {
    const int lane = threadIdx.x & 31;
    int lo = -1, hi = n_seq + 1;
    while (hi - lo > 1) {
        const int step = (int)(((int64_t)hi - lo + 32) / 33);
        const int64_t at = lo + (int64_t)(lane + 1) * step;
        const bool le = at < hi && offsets[at] <= t;
        const uint32_t no = ~__ballot_sync(0xFFFFFFFFu, le);
        const int yes = no ? __ffs(no) - 1 : 32;  // probes up to the first that is behind t
        const int64_t behind = lo + (int64_t)(yes + 1) * step;
        lo += yes * step;
        hi = behind < hi ? (int)behind : hi;
    }
    return lo;
}

// Offsets of a sequence, kept inside the batch.  offsets == nullptr: one
// sequence of all T tokens.
__device__ __forceinline__ void sequence_range(const int32_t *offsets, int s, int T, int *lo,
                                               int *hi) {
    *lo = offsets ? max(0, min(T, offsets[s])) : 0;
    *hi = offsets ? max(0, min(T, offsets[s + 1])) : T;
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

// The sequence that starts in tile b and goes on, if there is one, by one block of
// THREADS threads, which lie over the experts and, where these are fewer, over equal
// shares of the tiles.  `ready` waits for the tiles' shares; every block calls it.
template <int THREADS, class Ready>
__device__ __forceinline__ void join_sequence(const BalanceArgs &a, int b, Ready ready) {
    __shared__ float sp[THREADS];
    __shared__ int sn[THREADS];
    __shared__ double scratch[THREADS / 32];
    const int lo_tile = b * a.tile;
    const int64_t hi_tile = (int64_t)lo_tile + a.tile;
    int s = 0, s_lo = 0, s_hi = a.T;
    if (a.offsets && hi_tile < a.T) {
        s = warp_find_sequence(a.offsets, a.n_seq, (int)hi_tile - 1);
        if (s < 0 || s >= a.n_seq) s_hi = 0;
        else sequence_range(a.offsets, s, a.T, &s_lo, &s_hi);
    }
    ready();
    if (s_lo < lo_tile || s_hi <= hi_tile) return;
    const int last = (s_hi - 1) / a.tile;
    const int len = s_hi - s_lo;
    double dot = 0.0;
    for (int i0 = 0; i0 < a.E; i0 += THREADS) {
        const int cols = min(THREADS, (a.E - i0 + 31) / 32 * 32);
        const int parts = THREADS / cols;
        const int part = threadIdx.x / cols, i = threadIdx.x - part * cols;
        const bool in = i0 + i < a.E && part < parts;
        float p = 0.f;
        int n = 0;
        if (in) {
#pragma unroll 8
            for (int k = b + part; k <= last; k += parts) {
                const size_t at = ((size_t)k * 2 + (k == b)) * a.E + i0 + i;
                p += __ldcg(a.part + at);
                n += __ldcg(a.part_n + at);
            }
        }
        sp[threadIdx.x] = p;
        sn[threadIdx.x] = n;
        __syncthreads();
        if (in && part == 0) {
            for (int k = 1; k < parts; ++k) p += sp[k * cols + i], n += sn[k * cols + i];
            a.counts[(size_t)s * a.E + i0 + i] = n;
            a.prob[(size_t)s * a.E + i0 + i] = p / (float)len;
            dot += (double)n * p;
        }
        __syncthreads();
    }
    dot = block_sum(dot, scratch);
    if (threadIdx.x == 0)
        a.loss[s] = (float)((double)a.alpha * a.E / ((double)a.K * len * len) * dot);
}

// Dynamic shared memory of a tile's block: the warps' sums and the counts.
constexpr size_t balance_smem(int E) { return sizeof(float) * (BAL_WARPS + 1) * (size_t)E; }

// One tile of tokens per block.  CLUSTER: the blocks are one cluster, and join the
// crossing sequences themselves.
template <class R, bool CLUSTER>
__global__ void __launch_bounds__(BAL_THREADS, R::kValues <= 16 ? 2 : 1)
balance_tile_kernel(const BalanceArgs a) {
    extern __shared__ float red[];             // [BAL_WARPS, E]
    int *hist = reinterpret_cast<int *>(red + BAL_WARPS * a.E);  // [E]
    __shared__ double scratch[BAL_WARPS];
    constexpr int NV = R::kValues, GROUPS = BAL_THREADS / R::kGroup;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int glane = lane % R::kGroup, group = threadIdx.x / R::kGroup;
    dependency_wait();
    dependency_release();  // the join's blocks may take their places
    const int lo_tile = blockIdx.x * a.tile;
    const int hi_tile = (int)min((int64_t)a.T, (int64_t)lo_tile + a.tile);

    // empty sequences, and offsets that are not monotone or leave the batch
    for (int s = blockIdx.x * BAL_WARPS + warp; s < a.n_seq; s += gridDim.x * BAL_WARPS) {
        int lo = 0, hi = a.T;
        if (a.offsets) {
            lo = a.offsets[s], hi = a.offsets[s + 1];
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
            s = warp_find_sequence(a.offsets, a.n_seq, t);
            if (s >= a.n_seq) break;  // padding behind the last sequence
            if (s < 0) {              // ... or in front of the first
                t = max(t + 1, a.offsets[0]);
                continue;
            }
            sequence_range(a.offsets, s, a.T, &s_lo, &s_hi);
        }
        const int end = min(hi_tile, s_hi);
        float v[NV];  // the first rows come in beside the ids
        R::load(a.scores, t + group, end, glane, a.E, v);
        for (int i = threadIdx.x; i < a.E; i += BAL_THREADS) hist[i] = 0;
        __syncthreads();
        // ids in batches whose loads are in flight together (one by one they took 6 us of
        // the 58 of 262144 tokens)
        constexpr int BATCH = 8;
        const int64_t last_id = (int64_t)end * a.K;
        for (int64_t c = (int64_t)t * a.K + threadIdx.x; c < last_id; c += BATCH * BAL_THREADS) {
            int id[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                id[k] = c + k * BAL_THREADS < last_id ? a.topk_idx[c + k * BAL_THREADS] : INT_MIN;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                if (id[k] >= 0 && id[k] < a.E) atomicAdd(hist + id[k], 1);
                else if (c + k * BAL_THREADS < last_id) record_status(a.status, MOE_ERR_DEVICE_FAULT);
            }
        }
        float acc[NV];
#pragma unroll
        for (int q = 0; q < NV; ++q) acc[q] = 0.f;
        // whole warps stay in the loop: the sums are shuffles
        for (uint32_t u = t; u < (uint32_t)end; u += GROUPS) {
            float next[NV];
            R::load(a.scores, u + GROUPS + group, end, glane, a.E, next);
            float down;
            const float inv = R::inverse_sum(v, &down);
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                acc[q] = fmaf(v[q], inv, acc[q]);
                v[q] = next[q];
            }
        }
#pragma unroll
        for (int o = R::kGroup; o < 32; o <<= 1)
#pragma unroll
            for (int q = 0; q < NV; ++q) acc[q] += __shfl_xor_sync(0xFFFFFFFFu, acc[q], o);
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
    if constexpr (CLUSTER) join_sequence<BAL_THREADS>(a, blockIdx.x, [] { cluster_sync_all(); });
}

// The crossing sequences of the batches that fill more than one cluster, a block for
// each tile but the last.
__global__ void __launch_bounds__(BAL_JOIN_THREADS)
balance_join_kernel(const BalanceArgs a) {
    // blocks without a sequence wait too: what follows on the stream waits for this
    // kernel alone
    join_sequence<BAL_JOIN_THREADS>(a, blockIdx.x, [] { dependency_wait(); });
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
    int T, E, K, tile;
    float *d_logits;
    int32_t *status;
};

// (1 - e^-x) / (2 x), x = s^2: its Taylor series below 1/4 (the first term left out
// is 2^-24 of it), where the difference would lose digits.
__device__ __forceinline__ float softplus_ratio(float s) {
    const float x = s * s;
    float y = -1.0f / 1440.0f;
    y = fmaf(y, x, 1.0f / 240.0f);
    y = fmaf(y, x, -1.0f / 48.0f);
    y = fmaf(y, x, 1.0f / 12.0f);
    y = fmaf(y, x, -0.25f);
    y = fmaf(y, x, 0.5f);
    return x < 0.25f ? y : __fdividef(0.5f - 0.5f * __expf(-x), x);
}

// Blocks an SM (four cost spills where a lane holds 16 values: 131072 x 256 takes 54 us
// with four, 51 with three; 196601 x 64 with 8 values 35.6 and 37.8).
template <class R>
__host__ __device__ constexpr int grad_blocks() {
    return R::kValues <= 8 ? 4 : R::kValues <= 16 ? 3 : 1;
}

// SLOTS: gates of a lane (1 where a group has a lane for each of a token's K).
template <class R, int SLOTS, bool SOFTPLUS>
__global__ void __launch_bounds__(GRAD_THREADS, grad_blocks<R>())
route_backward_kernel(const RouteGradArgs a) {
    extern __shared__ float gates[];  // [GROUPS, E]: the gates' part of a token's row
    constexpr int NV = R::kValues, GROUPS = GRAD_THREADS / R::kGroup;
    const int lane = threadIdx.x & 31, glane = lane % R::kGroup;
    const int group = threadIdx.x / R::kGroup;
    float *mine = gates + group * a.E;
    const bool gate = a.d_topk_w != nullptr, balance = a.d_loss != nullptr;
    if (gate) {
        for (int i = threadIdx.x; i < GROUPS * a.E; i += GRAD_THREADS) gates[i] = 0.f;
        __syncthreads();
    }
    const int lo_tile = blockIdx.x * a.tile;
    const uint32_t hi_tile = (uint32_t)min((int64_t)a.T, (int64_t)lo_tile + a.tile);
    float pull[NV];  // g_s (c_i - mean c) of the current sequence
#pragma unroll
    for (int q = 0; q < NV; ++q) pull[q] = 0.f;
    int cur_lo = 0, cur_hi = 0;  // tokens for which `pull` holds
    bool counted = false;        // ... and whether they lie in a sequence
    float v[NV], dw[SLOTS];
    int idx[SLOTS];
    auto load_gates = [&](uint32_t tok, int (&i)[SLOTS], float (&d)[SLOTS]) {
#pragma unroll
        for (int h = 0; h < SLOTS; ++h) {
            const int j = h * R::kGroup + glane;
            const bool in = gate && tok < hi_tile && j < a.K;
            i[h] = in ? a.topk_idx[(size_t)tok * a.K + j] : -1;
            d[h] = in ? a.d_topk_w[(size_t)tok * a.K + j] : 0.f;
            if (in && (i[h] < 0 || i[h] >= a.E)) {
                record_status(a.status, MOE_ERR_DEVICE_FAULT);
                i[h] = -1;
                d[h] = 0.f;
            }
        }
    };
    dependency_wait();
    dependency_release();
    R::load(a.scores, lo_tile + group, hi_tile, glane, a.E, v);
    load_gates(lo_tile + group, idx, dw);
    int seq = 0;  // of the warp's first token: found by 32 probes at a time
    if (balance && a.offsets)
        seq = warp_find_sequence(a.offsets, a.n_seq, lo_tile + (int)(threadIdx.x & ~31u) / R::kGroup);
    for (uint32_t u = lo_tile; u < hi_tile; u += GROUPS) {
        const uint32_t tok = u + group;
        const bool in = tok < hi_tile;
        // a sequence begins for this token's group (before the loads below: behind them
        // 131072 x 256 takes 53.4 us for 51.7)
        const bool enters = balance && in && ((int)tok < cur_lo || (int)tok >= cur_hi);
        if (__any_sync(0xFFFFFFFFu, enters)) {
            int s = seq;
            double g = 0.0;
            if (enters) {
                for (int look = 0; look < 2; ++look) {  // the sequence at hand, else the search
                    if (look) s = find_sequence(a.offsets, a.n_seq, (int)tok);
                    cur_lo = !a.offsets || s < 0 ? 0 : a.offsets[s];
                    cur_hi = !a.offsets || s >= a.n_seq ? a.T : a.offsets[s + 1];
                    if (!a.offsets || ((int)tok >= cur_lo && (int)tok < cur_hi)) break;
                }
                counted = s >= 0 && s < a.n_seq;
                const int s_lo = max(0, cur_lo), len = min(a.T, cur_hi) - s_lo;
                if (counted) g = (double)a.d_loss[s] * a.alpha / ((double)a.K * len * len);
            }
            // sum_i p_i = 1, so any constant taken off the counts leaves the gradient as it
            // is; their mean takes the cancellation out of it.  It is that of the counts given:
            // K N_s / E for this batch's own, but not for sums over ranks.
            int64_t total = 0;
            if (enters) {
#pragma unroll
                for (int q = 0; q < NV; ++q) {  // the counts, in pull's registers: others spill
                    const int i = R::expert(glane, q / R::kVec) + q % R::kVec;
                    const int n = counted && i < a.E ? a.counts[(size_t)s * a.E + i] : 0;
                    total += n;
                    pull[q] = __int_as_float(n);
                }
            }
#pragma unroll
            for (int o = R::kGroup / 2; o > 0; o >>= 1)
                total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
            if (enters) {
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    const int i = R::expert(glane, q / R::kVec) + q % R::kVec;
                    const int64_t off = (int64_t)__float_as_int(pull[q]) * a.E - total;
                    pull[q] = i < a.E ? (float)(g * (double)off) : 0.f;
                }
            }
        }

        // this token's chosen affinities (its row is in L1) and the next token's loads
        float sj[SLOTS], next[NV], next_dw[SLOTS];
        int next_idx[SLOTS];
#pragma unroll
        for (int h = 0; h < SLOTS; ++h)
            sj[h] = idx[h] >= 0 ? a.scores[(size_t)tok * a.E + idx[h]] : 0.f;
        R::load(a.scores, tok + GROUPS, hi_tile, glane, a.E, next);
        load_gates(tok + GROUPS, next_idx, next_dw);

        // Without a sequence `pull` and so the sums are 0: what is left to keep out of
        // the row are values that 0 times is not 0.
        if (!counted) {
#pragma unroll
            for (int q = 0; q < NV; ++q) v[q] = fabsf(v[q]) < INFINITY ? v[q] : 0.f;
        }
        // The gates' gradients less that of the largest gate: their mean is taken off them
        // below, so it makes no difference but that equal ones (or a single one) cancel
        // exactly.  The largest gate's weight is at least 1 / K, so what is taken off is at
        // most K times the mean size of the gradients; that of a small gate, which hardly enters
        // the mean, could be any size and round the others' digits away.  The slot comes with the
        // affinity in one key (its last five bits, 2^-18 of it; the lowest of equal ones).
        if (gate) {
            uint32_t top = 0;
#pragma unroll
            for (int h = 0; h < SLOTS; ++h)
                top = max(top, (__float_as_uint(sj[h]) | 31u) - (uint32_t)(h * R::kGroup + glane));
            const int from = (int)(~R::largest(top) & 31u);
            float dwt = dw[0];
#pragma unroll
            for (int h = 1; h < SLOTS; ++h)
                if (from / R::kGroup == h) dwt = dw[h];
            dwt = __shfl_sync(0xFFFFFFFFu, dwt, lane - glane + from % R::kGroup);
#pragma unroll
            for (int h = 0; h < SLOTS; ++h) dw[h] -= dwt;
        }
        // the four sums of a token side by side: S, pull . s, Z, dw . s_chosen
        float sum = 0.f, dot = 0.f, z = 0.f, zdw = 0.f, down = 1.0f;
        auto sums = [&] {
            sum = dot = 0.f;
            if (balance) {
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    sum += v[q];
                    dot = fmaf(pull[q], v[q], dot);
                }
            }
            z = zdw = 0.f;
            if (gate) {
#pragma unroll
                for (int h = 0; h < SLOTS; ++h) {
                    z += sj[h];
                    zdw = fmaf(dw[h], sj[h], zdw);
                }
            }
#pragma unroll
            for (int o = R::kGroup / 2; o > 0; o >>= 1) {
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
                z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
                zdw += __shfl_xor_sync(0xFFFFFFFFu, zdw, o);
            }
        };
        sums();
        // a row or a choice whose sum is tiny: scaled up first, or its reciprocal would
        // overflow and its products lose digits
        const bool tiny = (balance && fabsf(sum) < 0x1p-60f) || (gate && fabsf(z) < 0x1p-60f);
        if (__any_sync(0xFFFFFFFFu, in && tiny)) {
            if (balance && fabsf(sum) < 0x1p-60f) {
                down = 0x1p-80f;
#pragma unroll
                for (int q = 0; q < NV; ++q) v[q] *= 0x1p80f;
            }
            if (gate && fabsf(z) < 0x1p-60f) {
#pragma unroll
                for (int h = 0; h < SLOTS; ++h) sj[h] *= 0x1p80f;
            }
            sums();
        }
        const float inv = reciprocal(sum), zinv = reciprocal(z);
        dot *= inv;
        if (gate) {
            // an expert listed twice has two gates: added then, stored otherwise
            bool twice = SLOTS > 1;  // (then a lane holds several, and all are added)
            if (SLOTS == 1) {
                const uint32_t key = idx[0] >= 0 ? (uint32_t)(idx[0] + group * 1024)
                                                 : 0x80000000u + lane;
                twice = __any_sync(0xFFFFFFFFu, __popc(__match_any_sync(0xFFFFFFFFu, key)) > 1);
            }
#pragma unroll
            for (int h = 0; h < SLOTS; ++h) {
                const float g = (dw[h] - zdw * zinv) * (sj[h] * zinv);
                if (idx[h] >= 0) {
                    if (twice) atomicAdd(mine + idx[h], g);
                    else mine[idx[h]] = g;
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int q = 0; q < R::kN; ++q) {
            const int i = R::expert(glane, q);
            float gt[R::kVec], o[R::kVec];
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
                const float d = fmaf(pull[n] - dot, v[n] * inv, gt[k]);
                o[k] = d * (SOFTPLUS ? softplus_ratio(v[n] * down) : fmaf(-down, v[n], 1.0f));
                v[n] = next[n];
            }
            if (in && i < a.E) {
                float *dst = a.d_logits + (size_t)tok * a.E + i;
                if constexpr (R::kVec == 4)
                    *reinterpret_cast<float4 *>(dst) = make_float4(o[0], o[1], o[2], o[3]);
                else
                    *dst = o[0];
            }
        }
#pragma unroll
        for (int h = 0; h < SLOTS; ++h) idx[h] = next_idx[h], dw[h] = next_dw[h];
        if (gate) __syncwarp();  // the zeroed gates are seen before the next token's
    }
}

// Calls f with the row layout for E experts.  Four experts a load where E allows it,
// and as few lanes a token as hold its row in at most 16 values each (32 from 513
// experts): a warp's steps are then shared by more tokens.  The router gradient of
// 8.4 M affinities with twice the lanes (and half the values), in us: E = 64 34.9 for
// 17.4, 128 17.4 for 14.5, 256 17.0 for 14.5; at 512, half the lanes 16.4 for 14.5.
// Other E go one expert a load: 32768 tokens of 62 experts 16.5 us for 6.9 at 64, of 254
// 18.9 for 14.4 at 256; above 256 a lane holds 32 values and an SM one block, 258
// experts 66 us where 300, four a load, take 22.
template <class F>
cudaError_t with_row(int E, F f) {
    if (E % 4 == 0) {
        if (E <= 64) return f(Row<8, 4, 2>{});
        if (E <= 128) return f(Row<8, 4, 4>{});
        if (E <= 256) return f(Row<16, 4, 4>{});
        if (E <= 512) return f(Row<32, 4, 4>{});
        return f(Row<32, 4, 8>{});
    }
    if (E <= 64) return f(Row<32, 1, 2>{});
    if (E <= 256) return f(Row<32, 1, 8>{});
    return f(Row<32, 1, 32>{});
}

}  // namespace

cudaError_t launch_balance_loss(const float *scores, const int32_t *topk_idx,
                                const int32_t *offsets, int n_seq, float alpha, int T, int E,
                                int K, int32_t *counts, float *prob, float *loss, float *part,
                                int32_t *part_n, int32_t *status, cudaStream_t st) {
    if (n_seq == 0) return cudaSuccess;
    BalanceArgs a{scores, topk_idx, offsets, n_seq, T, E, K, balance_tile(T, n_seq), alpha,
                  counts, prob, loss, part, part_n, status};
    const int tiles = T > 0 ? (T + a.tile - 1) / a.tile : 1;
    const size_t smem = balance_smem(E);
    cudaError_t err = with_row(E, [&](auto row) {
        // up to BAL_CLUSTER tiles are one cluster and one launch (520 tokens of 40 experts:
        // 8.2 us a call, 10.3 with the second launch)
        const bool one = tiles > 1 && tiles <= BAL_CLUSTER;
        auto kern = one ? balance_tile_kernel<decltype(row), true>
                        : balance_tile_kernel<decltype(row), false>;
        // Beside what the kernel declares (4352 bytes with the join, 128 without), rows of
        // more than 658 experts pass the 48 KB that need no leave.  It is asked for
        // the layout's largest E, whatever this call's: no call depends on another's.
        constexpr size_t most = balance_smem(decltype(row)::kMaxE);
        if (most > 40 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(
                kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
            if (e != cudaSuccess) return e;
        }
        if (one) return launch_dependent(kern, tiles, BAL_THREADS, smem, tiles, st, a);
        return launch_dependent(kern, tiles, BAL_THREADS, smem, 1, st, a);
    });
    if (err != cudaSuccess || tiles <= BAL_CLUSTER) return err;
    return launch_dependent(balance_join_kernel, tiles - 1, BAL_JOIN_THREADS, 0, 1, st, a);
}

cudaError_t launch_route_backward(const float *scores, const int32_t *topk_idx,
                                  const float *d_topk_w, const int32_t *offsets, int n_seq,
                                  const int32_t *counts, const float *d_loss, float alpha, int T,
                                  int E, int K, bool softplus, float *d_logits, int32_t *status,
                                  cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    RouteGradArgs a{scores, topk_idx, d_topk_w, offsets, n_seq, counts, d_loss, alpha,
                    T, E, K, 0, d_logits, status};
    return with_row(E, [&](auto row) {
        using R = decltype(row);
        constexpr int many = 32 / R::kGroup;
        auto kern = K <= R::kGroup ? (softplus ? route_backward_kernel<R, 1, true>
                                               : route_backward_kernel<R, 1, false>)
                                   : (softplus ? route_backward_kernel<R, many, true>
                                               : route_backward_kernel<R, many, false>);
        constexpr int groups = GRAD_THREADS / R::kGroup;
        static_assert(sizeof(float) * R::kMaxE * groups <= 32 * 1024);
        const size_t smem = d_topk_w ? sizeof(float) * (size_t)E * groups : 0;
        // consecutive tokens to a block, the same number to each of its groups: one wave
        // of blocks for long batches, a token a group for short ones
        const int64_t round = (int64_t)groups * grad_blocks<R>() * 148;
        a.tile = (int)((T + round - 1) / round) * groups;
        return launch_dependent(kern, (unsigned)(((int64_t)T + a.tile - 1) / a.tile), GRAD_THREADS,
                                smem, 1, st, a);
    });
}

}  // namespace moe
