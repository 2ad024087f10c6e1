// combine.cu -- gate-weighted un-permute and reduce back to token order.
//
// The combine all-to-all ("moe-node-limited-routing", "Why all to all
// dominates MoE step time": outputs return to the token's origin) is a
// gather-reduce on one GPU:
//   out[t] = y_shared[t] + sum_j w[t, j] * y_perm[inv_perm[t, j]]
// in fp32, rounded once to bf16.  HBM-bound: per token K + 1 rows read, one
// written; every thread moves 16-byte chunks and keeps K + 1 loads in flight.
#include "kernels.h"

namespace moe {

namespace {
constexpr int CB_THREADS = 256;

__device__ __forceinline__ void acc_row(float (&acc)[8], float wj, const uint4 &v) {
    acc[0] = fmaf(wj, bf16_lo(v.x), acc[0]); acc[1] = fmaf(wj, bf16_hi(v.x), acc[1]);
    acc[2] = fmaf(wj, bf16_lo(v.y), acc[2]); acc[3] = fmaf(wj, bf16_hi(v.y), acc[3]);
    acc[4] = fmaf(wj, bf16_lo(v.z), acc[4]); acc[5] = fmaf(wj, bf16_hi(v.z), acc[5]);
    acc[6] = fmaf(wj, bf16_lo(v.w), acc[6]); acc[7] = fmaf(wj, bf16_hi(v.w), acc[7]);
}
}  // namespace

// KB = slots loaded per batch (all K at once when K <= 8, so that every row
// load of a chunk is in flight together); slots are accumulated in slot order.
template <int KB>
__global__ void __launch_bounds__(CB_THREADS)
combine_kernel(const uint4 *__restrict__ y_perm, const int32_t *__restrict__ inv_perm,
               const float *__restrict__ topk_w, const uint4 *__restrict__ y_shared, int T,
               int chunks, int K, int64_t n_rows, uint4 *__restrict__ out) {
    const int64_t total = (int64_t)T * chunks;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = i / chunks;
        const int c = (int)(i - t * chunks);
        float acc[8];
        if (y_shared) {
            const uint4 v = __ldg(y_shared + i);
            acc[0] = bf16_lo(v.x); acc[1] = bf16_hi(v.x);
            acc[2] = bf16_lo(v.y); acc[3] = bf16_hi(v.y);
            acc[4] = bf16_lo(v.z); acc[5] = bf16_hi(v.z);
            acc[6] = bf16_lo(v.w); acc[7] = bf16_hi(v.w);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] = 0.f;
        }
        for (int j0 = 0; j0 < K; j0 += KB) {
            uint4 rows[KB];
            float w[KB];
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                const int j = j0 + q;
                rows[q] = make_uint4(0, 0, 0, 0);
                w[q] = 0.f;
                if (j < K) {
                    const int r = __ldg(inv_perm + t * K + j);
                    w[q] = __ldg(topk_w + t * K + j);
                    if (r >= 0 && r < n_rows) rows[q] = __ldg(y_perm + (int64_t)r * chunks + c);
                }
            }
#pragma unroll
            for (int q = 0; q < KB; ++q)
                if (j0 + q < K) acc_row(acc, w[q], rows[q]);
        }
        uint4 o;
        o.x = pack_bf16x2(acc[0], acc[1]);
        o.y = pack_bf16x2(acc[2], acc[3]);
        o.z = pack_bf16x2(acc[4], acc[5]);
        o.w = pack_bf16x2(acc[6], acc[7]);
        out[i] = o;
    }
}

cudaError_t launch_combine(const void *y_perm, const int32_t *inv_perm, const float *topk_w,
                           const void *y_shared, int T, int d, int K, int64_t n_rows, void *out,
                           cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const int chunks = d / 8;
    const int64_t total = (int64_t)T * chunks;
    int sms = 148, dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t want = (total + CB_THREADS - 1) / CB_THREADS;
    const int grid = (int)(want < (int64_t)sms * 8 ? want : (int64_t)sms * 8);
    const uint4 *yp = static_cast<const uint4 *>(y_perm);
    const uint4 *ys = static_cast<const uint4 *>(y_shared);
    uint4 *o = static_cast<uint4 *>(out);
    if (K <= 4)
        combine_kernel<4><<<grid, CB_THREADS, 0, st>>>(yp, inv_perm, topk_w, ys, T, chunks, K, n_rows, o);
    else
        combine_kernel<8><<<grid, CB_THREADS, 0, st>>>(yp, inv_perm, topk_w, ys, T, chunks, K, n_rows, o);
    count_launch();
    return cudaGetLastError();
}

// Gradients of the combine (out_t = y_shared_t + sum_j w_j y_row(t,j)) with
// respect to the expert rows and the gates:
//   d_y_perm[row(t,j)] = bf16(w_(t,j) d_out[t]),  d_topk_w[t][j] = d_out[t] . y_perm[row(t,j)]
// (y_shared's gradient is d_out itself.)  HBM-bound: per copy one row read and
// one written, and d_out once per token: the K warps of a token run side by
// side in a block, so that K - 1 of them find its row in L1.  8192 tokens of 7168
// with K = 8 take 326 us, 6.1 TB/s of the 1.99 GB.  WARPS warps share a copy's
// row: one, which has no sum across warps to wait for, or, for few or long rows,
// eight, whose loads are all in flight at once.
template <int WARPS, bool DY, bool DW>
__global__ void __launch_bounds__(CB_THREADS)
combine_backward_kernel(const uint4 *__restrict__ d_out, const uint4 *__restrict__ y_perm,
                        const int32_t *__restrict__ inv_perm, const float *__restrict__ topk_w,
                        int chunks, int K, int64_t copies, uint4 *__restrict__ d_y_perm,
                        float *__restrict__ d_topk_w) {
    constexpr int TEAM = WARPS * 32, UNROLL = 4;
    const int64_t copy = blockIdx.x * (int64_t)(CB_THREADS / TEAM) + threadIdx.x / TEAM;
    if (copy >= copies) return;  // whole warps; with WARPS > 1 the block is one copy
    const int at = threadIdx.x % TEAM;
    const int row = __ldg(inv_perm + copy);
    const bool have = row >= 0 && row < copies;
    float dot = 0.f;
    if (have) {
        const uint4 *g_row = d_out + copy / K * chunks;
        const uint4 *y_row = y_perm + (int64_t)row * chunks;
        uint4 *dy_row = d_y_perm + (int64_t)row * chunks;
        const float w = DY ? __ldg(topk_w + copy) : 0.f;
        for (int c0 = at; c0 < chunks; c0 += UNROLL * TEAM) {
            uint4 g[UNROLL], y[UNROLL];
#pragma unroll
            for (int q = 0; q < UNROLL; ++q) {
                const int c = c0 + q * TEAM;
                g[q] = y[q] = make_uint4(0u, 0u, 0u, 0u);
                if (c < chunks) {
                    g[q] = __ldg(g_row + c);
                    if (DW) y[q] = __ldcs(y_row + c);
                }
            }
#pragma unroll
            for (int q = 0; q < UNROLL; ++q) {
                const int c = c0 + q * TEAM;
                const uint32_t gw[4] = {g[q].x, g[q].y, g[q].z, g[q].w};
                const uint32_t yw[4] = {y[q].x, y[q].y, y[q].z, y[q].w};
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float lo = bf16_lo(gw[k]), hi = bf16_hi(gw[k]);
                    if (DY) o[k] = pack_bf16x2(w * lo, w * hi);
                    if (DW) dot = fmaf(hi, bf16_hi(yw[k]), fmaf(lo, bf16_lo(yw[k]), dot));
                }
                if (DY && c < chunks) __stcs(dy_row + c, make_uint4(o[0], o[1], o[2], o[3]));
            }
        }
    }
    if constexpr (DW) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
        if (WARPS > 1) {
            __shared__ float part[CB_THREADS / 32];
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
            __syncthreads();
            dot = 0.f;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) dot += part[k];
        }
        if (at == 0) d_topk_w[copy] = dot;
    }
}

namespace {
template <int WARPS>
void run_combine_backward(const uint4 *g, const uint4 *y, const int32_t *inv_perm,
                          const float *topk_w, int chunks, int K, int64_t copies, uint4 *dy,
                          float *dw, cudaStream_t st) {
    constexpr int PER = CB_THREADS / (WARPS * 32);
    const unsigned grid = (unsigned)((copies + PER - 1) / PER);
    if (dy && dw)
        combine_backward_kernel<WARPS, true, true>
            <<<grid, CB_THREADS, 0, st>>>(g, y, inv_perm, topk_w, chunks, K, copies, dy, dw);
    else if (dy)
        combine_backward_kernel<WARPS, true, false>
            <<<grid, CB_THREADS, 0, st>>>(g, y, inv_perm, topk_w, chunks, K, copies, dy, dw);
    else
        combine_backward_kernel<WARPS, false, true>
            <<<grid, CB_THREADS, 0, st>>>(g, y, inv_perm, topk_w, chunks, K, copies, dy, dw);
}
}  // namespace

cudaError_t launch_combine_backward(const void *d_out, const void *y_perm,
                                    const int32_t *inv_perm, const float *topk_w, int T, int d,
                                    int K, int64_t n_rows, void *d_y_perm, float *d_topk_w,
                                    cudaStream_t st) {
    if (T == 0 || (!d_y_perm && !d_topk_w)) return cudaSuccess;
    const uint4 *g = static_cast<const uint4 *>(d_out), *y = static_cast<const uint4 *>(y_perm);
    uint4 *dy = static_cast<uint4 *>(d_y_perm);
    // Eight warps a row and one, in us, by d and copies: 2048: 256 2.2 and 3.2, 512 3.0 and
    // 3.3, 1024 4.4 and 3.4; 4096: 1024 4.9 and 5.5, 8192 30 and 21; 7168: 1024 5.4 and 8.3,
    // 8192 44 and 45, 65536 354 and 323.  The crossing grows as d^2.
    if (n_rows * 8192 <= (int64_t)d * d)
        run_combine_backward<8>(g, y, inv_perm, topk_w, d / 8, K, n_rows, dy, d_topk_w, st);
    else
        run_combine_backward<1>(g, y, inv_perm, topk_w, d / 8, K, n_rows, dy, d_topk_w, st);
    count_launch();
    return cudaGetLastError();
}

}  // namespace moe
