// quant_int8.cu -- rows to signed 8-bit codes with one fp32 scale per row:
//   s = amax / 127 (fp32 division),  q = rint(x / s) (fp32 division, nearest even)
// so that x ~ s q and the row's largest magnitude is +-127.  A row of zeros has
// s = 0 and codes 0; a row that holds a NaN or an infinity has s = NaN (and
// codes 0), so that whatever is computed from it is NaN as it would be from x.
//
// Used for the dispatch payload (a token's codes go to its K permuted rows), the
// shared experts' input, the SwiGLU intermediate and, once at load, the
// weights (a row = an output channel).  HBM-bound: each row is read once and kept
// in registers between the maximum and the rounding (rows of up to 8192 values;
// longer ones are read twice).  A warp takes a row of up to 2048 values, a block
// of four warps a longer one.
#include <type_traits>

#include "kernels.h"

namespace moe {
namespace {

constexpr int Q_THREADS = 128;

struct QuantArgs {
    const void *src;          // rows of `segs` runs of `seg_len` values
    int64_t rows;
    int segs, seg_len;
    int64_t row_stride, seg_stride;  // in values, for src and for the codes beside it
    int8_t *q;                // codes in src's layout, or nullptr
    float *scale;             // [rows], with q
    const int32_t *inv_perm;  // [rows, K] or nullptr: rows of q_perm that get the codes too
    int K;
    int64_t n_perm;
    int8_t *q_perm;           // [n_perm, seg_len], one segment only
    float *scale_perm;        // [n_perm]
};

// One 16-byte load: 8 bf16 or 4 fp32 values, as fp32.
template <bool BF16>
struct Unit {
    static constexpr int N = BF16 ? 8 : 4;
    static __device__ __forceinline__ float get(const uint4 &v, int i) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (BF16) return (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        else return __uint_as_float(w[i]);
    }
};

__device__ __forceinline__ uint32_t code(float x, float s) {
    const float r = rintf(__fdiv_rn(x, s));
    return (uint32_t)(int)fminf(fmaxf(r, -127.f), 127.f) & 0xFFu;  // (a denormal s is coarse)
}

template <bool BF16, int TEAM, int UNITS>
__global__ void __launch_bounds__(Q_THREADS)
quantize_rows_kernel(const QuantArgs a) {
    using U = Unit<BF16>;
    const int at = threadIdx.x % TEAM;
    const int64_t row = blockIdx.x * (int64_t)(Q_THREADS / TEAM) + threadIdx.x / TEAM;
    if (row >= a.rows) return;  // whole teams
    const int per_seg = a.seg_len / U::N, total = per_seg * a.segs;
    const uint4 *src = static_cast<const uint4 *>(a.src);
    auto place = [&](int u) {  // 16-byte units from the start of src
        const int seg = a.segs == 1 ? 0 : u / per_seg;
        return (row * a.row_stride + seg * a.seg_stride) / U::N + (u - seg * per_seg);
    };
    uint4 v[UNITS];
    uint32_t top = 0;  // bits of the largest magnitude: NaN above infinity above the rest
    for (int base = 0; base < total; base += TEAM * UNITS) {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const int u = base + k * TEAM + at;
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (u < total) v[k] = __ldg(src + place(u));
        }
#pragma unroll
        for (int k = 0; k < UNITS; ++k)
#pragma unroll
            for (int i = 0; i < U::N; ++i)
                top = max(top, __float_as_uint(U::get(v[k], i)) & 0x7FFFFFFFu);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (TEAM > 32) {
        __shared__ uint32_t tops[Q_THREADS / 32];
        if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < Q_THREADS / 32; ++w) top = max(top, tops[w]);
    }
    const float s = top >= 0x7F800000u ? __uint_as_float(0x7FFFFFFFu)
                                       : __fdiv_rn(__uint_as_float(top), 127.0f);
    if (at == 0 && a.q) a.scale[row] = s;
    if (a.inv_perm)
        for (int j = at; j < a.K; j += TEAM) {
            const int r = __ldg(a.inv_perm + row * a.K + j);
            if (r >= 0 && r < a.n_perm) a.scale_perm[r] = s;
        }
    const bool again = total > TEAM * UNITS;
    for (int base = 0; base < total; base += TEAM * UNITS) {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const int u = base + k * TEAM + at;
            if (u >= total) continue;
            if (again) v[k] = __ldg(src + place(u));
            uint32_t c[2] = {0u, 0u};
            if (s > 0.f) {
#pragma unroll
                for (int i = 0; i < U::N; ++i)
                    c[i >> 2] |= code(U::get(v[k], i), s) << (8 * (i & 3));
            }
            using Out = typename std::conditional<BF16, uint2, uint32_t>::type;
            Out o;
            if constexpr (BF16) o = make_uint2(c[0], c[1]);
            else o = c[0];
            if (a.q) reinterpret_cast<Out *>(a.q)[place(u)] = o;
            if (a.inv_perm)
                for (int j = 0; j < a.K; ++j) {
                    const int r = __ldg(a.inv_perm + row * a.K + j);
                    if (r >= 0 && r < a.n_perm)
                        reinterpret_cast<Out *>(a.q_perm)[(int64_t)r * total + u] = o;
                }
        }
    }
}

template <bool BF16>
cudaError_t run(const QuantArgs &a, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    constexpr int UNITS = BF16 ? 8 : 16;  // 2048 values a warp, 8192 a block
    if ((int64_t)a.segs * a.seg_len <= 2048) {
        const int64_t per = Q_THREADS / 32;
        quantize_rows_kernel<BF16, 32, UNITS>
            <<<(unsigned)((a.rows + per - 1) / per), Q_THREADS, 0, st>>>(a);
    } else {
        quantize_rows_kernel<BF16, Q_THREADS, UNITS><<<(unsigned)a.rows, Q_THREADS, 0, st>>>(a);
    }
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_rows_bf16(const void *x, int64_t rows, int cols, int8_t *q,
                                      float *scale, cudaStream_t st) {
    QuantArgs a{};
    a.src = x; a.rows = rows; a.segs = 1; a.seg_len = cols; a.row_stride = cols;
    a.q = q; a.scale = scale;
    return run<true>(a, st);
}

cudaError_t launch_quantize_rows_f32(const float *x, int64_t rows, int cols, int8_t *q,
                                     float *scale, cudaStream_t st) {
    QuantArgs a{};
    a.src = x; a.rows = rows; a.segs = 1; a.seg_len = cols; a.row_stride = cols;
    a.q = q; a.scale = scale;
    return run<false>(a, st);
}

cudaError_t launch_quantize_joint_bf16(const void *x, int n_mat, int64_t rows, int cols,
                                       int8_t *q, float *scale, cudaStream_t st) {
    QuantArgs a{};
    a.src = x; a.rows = rows; a.segs = n_mat; a.seg_len = cols; a.row_stride = cols;
    a.seg_stride = rows * cols;
    a.q = q; a.scale = scale;
    return run<true>(a, st);
}

cudaError_t launch_gather_int8(const void *x, const int32_t *inv_perm, int T, int d, int K,
                               int8_t *x_perm_q, float *x_scale, int8_t *x_q, float *x_q_scale,
                               cudaStream_t st) {
    QuantArgs a{};
    a.src = x; a.rows = T; a.segs = 1; a.seg_len = d; a.row_stride = d;
    a.q = x_q; a.scale = x_q_scale;
    a.inv_perm = inv_perm; a.K = K; a.n_perm = (int64_t)T * K;
    a.q_perm = x_perm_q; a.scale_perm = x_scale;
    return run<true>(a, st);
}

}  // namespace moe
