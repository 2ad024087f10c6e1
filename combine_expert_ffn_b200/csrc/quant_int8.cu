// quant_int8.cu -- rows to signed 8-bit codes with one fp32 scale per row:
//   s = amax / 127 (fp32 division)
//   q = rint(x / s) (fp32 division, nearest even)               bf16 rows
//   q = rint(x * fp32(1 / s)) (exact product, nearest even)     fp32 rows: h
// so that x ~ s q and the row's largest magnitude is +-127.  (The two differ only where
// x / s lies within 2^-22 of its size of a half.)  A row of zeros has s = 0 and
// codes 0; a row that holds a NaN or an infinity has s = NaN (and codes 0), so that
// whatever is computed from it is NaN as it would be from x.
//
// Used for the dispatch payload (a token's codes go to its K permuted rows), the
// shared experts' input, the SwiGLU intermediate and, once at load, the
// weights (a row = an output channel).  HBM-bound: each row is read once and kept
// in registers between the maximum and the rounding (rows of up to 8192 values;
// longer ones are read twice), by as many lanes as it takes to hold four 16-byte
// loads each: a warp, four warps or a block.
#include <type_traits>

#include "kernels.h"

namespace moe {
namespace {

constexpr int Q_UNITS = 4;  // 16-byte loads of a lane that stay in registers

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
    // fp32: a second matrix of one-run rows, worked on by the blocks behind
    const void *src2;
    int64_t rows2;
    int len2;
    int8_t *q2;
    float *scale2;
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

// The codes of N values (N / 4 words), and whether each is sure.  With inv = 1 / s,
// x * inv is within 1.5 * 2^-23 |x / s| of the fp32 quotient, so it rounds to the same
// code unless it lies that near a half.  Adding 1.5 * 2^23 leaves the integer, rounded
// to nearest even, in the low byte: no conversion instructions, which run at a
// quarter of the rate.
// TIE: bf16 rows hold half of their largest magnitude often enough (the only
// quotient near a half, 63.5, that 8-bit mantissas give to most rows: 1 value in 600
// of a normal row) to be told apart: |x| = half gets at_half, 63.25 or 63.75 as the
// division says.
// Rows in fp32 are the library's own h, whose 24-bit rounding moves codes that near a
// half either way already: their codes are the product's, by definition (65536 rows of
// 2048 values with the division's: 144 us, without 98, as long as a copy of the bytes takes).
// Where 1 / s is no normal number they are the division's.
template <bool TIE, int N>
__device__ __forceinline__ bool codes(const float (&x)[N], float inv, float half, float at_half,
                                      uint32_t (&c)[N / 4]) {
    constexpr float kMagic = 12582912.0f;
    uint32_t b[N];
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (!TIE) {
            b[i] = __float_as_uint(fmaf(x[i], inv, kMagic));
            continue;
        }
        const float t = fabsf(x[i]) == half ? copysignf(at_half, x[i]) : x[i] * inv;
        const float r = t + kMagic;
        far = fmaxf(far, fmaf(fabsf(t), 0x1p-22f, fabsf(t - (r - kMagic))));
        b[i] = __float_as_uint(r);
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        c[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                           __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
    return far < 0.5f;
}

// The larger magnitude; a NaN wins.
__device__ __forceinline__ float max_magnitude(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
    return m;
}

template <int TEAM>
__host__ __device__ constexpr int block_threads() { return TEAM < 128 ? 128 : TEAM; }

// TEAM threads a row.
// JOINT: rows of more than one run.
template <bool BF16, int TEAM, bool JOINT>
__global__ void __launch_bounds__(block_threads<TEAM>())
quantize_rows_kernel(const QuantArgs a) {
    using U = Unit<BF16>;
    constexpr int UNITS = Q_UNITS, Q_THREADS = block_threads<TEAM>();
    const int at = threadIdx.x % TEAM;
    int64_t row = blockIdx.x * (int64_t)(Q_THREADS / TEAM) + threadIdx.x / TEAM;
    dependency_wait();
    dependency_release();
    const bool second = !BF16 && row >= a.rows;
    if (second) row -= a.rows;
    if (row >= (second ? a.rows2 : a.rows)) return;  // whole teams
    const int per_seg = (second ? a.len2 : a.seg_len) / U::N;
    const int total = JOINT ? per_seg * a.segs : per_seg;
    // in 16-byte units from the start of src
    const int64_t row0 = row * ((second ? a.len2 : a.row_stride) / U::N);
    const uint4 *src = static_cast<const uint4 *>(second ? a.src2 : a.src) + row0;
    int8_t *const q_out = second ? a.q2 : a.q;
    auto place = [&](int u) {
        if (!JOINT) return (int64_t)u;
        const int seg = u / per_seg;
        return seg * (a.seg_stride / U::N) + (u - seg * per_seg);
    };
    uint4 v[UNITS];
    float most = 0.f;
    __nv_bfloat162 most2 = __floats2bfloat162_rn(0.f, 0.f);
    for (int base = 0; base < total; base += TEAM * UNITS) {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const int u = base + k * TEAM + at;
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (u < total) v[k] = __ldcg(src + place(u));
        }
#pragma unroll
        for (int k = 0; k < UNITS; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t w = i == 0 ? v[k].x : i == 1 ? v[k].y : i == 2 ? v[k].z : v[k].w;
                if constexpr (BF16)
                    most2 = __hmax2_nan(most2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w)));
                else
                    most = max_magnitude(most, __uint_as_float(w));
            }
    }
    if (BF16) most = max_magnitude(__low2float(most2), __high2float(most2));
    // as bits: NaN above infinity above the rest
    uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
    if (TEAM > 32) {
        __shared__ uint32_t tops[Q_THREADS / 32];
        if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < Q_THREADS / 32; ++w) top = max(top, tops[w]);
    }
    const float s = top >= 0x7F800000u ? __uint_as_float(0x7FFFFFFFu)
                                       : __fdiv_rn(__uint_as_float(top), 127.0f);
    if (at == 0 && q_out) (second ? a.scale2 : a.scale)[row] = s;
    if (BF16 && a.inv_perm)
        for (int j = at; j < a.K; j += TEAM) {
            const int r = a.inv_perm[row * a.K + j];
            if (r >= 0 && r < a.n_perm) a.scale_perm[r] = s;
        }
    using Out = typename std::conditional<BF16, uint2, uint32_t>::type;
    auto store = [&](int u, const uint32_t (&c)[U::N / 4]) {
        Out o;
        if constexpr (BF16) o = make_uint2(c[0], c[1]);
        else o = c[0];
        if (q_out) reinterpret_cast<Out *>(q_out)[row0 + place(u)] = o;
        if (BF16 && a.inv_perm)
            for (int j = 0; j < a.K; ++j) {
                const int r = a.inv_perm[row * a.K + j];
                if (r >= 0 && r < a.n_perm)
                    reinterpret_cast<Out *>(a.q_perm)[(int64_t)r * total + u] = o;
            }
    };
    // a scale whose reciprocal is no normal float (0 and NaN among them): every code
    // is unsure, from values of inv = 0
    const float inv = s > 0x1p-120f && s < 0x1p120f ? 1.0f / s : 0.f;
    const float half = 0.5f * __uint_as_float(top);
    const float at_half = rintf(__fdiv_rn(half, s)) > 63.5f ? 63.75f : 63.25f;
    const bool again = total > TEAM * UNITS;
    for (int base = 0; base < total; base += TEAM * UNITS) {
        uint32_t unsure = 0;
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const int u = base + k * TEAM + at;
            if (u >= total) continue;
            if (again) v[k] = __ldcg(src + place(u));
            float f[U::N];
#pragma unroll
            for (int i = 0; i < U::N; ++i) f[i] = U::get(v[k], i);
            uint32_t c[U::N / 4];
            if (!codes<BF16, U::N>(f, inv, half, at_half, c) || inv == 0.f) unsure |= 1u << k;
            else store(u, c);
        }
        // Units with a value near a half divide.
        // A rolled loop that reads them again: with the divisions of every unit inlined
        // above, the kernel's instruction fetches alone took 11 us a block.
#pragma unroll 1
        for (; unsure; unsure &= unsure - 1) {
            const int u = base + (__ffs(unsure) - 1) * TEAM + at;
            const uint4 w = __ldcg(src + place(u));
            uint32_t c[U::N / 4];
#pragma unroll
            for (int i = 0; i < U::N / 4; ++i) c[i] = 0u;
            if (s > 0.f) {
#pragma unroll
                for (int i = 0; i < U::N; ++i) c[i / 4] |= code(U::get(w, i), s) << (8 * (i % 4));
            }
            store(u, c);
        }
    }
}

// The whole int8 dispatch of a batch of at most 256 tokens in one launch, a block a
// token.  Every block builds the plan for itself -- a bit for each (expert, token), whose
// counts over all tokens, scanned over the experts, are the offsets, and over the tokens
// below its own the ranks -- and then writes its token's codes to its K rows; block 0
// writes what belongs to the batch.  The ids (at most 8192) come from L2 for each block,
// which is less than the two launches it saves: 1, 128 and 256 tokens of 7168, K = 8, 256
// experts take 5.6, 8.8 and 10.0 us, the plan's two kernels and the gather 11.7, 17.4 and 19.2.
struct SmallDispatch {
    QuantArgs q;  // the token rows, codes and permuted rows
    const int32_t *topk_idx;
    int T, E, G;
    int32_t *counts, *offsets, *send, *send_tok, *perm_token, *inv_perm, *status;
};

// Its dynamic shared memory: the tokens' bits, the offsets, and the two send matrices.
constexpr size_t small_dispatch_smem(int E, int G) {
    return sizeof(uint32_t) * ((size_t)E * (DISPATCH_BLOCK / 32) + E + 1 + 2 * G * G);
}

__global__ void __launch_bounds__(DISPATCH_BLOCK)
dispatch_int8_small_kernel(const SmallDispatch a) {
    constexpr int BLK = DISPATCH_BLOCK, WORDS = BLK / 32, KMAX = 32;
    extern __shared__ __align__(16) uint32_t sm[];
    const int E = a.E, G = a.G, K = a.q.K;
    uint32_t *masks = sm;                                        // [E, WORDS]
    int *offs = reinterpret_cast<int *>(masks + E * WORDS);      // [E + 1]
    int *send_s = offs + E + 1, *sendtok_s = send_s + G * G;     // [G, G] each, block 0
    __shared__ int wsum[WORDS], rows[KMAX];
    __shared__ uint32_t tops[WORDS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = blockIdx.x;
    const bool first = t == 0;
    dependency_wait();
    dependency_release();

    // loads first: this thread's token's ids, and this block's row
    int ev[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
        ev[j] = tid < a.T && j < K ? a.topk_idx[tid * K + j] : -1;
    const int total = a.q.seg_len / 8;
    const uint4 *src = static_cast<const uint4 *>(a.q.src) + (int64_t)t * total;
    uint4 v[Q_UNITS];
    auto load = [&](int base) {
#pragma unroll
        for (int k = 0; k < Q_UNITS; ++k) {
            const int u = base + k * BLK + tid;
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (u < total) v[k] = __ldcg(src + u);
        }
    };
    load(0);
    for (int i = tid; i < E * WORDS; i += BLK) masks[i] = 0u;
    if (first)
        for (int i = tid; i < 2 * G * G; i += BLK) send_s[i] = 0;
    __syncthreads();
    if (tid < a.T) {
        uint64_t hit = 0;
        const int gsz = E / G, from = tid / (a.T / G);
#pragma unroll
        for (int j = 0; j < KMAX; ++j) {
            if (j >= K) break;
            const int e = ev[j];
            if (e < 0 || e >= E) {
                if (first) record_status(a.status, MOE_ERR_DEVICE_FAULT);
                continue;
            }
            const uint32_t old = atomicOr(&masks[e * WORDS + warp], 1u << lane);
            if (first) {
                if (old >> lane & 1u) record_status(a.status, MOE_ERR_DEVICE_FAULT);
                atomicAdd(&send_s[from * G + e / gsz], 1);
                hit |= 1ull << (e / gsz);
            }
        }
        for (; hit; hit &= hit - 1) atomicAdd(&sendtok_s[from * G + __ffsll((long long)hit) - 1], 1);
    }
    __syncthreads();
    // offsets: each thread a run of experts
    const int per = (E + BLK - 1) / BLK;
    int run = 0;
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e >= E) break;
        int c = 0;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) c += __popc(masks[e * WORDS + w]);
        offs[e] = c;
        run += c;
    }
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) wsum[warp] = incl;
    // the row's largest magnitude meanwhile (as bits: NaN above infinity above the rest)
    __nv_bfloat162 most2 = __floats2bfloat162_rn(0.f, 0.f);
    for (int base = 0;;) {
#pragma unroll
        for (int k = 0; k < Q_UNITS; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                most2 = __hmax2_nan(most2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(w + i)));
        }
        base += BLK * Q_UNITS;
        if (base >= total) break;
        load(base);
    }
    uint32_t top = __reduce_max_sync(
        0xFFFFFFFFu, __float_as_uint(max_magnitude(__low2float(most2), __high2float(most2))));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    int at = incl - run;
    for (int w = 0; w < warp; ++w) at += wsum[w];
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e >= E) break;
        const int c = offs[e];
        offs[e] = at;
        if (first) {
            a.counts[e] = c;
            a.offsets[e] = at;
        }
        at += c;
    }
    if (first && tid == BLK - 1) a.offsets[E] = at;
    if (first)
        for (int i = tid; i < G * G; i += BLK) {
            a.send[i] = send_s[i];
            if (a.send_tok) a.send_tok[i] = sendtok_s[i];
        }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WORDS; ++w) top = max(top, tops[w]);
    const float s = top >= 0x7F800000u ? __uint_as_float(0x7FFFFFFFu)
                                       : __fdiv_rn(__uint_as_float(top), 127.0f);
    if (tid < K) {  // this token's rows
        const int e = a.topk_idx[t * K + tid];
        int row = -1;
        if (e >= 0 && e < E) {
            row = offs[e] + __popc(masks[e * WORDS + (t >> 5)] & ((1u << (t & 31)) - 1u));
            for (int w = 0; w < t >> 5; ++w) row += __popc(masks[e * WORDS + w]);
            a.perm_token[row] = t;
            a.q.scale_perm[row] = s;
        }
        a.inv_perm[t * K + tid] = row;
        rows[tid] = row;
    }
    if (tid == 0 && a.q.q) a.q.scale[t] = s;
    __syncthreads();
    auto store = [&](int u, const uint32_t (&c)[2]) {
        const uint2 o = make_uint2(c[0], c[1]);
        if (a.q.q) reinterpret_cast<uint2 *>(a.q.q)[(int64_t)t * total + u] = o;
        for (int j = 0; j < K; ++j)
            if (rows[j] >= 0) reinterpret_cast<uint2 *>(a.q.q_perm)[(int64_t)rows[j] * total + u] = o;
    };
    const float inv = s > 0x1p-120f && s < 0x1p120f ? 1.0f / s : 0.f;
    const float half = 0.5f * __uint_as_float(top);
    const float at_half = rintf(__fdiv_rn(half, s)) > 63.5f ? 63.75f : 63.25f;
    for (int base = 0; base < total; base += BLK * Q_UNITS) {
        if (total > BLK * Q_UNITS) load(base);
        uint32_t unsure = 0;
#pragma unroll
        for (int k = 0; k < Q_UNITS; ++k) {
            const int u = base + k * BLK + tid;
            if (u >= total) continue;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = Unit<true>::get(v[k], i);
            uint32_t c[2];
            if (!codes<true, 8>(f, inv, half, at_half, c) || inv == 0.f) unsure |= 1u << k;
            else store(u, c);
        }
#pragma unroll 1
        for (; unsure; unsure &= unsure - 1) {  // values near a half
            const int u = base + (__ffs(unsure) - 1) * BLK + tid;
            const uint4 w = __ldcg(src + u);
            uint32_t c[2] = {0u, 0u};
            if (s > 0.f) {
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i / 4] |= code(Unit<true>::get(w, i), s) << (8 * (i % 4));
            }
            store(u, c);
        }
    }
}

template <bool BF16, int TEAM>
cudaError_t run_team(const QuantArgs &a, cudaStream_t st) {
    constexpr int per = block_threads<TEAM>() / TEAM;
    const unsigned grid = (unsigned)((a.rows + a.rows2 + per - 1) / per);
    if (BF16 && a.segs > 1)  // the shared experts' down projection; never fp32
        return launch_dependent(quantize_rows_kernel<BF16, TEAM, BF16>, grid, block_threads<TEAM>(),
                                0, 1, st, a);
    return launch_dependent(quantize_rows_kernel<BF16, TEAM, false>, grid, block_threads<TEAM>(), 0,
                            1, st, a);
}

template <bool BF16>
cudaError_t run(const QuantArgs &a, cudaStream_t st) {
    if (a.rows + a.rows2 == 0) return cudaSuccess;
    const int64_t lanes = (int64_t)a.segs * a.seg_len / (Unit<BF16>::N * Q_UNITS);
    if (lanes <= 32) return run_team<BF16, 32>(a, st);
    if (lanes <= 128) return run_team<BF16, 128>(a, st);
    if (BF16 || lanes <= 256) return run_team<BF16, 256>(a, st);
    return run_team<BF16, BF16 ? 256 : 512>(a, st);
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
                                     float *scale, const float *x2, int64_t rows2, int cols2,
                                     int8_t *q2, float *scale2, cudaStream_t st) {
    QuantArgs a{};
    a.src = x; a.rows = rows; a.segs = 1; a.seg_len = cols; a.row_stride = cols;
    a.q = q; a.scale = scale;
    QuantArgs b{};
    b.src = x2; b.rows = rows2; b.segs = 1; b.seg_len = cols2; b.row_stride = cols2;
    b.q = q2; b.scale = scale2;
    // one launch where both take the same number of lanes a row (a launch saved is 2 us
    // of a single token's 84)
    auto lanes = [](int c) { return c <= 512 ? 32 : c <= 2048 ? 128 : c <= 4096 ? 256 : 512; };
    if (rows2 > 0 && lanes(cols) != lanes(cols2)) {
        const cudaError_t err = run<false>(b, st);
        if (err != cudaSuccess) return err;
    } else {
        a.src2 = x2; a.rows2 = rows2; a.len2 = cols2; a.q2 = q2; a.scale2 = scale2;
    }
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

cudaError_t launch_dispatch_int8(const void *x, const int32_t *topk_idx, int T, int d, int E, int G,
                                 int K, int32_t *counts, int32_t *offsets, int32_t *send,
                                 int32_t *send_tok, int32_t *perm_token, int32_t *inv_perm,
                                 int8_t *x_perm_q, float *x_scale, int8_t *x_q, float *x_q_scale,
                                 const DispatchWs &ws, int32_t *status, cudaStream_t st) {
    QuantArgs q{};
    q.src = x; q.rows = T; q.segs = 1; q.seg_len = d; q.row_stride = d;
    q.q = x_q; q.scale = x_q_scale;
    q.inv_perm = inv_perm; q.K = K; q.n_perm = (int64_t)T * K;
    q.q_perm = x_perm_q; q.scale_perm = x_scale;
    if (dispatch_int8_in_one(T)) {
        SmallDispatch a{q, topk_idx, T, E, G, counts, offsets, send, send_tok, perm_token, inv_perm,
                        status};
        // Beside the 192 bytes that the kernel declares, 48 KB need no leave.  It is
        // asked for the largest E and G, whatever this call's: no call depends on another's.
        const size_t smem = small_dispatch_smem(E, G);
        if (smem > 40 * 1024) {
            const cudaError_t err = cudaFuncSetAttribute(
                dispatch_int8_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                (int)small_dispatch_smem(1024, 64));
            if (err != cudaSuccess) return err;
        }
        return launch_dependent(dispatch_int8_small_kernel, T, DISPATCH_BLOCK, smem, 1, st, a);
    }
    const cudaError_t err = launch_dispatch(x, topk_idx, T, d, E, G, K, counts, offsets, send, send_tok,
                                            perm_token, inv_perm, nullptr, ws, status, st);
    return err != cudaSuccess ? err : run<true>(q, st);
}

}  // namespace moe
