// gemm_int8.cu -- the grouped expert FFN as int8 matrix products on the
// 5th-generation tensor cores (tcgen05.mma kind::i8, 32-bit integer accumulators
// in TMEM, operands by TMA).
//
// Per routed expert e with rows R_e = [offsets[e], offsets[e+1]) of the codes
// x_perm_q (row scale sx) and for the shared experts on all T rows:
//   GEMM1:  g = (Xq Wq_g^T) sx sg,  u = (Xq Wq_u^T) sx su,  h = SiLU(g) u  (fp32)
//   rows:   sh = max|h| / 127,  Hq = rint(h / sh)
//   GEMM2:  y = (Hq Wq_d^T) sh sd                                          (bf16)
// sg, su, sd are per output channel.  The integer sums are exact (reductions of
// less than 2^17 keep |sum| < 2^31); h is kept in fp32 because a rounding to 16
// bits would move about one code in seventy of its row to a neighbour, an error
// several times the final bf16 rounding.  The n_shared shared experts are one
// expert of width n_shared * d_ff_shared.
//
// One persistent kernel per GEMM, one CTA per SM, 192 threads: warp 0 the TMA
// producer (A 128 x 128 bytes, B 256 x 128 bytes a stage), warp 1 the MMA issuer
// (M = 128, N = 256, K = 32), warps 2..5 the epilogue, over two accumulators so
// that the epilogue of a tile overlaps the next tile's MMAs.  Rows of a tile past
// its segment are computed and never stored.  Every wait is bounded.
#include <cstring>

#include "kernels.h"

namespace moe {
namespace gemm_i8 {

constexpr int BM = 128;
constexpr int BK = 128;      // bytes = codes per k block
constexpr int BN_ACC = 256;  // accumulator columns
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK;
constexpr int B_BYTES = BN_ACC * BK;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int NUM_THREADS = 192;
constexpr int TMEM_COLS = 512;
constexpr int MAX_E = 1024;
constexpr int SMEM_DYN = STAGES * STAGE_BYTES + 1024;

enum { EPI_SWIGLU = 0, EPI_STORE = 1 };
template <int EPI>
__host__ __device__ constexpr int bn_out() { return EPI == EPI_SWIGLU ? 128 : 256; }

struct Maps {
    CUtensorMap a_r, a_s;    // codes [rows, k], box 128 x 128
    CUtensorMap b0_r, b1_r;  // routed weights [E, n, k], box 128 x (128 | 256): gate | down, up
    CUtensorMap b0_s, b1_s;  // shared weights
};

struct Params {
    const int32_t *offsets;
    int E, rows_r, T;        // T = 0: no shared experts
    int n_out_r, n_out_s;    // output columns
    int k_r, k_s;            // reduction lengths; the shared one is n_seg_s runs of k_s
    int n_seg_s;
    const float *a_scale_r, *a_scale_s;    // per row
    const float *b0_scale_r, *b1_scale_r;  // per output channel, [E, n_out_r]
    const float *b0_scale_s, *b1_scale_s;
    void *out_r, *out_s;     // fp32 (SwiGLU) or bf16
    int32_t *status;
    int64_t timeout_ns;
};

struct Tile {
    int row0, rows_valid, n0, e, kblocks;  // e < 0: the shared experts
};

template <int EPI>
__device__ __forceinline__ Tile decode_tile(int idx, const int *tile_base, const int *seg,
                                            const int *segc, const Params &p, int ntr, int nt_s) {
    Tile t;
    if (idx < ntr) {
        int lo = 0, hi = p.E;  // tile_base[lo] <= idx < tile_base[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tile_base[mid] <= idx) lo = mid; else hi = mid;
        }
        const int cnt = segc[lo], mt = (cnt + BM - 1) / BM;
        const int local = idx - tile_base[lo];
        const int n = local / mt, m = local - n * mt;  // row tiles of a weight tile side by side
        t.row0 = seg[lo] + m * BM;
        t.rows_valid = min(BM, cnt - m * BM);
        t.n0 = n * bn_out<EPI>();
        t.e = lo;
        t.kblocks = (p.k_r + BK - 1) / BK;
    } else {
        const int local = idx - ntr;
        const int m = local / nt_s, n = local - m * nt_s;
        t.row0 = m * BM;
        t.rows_valid = min(BM, p.T - m * BM);
        t.n0 = n * bn_out<EPI>();
        t.e = -1;
        t.kblocks = p.n_seg_s * ((p.k_s + BK - 1) / BK);
    }
    return t;
}

// Wait while winding down: ignores the abort flag, so that copies and MMAs in
// flight are waited for before the CTA exits.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, int64_t timeout_ns,
                                           int32_t *status) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if ((int64_t)(globaltimer_ns() - t0) > timeout_ns) {
            record_status(status, MOE_ERR_DEVICE_TIMEOUT);
            return;
        }
    }
}

__device__ __forceinline__ float silu_mul(float g, float u) {
    return g * __frcp_rn(1.0f + __expf(-g)) * u;
}

template <int EPI>
__global__ void __launch_bounds__(NUM_THREADS, 1)
grouped_int8_kernel(const __grid_constant__ Maps maps, const Params p) {
    constexpr int BN_OUT = bn_out<EPI>();
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[STAGES], empty_bar[STAGES];
    __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2], done_bar;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;
    __shared__ int tile_base[MAX_E + 1], seg[MAX_E], segc[MAX_E];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t smem0 = smem_u32(smem);
    volatile int *abort_flag = &abort_s;

    if (warp == 0) {
        // tile_base[e] = sum over experts < e of (row tiles x column tiles)
        const int nt_r = (p.n_out_r + BN_OUT - 1) / BN_OUT;
        int carry = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int lo = 0, cnt = 0;
            if (e < p.E) {
                lo = p.offsets[e];
                const int64_t n = (int64_t)p.offsets[e + 1] - lo;
                // a segment that leaves the buffer or has a negative length is
                // treated as empty and reported
                if (lo < 0 || n < 0 || lo + n > p.rows_r) {
                    record_status(p.status, MOE_ERR_DEVICE_FAULT);
                    lo = 0;
                } else {
                    cnt = (int)n;
                }
                seg[e] = lo;
                segc[e] = cnt;
            }
            const int v = (int)(((int64_t)cnt + BM - 1) / BM) * nt_r;
            int incl = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += n;
            }
            if (e < p.E) tile_base[e] = carry + incl - v;
            carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (lane == 0) {
            tile_base[p.E] = carry;
            tma_prefetch_desc(&maps.a_r);
            tma_prefetch_desc(&maps.b0_r);
            if (EPI == EPI_SWIGLU) tma_prefetch_desc(&maps.b1_r);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < STAGES; ++s) {
                mbar_init(smem_u32(&full_bar[s]), 1);
                mbar_init(smem_u32(&empty_bar[s]), 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&tfull_bar[b]), 1);
                mbar_init(smem_u32(&tempty_bar[b]), 128);
            }
            mbar_init(smem_u32(&done_bar), 1);
            abort_s = 0;
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc<TMEM_COLS>(smem_u32(&tmem_base_s));
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_s;

    const int ntr = tile_base[p.E];
    const int mt_s = p.T > 0 ? (p.T + BM - 1) / BM : 0;
    const int nt_s = p.T > 0 ? (p.n_out_s + BN_OUT - 1) / BN_OUT : 0;
    const int total = ntr + mt_s * nt_s;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, n_issued = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < total && ok; idx += gridDim.x) {
                const Tile t = decode_tile<EPI>(idx, tile_base, seg, segc, p, ntr, nt_s);
                const bool shared = t.e < 0;
                const CUtensorMap *am = shared ? &maps.a_s : &maps.a_r;
                const CUtensorMap *b0 = shared ? &maps.b0_s : &maps.b0_r;
                const CUtensorMap *b1 = shared ? &maps.b1_s : &maps.b1_r;
                const int k_len = shared ? p.k_s : p.k_r;
                int mat = shared ? 0 : t.e, k = 0, a_col = 0;
                for (int kb = 0; kb < t.kblocks; ++kb) {
                    if (!mbar_wait_bounded(smem_u32(&empty_bar[stage]), phase ^ 1u, abort_flag,
                                           p.status, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&full_bar[stage]);
                    const uint32_t a_dst = smem0 + stage * STAGE_BYTES;
                    const uint32_t b_dst = a_dst + A_BYTES;
                    mbar_arrive_expect_tx(fb, STAGE_BYTES);
                    tma_load_2d(a_dst, am, fb, a_col + k, t.row0);
                    tma_load_3d(b_dst, b0, fb, k, t.n0, mat);
                    if (EPI == EPI_SWIGLU) tma_load_3d(b_dst + B_BYTES / 2, b1, fb, k, t.n0, mat);
                    // a run's last block may pass its end: B reads zeros there
                    k += BK;
                    if (shared && k >= k_len) {
                        k = 0;
                        ++mat;
                        a_col += k_len;
                    }
                    ++n_issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            // wind down: every load issued into a stage has landed
            for (int s = 0; s < STAGES; ++s) {
                if (n_issued > (uint32_t)s) {
                    const uint32_t uses = (n_issued - 1 - s) / STAGES + 1;
                    drain_wait(smem_u32(&full_bar[s]), (uses - 1) & 1u, p.timeout_ns, p.status);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_s8_s32<BM, BN_ACC>();
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < total && ok; idx += gridDim.x) {
                const Tile t = decode_tile<EPI>(idx, tile_base, seg, segc, p, ntr, nt_s);
                if (!mbar_wait_bounded(smem_u32(&tempty_bar[acc]), acc_phase ^ 1u, abort_flag,
                                       p.status, p.timeout_ns))
                    break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * BN_ACC;
                for (int kb = 0; kb < t.kblocks; ++kb) {
                    if (!mbar_wait_bounded(smem_u32(&full_bar[stage]), phase, abort_flag, p.status,
                                           p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem0 + stage * STAGE_BYTES;
                    const uint64_t a_desc = smem_desc_sw128(a_addr);
                    const uint64_t b_desc = smem_desc_sw128(a_addr + A_BYTES);
#pragma unroll
                    for (int ks = 0; ks < BK / 32; ++ks)
                        tc_mma_s8(d_tmem, a_desc + 2 * ks, b_desc + 2 * ks, idesc,
                                  (kb | ks) != 0 ? 1u : 0u);
                    tc_commit(smem_u32(&empty_bar[stage]));
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                tc_commit(smem_u32(&tfull_bar[acc]));
                if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
            }
            // wind down: every MMA issued has completed
            tc_commit(smem_u32(&done_bar));
            drain_wait(smem_u32(&done_bar), 0, p.timeout_ns, p.status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int idx = blockIdx.x; idx < total; idx += gridDim.x) {
            const Tile t = decode_tile<EPI>(idx, tile_base, seg, segc, p, ntr, nt_s);
            const bool shared = t.e < 0;
            const int n_out = shared ? p.n_out_s : p.n_out_r;
            const int row = q * 32 + lane;
            const bool row_ok = row < t.rows_valid;
            const size_t grow = (size_t)t.row0 + row;
            float sa = 0.f;
            if (row_ok) sa = __ldg((shared ? p.a_scale_s : p.a_scale_r) + grow);
            const size_t ch = (size_t)(shared ? 0 : t.e) * n_out + t.n0;
            const float *s0 = (shared ? p.b0_scale_s : p.b0_scale_r) + ch;
            const float *s1 = (shared ? p.b1_scale_s : p.b1_scale_r) + ch;
            if (!mbar_wait_bounded(smem_u32(&tfull_bar[acc]), acc_phase, abort_flag, p.status,
                                   p.timeout_ns))
                break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * BN_ACC;
            // columns past n_out come in whole chunks: n_out is a multiple of 64
#pragma unroll 1
            for (int c = 0; c < BN_OUT && t.n0 + c < n_out; c += 32) {
                if (EPI == EPI_SWIGLU) {
                    uint32_t g[32], u[32];
                    tmem_ld32(taddr + c, g);
                    tmem_ld32(taddr + BN_ACC / 2 + c, u);
                    tc_wait_ld();
                    if (row_ok) {
                        float *dst = static_cast<float *>(shared ? p.out_s : p.out_r) +
                                     grow * n_out + t.n0 + c;
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const float4 sg = __ldg(reinterpret_cast<const float4 *>(s0 + c) + v);
                            const float4 su = __ldg(reinterpret_cast<const float4 *>(s1 + c) + v);
                            float4 o;
                            o.x = silu_mul((float)(int)g[4 * v] * sa * sg.x,
                                           (float)(int)u[4 * v] * sa * su.x);
                            o.y = silu_mul((float)(int)g[4 * v + 1] * sa * sg.y,
                                           (float)(int)u[4 * v + 1] * sa * su.y);
                            o.z = silu_mul((float)(int)g[4 * v + 2] * sa * sg.z,
                                           (float)(int)u[4 * v + 2] * sa * su.z);
                            o.w = silu_mul((float)(int)g[4 * v + 3] * sa * sg.w,
                                           (float)(int)u[4 * v + 3] * sa * su.w);
                            reinterpret_cast<float4 *>(dst)[v] = o;
                        }
                    }
                } else {
                    uint32_t r[32];
                    tmem_ld32(taddr + c, r);
                    tc_wait_ld();
                    if (row_ok) {
                        __nv_bfloat16 *dst =
                            static_cast<__nv_bfloat16 *>(shared ? p.out_s : p.out_r) +
                            grow * n_out + t.n0 + c;
                        float f[32];
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const float4 sd = __ldg(reinterpret_cast<const float4 *>(s0 + c) + v);
                            f[4 * v] = (float)(int)r[4 * v] * sa * sd.x;
                            f[4 * v + 1] = (float)(int)r[4 * v + 1] * sa * sd.y;
                            f[4 * v + 2] = (float)(int)r[4 * v + 2] * sa * sd.z;
                            f[4 * v + 3] = (float)(int)r[4 * v + 3] * sa * sd.w;
                        }
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            reinterpret_cast<uint4 *>(dst)[v] =
                                make_uint4(pack_bf16x2(f[8 * v], f[8 * v + 1]),
                                           pack_bf16x2(f[8 * v + 2], f[8 * v + 3]),
                                           pack_bf16x2(f[8 * v + 4], f[8 * v + 5]),
                                           pack_bf16x2(f[8 * v + 6], f[8 * v + 7]));
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&tempty_bar[acc]));
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<TMEM_COLS>(tmem_base);
    }
}

namespace {
int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    return sms;
}

template <int EPI>
cudaError_t launch(const Maps &maps, const Params &p, cudaStream_t st) {
    auto kern = grouped_int8_kernel<EPI>;
    cudaError_t err =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_DYN);
    if (err != cudaSuccess) return err;
    kern<<<sm_count(), NUM_THREADS, SMEM_DYN, st>>>(maps, p);
    count_launch();
    return cudaGetLastError();
}
}  // namespace
}  // namespace gemm_i8

cudaError_t launch_expert_ffn_int8(const FfnInt8Args &a, cudaStream_t st) {
    using namespace gemm_i8;
    if (!tensor_maps_available()) return cudaErrorNotSupported;
    const uint64_t rows = (uint64_t)a.T * a.K;
    if (rows == 0) return cudaSuccess;
    const bool has_shared = a.n_shared > 0;
    const int ffs = a.n_shared * a.d_ff_shared;

    Maps m;
    std::memset(&m, 0, sizeof(m));
    bool ok = tensor_map_2d_u8(&m.a_r, a.x_perm_q, rows, a.d, BK, BM, 128) &&
              tensor_map_3d_u8(&m.b0_r, a.w.w_gate, a.E, a.d_ff, a.d, BK, BN_ACC / 2, 128) &&
              tensor_map_3d_u8(&m.b1_r, a.w.w_up, a.E, a.d_ff, a.d, BK, BN_ACC / 2, 128);
    if (has_shared)
        ok = ok && tensor_map_2d_u8(&m.a_s, a.x_q, a.T, a.d, BK, BM, 128) &&
             tensor_map_3d_u8(&m.b0_s, a.w.ws_gate, 1, ffs, a.d, BK, BN_ACC / 2, 128) &&
             tensor_map_3d_u8(&m.b1_s, a.w.ws_up, 1, ffs, a.d, BK, BN_ACC / 2, 128);
    if (!ok) return cudaErrorInvalidValue;
    Params p{};
    p.offsets = a.offsets;
    p.E = a.E;
    p.rows_r = (int)rows;
    p.T = has_shared ? a.T : 0;
    p.n_out_r = a.d_ff;
    p.n_out_s = ffs;
    p.k_r = p.k_s = a.d;
    p.n_seg_s = 1;
    p.a_scale_r = a.x_scale;
    p.a_scale_s = a.x_q_scale;
    p.b0_scale_r = a.w.w_gate_scale;
    p.b1_scale_r = a.w.w_up_scale;
    p.b0_scale_s = a.w.ws_gate_scale;
    p.b1_scale_s = a.w.ws_up_scale;
    p.out_r = a.h;
    p.out_s = a.h_shared;
    p.status = a.status;
    p.timeout_ns = a.timeout_ns;
    cudaError_t err = launch<EPI_SWIGLU>(m, p, st);
    if (err != cudaSuccess) return err;

    err = launch_quantize_rows_f32(a.h, (int64_t)rows, a.d_ff, a.h_q, a.h_scale, st);
    if (err != cudaSuccess) return err;
    if (has_shared) {
        err = launch_quantize_rows_f32(a.h_shared, a.T, ffs, a.h_shared_q, a.h_shared_scale, st);
        if (err != cudaSuccess) return err;
    }

    std::memset(&m, 0, sizeof(m));
    ok = tensor_map_2d_u8(&m.a_r, a.h_q, rows, a.d_ff, BK, BM, 128) &&
         tensor_map_3d_u8(&m.b0_r, a.w.w_down, a.E, a.d, a.d_ff, BK, BN_ACC, 128);
    if (has_shared)
        ok = ok && tensor_map_2d_u8(&m.a_s, a.h_shared_q, a.T, ffs, BK, BM, 128) &&
             tensor_map_3d_u8(&m.b0_s, a.w.ws_down, a.n_shared, a.d, a.d_ff_shared, BK, BN_ACC, 128);
    if (!ok) return cudaErrorInvalidValue;
    p.n_out_r = p.n_out_s = a.d;
    p.k_r = a.d_ff;
    p.k_s = a.d_ff_shared;
    p.n_seg_s = a.n_shared;
    p.a_scale_r = a.h_scale;
    p.a_scale_s = a.h_shared_scale;
    p.b0_scale_r = p.b1_scale_r = a.w.w_down_scale;
    p.b0_scale_s = p.b1_scale_s = a.w.ws_down_scale;
    p.out_r = a.y_perm;
    p.out_s = a.y_shared;
    return launch<EPI_STORE>(m, p, st);
}

}  // namespace moe
