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
// Weight channels lie on the MMA's M side and token rows on N, on pairs of SMs (a
// cluster of 2 CTAs, tcgen05.mma.cta_group::2, M = 256): a tile is one expert's
// 256 weight rows x up to 256 tokens, in steps of 32.  CTA r holds half of the
// weight rows (128 TMEM lanes) and loads half of the tokens, so a k block of 128
// codes brings 32 KB into each SM for 512 cycles of MMA at N = 256, and the two
// accumulators of 256 columns let the epilogue of a tile overlap the next one's
// products.  An expert's tokens are cut into equal tiles of at most 256, so at
// most 31 padding columns are computed per expert: with the tokens on M, in tiles
// of 128, a quarter of the MMA work of a 256-token expert was padding, and a
// decode step's (a few tokens per expert) nearly all of it.  An expert of little more
// than 256 tokens would have two small tiles that each load all its weights: the WIDE
// kernel makes one of them, over both accumulators; a k block then takes two stages, the
// second one with tokens only, and both products read the first one's weights.
//   GEMM1  a tile's 256 weight rows are 128 channels' gate and up rows, 16 and 16
//          in turn (one 16 KB TMA box over both tensors: boxes of 16 rows each made
//          this GEMM 1.5 times slower at a decode step, 1745 against 1149 us): one
//          half of a TMEM quarter's lanes holds a channel's gate, the other its up,
//          and one shuffle per two tokens joins them
//   GEMM2  256 channels; pairs of lanes exchange one of two tokens so that each
//          stores two neighbouring channels of one
// One persistent kernel per GEMM, 320 threads a CTA: warp 0 the TMA producer, warp
// 1 (of the leading CTA) the MMA issuer, warps 2..9 the epilogue.  Producer and issuer
// are converged warps of which one elected lane issues: under a test of the lane number
// each TMA and MMA instruction loops over the lanes, and a k block took 340 ns to issue
// where its products take 270.  Rows of a tile past its segment are computed and never
// stored.  Every wait on a barrier is bounded.
//
// Measured with d = 7168, 256 experts of d_ff 2048, K = 8 and one shared expert:
//   128 tokens   1.69 ms for 11.2 GB, 6.6 TB/s: HBM bounds it
//   1 token      79 us for 0.40 GB, 5.0 TB/s: the first loads of each GEMM and the last,
//                partly filled round of tiles (252 of GEMM2 over 74 pairs)
//   8192 tokens  3.8 to 4.2 ms (by the GPU), 1.6 POP/s: the power limit.  Back to back
//                passes run at 1.05 to 1.1 GHz, the first ones at up to 1.9 GHz.  Of 4.1 ms
//                before the wide tiles (which saved 0.23) the products alone would take 2.3
//                at the same power, the token loads cost 0.7, the weight loads 1.4,
//                epilogue and h 0.6
#include <cstring>

#include "kernels.h"

namespace moe {
namespace gemm_i8 {

constexpr int BK = 128;            // codes (bytes) per k block
constexpr int M_CTA = 128;         // weight rows of a CTA; the pair has twice as many
constexpr int N_MAX = 256;         // tokens of an accumulator
constexpr int WIDE_MAX = 2 * N_MAX;  // ... and of a tile that takes both
constexpr int N_STEP = 32;
constexpr int STAGES = 6;
constexpr int A_BYTES = M_CTA * BK;
constexpr int B_BYTES = N_MAX / 2 * BK;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 8;       // two per TMEM lane quarter, on alternate chunks of 32 tokens
constexpr int NUM_THREADS = 64 + EPI_WARPS * 32;
constexpr int TMEM_COLS = 512;
constexpr int MAX_E = 1024;
constexpr int SMEM_DYN = STAGES * STAGE_BYTES + 1024;

enum { EPI_SWIGLU = 0, EPI_STORE = 1 };
// output channels of a pair tile
template <int EPI>
__host__ __device__ constexpr int channels() { return EPI == EPI_SWIGLU ? M_CTA : 2 * M_CTA; }

struct Maps {
    CUtensorMap w_r, w_s;        // weights: gate and up as a pair, or down; 16 KB boxes
    CUtensorMap x_r[3], x_s[3];  // token codes [rows, k], boxes of 64, 32 and 16 rows
};

struct Params {
    const int32_t *offsets;
    int E, rows_r, T;            // T = 0: no shared experts
    int n_out_r, n_out_s;        // output channels
    int k_r, k_s;                // reduction lengths; the shared one is n_seg_s runs of k_s
    int n_seg_s;
    const float *x_scale_r, *x_scale_s;    // per token row
    // per channel, [E, n_out_r]: the first and the second 16 lanes' (GEMM1), or both
    // the same (GEMM2); gate_r, gate_s: which half holds the gate
    const float *w0_scale_r, *w1_scale_r, *w0_scale_s, *w1_scale_s;
    int gate_r, gate_s;
    void *out_r, *out_s;         // fp32 (SwiGLU) or bf16
    int early;                   // only the token codes and scales wait for the kernel before
    int32_t *status;
    int64_t timeout_ns;
};

struct Tile {
    int e;           // expert, or -1: the shared experts
    int c0;          // first channel of the pair
    int t0, valid;   // first token row, rows to store
    int n, n1;       // MMA columns of the first and the second (or 0) accumulator
    int kblocks;
};

// Token tiles of an expert: the fewest of at most N_MAX, equal up to N_STEP.  WIDE: a
// single one up to WIDE_MAX.
template <bool WIDE>
__device__ __forceinline__ int token_tiles(int cnt) {
    return WIDE && cnt <= WIDE_MAX ? cnt > 0 : (cnt + N_MAX - 1) / N_MAX;
}
template <bool WIDE>
__device__ __forceinline__ void token_range(int cnt, int tiles, int i, Tile &t) {
    const int units = (cnt + N_STEP - 1) / N_STEP;
    const int each = units / tiles, more = units - each * tiles;
    const int u0 = i * each + min(i, more);
    t.t0 = u0 * N_STEP;
    const int mine = each + (i < more);
    t.n1 = WIDE && mine * N_STEP > N_MAX ? mine / 2 * N_STEP : 0;
    t.n = mine * N_STEP - t.n1;
    t.valid = min(mine * N_STEP, cnt - t.t0);
}

template <int EPI, bool WIDE>
__device__ __forceinline__ Tile decode_tile(int idx, const int *tile_base, const int *seg,
                                            const int *segc, const Params &p, int ntr, int nc_s) {
    Tile t;
    if (idx < ntr) {
        int lo = 0, hi = p.E;  // tile_base[lo] <= idx < tile_base[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tile_base[mid] <= idx) lo = mid; else hi = mid;
        }
        const int cnt = segc[lo], nt = token_tiles<WIDE>(cnt);
        const int local = idx - tile_base[lo];
        const int c = local / nt;  // token tiles of the same weights side by side
        token_range<WIDE>(cnt, nt, local - c * nt, t);
        t.t0 += seg[lo];
        t.c0 = c * channels<EPI>();
        t.e = lo;
        t.kblocks = (p.k_r + BK - 1) / BK;
    } else {
        const int local = idx - ntr;
        const int i = local / nc_s;
        token_range<WIDE>(p.T, token_tiles<WIDE>(p.T), i, t);
        t.c0 = (local - i * nc_s) * channels<EPI>();
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

// A bounded wait by a converged warp: every lane sees the barrier's phase, and all
// agree on the outcome.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort,
                                          const Params &p) {
    return __all_sync(0xFFFFFFFFu,
                      mbar_wait_bounded(bar, parity, abort, p.status, p.timeout_ns));
}

__device__ __forceinline__ float silu_mul(float g, float u) {
    // approximate division (2 ulp; 0 where 1 + e^-g passes 2^126): the rounded one
    // branches, and the values of a chunk would not overlap
    return __fdividef(g, 1.0f + __expf(-g)) * u;
}

template <int EPI, bool WIDE>
__global__ void __launch_bounds__(NUM_THREADS, 1)
grouped_int8_kernel(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[STAGES];   // used in the leader
    __shared__ __align__(8) uint64_t empty_bar[STAGES];
    __shared__ __align__(8) uint64_t tfull_bar[2];
    __shared__ __align__(8) uint64_t tempty_bar[2];      // used in the leader
    __shared__ __align__(8) uint64_t done_bar;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;
    __shared__ int tile_base[MAX_E + 1], seg[MAX_E], segc[MAX_E];
    __shared__ __align__(16) float x_scale[EPI_WARPS][N_MAX];  // a copy per warp

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t smem0 = smem_u32(smem);
    volatile int *abort_flag = &abort_s;

    if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < STAGES; ++s) {
                mbar_init(smem_u32(&full_bar[s]), 1);
                mbar_init(smem_u32(&empty_bar[s]), 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&tfull_bar[b]), 1);
                mbar_init(smem_u32(&tempty_bar[b]), 2 * EPI_WARPS);
            }
            mbar_init(smem_u32(&done_bar), 1);
            abort_s = 0;
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc_pair<TMEM_COLS>(smem_u32(&tmem_base_s));
        tc_fence_before();
    } else if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&maps.w_r);
        for (int i = 0; i < 3; ++i) tma_prefetch_desc(&maps.x_r[i]);
    }
    // From here on the kernel reads what the ones before it wrote.  Where the kernel
    // right before only writes the token codes and scales, the first weights are
    // requested while it still runs.
    if (!p.early) dependency_wait();
    dependency_release();
    for (int e = threadIdx.x; e < p.E; e += NUM_THREADS) {
        int lo = __ldcg(p.offsets + e), cnt = 0;
        const int64_t n = (int64_t)__ldcg(p.offsets + e + 1) - lo;
        // a segment that leaves the buffer or has a negative length is treated as
        // empty and reported
        if (lo < 0 || n < 0 || lo + n > p.rows_r) {
            record_status(p.status, MOE_ERR_DEVICE_FAULT);
            lo = 0;
        } else {
            cnt = (int)n;
        }
        seg[e] = lo;
        segc[e] = cnt;
    }
    __syncthreads();
    if (warp == 0) {
        // tile_base[e] = sum over experts < e of (token tiles x channel blocks): a lane
        // sums the experts of its share, the warp the shares
        const int nc_r = (p.n_out_r + channels<EPI>() - 1) / channels<EPI>();
        const int per = (p.E + 31) / 32;
        const int e0 = min(p.E, lane * per), e1 = min(p.E, e0 + per);
        int mine = 0;
        for (int e = e0; e < e1; ++e) mine += token_tiles<WIDE>(segc[e]) * nc_r;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += n;
        }
        int at = incl - mine;
        for (int e = e0; e < e1; ++e) {
            tile_base[e] = at;
            at += token_tiles<WIDE>(segc[e]) * nc_r;
        }
        if (lane == 31) tile_base[p.E] = incl;
    }
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers are initialised and TMEM is allocated
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_s;

    const int ntr = tile_base[p.E];
    const int nc_s = p.T > 0 ? (p.n_out_s + channels<EPI>() - 1) / channels<EPI>() : 0;
    const int total = ntr + (p.T > 0 ? token_tiles<WIDE>(p.T) * nc_s : 0);
    const int pair_id = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer (both CTAs)
        // The whole warp walks the tiles and waits; one elected lane issues.
        int stage = 0;
        uint32_t phase = 0, n_issued = 0;
        bool ok = true;
        const uint32_t full0 = mapa_shared(smem_u32(&full_bar[0]), 0);  // the leader's
        for (int idx = pair_id; idx < total && ok; idx += n_pairs) {
            const Tile t = decode_tile<EPI, WIDE>(idx, tile_base, seg, segc, p, ntr, nc_s);
            const bool shared = t.e < 0;
            const CUtensorMap *w = shared ? &maps.w_s : &maps.w_r;
            const CUtensorMap *x = shared ? maps.x_s : maps.x_r;
            const int k_len = shared ? p.k_s : p.k_r;
            const int ch = t.c0 + rank * (channels<EPI>() / 2);
            const int runs = WIDE && t.n1 ? 2 : 1;  // stages of a k block
            int mat = shared ? 0 : t.e, k = 0, x_col = 0;
            const uint32_t tx = 2 * A_BYTES + (uint32_t)t.n * BK;
            auto load_weights = [&](int s) {
                const uint32_t fb = full0 + 8 * s, a_dst = smem0 + s * STAGE_BYTES;
                if (leader) mbar_arrive_expect_tx(smem_u32(&full_bar[s]), tx);
                if (EPI == EPI_SWIGLU)
                    tma_load_5d_pair(a_dst, w, fb, k, 0, 0, ch / 16, mat);
                else
                    tma_load_3d_pair(a_dst, w, fb, k, ch, mat);
            };
            // a run's last block may pass its end: the weights read zeros there
            auto advance = [&] {
                k += BK;
                if (shared && k >= k_len) {
                    k = 0;
                    ++mat;
                    x_col += k_len;
                }
            };
            int ahead = 0;  // k blocks of the first tile whose weights are on their way
            if (p.early && idx == pair_id) {
                for (; ahead < min(STAGES / runs, t.kblocks); ++ahead) {
                    if (elect_one()) load_weights(ahead * runs);
                    __syncwarp();
                    advance();
                }
                mat = shared ? 0 : t.e, k = 0, x_col = 0;
                dependency_wait();
            }
            // this CTA's half of an accumulator's tokens as boxes of 64, 32 and 16 rows
            auto load_tokens = [&](int first, int half) {
                const uint32_t fb = full0 + 8 * stage;
                const uint32_t b_dst = smem0 + stage * STAGE_BYTES + A_BYTES;
                const int r32 = half & ~63, r16 = half & ~31, tok = first + rank * half;
                if (half & 16) tma_load_2d_pair(b_dst + r16 * BK, x + 2, fb, x_col + k, tok + r16);
                if (half & 32) tma_load_2d_pair(b_dst + r32 * BK, x + 1, fb, x_col + k, tok + r32);
                if (half >= 64) tma_load_2d_pair(b_dst, x, fb, x_col + k, tok);
                if (half == 128) tma_load_2d_pair(b_dst + 64 * BK, x, fb, x_col + k, tok + 64);
            };
            for (int kb = 0; kb < t.kblocks; ++kb) {
                if (!warp_wait(smem_u32(&empty_bar[stage]), phase ^ 1u, abort_flag, p)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    if (kb >= ahead) load_weights(stage);
                    load_tokens(t.t0, t.n / 2);
                }
                __syncwarp();
                ++n_issued;
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                if (WIDE && t.n1) {
                    if (!warp_wait(smem_u32(&empty_bar[stage]), phase ^ 1u, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        if (leader) mbar_arrive_expect_tx(smem_u32(&full_bar[stage]), t.n1 * BK);
                        load_tokens(t.t0 + t.n, t.n1 / 2);
                    }
                    __syncwarp();
                    ++n_issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                advance();
            }
        }
        if (p.early && pair_id >= total) dependency_wait();
        // Wind down: every load of both CTAs has landed (the leader's barriers count both),
        // and every stage's last release has arrived in this CTA.  The commits behind those
        // releases are arrivals from the leader's tensor core, in both CTAs and asynchronous:
        // no barrier of the threads orders them, and one that came late would hit the shared
        // memory of a CTA that is gone or of the block in its place.  Where a wait ran out,
        // no commit of the last two seconds is under way, and stages may never be released.
        for (int s = 0; s < min(STAGES, (int)n_issued); ++s) {
            const uint32_t last = ((n_issued - 1 - s) / STAGES) & 1u;  // parity of its last use
            if (leader) drain_wait(smem_u32(&full_bar[s]), last, p.timeout_ns, p.status);
            ok = ok && warp_wait(smem_u32(&empty_bar[s]), last, abort_flag, p);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer (leader)
        // The whole warp walks the tiles and waits; one elected lane issues.
        if (leader) {
            int stage = 0;
            uint32_t phase = 0, use = 0;  // accumulators so far, in turn
            bool ok = true;
            for (int idx = pair_id; idx < total && ok; idx += n_pairs) {
                const Tile t = decode_tile<EPI, WIDE>(idx, tile_base, seg, segc, p, ntr, nc_s);
                const uint32_t idesc = idesc_s8_s32(2 * M_CTA, t.n);
                const uint32_t idesc1 = idesc_s8_s32(2 * M_CTA, t.n1);
                const uint32_t d_tmem = tmem_base + (use & 1u) * N_MAX;
                const uint32_t d1_tmem = tmem_base + (~use & 1u) * N_MAX;
                if (!warp_wait(smem_u32(&tempty_bar[use & 1u]), (use >> 1 & 1u) ^ 1u, abort_flag, p))
                    break;
                for (int kb = 0; kb < t.kblocks; ++kb) {
                    if (!warp_wait(smem_u32(&full_bar[stage]), phase, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int first = stage;
                    const uint32_t a_addr = smem0 + stage * STAGE_BYTES;
                    const uint64_t a_desc = smem_desc_sw128(a_addr);
                    if (elect_one()) {
                        const uint64_t b_desc = smem_desc_sw128(a_addr + A_BYTES);
#pragma unroll
                        for (int ks = 0; ks < BK / 32; ++ks)
                            tc_mma_s8_pair(d_tmem, a_desc + 2 * ks, b_desc + 2 * ks, idesc,
                                           (kb | ks) != 0 ? 1u : 0u);
                        if (!WIDE || !t.n1) tc_commit_pair_both(smem_u32(&empty_bar[stage]));
                    }
                    __syncwarp();
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (WIDE && t.n1) {  // the same weights with the second accumulator's tokens
                        if ((kb == 0 && !warp_wait(smem_u32(&tempty_bar[~use & 1u]),
                                                   ((use + 1) >> 1 & 1u) ^ 1u, abort_flag, p)) ||
                            !warp_wait(smem_u32(&full_bar[stage]), phase, abort_flag, p)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t b_desc =
                                smem_desc_sw128(smem0 + stage * STAGE_BYTES + A_BYTES);
#pragma unroll
                            for (int ks = 0; ks < BK / 32; ++ks)
                                tc_mma_s8_pair(d1_tmem, a_desc + 2 * ks, b_desc + 2 * ks, idesc1,
                                               (kb | ks) != 0 ? 1u : 0u);
                            tc_commit_pair_both(smem_u32(&empty_bar[first]));
                            tc_commit_pair_both(smem_u32(&empty_bar[stage]));
                        }
                        __syncwarp();
                        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    }
                }
                if (!ok) break;
                if (elect_one()) {
                    tc_commit_pair_both(smem_u32(&tfull_bar[use & 1u]));
                    if (WIDE && t.n1) tc_commit_pair_both(smem_u32(&tfull_bar[(use + 1) & 1u]));
                }
                __syncwarp();
                use += WIDE && t.n1 ? 2 : 1;
            }
            // wind down: every MMA issued has completed
            if (elect_one()) tc_commit_pair(smem_u32(&done_bar));
            __syncwarp();
            drain_wait(smem_u32(&done_bar), 0, p.timeout_ns, p.status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue (both CTAs)
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const int part = (warp - 2) >> 2;
        float *xs = x_scale[warp - 2];
        if (p.early) dependency_wait();
        uint32_t use = 0;
        int second = 0;  // the tokens that a tile's second accumulator has yet
        for (int idx = pair_id; idx < total; idx += WIDE && second ? 0 : n_pairs, ++use) {
            Tile t = decode_tile<EPI, WIDE>(idx, tile_base, seg, segc, p, ntr, nc_s);
            const uint32_t acc = use & 1u;
            if (WIDE && second) {
                t.t0 += t.n;
                t.valid -= t.n;
                t.n = t.n1;
                second = 0;
            } else if (WIDE) {
                second = t.n1;
                t.valid = min(t.valid, t.n);
            }
            const bool shared = t.e < 0;
            const int n_out = shared ? p.n_out_s : p.n_out_r;
            const float *xs_g = (shared ? p.x_scale_s : p.x_scale_r) + t.t0;
            for (int j = lane; j < t.n; j += 32) xs[j] = j < t.valid ? __ldcg(xs_g + j) : 0.f;
            // this lane's channel (whole warps are inside or outside n_out, a multiple of 64)
            const int ch = EPI == EPI_SWIGLU ? t.c0 + rank * 64 + q * 16 + (lane & 15)
                                             : t.c0 + rank * 128 + q * 32 + lane;
            const bool ch_ok = ch < n_out;
            float ws = 0.f;
            if (ch_ok) {
                const float *s0 = shared ? p.w0_scale_s : p.w0_scale_r;
                const float *s1 = shared ? p.w1_scale_s : p.w1_scale_r;
                ws = (EPI == EPI_SWIGLU && lane >= 16 ? s1 : s0)[(size_t)(shared ? 0 : t.e) * n_out +
                                                                 ch];
            }
            __syncwarp();
            // (the TMEM loads want the warp together)
            if (!warp_wait(smem_u32(&tfull_bar[acc]), use >> 1 & 1u, abort_flag, p)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * N_MAX;
            // which of two neighbouring tokens this lane stores
            const int mine = EPI == EPI_SWIGLU ? lane >> 4 : lane & 1;
            const int partner = EPI == EPI_SWIGLU ? 16 : 1;
            // whether this lane's own accumulator is the gate
            const bool own_gate = mine == (shared ? p.gate_s : p.gate_r);
#pragma unroll 1
            for (int c = part * 32; c < t.valid; c += EPI_WARPS / 4 * 32) {
                uint32_t r[32];
                tmem_ld32(taddr + c, r);
                tc_wait_ld();
                if (!ch_ok) continue;
                // the values of a chunk first, free of branches, so that their shuffles and
                // exponentials overlap; then its stores
                uint32_t o[16];
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 s4 = *reinterpret_cast<const float4 *>(xs + c + j);
                    const float sx[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                    for (int h = 0; h < 4; h += 2) {
                        const float a = (float)(int)r[j + h] * sx[h] * ws;
                        const float b = (float)(int)r[j + h + 1] * sx[h + 1] * ws;
                        const float got = __shfl_xor_sync(0xFFFFFFFFu, mine ? a : b, partner);
                        const float own = mine ? b : a;
                        if (EPI == EPI_SWIGLU)
                            o[(j + h) / 2] = __float_as_uint(silu_mul(own_gate ? own : got,
                                                                      own_gate ? got : own));
                        else
                            o[(j + h) / 2] = mine ? pack_bf16x2(got, own) : pack_bf16x2(own, got);
                    }
                }
                // fp32: one channel; bf16: two, a 4-byte word either way
                const size_t words = EPI == EPI_SWIGLU ? (size_t)n_out : (size_t)n_out / 2;
                uint32_t *dst = static_cast<uint32_t *>(shared ? p.out_s : p.out_r) +
                                (size_t)(t.t0 + c + mine) * words +
                                (EPI == EPI_SWIGLU ? ch : ch / 2);
                if (c + 32 <= t.valid) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) dst[2 * j * words] = o[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + 2 * j + mine < t.valid) dst[2 * j * words] = o[j];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty_bar[acc]), 0));
        }
    }

    tc_fence_before();
    __syncthreads();
    // the leader's MMAs into this CTA's TMEM, every load into this CTA's shared memory
    // and every arrival on its barriers are done before either CTA frees TMEM or exits
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair<TMEM_COLS>(tmem_base);
    }
    __syncwarp();
    cluster_sync_all();  // neither CTA is gone while the other still frees the pair's TMEM
}

namespace {
int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    return sms;
}

template <int EPI>
cudaError_t launch(const Maps &maps, const Params &p, const FfnInt8Args &a, cudaStream_t st) {
    const int sms = sm_count() / 2 * 2;
    // Wide tiles pay where most experts have 257 to 512 tokens or little less, whose
    // weights would be loaded twice and in smaller tiles, where the reduction is long (an
    // epilogue no longer runs beside the next tile's products) and where each pair gets
    // many tiles (they are coarser).  us without and with:
    //   256 experts of 7168 x 2048, K = 8: 8192 tokens 4230 4040, 9216 4980 4370, 12288
    //   5820 5250; in both products 4096 2400 2530 and 16384 (512 an expert and more) 6910
    //   7600 (64 of 2048 x 1408, 4096 tokens of 6: 320 360; 32 of 7168 x 2048, 1024 of 8:
    //   424 469)
    const int64_t rows = (int64_t)a.T * a.K, blocks = (p.n_out_r + channels<EPI>() - 1) / channels<EPI>();
    const bool wide = rows >= 192ll * a.E && rows <= 448ll * a.E && p.k_r >= 32 * BK &&
                      a.E * blocks >= 32ll * (sms / 2);
    auto kern = wide ? grouped_int8_kernel<EPI, true> : grouped_int8_kernel<EPI, false>;
    cudaError_t err =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_DYN);
    if (err != cudaSuccess) return err;
    // one wave of pairs, one CTA per SM (pairs that do not fit at once would take
    // their share of the tiles later)
    return launch_dependent(kern, sms, NUM_THREADS, SMEM_DYN, 2, st, maps, p);
}

// Token codes [rows, cols] in boxes of 64, 32 and 16 rows.
bool token_maps(CUtensorMap *x, const int8_t *q, uint64_t rows, uint64_t cols) {
    return tensor_map_2d_u8(x, q, rows, cols, BK, 64, 128) &&
           tensor_map_2d_u8(x + 1, q, rows, cols, BK, 32, 128) &&
           tensor_map_2d_u8(x + 2, q, rows, cols, BK, 16, 128);
}
// Gate and up codes [n_mat, rows, cols] as a pair, the lower address first;
// *gate: the place of the gate.
bool gate_up_map(CUtensorMap *m, const int8_t *gate_w, const int8_t *up_w, uint64_t n_mat,
                 uint64_t rows, uint64_t cols, int *gate) {
    *gate = gate_w < up_w ? 0 : 1;
    const int8_t *first = *gate ? up_w : gate_w, *second = *gate ? gate_w : up_w;
    return tensor_map_pair_u8(m, first, (uint64_t)(second - first), n_mat, rows, cols, BK, 16, 4);
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
    Params p{};
    bool ok = token_maps(m.x_r, a.x_perm_q, rows, a.d) &&
              gate_up_map(&m.w_r, a.w.w_gate, a.w.w_up, a.E, a.d_ff, a.d, &p.gate_r);
    if (has_shared)
        ok = ok && token_maps(m.x_s, a.x_q, a.T, a.d) &&
             gate_up_map(&m.w_s, a.w.ws_gate, a.w.ws_up, 1, ffs, a.d, &p.gate_s);
    if (!ok) return cudaErrorInvalidValue;
    p.offsets = a.offsets;
    p.E = a.E;
    p.rows_r = (int)rows;
    p.T = has_shared ? a.T : 0;
    p.n_out_r = a.d_ff;
    p.n_out_s = ffs;
    p.k_r = p.k_s = a.d;
    p.n_seg_s = 1;
    p.x_scale_r = a.x_scale;
    p.x_scale_s = a.x_q_scale;
    p.w0_scale_r = p.gate_r ? a.w.w_up_scale : a.w.w_gate_scale;
    p.w1_scale_r = p.gate_r ? a.w.w_gate_scale : a.w.w_up_scale;
    p.w0_scale_s = p.gate_s ? a.w.ws_up_scale : a.w.ws_gate_scale;
    p.w1_scale_s = p.gate_s ? a.w.ws_gate_scale : a.w.ws_up_scale;
    p.out_r = a.h;
    p.out_s = a.h_shared;
    p.status = a.status;
    p.timeout_ns = a.timeout_ns;
    p.early = a.after_quantize;
    cudaError_t err = launch<EPI_SWIGLU>(m, p, a, st);
    if (err != cudaSuccess) return err;

    err = launch_quantize_rows_f32(a.h, (int64_t)rows, a.d_ff, a.h_q, a.h_scale, a.h_shared,
                                   has_shared ? a.T : 0, ffs, a.h_shared_q, a.h_shared_scale, st);
    if (err != cudaSuccess) return err;

    std::memset(&m, 0, sizeof(m));
    ok = token_maps(m.x_r, a.h_q, rows, a.d_ff) &&
         tensor_map_3d_u8(&m.w_r, a.w.w_down, a.E, a.d, a.d_ff, BK, M_CTA, 128);
    if (has_shared)
        ok = ok && token_maps(m.x_s, a.h_shared_q, a.T, ffs) &&
             tensor_map_3d_u8(&m.w_s, a.w.ws_down, a.n_shared, a.d, a.d_ff_shared, BK, M_CTA, 128);
    if (!ok) return cudaErrorInvalidValue;
    p.n_out_r = p.n_out_s = a.d;
    p.k_r = a.d_ff;
    p.k_s = a.d_ff_shared;
    p.n_seg_s = a.n_shared;
    p.x_scale_r = a.h_scale;
    p.x_scale_s = a.h_shared_scale;
    p.w0_scale_r = p.w1_scale_r = a.w.w_down_scale;
    p.w0_scale_s = p.w1_scale_s = a.w.ws_down_scale;
    p.out_r = a.y_perm;
    p.out_s = a.y_shared;
    p.early = 1;  // (behind the quantization of h)
    return launch<EPI_STORE>(m, p, a, st);
}

}  // namespace moe
