// The matrix product with bias, activation and residual in its epilogue, and
// its gradients, on the 5th-generation tensor cores:
//   z = x W^T + b, y = act(z) + r            x: m x k, W: n x k
//   dz = dy act'(z), dx = dz W, dW = dz^T x, db = sum over rows of dz
// and the gated form with two weights,
//   y = act(x Wg^T + bg) (x Wu^T + bu), dx = dzg Wg + dzu Wu, dWg = dzg^T x, dWu = dzu^T x
// All products are one kernel, D(i, j) = sum_k A(i, k) B(j, k), for
// operands that are contiguous along k ("K-major": x and W forward, dz for
// dx) or along their rows ("MN-major": W for dx, both for dW), so nothing is
// transposed in memory.  kind::f16 MMAs of 128 x BN x 16 with float32
// accumulators in TMEM; operands come by TMA in 128-byte swizzled tiles of 64
// along k, zero-filled beyond the matrices' ends, so ragged sizes need no
// code in the main loop.
//
// Warp roles (320 threads, persistent over the output tiles): warp 0 issues
// the TMA loads into a ring of stages, warp 1 the MMAs (one thread), warps 2-9
// drain the accumulator while the next tile's MMAs fill the other half of TMEM.
// Products with fewer tiles than SMs are split along k: each part leaves its
// float32 partial sums in the workspace and a second kernel adds them in a
// fixed order and applies the epilogue.  Every mbarrier wait is bounded: on
// give-up the kernel raises the handle's status word, stops all roles, waits
// (bounded) for its own copies and MMAs and frees TMEM.
#pragma once

#include <algorithm>

#include "linear.cuh"
#include "tcgen05.cuh"

namespace {

using namespace zs;

constexpr int BM = 128;       // rows of an output tile
constexpr int BK = 64;        // k values of a stage: 128 bytes, one swizzle row
constexpr int kDrain = 8;  // epilogue warps: two for each quarter of the TMEM lanes
constexpr int kThreads = 64 + 32 * kDrain;
constexpr uint32_t kTmemCols = 512;

constexpr int BN = 128;       // columns of an output tile of one CTA
// Bytes in which the epilogue warps turn their values over where the results' rows
// start anywhere.  Those kernels are apart: the others need the registers, and L1, whose
// room this takes, for the other half of each sector of the residual (8192 x 8192 x 1024:
// 125 us, 134 with both ways in one kernel, 166 with the memory taken as well).
constexpr int kTurn = kDrain * 32 * kTurnLd * 4;
inline bool turned(const Epilogue &e) { return !e.vec && !e.part; }
struct Cfg {
    static constexpr int A_BYTES = BM * BK * 2;
    static constexpr int B_BYTES = BN * BK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = 6;
    static constexpr int SMEM = STAGES * STAGE + 1024;  // + alignment slack
};

constexpr uint32_t kBox = 64 * 128;  // bytes of an MN-major box: 64 k rows
template <bool MN>
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) { return zs::smem_desc<MN>(addr, kBox); }

// ---------------------------------------------------------------- the gated form

// What the products of the gated form have beside the plain ones' arguments.  dzg
// and dzu are the halves of one matrix, `apart` columns from one to the other (a multiple of a
// tile's rows): dx is a sum over the k blocks of the first half and then over those of
// the second, whose other factor is the second weight; dW has the rows of both
// halves, and a tile's rows are of one of them.
enum { GLU_NONE, GLU_FWD, GLU_DX, GLU_DW };
struct GluMore {
    CUtensorMap b2;   // forward, dx: the second weight
    Epilogue second;  // dW: that of the second weight's gradient
    int64_t rows;     // dW: rows of each weight
    int apart;
    int kfirst;       // dx: k blocks of the first half
};
struct Nothing {};
template <int GLU>
using MoreOf = typename std::conditional<GLU != GLU_NONE, GluMore, Nothing>::type;
template <int GLU>
using EpiOf = typename std::conditional<GLU == GLU_FWD, GluEpilogue, Epilogue>::type;
inline bool turned(const GluEpilogue &e) { return !e.vec && !e.part; }

// ---------------------------------------------------------------- product

// Output tile t of the launch: bands of kBand row tiles, column by column
// within a band, so that the blocks at work at one time share few operand
// rows and find most of them in L2.
constexpr int kBand = 16;
struct TileAt {
    int tm, tn, split;
};
__device__ __forceinline__ TileAt tile_at(int t, int mt, int nt) {
    TileAt x;
    const int per = mt * nt;
    x.split = t / per;
    t -= x.split * per;
    const int band = t / (kBand * nt), in = t - band * kBand * nt;
    const int rows = min(kBand, mt - band * kBand);
    x.tm = band * kBand + in % rows;
    x.tn = in / rows;
    return x;
}

// One warp's part of a finished accumulator: 32 rows (a lane a row), CHUNKS x 32
// columns from `col` on.  ready(): waits for the accumulator, false if that gave up;
// release(): called once it is read.  Four warps that loaded the residual and the bias
// where they were added took 20 us for a 128 x 256 part, more than the MMAs of 4096 k
// values; eight that load a step ahead: 8192 x 8192 x 1024 with SiLU 318 -> 125 us,
// 8192 x 8192 x 4096 364 -> 324.
// TURN: for rows of results that start anywhere (5000 x 1001 x 700: 96 us with a row's
// values stored one by one by its lane, 46 so).
template <typename T, int CHUNKS, bool TURN, typename Ready, typename Release>
__device__ __forceinline__ bool drain(const Epilogue &epi, int64_t M, int64_t N, int64_t row, int64_t col, int split,
                                      uint32_t taddr, float *turn, Ready ready, Release release) {
    Ahead<T> in;
    auto whole = [&](int64_t c) { return !TURN && row < M && c + 32 <= N && epi.vec && !epi.part; };
    if (whole(col)) in.load(epi, row, col);
    if (!ready()) return false;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int c = 0; c < CHUNKS; c++, col += 32) {
        float v[32];
        __syncwarp();  // lanes beyond the last row come back
        tmem_ld32(taddr + (uint32_t)(c * 32), v);
        if (c == CHUNKS - 1) release();
        if (TURN) {
            if (row - lane < M && col < N)
                finish_turned<T>(epi, row - lane, (int)min((int64_t)32, M - (row - lane)), col,
                                 (int)min((int64_t)32, N - col), v, turn);
            continue;
        }
        if (whole(col)) {
            const Ahead<T> now = in;
            if (c + 1 < CHUNKS && whole(col + 32)) in.load(epi, row, col + 32);
            finish32<T>(epi, row, col, now, v);
            continue;
        }
        if (row >= M) continue;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int64_t cj = col + j * 8;
            const int nc = (int)min((int64_t)8, N - cj);
            if (nc <= 0) break;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; i++) f[i] = v[j * 8 + i];
            if (epi.part) {  // ldp is a multiple of 8 and the padding is ours
                float4 *p = reinterpret_cast<float4 *>(epi.part + ((int64_t)split * M + row) * epi.ldp + cj);
                p[0] = make_float4(f[0], f[1], f[2], f[3]);
                p[1] = make_float4(f[4], f[5], f[6], f[7]);
            } else {
                finish8<T>(epi, row, cj, nc, f);
            }
        }
    }
    return true;
}

// The same for the gated form: the gate's columns at taddr, the other factor's `apart`
// columns on.
template <typename T, int CHUNKS, bool TURN, typename Ready, typename Release>
__device__ __forceinline__ bool drain_glu(const GluEpilogue &epi, int64_t M, int64_t N, int64_t row, int64_t col, int split,
                                          uint32_t taddr, uint32_t apart, float *turn, Ready ready, Release release) {
    GluAhead<T> in;
    auto whole = [&](int64_t c) { return !TURN && row < M && c + 32 <= N && epi.vec && !epi.part; };
    if (whole(col)) in.load(epi, col);
    if (!ready()) return false;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int c = 0; c < CHUNKS; c++, col += 32) {
        float g[32], u[32];
        __syncwarp();  // lanes beyond the last row come back
        tmem_ld32(taddr + (uint32_t)(c * 32), g);
        tmem_ld32(taddr + apart + (uint32_t)(c * 32), u);
        if (c == CHUNKS - 1) release();
        if (TURN) {
            if (row - lane < M && col < N)
                glu_turned<T>(epi, row - lane, (int)min((int64_t)32, M - (row - lane)), col, (int)min((int64_t)32, N - col), g, u,
                              turn);
            continue;
        }
        if (whole(col)) {
            const GluAhead<T> now = in;
            if (c + 1 < CHUNKS && whole(col + 32)) in.load(epi, col + 32);
            glu_finish32<T>(epi, row, col, now, g, u);
            continue;
        }
        if (row >= M) continue;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int64_t cj = col + j * 8;
            const int nc = (int)min((int64_t)8, N - cj);
            if (nc <= 0) break;
            float f[8], h[8];
#pragma unroll
            for (int i = 0; i < 8; i++) f[i] = g[j * 8 + i], h[i] = u[j * 8 + i];
            if (epi.part) {  // ldp is a multiple of 8 and the padding is ours
                float *q = epi.part + ((int64_t)split * M + row) * 2 * epi.ldp + cj;
                float4 *p = reinterpret_cast<float4 *>(q);
                p[0] = make_float4(f[0], f[1], f[2], f[3]);
                p[1] = make_float4(f[4], f[5], f[6], f[7]);
                p = reinterpret_cast<float4 *>(q + epi.ldp);
                p[0] = make_float4(h[0], h[1], h[2], h[3]);
                p[1] = make_float4(h[4], h[5], h[6], h[7]);
            } else {
                glu_finish8<T>(epi, row, cj, nc, f, h);
            }
        }
    }
    return true;
}

// GLU: the plain product, or one of the gated form's.  Its forward tiles are 64 columns of each
// of the two products, side by side.
template <typename T, bool A_MN, bool B_MN, bool TURN, int GLU>
__global__ void __launch_bounds__(kThreads, 1)
k_linear_tc(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, int64_t M, int64_t N,
            int kblocks, int splits, const EpiOf<GLU> epi, unsigned *__restrict__ status,
            const __grid_constant__ MoreOf<GLU> more) {
    using C = Cfg;
    constexpr int TN = GLU == GLU_FWD ? BN / 2 : BN;  // columns of the result that a tile has
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[C::STAGES], bar_empty[C::STAGES], bar_accf[2], bar_acce[2], bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mt = (int)((M + BM - 1) / BM), nt = (int)((N + TN - 1) / TN);
    const int total = mt * nt * splits;
    // kind::f16: D float32, A and B of one type, majors, N, M
    constexpr uint32_t fmt = sizeof(T) == 2 && std::is_same<T, bf16>::value ? 1u : 0u;
    constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((A_MN ? 1u : 0u) << 15) |
                               ((B_MN ? 1u : 0u) << 16) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);

    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < C::STAGES; s++) {
            bar_init(&bar_full[s], 1);
            bar_init(&bar_empty[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            bar_init(&bar_accf[b], 1);
            bar_init(&bar_acce[b], kDrain);
        }
        bar_init(&bar_drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    after_previous();
    may_start_next();
    const uint32_t tmem = s_tmem;
    // k blocks of split s: an equal share, the first ones one more
    auto kfirst = [&](int s) { return (int)((int64_t)kblocks * s / splits); };

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&amap) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&bmap) : "memory");
            uint32_t g = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const TileAt x = tile_at(t, mt, nt);
                const int k1 = kfirst(x.split + 1);
                for (int kb = kfirst(x.split); kb < k1; kb++, g++) {
                    const uint32_t st = g % C::STAGES, ph = (g / C::STAGES) & 1u;
                    if (!bar_wait(&bar_empty[st], ph ^ 1u, &s_abort, status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&bar_full[st]);
                    bar_expect(&bar_full[st], C::STAGE);
                    const uint32_t sa = base + st * C::STAGE, sb = sa + C::A_BYTES;
                    if (A_MN) {
#pragma unroll
                        for (int i = 0; i < BM / 64; i++)
                            tma_load_2d(sa + i * kBox, &amap, x.tm * BM + i * 64, kb * BK, fb);
                    } else {
                        int ca = kb * BK;
                        if constexpr (GLU == GLU_DX)
                            if (kb >= more.kfirst) ca = more.apart + (kb - more.kfirst) * BK;
                        tma_load_2d(sa, &amap, ca, x.tm * BM, fb);
                    }
                    if constexpr (GLU == GLU_FWD) {
                        tma_load_2d(sb, &bmap, kb * BK, x.tn * TN, fb);
                        tma_load_2d(sb + TN * BK * 2, &more.b2, kb * BK, x.tn * TN, fb);
                    } else if (B_MN) {
                        const CUtensorMap *mb = &bmap;
                        int rb = kb * BK;
                        if constexpr (GLU == GLU_DX)
                            if (kb >= more.kfirst) mb = &more.b2, rb = (kb - more.kfirst) * BK;
#pragma unroll
                        for (int i = 0; i < BN / 64; i++)
                            tma_load_2d(sb + i * kBox, mb, x.tn * BN + i * 64, rb, fb);
                    } else {
                        tma_load_2d(sb, &bmap, kb * BK, x.tn * BN, fb);
                    }
                }
            }
            // our own copies in flight: wait (bounded) for the last stages to land
            for (uint32_t q = g > (uint32_t)C::STAGES ? g - C::STAGES : 0; q < g; q++) {
                uint32_t it = 0;
                while (!bar_try(&bar_full[q % C::STAGES], (q / C::STAGES) & 1u) && ++it < kWaitLimit) {
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (lane == 0) {
            uint32_t g = 0, it = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x, it++) {
                const TileAt x = tile_at(t, mt, nt);
                const int k0 = kfirst(x.split), k1 = kfirst(x.split + 1);
                const uint32_t buf = it & 1u, aph = (it >> 1) & 1u;
                if (!bar_wait(&bar_acce[buf], aph ^ 1u, &s_abort, status)) break;
                tc_fence_after();
                const uint32_t d = tmem + buf * 256u;
                for (int kb = k0; kb < k1; kb++, g++) {
                    const uint32_t st = g % C::STAGES, ph = (g / C::STAGES) & 1u;
                    if (!bar_wait(&bar_full[st], ph, &s_abort, status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = base + st * C::STAGE, sb = sa + C::A_BYTES;
#pragma unroll
                    for (int ks = 0; ks < BK / 16; ks++)  // 16 k: 32 bytes of a K-major row, 16 rows of an MN-major box
                        mma_f16(d, smem_desc<A_MN>(sa + ks * (A_MN ? 2048 : 32)),
                                smem_desc<B_MN>(sb + ks * (B_MN ? 2048 : 32)), idesc, (kb > k0 || ks) ? 1u : 0u);
                    mma_commit(smem_u32(&bar_empty[st]));  // stage free once these MMAs finish
                }
                if (!ok) break;
                mma_commit(smem_u32(&bar_accf[buf]));  // accumulator ready
            }
            // every MMA issued so far completes before TMEM is freed
            mma_commit(smem_u32(&bar_drain));
            uint32_t w = 0;
            while (!bar_try(&bar_drain, 0) && ++w < kWaitLimit) {
            }
        }
    } else {
        // ------------------------------------------------ epilogue (warps 2-9)
        const int quad = warp & 3, half = (warp - 2) >> 2;  // TMEM lanes 32 quad .. 32 quad + 31, half the columns
        float *turn = reinterpret_cast<float *>(smem_raw + (base - smem_u32(smem_raw)) + C::STAGES * C::STAGE) + (warp - 2) * 32 * kTurnLd;
        uint32_t it = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x, it++) {
            const TileAt x = tile_at(t, mt, nt);
            const uint32_t buf = it & 1u, aph = (it >> 1) & 1u;
            auto ready = [&] {
                const bool in = __all_sync(0xffffffffu, bar_wait(&bar_accf[buf], aph, &s_abort, status));
                tc_fence_after();
                return in;
            };
            auto release = [&] {  // accumulator fully read: hand it back to the MMA warp
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&bar_acce[buf]);
            };
            const int64_t row = (int64_t)x.tm * BM + quad * 32 + lane, col = (int64_t)x.tn * TN + half * (TN / 2);
            const uint32_t at = tmem + buf * 256u + (uint32_t)(half * (TN / 2)) + ((uint32_t)(quad * 32) << 16);
            bool ok;
            if constexpr (GLU == GLU_FWD) {
                ok = drain_glu<T, TN / 64, TURN>(epi, M, N, row, col, x.split, at, TN, turn, ready, release);
            } else if constexpr (GLU == GLU_DW) {  // parts keep the rows of both halves
                const bool second = x.tm * BM >= more.apart && !epi.part;
                const Epilogue &e = second ? more.second : epi;
                ok = drain<T, BN / 64, TURN>(e, e.part ? M : e.y ? more.rows : 0, N, second ? row - more.apart : row, col, x.split, at,
                                             turn, ready, release);
            } else {
                ok = drain<T, BN / 64, TURN>(epi, M, N, row, col, x.split, at, turn, ready, release);
            }
            if (!ok) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// The same for large products on pairs of SMs (cta_group::2): a pair's MMA is 256
// x 256 x 16, each CTA holds its 128 rows of A and of B and drains its 128 rows of
// the result.  A CTA then stages 32 KB a k block for the 48 KB of a 128 x 256 tile
// of its own, and shared memory, which feeds the MMAs and takes the copies, no
// longer bounds the rate.  The leader's threads issue the MMAs and own the
// barriers of full stages and of free accumulators; a stage's release and a
// finished accumulator are told to both.  16384 x 8192 x 4096 with bias, SiLU and
// residual back to back: 732 us, 1500 TFLOP/s, where the power limit lowers the clock (a
// library's plain product: 1685).
constexpr int kPairStages = 6;
constexpr int kPairStage = 2 * BM * BK * 2;  // A and B rows of one CTA
constexpr int kPairSmem = kPairStages * kPairStage + 1024;
static_assert(kPairSmem + kTurn + 512 <= 232448 && Cfg::SMEM + kTurn + 512 <= 232448, "shared memory of a block");

__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(cluster_bar)
        : "memory");
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// arrive on the barrier at this offset in both CTAs
__device__ __forceinline__ void mma_commit_both(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One product, or two whose tiles are dealt together, so that the second fills the
// SMs that the first's last round leaves idle (both gradients of 8192 x 4096 x 2048:
// 193 us in two launches).
enum { PAIR_FWD, PAIR_DX, PAIR_DW, PAIR_GRADS,  // x W^T, dz W, dz^T x, and the last two together
       PAIR_GLU_FWD, PAIR_GLU_DX, PAIR_GLU_DW, PAIR_GLU_GRADS };  // the gated form's
template <int FORM>
constexpr bool pair_both() { return FORM == PAIR_GRADS || FORM == PAIR_GLU_GRADS; }
template <int FORM>
constexpr int pair_glu() { return FORM < PAIR_GLU_FWD ? GLU_NONE : FORM == PAIR_GLU_FWD ? GLU_FWD : GLU_DX; }  // the last for all gradients
struct PairSecond {
    CUtensorMap a, b;
    int64_t M, N;
    int kblocks;
    bool first_mn;  // A of the first product is stored k x M, that of this one M x k; or the reverse
    int extra;      // tiles of the second that a pair of SMs takes for a tile of the first it has fewer
    Epilogue epi;
};
// Tile i of pair p of the P, of products of t0 and t1 tiles: true, which product and
// which of its tiles; or false
template <bool TWO>
__device__ __forceinline__ bool pair_tile(int t0, int t1, int extra, int p, int P, int i, int *job, int *tile) {
    if (!TWO) {
        *job = 0;
        *tile = i * P + p;
        return *tile < t0;
    }
    const int more = t0 % P, own = t0 / P + (p < more);
    *job = i >= own;
    if (i < own) {
        *tile = i * P + p;
        return true;
    }
    const int r = i - own, fewer = P - more;
    if (p >= more && r < extra)
        *tile = r * fewer + p - more;
    else
        *tile = extra * fewer + (r - (p >= more ? extra : 0)) * P + p;
    return *tile < t1;
}

// FORM: which; the operands' orders and the one product's place are constants but for
// PAIR_GRADS (read from the arguments for all of them, x W^T took 834 us for 758 at
// 16384 x 8192 x 4096).
template <typename T, int FORM, bool TURN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
k_linear_pair(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, int64_t M0, int64_t N0,
              int kblocks0, const EpiOf<pair_glu<FORM>()> epi0, const __grid_constant__ PairSecond two, unsigned *__restrict__ status,
              const __grid_constant__ MoreOf<pair_glu<FORM>()> more) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[kPairStages], bar_empty[kPairStages], bar_accf[2], bar_acce[2], bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1u;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    constexpr uint32_t fmt = std::is_same<T, bf16>::value ? 1u : 0u;
    constexpr uint32_t shape = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(256 >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
    constexpr bool BOTH = pair_both<FORM>(), FWD2 = FORM == PAIR_GLU_FWD, GRAD2 = FORM > PAIR_GLU_FWD;
    constexpr bool b_mn = FORM != PAIR_FWD && !FWD2;
    constexpr int TN = FWD2 ? 128 : 256;  // columns of the result that a tile has: in the gated form of each product
    const int mt0 = (int)((M0 + 2 * BM - 1) / (2 * BM)), nt0 = (int)((N0 + TN - 1) / TN);
    const int mt1 = BOTH ? (int)((two.M + 2 * BM - 1) / (2 * BM)) : 0, nt1 = BOTH ? (int)((two.N + 255) / 256) : 0;
    int job, tile;
    auto next = [&](uint32_t i) {  // the pair's tile i, if there is one
        return pair_tile<BOTH>(mt0 * nt0, mt1 * nt1, BOTH ? two.extra : 0, pair, pairs, (int)i, &job, &tile);
    };
    auto place = [&] { return BOTH && job ? tile_at(tile, mt1, nt1) : tile_at(tile, mt0, nt0); };
    auto a_major = [&] { return BOTH ? two.first_mn == !job : FORM == PAIR_DW || FORM == PAIR_GLU_DW; };

    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < kPairStages; s++) {
            bar_init(&bar_full[s], 1);
            bar_init(&bar_empty[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            bar_init(&bar_accf[b], 1);
            bar_init(&bar_acce[b], 2 * kDrain);  // the epilogue warps of both CTAs
        }
        bar_init(&bar_drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are there before anything arrives on them
    tc_fence_after();
    after_previous();
    may_start_next();
    const uint32_t tmem = s_tmem;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer, of its CTA's rows
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&amap) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&bmap) : "memory");
            uint32_t g = 0;
            bool ok = true;
            for (uint32_t i = 0; ok && next(i); i++) {
                const TileAt x = place();
                const CUtensorMap *ma = BOTH && job ? &two.a : &amap, *mb = BOTH && job ? &two.b : &bmap;
                const int kblocks = BOTH && job ? two.kblocks : kblocks0;
                const bool a_mn = a_major();
                const int ra = x.tm * 2 * BM + (int)rank * BM, rb = x.tn * TN + (FWD2 ? 0 : (int)rank * 128);
                if constexpr (FWD2)  // the leader's half of the columns is the gate's
                    if (rank) mb = &more.b2;
                for (int kb = 0; kb < kblocks; kb++, g++) {
                    const uint32_t st = g % kPairStages, ph = (g / kPairStages) & 1u;
                    if (!bar_wait(&bar_empty[st], ph ^ 1u, &s_abort, status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = cluster_addr(smem_u32(&bar_full[st]), 0);
                    if (rank == 0) bar_expect(&bar_full[st], 2 * kPairStage);
                    const uint32_t sa = base + st * kPairStage, sb = sa + BM * BK * 2;
                    if (a_mn) {
                        tma_load_2d_pair(sa, ma, ra, kb * BK, fb);
                        tma_load_2d_pair(sa + kBox, ma, ra + 64, kb * BK, fb);
                    } else {
                        int ca = kb * BK;
                        if constexpr (GRAD2)
                            if (kb >= more.kfirst) ca = more.apart + (kb - more.kfirst) * BK;
                        tma_load_2d_pair(sa, ma, ca, ra, fb);
                    }
                    if (b_mn) {
                        int cb = kb * BK;
                        const CUtensorMap *m2 = mb;
                        if constexpr (GRAD2)
                            if (!a_mn && kb >= more.kfirst) m2 = &more.b2, cb = (kb - more.kfirst) * BK;
                        tma_load_2d_pair(sb, m2, rb, cb, fb);
                        tma_load_2d_pair(sb + kBox, m2, rb + 64, cb, fb);
                    } else {
                        tma_load_2d_pair(sb, mb, kb * BK, rb, fb);
                    }
                }
            }
            // the pair's copies in flight: the leader waits (bounded) for the last stages to land
            if (rank == 0)
                for (uint32_t q = g > (uint32_t)kPairStages ? g - kPairStages : 0; q < g; q++) {
                    uint32_t it = 0;
                    while (!bar_try(&bar_full[q % kPairStages], (q / kPairStages) & 1u) && ++it < kWaitLimit) {
                    }
                }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer, of the pair
        if (lane == 0 && rank == 0) {
            uint32_t g = 0, it = 0;
            bool ok = true;
            for (; ok && next(it); it++) {
                const int kblocks = BOTH && job ? two.kblocks : kblocks0;
                const bool a_mn = a_major();
                const uint32_t idesc = shape | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
                const uint64_t da = a_mn ? smem_desc<true>(0) : smem_desc<false>(0), db = b_mn ? smem_desc<true>(0) : smem_desc<false>(0);
                const uint32_t step_a = a_mn ? 2048 : 32, step_b = b_mn ? 2048 : 32;
                const uint32_t buf = it & 1u, aph = (it >> 1) & 1u;
                if (!bar_wait(&bar_acce[buf], aph ^ 1u, &s_abort, status)) break;
                tc_fence_after();
                const uint32_t d = tmem + buf * 256u;
                for (int kb = 0; kb < kblocks; kb++, g++) {
                    const uint32_t st = g % kPairStages, ph = (g / kPairStages) & 1u;
                    if (!bar_wait(&bar_full[st], ph, &s_abort, status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = base + st * kPairStage, sb = sa + BM * BK * 2;
#pragma unroll
                    for (int ks = 0; ks < BK / 16; ks++)
                        mma_f16_pair(d, da | ((sa + ks * step_a) >> 4 & 0x3FFF), db | ((sb + ks * step_b) >> 4 & 0x3FFF), idesc,
                                     (kb || ks) ? 1u : 0u);
                    mma_commit_both(smem_u32(&bar_empty[st]));
                }
                if (!ok) break;
                mma_commit_both(smem_u32(&bar_accf[buf]));
            }
            // every MMA issued so far completes before TMEM is freed
            mma_commit_pair(smem_u32(&bar_drain));
            uint32_t w = 0;
            while (!bar_try(&bar_drain, 0) && ++w < kWaitLimit) {
            }
        }
    } else {
        // ------------------------------------------------ epilogue (warps 2-9), of its CTA's rows
        const int quad = warp & 3, half = (warp - 2) >> 2;
        float *turn = reinterpret_cast<float *>(smem_raw + (base - smem_u32(smem_raw)) + kPairStages * kPairStage) + (warp - 2) * 32 * kTurnLd;
        uint32_t it = 0;
        for (; next(it); it++) {
            const TileAt x = place();
            const uint32_t buf = it & 1u, aph = (it >> 1) & 1u;
            auto ready = [&] {
                const bool in = __all_sync(0xffffffffu, bar_wait(&bar_accf[buf], aph, &s_abort, status));
                tc_fence_after();
                return in;
            };
            auto release = [&] {  // accumulator fully read: hand it back to the leader's MMA warp
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(cluster_addr(smem_u32(&bar_acce[buf]), 0));
            };
            const int64_t row = (int64_t)x.tm * 2 * BM + rank * BM + quad * 32 + lane, col = (int64_t)x.tn * TN + half * (TN / 2);
            const uint32_t at = tmem + buf * 256u + (uint32_t)(half * (TN / 2)) + ((uint32_t)(quad * 32) << 16);
            bool ok;
            if constexpr (FWD2) {
                ok = drain_glu<T, 2, TURN>(epi0, M0, N0, row, col, 0, at, TN, turn, ready, release);
            } else if constexpr (GRAD2) {
                const bool dw = a_major(), second = dw && x.tm * 2 * BM >= more.apart;
                const Epilogue &e = second ? more.second : BOTH && job ? two.epi : epi0;
                ok = drain<T, 4, TURN>(e, !dw ? BOTH && job ? two.M : M0 : e.y ? more.rows : 0, BOTH && job ? two.N : N0,
                                       second ? row - more.apart : row, col, 0, at, turn, ready, release);
            } else {
                ok = drain<T, 4, TURN>(BOTH && job ? two.epi : epi0, BOTH && job ? two.M : M0, BOTH && job ? two.N : N0, row, col, 0, at,
                                       turn, ready, release);
            }
            if (!ok) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still use its memory or barriers
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// The parts of a product split along k, `apart` rows each, added in order, and the
// epilogue; a thread for 8 columns of a row.  Bound by the latency of its loads, which L2 serves:
// 801 x 1000 in two parts 6 us, partly hidden behind the product's end.
template <typename T>
__global__ void __launch_bounds__(256)
k_linear_join(int64_t M, int64_t N, int splits, int64_t apart, const Epilogue epi) {
    after_previous();
    may_start_next();
    const int64_t groups = (N + 7) / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= M * groups) return;
    const int64_t row = i / groups, c = (i - row * groups) * 8;
    float v[8] = {};
    for (int s = 0; s < splits; s++) {
        const float4 *p = reinterpret_cast<const float4 *>(epi.part + (s * apart + row) * epi.ldp + c);
        const float4 a = p[0], b = p[1];
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
    finish8<T>(epi, row, c, (int)min((int64_t)8, N - c), v);
}

// Rows that TMA cannot address (base or row stride not a multiple of 16
// bytes) copied to rows that it can; 16-bit values, up to three matrices a launch.
struct PackJob {
    const uint16_t *src;
    uint16_t *dst;  // rows of whole 16 bytes
    int64_t ld, rows;
    int cols;
};
__global__ void __launch_bounds__(256)
k_linear_pack(const PackJob a, const PackJob b, const PackJob c3) {
    after_previous();
    may_start_next();
    const PackJob &j = blockIdx.y == 0 ? a : blockIdx.y == 1 ? b : c3;
    const int64_t ldd = (j.cols + 7) / 8 * 8, groups = ldd / 8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < j.rows * groups; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / groups;
        const int c = (int)(i - row * groups) * 8;
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; e++) u[e] = c + e < j.cols ? j.src[row * j.ld + c + e] : 0;
        *reinterpret_cast<uint4 *>(j.dst + row * ldd + c) =
            make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
    }
}

// The parts of the biases' gradients, added in order: `total` columns, the first n of them
// db's and the others db2's (either may be NULL).
template <typename T>
__global__ void __launch_bounds__(256)
k_linear_db(const float *__restrict__ parts, int nparts, int64_t total, int64_t n, T *__restrict__ db, T *__restrict__ db2) {
    __shared__ float red[8][32];
    after_previous();
    may_start_next();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    float s = 0.f;
    if (c < total)
        for (int p = ty; p < nparts; p += 8) s += parts[p * total + c];
    red[ty][tx] = s;
    __syncthreads();
    if (ty != 0 || c >= total) return;
#pragma unroll
    for (int r = 1; r < 8; r++) s += red[r][tx];
    T *to = c < n ? db : db2;
    if (to) to[c < n ? c : c - n] = from_f32<T>(s);
}

// ---------------------------------------------------------------- host

// Map of a matrix of `rows` rows of `cols` contiguous 16-bit values, row
// stride ld, in boxes of 64 values x box_rows.
cudaError_t encode(CUtensorMap *map, int type, const void *p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = get_encode();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    const CUresult r = enc(map, type == ZSOLVE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                           2, (void *)p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A 16-bit matrix as the kernels take it.
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
    bool tma_ok() const { return ((uintptr_t)p & 15) == 0 && ld % 8 == 0; }
    size_t packed_values() const { return (size_t)rows * ((cols + 7) / 8 * 8); }
};

// A product's tiles and parts along k.  Pairs of SMs on 256 x 256 tiles where
// there is a tile for every pair (and rows of tiles enough that a half empty last
// one does not matter), else single SMs on 128 x 128: four times the tiles.  Pairs
// against single SMs: 2048 x 2560 x 2048 (80 tiles for 76 pairs) 31.5 us and 38.2,
// 4096 x 4096 x 4096 95 and 153, 1100 x 4096 x 2048 (a last row of tiles 3/10 full)
// 30.7 and 27.5.  Parts are for what still leaves SMs idle, of 4 k blocks at least, so
// that a part's loads outweigh the pass that joins them.
struct Plan {
    bool pair;
    int splits, kblocks;
};
Plan plan_of(int64_t M, int64_t N, int64_t K, int num_sms) {
    Plan p;
    const int64_t mt = (M + BM - 1) / BM;
    p.kblocks = (int)((K + BK - 1) / BK);
    p.pair = (mt + 1) / 2 * ((N + 255) / 256) >= num_sms / 2 && (mt % 2 == 0 || mt >= 8);
    const int64_t tiles = mt * ((N + BN - 1) / BN);
    p.splits = p.pair ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>({num_sms / tiles, p.kblocks / 4, 32}));
    return p;
}
int64_t ld_part(int64_t N) { return (N + 7) / 8 * 8; }
size_t part_values(int64_t M, int64_t N, const Plan &p) {
    return p.splits > 1 ? (size_t)p.splits * M * ld_part(N) : 0;
}

template <typename T, bool A_MN, bool B_MN, bool TURN, int GLU = GLU_NONE>
cudaError_t launch_tc(const CUtensorMap &a, const CUtensorMap &b, int64_t M, int64_t N, const Plan &p,
                      const EpiOf<GLU> &epi, bool next, zsolve_seq *s, const MoreOf<GLU> &more = {}) {
    constexpr int TN = GLU == GLU_FWD ? BN / 2 : BN;
    constexpr int smem = Cfg::SMEM + (TURN ? kTurn : 0);
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_linear_tc<T, A_MN, B_MN, TURN, GLU>, smem);
    if (attr != cudaSuccess) return attr;
    const int64_t total = (M + BM - 1) / BM * ((N + TN - 1) / TN) * p.splits;
    s->launches++;
    return launch(next, k_linear_tc<T, A_MN, B_MN, TURN, GLU>, (unsigned)std::min<int64_t>(total, s->num_sms), kThreads, smem, s->st,
                  a, b, M, N, p.kblocks, p.splits, epi, s->d_status, more);
}

// D(i, j) = sum_k A(i, k) B(j, k) and the epilogue; a_mn: A is stored k x M, else M x k.
struct Product {
    int64_t M, N, K;
    Mat A, B;
    bool a_mn, b_mn;
    Epilogue epi;
};

cudaError_t maps(int type, const Product &p, CUtensorMap *a, CUtensorMap *b) {
    const cudaError_t e = encode(a, type, p.A.p, p.A.rows, p.A.cols, p.A.ld, p.a_mn ? 64 : BM);
    return e == cudaSuccess ? encode(b, type, p.B.p, p.B.rows, p.B.cols, p.B.ld, p.b_mn ? 64 : BN) : e;
}

// Products whose plan is pairs of SMs: one, or both gradients; the longer sums
// first, so that the last round is of short ones.
template <typename T, int FORM, bool TURN>
cudaError_t launch_pair_as(zsolve_seq *s, int type, const Product *p, bool next, const MoreOf<pair_glu<FORM>()> &more = {}) {
    constexpr int smem = kPairSmem + (TURN ? kTurn : 0);
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_linear_pair<T, FORM, TURN>, smem);
    if (attr != cudaSuccess) return attr;
    constexpr int n = pair_both<FORM>() ? 2 : 1;
    const int first = n == 2 && p[1].K > p[0].K;
    const Product &q = p[first];
    CUtensorMap ma, mb;
    cudaError_t e = maps(type, q, &ma, &mb);
    if (e != cudaSuccess) return e;
    auto tiles = [](const Product &p) { return (p.M + 2 * BM - 1) / (2 * BM) * ((p.N + 255) / 256); };
    auto kblocks = [](const Product &p) { return (int)((p.K + BK - 1) / BK); };
    int64_t total = tiles(q);
    PairSecond two{};
    if (n == 2) {
        const Product &r = p[first ^ 1];
        e = maps(type, r, &two.a, &two.b);
        if (e != cudaSuccess) return e;
        two.M = r.M, two.N = r.N, two.kblocks = kblocks(r);
        two.first_mn = q.a_mn, two.epi = r.epi;
        two.extra = kblocks(q) / kblocks(r);
        total += tiles(r);
    }
    const unsigned pairs = (unsigned)std::min<int64_t>(total, s->num_sms / 2);
    s->launches++;
    return launch(next, k_linear_pair<T, FORM, TURN>, 2 * pairs, kThreads, smem, s->st, ma, mb, q.M, q.N, kblocks(q), q.epi, two,
                  s->d_status, more);
}
template <typename T, int FORM>
cudaError_t launch_pair(zsolve_seq *s, int type, const Product *p, bool next, const MoreOf<pair_glu<FORM>()> &more = {}) {
    bool turn = turned(p[0].epi) || (pair_both<FORM>() && turned(p[1].epi));
    if constexpr (FORM == PAIR_GLU_DW || FORM == PAIR_GLU_GRADS) turn = turn || turned(more.second);
    return turn ? launch_pair_as<T, FORM, true>(s, type, p, next, more) : launch_pair_as<T, FORM, false>(s, type, p, next, more);
}

template <typename T>
cudaError_t product(zsolve_seq *s, int type, Product q, float *part, bool next) {
    const Plan p = plan_of(q.M, q.N, q.K, s->num_sms);
    if (p.pair)
        return !q.b_mn  ? launch_pair<T, PAIR_FWD>(s, type, &q, next)
               : q.a_mn ? launch_pair<T, PAIR_DW>(s, type, &q, next)
                        : launch_pair<T, PAIR_DX>(s, type, &q, next);
    CUtensorMap ma, mb;
    cudaError_t e = maps(type, q, &ma, &mb);
    if (e != cudaSuccess) return e;
    q.epi.part = p.splits > 1 ? part : nullptr;
    q.epi.ldp = ld_part(q.N);
#define LIN_GO(AM, BMN)                                                                        \
    e = turned(q.epi) ? launch_tc<T, AM, BMN, true>(ma, mb, q.M, q.N, p, q.epi, next, s) \
                      : launch_tc<T, AM, BMN, false>(ma, mb, q.M, q.N, p, q.epi, next, s)
    if (!q.a_mn && !q.b_mn) LIN_GO(false, false);
    else if (!q.a_mn) LIN_GO(false, true);
    else LIN_GO(true, true);
#undef LIN_GO
    if (e != cudaSuccess || p.splits == 1) return e;
    const int64_t n8 = q.M * ((q.N + 7) / 8);
    s->launches++;
    return launch(true, k_linear_join<T>, (unsigned)((n8 + 255) / 256), 256, 0, s->st, q.M, q.N, p.splits, q.M, q.epi);
}

// Matrices that TMA can address: themselves, or their copies (NULL: no third one).
cudaError_t packed(zsolve_seq *s, Mat *a, void *dsta, Mat *b, void *dstb, bool next, Mat *c = nullptr, void *dstc = nullptr) {
    PackJob job[3];
    int n = 0;
    int64_t most = 0;
    Mat *const mats[3] = {a, b, c};
    void *const dst[3] = {dsta, dstb, dstc};
    for (int i = 0; i < 3; i++) {
        Mat *m = mats[i];
        if (!m || !dst[i]) continue;
        const int64_t ldd = (m->cols + 7) / 8 * 8;
        job[n++] = PackJob{(const uint16_t *)m->p, (uint16_t *)dst[i], m->ld, m->rows, (int)m->cols};
        most = std::max(most, m->rows * (ldd / 8));
        m->p = dst[i];
        m->ld = ldd;
    }
    if (n == 0) return cudaSuccess;
    const unsigned blocks = (unsigned)std::min<int64_t>((most + 255) / 256, (int64_t)s->num_sms * 8);
    s->launches++;
    return launch(next, k_linear_pack, dim3(blocks, n), 256, 0, s->st, job[0], job[n > 1 ? 1 : 0], job[n - 1]);
}

bool vec8(const void *p, int64_t ld) { return !p || (((uintptr_t)p & 15) == 0 && ld % 8 == 0); }

}  // namespace
