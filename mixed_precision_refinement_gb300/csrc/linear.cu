// The matrix product with bias, activation and residual in its epilogue, and
// its gradients, on the 5th-generation tensor cores:
//   z = x W^T + b, y = act(z) + r            x: m x k, W: n x k
//   dz = dy act'(z), dx = dz W, dW = dz^T x, db = sum over rows of dz
// All three products are one kernel, D(i, j) = sum_k A(i, k) B(j, k), for
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
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "linear.cuh"

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

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 lanes x 32 consecutive float32 columns of the accumulator
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
          "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; i++) v[i] = __uint_as_float(r[i]);
}

// Shared-memory descriptor of a 128-byte swizzled operand.  K-major: rows of
// 128 bytes (64 k values), groups of 8 rows 1024 bytes apart (stride offset).
// MN-major: rows of 128 bytes hold 64 values along M or N for one k; groups of
// 8 k 1024 bytes apart (stride offset), the next 64 along M or N a box of
// 64 k rows further (leading offset).
constexpr uint32_t kBox = 64 * 128;  // bytes of an MN-major box: 64 k rows
template <bool MN>
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(MN ? kBox >> 4 : 1) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

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

template <typename T, bool A_MN, bool B_MN, bool TURN>
__global__ void __launch_bounds__(kThreads, 1)
k_linear_tc(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, int64_t M, int64_t N,
            int kblocks, int splits, const Epilogue epi, unsigned *__restrict__ status) {
    using C = Cfg;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[C::STAGES], bar_empty[C::STAGES], bar_accf[2], bar_acce[2], bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mt = (int)((M + BM - 1) / BM), nt = (int)((N + BN - 1) / BN);
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
                        tma_load_2d(sa, &amap, kb * BK, x.tm * BM, fb);
                    }
                    if (B_MN) {
#pragma unroll
                        for (int i = 0; i < BN / 64; i++)
                            tma_load_2d(sb + i * kBox, &bmap, x.tn * BN + i * 64, kb * BK, fb);
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
            const bool ok = drain<T, BN / 64, TURN>(
                epi, M, N, (int64_t)x.tm * BM + quad * 32 + lane, (int64_t)x.tn * BN + half * (BN / 2), x.split,
                tmem + buf * 256u + (uint32_t)(half * (BN / 2)) + ((uint32_t)(quad * 32) << 16), turn,
                [&] {
                    const bool in = __all_sync(0xffffffffu, bar_wait(&bar_accf[buf], aph, &s_abort, status));
                    tc_fence_after();
                    return in;
                },
                [&] {  // accumulator fully read: hand it back to the MMA warp
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&bar_acce[buf]);
                });
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
enum { PAIR_FWD, PAIR_DX, PAIR_DW, PAIR_GRADS };  // x W^T, dz W, dz^T x, and the last two together
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
              int kblocks0, const Epilogue epi0, const __grid_constant__ PairSecond two, unsigned *__restrict__ status) {
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
    constexpr bool BOTH = FORM == PAIR_GRADS, b_mn = FORM != PAIR_FWD;
    const int mt0 = (int)((M0 + 2 * BM - 1) / (2 * BM)), nt0 = (int)((N0 + 255) / 256);
    const int mt1 = BOTH ? (int)((two.M + 2 * BM - 1) / (2 * BM)) : 0, nt1 = BOTH ? (int)((two.N + 255) / 256) : 0;
    int job, tile;
    auto next = [&](uint32_t i) {  // the pair's tile i, if there is one
        return pair_tile<BOTH>(mt0 * nt0, mt1 * nt1, BOTH ? two.extra : 0, pair, pairs, (int)i, &job, &tile);
    };
    auto place = [&] { return BOTH && job ? tile_at(tile, mt1, nt1) : tile_at(tile, mt0, nt0); };
    auto a_major = [&] { return BOTH ? two.first_mn == !job : FORM == PAIR_DW; };

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
                const int ra = x.tm * 2 * BM + (int)rank * BM, rb = x.tn * 256 + (int)rank * 128;
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
                        tma_load_2d_pair(sa, ma, kb * BK, ra, fb);
                    }
                    if (b_mn) {
                        tma_load_2d_pair(sb, mb, rb, kb * BK, fb);
                        tma_load_2d_pair(sb + kBox, mb, rb + 64, kb * BK, fb);
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
            const bool ok = drain<T, 4, TURN>(
                BOTH && job ? two.epi : epi0, BOTH && job ? two.M : M0, BOTH && job ? two.N : N0,
                (int64_t)x.tm * 2 * BM + rank * BM + quad * 32 + lane, (int64_t)x.tn * 256 + half * 128, 0,
                tmem + buf * 256u + (uint32_t)(half * 128) + ((uint32_t)(quad * 32) << 16), turn,
                [&] {
                    const bool in = __all_sync(0xffffffffu, bar_wait(&bar_accf[buf], aph, &s_abort, status));
                    tc_fence_after();
                    return in;
                },
                [&] {  // accumulator fully read: hand it back to the leader's MMA warp
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(cluster_addr(smem_u32(&bar_acce[buf]), 0));
                });
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

// The parts of a product split along k, added in order, and the epilogue; a
// thread for 8 columns of a row.  Bound by the latency of its loads, which L2 serves:
// 801 x 1000 in two parts 6 us, partly hidden behind the product's end.
template <typename T>
__global__ void __launch_bounds__(256)
k_linear_join(int64_t M, int64_t N, int splits, const Epilogue epi) {
    after_previous();
    may_start_next();
    const int64_t groups = (N + 7) / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= M * groups) return;
    const int64_t row = i / groups, c = (i - row * groups) * 8;
    float v[8] = {};
    for (int s = 0; s < splits; s++) {
        const float4 *p = reinterpret_cast<const float4 *>(epi.part + ((int64_t)s * M + row) * epi.ldp + c);
        const float4 a = p[0], b = p[1];
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
    finish8<T>(epi, row, c, (int)min((int64_t)8, N - c), v);
}

// Rows that TMA cannot address (base or row stride not a multiple of 16
// bytes) copied to rows that it can; 16-bit values, up to two matrices a launch.
struct PackJob {
    const uint16_t *src;
    uint16_t *dst;  // rows of whole 16 bytes
    int64_t ld, rows;
    int cols;
};
__global__ void __launch_bounds__(256)
k_linear_pack(const PackJob a, const PackJob b) {
    after_previous();
    may_start_next();
    const PackJob &j = blockIdx.y ? b : a;
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

// dz = dy act'(z) into rows of stride ldo (a multiple of 8; NULL: not written)
// and, per block row, the columns' float32 sums of it before it is rounded
// (parts, one row of n a block row; NULL: not formed).  dz is rounded to the
// inputs' type because it is the tensor cores' operand: it adds one rounding
// of an input to each product's terms.  Bound by HBM: 8192 x 4096 bfloat16 in 45 us,
// 4.5 TB/s.
constexpr int kDzBlocks = 4;  // of an SM
template <typename T>
__global__ void __launch_bounds__(256, kDzBlocks)
k_linear_dz(const T *__restrict__ dy, int64_t lddy, const T *__restrict__ z, int64_t ldz, int act, int64_t m, int n,
            T *__restrict__ dz, int64_t ldo, float *__restrict__ parts, int vec) {
    __shared__ float red[8][32][9];
    after_previous();
    may_start_next();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = ((int64_t)blockIdx.x * 32 + tx) * 8;
    const int nc = (int)min((int64_t)8, (int64_t)n - c);
    float sum[8] = {};
    if (nc > 0) {
#pragma unroll 2
        for (int64_t row = (int64_t)blockIdx.y * 8 + ty; row < m; row += (int64_t)gridDim.y * 8) {
            float v[8], f[8];
            load8<T>(dy, row * lddy + c, nc, vec, v);
            if (z) {
                load8<T>(z, row * ldz + c, nc, vec, f);
#define SLOPE_CASE(A)                                                          \
    case A: {                                                                  \
        _Pragma("unroll") for (int i = 0; i < 8; i++) v[i] *= slope1<A>(f[i]); \
        break;                                                                 \
    }
                switch (act) {
                    SLOPE_CASE(ACT_RELU)
                    SLOPE_CASE(ACT_SILU)
                    SLOPE_CASE(ACT_GELU)
                    SLOPE_CASE(ACT_GELU_TANH)
                }
#undef SLOPE_CASE
            }
#pragma unroll
            for (int i = 0; i < 8; i++) {
                if (i >= nc) v[i] = 0.f;
                sum[i] += v[i];
            }
            if (dz) {
                Vec<T, 8> u;
                u.set(v);
                u.store(dz + row * ldo + c);
            }
        }
    }
    if (!parts) return;
#pragma unroll
    for (int i = 0; i < 8; i++) red[ty][tx][i] = sum[i];
    __syncthreads();
    // thread (ty, tx): column 8 tx + ty of the block's 256
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 8; r++) s += red[r][tx][ty];
    const int64_t col = ((int64_t)blockIdx.x * 32 + tx) * 8 + ty;
    if (col < n) parts[(int64_t)blockIdx.y * n + col] = s;
}

template <typename T>
__global__ void __launch_bounds__(256)
k_linear_db(const float *__restrict__ parts, int nparts, int n, T *__restrict__ db) {
    __shared__ float red[8][32];
    after_previous();
    may_start_next();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + tx;
    float s = 0.f;
    if (c < n)
        for (int p = ty; p < nparts; p += 8) s += parts[(int64_t)p * n + c];
    red[ty][tx] = s;
    __syncthreads();
    if (ty != 0 || c >= n) return;
#pragma unroll
    for (int r = 1; r < 8; r++) s += red[r][tx];
    db[c] = from_f32<T>(s);
}

// ---------------------------------------------------------------- host

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)p;
    }();
    return fn;
}

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

template <typename T, bool A_MN, bool B_MN, bool TURN>
cudaError_t launch_tc(const CUtensorMap &a, const CUtensorMap &b, int64_t M, int64_t N, const Plan &p,
                      const Epilogue &epi, bool next, zsolve_seq *s) {
    constexpr int smem = Cfg::SMEM + (TURN ? kTurn : 0);
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_linear_tc<T, A_MN, B_MN, TURN>, smem);
    if (attr != cudaSuccess) return attr;
    const int64_t total = (M + BM - 1) / BM * ((N + BN - 1) / BN) * p.splits;
    s->launches++;
    return launch(next, k_linear_tc<T, A_MN, B_MN, TURN>, (unsigned)std::min<int64_t>(total, s->num_sms), kThreads, smem, s->st,
                  a, b, M, N, p.kblocks, p.splits, epi, s->d_status);
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

// Products whose plan is pairs of SMs: one, or with PAIR_GRADS two; the longer sums
// first, so that the last round is of short ones.
template <typename T, int FORM, bool TURN>
cudaError_t launch_pair_as(zsolve_seq *s, int type, const Product *p, bool next) {
    constexpr int smem = kPairSmem + (TURN ? kTurn : 0);
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_linear_pair<T, FORM, TURN>, smem);
    if (attr != cudaSuccess) return attr;
    constexpr int n = FORM == PAIR_GRADS ? 2 : 1;
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
                  s->d_status);
}
template <typename T, int FORM>
cudaError_t launch_pair(zsolve_seq *s, int type, const Product *p, bool next) {
    return turned(p[0].epi) || (FORM == PAIR_GRADS && turned(p[1].epi)) ? launch_pair_as<T, FORM, true>(s, type, p, next)
                                                                        : launch_pair_as<T, FORM, false>(s, type, p, next);
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
    return launch(true, k_linear_join<T>, (unsigned)((n8 + 255) / 256), 256, 0, s->st, q.M, q.N, p.splits, q.epi);
}

// Matrices that TMA can address: themselves, or their copies.
cudaError_t packed(zsolve_seq *s, Mat *a, void *dsta, Mat *b, void *dstb, bool next) {
    PackJob job[2];
    int n = 0;
    int64_t most = 0;
    Mat *const mats[2] = {a, b};
    void *const dst[2] = {dsta, dstb};
    for (int i = 0; i < 2; i++) {
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
    return launch(next, k_linear_pack, dim3(blocks, n), 256, 0, s->st, job[0], job[n - 1]);
}

bool vec8(const void *p, int64_t ld) { return !p || (((uintptr_t)p & 15) == 0 && ld % 8 == 0); }

template <typename T>
int linear_fwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, Mat x, Mat w, const Epilogue &epi) {
    const Plan p = plan_of(m, n, k, s->num_sms);
    uint16_t *xp, *wp;
    float *part;
    int st = ZSOLVE_OK;
    auto carve = [&](void *base) {
        Carve c(base);
        xp = x.tma_ok() ? nullptr : c.take<uint16_t>(x.packed_values());
        wp = w.tma_ok() ? nullptr : c.take<uint16_t>(w.packed_values());
        part = p.splits > 1 ? c.take<float>(part_values(m, n, p)) : nullptr;
        return c.at;
    };
    const size_t bytes = carve(nullptr);
    if (bytes) {
        void *ws = seq_workspace(s, bytes, &st);
        if (!ws) return st;
        carve(ws);
    }
    const int64_t before = s->launches;
    SEQ_CU(packed(s, &x, xp, &w, wp, false));
    SEQ_CU(product<T>(s, type, Product{m, n, k, x, w, false, false, epi}, part, s->launches > before));
    return ZSOLVE_OK;
}

// Block rows of k_linear_dz, which are parts of db: as many blocks as the SMs hold at a time.
int dz_rows(int64_t m, int64_t n, int num_sms) {
    const int64_t most = std::max<int64_t>(1, (int64_t)num_sms * kDzBlocks / ((n + 255) / 256));
    return (int)std::min<int64_t>({(m + 7) / 8, most, 1024});
}

template <typename T>
int linear_bwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, Mat dy, Mat x, Mat w, int act, Mat z, void *dx,
               int64_t lddx, void *dw, int64_t lddw, void *db) {
    if (m == 0) {
        if (dw) SEQ_CU(cudaMemset2DAsync(dw, (size_t)lddw * 2, 0, (size_t)k * 2, (size_t)n, s->st));
        if (db) SEQ_CU(cudaMemsetAsync(db, 0, (size_t)n * 2, s->st));
        return ZSOLVE_OK;
    }
    const Plan px = plan_of(m, k, n, s->num_sms), pw = plan_of(n, k, m, s->num_sms);
    const bool has_act = act != ACT_NONE;
    const bool products = dx || dw;
    const bool form_dz = products && (has_act || !dy.tma_ok());
    const int dzrows = dz_rows(m, n, s->num_sms);
    const int64_t ldz8 = (n + 7) / 8 * 8;
    uint16_t *dzp = nullptr, *xp = nullptr, *wp = nullptr;
    float *part = nullptr, *sums = nullptr;
    int st = ZSOLVE_OK;
    auto carve = [&](void *base) {
        Carve c(base);
        dzp = form_dz ? c.take<uint16_t>((size_t)m * ldz8) : nullptr;
        xp = dw && !x.tma_ok() ? c.take<uint16_t>(x.packed_values()) : nullptr;
        wp = dx && !w.tma_ok() ? c.take<uint16_t>(w.packed_values()) : nullptr;
        const size_t parts = std::max(dx ? part_values(m, k, px) : 0, dw ? part_values(n, k, pw) : 0);
        part = parts ? c.take<float>(parts) : nullptr;
        sums = db ? c.take<float>((size_t)dzrows * n) : nullptr;
        return c.at;
    };
    const size_t bytes = carve(nullptr);
    if (bytes) {
        void *ws = seq_workspace(s, bytes, &st);
        if (!ws) return st;
        carve(ws);
    }
    const int64_t before = s->launches;
    if (form_dz || db) {
        const int vec = vec8(dy.p, dy.ld) && (!has_act || vec8(z.p, z.ld));
        k_linear_dz<T><<<dim3((unsigned)((n + 255) / 256), dzrows), 256, 0, s->st>>>(
            (const T *)dy.p, dy.ld, has_act ? (const T *)z.p : nullptr, z.ld, act, m, (int)n, (T *)dzp, ldz8, sums, vec);
        s->launches++;
        SEQ_CU(cudaGetLastError());
    }
    if (db) {
        s->launches++;
        SEQ_CU(launch(true, k_linear_db<T>, (unsigned)((n + 31) / 32), 256, 0, s->st, sums, dzrows, (int)n, (T *)db));
    }
    Mat dz = dy;
    if (form_dz) dz.p = dzp, dz.ld = ldz8;
    SEQ_CU(packed(s, &w, wp, &x, xp, s->launches > before));
    Product pr[2];
    int np = 0;
    if (dx) {
        Epilogue epi{};
        epi.y = dx, epi.ldy = lddx, epi.vec = vec8(dx, lddx);
        pr[np++] = Product{m, k, n, dz, w, false, true, epi};
    }
    if (dw) {
        Epilogue epi{};
        epi.y = dw, epi.ldy = lddw, epi.vec = vec8(dw, lddw);
        pr[np++] = Product{n, k, m, dz, x, true, true, epi};
    }
    if (np == 2 && px.pair && pw.pair) {
        SEQ_CU((launch_pair<T, PAIR_GRADS>(s, type, pr, s->launches > before)));
    } else {
        for (int i = 0; i < np; i++) SEQ_CU(product<T>(s, type, pr[i], part, s->launches > before));
    }
    return ZSOLVE_OK;
}

}  // namespace

int zs_linear(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx, const void *w,
              int64_t ldw, const void *b, int act, const void *r, int64_t ldr, void *y, int64_t ldy, void *z,
              int64_t ldz) {
    Epilogue epi{};
    epi.bias = b, epi.r = r, epi.y = y, epi.z = z;
    epi.ldr = ldr, epi.ldy = ldy, epi.ldz = ldz;
    epi.act = act;
    epi.vec = vec8(b, 0) && vec8(r, ldr) && vec8(y, ldy) && vec8(z, ldz);
    // One kernel for few rows, against a split product and its join.  4096 x 2048: 4.6 us
    // for 1 .. 8 rows, 6.6 for 16, against 10; 8192 x 4096: 16 and 19.7 against 18; rows
    // read value by value (1000 x 2157): 9.4 and 15.4 against 12.3.
    const bool aligned = Mat{x, m, k, ldx}.tma_ok() && Mat{w, n, k, ldw}.tma_ok();
    if (m <= 8 || (m <= kFewRows && aligned && n * k <= 1 << 24)) {
        SEQ_CU(zs_launch_linear_few(type, m, n, k, x, ldx, w, ldw, epi, s->st, &s->launches));
        return ZSOLVE_OK;
    }
    const Mat mx{x, m, k, ldx}, mw{w, n, k, ldw};
    return type == ZSOLVE_BF16 ? linear_fwd<bf16>(s, type, m, n, k, mx, mw, epi)
                               : linear_fwd<f16>(s, type, m, n, k, mx, mw, epi);
}

int zs_linear_bwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *dy, int64_t lddy,
                  const void *x, int64_t ldx, const void *w, int64_t ldw, int act, const void *z, int64_t ldz,
                  void *dx, int64_t lddx, void *dw, int64_t lddw, void *db) {
    const Mat md{dy, m, n, lddy}, mx{x, m, k, ldx}, mw{w, n, k, ldw}, mz{z, m, n, ldz};
    return type == ZSOLVE_BF16
               ? linear_bwd<bf16>(s, type, m, n, k, md, mx, mw, act, mz, dx, lddx, dw, lddw, db)
               : linear_bwd<f16>(s, type, m, n, k, md, mx, mw, act, mz, dx, lddx, dw, lddw, db);
}
