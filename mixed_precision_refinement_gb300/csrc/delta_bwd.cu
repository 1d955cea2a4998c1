// The gated delta rule in chunks of 64 tokens, backward (notation in
// delta.cuh).  With dO and dS', the gradients of a chunk's outputs and of the
// state after it,
//   dU = P^T dO + e K dS',  dX = T^T dU,
//   dS = c_64 dS' + scale (c Q)^T dO - (beta c K)^T dX                  (the recurrence)
// and then, chunk by chunk on its own, with w_ij = -(dX U^T)_ij e_ij (j < i),
// r_ij = scale (dO U^T)_ij e_ij (j <= i), E = dX S^T, F = scale dO S^T, H = U dS'^T:
//   dq = c F + r K,   dk = r^T Q + e H - beta c E + (beta w) K + (beta w)^T K,  dv = beta dX,
//   dbeta_i = dX_i . v_i - c_i k_i . E_i + sum_j w_ij (k_i . k_j),
//   db_i = c_i q_i . F_i - e_i k_i . H_i - beta_i c_i k_i . E_i + sum_j m_ij - sum_j m_ji,
//   m_ij = r_ij (q_i . k_j) + beta_i w_ij (k_i . k_j),
//   db_64 += sum_j e_j k_j . H_j + c_64 <S, dS'>,   dg_i = db_i + ... + db_64.
// The gates' gradients are float32 results built from these products, so they
// keep float32 accuracy throughout.
#include <algorithm>

#include "delta.cuh"

namespace {

using namespace zs;

// ---------------------------------------------------------------- chain backwards

// Laid out as the forward chain: a group of WK warps owns 16 value columns of
// dS^T, 32 key columns a warp, and one more warp fetches the chunks' operands;
// the exchanges are the partial sums of (K dS')^T, then dU^T, then dX^T and
// (scale c dO)^T, split where they are written.  A chunk of 128 x 128 heads takes 4.4
// us (bfloat16; 2 x 2048 tokens x 32 heads 284 us), bound by the latency of these steps.
template <typename T, int DK>
struct RChainCfg {
    static constexpr int WK = DK / 32;
    static constexpr int NV = DK == 32 ? 4 : 2;
    static constexpr int NC = 32 * WK * NV;  // threads of the groups
    static constexpr int NT = NC + 32;
    static constexpr int NTILE = 8 / WK;
    static constexpr int COLS = 16 * NV;
    static constexpr int STAGES = sizeof(T) == 2 || DK == 64 ? 2 : 1;  // as many as fit
};

template <typename T, int DK>
struct RChainStage {
    T k[kChunk * tile_ld<T>(DK)];
    T q[kChunk * tile_ld<T>(DK)];
    T dout[kChunk * tile_ld<T>(RChainCfg<T, DK>::COLS)];
    float tp[kSquare];
    float vec[kVec];
};

template <typename T, int DK>
struct RChainSmem {
    using C = RChainCfg<T, DK>;
    RChainStage<T, DK> st[C::STAGES];
    // the partial sums, then (scale c dO)^T: 16 rows of split pairs
    float part[C::NV][C::WK > 2 ? C::WK : 2][16 * kLdT];
    float4 u[C::NV][16 * kLdPair];  // dU^T
    float4 x[C::NV][16 * kLdPair];  // -(beta c dX)^T
    uint64_t full[C::STAGES], empty[C::STAGES];
    int abort_word;
};

// One value of a triangular product over later tokens: the sum of x(j) m[j ld] over the tokens j
// from `from` on.
template <typename FX>
__device__ __forceinline__ float later_again(FX x, const float *m, int ld, int from) {
    float sum = 0.f;
#pragma unroll 1
    for (int j = from; j < kChunk; j++) sum = fmaf(x(j), m[j * ld], sum);
    return sum;
}

template <typename T, int DK>
__global__ void __launch_bounds__(RChainCfg<T, DK>::NT, 1)
k_delta_rchain(const DeltaGeom geo, const DeltaTerms terms, const T *__restrict__ dout, int64_t lddo,
               const float *__restrict__ ds, float *__restrict__ dends, float *__restrict__ dxs, T *__restrict__ dv,
               float *__restrict__ ds0, unsigned *__restrict__ status) {
    using C = RChainCfg<T, DK>;
    constexpr int WK = C::WK, NTILE = C::NTILE;
    constexpr int LD = tile_ld<T>(DK), LDO = tile_ld<T>(C::COLS);
    constexpr bool EXACT = sizeof(T) == 2;
    static_assert(2 * 16 * kLdT * sizeof(float) >= 16 * kLdPair * sizeof(float4), "room for the split pairs");
    extern __shared__ __align__(16) uint8_t smem_raw[];
    RChainSmem<T, DK> &sm = *reinterpret_cast<RChainSmem<T, DK> *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int si = blockIdx.x / geo.hv, hv = blockIdx.x - si * geo.hv, hk = hv / (geo.hv / geo.hk);
    const int vb = (int)blockIdx.y * C::COLS;
    after_previous();
    may_start_next();
    const int cols = min(C::COLS, geo.dvp - vb);  // of the block's dO
    const int c0 = geo.first[si], c1 = geo.first[si + 1];

    if (tid == 0) {
        sm.abort_word = 0;
        for (int i = 0; i < C::STAGES; i++) {
            bar_init(&sm.full[i], 33);  // the fetching warp's lanes, and the bulk copies
            bar_init(&sm.empty[i], C::NC / 32);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();

    if (warp == C::NC / 32) {
        // ------------------------------------------------ the chunks' operands, the last chunk first
        const T *kp = (const T *)geo.k + (int64_t)hk * geo.dkp, *qp = (const T *)geo.q + (int64_t)hk * geo.dkp;
        const T *op = dout + (int64_t)hv * geo.dvp + vb;
        int it = 0;
        for (int c = c1 - 1; c >= c0; c--, it++) {
            const int stage = it % C::STAGES;
            if (!bar_wait(&sm.empty[stage], ((it / C::STAGES) & 1) ^ 1, &sm.abort_word, status)) break;
            const int2 ch = geo.chunk[c];
            RChainStage<T, DK> &s = sm.st[stage];
            const int64_t slot = (int64_t)c * geo.hv + hv;
            uint64_t *bar = &sm.full[stage];
            warp_tile<T, DK, 1>(s.k, kp + (int64_t)ch.x * geo.ldk, geo.ldk, ch.y, geo.dkp, 0);
            warp_tile<T, DK, 1>(s.q, qp + (int64_t)ch.x * geo.ldq, geo.ldq, ch.y, geo.dkp, 0);
            warp_tile<T, C::COLS, 1>(s.dout, op + (int64_t)ch.x * lddo, lddo, ch.y, cols, 0);
            cp_arrive(bar);
            if (lane == 0) {
                bar_expect(bar, (kSquare + kVec) * 4);
                bulk_load(s.tp, terms.tp + slot * kSquare, kSquare * 4, bar);
                bulk_load(s.vec, terms.vec + slot * kVec, kVec * 4, bar);
            }
        }
        bar_drain(sm.full, C::STAGES, it);  // copies in flight end before the block does
        return;
    }

    // ---------------------------------------------------- the groups
    const int grp = warp / WK, w = warp - grp * WK;
    const int v0 = vb + grp * 16, d0 = w * 32;
    const int64_t state_at = ((int64_t)si * geo.hv + hv) * geo.dk * geo.dv;
    float D[4][4];  // dS^T: rows v0 + g, + 8, columns d0 + 8 j + 2t, + 1
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int v = v0 + g + (e >> 1) * 8, d = d0 + 8 * j + 2 * t + (e & 1);
            D[j][e] = ds && v < geo.dv && d < geo.dk ? ds[state_at + (int64_t)d * geo.dv + v] : 0.f;
        }
    auto put_state = [&](float *dst) {
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int v = v0 + g + (e >> 1) * 8, d = d0 + 8 * j + 2 * t + (e & 1);
                if (v < geo.dv && d < geo.dk) dst[(int64_t)d * geo.dv + v] = D[j][e];
            }
    };

    for (int c = c1 - 1; c >= c0; c--) {
        const int it = c1 - 1 - c, stage = it % C::STAGES;
        bar_wait(&sm.full[stage], (it / C::STAGES) & 1, &sm.abort_word, status);
        RChainStage<T, DK> &st = sm.st[stage];
        const int2 ch = geo.chunk[c];
        const int64_t slot = (int64_t)c * geo.hv + hv;
        put_state(dends + slot * geo.dk * geo.dv);
        group_sync<WK>(grp);  // the group is done with the previous chunk's exchanges

        // partial (K dS')^T over the warp's key columns
        {
            StateSplit<T> a;
            a.set(D);
            float *part = sm.part[grp][w];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                float r[4][4];
                state_times_rows<T, LD>(a, st.k, 4 * h, d0, r);
#pragma unroll
                for (int n = 0; n < 4; n++) {
                    float *p = part + g * kLdT + (4 * h + n) * 8 + 2 * t;
                    *reinterpret_cast<float2 *>(p) = make_float2(r[n][0], r[n][1]);
                    *reinterpret_cast<float2 *>(p + 8 * kLdT) = make_float2(r[n][2], r[n][3]);
                }
            }
        }
        // (P^T dO)^T at the warp's token tiles: dO^T is the A operand, P's rows from the tile on
        float du[NTILE][4];
        triangular<WK, false, EXACT, false>(
            w, du,
            [&](int k, SplitA &a) {
                float2 f0, f1;
                frag2_col<T, LDO>(st.dout, k * 8, grp * 16, f0, f1);
                a.set(f0.x, f0.y, f1.x, f1.y);
            },
            [&](int k, int n) { return frag_p_later(st.tp, k, n); });
        group_sync<WK>(grp);
#pragma unroll
        for (int i = 0; i < NTILE; i++) {
            const int n = tile_of<WK>(w, i) * 8 + 2 * t;
            float2 lo = make_float2(0.f, 0.f), hi = lo;
#pragma unroll
            for (int p = 0; p < WK; p++) {
                const float2 y = *reinterpret_cast<const float2 *>(sm.part[grp][p] + g * kLdT + n);
                const float2 z = *reinterpret_cast<const float2 *>(sm.part[grp][p] + (g + 8) * kLdT + n);
                lo.x += y.x, lo.y += y.y, hi.x += z.x, hi.y += z.y;
            }
            const float2 ev = *reinterpret_cast<const float2 *>(st.vec + kChunk + n);
            float4 *u = sm.u[grp] + g * kLdPair + n / 2;
            u[0] = split_pair(fmaf(ev.x, lo.x, du[i][0]), fmaf(ev.y, lo.y, du[i][1]));
            u[8 * kLdPair] = split_pair(fmaf(ev.x, hi.x, du[i][2]), fmaf(ev.y, hi.y, du[i][3]));
        }
        // An infinity or NaN in dO is in the gradients of its token and those before it; in a
        // tile on the diagonal the zeros of P (and below of T) have made NaN of it for those
        // after it.  Put right as in the forward pass: one value at a time, from memory.
        if (not_finite(du)) {
#pragma unroll 1
            for (int b = 0; b < 4 * NTILE; b++) {
                const int r = g + (b & 2) * 4, n = tile_of<WK>(w, b >> 2) * 8 + 2 * t + (b & 1);
                if (isfinite(PairAt{sm.u[grp]}(r, n))) continue;
                const T *dot = st.dout + grp * 16 + r;
                float sum = later_again([&](int j) { return to_f32(dot[j * LDO]); }, st.tp + n * kLdT, 1, n), lo = 0.f;
                for (int p = 0; p < WK; p++) lo += sm.part[grp][p][r * kLdT + n];
                sum = fmaf(st.vec[kChunk + n], lo, sum);
                float *p = reinterpret_cast<float *>(sm.u[grp] + r * kLdPair + n / 2) + (n & 1);
                p[0] = __uint_as_float(tf32(sum));
                p[2] = __uint_as_float(tf32(sum - p[0]));
            }
        }
        group_sync<WK>(grp);
        // dX^T = dU^T T at the warp's token tiles: T's rows from the tile on
        {
            float x[NTILE][4];
            triangular<WK, false, false, false>(
                w, x, [&](int k, SplitA &a) { a.set(sm.u[grp][g * kLdPair + k * 4 + t], sm.u[grp][(g + 8) * kLdPair + k * 4 + t]); },
                [&](int k, int n) { return frag_t_later(st.tp, k, n); });
            // the partial sums' place is free: (scale c dO)^T, split, goes there
            float4 *y = reinterpret_cast<float4 *>(sm.part[grp][0]);
#pragma unroll
            for (int i = 0; i < NTILE; i++) {
                const int n = tile_of<WK>(w, i) * 8 + 2 * t, at = g * kLdPair + n / 2;
                const float2 cv = *reinterpret_cast<const float2 *>(st.vec + n);
                const float2 bv = *reinterpret_cast<const float2 *>(st.vec + 2 * kChunk + n);
                const float(&v)[4] = x[i];
                const float ba = -bv.x * cv.x, bb = -bv.y * cv.y;
                put_pair<T>(sm.x[grp] + at, ba * v[0], bb * v[1]);
                put_pair<T>(sm.x[grp] + at + 8 * kLdPair, ba * v[2], bb * v[3]);
                float2 f0, f1;
                frag2_col<T, LDO>(st.dout, n - 2 * t, grp * 16, f0, f1);
                const float ca = geo.scale * cv.x, cb = geo.scale * cv.y;
                put_pair<T>(y + at, ca * f0.x, cb * f0.y);
                put_pair<T>(y + at + 8 * kLdPair, ca * f1.x, cb * f1.y);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int vc = v0 + g + (e >> 1) * 8, tok = n + (e & 1);
                    if (vc < geo.dv) {
                        dxs[(slot * kChunk + tok) * geo.dv + vc] = v[e];
                        if (tok < ch.y)
                            dv[((int64_t)(ch.x + tok) * geo.hv + hv) * geo.dv + vc] =
                                from_f32<T>((e & 1 ? bv.y : bv.x) * v[e]);
                    }
                }
            }
            // dS needs no repair: its value column is not finite either way
            if (not_finite(x)) {
#pragma unroll 1
                for (int b = 0; b < 4 * NTILE; b++) {
                    const int r = g + (b & 2) * 4, n = tile_of<WK>(w, b >> 2) * 8 + 2 * t + (b & 1), vc = v0 + r;
                    float *p = dxs + (slot * kChunk + n) * geo.dv + vc;
                    if (vc >= geo.dv || isfinite(*p)) continue;
                    const PairAt u{sm.u[grp]};
                    *p = u(r, n) + later_again([&](int j) { return u(r, j); }, st.tp + n, kLdT, n + 1);
                    if (n < ch.y)
                        dv[((int64_t)(ch.x + n) * geo.hv + hv) * geo.dv + vc] = from_f32<T>(st.vec[2 * kChunk + n] * *p);
                }
            }
        }
        group_sync<WK>(grp);
        // dS^T = c_64 dS'^T + (scale c dO)^T Q - (beta c dX)^T K, each sum from zero
        float rk[4][4], rq[4][4];
        tokens_product<T, LD>(sm.x[grp], st.k, d0, rk);
        tokens_product<T, LD>(reinterpret_cast<const float4 *>(sm.part[grp][0]), st.q, d0, rq);
        const float cend = st.vec[kChunk - 1];
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) D[j][e] = fmaf(cend, D[j][e], rk[j][e] + rq[j][e]);
        __syncwarp();
        if (lane == 0) bar_arrive(&sm.empty[stage]);
    }
    if (ds0) put_state(ds0 + state_at);
}

// ---------------------------------------------------------------- gradients of a chunk

// One block for a chunk and a value head; warp (m, n): 16 tokens, key columns
// 32 n .. (of F, E, H, dq, dk) and 64 / NG of the 64 x 64 products' columns.  The
// products over the value columns run in slabs of 32 of them, two stages of slabs;
// the 64 x 64 matrices then take the slabs' place.  4096 tokens x 32 heads of 128,
// bfloat16: 480 us, 36 us a block; bound by the dependent steps of mma.sync (its pipe
// 39% busy) with the 16 warps an SM that registers and shared memory allow.
constexpr int kSlab = 32;
constexpr int kLdS = kSlab + 8;

template <typename T, int DK>
struct GradCfg {
    static constexpr int NG = DK / 32;
    // groups of 16 tokens, a warp's (32 a warp would share the B splits, but leave two warps a scheduler: 2104 us for 2047)
    static constexpr int MG = 4;
    static constexpr int NT = 32 * MG * NG;
    static constexpr int PT = 8 / NG;  // 8-column tiles of the 64 x 64 products a warp
    static constexpr int LD = tile_ld<T>(DK);
};

template <typename T, int DK>
struct GradSlab {
    float s[DK * kLdS];
    float ds[DK * kLdS];
    float u[kChunk * kLdS];
    float dx[kChunk * kLdS];
    T dout[kChunk * kLdS];
};

struct GradSquares {
    float r[kChunk * kLdT], w[kChunk * kLdT];  // r and beta w
};

template <typename T, int DK>
struct GradSmem {
    using C = GradCfg<T, DK>;
    T k[kChunk * C::LD];
    T q[kChunk * C::LD];
    union {
        GradSlab<T, DK> slab[2];
        GradSquares sq;
    };
    float vec[kVec];
    float row_kE[C::NG][kChunk], row_kH[C::NG][kChunk], row_qF[C::NG][kChunk];
    float row_m[C::NG][kChunk], row_w[C::NG][kChunk], col_m[C::MG][kChunk];
    float row_xv[kChunk];
    float dot[C::NG * C::MG];
};

// (X(r0 + g, c0 + 2t), X(r0 + g, c0 + 2t + 1))
template <typename T, int LD>
__device__ __forceinline__ float2 frag1(const T *x, int r0, int c0) {
    const int lane = threadIdx.x & 31;
    const T *p = x + (r0 + (lane >> 2)) * LD + c0 + 2 * (lane & 3);
    if constexpr (sizeof(T) == 2)
        return unpack2<T>(*reinterpret_cast<const uint32_t *>(p));
    else
        return *reinterpret_cast<const float2 *>(p);
}

// A 16 x 8 A operand from rows r0 .. of a tile: the parts, of which a 16-bit
// value has only the first.
template <typename T, int LD>
__device__ __forceinline__ SplitA rows_a(const T *x, int r0, int c0) {
    const float2 a = frag1<T, LD>(x, r0, c0), b = frag1<T, LD>(x, r0 + 8, c0);
    SplitA s;
    if constexpr (sizeof(T) == 2) {
        s.hi[0] = __float_as_uint(a.x), s.hi[1] = __float_as_uint(b.x), s.hi[2] = __float_as_uint(a.y), s.hi[3] = __float_as_uint(b.y);
        s.lo[0] = s.lo[1] = s.lo[2] = s.lo[3] = 0u;
    } else {
        s.set(a.x, a.y, b.x, b.y);
    }
    return s;
}

// A float32 B operand in two tf32 parts, for several products.
struct SplitB {
    uint32_t h0, h1, l0, l1;
};
__device__ __forceinline__ SplitB split_b(float2 b) {
    SplitB s;
    s.h0 = tf32(b.x), s.h1 = tf32(b.y);
    s.l0 = tf32(b.x - __uint_as_float(s.h0)), s.l1 = tf32(b.y - __uint_as_float(s.h1));
    return s;
}
template <bool A_EXACT>
__device__ __forceinline__ void mma_add(float (&c)[4], const SplitA &a, const SplitB &b) {
    float d[4];
    mma8_first(d, a.hi, b.l0, b.l1);
    if (!A_EXACT) mma8(d, a.lo, b.h0, b.h1);
    mma8(d, a.hi, b.h0, b.h1);
    add_to(c, d);
}

// Two neighbouring values as they lie in memory.
template <typename T>
struct alignas(2 * sizeof(T)) Pair {
    T x, y;
};
template <typename T>
__device__ __forceinline__ float2 pair_f32(const Pair<T> &p) {
    return make_float2(to_f32(p.x), to_f32(p.y));
}

// R rows of a slab: `cols` columns of rows at stride ld, zeros beyond
template <typename T, int R, int NT>
__device__ __forceinline__ void load_slab(T *dst, const T *src, int64_t ld, int rows, int cols, int vec) {
    if (vec) {
        constexpr int VE = 16 / (int)sizeof(T), PER = kSlab / VE;
        for (int i = threadIdx.x; i < R * PER; i += NT) {
            const int r = i / PER, c = (i - r * PER) * VE;
            const bool in = r < rows && c < cols;
            cp_async16(dst + r * kLdS + c, src + (in ? r * ld + c : 0), in ? 16 : 0);
        }
    } else {
        for (int i = threadIdx.x; i < R * kSlab; i += NT) {
            const int r = i / kSlab, c = i - r * kSlab;
            dst[r * kLdS + c] = r < rows && c < cols ? src[r * ld + c] : from_f32<T>(0.f);
        }
    }
}

template <typename T, int DK>
__global__ void __launch_bounds__(GradCfg<T, DK>::NT, 1)
k_delta_grads(const DeltaGeom geo, const DeltaTerms terms, const T *__restrict__ dout, int64_t lddo,
              const float *__restrict__ states, const float *__restrict__ dends, const float *__restrict__ us,
              const float *__restrict__ dxs, float *__restrict__ dqp, float *__restrict__ dkp, T *__restrict__ dq,
              T *__restrict__ dk, T *__restrict__ dv, float *__restrict__ dg, float *__restrict__ dbeta, int vecv) {
    using C = GradCfg<T, DK>;
    constexpr int NG = C::NG, MG = C::MG, NT = C::NT, PT = C::PT, LD = C::LD;
    constexpr bool EXACT = sizeof(T) == 2;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    GradSmem<T, DK> &sm = *reinterpret_cast<GradSmem<T, DK> *>(smem_raw);
    after_previous();
    may_start_next();
    const int2 ch = geo.chunk[blockIdx.x];
    const int n = ch.y, hv = blockIdx.y, hk = hv / (geo.hv / geo.hk);
    if (n == 0) {
        tokens_outside(geo, blockIdx.x, [&](int64_t t0, int64_t t1, int worker, int workers) {
            const int64_t at = (int64_t)hv * geo.dk, nk = (int64_t)geo.hv * geo.dk;
            zero_tokens(dv + (int64_t)hv * geo.dv, (int64_t)geo.hv * geo.dv, t0, t1, geo.dv, worker, workers);
            zero_tokens(dg + hv, geo.hv, t0, t1, 1, worker, workers);
            zero_tokens(dbeta + hv, geo.hv, t0, t1, 1, worker, workers);
            if (dqp) {
                zero_tokens(dqp + at, nk, t0, t1, geo.dk, worker, workers);
                zero_tokens(dkp + at, nk, t0, t1, geo.dk, worker, workers);
            } else {  // as many key heads as value heads
                zero_tokens(dq + at, nk, t0, t1, geo.dk, worker, workers);
                zero_tokens(dk + at, nk, t0, t1, geo.dk, worker, workers);
            }
        });
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int wm = warp % MG, wn = warp / MG, m0 = wm * 16, d0 = wn * 32, p0 = wn * PT * 8;
    const int64_t slot = (int64_t)blockIdx.x * geo.hv + hv;
    const float *S = states + slot * geo.dk * geo.dv, *DS = dends + slot * geo.dk * geo.dv;
    const float *Us = us + slot * kChunk * geo.dv, *DXs = dxs + slot * kChunk * geo.dv;
    const T *DO = dout + (int64_t)ch.x * lddo + (int64_t)hv * geo.dvp;
    const T *V = (const T *)geo.v + (int64_t)ch.x * geo.ldv + (int64_t)hv * geo.dvp;

    auto load = [&](int v, int stage) {
        GradSlab<T, DK> &s = sm.slab[stage];
        const int cols = geo.dv - v;
        load_slab<float, DK, NT>(s.s, S + v, geo.dv, geo.dk, cols, vecv);
        load_slab<float, DK, NT>(s.ds, DS + v, geo.dv, geo.dk, cols, vecv);
        load_slab<float, kChunk, NT>(s.u, Us + v, geo.dv, kChunk, cols, vecv);
        load_slab<float, kChunk, NT>(s.dx, DXs + v, geo.dv, kChunk, cols, vecv);
        load_slab<T, kChunk, NT>(s.dout, DO + v, lddo, n, geo.dvp - v, 1);
        cp_commit();
    };

    load_tile<T, DK, NT>(sm.k, (const T *)geo.k + (int64_t)ch.x * geo.ldk + (int64_t)hk * geo.dkp, geo.ldk, n, geo.dkp);
    load_tile<T, DK, NT>(sm.q, (const T *)geo.q + (int64_t)ch.x * geo.ldq + (int64_t)hk * geo.dkp, geo.ldq, n, geo.dkp);
    for (int i = tid; i < kVec / 4; i += NT) cp_async16(sm.vec + 4 * i, terms.vec + slot * kVec + 4 * i, 16);
    load(0, 0);
    if (tid < kChunk) sm.row_xv[tid] = 0.f;

    // the products over the value columns
    float F[4][4] = {}, E[4][4] = {}, H[4][4] = {}, dp[PT][4] = {}, da[PT][4] = {};
    float sds = 0.f;
    for (int v = 0, it = 0; v < geo.dv; v += kSlab, it++) {
        cp_wait<0>();
        __syncthreads();
        if (v + kSlab < geo.dv) load(v + kSlab, (it + 1) & 1);
        GradSlab<T, DK> &s = sm.slab[it & 1];
        // v for the dot products below: on its way during the products
        constexpr int NV2 = kChunk * kSlab / 2 / NT;
        Pair<T> vv[NV2];
#pragma unroll
        for (int i = 0; i < NV2; i++) {
            const int r = (tid >> 4) + i * (NT / 16), c = v + (tid & 15) * 2;
            vv[i] = Pair<T>{};
            if (r < n && c < geo.dvp) vv[i] = *reinterpret_cast<const Pair<T> *>(V + r * geo.ldv + c);  // dX is zero beyond dv
        }
#pragma unroll 1
        for (int c = 0; c < kSlab; c += 8) {
            const SplitA ao = rows_a<T, kLdS>(s.dout, m0, c), ax = rows_a<float, kLdS>(s.dx, m0, c), au = rows_a<float, kLdS>(s.u, m0, c);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const SplitB b = split_b(frag1<float, kLdS>(s.s, d0 + 8 * j, c)), e = split_b(frag1<float, kLdS>(s.ds, d0 + 8 * j, c));
                mma_add<EXACT>(F[j], ao, b);
                mma_add<false>(E[j], ax, b);
                mma_add<false>(H[j], au, e);
            }
#pragma unroll
            for (int j = 0; j < PT; j++) {
                if (p0 + 8 * j > m0 + 8) continue;  // above the diagonal
                const SplitB b = split_b(frag1<float, kLdS>(s.u, p0 + 8 * j, c));
                mma_add<EXACT>(dp[j], ao, b);
                mma_add<false>(da[j], ax, b);
            }
        }
        // dX_i . v_i, two columns a lane, and <S, dS'>
#pragma unroll
        for (int i = 0; i < NV2; i++) {
            const int r = (tid >> 4) + i * (NT / 16);
            const float2 x = *reinterpret_cast<const float2 *>(s.dx + r * kLdS + (tid & 15) * 2), y = pair_f32<T>(vv[i]);
            float sum = fmaf(x.x, y.x, x.y * y.y);
#pragma unroll
            for (int q = 1; q < 16; q <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, q);
            if ((tid & 15) == 0) sm.row_xv[r] += sum;  // one half warp a row
        }
        for (int i = tid; i < DK * kSlab / 4; i += NT) {
            const int r = i / (kSlab / 4), c = (i - r * (kSlab / 4)) * 4;
            const float4 x = *reinterpret_cast<const float4 *>(s.s + r * kLdS + c), y = *reinterpret_cast<const float4 *>(s.ds + r * kLdS + c);
            sds += fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w)));
        }
    }
    sds = warp_sum(sds);
    if (lane == 0) sm.dot[warp] = sds;
    __syncthreads();  // the slabs are read; the 64 x 64 matrices take their place

    // K K^T: the warp's tiles; of Q K^T only P is needed, which the terms have
    {
        const float *bh = sm.vec + 3 * kChunk, *bl = sm.vec + 4 * kChunk;
        float pt[PT][4];
#pragma unroll
        for (int j = 0; j < PT; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int y = m0 + g + (e >> 1) * 8, x = p0 + 8 * j + 2 * t + (e & 1);
                pt[j][e] = x <= y ? terms.tp[slot * kSquare + x * kLdT + y] : 0.f;
            }
        float kk[PT][4] = {};
#pragma unroll 4
        for (int c = 0; c < DK; c += 8) {
            const SplitA ak = rows_a<T, LD>(sm.k, m0, c);
#pragma unroll
            for (int j = 0; j < PT; j++) {
                const float2 b = frag1<T, LD>(sm.k, p0 + 8 * j, c);
                mma_add<EXACT, EXACT>(kk[j], ak, b);
            }
        }
        // r, beta w and their sums with the raw products
        float rm[2] = {}, rw[2] = {};
#pragma unroll
        for (int j = 0; j < PT; j++) {
            float cm[2] = {};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int y = m0 + g + (e >> 1) * 8, x = p0 + 8 * j + 2 * t + (e & 1);
                float r = 0.f, w = 0.f;
                if (x <= y) {
                    const float ex = expf((bh[y] - bh[x]) + (bl[y] - bl[x]));
                    r = geo.scale * ex * dp[j][e];
                    if (x < y) w = -ex * da[j][e];
                }
                const float bw = sm.vec[2 * kChunk + y] * w;
                sm.sq.r[y * kLdT + x] = r;
                sm.sq.w[y * kLdT + x] = bw;
                const float mm = x <= y ? fmaf(dp[j][e], pt[j][e], bw * kk[j][e]) : 0.f;
                rm[e >> 1] += mm;
                cm[e & 1] += mm;
                if (x < y) rw[e >> 1] = fmaf(w, kk[j][e], rw[e >> 1]);
            }
#pragma unroll
            for (int e = 0; e < 2; e++) {  // over the warp's rows
                cm[e] += __shfl_xor_sync(0xffffffffu, cm[e], 4);
                cm[e] += __shfl_xor_sync(0xffffffffu, cm[e], 8);
                cm[e] += __shfl_xor_sync(0xffffffffu, cm[e], 16);
                if (g == 0) sm.col_m[wm][p0 + 8 * j + 2 * t + e] = cm[e];
            }
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                rm[h] += __shfl_xor_sync(0xffffffffu, rm[h], o);
                rw[h] += __shfl_xor_sync(0xffffffffu, rw[h], o);
            }
            if (t == 0) {
                sm.row_m[wn][m0 + g + 8 * h] = rm[h];
                sm.row_w[wn][m0 + g + 8 * h] = rw[h];
            }
        }
    }
    // rows' products with k and q; then dq and dk begin with c F and e H - beta c E, in F's and H's place
    {
        float kE[2] = {}, kH[2] = {}, qF[2] = {};
        const int y0 = m0 + g;
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const float2 kv = frag1<T, LD>(sm.k, m0 + 8 * h, d0 + 8 * j), qv = frag1<T, LD>(sm.q, m0 + 8 * h, d0 + 8 * j);
                const int y = y0 + 8 * h, e = 2 * h;
                kE[h] = fmaf(kv.x, E[j][e], fmaf(kv.y, E[j][e + 1], kE[h]));
                kH[h] = fmaf(kv.x, H[j][e], fmaf(kv.y, H[j][e + 1], kH[h]));
                qF[h] = fmaf(qv.x, F[j][e], fmaf(qv.y, F[j][e + 1], qF[h]));
                const float c = sm.vec[y], en = sm.vec[kChunk + y], bc = sm.vec[2 * kChunk + y] * c;
#pragma unroll
                for (int q = e; q < e + 2; q++) {
                    F[j][q] *= geo.scale * c;
                    H[j][q] = fmaf(en, H[j][q], -bc * E[j][q]);
                }
            }
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                kE[h] += __shfl_xor_sync(0xffffffffu, kE[h], o);
                kH[h] += __shfl_xor_sync(0xffffffffu, kH[h], o);
                qF[h] += __shfl_xor_sync(0xffffffffu, qF[h], o);
            }
            if (t == 0) {
                sm.row_kE[wn][y0 + 8 * h] = kE[h];
                sm.row_kH[wn][y0 + 8 * h] = kH[h];
                sm.row_qF[wn][y0 + 8 * h] = qF[h];
            }
        }
    }
    __syncthreads();
    // dbeta, and dg as the sums of db from the end, on the last warp
    if (warp == NT / 32 - 1) {
        float db[2], endsum = 0.f, dots = 0.f;
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int i = 2 * lane + e;
            float kE = 0.f, kH = 0.f, qF = 0.f, rm = 0.f, rw = 0.f, cm = 0.f;
#pragma unroll
            for (int p = 0; p < NG; p++) {
                kE += sm.row_kE[p][i], kH += sm.row_kH[p][i], qF += sm.row_qF[p][i];
                rm += sm.row_m[p][i], rw += sm.row_w[p][i];
            }
#pragma unroll
            for (int p = 0; p < MG; p++) cm += sm.col_m[p][i];
            const float c = sm.vec[i], en = sm.vec[kChunk + i], b = sm.vec[2 * kChunk + i];
            db[e] = (geo.scale * c * qF - b * c * kE) + (rm - cm) - en * kH;
            endsum = fmaf(en, kH, endsum);
            if (i < n) dbeta[(int64_t)(ch.x + i) * geo.hv + hv] = sm.row_xv[i] - c * kE + rw;
        }
        for (int i = lane; i < NG * MG; i += 32) dots += sm.dot[i];
        const float last = fmaf(sm.vec[kChunk - 1], warp_sum(dots), warp_sum(endsum));
        if (lane == 31) db[1] += last;
        float s = db[0] + db[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_down_sync(0xffffffffu, s, o);
            if (lane + o < 32) s += x;
        }
        float after = __shfl_down_sync(0xffffffffu, s, 1);
        if (lane == 31) after = 0.f;
        const float d1 = db[1] + after;
        if (2 * lane < n) dg[(int64_t)(ch.x + 2 * lane) * geo.hv + hv] = db[0] + d1;
        if (2 * lane + 1 < n) dg[(int64_t)(ch.x + 2 * lane + 1) * geo.hv + hv] = d1;
    }
    // dq += r K, dk += (beta w) K: columns up to the diagonal
#pragma unroll 2
    for (int k = 0; k < 2 * (wm + 1); k++) {
        float2 b[4];
        frag4<T, LD, true>(sm.k, k * 8, d0, b);
        const SplitA ar = rows_a<float, kLdT>(sm.sq.r, m0, k * 8), aw = rows_a<float, kLdT>(sm.sq.w, m0, k * 8);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            mma_add<false, EXACT>(F[j], ar, b[j]);
            mma_add<false, EXACT>(H[j], aw, b[j]);
        }
    }
    // dk += r^T Q + (beta w)^T K: the transposes' rows, columns from the diagonal on
#pragma unroll 2
    for (int k = 2 * wm; k < 8; k++) {
        float2 bq[4], bk[4];
        frag4<T, LD, true>(sm.q, k * 8, d0, bq);
        frag4<T, LD, true>(sm.k, k * 8, d0, bk);
        const int at = (k * 8 + 2 * t) * kLdT + m0 + g;
        SplitA ar, aw;
        ar.set(sm.sq.r[at], sm.sq.r[at + kLdT], sm.sq.r[at + 8], sm.sq.r[at + kLdT + 8]);
        aw.set(sm.sq.w[at], sm.sq.w[at + kLdT], sm.sq.w[at + 8], sm.sq.w[at + kLdT + 8]);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            mma_add<false, EXACT>(H[j], ar, bq[j]);
            mma_add<false, EXACT>(H[j], aw, bk[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int y = m0 + g + 8 * h, d = d0 + 8 * j + 2 * t;
            if (y >= n) continue;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                if (d + e >= geo.dk) continue;
                if (dqp) {
                    const int64_t at = ((int64_t)(ch.x + y) * geo.hv + hv) * geo.dk + d + e;
                    dqp[at] = F[j][2 * h + e];
                    dkp[at] = H[j][2 * h + e];
                } else {
                    const int64_t at = ((int64_t)(ch.x + y) * geo.hk + hk) * geo.dk + d + e;
                    dq[at] = from_f32<T>(F[j][2 * h + e]);
                    dk[at] = from_f32<T>(H[j][2 * h + e]);
                }
            }
        }
}

// dq and dk of the key heads: the sums over the value heads that share them, in order.
// Bound by HBM: 4096 tokens x 32 value heads of 128 in 34 us, 4.3 TB/s.
template <typename T>
__global__ void __launch_bounds__(256)
k_delta_join(const float *__restrict__ dqp, const float *__restrict__ dkp, int64_t n, int group, int dk_,
             T *__restrict__ dq, T *__restrict__ dk) {
    after_previous();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t head = i / dk_, d = i - head * dk_;
        const int64_t at = head * group * dk_ + d;
        float a = 0.f, b = 0.f;
        for (int r = 0; r < group; r++) {
            a += dqp[at + (int64_t)r * dk_];
            b += dkp[at + (int64_t)r * dk_];
        }
        dq[i] = from_f32<T>(a);
        dk[i] = from_f32<T>(b);
    }
}

template <typename T, int DK>
cudaError_t rchain_dk(const DeltaGeom &g, const DeltaTerms &t, const void *dout, int64_t lddo, const float *ds,
                      float *dends, float *dxs, void *dv, float *ds0, unsigned *status, bool next, cudaStream_t st) {
    using C = RChainCfg<T, DK>;
    static_assert(sizeof(RChainSmem<T, DK>) <= 232448, "shared memory of a block");
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_delta_rchain<T, DK>, (int)sizeof(RChainSmem<T, DK>));
    if (attr != cudaSuccess) return attr;
    const dim3 grid((unsigned)(g.nseq * g.hv), (unsigned)((g.dv + C::COLS - 1) / C::COLS));
    return launch(next, k_delta_rchain<T, DK>, grid, C::NT, sizeof(RChainSmem<T, DK>), st, g, t, (const T *)dout, lddo, ds, dends,
                  dxs, (T *)dv, ds0, status);
}

template <typename T, int DK>
cudaError_t grads_dk(const DeltaGeom &g, const DeltaTerms &t, const void *dout, int64_t lddo, const float *states,
                     const float *dends, const float *us, const float *dxs, float *dqp, float *dkp, void *dq, void *dk,
                     void *dv, float *dg, float *dbeta, bool next, cudaStream_t st) {
    using C = GradCfg<T, DK>;
    static_assert(sizeof(GradSmem<T, DK>) <= 232448, "shared memory of a block");
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_delta_grads<T, DK>, (int)sizeof(GradSmem<T, DK>));
    if (attr != cudaSuccess) return attr;
    return launch(next, k_delta_grads<T, DK>, dim3(g.nchunks, g.hv), C::NT, sizeof(GradSmem<T, DK>), st, g, t, (const T *)dout,
                  lddo, states, dends, us, dxs, dqp, dkp, (T *)dq, (T *)dk, (T *)dv, dg, dbeta, (int)(g.dv % 4 == 0));
}

}  // namespace

cudaError_t zs_launch_delta_rchain(int type, const DeltaGeom &g, const DeltaTerms &t, const void *dout, int64_t lddo,
                                   const float *ds, float *dends, float *dxs, void *dv, float *ds0, unsigned *status,
                                   bool next, cudaStream_t st, int64_t *launches) {
    ++*launches;
    return DELTA_TYPE(rchain_dk, g, t, dout, lddo, ds, dends, dxs, dv, ds0, status, next, st);
}

cudaError_t zs_launch_delta_grads(int type, const DeltaGeom &g, const DeltaTerms &t, const void *dout, int64_t lddo,
                                  const float *states, const float *dends, const float *us, const float *dxs,
                                  float *dqp, float *dkp, void *dq, void *dk, void *dv, float *dg,
                                  float *dbeta, int num_sms, bool next, cudaStream_t st, int64_t *launches) {
    ++*launches;
    cudaError_t e = DELTA_TYPE(grads_dk, g, t, dout, lddo, states, dends, us, dxs, dqp, dkp, dq, dk, dv, dg, dbeta, next, st);
    if (e != cudaSuccess || !dqp) return e;
    const int64_t n = g.tokens * g.hk * g.dk;
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, (int64_t)num_sms * 16);
    const int group = g.hv / g.hk;
    ++*launches;
    auto join = [&](auto kernel, auto *q, auto *k) {
        return launch(true, kernel, blocks, 256, 0, st, (const float *)dqp, (const float *)dkp, n, group, g.dk, q, k);
    };
    return type == ZSOLVE_F32    ? join(k_delta_join<float>, (float *)dq, (float *)dk)
           : type == ZSOLVE_BF16 ? join(k_delta_join<bf16>, (bf16 *)dq, (bf16 *)dk)
                                 : join(k_delta_join<f16>, (f16 *)dq, (f16 *)dk);
}
