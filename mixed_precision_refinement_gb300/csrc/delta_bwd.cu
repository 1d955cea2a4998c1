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
// dS^T, 32 key columns a warp.
template <typename T, int DK>
struct RChainCfg {
    static constexpr int WK = DK / 32;
    static constexpr int NV = WK == 4 ? 2 : 4;
    static constexpr int NT = 32 * WK * NV;
    static constexpr int NTILE = 8 / WK;
    static constexpr int COLS = 16 * NV;
    static constexpr int STAGES = sizeof(T) == 2 || DK == 32 ? 2 : 1;  // as many as fit
};

template <typename T, int DK>
struct RChainStage {
    T k[kChunk * tile_ld<T>(DK)];
    T q[kChunk * tile_ld<T>(DK)];
    T dout[kChunk * tile_ld<T>(RChainCfg<T, DK>::COLS)];
    float t[kChunk * kLdT];
    float p[kChunk * kLdT];
    float vec[kVec];
};

template <typename T, int DK>
struct RChainSmem {
    using C = RChainCfg<T, DK>;
    RChainStage<T, DK> st[C::STAGES];
    float part[C::NV][C::WK][16 * kLdT];
    float x[C::NV][16 * kLdT];
    float u[C::NV][16 * kLdT];
};

// c += A B where A may be exact in tf32 (its lo part then is zero) and B is float32
template <bool EXACT_A>
__device__ __forceinline__ void mma_split_b(float (&c)[4], const SplitA &a, float2 b) {
    const uint32_t b0 = tf32(b.x), b1 = tf32(b.y);
    if (!EXACT_A) mma8(c, a.lo, b0, b1);
    mma8(c, a.hi, tf32(b.x - __uint_as_float(b0)), tf32(b.y - __uint_as_float(b1)));
    mma8(c, a.hi, b0, b1);
}

template <typename T, int DK>
__global__ void __launch_bounds__(RChainCfg<T, DK>::NT, 1)
k_delta_rchain(const DeltaGeom geo, const DeltaTerms terms, const T *__restrict__ dout, int64_t lddo,
               const float *__restrict__ ds, float *__restrict__ dends, float *__restrict__ dxs, T *__restrict__ dv,
               float *__restrict__ ds0, int vec, int veco) {
    using C = RChainCfg<T, DK>;
    constexpr int WK = C::WK, NV = C::NV, NT = C::NT, NTILE = C::NTILE;
    constexpr int LD = tile_ld<T>(DK), LDO = tile_ld<T>(C::COLS);
    constexpr bool EXACT = sizeof(T) == 2;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    RChainSmem<T, DK> &sm = *reinterpret_cast<RChainSmem<T, DK> *>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int grp = warp / WK, w = warp - grp * WK;
    const int si = blockIdx.x / geo.hv, hv = blockIdx.x - si * geo.hv, hk = hv / (geo.hv / geo.hk);
    const int vb = (int)blockIdx.y * C::COLS, v0 = vb + grp * 16, d0 = w * 32;
    const int64_t state_at = ((int64_t)si * geo.hv + hv) * geo.dk * geo.dv;

    auto load = [&](int c, int stage) {
        const int2 ch = geo.chunk[c];
        RChainStage<T, DK> &s = sm.st[stage];
        const int64_t slot = (int64_t)c * geo.hv + hv;
        load_tile<T, DK, NT>(s.k, (const T *)geo.k + (int64_t)ch.x * geo.ldk + (int64_t)hk * geo.dk, geo.ldk, ch.y, geo.dk, vec);
        load_tile<T, DK, NT>(s.q, (const T *)geo.q + (int64_t)ch.x * geo.ldq + (int64_t)hk * geo.dk, geo.ldq, ch.y, geo.dk, vec);
        load_tile<T, C::COLS, NT>(s.dout, dout + (int64_t)ch.x * lddo + (int64_t)hv * geo.dv + vb, lddo, ch.y, geo.dv - vb, veco);
        load_square<NT>(s.t, terms.t + slot * (kChunk * kChunk));
        load_square<NT>(s.p, terms.p + slot * (kChunk * kChunk));
        for (int i = threadIdx.x; i < kVec / 4; i += NT) cp_async16(s.vec + 4 * i, terms.vec + slot * kVec + 4 * i, 16);
        cp_commit();
    };

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

    const int c0 = geo.first[si], c1 = geo.first[si + 1];
    if (c0 < c1) load(c1 - 1, 0);
    for (int c = c1 - 1; c >= c0; c--) {
        const int stage = C::STAGES == 2 ? (c1 - 1 - c) & 1 : 0;
        cp_wait<0>();
        __syncthreads();  // the stage is complete, and every warp is done with the previous chunk
        if (C::STAGES == 2 && c > c0) load(c - 1, stage ^ 1);
        RChainStage<T, DK> &st = sm.st[stage];
        const int2 ch = geo.chunk[c];
        const int64_t slot = (int64_t)c * geo.hv + hv;
        put_state(dends + slot * geo.dk * geo.dv);

        // partial (K dS')^T over the warp's key columns
        {
            SplitA a[4];
#pragma unroll
            for (int j = 0; j < 4; j++) a[j].set(D[j]);
            float *part = sm.part[grp][w];
#pragma unroll
            for (int n = 0; n < 8; n++) {
                float2 b[4];
                float r[4] = {};
                frag4<T, LD, false>(st.k, n * 8, d0, b);
#pragma unroll
                for (int j = 0; j < 4; j++) mma_split<EXACT>(r, a[j], b[j]);
                *reinterpret_cast<float2 *>(part + g * kLdT + n * 8 + 2 * t) = make_float2(r[0], r[1]);
                *reinterpret_cast<float2 *>(part + (g + 8) * kLdT + n * 8 + 2 * t) = make_float2(r[2], r[3]);
            }
        }
        // dO^T as an A operand: rows v, columns the tokens of tile k
        auto dout_at = [&](int k, float (&f)[4]) {
            const T *x = st.dout + (k * 8 + 2 * t) * LDO + grp * 16 + g;
            f[0] = to_f32(x[0]), f[1] = to_f32(x[LDO]);
            f[2] = to_f32(x[8]), f[3] = to_f32(x[LDO + 8]);
        };
        // (P^T dO)^T at the warp's token tiles: P's rows from the tile on
        float du[NTILE][4] = {};
#pragma unroll
        for (int k = 0; k < 8; k++) {
            float f[4];
            dout_at(k, f);
            SplitA a;
            a.set(f);
#pragma unroll
            for (int i = 0; i < NTILE; i++) {
                const int n = tile_of<WK>(w, i);
                if (k < n) continue;
                const float *p = st.p + (k * 8 + 2 * t) * kLdT + n * 8 + g;
                mma_split_b<EXACT>(du[i], a, make_float2(p[0], p[kLdT]));
            }
        }
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
            const float ea = st.vec[kChunk + n], eb = st.vec[kChunk + n + 1];
            *reinterpret_cast<float2 *>(sm.u[grp] + g * kLdT + n) =
                make_float2(fmaf(ea, lo.x, du[i][0]), fmaf(eb, lo.y, du[i][1]));
            *reinterpret_cast<float2 *>(sm.u[grp] + (g + 8) * kLdT + n) =
                make_float2(fmaf(ea, hi.x, du[i][2]), fmaf(eb, hi.y, du[i][3]));
        }
        group_sync<WK>(grp);
        // dX^T = dU^T T at the warp's token tiles: T's rows from the tile on
        {
            float x[NTILE][4] = {};
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const float2 y = *reinterpret_cast<const float2 *>(sm.u[grp] + g * kLdT + k * 8 + 2 * t);
                const float2 z = *reinterpret_cast<const float2 *>(sm.u[grp] + (g + 8) * kLdT + k * 8 + 2 * t);
                SplitA a;
                a.set(y.x, y.y, z.x, z.y);
#pragma unroll
                for (int i = 0; i < NTILE; i++) {
                    const int n = tile_of<WK>(w, i);
                    if (k < n) continue;
                    const float *p = st.t + (k * 8 + 2 * t) * kLdT + n * 8 + g;
                    mma_split<false>(x[i], a, make_float2(p[0], p[kLdT]));
                }
            }
#pragma unroll
            for (int i = 0; i < NTILE; i++) {
                const int n = tile_of<WK>(w, i) * 8 + 2 * t;
                *reinterpret_cast<float2 *>(sm.x[grp] + g * kLdT + n) = make_float2(x[i][0], x[i][1]);
                *reinterpret_cast<float2 *>(sm.x[grp] + (g + 8) * kLdT + n) = make_float2(x[i][2], x[i][3]);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int v = v0 + g + (e >> 1) * 8, tok = n + (e & 1);
                    if (v < geo.dv) {
                        dxs[(slot * kChunk + tok) * geo.dv + v] = x[i][e];
                        if (tok < ch.y)
                            dv[((int64_t)(ch.x + tok) * geo.hv + hv) * geo.dv + v] =
                                from_f32<T>(st.vec[2 * kChunk + tok] * x[i][e]);
                    }
                }
            }
        }
        group_sync<WK>(grp);
        // dS^T = c_64 dS'^T + (scale c dO)^T Q - (beta c dX)^T K
        float acc[4][4] = {};
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const int tok = k * 8 + 2 * t;
            const float ca = st.vec[tok], cb = st.vec[tok + 1];
            const float ba = -ca * st.vec[2 * kChunk + tok], bb = -cb * st.vec[2 * kChunk + tok + 1];
            const float2 y = *reinterpret_cast<const float2 *>(sm.x[grp] + g * kLdT + tok);
            const float2 z = *reinterpret_cast<const float2 *>(sm.x[grp] + (g + 8) * kLdT + tok);
            SplitA a;
            float2 b[4];
            a.set(ba * y.x, bb * y.y, ba * z.x, bb * z.y);
            frag4<T, LD, true>(st.k, k * 8, d0, b);
#pragma unroll
            for (int j = 0; j < 4; j++) mma_split<EXACT>(acc[j], a, b[j]);
            float f[4];
            dout_at(k, f);
            const float sa = geo.scale * ca, sb = geo.scale * cb;
            a.set(sa * f[0], sb * f[1], sa * f[2], sb * f[3]);
            frag4<T, LD, true>(st.q, k * 8, d0, b);
#pragma unroll
            for (int j = 0; j < 4; j++) mma_split<EXACT>(acc[j], a, b[j]);
        }
        const float cend = st.vec[kChunk - 1];
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) D[j][e] = fmaf(cend, D[j][e], acc[j][e]);
        if (C::STAGES == 1) {
            __syncthreads();  // the only stage is free
            if (c > c0) load(c - 1, 0);
        }
    }
    if (ds0) put_state(ds0 + state_at);
}

// ---------------------------------------------------------------- gradients of a chunk

// One block for a chunk and a value head; warp (m, n): tokens 16 m .., key
// columns 32 n .. (of F, E, H, dq, dk) and 64 / NG of the 64 x 64 products'
// columns.  The products over the value columns run in slabs of 32 of them, two
// stages of slabs where they fit; the 64 x 64 matrices then take the slabs'
// place.
constexpr int kSlab = 32;
constexpr int kLdS = kSlab + 8;

template <typename T, int DK>
struct GradCfg {
    static constexpr int NG = DK / 32;
    static constexpr int NT = 128 * NG;
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
    float bh[kChunk], bl[kChunk];
    float row_kE[C::NG][kChunk], row_kH[C::NG][kChunk], row_qF[C::NG][kChunk];
    float row_m[C::NG][kChunk], row_w[C::NG][kChunk], col_m[4][kChunk];
    float row_xv[kChunk];
    float dot[C::NG * 4];
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
              T *__restrict__ dk, float *__restrict__ dg, float *__restrict__ dbeta, int vec, int vecv, int veco) {
    using C = GradCfg<T, DK>;
    constexpr int NG = C::NG, NT = C::NT, PT = C::PT, LD = C::LD;
    constexpr bool EXACT = sizeof(T) == 2;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    GradSmem<T, DK> &sm = *reinterpret_cast<GradSmem<T, DK> *>(smem_raw);
    const int2 ch = geo.chunk[blockIdx.x];
    const int n = ch.y;
    if (n == 0) return;
    const int hv = blockIdx.y, hk = hv / (geo.hv / geo.hk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int wm = warp & 3, wn = warp >> 2, m0 = wm * 16, d0 = wn * 32, p0 = wn * PT * 8;
    const int64_t slot = (int64_t)blockIdx.x * geo.hv + hv;
    const float *S = states + slot * geo.dk * geo.dv, *DS = dends + slot * geo.dk * geo.dv;
    const float *Us = us + slot * kChunk * geo.dv, *DXs = dxs + slot * kChunk * geo.dv;
    const T *DO = dout + (int64_t)ch.x * lddo + (int64_t)hv * geo.dv;
    const T *V = (const T *)geo.v + (int64_t)ch.x * geo.ldv + (int64_t)hv * geo.dv;

    auto load = [&](int v, int stage) {
        GradSlab<T, DK> &s = sm.slab[stage];
        const int cols = geo.dv - v;
        load_slab<float, DK, NT>(s.s, S + v, geo.dv, geo.dk, cols, vecv);
        load_slab<float, DK, NT>(s.ds, DS + v, geo.dv, geo.dk, cols, vecv);
        load_slab<float, kChunk, NT>(s.u, Us + v, geo.dv, kChunk, cols, vecv);
        load_slab<float, kChunk, NT>(s.dx, DXs + v, geo.dv, kChunk, cols, vecv);
        load_slab<T, kChunk, NT>(s.dout, DO + v, lddo, n, cols, veco);
        cp_commit();
    };

    load_tile<T, DK, NT>(sm.k, (const T *)geo.k + (int64_t)ch.x * geo.ldk + (int64_t)hk * geo.dk, geo.ldk, n, geo.dk, vec);
    load_tile<T, DK, NT>(sm.q, (const T *)geo.q + (int64_t)ch.x * geo.ldq + (int64_t)hk * geo.dk, geo.ldq, n, geo.dk, vec);
    for (int i = tid; i < kVec / 4; i += NT) cp_async16(sm.vec + 4 * i, terms.vec + slot * kVec + 4 * i, 16);
    load(0, 0);
    if (warp == 0) gate_sums(geo, ch, hv, sm.bh, sm.bl);
    if (tid < kChunk) sm.row_xv[tid] = 0.f;

    // the products over the value columns
    float F[4][4] = {}, E[4][4] = {}, H[4][4] = {}, dp[PT][4] = {}, da[PT][4] = {};
    float sds = 0.f;
    for (int v = 0, it = 0; v < geo.dv; v += kSlab, it++) {
        cp_wait<0>();
        __syncthreads();
        if (v + kSlab < geo.dv) load(v + kSlab, (it + 1) & 1);
        GradSlab<T, DK> &s = sm.slab[it & 1];
#pragma unroll
        for (int c = 0; c < kSlab; c += 8) {
            SplitA ao, ax, au;
            {
                const float2 a = frag1<T, kLdS>(s.dout, m0, c), b = frag1<T, kLdS>(s.dout, m0 + 8, c);
                ao.set(a.x, a.y, b.x, b.y);
            }
            {
                const float2 a = frag1<float, kLdS>(s.dx, m0, c), b = frag1<float, kLdS>(s.dx, m0 + 8, c);
                ax.set(a.x, a.y, b.x, b.y);
            }
            {
                const float2 a = frag1<float, kLdS>(s.u, m0, c), b = frag1<float, kLdS>(s.u, m0 + 8, c);
                au.set(a.x, a.y, b.x, b.y);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float2 b = frag1<float, kLdS>(s.s, d0 + 8 * j, c);
                mma_split_b<EXACT>(F[j], ao, b);
                mma_split<false>(E[j], ax, b);
                mma_split<false>(H[j], au, frag1<float, kLdS>(s.ds, d0 + 8 * j, c));
            }
#pragma unroll
            for (int j = 0; j < PT; j++) {
                if (p0 + 8 * j > m0 + 8) continue;  // above the diagonal
                const float2 b = frag1<float, kLdS>(s.u, p0 + 8 * j, c);
                mma_split_b<EXACT>(dp[j], ao, b);
                mma_split<false>(da[j], ax, b);
            }
        }
        // dX_i . v_i and <S, dS'>
        for (int i = tid; i < kChunk * kSlab; i += NT) {
            const int r = i / kSlab, c = i - r * kSlab;
            const float x = r < n && v + c < geo.dv ? s.dx[r * kLdS + c] * to_f32(V[r * geo.ldv + v + c]) : 0.f;
            const float sum = warp_sum(x);
            if (lane == 0) sm.row_xv[r] += sum;  // a warp is a row's 32 columns
        }
        for (int i = tid; i < DK * kSlab; i += NT) {
            const int r = i / kSlab, c = i - r * kSlab;
            sds = fmaf(s.s[r * kLdS + c], s.ds[r * kLdS + c], sds);
        }
    }
    sds = warp_sum(sds);
    if (lane == 0) sm.dot[warp] = sds;
    __syncthreads();  // the slabs are read; the 64 x 64 matrices take their place

    // K K^T and Q K^T: the warp's tiles
    {
        float kk[PT][4] = {}, qk[PT][4] = {};
#pragma unroll 1
        for (int c = 0; c < DK; c += 8) {
            SplitA ak, aq;
            {
                const float2 a = frag1<T, LD>(sm.k, m0, c), b = frag1<T, LD>(sm.k, m0 + 8, c);
                ak.set(a.x, a.y, b.x, b.y);
            }
            {
                const float2 a = frag1<T, LD>(sm.q, m0, c), b = frag1<T, LD>(sm.q, m0 + 8, c);
                aq.set(a.x, a.y, b.x, b.y);
            }
#pragma unroll
            for (int j = 0; j < PT; j++) {
                if (p0 + 8 * j > m0 + 8) continue;
                const float2 b = frag1<T, LD>(sm.k, p0 + 8 * j, c);
                mma_split<EXACT, EXACT>(kk[j], ak, b);
                mma_split<EXACT, EXACT>(qk[j], aq, b);
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
                    const float ex = expf((sm.bh[y] - sm.bh[x]) + (sm.bl[y] - sm.bl[x]));
                    r = geo.scale * ex * dp[j][e];
                    if (x < y) w = -ex * da[j][e];
                }
                const float bw = sm.vec[2 * kChunk + y] * w;
                sm.sq.r[y * kLdT + x] = r;
                sm.sq.w[y * kLdT + x] = bw;
                const float mm = x <= y ? fmaf(r, qk[j][e], bw * kk[j][e]) : 0.f;
                rm[e >> 1] += mm;
                cm[e & 1] += mm;
                if (x < y) rw[e >> 1] = fmaf(w, kk[j][e], rw[e >> 1]);
            }
#pragma unroll
            for (int e = 0; e < 2; e++) {  // over the 16 rows
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
    // rows' products with k and q, then dq and dk begin with c F and e H - beta c E
    float aq[4][4], ak[4][4];
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
                for (int i = e; i < e + 2; i++) {
                    aq[j][i] = geo.scale * c * F[j][i];
                    ak[j][i] = fmaf(en, H[j][i], -bc * E[j][i]);
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
    // dbeta, and dg as the sums of db from the end (float64: a few additions)
    if (warp == 0) {
        double db[2];
        float endsum = 0.f, dots = 0.f;
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
            for (int p = 0; p < 4; p++) cm += sm.col_m[p][i];
            const float c = sm.vec[i], en = sm.vec[kChunk + i], b = sm.vec[2 * kChunk + i];
            db[e] = (double)(geo.scale * c * qF) + (double)rm - (double)cm - (double)(en * kH) - (double)(b * c * kE);
            endsum = fmaf(en, kH, endsum);
            if (i < n) dbeta[(int64_t)(ch.x + i) * geo.hv + hv] = sm.row_xv[i] - c * kE + rw;
        }
        for (int i = lane; i < NG * 4; i += 32) dots += sm.dot[i];
        const float last = fmaf(sm.vec[kChunk - 1], warp_sum(dots), warp_sum(endsum));
        if (lane == 31) db[1] += (double)last;
        double s = db[0] + db[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_down_sync(0xffffffffu, s, o);
            if (lane + o < 32) s += x;
        }
        const double d0v = s, d1v = s - db[0];
        if (2 * lane < n) dg[(int64_t)(ch.x + 2 * lane) * geo.hv + hv] = (float)d0v;
        if (2 * lane + 1 < n) dg[(int64_t)(ch.x + 2 * lane + 1) * geo.hv + hv] = (float)d1v;
    }
    // dq += r K, dk += (beta w) K: rows of the tile, columns up to the diagonal
#pragma unroll 1
    for (int k = 0; k < 2 * wm + 2; k++) {
        float2 b[4];
        frag4<T, LD, true>(sm.k, k * 8, d0, b);
        SplitA ar, aw;
        {
            const float2 x = frag1<float, kLdT>(sm.sq.r, m0, k * 8), y = frag1<float, kLdT>(sm.sq.r, m0 + 8, k * 8);
            ar.set(x.x, x.y, y.x, y.y);
        }
        {
            const float2 x = frag1<float, kLdT>(sm.sq.w, m0, k * 8), y = frag1<float, kLdT>(sm.sq.w, m0 + 8, k * 8);
            aw.set(x.x, x.y, y.x, y.y);
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            mma_split<EXACT>(aq[j], ar, b[j]);
            mma_split<EXACT>(ak[j], aw, b[j]);
        }
    }
    // dk += r^T Q + (beta w)^T K: the transposes' rows, columns from the diagonal on
#pragma unroll 1
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
            mma_split<EXACT>(ak[j], ar, bq[j]);
            mma_split<EXACT>(ak[j], aw, bk[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int y = m0 + g + (e >> 1) * 8, d = d0 + 8 * j + 2 * t + (e & 1);
            if (y >= n || d >= geo.dk) continue;
            if (dqp) {
                const int64_t at = ((int64_t)(ch.x + y) * geo.hv + hv) * geo.dk + d;
                dqp[at] = aq[j][e];
                dkp[at] = ak[j][e];
            } else {
                const int64_t at = ((int64_t)(ch.x + y) * geo.hk + hk) * geo.dk + d;
                dq[at] = from_f32<T>(aq[j][e]);
                dk[at] = from_f32<T>(ak[j][e]);
            }
        }
}

// dq and dk of the key heads: the sums over the value heads that share them, in order.
template <typename T>
__global__ void __launch_bounds__(256)
k_delta_join(const float *__restrict__ dqp, const float *__restrict__ dkp, int64_t n, int group, int dk_,
             T *__restrict__ dq, T *__restrict__ dk) {
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
                      float *dends, float *dxs, void *dv, float *ds0, cudaStream_t st) {
    using C = RChainCfg<T, DK>;
    static_assert(sizeof(RChainSmem<T, DK>) <= 232448, "shared memory of a block");
    static const cudaError_t attr = cudaFuncSetAttribute(
        k_delta_rchain<T, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(RChainSmem<T, DK>));
    if (attr != cudaSuccess) return attr;
    const int vec = mult16(g.q, g.ldq, g.dk, sizeof(T)) && mult16(g.k, g.ldk, g.dk, sizeof(T));
    const int veco = mult16(dout, lddo, g.dv, sizeof(T));
    const dim3 grid((unsigned)(g.nseq * g.hv), (unsigned)((g.dv + C::COLS - 1) / C::COLS));
    k_delta_rchain<T, DK><<<grid, C::NT, sizeof(RChainSmem<T, DK>), st>>>(g, t, (const T *)dout, lddo, ds, dends, dxs,
                                                                          (T *)dv, ds0, vec, veco);
    return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t grads_dk(const DeltaGeom &g, const DeltaTerms &t, const void *dout, int64_t lddo, const float *states,
                     const float *dends, const float *us, const float *dxs, float *dqp, float *dkp, void *dq, void *dk,
                     float *dg, float *dbeta, cudaStream_t st) {
    using C = GradCfg<T, DK>;
    static_assert(sizeof(GradSmem<T, DK>) <= 232448, "shared memory of a block");
    static const cudaError_t attr = cudaFuncSetAttribute(
        k_delta_grads<T, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(GradSmem<T, DK>));
    if (attr != cudaSuccess) return attr;
    const int vec = mult16(g.q, g.ldq, g.dk, sizeof(T)) && mult16(g.k, g.ldk, g.dk, sizeof(T));
    const int veco = mult16(dout, lddo, g.dv, sizeof(T));
    k_delta_grads<T, DK><<<dim3(g.nchunks, g.hv), C::NT, sizeof(GradSmem<T, DK>), st>>>(
        g, t, (const T *)dout, lddo, states, dends, us, dxs, dqp, dkp, (T *)dq, (T *)dk, dg, dbeta, vec, g.dv % 4 == 0, veco);
    return cudaGetLastError();
}

}  // namespace

cudaError_t zs_launch_delta_rchain(int type, const DeltaGeom &g, const DeltaTerms &t, const void *dout, int64_t lddo,
                                   const float *ds, float *dends, float *dxs, void *dv, float *ds0, cudaStream_t st,
                                   int64_t *launches) {
    ++*launches;
    return DELTA_TYPE(rchain_dk, g, t, dout, lddo, ds, dends, dxs, dv, ds0, st);
}

cudaError_t zs_launch_delta_grads(int type, const DeltaGeom &g, const DeltaTerms &t, const void *dout, int64_t lddo,
                                  const float *states, const float *dends, const float *us, const float *dxs,
                                  float *dqp, float *dkp, void *dq, void *dk, float *dg, float *dbeta, cudaStream_t st,
                                  int64_t *launches) {
    ++*launches;
    cudaError_t e = DELTA_TYPE(grads_dk, g, t, dout, lddo, states, dends, us, dxs, dqp, dkp, dq, dk, dg, dbeta, st);
    if (e != cudaSuccess || !dqp) return e;
    const int64_t n = g.tokens * g.hk * g.dk;
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 152 * 16);
    const int group = g.hv / g.hk;
    ++*launches;
    if (type == ZSOLVE_F32)
        k_delta_join<float><<<blocks, 256, 0, st>>>(dqp, dkp, n, group, g.dk, (float *)dq, (float *)dk);
    else if (type == ZSOLVE_BF16)
        k_delta_join<bf16><<<blocks, 256, 0, st>>>(dqp, dkp, n, group, g.dk, (bf16 *)dq, (bf16 *)dk);
    else
        k_delta_join<f16><<<blocks, 256, 0, st>>>(dqp, dkp, n, group, g.dk, (f16 *)dq, (f16 *)dk);
    return cudaGetLastError();
}
