// The gated delta rule token by token, for decoding: a block holds 32 value
// columns of one state in registers, takes the sequence's tokens one after the
// other and writes the state back.  Bound by HBM, which the state crosses once
// each way; one pass over the registers gives both products of a token,
//   r = S^T k, y = S^T q,  u = beta (v - a r),  o = scale (a y + (q . k) u),
// so that a token costs one exchange between the warps.  64 sequences x 32 heads of
// 128 x 128: 268 MB in 54 us, 5.0 TB/s (a copy of as many bytes: 5.3 to 6.3).
#include "delta.cuh"

namespace {

using namespace zs;

constexpr int kCols = 32;     // value columns of a block
constexpr int kThreads = 256;

// VE: value columns of a thread (4: dv a multiple of 4), 32 / VE threads a
// row, ROWS rows a thread.
template <typename T, int VE>
__global__ void __launch_bounds__(kThreads, 5)
k_delta_step(const DeltaGeom geo, const int64_t *__restrict__ offsets, const float *__restrict__ s0,
             T *__restrict__ o, int64_t ldo, float *__restrict__ sn) {
    constexpr int TPR = kCols / VE;               // threads a row
    constexpr int RPP = kThreads / TPR;           // rows a pass
    constexpr int NR = 128 / RPP;                 // passes
    constexpr int NW = kThreads / 32;
    __shared__ float qs[128], ks[128];
    __shared__ __align__(16) float red[NW][2][kCols];
    __shared__ __align__(16) float dots[NW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int si = blockIdx.x / geo.hv, hv = blockIdx.x - si * geo.hv, hk = hv / (geo.hv / geo.hk);
    const int col = (tid % TPR) * VE, row = tid / TPR;
    const int v = blockIdx.y * kCols + col;
    const bool live = v < geo.dv;
    const int64_t at = ((int64_t)si * geo.hv + hv) * geo.dk * geo.dv;
    int64_t t0, t1;
    if (offsets) {
        t0 = offsets[si], t1 = offsets[si + 1];
        t0 = t0 < 0 ? 0 : t0 > geo.tokens ? geo.tokens : t0;
        t1 = t1 > geo.tokens ? geo.tokens : t1;
    } else {
        const int64_t len = geo.tokens / geo.nseq;
        t0 = si * len, t1 = t0 + len;
    }
    // tokens outside the sequences: their outputs are zero
    T *oh = o + (int64_t)hv * geo.dv + blockIdx.y * kCols;
    const int cols = min(kCols, geo.dv - (int)blockIdx.y * kCols);
    if (si == 0 && t0 > 0) zero_tokens(oh, ldo, 0, t0, cols, warp, NW);
    if (si == geo.nseq - 1 && t1 < geo.tokens) zero_tokens(oh, ldo, t1 > t0 ? t1 : t0, geo.tokens, cols, warp, NW);
    float S[NR][VE];
#pragma unroll
    for (int p = 0; p < NR; p++) {
        const int r = p * RPP + row;
        if (s0 && live && r < geo.dk) {
            Vec<float, VE> u;
            u.load(s0 + at + (int64_t)r * geo.dv + v);
            u.get(S[p]);
        } else {
#pragma unroll
            for (int e = 0; e < VE; e++) S[p][e] = 0.f;
        }
    }
    for (int64_t tok = t0; tok < t1; tok++) {
        if (tok > t0) __syncthreads();  // the previous token's readers are done
        if (tid < 128)
            qs[tid] = tid < geo.dk ? to_f32(((const T *)geo.q)[tok * geo.ldq + (int64_t)hk * geo.dk + tid]) : 0.f;
        else
            ks[tid - 128] = tid - 128 < geo.dk ? to_f32(((const T *)geo.k)[tok * geo.ldk + (int64_t)hk * geo.dk + tid - 128]) : 0.f;
        float gt = geo.g[tok * geo.hv + hv];
        const float a = expf(gt), beta = geo.beta[tok * geo.hv + hv];
        float vv[VE];
#pragma unroll
        for (int e = 0; e < VE; e++)
            vv[e] = live ? to_f32(((const T *)geo.v)[tok * geo.ldv + (int64_t)hv * geo.dv + v + e]) : 0.f;
        __syncthreads();
        float r1[VE] = {}, r2[VE] = {};
#pragma unroll
        for (int p = 0; p < NR; p++) {
            const float kr = ks[p * RPP + row], qr = qs[p * RPP + row];
#pragma unroll
            for (int e = 0; e < VE; e++) {
                r1[e] = fmaf(kr, S[p][e], r1[e]);
                r2[e] = fmaf(qr, S[p][e], r2[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < VE; e++)
#pragma unroll
            for (int s = TPR; s < 32; s <<= 1) {
                r1[e] += __shfl_xor_sync(0xffffffffu, r1[e], s);
                r2[e] += __shfl_xor_sync(0xffffffffu, r2[e], s);
            }
        if (lane < TPR)
#pragma unroll
            for (int e = 0; e < VE; e++) {
                red[warp][0][col + e] = r1[e];
                red[warp][1][col + e] = r2[e];
            }
        // q . k: 16 rows a warp
        const float d = lane < 16 ? qs[warp * 16 + lane] * ks[warp * 16 + lane] : 0.f;
        const float dot = warp_sum(d);
        if (lane == 0) dots[warp] = dot;
        __syncthreads();
        float qk = 0.f;
#pragma unroll
        for (int w = 0; w < NW; w++) qk += dots[w];
        float s1[VE] = {}, s2[VE] = {}, u[VE];
#pragma unroll
        for (int w = 0; w < NW; w++) {
            float x[VE], y[VE];
            Vec<float, VE> f;
            f.load(&red[w][0][col]);
            f.get(x);
            f.load(&red[w][1][col]);
            f.get(y);
#pragma unroll
            for (int e = 0; e < VE; e++) s1[e] += x[e], s2[e] += y[e];
        }
#pragma unroll
        for (int e = 0; e < VE; e++) {
            u[e] = beta * (vv[e] - a * s1[e]);
            if (row == 0 && live)
                o[tok * ldo + (int64_t)hv * geo.dv + v + e] = from_f32<T>(geo.scale * fmaf(a, s2[e], qk * u[e]));
        }
#pragma unroll
        for (int p = 0; p < NR; p++) {
            const float kr = ks[p * RPP + row];
#pragma unroll
            for (int e = 0; e < VE; e++) S[p][e] = fmaf(a, S[p][e], kr * u[e]);
        }
    }
    if (!sn) return;
#pragma unroll
    for (int p = 0; p < NR; p++) {
        const int r = p * RPP + row;
        if (live && r < geo.dk) {
            Vec<float, VE> u;
            u.set(S[p]);
            u.store(sn + at + (int64_t)r * geo.dv + v);
        }
    }
}

template <typename T>
cudaError_t step(const DeltaGeom &g, const int64_t *offsets, const float *s0, void *o, int64_t ldo, float *sn,
                 cudaStream_t st) {
    const dim3 grid((unsigned)(g.nseq * g.hv), (unsigned)((g.dv + kCols - 1) / kCols));
    if (g.dv % 4 == 0 && (((uintptr_t)s0 | (uintptr_t)sn) & 15) == 0)
        k_delta_step<T, 4><<<grid, kThreads, 0, st>>>(g, offsets, s0, (T *)o, ldo, sn);
    else
        k_delta_step<T, 1><<<grid, kThreads, 0, st>>>(g, offsets, s0, (T *)o, ldo, sn);
    return cudaGetLastError();
}

}  // namespace

cudaError_t zs_launch_delta_step(int type, const DeltaGeom &g, const int64_t *offsets, const float *s0, void *o,
                                 int64_t ldo, float *sn, cudaStream_t st, int64_t *launches) {
    ++*launches;
    if (type == ZSOLVE_F32) return step<float>(g, offsets, s0, o, ldo, sn, st);
    if (type == ZSOLVE_BF16) return step<bf16>(g, offsets, s0, o, ldo, sn, st);
    return step<f16>(g, offsets, s0, o, ldo, sn, st);
}
