// Linear attention with a decay for each head, token by token, for decoding: a block holds 32 value columns of one
// state in registers, takes the sequence's tokens one after the other,
//   S <- a S + k v^T,  o = scale S^T q,
// and writes the state back.  Bound by HBM, which the state crosses once each way; a token costs one exchange
// between the warps, for o.  64 sequences x 32 heads of 128 x 128: 44 us, 5.1 TB/s with what L2 keeps, 270 MB.
#include "decay.cuh"

namespace {

using namespace zs;

constexpr int kCols = 32;     // value columns of a block
constexpr int kThreads = 256;

// VE: value columns of a thread (4: dv a multiple of 4), 32 / VE threads a row.
template <typename T, int VE>
__global__ void __launch_bounds__(kThreads, 5)
k_decay_step(const DecayGeom geo, const int64_t *__restrict__ offsets, const float *s0, T *__restrict__ o, int64_t ldo, float *sn) {
    constexpr int TPR = kCols / VE, RPP = kThreads / TPR, NR = 128 / RPP, NW = kThreads / 32;
    __shared__ float qs[2][128], ks[2][128];
    __shared__ __align__(16) float red[2][NW][kCols];
    const DeltaGeom &d = geo.d;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int si = blockIdx.x / d.hv, hv = blockIdx.x - si * d.hv, hk = hv / (d.hv / d.hk);
    const int col = (tid % TPR) * VE, row = tid / TPR;
    const int v = blockIdx.y * kCols + col;
    const bool live = v < d.dv;
    const int64_t at = ((int64_t)si * d.hv + hv) * d.dk * d.dv;
    int64_t t0, t1;
    if (offsets) {
        t0 = offsets[si], t1 = offsets[si + 1];
        t0 = t0 < 0 ? 0 : t0 > d.tokens ? d.tokens : t0;
        t1 = t1 > d.tokens ? d.tokens : t1;
    } else {
        const int64_t len = d.tokens / d.nseq;
        t0 = si * len, t1 = t0 + len;
    }
    float S[NR][VE];
#pragma unroll
    for (int p = 0; p < NR; p++) {
        const int r = p * RPP + row;
        if (s0 && live && r < d.dk) {
            Vec<float, VE> u;
            u.load(s0 + at + (int64_t)r * d.dv + v);
            u.get(S[p]);
        } else {
#pragma unroll
            for (int e = 0; e < VE; e++) S[p][e] = 0.f;
        }
    }
    // tokens outside the sequences: their outputs are zero
    T *oh = o + (int64_t)hv * d.dv + blockIdx.y * kCols;
    const int cols = min(kCols, d.dv - (int)blockIdx.y * kCols);
    if (si == 0 && t0 > 0) zero_tokens(oh, ldo, 0, t0, cols, warp, NW);
    if (si == d.nseq - 1 && t1 < d.tokens) zero_tokens(oh, ldo, t1 > t0 ? t1 : t0, d.tokens, cols, warp, NW);
    int flip = 0;
    for (int64_t tok = t0; tok < t1; tok++, flip ^= 1) {
        if (tid < 128)
            qs[flip][tid] = tid < d.dk ? to_f32(((const T *)d.q)[tok * d.ldq + (int64_t)hk * d.dk + tid]) : 0.f;
        else
            ks[flip][tid - 128] = tid - 128 < d.dk ? to_f32(((const T *)d.k)[tok * d.ldk + (int64_t)hk * d.dk + tid - 128]) : 0.f;
        const float a = expf(d.g[tok * geo.ldg + hv]);
        float vv[VE];
#pragma unroll
        for (int e = 0; e < VE; e++) vv[e] = live ? to_f32(((const T *)d.v)[tok * d.ldv + (int64_t)hv * d.dv + v + e]) : 0.f;
        __syncthreads();
        float r[VE] = {};
#pragma unroll
        for (int p = 0; p < NR; p++) {
            const float kr = ks[flip][p * RPP + row], qr = qs[flip][p * RPP + row];
#pragma unroll
            for (int e = 0; e < VE; e++) {
                S[p][e] = fmaf(a, S[p][e], kr * vv[e]);
                r[e] = fmaf(qr, S[p][e], r[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < VE; e++)
#pragma unroll
            for (int s = TPR; s < 32; s <<= 1) r[e] += __shfl_xor_sync(0xffffffffu, r[e], s);
        if (lane < TPR)
#pragma unroll
            for (int e = 0; e < VE; e++) red[flip][warp][col + e] = r[e];
        __syncthreads();
        // the next token's values go to the other halves: one barrier lies between their use and their next writing
        if (tid < kCols && (int)blockIdx.y * kCols + tid < d.dv) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; w++) s += red[flip][w][tid];
            oh[tok * ldo + tid] = from_f32<T>(d.scale * s);
        }
    }
    if (!sn) return;
#pragma unroll
    for (int p = 0; p < NR; p++) {
        const int r = p * RPP + row;
        if (live && r < d.dk) {
            Vec<float, VE> u;
            u.set(S[p]);
            u.store(sn + at + (int64_t)r * d.dv + v);
        }
    }
}

template <typename T>
cudaError_t step(const DecayGeom &g, const int64_t *offsets, const float *s0, void *o, int64_t ldo, float *sn, cudaStream_t st) {
    const dim3 grid((unsigned)(g.d.nseq * g.d.hv), (unsigned)((g.d.dv + kCols - 1) / kCols));
    if (g.d.dv % 4 == 0 && (((uintptr_t)s0 | (uintptr_t)sn) & 15) == 0)
        k_decay_step<T, 4><<<grid, kThreads, 0, st>>>(g, offsets, s0, (T *)o, ldo, sn);
    else
        k_decay_step<T, 1><<<grid, kThreads, 0, st>>>(g, offsets, s0, (T *)o, ldo, sn);
    return cudaGetLastError();
}

}  // namespace

cudaError_t zs_launch_decay_step(int type, const DecayGeom &g, const int64_t *offsets, const float *s0, void *o, int64_t ldo, float *sn,
                                 cudaStream_t st, int64_t *launches) {
    ++*launches;
    if (type == ZSOLVE_F32) return step<float>(g, offsets, s0, o, ldo, sn, st);
    if (type == ZSOLVE_BF16) return step<bf16>(g, offsets, s0, o, ldo, sn, st);
    return step<f16>(g, offsets, s0, o, ldo, sn, st);
}
