// What the norms of rows share: a row's sums, loads of weights of two types, and the
// ring of rows in shared memory.
#pragma once

#include "seq.cuh"

namespace zs {

// Sum of v over the TPR threads of a row.  TPR = 32: one warp; else the row's
// warps exchange their sums through `red` (one slot a warp; `flip` alternates
// two sets, so that one barrier a reduction is enough).
template <int TPR>
__device__ __forceinline__ float2 row_sum(float2 v, float2 *red, int flip) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (TPR == 32) return v;
    constexpr int NW = TPR / 32;
    float2 *r = red + flip * NW;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) r[warp] = v;
    __syncthreads();
    // every thread adds the warps' sums itself: broadcast reads, without the
    // latency of five more shuffles
    float2 t = r[0], u = r[1];
#pragma unroll
    for (int w = 2; w < NW; w += 2) {
        t.x += r[w].x, t.y += r[w].y;
        u.x += r[w + 1].x, u.y += r[w + 1].y;
    }
    return make_float2(t.x + u.x, t.y + u.y);
}

// A load that stays where it is written: the next rows' mean and rstd, which the
// compiler would otherwise be free to move down to their use, a row later.
__device__ __forceinline__ float load_early(const float *p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

template <typename T>
__device__ __forceinline__ float load_w(const void *w, int wf32, int64_t i) {
    return wf32 ? reinterpret_cast<const float *>(w)[i] : to_f32(reinterpret_cast<const T *>(w)[i]);
}

// w at N consecutive columns (aligned as x is when N > 1)
template <typename T, int N>
__device__ __forceinline__ void load_wv(const void *w, int wf32, int64_t i, float *f) {
    if (N > 1 && !wf32) {
        Vec<T, N> v;
        v.load(reinterpret_cast<const T *>(w) + i);
        v.get(f);
        return;
    }
#pragma unroll
    for (int e = 0; e < N; e++) f[e] = load_w<T>(w, wf32, i + e);
}

// The same from shared memory, where both types of w are aligned.
template <typename T, int N>
__device__ __forceinline__ void load_ws(const void *w, int wf32, int i, float *f) {
    if (N > 1 && wf32) {
#pragma unroll
        for (int e = 0; e < N; e += 4)
            *reinterpret_cast<float4 *>(f + e) = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(w) + i + e);
    } else {
        load_wv<T, N>(w, wf32, i, f);
    }
}

// rs from mean (x - m)^2 and e = mean (x - m), whose square is at most the former but for
// rounding (NaN stays).
__device__ __forceinline__ float inv_std(float square, float e, float eps) {
    const float var = fmaf(-e, e, square);
    return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);
}

// A ring's row in shared memory: the values of d, and room for a start off 16 bytes.
template <typename T>
__host__ __device__ constexpr int ring_row(int d) {
    return (d + 2 * (16 / (int)sizeof(T)) - 1) / (16 / (int)sizeof(T)) * (16 / (int)sizeof(T));
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace zs
