// The epilogue of the matrix product: bias, activation, residual, stores.
#pragma once

#include "seq.cuh"

namespace zs {

enum { ACT_NONE = ZSOLVE_ACT_NONE, ACT_RELU = ZSOLVE_ACT_RELU, ACT_SILU = ZSOLVE_ACT_SILU, ACT_GELU = ZSOLVE_ACT_GELU, ACT_GELU_TANH = ZSOLVE_ACT_GELU_TANH };

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// The tanh form in the sigmoid: (1 + tanh u) / 2 = sigmoid(2 u), without the
// cancellation of 1 + tanh u for negative u.
constexpr float kTanhC = 0.7978845608028654f, kTanhA = 0.044715f;

// The exact form in the Gaussian's upper tail Q(y) = erfc(y / sqrt 2) / 2 of y = |z|: 1 + erf
// would leave no digits of a negative z's value.  With relu and sign,
//   z Phi(z) = relu(z) - y Q(y),  its slope = w or 1 - w, w = Q(y) - y phi(y),
// and Q(y) = exp(-y^2 / 2) gauss_tail(y): a smooth function between 1/2 and 0.03, here the
// polynomial of degree 7 in 1 / (1 + 0.35 y) whose largest relative error over 0 .. 14 is
// least (3e-7; 6e-7 in float32).  8192 x 8192 x 1024: 143 us, as with erff; with
// erfcf 212.
constexpr float kTailEnd = 16.f;  // from here on exp(-y^2 / 2) is 0
__device__ __forceinline__ float gauss_tail(float y) {
    const float t = __fdividef(1.f, fmaf(0.35f, y, 1.f));
    float p = 0.0489424467f;
    p = fmaf(p, t, -0.202119291f);
    p = fmaf(p, t, 0.240640819f);
    p = fmaf(p, t, -0.0170234367f);
    p = fmaf(p, t, 0.155961484f);
    p = fmaf(p, t, 0.133355096f);
    p = fmaf(p, t, 0.140270337f);
    return fmaf(p, t, -2.73155492e-05f);
}

template <int ACT>
__device__ __forceinline__ float act1(float z) {
    if (ACT == ACT_RELU) return z <= 0.f ? 0.f : z;
    if (ACT == ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
    if (ACT == ACT_GELU) {
        const float y = fminf(fabsf(z), kTailEnd);
        return fmaf(-y * __expf(-0.5f * y * y), gauss_tail(y), z <= 0.f ? 0.f : z);
    }
    if (ACT == ACT_GELU_TANH) return __fdividef(z, 1.f + __expf(-2.f * kTanhC * fmaf(kTanhA * z * z, z, z)));
    return z;
}
template <int ACT>
__device__ __forceinline__ float slope1(float z) {
    if (ACT == ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (ACT == ACT_SILU) {
        const float p = sigmoid(z);
        return p * fmaf(z, 1.f - p, 1.f);
    }
    if (ACT == ACT_GELU) {
        const float y = fabsf(z) > kTailEnd ? kTailEnd : fabsf(z);  // NaN stays
        const float w = __expf(-0.5f * y * y) * fmaf(-0.3989422804014327f, y, gauss_tail(y));
        return z < 0.f ? w : 1.f - w;
    }
    if (ACT == ACT_GELU_TANH) {
        const float p = sigmoid(2.f * kTanhC * fmaf(kTanhA * z * z, z, z));
        // beyond 32 p (1 - p) is 0, and z^2 may be infinite
        const float y = fminf(fmaxf(z, -32.f), 32.f);
        return fmaf(2.f * kTanhC * fmaf(3.f * kTanhA * y, y, 1.f), y * p * (1.f - p), p);
    }
    return 1.f;
}

template <int N>
__device__ __forceinline__ void act_all(float (&v)[N], int act) {
#define ACT_CASE(A)                                        \
    case A: {                                              \
        _Pragma("unroll") for (int i = 0; i < N; i++) v[i] = act1<A>(v[i]); \
        break;                                             \
    }
    switch (act) {
        ACT_CASE(ACT_RELU)
        ACT_CASE(ACT_SILU)
        ACT_CASE(ACT_GELU)
        ACT_CASE(ACT_GELU_TANH)
    }
#undef ACT_CASE
}

// What happens to a tile of the product: part (float32 partial sums, row
// stride ldp, one matrix of prows rows a split) or the finished result.
struct Epilogue {
    const void *bias;  // NULL: none
    const void *r;     // residual, NULL: none
    void *y;
    void *z;           // product and bias before the activation, NULL: not kept
    int64_t ldr, ldy, ldz;
    float *part;
    int64_t ldp;
    int act;
    int vec;           // 16-byte accesses allowed in bias, r, y, z
};

// 8 consecutive values of row `row` from column c on, of which nc (1..8) exist
template <typename T>
__device__ __forceinline__ void load8(const void *base, int64_t at, int nc, int vec, float (&f)[8]) {
    const T *p = reinterpret_cast<const T *>(base) + at;
    if (vec && nc == 8) {
        Vec<T, 8> u;
        u.load(p);
        u.get(f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = i < nc ? to_f32(p[i]) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store8(void *base, int64_t at, int nc, int vec, const float (&f)[8]) {
    T *p = reinterpret_cast<T *>(base) + at;
    if (vec && nc == 8) {
        Vec<T, 8> u;
        u.set(f);
        u.store(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < nc) p[i] = from_f32<T>(f[i]);
    }
}

// bias, activation, residual and the stores of 8 values
template <typename T>
__device__ __forceinline__ void finish8(const Epilogue &e, int64_t row, int64_t c, int nc, float (&v)[8]) {
    float f[8];
    if (e.bias) {
        load8<T>(e.bias, c, nc, e.vec, f);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] += f[i];
    }
    if (e.z) store8<T>(e.z, row * e.ldz + c, nc, e.vec, v);
    act_all(v, e.act);
    if (e.r) {
        load8<T>(e.r, row * e.ldr + c, nc, e.vec, f);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] += f[i];
    }
    store8<T>(e.y, row * e.ldy + c, nc, e.vec, v);
}

// 32 consecutive values of a row, all there and aligned: the residual and the bias
// are loaded a step ahead, so that their latency is not in the way of the stores.
template <typename T>
struct Ahead {
    Vec<T, 8> r[4], b[4];
    __device__ __forceinline__ void load(const Epilogue &e, int64_t row, int64_t c) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (e.r) r[j].load(reinterpret_cast<const T *>(e.r) + row * e.ldr + c + 8 * j);
            if (e.bias) b[j].load(reinterpret_cast<const T *>(e.bias) + c + 8 * j);
        }
    }
};
template <typename T>
__device__ __forceinline__ void finish32(const Epilogue &e, int64_t row, int64_t c, const Ahead<T> &in, float (&v)[32]) {
    float f[8];
    if (e.bias)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            in.b[j].get(f);
#pragma unroll
            for (int i = 0; i < 8; i++) v[8 * j + i] += f[i];
        }
    Vec<T, 8> u;
    if (e.z)
#pragma unroll
        for (int j = 0; j < 4; j++) u.set(v + 8 * j), u.store(reinterpret_cast<T *>(e.z) + row * e.ldz + c + 8 * j);
    act_all(v, e.act);
    if (e.r)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            in.r[j].get(f);
#pragma unroll
            for (int i = 0; i < 8; i++) v[8 * j + i] += f[i];
        }
#pragma unroll
    for (int j = 0; j < 4; j++) u.set(v + 8 * j), u.store(reinterpret_cast<T *>(e.y) + row * e.ldy + c + 8 * j);
}

// 32 x 32 values, a row a lane, of which `rows` x `cols` exist, at rows that start
// anywhere: turned over in shared memory (32 x kTurnLd floats of the warp's own), so that a
// warp's accesses are a row's neighbours.
constexpr int kTurnLd = 33;
template <typename T>
__device__ __forceinline__ void finish_turned(const Epilogue &e, int64_t row, int rows, int64_t c, int cols,
                                              const float (&v)[32], float *turn) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 32; i++) turn[lane * kTurnLd + i] = v[i];
    __syncwarp();
    const bool in = lane < cols;
    c += lane;
    const float bias = e.bias && in ? to_f32(reinterpret_cast<const T *>(e.bias)[c]) : 0.f;
#pragma unroll 1
    for (int r = 0; r < rows; r += 8) {
        float w[8], f[8];
#pragma unroll
        for (int u = 0; u < 8; u++) {
            f[u] = e.r && in && r + u < rows ? to_f32(reinterpret_cast<const T *>(e.r)[(row + r + u) * e.ldr + c]) : 0.f;
            w[u] = turn[(r + u) * kTurnLd + lane] + bias;
        }
        if (e.z)
#pragma unroll
            for (int u = 0; u < 8; u++)
                if (in && r + u < rows) reinterpret_cast<T *>(e.z)[(row + r + u) * e.ldz + c] = from_f32<T>(w[u]);
        act_all(w, e.act);
#pragma unroll
        for (int u = 0; u < 8; u++)
            if (in && r + u < rows) reinterpret_cast<T *>(e.y)[(row + r + u) * e.ldy + c] = from_f32<T>(w[u] + f[u]);
    }
    __syncwarp();  // read before the warp's next values come
}

}  // namespace zs

// linear_few.cu: y for at most kFewRows rows of x, in one kernel without a workspace.
constexpr int kFewRows = 16;
cudaError_t zs_launch_linear_few(int type, int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx, const void *w,
                                 int64_t ldw, const zs::Epilogue &epi, cudaStream_t st, int64_t *launches);
