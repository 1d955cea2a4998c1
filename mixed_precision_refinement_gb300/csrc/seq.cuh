// Shared helpers of the sequence-layer operators (layer norm, linear, delta
// rule): the handle, its workspace, and loads and stores of the three element
// types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "zsolve.h"

struct zsolve_seq {
    cudaStream_t st = nullptr;
    cudaEvent_t ev = nullptr;  // orders the workspace's users when the stream changes
    void *ws = nullptr;
    size_t ws_bytes = 0;
    int num_sms = 0;
    int dev = 0;
    int64_t launches = 0;
    unsigned *d_status = nullptr;  // device status word of the bounded waits
    char err[256] = "";
};

namespace zs {

// Records the message and returns the status.
int seq_fail(zsolve_seq *s, int status, const char *fmt, ...);

// The handle's workspace of at least `bytes` (256-byte aligned), or NULL with
// the failure recorded in *status.  Growing waits for the device, and is
// refused during a stream capture.
void *seq_workspace(zsolve_seq *s, size_t bytes, int *status);

// Parts of one workspace, each 256-byte aligned: first with base = NULL to
// add up the size, then with the workspace to place them.
struct Carve {
    char *base;
    size_t at = 0;
    explicit Carve(void *b) : base((char *)b) {}
    template <typename T>
    T *take(size_t n) {
        const size_t here = at;
        at += (n * sizeof(T) + 255) / 256 * 256;
        return base ? (T *)(base + here) : nullptr;
    }
};

#define SEQ_CU(expr)                                                                                          \
    do {                                                                                                      \
        const cudaError_t e_ = (expr);                                                                        \
        if (e_ != cudaSuccess) return zs::seq_fail(s, ZSOLVE_ECUDA, "%s: %s", #expr, cudaGetErrorString(e_)); \
    } while (0)

inline size_t type_bytes(int type) { return type == ZSOLVE_F32 ? 4 : 2; }
inline bool type_ok(int type) { return type == ZSOLVE_F32 || type == ZSOLVE_BF16 || type == ZSOLVE_F16; }

using bf16 = __nv_bfloat16;
using f16 = __half;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(f16 x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ f16 from_f32<f16>(float x) { return __float2half_rn(x); }

// Two floats of a packed pair of 16-bit values, and back.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<bf16>(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<f16>(uint32_t u) {
    return __half22float2(*reinterpret_cast<__half2 *>(&u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<bf16>(float a, float b) {
    __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&p);
}
template <>
__device__ __forceinline__ uint32_t pack2<f16>(float a, float b) {
    __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&p);
}

// N consecutive values (N * sizeof(T) = 4, 8 or 16 bytes, so aligned) as floats.
template <typename T, int N>
struct Vec {
    static constexpr int kWords = N * (int)sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T *p) {
        if (kWords == 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            w[0] = u.x, w[1 % kWords] = u.y, w[2 % kWords] = u.z, w[3 % kWords] = u.w;
        } else if (kWords == 2) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x, w[1 % kWords] = u.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if (kWords == 4)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1 % kWords], w[2 % kWords], w[3 % kWords]);
        else if (kWords == 2)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1 % kWords]);
        else
            *reinterpret_cast<uint32_t *>(p) = w[0];
    }
    __device__ __forceinline__ void get(float *f) const {
#pragma unroll
        for (int i = 0; i < kWords; i++) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else {
                const float2 v = unpack2<T>(w[i]);
                f[2 * i] = v.x, f[2 * i + 1] = v.y;
            }
        }
    }
    __device__ __forceinline__ void set(const float *f) {
#pragma unroll
        for (int i = 0; i < kWords; i++) {
            if constexpr (sizeof(T) == 4)
                w[i] = __float_as_uint(f[i]);
            else
                w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
        }
    }
};
// one value (any alignment of the element itself)
template <typename T>
struct Vec<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void store(T *p) const { *p = v; }
    __device__ __forceinline__ void get(float *f) const { f[0] = to_f32(v); }
    __device__ __forceinline__ void set(const float *f) { v = from_f32<T>(f[0]); }
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

}  // namespace zs

// ---------------------------------------------------------------- launchers
// All return cudaGetLastError() of the last launch and add to *launches.

// layernorm.cu.  w and b (NULL: 1 and 0) hold float32 when wf32, else the type of x.
cudaError_t zs_launch_layernorm(int type, int wf32, int64_t rows, int64_t d, const void *x, int64_t ldx,
                                const void *w, const void *b, float eps, void *y, int64_t ldy, float *mean,
                                float *rstd, cudaStream_t st, int64_t *launches);
// parts: float32 partial sums of the weight's and the bias's gradients, as many as
// zs_layernorm_bwd_parts says (both may be NULL: not formed).
int64_t zs_layernorm_bwd_parts(int type, int64_t rows, int64_t d, int num_sms);
cudaError_t zs_launch_layernorm_bwd(int type, int wf32, int64_t rows, int64_t d, const void *dy, int64_t lddy,
                                    const void *x, int64_t ldx, const float *mean, const float *rstd, const void *w,
                                    void *dx, int64_t lddx, void *dw, void *db, float *parts, int num_sms,
                                    cudaStream_t st, int64_t *launches);

// linear.cu: the whole call (arguments checked), a ZSOLVE_* status.
int zs_linear(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx, const void *w,
              int64_t ldw, const void *b, int act, const void *r, int64_t ldr, void *y, int64_t ldy, void *z,
              int64_t ldz);
int zs_linear_bwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *dy, int64_t lddy,
                  const void *x, int64_t ldx, const void *w, int64_t ldw, int act, const void *z, int64_t ldz,
                  void *dx, int64_t lddx, void *dw, int64_t lddw, void *db);
