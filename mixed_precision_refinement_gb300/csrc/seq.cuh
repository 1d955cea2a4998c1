// Shared helpers of the sequence-layer operators (layer norm, linear, delta
// rule): the handle, its workspace, and loads and stores of the three element
// types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <vector>

#include "device_once.h"
#include "zsolve.h"

struct zsolve_seq {
    cudaStream_t st = nullptr;
    cudaEvent_t ev = nullptr;  // orders the workspace's users when the stream changes
    cudaStream_t side = nullptr;           // beside st within a call; st waits for it before the call returns
    cudaEvent_t fork = nullptr, joined = nullptr;
    void *ws = nullptr;
    size_t ws_bytes = 0;
    bool ws_captured = false;      // a captured graph uses ws: it is kept until the handle goes
    std::vector<void *> retired;   // such workspaces that a larger one took the place of
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

// mbarriers and bulk copies.  Waits are bounded: on give-up the block's abort
// word and the status word are set, and every later wait of the block returns at
// once, so that all of its threads run to their end.
__device__ __forceinline__ void bar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"((uint32_t)__cvta_generic_to_shared(bar)), "r"(count)
                 : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"((uint32_t)__cvta_generic_to_shared(bar)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"((uint32_t)__cvta_generic_to_shared(bar)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"((uint32_t)__cvta_generic_to_shared(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
constexpr uint32_t kWaitLimit = 1u << 19;  // about a second
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, volatile int *abort_word, unsigned *status) {
    for (uint32_t it = 0; !bar_try(bar, parity); it++) {
        if (*abort_word) return false;
        if (it >= kWaitLimit) {
            *abort_word = 1;
            atomicOr(status, 1u);
            return false;
        }
    }
    return true;
}
// After a give-up, before the block ends: a bounded wait for the copies in flight
// among the last `stages` of `n` fills of a ring.
__device__ __forceinline__ void bar_drain(uint64_t *full, int stages, int n) {
    for (int q = n > stages ? n - stages : 0; q < n; q++)
        for (uint32_t i = 0; i < kWaitLimit && !bar_try(&full[q % stages], (q / stages) & 1); i++) {
        }
}
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(bytes), "r"((uint32_t)__cvta_generic_to_shared(bar))
                 : "memory");
}

// A kernel that follows another of the same call is launched with `next`: its blocks
// may be set up while the one before still runs, and wait in after_previous() until
// all of that one's results are there.  Every kernel that is launched so, or before
// one that is, calls after_previous() before it touches memory and may_start_next()
// when its own blocks are placed.  It hides the launches' gaps and set-up: linear of
// 801 x 1000 x 2157 (three kernels) 25.9 -> 20.5 us, layer norm backward of 6614 x 2157
// (two) 55.1 -> 51.3.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void may_start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... P, typename... A>
inline cudaError_t launch(bool next, void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid, cfg.blockDim = dim3((unsigned)threads), cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cfg.attrs = &attr, cfg.numAttrs = next ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// The kernel's limit of dynamic shared memory, which holds for the current device alone; a
// launcher keeps one OncePerDevice for each of its kernels.
template <typename K>
inline cudaError_t smem_limit(OncePerDevice &once, K kernel, int bytes) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return once.run(dev, [&] {
        const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (r != cudaSuccess) cudaGetLastError();  // told here, and not by the next launch
        return r;
    });
}

// Two float32 operations in one instruction, each rounded on its own: half the
// issue slots where those are what a kernel runs out of.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

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
                                    unsigned *status, cudaStream_t st, int64_t *launches);

// linear.cu: the whole call (arguments checked), a ZSOLVE_* status.
int zs_linear(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx, const void *w,
              int64_t ldw, const void *b, int act, const void *r, int64_t ldr, void *y, int64_t ldy, void *z,
              int64_t ldz);
int zs_linear_bwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *dy, int64_t lddy,
                  const void *x, int64_t ldx, const void *w, int64_t ldw, int act, const void *z, int64_t ldz,
                  void *dx, int64_t lddx, void *dw, int64_t lddw, void *db);
