// Layer norm of rows of d values, forward and backward.
//   forward:  mu = mean x, rs = (mean (x - mu)^2 + eps)^-1/2, h = (x - mu) rs,
//             y = h w + b
//   backward: a = dy w, dx = rs (a - mean a - h mean(a h)),
//             dw = sum over rows of dy h, db = sum over rows of dy
// Both are bound by HBM: each reads its inputs once and holds a row in
// registers between the reductions and the output.  All sums are float32; the
// variance is taken around the mean in a second pass over the registers, so a
// large common offset of a row costs no digits.
#include <algorithm>

#include "seq.cuh"

namespace {

using namespace zs;

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
    float2 t = lane < NW ? r[lane] : make_float2(0.f, 0.f);
    t.x = warp_sum(t.x);
    t.y = warp_sum(t.y);
    return t;
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

// Forward: TPR threads hold a row, VE consecutive values at a time (VE = 1
// where rows are not 16-byte aligned), NI times.  kRpb rows a block of at
// least 128 threads.
template <typename T, int VE, int TPR, int NI>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
k_layernorm(const T *__restrict__ x, int64_t ldx, const void *__restrict__ w, const void *__restrict__ b, int wf32,
            int64_t rows, int d, float eps, T *__restrict__ y, int64_t ldy, float *__restrict__ mean,
            float *__restrict__ rstd) {
    __shared__ float2 red[TPR == 32 ? 1 : 2 * (TPR / 32)];
    const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    const int t = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
    if (row >= rows) return;  // whole rows leave: no barrier is missed
    const T *xr = x + row * ldx;
    float v[NI * VE];
    Vec<T, VE> u[NI];
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = (i * TPR + t) * VE;
        if (c < d) u[i].load(xr + c);
    }
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = (i * TPR + t) * VE;
        if (c < d) {
            u[i].get(v + i * VE);
#pragma unroll
            for (int e = 0; e < VE; e++) s.x += v[i * VE + e];
        }
    }
    const float inv = 1.f / (float)d;
    const float mu = row_sum<TPR>(s, red, 0).x * inv;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = (i * TPR + t) * VE;
        if (c < d) {
#pragma unroll
            for (int e = 0; e < VE; e++) {
                const float z = v[i * VE + e] - mu;
                q = fmaf(z, z, q);
            }
        }
    }
    const float var = row_sum<TPR>(make_float2(q, 0.f), red, 1).x * inv;
    const float rs = 1.f / sqrtf(var + eps);
    if (t == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
    }
    T *yr = y + row * ldy;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = (i * TPR + t) * VE;
        if (c < d) {
            float o[VE], f[VE];
#pragma unroll
            for (int e = 0; e < VE; e++) o[e] = (v[i * VE + e] - mu) * rs;
            if (w) {
                load_wv<T, VE>(w, wf32, c, f);
#pragma unroll
                for (int e = 0; e < VE; e++) o[e] *= f[e];
            }
            if (b) {
                load_wv<T, VE>(b, wf32, c, f);
#pragma unroll
                for (int e = 0; e < VE; e++) o[e] += f[e];
            }
            Vec<T, VE> r;
            r.set(o);
            r.store(yr + c);
        }
    }
}

// Rows too long for the registers: one block a row, three passes (the second
// and third mostly from L2).
constexpr int kLongThreads = 1024;
template <typename T>
__global__ void __launch_bounds__(kLongThreads)
k_layernorm_long(const T *__restrict__ x, int64_t ldx, const void *__restrict__ w, const void *__restrict__ b,
                 int wf32, int64_t d, float eps, T *__restrict__ y, int64_t ldy, float *__restrict__ mean,
                 float *__restrict__ rstd) {
    __shared__ float2 red[2 * (kLongThreads / 32)];
    const int64_t row = blockIdx.x;
    const T *xr = x + row * ldx;
    float s = 0.f, q = 0.f;
    for (int64_t c = threadIdx.x; c < d; c += kLongThreads) s += to_f32(xr[c]);
    const float mu = row_sum<kLongThreads>(make_float2(s, 0.f), red, 0).x / (float)d;
    for (int64_t c = threadIdx.x; c < d; c += kLongThreads) {
        const float z = to_f32(xr[c]) - mu;
        q = fmaf(z, z, q);
    }
    const float rs = 1.f / sqrtf(row_sum<kLongThreads>(make_float2(q, 0.f), red, 1).x / (float)d + eps);
    if (threadIdx.x == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
    }
    for (int64_t c = threadIdx.x; c < d; c += kLongThreads) {
        float o = (to_f32(xr[c]) - mu) * rs;
        if (w) o *= load_w<T>(w, wf32, c);
        if (b) o += load_w<T>(b, wf32, c);
        y[row * ldy + c] = from_f32<T>(o);
    }
}

// Backward: a block takes every gridDim.x-th group of rows and keeps, in
// registers, its columns' sums of dy h and dy over them; they leave once, as
// one row of partial sums a block, and k_layernorm_bwd_sum adds those in a
// fixed order (no atomics: the same result every time).
template <typename T, int VE, int TPR, int NI>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
k_layernorm_bwd(const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx,
                const float *__restrict__ mean, const float *__restrict__ rstd, const void *__restrict__ w, int wf32,
                int64_t rows, int d, T *__restrict__ dx, int64_t lddx, float *__restrict__ parts) {
    constexpr int RPB = TPR == 32 ? 4 : 1;
    __shared__ float2 red[TPR == 32 ? 1 : 2 * (TPR / 32)];
    const int sub = TPR == 32 ? threadIdx.x >> 5 : 0;
    const int t = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
    const float inv = 1.f / (float)d;
    float aw[NI * VE], ab[NI * VE];
#pragma unroll
    for (int i = 0; i < NI * VE; i++) aw[i] = ab[i] = 0.f;
    Vec<T, VE> ux[NI], ud[NI];
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + sub;
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int c = (i * TPR + t) * VE;
            if (c < d && r < rows) {
                ux[i].load(x + r * ldx + c);
                ud[i].load(dy + r * lddy + c);
            }
        }
    };
    fetch(row);
    int flip = 0;
    for (; row < rows; row += step, flip ^= 1) {  // TPR > 32: the same rows in all of the block's threads
        const float mu = mean[row], rs = rstd[row];
        float h[NI * VE], a[NI * VE];
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int c = (i * TPR + t) * VE;
            if (c < d) {
                ux[i].get(h + i * VE);
                ud[i].get(a + i * VE);
            }
        }
        fetch(row + step);  // the next row's loads run during this row's reduction
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int c = (i * TPR + t) * VE;
            if (c < d) {
                float f[VE];
                if (w) load_wv<T, VE>(w, wf32, c, f);
#pragma unroll
                for (int e = 0; e < VE; e++) {
                    const int j = i * VE + e;
                    h[j] = (h[j] - mu) * rs;
                    aw[j] = fmaf(a[j], h[j], aw[j]);
                    ab[j] += a[j];
                    if (w) a[j] *= f[e];
                    s.x += a[j];
                    s.y = fmaf(a[j], h[j], s.y);
                }
            }
        }
        s = row_sum<TPR>(s, red, flip);
        const float m1 = s.x * inv, m2 = s.y * inv;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int c = (i * TPR + t) * VE;
            if (c < d) {
                float o[VE];
#pragma unroll
                for (int e = 0; e < VE; e++) {
                    const int j = i * VE + e;
                    o[e] = rs * (a[j] - m1 - h[j] * m2);
                }
                Vec<T, VE> r;
                r.set(o);
                r.store(dx + row * lddx + c);
            }
        }
    }
    if (!parts) return;
    float *pw = parts + ((int64_t)blockIdx.x * RPB + sub) * 2 * d;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = (i * TPR + t) * VE;
        if (c < d) {
#pragma unroll
            for (int e = 0; e < VE; e++) {
                pw[c + e] = aw[i * VE + e];
                pw[d + c + e] = ab[i * VE + e];
            }
        }
    }
}

// Rows too long for the registers: dx with one block a row in two passes ...
template <typename T>
__global__ void __launch_bounds__(kLongThreads)
k_layernorm_bwd_long(const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx,
                     const float *__restrict__ mean, const float *__restrict__ rstd, const void *__restrict__ w,
                     int wf32, int64_t d, T *__restrict__ dx, int64_t lddx) {
    __shared__ float2 red[2 * (kLongThreads / 32)];
    const int64_t row = blockIdx.x;
    const float mu = mean[row], rs = rstd[row];
    float2 s = make_float2(0.f, 0.f);
    for (int64_t c = threadIdx.x; c < d; c += kLongThreads) {
        const float h = (to_f32(x[row * ldx + c]) - mu) * rs;
        const float a = to_f32(dy[row * lddy + c]) * (w ? load_w<T>(w, wf32, c) : 1.f);
        s.x += a;
        s.y = fmaf(a, h, s.y);
    }
    s = row_sum<kLongThreads>(s, red, 0);
    const float m1 = s.x / (float)d, m2 = s.y / (float)d;
    for (int64_t c = threadIdx.x; c < d; c += kLongThreads) {
        const float h = (to_f32(x[row * ldx + c]) - mu) * rs;
        const float a = to_f32(dy[row * lddy + c]) * (w ? load_w<T>(w, wf32, c) : 1.f);
        dx[row * lddx + c] = from_f32<T>(rs * (a - m1 - h * m2));
    }
}

// ... and the columns' sums with a thread a column over a share of the rows.
template <typename T>
__global__ void __launch_bounds__(256)
k_layernorm_bwd_cols(const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx,
                     const float *__restrict__ mean, const float *__restrict__ rstd, int64_t rows, int64_t d,
                     float *__restrict__ parts) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= d) return;
    float aw = 0.f, ab = 0.f;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const float a = to_f32(dy[r * lddy + c]);
        aw = fmaf(a, (to_f32(x[r * ldx + c]) - mean[r]) * rstd[r], aw);
        ab += a;
    }
    parts[(int64_t)blockIdx.y * 2 * d + c] = aw;
    parts[(int64_t)blockIdx.y * 2 * d + d + c] = ab;
}

// dw and db: column sums of the partial sums, 32 columns a block, 32 threads a
// column, added in a fixed order.
template <typename T>
__global__ void __launch_bounds__(1024)
k_layernorm_bwd_sum(const float *__restrict__ parts, int64_t nparts, int64_t d, int wf32, void *__restrict__ dw,
                    void *__restrict__ db) {
    __shared__ float tile[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;  // column of [dw | db]
    float s = 0.f;
    if (c < 2 * d)
        for (int64_t p = ty; p < nparts; p += 32) s += parts[p * 2 * d + c];
    tile[ty][tx] = s;
    __syncthreads();
    const float v = warp_sum(tile[tx][ty]);
    const int64_t o = (int64_t)blockIdx.x * 32 + ty;
    if (tx != 0 || o >= 2 * d) return;
    void *dst = o < d ? dw : db;
    const int64_t i = o < d ? o : o - d;
    if (!dst) return;
    if (wf32)
        reinterpret_cast<float *>(dst)[i] = v;
    else
        reinterpret_cast<T *>(dst)[i] = from_f32<T>(v);
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Longest rows held in registers.
constexpr int64_t kMaxRow = 16384;
constexpr int64_t kMaxRowBwd = 8192;

template <typename T, int VE>
void launch_fwd(int64_t rows, int d, const T *x, int64_t ldx, const void *w, const void *b, int wf32, float eps, T *y,
                int64_t ldy, float *mean, float *rstd, cudaStream_t st) {
#define LN_GO(TPR, E)                                                                                              \
    k_layernorm<T, VE, TPR, (E) / VE>                                                                              \
        <<<(unsigned)((TPR) == 32 ? (rows + 3) / 4 : rows), (TPR) < 128 ? 128 : (TPR), 0, st>>>(                   \
            x, ldx, w, b, wf32, rows, d, eps, y, ldy, mean, rstd)
    if (d <= 256) LN_GO(32, 8);
    else if (d <= 512) LN_GO(32, 16);
    else if (d <= 1024) LN_GO(128, 8);
    else if (d <= 2048) LN_GO(256, 8);
    else if (d <= 4096) LN_GO(256, 16);
    else if (d <= 8192) LN_GO(512, 16);
    else LN_GO(1024, 16);
#undef LN_GO
}

// Blocks of the backward kernel for a row held by tpr threads.
int64_t bwd_blocks(int64_t rows, int tpr, int num_sms) {
    const int64_t groups = tpr == 32 ? (rows + 3) / 4 : rows;
    const int64_t per_sm = tpr <= 128 ? 8 : 1024 / tpr * 1;
    return std::max<int64_t>(1, std::min<int64_t>(groups, (int64_t)num_sms * std::max<int64_t>(1, per_sm)));
}

int bwd_tpr(int64_t d) { return d <= 256 ? 32 : d <= 1024 ? 128 : d <= 2048 ? 256 : d <= 4096 ? 512 : 1024; }

constexpr int64_t kColParts = 64;

template <typename T, int VE>
void launch_bwd(int64_t rows, int d, const T *dy, int64_t lddy, const T *x, int64_t ldx, const float *mean,
                const float *rstd, const void *w, int wf32, T *dx, int64_t lddx, float *parts, int64_t blocks,
                cudaStream_t st) {
#define LN_GO(TPR, E)                                                                                              \
    k_layernorm_bwd<T, VE, TPR, (E) / VE><<<(unsigned)blocks, (TPR) < 128 ? 128 : (TPR), 0, st>>>(                 \
        dy, lddy, x, ldx, mean, rstd, w, wf32, rows, d, dx, lddx, parts)
    if (d <= 256) LN_GO(32, 8);
    else if (d <= 1024) LN_GO(128, 8);
    else if (d <= 2048) LN_GO(256, 8);
    else if (d <= 4096) LN_GO(512, 8);
    else LN_GO(1024, 8);
#undef LN_GO
}

template <typename T>
cudaError_t fwd(int64_t rows, int64_t d, const void *x, int64_t ldx, const void *w, const void *b, int wf32, float eps,
                void *y, int64_t ldy, float *mean, float *rstd, cudaStream_t st) {
    constexpr int VE = 16 / (int)sizeof(T);
    const T *px = (const T *)x;
    T *py = (T *)y;
    const bool vec = d % VE == 0 && ldx % VE == 0 && ldy % VE == 0 && aligned16(x) && aligned16(y) &&
                     (wf32 || ((!w || aligned16(w)) && (!b || aligned16(b))));
    if (d > kMaxRow)
        k_layernorm_long<T><<<(unsigned)rows, kLongThreads, 0, st>>>(px, ldx, w, b, wf32, d, eps, py, ldy, mean, rstd);
    else if (vec)
        launch_fwd<T, VE>(rows, (int)d, px, ldx, w, b, wf32, eps, py, ldy, mean, rstd, st);
    else
        launch_fwd<T, 1>(rows, (int)d, px, ldx, w, b, wf32, eps, py, ldy, mean, rstd, st);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(int64_t rows, int64_t d, const void *dy, int64_t lddy, const void *x, int64_t ldx, const float *mean,
                const float *rstd, const void *w, int wf32, void *dx, int64_t lddx, void *dw, void *db, float *parts,
                int num_sms, cudaStream_t st, int64_t *launches) {
    constexpr int VE = 16 / (int)sizeof(T);
    const T *pd = (const T *)dy, *px = (const T *)x;
    T *po = (T *)dx;
    const bool sums = dw || db;
    int64_t nparts = 0;
    if (rows > 0 && d > kMaxRowBwd) {
        k_layernorm_bwd_long<T><<<(unsigned)rows, kLongThreads, 0, st>>>(pd, lddy, px, ldx, mean, rstd, w, wf32, d, po,
                                                                         lddx);
        ++*launches;
        if (sums) {
            nparts = std::min(rows, kColParts);
            k_layernorm_bwd_cols<T><<<dim3((unsigned)((d + 255) / 256), (unsigned)nparts), 256, 0, st>>>(
                pd, lddy, px, ldx, mean, rstd, rows, d, parts);
            ++*launches;
        }
    } else if (rows > 0) {
        const int64_t blocks = bwd_blocks(rows, bwd_tpr(d), num_sms);
        const bool vec = d % VE == 0 && ldx % VE == 0 && lddy % VE == 0 && lddx % VE == 0 && aligned16(x) &&
                         aligned16(dy) && aligned16(dx) && (wf32 || !w || aligned16(w));
        float *p = sums ? parts : nullptr;
        if (vec)
            launch_bwd<T, VE>(rows, (int)d, pd, lddy, px, ldx, mean, rstd, w, wf32, po, lddx, p, blocks, st);
        else
            launch_bwd<T, 1>(rows, (int)d, pd, lddy, px, ldx, mean, rstd, w, wf32, po, lddx, p, blocks, st);
        ++*launches;
        nparts = blocks * (bwd_tpr(d) == 32 ? 4 : 1);
    }
    if (sums) {
        k_layernorm_bwd_sum<T><<<(unsigned)((2 * d + 31) / 32), 1024, 0, st>>>(parts, nparts, d, wf32, dw, db);
        ++*launches;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t zs_launch_layernorm(int type, int wf32, int64_t rows, int64_t d, const void *x, int64_t ldx,
                                const void *w, const void *b, float eps, void *y, int64_t ldy, float *mean,
                                float *rstd, cudaStream_t st, int64_t *launches) {
    if (rows <= 0) return cudaSuccess;
    ++*launches;
    if (type == ZSOLVE_F32) return fwd<float>(rows, d, x, ldx, w, b, wf32, eps, y, ldy, mean, rstd, st);
    if (type == ZSOLVE_BF16) return fwd<bf16>(rows, d, x, ldx, w, b, wf32, eps, y, ldy, mean, rstd, st);
    return fwd<f16>(rows, d, x, ldx, w, b, wf32, eps, y, ldy, mean, rstd, st);
}

int64_t zs_layernorm_bwd_parts(int, int64_t rows, int64_t d, int num_sms) {
    if (rows <= 0) return 0;
    if (d > kMaxRowBwd) return std::min(rows, kColParts) * 2 * d;
    return bwd_blocks(rows, bwd_tpr(d), num_sms) * (bwd_tpr(d) == 32 ? 4 : 1) * 2 * d;
}

cudaError_t zs_launch_layernorm_bwd(int type, int wf32, int64_t rows, int64_t d, const void *dy, int64_t lddy,
                                    const void *x, int64_t ldx, const float *mean, const float *rstd, const void *w,
                                    void *dx, int64_t lddx, void *dw, void *db, float *parts, int num_sms,
                                    cudaStream_t st, int64_t *launches) {
    if (type == ZSOLVE_F32)
        return bwd<float>(rows, d, dy, lddy, x, ldx, mean, rstd, w, wf32, dx, lddx, dw, db, parts, num_sms, st, launches);
    if (type == ZSOLVE_BF16)
        return bwd<bf16>(rows, d, dy, lddy, x, ldx, mean, rstd, w, wf32, dx, lddx, dw, db, parts, num_sms, st, launches);
    return bwd<f16>(rows, d, dy, lddy, x, ldx, mean, rstd, w, wf32, dx, lddx, dw, db, parts, num_sms, st, launches);
}
