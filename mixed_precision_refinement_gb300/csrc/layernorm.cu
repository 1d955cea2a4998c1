// Layer norm of rows of d values, forward and backward.
//   forward:  mu = mean x, rs = (mean (x - mu)^2 + eps)^-1/2, h = (x - mu) rs,
//             y = h w + b
//   backward: a = dy w, dx = rs (a - mean a - h mean(a h)),
//             dw = sum over rows of dy h, db = sum over rows of dy
// Both are bound by HBM: each reads its inputs once and holds a row in
// registers between the reductions and the output.  All sums are float32.  The
// mean's own error, which grows with a row's common offset, is found again in
// the second pass over the registers: with m the float32 sum over d and
// e = mean (x - m), mu = m + e and mean (x - mu)^2 = mean (x - m)^2 - e^2, so h
// and rs lose no digits to an offset.  The backward pass has mu rounded to a
// float32, half a unit of its last place.
#include <algorithm>

#include "rownorm.cuh"

namespace {

using namespace zs;

// Forward: TPR threads hold a row, VE consecutive values at a time (VE = 1
// where rows are not 16-byte aligned), NI times; four rows a block of 128 threads
// where a warp holds one, else a row a block.  8 rows of 2048: 2.2 us, a launch;
// 32768 x 4096 bfloat16 111 us, 4.8 TB/s, bound by its instructions (3.2 of the 4
// issued a cycle: conversions, two passes of sums, the output; 107 us of it without the
// second reduction's sum of x - m).  A ring of rows as
// in the backward pass and packed float32 instructions were both slower: they
// take registers, and with them warps.
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
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = (i * TPR + t) * VE;
        if (c < d) {
#pragma unroll
            for (int e = 0; e < VE; e++) {
                const float z = v[i * VE + e] - mu;
                s.x = fmaf(z, z, s.x);
                s.y += z;
                v[i * VE + e] = z;
            }
        }
    }
    s = row_sum<TPR>(s, red, 1);
    const float off = s.y * inv, rs = inv_std(s.x * inv, off, eps), shift = -off * rs;
    if (t == 0) {
        if (mean) mean[row] = mu + off;
        if (rstd) rstd[row] = rs;
    }
    T *yr = y + row * ldy;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = (i * TPR + t) * VE;
        if (c < d) {
            float o[VE], f[VE];
#pragma unroll
            for (int e = 0; e < VE; e++) o[e] = fmaf(v[i * VE + e], rs, shift);
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

// Rows too long for the registers (1024 threads of 16 values each): one block a row,
// three passes (the second and third mostly from L2).
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
    s = 0.f;
    for (int64_t c = threadIdx.x; c < d; c += kLongThreads) {
        const float z = to_f32(xr[c]) - mu;
        q = fmaf(z, z, q);
        s += z;
    }
    const float2 r = row_sum<kLongThreads>(make_float2(q, s), red, 1);
    const float off = r.y / (float)d, rs = inv_std(r.x / (float)d, off, eps), shift = -off * rs;
    if (threadIdx.x == 0) {
        if (mean) mean[row] = mu + off;
        if (rstd) rstd[row] = rs;
    }
    for (int64_t c = threadIdx.x; c < d; c += kLongThreads) {
        float o = fmaf(to_f32(xr[c]) - mu, rs, shift);
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
    float mu_next = 0.f, rs_next = 0.f;
    if (row < rows) mu_next = mean[row], rs_next = rstd[row];
    fetch(row);
    int flip = 0;
    for (; row < rows; row += step, flip ^= 1) {  // TPR > 32: the same rows in all of the block's threads
        const float mu = mu_next, rs = rs_next;
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
        if (row + step < rows) mu_next = load_early(mean + row + step), rs_next = load_early(rstd + row + step);
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

// The same for longer rows, where registers alone do not keep enough bytes on
// their way: rows of x and dy arrive in a ring of kRing rows in shared memory, a
// bulk copy each, issued as soon as a row's reduction shows that every thread
// has read it.  A row need not start on 16 bytes (the tensors do): the copy takes
// the whole 16 bytes that begin in it, and the last values are read directly.
// mean and rstd are fetched two rows ahead.  32768 x 4096 bfloat16: 148 us and 7
// for the sums, 5.4 TB/s of the 6.8 that a copy reaches; 6614 x 2157 float32 46 and
// 5 us (a value at a time); without the ring 306 and 86 us in all.
constexpr int kRing = 4;
// threads of an SM that hold E values each: up to 85 or 64 registers
template <int E>
__host__ __device__ constexpr int ring_threads() {
    return E > 8 ? 768 : 1024;
}

template <typename T, int VE, int TPR, int NI>
__global__ void __launch_bounds__(TPR, ring_threads<NI * VE>() / TPR > 0 ? ring_threads<NI * VE>() / TPR : 1)
k_layernorm_bwd_ring(const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx,
                     const float *__restrict__ mean, const float *__restrict__ rstd, const void *__restrict__ w,
                     int wf32, int64_t rows, int d, T *__restrict__ dx, int64_t lddx, float *__restrict__ parts,
                     unsigned *__restrict__ status) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ float2 red[2 * (TPR / 32)];
    __shared__ __align__(8) uint64_t full[kRing];
    __shared__ volatile int s_abort;
    T *ring = reinterpret_cast<T *>(smem_raw);
    may_start_next();
    const int rr = ring_row<T>(d), t = threadIdx.x;
    void *ws = ring + 2 * kRing * rr;  // w, read again for every row
    if (w)
        for (int c = t; c < d; c += TPR) {
            if (wf32)
                reinterpret_cast<float *>(ws)[c] = reinterpret_cast<const float *>(w)[c];
            else
                reinterpret_cast<T *>(ws)[c] = reinterpret_cast<const T *>(w)[c];
        }
    constexpr int A = 16 / (int)sizeof(T);
    const float inv = 1.f / (float)d;
    if (t == 0) {
        s_abort = 0;
        for (int i = 0; i < kRing; i++) bar_init(&full[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    // a row that starts at value `at` begins `off` values into its ring row (at most
    // one group of 16 bytes); its values 0 .. whole - off - 1 are copied
    auto offset = [&](int64_t at) { return (int)((unsigned)at % A); };
    auto whole = [&](int off) { return (off + d) / A * A; };
    auto issue = [&](int64_t row, int i) {
        const int64_t ax = row * ldx, ad = row * lddy;
        const int ox = offset(ax), od = offset(ad);
        const uint32_t bx = (uint32_t)(whole(ox) * sizeof(T)), bd = (uint32_t)(whole(od) * sizeof(T));
        bar_expect(&full[i], bx + bd);
        bulk_load(ring + 2 * i * rr, x + (ax - ox), bx, &full[i]);
        bulk_load(ring + (2 * i + 1) * rr, dy + (ad - od), bd, &full[i]);
    };
    // a block's rows are neighbours: eight of them share a sector of mean and rstd
    const int64_t row0 = rows * blockIdx.x / gridDim.x, row1 = rows * (blockIdx.x + 1) / gridDim.x;
    if (t == 0)
        for (int i = 0; i < kRing; i++)
            if (row0 + i < row1) issue(row0 + i, i);
    constexpr int NP = NI * VE / 2;  // pairs of values a thread holds
    float2 aw[NP], ab[NP];
#pragma unroll
    for (int i = 0; i < NP; i++) aw[i] = ab[i] = make_float2(0.f, 0.f);
    float mu_next = 0.f, rs_next = 0.f, mu_later = 0.f, rs_later = 0.f;
    if (row0 < row1) mu_next = mean[row0], rs_next = rstd[row0];
    if (row0 + 1 < row1) mu_later = mean[row0 + 1], rs_later = rstd[row0 + 1];
    int it = 0;
    for (int64_t row = row0; row < row1; row++, it++) {
        const float mu = mu_next, rs = rs_next;
        mu_next = mu_later, rs_next = rs_later;
        if (row + 2 < row1) mu_later = load_early(mean + row + 2), rs_later = load_early(rstd + row + 2);
        const int slot = it % kRing;
        bar_wait(&full[slot], (it / kRing) & 1, &s_abort, status);
        const int offx = offset(row * ldx), nx = whole(offx) - offx, offd = offset(row * lddy), nd = whole(offd) - offd;
        const T *xs = ring + 2 * slot * rr + offx, *ds = ring + (2 * slot + 1) * rr + offd;
        // values beyond the row count as zeros of dy
        float2 h[NP], a[NP], sx = make_float2(0.f, 0.f), sy = sx;
        const float2 rs2 = make_float2(rs, rs), nmu2 = make_float2(-mu, -mu);
        constexpr int G = VE > 1 ? VE : 2;  // values at a time
#pragma unroll
        for (int i = 0; i < NI * VE / G; i++) {
            float hf[G], af[G], wf[G];
#pragma unroll
            for (int e = 0; e < G; e++) hf[e] = af[e] = 0.f, wf[e] = 1.f;
            if (VE > 1) {
                const int c = (i * TPR + t) * VE;
                if (c < d) {  // whole 16 bytes: all of them copied
                    Vec<T, VE> u;
                    u.load(xs + c);
                    u.get(hf);
                    u.load(ds + c);
                    u.get(af);
                    if (w) load_ws<T, VE>(ws, wf32, c, wf);
                }
            } else {
#pragma unroll
                for (int e = 0; e < G; e++) {
                    const int c = (i * G + e) * TPR + t;
                    if (c < d) {
                        hf[e] = to_f32(c < nx ? xs[c] : x[row * ldx + c]);
                        af[e] = to_f32(c < nd ? ds[c] : dy[row * lddy + c]);
                        if (w) wf[e] = load_w<T>(ws, wf32, c);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < G / 2; e++) {
                const int j = i * (G / 2) + e;
                const float2 v = make_float2(af[2 * e], af[2 * e + 1]);
                // x - mu first: x rs - mu rs would lose the digits of a large offset
                h[j] = mul2(add2(make_float2(hf[2 * e], hf[2 * e + 1]), nmu2), rs2);
                aw[j] = fma2(v, h[j], aw[j]);
                ab[j] = add2(v, ab[j]);
                a[j] = w ? mul2(v, make_float2(wf[2 * e], wf[2 * e + 1])) : v;
                sx = add2(a[j], sx);
                sy = fma2(a[j], h[j], sy);
            }
        }
        float2 s = make_float2(sx.x + sx.y, sy.x + sy.y);
        s = row_sum<TPR>(s, red, it & 1);
        if (t == 0 && row + kRing < row1) issue(row + kRing, slot);
        const float m1 = -rs * s.x * inv, m2 = -rs * s.y * inv;
        const float2 m12 = make_float2(m1, m1), m22 = make_float2(m2, m2);
#pragma unroll
        for (int j = 0; j < NP; j++) a[j] = fma2(h[j], m22, fma2(a[j], rs2, m12));
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int c = (i * TPR + t) * VE;
            if (c < d) {
                float o[VE];
#pragma unroll
                for (int e = 0; e < VE; e++) o[e] = (i * VE + e) & 1 ? a[(i * VE + e) / 2].y : a[(i * VE + e) / 2].x;
                Vec<T, VE> r;
                r.set(o);
                r.store(dx + row * lddx + c);
            }
        }
    }
    if (t == 0 && s_abort) bar_drain(full, kRing, it);
    if (!parts) return;
    float *pw = parts + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = (i * TPR + t) * VE;
        if (c < d) {
#pragma unroll
            for (int e = 0; e < VE; e++) {
                const int j = i * VE + e;
                pw[c + e] = j & 1 ? aw[j / 2].y : aw[j / 2].x;
                pw[d + c + e] = j & 1 ? ab[j / 2].y : ab[j / 2].x;
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
    after_previous();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;  // column of [dw | db]
    float s = 0.f;
    if (c < 2 * d) {
#pragma unroll 8
        for (int64_t p = ty; p < nparts; p += 32) s += parts[p * 2 * d + c];
    }
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

// Blocks of the backward kernel (at most) for a row held by tpr threads.
int64_t bwd_blocks(int64_t rows, int tpr, int num_sms) {
    const int64_t groups = tpr == 32 ? (rows + 3) / 4 : rows;
    const int64_t per_sm = tpr == 32 ? 8 : tpr <= 128 ? 12 : tpr == 256 ? 6 : tpr == 512 ? 3 : 1;
    return std::max<int64_t>(1, std::min<int64_t>(groups, (int64_t)num_sms * std::max<int64_t>(1, per_sm)));
}

int bwd_tpr(int64_t d) { return d <= 256 ? 32 : d <= 1024 ? 128 : d <= 2048 ? 256 : d <= 4096 ? 512 : 1024; }

constexpr int64_t kColParts = 64;

template <typename T, int VE>
cudaError_t launch_bwd(int64_t rows, int d, const T *dy, int64_t lddy, const T *x, int64_t ldx, const float *mean,
                const float *rstd, const void *w, int wf32, T *dx, int64_t lddx, float *parts, int64_t *blocks,
                int num_sms, unsigned *status, cudaStream_t st) {
    // Short rows and tensors that do not start on 16 bytes: without the ring (32768 rows of 256
    // bfloat16: 30 us, 40 with it; of 512: 46 and 38, of 1024: 66 and 56).
    if (d > 256 && aligned16(x) && aligned16(dy)) {
        const size_t smem = (size_t)2 * kRing * ring_row<T>(d) * sizeof(T) + (w ? (size_t)d * (wf32 ? 4 : sizeof(T)) : 0);
#define LN_RING(TPR, E)                                                                                             \
    do {                                                                                                           \
        constexpr int kMost = 2 * kRing * ring_row<T>((TPR) * (E)) * (int)sizeof(T) + (TPR) * (E) * 4;               \
        static OncePerDevice limit;                                                                                \
        const cudaError_t attr = smem_limit(limit, k_layernorm_bwd_ring<T, VE, TPR, (E) / VE>, kMost);             \
        if (attr != cudaSuccess) return attr;                                                                      \
        const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>(ring_threads<E>() / (TPR), 227 * 1024 / (smem + 1536))); \
        *blocks = std::min({*blocks, rows, per_sm * num_sms});                                                     \
        k_layernorm_bwd_ring<T, VE, TPR, (E) / VE><<<(unsigned)*blocks, TPR, smem, st>>>(                           \
            dy, lddy, x, ldx, mean, rstd, w, wf32, rows, d, dx, lddx, parts, status);                              \
        return cudaGetLastError();                                                                                 \
    } while (0)
        // values a thread: 16 of them share the cost of a row's reduction best, but
        // read one by one they leave too few threads to hide their loads (6614 rows
        // of 2157 float32: 63 us with 16, 50 us with 8)
        constexpr int E = VE > 1 ? 16 : 8, F = VE > 1 ? 1 : 2;
        if (d <= 1024) LN_RING(64 * F, E);
        if (d <= 2048) LN_RING(128 * F, E);
        if (d <= 4096) LN_RING(256 * F, E);
        if ((size_t)2 * kRing * ring_row<T>(8192) * sizeof(T) + 8192 * 4 <= 220 * 1024) LN_RING(512 * F, E);
#undef LN_RING
    }
#define LN_GO(TPR, E)                                                                                              \
    k_layernorm_bwd<T, VE, TPR, (E) / VE><<<(unsigned)*blocks, (TPR) < 128 ? 128 : (TPR), 0, st>>>(                 \
        dy, lddy, x, ldx, mean, rstd, w, wf32, rows, d, dx, lddx, parts)
    if (d <= 256) LN_GO(32, 8);
    else if (d <= 1024) LN_GO(128, 8);
    else if (d <= 2048) LN_GO(256, 8);
    else if (d <= 4096) LN_GO(512, 8);
    else LN_GO(1024, 8);
#undef LN_GO
    return cudaGetLastError();
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
                int num_sms, unsigned *status, cudaStream_t st, int64_t *launches) {
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
        int64_t blocks = bwd_blocks(rows, bwd_tpr(d), num_sms);
        const bool vec = d % VE == 0 && ldx % VE == 0 && lddy % VE == 0 && lddx % VE == 0 && aligned16(x) &&
                         aligned16(dy) && aligned16(dx) && (wf32 || !w || aligned16(w));
        float *p = sums ? parts : nullptr;
        const cudaError_t e =
            vec ? launch_bwd<T, VE>(rows, (int)d, pd, lddy, px, ldx, mean, rstd, w, wf32, po, lddx, p, &blocks, num_sms, status, st)
                : launch_bwd<T, 1>(rows, (int)d, pd, lddy, px, ldx, mean, rstd, w, wf32, po, lddx, p, &blocks, num_sms, status, st);
        if (e != cudaSuccess) return e;
        ++*launches;
        nparts = blocks * (bwd_tpr(d) == 32 ? 4 : 1);
    }
    if (sums) {
        ++*launches;
        return launch(nparts > 0, k_layernorm_bwd_sum<T>, (unsigned)((2 * d + 31) / 32), 1024, 0, st, parts, nparts, d, wf32, dw, db);
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
                                    unsigned *status, cudaStream_t st, int64_t *launches) {
    if (type == ZSOLVE_F32)
        return bwd<float>(rows, d, dy, lddy, x, ldx, mean, rstd, w, wf32, dx, lddx, dw, db, parts, num_sms, status, st,
                   launches);
    if (type == ZSOLVE_BF16)
        return bwd<bf16>(rows, d, dy, lddy, x, ldx, mean, rstd, w, wf32, dx, lddx, dw, db, parts, num_sms, status, st,
                   launches);
    return bwd<f16>(rows, d, dy, lddy, x, ldx, mean, rstd, w, wf32, dx, lddx, dw, db, parts, num_sms, status, st,
                   launches);
}
