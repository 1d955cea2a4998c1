// The join of a block and the residual stream: the norm of the block's output, its gate and
// residual scale, the sum, and the norm in front of the next block, in one pass.
//   h1 = (o - mu1) rs1, t = h1 w1 + b1, y = x + c act(z) t, h2 = (y - mu2) rs2, h = h2 w2 + b2
//   (layer norm: mu the row's mean, rs = (mean (v - mu)^2 + eps)^-1/2; root mean square: mu = 0;
//   without the first norm: mu1 = 0, rs1 = 1)
// and backwards, a2 = dh w2, norm'(a, h, rs) = rs (a - mean a - h mean(a h)) (root mean square:
// without mean a):
//   dx = dy + norm'(a2, h2, rs2), p = dx c act(z) (the gradient of t),
//   do = norm'(p w1, h1, rs1), dz = dx c t act'(z),
//   dw1 = sum p h1, db1 = sum p, dw2 = sum dh h2, db2 = sum dh over the rows,
//   dc = sum dx act(z) t.
// With u = dx act(z), Q = sum u h1 and R = sum u: dw1 = c Q, db1 = c R, dc = w1 Q + b1 R, so four
// sums a column serve all five.
// Both are bound by HBM: each tensor crosses it once, a row is held in registers between its
// reductions.  16384 x 4096 bfloat16 with a gate: 127 us, 5.0 TB/s; backwards, 32768 x 4096, 518 us and 7 for the weights' sums, 4.1 TB/s, bound by what a row's
// two reductions wait for with 16 warps an SM.  Sums, statistics and what lies between the norms are float32; y is rounded for
// memory alone, and h comes from the value before that rounding.  As in layernorm.cu, a mean's
// own error is found again in the second pass.
#include <algorithm>

#include "linear.cuh"
#include "rownorm.cuh"

namespace {

using namespace zs;

// What the kernels take beside the tensors' places.
struct ResGeom {
    const void *w1, *b1, *c, *w2, *b2;  // d values each; NULL: ones, zeros, ones, ...
    int wf32;                           // they are float32, else of the tensors' type
    int64_t rows;
    int d;
    float eps;
    int act, after, rms;
};

// 1 / sqrt(mean square + eps) and the correction of the mean, from the sums over a row of
// (v - m)^2 and v - m.
struct Stat {
    float rs, off;
};
__device__ __forceinline__ Stat stat_of(float2 s, float inv, float eps, int rms) {
    Stat r;
    r.off = rms ? 0.f : s.y * inv;
    r.rs = inv_std(s.x * inv, r.off, eps);
    return r;
}

// Two values at a time.  In both directions the instructions count as much as the bytes: a value of a row takes the share of a
// pair of each of its own, so they are held to pairs (packed float32) wherever neither memory nor the gate is concerned.
__device__ __forceinline__ float2 pair(const float *f, int j) { return make_float2(f[2 * j], f[2 * j + 1]); }
__device__ __forceinline__ void put(float *f, int j, float2 v) { f[2 * j] = v.x, f[2 * j + 1] = v.y; }
// f(j): each j of N / 2 pairs; g(e): the value left over
template <int N, typename F, typename G>
__device__ __forceinline__ void pairs(F f, G g) {
#pragma unroll
    for (int j = 0; j < N / 2; j++) f(j);
    if (N % 2) g(N - 1);
}
template <int N>
__device__ __forceinline__ void times(float *a, const float *b) {
    pairs<N>([&](int j) { put(a, j, mul2(pair(a, j), pair(b, j))); }, [&](int e) { a[e] *= b[e]; });
}
template <int N>
__device__ __forceinline__ void plus(float *a, const float *b) {
    pairs<N>([&](int j) { put(a, j, add2(pair(a, j), pair(b, j))); }, [&](int e) { a[e] += b[e]; });
}
// a = a s + b for two numbers s and b
template <int N>
__device__ __forceinline__ void scale_shift(float *a, float s, float b) {
    pairs<N>([&](int j) { put(a, j, fma2(pair(a, j), both(s), both(b))); }, [&](int e) { a[e] = fmaf(a[e], s, b); });
}

// Forward: TPR threads hold a row, VE consecutive values at a time (VE = 1 where rows are not
// 16-byte aligned), NI times; four rows a block where a warp holds one, else a row a block.  Sixteen values a thread: the sums over the
// threads are then a small part of the instructions, and half of an SM's threads have their rows in flight (eight a thread, in scalar
// arithmetic: 156 us for 127).
template <typename T, int VE, int TPR, int NI>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, TPR < 128 ? 8 : 1024 / TPR)
k_resnorm(const T *x, int64_t ldx, const T *__restrict__ o, int64_t ldo, const T *__restrict__ z, int64_t ldz, const ResGeom g,
          T *y, int64_t ldy, T *__restrict__ h, int64_t ldh, float *__restrict__ stats) {
    __shared__ float2 red[TPR == 32 ? 1 : 2 * (TPR / 32)];
    const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    const int t = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
    if (row >= g.rows) return;  // whole rows leave: no barrier is missed
    const int d = g.d;
    Vec<T, VE> ux[NI], uo[NI], uz[NI];
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = (i * TPR + t) * VE;
        if (c < d) {
            uo[i].load(o + row * ldo + c);
            ux[i].load(x + row * ldx + c);
            if (z) uz[i].load(z + row * ldz + c);
        }
    }
    const float inv = 1.f / (float)d;
    float v[NI * VE];
    auto each = [&](auto f) {  // f(i, c, values): the thread's pieces of the row
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int c = (i * TPR + t) * VE;
            if (c < d) f(i, c, v + i * VE);
        }
    };
    int flip = 0;
    // v - its mean, and the statistics: the mean first, unless it counts as zero
    auto standard = [&](float &mu) {
        float2 s = make_float2(0.f, 0.f);
        mu = 0.f;
        if (!g.rms) {
            each([&](int, int, float *a) { pairs<VE>([&](int j) { s = add2(s, pair(a, j)); }, [&](int e) { s.x += a[e]; }); });
            mu = row_sum<TPR>(make_float2(s.x + s.y, 0.f), red, flip).x * inv;
            flip ^= 1;
        }
        float2 q = make_float2(0.f, 0.f);
        s = q;
        each([&](int, int, float *a) {
            scale_shift<VE>(a, 1.f, -mu);
            pairs<VE>([&](int j) { q = fma2(pair(a, j), pair(a, j), q), s = add2(s, pair(a, j)); },
                      [&](int e) { q.x = fmaf(a[e], a[e], q.x), s.x += a[e]; });
        });
        s = row_sum<TPR>(make_float2(q.x + q.y, s.x + s.y), red, flip);
        flip ^= 1;
        return stat_of(s, inv, g.eps, g.rms);
    };
    each([&](int i, int, float *a) { uo[i].get(a); });
    float mu1 = 0.f, mu2;
    Stat s1 = {1.f, 0.f};
    if (g.after) s1 = standard(mu1);
    const float shift1 = -s1.off * s1.rs;
    each([&](int i, int c, float *a) {
        float f[VE], w[VE];
        if (g.after) scale_shift<VE>(a, s1.rs, shift1);
        if (g.w1) {
            load_ws<T, VE>(g.w1, g.wf32, c, f);
            times<VE>(a, f);
        }
        if (g.b1) {
            load_ws<T, VE>(g.b1, g.wf32, c, f);
            plus<VE>(a, f);
        }
        if (z) {
            float r[VE];
            uz[i].get(f);
            gates_all<false>(f, g.act, r, r);
            times<VE>(a, r);
        }
        if (g.c) {
            load_ws<T, VE>(g.c, g.wf32, c, f);
            times<VE>(a, f);
        }
        ux[i].get(w);
        plus<VE>(a, w);
        Vec<T, VE> r;
        r.set(a);
        r.store(y + row * ldy + c);
    });
    const Stat s2 = standard(mu2);
    const float shift2 = -s2.off * s2.rs;
    if (t == 0 && stats) {
        float *p = stats + 4 * row;
        p[0] = mu1 + s1.off, p[1] = s1.rs, p[2] = mu2 + s2.off, p[3] = s2.rs;
    }
    each([&](int, int c, float *a) {
        float f[VE];
        scale_shift<VE>(a, s2.rs, shift2);
        if (g.w2) {
            load_ws<T, VE>(g.w2, g.wf32, c, f);
            times<VE>(a, f);
        }
        if (g.b2) {
            load_ws<T, VE>(g.b2, g.wf32, c, f);
            plus<VE>(a, f);
        }
        Vec<T, VE> r;
        r.set(a);
        r.store(h + row * ldh + c);
    });
}

// Rows too long for the registers: one block a row in passes over it, mostly from L2.
constexpr int kLong = 1024;
template <typename T>
struct ResValue {  // y before its rounding
    const T *x, *o, *z;
    const ResGeom &g;
    float mu1, rs1;
    __device__ __forceinline__ float t(int64_t c) const {
        float a = (to_f32(o[c]) - mu1) * rs1;
        if (g.w1) a *= load_w<T>(g.w1, g.wf32, c);
        if (g.b1) a += load_w<T>(g.b1, g.wf32, c);
        return a;
    }
    __device__ __forceinline__ float operator()(int64_t c) const {
        float a[1] = {1.f};
        if (z) {
            a[0] = to_f32(z[c]);
            act_all(a, g.act);
        }
        const float v = a[0] * t(c);
        return fmaf(g.c ? load_w<T>(g.c, g.wf32, c) : 1.f, v, to_f32(x[c]));
    }
};
template <typename T>
__global__ void __launch_bounds__(kLong)
k_resnorm_long(const T *x, int64_t ldx, const T *__restrict__ o, int64_t ldo, const T *__restrict__ z, int64_t ldz, const ResGeom g,
               T *y, int64_t ldy, T *__restrict__ h, int64_t ldh, float *__restrict__ stats) {
    __shared__ float2 red[2 * (kLong / 32)];
    const int64_t row = blockIdx.x;
    ResValue<T> val{x + row * ldx, o + row * ldo, z ? z + row * ldz : nullptr, g, 0.f, 1.f};
    int flip = 0;
    auto standard = [&](auto f, float &mu) {
        float2 s = make_float2(0.f, 0.f);
        mu = 0.f;
        if (!g.rms) {
            for (int c = threadIdx.x; c < g.d; c += kLong) s.x += f(c);
            mu = row_sum<kLong>(s, red, flip).x / (float)g.d;
            flip ^= 1;
            s = make_float2(0.f, 0.f);
        }
        for (int c = threadIdx.x; c < g.d; c += kLong) {
            const float w = f(c) - mu;
            s.x = fmaf(w, w, s.x);
            s.y += w;
        }
        s = row_sum<kLong>(s, red, flip);
        flip ^= 1;
        const Stat r = stat_of(s, 1.f / (float)g.d, g.eps, g.rms);
        mu += r.off;
        return r.rs;
    };
    if (g.after) {
        float mu1;
        const float rs1 = standard([&](int c) { return to_f32(val.o[c]); }, mu1);
        val.mu1 = mu1, val.rs1 = rs1;
    }
    float mu2;
    const float rs2 = standard(val, mu2);
    if (threadIdx.x == 0 && stats) {
        float *p = stats + 4 * row;
        p[0] = val.mu1, p[1] = val.rs1, p[2] = mu2, p[3] = rs2;
    }
    for (int c = threadIdx.x; c < g.d; c += kLong) {
        const float w = val(c);
        y[row * ldy + c] = from_f32<T>(w);
        float a = (w - mu2) * rs2;
        if (g.w2) a *= load_w<T>(g.w2, g.wf32, c);
        if (g.b2) a += load_w<T>(g.b2, g.wf32, c);
        h[row * ldh + c] = from_f32<T>(a);
    }
}

// ---------------------------------------------------------------- backward

struct ResBack {
    const void *dh, *dy, *y, *o, *z;  // dy NULL: zeros; z NULL: no gate
    int64_t lddh, lddy, ldy, ldo, ldz;
    const float *stats;
    void *dx, *dout, *dz;             // dz NULL: not formed
    int64_t lddx, lddo, lddz;
};

// A block takes a share of the rows, which arrive in a ring of rows in shared memory, a bulk copy
// for each of the up to five tensors and the statistics, issued as soon as the row's second reduction shows that every
// thread has read it.  Two rows go side by side and share what a reduction waits for (32768 x 4096 bfloat16: 610 us one by one, 540).  A thread holds 8 values of a row (16 where the row has more than 4096) and its columns' four sums; the
// weights lie in shared memory.  A row need not start or end on 16 bytes (the tensors start there): the copy takes what lies around it
// too, but for a tensor's last values, which the threads put in place.
template <int N>
struct Count {
    static constexpr int value = N;
};
// Sums over the block of v[k], N rows' at once; `red`: N slots a warp, which the next sums may not use.  A shuffle moves two values
// that are still to be added up: lanes that differ in its bit keep one of them each.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float2 (&v)[N], float2 *red) {
    constexpr int NW = TPR / 32, V = 2 * N;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto fold = [&](float a, float b, int o) {  // of a pair of lanes the lower has the sum of a's, the upper that of b's
        const bool up = lane & o;
        return (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, o);
    };
    float x = N == 1 ? fold(v[0].x, v[0].y, 16) : fold(fold(v[0].x, v[N - 1].x, 16), fold(v[0].y, v[N - 1].y, 16), 8);
#pragma unroll
    for (int o = N == 1 ? 8 : 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    // value lane * V / 32: of row k its x, then its y
    if (TPR == 32) {
#pragma unroll
        for (int k = 0; k < N; k++) v[k] = make_float2(__shfl_sync(0xffffffffu, x, 32 / N * k), __shfl_sync(0xffffffffu, x, 32 / N * k + 32 / V));
        return;
    }
    float *to = reinterpret_cast<float *>(red);
    if (lane % (32 / V) == 0) to[warp * V + lane / (32 / V)] = x;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; k++) v[k] = red[k];
#pragma unroll
    for (int w = 1; w < NW; w++)
#pragma unroll
        for (int k = 0; k < N; k++) v[k] = add2(v[k], red[w * N + k]);
}
constexpr int ring_blocks(int tpr) {  // of an SM, as far as the registers go
    return std::max(1, 65536 / (tpr * 128));
}
template <typename T, int VE, int TPR, int E>
__global__ void __launch_bounds__(TPR, ring_blocks(TPR))
k_resnorm_bwd(const ResBack p, const ResGeom g, int stages, float *__restrict__ parts, unsigned *__restrict__ status) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr int kMost = 8;
    __shared__ float2 red[4 * (TPR / 32)];
    __shared__ __align__(8) uint64_t full[kMost];
    __shared__ __align__(16) float s_stats[kMost][4];
    __shared__ volatile int s_abort;
    may_start_next();
    const int d = g.d, rr = ring_row<T>(d), t = threadIdx.x;
    const T *const src[5] = {(const T *)p.dh, (const T *)p.y, (const T *)p.o, (const T *)p.dy, (const T *)p.z};
    const int64_t lds[5] = {p.lddh, p.ldy, p.ldo, p.lddy, p.ldz};
    const int place[5] = {0, 1, 2, 3, p.dy ? 4 : 3};
    const int tensors = 3 + (p.dy ? 1 : 0) + (p.z ? 1 : 0);
    T *const ring = reinterpret_cast<T *>(smem_raw);
    const int wsize = ((g.wf32 ? 4 : (int)sizeof(T)) * d + 15) / 16 * 16;
    uint8_t *const wbase = smem_raw + (size_t)stages * tensors * rr * sizeof(T);
    const void *const weights[4] = {g.w1, g.b1, g.c, g.w2};
    const void *ws[4];
    {
        int n = 0;
#pragma unroll
        for (int k = 0; k < 4; k++) {
            ws[k] = nullptr;
            if (!weights[k]) continue;
            uint8_t *const w = wbase + (size_t)n++ * wsize;
            ws[k] = w;
            for (int c = t; c < d; c += TPR) {
                if (g.wf32)
                    reinterpret_cast<float *>(w)[c] = reinterpret_cast<const float *>(weights[k])[c];
                else
                    reinterpret_cast<T *>(w)[c] = reinterpret_cast<const T *>(weights[k])[c];
            }
        }
    }
    constexpr int A = 16 / (int)sizeof(T);
    const float inv = 1.f / (float)d;
    if (t == 0) {
        s_abort = 0;
        for (int i = 0; i < stages; i++) bar_init(&full[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    auto offset = [&](int64_t at) { return VE > 1 ? 0 : (int)((unsigned)at % A); };
    // values from the 16 bytes that a row begins in to those that it ends in, or begins to end in where those are the tensor's last
    auto whole = [&](int64_t row, int k) {
        if (VE > 1) return d;
        const int64_t at = row * lds[k];
        const int off = offset(at), n = (off + d + A - 1) / A * A;
        return at - off + n <= (g.rows - 1) * lds[k] + d ? n : (off + d) / A * A;
    };
    auto slot_of = [&](int slot, int k) { return (slot * tensors + place[k]) * rr; };
    auto issue = [&](int64_t row, int slot) {
        uint32_t bytes = 16;
#pragma unroll
        for (int k = 0; k < 5; k++)
            if (src[k]) bytes += (uint32_t)(whole(row, k) * sizeof(T));
        bar_expect(&full[slot], bytes);
        bulk_load(s_stats[slot], p.stats + 4 * row, 16, &full[slot]);
#pragma unroll
        for (int k = 0; k < 5; k++) {
            if (!src[k]) continue;
            const int64_t at = row * lds[k];
            const int off = offset(at), n = whole(row, k);
            if (n) bulk_load(ring + slot_of(slot, k), src[k] + (at - off), (uint32_t)(n * sizeof(T)), &full[slot]);
        }
    };
    const int64_t row0 = g.rows * blockIdx.x / gridDim.x, row1 = g.rows * (blockIdx.x + 1) / gridDim.x;
    if (t == 0)
        for (int i = 0; i < stages; i++)
            if (row0 + i < row1) issue(row0 + i, i);
    constexpr int NP = E / 2;
    float2 aq[NP], ar[NP], aw[NP], ab[NP];
#pragma unroll
    for (int i = 0; i < NP; i++) aq[i] = ar[i] = aw[i] = ab[i] = make_float2(0.f, 0.f);
    // the value i of the thread: columns are VE together, so i and i + 1 (i even) are a pair of them
    auto column = [&](int i) { return VE > 1 ? ((i / VE) * TPR + t) * VE + i % VE : i * TPR + t; };
    constexpr int R = E > 8 ? 1 : 2;
    const int step = R == 2 && stages >= 4 ? 2 : 1;
    int it = 0;
    // N rows from `row` on, side by side
    auto rows = [&](auto count, int64_t row) {
        constexpr int N = decltype(count)::value;
        float mu1[N], rs1[N], mu2[N], rs2[N];
        int from[N][5];  // places in the ring
#pragma unroll
        for (int k = 0; k < N; k++) {
            const int slot = (it + k) % stages;
#pragma unroll
            for (int i = 0; i < 5; i++) from[k][i] = slot_of(slot, i) + offset((row + k) * lds[i]);
        }
#pragma unroll
        for (int k = 0; k < N; k++) bar_wait(&full[(it + k) % stages], ((it + k) / stages) & 1, &s_abort, status);
#pragma unroll
        for (int k = 0; k < N; k++) {
            const float4 v = *reinterpret_cast<const float4 *>(s_stats[(it + k) % stages]);
            mu1[k] = v.x, rs1[k] = v.y, mu2[k] = v.z, rs2[k] = v.w;
        }
        if (VE == 1 && row + N + A > g.rows) {  // the tensors' last values
#pragma unroll
            for (int k = 0; k < N; k++)
#pragma unroll
                for (int i = 0; i < 5; i++) {
                    if (!src[i]) continue;
                    const int c = whole(row + k, i) - offset((row + k) * lds[i]) + t;
                    if (t < A && c < d) ring[from[k][i] + c] = src[i][(row + k) * lds[i] + c];
                }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // of their places, before other copies into them
            __syncthreads();
        }
        // The thread's values from i on, G together.  Single columns beyond the row are the row's last, with weights of zero; where a
        // thread has several of them together, it has none beyond the row.
        // Four together hold less in registers than eight: those spill, 848 us for 527 at 32768 x 4096 bfloat16.
        constexpr int G = VE > 1 ? 4 : 2, U = VE > 1 ? 4 : 1;
        auto inside = [&](int i) { return column(i) < d; };
        auto any = [&](int i) { return VE == 1 || inside(i); };
        auto at = [&](int i) { return VE == 1 ? min(column(i), d - 1) : column(i); };
        auto read = [&](int k, int tensor, int i, float *f) {
#pragma unroll
            for (int e = 0; e < G; e += U) {
                Vec<T, U> u;
                u.load(ring + from[k][tensor] + at(i + e));
                u.get(f + e);
            }
        };
        auto weight = [&](int k, int i, float *f, float other) {
#pragma unroll
            for (int e = 0; e < G; e++) f[e] = other;
            if (ws[k])
#pragma unroll
                for (int e = 0; e < G; e += U) load_ws<T, U>(ws[k], g.wf32, at(i + e), f + e);
        };
        auto mask = [&](int i, float *f) {
            if (VE == 1)
#pragma unroll
                for (int e = 0; e < G; e++)
                    if (!inside(i + e)) f[e] = 0.f;
        };
        auto store = [&](void *to, int64_t row, int i, const float *f) {
#pragma unroll
            for (int e = 0; e < G; e += U)
                if (inside(i + e)) {
                    Vec<T, U> out;
                    out.set(f + e);
                    out.store((T *)to + row + column(i + e));
                }
        };
        float h[N][E], a[N][E], w[E];
#pragma unroll
        for (int i = 0; i < E; i += G) {
#pragma unroll
            for (int e = 0; e < G; e++) {
                w[i + e] = 0.f;
#pragma unroll
                for (int k = 0; k < N; k++) h[k][i + e] = a[k][i + e] = 0.f;
            }
            if (!any(i)) continue;
#pragma unroll
            for (int k = 0; k < N; k++) read(k, 1, i, h[k] + i), read(k, 0, i, a[k] + i);
            weight(3, i, w + i, 1.f);
            mask(i, w + i);
        }
        float2 s[N];
#pragma unroll
        for (int k = 0; k < N; k++) {
            const float2 r2 = make_float2(rs2[k], rs2[k]), nm2 = make_float2(-mu2[k], -mu2[k]);
            float2 sx = make_float2(0.f, 0.f), sy = sx;
#pragma unroll
            for (int j = 0; j < NP; j++) {
                const float2 v = pair(a[k], j);
                // values beyond the row: a = 0, and their h counts for nothing
                const float2 hj = mul2(add2(pair(h[k], j), nm2), r2);
                put(h[k], j, hj);
                aw[j] = fma2(v, hj, aw[j]);
                ab[j] = add2(v, ab[j]);
                const float2 x = mul2(v, pair(w, j));
                put(a[k], j, x);
                sx = add2(x, sx);
                sy = fma2(x, hj, sy);
            }
            s[k] = make_float2(sx.x + sx.y, sy.x + sy.y);
        }
        row_sums<TPR, N>(s, red);
#pragma unroll
        for (int k = 0; k < N; k++) {
            const float m1 = g.rms ? 0.f : -rs2[k] * s[k].x * inv, m2 = -rs2[k] * s[k].y * inv;
            const float2 r2 = make_float2(rs2[k], rs2[k]);
#pragma unroll
            for (int j = 0; j < NP; j++)  // dx but for dy
                put(a[k], j, fma2(pair(h[k], j), make_float2(m2, m2), fma2(pair(a[k], j), r2, make_float2(m1, m1))));
        }
        if (p.dy)
#pragma unroll
            for (int i = 0; i < E; i += G)
                if (any(i))
#pragma unroll
                    for (int k = 0; k < N; k++) {
                        float f[G];
                        read(k, 3, i, f);
                        plus<G>(a[k] + i, f);
                    }
        // the branch's gradients; where w1 is 0 beyond the row, the gradient of h1 is
#pragma unroll
        for (int i = 0; i < E; i += G) {
            if (!any(i)) {
#pragma unroll
                for (int k = 0; k < N; k++)
#pragma unroll
                    for (int e = 0; e < G; e++) a[k][i + e] = h[k][i + e] = 0.f;
                continue;
            }
            float w1[G], b1[G], cc[G], act[N * G], slope[N * G], z[N * G];
            weight(0, i, w1, 1.f), weight(1, i, b1, 0.f), weight(2, i, cc, 1.f);
            mask(i, w1);
#pragma unroll
            for (int e = 0; e < N * G; e++) act[e] = 1.f, slope[e] = 0.f;
            if (p.z) {
#pragma unroll
                for (int k = 0; k < N; k++) read(k, 4, i, z + k * G);
                gates_all<true>(z, g.act, act, slope);
            }
#pragma unroll
            for (int k = 0; k < N; k++) {
                store(p.dx, (row + k) * p.lddx, i, a[k] + i);
                float o[G];
                read(k, 2, i, o);
                float *const sl = slope + k * G;
#pragma unroll
                for (int j = 0; j < G / 2; j++) {
                    // the mean first: times rs1 it may be large beside h1
                    const float2 v = pair(a[k] + i, j), hj = mul2(add2(pair(o, j), both(-mu1[k])), both(rs1[k]));
                    const float2 u = mul2(v, pair(act + k * G, j)), wj = pair(w1, j), cj = pair(cc, j);
                    if (p.z) put(sl, j, mul2(mul2(pair(sl, j), mul2(v, cj)), fma2(hj, wj, pair(b1, j))));
                    float2 &q = aq[i / 2 + j], &r = ar[i / 2 + j];
                    q = fma2(u, hj, q);
                    r = add2(u, r);
                    put(a[k] + i, j, mul2(u, mul2(cj, wj))), put(h[k] + i, j, hj);
                }
                if (p.dz) store(p.dz, (row + k) * p.lddz, i, sl);
            }
        }
#pragma unroll
        for (int k = 0; k < N; k++) {
            float2 sx = make_float2(0.f, 0.f), sy = sx;
#pragma unroll
            for (int j = 0; j < NP; j++) sx = add2(pair(a[k], j), sx), sy = fma2(pair(a[k], j), pair(h[k], j), sy);
            s[k] = make_float2(sx.x + sx.y, sy.x + sy.y);
        }
        row_sums<TPR, N>(s, red + N * (TPR / 32));
        if (TPR == 32) __syncwarp();
        if (t == 0)
#pragma unroll
            for (int k = 0; k < N; k++)
                if (row + k + stages < row1) issue(row + k + stages, (it + k) % stages);
#pragma unroll
        for (int k = 0; k < N; k++) {
            const float k1 = g.after && !g.rms ? -rs1[k] * s[k].x * inv : 0.f, k2 = g.after ? -rs1[k] * s[k].y * inv : 0.f;
#pragma unroll
            for (int j = 0; j < NP; j++)
                put(a[k], j, fma2(pair(h[k], j), make_float2(k2, k2), fma2(pair(a[k], j), make_float2(rs1[k], rs1[k]), make_float2(k1, k1))));
        }
#pragma unroll
        for (int k = 0; k < N; k++)
#pragma unroll
            for (int i = 0; i < E; i += G) store(p.dout, (row + k) * p.lddo, i, a[k] + i);
        it += N;
    };
    int64_t row = row0;
    if (step == 2)
        for (; row + 1 < row1; row += 2) rows(Count<R>(), row);
    for (; row < row1; row++) rows(Count<1>(), row);
    if (t == 0 && s_abort) bar_drain(full, stages, it);
    if (!parts) return;
    float *q = parts + (int64_t)blockIdx.x * 4 * d;
#pragma unroll
    for (int i = 0; i < E; i++) {
        const int c = column(i);
        if (c < d) {
            q[c] = i & 1 ? aq[i / 2].y : aq[i / 2].x;
            q[d + c] = i & 1 ? ar[i / 2].y : ar[i / 2].x;
            q[2 * d + c] = i & 1 ? aw[i / 2].y : aw[i / 2].x;
            q[3 * d + c] = i & 1 ? ab[i / 2].y : ab[i / 2].x;
        }
    }
}

// Rows for which no ring has room, and tensors that do not start on 16 bytes: one block a row in
// passes over it (8192 x 8192 float32: 1787 us, 1.2 TB/s; bfloat16 with float32 weights, for which the ring has no room there, 1777, and with
// bfloat16 weights, from the ring, 290), and the columns' sums with a thread a column over a share of the rows, from the rows' means
// of the first reduction.
template <typename T>
struct ResGrad {
    const ResBack &p;
    const ResGeom &g;
    int64_t row;
    float mu1, rs1, mu2, rs2, m1, m2;  // m1, m2: the means, times -rs2
    __device__ __forceinline__ ResGrad(const ResBack &p_, const ResGeom &g_, int64_t r) : p(p_), g(g_), row(r), m1(0.f), m2(0.f) {
        const float *s = p.stats + 4 * r;
        mu1 = s[0], rs1 = s[1], mu2 = s[2], rs2 = s[3];
    }
    __device__ __forceinline__ float dh(int64_t c) const { return to_f32(((const T *)p.dh)[row * p.lddh + c]); }
    __device__ __forceinline__ float h2(int64_t c) const { return (to_f32(((const T *)p.y)[row * p.ldy + c]) - mu2) * rs2; }
    __device__ __forceinline__ float a2(int64_t c) const { return dh(c) * (g.w2 ? load_w<T>(g.w2, g.wf32, c) : 1.f); }
    __device__ __forceinline__ float dx(int64_t c) const {
        const float v = fmaf(h2(c), m2, fmaf(a2(c), rs2, m1));
        return p.dy ? v + to_f32(((const T *)p.dy)[row * p.lddy + c]) : v;
    }
    __device__ __forceinline__ float h1(int64_t c) const { return (to_f32(((const T *)p.o)[row * p.ldo + c]) - mu1) * rs1; }
    __device__ __forceinline__ float w1(int64_t c) const { return g.w1 ? load_w<T>(g.w1, g.wf32, c) : 1.f; }
    __device__ __forceinline__ float scale(int64_t c) const { return g.c ? load_w<T>(g.c, g.wf32, c) : 1.f; }
    __device__ __forceinline__ float2 gate(int64_t c) const {
        float z[1] = {p.z ? to_f32(((const T *)p.z)[row * p.ldz + c]) : 0.f}, a[1] = {1.f}, s[1] = {0.f};
        if (p.z) gates_all<true>(z, g.act, a, s);
        return make_float2(a[0], s[0]);
    }
};
template <typename T>
__global__ void __launch_bounds__(kLong)
k_resnorm_bwd_long(const ResBack p, const ResGeom g, float2 *__restrict__ means) {
    __shared__ float2 red[2 * (kLong / 32)];
    ResGrad<T> r(p, g, blockIdx.x);
    float2 s = make_float2(0.f, 0.f);
    for (int c = threadIdx.x; c < g.d; c += kLong) {
        const float a = r.a2(c);
        s.x += a;
        s.y = fmaf(a, r.h2(c), s.y);
    }
    s = row_sum<kLong>(s, red, 0);
    const float inv = 1.f / (float)g.d;
    r.m1 = g.rms ? 0.f : -r.rs2 * s.x * inv, r.m2 = -r.rs2 * s.y * inv;
    if (threadIdx.x == 0 && means) means[r.row] = make_float2(r.m1, r.m2);
    float k1 = 0.f, k2 = 0.f;
    if (g.after) {
        s = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < g.d; c += kLong) {
            const float a = r.dx(c) * r.gate(c).x * r.scale(c) * r.w1(c);
            s.x += a;
            s.y = fmaf(a, r.h1(c), s.y);
        }
        s = row_sum<kLong>(s, red, 1);
        k1 = g.rms ? 0.f : -r.rs1 * s.x * inv, k2 = -r.rs1 * s.y * inv;
    }
    for (int c = threadIdx.x; c < g.d; c += kLong) {
        const float dx = r.dx(c), h1 = r.h1(c), w1 = r.w1(c), b = dx * r.scale(c);
        const float2 a = r.gate(c);
        ((T *)p.dx)[r.row * p.lddx + c] = from_f32<T>(dx);
        if (p.dz) {
            const float t = fmaf(h1, w1, g.b1 ? load_w<T>(g.b1, g.wf32, c) : 0.f);
            ((T *)p.dz)[r.row * p.lddz + c] = from_f32<T>(b * t * a.y);
        }
        ((T *)p.dout)[r.row * p.lddo + c] = from_f32<T>(fmaf(h1, k2, fmaf(b * a.x * w1, r.rs1, k1)));
    }
}
template <typename T>
__global__ void __launch_bounds__(256)
k_resnorm_bwd_cols(const ResBack p, const ResGeom g, const float2 *__restrict__ means, float *__restrict__ parts) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= g.d) return;
    float q = 0.f, r = 0.f, w = 0.f, b = 0.f;
    for (int64_t row = blockIdx.y; row < g.rows; row += gridDim.y) {
        ResGrad<T> v(p, g, row);
        v.m1 = means[row].x, v.m2 = means[row].y;
        const float u = v.dx(c) * v.gate(c).x, dh = v.dh(c);
        q = fmaf(u, v.h1(c), q);
        r += u;
        w = fmaf(dh, v.h2(c), w);
        b += dh;
    }
    float *to = parts + (int64_t)blockIdx.y * 4 * g.d + c;
    to[0] = q, to[g.d] = r, to[2 * (int64_t)g.d] = w, to[3 * (int64_t)g.d] = b;
}

// The weights' gradients from the partial sums, which are added in a fixed order: 32 columns a
// block, 32 threads a column.
struct ResSums {
    void *dw1, *db1, *dc, *dw2, *db2;  // NULL: not formed
};
template <typename T>
__global__ void __launch_bounds__(1024)
k_resnorm_bwd_sum(const float *__restrict__ parts, int64_t nparts, const ResGeom g, const ResSums to) {
    __shared__ float tile[4][32][33];
    after_previous();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t d = g.d, c = (int64_t)blockIdx.x * 32 + tx;
    float s[4] = {};
    if (c < d) {
#pragma unroll 4
        for (int64_t p = ty; p < nparts; p += 32)
#pragma unroll
            for (int k = 0; k < 4; k++) s[k] += parts[(p * 4 + k) * d + c];
    }
#pragma unroll
    for (int k = 0; k < 4; k++) tile[k][ty][tx] = s[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; k++) s[k] = warp_sum(tile[k][tx][ty]);
    const int64_t o = (int64_t)blockIdx.x * 32 + ty;
    if (tx != 0 || o >= d) return;
    auto store = [&](void *p, float v) {
        if (!p) return;
        if (g.wf32)
            reinterpret_cast<float *>(p)[o] = v;
        else
            reinterpret_cast<T *>(p)[o] = from_f32<T>(v);
    };
    const float cc = g.c ? load_w<T>(g.c, g.wf32, o) : 1.f;
    store(to.dw1, cc * s[0]);
    store(to.db1, cc * s[1]);
    if (to.dc) {
        const float v = (g.w1 ? load_w<T>(g.w1, g.wf32, o) : 1.f) * s[0];
        store(to.dc, g.b1 ? fmaf(load_w<T>(g.b1, g.wf32, o), s[1], v) : v);
    }
    store(to.dw2, s[2]);
    store(to.db2, s[3]);
}

// ---------------------------------------------------------------- host

constexpr int64_t kMaxRow = 16384;  // of the forward pass in registers
constexpr int64_t kParts = 64;      // shares of the rows, where a thread takes a column

ResGeom geom_of(const zsolve_resnorm_args *a) {
    return ResGeom{a->w1, a->b1, a->c, a->w2, a->b2, a->wtype == ZSOLVE_F32, a->rows, (int)a->d, (float)a->eps, a->act, a->after != 0,
                   a->kind == ZSOLVE_NORM_RMS};
}
bool weights_aligned(const zsolve_resnorm_args *a) {
    return aligned16(a->w1) && aligned16(a->b1) && aligned16(a->c) && aligned16(a->w2) && aligned16(a->b2);
}

template <typename T>
int fwd(zsolve_seq *s, const zsolve_resnorm_args *a, const void *x, int64_t ldx, void *y, int64_t ldy, void *h, int64_t ldh, float *stats) {
    constexpr int V = 16 / (int)sizeof(T);
    const ResGeom g = geom_of(a);
    const int64_t d = a->d;
    const bool vec = d % V == 0 && ldx % V == 0 && a->ldo % V == 0 && (!a->z || a->ldz % V == 0) && ldy % V == 0 && ldh % V == 0 &&
                     aligned16(x) && aligned16(a->o) && aligned16(a->z) && aligned16(y) && aligned16(h) && weights_aligned(a);
    s->launches++;
#define RES_ARGS (const T *)x, ldx, (const T *)a->o, a->ldo, (const T *)a->z, a->ldz, g, (T *)y, ldy, (T *)h, ldh, stats
#define RES_GO(VE, TPR, E) \
    k_resnorm<T, VE, TPR, (E) / VE><<<(unsigned)((TPR) == 32 ? (a->rows + 3) / 4 : a->rows), (TPR) < 128 ? 128 : (TPR), 0, s->st>>>(RES_ARGS)
#define RES_SIZES(VE, E)                        \
    if (d <= 256) RES_GO(VE, 32, 8);            \
    else if (d <= 128 * E) RES_GO(VE, 128, E);  \
    else if (d <= 256 * E) RES_GO(VE, 256, E);  \
    else if (d <= 512 * E) RES_GO(VE, 512, E);  \
    else if (d <= 1024 * E) RES_GO(VE, 1024, E); \
    else RES_GO(VE, 1024, 16)
    if (d > kMaxRow) {
        k_resnorm_long<T><<<(unsigned)a->rows, kLong, 0, s->st>>>(RES_ARGS);
    } else if (vec) {
        RES_SIZES(V, 16);
    } else {
        RES_SIZES(1, 8);
    }
#undef RES_SIZES
#undef RES_GO
#undef RES_ARGS
    SEQ_CU(cudaGetLastError());
    return ZSOLVE_OK;
}

// The backward kernel's blocks and stages, or none where no ring has room.
struct RingPlan {
    int tpr = 0, stages = 0;
    int64_t blocks = 0;
    size_t smem = 0;
};
constexpr size_t kRingMost = 225 * 1024;  // beside the static shared memory
template <typename T>
RingPlan ring_plan(const zsolve_resnorm_args *a, const ResBack &p, int num_sms) {
    RingPlan r;
    const int64_t d = a->d;
    if (d > 8192 || !aligned16(p.stats) || !aligned16(p.dh) || !aligned16(p.dy) || !aligned16(p.y) || !aligned16(p.o) || !aligned16(p.z)) return r;
    const int e = d > 4096 ? 16 : 8;
    r.tpr = 32;
    while (r.tpr * e < d) r.tpr *= 2;
    const size_t row = (size_t)(3 + (p.dy != nullptr) + (p.z != nullptr)) * ring_row<T>((int)d) * sizeof(T);
    const int n = (a->w1 != nullptr) + (a->b1 != nullptr) + (a->c != nullptr) + (a->w2 != nullptr);
    const size_t weights = (size_t)n * ((d * (a->wtype == ZSOLVE_F32 ? 4 : sizeof(T)) + 15) / 16 * 16);
    if (2 * row + weights > kRingMost) return RingPlan{};
    // as many blocks as the registers allow, with four rows each or as many as there is room for
    const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>(ring_blocks(r.tpr), (int64_t)(kRingMost / (2 * row + weights + 1536))));
    r.stages = (int)std::max<int64_t>(2, std::min<int64_t>(4, ((int64_t)(kRingMost / per_sm) - (int64_t)weights - 1536) / (int64_t)row));
    r.smem = r.stages * row + weights;
    r.blocks = std::min(a->rows, per_sm * num_sms);
    return r;
}

template <typename T, int VE, int TPR, int E>
cudaError_t launch_ring(const ResBack &p, const ResGeom &g, const RingPlan &r, float *parts, unsigned *status, cudaStream_t st) {
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_resnorm_bwd<T, VE, TPR, E>, (int)kRingMost);
    if (attr != cudaSuccess) return attr;
    k_resnorm_bwd<T, VE, TPR, E><<<(unsigned)r.blocks, TPR, r.smem, st>>>(p, g, r.stages, parts, status);
    return cudaGetLastError();
}

template <typename T>
int bwd(zsolve_seq *s, const zsolve_resnorm_args *a, const ResBack &p, const ResSums &to) {
    constexpr int V = 16 / (int)sizeof(T);
    const ResGeom g = geom_of(a);
    const int64_t d = a->d;
    const bool sums = to.dw1 || to.db1 || to.dc || to.dw2 || to.db2;
    const RingPlan r = a->rows > 0 ? ring_plan<T>(a, p, s->num_sms) : RingPlan{};
    const int64_t nparts = !sums ? 0 : r.blocks ? r.blocks : std::min(a->rows, kParts);
    float *parts = nullptr;
    float2 *means = nullptr;
    if (nparts) {
        auto carve = [&](void *base) {
            Carve c(base);
            parts = c.take<float>((size_t)nparts * 4 * d);
            means = r.blocks ? nullptr : c.take<float2>((size_t)a->rows);
            return c.at;
        };
        int st = ZSOLVE_OK;
        void *ws = seq_workspace(s, carve(nullptr), &st);
        if (!ws) return st;
        carve(ws);
    }
    if (a->rows > 0) {
        s->launches++;
        if (r.blocks) {
            const bool vec = d % V == 0 && p.lddh % V == 0 && (!p.dy || p.lddy % V == 0) && p.ldy % V == 0 && p.ldo % V == 0 &&
                             (!p.z || p.ldz % V == 0) && p.lddx % V == 0 && p.lddo % V == 0 && (!p.dz || p.lddz % V == 0) &&
                             aligned16(p.dx) && aligned16(p.dout) && aligned16(p.dz);
#define RES_SINGLE(TPR, E) (launch_ring<T, 1, TPR, E>(p, g, r, parts, s->d_status, s->st))
#define RES_RING(TPR, E) (vec ? launch_ring<T, V, TPR, E>(p, g, r, parts, s->d_status, s->st) : launch_ring<T, 1, TPR, E>(p, g, r, parts, s->d_status, s->st))
            // Single columns: between four and six for each of 512 threads, six are enough, and the registers of two more are free (6614 rows of
            // 2157 float32 131 us, 156 with eight; of 2901 149 and 187; of 2501 bfloat16 141 and 162).  The like brackets of
            // fewer threads, 513 to 768 and 1025 to 1536 columns, have no such kernel.
            SEQ_CU(d > 4096       ? RES_RING(512, 16)
                   : !vec && d > 256 * 8 && d <= 512 * 6 ? RES_SINGLE(512, 6)
                   : r.tpr == 32  ? RES_RING(32, 8)
                   : r.tpr == 64  ? RES_RING(64, 8)
                   : r.tpr == 128 ? RES_RING(128, 8)
                   : r.tpr == 256 ? RES_RING(256, 8)
                                  : RES_RING(512, 8));
#undef RES_RING
#undef RES_SINGLE
        } else {
            k_resnorm_bwd_long<T><<<(unsigned)a->rows, kLong, 0, s->st>>>(p, g, means);
            SEQ_CU(cudaGetLastError());
            if (sums) {
                s->launches++;
                k_resnorm_bwd_cols<T><<<dim3((unsigned)((d + 255) / 256), (unsigned)nparts), 256, 0, s->st>>>(p, g, means, parts);
                SEQ_CU(cudaGetLastError());
            }
        }
    }
    if (!sums) return ZSOLVE_OK;
    s->launches++;
    SEQ_CU(launch(nparts > 0, k_resnorm_bwd_sum<T>, (unsigned)((d + 31) / 32), 1024, 0, s->st, parts, nparts, g, to));
    return ZSOLVE_OK;
}

}  // namespace

int zs_resnorm(zsolve_seq *s, const zsolve_resnorm_args *a, const void *x, int64_t ldx, void *y, int64_t ldy, void *h, int64_t ldh,
               float *stats) {
    if (a->type == ZSOLVE_F32) return fwd<float>(s, a, x, ldx, y, ldy, h, ldh, stats);
    return a->type == ZSOLVE_BF16 ? fwd<bf16>(s, a, x, ldx, y, ldy, h, ldh, stats) : fwd<f16>(s, a, x, ldx, y, ldy, h, ldh, stats);
}

int zs_resnorm_bwd(zsolve_seq *s, const zsolve_resnorm_args *a, const void *dh, int64_t lddh, const void *dy, int64_t lddy, const void *y,
                   int64_t ldy, const float *stats, void *dx, int64_t lddx, void *dout, int64_t lddo, void *dz, int64_t lddz, void *dw1,
                   void *db1, void *dc, void *dw2, void *db2) {
    const ResBack p{dh, dy, y, a->o, a->z, lddh, lddy, ldy, a->ldo, a->ldz, stats, dx, dout, a->z ? dz : nullptr, lddx, lddo, lddz};
    const ResSums to{dw1, db1, dc, dw2, db2};
    if (a->type == ZSOLVE_F32) return bwd<float>(s, a, p, to);
    return a->type == ZSOLVE_BF16 ? bwd<bf16>(s, a, p, to) : bwd<f16>(s, a, p, to);
}
