// Linear attention with a decay for each head: the spans' sums, the recurrence over the spans, and the
// gradients of the decays (formulas and geometry in decay.cuh).
#include <algorithm>

#include "decay.cuh"

namespace {

using namespace zs;

// ---------------------------------------------------------------- sums

// A block of warps holds DX x NB values of one span's sum in registers, 32 x 64 a warp, and goes through the
// span's tokens 64 at a time; their tiles come in two stages.  The weights enter x's side, whose
// product with y keeps float32 accuracy (two tf32 parts, added to nearest).  8 ragged sequences of 2467 tokens x 8 heads of
// 96 x 80 in float32: 27 us, a span's chain of products of mma.sync (tensor pipe 35 to 44 %).
template <typename T, int DX, int NB>
struct SumSmem {
    static constexpr int LDX = tile_ld<T>(DX), LDY = tile_ld<T>(NB);
    T x[2][kChunk * LDX];
    T y[2][kChunk * LDY];
    float2 b[kSpanMost];
    float w[kSpanMost];
};
template <int DX, int NB>
constexpr int sum_threads() { return DX * NB / 64; }

template <typename T, int DX, int NB>
__global__ void __launch_bounds__(sum_threads<DX, NB>(), DX * NB / 64 >= 256 ? 2 : 4)
k_decay_sums(const DecayGeom geo, const DecayRows x, const DecayRows y, int query, int gates, float *__restrict__ out) {
    using Smem = SumSmem<T, DX, NB>;
    constexpr int LDX = Smem::LDX, LDY = Smem::LDY, NT = sum_threads<DX, NB>();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    after_previous();
    may_start_next();
    const int span = blockIdx.x, hv = blockIdx.y, c0 = blockIdx.z * NB;
    const int2 sp = geo.d.chunk[span];
    if (sp.y == 0) return;
    const int group = geo.d.hv / geo.d.hk, hk = hv / group;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const T *px = (const T *)x.p + (int64_t)sp.x * x.ld + (int64_t)(x.key ? hk : hv) * x.dist;
    const T *py = (const T *)y.p + (int64_t)sp.x * y.ld + (int64_t)(y.key ? hk : hv) * y.dist + c0;
    const int ycols = min(NB, y.dist - c0), chunks = (sp.y + kChunk - 1) / kChunk;
    auto fetch = [&](int i) {
        const int n = min(kChunk, sp.y - i * kChunk);
        load_tile<T, DX, NT>(sm.x[i & 1], px + (int64_t)i * kChunk * x.ld, x.ld, n, x.dist);
        load_tile<T, NB, NT>(sm.y[i & 1], py + (int64_t)i * kChunk * y.ld, y.ld, n, ycols);
        cp_commit();
    };
    fetch(0);
    decay_loads(geo, sp, hv, sm.b, tid, NT);
    __syncthreads();
    if (warp == 0) decay_sums(sp, sm.b);
    __syncthreads();
    const float2 last = sm.b[sp.y - 1];
    for (int i = tid; i < chunks * kChunk; i += NT)
        sm.w[i] = i >= sp.y ? 0.f : query ? geo.d.scale * decay_exp(sm.b[i], make_float2(0.f, 0.f)) : decay_exp(last, sm.b[i]);
    if (gates && blockIdx.z == 0) {
        for (int i = tid; i < sp.y; i += NT) geo.gates[((int64_t)span * geo.d.hv + hv) * geo.span + i] = sm.b[i];
        if (tid == 0) geo.ends[(int64_t)span * geo.d.hv + hv] = decay_exp(last, make_float2(0.f, 0.f));
    }
    constexpr int WN = NB / 64;  // warps side by side
    const int d0 = warp / WN * 32, v0 = warp % WN * 64;
    float acc[2][8][4] = {};
    for (int i = 0; i < chunks; i++) {
        if (i + 1 < chunks) {
            fetch(i + 1);
            cp_wait<1>();
        } else {
            cp_wait<0>();
        }
        __syncthreads();
        const T *xs = sm.x[i & 1], *ys = sm.y[i & 1];
        const float *w = sm.w + i * kChunk;
#pragma unroll 2
        for (int k = 0; k < 8; k++) {
            const float2 wk = *reinterpret_cast<const float2 *>(w + k * 8 + 2 * t);
            float2 f[4];
            frag4<T, LDX, true>(xs, k * 8, d0, f);
            SplitA a[2];
#pragma unroll
            for (int m = 0; m < 2; m++)
                a[m].set(f[2 * m].x * wk.x, f[2 * m].y * wk.y, f[2 * m + 1].x * wk.x, f[2 * m + 1].y * wk.y);
#pragma unroll
            for (int n = 0; n < 2; n++) {
                frag4<T, LDY, true>(ys, k * 8, v0 + 32 * n, f);
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int m = 0; m < 2; m++) mma_add<false, sizeof(T) == 2>(acc[m][4 * n + j], a[m], f[j]);
            }
        }
        __syncthreads();  // the stage is free
    }
    float *po = out + ((int64_t)span * geo.d.hv + hv) * x.cols * y.cols;
#pragma unroll
    for (int m = 0; m < 2; m++)
#pragma unroll
        for (int j = 0; j < 8; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int r = d0 + 16 * m + g + (e >> 1) * 8, c = c0 + v0 + 8 * j + 2 * t + (e & 1);
                if (r < x.cols && c < y.cols) po[(int64_t)r * y.cols + c] = acc[m][j][e];
            }
}

// ---------------------------------------------------------------- the recurrence over the spans

constexpr int kScanThreads = 256;
constexpr int kAhead = 5;  // spans whose sums are on their way

__device__ __forceinline__ float span_decay(const DecayGeom &geo, int span, int hv) { return geo.ends[(int64_t)span * geo.d.hv + hv]; }

// A state's value as the next kernels take it: float32 in the place of the sum, or PARTS bfloat16 values that add up
// to it (16 or 24 bits), each part a matrix of its own.
template <int VE, int PARTS>
struct StatePut {
    __device__ __forceinline__ static void put(float *u, bf16 *planes, int64_t slot, int size, int at, const float (&s)[VE]) {
        if constexpr (PARTS == 0) {
            Vec<float, VE> v;
            v.set(s);
            v.store(u + slot * size + at);
        } else {
            float f[VE];
#pragma unroll
            for (int e = 0; e < VE; e++) f[e] = s[e];
            bf16 *p = planes + slot * PARTS * size + at;
#pragma unroll
            for (int i = 0; i < PARTS; i++, p += size) {
                Vec<bf16, VE> v;
                v.set(f);
                v.store(p);
                float g[VE];
                v.get(g);
#pragma unroll
                for (int e = 0; e < VE; e++) f[e] -= g[e];
            }
        }
    }
    __device__ __forceinline__ static void get(const float *u, const bf16 *planes, int64_t slot, int size, int at, float (&s)[VE]) {
        if constexpr (PARTS == 0) {
            Vec<float, VE> v;
            v.load(u + slot * size + at);
            v.get(s);
        } else {
            const bf16 *p = planes + slot * PARTS * size + at;
#pragma unroll
            for (int e = 0; e < VE; e++) s[e] = 0.f;
#pragma unroll
            for (int i = 0; i < PARTS; i++) {
                Vec<bf16, VE> v;
                v.load(p + (int64_t)(PARTS - 1 - i) * size);
                float g[VE];
                v.get(g);
#pragma unroll
                for (int e = 0; e < VE; e++) s[e] += g[e];
            }
        }
    }
};

// A thread VE neighbouring values of a state, the sums of the next spans on their way.  64 spans x 32 heads of 128 x 128: 48 us for 268 MB
// with two bfloat16 parts, 5.6 TB/s, bound by HBM.
template <int VE, int PARTS>
__global__ void __launch_bounds__(kScanThreads, 4)
k_decay_scan(const DecayGeom geo, float *u, bf16 *planes, const float *s0, float *sn) {
    after_previous();
    may_start_next();
    const int si = blockIdx.x / geo.d.hv, hv = blockIdx.x - si * geo.d.hv, size = geo.d.dk * geo.d.dv;
    const int at = ((int)blockIdx.y * kScanThreads + (int)threadIdx.x) * VE;
    if (at >= size) return;
    const int first = geo.d.first[si], n = geo.d.first[si + 1] - first;
    float s[VE] = {};
    Vec<float, VE> v;
    if (s0) v.load(s0 + (int64_t)blockIdx.x * size + at), v.get(s);
    Vec<float, VE> w[kAhead];
    float a[kAhead];
    auto fetch = [&](int k, int i) {
        if (i < n) w[k].load(u + ((int64_t)(first + i) * geo.d.hv + hv) * size + at), a[k] = span_decay(geo, first + i, hv);
    };
#pragma unroll
    for (int k = 0; k < kAhead; k++) fetch(k, k);
    for (int i = 0; i < n; i += kAhead) {
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            if (i + k >= n) break;
            float f[VE];
            w[k].get(f);
            const float ak = a[k];
            fetch(k, i + k + kAhead);
            StatePut<VE, PARTS>::put(u, planes, (int64_t)(first + i + k) * geo.d.hv + hv, size, at, s);
#pragma unroll
            for (int e = 0; e < VE; e++) s[e] = fmaf(ak, s[e], f[e]);
        }
    }
    if (sn) v.set(s), v.store(sn + (int64_t)blockIdx.x * size + at);
}

// PARTS: of the states and of their gradients.
template <int VE, int PARTS>
__global__ void __launch_bounds__(kScanThreads, 3)
k_decay_rscan(const DecayGeom geo, float *w, bf16 *planes, const float *__restrict__ states, const bf16 *__restrict__ splanes, const float *ds,
              float *ds0, float *__restrict__ dots) {
    after_previous();
    may_start_next();
    const int si = blockIdx.x / geo.d.hv, hv = blockIdx.x - si * geo.d.hv, size = geo.d.dk * geo.d.dv;
    const int at = ((int)blockIdx.y * kScanThreads + (int)threadIdx.x) * VE;
    const bool in = at < size;
    const int first = geo.d.first[si], n = geo.d.first[si + 1] - first;
    float s[VE] = {};
    Vec<float, VE> v;
    if (ds && in) v.load(ds + (int64_t)blockIdx.x * size + at), v.get(s);
    const int warps = kScanThreads / 32, parts = gridDim.y * warps;
    Vec<float, VE> x[kAhead];
    float y[kAhead][VE], a[kAhead];
    auto fetch = [&](int k, int i) {
        if (i < 0) return;
        const int64_t slot = (int64_t)(first + i) * geo.d.hv + hv;
        if (in) x[k].load(w + slot * size + at), StatePut<VE, PARTS>::get(states, splanes, slot, size, at, y[k]);
        a[k] = span_decay(geo, first + i, hv);
    };
#pragma unroll
    for (int k = 0; k < kAhead; k++) fetch(k, n - 1 - k);
    for (int i = n - 1; i >= 0; i -= kAhead) {
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            if (i - k < 0) break;
            const int64_t slot = (int64_t)(first + i - k) * geo.d.hv + hv;
            float dot = 0.f, f[VE], q[VE];
            const float ak = a[k];
#pragma unroll
            for (int e = 0; e < VE; e++) q[e] = y[k][e];
            x[k].get(f);
            fetch(k, i - k - kAhead);
            if (in) {
                StatePut<VE, PARTS>::put(w, planes, slot, size, at, s);
#pragma unroll
                for (int e = 0; e < VE; e++) dot = fmaf(q[e], s[e], dot), s[e] = fmaf(ak, s[e], f[e]);
            }
            dot = warp_sum(dot) * ak;
            if ((threadIdx.x & 31) == 0) dots[slot * parts + blockIdx.y * warps + (threadIdx.x >> 5)] = dot;
        }
    }
    if (ds0 && in) v.set(s), v.store(ds0 + (int64_t)blockIdx.x * size + at);
}

// ---------------------------------------------------------------- gradients of the decays

struct DecayDots {
    const float *xq, *rq, *xk, *rk;  // tokens x hv: the state's share and the pairs, as queries and as keys
    const float *dots;
    int parts;
};

// A block a span and eight heads: a thread has a thirty-second of the span's tokens of a head.  Within the span the sums
// over the tokens after and before t; float32, in pieces of at most 16 tokens and 32 pieces.
constexpr int kDgHeads = 8, kDgPieces = 32, kDgTokens = kSpanMost / kDgPieces;
__global__ void __launch_bounds__(kDgHeads * kDgPieces)
k_decay_dg(const DecayGeom geo, const DecayDots in, float *__restrict__ parts, float *__restrict__ dg) {
    __shared__ float s_later[kDgPieces + 1][kDgHeads], s_before[kDgPieces + 1][kDgHeads], s_z[kDgHeads];
    after_previous();
    may_start_next();
    const int h = threadIdx.x % kDgHeads, piece = threadIdx.x / kDgHeads, hv = (int)blockIdx.y * kDgHeads + h, span = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool live = hv < geo.d.hv;
    const int2 sp = geo.d.chunk[span];
    if (sp.y == 0) {
        if (parts) {
            if (live && piece == 0) parts[(int64_t)span * geo.d.hv + hv] = 0.f;
        } else if (live) {
            const int used = geo.d.first[geo.d.nseq], workers = (geo.d.nchunks - used) * kDgPieces, worker = (span - used) * kDgPieces + piece;
            const int2 last = geo.d.seq[geo.d.nseq - 1];
            for (int64_t t = worker; t < geo.d.seq[0].x; t += workers) dg[t * geo.d.hv + hv] = 0.f;
            for (int64_t t = (int64_t)last.x + last.y + worker; t < geo.d.tokens; t += workers) dg[t * geo.d.hv + hv] = 0.f;
        }
        return;
    }
    // exp(b_L) <S, D>: a warp a head
    {
        const int head = (int)blockIdx.y * kDgHeads + warp;
        float z = 0.f;
        if (head < geo.d.hv)
            for (int i = lane; i < in.parts; i += 32) z += in.dots[((int64_t)span * geo.d.hv + head) * in.parts + i];
        z = warp_sum(z);
        if (lane == 0) s_z[warp] = z;
    }
    const int per = (sp.y + kDgPieces - 1) / kDgPieces, i0 = min(piece * per, sp.y), i1 = min(i0 + per, sp.y);
    float own[kDgTokens], key[kDgTokens], later = 0.f, before = 0.f;
#pragma unroll
    for (int k = 0; k < kDgTokens; k++) {
        own[k] = key[k] = 0.f;
        if (live && i0 + k < i1) {
            const int64_t at = (int64_t)(sp.x + i0 + k) * geo.d.hv + hv;
            own[k] = in.xq[at] + (in.rq[at] - in.rk[at]);
            key[k] = in.xk[at];
        }
    }
#pragma unroll
    for (int k = 0; k < kDgTokens; k++) later += own[kDgTokens - 1 - k], before += key[k];
    s_later[piece][h] = later, s_before[piece][h] = before;
    __syncthreads();
    float tail = 0.f, head = 0.f;  // of the pieces after and before this one
    for (int w = kDgPieces - 1; w > piece; w--) tail += s_later[w][h];
    for (int w = 0; w < piece; w++) head += s_before[w][h];
    const float z = s_z[h];
    float total = 0.f, v[kDgTokens];
#pragma unroll
    for (int k = kDgTokens - 1; k >= 0; k--) tail += own[k], v[k] = tail;
#pragma unroll
    for (int k = 0; k < kDgTokens; k++) {
        if (live && i0 + k < i1) {
            v[k] += head + z;
            total += v[k];
            if (!parts) dg[(int64_t)(sp.x + i0 + k) * geo.d.hv + hv] = v[k];
        }
        head += key[k];
    }
    if (!parts) return;
    __syncthreads();
    s_later[piece][h] = total;
    __syncthreads();
    if (piece || !live) return;
    for (int w = 1; w < kDgPieces; w++) total += s_later[w][h];
    parts[(int64_t)span * geo.d.hv + hv] = total;
}

// One decay a head: the spans' parts, a warp a head.
__global__ void __launch_bounds__(128)
k_decay_dg_heads(const float *__restrict__ parts, int spans, int hv, float *__restrict__ dg) {
    after_previous();
    const int lane = threadIdx.x & 31, h = (int)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (h >= hv) return;
    float s = 0.f;
    for (int i = lane; i < spans; i += 32) s += parts[(int64_t)i * hv + h];
    s = warp_sum(s);
    if (lane == 0) dg[h] = s;
}

// ---------------------------------------------------------------- host

template <typename T, int DX, int NB>
cudaError_t sums_as(const DecayGeom &g, const DecayRows &x, const DecayRows &y, bool query, bool gates, float *out, bool next, cudaStream_t st) {
    constexpr int smem = (int)sizeof(SumSmem<T, DX, NB>);
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_decay_sums<T, DX, NB>, smem);
    if (attr != cudaSuccess) return attr;
    return launch(next, k_decay_sums<T, DX, NB>, dim3(g.d.nchunks, g.d.hv, (y.cols + NB - 1) / NB), sum_threads<DX, NB>(), smem, st, g, x, y,
                  (int)query, (int)gates, out);
}
template <typename T>
cudaError_t sums(const DecayGeom &g, const DecayRows &x, const DecayRows &y, bool query, bool gates, float *out, bool next, cudaStream_t st) {
#define SUM_GO(DX) (y.cols <= 64 ? sums_as<T, DX, 64>(g, x, y, query, gates, out, next, st) : sums_as<T, DX, 128>(g, x, y, query, gates, out, next, st))
    return x.cols <= 32 ? SUM_GO(32) : x.cols <= 64 ? SUM_GO(64) : SUM_GO(128);
#undef SUM_GO
}

}  // namespace

cudaError_t zs_launch_decay_sums(int type, const DecayGeom &g, const DecayRows &x, const DecayRows &y, bool query, bool gates, float *out,
                                 bool next, cudaStream_t st, int64_t *launches) {
    ++*launches;
    if (type == ZSOLVE_F32) return sums<float>(g, x, y, query, gates, out, next, st);
    if (type == ZSOLVE_BF16) return sums<bf16>(g, x, y, query, gates, out, next, st);
    return sums<f16>(g, x, y, query, gates, out, next, st);
}

cudaError_t zs_launch_decay_scan(const DecayGeom &g, float *u, void *planes, int parts, const float *s0, float *sn, bool next, cudaStream_t st,
                                 int64_t *launches) {
    ++*launches;
    const int size = g.d.dk * g.d.dv;
    const unsigned heads = (unsigned)(g.d.nseq * g.d.hv);
    bf16 *const pl = (bf16 *)planes;
#define SCAN_GO(VE, P) \
    launch(next, k_decay_scan<VE, P>, dim3(heads, (size + VE * kScanThreads - 1) / (VE * kScanThreads)), kScanThreads, 0, st, g, u, pl, s0, sn)
    if (zs_decay_vec(g, s0, sn)) return parts == 0 ? SCAN_GO(4, 0) : parts == 2 ? SCAN_GO(4, 2) : SCAN_GO(4, 3);
    return parts == 0 ? SCAN_GO(1, 0) : parts == 2 ? SCAN_GO(1, 2) : SCAN_GO(1, 3);
#undef SCAN_GO
}

cudaError_t zs_launch_decay_rscan(const DecayGeom &g, float *w, void *planes, int parts, const float *states, const void *splanes,
                                  const float *ds, float *ds0, float *dots, bool next, cudaStream_t st, int64_t *launches) {
    ++*launches;
    const int size = g.d.dk * g.d.dv;
    const unsigned heads = (unsigned)(g.d.nseq * g.d.hv);
    bf16 *const pl = (bf16 *)planes;
    const bf16 *const spl = (const bf16 *)splanes;
#define SCAN_GO(VE, P)                                                                                                              \
    launch(next, k_decay_rscan<VE, P>, dim3(heads, (size + VE * kScanThreads - 1) / (VE * kScanThreads)), kScanThreads, 0, st, g, w, pl, \
           states, spl, ds, ds0, dots)
    if (zs_decay_vec(g, ds, ds0)) return parts == 0 ? SCAN_GO(4, 0) : SCAN_GO(4, 3);
    return parts == 0 ? SCAN_GO(1, 0) : SCAN_GO(1, 3);
#undef SCAN_GO
}

cudaError_t zs_launch_decay_dg(const DecayGeom &g, const float *const from_q[2], const float *const from_k[2], const float *dots,
                               int ndots, float *parts, float *dg, cudaStream_t st, int64_t *launches) {
    const DecayDots in{from_q[0], from_q[1], from_k[0], from_k[1], dots, ndots};
    ++*launches;
    const cudaError_t e = launch(true, k_decay_dg, dim3(g.d.nchunks, (g.d.hv + kDgHeads - 1) / kDgHeads), kDgHeads * kDgPieces, 0, st, g, in, g.ldg ? (float *)nullptr : parts, dg);
    if (e != cudaSuccess || g.ldg) return e;
    ++*launches;
    return launch(true, k_decay_dg_heads, (unsigned)((g.d.hv + 3) / 4), 128, 0, st, parts, g.d.nchunks, g.d.hv, dg);
}
