// Linear attention with a decay for each head: the products of rows (formulas in decay.cuh),
//   out_i = f_i M^T x_i + scale sum_j e_ij (x_i . y_j) z_j
// over the tokens j of i's span up to i, or from i on.  A block of four warps takes 64 rows i of one
// head, 16 a warp: first the state's share, then the span's blocks of 64 tokens one after the other,
// the one on the diagonal among them.  A warp's scores stay in its registers: as accumulators they
// are, masked and decayed, the next product's A operand.
//
// Products keep float32 accuracy: an operand that is not exact in tf32 goes in two tf32 parts (delta.cuh), every sum is short and
// joins the others by float32 additions.
//
// 2467 tokens x 8 heads of 96 x 80 in float32, spans of 64: 44 us, bound by the products of a block in order (two warps a
// scheduler, which is what 255 registers allow; tensor pipe 34 %).  A state in four pieces, each waited for, was 6 us slower.
#include "decay.cuh"

namespace {

using namespace zs;

constexpr int kThreads = 128;

template <typename T, int CA, int CB, bool SELF>
struct RowSmem {
    static constexpr int LDA = tile_ld<T>(CA), LDB = tile_ld<T>(CB);
    static constexpr int LDM = CB + 8, LDMT = CA + 8;  // CA rows of a state's, or CB rows of CA columns
    T x[kChunk * LDA];
    T self[SELF ? kChunk * LDB : 8];
    union {
        struct {
            T y[kChunk * LDA];
            T z[kChunk * LDB];
        };
        float m[CA * LDM > CB * LDMT ? CA * LDM : CB * LDMT];
    };
    float2 b[kSpanMost];
};

// The rows of one column of z on the diagonal's tile that are an infinity or NaN: the first of them, or the last
// one (-1 or 64: none).
template <typename T, int LD>
__device__ __noinline__ int bad_row(const T *z, int c, bool back) {
    for (int i = 0; i < kChunk; i++) {
        const int r = back ? kChunk - 1 - i : i;
        if (!isfinite(to_f32(z[r * LD + c]))) return r;
    }
    return back ? -1 : kChunk;
}

// `rows` x `cols` float32 values at distance ld, of which those below n and d are there, zeros elsewhere.
template <int LD>
__device__ __forceinline__ void load_state(float *dst, const float *src, int64_t ld, int rows, int cols, int n, int d) {
    if (((uintptr_t)src & 15) == 0 && ld % 4 == 0 && d % 4 == 0) {
        const int per = cols / 4;
        for (int i = threadIdx.x; i < rows * per; i += kThreads) {
            const int r = i / per, c = (i - r * per) * 4;
            const bool in = r < n && c < d;
            cp_async16(dst + r * LD + c, src + (in ? r * ld + c : 0), in ? 16 : 0);
        }
    } else {
        for (int i = threadIdx.x; i < rows * cols; i += kThreads) {
            const int r = i / cols, c = i - r * cols;
            const bool in = r < n && c < d;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst + r * LD + c)),
                         "l"(src + (in ? r * ld + c : 0)), "r"(in ? 4 : 0)
                         : "memory");
        }
    }
}

template <typename T, int CA, int CB, bool SELF>
__global__ void __launch_bounds__(kThreads, 2)
k_decay_rows(const DecayGeom geo, const DecayProduct p, const DecayRows self) {
    using Smem = RowSmem<T, CA, CB, SELF>;
    constexpr bool EXACT = sizeof(T) == 2;
    constexpr int LDA = Smem::LDA, LDB = Smem::LDB, LDM = Smem::LDM, LDMT = Smem::LDMT, NB = CB / 8;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    after_previous();
    may_start_next();
    const int per = geo.span / kChunk, span = blockIdx.x / per, qb = blockIdx.x - span * per;
    const int head = blockIdx.y, c0 = blockIdx.z * CB, bcols = p.z.cols;
    const int2 sp = geo.d.chunk[span];
    T *const out = (T *)p.out + (int64_t)head * bcols + c0;
    const int cols = min(CB, bcols - c0);
    if (sp.y == 0) {
        if (qb == 0)
            tokens_outside(geo.d, span, [&](int64_t t0, int64_t t1, int worker, int workers) {
                zero_tokens(out, p.ldo, t0, t1, cols, worker, workers);
            });
        return;
    }
    const int i0 = qb * kChunk, n = sp.y;
    if (i0 >= n) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int group = geo.d.hv / geo.d.hk, blocks = (n + kChunk - 1) / kChunk;
    const int rows = min(kChunk, n - i0), m0 = warp * 16;
    const int acols = p.x.cols;
    const bool one = acols <= CA;  // x's columns in one piece
    auto at = [&](const DecayRows &r, int hv, int tok) {
        const int h = SELF && (&r == &self || r.key) ? head : r.key ? hv / group : hv;
        return (const T *)r.p + (int64_t)(sp.x + tok) * r.ld + (int64_t)h * r.dist;
    };
    float acc[NB][4] = {};
#pragma unroll 1
    for (int r = 0; r < (SELF ? group : 1); r++) {
        const int hv = SELF ? head * group + r : head;
        const int64_t slot = (int64_t)span * geo.d.hv + hv;
        __syncthreads();  // the last value head's tiles are read
        if (SELF && r == 0) load_tile<T, CB, kThreads>(sm.self, at(self, hv, i0), self.ld, rows, self.dist);
        // ---------------------------------------------------- the state's share
        const float *M = (const float *)p.m + slot * geo.d.dk * geo.d.dv;
        float share[SELF ? NB : 1][4] = {};
        float(&s)[SELF ? NB : NB][4] = *reinterpret_cast<float(*)[NB][4]>(SELF ? &share[0][0] : &acc[0][0]);
#pragma unroll 1
        for (int a0 = 0; a0 < acols; a0 += CA) {
            if (a0) __syncthreads();
            load_tile<T, CA, kThreads>(sm.x, at(p.x, hv, i0) + a0, p.x.ld, rows, min(CA, p.x.dist - a0));
            if (p.turned)  // M is CB's rows x acols
                load_state<LDMT>(sm.m, M + (int64_t)c0 * acols + a0, acols, CB, CA, bcols - c0, acols - a0);
            else
                load_state<LDM>(sm.m, M + (int64_t)a0 * bcols + c0, bcols, CA, CB, acols - a0, bcols - c0);
            cp_commit();
            if (a0 == 0)
                for (int i = tid; i < n; i += kThreads) sm.b[i] = geo.gates[slot * geo.span + i];
            cp_wait<0>();
            __syncthreads();
#pragma unroll 1
            for (int c = 0; c < CA && a0 + c < acols; c += 32) {
                float2 r0[4], r1[4];
                frag4<T, LDA, false>(sm.x, m0, c, r0);
                frag4<T, LDA, false>(sm.x, m0 + 8, c, r1);
                SplitA a[4];
#pragma unroll
                for (int i = 0; i < 4; i++) a[i].set(r0[i].x, r0[i].y, r1[i].x, r1[i].y);
#pragma unroll
                for (int j = 0; j < NB; j += 4) {
                    float2 f[4][4];  // [k step][column tile]
                    if (p.turned) {
#pragma unroll
                        for (int u = 0; u < 4; u++) {
                            float2 h[4];
                            frag4<float, LDMT, false>(sm.m, (j + u) * 8, c, h);
#pragma unroll
                            for (int i = 0; i < 4; i++) f[i][u] = h[i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; i++) frag4<float, LDM, true>(sm.m, c + i * 8, j * 8, f[i]);
                    }
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        Acc v;
                        v.zero();
#pragma unroll
                        for (int i = 0; i < 4; i++) mma_split<EXACT, false>(v, a[i], f[i][u]);
#pragma unroll
                        for (int e = 0; e < 4; e++) s[j + u][e] += v.get(e);
                    }
                }
            }
        }
        const int ra = m0 + g, rb = m0 + g + 8;  // the lane's rows
        const float2 ba = sm.b[min(i0 + ra, n - 1)], bb = sm.b[min(i0 + rb, n - 1)];
        {
            const float2 zero = make_float2(0.f, 0.f), last = sm.b[n - 1];
            const float fa = p.back ? decay_exp(last, ba) : geo.d.scale * decay_exp(ba, zero);
            const float fb = p.back ? decay_exp(last, bb) : geo.d.scale * decay_exp(bb, zero);
            float da = 0.f, db = 0.f;
#pragma unroll
            for (int j = 0; j < NB; j++) {
                s[j][0] *= fa, s[j][1] *= fa, s[j][2] *= fb, s[j][3] *= fb;
                if (SELF) {
                    const T *qa = sm.self + ra * LDB + j * 8 + 2 * t, *qc = sm.self + rb * LDB + j * 8 + 2 * t;
                    da = fmaf(s[j][0], to_f32(qa[0]), fmaf(s[j][1], to_f32(qa[1]), da));
                    db = fmaf(s[j][2], to_f32(qc[0]), fmaf(s[j][3], to_f32(qc[1]), db));
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[j][e] += s[j][e];
                }
            }
            if (SELF) {
                da += __shfl_xor_sync(0xffffffffu, da, 1), db += __shfl_xor_sync(0xffffffffu, db, 1);
                da += __shfl_xor_sync(0xffffffffu, da, 2), db += __shfl_xor_sync(0xffffffffu, db, 2);
                if (t == 0 && ra < rows) p.sums[0][(int64_t)(sp.x + i0 + ra) * geo.d.hv + hv] = da;
                if (t == 0 && rb < rows) p.sums[0][(int64_t)(sp.x + i0 + rb) * geo.d.hv + hv] = db;
            }
        }
        // ---------------------------------------------------- the span's tokens
        float pa = 0.f, pb = 0.f;
#pragma unroll 1
        for (int jb = p.back ? qb : 0; jb < (p.back ? blocks : qb + 1); jb++) {
            const int j0 = jb * kChunk, nj = min(kChunk, n - j0);
            Acc sc[8];
#pragma unroll
            for (int j = 0; j < 8; j++) sc[j].zero();
#pragma unroll 1
            for (int a0 = 0; a0 < acols; a0 += CA) {
                __syncthreads();  // the tiles of before are read
                if (!one) load_tile<T, CA, kThreads>(sm.x, at(p.x, hv, i0) + a0, p.x.ld, rows, min(CA, p.x.dist - a0));
                load_tile<T, CA, kThreads>(sm.y, at(p.y, hv, j0) + a0, p.y.ld, nj, min(CA, p.y.dist - a0));
                if (a0 == 0) load_tile<T, CB, kThreads>(sm.z, at(p.z, hv, j0) + c0, p.z.ld, nj, min(CB, p.z.dist - c0));
                cp_commit();
                cp_wait<0>();
                __syncthreads();
#pragma unroll 1
                for (int c = 0; c < CA; c += 32) {
                    float2 r0[4], r1[4], f[4];
                    frag4<T, LDA, false>(sm.x, m0, c, r0);
                    frag4<T, LDA, false>(sm.x, m0 + 8, c, r1);
                    SplitA a[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) a[i].set(r0[i].x, r0[i].y, r1[i].x, r1[i].y);
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        frag4<T, LDA, false>(sm.y, j * 8, c, f);
#pragma unroll
                        for (int i = 0; i < 4; i++) mma_split<EXACT, EXACT>(sc[j], a[i], f[i]);
                    }
                }
            }
            SplitA P[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int row = i0 + (e < 2 ? ra : rb), col = j0 + j * 8 + 2 * t + (e & 1);
                    const float2 bc = sm.b[min(col, n - 1)], br = e < 2 ? ba : bb;
                    const bool in = (p.back ? col >= row : col <= row) && col < n;
                    const float w = p.back ? decay_exp(bc, br) : decay_exp(br, bc);
                    v[e] = in ? geo.d.scale * sc[j].get(e) * w : 0.f;
                }
                P[j].set(v);
                if (SELF) {  // self's scores with z, pair by pair
                    Acc o;
                    o.zero();
#pragma unroll 1
                    for (int c = 0; c < CB; c += 32) {
                        float2 r0[4], r1[4], f[4];
                        frag4<T, LDB, false>(sm.self, m0, c, r0);
                        frag4<T, LDB, false>(sm.self, m0 + 8, c, r1);
                        frag4<T, LDB, false>(sm.z, j * 8, c, f);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            SplitA a;
                            a.set(r0[i].x, r0[i].y, r1[i].x, r1[i].y);
                            mma_split<EXACT, EXACT>(o, a, f[i]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int row = i0 + (e < 2 ? ra : rb), col = j0 + j * 8 + 2 * t + (e & 1);
                        if (row == col || (p.back ? col < row || col >= n : col > row)) continue;
                        if (e < 2)
                            pa = fmaf(v[e], o.get(e), pa);
                        else
                            pb = fmaf(v[e], o.get(e), pb);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < NB; j += 4) {
                Acc v[4];
                auto product = [&](bool clean) {
#pragma unroll
                    for (int u = 0; u < 4; u++) v[u].zero();
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        float2 f[4];
                        frag4<T, LDB, true>(sm.z, k * 8, j * 8, f);
                        if (clean)
#pragma unroll
                            for (int u = 0; u < 4; u++) f[u] = make_float2(isfinite(f[u].x) ? f[u].x : 0.f, isfinite(f[u].y) ? f[u].y : 0.f);
#pragma unroll
                        for (int u = 0; u < 4; u++) mma_split<false, EXACT>(v[u], P[k], f[u]);
                    }
                };
                product(false);
                if (jb == qb) {
                    // An infinity or NaN of a token that the mask leaves out has made NaN of its zeros: without those values,
                    // and NaN where they count.
                    float w[4][4];
#pragma unroll
                    for (int u = 0; u < 4; u++)
#pragma unroll
                        for (int e = 0; e < 4; e++) w[u][e] = v[u].get(e);
                    if (not_finite(w)) {
                        product(true);
#pragma unroll
                        for (int u = 0; u < 4; u++)
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                const int bad = bad_row<T, LDB>(sm.z, (j + u) * 8 + 2 * t + h, p.back);
                                if (p.back ? ra <= bad : ra >= bad) v[u].c[h] = __int_as_float(0x7fc00000);
                                if (p.back ? rb <= bad : rb >= bad) v[u].c[2 + h] = __int_as_float(0x7fc00000);
                            }
                    }
                }
#pragma unroll
                for (int u = 0; u < 4; u++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[j + u][e] += v[u].get(e);
            }
        }
        if (SELF) {
            pa += __shfl_xor_sync(0xffffffffu, pa, 1), pb += __shfl_xor_sync(0xffffffffu, pb, 1);
            pa += __shfl_xor_sync(0xffffffffu, pa, 2), pb += __shfl_xor_sync(0xffffffffu, pb, 2);
            if (t == 0 && ra < rows) p.sums[1][(int64_t)(sp.x + i0 + ra) * geo.d.hv + hv] = pa;
            if (t == 0 && rb < rows) p.sums[1][(int64_t)(sp.x + i0 + rb) * geo.d.hv + hv] = pb;
        }
    }
    T *po = out + (int64_t)(sp.x + i0) * p.ldo;
#pragma unroll
    for (int j = 0; j < NB; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int r = m0 + g + (e >> 1) * 8, c = j * 8 + 2 * t + (e & 1);
            if (r < rows && c < cols) po[(int64_t)r * p.ldo + c] = from_f32<T>(acc[j][e]);
        }
}

template <typename T, int CA, int CB, bool SELF>
cudaError_t rows_as(const DecayGeom &g, const DecayProduct &p, bool next, cudaStream_t st) {
    constexpr int smem = (int)sizeof(RowSmem<T, CA, CB, SELF>);
    static_assert(smem <= 232448, "shared memory of a block");
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_decay_rows<T, CA, CB, SELF>, smem);
    if (attr != cudaSuccess) return attr;
    const dim3 grid((unsigned)(g.d.nchunks * (g.span / kChunk)), (unsigned)p.heads, (unsigned)((p.z.cols + CB - 1) / CB));
    return launch(next, k_decay_rows<T, CA, CB, SELF>, grid, kThreads, smem, st, g, p, p.self ? *p.self : DecayRows{});
}
template <typename T, bool SELF>
cudaError_t rows(const DecayGeom &g, const DecayProduct &p, bool next, cudaStream_t st) {
#define ROWS_GO(CA) (p.z.cols <= 64 ? rows_as<T, CA, 64, SELF>(g, p, next, st) : rows_as<T, CA, 128, SELF>(g, p, next, st))
    return p.x.cols <= 64 ? ROWS_GO(64) : ROWS_GO(128);
#undef ROWS_GO
}

}  // namespace

cudaError_t zs_launch_decay_rows(int type, const DecayGeom &g, const DecayProduct &p, bool next, cudaStream_t st, int64_t *launches) {
    ++*launches;
#define ROWS_TYPE(T) (p.self ? rows<T, true>(g, p, next, st) : rows<T, false>(g, p, next, st))
    return type == ZSOLVE_F32 ? ROWS_TYPE(float) : type == ZSOLVE_BF16 ? ROWS_TYPE(bf16) : ROWS_TYPE(f16);
#undef ROWS_TYPE
}
