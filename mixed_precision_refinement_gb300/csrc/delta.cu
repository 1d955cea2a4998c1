// The gated delta rule in chunks of 64 tokens, forward: the chunk table, the
// terms of every chunk that do not depend on the state, and the recurrence
// over the chunks (the formulas are in delta.cuh).
#include <algorithm>

#include "delta.cuh"

namespace {

using namespace zs;

// ---------------------------------------------------------------- chunk table

// Sequences from their offsets (NULL: equal lengths), their first chunks, and
// the chunks' tokens.  Offsets that do not ascend within 0 .. tokens are
// brought into that range one after the other, so that no later access leaves
// the tensors.  One block: the sequences are few beside the tokens.
__global__ void __launch_bounds__(1024)
k_delta_plan(const int64_t *__restrict__ offsets, int nseq, int64_t tokens, int nchunks, int *__restrict__ first,
             int2 *__restrict__ seq, int2 *__restrict__ chunk) {
    __shared__ int64_t s_end[32];
    __shared__ int s_sum[32];
    __shared__ int64_t s_carry;
    __shared__ int s_chunks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) s_carry = 0, s_chunks = 0;
    for (int i = threadIdx.x; i < nchunks; i += 1024) chunk[i] = make_int2(0, 0);
    __syncthreads();
    for (int base = 0; base < nseq; base += 1024) {
        const int i = base + threadIdx.x;
        // the running maximum of the offsets: where sequence i ends
        int64_t end = 0;
        if (i < nseq) {
            end = offsets ? offsets[i + 1] : tokens / nseq * (i + 1);
            end = end < 0 ? 0 : end > tokens ? tokens : end;
        }
        int64_t lo = i == 0 && offsets ? (offsets[0] < 0 ? 0 : offsets[0] > tokens ? tokens : offsets[0]) : 0;
        if (end < lo) end = lo;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o && v > end) end = v;
        }
        if (lane == 31) s_end[warp] = end;
        __syncthreads();
        int64_t before = s_carry;
        for (int w = 0; w < warp; w++) before = s_end[w] > before ? s_end[w] : before;
        if (before > end) end = before;
        int64_t start = __shfl_up_sync(0xffffffffu, end, 1);
        if (lane == 0) start = before;
        if (start < lo) start = lo;
        int n = i < nseq ? (int)((end - start + kChunk - 1) / kChunk) : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane == 31) s_sum[warp] = sum;
        __syncthreads();
        int at = s_chunks + sum - n;
        for (int w = 0; w < warp; w++) at += s_sum[w];
        if (i < nseq) {
            first[i] = at;
            seq[i] = make_int2((int)start, (int)(end - start));
            for (int c = 0; c < n; c++) {
                const int64_t left = end - start - (int64_t)c * kChunk;
                chunk[at + c] = make_int2((int)start + c * kChunk, left < kChunk ? (int)left : kChunk);
            }
        }
        __syncthreads();
        if (threadIdx.x == 1023) {
            s_carry = end;
            s_chunks = at + n;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) first[nseq] = s_chunks;
}

// ---------------------------------------------------------------- terms

constexpr int kTermThreads = 256;
constexpr int kLdA = kChunk + 4;

// T <- inverse of I + A for a strictly lower A, both in shared memory (row
// stride kLdA), by blocks: the four 16 x 16 diagonal blocks by substitution,
// then pairs of blocks joined: [T1 0; -T2 A21 T1, T2].  tmp: 32 x kLdA.
__device__ void invert_unit_lower(const float *A, float *T, float *tmp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kChunk * kChunk; i += kTermThreads) {
        const int r = i >> 6, c = i & 63;
        if ((r >> 4) != (c >> 4)) T[r * kLdA + c] = 0.f;
    }
    if (warp < 4 && lane < 16) {  // column `lane` of diagonal block `warp`
        const float *a = A + (warp * 16) * kLdA + warp * 16;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; i++) {
            float s = i == lane ? 1.f : 0.f;
#pragma unroll
            for (int l = 0; l < i; l++) s = fmaf(-a[i * kLdA + l], x[l], s);
            x[i] = s;
            T[(warp * 16 + i) * kLdA + warp * 16 + lane] = s;
        }
    }
    __syncthreads();
    // 16 -> 32: both pairs at once, an output pair of columns a thread
    {
        const int p = tid >> 7, r = (tid >> 3) & 15, c = (tid & 7) * 2, o = p * 32;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int l = 0; l < 16; l++) {  // A21 T1
            const float a = A[(o + 16 + r) * kLdA + o + l];
            s0 = fmaf(a, T[(o + l) * kLdA + o + c], s0);
            s1 = fmaf(a, T[(o + l) * kLdA + o + c + 1], s1);
        }
        tmp[(p * 16 + r) * kLdA + c] = s0;
        tmp[(p * 16 + r) * kLdA + c + 1] = s1;
        __syncthreads();
        s0 = s1 = 0.f;
#pragma unroll
        for (int l = 0; l < 16; l++) {  // T2 (A21 T1)
            const float a = T[(o + 16 + r) * kLdA + o + 16 + l];
            s0 = fmaf(a, tmp[(p * 16 + l) * kLdA + c], s0);
            s1 = fmaf(a, tmp[(p * 16 + l) * kLdA + c + 1], s1);
        }
        T[(o + 16 + r) * kLdA + o + c] = -s0;
        T[(o + 16 + r) * kLdA + o + c + 1] = -s1;
    }
    __syncthreads();
    // 32 -> 64: four columns a thread
    {
        const int r = tid >> 3, c = (tid & 7) * 4;
        float s[4] = {};
#pragma unroll 8
        for (int l = 0; l < 32; l++) {
            const float a = A[(32 + r) * kLdA + l];
            const float4 b = *reinterpret_cast<const float4 *>(T + l * kLdA + c);
            s[0] = fmaf(a, b.x, s[0]), s[1] = fmaf(a, b.y, s[1]), s[2] = fmaf(a, b.z, s[2]), s[3] = fmaf(a, b.w, s[3]);
        }
        *reinterpret_cast<float4 *>(tmp + r * kLdA + c) = make_float4(s[0], s[1], s[2], s[3]);
        __syncthreads();
        s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll 8
        for (int l = 0; l < 32; l++) {
            const float a = T[(32 + r) * kLdA + 32 + l];
            const float4 b = *reinterpret_cast<const float4 *>(tmp + l * kLdA + c);
            s[0] = fmaf(a, b.x, s[0]), s[1] = fmaf(a, b.y, s[1]), s[2] = fmaf(a, b.z, s[2]), s[3] = fmaf(a, b.w, s[3]);
        }
        *reinterpret_cast<float4 *>(T + (32 + r) * kLdA + c) = make_float4(-s[0], -s[1], -s[2], -s[3]);
    }
    __syncthreads();
}

template <typename T, int DK>
struct TermSmem {
    T k[kChunk * tile_ld<T>(DK)];
    T q[kChunk * tile_ld<T>(DK)];
    float kk[kChunk * kLdA];
    float qk[kChunk * kLdA];
    float a[kChunk * kLdA];
    float t[kChunk * kLdA];
    float tmp[32 * kLdA];
    float bh[kChunk], bl[kChunk], beta[kChunk];
};

// One block for a chunk and a key head: K K^T and Q K^T once, then A, T, P and
// the vectors of each value head that shares the key head.
template <typename T, int DK>
__global__ void __launch_bounds__(kTermThreads)
k_delta_terms(const DeltaGeom geo, const DeltaTerms out, int vec) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    TermSmem<T, DK> &sm = *reinterpret_cast<TermSmem<T, DK> *>(smem_raw);
    constexpr bool EXACT = sizeof(T) == 2;
    constexpr int LD = tile_ld<T>(DK);
    const int2 ch = geo.chunk[blockIdx.x];
    const int n = ch.y;
    if (n == 0) return;
    const int hk = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    load_tile<T, DK, kTermThreads>(sm.k, (const T *)geo.k + (int64_t)ch.x * geo.ldk + (int64_t)hk * geo.dk, geo.ldk, n, geo.dk, vec);
    load_tile<T, DK, kTermThreads>(sm.q, (const T *)geo.q + (int64_t)ch.x * geo.ldq + (int64_t)hk * geo.dk, geo.ldq, n, geo.dk, vec);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    {
        // warps 0-3: rows 16 w of K K^T, warps 4-7: of Q K^T; tiles on and below the diagonal
        const int m = (warp & 3) * 16;
        const T *x = warp < 4 ? sm.k : sm.q;
        float *dst = warp < 4 ? sm.kk : sm.qk;
        float acc[8][4] = {};
#pragma unroll 1
        for (int c = 0; c < DK; c += 32) {
            float2 r0[4], r1[4], b[4];
            frag4<T, LD, false>(x, m, c, r0);
            frag4<T, LD, false>(x, m + 8, c, r1);
            SplitA a[4];
#pragma unroll
            for (int i = 0; i < 4; i++) a[i].set(r0[i].x, r0[i].y, r1[i].x, r1[i].y);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (j * 8 > m + 8) continue;
                frag4<T, LD, false>(sm.k, j * 8, c, b);
#pragma unroll
                for (int i = 0; i < 4; i++) mma_split<EXACT, EXACT>(acc[j], a[i], b[i]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (j * 8 > m + 8) continue;
            *reinterpret_cast<float2 *>(dst + (m + g) * kLdA + j * 8 + 2 * t) = make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2 *>(dst + (m + g + 8) * kLdA + j * 8 + 2 * t) = make_float2(acc[j][2], acc[j][3]);
        }
    }
    const int group = geo.hv / geo.hk;
    for (int r = 0; r < group; r++) {
        const int hv = hk * group + r;
        const int64_t slot = (int64_t)blockIdx.x * geo.hv + hv;
        __syncthreads();  // kk, qk complete; the previous head's readers done
        if (warp == 0) {
            gate_sums(geo, ch, hv, sm.bh, sm.bl);
        } else if (warp == 1) {
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int i = 2 * lane + e;
                sm.beta[i] = i < n ? geo.beta[(int64_t)(ch.x + i) * geo.hv + hv] : 0.f;
            }
        }
        __syncthreads();
        if (tid < kChunk) {
            float *v = out.vec + slot * kVec;
            v[tid] = expf(sm.bh[tid] + sm.bl[tid]);
            v[kChunk + tid] = expf((sm.bh[kChunk - 1] - sm.bh[tid]) + (sm.bl[kChunk - 1] - sm.bl[tid]));
            v[2 * kChunk + tid] = sm.beta[tid];
        }
        for (int i = tid; i < kChunk * kChunk; i += kTermThreads) {
            const int y = i >> 6, x = i & 63;
            float av = 0.f, pv = 0.f;
            if (x <= y) {
                const float e = expf((sm.bh[y] - sm.bh[x]) + (sm.bl[y] - sm.bl[x]));
                if (x < y) av = sm.beta[y] * sm.kk[y * kLdA + x] * e;
                pv = geo.scale * sm.qk[y * kLdA + x] * e;
            }
            sm.a[y * kLdA + x] = av;
            if (out.p) out.p[slot * (kChunk * kChunk) + i] = pv;
        }
        __syncthreads();
        invert_unit_lower(sm.a, sm.t, sm.tmp);
        for (int i = tid; i < kChunk * kChunk / 4; i += kTermThreads) {
            const int y = i >> 4, x = (i & 15) * 4;
            *reinterpret_cast<float4 *>(out.t + slot * (kChunk * kChunk) + y * kChunk + x) =
                *reinterpret_cast<const float4 *>(sm.t + y * kLdA + x);
        }
    }
}

// ---------------------------------------------------------------- chain

// The recurrence.  A block owns 16 NV value columns of one head of one
// sequence; a group of WK = DK / 32 warps owns 16 of them, and warp w of the
// group the 32 x 16 block of S^T for key columns 32 w ..: its accumulators,
// which are also its A operands.  Per chunk the group exchanges three small
// results through shared memory: the partial sums of S^T K^T (over the warps'
// key columns), X^T and U^T; token tiles of 8 are dealt so that the triangular
// products are equal shares (tile_of).
template <typename T, int DK>
struct ChainCfg {
    static constexpr int WK = DK / 32;
    static constexpr int NV = WK == 4 ? 2 : 4;
    static constexpr int NT = 32 * WK * NV;
    static constexpr int NTILE = 8 / WK;
    static constexpr int LD = tile_ld<T>(DK);
    // two stages of the chunk's operands where they fit
    static constexpr int STAGES = sizeof(T) == 2 || DK < 128 ? 2 : 1;
};

template <typename T, int DK>
struct ChainStage {
    T k[kChunk * tile_ld<T>(DK)];
    T q[kChunk * tile_ld<T>(DK)];
    float t[kChunk * kLdT];
    float p[kChunk * kLdT];
    float vec[kVec];
};

template <typename T, int DK>
struct ChainSmem {
    using C = ChainCfg<T, DK>;
    ChainStage<T, DK> st[C::STAGES];
    float part[C::NV][C::WK][16 * kLdT];
    float x[C::NV][16 * kLdT];
    float u[C::NV][16 * kLdT];
};

template <typename T, int DK, bool OUT>
__global__ void __launch_bounds__(ChainCfg<T, DK>::NT, 1)
k_delta_chain(const DeltaGeom geo, const DeltaTerms terms, const float *__restrict__ s0, T *__restrict__ o,
              int64_t ldo, float *__restrict__ sn, float *__restrict__ states, float *__restrict__ us, int vec) {
    using C = ChainCfg<T, DK>;
    constexpr int WK = C::WK, NV = C::NV, NT = C::NT, LD = C::LD, NTILE = C::NTILE;
    constexpr bool EXACT = sizeof(T) == 2;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    ChainSmem<T, DK> &sm = *reinterpret_cast<ChainSmem<T, DK> *>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int grp = warp / WK, w = warp - grp * WK;
    const int si = blockIdx.x / geo.hv, hv = blockIdx.x - si * geo.hv, hk = hv / (geo.hv / geo.hk);
    const int v0 = ((int)blockIdx.y * NV + grp) * 16;  // the group's value columns
    const int d0 = w * 32;                             // the warp's key columns
    const int64_t state_at = ((int64_t)si * geo.hv + hv) * geo.dk * geo.dv;

    auto load = [&](int c, int stage) {
        const int2 ch = geo.chunk[c];
        ChainStage<T, DK> &s = sm.st[stage];
        const int64_t slot = (int64_t)c * geo.hv + hv;
        load_tile<T, DK, NT>(s.k, (const T *)geo.k + (int64_t)ch.x * geo.ldk + (int64_t)hk * geo.dk, geo.ldk, ch.y, geo.dk, vec);
        load_square<NT>(s.t, terms.t + slot * (kChunk * kChunk));
        if (OUT) {
            load_tile<T, DK, NT>(s.q, (const T *)geo.q + (int64_t)ch.x * geo.ldq + (int64_t)hk * geo.dk, geo.ldq, ch.y, geo.dk, vec);
            load_square<NT>(s.p, terms.p + slot * (kChunk * kChunk));
        }
        for (int i = threadIdx.x; i < kVec / 4; i += NT) cp_async16(s.vec + 4 * i, terms.vec + slot * kVec + 4 * i, 16);
        cp_commit();
    };

    // S^T: rows v0 + g, v0 + g + 8, columns d0 + 8 j + 2t, + 1
    float S[4][4];
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int v = v0 + g + (e >> 1) * 8, d = d0 + 8 * j + 2 * t + (e & 1);
            S[j][e] = s0 && v < geo.dv && d < geo.dk ? s0[state_at + (int64_t)d * geo.dv + v] : 0.f;
        }
    auto put_state = [&](float *dst) {
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int v = v0 + g + (e >> 1) * 8, d = d0 + 8 * j + 2 * t + (e & 1);
                if (v < geo.dv && d < geo.dk) dst[(int64_t)d * geo.dv + v] = S[j][e];
            }
    };

    const int c0 = geo.first[si], c1 = geo.first[si + 1];
    if (c0 < c1) load(c0, 0);
    for (int c = c0; c < c1; c++) {
        const int stage = C::STAGES == 2 ? (c - c0) & 1 : 0;
        cp_wait<0>();
        __syncthreads();  // the stage is complete, and every warp is done with the previous chunk
        if (C::STAGES == 2 && c + 1 < c1) load(c + 1, stage ^ 1);
        ChainStage<T, DK> &st = sm.st[stage];
        const int2 ch = geo.chunk[c];
        const int64_t slot = (int64_t)c * geo.hv + hv;
        if (states) put_state(states + slot * geo.dk * geo.dv);

        // V^T of the warp's token tiles, for X (the loads run during the products)
        float vt[NTILE][4];
#pragma unroll
        for (int i = 0; i < NTILE; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int v = v0 + g + (e >> 1) * 8, tok = tile_of<WK>(w, i) * 8 + 2 * t + (e & 1);
                vt[i][e] = v < geo.dv && tok < ch.y
                               ? to_f32(((const T *)geo.v)[(int64_t)(ch.x + tok) * geo.ldv + (int64_t)hv * geo.dv + v])
                               : 0.f;
            }

        // partial S^T K^T and S^T Q^T over the warp's key columns
        float po[8][4];
        {
            SplitA a[4];
#pragma unroll
            for (int j = 0; j < 4; j++) a[j].set(S[j]);
            float *part = sm.part[grp][w];
#pragma unroll
            for (int n = 0; n < 8; n++) {
                float2 b[4];
                float r[4] = {};
                frag4<T, LD, false>(st.k, n * 8, d0, b);
#pragma unroll
                for (int j = 0; j < 4; j++) mma_split<EXACT>(r, a[j], b[j]);
                *reinterpret_cast<float2 *>(part + g * kLdT + n * 8 + 2 * t) = make_float2(r[0], r[1]);
                *reinterpret_cast<float2 *>(part + (g + 8) * kLdT + n * 8 + 2 * t) = make_float2(r[2], r[3]);
                if (OUT) {
                    frag4<T, LD, false>(st.q, n * 8, d0, b);
#pragma unroll
                    for (int e = 0; e < 4; e++) po[n][e] = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; j++) mma_split<EXACT, EXACT>(po[n], a[j], b[j]);
                }
            }
        }
        group_sync<WK>(grp);
        // X^T = beta (V - c K S)^T at the warp's token tiles
#pragma unroll
        for (int i = 0; i < NTILE; i++) {
            const int n = tile_of<WK>(w, i) * 8 + 2 * t;
            float2 lo = make_float2(0.f, 0.f), hi = lo;
#pragma unroll
            for (int p = 0; p < WK; p++) {
                const float2 y = *reinterpret_cast<const float2 *>(sm.part[grp][p] + g * kLdT + n);
                const float2 z = *reinterpret_cast<const float2 *>(sm.part[grp][p] + (g + 8) * kLdT + n);
                lo.x += y.x, lo.y += y.y, hi.x += z.x, hi.y += z.y;
            }
            const float ca = st.vec[n], cb = st.vec[n + 1], ba = st.vec[2 * kChunk + n], bb = st.vec[2 * kChunk + n + 1];
            *reinterpret_cast<float2 *>(sm.x[grp] + g * kLdT + n) =
                make_float2(ba * (vt[i][0] - ca * lo.x), bb * (vt[i][1] - cb * lo.y));
            *reinterpret_cast<float2 *>(sm.x[grp] + (g + 8) * kLdT + n) =
                make_float2(ba * (vt[i][2] - ca * hi.x), bb * (vt[i][3] - cb * hi.y));
        }
        group_sync<WK>(grp);
        if (OUT) {
            float *part = sm.part[grp][w];
#pragma unroll
            for (int n = 0; n < 8; n++) {
                *reinterpret_cast<float2 *>(part + g * kLdT + n * 8 + 2 * t) = make_float2(po[n][0], po[n][1]);
                *reinterpret_cast<float2 *>(part + (g + 8) * kLdT + n * 8 + 2 * t) = make_float2(po[n][2], po[n][3]);
            }
        }
        // U^T = X^T T^T at the warp's token tiles
        {
            float u[NTILE][4] = {};
#pragma unroll
            for (int k = 0; k < 8; k++) {
                SplitA a;
                const float2 y = *reinterpret_cast<const float2 *>(sm.x[grp] + g * kLdT + k * 8 + 2 * t);
                const float2 z = *reinterpret_cast<const float2 *>(sm.x[grp] + (g + 8) * kLdT + k * 8 + 2 * t);
                a.set(y.x, y.y, z.x, z.y);
#pragma unroll
                for (int i = 0; i < NTILE; i++) {
                    const int n = tile_of<WK>(w, i);
                    if (k > n) continue;
                    const float2 b = *reinterpret_cast<const float2 *>(st.t + (n * 8 + g) * kLdT + k * 8 + 2 * t);
                    mma_split<false>(u[i], a, b);
                }
            }
#pragma unroll
            for (int i = 0; i < NTILE; i++) {
                const int n = tile_of<WK>(w, i) * 8 + 2 * t;
                *reinterpret_cast<float2 *>(sm.u[grp] + g * kLdT + n) = make_float2(u[i][0], u[i][1]);
                *reinterpret_cast<float2 *>(sm.u[grp] + (g + 8) * kLdT + n) = make_float2(u[i][2], u[i][3]);
                if (us) {
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int v = v0 + g + (e >> 1) * 8;
                        if (v < geo.dv) us[(slot * kChunk + n + (e & 1)) * geo.dv + v] = u[i][e];
                    }
                }
            }
        }
        group_sync<WK>(grp);
        // S'^T = c_64 S^T + (e U)^T K: the chunk's sum starts from zero, so that
        // the state is rounded once a chunk; and O^T = scale c (Q S)^T + U^T P^T
        {
            float acc[4][4] = {}, oa[NTILE][4] = {};
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const float2 y = *reinterpret_cast<const float2 *>(sm.u[grp] + g * kLdT + k * 8 + 2 * t);
                const float2 z = *reinterpret_cast<const float2 *>(sm.u[grp] + (g + 8) * kLdT + k * 8 + 2 * t);
                const float ea = st.vec[kChunk + k * 8 + 2 * t], eb = st.vec[kChunk + k * 8 + 2 * t + 1];
                SplitA a;
                a.set(ea * y.x, eb * y.y, ea * z.x, eb * z.y);
                float2 b[4];
                frag4<T, LD, true>(st.k, k * 8, d0, b);
#pragma unroll
                for (int j = 0; j < 4; j++) mma_split<EXACT>(acc[j], a, b[j]);
                if (OUT) {
                    SplitA ua;
                    ua.set(y.x, y.y, z.x, z.y);
#pragma unroll
                    for (int i = 0; i < NTILE; i++) {
                        const int n = tile_of<WK>(w, i);
                        if (k > n) continue;
                        const float2 p = *reinterpret_cast<const float2 *>(st.p + (n * 8 + g) * kLdT + k * 8 + 2 * t);
                        mma_split<false, EXACT>(oa[i], ua, p);
                    }
                }
            }
            const float cend = st.vec[kChunk - 1];
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) S[j][e] = fmaf(cend, S[j][e], acc[j][e]);
            if (OUT) {
#pragma unroll
                for (int i = 0; i < NTILE; i++) {
                    const int n = tile_of<WK>(w, i) * 8 + 2 * t;
                    float2 lo = make_float2(0.f, 0.f), hi = lo;
#pragma unroll
                    for (int p = 0; p < WK; p++) {
                        const float2 y = *reinterpret_cast<const float2 *>(sm.part[grp][p] + g * kLdT + n);
                        const float2 z = *reinterpret_cast<const float2 *>(sm.part[grp][p] + (g + 8) * kLdT + n);
                        lo.x += y.x, lo.y += y.y, hi.x += z.x, hi.y += z.y;
                    }
                    const float ca = geo.scale * st.vec[n], cb = geo.scale * st.vec[n + 1];
                    const float r[4] = {fmaf(ca, lo.x, oa[i][0]), fmaf(cb, lo.y, oa[i][1]), fmaf(ca, hi.x, oa[i][2]),
                                        fmaf(cb, hi.y, oa[i][3])};
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int v = v0 + g + (e >> 1) * 8, tok = n + (e & 1);
                        if (v < geo.dv && tok < ch.y)
                            o[(int64_t)(ch.x + tok) * ldo + (int64_t)hv * geo.dv + v] = from_f32<T>(r[e]);
                    }
                }
            }
        }
        if (C::STAGES == 1) {
            __syncthreads();  // the only stage is free
            if (c + 1 < c1) load(c + 1, 0);
        }
    }
    if (sn) put_state(sn + state_at);
}

template <typename T, int DK>
cudaError_t terms_dk(const DeltaGeom &g, const DeltaTerms &t, cudaStream_t st) {
    const size_t smem = sizeof(TermSmem<T, DK>);
    static const cudaError_t attr = cudaFuncSetAttribute(
        k_delta_terms<T, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(TermSmem<T, DK>));
    if (attr != cudaSuccess) return attr;
    const int vec = mult16(g.q, g.ldq, g.dk, sizeof(T)) && mult16(g.k, g.ldk, g.dk, sizeof(T));
    k_delta_terms<T, DK><<<dim3(g.nchunks, g.hk), kTermThreads, smem, st>>>(g, t, vec);
    return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t chain_dk(const DeltaGeom &g, const DeltaTerms &t, const float *s0, void *o, int64_t ldo, float *sn,
                     float *states, float *us, cudaStream_t st) {
    using C = ChainCfg<T, DK>;
    const size_t smem = sizeof(ChainSmem<T, DK>);
    const int vec = mult16(g.q, g.ldq, g.dk, sizeof(T)) && mult16(g.k, g.ldk, g.dk, sizeof(T));
    const dim3 grid((unsigned)(g.nseq * g.hv), (unsigned)((g.dv + 16 * C::NV - 1) / (16 * C::NV)));
    if (o) {
        static const cudaError_t attr = cudaFuncSetAttribute(
            k_delta_chain<T, DK, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(ChainSmem<T, DK>));
        if (attr != cudaSuccess) return attr;
        k_delta_chain<T, DK, true><<<grid, C::NT, smem, st>>>(g, t, s0, (T *)o, ldo, sn, states, us, vec);
    } else {
        static const cudaError_t attr = cudaFuncSetAttribute(
            k_delta_chain<T, DK, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(ChainSmem<T, DK>));
        if (attr != cudaSuccess) return attr;
        k_delta_chain<T, DK, false><<<grid, C::NT, smem, st>>>(g, t, s0, nullptr, 0, sn, states, us, vec);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t zs_launch_delta_plan(const int64_t *offsets, int nseq, int64_t tokens, int nchunks, int *first, int2 *seq,
                                 int2 *chunk, cudaStream_t st, int64_t *launches) {
    k_delta_plan<<<1, 1024, 0, st>>>(offsets, nseq, tokens, nchunks, first, seq, chunk);
    ++*launches;
    return cudaGetLastError();
}

cudaError_t zs_launch_delta_terms(int type, const DeltaGeom &g, const DeltaTerms &t, cudaStream_t st,
                                  int64_t *launches) {
    ++*launches;
    return DELTA_TYPE(terms_dk, g, t, st);
}

cudaError_t zs_launch_delta_chain(int type, const DeltaGeom &g, const DeltaTerms &t, const float *s0, void *o,
                                  int64_t ldo, float *sn, float *states, float *us, cudaStream_t st,
                                  int64_t *launches) {
    ++*launches;
    return DELTA_TYPE(chain_dk, g, t, s0, o, ldo, sn, states, us, st);
}
