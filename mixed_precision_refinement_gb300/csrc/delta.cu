// The gated delta rule in chunks of 64 tokens, forward: the chunk table, the
// terms of every chunk that do not depend on the state, and the recurrence
// over the chunks (the formulas are in delta.cuh).
#include <algorithm>

#include "delta.cuh"

namespace {

using namespace zs;

// ---------------------------------------------------------------- chunk table

// Sequences from their offsets (NULL: equal lengths), their first chunks of `len` tokens, and
// the chunks' tokens.  Offsets that do not ascend within 0 .. tokens are
// brought into that range one after the other, so that no later access leaves
// the tensors.  One block: the sequences are few beside the tokens.
__global__ void __launch_bounds__(1024)
k_delta_plan(const int64_t *__restrict__ offsets, int nseq, int64_t tokens, int len, int nchunks, int *first, int2 *seq,
             int2 *chunk) {
    __shared__ int64_t s_end[32];
    __shared__ int s_sum[32];
    __shared__ int64_t s_carry;
    __shared__ int s_chunks;
    after_previous();
    may_start_next();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) s_carry = 0, s_chunks = 0;
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
        int n = i < nseq ? (int)((end - start + len - 1) / len) : 0;
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
        }
        __syncthreads();
        if (threadIdx.x == 1023) {
            s_carry = end;
            s_chunks = at + n;
        }
        __syncthreads();
    }
    const int used = s_chunks;
    if (threadIdx.x == 0) first[nseq] = used;
    // a thread a chunk: its sequence is the last whose first chunk is not after it
    // (among empty ones, which share their first chunk with the next)
    for (int c = threadIdx.x; c < nchunks; c += 1024) {
        int2 ch = make_int2(0, 0);
        if (c < used) {
            int lo = 0, hi = nseq;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= c)
                    lo = mid;
                else
                    hi = mid;
            }
            const int2 sq = seq[lo];
            const int at = (c - first[lo]) * len;
            ch = make_int2(sq.x + at, min(sq.y - at, len));
        }
        chunk[c] = ch;
    }
}

// ---------------------------------------------------------------- terms

// One block for a chunk and a key head: K K^T and Q K^T once (tensor cores),
// then, a half block of four warps a value head that shares the key head, A, T
// and P.  The inverse T of I + A by blocks of 16: the diagonal blocks by
// substitution, a lane a column; then warp j finds block column j below them,
//   T_ij = -T_ii (A_ij T_jj + ... + A_i,i-1 T_i-1,j),
// transposed, so that each finished block is, as an accumulator, the A operand
// of the next products.  Bound by the latency of these steps (1.9 of 4 instructions a
// cycle, tensor pipe 16%); two blocks an SM.  8192 tokens x 32 heads of 128, bfloat16:
// 88 us.
constexpr int kTermThreads = 256;
constexpr int kLdA = kChunk + 4;
constexpr int kLdD = 20;

template <typename T, int DK>
struct TermSmem {
    union {
        struct {
            T k[kChunk * tile_ld<T>(DK)];
            T q[kChunk * tile_ld<T>(DK)];
        };
        float a[2][kChunk * kLdT];  // a value head each, once the products are done
    };
    float kk[kChunk * kLdA];
    float kq[kChunk * kLdA];  // K Q^T: the transpose of Q K^T
    float diag[2][4][16 * kLdD];
    float bh[2][kChunk], bl[2][kChunk], beta[2][kChunk];
};

// A 16 x 16 block as two A operands' worth of accumulators
struct Block {
    Acc n[2];  // columns 0-7, 8-15
};

template <typename T, int DK>
__global__ void __launch_bounds__(kTermThreads, 2)
k_delta_terms(const DeltaGeom geo, const DeltaTerms out, T *__restrict__ o, int64_t ldo) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    TermSmem<T, DK> &sm = *reinterpret_cast<TermSmem<T, DK> *>(smem_raw);
    constexpr bool EXACT = sizeof(T) == 2;
    constexpr int LD = tile_ld<T>(DK);
    after_previous();
    may_start_next();
    const int2 ch = geo.chunk[blockIdx.x];
    const int n = ch.y, hk = blockIdx.y;
    if (n == 0) {
        const int cols = geo.hv / geo.hk * geo.dv;
        if (o)
            tokens_outside(geo, blockIdx.x, [&](int64_t t0, int64_t t1, int worker, int workers) {
                zero_tokens(o + (int64_t)hk * cols, ldo, t0, t1, cols, worker, workers);
            });
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    load_tile<T, DK, kTermThreads>(sm.k, (const T *)geo.k + (int64_t)ch.x * geo.ldk + (int64_t)hk * geo.dkp, geo.ldk, n, geo.dkp);
    load_tile<T, DK, kTermThreads>(sm.q, (const T *)geo.q + (int64_t)ch.x * geo.ldq + (int64_t)hk * geo.dkp, geo.ldq, n, geo.dkp);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    {
        // warps 0-3: rows 16 w of K K^T, warps 4-7: of Q K^T; tiles on and below the diagonal
        const int m = (warp & 3) * 16;
        const T *x = warp < 4 ? sm.k : sm.q;
        Acc acc[8];
#pragma unroll
        for (int j = 0; j < 8; j++) acc[j].zero();
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
            const float v[4] = {acc[j].get(0), acc[j].get(1), acc[j].get(2), acc[j].get(3)};
            if (warp < 4) {
                *reinterpret_cast<float2 *>(sm.kk + (m + g) * kLdA + j * 8 + 2 * t) = make_float2(v[0], v[1]);
                *reinterpret_cast<float2 *>(sm.kk + (m + g + 8) * kLdA + j * 8 + 2 * t) = make_float2(v[2], v[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++) sm.kq[(j * 8 + 2 * t + (e & 1)) * kLdA + m + g + (e >> 1) * 8] = v[e];
            }
        }
    }
    const int group = geo.hv / geo.hk, half = warp >> 2, w = warp & 3, ht = tid & 127;
    __syncthreads();  // kk, kq complete; k and q give way to A
    for (int r0 = 0; r0 < group; r0 += 2) {
        const int r = r0 + half;
        if (r < group) {  // the half blocks go their own way: barriers of 128 threads
            const int hv = hk * group + r;
            const int64_t slot = (int64_t)blockIdx.x * geo.hv + hv;
            float *A = sm.a[half], *bh = sm.bh[half], *bl = sm.bl[half], *beta = sm.beta[half];
            if (w == 0) {
                gate_sums(geo, ch, hv, bh, bl);
            } else if (w == 1) {
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int i = 2 * lane + e;
                    beta[i] = i < n ? geo.beta[(int64_t)(ch.x + i) * geo.hv + hv] : 0.f;
                }
            }
            asm volatile("bar.sync %0, 128;" ::"r"(half + 1) : "memory");
            if (ht < kChunk) {
                float *v = out.vec + slot * kVec;
                v[ht] = expf(bh[ht] + bl[ht]);
                v[kChunk + ht] = expf((bh[kChunk - 1] - bh[ht]) + (bl[kChunk - 1] - bl[ht]));
                v[2 * kChunk + ht] = beta[ht];
                v[3 * kChunk + ht] = bh[ht];
                v[4 * kChunk + ht] = bl[ht];
            }
            float *TP = out.tp + slot * kSquare;
#pragma unroll 4
            for (int i = ht; i < kChunk * kChunk; i += 128) {
                const int r = i >> 6, c = i & 63, y = max(r, c), x = min(r, c);
                const float e = expf((bh[y] - bh[x]) + (bl[y] - bl[x]));
                if (c < r)
                    A[r * kLdT + c] = beta[r] * sm.kk[r * kLdA + c] * e;
                else
                    TP[r * kLdT + c] = geo.scale * sm.kq[r * kLdA + c] * e;  // P(c, r)
            }
            asm volatile("bar.sync %0, 128;" ::"r"(half + 1) : "memory");
            {  // diagonal block w: lane l its column l (the upper half of the warp repeats the lower)
                const float *a = A + (w * 16) * kLdT + w * 16;
                const int c = lane & 15;
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    float s0 = i == c ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                    for (int l = 0; l + 1 < i; l += 2) {
                        const float2 al = *reinterpret_cast<const float2 *>(a + i * kLdT + l);
                        s0 = fmaf(-al.x, x[l], s0);
                        s1 = fmaf(-al.y, x[l + 1], s1);
                    }
                    if (i & 1) s0 = fmaf(-a[i * kLdT + i - 1], x[i - 1], s0);
                    x[i] = s0 + s1;
                }
                if (lane < 16) {
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        sm.diag[half][w][i * kLdD + c] = x[i];
                        if (i > c) TP[(w * 16 + i) * kLdT + w * 16 + c] = x[i];
                    }
                }
            }
            asm volatile("bar.sync %0, 128;" ::"r"(half + 1) : "memory");
            // block column w, transposed: Y_i = T_iw^T = -(sum over k of Y_k A_ik^T) T_ii^T
            SplitA y[4][2];
            {
                const float *d = sm.diag[half][w];  // Y_w = T_ww^T
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    const int at = (k * 8 + 2 * t) * kLdD + g;
                    const float c0 = d[at], c1 = d[at + kLdD], c2 = d[at + 8], c3 = d[at + kLdD + 8];
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (i == w) y[i][k].set(c0, c1, c2, c3);
                }
            }
#pragma unroll
            for (int i = 1; i < 4; i++) {
                if (i <= w) continue;
                Block s;
                s.n[0].zero(), s.n[1].zero();
#pragma unroll
                for (int k = 0; k < i; k++) {
                    if (k < w) continue;
#pragma unroll
                    for (int kk = 0; kk < 2; kk++)
#pragma unroll
                        for (int nn = 0; nn < 2; nn++)
                            mma_split<false, false>(s.n[nn], y[k][kk],
                                                    *reinterpret_cast<const float2 *>(A + (i * 16 + nn * 8 + g) * kLdT + k * 16 + kk * 8 + 2 * t));
                }
                // T_ii is zero above its diagonal: an infinity or NaN of a token counts as
                // zero there, and is put back in its own row (those after it have it from A)
                Block z;
                z.n[0].zero(), z.n[1].zero();
                float sv[2][4];
#pragma unroll
                for (int kk = 0; kk < 2; kk++) {
                    float neg[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        sv[kk][e] = s.n[kk].get(e);
                        neg[e] = isfinite(sv[kk][e]) ? -sv[kk][e] : 0.f;
                    }
                    SplitA a;
                    a.set(neg);
#pragma unroll
                    for (int nn = 0; nn < 2; nn++)
                        mma_split<false, false>(z.n[nn], a,
                                                *reinterpret_cast<const float2 *>(sm.diag[half][i] + (nn * 8 + g) * kLdD + kk * 8 + 2 * t));
                }
#pragma unroll
                for (int nn = 0; nn < 2; nn++) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) v[e] = z.n[nn].get(e) + (sv[nn][e] - sv[nn][e]);
                    if (i < 3) y[i][nn].set(v);
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        TP[(i * 16 + nn * 8 + 2 * t + (e & 1)) * kLdT + w * 16 + g + (e >> 1) * 8] = v[e];
                }
            }
            asm volatile("bar.sync %0, 128;" ::"r"(half + 1) : "memory");  // A, diag free for the next head
        }
    }
}

// ---------------------------------------------------------------- alignment

// Heads whose rows the bulk copies cannot address (16 bytes) copied to rows
// that they can, each head padded with zeros to dp values.
template <typename T>
__global__ void __launch_bounds__(256)
k_delta_pack(const T *__restrict__ src, int64_t ld, int64_t tokens, int heads, int d, int dp, T *__restrict__ dst) {
    after_previous();
    may_start_next();
    const int64_t n = tokens * heads * dp;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / dp, tok = row / heads;
        const int c = (int)(i - row * dp), h = (int)(row - tok * heads);
        dst[i] = c < d ? src[tok * ld + (int64_t)h * d + c] : from_f32<T>(0.f);
    }
}

// ---------------------------------------------------------------- chain

// The recurrence.  A block owns 16 NV value columns of one head of one
// sequence; a group of WK = DK / 32 warps owns 16 of them, and warp w of the
// group the 32 x 16 block of S^T for key columns 32 w ..: its accumulators,
// which are also its A operands.  Per chunk the group exchanges three small
// results through shared memory: the partial sums of S^T K^T (over the warps'
// key columns), X^T and U^T, the latter two already split by the warp that
// wrote them; token tiles of 8 are dealt so that the triangular products are
// equal shares.  What the next chunk does not wait for is done by helper warps
// beside the groups: they keep two stages of chunk operands filled, and form
// the outputs from S and U as the groups leave them in shared memory (with the
// outputs in the groups themselves a chunk took 4.0 us).  The groups do not wait
// for each other, so one's exchanges run beside the other's products.  A chunk of
// 128 x 128 heads takes 3.3 us (bfloat16), bound by shared memory (78% of its rate) and
// the latency from one product to the next; 32768 tokens x 32 heads 1.65 ms.
template <typename T, int DK>
struct ChainCfg {
    static constexpr int WK = DK / 32;
    static constexpr int NV = DK == 32 ? 4 : 2;
    static constexpr int NC = 32 * WK * NV;  // threads of the groups
    static constexpr int NTILE = 8 / WK;
    static constexpr int COLS = 16 * NV;  // delta_chain_blocks
    static constexpr int LD = tile_ld<T>(DK), LDV = tile_ld<T>(COLS);
    // two stages of the chunk's operands where they fit
    static constexpr int STAGES = sizeof(T) == 2 || DK == 64 ? 2 : 1;
    // bfloat16 outputs come from two bfloat16 parts of S and from U and P in tf32:
    // a quarter of their own rounding.  float16's would be as large as that rounding.
    static constexpr bool HALF = std::is_same<T, bf16>::value;
};
template <bool OUT>
constexpr int helpers() { return OUT ? 4 : 1; }

template <typename T, int DK>
struct ChainStage {
    T k[kChunk * tile_ld<T>(DK)];
    T q[kChunk * tile_ld<T>(DK)];
    T v[kChunk * tile_ld<T>(ChainCfg<T, DK>::COLS)];
    float tp[kSquare];
    float vec[kVec];
};

template <typename T, int DK>
struct ChainSmem {
    using C = ChainCfg<T, DK>;
    ChainStage<T, DK> st[C::STAGES];
    float part[C::NV][C::WK][16 * kLdT];
    float4 x[C::NV][16 * kLdPair];            // X^T
    float4 u[C::NV][16 * kLdPair];            // (e U)^T
    float2 un[C::NV][16 * kLdPair];           // U^T, for P U
    uint4 s[C::NV][C::WK][4][32];             // S^T, for Q S, as the lanes hold it
    T out[helpers<true>()][2][8 * 16];        // two tiles of outputs a helper
    uint64_t full[C::STAGES], empty[C::STAGES];
    uint64_t sfull[C::NV], sempty[C::NV], ufull[C::NV], uempty[C::NV];
    uint32_t bad[C::NV][4];                   // a warp's part of U^T is not finite
    int abort_word;
};

// Element (v, token) of U^T as the groups leave it for the outputs.
struct PlainAt {
    const float2 *u;
    __device__ __forceinline__ float operator()(int v, int j) const {
        const float2 p = u[v * kLdPair + j / 2];
        return j & 1 ? p.y : p.x;
    }
};

// U as P U takes it.
template <bool HALF>
__device__ __forceinline__ float2 out_pair(float a, float b) {
    return HALF ? make_float2(__uint_as_float(tf32(a)), __uint_as_float(tf32(b))) : make_float2(a, b);
}

// A warp's block of S^T for the outputs, four words of four registers a lane:
// bfloat16, two parts of each k step of 16; else the float32 values.
template <typename T>
__device__ __forceinline__ void put_parts(uint4 (*dst)[32], const StateSplit<T> &s, const float (&S)[4][4], int lane) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if constexpr (std::is_same<T, bf16>::value) {
            const uint32_t(&r)[4] = s.a[i >> 1].p[i & 1];
            dst[i][lane] = make_uint4(r[0], r[1], r[2], r[3]);
        } else {
            *reinterpret_cast<float4 *>(&dst[i][lane]) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
        }
    }
}

// acc[i] += S^T Q^T at token tiles n[i] over one warp's 32 key columns
template <typename T, int LD>
__device__ __forceinline__ void parts_times_rows(const uint4 (*src)[32], const T *q, const int (&n)[2], int d0, int lane,
                                                 Acc (&acc)[2]) {
    uint4 parts[4];
#pragma unroll
    for (int i = 0; i < 4; i++) parts[i] = src[i][lane];
    if constexpr (std::is_same<T, bf16>::value) {
        uint32_t b[2][4];
#pragma unroll
        for (int i = 0; i < 2; i++) ldmatrix4(b[i], q + (n[i] * 8 + (lane & 7)) * LD + d0 + 8 * (lane >> 3));
#pragma unroll
        for (int j = 3; j >= 0; j--) {  // part j & 1 of k step j >> 1
            const uint32_t a[4] = {parts[j].x, parts[j].y, parts[j].z, parts[j].w};
#pragma unroll
            for (int i = 0; i < 2; i++) mma16(j & 1 ? acc[i].l : acc[i].c, a, b[i][2 * (j >> 1)], b[i][2 * (j >> 1) + 1]);
        }
    } else {
        float2 b[2][4];
#pragma unroll
        for (int i = 0; i < 2; i++) frag4<T, LD, false>(q, n[i] * 8, d0, b[i]);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            SplitA a;
            a.set(__uint_as_float(parts[j].x), __uint_as_float(parts[j].y), __uint_as_float(parts[j].z), __uint_as_float(parts[j].w));
#pragma unroll
            for (int i = 0; i < 2; i++) mma_split<false, sizeof(T) == 2>(acc[i], a, b[i][j]);
        }
    }
}

template <typename T, int DK, bool OUT>
__global__ void __launch_bounds__(ChainCfg<T, DK>::NC + 32 * helpers<OUT>(), 1)
k_delta_chain(const DeltaGeom geo, const DeltaTerms terms, const float *__restrict__ s0, T *__restrict__ o,
              int64_t ldo, float *__restrict__ sn, float *__restrict__ states, float *__restrict__ us, int veco,
              unsigned *__restrict__ status) {
    using C = ChainCfg<T, DK>;
    constexpr int WK = C::WK, NV = C::NV, LD = C::LD, LDV = C::LDV, NTILE = C::NTILE, NH = helpers<OUT>();
    constexpr bool HALF = C::HALF;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    ChainSmem<T, DK> &sm = *reinterpret_cast<ChainSmem<T, DK> *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int si = blockIdx.x / geo.hv, hv = blockIdx.x - si * geo.hv, hk = hv / (geo.hv / geo.hk);
    const int vb = (int)blockIdx.y * C::COLS;
    after_previous();
    may_start_next();
    const int c0 = geo.first[si], c1 = geo.first[si + 1];

    if (tid == 0) {
        sm.abort_word = 0;
        for (int i = 0; i < C::STAGES; i++) {
            bar_init(&sm.full[i], 32 * NH + 1);  // the helpers' lanes, and the bulk copies
            bar_init(&sm.empty[i], C::NC / 32 + (OUT ? NH : 0));
        }
        for (int i = 0; i < NV; i++) {
            bar_init(&sm.sfull[i], WK);
            bar_init(&sm.sempty[i], NH);
            bar_init(&sm.ufull[i], WK);
            bar_init(&sm.uempty[i], NH);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    auto wait = [&](uint64_t *bar, int parity) { return bar_wait(bar, parity & 1, &sm.abort_word, status); };

    if (warp >= C::NC / 32) {
        // ------------------------------------------------ helpers
        const int hw = warp - C::NC / 32;
        const T *kp = (const T *)geo.k + (int64_t)hk * geo.dkp, *qp = (const T *)geo.q + (int64_t)hk * geo.dkp;
        const T *vp = (const T *)geo.v + (int64_t)hv * geo.dvp + vb;
        const int vcols = min(C::COLS, geo.dvp - vb), count = c1 - c0;
        int fetched = 0;
        auto fetch = [&]() {
            const int it = fetched++, stage = it % C::STAGES;
            if (!wait(&sm.empty[stage], it / C::STAGES + 1)) return;  // an early return: nothing more is fetched
            const int2 ch = geo.chunk[c0 + it];
            ChainStage<T, DK> &s = sm.st[stage];
            const int64_t slot = (int64_t)(c0 + it) * geo.hv + hv;
            uint64_t *bar = &sm.full[stage];
            warp_tile<T, DK, NH>(s.k, kp + (int64_t)ch.x * geo.ldk, geo.ldk, ch.y, geo.dkp, hw);
            if (OUT) warp_tile<T, DK, NH>(s.q, qp + (int64_t)ch.x * geo.ldq, geo.ldq, ch.y, geo.dkp, hw);
            warp_tile<T, C::COLS, NH>(s.v, vp + (int64_t)ch.x * geo.ldv, geo.ldv, ch.y, vcols, hw);
            cp_arrive(bar);
            if (hw == 0 && lane == 0) {
                bar_expect(bar, (kSquare + kVec) * 4);
                bulk_load(s.tp, terms.tp + slot * kSquare, kSquare * 4, bar);
                bulk_load(s.vec, terms.vec + slot * kVec, kVec * 4, bar);
            }
        };
        if (C::STAGES > 1 && count > 0) fetch();
        for (int it = 0; it < count && !*(volatile int *)&sm.abort_word; it++) {
            if (fetched < count) fetch();
            if (!OUT) continue;
            const int stage = it % C::STAGES;
            ChainStage<T, DK> &st = sm.st[stage];
            const int2 ch = geo.chunk[c0 + it];
            wait(&sm.full[stage], it / C::STAGES);
            // S^T Q^T at this helper's two token tiles
            Acc qs[NV][2];
#pragma unroll
            for (int grp = 0; grp < NV; grp++) {
                qs[grp][0].zero(), qs[grp][1].zero();
                wait(&sm.sfull[grp], it);
                const int n[2] = {tile_of<4>(hw, 0), tile_of<4>(hw, 1)};
#pragma unroll
                for (int w = 0; w < WK; w++) parts_times_rows<T, LD>(sm.s[grp][w], st.q, n, 32 * w, lane, qs[grp]);
                __syncwarp();
                if (lane == 0) bar_arrive(&sm.sempty[grp]);
            }
            // O^T = scale c (Q S)^T + U^T P^T
#pragma unroll
            for (int grp = 0; grp < NV; grp++) {
                wait(&sm.ufull[grp], it);
                float oa[2][4];
                triangular<4, true, false, HALF>(
                    hw, oa,
                    [&](int k, SplitA &a) {
                        const float2 y = sm.un[grp][g * kLdPair + k * 4 + t], z = sm.un[grp][(g + 8) * kLdPair + k * 4 + t];
                        if (HALF)
                            a.hi[0] = __float_as_uint(y.x), a.hi[1] = __float_as_uint(z.x), a.hi[2] = __float_as_uint(y.y), a.hi[3] = __float_as_uint(z.y);
                        else
                            a.set(y.x, y.y, z.x, z.y);
                    },
                    [&](int k, int n) { return frag_p_earlier(st.tp, k, n); });
                uint32_t bad = 0;
#pragma unroll
                for (int w = 0; w < WK; w++) bad |= sm.bad[grp][w];
                if (bad && not_finite(oa)) {
#pragma unroll
                    for (int i = 0; i < 2; i++)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (!isfinite(oa[i][e]))
                                oa[i][e] = row_again<true>(PlainAt{sm.un[grp]}, st.tp, g + (e >> 1) * 8,
                                                           tile_of<4>(hw, i) * 8 + 2 * t + (e & 1));
                }
                __syncwarp();
                if (lane == 0) bar_arrive(&sm.uempty[grp]);
                const int v0 = vb + grp * 16;
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int n = tile_of<4>(hw, i) * 8;
                    const float2 cv = *reinterpret_cast<const float2 *>(st.vec + n + 2 * t);
                    const float ca = geo.scale * cv.x, cb = geo.scale * cv.y;
                    const Acc &q = qs[grp][i];
                    const float r[4] = {fmaf(ca, q.get(0), oa[i][0]), fmaf(cb, q.get(1), oa[i][1]),
                                        fmaf(ca, q.get(2), oa[i][2]), fmaf(cb, q.get(3), oa[i][3])};
#pragma unroll
                    for (int e = 0; e < 4; e++) sm.out[hw][i][(2 * t + (e & 1)) * 16 + g + (e >> 1) * 8] = from_f32<T>(r[e]);
                }
                __syncwarp();
                T *op = o + (int64_t)hv * geo.dv + v0;
                if (veco) {  // 16 bytes a lane: rows of 16 values
                    constexpr int PIECE = 16 / (int)sizeof(T), PPR = 16 / PIECE;
#pragma unroll
                    for (int j = lane; j < 2 * 8 * PPR; j += 32) {
                        const int i = j / (8 * PPR), r = j / PPR % 8, c = j % PPR * PIECE, tok = tile_of<4>(hw, i) * 8 + r;
                        if (tok < ch.y && v0 + c < geo.dv)
                            *reinterpret_cast<uint4 *>(op + (int64_t)(ch.x + tok) * ldo + c) =
                                *reinterpret_cast<const uint4 *>(&sm.out[hw][i][r * 16 + c]);
                    }
                } else {
                    for (int j = lane; j < 2 * 8 * 16; j += 32) {
                        const int i = j / 128, r = j / 16 % 8, c = j % 16, tok = tile_of<4>(hw, i) * 8 + r;
                        if (tok < ch.y && v0 + c < geo.dv) op[(int64_t)(ch.x + tok) * ldo + c] = sm.out[hw][i][r * 16 + c];
                    }
                }
                __syncwarp();
            }
            if (lane == 0) bar_arrive(&sm.empty[stage]);
        }
        bar_drain(sm.full, C::STAGES, fetched);  // copies in flight end before the block does
        return;
    }

    // ---------------------------------------------------- the groups
    const int grp = warp / WK, w = warp - grp * WK;
    const int v0 = vb + grp * 16;  // the group's value columns
    const int d0 = w * 32;         // the warp's key columns
    const int64_t state_at = ((int64_t)si * geo.hv + hv) * geo.dk * geo.dv;

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

    for (int c = c0; c < c1; c++) {
        const int it = c - c0, stage = it % C::STAGES;
        StateSplit<T> a;
        a.set(S);
        if (OUT) {
            wait(&sm.sempty[grp], it + 1);
            put_parts<T>(sm.s[grp][w], a, S, lane);
            __syncwarp();
            if (lane == 0) bar_arrive(&sm.sfull[grp]);
        }
        wait(&sm.full[stage], it / C::STAGES);
        ChainStage<T, DK> &st = sm.st[stage];
        const int64_t slot = (int64_t)c * geo.hv + hv;
        if (!OUT) put_state(states + slot * geo.dk * geo.dv);
        group_sync<WK>(grp);  // the group is done with the previous chunk's exchanges

        // partial S^T K^T over the warp's key columns
        {
            float *part = sm.part[grp][w];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                float r[4][4];
                state_times_rows<T, LD>(a, st.k, 4 * h, d0, r);
#pragma unroll
                for (int n = 0; n < 4; n++) {
                    float *p = part + g * kLdT + (4 * h + n) * 8 + 2 * t;
                    *reinterpret_cast<float2 *>(p) = make_float2(r[n][0], r[n][1]);
                    *reinterpret_cast<float2 *>(p + 8 * kLdT) = make_float2(r[n][2], r[n][3]);
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
            const float2 cv = *reinterpret_cast<const float2 *>(st.vec + n);
            const float2 bv = *reinterpret_cast<const float2 *>(st.vec + 2 * kChunk + n);
            float2 va, vb8;
            frag2_col<T, LDV>(st.v, n - 2 * t, grp * 16, va, vb8);
            float4 *x = sm.x[grp] + g * kLdPair + n / 2;
            x[0] = split_pair(bv.x * (va.x - cv.x * lo.x), bv.y * (va.y - cv.y * lo.y));
            x[8 * kLdPair] = split_pair(bv.x * (vb8.x - cv.x * hi.x), bv.y * (vb8.y - cv.y * hi.y));
        }
        group_sync<WK>(grp);
        // U^T = X^T T^T at the warp's token tiles
        {
            float u[NTILE][4];
            triangular<WK, true, false, false>(
                w, u, [&](int k, SplitA &f) { f.set(sm.x[grp][g * kLdPair + k * 4 + t], sm.x[grp][(g + 8) * kLdPair + k * 4 + t]); },
                [&](int k, int n) { return frag_t_earlier(st.tp, k, n); });
            if (OUT) wait(&sm.uempty[grp], it + 1);
#pragma unroll
            for (int i = 0; i < NTILE; i++) {
                const int n = tile_of<WK>(w, i) * 8 + 2 * t, at = g * kLdPair + n / 2;
                const float2 ev = *reinterpret_cast<const float2 *>(st.vec + kChunk + n);
                const float(&v)[4] = u[i];
                put_pair<T>(sm.u[grp] + at, ev.x * v[0], ev.y * v[1]);
                put_pair<T>(sm.u[grp] + at + 8 * kLdPair, ev.x * v[2], ev.y * v[3]);
                if (OUT) {
                    sm.un[grp][at] = out_pair<HALF>(v[0], v[1]);
                    sm.un[grp][at + 8 * kLdPair] = out_pair<HALF>(v[2], v[3]);
                }
                if (!OUT) {
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int vc = v0 + g + (e >> 1) * 8;
                        if (vc < geo.dv) us[(slot * kChunk + n + (e & 1)) * geo.dv + vc] = v[e];
                    }
                }
            }
            // What an infinity or NaN of a later token made NaN is put right, one value at
            // a time and from memory: from the registers and unrolled, this branch that is
            // hardly ever taken took 10% of the loop (2230 us instead of 2003 at 32768
            // tokens x 32 heads).  S' needs no repair: its value column is not finite
            // either way.
            const bool bad = not_finite(u);
            if (bad) {
#pragma unroll 1
                for (int b = 0; b < 4 * NTILE; b++) {
                    const int r = g + (b & 2) * 4, n = tile_of<WK>(w, b >> 2) * 8 + 2 * t + (b & 1);
                    float *p = OUT ? reinterpret_cast<float *>(sm.un[grp]) + r * 2 * kLdPair + n
                                   : us + (slot * kChunk + n) * geo.dv + v0 + r;
                    if ((OUT || v0 + r < geo.dv) && !isfinite(*p)) {
                        const float v = row_again<false>(PairAt{sm.x[grp]}, st.tp, r, n);
                        *p = OUT ? out_pair<HALF>(v, v).x : v;
                    }
                }
            }
            if (OUT) {
                if (lane == 0) sm.bad[grp][w] = bad;
                __syncwarp();
                if (lane == 0) bar_arrive(&sm.ufull[grp]);
            }
        }
        group_sync<WK>(grp);
        // S'^T = c_64 S^T + (e U)^T K: the chunk's sum starts from zero, so that
        // the state is rounded once a chunk
        {
            float r[4][4];
            tokens_product<T, LD>(sm.u[grp], st.k, d0, r);
            const float cend = st.vec[kChunk - 1];
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) S[j][e] = fmaf(cend, S[j][e], r[j][e]);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&sm.empty[stage]);
    }
    if (sn) put_state(sn + state_at);
}

template <typename T, int DK>
cudaError_t terms_dk(const DeltaGeom &g, const DeltaTerms &t, void *o, int64_t ldo, bool next, cudaStream_t st) {
    const size_t smem = sizeof(TermSmem<T, DK>);
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_delta_terms<T, DK>, (int)sizeof(TermSmem<T, DK>));
    if (attr != cudaSuccess) return attr;
    return launch(next, k_delta_terms<T, DK>, dim3(g.nchunks, g.hk), kTermThreads, smem, st, g, t, (T *)o, ldo);
}

template <typename T, int DK>
cudaError_t chain_dk(const DeltaGeom &g, const DeltaTerms &t, const float *s0, void *o, int64_t ldo, float *sn,
                     float *states, float *us, unsigned *status, bool next, cudaStream_t st) {
    using C = ChainCfg<T, DK>;
    static_assert(sizeof(ChainSmem<T, DK>) <= 232448, "shared memory of a block");
    const size_t smem = sizeof(ChainSmem<T, DK>);
    const dim3 grid((unsigned)(g.nseq * g.hv), (unsigned)((g.dv + 16 * C::NV - 1) / (16 * C::NV)));
    if (o) {
        static OncePerDevice limit;
        const cudaError_t attr = smem_limit(limit, k_delta_chain<T, DK, true>, (int)sizeof(ChainSmem<T, DK>));
        if (attr != cudaSuccess) return attr;
        return launch(next, k_delta_chain<T, DK, true>, grid, C::NC + 32 * helpers<true>(), smem, st, g, t, s0, (T *)o, ldo, sn,
                      states, us, (int)mult16(o, ldo, g.dv, sizeof(T)), status);
    } else {
        static OncePerDevice limit;
        const cudaError_t attr = smem_limit(limit, k_delta_chain<T, DK, false>, (int)sizeof(ChainSmem<T, DK>));
        if (attr != cudaSuccess) return attr;
        return launch(next, k_delta_chain<T, DK, false>, grid, C::NC + 32 * helpers<false>(), smem, st, g, t, s0, (T *)nullptr,
                      (int64_t)0, sn, states, us, 0, status);
    }
}

}  // namespace

cudaError_t zs_launch_delta_plan(const int64_t *offsets, int nseq, int64_t tokens, int len, int nchunks, int *first, int2 *seq,
                                 int2 *chunk, cudaStream_t st, int64_t *launches) {
    k_delta_plan<<<1, 1024, 0, st>>>(offsets, nseq, tokens, len, nchunks, first, seq, chunk);
    ++*launches;
    return cudaGetLastError();
}

cudaError_t zs_launch_delta_pack(int type, const void *src, int64_t ld, int64_t tokens, int heads, int d, int dp,
                                 void *dst, int num_sms, cudaStream_t st, int64_t *launches) {
    ++*launches;
    const int64_t n = tokens * heads * dp;
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, (int64_t)num_sms * 8);
    if (type == ZSOLVE_F32)
        k_delta_pack<<<blocks, 256, 0, st>>>((const float *)src, ld, tokens, heads, d, dp, (float *)dst);
    else  // a copy: both 16-bit types alike
        k_delta_pack<<<blocks, 256, 0, st>>>((const bf16 *)src, ld, tokens, heads, d, dp, (bf16 *)dst);
    return cudaGetLastError();
}

cudaError_t zs_launch_delta_terms(int type, const DeltaGeom &g, const DeltaTerms &t, void *o, int64_t ldo, bool next,
                                  cudaStream_t st, int64_t *launches) {
    ++*launches;
    return DELTA_TYPE(terms_dk, g, t, o, ldo, next, st);
}

cudaError_t zs_launch_delta_chain(int type, const DeltaGeom &g, const DeltaTerms &t, const float *s0, void *o,
                                  int64_t ldo, float *sn, float *states, float *us, unsigned *status, bool next,
                                  cudaStream_t st, int64_t *launches) {
    ++*launches;
    return DELTA_TYPE(chain_dk, g, t, s0, o, ldo, sn, states, us, status, next, st);
}
