// The gated delta rule's shared parts: geometry of the chunks, the float32-class
// products on the tensor cores, operand fragments in shared memory.
//
// Per value head, with the state S (dk x dv), a_t = exp g_t and
//   S_t = a_t S_{t-1} + k_t u_t^T,  u_t = beta_t (v_t - a_t S_{t-1}^T k_t),  o_t = scale S_t^T q_t,
// a chunk of 64 tokens with b_i = g_1 + ... + g_i, c_i = exp b_i, e_ij = exp(b_i - b_j) is
//   A_ij = beta_i (k_i . k_j) e_ij (j < i),  T = (I + A)^-1,  X = beta (V - c K S),  U = T X,
//   O = scale (c Q S) + P U,  P_ij = scale (q_i . k_j) e_ij (j <= i),
//   S' = c_64 S + (e_64,j K)^T U
// : a unit lower-triangular solve and a rank-64 update, the two steps of the
// blocked factorisation.
//
// States, U and gradients of the gates are float32 results, so every product
// that feeds them keeps float32 accuracy on the tensor cores: an operand that
// is not exact in tf32 (float32 inputs, S, T, U, X) is split into a tf32 hi
// part and a tf32 lo part; the product is hi.hi + hi.lo + lo.hi, and
// hi.exact + lo.exact where the other operand is a bfloat16 or float16 input
// (exact in tf32).  The lo.lo term is below float32 rounding.  The
// instructions are mma.sync m16n8k8: a chunk's matrices are 64 wide and each
// step waits for the one before, so what counts is the latency from one
// product to the next, and register operands hand results on without a trip
// through TMEM (S^T, kept as the accumulator of S'^T = ... + U^T K, is the
// next chunk's A operand as it stands).
#pragma once

#include <type_traits>

#include "seq.cuh"

namespace zs {

constexpr int kChunk = 64;  // tokens of a chunk

// Inputs of a call and the chunk table.
struct DeltaGeom {
    const void *q, *k, *v;         // tokens x heads x d, token strides ld*
    int64_t ldq, ldk, ldv;
    int dkp, dvp;                  // dk, dv in whole 16 bytes: distance of two heads in the chunked form
                                   // (there q, k, v are aligned, or packed copies padded with zeros)
    const float *g, *beta;         // tokens x hv
    int hk, hv, dk, dv, nseq;
    int64_t tokens;
    float scale;
    const int *first;              // nseq + 1: first chunk of each sequence
    const int2 *seq;               // nseq: first token and length
    const int2 *chunk;             // per chunk: first token, tokens (1..64); 0 tokens: unused
    int nchunks;                   // room in the tables
};

// Per chunk and value head, what does not depend on the state (float32): T and P
// in one matrix of 64 rows of stride 72, T strictly below the diagonal (its
// diagonal is 1) and P transposed on and above it; and the vectors c_i, e_64,i,
// beta_i and b_i in two floats (64 each).
struct DeltaTerms {
    float *tp, *vec;
};
constexpr int kVec = 5 * kChunk;

// ---------------------------------------------------------------- products

__device__ __forceinline__ uint32_t tf32(float x) {
    uint32_t r;
    asm("cvt.rn.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void mma8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c = A B of one step, from zero
__device__ __forceinline__ void mma8_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// An A operand of 16 x 8 in two tf32 parts.  The instruction's k slots t and
// t + 4 hold the columns 2t and 2t + 1 (any order serves as long as A and B
// agree): the accumulator's columns, so an accumulator is an A operand, and a
// pair of neighbours in memory.
struct SplitA {
    uint32_t hi[4], lo[4];
    // c: (g, 2t), (g, 2t+1), (g+8, 2t), (g+8, 2t+1)
    __device__ __forceinline__ void set(float c0, float c1, float c2, float c3) {
        const float x[4] = {c0, c2, c1, c3};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            hi[i] = tf32(x[i]);
            lo[i] = tf32(x[i] - __uint_as_float(hi[i]));
        }
    }
    __device__ __forceinline__ void set(const float (&c)[4]) { set(c[0], c[1], c[2], c[3]); }
    // two rows of pairs as Pair keeps them
    __device__ __forceinline__ void set(float4 y, float4 z) {
        hi[0] = __float_as_uint(y.x), hi[2] = __float_as_uint(y.y), lo[0] = __float_as_uint(y.z), lo[2] = __float_as_uint(y.w);
        hi[1] = __float_as_uint(z.x), hi[3] = __float_as_uint(z.y), lo[1] = __float_as_uint(z.z), lo[3] = __float_as_uint(z.w);
    }
};

// Two neighbours split for later use as an A operand: (hi, hi, lo, lo).
__device__ __forceinline__ float4 split_pair(float a, float b) {
    const float ha = __uint_as_float(tf32(a)), hb = __uint_as_float(tf32(b));
    return make_float4(ha, hb, __uint_as_float(tf32(a - ha)), __uint_as_float(tf32(b - hb)));
}

// A product in two sums, c of the hi.hi terms and l of the small ones: the
// tensor cores round their sums toward zero, and apart the small terms do not
// add to how often c is rounded.
struct Acc {
    float c[4], l[4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < 4; e++) c[e] = l[e] = 0.f;
    }
    __device__ __forceinline__ float get(int e) const { return c[e] + l[e]; }
};

// acc += A B for one 16 x 8 x 8 step, b = (B(2t, g), B(2t+1, g)).  B_EXACT or
// A_EXACT: that operand is exact in tf32.
template <bool A_EXACT, bool B_EXACT>
__device__ __forceinline__ void mma_split(Acc &acc, const SplitA &a, float2 b) {
    uint32_t b0 = __float_as_uint(b.x), b1 = __float_as_uint(b.y);
    if (!B_EXACT) {
        b0 = tf32(b.x), b1 = tf32(b.y);
        mma8(acc.l, a.hi, tf32(b.x - __uint_as_float(b0)), tf32(b.y - __uint_as_float(b1)));
    }
    if (!A_EXACT) mma8(acc.l, a.lo, b0, b1);
    mma8(acc.c, a.hi, b0, b1);
}

__device__ __forceinline__ void add_to(float (&c)[4], const float (&d)[4]) {
    const float2 x = add2(make_float2(c[0], c[1]), make_float2(d[0], d[1]));
    const float2 y = add2(make_float2(c[2], c[3]), make_float2(d[2], d[3]));
    c[0] = x.x, c[1] = x.y, c[2] = y.x, c[3] = y.y;
}

// The same into one float32 sum that is rounded to nearest: the step's terms
// start from zero.
template <bool A_EXACT, bool B_EXACT>
__device__ __forceinline__ void mma_add(float (&c)[4], const SplitA &a, float2 b) {
    float d[4];
    uint32_t b0 = __float_as_uint(b.x), b1 = __float_as_uint(b.y);
    if (!B_EXACT) {
        b0 = tf32(b.x), b1 = tf32(b.y);
        mma8_first(d, a.hi, tf32(b.x - __uint_as_float(b0)), tf32(b.y - __uint_as_float(b1)));
        if (!A_EXACT) mma8(d, a.lo, b0, b1);
        mma8(d, a.hi, b0, b1);
    } else if (!A_EXACT) {
        mma8_first(d, a.lo, b0, b1);
        mma8(d, a.hi, b0, b1);
    } else {
        mma8_first(d, a.hi, b0, b1);
    }
    add_to(c, d);
}

// bfloat16 inputs: a float32 operand in three bfloat16 parts (24 bits), so that
// the other, exact operand needs no conversion and a step covers 16 k:
// m16n8k16, three products for the tf32 form's four.
struct Split3 {
    uint32_t p[3][4];
    // the accumulators of two neighbouring tiles of 8 columns
    __device__ __forceinline__ void set(const float (&c)[4], const float (&d)[4]) {
        split(c[0], c[1], 0), split(c[2], c[3], 1), split(d[0], d[1], 2), split(d[2], d[3], 3);
    }
    // as split3_pair left them: rows g and g + 8, pairs t and t + 4 of the tile
    __device__ __forceinline__ void set(uint4 a, uint4 b, uint4 c, uint4 d) {
        p[0][0] = a.x, p[1][0] = a.y, p[2][0] = a.z;
        p[0][1] = b.x, p[1][1] = b.y, p[2][1] = b.z;
        p[0][2] = c.x, p[1][2] = c.y, p[2][2] = c.z;
        p[0][3] = d.x, p[1][3] = d.y, p[2][3] = d.z;
    }
    static __device__ __forceinline__ uint32_t part(float &x, float &y) {
        const uint32_t u = pack2<bf16>(x, y);
        const float2 f = unpack2<bf16>(u);
        x -= f.x;
        y -= f.y;
        return u;
    }
    __device__ __forceinline__ void split(float x, float y, int i) {
        p[0][i] = part(x, y);
        p[1][i] = part(x, y);
        p[2][i] = pack2<bf16>(x, y);
    }
};

__device__ __forceinline__ uint4 split3_pair(float x, float y) {
    uint4 u;
    u.x = Split3::part(x, y);
    u.y = Split3::part(x, y);
    u.z = pack2<bf16>(x, y);
    u.w = 0u;
    return u;
}

__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// ---------------------------------------------------------------- fragments

__device__ __forceinline__ void ldmatrix4(uint32_t (&u)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                 : "r"((uint32_t)__cvta_generic_to_shared(p))
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&u)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                 : "r"((uint32_t)__cvta_generic_to_shared(p))
                 : "memory");
}

// Row stride (values) of a tile of D columns in shared memory: 16 bytes more
// for 16-bit values, 32 for float32, so that the eight rows of a fragment lie
// in different banks.
template <typename T>
__host__ __device__ constexpr int tile_ld(int d) {
    return d + 8;
}

// Four fragments of 8 x 8 from a tile X of row stride LD.
//   row: f[i] = (X(r0 + g, c0 + 8 i + 2t), X(r0 + g, c0 + 8 i + 2t + 1))
//   col: f[i] = (X(r0 + 2t, c0 + 8 i + g), X(r0 + 2t + 1, c0 + 8 i + g))
template <typename T, int LD, bool COL>
__device__ __forceinline__ void frag4(const T *x, int r0, int c0, float2 (&f)[4]) {
    const int lane = threadIdx.x & 31;
    if constexpr (sizeof(T) == 2) {
        const T *p = x + (r0 + (lane & 7)) * LD + c0 + 8 * (lane >> 3);
        uint32_t u[4];
        if (COL)
            ldmatrix4_trans(u, p);
        else
            ldmatrix4(u, p);
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = unpack2<T>(u[i]);
    } else {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (COL)
                f[i] = make_float2(x[(r0 + 2 * t) * LD + c0 + 8 * i + g], x[(r0 + 2 * t + 1) * LD + c0 + 8 * i + g]);
            else
                f[i] = *reinterpret_cast<const float2 *>(x + (r0 + g) * LD + c0 + 8 * i + 2 * t);
        }
    }
}

// (X(r0 + 2t, c0 + g), X(r0 + 2t + 1, c0 + g)) and the same eight columns on
template <typename T, int LD>
__device__ __forceinline__ void frag2_col(const T *x, int r0, int c0, float2 &f0, float2 &f1) {
    const int lane = threadIdx.x & 31;
    if constexpr (sizeof(T) == 2) {
        const uint32_t a = (uint32_t)__cvta_generic_to_shared(x + (r0 + (lane & 7)) * LD + c0 + 8 * ((lane >> 3) & 1));
        uint32_t u0, u1;
        asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(u0), "=r"(u1) : "r"(a) : "memory");
        f0 = unpack2<T>(u0);
        f1 = unpack2<T>(u1);
    } else {
        const T *p = x + (r0 + 2 * (lane & 3)) * LD + c0 + (lane >> 2);
        f0 = make_float2(p[0], p[LD]);
        f1 = make_float2(p[8], p[LD + 8]);
    }
}

// A 16 x 32 block of a state's transpose, as accumulators, split for the
// products with K and Q.
template <typename T>
struct StateSplit {
    SplitA a[4];
    __device__ __forceinline__ void set(const float (&s)[4][4]) {
#pragma unroll
        for (int j = 0; j < 4; j++) a[j].set(s[j]);
    }
};
template <>
struct StateSplit<bf16> {
    Split3 a[2];
    __device__ __forceinline__ void set(const float (&s)[4][4]) {
        a[0].set(s[0], s[1]);
        a[1].set(s[2], s[3]);
    }
};

// r[n] = S^T X^T at token tiles n0 .. n0 + 3 over key columns d0 .. d0 + 31 of
// the tile X.
template <typename T, int LD>
__device__ __forceinline__ void state_times_rows(const StateSplit<T> &s, const T *x, int n0, int d0, float (&r)[4][4]) {
    if constexpr (std::is_same<T, bf16>::value) {
        const int lane = threadIdx.x & 31;
        uint32_t b[4][4];
#pragma unroll
        for (int n = 0; n < 4; n++) ldmatrix4(b[n], x + ((n0 + n) * 8 + (lane & 7)) * LD + d0 + 8 * (lane >> 3));
        // the small parts first
#pragma unroll
        for (int i = 2; i >= 0; i--)
#pragma unroll
            for (int k = 0; k < 2; k++)
#pragma unroll
                for (int n = 0; n < 4; n++) {
                    if (i == 2 && k == 0)
                        mma16_first(r[n], s.a[k].p[i], b[n][2 * k], b[n][2 * k + 1]);
                    else
                        mma16(r[n], s.a[k].p[i], b[n][2 * k], b[n][2 * k + 1]);
                }
    } else {
        Acc acc[4];
        float2 b[4][4];
#pragma unroll
        for (int n = 0; n < 4; n++) {
            acc[n].zero();
            frag4<T, LD, false>(x, (n0 + n) * 8, d0, b[n]);
        }
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int n = 0; n < 4; n++) mma_split<false, sizeof(T) == 2>(acc[n], s.a[j], b[n][j]);
#pragma unroll
        for (int n = 0; n < 4; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) r[n][e] = acc[n].get(e);
    }
}

// Split pairs in shared memory: rows of 32 pairs of 16 bytes, 64 bytes more
// apart, so that the rows of a fragment's loads lie in different banks.
constexpr int kLdPair = 36;
template <typename T>
__device__ __forceinline__ void put_pair(float4 *p, float a, float b) {
    if constexpr (std::is_same<T, bf16>::value)
        *reinterpret_cast<uint4 *>(p) = split3_pair(a, b);
    else
        *p = split_pair(a, b);
}

// Element (v, token) of split pairs in shared memory.
struct PairAt {
    const float4 *x;
    __device__ __forceinline__ float operator()(int v, int j) const {
        const float *p = reinterpret_cast<const float *>(x + v * kLdPair + j / 2) + (j & 1);
        return p[0] + p[2];
    }
};

// r[j] = Y X over the chunk's 64 tokens: Y 16 x 64 from put_pair, X(tokens, key
// columns d0 + 8 j ..) of the tile, each sum from zero.
template <typename T, int LD>
__device__ __forceinline__ void tokens_product(const float4 *y, const T *x, int d0, float (&r)[4][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if constexpr (std::is_same<T, bf16>::value) {
        const uint4 *u = reinterpret_cast<const uint4 *>(y);
        float small[4][4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int at = g * kLdPair + k * 8 + t;
            Split3 a;
            a.set(u[at], u[at + 8 * kLdPair], u[at + 4], u[at + 8 * kLdPair + 4]);
            uint32_t b[2][4];
#pragma unroll
            for (int j = 0; j < 2; j++)
                ldmatrix4_trans(b[j], x + (k * 16 + (lane & 15)) * LD + d0 + 16 * j + 8 * (lane >> 4));
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t b0 = b[j >> 1][(j & 1) * 2], b1 = b[j >> 1][(j & 1) * 2 + 1];
                if (k == 0) {
                    mma16_first(small[j], a.p[2], b0, b1);
                    mma16_first(r[j], a.p[0], b0, b1);
                } else {
                    mma16(small[j], a.p[2], b0, b1);
                    mma16(r[j], a.p[0], b0, b1);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; j++) mma16(small[j], a.p[1], b[j >> 1][(j & 1) * 2], b[j >> 1][(j & 1) * 2 + 1]);
        }
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) r[j][e] += small[j][e];
    } else {
        Acc acc[4];
#pragma unroll
        for (int j = 0; j < 4; j++) acc[j].zero();
#pragma unroll
        for (int k = 0; k < 8; k++) {
            SplitA a;
            a.set(y[g * kLdPair + k * 4 + t], y[(g + 8) * kLdPair + k * 4 + t]);
            float2 b[4];
            frag4<T, LD, true>(x, k * 8, d0, b);
#pragma unroll
            for (int j = 0; j < 4; j++) mma_split<false, sizeof(T) == 2>(acc[j], a, b[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) r[j][e] = acc[j].get(e);
    }
}

// ---------------------------------------------------------------- loads

__device__ __forceinline__ void cp_async16(void *dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// By all NT threads: a tile of 64 rows x D columns from n rows of d values (whole
// 16 bytes) at stride ld; zeros elsewhere.
template <typename T, int D, int NT>
__device__ __forceinline__ void load_tile(T *dst, const T *src, int64_t ld, int n, int d) {
    constexpr int LD = tile_ld<T>(D), VE = 16 / (int)sizeof(T), PER = D / VE;
    for (int i = threadIdx.x; i < kChunk * PER; i += NT) {
        const int r = i / PER, c = (i - r * PER) * VE;
        const bool in = r < n && c < d;
        cp_async16(dst + r * LD + c, src + (in ? r * ld + c : 0), in ? 16 : 0);
    }
}

// Row stride of the matrix that holds T and P, in memory as in shared memory (a
// copy is one bulk copy, and a fragment's rows lie in different banks).
constexpr int kLdT = kChunk + 8;
constexpr int kSquare = kChunk * kLdT;

// B operands from it for the 8 x 8 tile of tokens k (the sum's) and n (the
// result's): T^T and P^T for products that run over earlier tokens (k <= n), T and
// P for those over later ones (k >= n).
__device__ __forceinline__ float2 frag_t_earlier(const float *m, int k, int n) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t2 = 2 * (lane & 3);
    float2 b = *reinterpret_cast<const float2 *>(m + (n * 8 + g) * kLdT + k * 8 + t2);  // T(n g, k t)
    if (k == n) {
        b.x = t2 < g ? b.x : t2 == g ? 1.f : 0.f;
        b.y = t2 + 1 < g ? b.y : t2 + 1 == g ? 1.f : 0.f;
    }
    return b;
}
__device__ __forceinline__ float2 frag_p_earlier(const float *m, int k, int n) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t2 = 2 * (lane & 3);
    const float *p = m + (k * 8 + t2) * kLdT + n * 8 + g;  // P(n g, k t), stored transposed
    float2 b = make_float2(p[0], p[kLdT]);
    if (k == n) {
        if (t2 > g) b.x = 0.f;
        if (t2 + 1 > g) b.y = 0.f;
    }
    return b;
}
__device__ __forceinline__ float2 frag_t_later(const float *m, int k, int n) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t2 = 2 * (lane & 3);
    const float *p = m + (k * 8 + t2) * kLdT + n * 8 + g;  // T(k t, n g)
    float2 b = make_float2(p[0], p[kLdT]);
    if (k == n) {
        b.x = t2 > g ? b.x : t2 == g ? 1.f : 0.f;
        b.y = t2 + 1 > g ? b.y : t2 + 1 == g ? 1.f : 0.f;
    }
    return b;
}
__device__ __forceinline__ float2 frag_p_later(const float *m, int k, int n) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t2 = 2 * (lane & 3);
    float2 b = *reinterpret_cast<const float2 *>(m + (n * 8 + g) * kLdT + k * 8 + t2);  // P(k t, n g), stored transposed
    if (k == n) {
        if (t2 < g) b.x = 0.f;
        if (t2 + 1 < g) b.y = 0.f;
    }
    return b;
}

// NW warps, of which this is warp w: a tile of 64 rows x D columns from n rows of d
// values (whole 16 bytes) at stride ld, by 16-byte copies that write zeros
// elsewhere (a bulk copy a row is issued a lane at a time, and 192 of them took
// longer than a chunk's products).
template <typename T, int D, int NW>
__device__ __forceinline__ void warp_tile(T *dst, const T *src, int64_t ld, int n, int d, int w) {
    constexpr int LD = tile_ld<T>(D), VE = 16 / (int)sizeof(T), PER = D / VE, ROWS = 32 / PER;
    const int lane = threadIdx.x & 31, r = w * (kChunk / NW) + lane / PER, c = (lane % PER) * VE;
    const T *p = src + (int64_t)r * ld + c;
    T *q = dst + r * LD + c;
#pragma unroll 8
    for (int i = 0; i < kChunk / NW; i += ROWS) {
        const bool in = i + r < n && c < d;
        cp_async16(q, in ? p : src, in ? 16 : 0);
        p += ROWS * ld;
        q += ROWS * LD;
    }
}

// Arrive on bar once the calling thread's copies so far are complete.
__device__ __forceinline__ void cp_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"((uint32_t)__cvta_generic_to_shared(bar))
                 : "memory");
}

// One warp: b_i of a chunk's tokens, summed in float64 (a few additions) and
// kept as two floats, so that the differences b_i - b_j keep their digits after
// a strong decay.  exp(-1e4) is 0, and finite sums leave no inf - inf.
__device__ __forceinline__ void gate_sums(const DeltaGeom &geo, int2 ch, int hv, float *bh, float *bl) {
    const int lane = threadIdx.x & 31;
    double x[2];
#pragma unroll
    for (int e = 0; e < 2; e++) {
        const int i = 2 * lane + e;
        float gi = i < ch.y ? geo.g[(int64_t)(ch.x + i) * geo.hv + hv] : 0.f;
        if (gi < -1e4f) gi = -1e4f;
        x[e] = gi;
    }
    double s = x[0] + x[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
    }
    double before = __shfl_up_sync(0xffffffffu, s, 1);
    if (lane == 0) before = 0.0;
    const double b0 = before + x[0], b1 = s;
    bh[2 * lane] = (float)b0, bl[2 * lane] = (float)(b0 - (double)(float)b0);
    bh[2 * lane + 1] = (float)b1, bl[2 * lane + 1] = (float)(b1 - (double)(float)b1);
}

// The tokens that belong to no sequence, before the first and after the last, have outputs
// and gradients that are zero.  The blocks of the chunk table's unused entries, of which
// `chunk` is one, write them (there is one at least where the sequences come from offsets),
// each its share of the tokens: zero(t0, t1, worker, workers), a worker a warp.
template <typename F>
__device__ __forceinline__ void tokens_outside(const DeltaGeom &geo, int chunk, F zero) {
    const int used = geo.first[geo.nseq], warps = blockDim.x >> 5;
    const int worker = (chunk - used) * warps + (threadIdx.x >> 5), workers = (geo.nchunks - used) * warps;
    const int2 last = geo.seq[geo.nseq - 1];
    zero((int64_t)0, (int64_t)geo.seq[0].x, worker, workers);
    zero((int64_t)last.x + last.y, geo.tokens, worker, workers);
}
// Zeros in `cols` values of the tokens t0 .. t1 - 1 at stride ld.
template <typename T>
__device__ __forceinline__ void zero_tokens(T *p, int64_t ld, int64_t t0, int64_t t1, int cols, int worker, int workers) {
    for (int64_t t = t0 + worker; t < t1; t += workers)
        for (int c = threadIdx.x & 31; c < cols; c += 32) p[t * ld + c] = from_f32<T>(0.f);
}

// ---------------------------------------------------------------- chains

// Token tile i (of 8) of warp w of WK: dealt so that triangular work is an
// equal share for every warp.
template <int WK>
__device__ __forceinline__ int tile_of(int w, int i) {
    return (i & 1) ? (i + 1) * WK - 1 - w : i * WK + w;
}

// The triangular products of a warp's pair p of token tiles, n0 < n1, one step of
// 8 x 8 x 8 after the other: as many for every warp of the group, so that the
// steps unroll without a branch and their loads run ahead.  EARLIER: tile n takes
// the tiles k = 0 .. n; else k = n .. 7.
template <int WK, bool EARLIER>
__host__ __device__ constexpr int steps_of(int p) {
    return EARLIER ? (4 * p + 2) * WK + 1 : 17 - (4 * p + 2) * WK;
}
template <int WK, bool EARLIER>
__device__ __forceinline__ void step_of(int w, int p, int s, int &k, int &n, bool &first) {
    const int n0 = tile_of<WK>(w, 2 * p), n1 = tile_of<WK>(w, 2 * p + 1);
    if (EARLIER) {
        first = s <= n0;
        k = first ? s : s - n0 - 1;
    } else {
        first = s < 8 - n0;
        k = first ? n0 + s : n1 + s - (8 - n0);
    }
    n = first ? n0 : n1;
}

// x[2p], x[2p + 1] = the pair's results: sums of steps, each from zero and rounded
// to nearest.  A(k): the step's A operand; B(k, n): its B operand; HALF: the hi
// parts alone.
template <int WK, bool EARLIER, bool A_EXACT, bool HALF, typename FA, typename FB>
__device__ __forceinline__ void triangular(int w, float (&x)[8 / WK][4], FA A, FB B) {
#pragma unroll
    for (int p = 0; p < 4 / WK; p++) {
        float a0[4] = {}, a1[4] = {};
#pragma unroll
        for (int s = 0; s < steps_of<WK, EARLIER>(p); s++) {
            int k, n;
            bool first;
            step_of<WK, EARLIER>(w, p, s, k, n, first);
            SplitA a;
            A(k, a);
            const float2 b = B(k, n);
            const uint32_t b0 = tf32(b.x), b1 = tf32(b.y);
            float d[4];
            if (HALF) {
                mma8_first(d, a.hi, b0, b1);
            } else {
                mma8_first(d, a.hi, tf32(b.x - __uint_as_float(b0)), tf32(b.y - __uint_as_float(b1)));
                if (!A_EXACT) mma8(d, a.lo, b0, b1);
                mma8(d, a.hi, b0, b1);
            }
            if (first) {
#pragma unroll
                for (int e = 0; e < 4; e++) a0[e] += d[e];
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++) a1[e] += d[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; e++) x[2 * p][e] = a0[e], x[2 * p + 1][e] = a1[e];
    }
}

// Whether any of the warp's values is an infinity or NaN.
template <int N>
__device__ __forceinline__ bool not_finite(const float (&x)[N][4]) {
    uint32_t most = 0;
#pragma unroll
    for (int q = 0; q < N; q++)
#pragma unroll
        for (int e = 0; e < 4; e++) most = max(most, __float_as_uint(x[q][e]) & 0x7fffffffu);
    return __any_sync(0xffffffffu, most >= 0x7f800000u);
}

// One value of a triangular product over earlier tokens once more: in a tile on the
// diagonal that holds an infinity or NaN, the zeros above T's and P's diagonal have
// made NaN of it for the tokens before it.  Row v, token i; xa(v, j): the other
// operand; tp as frag_*_earlier reads it, P: of P, else of T.
template <bool P, typename FX>
__device__ __forceinline__ float row_again(FX xa, const float *tp, int v, int i) {
    float sum = P ? 0.f : xa(v, i);
#pragma unroll 1
    for (int j = 0; j < (P ? i + 1 : i); j++) sum = fmaf(xa(v, j), P ? tp[j * kLdT + i] : tp[i * kLdT + j], sum);
    return sum;
}

// The warps of one column group wait for each other.
template <int WK>
__device__ __forceinline__ void group_sync(int group) {
    if (WK == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(WK * 32) : "memory");
}

inline bool mult16(const void *p, int64_t ld, int64_t d, size_t e) {
    return (((uintptr_t)p | (uint64_t)ld * e | (uint64_t)d * e) & 15) == 0;
}

}  // namespace zs

// FN<T, DK>(...) for the call's type and the key columns it needs (`type` and
// `g` in scope)
#define DELTA_DK(T, FN, ...) (g.dk <= 32 ? FN<T, 32>(__VA_ARGS__) : g.dk <= 64 ? FN<T, 64>(__VA_ARGS__) : FN<T, 128>(__VA_ARGS__))
#define DELTA_TYPE(FN, ...)                                                   \
    (type == ZSOLVE_F32    ? DELTA_DK(float, FN, __VA_ARGS__)                 \
     : type == ZSOLVE_BF16 ? DELTA_DK(bf16, FN, __VA_ARGS__)                  \
                           : DELTA_DK(f16, FN, __VA_ARGS__))

// ---------------------------------------------------------------- launchers

// next: the launch before on the stream is of the same call (seq.cuh).

// delta.cu
cudaError_t zs_launch_delta_plan(const int64_t *offsets, int nseq, int64_t tokens, int len, int nchunks, int *first, int2 *seq,
                                 int2 *chunk, cudaStream_t st, int64_t *launches);
// tokens x heads x d values at token stride ld into packed heads of dp values
cudaError_t zs_launch_delta_pack(int type, const void *src, int64_t ld, int64_t tokens, int heads, int d, int dp,
                                 void *dst, int num_sms, cudaStream_t st, int64_t *launches);
// The chunks' terms; and zeros in o (NULL: none) for the tokens outside the sequences.
cudaError_t zs_launch_delta_terms(int type, const zs::DeltaGeom &g, const zs::DeltaTerms &t, void *o, int64_t ldo, bool next,
                                  cudaStream_t st, int64_t *launches);
// The recurrence over the chunks.  o (NULL: not formed), sn (the last states;
// NULL: not written); states, us (NULL: not kept): the state each chunk
// starts from (per chunk and value head dk x dv) and U (64 x dv).  status: a
// word that a bounded wait sets when it gives up.
cudaError_t zs_launch_delta_chain(int type, const zs::DeltaGeom &g, const zs::DeltaTerms &t, const float *s0, void *o,
                                  int64_t ldo, float *sn, float *states, float *us, unsigned *status, bool next,
                                  cudaStream_t st, int64_t *launches);
// The recurrence backwards (delta_bwd.cu): from the gradients of o and of the
// last states (ds; NULL: zero), per chunk and value head the gradient of the
// state after the chunk (dends, dk x dv) and dX (64 x dv), dv, and the
// gradient of the first states (ds0; NULL: not written).
cudaError_t zs_launch_delta_rchain(int type, const zs::DeltaGeom &g, const zs::DeltaTerms &t, const void *dout,
                                   int64_t lddo, const float *ds, float *dends, float *dxs, void *dv, float *ds0,
                                   unsigned *status, bool next, cudaStream_t st, int64_t *launches);
// The blocks of either recurrence.
inline int64_t delta_chain_blocks(const zs::DeltaGeom &g) {
    const int cols = g.dk <= 32 ? 64 : 32;
    return (int64_t)g.nseq * g.hv * ((g.dv + cols - 1) / cols);
}
// The gradients that the chunks give on their own, and zeros in all of them (dv too) for
// the tokens outside the sequences.  parts (tokens x hv x dk
// float32, one for dq and one for dk) are needed where value heads share a key
// head; dq, dk: tokens x hk x dk.
cudaError_t zs_launch_delta_grads(int type, const zs::DeltaGeom &g, const zs::DeltaTerms &t, const void *dout,
                                  int64_t lddo, const float *states, const float *dends, const float *us,
                                  const float *dxs, float *dqp, float *dkp, void *dq, void *dk, void *dv,
                                  float *dg, float *dbeta, int num_sms, bool next, cudaStream_t st, int64_t *launches);
// Token by token (delta_step.cu): every sequence's tokens one after the other.
cudaError_t zs_launch_delta_step(int type, const zs::DeltaGeom &g, const int64_t *offsets, const float *s0, void *o,
                                 int64_t ldo, float *sn, cudaStream_t st, int64_t *launches);
