// Linear attention with a decay for each head: the geometry of its spans, and what its kernels share.
//
// Per value head, with the state S (dk x dv) and a_t = exp g_t,
//   S_t = a_t S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t.
// A span of up to L tokens with b_i = g_1 + ... + g_i:
//   U = sum_j exp(b_L - b_j) k_j v_j^T,  S' = exp(b_L) S + U,
//   o_i = scale (exp(b_i) S^T q_i + sum_{j <= i} exp(b_i - b_j) (q_i . k_j) v_j).
// Backwards, with D the gradient of the state after the span,
//   W = sum_i scale exp(b_i) q_i do_i^T,  D' (of the state before it) = exp(b_L) D + W,
//   dq_i = scale (exp(b_i) S do_i + sum_{j <= i} exp(b_i - b_j) (do_i . v_j) k_j)
//   dk_j = exp(b_L - b_j) D v_j + scale sum_{i >= j} exp(b_i - b_j) (do_i . v_j) q_i
//   dv_j = exp(b_L - b_j) D^T k_j + scale sum_{i >= j} exp(b_i - b_j) (q_i . k_j) do_i
//   dg_t = sum_{i >= t} q_i . dq_i|state + sum_{j < t} k_j . dk_j|state + exp(b_L) <S, D>
//          + sum_{i >= t > j} scale exp(b_i - b_j) (do_i . v_j)(q_i . k_j).
// U and W are one kernel (a weighted sum of outer products), and o, dq, dk and dv another: rows
// x_i against rows y_j, with the scores' products with rows z_j, and a state's share,
//   out_i = f_i M^T x_i + scale sum_j e_ij (x_i . y_j) z_j,
// forwards (j <= i) or backwards (j >= i) in time.  Between the two, the states of all spans are
// an elementwise recurrence over the spans.  So nothing but that recurrence goes token by token or
// span by span, and every span, head and block of rows is on its own.
//
// The terms of dg that cancel (pairs of tokens on the same side of t) are left out of its sums,
// not subtracted from them, but for those of one span.
#pragma once

#include "delta.cuh"

namespace zs {

constexpr int kSpanMost = 512;  // tokens of a span at most; a multiple of 64

struct DecayGeom {
    DeltaGeom d;        // its chunks are the spans; beta is not used
    int64_t ldg;        // tokens' distance in g: hv, or 0 where each head has one
    int span;           // tokens of a span, at most
    float2 *gates;      // per span and head `span` values: b_i / ln 2 in two floats
    float *ends;        // per span and head: exp(b_L)
};

// The state's or the score's rows: a tensor tokens x heads x cols.
struct DecayRows {
    const void *p;
    int64_t ld;
    int cols, dist;     // values of a head, and from one head to the next
    bool key;           // heads are hk
};

// The products of rows (the formulas above): out, tokens x heads x z's columns at token stride ldo.
//   m        per span and value head dk x dv; its rows meet x's columns, or (`turned`) its columns do
//   back     backwards in time
//   self     NULL, or what the gates' gradients need: out's heads are key heads, summed over the value heads that
//            share one; self's rows (tokens x hk x z's columns) times the state's share of out go to sums[0], and the sums
//            over j != i of scale e_ij (x_i . y_j)(self_i . z_j) to sums[1] (tokens x hv each)
struct DecayProduct {
    DecayRows x, y, z;
    const void *m;      // float32 (zs_launch_decay_rows)
    bool turned, back;
    void *out;
    int64_t ldo;
    int heads;
    const DecayRows *self;
    float *sums[2];
};

// exp(b - c) of two sums in two floats each (in units of ln 2).
__device__ __forceinline__ float decay_exp(float2 b, float2 c) { return exp2f((b.x - c.x) + (b.y - c.y)); }

// The sums b_i of a span's tokens into `b`, in units of ln 2 and in two floats, so that their differences keep their digits
// after a strong decay (float64 would do, but its additions are many times slower here).  exp(-1e4) is 0, and finite
// sums leave no inf - inf.  First the log decays by all of the block's `threads` threads (thread t of them), and then, once
// those are there, one warp the sums.
__device__ __forceinline__ void decay_loads(const DecayGeom &geo, int2 sp, int hv, float2 *b, int t, int threads) {
    for (int i = t; i < sp.y; i += threads) {
        float g = geo.d.g[(int64_t)(sp.x + i) * geo.ldg + hv];
        if (g < -1e4f) g = -1e4f;
        // 1 / ln 2 in two floats
        const float hi = g * 1.44269502f;
        b[i] = make_float2(hi, fmaf(g, 1.44269502f, -hi) + g * 1.92596299e-8f);
    }
}
// a + b of two floats each: the large parts' sum and its own rounding error exactly (Knuth), the small parts with it.
__device__ __forceinline__ float2 decay_add(float2 a, float2 b) {
    const float s = a.x + b.x, t = s - a.x, e = (a.x - (s - t)) + (b.x - t) + (a.y + b.y);
    const float hi = s + e;
    return make_float2(hi, e - (hi - s));
}
__device__ __forceinline__ void decay_sums(int2 sp, float2 *b) {
    const int lane = threadIdx.x & 31;
    const int per = (sp.y + 31) / 32, i0 = lane * per, i1 = min(i0 + per, sp.y);
    float2 s = make_float2(0.f, 0.f);
    for (int i = i0; i < i1; i++) s = decay_add(s, b[i]);
    float2 before = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float2 v = make_float2(__shfl_up_sync(0xffffffffu, before.x, o), __shfl_up_sync(0xffffffffu, before.y, o));
        if (lane >= o) before = decay_add(v, before);
    }
    before = make_float2(__shfl_up_sync(0xffffffffu, before.x, 1), __shfl_up_sync(0xffffffffu, before.y, 1));
    if (lane == 0) before = make_float2(0.f, 0.f);
    for (int i = i0; i < i1; i++) b[i] = before = decay_add(before, b[i]);
}

}  // namespace zs

// ---------------------------------------------------------------- launchers

// out (per span and value head xc x yc float32): the sum of w_j x_j y_j^T over the span's tokens;
// w_j = exp(b_L - b_j), or (`query`) scale exp(b_j).  The first launch of a call (`gates`) writes geo.gates.
cudaError_t zs_launch_decay_sums(int type, const zs::DecayGeom &g, const zs::DecayRows &x, const zs::DecayRows &y, bool query,
                                 bool gates, float *out, bool next, cudaStream_t st, int64_t *launches);
// The states in front of each span, of the spans' sums u and s0 (NULL: zero): in u's place (parts = 0), or in `parts` bfloat16 matrices
// each that add up to them (planes); and the last ones to sn (NULL: not written).
cudaError_t zs_launch_decay_scan(const zs::DecayGeom &g, float *u, void *planes, int parts, const float *s0, float *sn, bool next,
                                 cudaStream_t st, int64_t *launches);
// Their gradients after each span in the same forms (parts = 0 or 3, as the states have), of the sums w and ds (NULL: zero), the first
// ones' to ds0 (NULL: not written); and per span and head zs_decay_dots() partial sums of exp(b_L) <S, D> to dots.
cudaError_t zs_launch_decay_rscan(const zs::DecayGeom &g, float *w, void *planes, int parts, const float *states, const void *splanes,
                                  const float *ds, float *ds0, float *dots, bool next, cudaStream_t st, int64_t *launches);
inline bool zs_decay_vec(const zs::DecayGeom &g, const float *s, const float *t) {
    return g.d.dk * (int64_t)g.d.dv % 4 == 0 && (((uintptr_t)s | (uintptr_t)t) & 15) == 0;
}
inline int zs_decay_dots(const zs::DecayGeom &g, const float *ds, const float *ds0) {
    const int64_t block = zs_decay_vec(g, ds, ds0) ? 1024 : 256;
    return (int)(((int64_t)g.d.dk * g.d.dv + block - 1) / block) * 8;
}

cudaError_t zs_launch_decay_rows(int type, const zs::DecayGeom &g, const zs::DecayProduct &p, bool next, cudaStream_t st, int64_t *launches);
// The same for bfloat16 on the 5th-generation tensor cores (decay_tc.cu): dv a multiple of 8; x of at most 128 columns; spans of whole
// 128 tokens; and p.m `parts` bfloat16 matrices a state.  status: a word that a bounded wait sets when it gives up.
cudaError_t zs_launch_decay_sums_tc(const zs::DecayGeom &g, const zs::DecayRows &x, const zs::DecayRows &y, bool query, bool gates, float *out,
                                    unsigned *status, bool next, cudaStream_t st, int64_t *launches);
cudaError_t zs_launch_decay_rows_tc(const zs::DecayGeom &g, const zs::DecayProduct &p, int parts, int num_sms, unsigned *status, bool next,
                                    cudaStream_t st, int64_t *launches);
// dg from the sums of both directions and the dots: tokens x hv, or where each head has one decay (ldg = 0) per span in `parts`
// (spans x hv) and then in dg (hv).
cudaError_t zs_launch_decay_dg(const zs::DecayGeom &g, const float *const from_q[2], const float *const from_k[2], const float *dots,
                               int ndots, float *parts, float *dg, cudaStream_t st, int64_t *launches);
// Token by token (decay_step.cu).
cudaError_t zs_launch_decay_step(int type, const zs::DecayGeom &g, const int64_t *offsets, const float *s0, void *o, int64_t ldo, float *sn,
                                 cudaStream_t st, int64_t *launches);
