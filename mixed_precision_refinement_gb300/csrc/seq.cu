// The C-ABI of the sequence-layer operators: the handle, its workspace, and
// the argument checks in front of the kernels.
#include "decay.cuh"
#include "delta.cuh"
#include "seq.cuh"

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

namespace zs {

int seq_fail(zsolve_seq *s, int status, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(s->err, sizeof(s->err), fmt, ap);
    va_end(ap);
    return status;
}

void *seq_workspace(zsolve_seq *s, size_t bytes, int *status) {
    *status = ZSOLVE_OK;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(s->st, &cap);
    const bool capturing = e == cudaSuccess && cap != cudaStreamCaptureStatusNone;
    if (e == cudaSuccess && bytes <= s->ws_bytes) {
        s->ws_captured = s->ws_captured || capturing;
        return s->ws;
    }
    if (capturing) {
        *status = seq_fail(s, ZSOLVE_ESTATE,
                           "a workspace of %zu bytes is needed and cannot be allocated during a stream capture "
                           "(zsolve_seq_reserve before it)",
                           bytes);
        return nullptr;
    }
    // the old one may still be in use by work in flight, or by a graph
    if (e == cudaSuccess && s->ws && s->ws_captured) {
        try {
            s->retired.push_back(s->ws);
        } catch (...) {
            *status = seq_fail(s, ZSOLVE_ENOMEM, "out of host memory");
            return nullptr;
        }
    } else if (e == cudaSuccess && s->ws) {
        e = cudaDeviceSynchronize();
        if (e == cudaSuccess) e = cudaFree(s->ws);
    }
    if (e != cudaSuccess) {
        *status = seq_fail(s, ZSOLVE_ECUDA, "workspace: %s", cudaGetErrorString(e));
        return nullptr;
    }
    s->ws = nullptr;
    s->ws_bytes = 0;
    s->ws_captured = false;
    if (cudaMalloc(&s->ws, bytes) != cudaSuccess) {
        cudaGetLastError();  // not sticky: the next call may fit
        s->ws = nullptr;
        *status = seq_fail(s, ZSOLVE_ENOMEM, "a workspace of %zu bytes could not be allocated", bytes);
        return nullptr;
    }
    s->ws_bytes = bytes;
    return s->ws;
}

}  // namespace zs

using zs::seq_fail;

namespace {

// Whether the stream is in a capture (for the default stream: whether one
// elsewhere bars its use).
bool capturing(cudaStream_t st) {
    cudaStreamCaptureStatus c = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &c) != cudaSuccess) {
        cudaGetLastError();
        return true;
    }
    return c != cudaStreamCaptureStatusNone;
}

// The handle's device has to be the calling thread's current one.
int check_device(zsolve_seq *s) {
    int dev = 0;
    SEQ_CU(cudaGetDevice(&dev));
    if (dev != s->dev) return seq_fail(s, ZSOLVE_EINVAL, "the handle belongs to device %d, the current one is %d", s->dev, dev);
    return ZSOLVE_OK;
}

int check_linear(zsolve_seq *s, int type, int act, int64_t m, int64_t n, int64_t k) {
    if (type != ZSOLVE_BF16 && type != ZSOLVE_F16)
        return seq_fail(s, ZSOLVE_EINVAL, "type %d: ZSOLVE_BF16 or ZSOLVE_F16", type);
    if (act < ZSOLVE_ACT_NONE || act > ZSOLVE_ACT_GELU_TANH) return seq_fail(s, ZSOLVE_EINVAL, "act = %d", act);
    const int64_t most = 1 << 24;  // rows times tiles stay within 32 bits
    if (m < 0 || m > 0x7fffff00 || n < 1 || n > most || k < 1 || k > most ||
        ((m + 127) / 128) * ((n + 127) / 128) > 0x3ffffff || ((n + 127) / 128) * ((k + 127) / 128) > 0x3ffffff ||
        ((m + 127) / 128) * ((k + 127) / 128) > 0x3ffffff)
        return seq_fail(s, ZSOLVE_EINVAL, "m = %lld, n = %lld, k = %lld", (long long)m, (long long)n, (long long)k);
    return ZSOLVE_OK;
}

int check_resnorm(zsolve_seq *s, const zsolve_resnorm_args *a) {
    if (!a) return seq_fail(s, ZSOLVE_EINVAL, "NULL arguments");
    if (!zs::type_ok(a->type) || (a->wtype != a->type && a->wtype != ZSOLVE_F32))
        return seq_fail(s, ZSOLVE_EINVAL, "type %d, wtype %d: wtype is the type of the tensors or ZSOLVE_F32", a->type, a->wtype);
    if (a->kind != ZSOLVE_NORM_LAYER && a->kind != ZSOLVE_NORM_RMS) return seq_fail(s, ZSOLVE_EINVAL, "kind = %d", a->kind);
    if (a->act < ZSOLVE_ACT_NONE || a->act > ZSOLVE_ACT_GELU_TANH) return seq_fail(s, ZSOLVE_EINVAL, "act = %d", a->act);
    if (a->rows < 0 || a->rows > 0x7fffffff || a->d < 1 || a->d > 1 << 24)
        return seq_fail(s, ZSOLVE_EINVAL, "rows = %lld, d = %lld", (long long)a->rows, (long long)a->d);
    if (!(a->eps >= 0.0) || !std::isfinite(a->eps)) return seq_fail(s, ZSOLVE_EINVAL, "eps = %g", a->eps);
    if (a->rows > 0 && (!a->o || a->ldo < a->d || (a->z && a->ldz < a->d)))
        return seq_fail(s, ZSOLVE_EINVAL, "NULL o, or a row stride below d = %lld", (long long)a->d);
    return ZSOLVE_OK;
}

// The longest a sequence of the call can be.
int64_t longest(const zsolve_delta_args *a) {
    return a->nseq == 0 ? 0 : a->offsets ? a->tokens : a->tokens / a->nseq;
}

// Up to so many tokens a sequence, one kernel that takes them one by one
// (1.2 to 1.5 us each) is sooner done than the chunked form's three (20 us up to 64
// tokens; 8 tokens x 32 heads of 128 in bfloat16: 12.9 and 20.5, 16 tokens: 21.0 and 20.5).
constexpr int64_t kStepTokens = 8;

// The arguments of a delta rule call, checked, as the kernels take them.
int check_delta(zsolve_seq *s, const zsolve_delta_args *a, const void *o, int64_t ldo, zs::DeltaGeom *g) {
    if (!a) return seq_fail(s, ZSOLVE_EINVAL, "NULL arguments");
    if (!zs::type_ok(a->type)) return seq_fail(s, ZSOLVE_EINVAL, "type %d", a->type);
    if (a->hk < 1 || a->hv < 1 || a->hv % a->hk != 0 || a->hk > 65535)
        return seq_fail(s, ZSOLVE_EINVAL, "hk = %d, hv = %d: hv is a multiple of hk", a->hk, a->hv);
    if (a->dk < 1 || a->dk > ZSOLVE_DELTA_MAX_DK || a->dv < 1 || a->dv > 65536)
        return seq_fail(s, ZSOLVE_EINVAL, "dk = %d outside 1..%d or dv = %d outside 1..65536", a->dk, ZSOLVE_DELTA_MAX_DK, a->dv);
    if (a->nseq < 0 || a->tokens < 0 || a->tokens > 0x7fffff00 || (int64_t)a->nseq * a->hv > 0x7fffffff ||
        (a->nseq == 0 && a->tokens > 0) || (!a->offsets && a->nseq > 0 && a->tokens % a->nseq != 0))
        return seq_fail(s, ZSOLVE_EINVAL, "nseq = %d, tokens = %lld", a->nseq, (long long)a->tokens);
    if (!std::isfinite(a->scale)) return seq_fail(s, ZSOLVE_EINVAL, "scale = %g", a->scale);
    if (a->tokens > 0) {
        if (!a->q || !a->k || !a->v || !a->g || !a->beta || !o)
            return seq_fail(s, ZSOLVE_EINVAL, "NULL q, k, v, g, beta or output");
        const int64_t rk = (int64_t)a->hk * a->dk, rv = (int64_t)a->hv * a->dv;
        if (a->ldq < rk || a->ldk < rk || a->ldv < rv || ldo < rv)
            return seq_fail(s, ZSOLVE_EINVAL, "a token stride is below its heads' values");
    }
    const int ve = 16 / (int)zs::type_bytes(a->type);
    *g = zs::DeltaGeom{a->q, a->k, a->v, a->ldq, a->ldk, a->ldv, (a->dk + ve - 1) / ve * ve, (a->dv + ve - 1) / ve * ve, a->g, a->beta, a->hk, a->hv, a->dk, a->dv, a->nseq,
                       a->tokens, (float)a->scale, nullptr, nullptr, nullptr, 0};
    return ZSOLVE_OK;
}

// The chunked form's workspace.
struct DeltaWork {
    int nchunks = 0;
    int *first = nullptr;
    int2 *seq = nullptr, *chunk = nullptr;
    zs::DeltaTerms terms{};
    bool backward = false;
    void *qp = nullptr, *kp = nullptr, *vp = nullptr, *dop = nullptr;  // packed copies, where needed
    float *states = nullptr, *us = nullptr, *dends = nullptr, *dxs = nullptr, *dqp = nullptr, *dkp = nullptr;

    const void *dout = nullptr;  // backward: the gradient of o
    int64_t lddo = 0;

    static bool aligned(const void *p, int64_t ld, int64_t d, size_t e) {
        return (((uintptr_t)p | (uint64_t)ld * e | (uint64_t)d * e) & 15) == 0;
    }
    void carve(zs::Carve &c, const zsolve_delta_args *a) {
        const size_t slots = (size_t)(nchunks - (a->offsets ? 1 : 0)) * a->hv, sq = (size_t)zs::kSquare;
        first = c.take<int>((size_t)a->nseq + 1);
        seq = c.take<int2>((size_t)a->nseq);
        chunk = c.take<int2>((size_t)nchunks);
        terms.tp = c.take<float>(slots * sq);
        terms.vec = c.take<float>(slots * zs::kVec);
        const size_t e = zs::type_bytes(a->type), ve = 16 / e;
        const size_t nk = (size_t)a->tokens * a->hk * ((a->dk + ve - 1) / ve * ve) * e;
        const size_t nv = (size_t)a->tokens * a->hv * ((a->dv + ve - 1) / ve * ve) * e;
        qp = aligned(a->q, a->ldq, a->dk, e) ? nullptr : c.take<char>(nk);
        kp = aligned(a->k, a->ldk, a->dk, e) ? nullptr : c.take<char>(nk);
        vp = aligned(a->v, a->ldv, a->dv, e) ? nullptr : c.take<char>(nv);
        if (!backward) return;
        dop = aligned(dout, lddo, a->dv, e) ? nullptr : c.take<char>(nv);
        const size_t state = (size_t)a->dk * a->dv, rows = (size_t)zs::kChunk * a->dv;
        states = c.take<float>(slots * state);
        us = c.take<float>(slots * rows);
        dends = c.take<float>(slots * state);
        dxs = c.take<float>(slots * rows);
        if (a->hv == a->hk) return;
        dqp = c.take<float>((size_t)a->tokens * a->hv * a->dk);
        dkp = c.take<float>((size_t)a->tokens * a->hv * a->dk);
    }
    int place(zsolve_seq *s, const zsolve_delta_args *a) {
        // a sequence's last chunk may be short: one more each at most
        const int64_t most = a->tokens / zs::kChunk + a->nseq;
        if (most > 0x7fffffff / zs::kChunk) return seq_fail(s, ZSOLVE_EINVAL, "too many chunks");
        // and an unused entry, whose blocks write what belongs to the tokens outside the offsets
        nchunks = (int)most + (a->offsets ? 1 : 0);
        zs::Carve size(nullptr);
        carve(size, a);
        int st = ZSOLVE_OK;
        void *ws = zs::seq_workspace(s, size.at, &st);
        if (!ws) return st;
        zs::Carve c(ws);
        carve(c, a);
        return ZSOLVE_OK;
    }
    // The geometry on the workspace's tables and, where they are needed, packed copies.
    int bind(zsolve_seq *s, const zsolve_delta_args *a, zs::DeltaGeom *g) {
        struct {
            const void **p;
            int64_t *ld;
            void *copy;
            int heads, d, dp;
        } const t[4] = {{&g->q, &g->ldq, qp, a->hk, a->dk, g->dkp},
                        {&g->k, &g->ldk, kp, a->hk, a->dk, g->dkp},
                        {&g->v, &g->ldv, vp, a->hv, a->dv, g->dvp},
                        {&dout, &lddo, dop, a->hv, a->dv, g->dvp}};
        for (const auto &x : t) {
            if (!x.copy || a->tokens == 0) continue;
            SEQ_CU(zs_launch_delta_pack(a->type, *x.p, *x.ld, a->tokens, x.heads, x.d, x.dp, x.copy, s->num_sms, s->st,
                                        &s->launches));
            *x.p = x.copy;
            *x.ld = (int64_t)x.heads * x.dp;
        }
        g->first = first;
        g->seq = seq;
        g->chunk = chunk;
        g->nchunks = nchunks;
        return ZSOLVE_OK;
    }
};

// The arguments of a decayed attention call, checked, as the kernels take them.
int check_decay(zsolve_seq *s, const zsolve_decay_args *a, const void *o, int64_t ldo, zs::DecayGeom *g) {
    if (!a) return seq_fail(s, ZSOLVE_EINVAL, "NULL arguments");
    if (!zs::type_ok(a->type)) return seq_fail(s, ZSOLVE_EINVAL, "type %d", a->type);
    if (a->hk < 1 || a->hv < 1 || a->hv % a->hk != 0 || a->hv > 65535)
        return seq_fail(s, ZSOLVE_EINVAL, "hk = %d, hv = %d: hv is a multiple of hk up to 65535", a->hk, a->hv);
    if (a->dk < 1 || a->dk > ZSOLVE_DECAY_MAX_DK || a->dv < 1 || a->dv > 65536)
        return seq_fail(s, ZSOLVE_EINVAL, "dk = %d outside 1..%d or dv = %d outside 1..65536", a->dk, ZSOLVE_DECAY_MAX_DK, a->dv);
    if (a->nseq < 0 || a->tokens < 0 || a->tokens > 0x7fffff00 || (int64_t)a->nseq * a->hv > 0x7fffffff ||
        (a->nseq == 0 && a->tokens > 0) || (!a->offsets && a->nseq > 0 && a->tokens % a->nseq != 0))
        return seq_fail(s, ZSOLVE_EINVAL, "nseq = %d, tokens = %lld", a->nseq, (long long)a->tokens);
    if (!std::isfinite(a->scale)) return seq_fail(s, ZSOLVE_EINVAL, "scale = %g", a->scale);
    if (a->ldg != 0 && a->ldg != a->hv) return seq_fail(s, ZSOLVE_EINVAL, "ldg = %lld: hv, or 0 for one decay a head", (long long)a->ldg);
    if (a->tokens > 0) {
        if (!a->q || !a->k || !a->v || !a->g || !o) return seq_fail(s, ZSOLVE_EINVAL, "NULL q, k, v, g or output");
        const int64_t rk = (int64_t)a->hk * a->dk, rv = (int64_t)a->hv * a->dv;
        if (a->ldq < rk || a->ldk < rk || a->ldv < rv || ldo < rv)
            return seq_fail(s, ZSOLVE_EINVAL, "a token stride is below its heads' values");
    }
    const int ve = 16 / (int)zs::type_bytes(a->type);
    *g = zs::DecayGeom{};
    g->d = zs::DeltaGeom{a->q, a->k, a->v, a->ldq, a->ldk, a->ldv, (a->dk + ve - 1) / ve * ve, (a->dv + ve - 1) / ve * ve, a->g, nullptr,
                         a->hk, a->hv, a->dk, a->dv, a->nseq, a->tokens, (float)a->scale, nullptr, nullptr, nullptr, 0};
    g->ldg = a->ldg;
    return ZSOLVE_OK;
}

// The spans' workspace.
struct DecayWork {
    int *first = nullptr;
    int2 *seq = nullptr, *chunk = nullptr;
    float2 *gates = nullptr;
    float *ends = nullptr;
    float *u = nullptr, *w = nullptr, *dots = nullptr, *parts = nullptr, *sums[4] = {};
    void *copy[4] = {};  // packed q, k, v and dout, where needed
    int ndots = 0;
    int nparts = 0;      // bfloat16 matrices of a state, where the kernels of decay_tc.cu take them (else 0)
    void *uplanes = nullptr, *wplanes = nullptr;
    zs::DecayRows q{}, k{}, v{}, dout{};

    const void *states() const { return nparts ? uplanes : u; }
    const void *dstates() const { return nparts ? wplanes : w; }
    cudaError_t sums_of(zsolve_seq *s, const zsolve_decay_args *a, const zs::DecayGeom &g, const zs::DecayRows &x, const zs::DecayRows &y,
                        bool query, bool first_sums, float *out) const {
        return nparts ? zs_launch_decay_sums_tc(g, x, y, query, first_sums, out, s->d_status, true, s->st, &s->launches)
                      : zs_launch_decay_sums(a->type, g, x, y, query, first_sums, out, true, s->st, &s->launches);
    }
    cudaError_t rows_of(zsolve_seq *s, const zsolve_decay_args *a, const zs::DecayGeom &g, const zs::DecayProduct &p) const {
        return nparts ? zs_launch_decay_rows_tc(g, p, nparts, s->num_sms, s->d_status, true, s->st, &s->launches)
                      : zs_launch_decay_rows(a->type, g, p, true, s->st, &s->launches);
    }

    // Tokens of a span, by the rows (tokens x heads) of the call.  Short spans are short chains of products and many blocks, which is what few
    // tokens need; long ones are few states to write, read and hold, which is what many tokens cost.  One sequence, heads of 128 x 128,
    // us forwards / backwards (in brackets heads of 64 x 64):
    //   mma.sync, float32    rows  16000 (8 heads)    30000 (8)   40000 (8)   40000 (32)              80000 (32)   160000 (32)
    //     spans of  64       67 / 233 (37 / 132)      120 / 464   163 / 675   145 / 619 (65 / 215)    269 / 1058   502 / 1919 (215 / 660)
    //     spans of 128       69 / 280 (40 / 176)      121 / 528   156 / 639   148 / 622 (72 / 258)    273 / 1101   506 / 2017 (214 / 756)
    //     spans of 256       101 / 425 (56 / 283)     144 / 675   190 / 833   195 / 840 (87 / 353)    338 / 1462   610 / 2603 (267 / 1036)
    //   float16, 160000 rows:  64: 352 / 1034, 128: 326 / 1048.  So 64 is as fast or faster backwards at any size but one, and above 40000 rows the
    //   rule takes 128 for the workspace: half the states, 82 MB for 164 in float32 at 160000 rows (twice that backwards).
    //   tensor memory        rows  16000 (8 heads)    32000 (8)   64000 (8)   64000 (32)              160000 (32)             1048576 (32)
    //     spans of 128       31 / 103 (24 / 85)       46 / 148    81 / 275    66 / 233 (44 / 149)     164 / 530 (91 / 321)    993 / 2889 (530 / 1698)
    //     spans of 256       35 / 113 (27 / 92)       40 / 128    66 / 224    57 / 204 (42 / 150)     134 / 458 (87 / 321)    731 / 2327 (462 / 1645)
    //     spans of 512       46 / 149 (35 / 123)      49 / 156    67 / 224    64 / 228 (49 / 178)     137 / 484 (95 / 371)    670 / 2283 (461 / 1767)
    //   Forwards 512 costs 2 % (heads of 64: 9) at 160000 rows and gains 8 % at a million; where they cross was not looked for.
    static int span_of(const zsolve_decay_args *a, bool tc, bool backward) {
        const int64_t rows = a->tokens * a->hv;
        if (!tc) return rows <= 40000 ? 64 : 128;
        return rows <= 16384 ? 128 : rows <= 65536 || backward ? 256 : 512;
    }

    // Copies of rows that 16-byte loads cannot address, and the tables; dout NULL: the forward pass.
    int place(zsolve_seq *s, const zsolve_decay_args *a, zs::DecayGeom *g, const void *dout_p, int64_t lddo, bool backward, const float *ds,
              const float *ds0) {
        const bool tc = a->type == ZSOLVE_BF16 && a->dv % 8 == 0 && (!backward || a->dv <= 128);
        g->span = span_of(a, tc, backward);
        nparts = !tc ? 0 : backward ? 3 : 2;
        const int64_t most = a->tokens / g->span + a->nseq;
        if (most > 0x7fffffff / zs::kSpanMost) return seq_fail(s, ZSOLVE_EINVAL, "too many spans");
        // and an unused entry, whose blocks write what belongs to the tokens outside the offsets
        g->d.nchunks = (int)most + (a->offsets ? 1 : 0);
        const size_t slots = (size_t)most * a->hv, state = (size_t)a->dk * a->dv, e = zs::type_bytes(a->type);
        const void *src[4] = {a->q, a->k, a->v, dout_p};
        const int64_t ld[4] = {a->ldq, a->ldk, a->ldv, lddo};
        const int heads[4] = {a->hk, a->hk, a->hv, a->hv}, cols[4] = {a->dk, a->dk, a->dv, a->dv}, dist[4] = {g->d.dkp, g->d.dkp, g->d.dvp, g->d.dvp};
        ndots = backward ? zs_decay_dots(*g, ds, ds0) : 0;
        auto carve = [&](zs::Carve c) {
            first = c.take<int>((size_t)a->nseq + 1);
            seq = c.take<int2>((size_t)a->nseq);
            chunk = c.take<int2>((size_t)g->d.nchunks);
            gates = c.take<float2>(slots * g->span);
            ends = c.take<float>(slots);
            u = c.take<float>(slots * state);
            uplanes = nparts ? c.take<uint16_t>(slots * nparts * state) : nullptr;
            for (int i = 0; i < (backward ? 4 : 3); i++)
                copy[i] = zs::mult16(src[i], ld[i], cols[i], e) ? nullptr : c.take<char>((size_t)a->tokens * heads[i] * dist[i] * e);
            if (!backward) return c.at;
            w = c.take<float>(slots * state);
            wplanes = nparts ? c.take<uint16_t>(slots * nparts * state) : nullptr;
            dots = c.take<float>(slots * ndots);
            parts = a->ldg ? nullptr : c.take<float>((size_t)g->d.nchunks * a->hv);
            for (float *&x : sums) x = c.take<float>((size_t)a->tokens * a->hv);
            return c.at;
        };
        const size_t bytes = carve(zs::Carve(nullptr));
        int st = ZSOLVE_OK;
        void *ws = zs::seq_workspace(s, bytes, &st);
        if (!ws) return st;
        carve(zs::Carve(ws));
        zs::DecayRows *const rows[4] = {&q, &k, &v, &dout};
        for (int i = 0; i < (backward ? 4 : 3); i++) {
            *rows[i] = zs::DecayRows{src[i], ld[i], cols[i], copy[i] ? dist[i] : cols[i], i < 2};
            if (!copy[i] || a->tokens == 0) continue;
            SEQ_CU(zs_launch_delta_pack(a->type, src[i], ld[i], a->tokens, heads[i], cols[i], dist[i], copy[i], s->num_sms, s->st, &s->launches));
            rows[i]->p = copy[i];
            rows[i]->ld = (int64_t)heads[i] * dist[i];
        }
        g->d.first = first;
        g->d.seq = seq;
        g->d.chunk = chunk;
        g->gates = gates;
        g->ends = ends;
        SEQ_CU(zs_launch_delta_plan(a->offsets, a->nseq, a->tokens, g->span, g->d.nchunks, first, seq, chunk, s->st, &s->launches));
        return ZSOLVE_OK;
    }
};

}  // namespace

extern "C" {

int zsolve_seq_create(zsolve_seq **out) {
    if (!out) return ZSOLVE_EINVAL;
    *out = nullptr;
    zsolve_seq *s = new (std::nothrow) zsolve_seq;
    if (!s) return ZSOLVE_ENOMEM;
    auto bail = [&](int st) {
        zsolve_seq_destroy(s);
        return st;
    };
    if (cudaGetDevice(&s->dev) != cudaSuccess) return bail(ZSOLVE_ECUDA);
    if (cudaDeviceGetAttribute(&s->num_sms, cudaDevAttrMultiProcessorCount, s->dev) != cudaSuccess)
        return bail(ZSOLVE_ECUDA);
    if (cudaEventCreateWithFlags(&s->ev, cudaEventDisableTiming) != cudaSuccess) return bail(ZSOLVE_ECUDA);
    if (cudaStreamCreateWithFlags(&s->side, cudaStreamNonBlocking) != cudaSuccess ||
        cudaEventCreateWithFlags(&s->fork, cudaEventDisableTiming) != cudaSuccess ||
        cudaEventCreateWithFlags(&s->joined, cudaEventDisableTiming) != cudaSuccess)
        return bail(ZSOLVE_ECUDA);
    if (cudaMalloc(&s->d_status, sizeof(unsigned)) != cudaSuccess) return bail(ZSOLVE_ENOMEM);
    if (cudaMemset(s->d_status, 0, sizeof(unsigned)) != cudaSuccess) return bail(ZSOLVE_ECUDA);
    *out = s;
    return ZSOLVE_OK;
}

int zsolve_seq_set_stream(zsolve_seq *s, void *stream) {
    if (!s) return ZSOLVE_EINVAL;
    cudaStream_t st = (cudaStream_t)stream;
    if (st == s->st) return ZSOLVE_OK;
    // The workspace is shared: the new stream's work comes after the old
    // stream's.  A capture cannot wait for work outside it; the caller has
    // waited for that work before the capture began.
    if (s->launches > 0 && !capturing(s->st) && !capturing(st)) {
        SEQ_CU(cudaEventRecord(s->ev, s->st));
        SEQ_CU(cudaStreamWaitEvent(st, s->ev, 0));
    }
    s->st = st;
    return ZSOLVE_OK;
}

int zsolve_seq_reserve(zsolve_seq *s, int64_t bytes) {
    if (!s) return ZSOLVE_EINVAL;
    if (bytes < 0) return seq_fail(s, ZSOLVE_EINVAL, "bytes = %lld is negative", (long long)bytes);
    int st = check_device(s);
    if (st == ZSOLVE_OK && bytes > 0) zs::seq_workspace(s, (size_t)bytes, &st);
    return st;
}

int64_t zsolve_seq_workspace_bytes(const zsolve_seq *s) { return s ? (int64_t)s->ws_bytes : 0; }

int64_t zsolve_seq_launches(const zsolve_seq *s) { return s ? s->launches : 0; }

const char *zsolve_seq_last_error(const zsolve_seq *s) { return s ? s->err : "NULL handle"; }

void zsolve_seq_destroy(zsolve_seq *s) {
    if (!s) return;
    cudaFree(s->ws);  // waits for the work in flight
    for (void *p : s->retired) cudaFree(p);
    cudaFree(s->d_status);
    if (s->ev) cudaEventDestroy(s->ev);
    if (s->fork) cudaEventDestroy(s->fork);
    if (s->joined) cudaEventDestroy(s->joined);
    if (s->side) cudaStreamDestroy(s->side);
    delete s;
}

int zsolve_layernorm(zsolve_seq *s, int type, int wtype, int64_t rows, int64_t d, const void *x, int64_t ldx,
                     const void *w, const void *b, double eps, void *y, int64_t ldy, float *mean, float *rstd) {
    if (!s) return ZSOLVE_EINVAL;
    if (!zs::type_ok(type) || (wtype != type && wtype != ZSOLVE_F32))
        return seq_fail(s, ZSOLVE_EINVAL, "type %d, wtype %d: wtype is the type of x or ZSOLVE_F32", type, wtype);
    if (rows < 0 || rows > 0x7fffffff || d < 1 || d > 0x7fffffff)
        return seq_fail(s, ZSOLVE_EINVAL, "rows = %lld, d = %lld", (long long)rows, (long long)d);
    if (!(eps >= 0.0) || !std::isfinite(eps)) return seq_fail(s, ZSOLVE_EINVAL, "eps = %g", eps);
    if (rows == 0) return ZSOLVE_OK;
    if (!x || !y) return seq_fail(s, ZSOLVE_EINVAL, "NULL x or y");
    if (ldx < d || ldy < d) return seq_fail(s, ZSOLVE_EINVAL, "ldx = %lld or ldy = %lld is below d = %lld", (long long)ldx, (long long)ldy, (long long)d);
    int st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    SEQ_CU(zs_launch_layernorm(type, wtype == ZSOLVE_F32, rows, d, x, ldx, w, b, (float)eps, y, ldy, mean, rstd, s->st,
                               &s->launches));
    return ZSOLVE_OK;
}

int zsolve_layernorm_bwd(zsolve_seq *s, int type, int wtype, int64_t rows, int64_t d, const void *dy, int64_t lddy,
                         const void *x, int64_t ldx, const float *mean, const float *rstd, const void *w, void *dx,
                         int64_t lddx, void *dw, void *db) {
    if (!s) return ZSOLVE_EINVAL;
    if (!zs::type_ok(type) || (wtype != type && wtype != ZSOLVE_F32))
        return seq_fail(s, ZSOLVE_EINVAL, "type %d, wtype %d: wtype is the type of x or ZSOLVE_F32", type, wtype);
    if (rows < 0 || rows > 0x7fffffff || d < 1 || d > 0x7fffffff)
        return seq_fail(s, ZSOLVE_EINVAL, "rows = %lld, d = %lld", (long long)rows, (long long)d);
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return seq_fail(s, ZSOLVE_EINVAL, "NULL dy, x, mean, rstd or dx");
    if (rows > 0 && (lddy < d || ldx < d || lddx < d))
        return seq_fail(s, ZSOLVE_EINVAL, "a row stride (%lld, %lld, %lld) is below d = %lld", (long long)lddy, (long long)ldx, (long long)lddx, (long long)d);
    int st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    float *parts = nullptr;
    if (dw || db) {
        const int64_t n = zs_layernorm_bwd_parts(type, rows, d, s->num_sms);
        if (n > 0) parts = (float *)zs::seq_workspace(s, (size_t)n * 4, &st);
        if (st != ZSOLVE_OK) return st;
    }
    SEQ_CU(zs_launch_layernorm_bwd(type, wtype == ZSOLVE_F32, rows, d, dy, lddy, x, ldx, mean, rstd, w, dx, lddx, dw,
                                   db, parts, s->num_sms, s->d_status, s->st, &s->launches));
    return ZSOLVE_OK;
}

int zsolve_resnorm(zsolve_seq *s, const zsolve_resnorm_args *a, const void *x, int64_t ldx, void *y, int64_t ldy, void *h, int64_t ldh,
                   float *stats) {
    if (!s) return ZSOLVE_EINVAL;
    int st = check_resnorm(s, a);
    if (st != ZSOLVE_OK || a->rows == 0) return st;
    if (!x || !y || !h) return seq_fail(s, ZSOLVE_EINVAL, "NULL x, y or h");
    if (ldx < a->d || ldy < a->d || ldh < a->d) return seq_fail(s, ZSOLVE_EINVAL, "a row stride is below d = %lld", (long long)a->d);
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    return zs_resnorm(s, a, x, ldx, y, ldy, h, ldh, stats);
}

int zsolve_resnorm_bwd(zsolve_seq *s, const zsolve_resnorm_args *a, const void *dh, int64_t lddh, const void *dy, int64_t lddy,
                       const void *y, int64_t ldy, const float *stats, void *dx, int64_t lddx, void *dout, int64_t lddo, void *dz,
                       int64_t lddz, void *dw1, void *db1, void *dc, void *dw2, void *db2) {
    if (!s) return ZSOLVE_EINVAL;
    int st = check_resnorm(s, a);
    if (st != ZSOLVE_OK) return st;
    if (a->rows > 0 && (!dh || !y || !stats || !dx || !dout)) return seq_fail(s, ZSOLVE_EINVAL, "NULL dh, y, stats, dx or do");
    if (dz && !a->z) return seq_fail(s, ZSOLVE_EINVAL, "dz without z");
    if (a->rows > 0 && (lddh < a->d || ldy < a->d || lddx < a->d || lddo < a->d || (dy && lddy < a->d) || (dz && lddz < a->d)))
        return seq_fail(s, ZSOLVE_EINVAL, "a row stride is below d = %lld", (long long)a->d);
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    return zs_resnorm_bwd(s, a, dh, lddh, dy, lddy, y, ldy, stats, dx, lddx, dout, lddo, dz, lddz, dw1, db1, dc, dw2, db2);
}

int zsolve_seq_check(zsolve_seq *s) {
    if (!s) return ZSOLVE_EINVAL;
    int st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    unsigned word = 0;
    SEQ_CU(cudaMemcpyAsync(&word, s->d_status, sizeof(word), cudaMemcpyDeviceToHost, s->st));
    SEQ_CU(cudaStreamSynchronize(s->st));
    if (!word) return ZSOLVE_OK;
    SEQ_CU(cudaMemsetAsync(s->d_status, 0, sizeof(word), s->st));
    return seq_fail(s, ZSOLVE_ETIMEOUT, "a bounded device-side wait gave up");
}

int zsolve_linear(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx, const void *w,
                  int64_t ldw, const void *b, int act, const void *r, int64_t ldr, void *y, int64_t ldy, void *z,
                  int64_t ldz) {
    if (!s) return ZSOLVE_EINVAL;
    int st = check_linear(s, type, act, m, n, k);
    if (st != ZSOLVE_OK || m == 0) return st;
    if (!x || !w || !y) return seq_fail(s, ZSOLVE_EINVAL, "NULL x, w or y");
    if (ldx < k || ldw < k || ldy < n || (r && ldr < n) || (z && ldz < n))
        return seq_fail(s, ZSOLVE_EINVAL, "a row stride is below its row's length");
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    return zs_linear(s, type, m, n, k, x, ldx, w, ldw, b, act, r, ldr, y, ldy, z, ldz);
}

int zsolve_linear_bwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *dy, int64_t lddy,
                      const void *x, int64_t ldx, const void *w, int64_t ldw, int act, const void *z, int64_t ldz,
                      void *dx, int64_t lddx, void *dw, int64_t lddw, void *db) {
    if (!s) return ZSOLVE_EINVAL;
    int st = check_linear(s, type, act, m, n, k);
    if (st != ZSOLVE_OK) return st;
    if (m > 0 && (!dy || (dw && !x) || (dx && !w) || (act != ZSOLVE_ACT_NONE && !z)))
        return seq_fail(s, ZSOLVE_EINVAL, "NULL dy, x, w or z that the gradients asked for need");
    if ((m > 0 && (lddy < n || (dw && ldx < k) || (dx && (ldw < k || lddx < k)) ||
                   (act != ZSOLVE_ACT_NONE && ldz < n))) || (dw && lddw < k))
        return seq_fail(s, ZSOLVE_EINVAL, "a row stride is below its row's length");
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    return zs_linear_bwd(s, type, m, n, k, dy, lddy, x, ldx, w, ldw, act, z, ldz, dx, lddx, dw, lddw, db);
}

int zsolve_glu(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx, const void *wg, int64_t ldwg,
               const void *wu, int64_t ldwu, const void *bg, const void *bu, int act, void *y, int64_t ldy, void *zg, int64_t ldzg,
               void *zu, int64_t ldzu) {
    if (!s) return ZSOLVE_EINVAL;
    int st = check_linear(s, type, act, m, n, k);
    if (st != ZSOLVE_OK || m == 0) return st;
    if (!x || !wg || !wu || !y || !zg != !zu) return seq_fail(s, ZSOLVE_EINVAL, "NULL x, wg, wu or y, or one of zg and zu without the other");
    if (ldx < k || ldwg < k || ldwu < k || ldy < n || (zg && (ldzg < n || ldzu < n)))
        return seq_fail(s, ZSOLVE_EINVAL, "a row stride is below its row's length");
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    return zs_glu(s, type, m, n, k, x, ldx, wg, ldwg, wu, ldwu, bg, bu, act, y, ldy, zg, ldzg, zu, ldzu);
}

int zsolve_glu_bwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                   const void *wg, int64_t ldwg, const void *wu, int64_t ldwu, int act, const void *zg, int64_t ldzg, const void *zu,
                   int64_t ldzu, void *dx, int64_t lddx, void *dwg, int64_t lddwg, void *dwu, int64_t lddwu, void *dbg, void *dbu) {
    if (!s) return ZSOLVE_EINVAL;
    int st = check_linear(s, type, act, m, n, k);
    if (st != ZSOLVE_OK) return st;
    const bool dw = dwg || dwu;
    if (m > 0 && (!dy || !zg || !zu || (dw && !x) || (dx && (!wg || !wu))))
        return seq_fail(s, ZSOLVE_EINVAL, "NULL dy, zg, zu, or an x, wg or wu that the gradients asked for need");
    if ((m > 0 && (lddy < n || ldzg < n || ldzu < n || (dw && ldx < k) || (dx && (ldwg < k || ldwu < k || lddx < k)))) ||
        (dwg && lddwg < k) || (dwu && lddwu < k))
        return seq_fail(s, ZSOLVE_EINVAL, "a row stride is below its row's length");
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    return zs_glu_bwd(s, type, m, n, k, dy, lddy, x, ldx, wg, ldwg, wu, ldwu, act, zg, ldzg, zu, ldzu, dx, lddx, dwg, lddwg, dwu, lddwu,
                      dbg, dbu);
}

int zsolve_delta(zsolve_seq *s, const zsolve_delta_args *a, void *o, int64_t ldo, float *sn) {
    if (!s) return ZSOLVE_EINVAL;
    zs::DeltaGeom g;
    int st = check_delta(s, a, o, ldo, &g);
    if (st != ZSOLVE_OK || a->nseq == 0) return st;
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    if (longest(a) <= kStepTokens) {
        SEQ_CU(zs_launch_delta_step(a->type, g, a->offsets, a->s0, o, ldo, sn, s->st, &s->launches));
        return ZSOLVE_OK;
    }
    DeltaWork w;
    st = w.place(s, a);
    if (st == ZSOLVE_OK) st = w.bind(s, a, &g);
    if (st != ZSOLVE_OK) return st;
    SEQ_CU(zs_launch_delta_plan(a->offsets, a->nseq, a->tokens, zs::kChunk, w.nchunks, w.first, w.seq, w.chunk, s->st, &s->launches));
    SEQ_CU(zs_launch_delta_terms(a->type, g, w.terms, o, ldo, true, s->st, &s->launches));
    SEQ_CU(zs_launch_delta_chain(a->type, g, w.terms, a->s0, o, ldo, sn, nullptr, nullptr, s->d_status, true, s->st,
                                 &s->launches));
    return ZSOLVE_OK;
}

int zsolve_delta_step(zsolve_seq *s, const zsolve_delta_args *a, void *o, int64_t ldo, float *sn) {
    if (!s) return ZSOLVE_EINVAL;
    zs::DeltaGeom g;
    int st = check_delta(s, a, o, ldo, &g);
    if (st != ZSOLVE_OK || a->nseq == 0) return st;
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    SEQ_CU(zs_launch_delta_step(a->type, g, a->offsets, a->s0, o, ldo, sn, s->st, &s->launches));
    return ZSOLVE_OK;
}

int zsolve_decay(zsolve_seq *s, const zsolve_decay_args *a, void *o, int64_t ldo, float *sn) {
    if (!s) return ZSOLVE_EINVAL;
    zs::DecayGeom g;
    int st = check_decay(s, a, o, ldo, &g);
    if (st != ZSOLVE_OK || a->nseq == 0) return st;
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    const int64_t longest = a->offsets ? a->tokens : a->tokens / a->nseq;
    // The delta rule's bound.  Here the two cross later: heads of 128 x 128 in bfloat16, token by token / in spans, 8 tokens of one sequence
    // x 32 heads 7.2 / 22.4 us, 16 tokens 12.0 / 22.4, 32 tokens 21.8 / 22.4; 64 such sequences 133 / 233, 242 / 238, 462 / 243.
    if (longest <= kStepTokens) {
        SEQ_CU(zs_launch_decay_step(a->type, g, a->offsets, a->s0, o, ldo, sn, s->st, &s->launches));
        return ZSOLVE_OK;
    }
    DecayWork w;
    st = w.place(s, a, &g, nullptr, 0, false, nullptr, nullptr);
    if (st != ZSOLVE_OK) return st;
    SEQ_CU(w.sums_of(s, a, g, w.k, w.v, false, true, w.u));
    SEQ_CU(zs_launch_decay_scan(g, w.u, w.uplanes, w.nparts, a->s0, sn, true, s->st, &s->launches));
    SEQ_CU(w.rows_of(s, a, g, {w.q, w.k, w.v, w.states(), false, false, o, ldo, a->hv, nullptr, {nullptr, nullptr}}));
    return ZSOLVE_OK;
}

int zsolve_decay_step(zsolve_seq *s, const zsolve_decay_args *a, void *o, int64_t ldo, float *sn) {
    if (!s) return ZSOLVE_EINVAL;
    zs::DecayGeom g;
    int st = check_decay(s, a, o, ldo, &g);
    if (st != ZSOLVE_OK || a->nseq == 0) return st;
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    SEQ_CU(zs_launch_decay_step(a->type, g, a->offsets, a->s0, o, ldo, sn, s->st, &s->launches));
    return ZSOLVE_OK;
}

int zsolve_decay_bwd(zsolve_seq *s, const zsolve_decay_args *a, const void *dout, int64_t lddo, const float *ds, void *dq, void *dk,
                     void *dv, float *dg, float *ds0) {
    if (!s) return ZSOLVE_EINVAL;
    zs::DecayGeom g;
    int st = check_decay(s, a, dout, lddo, &g);
    if (st != ZSOLVE_OK) return st;
    if ((a->tokens > 0 && (!dq || !dk || !dv || !dg)) || (a->ldg == 0 && !dg)) return seq_fail(s, ZSOLVE_EINVAL, "NULL dq, dk, dv or dg");
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    if (a->nseq == 0 || a->tokens == 0) {  // sums over nothing, and the states' gradients as they are
        const size_t states = (size_t)a->nseq * a->hv * a->dk * a->dv * sizeof(float);
        if (a->ldg == 0) SEQ_CU(cudaMemsetAsync(dg, 0, (size_t)a->hv * sizeof(float), s->st));
        if (ds0 && states && ds0 != ds) {
            if (ds)
                SEQ_CU(cudaMemcpyAsync(ds0, ds, states, cudaMemcpyDeviceToDevice, s->st));
            else
                SEQ_CU(cudaMemsetAsync(ds0, 0, states, s->st));
        }
        return ZSOLVE_OK;
    }
    DecayWork w;
    st = w.place(s, a, &g, dout, lddo, true, ds, ds0);
    if (st != ZSOLVE_OK) return st;
    SEQ_CU(w.sums_of(s, a, g, w.k, w.v, false, true, w.u));
    SEQ_CU(w.sums_of(s, a, g, w.q, w.dout, true, false, w.w));
    SEQ_CU(zs_launch_decay_scan(g, w.u, w.uplanes, w.nparts, a->s0, nullptr, true, s->st, &s->launches));
    SEQ_CU(zs_launch_decay_rscan(g, w.w, w.wplanes, w.nparts, w.u, w.uplanes, ds, ds0, w.dots, true, s->st, &s->launches));
    const int64_t rk = (int64_t)a->hk * a->dk, rv = (int64_t)a->hv * a->dv;
    SEQ_CU(w.rows_of(s, a, g, {w.dout, w.v, w.k, w.states(), true, false, dq, rk, a->hk, &w.q, {w.sums[0], w.sums[1]}}));
    SEQ_CU(w.rows_of(s, a, g, {w.v, w.dout, w.q, w.dstates(), true, true, dk, rk, a->hk, &w.k, {w.sums[2], w.sums[3]}}));
    SEQ_CU(w.rows_of(s, a, g, {w.k, w.q, w.dout, w.dstates(), false, true, dv, rv, a->hv, nullptr, {nullptr, nullptr}}));
    const float *const from_q[2] = {w.sums[0], w.sums[1]}, *const from_k[2] = {w.sums[2], w.sums[3]};
    SEQ_CU(zs_launch_decay_dg(g, from_q, from_k, w.dots, w.ndots, w.parts, dg, s->st, &s->launches));
    return ZSOLVE_OK;
}

int zsolve_delta_bwd(zsolve_seq *s, const zsolve_delta_args *a, const void *dout, int64_t lddo, const float *ds,
                     void *dq, void *dk, void *dv, float *dg, float *dbeta, float *ds0) {
    if (!s) return ZSOLVE_EINVAL;
    zs::DeltaGeom g;
    int st = check_delta(s, a, dout, lddo, &g);
    if (st != ZSOLVE_OK || a->nseq == 0) return st;
    if (a->tokens > 0 && (!dq || !dk || !dv || !dg || !dbeta))
        return seq_fail(s, ZSOLVE_EINVAL, "NULL dq, dk, dv, dg or dbeta");
    if (a->hv > 65535) return seq_fail(s, ZSOLVE_EINVAL, "hv = %d", a->hv);
    st = check_device(s);
    if (st != ZSOLVE_OK) return st;
    DeltaWork w;
    w.backward = true;
    w.dout = dout;
    w.lddo = lddo;
    st = w.place(s, a);
    if (st == ZSOLVE_OK) st = w.bind(s, a, &g);
    if (st != ZSOLVE_OK) return st;
    SEQ_CU(zs_launch_delta_plan(a->offsets, a->nseq, a->tokens, zs::kChunk, w.nchunks, w.first, w.seq, w.chunk, s->st, &s->launches));
    if (a->tokens > 0) SEQ_CU(zs_launch_delta_terms(a->type, g, w.terms, nullptr, 0, true, s->st, &s->launches));
    auto backwards = [&](bool next, cudaStream_t on) {
        return zs_launch_delta_rchain(a->type, g, w.terms, w.dout, w.lddo, ds, w.dends, w.dxs, dv, ds0, s->d_status, next, on,
                                      &s->launches);
    };
    // the states and U once more: keeping them from the forward pass would hold 96 KB a chunk and head
    // at 128 x 128 until the backward pass
    auto forwards = [&](bool next) {
        return zs_launch_delta_chain(a->type, g, w.terms, a->s0, nullptr, 0, nullptr, w.states, w.us, s->d_status, next, s->st,
                                     &s->launches);
    };
    if (a->tokens == 0) {
        SEQ_CU(backwards(true, s->st));
        return ZSOLVE_OK;
    }
    // The two recurrences do not need each other.  They run side by side where the SMs
    // hold both, a block each (24 blocks each, 4000 tokens, float32: 966 -> 640 us; 8 blocks,
    // 300 tokens: 81 -> 66), else one after the other (128 blocks each, 4096 tokens,
    // bfloat16: 1057 us side by side, 1043 so), as for a chunk or two, where the events
    // cost more (20 tokens: 56 us for 53).
    const bool both = 2 * delta_chain_blocks(g) <= s->num_sms && a->tokens > 2 * zs::kChunk;
    if (both) {
        SEQ_CU(cudaEventRecord(s->fork, s->st));
        SEQ_CU(cudaStreamWaitEvent(s->side, s->fork, 0));
        const cudaError_t e = backwards(false, s->side), e2 = forwards(false);
        // joined also after a failed launch: the workspace's next user comes after both
        SEQ_CU(cudaEventRecord(s->joined, s->side));
        SEQ_CU(cudaStreamWaitEvent(s->st, s->joined, 0));
        SEQ_CU(e);
        SEQ_CU(e2);
    } else {
        SEQ_CU(forwards(true));
        SEQ_CU(backwards(true, s->st));
    }
    SEQ_CU(zs_launch_delta_grads(a->type, g, w.terms, w.dout, w.lddo, w.states, w.dends, w.us, w.dxs, w.dqp, w.dkp, dq, dk,
                                 dv, dg, dbeta, s->num_sms, !both, s->st, &s->launches));
    return ZSOLVE_OK;
}

}  // extern "C"
