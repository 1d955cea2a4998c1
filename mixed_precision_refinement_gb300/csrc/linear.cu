// The matrix product with bias, activation and residual in its epilogue, and
// its gradients (kernels and formulas in linear_tc.cuh).
#include "linear_tc.cuh"

namespace {

using namespace zs;

// dz = dy act'(z) into rows of stride ldo (a multiple of 8; NULL: not written)
// and, per block row, the columns' float32 sums of it before it is rounded
// (parts, one row of n a block row; NULL: not formed).  dz is rounded to the
// inputs' type because it is the tensor cores' operand: it adds one rounding
// of an input to each product's terms.  Bound by HBM: 8192 x 4096 bfloat16 in 45 us,
// 4.5 TB/s.
constexpr int kDzBlocks = 4;  // of an SM
template <typename T>
__global__ void __launch_bounds__(256, kDzBlocks)
k_linear_dz(const T *__restrict__ dy, int64_t lddy, const T *__restrict__ z, int64_t ldz, int act, int64_t m, int n,
            T *__restrict__ dz, int64_t ldo, float *__restrict__ parts, int vec) {
    __shared__ float red[8][32][9];
    after_previous();
    may_start_next();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = ((int64_t)blockIdx.x * 32 + tx) * 8;
    const int nc = (int)min((int64_t)8, (int64_t)n - c);
    float sum[8] = {};
    if (nc > 0) {
#pragma unroll 2
        for (int64_t row = (int64_t)blockIdx.y * 8 + ty; row < m; row += (int64_t)gridDim.y * 8) {
            float v[8], f[8];
            load8<T>(dy, row * lddy + c, nc, vec, v);
            if (z) {
                load8<T>(z, row * ldz + c, nc, vec, f);
#define SLOPE_CASE(A)                                                          \
    case A: {                                                                  \
        _Pragma("unroll") for (int i = 0; i < 8; i++) v[i] *= slope1<A>(f[i]); \
        break;                                                                 \
    }
                switch (act) {
                    SLOPE_CASE(ACT_RELU)
                    SLOPE_CASE(ACT_SILU)
                    SLOPE_CASE(ACT_GELU)
                    SLOPE_CASE(ACT_GELU_TANH)
                }
#undef SLOPE_CASE
            }
#pragma unroll
            for (int i = 0; i < 8; i++) {
                if (i >= nc) v[i] = 0.f;
                sum[i] += v[i];
            }
            if (dz) {
                Vec<T, 8> u;
                u.set(v);
                u.store(dz + row * ldo + c);
            }
        }
    }
    if (!parts) return;
#pragma unroll
    for (int i = 0; i < 8; i++) red[ty][tx][i] = sum[i];
    __syncthreads();
    // thread (ty, tx): column 8 tx + ty of the block's 256
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 8; r++) s += red[r][tx][ty];
    const int64_t col = ((int64_t)blockIdx.x * 32 + tx) * 8 + ty;
    if (col < n) parts[(int64_t)blockIdx.y * n + col] = s;
}

template <typename T>
int linear_fwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, Mat x, Mat w, const Epilogue &epi) {
    const Plan p = plan_of(m, n, k, s->num_sms);
    uint16_t *xp, *wp;
    float *part;
    int st = ZSOLVE_OK;
    auto carve = [&](void *base) {
        Carve c(base);
        xp = x.tma_ok() ? nullptr : c.take<uint16_t>(x.packed_values());
        wp = w.tma_ok() ? nullptr : c.take<uint16_t>(w.packed_values());
        part = p.splits > 1 ? c.take<float>(part_values(m, n, p)) : nullptr;
        return c.at;
    };
    const size_t bytes = carve(nullptr);
    if (bytes) {
        void *ws = seq_workspace(s, bytes, &st);
        if (!ws) return st;
        carve(ws);
    }
    const int64_t before = s->launches;
    SEQ_CU(packed(s, &x, xp, &w, wp, false));
    SEQ_CU(product<T>(s, type, Product{m, n, k, x, w, false, false, epi}, part, s->launches > before));
    return ZSOLVE_OK;
}

// Block rows of k_linear_dz, which are parts of db: as many blocks as the SMs hold at a time.
int dz_rows(int64_t m, int64_t n, int num_sms) {
    const int64_t most = std::max<int64_t>(1, (int64_t)num_sms * kDzBlocks / ((n + 255) / 256));
    return (int)std::min<int64_t>({(m + 7) / 8, most, 1024});
}

template <typename T>
int linear_bwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, Mat dy, Mat x, Mat w, int act, Mat z, void *dx,
               int64_t lddx, void *dw, int64_t lddw, void *db) {
    if (m == 0) {
        if (dw) SEQ_CU(cudaMemset2DAsync(dw, (size_t)lddw * 2, 0, (size_t)k * 2, (size_t)n, s->st));
        if (db) SEQ_CU(cudaMemsetAsync(db, 0, (size_t)n * 2, s->st));
        return ZSOLVE_OK;
    }
    const Plan px = plan_of(m, k, n, s->num_sms), pw = plan_of(n, k, m, s->num_sms);
    const bool has_act = act != ACT_NONE;
    const bool products = dx || dw;
    const bool form_dz = products && (has_act || !dy.tma_ok());
    const int dzrows = dz_rows(m, n, s->num_sms);
    const int64_t ldz8 = (n + 7) / 8 * 8;
    uint16_t *dzp = nullptr, *xp = nullptr, *wp = nullptr;
    float *part = nullptr, *sums = nullptr;
    int st = ZSOLVE_OK;
    auto carve = [&](void *base) {
        Carve c(base);
        dzp = form_dz ? c.take<uint16_t>((size_t)m * ldz8) : nullptr;
        xp = dw && !x.tma_ok() ? c.take<uint16_t>(x.packed_values()) : nullptr;
        wp = dx && !w.tma_ok() ? c.take<uint16_t>(w.packed_values()) : nullptr;
        const size_t parts = std::max(dx ? part_values(m, k, px) : 0, dw ? part_values(n, k, pw) : 0);
        part = parts ? c.take<float>(parts) : nullptr;
        sums = db ? c.take<float>((size_t)dzrows * n) : nullptr;
        return c.at;
    };
    const size_t bytes = carve(nullptr);
    if (bytes) {
        void *ws = seq_workspace(s, bytes, &st);
        if (!ws) return st;
        carve(ws);
    }
    const int64_t before = s->launches;
    if (form_dz || db) {
        const int vec = vec8(dy.p, dy.ld) && (!has_act || vec8(z.p, z.ld));
        k_linear_dz<T><<<dim3((unsigned)((n + 255) / 256), dzrows), 256, 0, s->st>>>(
            (const T *)dy.p, dy.ld, has_act ? (const T *)z.p : nullptr, z.ld, act, m, (int)n, (T *)dzp, ldz8, sums, vec);
        s->launches++;
        SEQ_CU(cudaGetLastError());
    }
    if (db) {
        s->launches++;
        SEQ_CU(launch(true, k_linear_db<T>, (unsigned)((n + 31) / 32), 256, 0, s->st, sums, dzrows, n, n, (T *)db, (T *)nullptr));
    }
    Mat dz = dy;
    if (form_dz) dz.p = dzp, dz.ld = ldz8;
    SEQ_CU(packed(s, &w, wp, &x, xp, s->launches > before));
    Product pr[2];
    int np = 0;
    if (dx) {
        Epilogue epi{};
        epi.y = dx, epi.ldy = lddx, epi.vec = vec8(dx, lddx);
        pr[np++] = Product{m, k, n, dz, w, false, true, epi};
    }
    if (dw) {
        Epilogue epi{};
        epi.y = dw, epi.ldy = lddw, epi.vec = vec8(dw, lddw);
        pr[np++] = Product{n, k, m, dz, x, true, true, epi};
    }
    if (np == 2 && px.pair && pw.pair) {
        SEQ_CU((launch_pair<T, PAIR_GRADS>(s, type, pr, s->launches > before)));
    } else {
        for (int i = 0; i < np; i++) SEQ_CU(product<T>(s, type, pr[i], part, s->launches > before));
    }
    return ZSOLVE_OK;
}

}  // namespace

int zs_linear(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx, const void *w,
              int64_t ldw, const void *b, int act, const void *r, int64_t ldr, void *y, int64_t ldy, void *z,
              int64_t ldz) {
    Epilogue epi{};
    epi.bias = b, epi.r = r, epi.y = y, epi.z = z;
    epi.ldr = ldr, epi.ldy = ldy, epi.ldz = ldz;
    epi.act = act;
    epi.vec = vec8(b, 0) && vec8(r, ldr) && vec8(y, ldy) && vec8(z, ldz);
    // One kernel for few rows, against a split product and its join.  4096 x 2048: 4.6 us
    // for 1 .. 8 rows, 6.6 for 16, against 10; 8192 x 4096: 16 and 19.7 against 18; rows
    // read value by value (1000 x 2157): 9.4 and 15.4 against 12.3.
    const bool aligned = Mat{x, m, k, ldx}.tma_ok() && Mat{w, n, k, ldw}.tma_ok();
    if (m <= 8 || (m <= kFewRows && aligned && n * k <= 1 << 24)) {
        SEQ_CU(zs_launch_linear_few(type, m, n, k, x, ldx, w, ldw, epi, s->st, &s->launches));
        return ZSOLVE_OK;
    }
    const Mat mx{x, m, k, ldx}, mw{w, n, k, ldw};
    return type == ZSOLVE_BF16 ? linear_fwd<bf16>(s, type, m, n, k, mx, mw, epi)
                               : linear_fwd<f16>(s, type, m, n, k, mx, mw, epi);
}

int zs_linear_bwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *dy, int64_t lddy,
                  const void *x, int64_t ldx, const void *w, int64_t ldw, int act, const void *z, int64_t ldz,
                  void *dx, int64_t lddx, void *dw, int64_t lddw, void *db) {
    const Mat md{dy, m, n, lddy}, mx{x, m, k, ldx}, mw{w, n, k, ldw}, mz{z, m, n, ldz};
    return type == ZSOLVE_BF16
               ? linear_bwd<bf16>(s, type, m, n, k, md, mx, mw, act, mz, dx, lddx, dw, lddw, db)
               : linear_bwd<f16>(s, type, m, n, k, md, mx, mw, act, mz, dx, lddx, dw, lddw, db);
}
