// The gated feed-forward projections and their gradients:
//   zg = x Wg^T + bg, zu = x Wu^T + bu, y = act(zg) zu         x: m x k, Wg, Wu: n x k
//   dzg = dy zu act'(zg), dzu = dy act(zg)
//   dx = dzg Wg + dzu Wu, dWg = dzg^T x, dWu = dzu^T x, db: the sums of dz over the rows
// Forward, both products are one launch: an output tile is 128 (or 64) columns of each, side by
// side in one accumulator, and the epilogue multiplies what it reads (linear_tc.cuh).  Nothing
// but y is written unless zg and zu are kept.  Backward, dzg and dzu are the halves of one
// matrix, so that dx is one sum over both and dW one product with the rows of both.  16384 x 8192 x 4096 bfloat16: 1187 us alone,
// 1345 to 1380 back to back under the power limit (1635 to 1590 TFLOP/s); backwards 8192 x 4096 x 2048 390 to 404 us, 307 of them the products.
#include "linear_tc.cuh"

namespace {

using namespace zs;

// dzg and dzu into the halves of a matrix of rows of 2 nz values (NULL: not written), zeros from
// column n to the next multiple of 64 (they are factors of dx's sums), and per block row the
// columns' float32 sums before the rounding (parts, 2 n a block row; NULL: not formed).  The
// rounding to the inputs' type, which the tensor cores need, adds one of an input's size.  8192 x 4096 bfloat16: 53 us, 5.4 TB/s (two
// blocks an SM 62, four 59; an exponential each for the gate and its slope 94).
constexpr int kDzBlocks = 3;  // of an SM
template <typename T>
__global__ void __launch_bounds__(256, kDzBlocks)
k_glu_dz(const T *__restrict__ dy, int64_t lddy, const T *__restrict__ zg, int64_t ldzg, const T *__restrict__ zu, int64_t ldzu,
         int act, int64_t m, int n, T *__restrict__ dz, int64_t nz, float *__restrict__ parts, int vec) {
    __shared__ float red[2][8][32][9];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = ((int64_t)blockIdx.x * 32 + tx) * 8;
    const int nc = (int)min((int64_t)8, (int64_t)n - c);
    float2 sg[4] = {}, su[4] = {};
    // behind the last column d is zero, and with it everything
    auto one = [&](int64_t row, const float (&d)[8], float (&g)[8], float (&u)[8]) {
        float a[8], s[8];
        gates_all<true>(g, act, a, s);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 di = make_float2(d[i], d[i + 1]);
            const float2 x = mul2(mul2(di, make_float2(u[i], u[i + 1])), make_float2(s[i], s[i + 1])), y = mul2(di, make_float2(a[i], a[i + 1]));
            g[i] = x.x, g[i + 1] = x.y, u[i] = y.x, u[i + 1] = y.y;
            sg[i / 2] = add2(sg[i / 2], x), su[i / 2] = add2(su[i / 2], y);
        }
        if (!dz) return;
        Vec<T, 8> w;
        w.set(g);
        w.store(dz + row * 2 * nz + c);
        w.set(u);
        w.store(dz + row * 2 * nz + nz + c);
    };
    const int64_t first = (int64_t)blockIdx.y * 8 + ty, step = (int64_t)gridDim.y * 8;
    if (vec && nc == 8) {
#pragma unroll 2
        for (int64_t row = first; row < m; row += step) {
            Vec<T, 8> vd, vg, vu;
            vd.load(dy + row * lddy + c), vg.load(zg + row * ldzg + c), vu.load(zu + row * ldzu + c);
            float d[8], g[8], u[8];
            vd.get(d), vg.get(g), vu.get(u);
            one(row, d, g, u);
        }
    } else if (c < (n + 63) / 64 * 64) {
#pragma unroll 1
        for (int64_t row = first; row < m; row += step) {
            float d[8] = {}, g[8] = {}, u[8] = {};
            if (nc > 0) {
                load8<T>(dy, row * lddy + c, nc, 0, d);
                load8<T>(zg, row * ldzg + c, nc, 0, g);
                load8<T>(zu, row * ldzu + c, nc, 0, u);
            }
            one(row, d, g, u);
        }
    }
    if (!parts) return;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        red[0][ty][tx][2 * i] = sg[i].x, red[0][ty][tx][2 * i + 1] = sg[i].y;
        red[1][ty][tx][2 * i] = su[i].x, red[1][ty][tx][2 * i + 1] = su[i].y;
    }
    __syncthreads();
    // thread (ty, tx): column 8 tx + ty of the block's 256, of both
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int r = 0; r < 8; r++) a += red[0][r][tx][ty], b += red[1][r][tx][ty];
    const int64_t col = ((int64_t)blockIdx.x * 32 + tx) * 8 + ty;
    if (col < n) parts[(int64_t)blockIdx.y * 2 * n + col] = a, parts[((int64_t)blockIdx.y * 2 + 1) * n + col] = b;
}

// The parts of a forward product split along k, added in order, and the epilogue.
template <typename T>
__global__ void __launch_bounds__(256)
k_glu_join(int64_t M, int64_t N, int splits, const GluEpilogue epi) {
    after_previous();
    may_start_next();
    const int64_t groups = (N + 7) / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= M * groups) return;
    const int64_t row = i / groups, c = (i - row * groups) * 8;
    float v[2][8] = {};
    for (int s = 0; s < splits; s++) {
        const float *q = epi.part + ((int64_t)s * M + row) * 2 * epi.ldp + c;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const float4 *p = reinterpret_cast<const float4 *>(q + h * epi.ldp);
            const float4 a = p[0], b = p[1];
            v[h][0] += a.x, v[h][1] += a.y, v[h][2] += a.z, v[h][3] += a.w;
            v[h][4] += b.x, v[h][5] += b.y, v[h][6] += b.z, v[h][7] += b.w;
        }
    }
    glu_finish8<T>(epi, row, c, (int)min((int64_t)8, N - c), v[0], v[1]);
}

// ---------------------------------------------------------------- host

template <typename T, bool TURN>
cudaError_t launch_pair_fwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const Mat &x, const Mat &wg, const Mat &wu,
                            const GluEpilogue &epi, bool next) {
    constexpr int smem = kPairSmem + (TURN ? kTurn : 0);
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_linear_pair<T, PAIR_GLU_FWD, TURN>, smem);
    if (attr != cudaSuccess) return attr;
    CUtensorMap ma, mb;
    GluMore more{};
    cudaError_t e = encode(&ma, type, x.p, x.rows, x.cols, x.ld, BM);
    if (e == cudaSuccess) e = encode(&mb, type, wg.p, wg.rows, wg.cols, wg.ld, 128);
    if (e == cudaSuccess) e = encode(&more.b2, type, wu.p, wu.rows, wu.cols, wu.ld, 128);
    if (e != cudaSuccess) return e;
    const int64_t total = (m + 2 * BM - 1) / (2 * BM) * ((n + 127) / 128);
    s->launches++;
    return launch(next, k_linear_pair<T, PAIR_GLU_FWD, TURN>, 2 * (unsigned)std::min<int64_t>(total, s->num_sms / 2), kThreads, smem,
                  s->st, ma, mb, m, n, (int)((k + BK - 1) / BK), epi, PairSecond{}, s->d_status, more);
}

template <typename T>
int glu_fwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, Mat x, Mat wg, Mat wu, GluEpilogue epi) {
    const Plan p = plan_of(m, 2 * n, k, s->num_sms);
    uint16_t *xp, *gp, *up;
    float *part;
    int st = ZSOLVE_OK;
    auto carve = [&](void *base) {
        Carve c(base);
        xp = x.tma_ok() ? nullptr : c.take<uint16_t>(x.packed_values());
        gp = wg.tma_ok() ? nullptr : c.take<uint16_t>(wg.packed_values());
        up = wu.tma_ok() ? nullptr : c.take<uint16_t>(wu.packed_values());
        part = p.splits > 1 ? c.take<float>((size_t)p.splits * m * 2 * ld_part(n)) : nullptr;
        return c.at;
    };
    const size_t bytes = carve(nullptr);
    if (bytes) {
        void *ws = seq_workspace(s, bytes, &st);
        if (!ws) return st;
        carve(ws);
    }
    const int64_t before = s->launches;
    SEQ_CU(packed(s, &x, xp, &wg, gp, false, &wu, up));
    const bool next = s->launches > before;
    if (p.pair) {
        if (turned(epi))
            SEQ_CU((launch_pair_fwd<T, true>(s, type, m, n, k, x, wg, wu, epi, next)));
        else
            SEQ_CU((launch_pair_fwd<T, false>(s, type, m, n, k, x, wg, wu, epi, next)));
        return ZSOLVE_OK;
    }
    CUtensorMap ma, mb;
    GluMore more{};
    SEQ_CU(encode(&ma, type, x.p, x.rows, x.cols, x.ld, BM));
    SEQ_CU(encode(&mb, type, wg.p, wg.rows, wg.cols, wg.ld, 64));
    SEQ_CU(encode(&more.b2, type, wu.p, wu.rows, wu.cols, wu.ld, 64));
    epi.part = part;
    epi.ldp = ld_part(n);
    if (turned(epi))
        SEQ_CU((launch_tc<T, false, false, true, GLU_FWD>(ma, mb, m, n, p, epi, next, s, more)));
    else
        SEQ_CU((launch_tc<T, false, false, false, GLU_FWD>(ma, mb, m, n, p, epi, next, s, more)));
    if (p.splits == 1) return ZSOLVE_OK;
    const int64_t n8 = m * ((n + 7) / 8);
    s->launches++;
    SEQ_CU(launch(true, k_glu_join<T>, (unsigned)((n8 + 255) / 256), 256, 0, s->st, m, n, p.splits, epi));
    return ZSOLVE_OK;
}

template <typename T>
int glu_bwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, Mat dy, Mat x, Mat wg, Mat wu, int act, Mat zg, Mat zu,
            void *dx, int64_t lddx, void *dwg, int64_t lddwg, void *dwu, int64_t lddwu, void *dbg, void *dbu) {
    const bool dw = dwg || dwu, db = dbg || dbu;
    if (m == 0) {
        if (dwg) SEQ_CU(cudaMemset2DAsync(dwg, (size_t)lddwg * 2, 0, (size_t)k * 2, (size_t)n, s->st));
        if (dwu) SEQ_CU(cudaMemset2DAsync(dwu, (size_t)lddwu * 2, 0, (size_t)k * 2, (size_t)n, s->st));
        if (dbg) SEQ_CU(cudaMemsetAsync(dbg, 0, (size_t)n * 2, s->st));
        if (dbu) SEQ_CU(cudaMemsetAsync(dbu, 0, (size_t)n * 2, s->st));
        return ZSOLVE_OK;
    }
    if (!dx && !dw && !db) return ZSOLVE_OK;
    // a tile of dW has rows of one half: 256 in pairs of SMs
    const int64_t kfirst = (n + BK - 1) / BK;
    Plan pw = plan_of(2 * ((n + 255) / 256 * 256), k, m, s->num_sms);
    const int64_t nz = pw.pair ? (n + 255) / 256 * 256 : (n + 127) / 128 * 128;
    if (!pw.pair) pw = plan_of(2 * nz, k, m, s->num_sms);  // fewer tiles: pairs no more than before
    const Plan px = plan_of(m, k, 2 * kfirst * BK, s->num_sms);
    const int64_t per = (n + 255) / 256;
    const int dzrows = (int)std::min<int64_t>({(m + 7) / 8, std::max<int64_t>(1, (int64_t)s->num_sms * kDzBlocks / per), 1024});
    uint16_t *dzp = nullptr, *xp = nullptr, *gp = nullptr, *up = nullptr;
    float *part = nullptr, *sums = nullptr;
    int st = ZSOLVE_OK;
    auto carve = [&](void *base) {
        Carve c(base);
        dzp = dx || dw ? c.take<uint16_t>((size_t)m * 2 * nz) : nullptr;
        xp = dw && !x.tma_ok() ? c.take<uint16_t>(x.packed_values()) : nullptr;
        gp = dx && !wg.tma_ok() ? c.take<uint16_t>(wg.packed_values()) : nullptr;
        up = dx && !wu.tma_ok() ? c.take<uint16_t>(wu.packed_values()) : nullptr;
        const size_t parts = std::max(dx ? part_values(m, k, px) : 0, dw ? part_values(2 * nz, k, pw) : 0);
        part = parts ? c.take<float>(parts) : nullptr;
        sums = db ? c.take<float>((size_t)dzrows * 2 * n) : nullptr;
        return c.at;
    };
    void *ws = seq_workspace(s, carve(nullptr), &st);
    if (!ws) return st;
    carve(ws);
    const int vec = vec8(dy.p, dy.ld) && vec8(zg.p, zg.ld) && vec8(zu.p, zu.ld);
    k_glu_dz<T><<<dim3((unsigned)per, dzrows), 256, 0, s->st>>>((const T *)dy.p, dy.ld, (const T *)zg.p, zg.ld, (const T *)zu.p, zu.ld,
                                                                 act, m, (int)n, (T *)dzp, nz, sums, vec);
    s->launches++;
    SEQ_CU(cudaGetLastError());
    if (db) {
        s->launches++;
        SEQ_CU(launch(true, k_linear_db<T>, (unsigned)((2 * n + 31) / 32), 256, 0, s->st, sums, dzrows, 2 * n, n, (T *)dbg, (T *)dbu));
    }
    if (!dx && !dw) return ZSOLVE_OK;
    SEQ_CU(packed(s, &wg, gp, &wu, up, true, &x, xp));
    const Mat dz{dzp, m, 2 * nz, 2 * nz};
    GluMore more{};
    more.rows = n;
    more.apart = (int)nz;
    more.kfirst = (int)kfirst;
    Product pdx{m, k, 2 * kfirst * BK, dz, wg, false, true, {}}, pdw{2 * nz, k, m, dz, x, true, true, {}};
    if (dx) {
        pdx.epi.y = dx, pdx.epi.ldy = lddx, pdx.epi.vec = vec8(dx, lddx);
        SEQ_CU(encode(&more.b2, type, wu.p, wu.rows, wu.cols, wu.ld, 64));
    }
    if (dw) {
        // one of the two alone: the other's rows are formed and left
        pdw.epi.y = dwg, pdw.epi.ldy = lddwg, pdw.epi.vec = vec8(dwg, lddwg) && vec8(dwu, lddwu);
        more.second = pdw.epi;
        more.second.y = dwu, more.second.ldy = lddwu;
    }
    if (dx && dw && px.pair && pw.pair) {
        const Product two[2] = {pdx, pdw};
        SEQ_CU((launch_pair<T, PAIR_GLU_GRADS>(s, type, two, true, more)));
        return ZSOLVE_OK;
    }
    CUtensorMap ma, mb;
#define GLU_TC(AM, BMN, G, Q, P)                                                                        \
    do {                                                                                                \
        if (turned((Q).epi) || ((G) == GLU_DW && turned(more.second)))                                  \
            SEQ_CU((launch_tc<T, AM, BMN, true, G>(ma, mb, (Q).M, (Q).N, P, (Q).epi, true, s, more)));   \
        else                                                                                            \
            SEQ_CU((launch_tc<T, AM, BMN, false, G>(ma, mb, (Q).M, (Q).N, P, (Q).epi, true, s, more)));  \
    } while (0)
    auto join = [&](const Epilogue &epi, int64_t rows, int splits, int64_t apart) {
        const int64_t n8 = rows * ((k + 7) / 8);
        s->launches++;
        return launch(true, k_linear_join<T>, (unsigned)((n8 + 255) / 256), 256, 0, s->st, rows, k, splits, apart, epi);
    };
    if (dx && px.pair) {
        SEQ_CU((launch_pair<T, PAIR_GLU_DX>(s, type, &pdx, true, more)));
    } else if (dx) {
        SEQ_CU(maps(type, pdx, &ma, &mb));
        pdx.epi.part = px.splits > 1 ? part : nullptr;
        pdx.epi.ldp = ld_part(k);
        GLU_TC(false, true, GLU_DX, pdx, px);
        if (px.splits > 1) SEQ_CU(join(pdx.epi, m, px.splits, m));
    }
    if (dw && pw.pair) {
        SEQ_CU((launch_pair<T, PAIR_GLU_DW>(s, type, &pdw, true, more)));
    } else if (dw) {
        SEQ_CU(maps(type, pdw, &ma, &mb));
        pdw.epi.part = more.second.part = pw.splits > 1 ? part : nullptr;
        pdw.epi.ldp = more.second.ldp = ld_part(k);
        GLU_TC(true, true, GLU_DW, pdw, pw);
        if (pw.splits > 1) {
            more.second.part += nz * ld_part(k);
            if (dwg) SEQ_CU(join(pdw.epi, n, pw.splits, 2 * nz));
            if (dwu) SEQ_CU(join(more.second, n, pw.splits, 2 * nz));
        }
    }
#undef GLU_TC
    return ZSOLVE_OK;
}

}  // namespace

int zs_glu(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx, const void *wg, int64_t ldwg,
           const void *wu, int64_t ldwu, const void *bg, const void *bu, int act, void *y, int64_t ldy, void *zg, int64_t ldzg,
           void *zu, int64_t ldzu) {
    GluEpilogue epi{};
    epi.bg = bg, epi.bu = bu, epi.y = y, epi.zg = zg, epi.zu = zu;
    epi.ldy = ldy, epi.ldzg = ldzg, epi.ldzu = ldzu;
    epi.act = act;
    epi.vec = vec8(bg, 0) && vec8(bu, 0) && vec8(y, ldy) && vec8(zg, ldzg) && vec8(zu, ldzu);
    const Mat mx{x, m, k, ldx}, mg{wg, n, k, ldwg}, mu{wu, n, k, ldwu};
    const bool aligned = mx.tma_ok() && mg.tma_ok() && mu.tma_ok();
    // Few rows: one kernel that reads each weight once and waits for its loads, against tiles of 128 rows.  The small kernel and the tiles at
    // 16 rows, bfloat16, weights from HBM, us: 1024 x 1024 6.5 and 8.0, 2048 x 2048 11.1 and 10.3, 4096 x 2048 12.7 and 14.1,
    // 4096 x 4096 22.1 and 17.9 (9 rows: 21.3 and 22.7), 8192 x 4096 43.2 and 29.6.
    if (m <= 8 || (m <= kFewRows && aligned && n * k <= 1 << 23)) {
        SEQ_CU(zs_launch_glu_few(type, m, n, k, x, ldx, wg, ldwg, wu, ldwu, epi, s->st, &s->launches));
        return ZSOLVE_OK;
    }
    return type == ZSOLVE_BF16 ? glu_fwd<bf16>(s, type, m, n, k, mx, mg, mu, epi) : glu_fwd<f16>(s, type, m, n, k, mx, mg, mu, epi);
}

int zs_glu_bwd(zsolve_seq *s, int type, int64_t m, int64_t n, int64_t k, const void *dy, int64_t lddy, const void *x, int64_t ldx,
               const void *wg, int64_t ldwg, const void *wu, int64_t ldwu, int act, const void *zg, int64_t ldzg, const void *zu,
               int64_t ldzu, void *dx, int64_t lddx, void *dwg, int64_t lddwg, void *dwu, int64_t lddwu, void *dbg, void *dbu) {
    const Mat md{dy, m, n, lddy}, mx{x, m, k, ldx}, mg{wg, n, k, ldwg}, mu{wu, n, k, ldwu}, mzg{zg, m, n, ldzg}, mzu{zu, m, n, ldzu};
    return type == ZSOLVE_BF16
               ? glu_bwd<bf16>(s, type, m, n, k, md, mx, mg, mu, act, mzg, mzu, dx, lddx, dwg, lddwg, dwu, lddwu, dbg, dbu)
               : glu_bwd<f16>(s, type, m, n, k, md, mx, mg, mu, act, mzg, mzu, dx, lddx, dwg, lddwg, dwu, lddwu, dbg, dbu);
}
