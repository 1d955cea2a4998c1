// The matrix product with its epilogue for a few rows of x, as in decoding:
// bound by reading the weight once.  A block owns 16 outputs and its eight warps
// a share of k each; a warp reads its weights straight into the fragments of
// m16n8k16 (weights as A, the rows of x as B), 16 bytes a lane: a lane's eight
// neighbours along k serve two steps, since any order of k serves as long as A
// and B agree.  The warps' partial sums meet in shared memory, so one launch does
// all of it, without tensor maps or a workspace.  One row, 4096 x 2048: 4.6 us with the
// weight in L2, 3.6 TB/s; 10.7 us from HBM, bound by the loads' latency.
#include <type_traits>

#include "linear.cuh"

namespace {

using namespace zs;

constexpr int kWarps = 8;
constexpr int kOut = 16;  // outputs of a block

template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, bf16>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight values of a row from column c on, of which those before k exist
template <bool VEC>
__device__ __forceinline__ uint4 row8(const uint16_t *p, int64_t c, int64_t k, bool in) {
    if (!in || c >= k) return make_uint4(0, 0, 0, 0);
    if (VEC && c + 8 <= k) return *reinterpret_cast<const uint4 *>(p + c);
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; i++) u[i] = c + i < k ? p[c + i] : 0;
    return make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
}

// NT: tiles of 8 rows of x; VEC: rows start on 16 bytes
template <typename T, int NT, bool VEC>
__global__ void __launch_bounds__(kWarps * 32)
k_linear_few(const uint16_t *__restrict__ x, int64_t ldx, const uint16_t *__restrict__ w, int64_t ldw, int m, int64_t n,
             int64_t k, const Epilogue epi) {
    __shared__ float part[kWarps][8 * NT][kOut + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t n0 = (int64_t)blockIdx.x * kOut;
    const bool in0 = n0 + g < n, in1 = n0 + g + 8 < n;
    const uint16_t *w0 = w + (in0 ? n0 + g : 0) * ldw, *w1 = w + (in1 ? n0 + g + 8 : 0) * ldw;
    const uint16_t *xr[NT];
    bool xin[NT];
#pragma unroll
    for (int j = 0; j < NT; j++) {
        xin[j] = j * 8 + g < m;
        xr[j] = x + (xin[j] ? j * 8 + g : 0) * ldx;
    }
    float acc[NT][4] = {};
    // 32 k a step; the warps take steps in turn, so that they read neighbouring memory
#pragma unroll 4
    for (int64_t c = warp * 32 + t * 8; c < (k + 31) / 32 * 32; c += kWarps * 32) {
        const uint4 a = row8<VEC>(w0, c, k, in0), b = row8<VEC>(w1, c, k, in1);
        const uint32_t a0[4] = {a.x, b.x, a.y, b.y}, a1[4] = {a.z, b.z, a.w, b.w};
#pragma unroll
        for (int j = 0; j < NT; j++) {
            const uint4 v = row8<VEC>(xr[j], c, k, xin[j]);
            mma16<T>(acc[j], a0, v.x, v.y);
            mma16<T>(acc[j], a1, v.z, v.w);
        }
    }
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) part[warp][j * 8 + 2 * t + (e & 1)][g + (e >> 1) * 8] = acc[j][e];
    __syncthreads();
    // output (row r of x, column n0 + c): a thread each
    for (int i = threadIdx.x; i < 8 * NT * kOut; i += kWarps * 32) {
        const int r = i / kOut, c = i - r * kOut;
        if (r >= m || n0 + c >= n) continue;
        float v[1] = {0.f};
#pragma unroll
        for (int q = 0; q < kWarps; q++) v[0] += part[q][r][c];
        const int64_t col = n0 + c;
        if (epi.bias) v[0] += to_f32(reinterpret_cast<const T *>(epi.bias)[col]);
        if (epi.z) reinterpret_cast<T *>(epi.z)[r * epi.ldz + col] = from_f32<T>(v[0]);
        act_all(v, epi.act);
        if (epi.r) v[0] += to_f32(reinterpret_cast<const T *>(epi.r)[r * epi.ldr + col]);
        reinterpret_cast<T *>(epi.y)[r * epi.ldy + col] = from_f32<T>(v[0]);
    }
}

template <typename T>
cudaError_t few(int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx, const void *w, int64_t ldw,
                const Epilogue &epi, cudaStream_t st) {
    const uint16_t *px = (const uint16_t *)x, *pw = (const uint16_t *)w;
    const bool vec = (((uintptr_t)x | (uintptr_t)w | (uint64_t)ldx * 2 | (uint64_t)ldw * 2) & 15) == 0;
    const unsigned grid = (unsigned)((n + kOut - 1) / kOut);
#define FEW_GO(NT, V) k_linear_few<T, NT, V><<<grid, kWarps * 32, 0, st>>>(px, ldx, pw, ldw, (int)m, n, k, epi)
    if (m <= 8) {
        if (vec) FEW_GO(1, true);
        else FEW_GO(1, false);
    } else {
        if (vec) FEW_GO(2, true);
        else FEW_GO(2, false);
    }
#undef FEW_GO
    return cudaGetLastError();
}

}  // namespace

cudaError_t zs_launch_linear_few(int type, int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx, const void *w,
                                 int64_t ldw, const Epilogue &epi, cudaStream_t st, int64_t *launches) {
    ++*launches;
    return type == ZSOLVE_BF16 ? few<bf16>(m, n, k, x, ldx, w, ldw, epi, st) : few<f16>(m, n, k, x, ldx, w, ldw, epi, st);
}
