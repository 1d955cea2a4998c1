// Linear attention with a decay for each head on the 5th-generation tensor cores, bfloat16 (formulas and
// geometry in decay.cuh): the spans' sums of outer products, and the products of rows.
//
// A bfloat16 input is an exact operand.  What is float32 goes in bfloat16 parts that add up to it:
// three (24 bits) where the result is float32 (the states, and what the gradients of the decays are summed from),
// two (16 bits, 2^-17 of a term) where it is rounded to bfloat16 right after.  The tensor cores
// cut their sums instead of rounding, so a float32 result's sums are short (8 steps), small parts
// apart or first, and join the others by float32 additions.
//
// Every mbarrier wait is bounded: on give-up the kernel raises the handle's status word, stops all
// roles, waits (bounded) for its own copies and MMAs and frees TMEM.
#include <algorithm>

#include "decay.cuh"
#include "tcgen05.cuh"

namespace {

using namespace zs;

constexpr int kRow = 128;  // bytes of a swizzled row: 64 values

// Place of the 16 bytes `c` (of 8) of row r in a box of swizzled rows.
__device__ __forceinline__ uint32_t swizzled(int r, int c) { return (uint32_t)(r * kRow + ((c ^ (r & 7)) << 4)); }

// Whether one of eight bfloat16 values is an infinity or NaN: its exponent and one more carry into the sign's place.
__device__ __forceinline__ bool not_finite8(uint4 u) {
    const uint32_t m = 0x7f807f80u, one = 0x00800080u;
    return ((((u.x & m) + one) | ((u.y & m) + one) | ((u.z & m) + one) | ((u.w & m) + one)) & 0x80008000u) != 0;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 2^x, results below 2^-126 flushed to zero
__device__ __forceinline__ float exp2_flush(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two values in two bfloat16 parts each
__device__ __forceinline__ void split2(float2 v, uint32_t &hi, uint32_t &lo) {
    hi = pack2<bf16>(v.x, v.y);
    const float2 r = fma2(unpack2<bf16>(hi), make_float2(-1.f, -1.f), v);
    lo = pack2<bf16>(r.x, r.y);
}
__device__ __forceinline__ void load4(const float *p, float2 &a, float2 &b) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    a = make_float2(v.x, v.y), b = make_float2(v.z, v.w);
}

// ---------------------------------------------------------------- sums

// U = sum over a span's tokens of w_j x_j y_j^T, 128 x 128 in TMEM.  x's tiles of 64 tokens are scaled and split in
// three parts by eight warps, in shared memory, where they are the MN-major A operand (the large part in the tile's own
// place); y's are the B operand as TMA leaves them.  Two accumulators, one for the small parts; after 128 tokens both are
// added to the float32 sums in the warps' registers.  Two blocks an SM, so that one's
// conversions run beside the other's products.  32768 tokens x 32 heads of 128 x 128 in spans of 512: 204 us, the tensor pipe busy
// 19 % of the time; what a chunk waits for is the way from its tile over its parts to the products, and two blocks are what
// shared memory holds.
constexpr int kSumWorkers = 256, kSumThreads = kSumWorkers + 32;
constexpr int kSumChunk = 64;
constexpr uint32_t kSumBox = kSumChunk * kRow, kSumTile = 2 * kSumBox;
constexpr uint32_t kSumSmem = kSumTile * 6 + 1024;  // two stages of x and y, two small parts

__global__ void __launch_bounds__(kSumThreads, 2)
k_decay_sums_tc(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap ymap, const DecayGeom geo, int xcols, int ycols,
                int xkey, int ykey, int query, int gates, float *__restrict__ out, unsigned *__restrict__ status) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_in[2], bar_parts, bar_used, bar_acc, bar_acc_free, bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ float2 s_b[kSpanMost];
    __shared__ float s_w[kSpanMost];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int span = blockIdx.x, hv = blockIdx.y, c0 = blockIdx.z * 128;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sx = base, sy = base + 2 * kSumTile, sp_ = base + 4 * kSumTile;
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 2; i++) bar_init(&bar_in[i], 1);
        bar_init(&bar_parts, kSumWorkers / 32);
        bar_init(&bar_used, 1);
        bar_init(&bar_acc, 1);
        bar_init(&bar_acc_free, kSumWorkers / 32);
        bar_init(&bar_drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(256) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    after_previous();
    may_start_next();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    const int2 sp = geo.d.chunk[span];
    const int n = sp.y, group = geo.d.hv / geo.d.hk, hk = hv / group;
    const int chunks = (n + kSumChunk - 1) / kSumChunk, xboxes = (xcols + 63) / 64, yboxes = min(2, (ycols - c0 + 63) / 64);
    auto load = [&](int i) {  // by one thread: chunk i into its stage
        const uint32_t bar = smem_u32(&bar_in[i & 1]);
        bar_expect(&bar_in[i & 1], (uint32_t)(xboxes + yboxes) * kSumBox);
        for (int b = 0; b < xboxes; b++)
            tma_load_3d(sx + (i & 1) * kSumTile + b * kSumBox, &xmap, b * 64, xkey ? hk : hv, sp.x + i * kSumChunk, bar);
        for (int b = 0; b < yboxes; b++)
            tma_load_3d(sy + (i & 1) * kSumTile + b * kSumBox, &ymap, c0 + b * 64, ykey ? hk : hv, sp.x + i * kSumChunk, bar);
    };
    if (tid == kSumWorkers) {
        for (int i = 0; i < min(2, chunks); i++) load(i);
        for (int i = 2; i < chunks; i++) {  // the others on their way to L2
            for (int b = 0; b < xboxes; b++) tma_prefetch_3d(&xmap, b * 64, xkey ? hk : hv, sp.x + i * kSumChunk);
            for (int b = 0; b < yboxes; b++) tma_prefetch_3d(&ymap, c0 + b * 64, ykey ? hk : hv, sp.x + i * kSumChunk);
        }
    }
    if (tid < kSumWorkers) decay_loads(geo, sp, hv, s_b, tid, kSumWorkers);
    __syncthreads();
    if (warp == 0 && n > 0) decay_sums(sp, s_b);
    __syncthreads();
    if (tid < kSumWorkers && n > 0) {
        const float2 last = s_b[n - 1];
        for (int i = tid; i < chunks * kSumChunk; i += kSumWorkers)
            s_w[i] = i >= n ? 0.f : query ? geo.d.scale * decay_exp(s_b[i], make_float2(0.f, 0.f)) : decay_exp(last, s_b[i]);
        if (gates && blockIdx.z == 0) {
            for (int i = tid; i < n; i += kSumWorkers) geo.gates[((int64_t)span * geo.d.hv + hv) * geo.span + i] = s_b[i];
            if (tid == 0) geo.ends[(int64_t)span * geo.d.hv + hv] = decay_exp(last, make_float2(0.f, 0.f));
        }
        if (xboxes == 1) {  // the rows beyond x's columns: zeros in all parts
            for (int i = tid; i < 4 * (int)kSumBox / 16; i += kSumWorkers) {
                const uint32_t tile = (uint32_t)(i / ((int)kSumBox / 16)), at = (uint32_t)(i % ((int)kSumBox / 16)) * 16;
                sts128((tile < 2 ? sx + tile * kSumTile : sp_ + (tile - 2) * kSumTile) + kSumBox + at, make_uint4(0, 0, 0, 0));
            }
        }
    }
    __syncthreads();
    if (warp == 8) {  // the whole warp, uniformly
        int loaded = min(2, chunks);
        const uint32_t idesc = f16_idesc<bf16>(128, yboxes * 64, true, true);
        auto wait = [&](uint64_t *bar, int phase) { return __all_sync(0xffffffffu, bar_wait(bar, phase & 1, &s_abort, status)); };
#pragma unroll 1
        for (int i = 0; i < chunks; i++) {
            if (!wait(&bar_parts, i)) break;
            const bool first = !(i & 1);
            if (first && !wait(&bar_acc_free, (i >> 1) + 1)) break;
            tc_fence_after();
            const uint64_t y = smem_desc<true>(sy + (i & 1) * kSumTile, kSumBox);
            // the small parts, smallest first, then the large one
#pragma unroll
            for (int part = 2; part >= 0; part--) {
                const uint64_t x = smem_desc<true>(part ? sp_ + (part - 1) * kSumTile : sx + (i & 1) * kSumTile, kSumBox);
#pragma unroll
                for (int ks = 0; ks < kSumChunk / 16; ks++)
                    mma_f16_warp(tmem + (part ? 128u : 0u), x + 128 * ks, y + 128 * ks, idesc, !first || ks || part == 1 ? 1u : 0u);
            }
            if (!first || i + 1 == chunks) mma_commit_warp(smem_u32(&bar_acc));
            mma_commit_warp(smem_u32(&bar_used));
            if (i + 2 >= chunks) continue;
            if (!wait(&bar_used, i)) break;
            if (lane == 0) load(i + 2);
            loaded = i + 3;
        }
        mma_commit_warp(smem_u32(&bar_drain));
        for (uint32_t w = 0; w < kWaitLimit && !__all_sync(0xffffffffu, bar_try(&bar_drain, 0)); w++) {
        }
        for (int i = std::max(0, loaded - 2); i < loaded; i++)  // the copies in flight
            for (uint32_t w = 0; w < kWaitLimit && !__all_sync(0xffffffffu, bar_try(&bar_in[i & 1], (i >> 1) & 1)); w++) {
            }
    } else {
        const int quad = warp & 3, half = warp >> 2;
        float acc[64];
#pragma unroll
        for (int e = 0; e < 64; e++) acc[e] = 0.f;
        const int row = quad * 32 + lane, cols = yboxes * 32;  // a thread's columns: its half
        for (int i = 0; i < chunks; i++) {
            if (!bar_wait(&bar_in[i & 1], (i >> 1) & 1, &s_abort, status)) break;
            if (!bar_wait(&bar_used, (i & 1) ^ 1, &s_abort, status)) break;
            const int rest = n - i * kSumChunk;
            const uint32_t xb = sx + (i & 1) * kSumTile;
            for (int j = tid; j < kSumChunk * 8 * xboxes; j += kSumWorkers) {
                const int c = j & 7, b = xboxes == 2 ? (j >> 3) & 1 : 0, r = xboxes == 2 ? j >> 4 : j >> 3;
                const uint32_t at = b * kSumBox + swizzled(r, c);
                const uint4 u = lds128(xb + at);
                const float w = s_w[i * kSumChunk + r];
                const uint32_t in[4] = {u.x, u.y, u.z, u.w};
                uint32_t p0[4], p1[4], p2[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    float2 f = mul2(unpack2<bf16>(in[e]), make_float2(w, w));
                    if (r >= rest) f = make_float2(0.f, 0.f);
                    p0[e] = pack2<bf16>(f.x, f.y);
                    split2(fma2(unpack2<bf16>(p0[e]), make_float2(-1.f, -1.f), f), p1[e], p2[e]);
                }
                sts128(xb + at, make_uint4(p0[0], p0[1], p0[2], p0[3]));
                sts128(sp_ + at, make_uint4(p1[0], p1[1], p1[2], p1[3]));
                sts128(sp_ + kSumTile + at, make_uint4(p2[0], p2[1], p2[2], p2[3]));
            }
            // what lies behind the span meets zeros of x, and must be finite
            for (int j = tid; j < (kSumChunk - rest) * 8 * yboxes; j += kSumWorkers) {
                const int c = j & 7, b = (j >> 3) % yboxes, r = rest + (j >> 3) / yboxes;
                sts128(sy + (i & 1) * kSumTile + b * kSumBox + swizzled(r, c), make_uint4(0, 0, 0, 0));
            }
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(&bar_parts);
            if ((i & 1) || i + 1 == chunks) {
                if (!__all_sync(0xffffffffu, bar_wait(&bar_acc, (i >> 1) & 1, &s_abort, status))) break;
                tc_fence_after();
                const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16) + half * cols;
#pragma unroll
                for (int c = 0; c < 64; c += 16) {
                    if (c >= cols) break;
                    float hi[16], lo[16];
                    tmem_ld16(at + c, hi);
                    tmem_ld16(at + 128 + c, lo);
#pragma unroll
                    for (int e = 0; e < 16; e++) acc[c + e] += hi[e] + lo[e];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&bar_acc_free);
            }
        }
        if (n > 0 && row < xcols) {
            const int first = c0 + half * cols;
            float *p = out + (((int64_t)span * geo.d.hv + hv) * xcols + row) * ycols + first;
            const bool vec = ycols % 4 == 0;  // 16 bytes
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                if (c >= cols || first + c >= ycols) break;
                if (vec)
                    *reinterpret_cast<float4 *>(p + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
                else
                    for (int e = 0; e < 4; e++)
                        if (first + c + e < ycols) p[c + e] = acc[c + e];
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(256) : "memory");
}

// ---------------------------------------------------------------- rows

// The products of rows, 128 rows i of one head at a time, against the span's tokens 128 at a time:
//   S = X Y^T in TMEM; the warps read it, mask and weigh it, and put it back in two bfloat16 parts, in its
//   place, as the A operand of O += P Z; the state's share X M comes first and, scaled in TMEM, is what O starts from.
// What a step waits for is the way from one product over the weights to the next, so two of them are on their way at a time:
// two events of one block of threads, or two blocks of threads an SM.
constexpr int kTile = 128;
constexpr uint32_t kBoxBytes = kTile * kRow, kTileBytes = 2 * kBoxBytes;
constexpr int kRowThreads = 64 + 512;
constexpr int kRing = 4;

struct RowsTc {
    int xcols, ncols;      // columns of x and y, and of z
    int xkey, ykey, zkey;  // heads are key heads
    int turned, back, parts;
    bf16 *out;
    int64_t ldo;
    int vec;               // stores of 16 (1) or 32 bytes (2)
    float *sums[2];
};

struct Item {
    int span, rb, head, c0;  // which of the span's blocks of rows
    int2 sp;
    int n, tiles, live;    // tokens and their blocks; whether there is anything to do
};
// Quotients by a divisor of up to 2^31, of dividends below 2^31: a multiplication (2^(31 + l) / d rounded up, 2^l >= d, is off by
// less than 1 / d of a quotient).
struct FastDiv {
    uint32_t d, mul, shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t n) : d(n), mul(0), shift(31) {
        while ((1ull << (shift - 31)) < n) shift++;
        mul = (uint32_t)(((1ull << shift) + n - 1) / n);
    }
    __device__ __forceinline__ int div(int i) const { return (int)(((uint64_t)(uint32_t)i * mul) >> shift); }
};
struct Items {
    FastDiv heads, zblocks, per;  // `per` items a span and head
    int total;
    template <bool UNIFORM = false>  // for a whole warp, which then keeps it in uniform registers
    __device__ __forceinline__ Item at(const DecayGeom &geo, int i) const {
        Item x;
        if (i >= total) {
            x.span = x.rb = x.head = x.c0 = x.n = x.tiles = x.live = 0, x.sp = make_int2(0, 0);
            return x;
        }
        int j = heads.div(i);
        x.head = i - j * (int)heads.d;
        i = j, j = zblocks.div(i);
        x.c0 = (i - j * (int)zblocks.d) * 128;
        x.span = per.div(j);
        x.rb = j - x.span * (int)per.d;
        x.sp = geo.d.chunk[x.span];
        if (UNIFORM) x.sp.x = __shfl_sync(0xffffffffu, x.sp.x, 0), x.sp.y = __shfl_sync(0xffffffffu, x.sp.y, 0);
        x.n = x.sp.y;
        x.tiles = (x.n + kTile - 1) / kTile;
        x.live = x.rb < x.tiles;
        return x;
    }
};

// A warp's share of zeros in the results of the tokens outside the sequences.
__device__ __forceinline__ void zero_outside(const DecayGeom &geo, const RowsTc &p, const Item &x, int warp, int warps) {
    const int used = geo.d.first[geo.d.nseq], workers = (geo.d.nchunks - used) * warps, worker = (x.span - used) * warps + warp;
    const int2 last = geo.d.seq[geo.d.nseq - 1];
    bf16 *o = p.out + (int64_t)x.head * p.ncols + x.c0;
    const int cols = min(128, p.ncols - x.c0);
    zero_tokens(o, p.ldo, 0, geo.d.seq[0].x, cols, worker, workers);
    zero_tokens(o, p.ldo, (int64_t)last.x + last.y, geo.d.tokens, cols, worker, workers);
}

// `boxes` times 64 along k of a product of two tiles: operands K-major (a box a 64) or MN-major (16 k values 2048 bytes apart).  The
// columns beyond a head's are zeros.
template <bool MN>
__device__ __forceinline__ uint64_t tile_desc(uint32_t tile) { return smem_desc<MN>(tile, kBoxBytes); }
template <bool B_MN>
__device__ __forceinline__ void mma_tiles(uint32_t d, uint32_t a, uint32_t b, int boxes, uint32_t idesc, bool more) {
    uint64_t da = tile_desc<false>(a), db = tile_desc<B_MN>(b);
    uint32_t acc = more ? 1u : 0u;
#pragma unroll 1
    for (int i = 0; i < boxes; i++) {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            mma_f16_warp(d, da + 2 * k, db + (B_MN ? 128 : 2) * k, idesc, acc);
            acc = 1u;
        }
        da += kBoxBytes >> 4;
        db += B_MN ? 512 : kBoxBytes >> 4;
    }
}
// O += P Z over a block's tokens, P in its two parts
__device__ __forceinline__ void mma_weights(uint32_t o, uint32_t p, uint32_t z, uint32_t idesc) {
    uint64_t dz = tile_desc<true>(z);
#pragma unroll 1
    for (int i = 0; i < 2; i++, p += 64, dz += 512)
#pragma unroll
        for (int k = 0; k < 4; k++) {
            mma_f16_ta_warp(o, p + k * 16, dz + 128 * k, idesc, 1u);
            mma_f16_ta_warp(o, p + k * 16 + 8, dz + 128 * k, idesc, 1u);
        }
}

// All of `THREADS` threads (whole warps) wait for each other; whether one of them says so.
template <int THREADS>
__device__ __forceinline__ bool group_or(bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)x), "n"(THREADS)
                 : "memory");
    return r != 0;
}

// A tile of Z looked over by `threads` threads (this is thread t): rows from `rest` on, behind the span, become zeros.  On the
// diagonal, an infinity or NaN would meet the zeros of the rows that the mask keeps from it: it is taken out, and its column's
// entry of `bad` has the first such row (or, back, the last one), `token` (if any) that of all columns.
__device__ __forceinline__ void look_over(uint32_t tile, int boxes, int rest, bool diag, bool back, volatile int *bad, volatile int *any,
                                          volatile int *token, int t, int threads) {
    bool wrote = false;
    for (int j = t; j < kTile * 8 * boxes; j += threads) {
        const int c = j & 7, b = boxes == 2 ? (j >> 3) & 1 : 0, rr = boxes == 2 ? j >> 4 : j >> 3;
        const uint32_t at = tile + b * kBoxBytes + swizzled(rr, c);
        if (rr >= rest) {
            sts128(at, make_uint4(0, 0, 0, 0));
            wrote = true;
            continue;
        }
        if (!diag) continue;
        const uint4 u = lds128(at);
        if (!not_finite8(u)) continue;
        wrote = true;
        uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if (((w[e >> 1] >> (16 * (e & 1))) & 0x7f80u) != 0x7f80u) continue;
            w[e >> 1] &= e & 1 ? 0xffffu : 0xffff0000u;
            int *to = const_cast<int *>(bad + b * 64 + c * 8 + e), *tok = const_cast<int *>(token);
            back ? atomicMax(to, rr) : atomicMin(to, rr);
            if (tok) back ? atomicMax(tok, rr) : atomicMin(tok, rr);
        }
        *any = 1;
        sts128(at, make_uint4(w[0], w[1], w[2], w[3]));
    }
    if (wrote) fence_async();
}

// Weights of 16 tokens from j on for a row, in pairs: for each of its own, or both factors across the border.
struct RowWeights {
    float2 r, h, l, scale;  // the row's factor, its sum in two floats, each twice
    __device__ __forceinline__ RowWeights(const RowsTc &p, float ri, float2 bi, float sc) {
        r = make_float2(ri, ri), scale = make_float2(sc, sc);
        h = p.back ? make_float2(-bi.x, -bi.x) : make_float2(bi.x, bi.x);
        l = p.back ? make_float2(-bi.y, -bi.y) : make_float2(bi.y, bi.y);
    }
    __device__ __forceinline__ void get(bool each, const float *bh, const float *bl, const float *c, float2 (&w)[8]) const {
        if (each) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float2 h0, h1, l0, l1;
                load4(bh + 2 * e, h0, h1);
                load4(bl + 2 * e, l0, l1);
                h0 = add2(add2(h, h0), add2(l, l0)), h1 = add2(add2(h, h1), add2(l, l1));
                w[e] = mul2(make_float2(exp2_flush(h0.x), exp2_flush(h0.y)), scale);
                w[e + 1] = mul2(make_float2(exp2_flush(h1.x), exp2_flush(h1.y)), scale);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                load4(c + 2 * e, w[e], w[e + 1]);
                w[e] = mul2(w[e], r), w[e + 1] = mul2(w[e + 1], r);
            }
        }
    }
};

// 16 values of a row of results, columns c .. c + 15, of which those below `cols` are there; vec: of 32 or 16 bytes.  A warp's
// store is 32 rows, and what it takes is a pass a row.
__device__ __forceinline__ void put_row(bf16 *o, int c, int cols, int vec, const float (&v)[16]) {
    uint32_t u[8];
#pragma unroll
    for (int e = 0; e < 8; e++) u[e] = pack2<bf16>(v[2 * e], v[2 * e + 1]);
    if (vec == 2 && c + 16 <= cols) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o + c), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]),
                     "r"(u[5]), "r"(u[6]), "r"(u[7])
                     : "memory");
        return;
    }
#pragma unroll
    for (int h = 0; h < 16; h += 8) {
        if (vec && c + h + 8 <= cols) {
            *reinterpret_cast<uint4 *>(o + c + h) = make_uint4(u[h / 2], u[h / 2 + 1], u[h / 2 + 2], u[h / 2 + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++)
                if (c + h + e < cols) o[c + h + e] = from_f32<bf16>(v[h + e]);
        }
    }
}

// With SELF (dq and dk): the value heads that share out's key head one after the other, whose gradients add up in O, and
// beside S the other scores S2 = self Z^T, for the sums of pairs.  One block of threads an SM, sixteen warps, a quarter of a row a
// thread.  Its events, a state's share or a block of tokens each, use two places for S in turn: the next one's product is
// under way while this one's weights are found; S2 has one place and follows once it is read.  2 x 4096 tokens x 32 heads (16 key heads)
// of 128: 142 us, the tensor pipe busy 21 %: the way from an event to the next.  TMEM has no room for a second block beside
// its 512 columns.
constexpr uint32_t kSelfSmem = kTileBytes * (2 + kRing) + 1024;

__global__ void __launch_bounds__(kRowThreads, 1)
k_decay_rows_self(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap ymap, const __grid_constant__ CUtensorMap zmap,
                  const __grid_constant__ CUtensorMap mmap, const __grid_constant__ CUtensorMap qmap, const DecayGeom geo, const RowsTc p,
                  const Items items, unsigned *__restrict__ status) {
    extern __shared__ uint8_t smem_raw[];
    // Two each, in turn, where one warp may be a phase ahead of another: with one barrier, its second arrival would count for the
    // first phase, and a warp that looks for a phase when the next is over too would wait for ever.  No warp is two phases ahead.
    __shared__ __align__(8) uint64_t bar_x, bar_x_free, bar_full[kRing], bar_empty[kRing], bar_s, bar_p, bar_pv[2], bar_checked[2], bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    // sums b_j in two floats, negative where time runs forwards: the exponent of a row i and a token j is the sum of theirs;
    // and the weights of the tokens outside the rows' own block, up to its border
    __shared__ __align__(16) float s_bh[kSpanMost], s_bl[kSpanMost], s_c[kSpanMost];
    __shared__ volatile int s_bad[128], s_anybad, s_badtok;
    __shared__ int s_exact;
    __shared__ float s_dot[4][2][kTile];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u, sx = base, sq = base + kTileBytes, ring = base + 2 * kTileBytes;
    if (tid == 0) {
        s_abort = 0;
        bar_init(&bar_x, 1), bar_init(&bar_x_free, 1 + 16);
        for (int i = 0; i < kRing; i++) bar_init(&bar_full[i], 1), bar_init(&bar_empty[i], 1);
        bar_init(&bar_s, 1), bar_init(&bar_p, 16), bar_init(&bar_drain, 1);
        for (int i = 0; i < 2; i++) bar_init(&bar_checked[i], 16), bar_init(&bar_pv[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    after_previous();
    may_start_next();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0), t_s2 = tmem + 256, t_o = tmem + 384;  // two places of S, then S2 and O
    const int group = geo.d.hv / geo.d.hk, xboxes = (p.xcols + 63) / 64;
    const int zboxes = (p.ncols + 63) / 64, mboxes = p.turned ? xboxes : zboxes;
    auto first_jb = [&](const Item &x) { return p.back ? x.rb : 0; };
    auto end_jb = [&](const Item &x) { return p.back ? x.tiles : x.rb + 1; };
    auto checked = [&](const Item &x, int jb) { return jb == x.rb || (jb + 1) * kTile > x.n; };

    if (warp == 0) {
        // ------------------------------------------------ TMA
        if (lane == 0) {
            uint32_t q = 0, cx = 0;
            bool ok = true;
            auto load = [&](uint32_t to, const CUtensorMap *map, int boxes, int c, int h, int row, uint64_t *bar) {
                for (int b = 0; b < boxes; b++) tma_load_3d(to + b * kBoxBytes, map, c + b * 64, h, row, smem_u32(bar));
            };
            auto next = [&](const CUtensorMap *map, int boxes, int h, int row) {
                const uint32_t st = q % kRing;
                ok = ok && bar_wait(&bar_empty[st], ((q / kRing) & 1u) ^ 1u, &s_abort, status);
                if (!ok) return;
                bar_expect(&bar_full[st], (uint32_t)boxes * kBoxBytes);
                load(ring + st * kTileBytes, map, boxes, 0, h, row, &bar_full[st]);
                q++;
            };
            // a round's tiles on their way to L2 while the one before is at work
            auto prefetch = [&](const Item &x, int r) {
                if (!x.live) return;
                const int hv = x.head * group + r;
                auto ask = [&](const CUtensorMap *map, int boxes, int h, int row) {
                    for (int b = 0; b < boxes; b++) tma_prefetch_3d(map, b * 64, h, row);
                };
                for (int part = 0; part < 3; part++) ask(&mmap, mboxes, 0, (x.span * geo.d.hv + hv) * 3 + part);
                ask(&xmap, xboxes, p.xkey ? x.head : hv, x.sp.x + x.rb * kTile);
                ask(&qmap, zboxes, x.head, x.sp.x + x.rb * kTile);
                for (int jb = first_jb(x); jb < end_jb(x); jb++) {
                    ask(&ymap, xboxes, p.ykey ? x.head : hv, x.sp.x + jb * kTile);
                    ask(&zmap, zboxes, p.zkey ? x.head : hv, x.sp.x + jb * kTile);
                }
            };
            for (int it = blockIdx.x; ok && it < items.total; it += gridDim.x) {
                const Item x = items.at(geo, it);
                if (!x.live) continue;
                for (int r = 0; ok && r < group; r++) {
                    if (r + 1 < group)
                        prefetch(x, r + 1);
                    else
                        prefetch(items.at(geo, it + gridDim.x), 0);
                    const int hv = x.head * group + r;
                    auto head_of = [&](int key) { return key ? x.head : hv; };
                    for (int part = 0; part < 3; part++) next(&mmap, mboxes, 0, (x.span * geo.d.hv + hv) * 3 + part);
                    for (int jb = first_jb(x); ok && jb < end_jb(x); jb++) {
                        next(&ymap, xboxes, head_of(p.ykey), x.sp.x + jb * kTile);
                        if (jb == first_jb(x)) {  // x's place is free later than the ring's
                            ok = ok && bar_wait(&bar_x_free, (cx & 1u) ^ 1u, &s_abort, status);
                            if (!ok) break;
                            bar_expect(&bar_x, (uint32_t)(xboxes + zboxes) * kBoxBytes);
                            load(sx, &xmap, xboxes, 0, head_of(p.xkey), x.sp.x + x.rb * kTile, &bar_x);
                            load(sq, &qmap, zboxes, 0, x.head, x.sp.x + x.rb * kTile, &bar_x);
                            cx++;
                        }
                        next(&zmap, zboxes, head_of(p.zkey), x.sp.x + jb * kTile);
                    }
                }
            }
            // the copies in flight: wait (bounded) for the last of each
            for (uint32_t i = q > (uint32_t)kRing ? q - kRing : 0; i < q; i++)
                for (uint32_t w = 0; w < kWaitLimit && !bar_try(&bar_full[i % kRing], (i / kRing) & 1u); w++) {
                }
            for (uint32_t w = 0; cx && w < kWaitLimit && !bar_try(&bar_x, (cx - 1) & 1u); w++) {
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (the whole warp, uniformly)
        uint32_t cx = 0, ck = 0, cp = 0, cpv = 0, e = 0;  // e: events issued
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t count) {
            ok = ok && __all_sync(0xffffffffu, bar_wait(bar, count & 1u, &s_abort, status));
            tc_fence_after();
            return ok;
        };
        auto tile = [&](uint32_t i) { return ring + i % kRing * kTileBytes; };
        auto arrived = [&](uint32_t i) { return wait(&bar_full[i % kRing], i / kRing); };
        auto free = [&](uint32_t i) { mma_commit_warp(smem_u32(&bar_empty[i % kRing])); };
        const uint32_t id_s = f16_idesc<bf16>(128, 128, false, false), id_o = f16_idesc<bf16>(128, zboxes * 64, false, true);
        const uint32_t id_m = f16_idesc<bf16>(128, p.turned ? 128 : zboxes * 64, false, !p.turned);
        uint32_t m = 0;  // the round's first tile
        Item x = items.at<true>(geo, blockIdx.x);
        for (int it = blockIdx.x; ok && it < items.total; it += gridDim.x) {
            const Item after = items.at<true>(geo, it + gridDim.x);
            const int first = first_jb(x), end = end_jb(x);
            for (int r = 0; ok && x.live && r < group; r++) {
                // the state's share, the smallest part first
                if (!wait(&bar_x, cx++)) break;
                if (!arrived(m) || !arrived(m + 1) || !arrived(m + 2)) break;
#pragma unroll 1
                for (int part = 2; part >= 0; part--)
                    if (p.turned)
                        mma_tiles<false>(tmem + (e & 1) * 128, sx, tile(m + part), xboxes, id_m, part < 2);
                    else
                        mma_tiles<true>(tmem + (e & 1) * 128, sx, tile(m + part), xboxes, id_m, part < 2);
                free(m), free(m + 1), free(m + 2);
                mma_commit_warp(smem_u32(&bar_s));
                e++;
                bool block = false;  // the event before is one of tokens: its P Z is to come
                for (int jb = first; ok && jb <= end; jb++) {
                    const uint32_t y = m + 3 + 2 * (jb - first), z = y + 1;
                    if (jb < end) {  // the next scores beside the last event's weights
                        if (!arrived(y)) break;
                        mma_tiles<false>(tmem + (e & 1) * 128, sx, tile(y), xboxes, id_s, false);
                        free(y);
                    }
                    if (!wait(&bar_p, cp++)) break;  // the last event is read, or its P there
                    if (jb < end) {
                        if (!arrived(z)) break;
                        if (checked(x, jb)) {
                            if (!wait(&bar_checked[ck & 1], ck >> 1)) break;
                            ck++;
                        }
                        mma_tiles<false>(t_s2, sq, tile(z), zboxes, id_s, false);
                        if (jb + 1 == end) mma_commit_warp(smem_u32(&bar_x_free));
                        mma_commit_warp(smem_u32(&bar_s));
                    }
                    if (block) {
                        const uint32_t t_p = tmem + ((e - 1) & 1) * 128, zp = z - 2;
                        mma_weights(t_o, t_p, tile(zp), id_o);
                        free(zp);
                        mma_commit_warp(smem_u32(&bar_pv[cpv & 1]));
                        // its place is the next but one event's
                        if (!wait(&bar_pv[cpv & 1], cpv >> 1)) break;
                        cpv++;
                    }
                    block = true;
                    if (jb < end) e++;
                }
                m += 3 + 2 * (end - first);
            }
            x = after;
        }
        // every MMA issued so far completes before TMEM is freed
        mma_commit_warp(smem_u32(&bar_drain));
        for (uint32_t w = 0; w < kWaitLimit && !__all_sync(0xffffffffu, bar_try(&bar_drain, 0)); w++) {
        }
    } else {
        // ------------------------------------------------ weights and results (warps 2-17)
        const int quad = warp & 3, quarter = (warp - 2) >> 2, et = tid - 64;
        const int row = quad * 32 + lane, hcols = zboxes * 16;  // a thread's columns of O
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        uint32_t m = 0, e = 0, cpv = 0, cx = 0, ck = 0;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t count) {
            ok = ok && __all_sync(0xffffffffu, bar_wait(bar, count & 1u, &s_abort, status));
            tc_fence_after();
            return ok;
        };
        auto arrive = [&](uint64_t *bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar);
        };
        const float2 zero = make_float2(0.f, 0.f);
        float2 ahead = zero;  // the next round's sums
        auto fetch = [&](const Item &x, int r) {
            if (x.live && et < x.tiles * kTile)
                ahead = geo.gates[((int64_t)x.span * geo.d.hv + x.head * group + r) * geo.span + min(et, x.n - 1)];
        };
        Item x = items.at(geo, blockIdx.x), after = x;
        fetch(x, 0);
        int it = blockIdx.x, r = 0;
        // a round each: a value head of an item
        for (; it < items.total; r + 1 < group && x.live ? r++ : (r = 0, it += gridDim.x, x = after, 0)) {
            if (r == 0) after = items.at(geo, it + gridDim.x);
            if (!x.live) {
                if (x.n == 0 && x.rb == 0) zero_outside(geo, p, x, warp - 2, 16);
                fetch(after, 0);
                continue;
            }
            const int n = x.n, rb = x.rb, i0 = rb * kTile, i = i0 + row, i1 = min(i0 + kTile, n) - 1, hv = x.head * group + r;
            const int first = first_jb(x), end = end_jb(x);
            if (group_or<512>(!ok)) break;  // and the last round's sums are read
            if (et < x.tiles * kTile) s_bh[et] = p.back ? ahead.x : -ahead.x, s_bl[et] = p.back ? ahead.y : -ahead.y;
            if (r == 0 && et < 128) s_bad[et] = p.back ? -1 : kTile;
            if (et == 0) {
                s_exact = 0;
                if (r == 0) s_anybad = 0, s_badtok = p.back ? -1 : kTile;
            }
            group_or<512>(false);
            if (r + 1 < group)
                fetch(x, r + 1);
            else
                fetch(after, 0);
            auto sum = [&](int j) { return p.back ? make_float2(s_bh[j], s_bl[j]) : make_float2(-s_bh[j], -s_bl[j]); };
            // weights across the border of the rows: both factors of a decay are at most 1; where they grow beyond float32
            // (positive g), every weight is found for itself
            const float2 border = p.back ? sum(i1) : i0 ? sum(i0 - 1) : zero, bi = sum(min(i, n - 1));
            if (et < x.tiles * kTile && (p.back ? et > i1 : et < i0)) {
                const float c = et >= n ? 0.f : p.back ? decay_exp(sum(et), border) : decay_exp(border, sum(et));
                s_c[et] = c;
                if (isinf(c)) s_exact = 1;
            }
            const float ri = geo.d.scale * (p.back ? decay_exp(border, bi) : decay_exp(bi, border));
            if (i < n && isinf(ri)) s_exact = 1;
            const float f = p.back ? decay_exp(sum(n - 1), bi) : geo.d.scale * decay_exp(bi, zero);
            group_or<512>(false);
            const bool exact = s_exact;
            const RowWeights weights(p, ri, bi, geo.d.scale);
            float dot = 0.f, pair = 0.f;
            // ---------------------------------------- the state's share
            if (wait(&bar_x, cx++) && wait(&bar_s, e)) {
#pragma unroll 1
                for (int c = quarter * hcols; c < (quarter + 1) * hcols; c += 16) {
                    float v[16];
                    tmem_ld16(tmem + (e & 1) * 128 + lanes + c, v);
#pragma unroll
                    for (int k = 0; k < 16; k++) v[k] *= f;
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int cc = c + 8 * h;
                        const uint4 q = lds128(sq + (cc >> 6) * kBoxBytes + swizzled(row, (cc >> 3) & 7));
                        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const float2 s = unpack2<bf16>(w[k]);
                            dot = fmaf(v[8 * h + 2 * k], s.x, fmaf(v[8 * h + 2 * k + 1], s.y, dot));
                        }
                    }
                    if (r > 0) {
                        float o[16];
                        tmem_ld16(t_o + lanes + c, o);
#pragma unroll
                        for (int k = 0; k < 16; k++) v[k] += o[k];
                    }
                    uint32_t u[16];
#pragma unroll
                    for (int k = 0; k < 16; k++) u[k] = __float_as_uint(v[k]);
                    tmem_st16(t_o + lanes + c, u);
                }
                tmem_wait_st();
                arrive(&bar_p);
                if (lane == 0) bar_arrive(&bar_x_free);  // self's rows are read
            }
            e++;
            // ---------------------------------------- the span's tokens
            for (int jb = first; ok && jb < end; jb++, e++) {
                const int j0 = jb * kTile, rest = n - j0;
                const bool diag = jb == rb;
                if (checked(x, jb)) {
                    // the tile before it in its place has arrived: it is one of the state's, or one that S2 was formed from, and the
                    // warps have waited for those products
                    const uint32_t z = m + 4 + 2 * (jb - first);
                    if (!wait(&bar_full[z % kRing], z / kRing)) break;
                    look_over(ring + z % kRing * kTileBytes, zboxes, rest, diag, p.back, s_bad, &s_anybad, &s_badtok, et, 512);
                    arrive(&bar_checked[ck++ & 1]);
                }
                if (!wait(&bar_s, e)) break;
                // the row's tokens of this block: of 128 columns those below `to`, and from `from` on
                const int last = min(rest, kTile), from = diag && p.back ? row : 0, to = diag && !p.back ? min(row + 1, last) : last;
                const uint32_t t_s = tmem + (e & 1) * 128 + lanes;
#pragma unroll 1
                for (int c = quarter * 32; c < quarter * 32 + 32; c += 16) {
                    float v[16], s2[16];
                    float2 w[8];
                    tmem_ld16(t_s + c, v);
                    tmem_ld16(t_s2 + lanes + c, s2);
                    weights.get(diag || exact, s_bh + j0 + c, s_bl + j0 + c, s_c + j0 + c, w);
                    uint32_t u[16];
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        w[k] = mul2(make_float2(v[2 * k], v[2 * k + 1]), w[k]);
                        // the mask, and the columns behind the span, whose scores may be anything
                        const int a = c + 2 * k, b = a + 1;
                        if (a < from || a >= to) w[k].x = 0.f, s2[2 * k] = 0.f;
                        if (b < from || b >= to) w[k].y = 0.f, s2[2 * k + 1] = 0.f;
                        // a step's 16 tokens: eight columns of the large parts, eight of the small ones, where the scores were
                        split2(w[k], u[k], u[8 + k]);
                        if (!diag || a != row) pair = fmaf(w[k].x, s2[2 * k], pair);
                        if (!diag || b != row) pair = fmaf(w[k].y, s2[2 * k + 1], pair);
                    }
                    tmem_st16(t_s + c, u);
                }
                tmem_wait_st();
                arrive(&bar_p);
                // every phase of the products in turn: the one before this block's
                if (jb > first) {
                    if (!wait(&bar_pv[cpv & 1], cpv >> 1)) break;
                    cpv++;
                }
            }
            m += 3 + 2 * (end - first);
            s_dot[quarter][0][row] = dot, s_dot[quarter][1][row] = pair;
            if (ok) wait(&bar_pv[cpv & 1], cpv >> 1), cpv++;  // O is complete, up to this head
            group_or<512>(false);           // and every value that was taken out is known
            if (!ok) continue;
            const float nan = __int_as_float(0x7fc00000);
            if (quarter < 2 && i < n) {
                float v = (s_dot[0][quarter][row] + s_dot[1][quarter][row]) + (s_dot[2][quarter][row] + s_dot[3][quarter][row]);
                if (quarter == 1 && (p.back ? row < s_badtok : row > s_badtok)) v = nan;
                p.sums[quarter][(int64_t)(x.sp.x + i) * geo.d.hv + hv] = v;
            }
            if (r + 1 < group) continue;
            // ---------------------------------------- results
            bf16 *o = p.out + (int64_t)(x.sp.x + i) * p.ldo + (int64_t)x.head * p.ncols;
            const bool patch = s_anybad;
#pragma unroll 1
            for (int c = quarter * hcols; c < (quarter + 1) * hcols; c += 16) {
                float v[16];
                tmem_ld16(t_o + lanes + c, v);
                if (patch) {
#pragma unroll
                    for (int k = 0; k < 16; k++)
                        if (p.back ? row <= s_bad[c + k] : row >= s_bad[c + k]) v[k] = nan;
                }
                if (i < n) put_row(o, c, p.ncols, p.vec, v);
            }
            __syncwarp();
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Without SELF (o and dv): two blocks of threads an SM, of eight warps each, half a row a thread; their items are 128 rows of a span
// and head.  An item is a chain (the state's share, scores, weights, products, results), and each block has one at a time:
// what runs side by side is the two blocks' chains.  32768 tokens x 32 heads of 128 in spans of 512: 402 us.  One block of sixteen warps whose
// chains overlap by two places for S and O was slower: the call 778 us for 742 when both took spans of 256, backwards 675 for 656.
constexpr int kHalfThreads = 64 + 256;
constexpr int kHalfRing = 2;
constexpr uint32_t kRowsSmem = kTileBytes * (1 + kHalfRing) + 1024;

__global__ void __launch_bounds__(kHalfThreads, 2)
k_decay_rows_tc(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap ymap, const __grid_constant__ CUtensorMap zmap,
                const __grid_constant__ CUtensorMap mmap, const DecayGeom geo, const RowsTc p, const Items items, unsigned *__restrict__ status) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_x, bar_x_free, bar_full[kHalfRing], bar_empty[kHalfRing], bar_state[2], bar_s[2], bar_p[2], bar_pv, bar_o[2],
        bar_o_free[2], bar_checked[2], bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    // as above, of this item and the next; and what the diagonal's tile held, of an item, the next, and the one whose results are to leave
    __shared__ __align__(16) float s_bh[2][kSpanMost], s_bl[2][kSpanMost], s_c[2][kSpanMost];
    __shared__ volatile int s_bad[3][128], s_anybad[3], s_exact[3];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u, ring = base + kTileBytes;
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 2; i++) bar_init(&bar_o_free[i], 8), bar_init(&bar_p[i], 8), bar_init(&bar_checked[i], 8);
        for (int i = 0; i < kHalfRing; i++) bar_init(&bar_full[i], 1), bar_init(&bar_empty[i], 1);
        for (int i = 0; i < 2; i++) bar_init(&bar_state[i], 1), bar_init(&bar_s[i], 1), bar_init(&bar_o[i], 1);
        bar_init(&bar_x, 1), bar_init(&bar_x_free, 1), bar_init(&bar_pv, 1), bar_init(&bar_drain, 1);
        for (int i = 0; i < 3; i++) s_exact[i] = 0, s_anybad[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < 3 * 128; i += kHalfThreads) s_bad[i >> 7][i & 127] = p.back ? -1 : kTile;
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(256) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    after_previous();
    may_start_next();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);  // S and O of 128 columns
    const int group = geo.d.hv / geo.d.hk, xboxes = (p.xcols + 63) / 64;
    auto first_jb = [&](const Item &x) { return p.back ? x.rb : 0; };
    auto end_jb = [&](const Item &x) { return p.back ? x.tiles : x.rb + 1; };
    auto checked = [&](const Item &x, int jb) { return jb == x.rb || (jb + 1) * kTile > x.n; };
    auto zboxes_of = [&](const Item &x) { return (min(128, p.ncols - x.c0) + 63) / 64; };

    if (warp == 0) {
        // ------------------------------------------------ TMA
        if (lane == 0) {
            uint32_t q = 0, i = 0;
            bool ok = true;
            auto load = [&](uint32_t to, const CUtensorMap *map, int boxes, int c, int h, int row, uint64_t *bar) {
                bar_expect(bar, (uint32_t)boxes * kBoxBytes);
                for (int b = 0; b < boxes; b++) tma_load_3d(to + b * kBoxBytes, map, c + b * 64, h, row, smem_u32(bar));
            };
            auto next = [&](const CUtensorMap *map, int boxes, int c, int h, int row) {
                const uint32_t st = q % kHalfRing;
                ok = ok && bar_wait(&bar_empty[st], ((q / kHalfRing) & 1u) ^ 1u, &s_abort, status);
                if (!ok) return;
                load(ring + st * kTileBytes, map, boxes, c, h, row, &bar_full[st]);
                q++;
            };
            // an item's tiles on their way to L2 while the one before is at work: the ring alone holds too little of what HBM has to be
            // asked for in time
            auto prefetch = [&](const Item &x) {
                if (!x.live) return;
                const int zboxes = zboxes_of(x), mboxes = p.turned ? xboxes : zboxes, key = x.head / group;
                auto ask = [&](const CUtensorMap *map, int boxes, int c, int h, int row) {
                    for (int b = 0; b < boxes; b++) tma_prefetch_3d(map, c + b * 64, h, row);
                };
                const int plane = (x.span * geo.d.hv + x.head) * p.parts;
                for (int part = 0; part < 2; part++) ask(&mmap, mboxes, p.turned ? 0 : x.c0, p.turned ? x.c0 : 0, plane + part);
                ask(&xmap, xboxes, 0, p.xkey ? key : x.head, x.sp.x + x.rb * kTile);
                for (int jb = first_jb(x); jb < end_jb(x); jb++) {
                    ask(&ymap, xboxes, 0, p.ykey ? key : x.head, x.sp.x + jb * kTile);
                    ask(&zmap, zboxes, x.c0, p.zkey ? key : x.head, x.sp.x + jb * kTile);
                }
            };
            for (int it = blockIdx.x; ok && it < items.total; it += gridDim.x) {
                const Item x = items.at(geo, it);
                prefetch(items.at(geo, it + gridDim.x));
                if (!x.live) continue;
                const int zboxes = zboxes_of(x), mboxes = p.turned ? xboxes : zboxes, key = x.head / group;
                const int plane = (x.span * geo.d.hv + x.head) * p.parts;
                for (int part = 0; part < 2; part++) {
                    next(&mmap, mboxes, p.turned ? 0 : x.c0, p.turned ? x.c0 : 0, plane + part);
                    if (part) break;
                    ok = ok && bar_wait(&bar_x_free, (i & 1u) ^ 1u, &s_abort, status);
                    if (!ok) break;
                    load(base, &xmap, xboxes, 0, p.xkey ? key : x.head, x.sp.x + x.rb * kTile, &bar_x);
                    i++;
                }
                for (int jb = first_jb(x); ok && jb < end_jb(x); jb++) {
                    next(&ymap, xboxes, 0, p.ykey ? key : x.head, x.sp.x + jb * kTile);
                    next(&zmap, zboxes, x.c0, p.zkey ? key : x.head, x.sp.x + jb * kTile);
                }
            }
            // the copies in flight: wait (bounded) for the last of each
            for (uint32_t j = q > (uint32_t)kHalfRing ? q - kHalfRing : 0; j < q; j++)
                for (uint32_t w = 0; w < kWaitLimit && !bar_try(&bar_full[j % kHalfRing], (j / kHalfRing) & 1u); w++) {
                }
            for (uint32_t w = 0; i && w < kWaitLimit && !bar_try(&bar_x, (i - 1) & 1u); w++) {
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (the whole warp, uniformly)
        uint32_t ck = 0, k = 0;  // tiles looked over, blocks of tokens
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t count) {
            ok = ok && __all_sync(0xffffffffu, bar_wait(bar, count & 1u, &s_abort, status));
            tc_fence_after();
            return ok;
        };
        auto tile = [&](uint32_t j) { return ring + j % kHalfRing * kTileBytes; };
        auto arrived = [&](uint32_t j) { return wait(&bar_full[j % kHalfRing], j / kHalfRing); };
        auto free = [&](uint32_t j) { mma_commit_warp(smem_u32(&bar_empty[j % kHalfRing])); };
        const uint32_t id_s = f16_idesc<bf16>(128, 128, false, false);
        const uint32_t t_s = tmem, t_o = tmem + 128;
        uint32_t i = 0, m = 0;  // items, the item's first tile
        Item x = items.at<true>(geo, blockIdx.x);
        for (int it = blockIdx.x; ok && it < items.total; it += gridDim.x) {
            const Item after = items.at<true>(geo, it + gridDim.x);
            if (x.live) {
                const int first = first_jb(x), end = end_jb(x), zboxes = zboxes_of(x);
                const uint32_t id_o = f16_idesc<bf16>(128, zboxes * 64, false, true);
                const uint32_t id_m = f16_idesc<bf16>(128, p.turned ? 128 : zboxes * 64, false, !p.turned);
                // the state's share, the smaller part first
                if (!arrived(m + 1) || !arrived(m) || !wait(&bar_x, i)) break;
                if (i && !wait(&bar_o_free[(i - 1) & 1], (i - 1) >> 1)) break;  // O's last results are read
#pragma unroll 1
                for (int part = 1; part >= 0; part--)
                    if (p.turned)
                        mma_tiles<false>(t_o, base, tile(m + part), xboxes, id_m, part == 0);
                    else
                        mma_tiles<true>(t_o, base, tile(m + part), xboxes, id_m, part == 0);
                free(m), free(m + 1);
                mma_commit_warp(smem_u32(&bar_state[i & 1]));
                for (int jb = first; ok && jb < end; jb++, k++) {
                    const uint32_t y = m + 2 + 2 * (jb - first), z = y + 1;
                    if (k && !wait(&bar_pv, k - 1)) break;  // P's place is the scores'
                    if (!arrived(y)) break;
                    mma_tiles<false>(t_s, base, tile(y), xboxes, id_s, false);
                    mma_commit_warp(smem_u32(&bar_s[k & 1]));
                    free(y);
                    if (jb + 1 == end) mma_commit_warp(smem_u32(&bar_x_free));
                    if (!arrived(z)) break;
                    if (checked(x, jb)) {
                        if (!wait(&bar_checked[ck & 1], ck >> 1)) break;
                        ck++;
                    }
                    if (!wait(&bar_p[k & 1], k >> 1)) break;
                    mma_weights(t_o, t_s, tile(z), id_o);
                    mma_commit_warp(smem_u32(&bar_pv));
                    if (jb + 1 == end) mma_commit_warp(smem_u32(&bar_o[i & 1]));
                    free(z);
                }
                m += 2 + 2 * (end - first), i++;
            }
            x = after;
        }
        // every MMA issued so far completes before TMEM is freed
        mma_commit_warp(smem_u32(&bar_drain));
        for (uint32_t w = 0; w < kWaitLimit && !__all_sync(0xffffffffu, bar_try(&bar_drain, 0)); w++) {
        }
    } else {
        // ------------------------------------------------ weights and results (warps 2-9)
        const int quad = warp & 3, half = (warp - 2) >> 2, et = tid - 64;
        const int row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        uint32_t m = 0, k = 0, i = 0, ck = 0;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t count) {
            ok = ok && __all_sync(0xffffffffu, bar_wait(bar, count & 1u, &s_abort, status));
            tc_fence_after();
            return ok;
        };
        auto arrive = [&](uint64_t *bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar);
        };
        const float2 zero = make_float2(0.f, 0.f);
        // the next item's sums: of the thread's tokens, its row, the rows' border, and the last one
        constexpr int kTokens = kSpanMost / 256;
        float2 of_token[kTokens], of_row = zero, border = zero, last_sum = zero;
        auto fetch = [&](const Item &x) {
            if (!x.live) return;
            const float2 *g = geo.gates + ((int64_t)x.span * geo.d.hv + x.head) * geo.span;
            const int i0 = x.rb * kTile;
#pragma unroll
            for (int j = 0; j < kTokens; j++)
                if (et + 256 * j < x.tiles * kTile) of_token[j] = g[min(et + 256 * j, x.n - 1)];
            of_row = g[min(i0 + row, x.n - 1)];
            border = p.back ? g[min(i0 + kTile, x.n) - 1] : i0 ? g[i0 - 1] : zero;
            last_sum = g[x.n - 1];
        };
        // the results of an item whose products are done: item j
        auto results = [&](const Item &x, uint32_t j) {
            if (!wait(&bar_o[j & 1], j >> 1)) return;
            const int r = x.rb * kTile + row, cols = min(128, p.ncols - x.c0), hcols = zboxes_of(x) * 32;
            bf16 *o = p.out + (int64_t)(x.sp.x + r) * p.ldo + (int64_t)x.head * p.ncols + x.c0;
            const bool patch = s_anybad[j % 3];
#pragma unroll 1
            for (int c = half * hcols; c < (half + 1) * hcols; c += 16) {
                float v[16];
                tmem_ld16(tmem + 128 + lanes + c, v);
                if (patch) {
#pragma unroll
                    for (int e = 0; e < 16; e++)
                        if (p.back ? row <= s_bad[j % 3][c + e] : row >= s_bad[j % 3][c + e]) v[e] = __int_as_float(0x7fc00000);
                }
                if (r < x.n) put_row(o, c, cols, p.vec, v);
            }
            __syncwarp();
            arrive(&bar_o_free[j & 1]);
        };
        Item x = items.at(geo, blockIdx.x), after = items.at(geo, blockIdx.x + gridDim.x), done = x;
        done.live = 0;  // the item whose results are to leave
        fetch(x);
        for (int it = blockIdx.x; it < items.total; it += gridDim.x) {
            const Item later = items.at(geo, it + 2 * gridDim.x);
            if (!x.live) {
                if (x.n == 0 && x.rb == 0) zero_outside(geo, p, x, warp - 2, 8);
                fetch(after);
                x = after, after = later;
                continue;
            }
            const int n = x.n, rb = x.rb, i0 = rb * kTile, r = i0 + row, i1 = min(i0 + kTile, n) - 1, first = first_jb(x), end = end_jb(x);
            const int zboxes = zboxes_of(x), b = i & 1;
            // sums and weights of the item: the places are those of the item before the last
#pragma unroll
            for (int j = 0; j < kTokens; j++) {
                const int t = et + 256 * j;
                if (t >= x.tiles * kTile) break;
                s_bh[b][t] = p.back ? of_token[j].x : -of_token[j].x, s_bl[b][t] = p.back ? of_token[j].y : -of_token[j].y;
                // weights across the border of the rows: both factors of a decay are at most 1; where they grow beyond float32
                // (positive g), every weight is found for itself
                if (p.back ? t > i1 : t < i0) {
                    const float c = t >= n ? 0.f : p.back ? decay_exp(of_token[j], border) : decay_exp(border, of_token[j]);
                    s_c[b][t] = c;
                    if (isinf(c)) s_exact[i % 3] = 1;
                }
            }
            const float ri = geo.d.scale * (p.back ? decay_exp(border, of_row) : decay_exp(of_row, border));
            if (r < n && isinf(ri)) s_exact[i % 3] = 1;
            const float f = p.back ? decay_exp(last_sum, of_row) : geo.d.scale * decay_exp(of_row, zero);
            const RowWeights weights(p, ri, of_row, geo.d.scale);
            if (group_or<256>(!ok)) break;
            const bool exact = s_exact[i % 3];
            if (et < 128) s_bad[(i + 1) % 3][et] = p.back ? -1 : kTile;
            if (et == 0) s_exact[(i + 2) % 3] = 0, s_anybad[(i + 1) % 3] = 0;
            if (done.live) results(done, i - 1);  // their products ended beside the above
            fetch(after);
            // ---------------------------------------- the state's share
            if (wait(&bar_state[b], i >> 1)) {
                const int hcols = zboxes * 32;
#pragma unroll 1
                for (int c = half * hcols; c < (half + 1) * hcols; c += 16) {
                    float v[16];
                    uint32_t u[16];
                    tmem_ld16(tmem + 128 + lanes + c, v);
#pragma unroll
                    for (int e = 0; e < 16; e++) u[e] = __float_as_uint(v[e] * f);
                    tmem_st16(tmem + 128 + lanes + c, u);
                }
                tmem_wait_st();
            }
            // ---------------------------------------- the span's tokens
            for (int jb = first; ok && jb < end; jb++, k++) {
                const int j0 = jb * kTile, rest = n - j0;
                const bool diag = jb == rb;
                // Every tile of z takes the place of the one before it, and the warps wait for each of them, also where there is nothing to
                // look over: with the one before still on its way, a wait for this one would be told of the fill before both.
                const uint32_t z = m + 3 + 2 * (jb - first);
                if (checked(x, jb)) {
                    if (!wait(&bar_full[z % kHalfRing], z / kHalfRing)) break;
                    look_over(ring + z % kHalfRing * kTileBytes, zboxes, rest, diag, p.back, s_bad[i % 3], &s_anybad[i % 3], nullptr, et, 256);
                    arrive(&bar_checked[ck++ & 1]);
                }
                if (!wait(&bar_s[k & 1], k >> 1)) break;
                // the row's tokens of this block: of 128 columns those below `to`, and from `from` on
                const int last = min(rest, kTile), from = diag && p.back ? row : 0, to = diag && !p.back ? min(row + 1, last) : last;
                const uint32_t t_s = tmem + lanes;
#pragma unroll 1
                for (int c = half * 64; c < half * 64 + 64; c += 16) {
                    float v[16];
                    float2 w[8];
                    uint32_t u[16];
                    tmem_ld16(t_s + c, v);
                    weights.get(diag || exact, s_bh[b] + j0 + c, s_bl[b] + j0 + c, s_c[b] + j0 + c, w);
#pragma unroll
                    for (int e = 0; e < 8; e++) w[e] = mul2(make_float2(v[2 * e], v[2 * e + 1]), w[e]);
                    if (diag || rest < kTile) {  // the mask, and the columns behind the span, whose scores may be anything
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            if (c + 2 * e < from || c + 2 * e >= to) w[e].x = 0.f;
                            if (c + 2 * e + 1 < from || c + 2 * e + 1 >= to) w[e].y = 0.f;
                        }
                    }
                    // a step's 16 tokens: eight columns of the large parts, eight of the small ones, where the scores were
#pragma unroll
                    for (int e = 0; e < 8; e++) split2(w[e], u[e], u[8 + e]);
                    tmem_st16(t_s + c, u);
                }
                tmem_wait_st();
                // before the weights are handed over: z's place is not free, nor filled again, until all warps have done so
                if (!checked(x, jb) && !wait(&bar_full[z % kHalfRing], z / kHalfRing)) break;
                arrive(&bar_p[k & 1]);
            }
            m += 2 + 2 * (end - first);
            done = x, x = after, after = later, i++;
        }
        if (ok && done.live) results(done, i - 1);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(256) : "memory");
}

// ---------------------------------------------------------------- host

// Map of a tensor tokens x heads x cols (or planes x rows x cols) in boxes of 64 columns x `box` rows of its tokens (or rows).
cudaError_t map3(CUtensorMap *map, const void *p, const uint64_t (&dims)[3], const uint64_t (&strides)[2], const uint32_t (&box)[3]) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = get_encode();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t d[3] = {dims[0], dims[1], dims[2]}, s[2] = {strides[0], strides[1]};
    const cuuint32_t b[3] = {box[0], box[1], box[2]}, estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, (void *)p, d, s, b, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t map_rows(CUtensorMap *map, const DecayGeom &g, const DecayRows &r, uint32_t box) {
    const uint64_t heads = r.key ? g.d.hk : g.d.hv;
    return map3(map, r.p, {(uint64_t)r.dist, heads, (uint64_t)g.d.tokens}, {(uint64_t)r.dist * 2, (uint64_t)r.ld * 2}, {64, 1, box});
}

cudaError_t rows_go(const DecayGeom &g, const DecayProduct &p, int parts, int num_sms, unsigned *status, bool next, cudaStream_t st) {
    CUtensorMap x, y, z, m, q;
    cudaError_t e = map_rows(&x, g, p.x, kTile);
    if (e == cudaSuccess) e = map_rows(&y, g, p.y, kTile);
    if (e == cudaSuccess) e = map_rows(&z, g, p.z, kTile);
    if (e == cudaSuccess && p.self) e = map_rows(&q, g, *p.self, kTile);
    const uint64_t planes = (uint64_t)g.d.nchunks * g.d.hv * parts;
    if (e == cudaSuccess)
        e = map3(&m, p.m, {(uint64_t)g.d.dv, (uint64_t)g.d.dk, planes}, {(uint64_t)g.d.dv * 2, (uint64_t)g.d.dv * g.d.dk * 2}, {64, kTile, 1});
    if (e != cudaSuccess) return e;
    RowsTc r{};
    r.xcols = p.x.cols, r.ncols = p.z.cols;
    r.xkey = p.x.key, r.ykey = p.y.key, r.zkey = p.z.key;
    r.turned = p.turned, r.back = p.back, r.parts = parts;
    r.out = (bf16 *)p.out, r.ldo = p.ldo;
    r.vec = !mult16(p.out, p.ldo, p.z.cols, 2) ? 0 : (((uintptr_t)p.out | (uint64_t)p.ldo * 2 | (uint64_t)p.z.cols * 2) & 31) == 0 ? 2 : 1;
    r.sums[0] = p.sums[0], r.sums[1] = p.sums[1];
    const int zb = (p.z.cols + 127) / 128;
    const int per = g.span / kTile;
    Items items{FastDiv((uint32_t)p.heads), FastDiv((uint32_t)zb), FastDiv((uint32_t)per), 0};
    const int64_t total = (int64_t)g.d.nchunks * per * p.heads * zb;
    if (total > 0x7fffffff - 4 * num_sms) return cudaErrorInvalidValue;
    items.total = (int)total;
    const unsigned blocks = (unsigned)std::min<int64_t>(total, num_sms);
    if (p.self) {
        static OncePerDevice limit;
        const cudaError_t attr = smem_limit(limit, k_decay_rows_self, (int)kSelfSmem);
        if (attr != cudaSuccess) return attr;
        return launch(next, k_decay_rows_self, blocks, kRowThreads, kSelfSmem, st, x, y, z, m, q, g, r, items, status);
    }
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_decay_rows_tc, (int)kRowsSmem);
    if (attr != cudaSuccess) return attr;
    return launch(next, k_decay_rows_tc, (unsigned)std::min<int64_t>(total, 2 * num_sms), kHalfThreads, kRowsSmem, st, x, y, z, m, g, r, items, status);
}

}  // namespace

cudaError_t zs_launch_decay_sums_tc(const DecayGeom &g, const DecayRows &x, const DecayRows &y, bool query, bool gates, float *out,
                                    unsigned *status, bool next, cudaStream_t st, int64_t *launches) {
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_decay_sums_tc, (int)kSumSmem);
    if (attr != cudaSuccess) return attr;
    CUtensorMap mx, my;
    cudaError_t e = map_rows(&mx, g, x, kSumChunk);
    if (e == cudaSuccess) e = map_rows(&my, g, y, kSumChunk);
    if (e != cudaSuccess) return e;
    ++*launches;
    return launch(next, k_decay_sums_tc, dim3(g.d.nchunks, g.d.hv, (y.cols + 127) / 128), kSumThreads, kSumSmem, st, mx, my, g, x.cols, y.cols,
                  (int)x.key, (int)y.key, (int)query, (int)gates, out, status);
}

cudaError_t zs_launch_decay_rows_tc(const DecayGeom &g, const DecayProduct &p, int parts, int num_sms, unsigned *status, bool next,
                                    cudaStream_t st, int64_t *launches) {
    ++*launches;
    return rows_go(g, p, parts, num_sms, status, next, st);
}
