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

__device__ __forceinline__ bool finite_pair(uint32_t w) { return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u; }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// ---------------------------------------------------------------- sums

// U = sum over a span's tokens of w_j x_j y_j^T, 128 x 128 in TMEM.  x's tiles of 64 tokens are scaled and split in
// three parts by eight warps, in shared memory, where they are the MN-major A operand; y's are the
// B operand as TMA leaves them.  Two accumulators, one for the small parts; after 128 tokens both are
// added to the float32 sums in the warps' registers.  Two blocks an SM, so that one's
// conversions run beside the other's products.
constexpr int kSumWorkers = 256, kSumThreads = kSumWorkers + 32;
constexpr int kSumChunk = 64;
constexpr uint32_t kSumBox = kSumChunk * kRow, kSumTile = 2 * kSumBox;
constexpr uint32_t kSumSmem = kSumTile * 6 + 1024;  // x, two of y, three parts

__global__ void __launch_bounds__(kSumThreads, 2)
k_decay_sums_tc(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap ymap, const DecayGeom geo, int xcols, int ycols,
                int xkey, int ykey, int query, int gates, float *__restrict__ out, unsigned *__restrict__ status) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_x, bar_y[2], bar_parts, bar_parts_free, bar_y_free[2], bar_acc, bar_acc_free, bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ float2 s_b[kSpanMost];
    __shared__ float s_w[kSpanMost];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int span = blockIdx.x, hv = blockIdx.y, c0 = blockIdx.z * 128;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sx = base, sy = base + kSumTile, sp_ = base + 3 * kSumTile;
    if (tid == 0) {
        s_abort = 0;
        bar_init(&bar_x, 1);
        for (int i = 0; i < 2; i++) bar_init(&bar_y[i], 1), bar_init(&bar_y_free[i], 1);
        bar_init(&bar_parts, kSumWorkers / 32);
        bar_init(&bar_parts_free, 1);
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
    const uint32_t tmem = s_tmem;
    const int2 sp = geo.d.chunk[span];
    const int n = sp.y, group = geo.d.hv / geo.d.hk, hk = hv / group;
    const int chunks = (n + kSumChunk - 1) / kSumChunk, xboxes = (xcols + 63) / 64, yboxes = min(2, (ycols - c0 + 63) / 64);
    if (warp == 0 && n > 0) decay_sums(geo, sp, hv, s_b);
    __syncthreads();
    if (tid < kSumWorkers && n > 0) {
        const float2 last = s_b[n - 1];
        for (int i = tid; i < chunks * kSumChunk; i += kSumWorkers)
            s_w[i] = i >= n ? 0.f : query ? geo.d.scale * decay_exp(s_b[i], make_float2(0.f, 0.f)) : decay_exp(last, s_b[i]);
        if (gates && blockIdx.z == 0)
            for (int i = tid; i < n; i += kSumWorkers) geo.gates[((int64_t)span * geo.d.hv + hv) * geo.span + i] = s_b[i];
        if (xboxes == 1)  // the rows beyond x's columns: zeros in all parts
            for (int i = tid; i < 3 * (int)kSumBox / 16; i += kSumWorkers)
                sts128(sp_ + (uint32_t)(i / ((int)kSumBox / 16)) * kSumTile + kSumBox + (uint32_t)(i % ((int)kSumBox / 16)) * 16, make_uint4(0, 0, 0, 0));
    }
    __syncthreads();
    if (warp == 8) {
        if (lane == 0) {
            int loaded = 0;
            bool ok = true;
            auto load_x = [&](int i) {
                bar_expect(&bar_x, (uint32_t)xboxes * kSumBox);
                for (int b = 0; b < xboxes; b++)
                    tma_load_3d(sx + b * kSumBox, &xmap, b * 64, xkey ? hk : hv, sp.x + i * kSumChunk, smem_u32(&bar_x));
            };
            auto load_y = [&](int i) {
                const int st = i & 1;
                if (!bar_wait(&bar_y_free[st], ((i >> 1) & 1) ^ 1, &s_abort, status)) return false;
                bar_expect(&bar_y[st], (uint32_t)yboxes * kSumBox);
                for (int b = 0; b < yboxes; b++)
                    tma_load_3d(sy + st * kSumTile + b * kSumBox, &ymap, c0 + b * 64, ykey ? hk : hv, sp.x + i * kSumChunk, smem_u32(&bar_y[st]));
                return true;
            };
            if (chunks > 0) {
                load_x(0);
                ok = load_y(0);
                loaded = 1;
            }
            const uint32_t idesc = f16_idesc<bf16>(128, yboxes * 64, true, true);
            for (int i = 0; ok && i < chunks; i++) {
                if (!bar_wait(&bar_parts, i & 1, &s_abort, status)) break;  // x is read, its parts are there
                if (i + 1 < chunks) {
                    load_x(i + 1);
                    if (!load_y(i + 1)) break;
                    loaded = i + 2;
                }
                if (!bar_wait(&bar_y[i & 1], (i >> 1) & 1, &s_abort, status)) break;
                const bool first = !(i & 1);
                if (first && !bar_wait(&bar_acc_free, ((i >> 1) & 1) ^ 1, &s_abort, status)) break;
                tc_fence_after();
                const uint32_t yb = sy + (i & 1) * kSumTile;
                // the small parts, smallest first, then the large one
#pragma unroll
                for (int part = 2; part >= 0; part--)
#pragma unroll
                    for (int ks = 0; ks < kSumChunk / 16; ks++)
                        mma_f16(tmem + (part ? 128u : 0u), smem_desc<true>(sp_ + part * kSumTile + ks * 2048, kSumBox),
                                smem_desc<true>(yb + ks * 2048, kSumBox), idesc, !first || ks || part == 1 ? 1u : 0u);
                mma_commit(smem_u32(&bar_parts_free));
                mma_commit(smem_u32(&bar_y_free[i & 1]));
                if (!first || i + 1 == chunks) mma_commit(smem_u32(&bar_acc));
            }
            mma_commit(smem_u32(&bar_drain));
            for (uint32_t w = 0; w < kWaitLimit && !bar_try(&bar_drain, 0); w++) {
            }
            if (loaded) {  // the copies in flight
                for (uint32_t w = 0; w < kWaitLimit && !bar_try(&bar_x, (loaded - 1) & 1); w++) {
                }
                for (int i = std::max(0, loaded - 2); i < loaded; i++)
                    for (uint32_t w = 0; w < kWaitLimit && !bar_try(&bar_y[i & 1], (i >> 1) & 1); w++) {
                    }
            }
        }
    } else {
        const int quad = warp & 3, half = warp >> 2;
        float acc[64];
#pragma unroll
        for (int e = 0; e < 64; e++) acc[e] = 0.f;
        const int row = quad * 32 + lane, cols = yboxes * 32;  // a thread's columns: its half
        for (int i = 0; i < chunks; i++) {
            if (!bar_wait(&bar_x, i & 1, &s_abort, status)) break;
            if (!bar_wait(&bar_parts_free, (i & 1) ^ 1, &s_abort, status)) break;
            const int rest = n - i * kSumChunk;
            for (int j = tid; j < kSumChunk * 8 * xboxes; j += kSumWorkers) {
                const int c = j & 7, b = xboxes == 2 ? (j >> 3) & 1 : 0, r = xboxes == 2 ? j >> 4 : j >> 3;
                const uint32_t at = b * kSumBox + swizzled(r, c);
                const uint4 u = lds128(sx + at);
                const float w = s_w[i * kSumChunk + r];
                const uint32_t in[4] = {u.x, u.y, u.z, u.w};
                uint32_t p0[4], p1[4], p2[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    float2 f = unpack2<bf16>(in[e]);
                    f.x = r < rest ? f.x * w : 0.f;
                    f.y = r < rest ? f.y * w : 0.f;
                    p0[e] = Split3::part(f.x, f.y);
                    p1[e] = Split3::part(f.x, f.y);
                    p2[e] = pack2<bf16>(f.x, f.y);
                }
                sts128(sp_ + at, make_uint4(p0[0], p0[1], p0[2], p0[3]));
                sts128(sp_ + kSumTile + at, make_uint4(p1[0], p1[1], p1[2], p1[3]));
                sts128(sp_ + 2 * kSumTile + at, make_uint4(p2[0], p2[1], p2[2], p2[3]));
            }
            if (rest < kSumChunk) {  // what lies behind the span meets zeros of x, and must be finite
                if (!bar_wait(&bar_y[i & 1], (i >> 1) & 1, &s_abort, status)) break;
                for (int j = tid; j < (kSumChunk - rest) * 8 * yboxes; j += kSumWorkers) {
                    const int c = j & 7, b = (j >> 3) % yboxes, r = rest + (j >> 3) / yboxes;
                    sts128(sy + (i & 1) * kSumTile + b * kSumBox + swizzled(r, c), make_uint4(0, 0, 0, 0));
                }
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
//   S = X Y^T in TMEM; eight warps read it, mask and weigh it, and put it back in two bfloat16 parts, in its
//   place, as the A operand of O += P Z; the state's share X M comes first and, scaled in TMEM, is what O starts from.
// Two blocks an SM (256 columns of TMEM each), so that one's weights are found beside the other's products.  SELF: one
// block an SM, which also has the other scores self Z^T, for the sums of pairs, and goes through the value heads that
// share its key head; their gradients add up in O.
constexpr int kTile = 128;
constexpr uint32_t kBoxBytes = kTile * kRow, kTileBytes = 2 * kBoxBytes;
constexpr int kRowThreads = 64 + 256;

struct RowsTc {
    int xcols, ncols;      // columns of x and y, and of z
    int xkey, ykey, zkey;  // heads are key heads
    int turned, back, parts;
    int blocks;            // of rows, a block of threads takes one after the other
    bf16 *out;
    int64_t ldo;
    int vec;               // 16-byte stores
    float *sums[2];
};

template <bool SELF>
constexpr uint32_t rows_smem() { return kTileBytes * (SELF ? 5 : 3) + 1024; }

template <bool SELF>
__global__ void __launch_bounds__(kRowThreads, SELF ? 1 : 2)
k_decay_rows_tc(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap ymap, const __grid_constant__ CUtensorMap zmap,
                const __grid_constant__ CUtensorMap mmap, const __grid_constant__ CUtensorMap qmap, const DecayGeom geo, const RowsTc p,
                unsigned *__restrict__ status) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_x, bar_x_free, bar_y, bar_y_free, bar_z, bar_z_free, bar_w, bar_w_free, bar_checked, bar_state, bar_begun,
        bar_s, bar_p, bar_o, bar_o_free, bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ float2 s_b[kSpanMost];
    __shared__ float s_c[kSpanMost];          // weights of the tokens outside the rows' own block, up to its border
    __shared__ int s_bad[128], s_anybad, s_badtok, s_exact;
    __shared__ float s_dot[SELF ? 2 : 1][2][kTile];
    constexpr uint32_t kCols = SELF ? 512 : 256;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sx = base, sy = base + kTileBytes, sz = base + 2 * kTileBytes, sw = base + 3 * kTileBytes, sq = base + 4 * kTileBytes;
    if (tid == 0) {
        s_abort = 0;
        bar_init(&bar_x, 1), bar_init(&bar_x_free, 1 + (SELF ? 8 : 0));
        bar_init(&bar_y, 1), bar_init(&bar_y_free, 1);
        bar_init(&bar_z, 1), bar_init(&bar_z_free, 1);
        bar_init(&bar_w, 1), bar_init(&bar_w_free, 1);
        bar_init(&bar_checked, 8), bar_init(&bar_state, 1), bar_init(&bar_begun, 8);
        bar_init(&bar_s, 1), bar_init(&bar_p, 8), bar_init(&bar_o, 1), bar_init(&bar_o_free, 8);
        bar_init(&bar_drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    after_previous();
    may_start_next();
    const uint32_t tmem = s_tmem;
    const int all = geo.span / kTile, per = (all + p.blocks - 1) / p.blocks;  // blocks of threads a span
    const int span = blockIdx.x / per, rb0 = (blockIdx.x - span * per) * p.blocks;
    const int head = blockIdx.y, c0 = blockIdx.z * 128;
    const int2 sp = geo.d.chunk[span];
    const int n = sp.y, tiles = (n + kTile - 1) / kTile, rb1 = min(tiles, rb0 + p.blocks);
    const int group = geo.d.hv / geo.d.hk, rounds = SELF ? group : 1;
    const int xboxes = (p.xcols + 63) / 64, cols = min(128, p.ncols - c0), zboxes = (cols + 63) / 64, ksteps = (p.xcols + 15) / 16;
    const int mboxes = p.turned ? xboxes : zboxes;
    auto head_of = [&](int key, int r) { return SELF ? (key ? head : head * group + r) : (key ? head / group : head); };
    auto jb0 = [&](int rb) { return p.back ? rb : 0; };
    auto jb1 = [&](int rb) { return p.back ? tiles : rb + 1; };
    auto checked = [&](int rb, int jb) { return jb == rb || (jb + 1) * kTile > n; };
    const uint32_t t_s = tmem, t_o = tmem + 128, t_s2 = tmem + 256;
    const uint32_t t_m = SELF ? t_s : t_o;  // where the state's share arrives

    if (n == 0 && rb0 == 0 && warp >= 2) {
        // tokens outside the sequences
        const int used = geo.d.first[geo.d.nseq], workers = (geo.d.nchunks - used) * 8, worker = (span - used) * 8 + warp - 2;
        const int2 last = geo.d.seq[geo.d.nseq - 1];
        bf16 *o = p.out + (int64_t)head * p.ncols + c0;
        zero_tokens(o, p.ldo, 0, geo.d.seq[0].x, cols, worker, workers);
        zero_tokens(o, p.ldo, (int64_t)last.x + last.y, geo.d.tokens, cols, worker, workers);
    } else if (warp == 0) {
        // ------------------------------------------------ TMA
        if (lane == 0) {
            uint32_t cx = 0, cy = 0, cz = 0, cw = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t count) { return ok = ok && bar_wait(bar, (count & 1u) ^ 1u, &s_abort, status); };
            // `boxes` boxes of 64 columns from column c on, all into one tile
            auto load = [&](uint32_t to, const CUtensorMap *map, int boxes, int c, int h, int row, uint64_t *bar) {
                for (int b = 0; b < boxes; b++) tma_load_3d(to + b * kBoxBytes, map, c + b * 64, h, row, smem_u32(bar));
            };
            auto load_m = [&](uint32_t to, int part, int hv, uint64_t *bar) {
                bar_expect(bar, (uint32_t)mboxes * kBoxBytes);
                const int plane = (span * geo.d.hv + hv) * p.parts + part;
                load(to, &mmap, mboxes, p.turned ? 0 : c0, p.turned ? c0 : 0, plane, bar);
            };
            for (int rb = rb0; ok && rb < rb1; rb++)
                for (int r = 0; ok && r < rounds; r++) {
                    const int hv = SELF ? head * group + r : head, row = sp.x + rb * kTile;
                    if (!wait(&bar_x_free, cx)) break;
                    bar_expect(&bar_x, (uint32_t)(xboxes + (SELF ? zboxes : 0)) * kBoxBytes);
                    load(sx, &xmap, xboxes, 0, head_of(p.xkey, r), row, &bar_x);
                    if (SELF) load(sq, &qmap, zboxes, 0, head, row, &bar_x);
                    cx++;
                    if (!wait(&bar_y_free, cy)) break;
                    load_m(sy, 0, hv, &bar_y), cy++;
                    if (!wait(&bar_z_free, cz)) break;
                    load_m(sz, 1, hv, &bar_z), cz++;
                    if (SELF) {
                        if (!wait(&bar_w_free, cw)) break;
                        load_m(sw, 2, hv, &bar_w), cw++;
                    }
                    for (int jb = jb0(rb); jb < jb1(rb); jb++) {
                        if (!wait(&bar_y_free, cy)) break;
                        bar_expect(&bar_y, (uint32_t)xboxes * kBoxBytes);
                        load(sy, &ymap, xboxes, 0, head_of(p.ykey, r), sp.x + jb * kTile, &bar_y), cy++;
                        if (!wait(&bar_z_free, cz)) break;
                        bar_expect(&bar_z, (uint32_t)zboxes * kBoxBytes);
                        load(sz, &zmap, zboxes, c0, head_of(p.zkey, r), sp.x + jb * kTile, &bar_z), cz++;
                    }
                }
            // the copies in flight: wait (bounded) for the last of each
            auto drain = [&](uint64_t *bar, uint32_t count) {
                for (uint32_t w = 0; count && w < kWaitLimit && !bar_try(bar, (count - 1) & 1u); w++) {
                }
            };
            drain(&bar_x, cx), drain(&bar_y, cy), drain(&bar_z, cz), drain(&bar_w, cw);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (lane == 0) {
            uint32_t cx = 0, cy = 0, cz = 0, cw = 0, ck = 0, cp = 0, co = 0, cb = 0, crb = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t count) {
                ok = ok && bar_wait(bar, count & 1u, &s_abort, status);
                tc_fence_after();
                return ok;
            };
            const uint32_t id_s = f16_idesc<bf16>(128, 128, false, false), id_o = f16_idesc<bf16>(128, zboxes * 64, false, true);
            const uint32_t id_m = f16_idesc<bf16>(128, p.turned ? 128 : zboxes * 64, false, !p.turned);
            auto kmajor = [&](uint32_t tile, int ks) { return smem_desc<false>(tile + (ks >> 2) * kBoxBytes + (ks & 3) * 32, kBoxBytes); };
            auto mnmajor = [&](uint32_t tile, int ks) { return smem_desc<true>(tile + ks * 2048, kBoxBytes); };
            for (int rb = rb0; ok && rb < rb1; rb++, crb++)
                for (int r = 0; ok && r < rounds; r++) {
                    if (!wait(&bar_x, cx++)) break;
                    if (r == 0 && !wait(&bar_o_free, crb ^ 1u)) break;  // the rows before are read
                    // the state's share, the smallest part first
                    if (!wait(&bar_y, cy++) || !wait(&bar_z, cz++)) break;
                    if (SELF && !wait(&bar_w, cw++)) break;
                    bool first = true;
                    for (int part = SELF ? 2 : 1; part >= 0; part--) {
                        const uint32_t m = part == 0 ? sy : part == 1 ? sz : sw;
                        for (int ks = 0; ks < ksteps; ks++, first = false)
                            mma_f16(t_m, kmajor(sx, ks), p.turned ? kmajor(m, ks) : mnmajor(m, ks), id_m, first ? 0u : 1u);
                    }
                    mma_commit(smem_u32(&bar_y_free));
                    mma_commit(smem_u32(&bar_z_free));
                    if (SELF) mma_commit(smem_u32(&bar_w_free));
                    mma_commit(smem_u32(&bar_state));
                    if (!wait(&bar_begun, cb++)) break;  // O holds it, scaled
                    for (int jb = jb0(rb); jb < jb1(rb); jb++) {
                        if (!wait(&bar_y, cy++)) break;
                        for (int ks = 0; ks < ksteps; ks++) mma_f16(t_s, kmajor(sx, ks), kmajor(sy, ks), id_s, ks ? 1u : 0u);
                        mma_commit(smem_u32(&bar_y_free));
                        const bool check = checked(rb, jb);
                        if (SELF) {
                            if (!wait(&bar_z, cz++)) break;
                            if (check && !wait(&bar_checked, ck++)) break;
                            for (int ks = 0; ks < (cols + 15) / 16; ks++) mma_f16(t_s2, kmajor(sq, ks), kmajor(sz, ks), id_s, ks ? 1u : 0u);
                        }
                        if (jb + 1 == jb1(rb)) mma_commit(smem_u32(&bar_x_free));
                        mma_commit(smem_u32(&bar_s));
                        if (!SELF) {
                            if (!wait(&bar_z, cz++)) break;
                            if (check && !wait(&bar_checked, ck++)) break;
                        }
                        if (!wait(&bar_p, cp++)) break;
                        for (int part = 0; part < 2; part++)
                            for (int ks = 0; ks < kTile / 16; ks++)
                                mma_f16_ta(t_o, t_s + ks * 16 + part * 8, mnmajor(sz, ks), id_o, 1u);
                        mma_commit(smem_u32(&bar_z_free));
                        mma_commit(smem_u32(&bar_o));
                        if (!wait(&bar_o, co++)) break;  // P's place is the next scores'
                    }
                }
            // every MMA issued so far completes before TMEM is freed
            mma_commit(smem_u32(&bar_drain));
            for (uint32_t w = 0; w < kWaitLimit && !bar_try(&bar_drain, 0); w++) {
            }
        }
    } else {
        // ------------------------------------------------ weights and results (warps 2-9)
        const int quad = warp & 3, half = (warp - 2) >> 2, et = tid - 64;
        const int row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const int hcols = zboxes * 32;  // a thread's columns of O: its half
        uint32_t cs = 0, cz = 0, cst = 0, co = 0;
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
        // the eight warps wait for each other; whether one of them has given up
        auto all_or = [](bool bad) {
            uint32_t r;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(r)
                         : "r"((uint32_t)bad)
                         : "memory");
            return r != 0;
        };
        const float2 zero = make_float2(0.f, 0.f);
        for (int rb = rb0, r = 0; rb < rb1; r + 1 < rounds ? r++ : (r = 0, rb++)) {
            const int i0 = rb * kTile, i1 = min(i0 + kTile, n) - 1, i = i0 + row;
            const int hv = SELF ? head * group + r : head;
            const int64_t slot = (int64_t)span * geo.d.hv + hv;
            if (all_or(!ok)) break;  // and the last round's sums are read
            for (int j = et; j < n; j += 256) s_b[j] = geo.gates[slot * geo.span + j];
            if (r == 0) {
                if (et < 128) s_bad[et] = p.back ? -1 : kTile;
                if (et == 0) s_anybad = 0, s_badtok = p.back ? -1 : kTile;
            }
            if (et == 0) s_exact = 0;
            all_or(false);
            // weights across the border of the rows' own block: both factors of a decay are at most 1; where they grow
            // beyond float32 (positive g), every weight is found for itself
            const float2 border = p.back ? s_b[i1] : i0 ? s_b[i0 - 1] : zero;
            for (int j = et; j < n; j += 256) {
                if (p.back ? j <= i1 : j >= i0) continue;
                const float c = p.back ? decay_exp(s_b[j], border) : decay_exp(border, s_b[j]);
                s_c[j] = c;
                if (isinf(c)) s_exact = 1;
            }
            const float2 bi = s_b[min(i, n - 1)], bl = s_b[n - 1];
            const float ri = geo.d.scale * (p.back ? decay_exp(border, bi) : decay_exp(bi, border));
            if (i < n && isinf(ri)) s_exact = 1;
            const float f = p.back ? decay_exp(bl, bi) : geo.d.scale * decay_exp(bi, zero);
            all_or(false);
            const bool exact = s_exact;
            float dot = 0.f, pair = 0.f;
            // ---------------------------------------- the state's share
            if (wait(&bar_state, cst++)) {
#pragma unroll 1
                for (int c = 0; c < hcols; c += 16) {
                    float v[16];
                    const int col = half * hcols + c;
                    tmem_ld16(t_m + lanes + col, v);
#pragma unroll
                    for (int e = 0; e < 16; e++) v[e] *= f;
                    if (SELF) {
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int cc = col + 8 * h;
                            const uint4 q = lds128(sq + (cc >> 6) * kBoxBytes + swizzled(row, (cc >> 3) & 7));
                            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const float2 s = unpack2<bf16>(w[e]);
                                dot = fmaf(v[8 * h + 2 * e], s.x, fmaf(v[8 * h + 2 * e + 1], s.y, dot));
                            }
                        }
                        if (r > 0) {
                            float o[16];
                            tmem_ld16(t_o + lanes + col, o);
#pragma unroll
                            for (int e = 0; e < 16; e++) v[e] += o[e];
                        }
                    }
                    uint32_t u[16];
#pragma unroll
                    for (int e = 0; e < 16; e++) u[e] = __float_as_uint(v[e]);
                    tmem_st16(t_o + lanes + col, u);
                }
                tmem_wait_st();
                arrive(&bar_begun);
                if (SELF && lane == 0) bar_arrive(&bar_x_free);  // self's rows are read
            }
            cz++;  // z's place held a part of the state
            // ---------------------------------------- the span's tokens
            for (int jb = jb0(rb); ok && jb < jb1(rb); jb++, cz++, co++) {
                const int j0 = jb * kTile, rest = n - j0;
                if (!wait(&bar_z, cz)) break;
                if (checked(rb, jb)) {
                    // Tokens behind the span count as zeros.  On the diagonal, an infinity or NaN would meet the zeros of the rows that
                    // the mask keeps from it: it is taken out, and put into the results of the others.
                    for (int j = et; j < kTile * 8 * zboxes; j += 256) {
                        const int c = j & 7, b = zboxes == 2 ? (j >> 3) & 1 : 0, rr = zboxes == 2 ? j >> 4 : j >> 3;
                        const uint32_t at = sz + b * kBoxBytes + swizzled(rr, c);
                        if (rr >= rest) {
                            sts128(at, make_uint4(0, 0, 0, 0));
                            continue;
                        }
                        if (jb != rb) continue;
                        const uint4 u = lds128(at);
                        if (finite_pair(u.x) && finite_pair(u.y) && finite_pair(u.z) && finite_pair(u.w)) continue;
                        uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            if (((w[e >> 1] >> (16 * (e & 1))) & 0x7f80u) != 0x7f80u) continue;
                            w[e >> 1] &= e & 1 ? 0xffffu : 0xffff0000u;
                            int *bad = &s_bad[b * 64 + c * 8 + e];
                            if (p.back)
                                atomicMax(bad, rr), atomicMax(&s_badtok, rr);
                            else
                                atomicMin(bad, rr), atomicMin(&s_badtok, rr);
                        }
                        s_anybad = 1;
                        sts128(at, make_uint4(w[0], w[1], w[2], w[3]));
                    }
                    fence_async();
                    arrive(&bar_checked);
                }
                if (!wait(&bar_s, cs++)) break;
                const bool each = jb == rb || exact;
#pragma unroll 1
                for (int c = 0; c < 64; c += 16) {
                    float v[16], s2[SELF ? 16 : 1];
                    const int cc = half * 64 + c, j = j0 + cc;
                    tmem_ld16(t_s + lanes + cc, v);
                    if constexpr (SELF) tmem_ld16(t_s2 + lanes + cc, s2);
                    if (each) {
#pragma unroll
                        for (int e = 0; e < 16; e++) {
                            const float2 bj = s_b[min(j + e, n - 1)];
                            const bool in = (p.back ? j + e >= i : j + e <= i) && j + e < n;
                            v[e] = in ? v[e] * (geo.d.scale * (p.back ? decay_exp(bj, bi) : decay_exp(bi, bj))) : 0.f;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e++) v[e] = j + e < n ? v[e] * (ri * s_c[min(j + e, n - 1)]) : 0.f;
                    }
                    if constexpr (SELF) {
#pragma unroll
                        for (int e = 0; e < 16; e++)
                            if ((p.back ? j + e > i : j + e < i) && j + e < n) pair = fmaf(v[e], s2[e], pair);
                    }
                    // a step's 16 tokens: eight columns of the large parts, eight of the small ones, where the scores were
                    uint32_t u[16];
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        u[e] = Split3::part(v[2 * e], v[2 * e + 1]);
                        u[8 + e] = pack2<bf16>(v[2 * e], v[2 * e + 1]);
                    }
                    tmem_st16(t_s + lanes + cc, u);
                }
                tmem_wait_st();
                arrive(&bar_p);
            }
            if (SELF) s_dot[half][0][row] = dot, s_dot[half][SELF ? 1 : 0][row] = pair;
            all_or(false);  // and every value that was taken out is known
            if (!ok) continue;
            const float nan = __int_as_float(0x7fc00000);
            if (SELF && half == 0 && i < n) {
                const int64_t at = (int64_t)(sp.x + i) * geo.d.hv + hv;
                float pairs = s_dot[0][1][row] + s_dot[SELF ? 1 : 0][1][row];
                if (p.back ? row < s_badtok : row > s_badtok) pairs = nan;
                p.sums[0][at] = s_dot[0][0][row] + s_dot[SELF ? 1 : 0][0][row];
                p.sums[1][at] = pairs;
            }
            if (r + 1 < rounds) continue;
            // ---------------------------------------- results
            if (!wait(&bar_o, co - 1)) continue;
            bf16 *o = p.out + (int64_t)(sp.x + i) * p.ldo + (int64_t)head * p.ncols + c0;
#pragma unroll 1
            for (int c = 0; c < hcols; c += 16) {
                float v[16];
                const int col = half * hcols + c;
                tmem_ld16(t_o + lanes + col, v);
                if (s_anybad)
#pragma unroll
                    for (int e = 0; e < 16; e++)
                        if (p.back ? row <= s_bad[col + e] : row >= s_bad[col + e]) v[e] = nan;
                if (i >= n) continue;
#pragma unroll
                for (int h = 0; h < 16; h += 8) {
                    if (p.vec && col + h + 8 <= cols) {
                        *reinterpret_cast<uint4 *>(o + col + h) = make_uint4(pack2<bf16>(v[h], v[h + 1]), pack2<bf16>(v[h + 2], v[h + 3]),
                                                                             pack2<bf16>(v[h + 4], v[h + 5]), pack2<bf16>(v[h + 6], v[h + 7]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            if (col + h + e < cols) o[col + h + e] = from_f32<bf16>(v[h + e]);
                    }
                }
            }
            __syncwarp();
            arrive(&bar_o_free);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
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

template <bool SELF>
cudaError_t rows_go(const DecayGeom &g, const DecayProduct &p, int parts, int num_sms, unsigned *status, bool next, cudaStream_t st) {
    static OncePerDevice limit;
    const cudaError_t attr = smem_limit(limit, k_decay_rows_tc<SELF>, (int)rows_smem<SELF>());
    if (attr != cudaSuccess) return attr;
    CUtensorMap x, y, z, m, q;
    cudaError_t e = map_rows(&x, g, p.x, kTile);
    if (e == cudaSuccess) e = map_rows(&y, g, p.y, kTile);
    if (e == cudaSuccess) e = map_rows(&z, g, p.z, kTile);
    if (e == cudaSuccess) e = map_rows(&q, g, p.self ? *p.self : p.z, kTile);
    const uint64_t planes = (uint64_t)g.d.nchunks * g.d.hv * parts;
    if (e == cudaSuccess)
        e = map3(&m, p.m, {(uint64_t)g.d.dv, (uint64_t)g.d.dk, planes}, {(uint64_t)g.d.dv * 2, (uint64_t)g.d.dv * g.d.dk * 2}, {64, kTile, 1});
    if (e != cudaSuccess) return e;
    RowsTc r{};
    r.xcols = p.x.cols, r.ncols = p.z.cols;
    r.xkey = p.x.key, r.ykey = p.y.key, r.zkey = p.z.key;
    r.turned = p.turned, r.back = p.back, r.parts = parts;
    r.out = (bf16 *)p.out, r.ldo = p.ldo;
    r.vec = mult16(p.out, p.ldo, p.z.cols, 2);
    r.sums[0] = p.sums[0], r.sums[1] = p.sums[1];
    const int all = g.span / kTile, zb = (p.z.cols + 127) / 128;
    // a block of threads takes all of a span's rows where there are blocks enough without parting them
    r.blocks = (int64_t)g.d.nchunks * p.heads * zb >= (SELF ? 2 : 4) * num_sms ? all : 1;
    const dim3 grid((unsigned)(g.d.nchunks * ((all + r.blocks - 1) / r.blocks)), (unsigned)p.heads, (unsigned)zb);
    return launch(next, k_decay_rows_tc<SELF>, grid, kRowThreads, rows_smem<SELF>(), st, x, y, z, m, q, g, r, status);
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
    return p.self ? rows_go<true>(g, p, parts, num_sms, status, next, st) : rows_go<false>(g, p, parts, num_sms, status, next, st);
}
