// glu_tc.cuh -- the matrix products of the gated feed-forward on the tensor cores
// (tcgen05, 16-bit operands, fp32 accumulators), with what is done to their results.
//
// A pair of blocks on two SMs works on one tile of 256 x 256 (cta_group::2): each has
// 128 of the tile's rows in its tensor memory and half of either operand in its shared
// memory, so that a K-step of 64 takes 32 KB of each block (of single blocks on 128 x 256
// 48).  Persistent; per block a warp that loads
// (TMA, six stages), a warp whose first thread issues the products (in the pair's first
// block) and eight warps that take the finished accumulators (two of them, so that the
// next tile's products run meanwhile) out of tensor memory.
//
// Forward: the 256 columns are 128 of the gate and the same 128 of the up projection (the
// first block of the pair loads w_gate's rows, the second w_up's), so both factors of an
// output meet in one thread.  Backward: dx sums over two pairs of operands, d_g w_gate and
// d_u w_up, in one accumulator; the weights' gradients take d^T and x as they lie in memory,
// both with K (the tokens) as their outer dimension.  Both are one launch, so that
// the tiles of one fill what those of the other leave of the device.
//
// 16384 x 2048 x 6144 bf16: forward 430 us alone (1.92 PFLOP/s) and 496 in a row of them, which
// the card's power bounds (1.66); the training pass 1764 with its element-wise part.  With few
// K-steps a tile's results bound it: 32768 x 512 x 1536 69 us (1.49), with kept gates 101
// (they are 300 MB).
//
// Where there are few tiles, each is cut into stretches of K, whose sums go to memory in
// fp32 and are added up by a kernel of their own, in one order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "glu_launch.h"
#include "glu_math.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace gdn {
namespace glu {

constexpr int kHalf = 16384;  // bytes of a block's share of an operand's stage
constexpr int kStageBytes = 2 * kHalf;
constexpr int kEpilogueWarps = 8, kProductThreads = 32 * (2 + kEpilogueWarps);
constexpr int kBox = 4096;  // 32 rows of 64 results
// Six stages leave each of these warps one box, which is what a tile needs: with two, and
// five stages, 16384 x 2048 x 6144 with kept gates took 486 us in place of 471.
constexpr int kStages = 6;
constexpr int kProductSmem = 1024 + kStages * kStageBytes + kEpilogueWarps * kBox + 256;
template <typename Call>
struct Shape {
    static constexpr bool kForward = false, kKeep = false, kShares = false;
};
template <bool KEEP>
struct Shape<Forward<KEEP>> {
    static constexpr bool kForward = true, kKeep = KEEP, kShares = false;
};
template <>
struct Shape<ForwardShares> {
    static constexpr bool kForward = true, kKeep = false, kShares = true;
};
constexpr int kGroup = 8;  // tiles along the rows that are taken side by side

struct Barriers {
    uint64_t full[kStages], empty[kStages], done[2], taken[2];
    uint32_t tmem;
};

struct TileAt {
    int m, n, z, part;  // of the results' tiles, which result, which stretch of K
    int begin, end;     // its K-steps
};
// Tiles in groups of kGroup along the rows, so that those worked on at once share their
// operands in L2.
__device__ __forceinline__ TileAt tile_at(const Job &p, uint32_t i) {
    TileAt t;
    const uint32_t wide = (uint32_t)p.tiles_n, tall = (uint32_t)p.tiles_m, per = wide * tall;
    const uint32_t plane = i / per;
    i -= plane * per;
    t.part = (int)plane / p.results, t.z = (int)plane - t.part * p.results;
    const uint32_t group = i / (kGroup * wide), first = group * kGroup;
    const uint32_t rows = tall - first < kGroup ? tall - first : kGroup;
    i -= first * wide;
    t.n = (int)(i / rows);
    t.m = (int)(first + (i - (uint32_t)t.n * rows));
    const int all = p.pairs * p.blocks_k, end = (t.part + 1) * p.per_part;
    t.begin = t.part * p.per_part, t.end = end < all ? end : all;
    return t;
}
// The job of a tile, which is then counted from the job's first.
__device__ __forceinline__ const Job &job_of(const ForwardArgs &p, uint32_t &) { return p.job; }
__device__ __forceinline__ const Job &job_of(const Backward &p, uint32_t &i) {
    const bool second = i >= p.job[0].tiles;
    if (second) i -= p.job[0].tiles;
    return p.job[second];
}
__host__ __device__ inline uint32_t tiles_of(const ForwardArgs &p) { return p.job.tiles; }
__host__ __device__ inline uint32_t tiles_of(const Backward &p) { return p.job[0].tiles + p.job[1].tiles; }

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 32 results of a lane's row, rounded, and their place in its row of 64 of a box: 16-byte
// pieces where the 128-byte swizzle has them.
struct Packed {
    uint32_t w[16];
};
template <typename T>
__device__ __forceinline__ Packed pack(const uint32_t (&r)[32]) {
    Packed p;
#pragma unroll
    for (int i = 0; i < 16; ++i) p.w[i] = pack2<T>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    return p;
}
__device__ __forceinline__ void put(unsigned char *box, int lane, const Packed (&p)[2]) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint32_t *w = p[c >> 2].w + 4 * (c & 3);
        *reinterpret_cast<uint4 *>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Sends a warp's box of 32 rows x 64 columns to its place; what lies outside is left out.
__device__ __forceinline__ void send(const Job &p, const Result &c, const unsigned char *box, int64_t row, int col,
                                     int lane) {
    if (c.by_map) {
        ptx::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            ptx::tma_store_2d(&c.map, col, (int)row, box);
            ptx::bulk_commit();
        }
        return;
    }
    __syncwarp();
    const int rows = p.rows - row < 32 ? (int)(p.rows - row) : 32;
    uint16_t *to = static_cast<uint16_t *>(c.at) + row * c.stride + col;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = lane + 32 * h;
        if (col + e >= p.cols) continue;
#pragma unroll 16
        for (int r = 0; r < 32; ++r) {
            const uint16_t v = *reinterpret_cast<const uint16_t *>(box + r * 128 + (((e >> 3) ^ (r & 7)) << 4) + (e & 7) * 2);
            if (r < rows) to[r * c.stride + e] = v;
        }
    }
    __syncwarp();
}
// Before a warp's box is filled anew: its store has read it.
__device__ __forceinline__ void reuse(int lane) {
    if (lane == 0) ptx::bulk_wait_read();
    __syncwarp();
}

// 32 fp32 columns of a lane's row: a share of a result that is summed over stretches of K.
__device__ __forceinline__ void put_share(unsigned char *box, int lane, const uint32_t (&r)[32]) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4 *>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) =
            make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]);
}

__device__ __forceinline__ void send_share(const Job &p, const uint32_t (&r)[32], unsigned char *box, int64_t row,
                                           int col, int plane, int lane) {
    reuse(lane);
    put_share(box, lane, r);
    ptx::fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        ptx::tma_store_3d(&p.shares, col, (int)row, plane, box);
        ptx::bulk_commit();
    }
}

// An accumulator's 128 columns of one of two groups of warps, `half`: taken into registers,
// after which it is free for the next tile but one, and sent to their results.
template <typename T, typename Call>
__device__ __forceinline__ void take(const Call &call, const Job &p, const TileAt &t, uint32_t acc, uint32_t taken,
                                     int64_t row, unsigned char *box, int half, int lane) {
    constexpr bool FORWARD = Shape<Call>::kForward, KEEP = Shape<Call>::kKeep;
    auto release = [&] {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(taken);
    };
    if constexpr (Shape<Call>::kShares) {  // 64 columns of the gate and the same of up, not yet joined
        const int col = t.n * 128 + 64 * half;
        uint32_t r[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k) tc::ld32_begin(acc + 128 * (k >> 1) + 64 * half + 32 * (k & 1), r[k]);
        tc::wait_ld(r);
        release();
        if (row >= p.rows) return;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (col + 32 * (k & 1) < p.cols) send_share(p, r[k], box, row, col + 32 * (k & 1), 2 * t.part + (k >> 1), lane);
    } else if constexpr (FORWARD) {  // 64 columns of the gate and the same 64 of up
        const int col = t.n * 128 + 64 * half;
        const bool kept = row < p.rows && col < p.cols;
        Packed v[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t r[2][32];
            tc::ld32_begin(acc + 64 * half + 32 * q, r[0]);
            tc::ld32_begin(acc + 128 + 64 * half + 32 * q, r[1]);
            tc::wait_ld(r);
            if (!KEEP && q == 1) release();
            with_activation(call.act, [&](auto act) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[q].w[i] = pack2<T>(
                        activation<act>(__uint_as_float(r[0][2 * i])) * __uint_as_float(r[1][2 * i]),
                        activation<act>(__uint_as_float(r[0][2 * i + 1])) * __uint_as_float(r[1][2 * i + 1]));
            });
        }
        if (kept) {
            reuse(lane);
            put(box, lane, v);
            send(p, p.c[0], box, row, col, lane);
        }
        if constexpr (KEEP) {  // cut to 24 bits, which no number leaves and no NaN
            uint32_t lower[2][16];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t r[2][32];
                tc::ld32_begin(acc + 128 * k + 64 * half, r[0]);
                tc::ld32_begin(acc + 128 * k + 64 * half + 32, r[1]);
                tc::wait_ld(r);
                if (k == 1) release();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[q].w[i] = __byte_perm(r[q][2 * i], r[q][2 * i + 1], 0x7632);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        lower[k][8 * q + i] = __byte_perm(__byte_perm(r[q][4 * i], r[q][4 * i + 1], 0x0051),
                                                          __byte_perm(r[q][4 * i + 2], r[q][4 * i + 3], 0x0051), 0x5410);
                }
                if (!kept) continue;
                reuse(lane);
                put(box, lane, v);
                send(p, p.c[1 + k], box, row, col, lane);
            }
            if (!kept) return;
            reuse(lane);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint32_t *w = lower[c >> 2] + 4 * (c & 3);
                *reinterpret_cast<uint4 *>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            ptx::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::tma_store_2d(&call.lower, 2 * col, (int)row, box);
                ptx::bulk_commit();
            }
        }
    } else {
        const int col = t.n * 256 + 128 * half;
        uint32_t r[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k) tc::ld32_begin(acc + 128 * half + 32 * k, r[k]);
        tc::wait_ld(r);
        release();
        if (row >= p.rows) return;
        if (p.parts > 1) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                if (col + 32 * h >= p.cols) return;
                send_share(p, r[h], box, row, col + 32 * h, t.part * p.results + t.z, lane);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (col + 64 * h >= p.cols) return;
                const Packed v[2] = {pack<T>(r[2 * h]), pack<T>(r[2 * h + 1])};
                reuse(lane);
                put(box, lane, v);
                send(p, p.c[t.z], box, row, col + 64 * h, lane);
            }
        }
    }
}

template <typename T, typename Call>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kProductThreads, 1)
    product_kernel(const __grid_constant__ Call p) {
    extern __shared__ unsigned char raw[];
    constexpr bool FORWARD = Shape<Call>::kForward;
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *boxes = sm + kStages * kStageBytes;
    Barriers &bar = *reinterpret_cast<Barriers *>(boxes + kEpilogueWarps * kBox);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&bar.full[s], 1);
            ptx::mbar_init(&bar.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(&bar.done[a], 1);
            ptx::mbar_init(&bar.taken[a], 2 * kEpilogueWarps);
        }
        ptx::fence_mbar_init();
    }
    if (warp == 1) tc::tmem_alloc_pair(&bar.tmem, 512);
    tc::fence_before();
    __syncthreads();
    ptx::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = bar.tmem;
    ptx::grid_wait();

    const uint32_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const uint32_t tiles = tiles_of(p);
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            int64_t filled = 0;
            for (uint32_t i = first; ok && i < tiles; i += step) {
                uint32_t at = i;
                const Job &job = job_of(p, at);
                const TileAt t = tile_at(job, at);
                const int m = t.m * 256 + 128 * (int)rank;
                const int n = FORWARD ? t.n * 128 : t.n * 256 + 128 * (int)rank;
                for (int kb = t.begin; kb < t.end; ++kb) {
                    if (!ptx::mbar_wait_sleep(&bar.empty[s], ph ^ 1)) {
                        ok = false;
                        break;
                    }
                    unsigned char *a = sm + s * kStageBytes, *b = a + kHalf;
                    const uint32_t full = ptx::cluster_address(&bar.full[s], 0);
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&bar.full[s], 2 * kStageBytes);
                    const int pair = kb >= job.blocks_k ? 1 : 0, k = (kb - pair * job.blocks_k) * 64;
                    const CUtensorMap *ma = &job.a[t.z + pair];
                    const CUtensorMap *mb = &job.b[FORWARD ? rank : pair];
                    if (!FORWARD && job.a_outer) {
                        ptx::tma_load_2d_pair(a, ma, m, k, full);
                        ptx::tma_load_2d_pair(a + kHalf / 2, ma, m + 64, k, full);
                    } else {
                        ptx::tma_load_2d_pair(a, ma, k, m, full);
                    }
                    if (FORWARD) {
                        ptx::tma_load_2d_pair(b, mb, k, n, full);
                    } else {
                        ptx::tma_load_2d_pair(b, mb, n, k, full);
                        ptx::tma_load_2d_pair(b + kHalf / 2, mb, n + 64, k, full);
                    }
                    ++filled;
                    if (++s == kStages) s = 0, ph ^= 1;
                }
            }
            // what was loaded has been read, and the pair's arrivals are in, before either block ends
            for (int j = 0; j < kStages && j < filled; ++j) {
                if (--s < 0) s = kStages - 1, ph ^= 1;
                ok = ptx::mbar_wait_sleep(&bar.empty[s], ph) && ok;
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? tc::kIdescBf16 : 0u;
            // operands with K as the inner and as the outer dimension, and 16 of K in bytes
            const uint32_t base = ptx::smem_u32(sm);
            const uint64_t inner = tc::desc_sw128(base, 16), outer = tc::desc_sw128(base, kHalf / 2);
            const uint64_t db = tc::desc_adv(FORWARD ? inner : outer, kHalf);
            constexpr uint32_t sb = FORWARD ? 32 : 2048;
            int s = 0;
            uint32_t ph = 0, turn = 0;
            for (uint32_t i = first; ok && i < tiles; i += step, ++turn) {
                const uint32_t a = turn & 1;
                uint32_t at = i;
                const Job &job = job_of(p, at);
                const TileAt t = tile_at(job, at);
                const bool a_outer = !FORWARD && job.a_outer;
                const uint64_t da = a_outer ? outer : inner;
                const uint32_t sa = a_outer ? 2048 : 32;
                const uint32_t id = tc::idesc_f16(256, 256, a_outer, !FORWARD) | type;
                if (!ptx::mbar_wait(&bar.taken[a], ((turn >> 1) & 1) ^ 1, 1u << 22)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                for (int kb = t.begin; kb < t.end; ++kb) {
                    if (!ptx::mbar_wait(&bar.full[s], ph, 1u << 22)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma_f16_pair(tmem + a * 256, tc::desc_adv(da, s * kStageBytes + k * sa),
                                         tc::desc_adv(db, s * kStageBytes + k * sb), id, kb > t.begin || k > 0);
                    tc::commit_pair(&bar.empty[s]);
                    if (++s == kStages) s = 0, ph ^= 1;
                }
                tc::commit_pair(&bar.done[a]);
            }
        }
    } else {
        const int quarter = warp & 3;  // of the tensor memory's lanes, by the warp's number
        unsigned char *mine = boxes + (warp - 2) * kBox;
        uint32_t turn = 0;
        const uint32_t taken[2] = {ptx::cluster_address(&bar.taken[0], 0), ptx::cluster_address(&bar.taken[1], 0)};
        for (uint32_t i = first; i < tiles; i += step, ++turn) {
            uint32_t at = i;
            const Job &job = job_of(p, at);
            const TileAt t = tile_at(job, at);
            const uint32_t a = turn & 1;
            ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(&bar.done[a], (turn >> 1) & 1));
            if (!ok) break;
            tc::fence_after();
            const int64_t row = (int64_t)t.m * 256 + 128 * rank + 32 * quarter;
            take<T>(p, job, t, tmem + a * 256 + ((uint32_t)(32 * quarter) << 16), taken[a], row, mine, (warp - 2) >> 2,
                    lane);
        }
        if (lane == 0) ptx::bulk_wait_read();
    }
    if (!ok) {
        if (p.err) atomicOr(p.err, kErrTimeout);
        // what the block still has in flight ends meanwhile
        for (int i = 0; i < 100; ++i) __nanosleep(10000);
    }
    __syncthreads();
    ptx::cluster_sync();
    if (warp == 1) tc::tmem_dealloc_pair(tmem, 512);
}

template <typename T, typename Call>
cudaError_t launch_product(const Call &p, cudaStream_t stream) {
    const auto kernel = product_kernel<T, Call>;
    const cudaError_t e = smem_attr((const void *)kernel, kProductSmem);
    if (e != cudaSuccess) return e;
    const uint32_t tiles = tiles_of(p), pairs = (uint32_t)sm_count() / 2;
    return launch_early(kernel, 2 * (tiles < pairs ? tiles : pairs), kProductThreads, kProductSmem, stream, p);
}

template <typename T>
cudaError_t launch_forward(const ForwardArgs &p, bool keep, cudaStream_t stream) {
    if (p.job.parts > 1) return launch_product<T>(ForwardShares{p}, stream);
    return keep ? launch_product<T>(Forward<true>{p}, stream) : launch_product<T>(Forward<false>{p}, stream);
}

}  // namespace glu
}  // namespace gdn
