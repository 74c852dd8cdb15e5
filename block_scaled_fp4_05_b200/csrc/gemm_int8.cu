// INT8 matrix products with a scale for each token and each output channel,
//   D[m, n] = round16( (sum_k qA[m, k] qB[n, k]) sA[m] sB[n] + bias[n] ),
// dense, or grouped by expert: the rows [offsets[e], offsets[e + 1]) of A and
// D belong to expert e's weights B[e], and the offsets are read on the device.
// The sums are exact 32-bit integers (tcgen05.mma kind::i8; K <= 131071 keeps
// them in range for any codes); the scales and the bias are applied in FP32
// and the result is rounded once, to BF16 or FP16.
//
// Two kernels:
//   int8_pair_kernel   many tokens: persistent CTA pairs, tiles of 256
//                      channels x 32 to 256 tokens.  Bound by the tensor pipe.
//   int8_swap_kernel   few tokens: tiles of 128 channels x 16 to 128 tokens,
//                      K split over a cluster whose CTAs join their sums
//                      through distributed shared memory.  Bound by HBM (the
//                      weights are read once).
// Both have the weights on the MMA's fixed side and the tokens on the other.
// (gemv_int8.cu has a third, dot products, for the smallest.)
// Scales, bias and offsets are read past L1 (they may be written by the kernel
// before, which can still be running when these kernels start).
// Both take a grouped launch's tile list from the offsets themselves, so a
// call needs no size from the device and can be captured in a graph.  Offsets
// are clamped to [0, T] and made non-decreasing before use: whatever they
// hold, no access leaves the tensors.
//
// K needs no padding: the tensor maps end at K, what a box reads behind it is
// zero in shared memory, and zero codes add nothing.

#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "fp4_internal.h"
#include "int8_device.cuh"
#include "tc_device.cuh"

namespace fp4 {
namespace {

using i8::pack16;
using i8::scaled;

constexpr int I8_BM = 128;          // rows of the A-side operand per CTA
constexpr int I8_BK = 128;          // K elements (and bytes a row) per stage
constexpr int I8_MMA_K = 32;        // K per tcgen05.mma kind::i8
constexpr int I8_TILE = I8_BM * I8_BK;
constexpr int kMaxExperts = kInt8MaxExperts;
constexpr int kMaxSmem = 232448;    // dynamic shared memory of a block
constexpr int kSmSmem = 233472;     // of an SM; each block there takes 1 KB more than it asks for
constexpr int64_t kI8GroupBytes = int64_t(32) << 20;

struct I8Params {
    const float* sa;         // [M]
    const float* sb;         // [E x N]
    const float* bias;       // [E x N] or NULL
    uint16_t* D;             // [M x N], leading dimension ldd
    int64_t ldd;
    int32_t M, N;            // rows of A and D, output channels
    int32_t ks_total;        // stages of a tile (0: K = 0, the sums are zero)
    int32_t tiles_n;         // channel tiles
    int32_t stages;          // of the ring
    // pair kernel: most tokens of a tile, token tiles per group of the tile order
    int32_t bt, raster_gm;
    int32_t E;               // experts (dense: 1)
    const int32_t* offsets;  // [E + 1] (dense: NULL, one group of all M rows)
    int32_t b_static;        // B is not written by the previous kernel
};

// ------------------------------------------------------------------------
// PTX wrappers of this file
// ------------------------------------------------------------------------
// D (+)= A B^T in 32-bit integers, both operands signed 8-bit, K-major.
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_i8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::i8: signed 8-bit A and B (1 in bits 7 and
// 10), 32-bit integer D (2 in bits 4-5), K-major operands, no saturation.
__host__ __device__ constexpr uint32_t idesc_i8(int m, int n)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint32_t bar, uint32_t dst, int32_t x,
                                            int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(const CUtensorMap* map, uint32_t bar_cluster, uint32_t dst,
                                                 int32_t x, int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// One thread of a converged warp, the same one each time.  Unlike a test of
// the lane it tells the compiler that a single thread runs the branch, whose
// tensor-memory and TMA instructions take their operands from uniform
// registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t cluster_addr)
{
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

// Inclusive prefix sum / maximum over the lanes of a warp.
__device__ __forceinline__ int warp_scan_add(int v, int lane)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}
__device__ __forceinline__ int warp_scan_max(int v, int lane)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v = max(v, o);
    }
    return v;
}

// Bounds of the 32 experts from e0 (one a lane), clamped to [0, M] and made
// non-decreasing: first and end row of the lane's expert (empty past E).
// `reached` carries the largest bound of the experts before e0, and leaves as
// the largest up to here.
__device__ __forceinline__ void expert_bounds(const I8Params& p, int e0, int lane, int& reached, int& first, int& end)
{
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < p.E) {
        lo = min(max(__ldcg(p.offsets + e), 0), p.M);
        hi = min(max(__ldcg(p.offsets + e + 1), 0), p.M);
    }
    const int top = warp_scan_max(max(lo, hi), lane);   // the largest bound up to and with e + 1
    int before = __shfl_up_sync(0xFFFFFFFFu, top, 1);
    if (lane == 0) before = 0;
    first = max(max(before, reached), lo);
    end = e < p.E ? max(max(first, hi), reached) : first;
    reached = max(reached, __shfl_sync(0xFFFFFFFFu, top, 31));
}

// ------------------------------------------------------------------------
// Few tokens: one CTA computes 128 output channels of up to NT tokens over
// its share of K; the S CTAs of a cluster share the tile's K.
//   warp 0     producer: weight and token tiles of each stage by TMA
//   warp 1     tensor-memory allocation, MMA issue (128 x NT x 32)
//   warps 2-5  move the accumulator to shared memory as [token][channel]
//   warp 7     grouped: finds the next item in the offsets; warps 6 and 7
//              else only help with the end:
// then all threads add the S CTAs' sums (integers: any order gives the same
// result), each CTA for 128 / S channels, scale, and store 8 bytes at a time.
// ------------------------------------------------------------------------
constexpr int kSwapThreads = 256;
constexpr int swap_resident(int nt) { return nt == 16 ? 3 : 2; }   // CTAs an SM holds, at most

template <int NT>
struct SwapCfg {
    static constexpr int MAX_STAGES = 12;
    static constexpr int STAGE_BYTES = I8_TILE + NT * I8_BK;
    static constexpr int OFF_T = I8_TILE;
    // before the stages: barriers, sA of the tokens, sB and bias of the channels
    static constexpr int OFF_SCALE = 256;
    static constexpr int FIXED = (OFF_SCALE + (NT + 2 * I8_BM) * 4 + 1023) / 1024 * 1024;
    static constexpr int TMEM_COLS = NT < 32 ? 32 : NT;
    static constexpr int smem(int stages) { return 1024 + FIXED + stages * STAGE_BYTES; }
    static_assert((2 * MAX_STAGES + 1) * 8 + 40 <= OFF_SCALE, "barrier area");
};

// Adds the S CTAs' sums for this CTA's channels, scales and stores.  A thread
// has four channels (the same ones for all its tokens) and every
// (kSwapThreads / pieces)-th token, U of them at a time: a read of another
// CTA's memory takes about a microsecond, so many are kept in flight.
template <int S, bool HALF>
__device__ __forceinline__ void swap_finish(const I8Params& p, uint32_t sums, const float* sas, const float* sbs,
                                            int rank, int row0, int ntok, int n0)
{
    constexpr int PIECES = I8_BM / 4 / S;
    constexpr int STEP = kSwapThreads / PIECES;
    constexpr int U = S == 8 ? 1 : S == 4 ? 2 : 4;
    static_assert(kSwapThreads % PIECES == 0, "a thread keeps its channels");
    const int ch = (rank * PIECES + threadIdx.x % PIECES) * 4;   // within the tile
    const int n = n0 + ch;
    if (n >= p.N) return;
    const float4 sb = *reinterpret_cast<const float4*>(sbs + ch);
    const float4 bias = *reinterpret_cast<const float4*>(sbs + I8_BM + ch);
    uint32_t from[S];
#pragma unroll
    for (int r = 0; r < S; ++r) from[r] = map_to_rank(sums + ch * 4u, r);
    for (int tok0 = threadIdx.x / PIECES; tok0 < ntok; tok0 += U * STEP) {
        int4 v[U][S];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < S; ++r)
                if (u == 0 || tok0 + u * STEP < ntok)
                    v[u][r] = ld_cluster_v4(from[r] + (uint32_t)(tok0 + u * STEP) * (I8_BM * 4));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int tok = tok0 + u * STEP;
            if (tok >= ntok) break;
            int4 sum = v[u][0];
#pragma unroll
            for (int r = 1; r < S; ++r) {
                sum.x += v[u][r].x;
                sum.y += v[u][r].y;
                sum.z += v[u][r].z;
                sum.w += v[u][r].w;
            }
            const float sa = sas[tok];
            const uint32_t lo = pack16<HALF>(scaled(sum.x, sa, sb.x, bias.x), scaled(sum.y, sa, sb.y, bias.y));
            const uint32_t hi = pack16<HALF>(scaled(sum.z, sa, sb.z, bias.z), scaled(sum.w, sa, sb.w, bias.w));
            uint16_t* d = p.D + (int64_t)(row0 + tok) * p.ldd + n;
            if (n + 4 <= p.N) {
                *reinterpret_cast<uint2*>(d) = make_uint2(lo, hi);
            } else {
                d[0] = (uint16_t)lo;
                if (n + 1 < p.N) d[1] = (uint16_t)(lo >> 16);
                if (n + 2 < p.N) d[2] = (uint16_t)hi;
            }
        }
    }
}

template <int NT, bool HALF>
__global__ void __launch_bounds__(kSwapThreads)
int8_swap_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                 const I8Params p)
{
    using C = SwapCfg<NT>;
    const int stages = p.stages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
    // [0,12) full, [12,24) empty, [24] accumulator full
    int* shared_word = reinterpret_cast<int*>(bars + 2 * C::MAX_STAGES + 1);
    // [0] tensor-memory base, [1] abort; [2..5] and [6..9] the item (grouped,
    // even and odd ones): expert (-1: none), first row, rows, tile within the expert
    volatile int* abort_flag = shared_word + 1;
    float* sas = reinterpret_cast<float*>(smem + C::OFF_SCALE);   // [NT]
    float* sbs = sas + NT;                                        // [128], then the bias [128]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint32_t split;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    const int rank = (int)cluster_rank();
    const int kb = (int)((int64_t)p.ks_total * rank / (int)split);
    const int ke = (int)((int64_t)p.ks_total * (rank + 1) / (int)split);
    const uint32_t smem0 = smem_u32(smem) + C::FIXED;   // first stage
    const uint32_t bar0 = smem_u32(bars);
    auto FULL = [&](int s) { return bar0 + 8u * s; };
    auto EMPTY = [&](int s) { return bar0 + 8u * (C::MAX_STAGES + s); };
    const uint32_t acc_full = bar0 + 8u * (2 * C::MAX_STAGES);
    // Items: the tiles (expert, channel tile, token tile), token tiles
    // fastest so that clusters that share weights run next to each other,
    // dealt round-robin to the clusters.
    const int cluster = (int)(blockIdx.x / split), clusters = (int)(gridDim.x / split);
    const int dense_mt = (p.M + NT - 1) / NT;
    // Weight tiles requested before the dependency wait (static weights of a
    // dense product): those of the first stages, their token tiles follow.
    int pre = !p.offsets && p.b_static ? min(stages, ke - kb) : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(FULL(s), 1);
            mbar_init(EMPTY(s), 1);
        }
        mbar_init(acc_full, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        for (int i = 0; i < pre; ++i) {
            mbar_arrive_expect_tx(FULL(i), C::STAGE_BYTES);
            tma_load_3d(&tmW, FULL(i), smem0 + i * C::STAGE_BYTES, (kb + i) * I8_BK, cluster / dense_mt * I8_BM, 0);
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(shared_word)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // Item c of a grouped launch, found by one warp (into the words of its parity).
    auto find_item = [&](int64_t c, int odd) {
        int* word = shared_word + 2 + 4 * odd;
        int64_t seen = 0;   // tiles of the experts before e0
        int reached = 0, found = 0;
        for (int e0 = 0; e0 < p.E && !found; e0 += 32) {
            int first, end;
            expert_bounds(p, e0, lane, reached, first, end);
            const int mt = (end - first + NT - 1) / NT;
            const int upto = warp_scan_add(mt, lane);   // token tiles up to this expert
            const int64_t from = seen + (int64_t)(upto - mt) * p.tiles_n;
            const bool mine = c >= from && c < from + (int64_t)mt * p.tiles_n;
            if (mine) {
                word[0] = e0 + lane;
                word[1] = first;
                word[2] = end - first;
                word[3] = (int)(c - from);
            }
            found = __any_sync(0xFFFFFFFFu, mine);
            seen += (int64_t)__shfl_sync(0xFFFFFFFFu, upto, 31) * p.tiles_n;
        }
        if (!found && lane == 0) word[0] = -1;
    };
    __syncwarp();
    if (p.offsets && warp == 7) {
        pdl_wait();
        find_item(cluster, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = (uint32_t)shared_word[0];
    pdl_wait();

    int stage = 0, odd = 0;
    uint32_t phase = 0, acc_phase = 0;
    for (int64_t c = cluster;; c += clusters, odd ^= 1) {
        int expert = 0, first = 0, rows = p.M, tile = (int)c;
        if (p.offsets) {
            const int* word = shared_word + 2 + 4 * odd;
            expert = word[0];
            first = word[1];
            rows = word[2];
            tile = word[3];
            if (expert < 0) break;   // no rows at all (the same in every CTA of the cluster)
        }
        const int mt = (rows + NT - 1) / NT;
        const int tm = tile % mt, tn = tile / mt;
        const int row0 = first + tm * NT;        // first token
        const int ntok = min(NT, rows - tm * NT);

        if (warp == 0) {
            if (elect_one()) {
                bool ok = true;
                for (int ks = kb; ks < ke; ++ks) {
                    const uint32_t st = smem0 + stage * C::STAGE_BYTES;
                    if (pre > 0) {
                        --pre;   // this stage's weight tile is on its way
                    } else {
                        if (!wait_fast(EMPTY(stage), phase ^ 1u, abort_flag, ERR_EMPTY)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(FULL(stage), C::STAGE_BYTES);
                        tma_load_3d(&tmW, FULL(stage), st, ks * I8_BK, tn * I8_BM, expert);
                    }
                    tma_load_2d(&tmX, FULL(stage), st + C::OFF_T, ks * I8_BK, row0);
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                // Once the first item's loads are issued the next kernel may
                // start: before them, its first weight loads beside this
                // one's cost more than they hid (1x28672x8192, call after
                // call: 39.8 us, 48 with the trigger at the start).  Where a
                // cluster takes several items in turn, waiting for the last
                // one's gains nothing: 16x28672x1024 6.5 -> 6.7 us, 16 rows
                // over 8 experts of 14336x4096 72 -> 76, 500 over 64 of
                // 4096x1024 45.3 -> 44.7.
                pdl_trigger();
                if (!ok || *abort_flag) spin_ns(200000);   // loads in flight land before the memory is used again
            }
            __syncwarp();
        } else if (warp == 1) {
            if (kb < ke && elect_one()) {
                const uint64_t adesc0 = desc_sw128(smem0);
                const uint64_t bdesc0 = desc_sw128(smem0 + C::OFF_T);
                for (int ks = kb; ks < ke; ++ks) {
                    if (!wait_fast(FULL(stage), phase, abort_flag, ERR_FULL)) break;
                    tc_fence_after();
                    const uint64_t step = (uint64_t)(stage * (C::STAGE_BYTES >> 4));
#pragma unroll
                    for (int j = 0; j < I8_BK / I8_MMA_K; ++j)
                        mma_i8(tmem_base, adesc0 + step + 2 * j, bdesc0 + step + 2 * j, idesc_i8(I8_BM, NT),
                               (ks > kb || j > 0) ? 1u : 0u);
                    tc_commit(EMPTY(stage));
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                // completes when every MMA issued here has
                tc_commit(acc_full);
            }
            __syncwarp();
        } else if (warp < 6) {
            const int i = threadIdx.x - 64;
            const int64_t chan = (int64_t)expert * p.N + tn * I8_BM + i;
            const bool in = tn * I8_BM + i < p.N;
            if (i < ntok) sas[i] = __ldcg(p.sa + row0 + i);
            sbs[i] = in ? __ldcg(p.sb + chan) : 0.0f;
            sbs[I8_BM + i] = in && p.bias ? __ldcg(p.bias + chan) : 0.0f;
            const int q = warp & 3;   // tensor-memory lane quadrant: channels [32 q, 32 q + 32)
            const uint32_t dst = smem0 + (uint32_t)(q * 32 + lane) * 4u;
            const bool have = kb < ke && warp_wait(acc_full, acc_phase, abort_flag, ERR_ACC_FULL);
            acc_phase ^= 1u;
            tc_fence_after();
            // Every stage has been read by then (the MMAs are complete) and
            // none is being filled, so the sums take their place.
#pragma unroll
            for (int col = 0; col < NT; col += 16) {
                if (col >= ntok) break;
                uint32_t r[16];
                if (have) {
                    tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + col, r);
                    tmem_wait_ld(r);
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) r[k] = 0u;
                }
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + (uint32_t)(col + k) * (I8_BM * 4)), "r"(r[k])
                                 : "memory");
            }
        } else if (warp == 7 && p.offsets) {
            find_item(c + clusters, odd ^ 1);
        }
        tc_fence_before();
        __syncwarp();
        if (split > 1)
            cluster_sync();
        else
            __syncthreads();
        tc_fence_after();
        if (split == 1)
            swap_finish<1, HALF>(p, smem0, sas, sbs, rank, row0, ntok, tn * I8_BM);
        else if (split == 2)
            swap_finish<2, HALF>(p, smem0, sas, sbs, rank, row0, ntok, tn * I8_BM);
        else if (split == 4)
            swap_finish<4, HALF>(p, smem0, sas, sbs, rank, row0, ntok, tn * I8_BM);
        else
            swap_finish<8, HALF>(p, smem0, sas, sbs, rank, row0, ntok, tn * I8_BM);
        const bool more = p.offsets ? shared_word[2 + 4 * (odd ^ 1)] >= 0 : c + clusters < (int64_t)dense_mt * p.tiles_n;
        // The sums have been read, by the other CTAs too, before the next
        // item's loads (or this CTA's end) touch their memory.
        if (more) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (split > 1)
            cluster_sync();
        else if (more)
            __syncthreads();
        if (!more) break;
    }
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(C::TMEM_COLS)
                     : "memory");
}

// ------------------------------------------------------------------------
// Many tokens: a cluster of two CTAs computes 256 channels of up to bt tokens
// with pair MMAs (M = 256 channels, N = a multiple of 32 tokens up to 256):
// each CTA stages its own 128 rows of weights and half of the tile's tokens.
// The weights are on the MMA's fixed side, so that a group's last tile can be
// as narrow as its rows: 8192 rows over 8 experts of 14336x4096 332 us, 352
// with the tokens on that side; 7104 over 64 of 6103x1024 85 against 110 us;
// one group of whole tiles the same within 3 %.  Two accumulators in tensor memory, so that a
// tile's epilogue runs beside the next tile's MMAs.
//   warp 0      producer (both CTAs; loads complete on the leader's full[s])
//   warp 1      MMA issue (leader): passes a stage's named barrier, issues
//               four MMAs and the commit that releases the stage in both
//               CTAs; it touches no mbarrier, since a probe between two
//               stages' MMAs leaves the tensor pipe idle
//   warp 2      gatekeeper (leader): waits for the accumulator's release and
//               for each stage, then opens the stage's named barrier
//   warp 3      grouped: the tile list from the offsets
//   warps 4-11  epilogue: two warps a tensor-memory lane quadrant (32
//               channels), 32 tokens in turn; scaled, rounded, turned into
//               rows through the warp's block of shared memory, stored four
//               lanes a row
// Every wait is bounded; a CTA that gives up records it in the error word.
// ------------------------------------------------------------------------
constexpr int kI8EpiWarps = 8;
constexpr int kI8PairThreads = 128 + 32 * kI8EpiWarps;
constexpr int kI8PairMaxStages = 12;

struct I8Pair {
    static constexpr int OFF_EPI = 0;                                         // a warp's 32 tokens x 32 channels of results
    static constexpr int OFF_SA = OFF_EPI + kI8EpiWarps * 32 * 32 * 2;        // sA of a warp's tokens
    static constexpr int OFF_LIST = OFF_SA + kI8EpiWarps * 128 * 4;           // experts' first tiles and rows
    static constexpr int OFF_BARS = OFF_LIST + 2 * (kMaxExperts + 2) * 4;
    static constexpr int NBARS = 2 * kI8PairMaxStages + 5;
    static constexpr int FIXED = (OFF_BARS + 256 + 1023) / 1024 * 1024;       // what lies before the stages
    static constexpr int SMEM = kMaxSmem;
    static constexpr int STAGE_ROOM = SMEM - 1024 - FIXED;
    static_assert(NBARS * 8 + 8 <= 256, "barrier area");
    static_assert(OFF_BARS % 16 == 0, "barrier alignment");
    static_assert(kI8PairMaxStages + 1 <= 16, "one named barrier per stage (ids from 1)");
    static_assert(STAGE_ROOM >= 6 * (I8_TILE + 128 * I8_BK), "six stages of the widest tile");
    // a CTA's share of a stage with `width` tokens
    __host__ __device__ static constexpr int stage_bytes(int width) { return I8_TILE + width / 2 * I8_BK; }
    static constexpr int stages(int bt)
    {
        const int n = STAGE_ROOM / stage_bytes(bt);
        return n < kI8PairMaxStages ? n : kI8PairMaxStages;
    }
};

// The tokens with boxes of one to four quarters of a CTA's share of the widest
// tile: a narrower tile is loaded by the smallest that holds it, in one piece
// (pieces of 16 rows cost more: a tile half as wide 18.6 instead of 12.3 us).
struct TokenMaps {
    CUtensorMap q[4];
};

template <bool HALF, bool GROUPED>
__global__ void __launch_bounds__(kI8PairThreads, 1)
int8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ TokenMaps tmX, const I8Params p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + I8Pair::OFF_BARS);
    // [0,12) full (leader), [12,24) empty, [24..25] acc_full, [26..27] acc_empty (leader), [28] drain
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + I8Pair::NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* list = reinterpret_cast<int*>(smem + I8Pair::OFF_LIST);   // [E + 1] first tile of each expert
    int* bound = list + kMaxExperts + 2;                           // [E + 1] its first row

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int stages = p.stages;
    const uint32_t stage_bytes = (uint32_t)I8Pair::stage_bytes(p.bt);
    const uint32_t smem0 = smem_u32(smem) + I8Pair::FIXED;   // first stage
    const uint32_t bar0 = smem_u32(bars);
    auto FULL = [&](int s) { return bar0 + 8u * s; };
    auto EMPTY = [&](int s) { return bar0 + 8u * (kI8PairMaxStages + s); };
    auto ACC_FULL = [&](int b) { return bar0 + 8u * (2 * kI8PairMaxStages + b); };
    auto ACC_EMPTY = [&](int b) { return bar0 + 8u * (2 * kI8PairMaxStages + 2 + b); };
    const uint32_t drain = bar0 + 8u * (2 * kI8PairMaxStages + 4);

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(FULL(s), 1);
            mbar_init(EMPTY(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(ACC_FULL(b), 1);
            mbar_init(ACC_EMPTY(b), 2 * kI8EpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (GROUPED && warp == 3) {
        pdl_wait();
        int reached = 0, seen = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            int first, end;
            expert_bounds(p, e0, lane, reached, first, end);
            const int tiles = (end - first + p.bt - 1) / p.bt * p.tiles_n;
            const int upto = warp_scan_add(tiles, lane);
            if (e0 + lane < p.E) {
                list[e0 + lane] = seen + upto - tiles;
                bound[e0 + lane] = first;
                if (e0 + lane == p.E - 1) {
                    list[p.E] = seen + upto;
                    bound[p.E] = end;
                }
            }
            seen += __shfl_sync(0xFFFFFFFFu, upto, 31);
        }
    }
    tc_fence_before();
    cluster_sync();   // barriers of both CTAs initialised, TMEM allocated, tile list written
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const int pair = blockIdx.x >> 1;
    const int npairs = gridDim.x >> 1;
    const int tiles = GROUPED ? list[p.E] : (p.M + p.bt - 1) / p.bt * p.tiles_n;
    // Work items: the tiles, dealt round-robin.  A last, partial wave whose
    // halves fit on the pairs is computed as halves, of the tokens.
    const int rem = tiles % npairs;
    const int split_from = 2 * rem <= npairs ? tiles - rem : tiles;
    const int items = 2 * tiles - split_from;
    // Expert, first token, first channel and width (tokens rounded up to 32;
    // 0: nothing to do) of item t, and the end of the expert's rows.  Within
    // an expert groups of raster_gm consecutive token tiles sweep the channel
    // tiles together (token tiles fastest), so that a group's tokens stay in
    // L2 while the weights stream past them once.
    struct Place {
        int e, row, col, width, row_end;
    };
    auto locate = [&](int t) {
        Place w;
        int half = 0;
        const bool halved = t >= split_from;
        if (halved) {
            half = (t - split_from) & 1;
            t = split_from + ((t - split_from) >> 1);
        }
        int lo = 0, base = 0, end = p.M;
        if (GROUPED) {
            int hi = p.E;   // list[lo] <= t < list[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (list[mid] <= t) lo = mid;
                else hi = mid;
            }
            t -= list[lo];
            base = bound[lo];
            // an empty expert has no tile, so lo is the one that holds t; its
            // rows end where the next expert's begin
            end = bound[lo + 1];
        }
        const int tiles_m = (end - base + p.bt - 1) / p.bt;
        const int span = p.raster_gm * p.tiles_n;
        const int grp = t / span, in = t - grp * span;
        const int m0 = grp * p.raster_gm;
        const int gm = min(tiles_m - m0, p.raster_gm);
        w.e = lo;
        w.row = base + (m0 + in % gm) * p.bt;
        w.col = in / gm * 256;
        w.width = min(p.bt, (end - w.row + 31) & ~31);
        w.row_end = end;
        if (halved) {
            const int upper = (w.width / 2 + 31) & ~31;   // the first half's tokens
            w.row += half * upper;
            w.width = half ? w.width - upper : upper;
        }
        return w;
    };

    if (warp == 0) {
        if (elect_one()) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmW)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmX.q[3])) : "memory");
            auto box = [&](const Place& w) { return (w.width * 4 + p.bt - 1) / p.bt; };   // quarters
            auto load_w = [&](const Place& w, int s, int ks) {
                if (leader) mbar_arrive_expect_tx(FULL(s), 2u * (I8_TILE + box(w) * (p.bt / 8) * I8_BK));
                tma_load_3d_pair(&tmW, map_to_rank(FULL(s), 0), smem0 + s * stage_bytes, ks * I8_BK,
                                 w.col + (int)rank * I8_BM, w.e);
            };
            int stage = 0, pre = 0;
            uint32_t phase = 0;
            bool ok = true;
            if (!GROUPED && p.b_static && pair < items) {
                // static weights: those of the first stages are requested
                // before the dependency wait
                const Place w = locate(pair);
                if (w.width > 0)
                    for (; pre < stages && pre < p.ks_total; ++pre) load_w(w, pre, pre);
            }
            pdl_wait();
            for (int t = pair; ok && t < items; t += npairs) {
                const Place w = locate(t);
                if (w.width == 0) continue;
                const CUtensorMap* map = &tmX.q[box(w) - 1];
                const int y = w.row + (int)rank * (w.width / 2);   // this CTA's half of the tokens
                for (int ks = 0; ks < p.ks_total; ++ks) {
                    if (pre > 0) {
                        --pre;   // this stage's weights are on their way
                    } else {
                        if (!wait_fast(EMPTY(stage), phase ^ 1u, abort_flag, ERR_EMPTY)) {
                            ok = false;
                            break;
                        }
                        load_w(w, stage, ks);
                    }
                    tma_load_3d_pair(map, map_to_rank(FULL(stage), 0), smem0 + stage * stage_bytes + I8_TILE, ks * I8_BK, y,
                                     0);
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            pdl_trigger();
            if (!ok || *abort_flag) spin_ns(200000);   // loads in flight land before the CTAs meet
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            const uint64_t adesc0 = desc_sw128(smem0);
            const uint64_t bdesc0 = desc_sw128(smem0 + I8_TILE);
            int stage = 0, buf = 0;
            for (int t = pair; t < items; t += npairs) {
                const int width = locate(t).width;
                if (width == 0) continue;
                const uint32_t acc = tmem_base + (uint32_t)(buf * 256);
                const uint32_t idesc = idesc_i8(256, width);
                for (int ks = 0; ks < p.ks_total; ++ks) {
                    named_bar_sync(1 + stage, 64);
                    if (elect_one()) {
                        tc_fence_after();
                        const uint64_t step = (uint64_t)((uint32_t)stage * (stage_bytes >> 4));
#pragma unroll
                        for (int j = 0; j < I8_BK / I8_MMA_K; ++j)
                            mma_i8_pair(acc, adesc0 + step + 2 * j, bdesc0 + step + 2 * j, idesc,
                                        (ks > 0 || j > 0) ? 1u : 0u);
                        tc_commit_pair_both(EMPTY(stage));
                    }
                    __syncwarp();
                    if (++stage == stages) stage = 0;
                }
                if (elect_one()) tc_commit_pair_both(ACC_FULL(buf));
                __syncwarp();
                buf ^= 1;
            }
            if (elect_one()) {
                // every pair MMA issued here has completed before the TMEM is freed
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drain)
                             : "memory");
                wait_drain(drain, 0);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // After a wait that gave up the gatekeeper goes on opening barriers
        // without waiting, so that the MMA warp is never left blocked.
        if (leader) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int t = pair; t < items; t += npairs) {
                if (locate(t).width == 0) continue;
                if (ok && !warp_wait(ACC_EMPTY(buf), acc_phase ^ 1u, abort_flag, ERR_ACC_EMPTY)) ok = false;
                for (int ks = 0; ks < p.ks_total; ++ks) {
                    if (ok && !warp_wait(FULL(stage), phase, abort_flag, ERR_FULL)) ok = false;
                    named_bar_arrive(1 + stage, 64);
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                buf ^= 1;
                if (buf == 0) acc_phase ^= 1u;
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3;                  // tensor-memory lane quadrant
        const int half = (warp - 4) >> 2;        // the warp's 32-token chunks: half, half + 2, ...
        float* sas = reinterpret_cast<float*>(smem + I8Pair::OFF_SA) + (warp - 4) * 128;
        const uint32_t blk = smem_u32(smem) + I8Pair::OFF_EPI + (warp - 4) * (32 * 32 * 2);
        pdl_wait();
        // The scales of an item (this lane's channel, a token of each chunk)
        // are read while the item before it is worked on.
        Place next = {};
        float sb_next = 0.0f, bias_next = 0.0f, sa_next[4] = {};
        auto fetch = [&](int t) {
            if (t >= items) return;
            next = locate(t);
            const int n = next.col + (int)rank * I8_BM + q * 32 + lane;
            const int64_t chan = (int64_t)next.e * p.N + n;
            sb_next = n < p.N ? __ldcg(p.sb + chan) : 0.0f;
            bias_next = n < p.N && p.bias ? __ldcg(p.bias + chan) : 0.0f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int y = next.row + (half + 2 * c) * 32 + lane;
                sa_next[c] = (half + 2 * c) * 32 < next.width && y < next.row_end ? __ldcg(p.sa + y) : 0.0f;
            }
        };
        fetch(pair);
        uint32_t acc_phase = 0;
        int buf = 0;
        for (int t = pair; t < items; t += npairs) {
            const Place w = next;
            const float sb = sb_next, bias = bias_next;
            __syncwarp();   // the scales' memory has been read
#pragma unroll
            for (int c = 0; c < 4; ++c) sas[c * 32 + lane] = sa_next[c];
            __syncwarp();
            fetch(t + npairs);
            if (w.width == 0) continue;
            const int chunks = (w.width / 32 - half + 1) >> 1;   // 0 to 4
            const int x0 = w.col + (int)rank * I8_BM + q * 32;   // the warp's first channel
            if (!warp_wait(ACC_FULL(buf), acc_phase, abort_flag, ERR_ACC_FULL)) break;
            tc_fence_after();
            const uint32_t trow = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * 256 + half * 32);
            uint32_t r2[2][32];
            if (chunks > 0) tmem_ld32(trow, r2[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t (&r)[32] = r2[c & 1];
                if (c < chunks) tmem_wait_ld(r);
                if (c + 1 < chunks) {   // the next chunk's load overlaps this one's arithmetic
                    tmem_ld32(trow + (uint32_t)((c + 1) * 64), r2[(c + 1) & 1]);
                } else if (c == max(chunks - 1, 0)) {
                    // every column is in registers: hand the accumulator back
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (leader)
                            mbar_arrive(ACC_EMPTY(buf));
                        else
                            mbar_arrive_cluster_relaxed(map_to_rank(ACC_EMPTY(buf), 0));
                    }
                }
                const int y0 = w.row + (half + 2 * c) * 32;
                if (c < chunks && y0 < w.row_end && x0 < p.N) {
                    // 32 tokens x 32 channels of results: token i's in row i
                    // (64 bytes), whose 16-byte pieces are rotated so that the
                    // reads below are free of bank conflicts
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 sa = *reinterpret_cast<const float4*>(sas + c * 32 + i);
                        const uint32_t lo = pack16<HALF>(scaled((int)r[i], sa.x, sb, bias), scaled((int)r[i + 1], sa.y, sb, bias));
                        const uint32_t hi = pack16<HALF>(scaled((int)r[i + 2], sa.z, sb, bias), scaled((int)r[i + 3], sa.w, sb, bias));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t v = k < 2 ? lo : hi;
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(
                                             blk + (i + k) * 64 + (((lane >> 3) ^ (((i + k) >> 1) & 3)) << 4) + 2 * (lane & 7)),
                                         "h"((uint16_t)(k & 1 ? v >> 16 : v))
                                         : "memory");
                        }
                    }
                    __syncwarp();
                    const int x = x0 + 8 * (lane & 3);   // four lanes a token
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int i = 8 * k + (lane >> 2);
                        const uint4 v = ld_shared_v4(blk + i * 64 + (((lane & 3) ^ ((i >> 1) & 3)) << 4));
                        if (y0 + i >= w.row_end) break;   // the next expert's row, or none
                        uint16_t* d = p.D + (int64_t)(y0 + i) * p.ldd + x;
                        if (x + 8 <= p.N) {
                            *reinterpret_cast<uint4*>(d) = v;
                        } else {
                            const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (x + j < p.N) d[j] = (uint16_t)(word[j >> 1] >> (16 * (j & 1)));
                        }
                    }
                }
            }
            buf ^= 1;
            if (buf == 0) acc_phase ^= 1u;
        }
    }

    tc_fence_before();
    cluster_sync();   // all pair MMAs done, both epilogues finished reading TMEM
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
}

// ------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------
// [depth x rows x cols] bytes, boxes of 128 bytes x box_rows, 128-byte
// swizzle, zero outside.
bool make_map_i8(CUtensorMap* m, const void* base, int64_t depth, int64_t rows, int64_t cols, int64_t ld,
                 int64_t stride, int box_rows)
{
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)depth};
    cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)stride};
    cuuint32_t box[3] = {(cuuint32_t)I8_BK, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_map_i8_2d(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows)
{
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {(cuuint32_t)I8_BK, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Raises a kernel's dynamic shared-memory limit once per device; each caller
// passes a mask of its own.
cudaError_t raise_smem(const void* kernel, int bytes, uint64_t& done_mask)
{
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && ((done_mask >> dev) & 1ull)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done_mask |= 1ull << dev;
    return e;
}

void launch_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], unsigned grid, unsigned threads,
                   unsigned cluster, size_t smem, cudaStream_t s)
{
    cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
}

I8Params params_of(const Int8GemmArgs& a, int bn)
{
    I8Params p;
    p.sa = a.sA;
    p.sb = a.sB;
    p.bias = a.bias;
    p.D = a.D;
    p.ldd = a.ldd;
    p.M = (int32_t)a.M;
    p.N = (int32_t)a.N;
    p.ks_total = (int32_t)((a.K + I8_BK - 1) / I8_BK);
    p.tiles_n = (int32_t)((a.N + bn - 1) / bn);
    p.bt = 0;
    p.stages = 0;
    p.raster_gm = 1;
    p.E = (int32_t)a.E;
    p.offsets = a.offsets;
    p.b_static = a.b_static ? 1 : 0;
    return p;
}

// How many clusters of the few-token kernel run at once with one, two or three
// CTAs an SM (its share of the shared memory each).  Clusters do not cross the
// SMs' groups (GPCs), whose sizes are no multiples of 4 or 8 and differ from
// one GPU to the next: 148 SMs hold 15 clusters of 8 at a CTA each, not 18.
struct Held {
    int n[4][3];   // by log2 of the cluster's size and CTAs an SM
    int of(int split, int ctas) const { return n[split >= 8 ? 3 : split >= 4 ? 2 : split - 1][ctas - 1]; }
};

// The occupancy query counts one CTA an SM for any kernel with tensor memory,
// so it is asked about this one, which is never launched.
__global__ void __launch_bounds__(kSwapThreads) occupancy_stand_in() {}

Held query_held(int sm_count)
{
    Held h;
    static uint64_t done = 0;
    const void* kern = reinterpret_cast<const void*>(occupancy_stand_in);
    for (int i = 0; i < 12; ++i) {
        const int split = 1 << (i / 3), ctas = i % 3 + 1;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        launch_config(cfg, attr, (unsigned)(split * sm_count * ctas), kSwapThreads, (unsigned)split,
                      (size_t)(kSmSmem / ctas - 1024), nullptr);
        cfg.numAttrs = 1;
        int n = 0;
        if (raise_smem(kern, kMaxSmem, done) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = sm_count * ctas / split;   // (only a launch's speed hangs on it)
        }
        h.n[i / 3][i % 3] = n;
    }
    return h;
}

// Of the current device, asked once.
Held held_clusters(int sm_count)
{
    static std::mutex mu;
    static Held known[64];
    static uint64_t have = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return query_held(sm_count);
    std::lock_guard<std::mutex> lock(mu);
    if (!((have >> dev) & 1ull)) {
        known[dev] = query_held(sm_count);
        have |= 1ull << dev;
    }
    return known[dev];
}

// CTAs an SM of a launch, the fewest that run all its clusters at once.
int swap_ctas(int nt, int split, double clusters, const Held& held)
{
    int ctas = 1;
    while (ctas < swap_resident(nt) && clusters > held.of(split, ctas)) ++ctas;
    return ctas;
}

// Stages of the few-token kernel: those of a CTA's share of K, as far as they
// fit beside the other CTAs of the SM.
//
// A cluster asks for two at least, so that its CTAs never share an SM with
// those of the FP4 pair GEMM on another stream.  Both wait for tensor memory
// without a limit, and both wait for the rest of their cluster: with a CTA of
// each on two SMs, one ahead on either, none of the four would ever go on.
// (One stage: 21.5 KB, which fit beside the pair GEMM of MXFP4.  A CTA that is
// no cluster's waits for nothing but the tensor memory.)
constexpr int kClusterStages = 2;
static_assert(SwapCfg<16>::smem(kClusterStages) + 1024 + kFp4PairSmem + 1024 > kSmSmem, "no room for both on an SM");
constexpr int swap_stages(int nt, int split, int ctas, int share)
{
    const int bytes = I8_TILE + nt * I8_BK, fixed = 1024 + SwapCfg<128>::FIXED;
    const int room = (kSmSmem / ctas - 1024 - fixed) / bytes;
    const int sums = (nt * I8_BM * 4 + bytes - 1) / bytes;   // the sums take their memory
    const int least = split > 1 && sums < kClusterStages ? kClusterStages : sums;
    const int n = share < room ? share : room;
    return n < least ? least : n > SwapCfg<128>::MAX_STAGES ? SwapCfg<128>::MAX_STAGES : n;
}

// As many CTAs as an SM's shared memory holds, whatever their tiles, ask for no
// more than its 512 columns of tensor memory.
template <int NT>
constexpr bool columns_suffice(int split)
{
    return (int64_t)SwapCfg<NT>::TMEM_COLS * kSmSmem <= 512ll * (SwapCfg<NT>::smem(swap_stages(NT, split, 3, 1)) + 1024);
}
static_assert(columns_suffice<16>(1) && columns_suffice<32>(1) && columns_suffice<64>(1) && columns_suffice<128>(1),
              "tensor memory of the CTAs on an SM");

template <int NT, bool HALF>
cudaError_t launch_swap(const Int8GemmArgs& a, int split, int64_t clusters, const Held& held, cudaStream_t s)
{
    using C = SwapCfg<NT>;
    CUtensorMap tw = {}, tx = {};
    if (a.K > 0 && (!make_map_i8(&tw, a.B, a.E, a.N, a.K, a.ldb, a.stride_b, I8_BM) ||
                    !make_map_i8_2d(&tx, a.A, a.M, a.K, a.lda, NT))) {
        set_last_error("cuTensorMapEncodeTiled", cudaErrorInvalidValue);
        return cudaErrorInvalidValue;
    }
    static uint64_t done = 0;
    auto kern = int8_swap_kernel<NT, HALF>;
    constexpr int most = C::smem(C::MAX_STAGES) < kMaxSmem ? C::smem(C::MAX_STAGES) : kMaxSmem;
    cudaError_t e = raise_smem(reinterpret_cast<const void*>(kern), most, done);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        // as many clusters as the SMs hold take all tiles in turn
        const int64_t hold = held.of(split, swap_resident(NT));
        const unsigned grid = (unsigned)((clusters < hold ? clusters : hold) * split);
        I8Params p = params_of(a, I8_BM);
        p.stages = swap_stages(NT, split, swap_ctas(NT, split, (double)clusters, held), (p.ks_total + split - 1) / split);
        launch_config(cfg, attr, grid, kSwapThreads, (unsigned)split, C::smem(p.stages), s);
        e = cudaLaunchKernelEx(&cfg, kern, tw, tx, p);
    }
    if (e != cudaSuccess) set_last_error("INT8 GEMM launch (few tokens)", e);
    return e;
}

template <bool HALF, bool GROUPED>
cudaError_t launch_pair(const Int8GemmArgs& a, int bt, int64_t tiles, int sm_count, cudaStream_t s)
{
    I8Params p = params_of(a, 256);
    p.bt = bt;
    p.stages = I8Pair::stages(bt);
    const int64_t pairs = sm_count / 2, grid = tiles < pairs ? tiles : pairs;
    CUtensorMap tw;
    TokenMaps tx = {};
    // only the whole box where every tile is whole
    const bool narrow = GROUPED || a.M % bt != 0 || 2 * (tiles % grid) <= grid;
    bool ok = make_map_i8(&tw, a.B, a.E, a.N, a.K, a.ldb, a.stride_b, I8_BM);
    for (int q = narrow ? 1 : 4; q <= 4; ++q)
        ok = ok && make_map_i8(&tx.q[q - 1], a.A, 1, a.M, a.K, a.lda, a.lda, bt / 8 * q);
    if (!ok) {
        set_last_error("cuTensorMapEncodeTiled", cudaErrorInvalidValue);
        return cudaErrorInvalidValue;
    }
    // token tiles per group: as many as hold kI8GroupBytes of A, all of them
    // when A fits in half of the L2 cache
    const int64_t tile_bytes = bt * a.K, tiles_m = (a.M + bt - 1) / bt;
    int64_t rg = tiles_m;
    if (tile_bytes * tiles_m > 2 * kI8GroupBytes) rg = (kI8GroupBytes + tile_bytes / 2) / tile_bytes;
    p.raster_gm = (int32_t)(rg < 1 ? 1 : rg > tiles_m ? tiles_m : rg);
    static uint64_t done = 0;
    auto kern = int8_pair_kernel<HALF, GROUPED>;
    cudaError_t e = raise_smem(reinterpret_cast<const void*>(kern), I8Pair::SMEM, done);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        launch_config(cfg, attr, 2u * (unsigned)grid, kI8PairThreads, 2, I8Pair::SMEM, s);
        e = cudaLaunchKernelEx(&cfg, kern, tw, tx, p);
    }
    if (e != cudaSuccess) set_last_error("INT8 GEMM launch (CTA pairs)", e);
    return e;
}

template <int NT>
cudaError_t launch_swap_t(const Int8GemmArgs& a, int split, int64_t clusters, const Held& held, cudaStream_t s)
{
    return a.half_out ? launch_swap<NT, true>(a, split, clusters, held, s)
                      : launch_swap<NT, false>(a, split, clusters, held, s);
}

cudaError_t launch_pair_t(const Int8GemmArgs& a, int bt, int64_t tiles, int sm_count, cudaStream_t s)
{
    if (a.offsets)
        return a.half_out ? launch_pair<true, true>(a, bt, tiles, sm_count, s)
                          : launch_pair<false, true>(a, bt, tiles, sm_count, s);
    return a.half_out ? launch_pair<true, false>(a, bt, tiles, sm_count, s)
                      : launch_pair<false, false>(a, bt, tiles, sm_count, s);
}

// Token tiles of `nt` rows that a launch may need: a grouped one knows only
// the number of rows and experts.
int64_t most_token_tiles(const Int8GemmArgs& a, int nt)
{
    if (!a.offsets) return (a.M + nt - 1) / nt;
    return a.M / nt + (a.E < a.M ? a.E : a.M);
}

// Estimated microseconds of a product, to choose a kernel and its tile by.
// Fitted to times on a B200 (N of 64 to 28672, K of 104 to 14336, M = 7..829,
// weights from memory), which they meet within 8 % in the mean; what they
// choose takes 1.3 % longer there than the best choice, 1.19 times at most.
double either(double a, double b) { return std::sqrt(std::sqrt(a * a * a * a + b * b * b * b)); }   // the larger, or a bit more
double memory_us(double mb) { return mb / 6.4; }

// Few tokens: `tiles` tiles of 128 channels x nt tokens, `tokens` of them
// there, K split S ways.  A CTA takes a stage in 0.15 us at best and turns to
// its next tile in 0.9 us or more (2.5 with offsets to search), the CTAs of an
// SM together take 150 KB a microsecond, less where long rows start off a
// 128-byte line (`ragged`: 1, else 0).  The split costs its join, which grows
// with the tokens.  16x4096x4096: S = 1 8.4, 2 5.9, 4 6.4, 8 6.5 us;
// 64x4096x4096: 64 tokens S = 2 6.9, 32 tokens S = 4 7.4 us.
double swap_us(int nt, int split, double tiles, double tokens, int64_t ks, double mb, double ragged, bool grouped,
               const Held& held)
{
    const int ctas = swap_ctas(nt, split, tiles, held);
    const double at_once = held.of(split, ctas), share = (double)((ks + split - 1) / split);
    const double rounds = std::ceil(tiles / at_once - 1e-6);
    const double join = tokens * (1 + 0.26 * (ctas - 1)), sms = std::fmin(tiles, at_once) / held.of(1, 1);
    const double fixed = split == 1   ? 1.81 + 0.017 * join + 0.5 * sms
                         : split == 2 ? 2.30 + 0.019 * join + 1.7 * sms
                         : split == 4 ? 2.40 + 0.025 * join + 3.5 * sms
                                      : 2.46 + 0.035 * join + 6.9 * sms;
    // (rows past A are not loaded, the next expert's are)
    const double intake = rounds * share * ctas * (I8_BM + (grouped ? nt : tokens)) / 8 / 150 *
                          (1 + 0.8 * ragged * std::fmin(1, ks / 32.0));
    const double steps = rounds * share * 0.15 + (rounds - 1) * ((grouped ? 2.5 : 0.9) + 0.032 * tokens);
    return fixed + either(either(intake, steps), memory_us(mb));
}

// The groups of rows of a launch, as far as the host knows them: one, or some
// experts of which a launch knows the mean.  Experts' shares differ by several
// times, so three sizes stand for them.
struct Groups {
    double count;      // groups with rows, at most
    int kinds;
    double rows[3], share[3];
};

Groups groups_of(const Int8GemmArgs& a)
{
    if (!a.offsets) return {1, 1, {(double)a.M}, {1}};
    const double some = (double)(a.E < a.M ? a.E : a.M), mean = a.M / some;
    return {some, 3, {0.4 * mean, mean, 2.4 * mean}, {0.4, 0.35, 0.25}};
}

// Many tokens: tiles of 256 channels x bt tokens on the CTA pairs, the last of
// each group as narrow as its rows allow.  A stage takes 0.45 ns x (330 +
// width): the tensor pipe's time is proportional to the width, the loads' is
// not.  A tile's epilogue takes longer than the next tile's stages where K is
// short.  301x5003x4099: bt = 128 13.5, 160 14.5, 256 16.7 us; 1024x8192x8192:
// 256 52.9, 192 59.8 us; 7680 rows over 128 experts of 2283x896: 160 52.4, 192
// 56.8, 128 57.5 us.
double pair_us(int bt, const Groups& g, int64_t N, int64_t ks, double mb, double ragged, int sm_count)
{
    const double pairs = sm_count / 2, tiles_n = (double)((N + 255) / 256);
    double tiles = 0, columns = 0, widest = 0;
    for (int i = 0; i < g.kinds; ++i) {
        const double whole = std::floor(g.rows[i] / bt), rest = std::ceil((g.rows[i] - whole * bt) / 32) * 32;
        tiles += g.share[i] * (whole + (rest > 0 ? 1 : 0));
        columns += g.share[i] * (whole * (330 + bt) + (rest > 0 ? 330 + rest : 0));
        widest = std::fmax(widest, whole > 0 ? bt : rest);
    }
    tiles *= g.count * tiles_n;
    columns *= g.count * tiles_n;
    double longest = 330 + widest;   // of a pair
    if (tiles > pairs) {
        const double full = std::floor(tiles / pairs), rem = tiles - full * pairs;
        longest = full * columns / tiles + (rem == 0 ? 0 : 2 * rem <= pairs ? 330 + bt / 2 : 330 + widest);
    }
    const double products = 0.00045 * longest * ks * (1 + 0.27 * ragged);
    const double epilogues = (std::ceil(tiles / pairs - 1e-6) - 1) * (1.05 + 0.0092 * (columns / tiles - 330));
    return 2.06 + 0.0104 * widest + 1.6 * std::fmin(1, tiles / pairs) + either(either(products, epilogues), memory_us(mb));
}

Int8Form choose(const Int8GemmArgs& a, int kernel, const Held& held, int sm_count)
{
    const int64_t ks = (a.K + I8_BK - 1) / I8_BK, tiles_n = (a.N + I8_BM - 1) / I8_BM;
    const Groups g = groups_of(a);
    const double ragged = a.ldb % 128 != 0 ? 1 : 0;
    // (experts: some have no rows, and their weights are not read)
    const double mb = 1e-6 * ((a.offsets ? 0.8 : 1) * g.count * (double)a.N * (double)a.K + 2.0 * a.M * a.N);
    double rows = 0;
    for (int i = 0; i < g.kinds; ++i) rows += g.share[i] * g.rows[i];
    Int8Form few = {true, 128, 1}, many = {false, 256, 1};
    double best_swap = 1e30, best_pair = 1e30;
    for (int nt = 16; nt <= 128; nt *= 2) {
        double groups = 0;   // token tiles of a group, in the mean
        for (int i = 0; i < g.kinds; ++i) groups += g.share[i] * std::ceil(g.rows[i] / nt);
        const double tiles = groups * g.count * tiles_n;
        for (int split = 1; split <= 8; split *= 2) {
            if (split > 1 && (split > ks || tiles > held.of(split, swap_resident(nt)))) break;
            const double us = swap_us(nt, split, tiles, rows / groups, ks, mb, ragged, a.offsets != nullptr, held);
            // (a wider tile only for a gain)
            if (us < (nt == few.tile ? 1.0 : 0.94) * best_swap) {
                best_swap = us;
                few.tile = nt;
                few.split = split;
            }
        }
    }
    for (int bt = 256; bt >= 32; bt -= 32) {
        const double us = pair_us(bt, g, a.N, ks, mb, ragged, sm_count);
        if (us <= best_pair) {   // (of equal ones the narrowest: more stages fit)
            best_pair = us;
            many.tile = bt;
        }
    }
    return kernel == FP4_GEMM_DECODE || a.K == 0 || (kernel == FP4_GEMM_AUTO && best_swap <= best_pair) ? few : many;
}

}  // namespace

// Those that `choose` can return.
bool int8_form_applies(const Int8GemmArgs& a, const Int8Form& f)
{
    const int64_t ks = (a.K + I8_BK - 1) / I8_BK;
    if (f.swap)
        return (f.tile == 16 || f.tile == 32 || f.tile == 64 || f.tile == 128) &&
               (f.split == 1 || ((f.split == 2 || f.split == 4 || f.split == 8) && f.split <= ks));
    return f.tile >= 32 && f.tile <= 256 && f.tile % 32 == 0 && f.split == 1 && a.K > 0;
}

cudaError_t launch_gemm_int8(const Int8GemmArgs& a, int kernel, const Int8Form* form, const DeviceInfo& dev,
                             cudaStream_t s)
{
    if (!form && kernel != FP4_GEMM_PREFILL && gemv_int8_applies(a)) return launch_gemv_int8(a, dev, s);
    const Held held = held_clusters(dev.sm_count);
    const Int8Form f = form ? *form : choose(a, kernel, held, dev.sm_count);
    if (f.swap) {
        const int64_t clusters = most_token_tiles(a, f.tile) * ((a.N + I8_BM - 1) / I8_BM);
        if (f.tile == 16) return launch_swap_t<16>(a, f.split, clusters, held, s);
        if (f.tile == 32) return launch_swap_t<32>(a, f.split, clusters, held, s);
        if (f.tile == 64) return launch_swap_t<64>(a, f.split, clusters, held, s);
        return launch_swap_t<128>(a, f.split, clusters, held, s);
    }
    return launch_pair_t(a, f.tile, most_token_tiles(a, f.tile) * ((a.N + 255) / 256), dev.sm_count, s);
}

cudaError_t launch_int8_wait_selftest(cudaStream_t s)
{
    bounded_wait_selftest_kernel<<<1, 32, 0, s>>>();
    return cudaGetLastError();
}

cudaError_t read_and_clear_int8_error_word(unsigned int* word)
{
    cudaError_t e = cudaMemcpyFromSymbol(word, g_fp4_error_word, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    if (*word) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_fp4_error_word, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace fp4
