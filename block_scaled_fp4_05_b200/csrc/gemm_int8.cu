// INT8 matrix products with a scale for each token and each output channel,
//   D[m, n] = round16( (sum_k qA[m, k] qB[n, k]) sA[m] sB[n] + bias[n] ),
// dense, or grouped by expert: the rows [offsets[e], offsets[e + 1]) of A and
// D belong to expert e's weights B[e], and the offsets are read on the device.
// The sums are exact 32-bit integers (tcgen05.mma kind::i8; K <= 131071 keeps
// them in range for any codes); the scales and the bias are applied in FP32
// and the result is rounded once, to BF16 or FP16.
//
// Two kernels:
//   int8_pair_kernel   many tokens: persistent CTA pairs, 256 x 256 (or
//                      256 x 128) tiles.  Bound by the tensor pipe.
//   int8_swap_kernel   few tokens: the weights on the 128-row MMA side, 16 to
//                      128 tokens on the other, K split over a cluster whose
//                      CTAs join their sums through distributed shared
//                      memory.  Bound by HBM (the weights are read once).
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
#include "tc_device.cuh"

namespace fp4 {
namespace {

constexpr int I8_BM = 128;          // rows of the A-side operand per CTA
constexpr int I8_BK = 128;          // K elements (and bytes a row) per stage
constexpr int I8_MMA_K = 32;        // K per tcgen05.mma kind::i8
constexpr int I8_TILE = I8_BM * I8_BK;
constexpr int kMaxExperts = kInt8MaxExperts;
constexpr int64_t kI8GroupBytes = int64_t(32) << 20;

struct I8Params {
    const float* sa;         // [M]
    const float* sb;         // [E x N]
    const float* bias;       // [E x N] or NULL
    uint16_t* D;             // [M x N], leading dimension ldd
    int64_t ldd;
    int32_t M, N;            // rows of A and D, output channels
    int32_t ks_total;        // stages of a tile (0: K = 0, the sums are zero)
    int32_t tiles_n;
    // pair kernel: tile width and its stages, whether a partial last wave may
    // be halved, M tiles per group of the tile order
    int32_t bn, stages, halves;
    int32_t raster_gm;
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

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t cluster_addr)
{
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

// One step of a 4 x 4 transposition of 16-byte pieces (v[4 j .. 4 j + 3] is
// piece j) among the lanes of a quad: pieces and lanes whose numbers differ in
// bit `bit` (1 or 2) change places.
__device__ __forceinline__ void quad_transpose(uint32_t (&v)[16], int lane, int bit)
{
    const bool upper = lane & bit;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j & bit) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t &lo = v[4 * j + i], &hi = v[4 * (j | bit) + i];
            const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, upper ? lo : hi, bit);
            if (upper) lo = got;
            else hi = got;
        }
    }
}

template <bool HALF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    if constexpr (HALF) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    } else {
        return pack_bf16x2(lo, hi);
    }
}

// The scaled result of one sum; the token's scale first, so that the sum
// leaves the integer range before the channel's scale and bias are applied.
__device__ __forceinline__ float scaled(int acc, float sa, float sb, float bias)
{
    return __fmaf_rn(__fmul_rn(__int2float_rn(acc), sa), sb, bias);
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
constexpr int swap_resident(int nt) { return nt == 16 ? 3 : 2; }   // CTAs an SM holds

template <int NT>
struct SwapCfg {
    // Two to three CTAs share an SM, so that one's first loads and last
    // stores overlap another's stream: 72 to 100 KB each.
    static constexpr int STAGES = NT == 16 ? 4 : NT == 32 ? 5 : NT == 64 ? 4 : 3;
    static constexpr int STAGE_BYTES = I8_TILE + NT * I8_BK;
    static constexpr int OFF_T = I8_TILE;
    static constexpr int OFF_BARS = STAGES * STAGE_BYTES;
    static constexpr int OFF_SCALE = OFF_BARS + 256;   // sA of the tokens, sB and bias of the channels
    static constexpr int SMEM = OFF_SCALE + (NT + 2 * I8_BM) * 4 + 1024;
    static constexpr int TMEM_COLS = NT < 32 ? 32 : NT;
    static_assert(NT * I8_BM * 4 <= OFF_BARS, "the sums reuse the stages' memory");
    static_assert((2 * STAGES + 1) * 8 + 40 <= 256, "barrier area");
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
    constexpr int STAGES = C::STAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
    // [0,S) full, [S,2S) empty, [2S] accumulator full
    int* shared_word = reinterpret_cast<int*>(bars + 2 * STAGES + 1);
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
    const uint32_t smem0 = smem_u32(smem);
    const uint32_t bar0 = smem_u32(bars);
    auto FULL = [&](int s) { return bar0 + 8u * s; };
    auto EMPTY = [&](int s) { return bar0 + 8u * (STAGES + s); };
    const uint32_t acc_full = bar0 + 8u * (2 * STAGES);
    // Items: the tiles (expert, channel tile, token tile), token tiles
    // fastest so that clusters that share weights run next to each other,
    // dealt round-robin to the clusters.
    const int cluster = (int)(blockIdx.x / split), clusters = (int)(gridDim.x / split);
    const int dense_mt = (p.M + NT - 1) / NT;
    // Weight tiles requested before the dependency wait (static weights of a
    // dense product): those of the first stages, their token tiles follow.
    int pre = !p.offsets && p.b_static ? min(STAGES, ke - kb) : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
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
            if (lane == 0) {
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
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                // Only now may the next kernel start: its first weight loads
                // beside this one's cost more than they hid (1x28672x8192,
                // call after call: 39.8 us, 48 with the trigger at the start).
                pdl_trigger();
                if (!ok || *abort_flag) spin_ns(200000);   // loads in flight land before the memory is used again
            }
            __syncwarp();
        } else if (warp == 1) {
            if (lane == 0 && kb < ke) {
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
                    if (++stage == STAGES) {
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
// Many tokens: a cluster of two CTAs computes a 256 x bn tile with pair MMAs
// (M = 256, N = bn, a multiple of 32 up to 256 that the host chooses): each
// CTA stages its own 128 rows of A and half of the tile's B rows.  Two
// accumulators in tensor memory, so that a tile's epilogue runs beside the
// next tile's MMAs.
//   warp 0      producer (both CTAs; loads complete on the leader's full[s])
//   warp 1      MMA issue (leader): passes a stage's named barrier, issues
//               four MMAs and the commit that releases the stage in both
//               CTAs; it touches no mbarrier, since a probe between two
//               stages' MMAs leaves the tensor pipe idle
//   warp 2      gatekeeper (leader): waits for the accumulator's release and
//               for each stage, then opens the stage's named barrier
//   warp 3      grouped: the tile list from the offsets
//   warps 4-11  epilogue: two warps a tensor-memory lane quadrant, 32 columns
//               in turn; scales, bias, 16 bits, and from the registers to D,
//               four lanes a row (sixteen warps were 10 % faster where the
//               sums are short, K = 128 to 512, and 0.5 us slower a launch)
// Every wait is bounded; a CTA that gives up records it in the error word.
// ------------------------------------------------------------------------
constexpr int kI8EpiWarps = 8;
constexpr int kI8Parts = kI8EpiWarps / 4;        // epilogue warps a tensor-memory lane quadrant
constexpr int kI8Chunks = 256 / 32 / kI8Parts;   // 32-column chunks of each
constexpr int kI8PairThreads = 128 + 32 * kI8EpiWarps;
constexpr int kI8PairMaxStages = 12;

struct I8Pair {
    static constexpr int OFF_SCALE = 0;                                            // sB and bias of a warp's columns
    static constexpr int OFF_LIST = OFF_SCALE + 4 * 2 * 256 * 4;          // experts' first tiles and bounds
    static constexpr int OFF_BARS = OFF_LIST + 2 * (kMaxExperts + 2) * 4;
    static constexpr int NBARS = 2 * kI8PairMaxStages + 5;
    static constexpr int FIXED = (OFF_BARS + 256 + 1023) / 1024 * 1024;            // what lies before the stages
    static constexpr int SMEM = 232448;
    static constexpr int STAGE_ROOM = SMEM - 1024 - FIXED;
    static_assert(NBARS * 8 + 8 <= 256, "barrier area");
    static_assert(OFF_BARS % 16 == 0, "barrier alignment");
    static_assert(kI8PairMaxStages + 1 <= 16, "one named barrier per stage (ids from 1)");
    __host__ __device__ static constexpr int stage_bytes(int bn) { return I8_TILE + bn / 2 * I8_BK; }
    static constexpr int stages(int bn)
    {
        const int n = STAGE_ROOM / stage_bytes(bn);
        return n < kI8PairMaxStages ? n : kI8PairMaxStages;
    }
};

template <bool HALF, bool GROUPED>
__global__ void __launch_bounds__(kI8PairThreads, 1)
int8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmBh, const I8Params p)
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
    const uint32_t stage_bytes = (uint32_t)I8Pair::stage_bytes(p.bn);
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
            const int tiles = (end - first + 255) / 256 * p.tiles_n;
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
    const int tiles = GROUPED ? list[p.E] : (p.M + 255) / 256 * p.tiles_n;
    // Work items: the tiles, dealt round-robin.  A last, partial wave whose
    // halves fit on the pairs is computed as halves of bn / 2 columns.
    const int rem = tiles % npairs;
    const int split_from = p.halves && 2 * rem <= npairs ? tiles - rem : tiles;
    const int items = 2 * tiles - split_from;
    // Expert, first row and channel of item t, its width, and the end of the
    // expert's rows.  Within an expert groups of raster_gm consecutive M
    // tiles sweep the N tiles together (M fastest), so that a group's A rows
    // stay in L2 while B streams past them once.
    struct Place {
        int e, row, col, width, row_end;
    };
    auto locate = [&](int t) {
        Place w;
        int half = 0;
        w.width = p.bn;
        if (t >= split_from) {
            half = (t - split_from) & 1;
            t = split_from + ((t - split_from) >> 1);
            w.width = p.bn / 2;
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
        const int tiles_m = (end - base + 255) >> 8;
        const int span = p.raster_gm * p.tiles_n;
        const int grp = t / span, in = t - grp * span;
        const int m0 = grp * p.raster_gm;
        const int gm = min(tiles_m - m0, p.raster_gm);
        w.e = lo;
        w.row = base + (m0 + in % gm) * 256;
        w.col = in / gm * p.bn + half * w.width;
        w.row_end = end;
        return w;
    };

    if (warp == 0) {
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmA)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmB)) : "memory");
            // B rows of a stage: half of the item's columns in each CTA
            auto load_b = [&](const Place& w, int s, int ks) {
                if (leader) mbar_arrive_expect_tx(FULL(s), 2u * (uint32_t)I8Pair::stage_bytes(w.width));
                const int y = w.col + (int)rank * (w.width / 2);
                tma_load_3d_pair(w.width == p.bn ? &tmB : &tmBh, map_to_rank(FULL(s), 0),
                                 smem0 + s * stage_bytes + I8_TILE, ks * I8_BK, y, w.e);
            };
            int stage = 0, pre = 0;
            uint32_t phase = 0;
            bool ok = true;
            if (!GROUPED && p.b_static && pair < items) {
                // static weights: those of the first stages are requested
                // before the dependency wait
                const Place w = locate(pair);
                for (; pre < stages && pre < p.ks_total; ++pre) load_b(w, pre, pre);
            }
            pdl_wait();
            for (int t = pair; ok && t < items; t += npairs) {
                const Place w = locate(t);
                const int ya = w.row + (int)rank * I8_BM;
                for (int ks = 0; ks < p.ks_total; ++ks) {
                    if (pre > 0) {
                        --pre;   // this stage's B tile is on its way
                    } else {
                        if (!wait_fast(EMPTY(stage), phase ^ 1u, abort_flag, ERR_EMPTY)) {
                            ok = false;
                            break;
                        }
                        load_b(w, stage, ks);
                    }
                    tma_load_3d_pair(&tmA, map_to_rank(FULL(stage), 0), smem0 + stage * stage_bytes, ks * I8_BK, ya, 0);
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
                const uint32_t acc = tmem_base + (uint32_t)(buf * 256);
                const uint32_t idesc = idesc_i8(256, t >= split_from ? p.bn / 2 : p.bn);
                for (int ks = 0; ks < p.ks_total; ++ks) {
                    named_bar_sync(1 + stage, 64);
                    if (lane == 0) {
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
                if (lane == 0) tc_commit_pair_both(ACC_FULL(buf));
                __syncwarp();
                buf ^= 1;
            }
            if (lane == 0) {
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
        const int part = (warp - 4) >> 2;        // the warp's 32-column chunks: part, part + kI8Parts, ...
        float* sbs = reinterpret_cast<float*>(smem + I8Pair::OFF_SCALE) + (warp - 4) * (2 * 32 * kI8Chunks);
        float* bis = sbs + 32 * kI8Chunks;
        pdl_wait();
        // The scales of an item (this lane's row, a column of each chunk) are
        // read while the item before it is worked on.
        Place next = {};
        float sa_next = 0.0f, sb_next[kI8Chunks] = {}, bias_next[kI8Chunks] = {};
        auto fetch = [&](int t) {
            if (t >= items) return;
            next = locate(t);
            const int y = next.row + (int)rank * I8_BM + q * 32 + lane;
            if (y < next.row_end) sa_next = __ldcg(p.sa + y);
            const int64_t chan_base = (int64_t)next.e * p.N;
#pragma unroll
            for (int c = 0; c < kI8Chunks; ++c) {
                const int n = next.col + (part + kI8Parts * c) * 32 + lane;
                const bool in = (part + kI8Parts * c) * 32 < next.width && n < p.N;
                sb_next[c] = in ? __ldcg(p.sb + chan_base + n) : 0.0f;
                bias_next[c] = in && p.bias ? __ldcg(p.bias + chan_base + n) : 0.0f;
            }
        };
        fetch(pair);
        uint32_t acc_phase = 0;
        int buf = 0;
        for (int t = pair; t < items; t += npairs) {
            const Place w = next;
            const float sa = sa_next;
#pragma unroll
            for (int c = 0; c < kI8Chunks; ++c) {
                sbs[c * 32 + lane] = sb_next[c];
                bis[c * 32 + lane] = bias_next[c];
            }
            __syncwarp();
            fetch(t + npairs);
            const int y0 = w.row + (int)rank * I8_BM + q * 32;
            const int chunks = (w.width / 32 - part + kI8Parts - 1) / kI8Parts;   // 0 to kI8Chunks
            if (!warp_wait(ACC_FULL(buf), acc_phase, abort_flag, ERR_ACC_FULL)) break;
            tc_fence_after();
            const uint32_t trow = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * 256 + part * 32);
            uint32_t r2[2][32];
            if (chunks > 0) tmem_ld32(trow, r2[0]);
#pragma unroll
            for (int c = 0; c < kI8Chunks; ++c) {
                uint32_t (&r)[32] = r2[c & 1];
                if (c < chunks) tmem_wait_ld(r);
                if (c + 1 < chunks) {   // the next chunk's load overlaps this one's arithmetic
                    tmem_ld32(trow + (uint32_t)((c + 1) * kI8Parts * 32), r2[(c + 1) & 1]);
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
                const int x0 = w.col + (part + kI8Parts * c) * 32;
                if (c < chunks && y0 < w.row_end && x0 < p.N) {
                    uint32_t v[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 s4 = *reinterpret_cast<const float4*>(sbs + c * 32 + 4 * i);
                        const float4 b4 = *reinterpret_cast<const float4*>(bis + c * 32 + 4 * i);
                        v[2 * i] = pack16<HALF>(scaled((int)r[4 * i], sa, s4.x, b4.x),
                                                scaled((int)r[4 * i + 1], sa, s4.y, b4.y));
                        v[2 * i + 1] = pack16<HALF>(scaled((int)r[4 * i + 2], sa, s4.z, b4.z),
                                                    scaled((int)r[4 * i + 3], sa, s4.w, b4.w));
                    }
                    // Four lanes exchange their rows' 16-byte pieces, so that
                    // lane i has piece i of all four rows and they store 64
                    // bytes of one row at a time.
                    quad_transpose(v, lane, 1);
                    quad_transpose(v, lane, 2);
                    const int x = x0 + 8 * (lane & 3);
                    uint16_t* d = p.D + (int64_t)(y0 + (lane & 28)) * p.ldd + x;
#pragma unroll
                    for (int k = 0; k < 4; ++k, d += p.ldd) {
                        if (y0 + (lane & 28) + k >= w.row_end) break;   // the next expert's row, or none
                        if (x + 8 <= p.N) {
                            *reinterpret_cast<uint4*>(d) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (x + i < p.N) d[i] = (uint16_t)(v[4 * k + (i >> 1)] >> (16 * (i & 1)));
                        }
                    }
                }
                __syncwarp();   // (after the last chunk: the scales' memory is written again)
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
    p.bn = bn;
    p.stages = 0;
    p.halves = 0;
    p.raster_gm = 1;
    p.E = (int32_t)a.E;
    p.offsets = a.offsets;
    p.b_static = a.b_static ? 1 : 0;
    return p;
}

template <int NT, bool HALF>
cudaError_t launch_swap(const Int8GemmArgs& a, int split, int64_t clusters, int sm_count, cudaStream_t s)
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
    cudaError_t e = raise_smem(reinterpret_cast<const void*>(kern), C::SMEM, done);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        // as many clusters as the SMs hold take all tiles in turn
        const int64_t hold = (int64_t)swap_resident(NT) * sm_count / split;
        launch_config(cfg, attr, (unsigned)((clusters < hold ? clusters : hold) * split), kSwapThreads, (unsigned)split, C::SMEM, s);
        e = cudaLaunchKernelEx(&cfg, kern, tw, tx, params_of(a, I8_BM));
    }
    if (e != cudaSuccess) set_last_error("INT8 GEMM launch (few tokens)", e);
    return e;
}

template <bool HALF, bool GROUPED>
cudaError_t launch_pair(const Int8GemmArgs& a, int bn, int64_t tiles, int sm_count, cudaStream_t s)
{
    I8Params p = params_of(a, bn);
    p.stages = I8Pair::stages(bn);
    const int64_t pairs = sm_count / 2;
    const int64_t grid = tiles < pairs ? tiles : pairs;
    // halves are multiples of 32 columns
    p.halves = bn % 64 == 0 && (GROUPED || 2 * (tiles % grid) <= grid);
    CUtensorMap ta, tb, tbh = {};
    if (!make_map_i8(&ta, a.A, 1, a.M, a.K, a.lda, a.lda, I8_BM) ||
        !make_map_i8(&tb, a.B, a.E, a.N, a.K, a.ldb, a.stride_b, bn / 2) ||
        (p.halves && !make_map_i8(&tbh, a.B, a.E, a.N, a.K, a.ldb, a.stride_b, bn / 4))) {
        set_last_error("cuTensorMapEncodeTiled", cudaErrorInvalidValue);
        return cudaErrorInvalidValue;
    }
    // M tiles per group: as many as hold kI8GroupBytes of A, all of them when
    // A fits in half of the L2 cache
    const int64_t tile_bytes = 256 * a.K, tiles_m = (a.M + 255) / 256;
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
        e = cudaLaunchKernelEx(&cfg, kern, ta, tb, tbh, p);
    }
    if (e != cudaSuccess) set_last_error("INT8 GEMM launch (CTA pairs)", e);
    return e;
}

template <int NT>
cudaError_t launch_swap_t(const Int8GemmArgs& a, int split, int64_t clusters, int sm_count, cudaStream_t s)
{
    return a.half_out ? launch_swap<NT, true>(a, split, clusters, sm_count, s)
                      : launch_swap<NT, false>(a, split, clusters, sm_count, s);
}

cudaError_t launch_pair_t(const Int8GemmArgs& a, int bn, int64_t tiles, int sm_count, cudaStream_t s)
{
    if (a.offsets)
        return a.half_out ? launch_pair<true, true>(a, bn, tiles, sm_count, s)
                          : launch_pair<false, true>(a, bn, tiles, sm_count, s);
    return a.half_out ? launch_pair<true, false>(a, bn, tiles, sm_count, s)
                      : launch_pair<false, false>(a, bn, tiles, sm_count, s);
}

// Token tiles of `nt` rows that a launch may need: a grouped one knows only
// the number of rows and experts.
int64_t most_token_tiles(const Int8GemmArgs& a, int nt)
{
    if (!a.offsets) return (a.M + nt - 1) / nt;
    return a.M / nt + (a.E < a.M ? a.E : a.M);
}

// Estimated microseconds of a product, to choose a kernel and its tile by.
// Both are bound by what an SM takes in: 107 KB a microsecond at most, less
// with less of it in flight (a ring of stages turns over in 1.3 us or more).
// Fitted to times on a B200 over M = 1..8192, N = 320..57344, K = 300..8192,
// which they meet within about 15 % where HBM does not bind.
//
// Few tokens: `tiles` tiles of 128 channels x nt tokens, K split S ways.  The
// split costs its join, which grows with the tokens.  16x4096x4096: S = 1
// 12.2, 2 8.6, 4 6.5, 8 6.8 us; 64x4096x4096: 64 tokens S = 1 13.3, 4 8.3,
// 32 tokens S = 4 7.8 us; 16x28672x8192: S = 1 40.6, 2 45 us.
double swap_us(int nt, int split, double tiles, int64_t ks, int sm_count)
{
    const double resident = swap_resident(nt);
    const double ring_kb = nt == 16 ? 72 : nt == 32 ? 100 : 96;
    const double kb = (double)((ks + split - 1) / split) * (I8_BM + nt) / 8;   // a CTA's operands
    const double fixed = split == 1   ? 1.7 + 0.010 * nt
                         : split == 2 ? 2.7 + 0.023 * nt
                         : split == 4 ? 3.1 + 0.030 * nt
                                      : 4.1 + 0.044 * nt;
    const double n = tiles * split / sm_count;   // CTAs an SM
    if (n <= resident) return fixed + kb / std::fmin(ring_kb / 1.3, 107.0 / std::ceil(n));
    return 1.15 * n / resident * (fixed + kb / std::fmin(ring_kb / 1.3, 107.0 / resident));
}

// Many tokens: tiles of 256 tokens x bn channels on the CTA pairs.  A stage
// takes 0.53 ns x (400 + bn): the tensor pipe's time is proportional to bn,
// the loads' is not.  301x5003x4099 (2 M tiles): bn = 256 16.5, 160 14.2,
// 128 (two waves) 20.3 us; 1024x8192x8192: 256 48.9, 224 46.3, 192 63 us.
double pair_us(int bn, double tiles_m, int64_t N, int64_t ks, int sm_count)
{
    const double pairs = sm_count / 2;
    const double tiles = std::ceil(tiles_m * ((N + bn - 1) / bn));
    const double full = std::floor(tiles / pairs), rem = tiles - full * pairs;
    double columns = full * (400 + bn);
    if (rem > 0) columns += 400 + (full > 0 && bn % 64 == 0 && 2 * rem <= pairs ? bn / 2 : bn);
    return 3.4 + 0.0085 * bn + 0.00053 * columns * ks;
}

struct Choice {
    bool swap;
    int nt, split, bn;
};

Choice choose(const Int8GemmArgs& a, int kernel, int sm_count)
{
    const int64_t ks = (a.K + I8_BK - 1) / I8_BK, tiles_n = (a.N + I8_BM - 1) / I8_BM;
    const bool grouped = a.offsets != nullptr;
    const double mean = grouped ? (double)a.M / a.E : (double)a.M;   // rows an expert
    const double some = grouped ? (double)(a.E < a.M ? a.E : a.M) : 0;   // experts with rows, at most
    Choice c = {true, 16, 1, 256};
    double best_swap = 1e30, best_pair = 1e30;
    for (int nt = 16; nt <= 128; nt *= 2) {
        if (nt < 128 && 8 * nt <= mean) continue;
        // A grouped launch knows only the mean, and experts' shares differ by
        // several times: an expert of more than nt rows reads its weights
        // again for each tile, so the tile is wider than the mean.  64 experts
        // of 2056x2048, 1031 rows unevenly: 16 tokens 46.8, 64 43.1 us; 8 of
        // 4096x4096, 256 rows: 16 tokens 32.5, 64 25.5 us; but 8 of
        // 14336x4096, 16 rows: 16 tokens 62, 64 87 us.
        if (grouped && nt < 64 && nt < 2 * mean && !(nt == 32 && mean <= 20)) continue;
        if (grouped && nt > 16 && nt > 8 * mean) continue;
        const double tiles = (grouped ? std::fmax(a.M / nt + 0.5 * some, some) : (double)((a.M + nt - 1) / nt)) * tiles_n;
        for (int split = 1; split <= 8; split *= 2) {
            if (split > 1 && (split > ks || tiles * split > swap_resident(nt) * sm_count)) break;
            const double us = swap_us(nt, split, tiles, ks, sm_count);
            if (us < best_swap) {
                best_swap = us;
                c.nt = nt;
                c.split = split;
            }
        }
    }
    // a grouped launch has half an empty tile an expert, on the average
    const double tiles_m = grouped ? std::ceil(a.M / 256.0 + 0.5 * some) : std::ceil(a.M / 256.0);
    for (int bn = 256; bn >= 32; bn -= 32) {
        const double us = pair_us(bn, tiles_m, a.N, ks, sm_count);
        if (us < best_pair) {
            best_pair = us;
            c.bn = bn;
        }
    }
    // Where the weights' bytes bind, the few-token kernel reads them at 5.8
    // TB/s or more and the pair kernel, whose tiles are partly empty then, at
    // 5.0 (64 experts of 2056x2048, 1031 rows: 48 against 56 us).
    const double weight_mb = 1e-6 * (grouped ? some : 1) * (double)a.N * (double)a.K;
    best_swap = std::fmax(best_swap, weight_mb / 5.8 + 2);
    best_pair = std::fmax(best_pair, weight_mb / 5.0 + 4);
    c.swap = kernel == FP4_GEMM_DECODE || a.K == 0 || (kernel == FP4_GEMM_AUTO && best_swap <= best_pair);
    return c;
}

}  // namespace

cudaError_t launch_gemm_int8(const Int8GemmArgs& a, int kernel, const DeviceInfo& dev, cudaStream_t s)
{
    const Choice c = choose(a, kernel, dev.sm_count);
    if (c.swap) {
        const int64_t clusters = most_token_tiles(a, c.nt) * ((a.N + I8_BM - 1) / I8_BM);
        if (c.nt == 16) return launch_swap_t<16>(a, c.split, clusters, dev.sm_count, s);
        if (c.nt == 32) return launch_swap_t<32>(a, c.split, clusters, dev.sm_count, s);
        if (c.nt == 64) return launch_swap_t<64>(a, c.split, clusters, dev.sm_count, s);
        return launch_swap_t<128>(a, c.split, clusters, dev.sm_count, s);
    }
    return launch_pair_t(a, c.bn, most_token_tiles(a, 256) * ((a.N + c.bn - 1) / c.bn), dev.sm_count, s);
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
