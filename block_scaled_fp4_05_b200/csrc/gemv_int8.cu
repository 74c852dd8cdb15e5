// INT8 products of one to eight tokens with weights of a few megabytes:
//   D[m, n] = round16( (sum_k qA[m, k] qB[n, k]) sA[m] sB[n] + bias[n] ),
// the operation and the bits of gemm_int8.cu, as dot products on the ordinary
// cores.  Bound by HBM: every weight byte is read once and meets M codes.
//
// A warp has C channels; its lanes take 16 bytes each of 512 consecutive codes
// of a channel at a time, eight such loads in flight, against the tokens'
// codes in shared memory (__dp4a: four products an instruction), and the
// lanes' sums meet in one warp reduction a channel and token.  Where there are
// few channels, `ksplit` warps of a block share them, every ksplit-th piece
// of K each.  Blocks stay and take channels in turn.  Static weights of a
// warp's first pieces are requested before the dependency wait.
// Against the tensor-core form there is no tensor map, tensor memory or
// cluster to set up and no join between SMs.  (Loading a batch of pieces ahead
// of the one worked on cost more registers than it hid: 4096x4096 5.4 us
// instead of 5.1, 28672x8192 47 instead of 43.)

#include <cuda_runtime.h>
#include <cstdint>

#include "fp4_internal.h"
#include "int8_device.cuh"

namespace fp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPiece = 512;   // bytes of a channel that a warp takes at a time

struct GemvArgs {
    const int8_t* A;
    int64_t lda;
    const int8_t* B;
    int64_t ldb;
    const float *sa, *sb, *bias;
    uint16_t* D;
    int64_t ldd;
    int M, N, K, ksplit, b_static;
};

// Not through the read-only path: weights that are not static may be written
// by the kernel before, which can still be running when this one starts.
__device__ __forceinline__ int4 ld_stream(const int8_t* p)
{
    int4 v;
    asm volatile("ld.global.L1::no_allocate.v4.s32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// 16 codes from k on of a row of K, 0 behind it; nothing there is read.
__device__ __noinline__ int4 load_tail(const int8_t* row, int k, int K)
{
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (k + i < K) w[i >> 2] |= (uint32_t)(uint8_t)__ldcg(row + k + i) << (8 * (i & 3));
    return make_int4((int)w[0], (int)w[1], (int)w[2], (int)w[3]);
}

// MT: tokens computed (M of them stored); C * U pieces in flight a warp.
template <int MT, int C, int U, bool HALF>
__global__ void __launch_bounds__(kThreads, 3) int8_gemv_kernel(const GemvArgs p)
{
    extern __shared__ __align__(16) int8_t xs[];   // [MT][pieces * 512], zero behind K
    __shared__ int part[2][kWarps][C * MT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pieces = (p.K + kPiece - 1) / kPiece;
    const int per_block = kWarps / p.ksplit;       // channel groups of a block
    const int slot = warp / p.ksplit, share = warp % p.ksplit;
    const int groups = (p.N + C - 1) / C;
    const int passes = (groups + per_block - 1) / per_block;

    // U pieces from c on of the C channels from n0 on (a channel past the last
    // reads the last one's)
    auto load = [&](int n0, int c, int4 (&v)[U][C]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (c + u * p.ksplit) * kPiece + lane * 16;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                // What a row's last 16 bytes hold behind K meets zeros; they
                // are there for every row but the last.
                const int n = min(n0 + j, p.N - 1);
                const int8_t* row = p.B + (int64_t)n * p.ldb;
                if (k >= p.K) v[u][j] = make_int4(0, 0, 0, 0);
                else if (k + 16 <= p.K || n + 1 < p.N) v[u][j] = ld_stream(row + k);
                else v[u][j] = load_tail(row, k, p.K);
            }
        }
    };

    int4 v[U][C];
    int pass = blockIdx.x;
    int n0 = (pass * per_block + slot) * C;
    bool loaded = p.b_static && n0 < p.N;
    if (loaded) load(n0, share, v);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the tokens' codes, 16 bytes a thread, then what is left of each row by bytes
    const int row16 = pieces * (kPiece / 16), whole = p.K / 16;
    for (int i = threadIdx.x; i < MT * row16; i += kThreads) {
        const int m = i / row16, c = i % row16;
        reinterpret_cast<int4*>(xs)[i] =
            m < p.M && c < whole ? __ldcg(reinterpret_cast<const int4*>(p.A + m * p.lda) + c) : make_int4(0, 0, 0, 0);
    }
    if (p.K % 16) {   // (16 threads a row)
        __syncthreads();
        const int m = threadIdx.x / 16, k = whole * 16 + threadIdx.x % 16;
        if (m < p.M && k < p.K) xs[m * pieces * kPiece + k] = __ldcg(p.A + m * p.lda + k);
    }
    __syncthreads();
    for (int turn = 0; pass < passes; pass += gridDim.x, turn ^= 1) {
        n0 = (pass * per_block + slot) * C;
        int acc[C][MT] = {};
        if (n0 < p.N) {
            for (int c = share; c < pieces; c += U * p.ksplit) {
                if (!loaded) load(n0, c, v);
                loaded = false;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int piece = c + u * p.ksplit;
                    if (piece >= pieces) break;
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const int4 x = *reinterpret_cast<const int4*>(xs + (m * pieces + piece) * kPiece + lane * 16);
#pragma unroll
                        for (int j = 0; j < C; ++j) {
                            acc[j][m] = __dp4a(v[u][j].x, x.x, acc[j][m]);
                            acc[j][m] = __dp4a(v[u][j].y, x.y, acc[j][m]);
                            acc[j][m] = __dp4a(v[u][j].z, x.z, acc[j][m]);
                            acc[j][m] = __dp4a(v[u][j].w, x.w, acc[j][m]);
                        }
                    }
                }
            }
        }
        if (pass + gridDim.x >= passes) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int sum = __reduce_add_sync(0xFFFFFFFFu, acc[j][m]);
                if (lane == 0) part[turn][warp][m * C + j] = sum;
            }
        if (p.ksplit > 1) __syncthreads();   // (the other turn's sums have been read by then)
        else __syncwarp();
        const int m = lane / C, n = n0 + lane % C;
        static_assert(C * MT <= 32, "a lane a result");
        if (share == 0 && m < MT && m < p.M && n < p.N) {
            int sum = 0;
            for (int s = 0; s < p.ksplit; ++s) sum += part[turn][warp + s][lane];
            const float r = i8::scaled(sum, __ldcg(p.sa + m), __ldcg(p.sb + n), p.bias ? __ldcg(p.bias + n) : 0.0f);
            p.D[(int64_t)m * p.ldd + n] = (uint16_t)i8::pack16<HALF>(r, r);
        }
    }
}

// Tokens computed for M, channels of a warp and pieces in flight.
constexpr int kMaxTokens = 8;
int tokens_of(int64_t M) { return M <= 1 ? 1 : M <= 2 ? 2 : M <= 4 ? 4 : 8; }
constexpr int channels_of(int mt) { return mt <= 2 ? 4 : 2; }
constexpr int batch_of(int mt) { return mt == 4 ? 4 : 2; }

template <int MT>
cudaError_t launch(const GemvArgs& p, bool half, int smem, unsigned grid, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    constexpr int C = channels_of(MT), U = batch_of(MT);
    return half ? cudaLaunchKernelEx(&cfg, int8_gemv_kernel<MT, C, U, true>, p)
                : cudaLaunchKernelEx(&cfg, int8_gemv_kernel<MT, C, U, false>, p);
}

}  // namespace

bool gemv_int8_applies(const Int8GemmArgs& a)
{
    if (a.offsets || a.M > kMaxTokens || a.K == 0) return false;
    if (tokens_of(a.M) * ((a.K + kPiece - 1) / kPiece) * kPiece > 40960) return false;
    // The tensor-core form streams large weights faster; small ones are over
    // before it is set up.  One token: 512x512 2.0 against 3.3 us, 2048x4096
    // 3.9 / 5.6, 4096x4096 5.4 / 6.7, 8192x4096 8.6 / 8.4, 28672x8192 43.0 /
    // 38.6.  Four: 4096x4096 6.1 / 6.8, 8192x4096 9.7 / 8.5.  Eight: 2000x512
    // 2.4 / 3.4, 2048x2048 4.1 / 4.0, 4000x700 4.7 / 4.0.
    return a.N * a.K <= (a.M <= 4 ? 20000000 : 2000000);
}

cudaError_t launch_gemv_int8(const Int8GemmArgs& a, const DeviceInfo& dev, cudaStream_t s)
{
    GemvArgs p = {a.A, a.lda, a.B, a.ldb, a.sA, a.sB, a.bias, a.D, a.ldd, (int)a.M, (int)a.N, (int)a.K, 1, a.b_static ? 1 : 0};
    const int mt = tokens_of(a.M), channels = channels_of(mt);
    const int pieces = (p.K + kPiece - 1) / kPiece;
    const int64_t groups = (a.N + channels - 1) / channels;
    // warps that share channels: until the SMs have 16 warps each
    while (p.ksplit < kWarps && groups * p.ksplit < 16 * (int64_t)dev.sm_count && 2 * p.ksplit <= pieces) p.ksplit *= 2;
    const int64_t passes = (groups + kWarps / p.ksplit - 1) / (kWarps / p.ksplit);
    const unsigned grid = (unsigned)(passes < 3 * (int64_t)dev.sm_count ? passes : 3 * (int64_t)dev.sm_count);
    const int smem = mt * pieces * kPiece;
    const cudaError_t e = mt == 1   ? launch<1>(p, a.half_out, smem, grid, s)
                          : mt == 2 ? launch<2>(p, a.half_out, smem, grid, s)
                          : mt == 4 ? launch<4>(p, a.half_out, smem, grid, s)
                                    : launch<8>(p, a.half_out, smem, grid, s);
    if (e != cudaSuccess) set_last_error("INT8 GEMM launch (dot products)", e);
    return e;
}

}  // namespace fp4
