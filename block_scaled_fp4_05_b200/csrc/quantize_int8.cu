// Per-row symmetric INT8 quantization of BF16 or FP16 matrices, with an
// optional gather of the rows (the dispatch of tokens to experts).
//
//   amax = max_k |x_k|,  s = amax / 127 (1 for a zero row),
//   q_k  = RNE(127 x_k / amax)
//
// The codes are those of the exact quotient.  127 x_k and amax are short
// integers times powers of two, so 127 x_k / amax is either exactly halfway
// between two integers or at least 2^-19 (relative) away from it; an FP32
// quotient within an ulp rounds to the same integer unless it is a tie, and a
// tie has to come out exact.  With the row scaled by a power of two (exact,
// so that neither 127 x nor 1 / amax leaves the FP32 range) and r = RN(1/amax):
//   t = RN(a r), a = 127 x;  e = a - t amax (exact as an FMA: it cancels to a
//   few bits);  q = RN(t + e r)
// t + e r differs from the quotient by less than 2^-44 of it, so a quotient
// that FP32 holds (every tie does) comes out exactly.  Adding 1.5 * 2^23 rounds
// q to an integer, halves to even, and leaves its two's complement in the low
// byte.  Two elements go through these steps in one instruction each.
//
// Bound by HBM: 2 bytes read and 1 written an element.  A row stays in the
// registers of its threads between the maximum and the codes, so it is read
// once; rows above 32768 elements are read twice (the second time mostly from
// L2).  Short-lived blocks, one row each (a warp a row up to 2048 elements),
// keep more loads in flight than a resident ring would.

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "fp4_internal.h"
#include "quant_device.cuh"

namespace fp4 {
namespace {

// One row's multipliers: a = 127 x is x * c, the scaled maximum is m.
struct RowScale {
    float c;      // 127 * 2^p
    float m;      // amax * 2^p
    float r;      // RN(1 / m)
    float scale;  // what the codes are to be multiplied by
};

template <bool HALF>
__device__ __forceinline__ float widen(uint32_t bits16)
{
    return HALF ? __half2float(__ushort_as_half((unsigned short)bits16)) : __uint_as_float(bits16 << 16);
}

// amax_bits: the largest magnitude of the row as its 16-bit pattern.
template <bool HALF>
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits)
{
    RowScale s;
    const uint32_t inf = HALF ? 0x7C00u : 0x7F80u;
    if (amax_bits == 0u) {
        s.c = 0.0f;
        s.m = 1.0f;
        s.r = 1.0f;
        s.scale = 1.0f;
        return s;
    }
    if (amax_bits >= inf) {   // the products of the row come out NaN
        s.c = 0.0f;
        s.m = 1.0f;
        s.r = 1.0f;
        s.scale = __uint_as_float(0x7FC00000u);
        return s;
    }
    const float amax = widen<HALF>(amax_bits);
    // 2^p brings a normal maximum into [4, 8); p is capped at 120, so that
    // 127 * 2^p is finite (subnormal BF16 maxima then end below 4)
    const int eb = (int)(__float_as_uint(amax) >> 23);
    const float p = __uint_as_float((uint32_t)min(256 - eb, 247) << 23);
    s.c = 127.0f * p;
    s.m = amax * p;
    s.r = __frcp_rn(s.m);
    s.scale = __fdiv_rn(amax, 127.0f);
    return s;
}

// Two FP32 operations in one instruction (each rounded as its scalar form).
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The codes of two elements in the low bytes of the halves (other bytes: garbage).
__device__ __forceinline__ uint64_t code2(uint64_t x, uint64_t c, uint64_t neg_m, uint64_t r)
{
    const uint64_t a = mul2(x, c);
    const uint64_t t = mul2(a, r);
    const uint64_t q = fma2(fma2(t, neg_m, a), r, t);
    return add2(q, pair(12582912.0f, 12582912.0f));
}

template <bool HALF>
__device__ __forceinline__ uint2 codes8(uint4 v, const RowScale& s, bool finite)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const uint64_t c = pair(s.c, s.c), neg_m = pair(-s.m, -s.m), r = pair(s.r, s.r);
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        if (HALF) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            lo = f.x;
            hi = f.y;
        } else {
            lo = __uint_as_float(w[i] << 16);
            hi = __uint_as_float(w[i] & 0xFFFF0000u);
        }
        const uint64_t q = code2(pair(lo, hi), c, neg_m, r);
        b[i] = __byte_perm((uint32_t)q, (uint32_t)(q >> 32), 0x0040);
    }
    if (!finite) return make_uint2(0u, 0u);
    return make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
}

// Elements [k, k + 8) of a row of `cols`; nothing behind the row is read.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t k, int64_t cols)
{
    if (k + 8 <= cols) return qdev::ld_stream(reinterpret_cast<const uint4*>(row + k));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < cols) w[i >> 1] |= (uint32_t)__ldg(row + k + i) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(int8_t* row, int64_t k, int64_t cols, uint2 q)
{
    if (k + 8 <= cols) {
        *reinterpret_cast<uint2*>(row + k) = q;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < cols) row[k + i] = (int8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
}

struct QuantArgs {
    const uint16_t* x;
    int64_t rows_in, cols, ld;
    const int32_t* index;   // source row of each output row, or NULL
    int64_t rows;
    int8_t* codes;
    int64_t ldc;
    float* scales;
};

// TPR threads a row (32: a warp, several rows a block; else the block),
// CH 8-element chunks a thread; CH = 0: rows of any length, read twice.
template <bool HALF, int TPR, int CH, int THREADS>
__global__ void __launch_bounds__(THREADS) quantize_int8_kernel(const QuantArgs p)
{
    // The next kernel may start its set-up; this one starts before the one
    // before it has ended (0.5 us a launch) and touches nothing until then.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int ROWS = THREADS / TPR;
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    const bool have = ROWS == 1 || row < p.rows;   // the last block's rows may end before it
    int64_t src = row;
    bool inside = have;
    if (p.index && have) {
        src = __ldg(p.index + row);
        inside = src >= 0 && src < p.rows_in;   // an index outside gives a row of zeros
    }
    if (!inside) src = 0;
    const uint16_t* x = p.x + src * p.ld;
    const int64_t cols = inside ? p.cols : 0;
    uint4 v[CH > 0 ? CH : 1];
    uint32_t amax = 0;
    if (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int64_t k = ((int64_t)c * TPR + t) * 8;
            v[c] = k < cols ? load8(x, k, cols) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) amax = max(amax, qdev::absmax8(v[c]));
    } else {
        for (int64_t k = t * 8; k < cols; k += TPR * 8) amax = max(amax, qdev::absmax8(load8(x, k, cols)));
    }
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if (TPR > 32) {
        __shared__ uint32_t part[ROWS][TPR / 32];
        if ((t & 31) == 0) part[threadIdx.x / TPR][t >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) amax = max(amax, part[threadIdx.x / TPR][i]);
    }
    if (!have) return;
    const RowScale s = row_scale<HALF>(amax);
    const bool finite = amax < (HALF ? 0x7C00u : 0x7F80u);
    if (t == 0) p.scales[row] = s.scale;
    int8_t* out = p.codes + row * p.ldc;
    if (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int64_t k = ((int64_t)c * TPR + t) * 8;
            if (k < p.cols) store8(out, k, p.cols, codes8<HALF>(v[c], s, finite));
        }
    } else {
        for (int64_t k = t * 8; k < p.cols; k += TPR * 8)
            store8(out, k, p.cols,
                   codes8<HALF>(k < cols ? load8(x, k, cols) : make_uint4(0u, 0u, 0u, 0u), s, finite));
    }
}

template <bool HALF, int TPR, int CH, int THREADS>
cudaError_t launch(const QuantArgs& p, cudaStream_t s)
{
    constexpr int ROWS = THREADS / TPR;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.rows + ROWS - 1) / ROWS), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, quantize_int8_kernel<HALF, TPR, CH, THREADS>, p);
}

template <bool HALF>
cudaError_t dispatch(const QuantArgs& p, cudaStream_t s)
{
    if (p.cols <= 256) return launch<HALF, 32, 1, 128>(p, s);
    if (p.cols <= 512) return launch<HALF, 32, 2, 128>(p, s);
    if (p.cols <= 1024) return launch<HALF, 32, 4, 128>(p, s);
    if (p.cols <= 2048) return launch<HALF, 32, 8, 128>(p, s);
    const bool many = p.rows > 1024;
    if (p.cols <= 4096) return many ? launch<HALF, 128, 4, 128>(p, s) : launch<HALF, 256, 2, 256>(p, s);
    if (p.cols <= 8192) return many ? launch<HALF, 128, 8, 128>(p, s) : launch<HALF, 256, 4, 256>(p, s);
    if (p.cols <= 16384) return launch<HALF, 256, 8, 256>(p, s);
    if (p.cols <= 32768) return launch<HALF, 512, 8, 512>(p, s);
    return launch<HALF, 512, 0, 512>(p, s);
}

}  // namespace

cudaError_t launch_quantize_int8(int dtype, const uint16_t* x, int64_t rows_in, int64_t cols, int64_t ld,
                                 const int32_t* row_index, int64_t rows, int8_t* codes, int64_t ldc,
                                 float* scales, cudaStream_t s)
{
    const QuantArgs p = {x, rows_in, cols, ld, row_index, rows, codes, ldc, scales};
    const cudaError_t e = dtype == FP4_FP16 ? dispatch<true>(p, s) : dispatch<false>(p, s);
    if (e != cudaSuccess) set_last_error("INT8 quantizer launch", e);
    return e;
}

}  // namespace fp4
