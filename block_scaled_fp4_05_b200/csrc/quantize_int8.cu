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
// tie has to come out exactly.  So 127 / amax is held as the sum of two floats
// h + l, within 2^-44 of it (h the product with the approximate reciprocal, l
// from the residual 127 - h amax, which an FMA gives exactly), and
//   t = RN(x h + RN(x l))
// is a quotient that FP32 holds (every tie is one) exactly.  Adding 1.5 * 2^23
// rounds t to an integer, halves to even, and leaves its two's complement in
// the low byte.  Three instructions for two elements.
//
// Bound by HBM: 2 bytes read and 1 written an element.  A row stays in the
// registers of its threads between the maximum and the codes, so it is read
// once; rows above 32768 elements are read twice (the second time mostly from
// L2).  Short-lived blocks, one row each (a warp a row up to 2048 elements),
// keep more loads in flight than blocks that load a row ahead while they work
// on one (8194 rows of 4096, an earlier state of this kernel: two rows a block
// 3 % slower, eight 15 %).
// Measured on a B200 at 1965 MHz, launches of a graph over inputs larger than
// L2, of 6559 GB/s: 8192x8192 31.0 us (99 %), 8194x4096 16.3 (94 %),
// 16384x2048 16.4 (93 %); widths that leave some threads' last chunk empty
// 8192x7168 28.2 (95 %), 8192x5120 21.3 (90 %), 4096x28672 61.2 (88 %),
// 8192x2880 13.8 (78 %).  Gathered rows are read, searched and converted once
// a copy: 2 copies of 4097 rows of 4096 16.0 us of 10.2 for the bytes, 8 of
// 4096 rows 53.2 of 25.6, where latency and instructions bind (53 % of the
// issue slots), not HBM.

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "fp4_internal.h"
#include "quant_device.cuh"

namespace fp4 {
namespace {

// One row's multipliers: 127 / (amax * pre) = hi + lo, for elements times pre.
struct RowScale {
    float hi, lo;
    float pre;   // a power of two; 1 unless amax is so small or so large that hi or lo left the FP32 range
};

template <bool HALF>
__device__ __forceinline__ float widen(uint32_t bits16)
{
    return HALF ? __half2float(__ushort_as_half((unsigned short)bits16)) : __uint_as_float(bits16 << 16);
}

// amax_bits: the largest magnitude of the row as its 16-bit pattern, finite.
template <bool HALF>
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits)
{
    RowScale s;
    float m = amax_bits ? widen<HALF>(amax_bits) : 1.0f;   // a row of zeros: any
    s.pre = 1.0f;
    if (!HALF) {
        const int eb = (int)(__float_as_uint(m) >> 23);
        if (eb < 27 || eb > 242) {   // outside [2^-100, 2^116)
            // into [4, 8); a subnormal maximum ends below
            s.pre = __uint_as_float((uint32_t)min(256 - eb, 247) << 23);
            m *= s.pre;
        }
    }
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(m));
    s.hi = __fmul_rn(127.0f, r);
    s.lo = __fmul_rn(__fmaf_rn(-s.hi, m, 127.0f), r);
    return s;
}

// What the codes are to be multiplied by: amax / 127, 1 for a row of zeros,
// NaN for a row with an infinity or NaN (its products come out NaN).
template <bool HALF>
__device__ __forceinline__ float code_scale(uint32_t amax_bits)
{
    if (amax_bits == 0u) return 1.0f;
    if (amax_bits >= (HALF ? 0x7C00u : 0x7F80u)) return __uint_as_float(0x7FC00000u);
    return __fdiv_rn(widen<HALF>(amax_bits), 127.0f);
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

template <bool HALF>
__device__ __forceinline__ uint2 codes8(uint4 v, const RowScale& s, bool finite)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const uint64_t hi2 = pair(s.hi, s.hi), lo2 = pair(s.lo, s.lo), round2 = pair(12582912.0f, 12582912.0f);
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
        uint64_t x = pair(lo, hi);
        if (!HALF && s.pre != 1.0f) x = mul2(x, pair(s.pre, s.pre));   // (a row's choice)
        const uint64_t q = add2(fma2(x, hi2, mul2(x, lo2)), round2);
        b[i] = __byte_perm((uint32_t)q, (uint32_t)(q >> 32), 0x0040);
    }
    if (!finite) return make_uint2(0u, 0u);
    return make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
}

// Elements [k, k + 8) of a row of `cols`; nothing behind the row is read.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int k, int cols)
{
    if (k + 8 <= cols) return qdev::ld_stream_coherent(reinterpret_cast<const uint4*>(row + k));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < cols) w[i >> 1] |= (uint32_t)__ldcg(row + k + i) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(int8_t* row, int k, int cols, uint2 q)
{
    if (k + 8 <= cols) {
        *reinterpret_cast<uint2*>(row + k) = q;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < cols) row[k + i] = (int8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
}

// Largest magnitudes of two pairs of 16-bit floats, NaN where either has one
// (the sign of the result says nothing).
template <bool HALF>
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if (HALF)
        asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

struct QuantArgs {
    const uint16_t* x;
    int64_t rows_in, ld;
    int cols;
    const int32_t* index;   // source row of each output row, or NULL
    int64_t rows;
    int8_t* codes;
    int64_t ldc;
    float* scales;
};

// TPR threads a row (32: a warp, several rows a block; else the block),
// CH 8-element chunks a thread; CH = 0: rows of any length, read twice.
// FULL: a row is exactly TPR * CH * 8 elements.
template <bool HALF, int TPR, int CH, int THREADS, bool FULL>
__global__ void __launch_bounds__(THREADS) quantize_int8_kernel(const QuantArgs p)
{
    // This kernel starts before the one before it has ended (0.5 us a launch)
    // and touches nothing until then.  Only then may the next one start its
    // set-up: with the other order a product of static weights could request
    // them while the kernel before this one still writes them (a weight
    // quantized right before the layer's activation).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int ROWS = THREADS / TPR;
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    const bool have = ROWS == 1 || row < p.rows;   // the last block's rows may end before it
    int64_t src = row;
    bool inside = have;
    if (p.index && have) {
        src = __ldcg(p.index + row);   // (the kernel before may have written it)
        inside = src >= 0 && src < p.rows_in;   // an index outside gives a row of zeros
    }
    if (!inside) src = 0;
    const uint16_t* x = p.x + src * p.ld;
    const int cols = inside ? p.cols : 0;
    uint4 v[CH > 0 ? CH : 1];
    uint32_t top = 0;   // the magnitudes of even and odd elements
    auto raise = [&](uint4 u) { top = absmax2<HALF>(top, absmax2<HALF>(absmax2<HALF>(u.x, u.y), absmax2<HALF>(u.z, u.w))); };
    if (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = (c * TPR + t) * 8;
            if (FULL && inside)
                v[c] = qdev::ld_stream_coherent(reinterpret_cast<const uint4*>(x + k));
            else
                v[c] = !FULL && k < cols ? load8(x, k, cols) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) raise(v[c]);
    } else {
        for (int k = t * 8; k < cols; k += TPR * 8) raise(load8(x, k, cols));
    }
    top &= 0x7FFF7FFFu;
    uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
    if (TPR > 32) {
        __shared__ uint32_t part[ROWS][TPR / 32];
        if ((t & 31) == 0) part[threadIdx.x / TPR][t >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) amax = max(amax, part[threadIdx.x / TPR][i]);
    }
    if (!have) return;
    const bool finite = amax < (HALF ? 0x7C00u : 0x7F80u);
    const RowScale s = row_scale<HALF>(finite ? amax : 0u);
    if (t == 0) p.scales[row] = code_scale<HALF>(amax);
    int8_t* out = p.codes + row * p.ldc;
    if (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = (c * TPR + t) * 8;
            if (FULL)
                *reinterpret_cast<uint2*>(out + k) = codes8<HALF>(v[c], s, finite);
            else if (k < p.cols)
                store8(out, k, p.cols, codes8<HALF>(v[c], s, finite));
        }
    } else {
        for (int k = t * 8; k < p.cols; k += TPR * 8)
            store8(out, k, p.cols,
                   codes8<HALF>(k < cols ? load8(x, k, cols) : make_uint4(0u, 0u, 0u, 0u), s, finite));
    }
}

template <bool HALF, int TPR, int CH, int THREADS, bool FULL>
cudaError_t launch_kernel(const QuantArgs& p, cudaStream_t s)
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
    return cudaLaunchKernelEx(&cfg, quantize_int8_kernel<HALF, TPR, CH, THREADS, FULL>, p);
}

template <bool HALF, int TPR, int CH, int THREADS>
cudaError_t launch(const QuantArgs& p, cudaStream_t s)
{
    if (CH > 0 && p.cols == TPR * CH * 8) return launch_kernel<HALF, TPR, CH, THREADS, CH != 0>(p, s);
    return launch_kernel<HALF, TPR, CH, THREADS, false>(p, s);
}

template <bool HALF>
cudaError_t dispatch(const QuantArgs& p, cudaStream_t s)
{
    // A warp a row while it holds it: 16384 rows of 2048 16.5 us, 18.1 with a
    // block of 128 threads a row.
    if (p.cols <= 256) return launch<HALF, 32, 1, 128>(p, s);
    if (p.cols <= 512) return launch<HALF, 32, 2, 128>(p, s);
    if (p.cols <= 1024) return launch<HALF, 32, 4, 128>(p, s);
    if (p.cols <= 2048) return launch<HALF, 32, 8, 128>(p, s);
    // Then a block a row.  Many rows: more chunks a thread, so that more bytes
    // are in flight (8192 rows of 8192: 8 chunks 31.2, 4 30.9, 2 38.5 us; 8194
    // of 4096: 4 16.4, 2 18.1).  Few: more threads (one row of 4096: 2 chunks
    // 1.15, 4 1.23, 8 1.48 us; of 8192: 4 chunks 1.40, 8 1.49).  Gathered rows
    // come from L2 in part, and then the reductions' instructions count: half
    // as many threads (8194 rows of 4096 from 4097 17.1 -> 16.0 us, 4000 from
    // 2000 9.4 -> 8.7; 2000 from 1000 5.7 -> 5.6; in order 16.4 -> 16.6).
    const bool many = p.rows > 1024;
    if (p.cols <= 4096 && p.index && p.rows > 3000) return launch<HALF, 64, 8, 64>(p, s);
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
    const QuantArgs p = {x, rows_in, ld, (int)cols, row_index, rows, codes, ldc, scales};
    const cudaError_t e = dtype == FP4_FP16 ? dispatch<true>(p, s) : dispatch<false>(p, s);
    if (e != cudaSuccess) set_last_error("INT8 quantizer launch", e);
    return e;
}

}  // namespace fp4
