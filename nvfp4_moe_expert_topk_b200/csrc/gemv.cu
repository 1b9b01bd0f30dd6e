// gemv.cu -- products of a few bf16 rows with NVFP4 weights (the projections
// and the shared expert while few sequences are decoded):
//   out[m, n] = bf16( sum_k x[m, k] * e2m1(code[n, k]) * e4m3(scale[n, k / 16]) / gs[segment of n] )
// The activations are not quantised.  Products and sums in fp32.
#include "internal.h"
#include "quant.cuh"

namespace nvfp4 {

namespace {

// Two E2M1 nibbles of a byte -> exact fp32 pair (low nibble first).
__device__ __forceinline__ float2 e2m1x2_value(uint32_t byte)
{
    uint32_t h2;
    asm("{\n\t.reg .b8 b, z;\n\t.reg .b16 w;\n\tcvt.u16.u32 w, %1;\n\tmov.b16 {b, z}, w;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(h2)
        : "r"(byte));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h2));
}

} // namespace

// One warp per weight row; lane l takes the 16-element blocks l, l + 32, ...
__global__ void __launch_bounds__(256) gemv_kernel(const GemvArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (n >= a.N)
        return;
    float acc[kGemvMaxRows];
#pragma unroll
    for (int m = 0; m < kGemvMaxRows; ++m)
        acc[m] = 0.0f;
    const int nb = static_cast<int>(a.K / 16);
    for (int b = lane; b < nb; b += 32) {
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(a.codes + n * (a.K / 2)) + b);
        const float s = e4m3_value(__ldg(a.scales + mma_scale_offset(n, b >> 2, nb >> 2) + (b & 3)));
        float w[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 p = e2m1x2_value(((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 255u);
            w[2 * j] = p.x * s;
            w[2 * j + 1] = p.y * s;
        }
#pragma unroll
        for (int m = 0; m < kGemvMaxRows; ++m) {
            if (m < a.M) {
                const __nv_bfloat16 *xr = a.x + m * a.ldx + 16 * b;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    acc[m] = fmaf(__bfloat162float(xr[j]), w[j], acc[m]);
            }
        }
    }
    int seg = 0;
    while (seg + 1 < a.nseg && n >= a.seg_end[seg])
        ++seg;
    const float gs = __ldg(a.gs + seg);
#pragma unroll
    for (int m = 0; m < kGemvMaxRows; ++m) {
        if (m < a.M) {
            float v = acc[m];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0)
                a.out[m * a.ldo + n] = __float2bfloat16_rn(__fdiv_rn(v, gs));
        }
    }
}

cudaError_t launch_gemv(const GemvArgs &a, int, cudaStream_t s)
{
    return launch_pdl(gemv_kernel, dim3(static_cast<unsigned>((a.N + 7) / 8)), dim3(256), 0, s, a);
}

} // namespace nvfp4
