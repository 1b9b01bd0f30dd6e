// norm.cu -- residual addition + RMS norm with an optional quantised output:
// the step in front of the router, the MoE block and the projections.
//
//   h    = bf16(x + residual)                (stored as the new residual stream)
//   rstd = fp32(1 / sqrt(sum(h^2) / H + eps))
//   y    = fp32((h * rstd) * w)              -> bf16 row
//   NVFP4: the codes and scales nvfp4_quantize makes of the bf16 row
//   E4M3:  per 128 columns of the fp32 y:  a = max|y|, scale = a / 448,
//          q = E4M3(y * (a == 0 ? 0 : 448 / a))
//
// The norm reads the rounded h, so it can be recomputed from the stored
// residual stream.  The sum of squares is held in 64 bits: bf16 squares are
// exact there and the sum is off by ~1e-16, so rstd, y and the codes are the
// same bits whatever the order of summation (rows, threads, launch shape).
//
// Bound by HBM on long batches (10.6 bytes per element with a residual and
// NVFP4 rows), by launch and one pass over a row on short ones: a row stays in
// registers between its sum and its output, 16 columns per thread (one NVFP4
// block, an eighth of an E4M3 group), several rows in flight per SM.  What is
// exact in packed bf16 is done there: one add.bf16x2 rounds the exact sum once,
// as fp32 addition and rounding to bf16 do (fp32 keeps 16 bits below bf16, so
// its own rounding never moves a sum onto or over a border), and the largest
// magnitude of a block is the largest 15-bit pattern.
//
// Measured (one B200, per call in a CUDA graph of calls; from Python one after
// the other in brackets): 1 x 7168 with residual and NVFP4 rows 2.9 us (4.2), 64
// x 7168 to E4M3 3.1 us (4.2), 2041 x 1536 to NVFP4 4.6 us (4.8), 4096 x 7168
// with residual and NVFP4 rows 43.6 us (47.1), which is 5.8 TB/s or 88 % of a
// plain copy.  (One block per SM that loads its next row ahead was slower: 41 us
// against 27 without the residual.)
//
// The next kernel may start as soon as this one has (pdl_trigger): its blocks
// find their place and set up while the rows are worked on, although it reads
// memory only after all of them are done.  A few-row product behind a norm then
// ends 0.6 us earlier (1 x 7168, then 1 x 2048 x 7168: 9.5 instead of 10.2 us);
// norms that follow each other take up to 0.2 us longer (2041 x 1536: 4.6
// instead of 4.4).
#include "internal.h"
#include "quant.cuh"

namespace nvfp4 {

namespace {

__device__ __forceinline__ void unpack8(const uint4 &v, float *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float *f)
{
    uint4 v;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return v;
}

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint4 add8(const uint4 &a, const uint4 &b)
{
    return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z), add_bf16x2(a.w, b.w));
}

// Largest |value| of eight bf16, with the running one (bf16 pairs of magnitudes).
__device__ __forceinline__ uint32_t max8(uint32_t m, const uint4 &v)
{
    m = __vmaxu2(__vmaxu2(m, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
    return __vmaxu2(__vmaxu2(m, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
}

// fp32 pair -> two E4M3 bytes (a in the low byte), nearest even, saturating.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// quantize16 on sixteen bf16 values (quant.cuh), the same steps: only the
// largest magnitude is found in packed form.
__device__ __forceinline__ uint32_t quantize16_bf16(const uint4 &y0, const uint4 &y1, float gs, uint32_t &lo,
                                                    uint32_t &hi)
{
    const uint32_t m = max8(max8(0u, y0), y1);
    const float a = __uint_as_float(max(m & 0xFFFFu, m >> 16) << 16);
    const uint32_t s = cvt_e4m3(__fmul_rn(__fdiv_rn(a, 6.0f), gs));
    const float r = s == 0u ? 0.0f : __fdiv_rn(gs, e4m3_value(s));
    float p[16];
    unpack8(y0, p);
    unpack8(y1, p + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        p[i] = __fmul_rn(p[i], r);
    lo = cvt_e2m1x8(p);
    hi = cvt_e2m1x8(p + 8);
    return s;
}

// fp32(1 / sqrt(m)) by way of 64 bits: two Newton steps on the fp32 estimate
// leave 64-bit rounding errors (~2^-52), as division and square root in 64 bits
// do at five times the instructions; values that fp32 does not hold well take
// those.
__device__ __forceinline__ float inverse_sqrt(double m)
{
    const float mf = static_cast<float>(m);
    if (!(mf > 1e-30f && mf < 1e30f))
        return static_cast<float>(1.0 / sqrt(m));
    double y = rsqrtf(mf);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        y = fma(0.5 * y, fma(-m * y, y, 1.0), y);
    return static_cast<float>(y);
}

} // namespace

// `tpr` threads (a multiple of 32) per row, `blockDim.x / tpr` rows at a time;
// thread i of a row holds the 16-column blocks i, i + tpr, ... (VPT of them).
template <int VPT, int QUANT>
__global__ void __launch_bounds__(512, VPT == 1 ? 3 : VPT == 2 ? 2 : 1) add_rmsnorm_kernel(const NormArgs a, int tpr)
{
    __shared__ double part[16];
    pdl_wait();
    pdl_trigger();
    const int row_in_block = threadIdx.x / tpr;
    const int i0 = threadIdx.x - row_in_block * tpr;
    const int lane = threadIdx.x & 31;
    const int wpr = tpr >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + row_in_block;
    const bool live = t < a.T;
    uint4 h[VPT][2];
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int b = i0 + v * tpr;
        h[v][0] = h[v][1] = make_uint4(0, 0, 0, 0);
        if (live && b < a.nb) {
            const uint4 *xs = reinterpret_cast<const uint4 *>(a.x + t * a.ldx + 16 * b);
            h[v][0] = xs[0];
            h[v][1] = xs[1];
            if (a.residual != nullptr) {
                const uint4 *rs = reinterpret_cast<const uint4 *>(a.residual + t * a.ldr + 16 * b);
                const uint4 r0 = rs[0], r1 = rs[1];
                h[v][0] = add8(h[v][0], r0);
                h[v][1] = add8(h[v][1], r1);
                uint4 *ro = reinterpret_cast<uint4 *>(a.residual_out + t * a.ldro + 16 * b);
                ro[0] = h[v][0];
                ro[1] = h[v][1];
            }
        }
        float f[16];
        unpack8(h[v][0], f);
        unpack8(h[v][1], f + 8);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const double d = f[j];
            sum = fma(d, d, sum);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (wpr > 1) {
        if (lane == 0)
            part[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = 0.0;
        for (int w = 0; w < wpr; ++w)
            sum += part[row_in_block * wpr + w];
    }
    const float rstd = inverse_sqrt(fma(sum, a.inv_cols, a.eps));
    const float gs = QUANT == NVFP4_QUANT_NVFP4 ? __ldg(a.gs) : 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int b = i0 + v * tpr;
        const bool on = live && b < a.nb;
        float f[16], w[16];
        unpack8(h[v][0], f);
        unpack8(h[v][1], f + 8);
        if (on) {
            const uint4 *wp = reinterpret_cast<const uint4 *>(a.weight + 16 * b);
            unpack8(__ldg(wp), w);
            unpack8(__ldg(wp + 1), w + 8);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                w[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
            f[j] = __fmul_rn(__fmul_rn(f[j], rstd), w[j]);
        const uint4 y0 = pack8(f), y1 = pack8(f + 8);
        if (on && a.y != nullptr) {
            uint4 *yo = reinterpret_cast<uint4 *>(a.y + t * a.ldy + 16 * b);
            yo[0] = y0;
            yo[1] = y1;
        }
        if (QUANT == NVFP4_QUANT_NVFP4 && on) {
            uint32_t lo, hi;
            const uint32_t s = quantize16_bf16(y0, y1, gs, lo, hi);
            reinterpret_cast<uint2 *>(a.codes)[t * a.nb + b] = make_uint2(lo, hi);
            uint8_t *sc = static_cast<uint8_t *>(a.scales);
            if (a.layout == NVFP4_SCALES_MMA)
                sc[mma_scale_offset(t, b >> 2, a.nb >> 2) + (b & 3)] = static_cast<uint8_t>(s);
            else
                sc[t * a.nb + b] = static_cast<uint8_t>(s);
        }
        if (QUANT == NVFP4_QUANT_E4M3) {
            // a group of 128 columns = 8 consecutive blocks = 8 lanes
            float m = 0.0f;
            if (on)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    m = fmaxf(m, fabsf(f[j]));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (on) {
                float top = m;
                if (m < 0x1p-100f) {               // 448 / m may not be an fp32 number: both sides times 2^100, exactly
                    top *= 0x1p100f;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        f[j] *= 0x1p100f;
                }
                const float r = m == 0.0f ? 0.0f : __fdiv_rn(448.0f, top);
                uint32_t q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    q[j] = cvt_e4m3x2(__fmul_rn(f[4 * j], r), __fmul_rn(f[4 * j + 1], r)) |
                           cvt_e4m3x2(__fmul_rn(f[4 * j + 2], r), __fmul_rn(f[4 * j + 3], r)) << 16;
                reinterpret_cast<uint4 *>(a.codes)[t * a.nb + b] = make_uint4(q[0], q[1], q[2], q[3]);
                if ((b & 7) == 0)
                    static_cast<float *>(a.scales)[t * ((a.nb + 7) >> 3) + (b >> 3)] = __fdiv_rn(m, 448.0f);
            }
        }
    }
}

namespace {

template <int VPT>
cudaError_t launch_vpt(const NormArgs &a, int tpr, int rpb, cudaStream_t s)
{
    const dim3 grid(static_cast<unsigned>((a.T + rpb - 1) / rpb)), block(static_cast<unsigned>(tpr * rpb));
    switch (a.quant) {
    case NVFP4_QUANT_NVFP4:
        return launch_pdl(add_rmsnorm_kernel<VPT, NVFP4_QUANT_NVFP4>, grid, block, 0, s, a, tpr);
    case NVFP4_QUANT_E4M3:
        return launch_pdl(add_rmsnorm_kernel<VPT, NVFP4_QUANT_E4M3>, grid, block, 0, s, a, tpr);
    default:
        return launch_pdl(add_rmsnorm_kernel<VPT, NVFP4_QUANT_NONE>, grid, block, 0, s, a, tpr);
    }
}

} // namespace

cudaError_t launch_add_rmsnorm(const NormArgs &a, int, cudaStream_t s)
{
    const int vpt = a.nb <= 512 ? 1 : a.nb <= 1024 ? 2 : 4;
    const int tpr = ((a.nb + vpt - 1) / vpt + 31) / 32 * 32;
    const int rpb = tpr >= 256 ? 1 : 256 / tpr;
    switch (vpt) {
    case 1: return launch_vpt<1>(a, tpr, rpb, s);
    case 2: return launch_vpt<2>(a, tpr, rpb, s);
    default: return launch_vpt<4>(a, tpr, rpb, s);
    }
}

} // namespace nvfp4
