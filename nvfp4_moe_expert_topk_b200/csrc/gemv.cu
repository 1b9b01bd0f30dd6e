// gemv.cu -- products of a few bf16 rows with NVFP4 weights (the projections
// and the shared expert while few sequences are decoded):
//   out[m, n] = bf16( sum_k x[m, k] * e2m1(code[n, k]) * e4m3(scale[n, k / 16]) / gs[segment of n] )
// The activations are not quantised.
//
// What bounds it: the weights are read once (9/16 byte each) and every one has
// to be turned from a nibble and a scale byte into a tensor-core operand.  A
// weight times its scale has 6 significant bits, so it is exact in bf16, and
// bf16 x bf16 products are exact in the fp32 accumulators of
// mma.sync.m16n8k16: the weights are its 16-row operand, the x rows (up to 8,
// or two sets of 8) its 8 columns.  (mma.sync and not tcgen05: the operand is
// made in registers, and at 8 or 16 columns the tensor pipe idles either way.)
//
// Decoding.  A nibble s.ee.m placed at bits 15 | 8..6 of a bf16 is the value
// e2m1 * 2^-126 (subnormal where ee = 0), and an E4M3 byte at bits 11..4 is
// e4m3 * 2^-120, so both conversions are shifts and masks and one packed
// product joins them: (e2m1 * 2^-126) * (e4m3 * 2^118) = weight * 2^-8, exact.
// Two nibbles 16 bits apart are handled at once, which pairs elements i and
// i + 4 of a group of eight; x is paired the same way (a permutation of k
// inside a group does not change the sum).
//
// Tiles.  A warp owns 32 rows, 8 consecutive ones g in each 32-row quarter of
// a 128-row scale block: the four rows' scales of 64 columns then are 16
// consecutive bytes of the layout.  Per step of 128 columns lane (g, t) loads
// 16 bytes of codes of each of its rows (two scale blocks per row) and one
// 16-byte piece of scales; the next step's loads are issued before the current
// step is used.  The steps of a row tile are split over the warps of a block
// and over the blocks of a cluster, whose partial sums meet in shared memory
// in a fixed order.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kStep = 128;               // columns per step

// Nibble pairs (i, i + 4) of eight packed codes as bf16 pairs scaled by 2^-126.
__device__ __forceinline__ void e2m1_pairs(uint32_t q, uint32_t (&p)[4])
{
    const uint32_t r = q >> 8;
    p[0] = ((q << 6) & 0x01C001C0u) | ((q << 12) & 0x80008000u);
    p[1] = ((q << 2) & 0x01C001C0u) | ((q << 8) & 0x80008000u);
    p[2] = ((r << 6) & 0x01C001C0u) | ((r << 12) & 0x80008000u);
    p[3] = ((r << 2) & 0x01C001C0u) | ((r << 8) & 0x80008000u);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// E4M3 byte `byte` of a word, twice, as bf16 * 2^118.
__device__ __forceinline__ uint32_t scale_pair(uint32_t word, int byte)
{
    constexpr uint32_t k2p119 = 0x7B007B00u;
    const uint32_t v = __byte_perm(word, 0u, 0x4040u | byte | byte << 8) << 4;
    return mul_bf16x2(mul_bf16x2(v, k2p119), k2p119);
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One step's weights of a lane: 16 bytes of codes of its four rows, and the
// four rows' scales of the 64 columns that hold its two blocks.
struct WStep {
    uint4 c[4];
    uint4 s;
};

} // namespace

// blockDim = 32 * row_tiles * slices; gridDim = cluster * row groups.
template <int MT>
__global__ void __launch_bounds__(512) gemv_kernel(const GemvArgs a, int slices, int cluster)
{
    extern __shared__ float red[];                 // [warps][8 * MT][32]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int tiles = (blockDim.x >> 5) / slices;  // row tiles of this block
    const int tile = warp / slices, slice = warp - tile * slices;
    const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t tile_id = static_cast<int64_t>(blockIdx.x / cluster) * tiles + tile;
    const int64_t row0 = (tile_id >> 2) * 128 + (tile_id & 3) * 8 + g;
    const int steps = static_cast<int>((a.K + kStep - 1) / kStep);
    const int part = rank * slices + slice, parts = slices * cluster;
    const int s0 = static_cast<int>(static_cast<int64_t>(steps) * part / parts);
    const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (part + 1) / parts);

    const uint8_t *cp[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)                    // rows past N read row N - 1; their sums are not stored
        cp[j] = a.codes + min(row0 + 32 * j, a.N - 1) * (a.K / 2) + 16 * t;
    const uint8_t *sp = a.scales + (min(row0, a.N - 1) >> 7) * (a.K / 64) * 512 + ((tile_id & 3) * 8 + g) * 16;
    float acc[2][MT][4];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[p][m][i] = 0.0f;

    pdl_wait();
    pdl_trigger();
    auto load = [&](WStep &w, int step) {
        const bool on = step < s1 && step * kStep + 32 * t < a.K;
        const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w.c[j] = on ? __ldg(reinterpret_cast<const uint4 *>(cp[j] + static_cast<int64_t>(step) * (kStep / 2))) : z;
        w.s = on ? __ldg(reinterpret_cast<const uint4 *>(sp + (2 * static_cast<int64_t>(step) + (t >> 1)) * 512)) : z;
    };
    WStep cur, nxt;
    load(cur, s0);
    for (int step = s0; step < s1; ++step) {
        load(nxt, step + 1);
        uint4 x[MT][4];
        const int k = step * kStep + 32 * t;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const bool on = 8 * m + g < a.M && k < a.K;
            const uint4 *xs = reinterpret_cast<const uint4 *>(a.x + (8 * m + g) * a.ldx + k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[m][i] = on ? __ldg(xs + i) : make_uint4(0, 0, 0, 0);
        }
        const uint32_t sw[4] = {cur.s.x, cur.s.y, cur.s.z, cur.s.w};
        const int sb = 2 * (t & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {              // eight columns of each lane's 32
            uint32_t b[MT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                b[m][0] = __byte_perm(x[m][i].x, x[m][i].z, 0x5410);
                b[m][1] = __byte_perm(x[m][i].x, x[m][i].z, 0x7632);
                b[m][2] = __byte_perm(x[m][i].y, x[m][i].w, 0x5410);
                b[m][3] = __byte_perm(x[m][i].y, x[m][i].w, 0x7632);
            }
            uint32_t w[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t q = i == 0 ? cur.c[j].x : i == 1 ? cur.c[j].y : i == 2 ? cur.c[j].z : cur.c[j].w;
                const uint32_t sc = scale_pair(sw[j], sb + (i >> 1));
                e2m1_pairs(q, w[j]);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    w[j][u] = mul_bf16x2(w[j][u], sc);
            }
#pragma unroll
            for (int h = 0; h < 4; h += 2)
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        mma_bf16(acc[p][m], w[2 * p][h], w[2 * p + 1][h], w[2 * p][h + 1], w[2 * p + 1][h + 1],
                                 b[m][h], b[m][h + 1]);
        }
        cur = nxt;
    }

    // sums over the slices of a block, then over the blocks of the cluster
    constexpr int kVals = 8 * MT;
    if (slices > 1 || cluster > 1) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    red[(warp * kVals + (p * MT + m) * 4 + i) * 32 + lane] = acc[p][m][i];
        __syncthreads();
        if (slice == 0) {
#pragma unroll
            for (int v = 0; v < kVals; ++v) {
                float s = red[(warp * kVals + v) * 32 + lane];
                for (int w = 1; w < slices; ++w)
                    s += red[((warp + w) * kVals + v) * 32 + lane];
                acc[v / (4 * MT)][v / 4 % MT][v % 4] = s;
                red[(warp * kVals + v) * 32 + lane] = s;
            }
        }
        if (cluster > 1) {
            cluster_sync();
            if (rank == 0 && slice == 0) {
                for (int r = 1; r < cluster; ++r) {
                    const uint32_t peer = map_shared_to_cta(smem_u32(red), r);
#pragma unroll
                    for (int v = 0; v < kVals; ++v) {
                        float s;
                        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                     : "=f"(s)
                                     : "r"(peer + 4u * ((warp * kVals + v) * 32 + lane)));
                        acc[v / (4 * MT)][v / 4 % MT][v % 4] += s;
                    }
                }
            }
            cluster_sync();                        // the peers' shared memory stays until it is read
        }
        if (rank != 0 || slice != 0)
            return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t n = row0 + 32 * j;
        if (n >= a.N)
            continue;
        int seg = 0;
        while (seg + 1 < a.nseg && n >= a.seg_end[seg])
            ++seg;
        const float gs = __ldg(a.gs + seg);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 8 * m + 2 * t + c;
                if (row < a.M)
                    a.out[row * a.ldo + n] =
                        __float2bfloat16_rn(__fdiv_rn(acc[j >> 1][m][2 * (j & 1) + c] * 256.0f, gs));
            }
    }
}

template <int MT>
static cudaError_t launch_mt(const GemvArgs &a, int tiles, int slices, int cluster, cudaStream_t s)
{
    const int warps = tiles * slices;
    const int64_t row_tiles = (a.N + 127) / 128 * 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((row_tiles + tiles - 1) / tiles * cluster));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = warps > tiles || cluster > 1 ? sizeof(float) * 32 * 8 * MT * warps : 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, gemv_kernel<MT>, a, slices, cluster);
}

cudaError_t launch_gemv_as(const GemvArgs &a, int tiles, int slices, int cluster, cudaStream_t s)
{
    return a.M <= 8 ? launch_mt<1>(a, tiles, slices, cluster, s) : launch_mt<2>(a, tiles, slices, cluster, s);
}

cudaError_t launch_gemv(const GemvArgs &a, int num_sms, cudaStream_t s)
{
    const int64_t row_tiles = (a.N + 127) / 128 * 4;
    const int64_t steps = (a.K + kStep - 1) / kStep;
    int64_t parts = std::min<int64_t>(steps, 16LL * num_sms / row_tiles);
    int cluster = 1, slices = 1, tiles = 4;
    if (parts > 1) {
        while (parts > 8 * cluster && cluster < 8)
            cluster *= 2;
        slices = static_cast<int>(std::min<int64_t>(8, (parts + cluster - 1) / cluster));
        tiles = slices >= 3 ? 1 : 2;
    }
    return launch_gemv_as(a, tiles, slices, cluster, s);
}

} // namespace nvfp4
