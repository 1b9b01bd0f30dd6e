// gemv.cu -- products of a few bf16 rows with NVFP4 weights (the projections
// and the shared expert while few sequences are decoded):
//   out[m, n] = bf16( sum_k x[m, k] * e2m1(code[n, k]) * e4m3(scale[n, k / 16]) / gs[segment of n] )
// The activations are not quantised.
//
// What bounds it: the weights are read once (9/16 byte each), and every one
// has to be turned from a nibble and a scale byte into a tensor-core operand.
// A weight times its scale has 6 significant bits and at most 2688 in value,
// so it is exact in f16: cvt.f16x2.e2m1x2 and one packed product per two
// weights, half the instructions that making bf16 operands with shifts and
// masks takes (measured: 64 lanes a clock and SM for the conversion as for
// the product).  The products run on mma.sync.m16n8k16 (f16, fp32
// accumulators), the weights as its 16-row operand, the x rows (up to 8, or
// two sets of 8) as its columns.  (mma.sync and not tcgen05: the operand is
// made in registers, and at 8 or 16 columns the tensor pipe idles either way.)
//
// x in f16: each row's piece of k that a block sums is scaled by a power of two
// that brings its largest magnitude into [2^14, 2^15); f16 then holds a bf16
// value exactly down to 2^-31 of that largest one.  The power of two is undone
// in fp32.  A block one of whose rows holds a smaller value (not zero) works on
// bf16 operands instead: x as it is, and the weights (6 significant bits) turned
// from f16 to bf16 at three more instructions a pair.  Such a value may be all
// that a sum consists of, if the large ones meet weights of zero.  So x is never
// rounded, whatever it holds.  (Of normally distributed rows one launch in some
// thousands has such a block.)
//
// Tiles.  A warp works on row tiles of 32 rows, 8 consecutive ones g in each
// 32-row quarter of a 128-row scale block: the four rows' scales of 64 columns
// then are 16 consecutive bytes of the layout.  Per step of 256 columns one
// lane brings the tile's codes (a TMA box of 4 quarters x 8 rows x 128 bytes)
// and its scales (4 atoms x 128 bytes) into the warp's own ring in shared
// memory, on into the next tile (the same loads with cp.async by every lane
// stopped at 4 TB/s, from L2 too).  Lane (g, t) owns columns 64 t .. 64 t + 63 of the step,
// in two halves of 32: 16-byte pieces 2 t + h of its rows, which the 128-byte
// swizzle of the boxes puts on distinct banks for every eight lanes, and the
// scale word of atom t.  (Which k goes to which place of the instruction does
// not matter as long as weights and x agree.)
//
// Blocks are persistent (one per SM): each converts its piece of x once, in
// the order its lanes read it, and walks over row tiles.  k is split over the
// blocks of a cluster and over the `slices` warps of a tile; partial sums meet
// in shared memory in a fixed order.  Every wait on a copy is bounded: a warp
// that gives up stops loading, and the sums it has a share in become NaN.
//
// Measured (one B200, per call in a CUDA graph of calls): 3 x 200 x 256 (M x N x
// K) 3.5 us, 1 x 2048 x 7168 7.0 us, 5 x 7168 x 8192 14.1 us (2.4 TB/s), 16 x
// 65536 x 1536 20.5 us (2.9 TB/s); with bf16 operands in every block, the weights
// in L2, 4.7, 9.0, 18.3 and 25.7 us instead of 3.6, 7.2, 13.3 and 18.4.  Of the
// last one 1 us is the launch, 5 us the x phase (loads, largest and smallest
// magnitudes, conversion) and 12 us six steps per warp: 3900 cycles a step and
// scheduler, of which its 3.5 warps' conversions, products and MMAs take 2000
// each at the rates measured alone (2.25, 2 and 8 cycles an instruction).
// More warps (20, 24), another order of the loop's parts or more accumulators
// did not shorten a step; a loop of half the code lengthened it by 3 %.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kStep = 256;               // columns per step: 128 bytes of codes per row

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight packed codes -> four f16 pairs (elements 2 i, 2 i + 1), exact.
__device__ __forceinline__ void e2m1_pairs(uint32_t q, uint32_t (&p)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
        : "r"(q));
}

// Two E4M3 bytes (the low half of v) -> two f16 pairs, each scale twice.
__device__ __forceinline__ void scale_pairs(uint32_t v, uint32_t (&s)[2])
{
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(v));
    s[0] = __byte_perm(h, 0u, 0x1010);
    s[1] = __byte_perm(h, 0u, 0x3232);
}

// f16 pair -> bf16 pair.
__device__ __forceinline__ uint32_t to_bf16x2(uint32_t h)
{
    uint32_t d;
    asm("{\n\t.reg .b16 lo, hi;\n\t.reg .f32 a, b;\n\tmov.b32 {lo, hi}, %1;\n\t"
        "cvt.f32.f16 a, lo;\n\tcvt.f32.f16 b, hi;\n\tcvt.rn.bf16x2.f32 %0, b, a;\n\t}"
        : "=r"(d)
        : "r"(h));
    return d;
}

// bf16 pair times a power of two (both halves of p2) -> f16 pair.
__device__ __forceinline__ uint32_t to_f16x2(uint32_t x, uint32_t p2)
{
    const uint32_t v = mul_bf16x2(x, p2);
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;"
        : "=r"(d)
        : "f"(__uint_as_float(v & 0xFFFF0000u)), "f"(__uint_as_float(v << 16)));
    return d;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kCodeStage = 4096, kScaleStage = 512;            // bytes per ring stage of a warp
constexpr int kMaxWarps = 16, kMaxDepth = 4;
constexpr int kKeep = 4;                           // pieces of x per lane kept from the maximum to the conversion

// A launch's split, and its shared memory in bytes: the rings, the converted x
// of one panel of k, the partial sums of the tiles' slices and those of the
// cluster's blocks.
struct GemvPlan {
    int groups, slices, cluster;                   // row tiles and k slices at a time per block; blocks per cluster
    int clusters;                                  // in the grid
    int depth;                                     // ring stages per warp
    int panel;                                     // steps of x held at a time
    int rounds;                                    // tiles per group
    int rows;                                      // of x
    __host__ __device__ int warps() const { return groups * slices; }
    __host__ __device__ int codes() const { return warps() * depth * kCodeStage; }
    __host__ __device__ int ring() const { return codes() + warps() * depth * kScaleStage; }
    __host__ __device__ int step_x() const { return rows * kStep * 2; }
    __host__ __device__ int x() const { return panel * step_x(); }
    __host__ __device__ int red(int mt) const { return slices > 1 ? warps() * mt * 1024 : 0; }
    __host__ __device__ int owned() const { return (rounds + cluster - 1) / cluster; }
    __host__ __device__ int sums(int mt) const { return cluster > 1 ? cluster * owned() * groups * mt * 1024 : 0; }
    __host__ __device__ int total(int mt) const { return ring() + x() + red(mt) + sums(mt); }
};

// The launch's tensor maps: codes as [N / 32][32][K / 2] (whole blocks of 128
// rows), codes as [N][K / 2] (the last, partial block), scale atoms as
// [blocks * K / 64][512].
struct GemvMaps {
    CUtensorMap blocks, rows, scales;
};

__device__ __forceinline__ void tma_load_3d(void *smem_dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z,
                                           uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Bytes to wait for in the barrier's current phase, without an arrival.
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// All threads of the `n` warps that share barrier `id`.
__device__ __forceinline__ void bar_group(int id, int n)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * n) : "memory");
}

} // namespace

template <int MT>
__global__ void __launch_bounds__(32 * kMaxWarps)
    gemv_kernel(const __grid_constant__ GemvMaps maps, const GemvArgs a, const GemvPlan pl)
{
    extern __shared__ uint8_t sm_raw[];
    __shared__ uint32_t expo[8 * MT];
    __shared__ uint64_t bars[kMaxWarps * kMaxDepth];
    __shared__ float inv_gs[4];
    __shared__ int never_abort;
    constexpr int kVals = 8 * MT;                  // sums per lane and row tile
    // four accumulators in turn, so that an instruction does not wait for the previous one's sums
    constexpr int kChains = MT == 1 ? 2 : 1;
    uint8_t *sm = sm_raw + (-smem_u32(sm_raw) & 1023u);        // (the swizzle's period; still a shared-memory address)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = pl.warps();
    const int g = lane >> 2, t = lane & 3;
    const int group = warp / pl.slices, slice = warp - group * pl.slices;
    const int cluster = pl.cluster, rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cid = blockIdx.x / cluster;
    const int K = static_cast<int>(a.K);
    const int steps = (K + kStep - 1) / kStep;
    const int b0 = steps * rank / cluster, b1 = steps * (rank + 1) / cluster;       // the block's steps
    const int full_blocks = static_cast<int>(a.N >> 7);

    if (cluster > 1)
        cluster_arrive();                          // waited for before the first store to a peer
    if (threadIdx.x < 8 * MT)
        expo[threadIdx.x] = 15u;                   // smallest exponent field: both powers of two stay normal
    uint64_t *bar = bars + warp * kMaxDepth;
    if (lane == 0) {
        for (int d = 0; d < pl.depth; ++d)
            mbar_init(&bar[d], 1);
        never_abort = 0;
        fence_mbar_init();
        if (warp == 0) {
            tma_prefetch_map(&maps.blocks);
            tma_prefetch_map(&maps.scales);
        }
    }
    uint8_t *codes_s = sm + warp * pl.depth * kCodeStage;
    uint8_t *scales_s = sm + pl.codes() + warp * pl.depth * kScaleStage;
    uint4 *xs = reinterpret_cast<uint4 *>(sm + pl.ring());
    float *red = reinterpret_cast<float *>(sm + pl.ring() + pl.x()) + group * pl.slices * (kVals * 32) + lane;
    float *sums = reinterpret_cast<float *>(sm + pl.ring() + pl.x() + pl.red(MT));

    // Tile of round `it` (past the last: rows that do not exist, zeros).
    auto tile_of = [&](int it) { return (it * pl.clusters + cid) * pl.groups + group; };
    // Prefetch cursor over (round, step) up to f_end rounds; lane 0 brings one
    // step into a ring slot; columns past K and rows past N arrive as zeros.
    int f_it = 0, f_end = 0, f_step = 0, f_slot = 0, first = 0, last = 0;
    auto fetch = [&]() {
        if (f_it < f_end && first < last) {
            if (lane == 0) {
                const int tile = tile_of(f_it), blk = tile >> 2, row = (tile & 3) * 8;
                uint64_t *full = &bar[f_slot];
                uint8_t *dst = codes_s + f_slot * kCodeStage;
                mbar_arrive_expect_tx(full, kCodeStage + kScaleStage);
                if (blk < full_blocks)
                    tma_load_3d(dst, &maps.blocks, f_step * (kStep / 2), row, 4 * blk, full);
                else
                    for (int j = 0; j < 4; ++j)
                        tma_load_2d(dst + 1024 * j, &maps.rows, f_step * (kStep / 2), blk * 128 + row + 32 * j, full);
                // (atoms past K are the next block's, or zeros past the last: masked when they are used)
                tma_load_2d(scales_s + f_slot * kScaleStage, &maps.scales, row * 16, blk * (K / 64) + 4 * f_step, full);
            }
            if (++f_step == last) {
                f_step = first;
                ++f_it;
            }
            f_slot = f_slot + 1 == pl.depth ? 0 : f_slot + 1;
        }
    };

    // Pieces of x: for each set m of 8 rows, piece i is 8 columns of each lane's
    // 64 in one step (i / 8, i % 8); warp w takes the pieces w, w + warps, ...
    auto piece = [&](int m, int p0, int i) -> uint4 {
        const int row = 8 * m + g, k = (p0 + (i >> 3)) * kStep + 64 * t + 8 * (i & 7);
        return row < a.M && k < K ? __ldg(reinterpret_cast<const uint4 *>(a.x + row * a.ldx + k))
                                  : make_uint4(0, 0, 0, 0);
    };
    auto put = [&](int m, int i, const uint4 &v, uint32_t p2) {
        xs[(i * pl.rows + 8 * m + g) * 4 + t] =
            make_uint4(to_f16x2(v.x, p2), to_f16x2(v.y, p2), to_f16x2(v.z, p2), to_f16x2(v.w, p2));
    };
    // the same on bf16 operands: x as it is
    auto copy = [&](int p0, int n) {
        for (int m = 0; m < MT; ++m)
            if (8 * m + g < a.M)
                for (int i = warp; i < 8 * n; i += warps)
                    xs[(i * pl.rows + 8 * m + g) * 4 + t] = piece(m, p0, i);
    };
    // 2^(141 - exponent) in bf16, twice
    auto power = [&](int m) { return (268u - expo[8 * m + g]) * 0x00800080u; };
    auto convert = [&](int p0, int n, int from) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if (8 * m + g < a.M) {
                const uint32_t p2 = power(m);
#pragma unroll 4
                for (int i = from; i < 8 * n; i += warps)
                    put(m, i, piece(m, p0, i), p2);
            }
    };
    // this warp's steps of the panel [p0, p0 + n)
    auto share = [&](int p0, int n) {
        first = f_step = p0 + n * slice / pl.slices;
        last = p0 + n * (slice + 1) / pl.slices;
    };

    const bool whole = b1 - b0 <= pl.panel;        // the block's x stays: the ring runs on from tile to tile
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    // the largest exponent of each row's piece of k; the first pieces stay in
    // registers until they are converted.  (Their loads go out before the
    // weights', which would keep them waiting.)
    uint4 keep[MT][kKeep];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int u = 0; u < kKeep; ++u)
            keep[m][u] = warp + u * warps < (b1 - b0) * 8 ? piece(m, b0, warp + u * warps) : make_uint4(0, 0, 0, 0);
    asm volatile("" ::: "memory");
    if (a.withhold && blockIdx.x == 0 && threadIdx.x == 0)
        mbar_expect_tx(&bar[0], 16);               // bytes that never come
    if (whole) {
        share(b0, b1 - b0);
        f_end = pl.rounds;
        for (int d = 0; d < pl.depth; ++d)
            fetch();
    }
    if (threadIdx.x < a.nseg)
        inv_gs[threadIdx.x] = __fdiv_rn(1.0f, __ldg(a.gs + threadIdx.x));
    __syncthreads();                               // expo is initialised
    uint32_t low[MT];                              // the lane's smallest magnitude but 0, less 1
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        uint32_t mx = 0, mn = 0xFFFFFFFFu;
        auto top = [&](const uint4 &v) {
            const uint32_t w[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mx = __vmaxu2(mx, w[i]);
                mn = __viaddmin_u16x2(w[i], 0xFFFFFFFFu, mn);      // (0 becomes the largest)
            }
        };
#pragma unroll
        for (int u = 0; u < kKeep; ++u)
            top(keep[m][u]);
#pragma unroll 4
        for (int i = warp + kKeep * warps; i < (b1 - b0) * 8; i += warps)
            top(piece(m, b0, i));
        mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        mx = max(mx & 0xFFFFu, mx >> 16) >> 7;
        if (t == 0 && mx > 15u)
            atomicMax(&expo[8 * m + g], mx);
        low[m] = min(mn & 0xFFFFu, mn >> 16);
    }
    __syncthreads();
    // a value more than 31 binades below its row's largest (of a row that is finite)
    int far = 0;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int e = static_cast<int>(expo[8 * m + g]);
        far |= e < 255 && static_cast<int>(low[m]) + 1 < (e - 31) * 128;
    }
    if (whole) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int u = 0; u < kKeep; ++u)
                if (8 * m + g < a.M && warp + u * warps < (b1 - b0) * 8)
                    put(m, warp + u * warps, keep[m][u], power(m));
        convert(b0, b1 - b0, warp + kKeep * warps);
    }
    const bool wide = __syncthreads_or(far) != 0;  // bf16 operands
    if (__builtin_expect(wide, 0)) {
        if (threadIdx.x < 8 * MT)
            expo[threadIdx.x] = 141u;              // nothing to undo
        if (whole)
            copy(b0, b1 - b0);
        __syncthreads();
    }

    // value v of a lane: its weight row's place in the tile and its x row
    auto store = [&](int tile, int v, float s) {
        const int j = 2 * (v / (4 * MT)) + ((v >> 1) & 1), row = 8 * (v / 4 % MT) + 2 * t + (v & 1);
        const int64_t n = static_cast<int64_t>(tile >> 2) * 128 + (tile & 3) * 8 + g + 32 * j;
        if (n < a.N && row < a.M) {
            const int seg = (a.nseg > 1 && n >= a.seg_end[0]) + (a.nseg > 2 && n >= a.seg_end[1]) +
                            (a.nseg > 3 && n >= a.seg_end[2]);
            a.out[row * a.ldo + n] = __float2bfloat16_rn(s * inv_gs[seg]);
        }
    };

    // undoes the x row's power of two (each block of a cluster has its own)
    auto unscale = [&](int v, float s) {
        return s * __uint_as_float((expo[8 * (v / 4 % MT) + 2 * t + (v & 1)] - 14u) << 23);
    };

    bool peers_up = cluster == 1, ok = true;
    int slot = 0;
    uint32_t phase = 0;
    for (int it = 0; it < pl.rounds; ++it) {
        float acc[2][MT][kChains][4];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int v = 0; v < 4 * kChains; ++v)
                    acc[p][m][v >> 2][v & 3] = 0.0f;
        // the tile's sums over this warp's steps, on f16 or on bf16 operands
        auto sum_steps = [&](auto form) {
            constexpr bool kWide = decltype(form)::value;
            const auto mma = [](auto &...v) {
                if (kWide)
                    mma_bf16(v...);
                else
                    mma_f16(v...);
            };
            for (int p0 = b0; p0 < b1; p0 += pl.panel) {
                if (!whole) {                          // x does not fit: panel by panel, again for every tile
                    const int n = min(pl.panel, b1 - p0);
                    __syncthreads();                   // the previous panel of x is read
                    if (kWide)
                        copy(p0, n);
                    else
                        convert(p0, n, warp);
                    __syncthreads();
                    share(p0, n);
                    f_it = it;
                    f_end = it + 1;
                    for (int d = 0; d < pl.depth; ++d)
                        if (ok)
                            fetch();
                }
                for (int step = first; step < last && ok; ++step) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&bar[slot], phase, &never_abort));
                    if (!ok)
                        break;
                    const uint8_t *cs = codes_s + slot * kCodeStage + g * 128;
                    uint4 s4 = *reinterpret_cast<const uint4 *>(scales_s + slot * kScaleStage + t * 128 + g * 16);
                    if (step * kStep + 64 * t >= K)
                        s4 = make_uint4(0, 0, 0, 0);   // scales past K are not loaded
                    const uint32_t sw[4] = {s4.x, s4.y, s4.z, s4.w};
                    const uint4 *xp[MT];
#pragma unroll
                    for (int m = 0; m < MT; ++m)       // columns past M repeat row M - 1; their sums are not stored
                        xp[m] = xs + ((step - p0) * 8 * pl.rows + min(8 * m + g, pl.rows - 1)) * 4 + t;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {      // 32 of the lane's 64 columns
                        uint32_t sc[4][2];
                        uint4 c[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            scale_pairs(h ? sw[j] >> 16 : sw[j], sc[j]);
                            c[j] = *reinterpret_cast<const uint4 *>(cs + 1024 * j + (((2 * t + h) ^ g) << 4));
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {  // eight of them
                            uint32_t v[4][4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                e2m1_pairs(q == 0 ? c[j].x : q == 1 ? c[j].y : q == 2 ? c[j].z : c[j].w, v[j]);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                {
                                    v[j][e] = mul_f16x2(v[j][e], sc[j][q >> 1]);
                                    if (kWide)
                                        v[j][e] = to_bf16x2(v[j][e]);
                                }
                            }
                            uint4 x[MT];
#pragma unroll
                            for (int m = 0; m < MT; ++m)
                                x[m] = xp[m][(4 * h + q) * 4 * pl.rows];
#pragma unroll
                            for (int p = 0; p < 2; ++p)                // rows 64 p and 64 p + 32 of the block
#pragma unroll
                                for (int m = 0; m < MT; ++m)
                                    mma(acc[p][m][0], v[2 * p][0], v[2 * p + 1][0], v[2 * p][1], v[2 * p + 1][1], x[m].x,
                                        x[m].y);
#pragma unroll
                            for (int p = 0; p < 2; ++p)
#pragma unroll
                                for (int m = 0; m < MT; ++m)
                                    mma(acc[p][m][kChains - 1], v[2 * p][2], v[2 * p + 1][2], v[2 * p][3], v[2 * p + 1][3],
                                        x[m].z, x[m].w);
                        }
                    }
                    __syncwarp();                      // every lane has read the slot
                    fetch();
                    if (++slot == pl.depth) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
        };
        if (__builtin_expect(!wide, 1))
            sum_steps(std::false_type{});
        else
            sum_steps(std::true_type{});
        if (kChains == 2)
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    acc[p][0][0][v] += acc[p][0][kChains - 1][v];
        if (__builtin_expect(!ok, 0))              // not all of the weights came
#pragma unroll
            for (int v = 0; v < kVals; ++v)
                acc[v / (4 * MT)][v / 4 % MT][0][v & 3] = __int_as_float(0x7FC00000);
        const int tile = tile_of(it);
        if (pl.slices == 1 && cluster == 1) {
            // nothing to add up: straight from the registers
            const int64_t n0 = static_cast<int64_t>(tile >> 2) * 128 + (tile & 3) * 8 + g;
            const bool one = a.nseg == 1 && n0 + 96 < a.N;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int row = 8 * m + 2 * t + c;
                    if (row < a.M) {
                        if (one) {
                            const float q = unscale(4 * m + c, 1.0f), inv = inv_gs[0];
                            __nv_bfloat16 *o = a.out + row * a.ldo + n0;
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                o[32 * j] = __float2bfloat16_rn(acc[j >> 1][m][0][2 * (j & 1) + c] * q * inv);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int v = ((j >> 1) * MT + m) * 4 + 2 * (j & 1) + c;
                                store(tile, v, unscale(v, acc[j >> 1][m][0][2 * (j & 1) + c]));
                            }
                        }
                    }
                }
            continue;
        }
        // The tile's sums over its slices (value v by slice v mod slices), then
        // to the block of the cluster that owns the round.
        if (pl.slices > 1) {
            if (it > 0)
                bar_group(1 + group, pl.slices);   // the previous round's sums are read
#pragma unroll
            for (int v = 0; v < kVals; ++v)
                red[(slice * kVals + v) * 32] = acc[v / (4 * MT)][v / 4 % MT][0][v & 3];
            bar_group(1 + group, pl.slices);
        }
        float *dst_own = sums + ((rank * pl.owned() + it / cluster) * pl.groups + group) * (kVals * 32) + lane;
        uint32_t dst = 0;
        if (cluster > 1) {
            if (!peers_up) {
                cluster_wait();                    // every block of the cluster has started
                peers_up = true;
            }
            dst = map_shared_to_cta(smem_u32(dst_own), it % cluster);
        }
        auto pass_on = [&](int v, float s) {
            s = unscale(v, s);
            if (cluster > 1)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + 128 * v), "f"(s) : "memory");
            else
                store(tile, v, s);
        };
        if (pl.slices == 1) {
#pragma unroll
            for (int v = 0; v < kVals; ++v)
                pass_on(v, acc[v / (4 * MT)][v / 4 % MT][0][v & 3]);
        } else {
            // two values at a time, all loads first, then the sums in order
            for (int v = slice; v < kVals; v += 2 * pl.slices) {
                const int w = v + pl.slices;
                const float *r0 = red + v * 32, *r1 = red + (w < kVals ? w : v) * 32;
                float p0[kMaxWarps], p1[kMaxWarps];
#pragma unroll
                for (int k = 0; k < kMaxWarps; ++k) {
                    p0[k] = k < pl.slices ? r0[k * (kVals * 32)] : 0.0f;
                    p1[k] = k < pl.slices ? r1[k * (kVals * 32)] : 0.0f;
                }
#pragma unroll
                for (int k = 1; k < kMaxWarps; ++k) {
                    p0[0] += p0[k];
                    p1[0] += p1[k];
                }
                pass_on(v, p0[0]);
                if (w < kVals)
                    pass_on(w, p1[0]);
            }
        }
    }
    if (!ok && lane == 0)                          // copies still in flight have landed before the block ends
        for (int d = 0; d < pl.depth; ++d)
            mbar_wait(&bar[(slot + d) % pl.depth], slot + d < pl.depth ? phase : phase ^ 1u, &never_abort);
    if (cluster > 1) {
        if (!peers_up)
            cluster_wait();
        cluster_arrive();
        cluster_wait();
        // the owned rounds: sums over the cluster's blocks in rank order
        for (int it = rank; it < pl.rounds; it += cluster)
            for (int v = slice; v < kVals; v += pl.slices) {
                const float *p = sums + ((it / cluster) * pl.groups + group) * (kVals * 32) + v * 32 + lane;
                const int ld = pl.owned() * pl.groups * (kVals * 32);
                float part[8];                     // (a cluster has 8 blocks at most)
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    part[r] = r < cluster ? p[r * ld] : 0.0f;
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    part[0] += part[r];
                store(tile_of(it), v, part[0]);
            }
    }
}

constexpr int kMaxBytes = 225 * 1024;              // dynamic shared memory of a block

// Clusters of `cluster` blocks (a power of two up to 8) that fit on the current
// device at once, one block per SM; asked once per device and size.  A cluster
// lies in one group of SMs, so fewer fit than SMs / cluster.
int gemv_clusters(int cluster, int num_sms)
{
    constexpr int kMaxDev = 64;
    static int cached[kMaxDev][4];                 // 0: not yet asked
    static std::mutex mu;
    if (cluster == 1)
        return num_sms;
    const int size = cluster == 2 ? 1 : cluster == 4 ? 2 : 3;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev)
        return num_sms / cluster;
    std::lock_guard<std::mutex> lock(mu);
    if (cached[dev][size] > 0)
        return cached[dev][size];
    int n = 0;
    if (cudaFuncSetAttribute(gemv_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxBytes + 1024) ==
        cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(num_sms / cluster * cluster));
        cfg.blockDim = dim3(32 * kMaxWarps);
        cfg.dynamicSmemBytes = kMaxBytes + 1024;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, gemv_kernel<2>, &cfg) != cudaSuccess)
            n = 0;
    }
    (void)cudaGetLastError();
    if (n <= 0 || n > num_sms / cluster)
        n = num_sms / cluster;
    cached[dev][size] = n;
    return n;
}

// The split (groups, slices, cluster) completed for a shape, `fit` clusters at
// a time; panel < 1: it does not fit into shared memory.
static GemvPlan complete_plan(const GemvArgs &a, int groups, int slices, int cluster, int fit)
{
    const int mt = a.M <= 8 ? 1 : 2;
    const int row_tiles = static_cast<int>((a.N + 127) / 128 * 4);
    const int steps = static_cast<int>((a.K + kStep - 1) / kStep);
    const int block_steps = (steps + cluster - 1) / cluster;
    GemvPlan p{};
    p.groups = groups;
    p.slices = slices;
    p.cluster = cluster;
    p.rows = static_cast<int>(a.M);
    const int tiles = (row_tiles + groups - 1) / groups;
    p.rounds = (tiles + fit - 1) / fit;
    p.clusters = (tiles + p.rounds - 1) / p.rounds;
    p.depth = 2;                                           // deeper beside the whole x where there is room
    const int room = kMaxBytes - p.total(mt);
    p.depth += std::min(kMaxDepth - 2, std::max(0, (room - block_steps * p.step_x()) / (p.ring() / 2)));
    p.panel = std::min(block_steps, (kMaxBytes - p.total(mt)) / p.step_x());
    return p;
}

// Estimated time of a plan in 10 ns, less what all plans share.  The weights of
// the terms are a fit to the device times of all splits of 22 shapes (M 1 to
// 16, N 33 to 65536, K 64 to 16384; off by 10 % rms, and the split it picks
// within 3 % of the best one tried for 17 of them, 13 % at worst): a round's
// steps cost a latency and a share per warp, plus the meeting of the slices,
// the block's pieces of x per warp, and the meeting of the cluster.
static int plan_cost(const GemvPlan &p, int mt, int steps)
{
    const int block_steps = (steps + p.cluster - 1) / p.cluster;
    const int s = (block_steps + p.slices - 1) / p.slices, w = p.warps();
    const int pieces = (block_steps * 8 + w - 1) / w;
    const bool sl = p.slices > 1, cl = p.cluster > 1;
    if (p.panel < block_steps)                             // x converted again for every tile
        return (1 << 28) + p.rounds * block_steps;
    return mt == 1 ? p.rounds * (s * (26 + 12 * w) + 5 * cl + 83) + 21 * pieces + 119 * cl
                   : p.rounds * (s * (80 + 13 * w) + 53 * sl) + 26 * pieces + 232 * cl;
}

template <int MT>
static cudaError_t launch_mt(const GemvArgs &a, const GemvPlan &p, cudaStream_t s)
{
    static unsigned long long attr_done = 0;
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(gemv_kernel<MT>), kMaxBytes + 1024, &attr_done);
    if (e != cudaSuccess)
        return e;
    GemvMaps maps;
    const uint64_t ld = static_cast<uint64_t>(a.K / 2);
    if (code_map(&maps.rows, a.codes, a.N, a.K / 2, 8) != NVFP4_OK)
        return cudaErrorInvalidValue;
    maps.blocks = maps.rows;
    if (a.N >= 128) {
        const uint64_t dims[3] = {ld, 32, static_cast<uint64_t>(a.N / 32)}, strides[2] = {ld, 32 * ld};
        const uint32_t box[3] = {128, 8, 4};
        if (byte_map(&maps.blocks, a.codes, 3, dims, strides, box, true) != NVFP4_OK)
            return cudaErrorInvalidValue;
    }
    {
        const uint64_t dims[2] = {512, static_cast<uint64_t>((a.N + 127) / 128 * (a.K / 64))}, strides[1] = {512};
        const uint32_t box[2] = {128, 4};
        if (byte_map(&maps.scales, a.scales, 2, dims, strides, box, false) != NVFP4_OK)
            return cudaErrorInvalidValue;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.clusters * p.cluster));
    cfg.blockDim = dim3(32 * p.warps());
    cfg.dynamicSmemBytes = p.total(MT) + 1024;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, gemv_kernel<MT>, maps, a, p);
}

static cudaError_t launch_plan(const GemvArgs &a, const GemvPlan &p, cudaStream_t s)
{
    if (p.panel < 1)
        return cudaErrorInvalidValue;
    return a.M <= 8 ? launch_mt<1>(a, p, s) : launch_mt<2>(a, p, s);
}

cudaError_t launch_gemv(const GemvArgs &a, int num_sms, cudaStream_t s)
{
    const int steps = static_cast<int>((a.K + kStep - 1) / kStep);
    GemvPlan best{};
    int least = 0;
    for (int cluster = 1; cluster <= 8 && cluster <= steps; cluster *= 2) {
        const int fit = gemv_clusters(cluster, num_sms);
        for (int groups = 1; groups <= kMaxWarps; ++groups)
            for (int slices = 1; slices * groups <= kMaxWarps && slices * cluster <= steps; ++slices) {
                const GemvPlan p = complete_plan(a, groups, slices, cluster, fit);
                const int cost = p.panel < 1 ? 1 << 30 : plan_cost(p, a.M <= 8 ? 1 : 2, steps);
                if (best.groups == 0 || cost < least) {
                    best = p;
                    least = cost;
                }
            }
    }
    return launch_plan(a, best, s);
}

} // namespace nvfp4
