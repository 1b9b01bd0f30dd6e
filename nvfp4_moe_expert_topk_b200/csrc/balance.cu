// balance.cu -- load statistics of the router, its balance loss and the
// gradient with respect to the logits.
//
// Per token:  p = softmax(l), or sigmoid(l) / sum sigmoid(l).
// Per sequence s (tokens [offsets[s], offsets[s + 1])), over the n tokens that
// have a slot (an id in [0, E)):
//   counts[e] = number of slots with expert e,   P[e] = sum_t p[t, e],
//   loss = E / (k n^2) * sum_e counts[e] * P[e]        (0 when n = 0).
// Gradient, c = grad_loss[s] * E / (k n^2):
//   softmax  d[e] = c * p[e] * (counts[e] - sum_j p[j] counts[j])
//   sigmoid  d[e] = the same * (1 - sigmoid(l[e])),
// plus, for the renormalised weights w_j over the row's slots with gradient
// g_j:  d[id_j] += w_j * (g_j - sum_i g_i w_i), for sigmoid * (1 - sigmoid(l)).
//
// The tokens are cut into chunks that never cross a sequence: with C tokens
// per chunk, sequence s owns the chunk slots off(s) / C + s onwards (one per
// multiple of C that it touches), so a block finds its sequence by a binary
// search, and a ragged batch needs no host-side plan.  Every chunk leaves its
// sums in the workspace and a second kernel adds them in slot order: no
// floating-point atomics, so results do not depend on timing.
//
// Both directions stream the logits once (4 bytes read per logit, 4 written
// by the gradient) and are bound by HBM on long batches and by latency on
// short ones: one warp per token with the row in registers, and the next
// token's row, ids and weight gradients are loaded while the current one is
// worked on.
//
// Measured (one B200, per call in a CUDA graph of calls; softmax where nothing
// else is said): loss of 64 x 48 3.3 us (sigmoid), of 4096 x 384 in 7 sequences
// 7.6 us, of 65536 x 384 24.7 us (4.1 TB/s; sigmoid 27.2); gradient with weight
// gradients of 4096 x 384 5.5 us (sigmoid), of 65536 x 384 46.4 us (4.4 TB/s;
// sigmoid 48.7).  The long ones execute 173 and 380 instructions a token and warp
// (scores, sums, the slots' part of the gradient) at 55 % of the issue rate, and
// wait for loads (the largest stall) between them.  Rows of sigmoids that fp32
// does not hold cost their warp a second pass: with one in a thousand 65536 x 384
// takes 33 and 80 us, with nothing else 84 and 250.  Rows of 64 experts or fewer
// leave half the lanes idle: 65536 x 48 takes 13.4 us and 24 us.
#include "internal.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 8;                   // block of the gradient
constexpr int kThreads = 32 * kWarps;
constexpr int kSumThreads = 512;            // block that adds chunks up
constexpr unsigned kAll = 0xffffffffu;

// Columns of a chunk's row of sums, so that rows start on 16 bytes.
__host__ __device__ constexpr int padded(int E) { return (E + 3) & ~3; }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Sums over the warp of four values at once (each lane gets all four): the
// first two exchanges halve the values a lane carries, so that ten exchanges
// do what four separate sums take twenty for, in six dependent steps.
__device__ __forceinline__ void warp_sum4(float (&v)[4])
{
    const int lane = threadIdx.x & 31;
    const bool up16 = (lane & 16) != 0, up8 = (lane & 8) != 0;
    const float a = (up16 ? v[2] : v[0]) + __shfl_xor_sync(kAll, up16 ? v[0] : v[2], 16);
    const float b = (up16 ? v[3] : v[1]) + __shfl_xor_sync(kAll, up16 ? v[1] : v[3], 16);
    float s = (up8 ? b : a) + __shfl_xor_sync(kAll, up8 ? a : b, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        s += __shfl_xor_sync(kAll, s, o);
#pragma unroll
    for (int i = 0; i < 4; ++i)                    // value i is in the lanes 8 i .. 8 i + 7
        v[i] = __shfl_sync(kAll, s, 8 * i);
}

__device__ __forceinline__ float warp_max(float v)
{
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// All threads of the cluster; what was stored before an arrival is seen after
// the wait.
__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// exp(x), x <= 0 or moderate: 2^(x log2 e) on the special-function unit, off by
// 2 ulp and by the rounding of the product (|x| 2^-24 relative); results below
// 2^-126 are 0.
__device__ __forceinline__ float exp_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// 1 / x within 1 ulp; 0 for infinity.
__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float sigmoid_fast(float x)
{
    return rcp_fast(1.0f + exp_fast(-x));
}

// sigmoid(x) and 1 - sigmoid(x) = sigmoid(-x), neither by subtraction: the smaller one is
// e^-|x| / (1 + e^-|x|).
__device__ __forceinline__ void sigmoid_pair(float x, float &s, float &complement)
{
    const float t = exp_fast(-fabsf(x)), large = rcp_fast(1.0f + t), small = t * large;
    s = x < 0.0f ? small : large;
    complement = x < 0.0f ? large : small;
}

// 1 / x, 0 for 0.
__device__ __forceinline__ float inverse(float x)
{
    return x == 0.0f ? 0.0f : __frcp_rn(x);
}

// Rows of low sigmoids.  Where sigmoids that are to be divided by their sum are
// all below kTiny (a sum below it says so), they are e^l to fp32 accuracy and
// their slopes 1: e^(l - max l) then takes their place, which fp32 holds however
// low the logits are.  Below kMasked (a mask of the type's lowest value) a logit
// counts as -inf.  Such rows are rare: the main loops leave them out, and a warp
// that met one goes over its tokens again behind its loop (handled in the loop
// they cost all other rows 3 to 8 %).  Both times the sum is taken by the same
// steps, so that they agree on which rows these are.
constexpr float kTiny = 1.0f / (1 << 30), kMasked = -1e30f;

// 1 / sum of a row's scores, 0 for a row that is left out.
template <bool SIG>
__device__ __forceinline__ float inverse_sum(float sum)
{
    return SIG ? (sum < kTiny ? 0.0f : __frcp_rn(sum)) : inverse(sum);
}

__device__ __forceinline__ float low_score(float l, float m)
{
    return l < kMasked ? 0.0f : exp_fast(l - m);
}

// out[e] += the row's share of e (counts null), or its gradient of the loss for
// counts and their coefficient; the whole warp.
__device__ __forceinline__ void add_low_row(const float *row, int E, int lane, const int32_t *counts, float coef,
                                            float *out)
{
    float m = -INFINITY, sum = 0.0f, dot = 0.0f;
#pragma unroll 1
    for (int c = lane; c < E; c += 32)
        m = row[c] < kMasked ? m : fmaxf(m, row[c]);
    m = warp_max(m);
    if (m == -INFINITY)                            // nothing but masks
        return;
#pragma unroll 1
    for (int c = lane; c < E; c += 32) {
        const float v = low_score(row[c], m);
        sum += v;
        if (counts != nullptr)
            dot = fmaf(v, coef * static_cast<float>(counts[c]), dot);
    }
    const float inv = inverse(warp_sum(sum));
    dot = warp_sum(dot) * inv;
#pragma unroll 1
    for (int c = lane; c < E; c += 32) {
        const float p = low_score(row[c], m) * inv;
        out[c] += counts == nullptr ? p : p * (coef * static_cast<float>(counts[c]) - dot);
    }
}

// Start of sequence s (s = S: end of the last), clamped into [0, T].
__device__ __forceinline__ int seq_start(const BalanceArgs &a, int s)
{
    if (a.offsets == nullptr)
        return s == 0 ? 0 : static_cast<int>(a.T);
    const int v = __ldg(a.offsets + s);
    return min(max(v, 0), static_cast<int>(a.T));
}

__device__ __forceinline__ int first_slot(const BalanceArgs &a, int s)
{
    return seq_start(a, s) / a.chunk + s;
}

// The last s in [0, S) with before(s), where before holds up to some s (and is
// taken to hold for 0); the whole warp looks at 32 places at a time.
template <typename F>
__device__ __forceinline__ int last_sequence(int S, int lane, F before)
{
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const int n = __popc(__ballot_sync(kAll, at < hi && (at == lo || before(at))));
        lo += (n - 1) * step;
        hi = min(lo + step, hi);
    }
    return lo;
}

// Tokens [t0, t1) of chunk slot `slot` of sequence s (empty: t0 >= t1).
__device__ __forceinline__ void slot_tokens(const BalanceArgs &a, int s, int slot, int &t0, int &t1)
{
    const int o0 = seq_start(a, s), o1 = seq_start(a, s + 1);
    const int64_t c = static_cast<int64_t>(slot - s) * a.chunk;
    t0 = static_cast<int>(max(static_cast<int64_t>(o0), c));
    t1 = static_cast<int>(min(static_cast<int64_t>(o1), c + a.chunk));
}

// One row in a warp's registers, 4 * P values per lane.  V4: 16-byte loads,
// lane l holds columns 4 (l + 32 i) .. + 3; else columns l + 32 j.  Columns
// past E hold -inf.
template <int P, bool V4>
struct Row {
    float v[4 * P];
    static __device__ __forceinline__ int col(int lane, int q)
    {
        return V4 ? 4 * (lane + 32 * (q >> 2)) + (q & 3) : lane + 32 * q;
    }
    __device__ __forceinline__ void load(const float *row, int E, int lane)
    {
        if (V4) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = 4 * (lane + 32 * i);
                // (P is E / 128 rounded up, up to 4: only the last piece can be short)
                const bool in = (P <= 4 && i < P - 1) || c < E;
                const float4 f = in ? __ldg(reinterpret_cast<const float4 *>(row + c))
                                    : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4 * P; ++q)
                v[q] = col(lane, q) < E ? __ldg(row + col(lane, q)) : -INFINITY;
        }
    }
    // scores (exp(l - max) or sigmoid(l)) in place; returns the lane's part of
    // their sum (which is 0 for a row of -inf: no probability anywhere)
    template <bool SIG>
    __device__ __forceinline__ float scores()
    {
        float sum = 0.0f;
        if (!SIG) {
            float m = v[0];
#pragma unroll
            for (int q = 1; q < 4 * P; ++q)
                m = fmaxf(m, v[q]);
            m = warp_max(m);
            if (m == -INFINITY)
                m = 0.0f;
#pragma unroll
            for (int q = 0; q < 4 * P; ++q) {
                v[q] = exp_fast(v[q] - m);
                sum += v[q];
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4 * P; ++q) {
                v[q] = sigmoid_fast(v[q]);
                sum += v[q];
            }
        }
        return sum;
    }
    // sigmoids, each passed to f, and the lane's part of their sum; in place stays the smaller one of the score and
    // its complement (their product is the slope)
    template <typename F>
    __device__ __forceinline__ float sigmoids(F f)
    {
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < 4 * P; ++q) {
            float s, complement;
            sigmoid_pair(v[q], s, complement);
            sum += s;
            f(q, s);
            v[q] = fminf(s, complement);
        }
        return sum;
    }
};

} // namespace

// Tokens a warp holds at a time: one is worked on in place while the others are
// on their way (short rows need several to fill the memory's latency; of the
// longest rows one alone leaves registers for half as many warps more, which
// runs the gradient at 24000 x 1024 in 64 us instead of about 90).
__host__ __device__ constexpr int tokens_held(int P) { return P == 1 ? 4 : P <= 4 ? 2 : 1; }

// Blocks per SM, by the registers that a row of up to 128 P columns takes.
// (Few blocks of many warps: half as many chunks to add up as with eight warps each.)
__host__ __device__ constexpr int chunk_warps(int P, bool whole) { return P == 4 && !whole ? 12 : 16; }
__host__ __device__ constexpr int chunk_blocks(int P) { return P <= 4 ? 2 : 1; }
__host__ __device__ constexpr int backward_blocks(int P) { return P <= 2 ? 4 : P == 4 ? 2 : 3; }

// Sums of a run of tokens of one sequence: a chunk's, left in the workspace, or
// (WHOLE, short batches) a whole sequence's, with its loss, in one launch.
template <int P, bool V4, bool SIG, bool WHOLE>
__global__ void __launch_bounds__(32 * chunk_warps(P, WHOLE), WHOLE ? 1 : chunk_blocks(P)) balance_chunk_kernel(const BalanceArgs a)
{
    constexpr int W = chunk_warps(P, WHOLE), D = tokens_held(P);
    extern __shared__ float sm[];                 // [W][E] probability sums, then [E] int counts
    __shared__ int tokens_s;
    __shared__ double red[W];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E, slot = blockIdx.x;
    int seq, t0, t1;
    if (WHOLE) {
        seq = slot;
        t0 = seq_start(a, seq);
        t1 = seq_start(a, seq + 1);
    } else {
        seq = last_sequence(a.S, lane, [&](int s) { return first_slot(a, s) <= slot; });
        slot_tokens(a, seq, slot, t0, t1);
        if (t0 >= t1)
            return;
    }
    // (a padded token's logits are not used, but they are there to be read)
    Row<P, V4> ring[D];
    int ids[D];
    int tf = t0 + warp;                            // next token to fetch, its row and its ids
    const float *lf = a.logits + static_cast<int64_t>(tf) * E;
    const int32_t *idf = a.ids + static_cast<int64_t>(tf) * a.ld_ids + lane;
    auto fetch = [&](int u) {
        if (tf < t1) {
            ids[u] = lane < a.k ? __ldg(idf) : -1;
            ring[u].load(lf, E, lane);
        }
        tf += W;
        lf += W * E;
        idf += W * a.ld_ids;
    };
#pragma unroll
    for (int u = 0; u < D; ++u)
        fetch(u);
    int *hist = reinterpret_cast<int *>(sm + W * E);
    for (int e = threadIdx.x; e < E; e += 32 * W)
        hist[e] = 0;
    if (threadIdx.x == 0)
        tokens_s = 0;
    __syncthreads();
    float acc[4 * P];
#pragma unroll
    for (int q = 0; q < 4 * P; ++q)
        acc[q] = 0.0f;
    int tokens = 0;
    bool low = false;
    for (int tb = t0 + warp; tb < t1; tb += D * W) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
            const int t = tb + u * W;
            if (t >= t1)
                break;
            Row<P, V4> &r = ring[u];
            const int id = ids[u];
            const bool on = id >= 0 && id < E;
            if (__any_sync(kAll, on)) {            // not a padded token
                ++tokens;
                if (on)
                    atomicAdd(hist + id, 1);
                const float sum = warp_sum(r.template scores<SIG>()), inv = inverse_sum<SIG>(sum);
                low |= SIG && sum < kTiny;
#pragma unroll
                for (int q = 0; q < 4 * P; ++q)
                    acc[q] = fmaf(r.v[q], inv, acc[q]);
            }
            fetch(u);
        }
    }
    if (lane == 0 && tokens)
        atomicAdd(&tokens_s, tokens);
#pragma unroll
    for (int q = 0; q < 4 * P; ++q) {
        const int c = Row<P, V4>::col(lane, q);
        if (c < E)
            sm[warp * E + c] = acc[q];
    }
    if (SIG && low) {
        __syncwarp();
#pragma unroll 1
        for (int t = t0 + warp; t < t1; t += W) {
            const int id = lane < a.k ? __ldg(a.ids + static_cast<int64_t>(t) * a.ld_ids + lane) : -1;
            const float *row = a.logits + static_cast<int64_t>(t) * E;
            if (!__any_sync(kAll, id >= 0 && id < E))
                continue;
            Row<P, V4> r;
            r.load(row, E, lane);
            if (warp_sum(r.template scores<true>()) < kTiny)
                add_low_row(row, E, lane, nullptr, 0.0f, sm + warp * E);
        }
    }
    __syncthreads();
    pdl_trigger();                                 // (the next kernel's blocks would only be in the way before)
    const int Ep = padded(E);
    double dot = 0.0;
    for (int e = threadIdx.x; e < E; e += 32 * W) {
        float p = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w)
            p += sm[w * E + e];
        if (WHOLE) {
            a.counts[static_cast<int64_t>(seq) * E + e] = hist[e];
            a.probs[static_cast<int64_t>(seq) * E + e] = p;
            dot += static_cast<double>(hist[e]) * p;
        } else {
            a.part_p[static_cast<int64_t>(slot) * Ep + e] = p;
            a.part_c[static_cast<int64_t>(slot) * Ep + e] = hist[e];
        }
    }
    if (WHOLE) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            dot += __shfl_xor_sync(kAll, dot, o);
        if (lane == 0)
            red[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < W; ++w)
                dot += red[w];
            const double n = tokens_s;
            a.tokens[seq] = tokens_s;
            a.loss[seq] = tokens_s == 0 ? 0.0f : static_cast<float>(dot * E / (a.k * n * n));
        }
    } else if (threadIdx.x == 0) {
        a.part_n[slot] = tokens_s;
    }
}

// Sums over a sequence's chunks and its loss: one cluster of blocks per
// sequence, block x for the experts [x, x + 1) * cols; one half of its threads
// adds probabilities, the other counts, thread (i, c) four experts' in the
// chunks i, i + rows, ...; the rows' sums and the blocks' parts of the loss
// (through shared memory of the cluster's first block) are added in order.
// Bound by latency: the offsets, then up to kSumLoads loads of a thread at once
// (four arrays' worth of half as many took 0.5 to 3 us more), then two
// meetings.
constexpr int kSumLoads = 8;
constexpr int kSumRows = 32;                       // at most

__global__ void __launch_bounds__(kSumThreads, 2) balance_sum_kernel(const BalanceArgs a, int cols)
{
    constexpr int kHalf = kSumThreads / 2;
    __shared__ double sp[4 * kHalf];
    __shared__ int sc[4 * kHalf];
    __shared__ int sn[kSumThreads / 32];
    __shared__ double red[kSumThreads / 32], dots[8];
    const int blocks = gridDim.x, rank = blockIdx.x;
    if (blocks > 1)
        cluster_arrive();                          // waited for before the store to the first block
    const int quads = cols / 4, rows = min(kHalf / quads, kSumRows);
    const int half = threadIdx.x % kHalf, row = half / quads, c4 = 4 * (half - row * quads);
    const int s = blockIdx.y, E = a.E, Ep = padded(E), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    const int o0 = seq_start(a, s), o1 = seq_start(a, s + 1);
    const int slot0 = o0 / a.chunk + s;
    const int nslots = o1 > o0 ? (o1 - 1) / a.chunk - o0 / a.chunk + 1 : 0;    // non-empty ones
    int n = 0;
    for (int i = threadIdx.x; i < nslots; i += kSumThreads)
        n += __ldcg(a.part_n + slot0 + i);
    const bool mine = row < rows && rank * cols + c4 < E;
    const int64_t first = static_cast<int64_t>(slot0) * Ep + rank * cols + c4;
    const int at = row * cols + c4;
    if (threadIdx.x < kHalf) {
        double p[4] = {0.0, 0.0, 0.0, 0.0};
        for (int i = row; mine && i < nslots; i += kSumLoads * rows) {
            float4 f[kSumLoads];
#pragma unroll
            for (int u = 0; u < kSumLoads; ++u)
                f[u] = i + u * rows < nslots ? __ldcg(reinterpret_cast<const float4 *>(
                                                   a.part_p + first + static_cast<int64_t>(i + u * rows) * Ep))
                                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int u = 0; u < kSumLoads; ++u)
                p[0] += f[u].x, p[1] += f[u].y, p[2] += f[u].z, p[3] += f[u].w;
        }
        if (row < rows)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sp[at + j] = p[j];
    } else {
        int c[4] = {0, 0, 0, 0};
        for (int i = row; mine && i < nslots; i += kSumLoads * rows) {
            int4 m[kSumLoads];
#pragma unroll
            for (int u = 0; u < kSumLoads; ++u)
                m[u] = i + u * rows < nslots ? __ldcg(reinterpret_cast<const int4 *>(
                                                   a.part_c + first + static_cast<int64_t>(i + u * rows) * Ep))
                                             : make_int4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < kSumLoads; ++u)
                c[0] += m[u].x, c[1] += m[u].y, c[2] += m[u].z, c[3] += m[u].w;
        }
        if (row < rows)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sc[at + j] = c[j];
    }
    pdl_trigger();
    n = __reduce_add_sync(kAll, n);
    if (lane == 0)
        sn[warp] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < kSumThreads / 32; ++w)
        n += sn[w];
    const int e = rank * cols + threadIdx.x;
    double dot = 0.0;
    if (threadIdx.x < cols && e < E) {
        double ps = 0.0;
        int cs = 0;
#pragma unroll 8
        for (int i = 0; i < rows; ++i) {
            ps += sp[i * cols + threadIdx.x];
            cs += sc[i * cols + threadIdx.x];
        }
        a.counts[static_cast<int64_t>(s) * E + e] = cs;
        a.probs[static_cast<int64_t>(s) * E + e] = static_cast<float>(ps);
        dot = cs * ps;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        dot += __shfl_xor_sync(kAll, dot, o);
    if (lane == 0)
        red[warp] = dot;
    __syncthreads();
    if (blocks > 1)
        cluster_wait();
    if (threadIdx.x == 0) {
        dot = 0.0;
        for (int w = 0; w < kSumThreads / 32; ++w)
            dot += red[w];
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(map_shared_to_cta(smem_u32(dots + rank), 0)), "d"(dot)
                     : "memory");
    }
    if (blocks > 1) {
        cluster_arrive();
        cluster_wait();
    }
    if (rank == 0 && threadIdx.x == 0) {
        dot = 0.0;
        for (int i = 0; i < blocks; ++i)
            dot += dots[i];
        a.tokens[s] = n;
        a.loss[s] = n == 0 ? 0.0f : static_cast<float>(dot * E / (static_cast<double>(a.k) * n * n));
    }
}

// Gradient: one warp per token, consecutive tokens per warp.  The next kernel's
// blocks come when this one's leave: they would take issue slots for nothing
// (4096 x 384: 5.5 us, about 6.4 with an early trigger).
template <int P, bool V4, bool SIG>
__global__ void __launch_bounds__(kThreads, backward_blocks(P)) balance_backward_kernel(const BalanceArgs a, int per_warp)
{
    extern __shared__ __align__(16) float sm[];   // [kWarps][E]: the weights' part of a row; [kWarps][E] bytes: slots
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E;
    float *extra = sm + warp * E;
    uint8_t *slot_of = reinterpret_cast<uint8_t *>(sm + kWarps * E) + warp * E;
    for (int e = lane; e < E; e += 32)
        extra[e] = 0.0f;
    const int64_t tw = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * per_warp;
    if (tw >= a.T)
        return;
    const int t_end = static_cast<int>(min(tw + per_warp, a.T));
    // The sequence's counts (times its coefficient) stay in registers for rows of up to 384 columns;
    // longer rows read them again for every token (from L1), which leaves
    // registers for twice the warps.
    constexpr bool kHold = P <= 3;
    int s = -1, s_end = 0;
    float cnt[kHold ? 4 * P : 1] = {}, coef = 0.0f;
    // the last sequence that starts at or before t (and is not empty there), its coefficient; false: t is outside
    // every sequence, or the sequence has no tokens
    auto enter = [&](int t) {
        s = last_sequence(a.S, lane, [&](int i) { return seq_start(a, i) <= t; });
        s_end = seq_start(a, s + 1);
        const int n = __ldg(a.tokens + s);
        const bool in = t >= seq_start(a, s) && t < s_end && n > 0;
        coef = in ? static_cast<float>(static_cast<double>(__ldg(a.grad_loss + s)) * E /
                                       (static_cast<double>(a.k) * n * n))
                  : 0.0f;
        return in;
    };
    bool low = false;                              // a row's scores or its selected ones are left for later
    auto count = [&](int q) -> float {
        if (kHold)
            return cnt[kHold ? q : 0];
        const int c = Row<P, V4>::col(lane, q);
        return c < E ? coef * static_cast<float>(__ldg(a.counts + static_cast<int64_t>(s) * E + c)) : 0.0f;
    };
    constexpr int D = tokens_held(P);
    Row<P, V4> ring[D];
    int ids[D];
    float grads[D];                                // slot lane's weight gradient
    int64_t at = tw * E, id_at = tw * a.ld_ids + lane;         // the current token's row and its slot lane
    auto fetch = [&](int u, int ahead, int t) {
        if (t < t_end) {
            ids[u] = lane < a.k ? __ldg(a.ids + id_at + ahead * a.ld_ids) : -1;
            grads[u] = a.grad_weights != nullptr && lane < a.k
                           ? __ldg(a.grad_weights + static_cast<int64_t>(t) * a.k + lane)
                           : 0.0f;
            ring[u].load(a.logits + at + ahead * E, E, lane);
        }
    };
#pragma unroll
    for (int u = 0; u < D; ++u)
        fetch(u, u, static_cast<int>(tw) + u);
    for (int tb = static_cast<int>(tw); tb < t_end; tb += D)
#pragma unroll
    for (int u = 0; u < D; ++u) {
        const int t = tb + u;
        if (t >= t_end)
            break;
        if (s < 0 || t >= s_end) {
            const bool in = enter(t);
            if (kHold)
#pragma unroll
                for (int q = 0; q < 4 * P; ++q) {
                    const int c = Row<P, V4>::col(lane, q);
                    cnt[kHold ? q : 0] =
                        in && c < E ? coef * static_cast<float>(__ldg(a.counts + static_cast<int64_t>(s) * E + c)) : 0.0f;
                }
            if (!in)
                s = -1;                            // outside every sequence: looked up again for the next token
        }
        Row<P, V4> &r = ring[u];
        const int id = ids[u];
        const float g = grads[u];
        const bool on = s >= 0 && id >= 0 && id < E;
        // (from L1: the row has just been read)
        const float l = on && a.grad_weights != nullptr ? __ldg(a.logits + at + id) : 0.0f;
        if (on && a.grad_weights != nullptr)
            slot_of[id] = static_cast<uint8_t>(lane);      // of slots of one expert, one stays
        if (__any_sync(kAll, on)) {
            // the row's scores, and the selected slots' for the weights' part
            float sums[4];
            sums[1] = 0.0f;
            if (SIG) {
                sums[0] = r.sigmoids([&](int q, float sc) { sums[1] = fmaf(sc, count(q), sums[1]); });
            } else {
                sums[0] = r.template scores<false>();
#pragma unroll
                for (int q = 0; q < 4 * P; ++q)
                    sums[1] = fmaf(r.v[q], count(q), sums[1]);
            }
            float v = 0.0f, slope = 1.0f;
            if (a.grad_weights != nullptr) {
                if (!SIG) {
                    const float m = warp_max(on ? l : -INFINITY);
                    v = on && m != -INFINITY ? exp_fast(l - m) : 0.0f;
                } else {
                    sigmoid_pair(l, v, slope);
                    v = on ? v : 0.0f;
                }
            }
            sums[2] = v;
            sums[3] = on ? g * v : 0.0f;
            warp_sum4(sums);
            // p (c - sum p c) coef with p = score * inv and the counts scaled by coef: score (inv c' - inv dot)
            const float inv = inverse_sum<SIG>(sums[0]);
            const float dot = -sums[1] * inv * inv;
            low |= SIG && (sums[0] < kTiny || (a.grad_weights != nullptr && sums[2] < kTiny));
#pragma unroll
            for (int q = 0; q < 4 * P; ++q) {
                const float sc = r.v[q];
                r.v[q] = sc * fmaf(inv, count(q), dot);
                if (SIG)
                    r.v[q] *= 1.0f - sc;           // (sc is 1/2 at most here: nothing cancels)
            }
            if (a.grad_weights != nullptr) {
                // w (g - sum g w) with w = v / sum v
                const float q = inverse_sum<SIG>(sums[2]);
                const float d = v * q * (g - sums[3] * q) * slope;
                // into the row by way of shared memory; slots of one expert add up in slot order
                // (found by the slots' numbers: comparing them by shuffles took 40 instructions more, 48.5 us
                // instead of 46.3 at 65536 x 384)
                __syncwarp();
                if (!__any_sync(kAll, on && slot_of[id] != lane)) {
                    if (on)
                        extra[id] = d;
                } else {
                    for (int j = 0; j < a.k; ++j) {
                        if (lane == j && on)
                            extra[id] += d;
                        __syncwarp();
                    }
                }
                __syncwarp();
                if (V4) {
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const int c = 4 * (lane + 32 * i);
                        const float4 f =
                            c < E ? *reinterpret_cast<const float4 *>(extra + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        r.v[4 * i] += f.x, r.v[4 * i + 1] += f.y, r.v[4 * i + 2] += f.z, r.v[4 * i + 3] += f.w;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 4 * P; ++q) {
                        const int c = Row<P, V4>::col(lane, q);
                        if (c < E)
                            r.v[q] += extra[c];
                    }
                }
                __syncwarp();
                if (on)
                    extra[id] = 0.0f;
                __syncwarp();
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4 * P; ++q)
                r.v[q] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < (V4 ? P : 4 * P); ++i) {
            const int c = Row<P, V4>::col(lane, V4 ? 4 * i : i);
            if (c < E) {
                if (V4)
                    *reinterpret_cast<float4 *>(a.grad_logits + at + c) =
                        make_float4(r.v[4 * i], r.v[4 * i + 1], r.v[4 * i + 2], r.v[4 * i + 3]);
                else
                    a.grad_logits[at + c] = r.v[i];
            }
        }
        fetch(u, D, t + D);
        at += E;
        id_at += a.ld_ids;
    }
    if (SIG && low) {
#pragma unroll 1
        for (int t = static_cast<int>(tw); t < t_end; ++t) {
            const int id = lane < a.k ? __ldg(a.ids + static_cast<int64_t>(t) * a.ld_ids + lane) : -1;
            const bool on = id >= 0 && id < E;
            if (!__any_sync(kAll, on) || !enter(t))
                continue;
            const float *row = a.logits + static_cast<int64_t>(t) * E;
            float *out = a.grad_logits + static_cast<int64_t>(t) * E;
            const float l = on ? __ldg(row + id) : -INFINITY;
            Row<P, V4> r;
            r.load(row, E, lane);
            float sums[4] = {r.sigmoids([](int, float) {}), 0.0f, 0.0f, 0.0f}, slope;
            sigmoid_pair(l, sums[2], slope);
            warp_sum4(sums);
            __syncwarp();                          // (the row as it was stored above)
            if (sums[0] < kTiny)
                add_low_row(row, E, lane, a.counts + static_cast<int64_t>(s) * E, coef, out);
            const float m = warp_max(l < kMasked ? -INFINITY : l);
            if (a.grad_weights == nullptr || !(sums[2] < kTiny) || m == -INFINITY)
                continue;
            const float g = on ? __ldg(a.grad_weights + static_cast<int64_t>(t) * a.k + lane) : 0.0f;
            const float v = low_score(l, m), q = inverse(warp_sum(v)), dot = warp_sum(g * v) * q;
            for (int j = 0; j < a.k; ++j) {        // in slot order
                __syncwarp();
                if (lane == j && on)
                    out[id] += v * q * (g - dot);
            }
        }
    }
}

// Tokens per chunk: about as many chunks as blocks fit on the 148 SMs of the
// device (more, shorter ones pay each block's start and end; fewer leave SMs
// idle), but a token per warp at least, and two where one would leave more
// chunks of a sequence than its second kernel reads at once (4096 x 384: one
// sequence 6.7 us with two and 8.2 with one, seven sequences 8.3 and 7.6).
int balance_chunk(int64_t T, int64_t S, int E)
{
    const int P = (E + 127) / 128;
    const int64_t fit = 148 * chunk_blocks(P), warps = chunk_warps(P, false);
    const int64_t blocks = S < fit / 2 ? fit - S : fit / 2;    // (every sequence may add a chunk)
    const int64_t c = (T + blocks - 1) / blocks, least = T > 128 * warps * S ? 2 * warps : warps;
    return static_cast<int>(c < least ? least : c);
}

int64_t balance_slots(int64_t T, int64_t S, int E)
{
    return T / balance_chunk(T, S, E) + S;
}

// At least as many as any batch of up to T tokens in up to S sequences takes,
// for any E (12 tokens per chunk at least, at most 2 blocks per SM): what the
// workspace holds.  It does not shrink as T or S grow, which the slots of one
// batch do where its chunks get longer.
int64_t balance_slots_most(int64_t T, int64_t S)
{
    constexpr int64_t fit = 148 * 2;
    const int64_t blocks = S < fit / 2 ? fit - S : fit / 2;
    return (T / 12 < blocks ? T / 12 : blocks) + S;
}

// 16-byte loads and stores need every row to start on a 16-byte boundary.
static bool aligned_rows(const BalanceArgs &a)
{
    return ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.grad_logits)) & 15) == 0;
}

// F(P, V4, SIG) of the smallest P that holds a row.
#define NVFP4_BALANCE_ROWS(F, V, S)                                                                              \
    (p4 <= 1 ? F(1, V, S) : p4 <= 2 ? F(2, V, S) : p4 <= 3 ? F(3, V, S) : p4 <= 4 ? F(4, V, S) : F(8, V, S))
#define NVFP4_BALANCE_CASES(F)                                                                                   \
    const int p4 = (a.E + 127) / 128;                                                                            \
    const bool v4 = a.E % 4 == 0 && aligned_rows(a);                                                             \
    if (a.scoring == NVFP4_SCORING_SOFTMAX)                                                                      \
        return v4 ? NVFP4_BALANCE_ROWS(F, true, false) : NVFP4_BALANCE_ROWS(F, false, false);                    \
    return v4 ? NVFP4_BALANCE_ROWS(F, true, true) : NVFP4_BALANCE_ROWS(F, false, true);

namespace {

template <int P, bool V4, bool SIG, bool WHOLE>
cudaError_t chunk_launch(const BalanceArgs &a, cudaStream_t s)
{
    const int64_t blocks = WHOLE ? a.S : balance_slots(a.T, a.S, a.E);
    static unsigned long long attr_done = 0;
    constexpr int W = chunk_warps(P, WHOLE);
    const auto kernel = balance_chunk_kernel<P, V4, SIG, WHOLE>;
    const cudaError_t e =
        ensure_smem_limit(reinterpret_cast<const void *>(kernel), sizeof(float) * (W + 1) * 128 * P, &attr_done);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(32 * W), sizeof(float) * (W + 1) * a.E, s, a);
}

template <int P, bool V4, bool SIG>
cudaError_t backward_launch(const BalanceArgs &a, cudaStream_t s)
{
    // consecutive tokens per warp, one wave of blocks
    const int64_t warps = 148LL * kWarps * backward_blocks(P);
    const int64_t per = (a.T + warps - 1) / warps;
    const int64_t grid = (a.T + kWarps * per - 1) / (kWarps * per);
    return launch_pdl(balance_backward_kernel<P, V4, SIG>, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                      (sizeof(float) + 1) * kWarps * a.E, s, a, static_cast<int>(per));
}

cudaError_t launch_chunks(const BalanceArgs &a, cudaStream_t s)
{
#define F(P, V, S) chunk_launch<P, V, S, false>(a, s)
    NVFP4_BALANCE_CASES(F)
#undef F
}

cudaError_t launch_whole(const BalanceArgs &a, cudaStream_t s)
{
#define F(P, V, S) chunk_launch<P, V, S, true>(a, s)
    NVFP4_BALANCE_CASES(F)
#undef F
}

} // namespace

cudaError_t launch_balance(const BalanceArgs &a, cudaStream_t s)
{
    // One launch for short batches, a block per sequence.  With all tokens in one
    // sequence it takes as long as two launches at 190 tokens of 48 or 128
    // experts, 160 of 256, 150 of 384, 128 of 512 and 95 of 1024 (6 to 8 us;
    // 64 x 48: 3.3 us instead of 5.8; 512 x 512: 19.2 instead of 6.9).
    if (a.T * (a.E + 700) <= 128 * (512 + 700))
        return launch_whole(a, s);
    const cudaError_t e = launch_chunks(a, s);
    if (e != cudaSuccess)
        return e;
    // up to 8 blocks per sequence, 32 experts each at least
    const int blocks = a.E <= 32 ? 1 : a.E <= 64 ? 2 : a.E <= 128 ? 4 : 8;
    const int cols = padded((a.E + blocks - 1) / blocks);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(a.S));
    cfg.blockDim = dim3(kSumThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, balance_sum_kernel, a, cols);
}

cudaError_t launch_balance_backward(const BalanceArgs &a, cudaStream_t s)
{
#define F(P, V, S) backward_launch<P, V, S>(a, s)
    NVFP4_BALANCE_CASES(F)
#undef F
}

} // namespace nvfp4
