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
#include "internal.h"
#include "quant.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
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
                const float4 f = c < E ? __ldg(reinterpret_cast<const float4 *>(row + c))
                                       : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4 * P; ++q)
                v[q] = col(lane, q) < E ? __ldg(row + col(lane, q)) : -INFINITY;
        }
    }
    // scores (exp(l - max) or sigmoid(l)) in place; returns 1 / their sum, or 0
    // where the sum is 0 (a row of -inf: no probability anywhere)
    __device__ __forceinline__ float scores(int scoring)
    {
        float sum = 0.0f;
        if (scoring == NVFP4_SCORING_SOFTMAX) {
            float m = v[0];
#pragma unroll
            for (int q = 1; q < 4 * P; ++q)
                m = fmaxf(m, v[q]);
            m = warp_max(m);
            if (m == -INFINITY)
                m = 0.0f;
#pragma unroll
            for (int q = 0; q < 4 * P; ++q) {
                v[q] = expf(v[q] - m);
                sum += v[q];
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4 * P; ++q) {
                v[q] = __frcp_rn(1.0f + expf(-v[q]));
                sum += v[q];
            }
        }
        sum = warp_sum(sum);
        return sum == 0.0f ? 0.0f : __frcp_rn(sum);
    }
};

} // namespace

// Sums of one chunk slot: counts, tokens and probabilities.
template <int P, bool V4>
__global__ void __launch_bounds__(kThreads) balance_chunk_kernel(const BalanceArgs a)
{
    extern __shared__ float sm[];                 // [kWarps][E] probability sums, then [E] int counts
    __shared__ int tokens_s;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E, slot = blockIdx.x;
    // the last sequence whose first slot is <= slot
    int lo = 0, hi = a.S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_slot(a, mid) <= slot)
            lo = mid;
        else
            hi = mid;
    }
    int t0, t1;
    slot_tokens(a, lo, slot, t0, t1);
    if (t0 >= t1)
        return;
    int *hist = reinterpret_cast<int *>(sm + kWarps * E);
    for (int e = threadIdx.x; e < E; e += kThreads)
        hist[e] = 0;
    if (threadIdx.x == 0)
        tokens_s = 0;
    __syncthreads();
    float acc[4 * P];
#pragma unroll
    for (int q = 0; q < 4 * P; ++q)
        acc[q] = 0.0f;
    int tokens = 0;
    for (int t = t0 + warp; t < t1; t += kWarps) {
        const int id = lane < a.k ? __ldg(a.ids + static_cast<int64_t>(t) * a.ld_ids + lane) : -1;
        const bool on = id >= 0 && id < E;
        if (!__any_sync(kAll, on))
            continue;                              // a padded token
        ++tokens;
        if (on)
            atomicAdd(hist + id, 1);
        Row<P, V4> r;
        r.load(a.logits + static_cast<int64_t>(t) * E, E, lane);
        const float inv = r.scores(a.scoring);
#pragma unroll
        for (int q = 0; q < 4 * P; ++q)
            acc[q] = fmaf(r.v[q], inv, acc[q]);
    }
    if (lane == 0 && tokens)
        atomicAdd(&tokens_s, tokens);
#pragma unroll
    for (int q = 0; q < 4 * P; ++q) {
        const int c = Row<P, V4>::col(lane, q);
        if (c < E)
            sm[warp * E + c] = acc[q];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
        float p = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            p += sm[w * E + e];
        a.part_p[static_cast<int64_t>(slot) * E + e] = p;
        a.part_c[static_cast<int64_t>(slot) * E + e] = hist[e];
    }
    if (threadIdx.x == 0)
        a.part_n[slot] = tokens_s;
}

// One block per sequence: its chunks' sums in slot order, and the loss.
__global__ void __launch_bounds__(kThreads) balance_sum_kernel(const BalanceArgs a)
{
    __shared__ double red[kWarps];
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.x, E = a.E;
    const int o0 = seq_start(a, s), o1 = seq_start(a, s + 1);
    const int slot0 = first_slot(a, s);
    const int nslots = o1 > o0 ? (o1 - 1) / a.chunk - o0 / a.chunk + 1 : 0;    // non-empty ones
    int n = 0;
    for (int i = 0; i < nslots; ++i)
        n += a.part_n[slot0 + i];
    double dot = 0.0;
    for (int e = threadIdx.x; e < E; e += kThreads) {
        double p = 0.0;
        int c = 0;
        for (int i = 0; i < nslots; ++i) {
            p += a.part_p[static_cast<int64_t>(slot0 + i) * E + e];
            c += a.part_c[static_cast<int64_t>(slot0 + i) * E + e];
        }
        a.counts[static_cast<int64_t>(s) * E + e] = c;
        a.probs[static_cast<int64_t>(s) * E + e] = static_cast<float>(p);
        dot += c * p;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        dot += __shfl_xor_sync(kAll, dot, o);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        dot = 0.0;
        for (int w = 0; w < kWarps; ++w)
            dot += red[w];
        a.tokens[s] = n;
        a.loss[s] = n == 0 ? 0.0f : static_cast<float>(dot * E / (static_cast<double>(a.k) * n * n));
    }
}

// Gradient: one warp per token, consecutive tokens per warp.
template <int P, bool V4>
__global__ void __launch_bounds__(kThreads) balance_backward_kernel(const BalanceArgs a, int per_warp)
{
    extern __shared__ float sm[];                 // [kWarps][E]: the weights' part of a row
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E;
    float *extra = sm + warp * E;
    for (int e = lane; e < E; e += 32)
        extra[e] = 0.0f;
    const int64_t tw = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * per_warp;
    if (tw >= a.T)
        return;
    const int t_end = static_cast<int>(min(tw + per_warp, a.T));
    int s = -1, s_end = 0;
    float cnt[4 * P], coef = 0.0f;
    for (int t = static_cast<int>(tw); t < t_end; ++t) {
        if (s < 0 || t >= s_end) {
            // the last sequence that starts at or before t (and is not empty there)
            int lo = 0, hi = a.S;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (seq_start(a, mid) <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            s = lo;
            s_end = seq_start(a, s + 1);
            const int n = __ldg(a.tokens + s);
            const bool in = t >= seq_start(a, s) && t < s_end && n > 0;
            coef = in ? static_cast<float>(static_cast<double>(__ldg(a.grad_loss + s)) * E /
                                           (static_cast<double>(a.k) * n * n))
                      : 0.0f;
#pragma unroll
            for (int q = 0; q < 4 * P; ++q) {
                const int c = Row<P, V4>::col(lane, q);
                cnt[q] = in && c < E ? static_cast<float>(__ldg(a.counts + static_cast<int64_t>(s) * E + c)) : 0.0f;
            }
            if (!in)
                s = -1;                            // outside every sequence: looked up again for the next token
        }
        float *out = a.grad_logits + static_cast<int64_t>(t) * E;
        const int id = lane < a.k && s >= 0 ? __ldg(a.ids + static_cast<int64_t>(t) * a.ld_ids + lane) : -1;
        const bool on = id >= 0 && id < E;
        Row<P, V4> r;
        if (__any_sync(kAll, on)) {
            const float *row = a.logits + static_cast<int64_t>(t) * E;
            r.load(row, E, lane);
            const float inv = r.scores(a.scoring);
            float dot = 0.0f;
#pragma unroll
            for (int q = 0; q < 4 * P; ++q)
                dot = fmaf(r.v[q], cnt[q], dot);
            dot = warp_sum(dot) * inv;
            const float ci = coef * inv;
#pragma unroll
            for (int q = 0; q < 4 * P; ++q) {
                const float sc = r.v[q];
                r.v[q] = ci * sc * (cnt[q] - dot);
                if (a.scoring != NVFP4_SCORING_SOFTMAX)
                    r.v[q] *= 1.0f - sc;
            }
            if (a.grad_weights != nullptr) {
                const float l = on ? __ldg(row + id) : -INFINITY;
                float v, slope = 1.0f;
                if (a.scoring == NVFP4_SCORING_SOFTMAX) {
                    const float m = warp_max(l);
                    v = on && m != -INFINITY ? expf(l - m) : 0.0f;
                } else {
                    v = on ? __frcp_rn(1.0f + expf(-l)) : 0.0f;
                    slope = 1.0f - v;
                }
                const float sum = warp_sum(v);
                const float w = sum == 0.0f ? 0.0f : __fdiv_rn(v, sum);
                const float g = on ? __ldg(a.grad_weights + static_cast<int64_t>(t) * a.k + lane) : 0.0f;
                const float d = w * (g - warp_sum(g * w)) * slope;
                // slots of one expert add up in slot order
                for (int j = 0; j < a.k; ++j) {
                    if (lane == j && on)
                        extra[id] += d;
                    __syncwarp();
                }
#pragma unroll
                for (int q = 0; q < 4 * P; ++q) {
                    const int c = Row<P, V4>::col(lane, q);
                    if (c < E)
                        r.v[q] += extra[c];
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
                    *reinterpret_cast<float4 *>(out + c) =
                        make_float4(r.v[4 * i], r.v[4 * i + 1], r.v[4 * i + 2], r.v[4 * i + 3]);
                else
                    out[c] = r.v[i];
            }
        }
    }
}

int balance_chunk(int64_t T)
{
    const int64_t c = (T + 511) / 512;
    return static_cast<int>(c < 8 ? 8 : c);
}

int64_t balance_slots(int64_t T, int64_t S)
{
    return T / balance_chunk(T) + S;
}

// 16-byte loads and stores need every row to start on a 16-byte boundary.
static bool aligned_rows(const BalanceArgs &a)
{
    return ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.grad_logits)) & 15) == 0;
}

#define NVFP4_BALANCE_CASES(F)                                                                                   \
    const int p4 = (a.E + 127) / 128;                                                                            \
    const bool v4 = a.E % 4 == 0 && aligned_rows(a);                                                             \
    if (v4)                                                                                                      \
        return p4 <= 1 ? F(1, true) : p4 <= 2 ? F(2, true) : p4 <= 3 ? F(3, true) : p4 <= 4 ? F(4, true)         \
               : F(8, true);                                                                                     \
    return p4 <= 1 ? F(1, false) : p4 <= 3 ? F(3, false) : F(8, false);

namespace {

template <int P, bool V4>
cudaError_t chunk_launch(const BalanceArgs &a, cudaStream_t s)
{
    return launch_pdl(balance_chunk_kernel<P, V4>, dim3(static_cast<unsigned>(balance_slots(a.T, a.S))),
                      dim3(kThreads), sizeof(float) * (kWarps + 1) * a.E, s, a);
}

template <int P, bool V4>
cudaError_t backward_launch(const BalanceArgs &a, cudaStream_t s)
{
    int64_t per = (a.T + 148 * 32 - 1) / (148 * 32);
    if (per < 1)
        per = 1;
    const int64_t grid = (a.T + kWarps * per - 1) / (kWarps * per);
    return launch_pdl(balance_backward_kernel<P, V4>, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                      sizeof(float) * kWarps * a.E, s, a, static_cast<int>(per));
}

cudaError_t launch_chunks(const BalanceArgs &a, cudaStream_t s)
{
#define F(P, V) chunk_launch<P, V>(a, s)
    NVFP4_BALANCE_CASES(F)
#undef F
}

} // namespace

cudaError_t launch_balance(const BalanceArgs &a, cudaStream_t s)
{
    cudaError_t e = a.T > 0 ? launch_chunks(a, s) : cudaSuccess;
    if (e == cudaSuccess)
        e = launch_pdl(balance_sum_kernel, dim3(static_cast<unsigned>(a.S)), dim3(kThreads), 0, s, a);
    return e;
}

cudaError_t launch_balance_backward(const BalanceArgs &a, cudaStream_t s)
{
#define F(P, V) backward_launch<P, V>(a, s)
    NVFP4_BALANCE_CASES(F)
#undef F
}

} // namespace nvfp4
