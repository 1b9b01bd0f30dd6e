// api_layer.cu -- the C ABI of the operators around the routed block
// (declared in include/nvfp4moe.h): argument checks and launches of the norm,
// the few-row products and the router's balance loss.  No allocation, no host
// synchronisation, everything on the caller's stream.
#include "internal.h"

using namespace nvfp4;

namespace {

bool aligned(const void *p, uintptr_t bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

int status_of(cudaError_t e)
{
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

// Workspace of nvfp4_moe_balance: per chunk slot E probability sums and E
// counts (padded to 4) and the token count; as many slots as any batch that is
// no larger takes.
struct BalanceLayout {
    int64_t part_c, part_n, total;
};

BalanceLayout balance_layout(int64_t T, int64_t S, int64_t E)
{
    BalanceLayout L;
    const int64_t slots = balance_slots_most(T, S), row = (E + 3) / 4 * 16;
    L.part_c = slots * row;
    L.part_n = 2 * L.part_c;
    L.total = L.part_n + 4 * slots;
    return L;
}

int check_balance(int64_t T, int64_t S, int E, int k, int64_t ld_ids, int scoring)
{
    if (T < 0 || S < 1 || E < 1 || k < 1 || ld_ids < k)
        return NVFP4_ERR_INVALID_ARG;
    if (scoring != NVFP4_SCORING_SOFTMAX && scoring != NVFP4_SCORING_SIGMOID)
        return NVFP4_ERR_INVALID_ARG;
    if (E > 1024 || k > 32 || k > E || T >= (1LL << 31) - 1024 || S > 65535)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    return NVFP4_OK;
}

int gemv(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *b_codes, const uint8_t *b_scales, const float *b_gs,
         const int64_t *seg_end, int nseg, int64_t N, int64_t K, uint16_t *out, int64_t ldo, int withhold, void *stream)
{
    if (M < 0 || N < 1 || K < 1 || nseg < 1 || seg_end == nullptr)
        return NVFP4_ERR_INVALID_ARG;
    if (b_codes == nullptr || b_scales == nullptr || b_gs == nullptr)
        return NVFP4_ERR_INVALID_ARG;
    if (M > 0 && (x == nullptr || out == nullptr || ldx < K || ldo < N))
        return NVFP4_ERR_INVALID_ARG;
    if (M > kGemvMaxRows || K % 64 != 0 || K > (1LL << 20) || N > (1LL << 30) || nseg > 4 ||
        (N + 127) / 128 * (K / 64) >= (1LL << 31))
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    int64_t prev = 0;
    for (int i = 0; i < nseg; ++i) {
        if (seg_end[i] <= prev)
            return NVFP4_ERR_INVALID_ARG;
        prev = seg_end[i];
    }
    if (prev != N)
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned(b_codes, 16) || !aligned(b_scales, 16) || !aligned(b_gs, 4))
        return NVFP4_ERR_MISALIGNED;
    if (M > 0 && (!aligned(x, 16) || !aligned(out, 2) || ldx % 8 != 0))
        return NVFP4_ERR_MISALIGNED;
    int sms = 0;
    const int st = device_status(&sms);
    if (st != NVFP4_OK)
        return st;
    if (M == 0)
        return NVFP4_OK;
    GemvArgs g{};
    g.x = reinterpret_cast<const __nv_bfloat16 *>(x);
    g.M = M;
    g.ldx = ldx;
    g.codes = b_codes;
    g.scales = b_scales;
    g.gs = b_gs;
    g.nseg = nseg;
    for (int i = 0; i < nseg; ++i)
        g.seg_end[i] = seg_end[i];
    g.N = N;
    g.K = K;
    g.out = reinterpret_cast<__nv_bfloat16 *>(out);
    g.ldo = ldo;
    g.withhold = withhold;
    return status_of(launch_gemv(g, sms, static_cast<cudaStream_t>(stream)));
}

} // namespace

extern "C" {

int nvfp4_add_rmsnorm(const nvfp4_norm_args *a, void *stream)
{
    if (a == nullptr || a->T < 0 || a->H < 1 || a->eps < 0.0 || a->eps != a->eps)
        return NVFP4_ERR_INVALID_ARG;
    if (a->quant != NVFP4_QUANT_NONE && a->quant != NVFP4_QUANT_NVFP4 && a->quant != NVFP4_QUANT_E4M3)
        return NVFP4_ERR_INVALID_ARG;
    const bool q4 = a->quant == NVFP4_QUANT_NVFP4, q = a->quant != NVFP4_QUANT_NONE;
    if (q4 && a->scale_layout != NVFP4_SCALES_ROWMAJOR && a->scale_layout != NVFP4_SCALES_MMA)
        return NVFP4_ERR_INVALID_ARG;
    if (a->T > 0) {
        if (a->x == nullptr || a->weight == nullptr || (a->y == nullptr && !q) ||
            (a->residual == nullptr) != (a->residual_out == nullptr) ||
            (q && (a->codes == nullptr || a->scales == nullptr)) || (q4 && a->gs == nullptr))
            return NVFP4_ERR_INVALID_ARG;
        if (a->ldx < a->H || (a->residual != nullptr && (a->ldr < a->H || a->ldro < a->H)) ||
            (a->y != nullptr && a->ldy < a->H))
            return NVFP4_ERR_INVALID_ARG;
    }
    if (a->H % 16 != 0 || a->H > kNormMaxCols || a->T >= (1LL << 31) ||
        (q4 && a->scale_layout == NVFP4_SCALES_MMA && a->H % 64 != 0))
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (a->T > 0) {
        const void *p16[] = {a->x, a->residual, a->residual_out, a->weight, a->y, q ? a->codes : nullptr};
        for (const void *p : p16)
            if (!aligned(p, 16))
                return NVFP4_ERR_MISALIGNED;
        if (q && !aligned(a->scales, 4))
            return NVFP4_ERR_MISALIGNED;
        if (a->ldx % 8 != 0 || (a->residual != nullptr && (a->ldr % 8 != 0 || a->ldro % 8 != 0)) ||
            (a->y != nullptr && a->ldy % 8 != 0))
            return NVFP4_ERR_MISALIGNED;
    }
    int sms = 0;
    const int st = device_status(&sms);
    if (st != NVFP4_OK)
        return st;
    if (a->T == 0)
        return NVFP4_OK;
    NormArgs n{};
    n.x = reinterpret_cast<const __nv_bfloat16 *>(a->x);
    n.residual = reinterpret_cast<const __nv_bfloat16 *>(a->residual);
    n.weight = reinterpret_cast<const __nv_bfloat16 *>(a->weight);
    n.residual_out = reinterpret_cast<__nv_bfloat16 *>(a->residual_out);
    n.y = reinterpret_cast<__nv_bfloat16 *>(a->y);
    n.ldx = a->ldx;
    n.ldr = a->ldr;
    n.ldro = a->ldro;
    n.ldy = a->ldy;
    n.T = a->T;
    n.nb = static_cast<int>(a->H / 16);
    n.inv_cols = 1.0 / static_cast<double>(a->H);
    n.eps = a->eps;
    n.quant = a->quant;
    n.layout = a->scale_layout;
    n.gs = a->gs;
    n.codes = a->codes;
    n.scales = a->scales;
    return status_of(launch_add_rmsnorm(n, sms, static_cast<cudaStream_t>(stream)));
}

int nvfp4_gemv(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *b_codes, const uint8_t *b_scales,
               const float *b_gs, const int64_t *seg_end, int nseg, int64_t N, int64_t K, uint16_t *out, int64_t ldo,
               void *stream)
{
    return gemv(x, M, ldx, b_codes, b_scales, b_gs, seg_end, nseg, N, K, out, ldo, 0, stream);
}

int nvfp4_debug_gemv_timeout(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *b_codes, const uint8_t *b_scales,
                             const float *b_gs, const int64_t *seg_end, int nseg, int64_t N, int64_t K, uint16_t *out,
                             int64_t ldo, void *stream)
{
    return gemv(x, M, ldx, b_codes, b_scales, b_gs, seg_end, nseg, N, K, out, ldo, 1, stream);
}

size_t nvfp4_moe_balance_workspace_size(int64_t T, int64_t S, int E)
{
    if (check_balance(T, S, E, 1, 1, NVFP4_SCORING_SOFTMAX) != NVFP4_OK)
        return 0;
    return static_cast<size_t>(balance_layout(T, S, E).total);
}

int nvfp4_moe_balance(const float *logits, const int32_t *topk_ids, int64_t ld_ids, int64_t T, int E, int k,
                      const int32_t *seq_offsets, int64_t S, int scoring, int32_t *counts, int32_t *tokens,
                      float *probs, float *loss, void *workspace, size_t ws_bytes, void *stream)
{
    int st = check_balance(T, S, E, k, ld_ids, scoring);
    if (st != NVFP4_OK)
        return st;
    if (T > 0 && (logits == nullptr || topk_ids == nullptr))
        return NVFP4_ERR_INVALID_ARG;
    if (counts == nullptr || tokens == nullptr || probs == nullptr || loss == nullptr || workspace == nullptr ||
        (seq_offsets == nullptr && S != 1))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned(workspace, 16))
        return NVFP4_ERR_MISALIGNED;
    const BalanceLayout L = balance_layout(T, S, E);
    if (ws_bytes < static_cast<size_t>(L.total))
        return NVFP4_ERR_WORKSPACE_TOO_SMALL;
    st = device_status(nullptr);
    if (st != NVFP4_OK)
        return st;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    BalanceArgs a{};
    a.logits = logits;
    a.ids = topk_ids;
    a.ld_ids = ld_ids;
    a.k = k;
    a.T = T;
    a.E = E;
    a.S = static_cast<int>(S);
    a.offsets = seq_offsets;
    a.scoring = scoring;
    a.chunk = balance_chunk(T, S, E);
    a.counts = counts;
    a.tokens = tokens;
    a.probs = probs;
    a.loss = loss;
    a.part_p = reinterpret_cast<float *>(ws);
    a.part_c = reinterpret_cast<int32_t *>(ws + L.part_c);
    a.part_n = reinterpret_cast<int32_t *>(ws + L.part_n);
    return status_of(launch_balance(a, static_cast<cudaStream_t>(stream)));
}

int nvfp4_moe_balance_backward(const float *logits, const int32_t *topk_ids, int64_t ld_ids, int64_t T, int E, int k,
                               const int32_t *seq_offsets, int64_t S, int scoring, const int32_t *counts,
                               const int32_t *tokens, const float *grad_loss, const float *grad_weights,
                               float *grad_logits, void *stream)
{
    int st = check_balance(T, S, E, k, ld_ids, scoring);
    if (st != NVFP4_OK)
        return st;
    if (T > 0 && (logits == nullptr || topk_ids == nullptr || grad_logits == nullptr))
        return NVFP4_ERR_INVALID_ARG;
    if (counts == nullptr || tokens == nullptr || grad_loss == nullptr || (seq_offsets == nullptr && S != 1))
        return NVFP4_ERR_INVALID_ARG;
    st = device_status(nullptr);
    if (st != NVFP4_OK)
        return st;
    if (T == 0)
        return NVFP4_OK;
    BalanceArgs a{};
    a.logits = logits;
    a.ids = topk_ids;
    a.ld_ids = ld_ids;
    a.k = k;
    a.T = T;
    a.E = E;
    a.S = static_cast<int>(S);
    a.offsets = seq_offsets;
    a.scoring = scoring;
    a.counts = const_cast<int32_t *>(counts);
    a.tokens = const_cast<int32_t *>(tokens);
    a.grad_loss = grad_loss;
    a.grad_weights = grad_weights;
    a.grad_logits = grad_logits;
    return status_of(launch_balance_backward(a, static_cast<cudaStream_t>(stream)));
}

} // extern "C"
