// rmsq_rope.cu -- C ABI of the per-head norm with rotation and of its gradient: argument checks, the choice of
// vectors and the launches (declared in include/rmsq.h).
#include <cmath>
#include <cstdint>

#include "rmsq_ops.h"
#include "rmsq_rope.cuh"

namespace rmsq {

static bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

// Whether [tokens][heads][dim] elements with these strides lie apart from one another.
static bool apart(long long tokens, long long heads, long long dim, long long st, long long sh)
{
    if (tokens == 1) st = 0;
    if (heads == 1) sh = 0;
    if ((tokens > 1 && st < dim) || (heads > 1 && sh < dim)) return false;
    return tokens == 1 || heads == 1 || st >= (heads - 1) * sh + dim || sh >= (tokens - 1) * st + dim;
}

// Strides past this would leave 64 bits once multiplied by a count of heads or tokens.
constexpr long long kMostStride = 1LL << 31;

static rmsq_status check_side(const rmsq_heads* s, int64_t tokens, int64_t dim, int es, bool output, int* vec)
{
    if (s == nullptr) return RMSQ_ERR_NULL;
    if (s->heads < 1 || s->heads > 65536 || s->token_stride < 0 || s->head_stride < 0 || s->token_stride >= kMostStride ||
        s->head_stride >= kMostStride)
        return RMSQ_ERR_SHAPE;
    if (tokens == 0) return RMSQ_OK;
    if (s->data == nullptr) return RMSQ_ERR_NULL;
    if (!aligned(s->data, es)) return RMSQ_ERR_ALIGN;
    if (output && !apart(tokens, s->heads, dim, s->token_stride, s->head_stride)) return RMSQ_ERR_SHAPE;
    // elements that every row starts at a multiple of, in memory
    while (*vec > 1 && (!aligned(s->data, *vec * es) || (tokens > 1 && s->token_stride % *vec != 0) ||
                        (s->heads > 1 && s->head_stride % *vec != 0)))
        *vec /= 2;
    return RMSQ_OK;
}

template <int DT, int V, bool BOTH> static const void* rope_at(bool inter, bool backward)
{
    if (inter)
        return backward ? reinterpret_cast<const void*>(&rmsq_rope_bwd_kernel<DT, V, true, BOTH>)
                        : reinterpret_cast<const void*>(&rmsq_rope_kernel<DT, V, true, BOTH>);
    return backward ? reinterpret_cast<const void*>(&rmsq_rope_bwd_kernel<DT, V, false, BOTH>)
                    : reinterpret_cast<const void*>(&rmsq_rope_kernel<DT, V, false, BOTH>);
}

template <int DT, bool BOTH> static const void* rope_fn(int vec, bool inter, bool backward)
{
    if constexpr (DT != DT_F32)
        if (vec == 8) return rope_at<DT, 8, BOTH>(inter, backward);
    if (vec == 4) return rope_at<DT, 4, BOTH>(inter, backward);
    // (narrow vectors, of odd sizes and places, are slow for other reasons)
    return vec == 2 ? rope_at<DT, 2, true>(inter, backward) : rope_at<DT, 1, true>(inter, backward);
}

struct RopeCall {
    const rmsq_heads *dq, *dk;                   // backward: gradients that come
    const rmsq_heads *q, *k;
    const void *gq, *gk;
    const rmsq_rotation* rot;
    int64_t tokens, dim;
    int dtype;
    float eps, offset;
    const rmsq_heads *oq, *ok;
};

// Checks a call and fills in everything but the launch; *vec: the elements a vector holds.
static rmsq_status prepare_rope(const RopeCall& c, RopeParams* p, int* vec)
{
    if (c.dtype != RMSQ_BF16 && c.dtype != RMSQ_FP16 && c.dtype != RMSQ_F32) return RMSQ_ERR_DTYPE;
    if (c.rot == nullptr || c.q == nullptr || c.k == nullptr || c.oq == nullptr || c.ok == nullptr) return RMSQ_ERR_NULL;
    const rmsq_rotation& r = *c.rot;
    if (r.position_bits != 32 && r.position_bits != 64) return RMSQ_ERR_DTYPE;
    if (c.tokens < 0 || c.tokens > RMSQ_ROPE_MAX_TOKENS || c.dim < 2 || c.dim > RMSQ_ROPE_MAX_DIM || c.dim % 2 != 0 ||
        r.rotated < 2 || r.rotated > c.dim || r.rotated % 2 != 0 || r.places < 1 || r.axes < 1 || r.axes > kRopeAxes)
        return RMSQ_ERR_SHAPE;
    int sum = 0;
    for (int a = 0; a < r.axes && r.axes > 1; ++a) {
        if (r.sections[a] < 0 || r.sections[a] > r.rotated / 2) return RMSQ_ERR_SHAPE;
        sum += r.sections[a];
    }
    if (r.axes > 1 && sum != r.rotated / 2) return RMSQ_ERR_SHAPE;
    if (!(c.eps >= 0.0f) || !std::isfinite(c.eps) || !std::isfinite(c.offset)) return RMSQ_ERR_VALUE;
    if (c.q->heads != c.oq->heads || c.k->heads != c.ok->heads) return RMSQ_ERR_SHAPE;
    const int es = c.dtype == RMSQ_F32 ? 4 : 2, half = r.rotated / 2;
    *vec = 16 / es;
    rmsq_status st = check_side(c.q, c.tokens, c.dim, es, false, vec);
    if (st == RMSQ_OK) st = check_side(c.k, c.tokens, c.dim, es, false, vec);
    if (st == RMSQ_OK) st = check_side(c.oq, c.tokens, c.dim, es, true, vec);
    if (st == RMSQ_OK) st = check_side(c.ok, c.tokens, c.dim, es, true, vec);
    if (st != RMSQ_OK) return st;
    if (c.tokens > 0) {
        if (!c.gq || !c.gk || !r.cos || !r.sin || !r.positions) return RMSQ_ERR_NULL;
        if (!aligned(c.gq, es) || !aligned(c.gk, es) || !aligned(r.cos, 4) || !aligned(r.sin, 4) ||
            !aligned(r.positions, r.position_bits / 8))
            return RMSQ_ERR_ALIGN;
    }
    // vectors end where the pairs' halves and the rotation do
    const auto whole = [&](int v) {
        return r.neighbours ? c.dim % v == 0 && r.rotated % v == 0 : half % v == 0 && (c.dim / 2 - half) % v == 0;
    };
    while (*vec > 1 && !whole(*vec)) *vec /= 2;
    *p = {};
    const rmsq_heads* in[2] = {c.q, c.k};
    const rmsq_heads* out[2] = {c.oq, c.ok};
    const void* gamma[2] = {c.gq, c.gk};
    for (int s = 0; s < 2; ++s) {
        RopeSide& d = p->side[s];
        d.x = in[s]->data;
        d.xt = static_cast<unsigned>(in[s]->token_stride);
        d.xh = static_cast<unsigned>(in[s]->head_stride);
        d.out = out[s]->data;
        d.ot = static_cast<unsigned>(out[s]->token_stride);
        d.oh = static_cast<unsigned>(out[s]->head_stride);
        d.gamma = gamma[s];
        d.heads = static_cast<int>(in[s]->heads);
    }
    p->cos = r.cos;
    p->sin = r.sin;
    p->positions = r.positions;
    p->tokens = static_cast<int>(c.tokens);
    p->places = r.places;
    p->dim = static_cast<int>(c.dim);
    p->half = half;
    p->wide = r.position_bits == 64;
    p->axes = r.axes;
    for (int a = 0, end = 0; a < kRopeAxes; ++a) {
        end += r.axes > 1 && a < r.axes ? r.sections[a] : 0;
        p->until[a] = a < r.axes - 1 ? end : half;
    }
    p->vec_table = half % 4 == 0 && aligned(r.cos, 16) && aligned(r.sin, 16);
    p->eps = c.eps;
    p->offset = c.offset;
    p->inv_dim = 1.0f / static_cast<float>(c.dim);
    return RMSQ_OK;
}

// Lanes per row, a token's groups, and the CTAs: `most` at most, those of the queries and of the keys by their turns, and no more
// than have a turn for every warp.
static unsigned deal_rope(RopeParams* p, int vec, bool neighbours, long long most, int warps)
{
    // a lane holds 8 pairs, in steps of a vector (neighbours: of a pair at least)
    const int step = neighbours ? (vec > 2 ? vec / 2 : 1) : vec;
    const int units = (p->dim / 2 / step + 8 / step - 1) / (8 / step);
    p->lanes = 1;
    while (p->lanes < units) p->lanes *= 2;
    const int rows = 32 / p->lanes;
    long long turns[2];
    for (int s = 0; s < 2; ++s) {
        RopeSide& d = p->side[s];
        d.groups = (d.heads + rows - 1) / rows;
        turns[s] = (static_cast<long long>(p->tokens) * d.groups + kRopeRows - 1) / kRopeRows;
    }
    const long long all = turns[0] + turns[1];
    long long need[2] = {(turns[0] + warps - 1) / warps, (turns[1] + warps - 1) / warps};
    long long q = need[0];
    if (need[0] + need[1] > most) {
        q = (most * turns[0] + all / 2) / all;
        q = q < 1 ? 1 : q > most - 1 ? most - 1 : q;
        if (q > need[0]) q = need[0];
        if (q < most - need[1]) q = most - need[1];
        need[1] = most - q;
    }
    p->split = static_cast<int>(q);
    return static_cast<unsigned>(q + need[1]);
}

template <bool BOTH> static const void* rope_kernel(int dtype, int vec, bool neighbours, bool backward)
{
    return dtype == RMSQ_BF16   ? rope_fn<DT_BF16, BOTH>(vec, neighbours, backward)
           : dtype == RMSQ_FP16 ? rope_fn<DT_FP16, BOTH>(vec, neighbours, backward)
                                : rope_fn<DT_F32, BOTH>(vec, neighbours, backward);
}

// Whether a turn may have rows of two tokens, or the kernel allows for it.
static bool two_tokens(const RopeParams& p, int vec) { return vec < 4 || p.side[0].groups % 2 != 0 || p.side[1].groups % 2 != 0; }

static const void* rope_kernel(const RopeParams& p, int dtype, int vec, bool neighbours, bool backward)
{
    return two_tokens(p, vec) ? rope_kernel<true>(dtype, vec, neighbours, backward) : rope_kernel<false>(dtype, vec, neighbours, backward);
}

static rmsq_status status_of(cudaError_t e)
{
    if (e == cudaSuccess) return RMSQ_OK;
    cudaGetLastError();
    return RMSQ_ERR_LAUNCH;
}

template <bool BACKWARD> static int rope_smem(const RopeParams& p, int dtype, int vec)
{
    using S = RopeShape<BACKWARD>;
    return S::STAGES * 16 * (dtype == RMSQ_F32 ? 4 : 2) * S::THREADS * kRopeRows * (BACKWARD ? 2 : 1) +
           S::THREADS / 32 * (two_tokens(p, vec) ? RopeAngles<S::STAGES, true>::bytes(p.half) : RopeAngles<S::STAGES, false>::bytes(p.half)) +
           (p.dim + 3) / 4 * 16;
}

}  // namespace rmsq

using namespace rmsq;

extern "C" rmsq_status rmsnorm_rope(const rmsq_heads* query, const rmsq_heads* key, const void* query_gamma,
                                    const void* key_gamma, const rmsq_rotation* rotation, int64_t tokens, int64_t dim,
                                    int dtype, float epsilon, float weight_offset, const rmsq_heads* query_output,
                                    const rmsq_heads* key_output, void* stream)
{
    RopeParams p;
    int vec = 0;
    const rmsq_status st = prepare_rope({nullptr, nullptr, query, key, query_gamma, key_gamma, rotation, tokens, dim, dtype,
                                         epsilon, weight_offset, query_output, key_output}, &p, &vec);
    if (st != RMSQ_OK || tokens == 0) return st;
    DeviceView dv;
    if (!device_view(&dv)) return RMSQ_ERR_DEVICE;
    const bool neighbours = rotation->neighbours != 0;
    using S = RopeShape<false>;
    const unsigned grid = deal_rope(&p, vec, neighbours, dv.sms * S::CTAS, S::THREADS / 32);
    void* args[] = {&p};
    return status_of(launch_kernel(rope_kernel(p, dtype, vec, neighbours, false), dim3(grid), S::THREADS, rope_smem<false>(p, dtype, vec), 1,
                                   static_cast<cudaStream_t>(stream), args));
}

extern "C" int64_t rmsnorm_rope_backward_workspace(int64_t tokens, int64_t dim)
{
    if (tokens <= 0 || dim <= 0 || dim > RMSQ_ROPE_MAX_DIM) return 0;
    return RMSQ_ROPE_PARTS * dim * static_cast<int64_t>(sizeof(float));
}

extern "C" rmsq_status rmsnorm_rope_backward(const rmsq_heads* grad_query, const rmsq_heads* grad_key,
                                             const rmsq_heads* query, const rmsq_heads* key, const void* query_gamma,
                                             const void* key_gamma, const rmsq_rotation* rotation, int64_t tokens,
                                             int64_t dim, int dtype, float epsilon, float weight_offset,
                                             const rmsq_heads* query_output, const rmsq_heads* key_output,
                                             void* grad_query_gamma, void* grad_key_gamma, int param_grad_dtype,
                                             void* workspace, int64_t workspace_bytes, void* stream)
{
    RopeParams p;
    int vec = 0;
    rmsq_status st = prepare_rope({grad_query, grad_key, query, key, query_gamma, key_gamma, rotation, tokens, dim, dtype,
                                   epsilon, weight_offset, query_output, key_output}, &p, &vec);
    if (st != RMSQ_OK) return st;
    if (param_grad_dtype != dtype && param_grad_dtype != RMSQ_F32) return RMSQ_ERR_DTYPE;
    const int es = dtype == RMSQ_F32 ? 4 : 2;
    const rmsq_heads* grads[2] = {grad_query, grad_key};
    for (int s = 0; s < 2; ++s) {
        st = check_side(grads[s], tokens, dim, es, false, &vec);
        if (st != RMSQ_OK) return st;
        if (grads[s]->heads != p.side[s].heads) return RMSQ_ERR_SHAPE;
        p.side[s].dy = grads[s]->data;
        p.side[s].dt = static_cast<unsigned>(grads[s]->token_stride);
        p.side[s].dh = static_cast<unsigned>(grads[s]->head_stride);
    }
    if (!grad_query_gamma || !grad_key_gamma) return RMSQ_ERR_NULL;
    if (!aligned(grad_query_gamma, 16) || !aligned(grad_key_gamma, 16)) return RMSQ_ERR_ALIGN;
    if (tokens > 0) {
        if (!workspace) return RMSQ_ERR_NULL;
        if (!aligned(workspace, 16)) return RMSQ_ERR_ALIGN;
        if (workspace_bytes < rmsnorm_rope_backward_workspace(tokens, dim)) return RMSQ_ERR_SHAPE;
    }
    DeviceView dv;
    if (!device_view(&dv)) return RMSQ_ERR_DEVICE;
    RopeReduceParams r = {};
    r.part = static_cast<const float*>(workspace);
    r.out[0] = grad_query_gamma;
    r.out[1] = grad_key_gamma;
    r.dim = static_cast<int>(dim);
    r.dt = param_grad_dtype;
    if (tokens > 0) {
        const bool neighbours = rotation->neighbours != 0;
        using S = RopeShape<true>;
        const int ctas = dv.sms * S::CTAS < RMSQ_ROPE_PARTS ? dv.sms * S::CTAS : RMSQ_ROPE_PARTS;
        const unsigned grid = deal_rope(&p, vec, neighbours, ctas, S::THREADS / 32);
        p.part = static_cast<float*>(workspace);
        r.rows[0] = p.split;
        r.rows[1] = static_cast<int>(grid) - p.split;
        void* args[] = {&p};
        st = status_of(launch_kernel(rope_kernel(p, dtype, vec, neighbours, true), dim3(grid), S::THREADS, rope_smem<true>(p, dtype, vec), 1,
                                     static_cast<cudaStream_t>(stream), args));
        if (st != RMSQ_OK) return st;
    }
    void* args[] = {&r};
    return status_of(launch_kernel(reinterpret_cast<const void*>(&rmsq_rope_reduce_kernel),
                                   dim3(static_cast<unsigned>((dim + 31) / 32), 2), 1024, 0, 1, static_cast<cudaStream_t>(stream), args));
}
