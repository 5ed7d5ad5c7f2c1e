// lm_api.cu -- C ABI of the language-model operators: the window handle, the norm and rotation, and
// the paged cache (argument checks and launches).
#include <math.h>
#include <string.h>

#include <new>

#include "kernels.h"
#include "lm.h"
#include "paged_decode.h"
#include "plan.h"
#include "rope.h"

namespace {

using st::aligned_to;
using st::check_strides;
using st::elem_bytes;
using st::MAX_POS;
using st::round256;

bool known_dtype(int32_t t) { return t == ST_BF16 || t == ST_FP32 || t == ST_FP16; }

st::RopeTensor tensor(const void *p, const st_strides_t &s, int es)
{
    return {static_cast<char *>(const_cast<void *>(p)), s.batch * es, s.head * es, s.row * es};
}

st_status_t check_rope(const st_rope_desc_t *d)
{
    if (!d) return ST_ERR_INVALID_ARG;
    if (d->batch < 1 || d->heads < 1 || d->kv_heads < 1 || d->n < 1 || d->d < 1 || d->pos_batch < 0 ||
        !known_dtype(d->dtype) || (d->wdtype != d->dtype && d->wdtype != ST_FP32) || !(d->eps >= 0.f) ||
        d->rot < 1 || d->rot > d->d || (d->interleaved != 0 && d->interleaved != 1))
        return ST_ERR_INVALID_ARG;
    if (d->d > 256 || d->d % 16 != 0 || d->rot % 16 != 0 || d->batch > MAX_POS || d->n > MAX_POS ||
        d->batch * d->n > MAX_POS || d->heads > 4096 || d->kv_heads > 4096 ||
        d->batch * d->n * ((d->heads + 2 * d->kv_heads + 1) / 2) > INT32_MAX)
        return ST_ERR_UNSUPPORTED;
    return ST_OK;
}

st::RopeParams rope_params(const st_rope_desc_t *d, const void *wq, const void *wk, const uint64_t *turns,
                           const int32_t *positions)
{
    st::RopeParams p;
    memset(&p, 0, sizeof(p));
    p.wq = wq;
    p.wk = wk;
    p.turns = turns;
    p.positions = positions;
    p.n = d->n;
    p.start = d->start;
    p.pos_batch = d->pos_batch;
    p.batch = d->batch;
    p.heads = static_cast<int32_t>(d->heads);
    p.kv = static_cast<int32_t>(d->kv_heads);
    p.d = static_cast<int32_t>(d->d);
    p.rot = d->rot;
    p.interleaved = d->interleaved;
    p.w_f32 = d->wdtype == ST_FP32;
    p.eps = d->eps;
    p.mscale = d->mscale;
    p.inv_d = 1.0f / static_cast<float>(d->d);
    return p;
}

// Strides of a q-shaped and a k-shaped tensor.
st_status_t check_pair(const st_rope_desc_t *d, const st_strides_t &q, const st_strides_t &k)
{
    const int es = elem_bytes(d->dtype);
    const st_status_t s = check_strides(q, d->batch, d->heads, d->n, d->d, es);
    return s != ST_OK ? s : check_strides(k, d->batch, d->kv_heads, d->n, d->d, es);
}

st_status_t check_pages(const st_pages_t *g, int64_t kv, int64_t d, int es)
{
    if (!g || g->num_pages < 1 || g->page_size < 1 || g->num_pages > INT32_MAX / g->page_size) return ST_ERR_INVALID_ARG;
    const st_status_t s = check_strides(g->k, g->num_pages, kv, g->page_size, d, es);
    return s != ST_OK ? s : check_strides(g->v, g->num_pages, kv, g->page_size, d, es);
}

}  // namespace

extern "C" {

// ---- the window handle --------------------------------------------------------------------------

st_status_t st_window_create(int32_t heads, int32_t kv_heads, int64_t window, int64_t sinks, st_window_t **out)
{
    if (!out || heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || window < 0 || window > MAX_POS || sinks < 0 ||
        sinks > MAX_POS)
        return ST_ERR_INVALID_ARG;
    st_window *w = new (std::nothrow) st_window();
    if (!w) return ST_ERR_OOM;
    w->heads = heads;
    w->kv_heads = kv_heads;
    w->window = window;
    w->sinks = sinks;
    *out = w;
    return ST_OK;
}

st_status_t st_window_upload(st_window_t *w, st_stream_t stream)
{
    if (!w) return ST_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return ST_ERR_CUDA;
    if (w->uploaded) return dev == w->device ? ST_OK : ST_ERR_INVALID_ARG;
    if (cudaMalloc(&w->d_err, 256) != cudaSuccess) {
        w->d_err = nullptr;
        return ST_ERR_OOM;
    }
    // the word is zero before any stream's kernel can use it
    if (cudaMemsetAsync(w->d_err, 0, 256, stream) != cudaSuccess || cudaStreamSynchronize(stream) != cudaSuccess) {
        cudaFree(w->d_err);
        w->d_err = nullptr;
        return ST_ERR_CUDA;
    }
    w->device = dev;
    w->uploaded = true;
    return ST_OK;
}

st_status_t st_window_check(st_window_t *w, st_stream_t stream)
{
    const st_status_t cs = st::check_window(w);
    if (cs != ST_OK) return cs;
    int32_t err = 0;
    if (cudaMemcpyAsync(&err, w->d_err, sizeof(err), cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
        return ST_ERR_CUDA;
    if (err == 0) return ST_OK;
    if (cudaMemsetAsync(w->d_err, 0, sizeof(err), stream) != cudaSuccess || cudaStreamSynchronize(stream) != cudaSuccess)
        return ST_ERR_CUDA;
    return (err & 1) ? ST_ERR_DEVICE_TIMEOUT : ((err & st::ERR_PAGE) ? ST_ERR_BAD_PAGE : ST_ERR_INTERNAL);
}

void st_window_destroy(st_window_t *w)
{
    if (!w) return;
    if (w->d_err) cudaFree(w->d_err);
    delete w;
}

// ---- norm and rotation --------------------------------------------------------------------------

st_status_t st_rope_turns(int32_t rot, double base, int32_t scaling, double factor, double original, uint64_t *turns,
                          float *mscale)
{
    if (!turns || !mscale || rot < 2 || rot % 2 != 0 || !(base > 1.0) || !isfinite(base) || !(factor >= 1.0) ||
        !isfinite(factor) || scaling < ST_ROPE_NONE || scaling > ST_ROPE_YARN ||
        (scaling == ST_ROPE_YARN && !(original > 0.0 && isfinite(original))) || (scaling == ST_ROPE_NTK && rot < 4))
        return ST_ERR_INVALID_ARG;
    const long double two_pi = 6.283185307179586476925286766559L;
    long double theta = base;
    if (scaling == ST_ROPE_NTK) theta *= powl(factor, static_cast<long double>(rot) / (rot - 2));
    for (int32_t i = 0; i < rot / 2; ++i) {
        long double w = powl(theta, -2.0L * i / rot);
        if (scaling == ST_ROPE_LINEAR) w /= factor;
        if (scaling == ST_ROPE_YARN) {
            const long double t = fminl(1.0L, fmaxl(0.0L, (original * w / two_pi - 1.0L) / 31.0L));
            w *= t + (1.0L - t) / factor;
        }
        turns[i] = static_cast<uint64_t>(w / two_pi * 0x1p64L + 0.5L);  // w <= 1: under 2^62
    }
    *mscale = scaling == ST_ROPE_YARN ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
    return ST_OK;
}

st_status_t st_qk_norm_rope(const void *q, const void *k, const void *wq, const void *wk, const uint64_t *turns,
                            const int32_t *positions, void *q_out, void *k_out, const st_rope_desc_t *desc,
                            st_stream_t stream)
{
    if (!q || !k || !turns || !q_out || !k_out || (!wq != !wk)) return ST_ERR_INVALID_ARG;
    st_status_t cs = check_rope(desc);
    if (cs != ST_OK || (cs = check_pair(desc, desc->q, desc->k)) != ST_OK ||
        (cs = check_pair(desc, desc->q_out, desc->k_out)) != ST_OK)
        return cs;
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(q_out, 16) || !aligned_to(k_out, 16) ||
        !aligned_to(wq, 16) || !aligned_to(wk, 16) || !aligned_to(turns, 8) || !aligned_to(positions, 4))
        return ST_ERR_ALIGNMENT;
    if (st::same_start<2, 4>({q_out, k_out}, {wq, wk, turns, positions}) || q_out == k || k_out == q ||
        (q_out == q && !st::same_strides(desc->q_out, desc->q, desc->batch, desc->heads, desc->n)) ||
        (k_out == k && !st::same_strides(desc->k_out, desc->k, desc->batch, desc->kv_heads, desc->n)))
        return ST_ERR_INVALID_ARG;
    const int es = elem_bytes(desc->dtype);
    st::RopeParams p = rope_params(desc, wq, wk, turns, positions);
    p.q = tensor(q, desc->q, es);
    p.k = tensor(k, desc->k, es);
    p.qo = tensor(q_out, desc->q_out, es);
    p.ko = tensor(k_out, desc->k_out, es);
    return st::launch_rope(p, desc->dtype, st::ROPE_FWD, nullptr, nullptr, stream) == cudaSuccess ? ST_OK : ST_ERR_CUDA;
}

size_t st_qk_norm_rope_bwd_workspace_bytes(const st_rope_desc_t *desc)
{
    if (check_rope(desc) != ST_OK) return 0;
    const st::RopeCtas c = st::rope_bwd_ctas(desc->batch * desc->n, static_cast<int>(desc->heads),
                                             static_cast<int>(desc->kv_heads), static_cast<int>(desc->d));
    return round256(static_cast<size_t>(c.q + c.k) * desc->d * sizeof(float));
}

st_status_t st_qk_norm_rope_bwd(const void *q, const void *k, const void *gq, const void *gk, const void *wq,
                                const void *wk, const uint64_t *turns, const int32_t *positions, void *dq, void *dk,
                                float *dwq, float *dwk, void *workspace, size_t workspace_bytes,
                                const st_rope_desc_t *desc, st_stream_t stream)
{
    if (!q || !k || !gq || !gk || !turns || !dq || !dk || (!wq != !wk) || (wq && (!dwq || !dwk)))
        return ST_ERR_INVALID_ARG;
    st_status_t cs = check_rope(desc);
    if (cs != ST_OK || (cs = check_pair(desc, desc->q, desc->k)) != ST_OK ||
        (cs = check_pair(desc, desc->q_out, desc->k_out)) != ST_OK || (cs = check_pair(desc, desc->dq, desc->dk)) != ST_OK)
        return cs;
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(gq, 16) || !aligned_to(gk, 16) || !aligned_to(dq, 16) ||
        !aligned_to(dk, 16) || !aligned_to(wq, 16) || !aligned_to(wk, 16) || !aligned_to(turns, 8) ||
        !aligned_to(positions, 4) || !aligned_to(dwq, 4) || !aligned_to(dwk, 4))
        return ST_ERR_ALIGNMENT;
    if (wq) {
        if (!workspace || workspace_bytes < st_qk_norm_rope_bwd_workspace_bytes(desc)) return ST_ERR_WORKSPACE;
        if (!aligned_to(workspace, 256)) return ST_ERR_ALIGNMENT;
        if (st::same_start<3, 10>({dwq, dwk, workspace}, {q, k, gq, gk, wq, wk, turns, positions, dq, dk}))
            return ST_ERR_INVALID_ARG;
    }
    if (st::same_start<2, 6>({dq, dk}, {q, k, wq, wk, turns, positions}) || dq == gk || dk == gq ||
        (dq == gq && !st::same_strides(desc->dq, desc->q_out, desc->batch, desc->heads, desc->n)) ||
        (dk == gk && !st::same_strides(desc->dk, desc->k_out, desc->batch, desc->kv_heads, desc->n)))
        return ST_ERR_INVALID_ARG;
    const int es = elem_bytes(desc->dtype);
    st::RopeParams p = rope_params(desc, wq, wk, turns, positions);
    p.q = tensor(q, desc->q, es);
    p.k = tensor(k, desc->k, es);
    p.gq = tensor(gq, desc->q_out, es);
    p.gk = tensor(gk, desc->k_out, es);
    p.qo = tensor(dq, desc->dq, es);
    p.ko = tensor(dk, desc->dk, es);
    p.partial = static_cast<float *>(workspace);
    return st::launch_rope(p, desc->dtype, st::ROPE_BWD, dwq, dwk, stream) == cudaSuccess ? ST_OK : ST_ERR_CUDA;
}

// ---- paged cache --------------------------------------------------------------------------------

st_status_t st_paged_plan(const int32_t *lens, const int32_t *new_tokens, int32_t *block_table, const int32_t *free_pages,
                          const int32_t *free_count, int32_t *lens_out, int32_t *free_left, int32_t *offsets,
                          int32_t *slots, int32_t *positions, int32_t *status, const st_plan_desc_t *desc,
                          st_stream_t stream)
{
    const void *ptrs[] = {lens, new_tokens, block_table, free_pages, free_count, lens_out,
                          free_left, offsets, slots, positions, status};
    if (!desc) return ST_ERR_INVALID_ARG;
    for (int i = 0; i < 11; ++i)
        if (!ptrs[i] && !(i == 3 && desc->free_capacity == 0)) return ST_ERR_INVALID_ARG;  // (an empty list is not read)
    if (desc->requests < 1 || desc->tokens < 1 || desc->tokens > MAX_POS || desc->max_pages < 1 ||
        desc->max_pages > (1 << 24) || desc->page_size < 1 || desc->page_size > (1 << 20) || desc->free_capacity < 0 ||
        desc->free_capacity > INT32_MAX || (desc->requests > 1 && desc->table_stride < desc->max_pages) ||
        desc->table_stride > (1ll << 38))
        return ST_ERR_INVALID_ARG;
    if (desc->requests > st::PLAN_MAX_REQUESTS) return ST_ERR_UNSUPPORTED;
    // an output that shares memory with another array would be read while it is written
    const int64_t R = desc->requests;
    const int64_t words[] = {R, R, (R - 1) * (R > 1 ? desc->table_stride : 0) + desc->max_pages, desc->free_capacity, 1, R, 1,
                             R + 1, desc->tokens, desc->tokens, R};
    for (int i = 0; i < 11; ++i) {
        if (!aligned_to(ptrs[i], 4)) return ST_ERR_ALIGNMENT;
        for (int j = 0; j < i; ++j) {
            if ((i < 5 && i != 2 && j != 2) || words[i] == 0 || words[j] == 0) continue;  // two inputs, or no elements
            const auto a = reinterpret_cast<uintptr_t>(ptrs[i]), b = reinterpret_cast<uintptr_t>(ptrs[j]);
            if (a < b + 4 * words[j] && b < a + 4 * words[i]) return ST_ERR_INVALID_ARG;
        }
    }
    st::PlanParams p{lens, new_tokens, free_pages, free_count, block_table, lens_out, free_left, offsets, slots, positions,
                     status, desc->tokens, desc->max_pages, desc->table_stride, desc->page_size, desc->free_capacity,
                     static_cast<int32_t>(R)};
    return st::launch_plan(p, stream) == cudaSuccess ? ST_OK : ST_ERR_CUDA;
}

st_status_t st_paged_append(const void *q, const void *k, const void *v, const void *wq, const void *wk,
                            const uint64_t *turns, const int32_t *positions, const int32_t *slots, void *q_out,
                            void *k_pages, void *v_pages, const st_strides_t *v_strides, const st_pages_t *pages,
                            const st_rope_desc_t *desc, st_stream_t stream)
{
    if (!q || !k || !v || !turns || !positions || !slots || !q_out || !k_pages || !v_pages || !v_strides || (!wq != !wk))
        return ST_ERR_INVALID_ARG;
    st_status_t cs = check_rope(desc);
    if (cs != ST_OK) return cs;
    if (desc->batch != 1) return ST_ERR_INVALID_ARG;
    const int es = elem_bytes(desc->dtype);
    if ((cs = check_pair(desc, desc->q, desc->k)) != ST_OK || (cs = check_pair(desc, desc->q_out, *v_strides)) != ST_OK ||
        (cs = check_pages(pages, desc->kv_heads, desc->d, es)) != ST_OK)
        return cs;
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(q_out, 16) ||
        !aligned_to(k_pages, 16) || !aligned_to(v_pages, 16) || !aligned_to(wq, 16) || !aligned_to(wk, 16) ||
        !aligned_to(turns, 8) || !aligned_to(positions, 4) || !aligned_to(slots, 4))
        return ST_ERR_ALIGNMENT;
    if (st::same_start<3, 7>({q_out, k_pages, v_pages}, {k, v, wq, wk, turns, positions, slots}) || k_pages == q ||
        v_pages == q || (q_out == q && !st::same_strides(desc->q_out, desc->q, 1, desc->heads, desc->n)))
        return ST_ERR_INVALID_ARG;
    st::RopeParams p = rope_params(desc, wq, wk, turns, positions);
    p.q = tensor(q, desc->q, es);
    p.k = tensor(k, desc->k, es);
    p.v = tensor(v, *v_strides, es);
    p.qo = tensor(q_out, desc->q_out, es);
    p.ko = tensor(k_pages, pages->k, es);
    p.vo = tensor(v_pages, pages->v, es);
    p.slots = slots;
    p.page_size = pages->page_size;
    p.nslots = pages->num_pages * pages->page_size;
    return st::launch_rope(p, desc->dtype, st::ROPE_APPEND, nullptr, nullptr, stream) == cudaSuccess ? ST_OK : ST_ERR_CUDA;
}

namespace {

// Sizes of a decode call: one error for what no kernel could mean, another for what these do not take.
st_status_t check_paged(const st_paged_desc_t *d, const st_window_t *w)
{
    if (!d || !w || d->requests < 1 || d->max_pages < 1 || d->d < 1 || d->pages.num_pages < 1 ||
        d->pages.page_size < 1 || d->pages.num_pages > INT32_MAX / d->pages.page_size ||
        (d->dtype != ST_BF16 && d->dtype != ST_FP16 && d->dtype != ST_FP32) ||
        (d->requests > 1 && d->table_stride < d->max_pages) || d->table_stride > (1ll << 38))
        return ST_ERR_INVALID_ARG;
    if (d->dtype == ST_FP32 || (d->d != 64 && d->d != 128) || d->pages.page_size % st::PD_TILE != 0 ||
        w->heads / w->kv_heads > 64 || d->requests > st::PD_MAX_REQUESTS || d->max_pages > MAX_POS / d->pages.page_size ||
        d->requests * (d->max_pages * (d->pages.page_size / st::PD_TILE) + 1) > INT32_MAX)
        return ST_ERR_UNSUPPORTED;
    return ST_OK;
}

int32_t paged_grid()
{
    const int32_t n = st::sm_count() * st::PD_CTAS_PER_SM;
    return n < st::PD_MAX_GRID ? n : st::PD_MAX_GRID;
}

}  // namespace

size_t st_paged_decode_workspace_bytes(const st_paged_desc_t *desc, const st_window_t *w)
{
    if (check_paged(desc, w) != ST_OK) return 0;
    const size_t part = static_cast<size_t>(st::pd_part(w->heads / w->kv_heads, static_cast<int>(desc->d)));
    return round256((desc->requests + 1) * sizeof(int32_t)) + round256(2 * paged_grid() * part * sizeof(float));
}

st_status_t st_paged_decode(const void *q, const void *k_pages, const void *v_pages, const int32_t *block_table,
                            const int32_t *lens, const st_window_t *w, void *o, float *lse, void *workspace,
                            size_t workspace_bytes, const st_paged_desc_t *desc, st_stream_t stream)
{
    if (!q || !k_pages || !v_pages || !block_table || !lens || !o || !lse) return ST_ERR_INVALID_ARG;
    st_status_t cs = check_paged(desc, w);
    if (cs != ST_OK || (cs = check_pages(&desc->pages, w->kv_heads, desc->d, 2)) != ST_OK) return cs;
    if (!aligned_to(q, 16) || !aligned_to(k_pages, 16) || !aligned_to(v_pages, 16) || !aligned_to(o, 16) ||
        !aligned_to(block_table, 4) || !aligned_to(lens, 4) || !aligned_to(lse, 4))
        return ST_ERR_ALIGNMENT;
    if ((cs = st::check_window(w)) != ST_OK) return cs;
    if (!workspace || workspace_bytes < st_paged_decode_workspace_bytes(desc, w)) return ST_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return ST_ERR_ALIGNMENT;
    if (st::same_start<3, 5>({o, lse, workspace}, {q, k_pages, v_pages, block_table, lens})) return ST_ERR_INVALID_ARG;
    st::PagedParams p;
    memset(&p, 0, sizeof(p));
    p.q = q;
    p.k = static_cast<const char *>(k_pages);
    p.v = static_cast<const char *>(v_pages);
    p.k_page = desc->pages.k.batch * 2;
    p.k_head = desc->pages.k.head * 2;
    p.k_row = desc->pages.k.row * 2;
    p.v_page = desc->pages.v.batch * 2;
    p.v_head = desc->pages.v.head * 2;
    p.v_row = desc->pages.v.row * 2;
    p.table = block_table;
    p.lens = lens;
    p.o = o;
    p.lse = lse;
    p.prefix = static_cast<int32_t *>(workspace);
    p.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + round256((desc->requests + 1) * sizeof(int32_t)));
    p.err = w->d_err;
    p.table_stride = desc->table_stride;
    p.num_pages = desc->pages.num_pages;
    p.capacity = static_cast<int32_t>(desc->max_pages * desc->pages.page_size);
    p.window = static_cast<int32_t>(w->window);
    p.sinks = static_cast<int32_t>(w->sinks);
    p.requests = static_cast<int32_t>(desc->requests);
    p.heads = w->heads;
    p.kv = w->kv_heads;
    p.group = w->heads / w->kv_heads;
    const int hb = st::pd_heads(p.group);
    p.blocks = (p.group + hb - 1) / hb;
    p.page_size = static_cast<int32_t>(desc->pages.page_size);
    p.grid = paged_grid();
    p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(desc->d));
    return st::launch_paged_decode(p, desc->dtype, static_cast<int>(desc->d), stream) == cudaSuccess ? ST_OK : ST_ERR_CUDA;
}

}  // extern "C"
