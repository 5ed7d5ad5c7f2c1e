// window_api.cu -- C ABI of sliding-window attention: argument checks, tensor maps, launches.
#include <math.h>
#include <string.h>

#include "kernels.h"
#include "lm.h"
#include "tensor_map.h"
#include "window.h"

namespace {

using st::aligned_to;
using st::check_strides;
using st::MAX_POS;

// Sizes of a window call: one error for what no kernel could mean, another for what these do not take.
st_status_t check_sizes(const st_window_desc_t *d, const st_window_t *w)
{
    if (!d || !w || d->batch < 1 || d->nq < 1 || d->nk < 1 || d->d < 1 || d->q_start < 0 ||
        (d->dtype != ST_BF16 && d->dtype != ST_FP16 && d->dtype != ST_FP32))
        return ST_ERR_INVALID_ARG;
    if (d->dtype == ST_FP32 || (d->d != 64 && d->d != 128) || d->nq > MAX_POS || d->nk > MAX_POS || d->q_start > MAX_POS ||
        d->q_start + d->nq > MAX_POS || d->batch > (1 << 20) || w->heads > (1 << 20) ||
        d->batch * w->heads > INT32_MAX / ((d->nq + 127) / 128) || d->batch * w->heads > INT32_MAX / ((d->nk + 127) / 128))
        return ST_ERR_UNSUPPORTED;
    return ST_OK;
}

// Tensor map of a 16-bit [batch, heads, rows, d] tensor: boxes of 64 columns by 128 rows.
bool make_map(CUtensorMap *m, const void *p, const st_strides_t &s, const st_window_desc_t *d, int64_t heads, int64_t rows)
{
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d->d), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(d->batch)};
    // the stride of a dimension of extent 1 is not used, but must be valid
    const cuuint64_t any = static_cast<cuuint64_t>(d->d) * 2;
    const cuuint64_t str[3] = {rows > 1 ? static_cast<cuuint64_t>(s.row) * 2 : any, heads > 1 ? static_cast<cuuint64_t>(s.head) * 2 : any,
                               d->batch > 1 ? static_cast<cuuint64_t>(s.batch) * 2 : any};
    const cuuint32_t box[4] = {64, 128, 1, 1};
    return st::encode(m, p, d->dtype == ST_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, dims,
                      str, box);
}

st::RawTensor raw(const void *p, const st_strides_t &s)
{
    return {static_cast<const char *>(p), s.batch * 2, s.head * 2, s.row * 2};
}

st::WindowGeom geometry(const st_window_desc_t *d, const st_window_t *w, const int32_t *lens)
{
    st::WindowGeom g;
    memset(&g, 0, sizeof(g));
    g.lens = lens;
    g.batch = static_cast<int32_t>(d->batch);
    g.heads = w->heads;
    g.kv = w->kv_heads;
    g.group = w->heads / w->kv_heads;
    g.nq = static_cast<int32_t>(d->nq);
    g.nk = static_cast<int32_t>(d->nk);
    g.q_start = static_cast<int32_t>(d->q_start);
    g.window = static_cast<int32_t>(w->window);
    g.sinks = static_cast<int32_t>(w->sinks);
    g.nqt = (g.nq + 127) / 128;
    g.nkt = (g.nk + 127) / 128;
    g.scale = 1.0f / sqrtf(static_cast<float>(d->d));
    g.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(d->d));
    g.err = w->d_err;
    return g;
}

}  // namespace

extern "C" {

st_status_t st_window_fwd(const void *q, const void *k, const void *v, const int32_t *lens, const st_window_t *w, void *o,
                          float *lse, const st_window_desc_t *desc, st_stream_t stream)
{
    if (!q || !k || !v || !o || !lse) return ST_ERR_INVALID_ARG;
    st_status_t cs = check_sizes(desc, w);
    if (cs != ST_OK || (cs = check_strides(desc->q, desc->batch, w->heads, desc->nq, desc->d, 2)) != ST_OK ||
        (cs = check_strides(desc->k, desc->batch, w->kv_heads, desc->nk, desc->d, 2)) != ST_OK ||
        (cs = check_strides(desc->v, desc->batch, w->kv_heads, desc->nk, desc->d, 2)) != ST_OK ||
        (cs = check_strides(desc->o, desc->batch, w->heads, desc->nq, desc->d, 2)) != ST_OK)
        return cs;
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(o, 16) || !aligned_to(lse, 4) ||
        !aligned_to(lens, 4))
        return ST_ERR_ALIGNMENT;
    if ((cs = st::check_window(w)) != ST_OK) return cs;
    if (!st::encode_fn()) return ST_ERR_CUDA;
    st::WindowFwdParams p;
    memset(&p, 0, sizeof(p));
    if (!make_map(&p.q, q, desc->q, desc, w->heads, desc->nq) || !make_map(&p.k, k, desc->k, desc, w->kv_heads, desc->nk) ||
        !make_map(&p.v, v, desc->v, desc, w->kv_heads, desc->nk))
        return ST_ERR_CUDA;
    p.g = geometry(desc, w, lens);
    p.vraw = raw(v, desc->v);
    p.o = static_cast<char *>(o);
    p.o_batch = desc->o.batch * 2;
    p.o_head = desc->o.head * 2;
    p.o_row = desc->o.row * 2;
    p.lse = lse;
    p.pair_rows = p.g.group % 2 != 0;
    p.units = p.g.batch * (p.pair_rows ? p.g.heads * ((p.g.nqt + 1) / 2) : p.g.heads / 2 * p.g.nqt);
    return st::launch_window_fwd(p, desc->dtype, static_cast<int>(desc->d), stream) == cudaSuccess ? ST_OK : ST_ERR_CUDA;
}

}  // extern "C"
extern "C" {
size_t st_window_bwd_workspace_bytes(const st_window_desc_t *, const st_window_t *) { return 0; }
st_status_t st_window_bwd(const void *, const void *, const void *, const void *, const float *, const void *, const int32_t *,
                          const st_window_t *, void *, void *, void *, void *, size_t, const st_window_desc_t *, st_stream_t)
{
    return ST_ERR_UNSUPPORTED;
}
}
