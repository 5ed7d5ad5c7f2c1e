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

// The units of the dK, dV kernel: steps a chunk may have, entries a key head, chunked ones among them.
struct Units {
    int32_t chunk, entries, split;
};

Units plan_units(const st::WindowGeom &g)
{
    // A chunk's partial sums cost about five steps' time to write and add (128 KB at d = 128), so
    // chunks have at least 32, or where the SMs would have less than 16 each, down to 8; beyond that
    // enough of them for four rounds of the SMs.
    int64_t total = 0;
    for (int32_t t = 0; t < g.nkt; ++t) {
        int32_t i0, i1;
        st::query_range(g, t, i0, i1);
        if (i1 >= i0) total += static_cast<int64_t>(i1 - i0 + 1) * g.group;
    }
    total *= static_cast<int64_t>(g.batch) * g.kv;
    const int64_t each = total / st::sm_count(), least = each >= 16 ? 32 : (each <= 4 ? 8 : 2 * each), rounds = each / 4;
    Units u{static_cast<int32_t>(rounds < least ? least : (rounds > MAX_POS ? MAX_POS : rounds)), 0, 0};
    for (int32_t t = 0; t < g.nkt; ++t) {
        int32_t i0, i1;
        st::query_range(g, t, i0, i1);
        const int32_t c = st::chunks_of(i1 < i0 ? 0 : (i1 - i0 + 1) * g.group, u.chunk);
        u.entries += c;
        if (c > 1) u.split += c;
    }
    return u;
}

struct BwdSizes {
    size_t delta, entries, parts, maxima, counters;
    size_t total() const { return delta + entries + parts + maxima + counters; }
};

BwdSizes bwd_sizes(const st::WindowGeom &g, const Units &u, int64_t d)
{
    const size_t bk = static_cast<size_t>(g.batch) * g.kv;
    return {st::round256(static_cast<size_t>(g.batch) * g.heads * g.nq * sizeof(float)), st::round256(u.entries * sizeof(int2)),
            bk * u.split * 2 * 128 * d * sizeof(float), st::round256(bk * 2 * sizeof(uint32_t)),
            256};
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
    if (st::same_start<2, 4>({o, lse}, {q, k, v, lens})) return ST_ERR_INVALID_ARG;
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

size_t st_window_bwd_workspace_bytes(const st_window_desc_t *desc, const st_window_t *w)
{
    if (check_sizes(desc, w) != ST_OK) return 0;
    const st::WindowGeom g = geometry(desc, w, nullptr);
    return bwd_sizes(g, plan_units(g), desc->d).total();
}

st_status_t st_window_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dO,
                          const int32_t *lens, const st_window_t *w, void *dq, void *dk, void *dv, void *workspace,
                          size_t workspace_bytes, const st_window_desc_t *desc, st_stream_t stream)
{
    if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return ST_ERR_INVALID_ARG;
    st_status_t cs = check_sizes(desc, w);
    if (cs != ST_OK) return cs;
    const st_strides_t *qs[] = {&desc->q, &desc->o, &desc->dout, &desc->dq}, *ks[] = {&desc->k, &desc->v, &desc->dk, &desc->dv};
    for (int i = 0; i < 4; ++i)
        if ((cs = check_strides(*qs[i], desc->batch, w->heads, desc->nq, desc->d, 2)) != ST_OK ||
            (cs = check_strides(*ks[i], desc->batch, w->kv_heads, desc->nk, desc->d, 2)) != ST_OK)
            return cs;
    for (const void *p : {q, k, v, o, dO, static_cast<const void *>(dq), static_cast<const void *>(dk), static_cast<const void *>(dv)})
        if (!aligned_to(p, 16)) return ST_ERR_ALIGNMENT;
    if (!aligned_to(lse, 4) || !aligned_to(lens, 4)) return ST_ERR_ALIGNMENT;
    if ((cs = st::check_window(w)) != ST_OK) return cs;
    st::WindowBwdParams p;
    memset(&p, 0, sizeof(p));
    p.g = geometry(desc, w, lens);
    const Units u = plan_units(p.g);
    const BwdSizes z = bwd_sizes(p.g, u, desc->d);
    if (static_cast<int64_t>(u.entries) * p.g.batch * p.g.kv > INT32_MAX ||
        static_cast<int64_t>(u.split) * p.g.batch * p.g.kv * (desc->d / 4) > INT32_MAX)
        return ST_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < z.total()) return ST_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return ST_ERR_ALIGNMENT;
    if (st::same_start<4, 7>({dq, dk, dv, workspace}, {q, k, v, o, lse, dO, lens})) return ST_ERR_INVALID_ARG;
    if (!st::encode_fn()) return ST_ERR_CUDA;
    if (!make_map(&p.q, q, desc->q, desc, w->heads, desc->nq) || !make_map(&p.k, k, desc->k, desc, w->kv_heads, desc->nk) ||
        !make_map(&p.v, v, desc->v, desc, w->kv_heads, desc->nk) || !make_map(&p.dout, dO, desc->dout, desc, w->heads, desc->nq))
        return ST_ERR_CUDA;
    p.qraw = raw(q, desc->q);
    p.kraw = raw(k, desc->k);
    p.vraw = raw(v, desc->v);
    p.oraw = raw(o, desc->o);
    p.doraw = raw(dO, desc->dout);
    p.dq = {static_cast<char *>(dq), desc->dq.batch * 2, desc->dq.head * 2, desc->dq.row * 2};
    p.dk = {static_cast<char *>(dk), desc->dk.batch * 2, desc->dk.head * 2, desc->dk.row * 2};
    p.dv = {static_cast<char *>(dv), desc->dv.batch * 2, desc->dv.head * 2, desc->dv.row * 2};
    p.lse = lse;
    char *ws = static_cast<char *>(workspace);
    p.delta = reinterpret_cast<float *>(ws);
    p.entries = reinterpret_cast<int2 *>(ws + z.delta);
    p.parts = reinterpret_cast<float *>(ws + z.delta + z.entries);
    p.maxima = reinterpret_cast<uint32_t *>(ws + z.delta + z.entries + z.parts);
    p.counters = reinterpret_cast<int32_t *>(ws + z.delta + z.entries + z.parts + z.maxima);
    p.nentries = u.entries;
    p.nsplit = u.split;
    p.chunk = u.chunk;
    return st::launch_window_bwd(p, desc->dtype, static_cast<int>(desc->d), stream) == cudaSuccess ? ST_OK : ST_ERR_CUDA;
}

}  // extern "C"
