// pn_attend.hip -- pn_attend's arguments, how a call is cut into workgroups, and its entry points.
// The kernels are in pn_attend.h.
#include "pn_attend.h"

namespace pn {

template <>
int launch_format<PN_CACHE_MXFP8>(const AttendArgs &A, int dim, int parts, hipStream_t s);
template <>
int launch_format<PN_CACHE_MXFP4>(const AttendArgs &A, int dim, int parts, hipStream_t s);

static int parts_of(int type) { return type == PN_BF16 ? 1 : type == PN_F16 ? 2 : 3; }

// How a call is cut: rows a wave or workgroup holds, row blocks and token ranges (as in AttendArgs).
struct Cut {
    int shared_tiles, prefix_tiles, own_tiles;
    int prefix_splits, prefix_blocks, own_splits, own_blocks;
    bool direct;
    int64_t rows;
    int64_t workspace;
};

static int attend_check(const pn_cache *cache, const pn_attend_args *a, CacheView &c)
{
    const int st = cache_view(cache, c);
    if (st != PN_OK)
        return st;
    if (!a)
        return PN_ERR_NULL;
    if (elem_bytes(a->type) == 0)
        return PN_ERR_FORMAT;
    const int64_t most = INT32_MAX - 64;  // tokens, rows and workgroups are counted in 32 bits
    if (a->B < 0 || a->Q < 0 || a->Hq < 1 || a->Hq % cache->heads || a->table_width < 0 ||
        a->prefix_len < 0 || a->prefix_len > most || (int64_t)a->table_width * cache->page > most ||
        !isfinite(a->scale))
        return PN_ERR_SHAPE;
    if ((int64_t)a->B * a->Q > most / a->Hq)
        return PN_ERR_SHAPE;
    return PN_OK;
}

static Cut attend_cut(const pn_cache *cache, const pn_attend_args *a)
{
    const int G = a->Hq / cache->heads;
    Cut t = {};
    const int64_t own_rows = (int64_t)a->Q * G, prefix_rows = own_rows * a->B;
    const int64_t own_records = (int64_t)a->table_width * (cache->page / kTile);
    const int64_t prefix_records = (a->prefix_len + kTile - 1) / kTile;
    // One workgroup a CU: what 256 channels (134 KB of LDS) and 32 rows a wave (over 128 registers) leave
    // room for. Of the smaller ones two would fit; cutting for two is not measured.
    const int64_t cus = device_cus();
    const auto stream_tiles = [](int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; };
    const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    t.own_tiles = stream_tiles(own_rows);
    t.own_blocks = (int)up(own_rows, 16 * t.own_tiles);
    // At least one record a wave. One range in all is written out at once; the second kernel that joins
    // several takes 4 to 5 us with its launch, what a wave needs for about 512 / (dim * parts) records:
    // 16 sequences of up to 777 tokens, 128 channels, bf16 9.3 us in one range, 8.5 + 4.7 in two; one of
    // 1000 tokens, 256 channels, fp32 16.5 us in one, 9.6 + 3.7 in four.
    const int64_t a_wave = up(own_records * t.own_tiles, kWaves);
    const bool one = prefix_records == 0 && a_wave * cache->dim * parts_of(a->type) <= 512;
    t.own_splits = one ? 1
                       : (int)std::max<int64_t>(1, std::min(up(cus, (int64_t)a->B * cache->heads * t.own_blocks),
                                                            a_wave));
    if (prefix_records > 0 && prefix_rows <= 64) {
        t.prefix_tiles = stream_tiles(prefix_rows);
        t.prefix_blocks = 1;
        t.prefix_splits = (int)std::min(up(cus, cache->heads), up(prefix_records * t.prefix_tiles, kWaves));
    } else if (prefix_records > 0) {
        const int most = shared_tiles(cache->dim, parts_of(a->type));
        t.shared_tiles = prefix_rows <= 128 ? 1 : prefix_rows <= 256 ? std::min(2, most) : most;
        t.prefix_blocks = (int)up(prefix_rows, 128 * t.shared_tiles);
        // one round of workgroups, at least eight records each
        t.prefix_splits = (int)std::max<int64_t>(1, std::min(cus / ((int64_t)cache->heads * t.prefix_blocks),
                                                             up(prefix_records, 8)));
    }
    t.direct = t.own_splits + t.prefix_splits == 1;
    t.rows = (int64_t)a->B * a->Q * a->Hq;
    t.workspace = t.direct ? 0 : (t.own_splits + t.prefix_splits) * t.rows * (cache->dim + 2) * 4;
    return t;
}

}  // namespace pn

using namespace pn;

extern "C" int64_t pn_attend_workspace_bytes(const pn_cache *cache, const pn_attend_args *a)
{
    CacheView c;
    if (attend_check(cache, a, c) != PN_OK || a->B == 0 || a->Q == 0)
        return 0;
    return attend_cut(cache, a).workspace;
}

extern "C" int pn_attend(const pn_cache *cache, const pn_attend_args *a, void *workspace,
                         int64_t workspace_bytes, void *stream)
{
    CacheView c;
    int st = attend_check(cache, a, c);
    if (st != PN_OK)
        return st;
    if (a->B == 0 || a->Q == 0)
        return PN_OK;
    const int size = elem_bytes(a->type);
    if (!a->q || !a->out || !a->lens || (a->table_width > 0 && !a->table) ||
        (a->prefix_len > 0 && !a->prefix_table))
        return PN_ERR_NULL;
    if (!aligned(a->q, size) || !aligned(a->out, 16) || !aligned(a->lens, 4) ||
        !aligned(a->table, 4) || !aligned(a->prefix_table, 4) || !aligned(a->q_lens, 4) ||
        !aligned(a->lse, 4))
        return PN_ERR_ALIGN;
    if (c.pages == 0 && (a->table_width > 0 || a->prefix_len > 0))
        return PN_ERR_SHAPE;  // no page to read
    const Cut t = attend_cut(cache, a);
    if (t.workspace > 0) {
        if (!workspace)
            return PN_ERR_NULL;
        if (!aligned(workspace, 16))
            return PN_ERR_ALIGN;
        if (workspace_bytes < t.workspace)
            return PN_ERR_WORKSPACE;
    }
    if ((st = check_device()) != PN_OK)
        return st;
    AttendArgs A;
    A.c = c;
    A.type = a->type;
    A.B = a->B;
    A.Q = a->Q;
    A.Hq = a->Hq;
    A.G = a->Hq / cache->heads;
    A.by_G = FastDiv(A.G);
    A.by_Q = FastDiv(A.Q);
    A.by_Hq = FastDiv(A.Hq);
    A.q = a->q;
    A.q_seq = a->q_seq_stride;
    A.q_tok = a->q_token_stride;
    A.q_head = a->q_head_stride;
    A.q_vec = aligned(a->q, 4 * size) && ((A.q_seq | A.q_tok | A.q_head) & 3) == 0;
    // a scale of zero and one that log2(e) would take past fp32 are made up in q, exactly
    const float by = fabsf(a->scale), more = by > 0x1p126f ? 2.0f : 1.0f;
    A.scale = fmaxf(by / more * kLog2e, 0x1p-126f);
    A.factor = a->scale > 0.0f ? more : a->scale < 0.0f ? -more : 0.0f;
    A.table = a->table;
    A.table_stride = a->table_stride;
    A.table_width = a->table_width;
    A.lens = a->lens;
    A.q_lens = a->q_lens;
    A.prefix_table = a->prefix_table;
    A.prefix_len = (int)a->prefix_len;
    A.shared_tiles = t.shared_tiles;
    A.prefix_tiles = t.prefix_tiles;
    A.own_tiles = t.own_tiles;
    A.prefix_splits = t.prefix_splits;
    A.prefix_blocks = t.prefix_blocks;
    A.own_splits = t.own_splits;
    A.own_blocks = t.own_blocks;
    A.direct = t.direct;
    A.part = (float *)workspace;
    A.part_ml = (float2 *)((float *)workspace + (int64_t)(t.own_splits + t.prefix_splits) * t.rows * cache->dim);
    A.out = a->out;
    A.lse = a->lse;
    hipStream_t s = (hipStream_t)stream;
    return cache->format == PN_CACHE_MXFP8
               ? launch_format<PN_CACHE_MXFP8>(A, cache->dim, parts_of(a->type), s)
               : launch_format<PN_CACHE_MXFP4>(A, cache->dim, parts_of(a->type), s);
}
