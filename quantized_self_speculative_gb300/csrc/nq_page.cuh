// nq_page.cuh -- the paged KV cache's layout and the argument checks its calls
// share (see nq_page_pool and nq_page_map in nq.h).
#pragma once

#include "nq_internal.cuh"

namespace nq {

struct Pool {
    uint8_t *data;        // of the layer, or of layer 0 with layer_bytes between layers
    int N, P, H, D, NG;   // NG groups of scales per row; 0 for BF16
    uint32_t rec;         // bytes of one (page, head)
    uint32_t base_block;  // bytes of a base block (NESTED44) or of a block (BF16)
    uint32_t resid_off;   // first refinement block within a record
    size_t layer_bytes;
};
struct Map {
    int S, W, N, P;
    int32_t *table, *held, *ref;
};

// Byte o of row r among 16 rows of rb bytes of nibbles.
__host__ __device__ __forceinline__ uint32_t nib_off(int rb, int r, int o)
{
    const int q = r * (rb >> 4) + (o >> 4), line = q >> 3;
    return static_cast<uint32_t>((line << 7) + (((q & 7) ^ (2 * (line & 3))) << 4) + (o & 15));
}
// Element i of row r among 16 rows of D bf16 values.
__host__ __device__ __forceinline__ uint32_t bf_off(int D, int r, int i)
{
    return static_cast<uint32_t>(r * D + (((i >> 3) ^ (r & 7)) << 3) + (i & 7));
}

inline nq_status pool_of(const nq_page_pool *p, Pool &out, bool need_data = true)
{
    if (!p || p->layers < 1 || p->n_pages < 1 || p->heads_kv < 1) return NQ_ERR_ARG;
    if (p->format != NQ_KV_NESTED44 && p->format != NQ_KV_BF16) return NQ_ERR_ARG;
    const int P = p->page_size, D = p->head_dim, G = p->group;
    if (!(P == 16 || P == 32 || P == 64 || P == 128 || P == 256) || !(D == 64 || D == 128)) return NQ_ERR_SHAPE;
    if (p->heads_kv > 4096) return NQ_ERR_SHAPE;
    out.N = p->n_pages;
    out.P = P;
    out.H = p->heads_kv;
    out.D = D;
    if (p->format == NQ_KV_BF16) {
        out.NG = 0;
        out.base_block = 2 * 16 * D * 2;
        out.resid_off = out.rec = P / 16 * out.base_block;
    } else {
        if (!(G == 64 || G == 128) || G > D) return NQ_ERR_SHAPE;
        out.NG = D / G;
        out.base_block = 16 * D + 64 * out.NG;
        out.resid_off = P / 16 * out.base_block;
        out.rec = out.resid_off + P / 16 * (16 * D);
    }
    // layers * n_pages * heads * record must not pass 2^62 bytes
    const double all = static_cast<double>(p->layers) * out.N * out.H * out.rec;
    if (all > 4.6e18) return NQ_ERR_SHAPE;
    out.layer_bytes = static_cast<size_t>(out.N) * out.H * out.rec;
    out.data = static_cast<uint8_t *>(p->data);
    if (need_data) {
        if (!p->data) return NQ_ERR_ARG;
        if (!aligned16(p->data)) return NQ_ERR_ALIGN;
    }
    return NQ_OK;
}

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// full: held and ref are needed as well as the table
inline nq_status map_of(const nq_page_map *m, Map &out, bool full)
{
    if (!m || m->max_seqs < 1 || m->max_pages < 1 || m->n_pages < 1 || !m->table) return NQ_ERR_ARG;
    if (full && (!m->held || !m->ref)) return NQ_ERR_ARG;
    const int P = m->page_size;
    if (!(P == 16 || P == 32 || P == 64 || P == 128 || P == 256)) return NQ_ERR_SHAPE;
    // rows are int32
    if (static_cast<long long>(m->max_pages) * P > 0x7fffffffll) return NQ_ERR_SHAPE;
    if (!aligned4(m->table) || !aligned4(m->held) || !aligned4(m->ref)) return NQ_ERR_ALIGN;
    out = Map{m->max_seqs, m->max_pages, m->n_pages, P, m->table, m->held, m->ref};
    return NQ_OK;
}
// A pool and the map of its pages.
inline nq_status pool_map_of(const nq_page_pool *p, const nq_page_map *m, Pool &po, Map &mo, bool full)
{
    nq_status st = pool_of(p, po);
    if (st != NQ_OK) return st;
    st = map_of(m, mo, full);
    if (st != NQ_OK) return st;
    return p->n_pages == m->n_pages && p->page_size == m->page_size ? NQ_OK : NQ_ERR_SHAPE;
}

}  // namespace nq
