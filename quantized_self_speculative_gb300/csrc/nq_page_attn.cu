// nq_page_attn.cu -- attention of the newest rows of each sequence over the
// paged KV cache.
//
// out = sum_t p_t V_t / sum_t p_t, p_t = 2^(s_t - m), s = log2(e) f(scale q.K_t):
// one pass over the rows with the running maximum m, sum and output.  Every
// K/V byte of the view that is read comes from HBM once; that is the bound.
//
// Work.  A (sequence, kv head, tile of query vectors) is a segment; its rows
// are cut into steps of SR rows.  All steps of a call form one flat list,
// dealt out in equal runs to a persistent grid, so ragged lengths balance
// whatever they are (they are only known on the device).  The four warps of a
// CTA take every fourth step of its run; each keeps its own softmax state and
// its own ring of stages, filled by bulk copies of whole blocks that its lanes
// issue ahead, a block each, across segment borders.  At a segment's end the
// warps' states merge; a segment cut by runs leaves partial states that a second,
// dependent launch joins.  More than 16 query vectors per kv head share a CTA's decoded
// rows instead: nq_page_attn_wide.cu, nq_page_attn_tc.cu (cols_of below).
//
// Arithmetic.  S^T = K Q^T and O^T = V^T P^T on the warp MMA (m16n8k16, fp32
// accumulators) with 16 cache rows or 16 dimensions as M and 8 query vectors
// as N, so that few queries waste nothing.  P^T goes from S^T's accumulators
// to the B operand by an 8x8 transpose between lanes (movmatrix).
// NESTED44: K's codes enter undequantised, an offset nibble (q4 + 8) or byte
// (16 q4 + r + 136) in the low bits of an fp16 half (code 2^-24), placed by
// masks; the offset leaves S through the accumulators' start.  The MMA adds such
// small halves with some 18 bits, which moves a score by 10^-5 or so.  In O that
// would show where large weights meet codes of zero, so V's codes become the
// signed numbers themselves: the code under an exponent of 2^10, and one fma on
// two halves that takes 2^10 and the offset off again.  K's scales multiply S, V's
// scales multiply P before it is rounded to fp16 (one rounding, 2^-11).  So that no
// V magnitude underflows there, m follows the running maximum of s + log2(scale of
// V) and P = 2^(s - m) scale <= 2^15.
// The query is brought to a largest magnitude of 2^10 by a power of two.
// BF16: K, V and the query as they are, P rounded to bf16 (2^-8); the sum is
// taken of the rounded P, which takes most of that error out again.
//
// Measured (GB300, 2070 MHz, one query row).  bf16, 4 sequences of 40001..131072
// rows, 8 kv heads of 128: 252 us, 6.8 TB/s, the measured copy rate.  131072 rows
// x 32 kv heads of 128: 8-bit view 171 us, 6.4 TB/s (94%); 4-bit view 121 us, 4.6
// TB/s (67%), bound by instruction issue: 298 warp instructions per block of 16
// rows (placing codes, scales, softmax) would need 3.0 per cycle and SM to keep up
// with HBM; the 12 warps that registers allow reach 2.1 (MMA pipe 23% busy).  32768
// rows of the 4-bit view: 39 us, some 10 of them launch, first fills, merge and join.
#include "nq_page_attn_warp.cuh"

namespace nq {
namespace {

constexpr int kJoinWarps = 8;

// ---------------------------------------------------------------- joining
// CTA (i, v): query vector v of the segment that run i begins and later runs
// end (if there is one): out = sum_r 2^(m_r - M) o_r / sum_r 2^(m_r - M) l_r
// over the runs' partial states, eight warps taking every eighth.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
join_kernel(const __grid_constant__ AttnArgs A)
{
    constexpr int E = D / 32;
    __shared__ float sm_m[kJoinWarps], sm_l[kJoinWarps], sm_o[kJoinWarps][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 in = A.info[blockIdx.x];
    if (in.x < 0) return;
    const int kvh = in.y / A.QT, v = (in.y % A.QT) * A.cols + blockIdx.y;
    if (v >= A.M * A.G) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = blockIdx.x, n = in.z - first + 1;
    float m = -INFINITY, l = 0.0f, o[E] = {};
    constexpr int U = 4;
    for (int r0 = warp; r0 < n; r0 += kJoinWarps * U) {
        float mm[U], ll[U], oo[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * kJoinWarps;
            mm[u] = -INFINITY;
            ll[u] = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) oo[u][e] = 0.0f;
            if (r < n) {
                const size_t at = (2 * static_cast<size_t>(first + r) + (r == 0 ? 1 : 0)) * A.cols + blockIdx.y;
                mm[u] = A.part_ml[at * 2];
                ll[u] = A.part_ml[at * 2 + 1];
                const float *p = A.part_o + at * D + lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) oo[u][e] = p[e];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float mn = fmaxf(m, mm[u]), mz = mn == -INFINITY ? 0.0f : mn, a = ex2(m - mz), f = ex2(mm[u] - mz);
            l = l * a + ll[u] * f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = o[e] * a + oo[u][e] * f;
            m = mn;
        }
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
    __syncthreads();
    if (threadIdx.x >= D / 2) return;
    float M2 = -INFINITY, x0 = 0.0f, x1 = 0.0f, den = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) M2 = fmaxf(M2, sm_m[w]);
    if (M2 == -INFINITY) M2 = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        const float f = ex2(sm_m[w] - M2);
        x0 = fmaf(f, sm_o[w][2 * threadIdx.x], x0);
        x1 = fmaf(f, sm_o[w][2 * threadIdx.x + 1], x1);
        den = fmaf(f, sm_l[w], den);
    }
    const float f = den == 0.0f ? 0.0f : 1.0f / den;
    const int mv = row_of_vector(A, v);
    const size_t row = (static_cast<size_t>(in.x) * A.M + mv) * A.Hq + kvh * A.G + v - mv * A.G;
    reinterpret_cast<uint32_t *>(A.out + row * D)[threadIdx.x] = pack_b(x0 * f, x1 * f);
}

// The same for trees, whose segments have many vectors: CTA (i, v) takes eight of them.  Of a
// segment in a few parts a warp takes a vector (a CTA per vector takes 29 us for 128 segments
// of 128 vectors in two or three parts each); of one in many the warps share each vector's.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
join_tree_kernel(const __grid_constant__ AttnArgs A)
{
    constexpr int E = D / 32, U = 4;
    __shared__ float sm_m[kJoinWarps][kJoinWarps], sm_l[kJoinWarps][kJoinWarps];
    __shared__ __align__(16) float sm_o[kJoinWarps][kJoinWarps][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 in = A.info[blockIdx.x];
    if (in.x < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = blockIdx.x, n = in.z - first + 1;
    const int kvh = in.y / A.QT, c0 = blockIdx.y * kJoinWarps, v0 = (in.y % A.QT) * A.cols, nv = min(A.cols, A.M * A.G - v0);
    struct State {
        float m, l, o[E];
    };
    auto add = [](State &s, float m, float l, const float (&o)[E]) {
        const float mn = fmaxf(s.m, m), mz = mn == -INFINITY ? 0.0f : mn, a = ex2(s.m - mz), f = ex2(m - mz);
        s.l = s.l * a + l * f;
#pragma unroll
        for (int e = 0; e < E; ++e) s.o[e] = s.o[e] * a + o[e] * f;
        s.m = mn;
    };
    auto parts = [&](int col, int r0, int step) {                // of parts r0, r0 + step, ..
        State s = {-INFINITY, 0.0f, {}};
        for (; r0 < n; r0 += U * step) {
            float mm[U], ll[U], oo[U][E];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * step;
                mm[u] = -INFINITY;
                ll[u] = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) oo[u][e] = 0.0f;
                if (r < n) {
                    const size_t at = (2 * static_cast<size_t>(first + r) + (r == 0 ? 1 : 0)) * A.cols + col;
                    const float2 ml = *reinterpret_cast<const float2 *>(A.part_ml + at * 2);
                    mm[u] = ml.x;
                    ll[u] = ml.y;
                    const float *p = A.part_o + at * D + lane * E;
#pragma unroll
                    for (int e = 0; e < E; ++e) oo[u][e] = p[e];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) add(s, mm[u], ll[u], oo[u]);
        }
        return s;
    };
    State s;
    if (n <= 2 * kJoinWarps) {
        if (c0 + warp >= nv) return;
        s = parts(c0 + warp, 0, 1);
    } else {
#pragma unroll 1
        for (int j = 0; j < kJoinWarps && c0 + j < nv; ++j) {
            s = parts(c0 + j, warp, kJoinWarps);
            if (lane == 0) {
                sm_m[j][warp] = s.m;
                sm_l[j][warp] = s.l;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) sm_o[j][warp][lane * E + e] = s.o[e];
        }
        __syncthreads();
        if (c0 + warp >= nv) return;
        s = {-INFINITY, 0.0f, {}};
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            float o[E];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = sm_o[warp][w][lane * E + e];
            add(s, sm_m[warp][w], sm_l[warp][w], o);
        }
    }
    const float f = s.l == 0.0f ? 0.0f : 1.0f / s.l;
    const int v = v0 + c0 + warp, mv = row_of_vector(A, v);
    uint32_t *to = reinterpret_cast<uint32_t *>(A.out + ((static_cast<size_t>(in.x) * A.M + mv) * A.Hq + kvh * A.G + v - mv * A.G) * D) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E; e += 2) to[e / 2] = pack_b(s.o[e] * f, s.o[e + 1] * f);
}

// ---------------------------------------------------------------- host side
cudaError_t launch_join(const AttnArgs &A, int grid, cudaStream_t s)
{
    // a programmatic dependent launch: it overlaps the end of the kernel before it
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int vectors = A.M * A.G < A.cols ? A.M * A.G : A.cols;
    const bool tree = A.tree_bits != nullptr;
    cfg.gridDim = dim3(grid, tree ? (vectors + kJoinWarps - 1) / kJoinWarps : vectors);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (tree) return cudaLaunchKernelEx(&cfg, A.p.D == 128 ? join_tree_kernel<128> : join_tree_kernel<64>, A);
    return cudaLaunchKernelEx(&cfg, A.p.D == 128 ? join_kernel<128> : join_kernel<64>, A);
}

// Columns (query vectors) per tile.  Up to 16 a warp holds them all and decodes
// for itself (16 vectors, 16 ragged sequences of the 8-bit view: 38 us against 53
// with a CTA's shared decoding; 5 to 16 vectors, all formats and head sizes: 0.5 to
// 0.9 of its time).  More share a CTA's decoded steps, 8 columns per warp, or
// the tensor cores where a row of the cache has one scale: these from 25 vectors
// on for heads of 128, from 33 on for heads of 64, whose steps decode half as much
// beside the same softmax.  us on the tensor cores / per warp, 8 kv heads, 8-bit
// view (the 4-bit view is alike):
//                        heads of 128: 24       28       32       36   heads of 64: 28       32       36
//   16 of 500..4000 rows       64 / 62  66 / 69  66 / 71  68 / 88       57 / 47  58 / 49  58 / 65
//   one of 32768 rows          46 / 49  46 / 55  47 / 56  47 / 67       41 / 38  42 / 40  42 / 50
bool tensor_cores(int vectors, int fmt, int ng, int D) { return vectors > (D == 64 ? 32 : 24) && fmt != kBf16 && ng == 1; }
int cols_of(int vectors, bool tc)
{
    if (tc) return vectors < 128 ? (vectors + 7) / 8 * 8 : 128;
    return vectors <= 8 ? 8 : vectors <= 16 ? 16 : vectors <= 32 ? 32 : 64;
}

// Trees have a tensor-core kernel of their own, which takes more than 16 vectors of a cache
// with one scale per row.  us on the tensor cores / per CTA, 8 kv heads, 4-bit | 8-bit view:
//                        heads of 128: 20               24       heads of 64: 20                24
//   16 of 500..4000 rows       47 / 62 | 49 / 66  47 / 63 | 49 / 68   39 / 37 | 41 / 41   39 / 39 | 41 / 41
//   one of 32768 rows          41 / 64 | 43 / 67  41 / 65 | 43 / 68   35 / 44 | 36 / 46   35 / 45 | 37 / 47
// on the tensor cores / per warp:
//                        heads of 128: 9                16       heads of 64: 9                 16
//   16 of 500..4000 rows       46 / 35 | 48 / 39  46 / 37 | 49 / 41   38 / 29 | 39 / 31   39 / 30 | 39 / 32
//   one of 32768 rows          41 / 39 | 43 / 43  41 / 39 | 43 / 43   35 / 32 | 35 / 35   35 / 33 | 35 / 35
//   one of 533, 32 kv heads                              - | 23 / 20
// (Plain scores.  Capped ones cost the tensor-core kernel more, see there.)
bool tree_tensor_cores(int vectors, int fmt, int ng) { return vectors > 16 && fmt != kBf16 && ng == 1; }
// Its tiles hold up to 256 vectors, even shares of what there is.
int tree_cols(int vectors, bool tc)
{
    const int tiles = (vectors + 255) / 256;
    return tc ? ((vectors + tiles - 1) / tiles + 7) / 8 * 8 : cols_of(vectors, false);
}

// Workspace: info, then partial states of two segments per CTA; enough for any
// of the kernels (4 CTAs per SM and 32 columns, 2 and 64, 1 and 128, ..).
struct Ws {
    size_t ml, o, total;
};
Ws ws_of(int vectors, int D, bool tree)
{
    const size_t ctas = 4 * static_cast<size_t>(sm_count()),
                 cols = 2 * static_cast<size_t>(sm_count()) * (vectors <= 8 ? 32 : vectors <= 16 ? 48 : tree && vectors > 128 ? 256 : 128);
    Ws w;
    w.ml = ctas * sizeof(int4);
    w.o = w.ml + cols * 8;
    w.total = w.o + cols * D * 4;
    return w;
}

}  // namespace
}  // namespace nq

extern "C" size_t nq_page_attn_workspace_bytes(int M, int heads_q, int heads_kv, int head_dim)
{
    if (M < 1 || heads_kv < 1 || heads_q < heads_kv || heads_q % heads_kv != 0 || !(head_dim == 64 || head_dim == 128)) return 0;
    if (static_cast<long long>(M) * (heads_q / heads_kv) > 65536) return 0;
    return nq::ws_of(M * (heads_q / heads_kv), head_dim, false).total;
}

// starve and wait_ns as in AttnArgs
static nq_status page_attn(const nq_page_pool *pool, int layer, const nq_page_map *map, const uint16_t *q, int64_t q_stride,
                           int batch, int M, int heads_q, const int32_t *seqs, const int32_t *len, int planes,
                           const nq_attn_opts *opts, const nq_tree *tree, uint16_t *out, void *ws, size_t ws_bytes, cudaStream_t stream,
                           int starve, unsigned long long wait_ns)
{
    nq::AttnArgs A{};
    const nq_status st = nq::pool_map_of(pool, map, A.p, A.m, false);
    if (st != NQ_OK) return st;
    const nq::Pool &p = A.p;
    if (layer < 0 || layer >= pool->layers || !q || !len || !out || !opts || batch < 1 || M < 1) return NQ_ERR_ARG;
    if (heads_q < p.H || heads_q % p.H != 0 || (planes != 1 && planes != 2) || (!seqs && batch > A.m.S)) return NQ_ERR_ARG;
    if (!(opts->scale > 0.0f && opts->scale <= 3.4028235e38f) || opts->window < 0) return NQ_ERR_ARG;
    if (opts->softcap != 0.0f && !(opts->softcap >= 0x1p-100f && opts->softcap <= 0x1p100f)) return NQ_ERR_ARG;
    if (tree && tree->window != opts->window) return NQ_ERR_ARG;
    const int G = heads_q / p.H;
    if (static_cast<long long>(M) * G > 65536) return NQ_ERR_SHAPE;
    if (q_stride < static_cast<int64_t>(heads_q) * p.D || q_stride % 8 != 0) return NQ_ERR_SHAPE;
    if (!nq::aligned16(q) || !nq::aligned16(out) || !nq::aligned16(ws) || !nq::aligned4(seqs) || !nq::aligned4(len) ||
        !nq::aligned4(opts->slopes))
        return NQ_ERR_ALIGN;
    const nq::Ws w = nq::ws_of(M * G, p.D, tree != nullptr);
    if (!ws || ws_bytes < w.total) return NQ_ERR_WORKSPACE;
    A.status = nq::device_status_ptr();
    if (!A.status) return NQ_ERR_CUDA;
    A.p.data += static_cast<size_t>(layer) * p.layer_bytes;
    A.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    A.q_stride = q_stride;
    A.B = batch;
    A.M = M;
    A.Hq = heads_q;
    A.G = G;
    A.g_mul = static_cast<unsigned>((0x100000000ull + G - 1) / G);
    const int fmt = p.NG == 0 ? nq::kBf16 : planes == 1 ? nq::kKv4 : nq::kKv8;
    const bool tc = tree ? nq::tree_tensor_cores(M * G, fmt, p.NG) : nq::tensor_cores(M * G, fmt, p.NG, p.D);
    const int cols = A.cols = tree ? nq::tree_cols(M * G, tc) : nq::cols_of(M * G, tc);
    A.QT = (M * G + cols - 1) / cols;
    // the kernel numbers the steps of all segments in 32 bits
    if (static_cast<double>(batch) * p.H * A.QT * (static_cast<double>(A.m.W) * A.m.P / 16 + 2) > 2.0e9) return NQ_ERR_SHAPE;
    // (trees count the begin and end of a segment as steps as well)
    if (tree && static_cast<double>(batch) * p.H * A.QT * (static_cast<double>(A.m.W) * A.m.P / 64 + 12) > 2.0e9) return NQ_ERR_SHAPE;
    A.seqs = seqs;
    A.len = len;
    A.scale = opts->scale;
    A.softcap = opts->softcap;
    A.window = opts->window;
    A.slopes = opts->slopes;
    A.out = reinterpret_cast<__nv_bfloat16 *>(out);
    A.wait_ns = wait_ns;
    A.starve = starve;
    if (tree) {
        A.tree_bits = tree->bits;
        A.tree_depth = tree->depth;
        A.tree_words = (M + 31) / 32;
    }
    uint8_t *wb = static_cast<uint8_t *>(ws);
    A.info = reinterpret_cast<int4 *>(wb);
    A.part_ml = reinterpret_cast<float *>(wb + w.ml);
    A.part_o = reinterpret_cast<float *>(wb + w.o);
    int grid = 0;
    cudaError_t e;
    if (tree && tc) e = nq::attn_tree_tc(fmt, A, stream, &grid);
    else if (tree) e = cols > 16 ? nq::attn_tree_wide(fmt, A, stream, &grid) : nq::attn_tree(fmt, A, stream, &grid);
    else if (tc) e = nq::attn_tc(fmt, A, stream, &grid);
    else if (cols > 16) e = nq::attn_wide(fmt, A, stream, &grid);
    else if (fmt == nq::kBf16) e = nq::launch_d<nq::kBf16, false>(cols / 8, A, stream, &grid);
    else if (fmt == nq::kKv4) e = nq::launch_d<nq::kKv4, false>(cols / 8, A, stream, &grid);
    else e = nq::launch_d<nq::kKv8, false>(cols / 8, A, stream, &grid);
    if (e != cudaSuccess) return NQ_ERR_CUDA;
    return nq::cuda_status(nq::launch_join(A, grid, stream));
}

extern "C" nq_status nq_page_attn(const nq_page_pool *pool, int layer, const nq_page_map *map, const uint16_t *q,
                                  int64_t q_stride, int batch, int M, int heads_q, const int32_t *seqs,
                                  const int32_t *len, int planes, const nq_attn_opts *opts, uint16_t *out, void *ws,
                                  size_t ws_bytes, cudaStream_t stream)
{
    return page_attn(pool, layer, map, q, q_stride, batch, M, heads_q, seqs, len, planes, opts, nullptr, out, ws, ws_bytes, stream, -1,
                     nq::kWaitNs);
}

extern "C" size_t nq_page_attn_tree_workspace_bytes(int nodes, int heads_q, int heads_kv, int head_dim)
{
    if (nodes > nq::kMaxNodes || nq_page_attn_workspace_bytes(nodes, heads_q, heads_kv, head_dim) == 0) return 0;
    return nq::ws_of(nodes * (heads_q / heads_kv), head_dim, true).total;
}

extern "C" nq_status nq_page_attn_tree(const nq_page_pool *pool, int layer, const nq_page_map *map, const uint16_t *q,
                                       int64_t q_stride, int heads_q, const int32_t *seqs, const int32_t *len, int planes,
                                       const nq_attn_opts *opts, const nq_tree *tree, uint16_t *out, void *ws,
                                       size_t ws_bytes, cudaStream_t stream)
{
    const nq_status st = nq::tree_of(tree);
    if (st != NQ_OK) return st;
    return page_attn(pool, layer, map, q, q_stride, tree->batch, tree->nodes, heads_q, seqs, len, planes, opts, tree, out, ws, ws_bytes, stream,
                     -1, nq::kWaitNs);
}

extern "C" nq_status nq_selftest_page_attn(const nq_page_pool *pool, int layer, const nq_page_map *map, const uint16_t *q,
                                           int64_t q_stride, int batch, int M, int heads_q, const int32_t *seqs,
                                           const int32_t *len, int planes, const nq_attn_opts *opts, uint16_t *out, void *ws,
                                           size_t ws_bytes, int steps, uint32_t limit_us, cudaStream_t stream)
{
    if (steps < 0 || limit_us < 1 || limit_us > 1000000u) return NQ_ERR_ARG;
    return page_attn(pool, layer, map, q, q_stride, batch, M, heads_q, seqs, len, planes, opts, nullptr, out, ws, ws_bytes, stream, steps,
                     limit_us * 1000ull);
}

extern "C" nq_status nq_selftest_page_attn_tree(const nq_page_pool *pool, int layer, const nq_page_map *map, const uint16_t *q,
                                                int64_t q_stride, int heads_q, const int32_t *seqs, const int32_t *len, int planes,
                                                const nq_attn_opts *opts, const nq_tree *tree, uint16_t *out, void *ws,
                                                size_t ws_bytes, int steps, uint32_t limit_us, cudaStream_t stream)
{
    if (steps < 0 || limit_us < 1 || limit_us > 1000000u) return NQ_ERR_ARG;
    const nq_status st = nq::tree_of(tree);
    if (st != NQ_OK) return st;
    return page_attn(pool, layer, map, q, q_stride, tree->batch, tree->nodes, heads_q, seqs, len, planes, opts, tree, out, ws, ws_bytes, stream,
                     steps, limit_us * 1000ull);
}
