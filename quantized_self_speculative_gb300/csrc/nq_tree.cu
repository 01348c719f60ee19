// nq_tree.cu -- trees of drafted tokens: their masks and depths, greedy
// acceptance along them, and keeping the accepted path's rows in the paged cache.
//
// Plan.  Node m's set is itself and what lies on the way up to the committed
// rows: a walk along parents, one thread per node, in shared memory.  As parents
// have lower numbers than their children the walk meets the set's bits from the
// highest word to the lowest, so each word is formed in a register and written
// once.
//
// Acceptance.  t_m = argmax of node m's logits; the walk starts at node 0 and
// goes on to the lowest child whose token is t of its parent.  Only the logits
// rows of the walk are read (an argmax of all nodes would read nodes / length
// times as much), one after another: a cluster of CTAs shares a row, so that one
// sequence has eight SMs' loads in flight, and every CTA learns the winner
// through distributed shared memory with one cluster barrier per row.
//
// Keep.  Row first + path[j] moves to row first + j.  path rises, so a row that is
// written is never read by a later move; a warp takes one (sequence, layer, head),
// reads a batch of rows into registers and then writes them.
//
// Measured (GB300): plan and acceptance of 64 trees over 152064 words, walks of up to
// eight nodes: 55 us (122 MB, 18 us at the copy rate; rows of a walk follow each other);
// of one tree over 32000 words, five nodes: 16 us.  Keep of 16 paths, 32 layers x 32
// heads: 12 us, of one path x 8 heads: 6 us, bound by its chain of dependent loads.
#include "nq_page.cuh"

namespace nq {
namespace {

// ---------------------------------------------------------------- plan
__global__ void __launch_bounds__(kMaxNodes)
plan_kernel(const int32_t *__restrict__ parents, int M, int words, int window, int32_t *__restrict__ depth,
            uint32_t *__restrict__ bits, unsigned int *status)
{
    __shared__ int up[kMaxNodes];
    const size_t at = static_cast<size_t>(blockIdx.x) * M;
    const int m = threadIdx.x;
    if (m < M) up[m] = parents[at + m];
    __syncthreads();
    if (m >= M) return;
    // down to -1 the chain is a node's way to the committed rows; any other end leaves the node unused
    int d = -1, cur = m;
    bool bad = false;
    while (cur >= 0) {
        const int p = up[cur];
        ++d;
        bad = p >= cur || (p < -1 && cur != m);
        cur = bad ? -2 : p;
    }
    if (bad) set_status(status, NQ_DEV_BAD_TREE);
    const bool used = cur == -1;
    depth[at + m] = used ? d : -1;
    uint32_t *row = bits + (at + m) * words;
    int left = used ? (window > 0 ? window : kMaxNodes) : 0;     // nodes of the set that the window holds
    cur = m;
    for (int w = words - 1; w >= 0; --w) {
        uint32_t x = 0;
        for (; left > 0 && cur >= 32 * w; cur = up[cur], --left) x |= 1u << (cur & 31);
        row[w] = x;
    }
}

// ---------------------------------------------------------------- acceptance
constexpr int kAccCluster = 8;            // the portable size
constexpr int kAccThreads = 256;
constexpr int kAccUnroll = 8;             // 16-byte loads in flight per thread

// Larger is better: the value in order (the zeros alike), then the lower index.  NaN is below all.
__device__ __forceinline__ unsigned long long order_of(float x, int i)
{
    const uint32_t u = __float_as_uint(x + 0.0f), k = x != x ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
    return (static_cast<unsigned long long>(k) << 32) | static_cast<uint32_t>(~i);
}
__device__ __forceinline__ unsigned long long shfl_max(unsigned long long v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long y = __shfl_xor_sync(0xffffffffu, v, o);
        v = y > v ? y : v;
    }
    return v;
}
__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__global__ void __launch_bounds__(kAccThreads, 4)
accept_tree_kernel(const int32_t *__restrict__ parents, const int32_t *__restrict__ depth, const int32_t *__restrict__ tokens,
                   const float *__restrict__ logits, int M, int V, int width, int32_t *__restrict__ out_tok,
                   int32_t *__restrict__ out_cnt, int32_t *__restrict__ path, unsigned int *status)
{
    __shared__ int up[kMaxNodes], tok[kMaxNodes];
    __shared__ unsigned long long part[kAccThreads / 32], slot[2][16];
    __shared__ int child[2];
    uint32_t ctas, rank;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int b = blockIdx.x / ctas, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t at = static_cast<size_t>(b) * M;
    bool bad_token = false;
    for (int m = threadIdx.x; m < M; m += kAccThreads) {
        const bool used = depth[at + m] >= 0;
        up[m] = used ? parents[at + m] : -2;
        tok[m] = tokens[at + m];
        bad_token |= used && m > 0 && static_cast<unsigned>(tok[m]) >= static_cast<unsigned>(V);
    }
    if (rank == 0) {
        if (bad_token) set_status(status, NQ_DEV_BAD_TOKEN);
        for (int j = threadIdx.x; j < width; j += kAccThreads) {
            out_tok[static_cast<size_t>(b) * width + j] = -1;
            path[static_cast<size_t>(b) * width + j] = -1;
        }
    }
    if (threadIdx.x < 2) child[threadIdx.x] = 0x7fffffff;
    // also: every CTA of the cluster runs before another writes into its shared memory
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
    bool odd = false;                     // a logit that is not finite
    int cur = up[0] >= -1 ? 0 : -1, n = 0;
    for (; cur >= 0; ++n) {
        // ---- this CTA's share of the row: 16-byte units of the whole array, of which the first and last may be cut
        const size_t f0 = (at + cur) * static_cast<size_t>(V), f1 = f0 + V;
        const size_t u0 = f0 >> 2, units = ((f1 + 3) >> 2) - u0, per = (units + ctas - 1) / ctas;
        const size_t lo = u0 + min(per * rank, units), hi = u0 + min(per * (rank + 1), units);
        unsigned long long best = 0;
        auto take = [&](float x, size_t f) {
            odd |= !(fabsf(x) <= 3.4028235e38f);
            const unsigned long long k = order_of(x, static_cast<int>(f - f0));
            best = k > best ? k : best;
        };
        // units wholly within the row: at most the first and the last are not
        const size_t in0 = max(lo, (f0 + 3) >> 2), in1 = min(hi, f1 >> 2);
        if (threadIdx.x == 0) {
            for (size_t u = lo; u < min(in0, hi); ++u)
                for (size_t f = max(4 * u, f0); f < min(4 * u + 4, f1); ++f) take(logits[f], f);
            for (size_t u = max(in1, in0); u < hi; ++u)
                for (size_t f = max(4 * u, f0); f < min(4 * u + 4, f1); ++f) take(logits[f], f);
        }
        for (size_t u = in0 + threadIdx.x; u < in1; u += kAccUnroll * kAccThreads) {
            float4 x[kAccUnroll];
#pragma unroll
            for (int i = 0; i < kAccUnroll; ++i) {
                x[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (u + i * kAccThreads < in1) x[i] = __ldcs(reinterpret_cast<const float4 *>(logits) + u + i * kAccThreads);
            }
#pragma unroll
            for (int i = 0; i < kAccUnroll; ++i) {
                if (u + i * kAccThreads >= in1) break;
                // the first of the four that equals their largest; NaN leaves fmaxf, and is looked for apart
                const float top = fmaxf(fmaxf(x[i].x, x[i].y), fmaxf(x[i].z, x[i].w));
                const int e = x[i].x == top ? 0 : x[i].y == top ? 1 : x[i].z == top ? 2 : 3;
                odd |= !(fabsf(x[i].x) <= 3.4028235e38f) || !(fabsf(x[i].y) <= 3.4028235e38f) ||
                       !(fabsf(x[i].z) <= 3.4028235e38f) || !(fabsf(x[i].w) <= 3.4028235e38f);
                const unsigned long long k = order_of(top, static_cast<int>(4 * (u + i * kAccThreads) + e - f0));
                best = k > best ? k : best;
            }
        }
        best = shfl_max(best);
        if (lane == 0) part[warp] = best;
        __syncthreads();
        if (warp == 0) {
            best = shfl_max(lane < kAccThreads / 32 ? part[lane] : 0);
            if (lane < ctas) {            // to slot [n & 1][rank] of CTA `lane`
                uint32_t to;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_addr(&slot[n & 1][rank])), "r"(lane));
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(best) : "memory");
            }
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        best = shfl_max(lane < ctas ? slot[n & 1][lane] : 0);
        const int t = static_cast<int>(~static_cast<uint32_t>(best));
        if (rank == 0 && threadIdx.x == 0) {
            out_tok[static_cast<size_t>(b) * width + n] = t;
            path[static_cast<size_t>(b) * width + n] = cur;
        }
        if (n + 1 == width) {
            ++n;
            break;
        }
        // ---- the lowest child with that token (children have higher numbers)
        for (int m = cur + 1 + threadIdx.x; m < M; m += kAccThreads)
            if (up[m] == cur && tok[m] == t) {
                atomicMin(&child[n & 1], m);
                break;
            }
        __syncthreads();
        const int next = child[n & 1];
        if (threadIdx.x == 0) child[(n + 1) & 1] = 0x7fffffff;   // of the next row: read last before the barrier above
        cur = next == 0x7fffffff ? -1 : next;
    }
    if (odd) set_status(status, NQ_DEV_NONFINITE);
    if (rank == 0 && threadIdx.x == 0) out_cnt[b] = n;
    // no CTA leaves while another may still write into its shared memory: all writes lie before the last barrier
}

// ---------------------------------------------------------------- keep
constexpr int kKeepWarps = 8;

struct RowAt {
    uint8_t *rec;         // of head 0
    int r;                // row within the page
};

template <int D, int NG>  // NG = 0: BF16
__global__ void __launch_bounds__(kKeepWarps * 32)
keep_kernel(Pool p, Map m, const int32_t *__restrict__ seqs, const int32_t *__restrict__ first, const int32_t *__restrict__ path,
            const int32_t *__restrict__ count, int n, int width, int layers, unsigned int *status)
{
    constexpr int RB = NG ? D / 2 : 2 * D;                       // bytes of a K (or V) row of one plane
    constexpr int CH = RB / 16, PARTS = NG ? 4 : 2;              // 16-byte chunks of one; K, V (and their refinement)
    constexpr int CPR = CH * PARTS, BATCH = 128 / CPR;           // chunks per row; rows that four registers per lane hold
    constexpr int NS = NG ? NG : 1;
    static_assert(BATCH * 2 * NS <= 32, "a lane holds at most one scale");
    const long long wi = static_cast<long long>(blockIdx.x) * kKeepWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, per = layers * p.H;
    const long long s = wi / per;
    if (s >= n) return;
    const int lh = static_cast<int>(wi - s * per), layer = lh / p.H, h = lh - layer * p.H;
    const bool report = lh == 0;
    const int lp = 31 - __clz(m.P);
    const int slot = seqs[s], base = first[s], cnt = count[s];
    const int32_t *pt = path + s * width;
    if (slot < 0 || slot >= m.S || base < 0 || cnt < 0 || cnt > width) {
        if (report && lane == 0) set_status(status, NQ_DEV_BAD_PAGE);
        return;
    }
    // a path that does not rise is left out whole
    bool bad = false;
    int j0 = cnt;                                                // the first row that does not lie where it belongs
    for (int j = lane; j < cnt; j += 32) {
        bad |= pt[j] < 0 || (j > 0 && pt[j] <= pt[j - 1]);
        if (pt[j] != j) j0 = min(j0, j);
    }
    j0 = __reduce_min_sync(0xffffffffu, j0);
    if (__any_sync(0xffffffffu, bad)) {
        if (report && lane == 0) set_status(status, NQ_DEV_BAD_PAGE);
        return;
    }
    uint8_t *data = p.data + static_cast<size_t>(layer) * p.layer_bytes + static_cast<size_t>(h) * p.rec;
    const int32_t *tab = m.table + static_cast<size_t>(slot) * m.W;
    auto row_at = [&](int off) {                                 // rec NULL: not there
        RowAt w{nullptr, 0};
        const long long row = static_cast<long long>(base) + off, j = row >> lp;
        if (j >= m.W) {
            if (report) set_status(status, NQ_DEV_SEQ_FULL);
            return w;
        }
        const int id = tab[j];
        if (id < 0 || id >= p.N) {
            if (report) set_status(status, NQ_DEV_BAD_PAGE);
            return w;
        }
        w.rec = data + static_cast<size_t>(id) * p.H * p.rec;
        w.r = static_cast<int>(row & (m.P - 1));
        return w;
    };
    auto chunk_at = [&](const RowAt &w, int part, int c) -> uint8_t * {
        const int blk = w.r >> 4, r = w.r & 15;
        if constexpr (NG == 0) return w.rec + static_cast<size_t>(blk) * p.base_block + part * 32 * D + 2 * bf_off(D, r, 8 * c);
        const int kv = part & 1;
        return w.rec + (part < 2 ? static_cast<size_t>(blk) * p.base_block : p.resid_off + static_cast<size_t>(blk) * (32 * RB)) + kv * 16 * RB +
               nib_off(RB, r, 16 * c);
    };
    auto scale_at = [&](const RowAt &w, int i) {                 // i = kv * NG + group
        return reinterpret_cast<uint16_t *>(w.rec + static_cast<size_t>(w.r >> 4) * p.base_block + 32 * RB + (i / NS) * 32 * NS) + (w.r & 15) * NS + i % NS;
    };
    for (; j0 < cnt; j0 += BATCH) {
        const int rows = min(BATCH, cnt - j0);
        uint4 x[4];
        uint8_t *to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = lane + 32 * i, j = e / CPR, c = e % CPR;
            to[i] = nullptr;
            if (j >= rows) continue;
            const RowAt a = row_at(pt[j0 + j]), d = row_at(j0 + j);
            if (!a.rec || !d.rec) continue;
            x[i] = *reinterpret_cast<const uint4 *>(chunk_at(a, c / CH, c % CH));
            to[i] = chunk_at(d, c / CH, c % CH);
        }
        uint16_t sc = 0, *sto = nullptr;
        if constexpr (NG != 0) {
            const int j = lane / (2 * NS);
            if (j < rows) {
                const RowAt a = row_at(pt[j0 + j]), d = row_at(j0 + j);
                if (a.rec && d.rec) {
                    sc = *scale_at(a, lane % (2 * NS));
                    sto = scale_at(d, lane % (2 * NS));
                }
            }
        }
        __syncwarp();                                            // all of the batch is read before any of it is written
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (to[i]) *reinterpret_cast<uint4 *>(to[i]) = x[i];
        if (sto) *sto = sc;
        __syncwarp();
    }
}

}  // namespace
}  // namespace nq

extern "C" nq_status nq_tree_plan(const nq_tree *tree, cudaStream_t stream)
{
    const nq_status st = nq::tree_of(tree);
    if (st != NQ_OK) return st;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    nq::plan_kernel<<<tree->batch, (tree->nodes + 31) / 32 * 32, 0, stream>>>(tree->parents, tree->nodes, (tree->nodes + 31) / 32, tree->window,
                                                                          tree->depth, tree->bits, status);
    return nq::cuda_status(cudaGetLastError());
}

extern "C" nq_status spec_accept_tree(const nq_tree *tree, const int32_t *tokens, const float *logits, int V, int width,
                                      int32_t *out_tok, int32_t *out_cnt, int32_t *path, cudaStream_t stream)
{
    const nq_status st = nq::tree_of(tree);
    if (st != NQ_OK) return st;
    if (!tokens || !logits || !out_tok || !out_cnt || !path || V < 1 || V > 524288 || width < 1 || width > tree->nodes) return NQ_ERR_ARG;
    if (tree->batch > 65535) return NQ_ERR_SHAPE;
    if (!nq::aligned16(logits) || !nq::aligned4(tokens) || !nq::aligned4(out_tok) || !nq::aligned4(out_cnt) || !nq::aligned4(path)) return NQ_ERR_ALIGN;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = nq::kAccCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tree->batch) * attr[0].val.clusterDim.x);
    cfg.blockDim = dim3(nq::kAccThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return nq::cuda_status(cudaLaunchKernelEx(&cfg, nq::accept_tree_kernel, tree->parents, static_cast<const int32_t *>(tree->depth), tokens, logits,
                                              tree->nodes, V, width, out_tok, out_cnt, path, status));
}

extern "C" nq_status nq_page_keep(const nq_page_pool *pool, const nq_page_map *map, const int32_t *seqs, const int32_t *first,
                                  const int32_t *path, const int32_t *count, int n, int width, cudaStream_t stream)
{
    nq::Pool p;
    nq::Map m;
    const nq_status st = nq::pool_map_of(pool, map, p, m, false);
    if (st != NQ_OK) return st;
    if (!seqs || !first || !path || !count || n < 1 || width < 1) return NQ_ERR_ARG;
    if (!nq::aligned4(seqs) || !nq::aligned4(first) || !nq::aligned4(path) || !nq::aligned4(count)) return NQ_ERR_ALIGN;
    if (static_cast<double>(pool->layers) * p.H > 2.0e9 || static_cast<double>(n) * pool->layers * p.H > 1.6e10) return NQ_ERR_SHAPE;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    const long long warps = static_cast<long long>(n) * pool->layers * p.H;
    const unsigned grid = static_cast<unsigned>((warps + nq::kKeepWarps - 1) / nq::kKeepWarps);
    auto go = [&](auto *kernel) { kernel<<<grid, nq::kKeepWarps * 32, 0, stream>>>(p, m, seqs, first, path, count, n, width, pool->layers, status); };
    if (p.D == 64) go(p.NG == 0 ? nq::keep_kernel<64, 0> : nq::keep_kernel<64, 1>);
    else go(p.NG == 0 ? nq::keep_kernel<128, 0> : p.NG == 1 ? nq::keep_kernel<128, 1> : nq::keep_kernel<128, 2>);
    return nq::cuda_status(cudaGetLastError());
}
