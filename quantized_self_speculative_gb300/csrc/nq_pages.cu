// nq_pages.cu -- which pages of the paged KV cache belong to which sequence:
// taking, sharing, releasing, moving and copying them.
//
// The state is a table of page ids per sequence slot, the number held, and a
// reference count per page (0 = free).  Counts change by atomic adds, whose
// order does not matter; ids are handed out lowest free first in the order of
// the requests, so the outcome is the same on every run.  The bookkeeping is a
// few KB of ids: bound by launches and the latency of scans (cutting back and
// extending 16 slots over 4096 pages: two calls, three launches, 11 us).  A request's
// pages are handed out by one thread: room for a prompt of 131072 rows in pages
// of 16 takes some 230 us, of 32768 rows 70 us, and 16 such at once 180 us.
#include "nq_page.cuh"

namespace nq {
namespace {

constexpr int kMapThreads = 256;
constexpr int kScanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;                                   // 16-byte loads in flight per thread
constexpr int kTile = kCopyThreads * kCopyUnroll;                // 16-byte units per copied tile

// ---------------------------------------------------------------- block scan
// Exclusive prefix sum of v over the block (1024 threads), total in `sum`.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *sm, T &sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    T w = sm[lane];                                              // 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    sum = __shfl_sync(0xffffffffu, w, 31);
    const T before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    __syncthreads();                                             // sm may be written again
    return before + x - v;
}

__device__ __forceinline__ int pages_of(int rows, int P) { return rows <= 0 ? 0 : (rows - 1) / P + 1; }

// ---------------------------------------------------------------- init
__global__ void init_kernel(Map m)
{
    const size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x, step = static_cast<size_t>(gridDim.x) * blockDim.x;
    const size_t nt = static_cast<size_t>(m.S) * m.W;
    for (size_t k = i; k < nt; k += step) m.table[k] = -1;
    for (size_t k = i; k < static_cast<size_t>(m.S); k += step) m.held[k] = 0;
    for (size_t k = i; k < static_cast<size_t>(m.N); k += step) m.ref[k] = 0;
}

// ---------------------------------------------------------------- truncate
// One CTA per request.  A slot may be named more than once: an entry is taken out by an
// exchange, so that one CTA releases its page whatever the others do, and `held` only falls.
__global__ void __launch_bounds__(kMapThreads)
truncate_kernel(Map m, const int32_t *__restrict__ seqs, const int32_t *__restrict__ rows, unsigned int *status)
{
    const int s = seqs[blockIdx.x];
    if (s < 0 || s >= m.S) {
        if (threadIdx.x == 0) set_status(status, NQ_DEV_BAD_PAGE);
        return;
    }
    const int held = min(max(m.held[s], 0), m.W), keep = min(pages_of(rows[blockIdx.x], m.P), held);
    int32_t *t = m.table + static_cast<size_t>(s) * m.W;
    for (int j = keep + threadIdx.x; j < held; j += kMapThreads) {
        const int p = atomicExch(t + j, -1);
        if (p >= 0 && p < m.N) atomicSub(m.ref + p, 1);
        else if (p != -1) set_status(status, NQ_DEV_BAD_PAGE);   // -1: another request for the slot has been here
    }
    // every thread has read `held`: the first CTA to lower it past an entry has taken that entry out
    __syncthreads();
    if (threadIdx.x == 0) atomicMin(m.held + s, keep);
}

// ---------------------------------------------------------------- fork
// First launch: every source row into the workspace ([n][2] page counts, then
// [n][W] ids), counts adjusted; nothing of the table changes.  Second launch:
// the rows to their slots.
__global__ void __launch_bounds__(kMapThreads)
fork_read_kernel(Map m, const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                 const int32_t *__restrict__ rows, int n_pairs, int32_t *__restrict__ ws, unsigned int *status)
{
    asm volatile("griddepcontrol.launch_dependents;");
    const int i = blockIdx.x, a = src[i], b = dst[i];
    if (a < 0 || a >= m.S || b < 0 || b >= m.S) {
        if (threadIdx.x == 0) set_status(status, NQ_DEV_BAD_PAGE);
        return;
    }
    const int ha = min(max(m.held[a], 0), m.W), hb = min(max(m.held[b], 0), m.W);
    const int want = pages_of(rows[i], m.P), n = min(want, ha);
    if (threadIdx.x == 0) {
        if (want > ha) set_status(status, NQ_DEV_BAD_PAGE);
        ws[2 * i] = n;
        ws[2 * i + 1] = hb;
    }
    const int32_t *ta = m.table + static_cast<size_t>(a) * m.W, *tb = m.table + static_cast<size_t>(b) * m.W;
    int32_t *out = ws + 2 * static_cast<size_t>(n_pairs) + static_cast<size_t>(i) * m.W;
    for (int j = threadIdx.x; j < max(n, hb); j += kMapThreads) {
        const int old = j < hb ? tb[j] : -1, p = j < n ? ta[j] : -1;
        if (p != old) {                       // a page that the slot keeps counts as before
            if (p >= 0 && p < m.N) atomicAdd(m.ref + p, 1);
            if (old >= 0 && old < m.N) atomicSub(m.ref + old, 1);
        }
        out[j] = p;
    }
}

__global__ void __launch_bounds__(kMapThreads)
fork_write_kernel(Map m, const int32_t *__restrict__ src, const int32_t *__restrict__ dst, int n_pairs,
                  const int32_t *__restrict__ ws)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int i = blockIdx.x, a = src[i], b = dst[i];
    if (a < 0 || a >= m.S || b < 0 || b >= m.S) return;
    const int n = ws[2 * i], hb = ws[2 * i + 1];
    int32_t *tb = m.table + static_cast<size_t>(b) * m.W;
    const int32_t *in = ws + 2 * static_cast<size_t>(n_pairs) + static_cast<size_t>(i) * m.W;
    for (int j = threadIdx.x; j < max(n, hb); j += kMapThreads) tb[j] = in[j];
    if (threadIdx.x == 0) m.held[b] = n;
}

// ---------------------------------------------------------------- copy
// Pages src -> dst in every layer, tiles of 32 KB over the whole grid.  The
// pairs are given as two lists; `count` (device) overrides n where not NULL.
// HBM bound: 512 MB moved by a compaction in 177 us with its plan, 5.8 TB/s (86%
// of the copy rate).
__global__ void __launch_bounds__(kCopyThreads)
copy_kernel(uint8_t *data, size_t layer_bytes, size_t page_bytes, int layers, int N, const int32_t *__restrict__ src,
            const int32_t *__restrict__ dst, int n, const int32_t *__restrict__ count, unsigned int *status)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (count) n = *count;
    const unsigned units = static_cast<unsigned>(page_bytes / 16), tiles = (units + kTile - 1) / kTile;
    const long long items = static_cast<long long>(n) * layers * tiles;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const unsigned tile = static_cast<unsigned>(it % tiles);
        const long long pl = it / tiles;
        const int layer = static_cast<int>(pl % layers), k = static_cast<int>(pl / layers);
        const int a = src[k], b = dst[k];
        if (a < 0 || a >= N || b < 0 || b >= N) {
            if (threadIdx.x == 0) set_status(status, NQ_DEV_BAD_PAGE);
            continue;
        }
        const uint8_t *from = data + layer * layer_bytes + a * page_bytes;
        uint8_t *to = data + layer * layer_bytes + b * page_bytes;
        uint4 v[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u) {
            const unsigned x = tile * kTile + u * kCopyThreads + threadIdx.x;
            if (x < units) v[u] = *reinterpret_cast<const uint4 *>(from + static_cast<size_t>(x) * 16);
        }
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u) {
            const unsigned x = tile * kTile + u * kCopyThreads + threadIdx.x;
            if (x < units) *reinterpret_cast<uint4 *>(to + static_cast<size_t>(x) * 16) = v[u];
        }
    }
}

// ---------------------------------------------------------------- reserve
// One CTA.  Workspace: asked[N], last[N] (of shared pages that requests touch),
// ids[N], before[n], then the copies: count, src[2n], dst[2n].
struct ReserveWs {
    int32_t *asked, *last, *ids, *before, *count, *src, *dst;
};
__host__ __device__ inline ReserveWs reserve_ws(int32_t *w, int N, int n)
{
    ReserveWs r;
    r.asked = w;
    r.last = w + N;
    r.ids = w + 2 * static_cast<size_t>(N);
    r.before = w + 3 * static_cast<size_t>(N);
    r.count = r.before + n;
    r.src = r.count + 4;
    r.dst = r.src + 2 * n;
    return r;
}

// The range of a request: pages lo .. need-1 hold its rows, held of them are there.
struct Want {
    int s, first, last, lo, need, held;
    bool ok;
};
__device__ __forceinline__ Want want_of(const Map &m, const int32_t *seqs, const int32_t *first, const int32_t *last,
                                        int i)
{
    Want w;
    w.s = seqs[i];
    w.first = first[i];
    w.last = last[i];
    const bool slot = w.s >= 0 && w.s < m.S && w.first >= 0;
    w.ok = slot && w.last <= m.W * m.P;
    w.held = slot ? min(max(m.held[w.s], 0), m.W) : 0;
    w.lo = w.need = 0;
    if (w.ok && w.last > w.first) {
        w.lo = w.first / m.P;
        w.need = pages_of(w.last, m.P);
    }
    return w;
}

__global__ void __launch_bounds__(kScanThreads, 1)
reserve_kernel(Map m, const int32_t *__restrict__ seqs, const int32_t *__restrict__ first,
               const int32_t *__restrict__ last, int n, int32_t *__restrict__ granted, int32_t *ws, unsigned int *status)
{
    __shared__ int sm[32], sm_copies;
    __shared__ long long sm_wide[32];
    asm volatile("griddepcontrol.launch_dependents;");
    const ReserveWs R = reserve_ws(ws, m.N, n);
    const int tid = threadIdx.x;
    if (tid == 0) sm_copies = 0;
    // ---- shared pages that requests write to: how many requests touch each, and the last of them
    for (int i = tid; i < n; i += kScanThreads) {
        const Want w = want_of(m, seqs, first, last, i);
        const int32_t *t = m.table + static_cast<size_t>(max(w.s, 0)) * m.W;
        for (int j = w.lo; j < min(w.held, w.need); ++j) {
            const int p = t[j];
            if (p >= 0 && p < m.N && m.ref[p] > 1) {
                R.asked[p] = 0;
                R.last[p] = -1;
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < n; i += kScanThreads) {
        const Want w = want_of(m, seqs, first, last, i);
        const int32_t *t = m.table + static_cast<size_t>(max(w.s, 0)) * m.W;
        for (int j = w.lo; j < min(w.held, w.need); ++j) {
            const int p = t[j];
            if (p >= 0 && p < m.N && m.ref[p] > 1) {
                atomicAdd(R.asked + p, 1);
                atomicMax(R.last + p, i);
            }
        }
    }
    __syncthreads();
    // ---- pages wanted per request; an entry to be copied is marked -(id + 2).  The requests of a call may
    // want more pages than 32 bits hold: a sum past them is kept as the largest number, which no pool covers
    long long total = 0;
    for (int i0 = 0; i0 < n; i0 += kScanThreads) {
        const int i = i0 + tid;
        int c = 0;
        if (i < n) {
            const Want w = want_of(m, seqs, first, last, i);
            if (w.s < 0 || w.s >= m.S || w.first < 0) set_status(status, NQ_DEV_BAD_PAGE);
            else if (!w.ok) set_status(status, NQ_DEV_SEQ_FULL);
            int32_t *t = m.table + static_cast<size_t>(max(w.s, 0)) * m.W;
            for (int j = w.lo; j < min(w.held, w.need); ++j) {
                const int p = t[j];
                if (p < 0 || p >= m.N) {
                    set_status(status, NQ_DEV_BAD_PAGE);
                } else if (m.ref[p] > 1 && !(R.asked[p] == m.ref[p] && R.last[p] == i)) {
                    t[j] = -(p + 2);
                    ++c;
                }
            }
            c += max(w.need - w.held, 0);
        }
        long long sum;
        const long long pre = total + block_scan(static_cast<long long>(c), sm_wide, sum);
        if (i < n) R.before[i] = static_cast<int>(min(pre, 0x7fffffffll));
        total += sum;
    }
    // ---- the lowest free ids, until there are enough
    constexpr int E = 8;
    int found = 0;
    for (int base = 0; base < m.N && found < total; base += kScanThreads * E) {
        unsigned z = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int p = base + tid * E + e;
            if (p < m.N && m.ref[p] == 0) z |= 1u << e;
        }
        int sum;
        int at = found + block_scan(__popc(z), sm, sum);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (z >> e & 1u) R.ids[at++] = base + tid * E + e;
        found += sum;
    }
    __syncthreads();
    // ---- hand them out
    for (int i = tid; i < n; i += kScanThreads) {
        const Want w = want_of(m, seqs, first, last, i);
        const int pre = R.before[i];
        int32_t *t = m.table + static_cast<size_t>(max(w.s, 0)) * m.W;
        int c = max(w.need - w.held, 0);
        for (int j = w.lo; j < min(w.held, w.need); ++j) c += t[j] < -1;
        const bool give = w.ok && static_cast<long long>(pre) + c <= found;
        if (w.ok && !give) set_status(status, NQ_DEV_POOL_FULL);
        int k = pre;
        for (int j = w.lo; j < min(w.held, w.need); ++j) {
            if (t[j] >= -1) continue;
            const int old = -t[j] - 2;
            if (!give) {
                t[j] = old;
                continue;
            }
            const int p = R.ids[k++];
            t[j] = p;
            m.ref[p] = 1;
            atomicSub(m.ref + old, 1);
            const long long r0 = static_cast<long long>(j) * m.P;
            if (r0 < w.first || r0 + m.P > w.last) {            // rows that this call's caller will not write
                const int at = atomicAdd(&sm_copies, 1);
                R.src[at] = old;
                R.dst[at] = p;
            }
        }
        if (give) {
            for (int j = w.held; j < w.need; ++j) {
                const int p = R.ids[k++];
                t[j] = p;
                m.ref[p] = 1;
            }
            if (w.need > w.held) m.held[w.s] = w.need;
        }
        if (granted) granted[i] = give ? 1 : 0;
    }
    __syncthreads();
    if (tid == 0) *R.count = sm_copies;
}

// ---------------------------------------------------------------- compact
// One CTA: `used`, the moves (from[k] -> to[k], ascending) and where each moved
// page went.  Workspace: count (4 words), from[N], to[N], where[N].
__global__ void __launch_bounds__(kScanThreads, 1)
compact_plan_kernel(Map m, int32_t *__restrict__ used, int32_t *ws)
{
    __shared__ int sm[32];
    asm volatile("griddepcontrol.launch_dependents;");
    int32_t *from = ws + 4, *to = from + m.N, *where = to + m.N;
    constexpr int E = 8;
    const int tid = threadIdx.x;
    int mine = 0;
    for (int p = tid; p < m.N; p += kScanThreads) mine += m.ref[p] > 0;
    int U;
    block_scan(mine, sm, U);
    int n_from = 0, n_to = 0;
    for (int base = 0; base < m.N; base += kScanThreads * E) {
        unsigned hole = 0, high = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int p = base + tid * E + e;
            if (p >= m.N) continue;
            const int r = m.ref[p];
            if (p < U && r <= 0) hole |= 1u << e;
            if (p >= U && r > 0) high |= 1u << e;
        }
        int sum;
        if (base < U) {
            int at = n_to + block_scan(__popc(hole), sm, sum);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (hole >> e & 1u) to[at++] = base + tid * E + e;
            n_to += sum;
        }
        if (base + kScanThreads * E > U) {
            int at = n_from + block_scan(__popc(high), sm, sum);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (high >> e & 1u) from[at++] = base + tid * E + e;
            n_from += sum;
        }
    }
    __syncthreads();
    for (int k = tid; k < n_from; k += kScanThreads) {
        const int a = from[k], b = to[k];
        where[a] = b;
        m.ref[b] = m.ref[a];
        m.ref[a] = 0;
    }
    if (tid == 0) {
        ws[0] = n_from;
        *used = U;
    }
}

__global__ void __launch_bounds__(kMapThreads)
compact_table_kernel(Map m, const int32_t *__restrict__ used, const int32_t *__restrict__ ws, unsigned int *status)
{
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t *where = ws + 4 + 2 * static_cast<size_t>(m.N);
    const int U = *used;
    if (ws[0] == 0) return;
    const size_t nt = static_cast<size_t>(m.S) * m.W;
    for (size_t k = static_cast<size_t>(blockIdx.x) * kMapThreads + threadIdx.x; k < nt; k += static_cast<size_t>(gridDim.x) * kMapThreads) {
        const int p = m.table[k];
        if (p < U || p >= m.N) continue;
        const int q = where[p];
        if (q >= 0 && q < U) m.table[k] = q;
        else set_status(status, NQ_DEV_BAD_PAGE);
    }
}

// ---------------------------------------------------------------- host side
template <typename... KA, typename... A>
cudaError_t launch_after(void (*kernel)(KA...), int grid, int threads, cudaStream_t s, A... args)
{
    // a programmatic dependent launch: it overlaps the kernel before it, and
    // griddepcontrol.wait orders its reads
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KA>(args)...);
}

size_t ws_words(const Map &m, int n)
{
    const size_t N = m.N, a = 3 * N + 5 * static_cast<size_t>(n) + 4, b = static_cast<size_t>(n) * (m.W + 2), c = 3 * N + 4;
    return (a > b ? a : b) > c ? (a > b ? a : b) : c;
}

int copy_grid(long long items) { return static_cast<int>(items < 8ll * sm_count() ? (items < 1 ? 1 : items) : 8ll * sm_count()); }
long long copy_items(const Pool &p, int layers, long long n)
{
    const long long units = static_cast<long long>(p.H) * p.rec / 16;
    return n * layers * ((units + kTile - 1) / kTile);
}

}  // namespace
}  // namespace nq

extern "C" nq_status nq_page_pool_bytes(int layers, int n_pages, int page_size, int heads_kv, int head_dim, int group,
                                        int format, size_t *bytes)
{
    nq_page_pool p{layers, n_pages, page_size, heads_kv, head_dim, group, format, 0, nullptr};
    nq::Pool o;
    const nq_status st = nq::pool_of(&p, o, false);
    if (st != NQ_OK) return st;
    if (!bytes) return NQ_ERR_ARG;
    *bytes = o.layer_bytes * layers;
    return NQ_OK;
}

extern "C" nq_status nq_page_map_init(const nq_page_map *map, cudaStream_t stream)
{
    nq::Map m;
    const nq_status st = nq::map_of(map, m, true);
    if (st != NQ_OK) return st;
    const size_t most = static_cast<size_t>(m.S) * m.W > static_cast<size_t>(m.N) ? static_cast<size_t>(m.S) * m.W : m.N;
    const size_t grid = (most + nq::kMapThreads - 1) / nq::kMapThreads;
    nq::init_kernel<<<static_cast<int>(grid < 1024 ? grid : 1024), nq::kMapThreads, 0, stream>>>(m);
    return nq::cuda_status(cudaGetLastError());
}

extern "C" size_t nq_page_workspace_bytes(const nq_page_map *map, int n)
{
    nq::Map m;
    if (nq::map_of(map, m, false) != NQ_OK || n < 1 || n > m.S) return 0;
    return nq::ws_words(m, n) * sizeof(int32_t);
}

namespace nq {
namespace {
// What reserve, fork and compact check alike.
nq_status check_ws(const Map &m, int n, const void *ws, size_t ws_bytes)
{
    if (n < 1 || n > m.S) return NQ_ERR_ARG;
    if (!ws || ws_bytes < ws_words(m, n) * sizeof(int32_t)) return NQ_ERR_WORKSPACE;
    return aligned16(ws) ? NQ_OK : NQ_ERR_ALIGN;
}
}  // namespace
}  // namespace nq

extern "C" nq_status nq_page_reserve(const nq_page_map *map, const nq_page_pool *pool, const int32_t *seqs,
                                     const int32_t *first, const int32_t *last, int n, int32_t *granted, void *ws,
                                     size_t ws_bytes, cudaStream_t stream)
{
    nq::Map m;
    nq::Pool p{};
    nq_status st = pool ? nq::pool_map_of(pool, map, p, m, true) : nq::map_of(map, m, true);
    if (st != NQ_OK) return st;
    if (!seqs || !first || !last) return NQ_ERR_ARG;
    if (!nq::aligned4(seqs) || !nq::aligned4(first) || !nq::aligned4(last) || !nq::aligned4(granted)) return NQ_ERR_ALIGN;
    st = nq::check_ws(m, n, ws, ws_bytes);
    if (st != NQ_OK) return st;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    int32_t *w = static_cast<int32_t *>(ws);
    nq::reserve_kernel<<<1, nq::kScanThreads, 0, stream>>>(m, seqs, first, last, n, granted, w, status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !pool) return nq::cuda_status(e);
    const nq::ReserveWs R = nq::reserve_ws(w, m.N, n);
    e = nq::launch_after(nq::copy_kernel, nq::copy_grid(nq::copy_items(p, pool->layers, 2ll * n)), nq::kCopyThreads, stream,
                         p.data, p.layer_bytes, static_cast<size_t>(p.H) * p.rec, pool->layers, p.N, R.src, R.dst, 0,
                         R.count, status);
    return nq::cuda_status(e);
}

extern "C" nq_status nq_page_fork(const nq_page_map *map, const int32_t *src, const int32_t *dst, const int32_t *rows,
                                  int n, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    nq::Map m;
    nq_status st = nq::map_of(map, m, true);
    if (st != NQ_OK) return st;
    if (!src || !dst || !rows) return NQ_ERR_ARG;
    if (!nq::aligned4(src) || !nq::aligned4(dst) || !nq::aligned4(rows)) return NQ_ERR_ALIGN;
    st = nq::check_ws(m, n, ws, ws_bytes);
    if (st != NQ_OK) return st;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    int32_t *w = static_cast<int32_t *>(ws);
    nq::fork_read_kernel<<<n, nq::kMapThreads, 0, stream>>>(m, src, dst, rows, n, w, status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return NQ_ERR_CUDA;
    e = nq::launch_after(nq::fork_write_kernel, n, nq::kMapThreads, stream, m, src, dst, n, w);
    return nq::cuda_status(e);
}

extern "C" nq_status nq_page_truncate(const nq_page_map *map, const int32_t *seqs, const int32_t *rows, int n,
                                      cudaStream_t stream)
{
    nq::Map m;
    const nq_status st = nq::map_of(map, m, true);
    if (st != NQ_OK) return st;
    if (!seqs || !rows || n < 1 || n > m.S) return NQ_ERR_ARG;
    if (!nq::aligned4(seqs) || !nq::aligned4(rows)) return NQ_ERR_ALIGN;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    nq::truncate_kernel<<<n, nq::kMapThreads, 0, stream>>>(m, seqs, rows, status);
    return nq::cuda_status(cudaGetLastError());
}

extern "C" nq_status nq_page_compact(const nq_page_map *map, const nq_page_pool *pool, int32_t *used, void *ws,
                                     size_t ws_bytes, cudaStream_t stream)
{
    nq::Map m;
    nq::Pool p;
    nq_status st = nq::pool_map_of(pool, map, p, m, true);
    if (st != NQ_OK) return st;
    if (!used) return NQ_ERR_ARG;
    if (!nq::aligned4(used)) return NQ_ERR_ALIGN;
    st = nq::check_ws(m, 1, ws, ws_bytes);
    if (st != NQ_OK) return st;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    int32_t *w = static_cast<int32_t *>(ws);
    nq::compact_plan_kernel<<<1, nq::kScanThreads, 0, stream>>>(m, used, w);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return NQ_ERR_CUDA;
    const size_t tg = (static_cast<size_t>(m.S) * m.W + nq::kMapThreads - 1) / nq::kMapThreads;
    e = nq::launch_after(nq::compact_table_kernel, static_cast<int>(tg < 1024 ? tg : 1024), nq::kMapThreads, stream, m,
                         used, w, status);
    if (e != cudaSuccess) return NQ_ERR_CUDA;
    e = nq::launch_after(nq::copy_kernel, nq::copy_grid(nq::copy_items(p, pool->layers, m.N)), nq::kCopyThreads, stream,
                         p.data, p.layer_bytes, static_cast<size_t>(p.H) * p.rec, pool->layers, p.N, w + 4, w + 4 + m.N,
                         0, w, status);
    return nq::cuda_status(e);
}

extern "C" nq_status nq_page_copy(const nq_page_pool *pool, const int32_t *src, const int32_t *dst, int n,
                                  cudaStream_t stream)
{
    nq::Pool p;
    const nq_status st = nq::pool_of(pool, p);
    if (st != NQ_OK) return st;
    if (!src || !dst || n < 1) return NQ_ERR_ARG;
    if (!nq::aligned4(src) || !nq::aligned4(dst)) return NQ_ERR_ALIGN;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    nq::copy_kernel<<<nq::copy_grid(nq::copy_items(p, pool->layers, n)), nq::kCopyThreads, 0, stream>>>(
        p.data, p.layer_bytes, static_cast<size_t>(p.H) * p.rec, pool->layers, p.N, src, dst, n, nullptr, status);
    return nq::cuda_status(cudaGetLastError());
}
