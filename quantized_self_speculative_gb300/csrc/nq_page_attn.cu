// nq_page_attn.cu -- attention of the newest rows of each sequence over the
// paged KV cache.
//
// out = sum_t p_t V_t / sum_t p_t, p_t = 2^(s_t - m), s = log2(e) f(scale q.K_t):
// one pass over the rows with the running maximum m, sum and output, rescaled
// when m grows.  One CTA of four warps per query vector, warp w takes rows w,
// w + 4, ..; lane l holds D / 32 of the row's values.
#include "nq_page.cuh"

namespace nq {
namespace {

constexpr int kWarps = 4;

template <int E>
__device__ __forceinline__ void row_values(const Pool &p, const uint8_t *rec, int r, int v, int planes, int lane,
                                           float (&x)[E])
{
    constexpr int D = 32 * E, RB = D / 2;
    const int blk = r >> 4, r16 = r & 15;
    const uint8_t *base = rec + blk * p.base_block;
    if (p.NG == 0) {
        const auto *src = reinterpret_cast<const __nv_bfloat16 *>(base) + v * 16 * D + bf_off(D, r16, lane * E);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = __bfloat162float(src[e]);
        return;
    }
    const uint32_t at = v * 16 * RB + nib_off(RB, r16, lane * E / 2);
    const uint8_t *resid = rec + p.resid_off + blk * (16 * D);
    const float s = __half2float(
        *reinterpret_cast<const __half *>(base + 32 * RB + v * 32 * p.NG + (r16 * p.NG + lane / (32 / p.NG)) * 2));
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int q4 = (base[at + e / 2] >> (4 * (e & 1)) & 15) - 8;
        const int rr = planes == 2 ? (resid[at + e / 2] >> (4 * (e & 1)) & 15) - 8 : 0;
        x[e] = s * (q4 + rr * 0.0625f);
    }
}

template <int E>
__global__ void __launch_bounds__(kWarps * 32)
attn_kernel(Pool p, Map m, const __nv_bfloat16 *__restrict__ q, long long q_stride, int M, int Hq,
            const int32_t *__restrict__ seqs, const int32_t *__restrict__ len, int planes, nq_attn_opts o,
            __nv_bfloat16 *__restrict__ out, unsigned int *status)
{
    constexpr int D = 32 * E;
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hq = blockIdx.x, mi = blockIdx.y, b = blockIdx.z, h = hq / (Hq / p.H);
    const int slot = seqs ? seqs[b] : b;
    const long long cap = static_cast<long long>(m.W) * m.P;
    int L = len[b];
    if (L > cap) {
        if (threadIdx.x == 0) set_status(status, NQ_DEV_SEQ_FULL);
        L = static_cast<int>(cap);
    }
    if (slot < 0 || slot >= m.S) {
        if (threadIdx.x == 0) set_status(status, NQ_DEV_BAD_PAGE);
        L = 0;
    }
    const int at = L - M + mi, lo = o.window > 0 ? max(0, at - o.window + 1) : 0;
    const __nv_bfloat16 *qr = q + (static_cast<long long>(b) * M + mi) * q_stride + hq * D + lane * E;
    float qv[E], acc[E], mx = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qv[e] = __bfloat162float(qr[e]);
        acc[e] = 0.0f;
    }
    for (int t = lo + warp; t <= at; t += kWarps) {
        const int id = m.table[static_cast<size_t>(slot) * m.W + t / m.P];
        if (id < 0 || id >= p.N) {
            set_status(status, NQ_DEV_BAD_PAGE);
            continue;
        }
        const uint8_t *rec = p.data + (static_cast<size_t>(id) * p.H + h) * p.rec;
        float kv[E], vv[E], s = 0.0f;
        row_values<E>(p, rec, t % m.P, 0, planes, lane, kv);
        row_values<E>(p, rec, t % m.P, 1, planes, lane, vv);
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(qv[e], kv[e], s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= o.scale;
        if (o.softcap > 0.0f) s = o.softcap * tanhf(s / o.softcap);
        if (o.slopes) s -= o.slopes[hq] * static_cast<float>(at - t);
        const float mn = fmaxf(mx, s), a = mx == -INFINITY ? 0.0f : expf(mx - mn), e1 = expf(s - mn);
        mx = mn;
        l = fmaf(l, a, e1);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], a, e1 * vv[e]);
    }
    if (lane == 0) {
        sm_m[warp] = mx;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = acc[e];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
        float M2 = -INFINITY, num = 0.0f, den = 0.0f;
        for (int w = 0; w < kWarps; ++w) M2 = fmaxf(M2, sm_m[w]);
        for (int w = 0; w < kWarps; ++w) {
            if (sm_m[w] == -INFINITY) continue;
            const float f = expf(sm_m[w] - M2);
            num = fmaf(f, sm_o[w][d], num);
            den = fmaf(f, sm_l[w], den);
        }
        const float r = at < lo ? 0.0f : num / den;
        out[((static_cast<long long>(b) * M + mi) * Hq + hq) * D + d] = __float2bfloat16_rn(r);
    }
}

}  // namespace
}  // namespace nq

extern "C" size_t nq_page_attn_workspace_bytes(int M, int heads_q, int heads_kv, int head_dim)
{
    if (M < 1 || heads_kv < 1 || heads_q < heads_kv || heads_q % heads_kv != 0 || !(head_dim == 64 || head_dim == 128)) return 0;
    return 16;
}

extern "C" nq_status nq_page_attn(const nq_page_pool *pool, int layer, const nq_page_map *map, const uint16_t *q,
                                  int64_t q_stride, int batch, int M, int heads_q, const int32_t *seqs,
                                  const int32_t *len, int planes, const nq_attn_opts *opts, uint16_t *out, void *ws,
                                  size_t ws_bytes, cudaStream_t stream)
{
    nq::Pool p;
    nq::Map m;
    const nq_status st = nq::pool_map_of(pool, map, p, m, false);
    if (st != NQ_OK) return st;
    if (layer < 0 || layer >= pool->layers || !q || !len || !out || !opts || batch < 1 || M < 1) return NQ_ERR_ARG;
    if (heads_q < p.H || heads_q % p.H != 0 || (planes != 1 && planes != 2) || (!seqs && batch > m.S)) return NQ_ERR_ARG;
    if (!(opts->scale > 0.0f) || !(opts->softcap >= 0.0f) || opts->window < 0) return NQ_ERR_ARG;
    if (M > 65535 || batch > 65535 || heads_q > 65536) return NQ_ERR_SHAPE;
    if (q_stride < static_cast<int64_t>(heads_q) * p.D || q_stride % 8 != 0) return NQ_ERR_SHAPE;
    if (!nq::aligned16(q) || !nq::aligned16(out) || !nq::aligned16(ws) || !nq::aligned4(seqs) || !nq::aligned4(len) ||
        !nq::aligned4(opts->slopes))
        return NQ_ERR_ALIGN;
    if (!ws || ws_bytes < nq_page_attn_workspace_bytes(M, heads_q, p.H, p.D)) return NQ_ERR_WORKSPACE;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    p.data += static_cast<size_t>(layer) * p.layer_bytes;
    auto *kernel = p.D == 128 ? nq::attn_kernel<4> : nq::attn_kernel<2>;
    kernel<<<dim3(heads_q, M, batch), nq::kWarps * 32, 0, stream>>>(
        p, m, reinterpret_cast<const __nv_bfloat16 *>(q), q_stride, M, heads_q, seqs, len, planes, *opts,
        reinterpret_cast<__nv_bfloat16 *>(out), status);
    return nq::cuda_status(cudaGetLastError());
}
